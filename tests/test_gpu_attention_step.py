"""attention_step with the caller's out and lse."""
import pytest
import torch

import workloads as W
from test_gpu_attention import DEV, F, _Step  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,most", [(5, 100), (2, 2500), (70, 4200)])         # whole, parts, the line
def test_step_into_given_outputs(F, B, most, out_dtype):
    s = _Step(F, W.gen(41, DEV), B=B, most=most)
    s.lt[B // 2] = 0
    s.slots[B // 2] = -1
    want = s.run(out_dtype=out_dtype)
    out, lse = torch.full_like(want, 7.0), torch.full((B, 8), 7.0, device=DEV)
    got = s.run(out_dtype=out_dtype, out=out, lse=lse)
    assert got.data_ptr() == out.data_ptr() and torch.equal(out, want)
    q, _ = F.fp8_qk_norm_rope(s.q, s.k, s.tab, s.pos, s.w, s.w)
    ref = torch.empty(B, 8, device=DEV)
    F.fp8_paged_attention(q, s.c, s.table, s.lt, out_dtype=out_dtype, lse=ref)
    assert torch.equal(lse, ref) and (lse[B // 2] == -float("inf")).all()
