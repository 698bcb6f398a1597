"""NaN rows that enter the cache stay NaN, whatever the row's magnitude, and reach the attention's output."""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import attention as A
from test_gpu_attention import DEV, F, _fresh, _np, _rows, _table  # noqa: F401

pytestmark = pytest.mark.gpu

# magnitudes on both sides of 2^-62, where the quotients go from multiplication to division
MAGNITUDES = [1.0, 2.0 ** -61, 2.0 ** -63, 2.0 ** -100, 2.0 ** -126, 0.0]


def _nan_rows(D, g):
    """[magnitudes, 3, D]: a NaN of either sign at one position of heads 0 and 1, head 2 wholly NaN."""
    x = torch.randn(len(MAGNITUDES), 3, D, generator=g, device=DEV)
    x = (x * torch.tensor(MAGNITUDES, device=DEV)[:, None, None]).bfloat16()
    x[:, 0, D // 3] = float("nan")
    x[:, 1, D - 1] = torch.tensor([-64], dtype=torch.int16, device=DEV).view(torch.bfloat16)[0]     # 0xffc0
    x[:, 2] = float("nan")
    return x


@pytest.mark.parametrize("fmt", ["e5m2", "e4m3"])
@pytest.mark.parametrize("D", [16, 64, 80, 128, 256])
@pytest.mark.parametrize("copies", [1, 500])          # a row slot each; slots that walk along tokens
def test_nan_rows_are_written_as_nan(F, D, fmt, copies):
    """The scale comes from the row's other values, their codes are as they would be without the NaN."""
    g = W.gen(D, DEV)
    rows = _nan_rows(D, g).repeat(copies, 1, 1)
    T, S = rows.shape[0], 16
    c = _fresh(F, -(-T // S), 3, S, D, fmt)
    F.fp8_kv_cache_write(rows, rows, torch.arange(T, device=DEV), c)
    k = _np(rows)
    nan = np.isnan(k)
    codes, d = A.quantise(np.where(nan, 0.0, k).astype(np.float32), fmt)
    meaning = A.code_values(fmt)
    for got, scales in ((c.k_codes, c.k_scales), (c.v_codes, c.v_scales)):
        got = got.transpose(1, 2).reshape(-1, 3, D)[:T].cpu().numpy()
        assert np.isnan(meaning[got][nan]).all()
        np.testing.assert_array_equal(got[~nan], codes[~nan])
        np.testing.assert_array_equal(scales.transpose(1, 2).reshape(-1, 3)[:T].cpu().numpy(), d)


@pytest.mark.parametrize("fmt", ["e5m2", "e4m3"])
@pytest.mark.parametrize("magnitude", [1.0, 2.0 ** -100, 0.0])
def test_a_step_on_nan_keys_gives_nan(F, magnitude, fmt):
    """A NaN in the new token's key of one KV head: that head's queries give NaN, the others are as they were."""
    g = W.gen(3, DEV)
    B, Hq, H, D, S = 2, 6, 3, 64, 16
    q, v = _rows(B, Hq, D, g), _rows(B, H, D, g)
    k = (_rows(B, H, D, g) * magnitude).bfloat16()
    tab, pos, slots = _table(D, 8), torch.tensor([2, 5], device=DEV), torch.tensor([2, S + 5], device=DEV)
    lens = torch.tensor([3, 6], dtype=torch.int32, device=DEV)
    table = torch.arange(B, dtype=torch.int32, device=DEV)[:, None]

    def step(k):
        c = F.KVCache(B, S, H, D, fmt, DEV)
        F.fp8_kv_cache_write(_rows(B * S, H, D, W.gen(4, DEV)), _rows(B * S, H, D, W.gen(5, DEV)),
                             torch.arange(B * S, device=DEV), c)
        return F.attention_step(q, k, v, tab, pos, slots, c, table, lens)

    want = step(k)
    bad = k.clone()
    bad[1, 2, 7] = float("nan")
    got = step(bad)
    assert torch.isfinite(want).all() and torch.isnan(got[1, 4:]).all()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1, :4], want[1, :4])


@pytest.mark.parametrize("fmt", ["e5m2", "e4m3"])
@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
def test_an_infinity_makes_the_rows_scale_nan(F, value, fmt):
    g = W.gen(6, DEV)
    c, clean = _fresh(F, 1, 2, 16, 64, fmt), _fresh(F, 1, 2, 16, 64, fmt)
    rows = _rows(16, 2, 64, g)
    bad = rows.clone()
    bad[3, 1, 5] = value
    slots = torch.arange(16, device=DEV)
    F.fp8_kv_cache_write(rows, rows, slots, clean)
    F.fp8_kv_cache_write(bad, bad, slots, c)
    at = torch.zeros(1, 2, 16, dtype=torch.bool, device=DEV)
    at[0, 1, 3] = True
    for a, b in ((c.k_scales, clean.k_scales), (c.v_scales, clean.v_scales)):
        assert torch.isnan(a[at]).all() and torch.equal(a[~at], b[~at])
    for a, b in ((c.k_codes, clean.k_codes), (c.v_codes, clean.v_codes)):
        assert torch.equal(a[~at], b[~at])


@pytest.mark.parametrize("max_context", [300, None])          # whole regions; parts
def test_values_that_are_not_finite_stay_in_their_position(F, max_context):
    """An infinite V code of a seen token: that position of its KV head's rows is not finite, all else is the same;
    an infinite V scale: every position of them."""
    g = W.gen(8, DEV)
    H, D, S, n = 2, 128, 16, 290
    c = F.KVCache(20, S, H, D, "e5m2", DEV)
    F.fp8_kv_cache_write(_rows(320, H, D, g), _rows(320, H, D, g), torch.arange(320, device=DEV), c)
    q = _rows(1, 6, D, g)
    table = torch.zeros(1, 200, dtype=torch.int32, device=DEV)
    table[0, :20] = torch.arange(20, device=DEV)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)

    def run():
        return F.fp8_paged_attention(q, c, table, lens, out_dtype=torch.float32, max_context=max_context)[0]

    want = run()
    c.v_codes[9, 1, 3, 77] = 0x7C
    got = run()
    bad = torch.zeros(6, D, dtype=torch.bool, device=DEV)
    bad[3:, 77] = True
    assert not torch.isfinite(got[bad]).any() and torch.equal(got[~bad], want[~bad])
    c.v_codes[9, 1, 3, 77] = 0
    c.v_scales[9, 1, 3] = float("inf")
    got = run()
    assert not torch.isfinite(got[3:]).any() and torch.equal(got[:3], want[:3])
