"""The weights of fp8_paged_attention keep 24 bits, for bf16 and fp32 output,
however the work is dealt out: whole regions, parts of regions, the line.

Each case leaves one rounding's worth of freedom (u = 2^-24): V is not zero
for one token only, so a product with V has one term a position, the weight
times a V scale of 24 bits times a power of two.  Weights cut to 16 bits
(two bf16 terms instead of three) miss by 64 u and more.
"""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import attention as A
from test_gpu_attention import DEV, U, F, _np  # noqa: F401

pytestmark = pytest.mark.gpu


def dealt(F, c, B, Hq, cols, max_context=None, window=0):
    """How a call deals out its work, from its workspace: 'whole' needs none, 'parts' a slot for each (regions
    times a power of two, at most 256), 'line' two for each of up to 512 pieces."""
    G, D = Hq // c.heads, c.head_dim
    most = 32 if G > 16 and D <= 128 else 16
    regions, rows = B * c.heads * -(-G // most), min(G, most)
    room = cols * c.page_size
    nbytes = F.attn_lib().fp8_paged_attention_workspace(c._ref, B, Hq, cols,
                                                        room if max_context is None else max_context, window)
    assert nbytes >= 0 and nbytes % (rows * (D + 2) * 4) == 0
    slots = nbytes // (rows * (D + 2) * 4)
    if slots == 0:
        return "whole"
    return "line" if slots > 256 else "parts" if slots in [regions << i for i in range(1, 9)] else "line"


def _cache(F, pages, H, S, D, fmt):
    """Codes 0, scales 1."""
    c = F.KVCache(pages, S, H, D, fmt, DEV)
    for t in (c.k_codes, c.v_codes):
        t.zero_()
    for t in (c.k_scales, c.v_scales):
        t.fill_(1.0)
    return c


def _code(fmt, x):
    """The code of a value that has one."""
    at = np.nonzero(A.code_values(fmt) == x)[0]
    return int(at[0])


# (sequences, KV heads, tokens of room): how the call is dealt out
WAYS = {"whole": (32, 4, 32), "parts": (16, 4, 3008), "line": (64, 4, 4800)}


@pytest.mark.parametrize("fmt", ["e5m2", "e4m3"])
@pytest.mark.parametrize("D", [64, 80, 128, 256])
@pytest.mark.parametrize("way", list(WAYS))
def test_one_token_is_its_value_rounded_once(F, way, D, fmt):
    """One token: weight 1, out = V.  The scales put V 2^-20 beside a tie of bf16, on the side that a rounding to
    16 bits first (to the tie, and from there to even) does not end on.  The three terms of a weight add up to it
    without a rounding, so bf16 output is V rounded to nearest and fp32 output is V."""
    B, H, room = WAYS[way]
    S = 16
    c = _cache(F, B, H, S, D, fmt)
    k = torch.arange(B * H, device=DEV).view(B, H) % 128
    side = torch.where(k % 2 == 0, 1.0, -1.0).double()
    scale = 1 + k * 2.0 ** -7 + 2.0 ** -8 + side * 2.0 ** -20
    c.v_scales[:, :, 0] = scale.float()
    assert torch.equal(c.v_scales[:, :, 0].double(), scale)
    powers = [1.0, 2.0, 0.5, -1.0, -4.0, 16.0, 0.25, -0.125]
    codes = torch.tensor([_code(fmt, powers[i % 8]) for i in range(D)], dtype=torch.uint8, device=DEV)
    c.v_codes[:, :, 0] = codes
    exact = scale[..., None] * torch.tensor([powers[i % 8] for i in range(D)], dtype=torch.float64, device=DEV)
    table = torch.zeros(B, room // S, dtype=torch.int32, device=DEV)
    table[:, 0] = torch.arange(B, device=DEV)
    lens = torch.ones(B, dtype=torch.int32, device=DEV)
    q = torch.randn(B, 2 * H, D, generator=W.gen(D, DEV), device=DEV).bfloat16()
    assert dealt(F, c, B, 2 * H, table.shape[1]) == way
    want = A.round_bf16(exact.cpu().numpy()).repeat(2, axis=1)
    np.testing.assert_array_equal(_np(F.fp8_paged_attention(q, c, table, lens)), want)
    got = F.fp8_paged_attention(q, c, table, lens, out_dtype=torch.float32)
    assert torch.equal(got.double(), exact.repeat_interleave(2, 1))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,H,room,way", [(3, 2, 700, "whole"), (3, 2, 2992, "parts"), (66, 2, 4800, "line")])
def test_equal_weights(F, B, H, room, way, D):
    """q = 0: every weight is 1 and their sum n, exactly; one token's V is not zero: out = V / n but for
    a reciprocal and a product, each rounded: 3 u; the terms' sum is exact and joining multiplies by 1."""
    S, n = 16, min(room, 2501)
    if way == "whole":
        n, room = 300, 304
    c = _cache(F, -(-n // S), H, S, D, "e5m2")
    scale = 1 + 5 * 2.0 ** -7 + 2.0 ** -9 + 2.0 ** -17
    for h, at in enumerate((n // 3, n - 1)):
        c.v_codes[at // S, h, at % S] = _code("e5m2", 1.0)
        c.v_scales[at // S, h, at % S] = scale
    cols = -(-room // S)
    table = torch.zeros(B, cols, dtype=torch.int32, device=DEV)
    table[:, :c.pages] = torch.arange(c.pages, device=DEV)
    lens = torch.full((B,), n, dtype=torch.int32, device=DEV)
    q = torch.zeros(B, 3 * H, D, device=DEV).bfloat16()
    assert dealt(F, c, B, 3 * H, cols) == way
    out = F.fp8_paged_attention(q, c, table, lens, out_dtype=torch.float32).double()
    assert ((out - scale / n).abs() <= 3 * U * scale / n).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,H,room,way", [(3, 2, 304, "whole"), (3, 2, 2992, "parts"), (66, 2, 4800, "line")])
@pytest.mark.parametrize("high_first", [False, True])
def test_rescaling_keeps_32_bits(F, B, H, room, way, D, high_first):
    """Two levels of scores, 0 and 1.25, the maximum growing along the sequence or not, one token's V not zero
    (of the low level for head 0, of the high one for head 1).

    A score of 1.25 is 1.8 in the log2 domain, off by 2 roundings of that (4 u); a weight or a rescaling factor by
    ln 2 of that and the exponential's ulp, 5 u and a product's 1; there are at most 4 factors (in the wave, between
    the waves, between pieces, between groups of pieces): 24 u.  The sum of the weights takes 8 additions a tile of
    a wave's quarter, 2 across lanes, 4 waves and at most 32 pieces.  V's product 3 u, division 3 u."""
    S, n = 16, {"whole": 300, "parts": 2501, "line": 2501}[way]
    c = _cache(F, -(-n // S), H, S, D, "e5m2")
    half = n // 2 + 5
    at = torch.arange(c.pages * S, device=DEV).view(c.pages, 1, S)
    high = (at < half) if high_first else (at >= half)
    c.k_codes[..., 0] = torch.where(high, _code("e5m2", 1.25), 0).to(torch.uint8).expand(c.pages, H, S)
    lo_at, hi_at = (n - 7, 11) if high_first else (11, n - 7)
    scale = 1 + 5 * 2.0 ** -7 + 2.0 ** -9 + 2.0 ** -17
    for h, t in enumerate((lo_at, hi_at)):
        c.v_codes[t // S, h, t % S] = _code("e5m2", 1.0)
        c.v_scales[t // S, h, t % S] = scale
    cols = -(-room // S)
    table = torch.zeros(B, cols, dtype=torch.int32, device=DEV)
    table[:, :c.pages] = torch.arange(c.pages, device=DEV)
    lens = torch.full((B,), n, dtype=torch.int32, device=DEV)
    q = torch.zeros(B, 2 * H, D, device=DEV).bfloat16()
    q[..., 0] = 1.0
    assert dealt(F, c, B, 2 * H, cols) == way
    out = F.fp8_paged_attention(q, c, table, lens, scale=1.0, out_dtype=torch.float32).double()
    n_high = half if high_first else n - half
    e = np.exp(1.25)
    total = n - n_high + n_high * e
    want = torch.tensor([scale / total, scale * e / total], dtype=torch.float64, device=DEV)
    want = want.repeat_interleave(2)[None, :, None]
    tol = (24 + 24 + 8 * -(-n // 128) + 2 + 4 + 32 + 6) * U     # (a factor in the numerator, in the denominator)
    assert ((out - want).abs() <= tol * want).all(), ((out - want).abs() / want).max() / U
