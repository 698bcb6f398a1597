"""The attention side of a decode step on the GPU against the 64-bit oracle.

Tolerances (u = 2^-24, a rounding of fp32; h = 2^-8, one of bf16):

* norm and rotation: the sum of D squares is off by D u at most (non-negative
  terms), the mean by 2 u more, eps by 1, all halved by the root; its
  reciprocal by an estimate and a Newton step is within 2 u, two products
  follow: a normed value is off by at most (D/2 + 6) u relative; the rotation
  adds 3 roundings of its two terms; then one rounding to bf16:
  |err| <= h |ref| + (D/2 + 12) u (|a c| + |b s|).
* codes, scales and values read back: equal bit for bit.
* attention: a score's fp32 sum of D exact products, the scale products (3) and
  the difference from the maximum are off by at most (D + 8) u S, S the largest
  sum of |q k| scale; the maximum cancels between numerator and denominator.
  A weight is off by twice that, relative, and 4 u for the exponential; its
  split into bf16 terms (2 or 3) by 2^-16 or 2^-24; both sums over n tokens by
  n u each, the joins by 16 u: with M the weighted mean of |v|,
  |err| <= M (4 (D + 8) u S + split + (2 n + 32) u), and h |ref| for bf16
  output (u |ref| for fp32).  lse: 2 (D + 8) u S + (n + 32) u + 4 u |lse|.
"""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import attention as A

pytestmark = pytest.mark.gpu
DEV = "cuda"
U, HB = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def F():
    import fp8_block_scaled_02_amd as F
    assert torch.cuda.is_available()
    return F


def _np(t):
    return t.detach().double().cpu().numpy()


def _rows(T, H, D, g, strided=False):
    """bf16 rows [T, H, D]; strided: a slice of wider storage in both strides."""
    if not strided:
        return torch.randn(T, H, D, generator=g, device=DEV).bfloat16()
    wide = torch.randn(T, H + 2, D + 24, generator=g, device=DEV).bfloat16()
    return wide[:, 1:H + 1, 8:D + 8]


def _table(rot, n, theta=10000.0):
    inv = theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    ang = torch.arange(n, dtype=torch.float64)[:, None] * inv
    return torch.cat((ang.cos(), ang.sin()), 1).float().to(DEV)


# ---- norm and rotation -------------------------------------------------------


def _check_rope(y, x, w, eps, tab, pos, inter):
    D = x.shape[2]
    ref, mag = A.norm_rope(_np(x), None if w is None else _np(w), eps, None if tab is None else _np(tab),
                           None if pos is None else pos.cpu().numpy(), inter)
    err = np.abs(_np(y) - ref)
    assert (err <= HB * np.abs(ref) + (D / 2 + 12) * U * mag + 2.0 ** -134).all(), err.max()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", [(16, 16), (64, 64), (64, 16), (80, 32), (96, 96), (128, 128), (128, 48), (160, 160),
                                   (192, 64), (256, 256), (240, 240)])
def test_norm_rope(F, D, rot, inter):
    g = W.gen(D + rot, DEV)
    T, Hq, Hk = 37, 7, 3
    q, k = _rows(T, Hq, D, g, True), _rows(T, Hk, D, g)
    tab = _table(rot, 500)
    pos = torch.randint(0, 500, (T,), generator=g, device=DEV)
    qw, kw = (torch.rand(D, generator=g, device=DEV).bfloat16() for _ in range(2))
    qo, ko = F.fp8_qk_norm_rope(q, k, tab, pos, qw, kw, 1e-5, inter)
    _check_rope(qo, q, qw, 1e-5, tab, pos, inter)
    _check_rope(ko, k, kw, 1e-5, tab, pos, inter)
    qo, ko = F.fp8_qk_norm_rope(q, k, tab, pos, None, kw, 1e-5, inter)     # one norm only
    _check_rope(qo, q, None, 1e-5, tab, pos, inter)
    _check_rope(ko, k, kw, 1e-5, tab, pos, inter)
    qo, _ = F.fp8_qk_norm_rope(q, k, None, None, qw, None, 1e-5, inter)    # no rotation
    _check_rope(qo, q, qw, 1e-5, None, None, inter)


@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 1), (1, 64, 8), (3, 0, 5), (3, 5, 0), (1025, 2, 1), (2500, 20, 5)])
def test_norm_rope_sizes(F, T, Hq, Hk):
    g = W.gen(T, DEV)
    q, k = _rows(T, Hq, 128, g), _rows(T, Hk, 128, g)
    tab, pos = _table(128, 64), torch.randint(0, 64, (T,), generator=g, device=DEV)
    w = torch.rand(128, generator=g, device=DEV).bfloat16()
    qo, ko = F.fp8_qk_norm_rope(q, k, tab, pos, w, w)
    if Hq:
        _check_rope(qo, q, w, 1e-6, tab, pos, False)
    if Hk:
        _check_rope(ko, k, w, 1e-6, tab, pos, False)


def test_norm_rope_in_place_on_the_projection(F):
    """q and k as slices of the fused projection, written over; the values beside them stay."""
    g = W.gen(1, DEV)
    T, Hq, Hk, D = 33, 6, 2, 128
    y = torch.randn(T, (Hq + 2 * Hk) * D, generator=g, device=DEV).bfloat16()
    before = y.clone()
    q, k = y[:, :Hq * D].view(T, Hq, D), y[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    tab, pos = _table(D, 64), torch.randint(0, 64, (T,), generator=g, device=DEV)
    want = F.fp8_qk_norm_rope(q, k, tab, pos)
    F.fp8_qk_norm_rope(q, k, tab, pos, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(y[:, (Hq + Hk) * D:], before[:, (Hq + Hk) * D:])


def test_norm_of_zeros_and_position_ends(F):
    q = torch.zeros(2, 1, 64, device=DEV).bfloat16()
    k = torch.ones(2, 1, 64, device=DEV).bfloat16()
    w = torch.ones(64, device=DEV).bfloat16()
    tab = _table(64, 8)
    pos = torch.tensor([0, 7], device=DEV)
    qo, ko = F.fp8_qk_norm_rope(q, k, tab, pos, w, w)
    assert not qo.any()
    _check_rope(ko, k, w, 1e-6, tab, pos, False)
    far = torch.tensor([-5, 1 << 40], device=DEV)        # outside the table: no fault, other rows unharmed
    F.fp8_qk_norm_rope(q, k, tab, far, w, w)
    torch.cuda.synchronize()


@pytest.mark.parametrize("D,rot,inter", [(64, 16, False), (128, 48, False), (256, 64, False), (80, 32, True)])
def test_infinities_beyond_the_rotation_pass(F, D, rot, inter):
    q = torch.ones(3, 2, D, device=DEV).bfloat16()
    q[1, 0, rot:] = float("inf")
    q[2, 1, rot + 1] = float("-inf")
    k = q.clone()
    tab, pos = _table(rot, 8), torch.tensor([1, 5, 7], device=DEV)
    for o in F.fp8_qk_norm_rope(q, k, tab, pos, interleaved=inter):
        assert torch.equal(o[..., rot:], q[..., rot:])
        assert torch.isfinite(o[..., :rot]).all()


# ---- writing and reading -----------------------------------------------------


def _fresh(F, pages, H, S, D, fmt, fill=0x5A):
    c = F.KVCache(pages, S, H, D, fmt, DEV)
    for t in (c.k_codes, c.v_codes):
        t.fill_(fill)
    for t in (c.k_scales, c.v_scales):
        t.fill_(-7.0)
    return c


def _expect_written(c, k, v, slots):
    """The whole cache as the oracle says it is after a write into a fresh one."""
    out = []
    for x in (k, v):
        codes = np.full((c.pages, c.heads, c.page_size, c.head_dim), 0x5A, np.uint8)
        scales = np.full((c.pages, c.heads, c.page_size), -7.0, np.float32)
        q, d = A.quantise(_np(x).astype(np.float32), c.fmt)
        for t, s in enumerate(slots.tolist()):
            if 0 <= s < c.pages * c.page_size:
                codes[s // c.page_size, :, s % c.page_size] = q[t]
                scales[s // c.page_size, :, s % c.page_size] = d[t]
        out.append((codes, scales))
    return out


def _assert_cache(c, want):
    for (codes, scales), got_c, got_s in zip(want, (c.k_codes, c.v_codes), (c.k_scales, c.v_scales)):
        np.testing.assert_array_equal(got_c.cpu().numpy(), codes)
        np.testing.assert_array_equal(got_s.cpu().numpy(), scales)


@pytest.mark.parametrize("fmt", ["e5m2", "e4m3"])
@pytest.mark.parametrize("H,S,D,T", [(1, 16, 16, 1), (3, 16, 64, 19), (8, 16, 128, 32), (5, 64, 80, 77), (2, 32, 112, 5),
                                     (1, 4096, 96, 40), (4, 128, 192, 131), (7, 16, 256, 23), (2, 16, 144, 1500)])
def test_cache_write(F, H, S, D, T, fmt):
    g = W.gen(H + D, DEV)
    c = _fresh(F, -(-T // S) + 3, H, S, D, fmt)
    mag = torch.exp2(60 * torch.rand(T, H, 1, generator=g, device=DEV) - 30)
    k = (torch.randn(T, H, D, generator=g, device=DEV) * mag).bfloat16()
    v = _rows(T, H, D, g, True)
    k[T // 2, 0] = 0                                                    # amax 0
    slots = torch.randperm(c.pages * S, generator=g, device=DEV)[:T]
    slots[::4] = -1
    if T > 5:
        slots[5] = c.pages * S                                          # past the end: nothing written
        slots[3] = -(1 << 40)
    F.fp8_kv_cache_write(k, v, slots, c)
    _assert_cache(c, _expect_written(c, k, v, slots))


@pytest.mark.parametrize("T,H,D,fmt", [(20011, 8, 128, "e5m2"), (9001, 8, 128, "e4m3"), (30011, 5, 256, "e4m3"),
                                       (12345, 1, 80, "e5m2")])
def test_large_write_is_the_small_writes(F, T, H, D, fmt):
    """Calls large enough for slots that walk along tokens and for non-temporal accesses, against calls of 700
    tokens; some tokens are padding."""
    g = W.gen(T, DEV)
    k, v = _rows(T, H, D, g), _rows(T, H, D, g)
    pages = -(-T // 64) + 1
    slots = torch.randperm(pages * 64, generator=g, device=DEV)[:T]
    slots[::7] = -1
    one, two = _fresh(F, pages, H, 64, D, fmt), _fresh(F, pages, H, 64, D, fmt)
    F.fp8_kv_cache_write(k, v, slots, one)
    for lo in range(0, T, 700):
        F.fp8_kv_cache_write(k[lo:lo + 700], v[lo:lo + 700], slots[lo:lo + 700], two)
    for a, b in zip((one.k_codes, one.v_codes, one.k_scales, one.v_scales),
                    (two.k_codes, two.v_codes, two.k_scales, two.v_scales)):
        assert torch.equal(a, b)


def test_large_norm_rope_is_the_small_ones(F):
    g = W.gen(17, DEV)
    T = 4100
    q, k = _rows(T, 20, 128, g), _rows(T, 3, 128, g)
    tab, pos = _table(128, 99), torch.randint(0, 99, (T,), generator=g, device=DEV)
    w = torch.rand(128, generator=g, device=DEV).bfloat16()
    qo, ko = F.fp8_qk_norm_rope(q, k, tab, pos, w, w)
    for lo in range(0, T, 500):
        a, b = F.fp8_qk_norm_rope(q[lo:lo + 500], k[lo:lo + 500], tab, pos[lo:lo + 500], w, w)
        assert torch.equal(qo[lo:lo + 500], a) and torch.equal(ko[lo:lo + 500], b)


def test_cache_write_into_a_layer_of_a_shared_allocation(F):
    """K and V of three layers in one allocation, page by page; neighbours stay."""
    g = W.gen(9, DEV)
    P, H, S, D, T = 6, 2, 16, 64, 30
    codes = torch.full((P, 3, 2, H, S, D), 0x5A, dtype=torch.uint8, device=DEV)
    scales = torch.full((P, 3, 2, H, S), -7.0, device=DEV)
    c = F.KVCache.from_tensors(codes[:, 1, 0], codes[:, 1, 1], scales[:, 1, 0], scales[:, 1, 1], "e4m3")
    k, v = _rows(T, H, D, g), _rows(T, H, D, g)
    slots = torch.randperm(P * S, generator=g, device=DEV)[:T]
    F.fp8_kv_cache_write(k, v, slots, c)
    _assert_cache(c, _expect_written(c, k, v, slots))
    rest = codes.clone()
    rest[:, 1] = 0x5A
    assert (rest == 0x5A).all() and (scales[:, [0, 2]] == -7.0).all()


def test_same_slot_twice_harms_no_other(F):
    g = W.gen(10, DEV)
    c = _fresh(F, 2, 2, 16, 64, "e5m2")
    k, v = _rows(4, 2, 64, g), _rows(4, 2, 64, g)
    slots = torch.tensor([3, 9, 9, 30], device=DEV)
    F.fp8_kv_cache_write(k, v, slots, c)
    want = _expect_written(c, k[[0, 1, 3]], v[[0, 1, 3]], slots[[0, 1, 3]])
    got = [t.cpu().numpy() for t in (c.k_codes, c.v_codes)]
    for (codes, _), have in zip(want, got):
        codes[0, :, 9] = have[0, :, 9]
        np.testing.assert_array_equal(have, codes)


@pytest.mark.parametrize("fmt", ["e5m2", "e4m3"])
@pytest.mark.parametrize("Hq,H,D,rot,inter", [(8, 2, 128, 128, False), (5, 5, 80, 32, True), (3, 1, 256, 64, False)])
def test_fused_write_is_the_two_calls(F, Hq, H, D, rot, inter, fmt):
    g = W.gen(D, DEV)
    for T in (1, 45):
        q, k, v = _rows(T, Hq, D, g, True), _rows(T, H, D, g), _rows(T, H, D, g, True)
        tab, pos = _table(rot, 99), torch.randint(0, 99, (T,), generator=g, device=DEV)
        qw, kw = (torch.rand(D, generator=g, device=DEV).bfloat16() for _ in range(2))
        slots = torch.randperm(80, generator=g, device=DEV)[:T]
        slots[T // 2] = -1
        one, two = _fresh(F, 5, H, 16, D, fmt), _fresh(F, 5, H, 16, D, fmt)
        qo = F.fp8_qkv_cache_write(q, k, v, tab, pos, slots, one, qw, kw, 1e-6, inter)
        q2, k2 = F.fp8_qk_norm_rope(q, k, tab, pos, qw, kw, 1e-6, inter)
        F.fp8_kv_cache_write(k2, v, slots, two)
        assert torch.equal(qo, q2)
        for a, b in zip((one.k_codes, one.v_codes, one.k_scales, one.v_scales),
                        (two.k_codes, two.v_codes, two.k_scales, two.v_scales)):
            assert torch.equal(a, b)


def _filled(F, pages, H, S, D, fmt, g):
    """A cache of N(0, 1) rows whose magnitudes differ from token to token."""
    c = F.KVCache(pages, S, H, D, fmt, DEV)
    for codes, scales in ((c.k_codes, c.k_scales), (c.v_codes, c.v_scales)):
        x = torch.randn(pages * S, H, D, generator=g, device=DEV)
        x = (x * torch.exp2(2 * torch.rand(pages * S, H, 1, generator=g, device=DEV) - 1)).bfloat16()
        q, d = A.quantise(_np(x).astype(np.float32), fmt)
        codes.copy_(torch.from_numpy(q).to(DEV).view(pages, S, H, D).transpose(1, 2))
        scales.copy_(torch.from_numpy(d).to(DEV).view(pages, S, H).transpose(1, 2))
    return c


def _values(c):
    """The cache's K and V in 64 bits, [pages, heads, page_size, D]."""
    t = torch.from_numpy(A.code_values(c.fmt)).to(DEV)
    return [t[x.long()] * s.double()[..., None] for x, s in ((c.k_codes, c.k_scales), (c.v_codes, c.v_scales))]


def _book(lens, S, g, spare=3, room=5000):
    """Pages in random order; table entries past a sequence's pages are no pages at all.  Room for contexts
    that are split, whatever these lengths."""
    need = [-(-n // S) for n in lens]
    order = torch.randperm(sum(need) + spare, generator=g, device=DEV).cpu()
    table = torch.full((len(lens), max(need + [-(-room // S)])), -(1 << 30), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n].int()
        table[b, n:] = (1 << 30) + b
        at += n
    return sum(need) + spare, table.to(DEV)


@pytest.mark.parametrize("fmt", ["e5m2", "e4m3"])
@pytest.mark.parametrize("lens,H,S,D", [([1], 1, 16, 16), ([0, 5, 0, 33, 16, 0], 3, 16, 64), ([129, 1, 64], 8, 64, 128),
                                        ([40] * 70, 2, 32, 96), ([500], 5, 128, 80), ([31, 17], 16, 16, 256)])
def test_cache_read(F, lens, H, S, D, fmt):
    g = W.gen(D + len(lens), DEV)
    pages, table = _book(lens, S, g)
    c = _filled(F, pages, H, S, D, fmt, g)
    offs = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV)
    R = sum(lens) + 9
    k, v = (torch.full((R, H, D), 123.0, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    F.fp8_kv_cache_read(c, table, offs, R, k, v)
    for got, val in zip((k, v), _values(c)):
        rows = [val[table[b, t // S], :, t % S] for b, n in enumerate(lens) for t in range(n)]
        want = torch.stack(rows).float().bfloat16()      # an fp32 product of an exact code and a scale, then bf16
        assert torch.equal(got[:sum(lens)], want)
        assert (got[sum(lens):] == 123.0).all()


def test_cache_read_of_nothing_and_of_bad_books(F):
    g = W.gen(11, DEV)
    c = _filled(F, 4, 2, 16, 64, "e5m2", g)
    offs = torch.zeros(3, dtype=torch.int32, device=DEV)
    table = torch.zeros(2, 2, dtype=torch.int32, device=DEV)
    assert F.fp8_kv_cache_read(c, table, offs, 0)[0].shape == (0, 2, 64)
    k, v = (torch.full((5, 2, 64), 3.0, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    F.fp8_kv_cache_read(c, table, offs, 5, k, v)
    assert (k == 3.0).all() and (v == 3.0).all()
    # longer than the table, pages that are none, offsets that fall: no fault
    for o in ([0, 50, 90], [0, 90, 20], [7, 8, 90]):
        bad = torch.tensor([[1 << 30, -1], [3, 7]], dtype=torch.int32, device=DEV)
        F.fp8_kv_cache_read(c, bad, torch.tensor(o, dtype=torch.int32, device=DEV), 90)
    torch.cuda.synchronize()


# ---- attention ---------------------------------------------------------------


def _check_attention(F, c, lens, q, table, window=0, out_dtype=torch.bfloat16, scale=None, max_context=None,
                     check=None):
    B, Hq, D = q.shape
    lt = torch.tensor(lens, dtype=torch.int32, device=DEV)
    lse = torch.full((B, Hq), 5.0, device=DEV)
    out = F.fp8_paged_attention(q, c, table, lt, scale, window, out_dtype, lse=lse, max_context=max_context)
    kv = _values(c)
    sc = D ** -0.5 if scale is None else scale
    S = c.page_size
    for b in (range(B) if check is None else check):
        n = max(0, min(lens[b], table.shape[1] * S))
        if max_context is not None:
            n = min(n, max_context)
        pages = table[b, :-(-n // S)].long()
        k, v = (x[pages].transpose(1, 2).reshape(-1, c.heads, D)[:n].cpu().numpy() for x in kv)
        ref, rl, mag, big = A.attention(_np(q[b]), k, v, sc, window)
        ds = (D + 8) * U * big
        split = 2.0 ** -16 if out_dtype == torch.bfloat16 else 2.0 ** -24
        tol = mag * (4 * ds + split + (2 * n + 32) * U)[:, None]
        tol += np.abs(ref) * (HB if out_dtype == torch.bfloat16 else U)
        err = np.abs(_np(out[b]) - ref)
        assert (err <= tol).all(), (b, n, err.max(), np.unravel_index(np.argmax(err - tol), err.shape))
        got = _np(lse[b])
        if n == 0:
            assert not out[b].any() and (got == -np.inf).all()
        else:
            assert (np.abs(got - rl) <= 2 * ds + (n + 32) * U + 4 * U * np.abs(rl)).all(), (b, got - rl)
    return out, lse


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", ["e5m2", "e4m3"])
@pytest.mark.parametrize("D", [16, 48, 64, 80, 96, 112, 128, 144, 160, 192, 208, 256])
def test_attention_head_dims(F, D, fmt, out_dtype):
    g = W.gen(D, DEV)
    lens = [1, 31, 32, 33, 0, 257, 700]
    pages, table = _book(lens, 16, g)
    c = _filled(F, pages, 2, 16, D, fmt, g)
    q = (2 * torch.randn(len(lens), 6, D, generator=g, device=DEV)).bfloat16()
    _check_attention(F, c, lens, q, table, out_dtype=out_dtype)
    _check_attention(F, c, lens, q, table, out_dtype=out_dtype, max_context=256)     # not split


@pytest.mark.parametrize("Hq,H,D", [(1, 1, 64), (7, 1, 64), (16, 1, 64), (17, 1, 64), (40, 1, 64), (5, 5, 64),
                                    (28, 4, 64), (24, 8, 64), (32, 16, 64), (96, 2, 64), (32, 1, 128), (33, 1, 128),
                                    (71, 1, 128), (24, 1, 80), (20, 1, 48), (16, 1, 256), (40, 2, 256), (34, 2, 192)])
def test_attention_head_layouts(F, Hq, H, D):
    g = W.gen(Hq, DEV)
    lens = [100, 513, 3]
    pages, table = _book(lens, 32, g)
    c = _filled(F, pages, H, 32, D, "e5m2", g)
    wide = torch.randn(3, Hq + 1, D + 16, generator=g, device=DEV).bfloat16()
    q = wide[:, 1:, 8:D + 8]                                             # strided
    _check_attention(F, c, lens, q, table)
    # one workgroup of 8 waves per region: the most shared memory
    _check_attention(F, c, lens, q, table, max_context=600, out_dtype=torch.float32)


@pytest.mark.parametrize("S", [16, 32, 64, 256, 4096])
@pytest.mark.parametrize("window", [0, 1, 2, 31, 33, 300, 5000])
def test_attention_pages_and_windows(F, S, window):
    g = W.gen(S + window, DEV)
    lens = [1, 2, 15, 16, 17, 48, 299, 300, 301, 1000, 0]
    pages, table = _book(lens, S, g)
    c = _filled(F, pages, 2, S, 64, "e4m3", g)
    q = (2 * torch.randn(len(lens), 4, 64, generator=g, device=DEV)).bfloat16()
    _check_attention(F, c, lens, q, table, window, torch.float32)
    _check_attention(F, c, lens, q, table, window, max_context=310)


def test_attention_long_context_is_split_and_joined(F):
    g = W.gen(2, DEV)
    lens = [20011, 7, 0, 12000]
    pages, table = _book(lens, 64, g)
    c = _filled(F, pages, 2, 64, 128, "e5m2", g)
    q = (2 * torch.randn(4, 16, 128, generator=g, device=DEV)).bfloat16()
    _check_attention(F, c, lens, q, table, out_dtype=torch.float32)
    _check_attention(F, c, lens, q, table, window=9999)
    _check_attention(F, c, lens, q, table, max_context=4096)


@pytest.mark.parametrize("fmt", ["e5m2", "e4m3"])
@pytest.mark.parametrize("Hq,H,D,window", [(8, 2, 128, 0), (4, 1, 64, 1700), (9, 3, 80, 0), (3, 1, 256, 0),
                                           (20, 1, 128, 0), (8, 2, 128, 1500)])
def test_attention_of_regions_in_parts(F, Hq, H, D, window, fmt):
    """Few regions of some length: each in equal parts, also where lengths leave most parts nothing."""
    g = W.gen(21, DEV)
    lens = [2000, 0, 1, 31, 33, 127, 129, 130, 640, 1999]
    pages, table = _book([2000] * len(lens), 32, g)
    c = _filled(F, pages, H, 32, D, fmt, g)
    q = torch.randn(len(lens), Hq, D, generator=g, device=DEV).bfloat16()
    _check_attention(F, c, lens, q, table, window=window, out_dtype=torch.float32)
    _check_attention(F, c, lens[:1], q[:1], table[:1], window=window)
    _check_attention(F, c, lens[2:5], q[2:5], table[2:5], window=window, max_context=1100)


def test_attention_many_sequences(F):
    """More sequences than a wave has lanes, and more regions than workgroups."""
    g = W.gen(3, DEV)
    lens = [int(x) for x in torch.randint(0, 400, (333,), generator=g, device=DEV)]
    pages, table = _book(lens, 16, g)
    c = _filled(F, pages, 4, 16, 64, "e5m2", g)
    q = torch.randn(333, 8, 64, generator=g, device=DEV).bfloat16()
    _check_attention(F, c, lens, q, table, check=range(0, 333, 7))
    _check_attention(F, c, lens, q, table, max_context=128, check=range(0, 333, 7))


@pytest.mark.parametrize("B", [63, 64, 65, 128, 129])
def test_attention_batches_at_a_waves_width(F, B):
    """The lengths are scanned 64 at a time; one sequence in the middle is far longer than the rest."""
    g = W.gen(B, DEV)
    lens = [int(x) for x in torch.randint(0, 60, (B,), generator=g, device=DEV)]
    lens[B // 2], lens[-1] = 4999, 333
    pages, table = _book(lens, 16, g)
    c = _filled(F, pages, 1, 16, 32, "e4m3", g)
    q = torch.randn(B, 3, 32, generator=g, device=DEV).bfloat16()
    _check_attention(F, c, lens, q, table, out_dtype=torch.float32)


def test_attention_outputs_and_strides(F):
    """Outputs given by the caller, one query for all rows, a table that is a slice of a wider one, no context at all."""
    g = W.gen(16, DEV)
    lens = [70, 300, 9]
    pages, table = _book(lens, 16, g)
    c = _filled(F, pages, 2, 16, 64, "e5m2", g)
    lt = torch.tensor(lens, dtype=torch.int32, device=DEV)
    one = torch.randn(1, 4, 64, generator=g, device=DEV).bfloat16()
    want = F.fp8_paged_attention(one.repeat(3, 1, 1), c, table, lt)
    assert torch.equal(F.fp8_paged_attention(one.expand(3, 4, 64), c, table, lt), want)
    wide = torch.full((3, table.shape[1] + 5), -9, dtype=torch.int32, device=DEV)
    wide[:, 2:-3] = table
    assert torch.equal(F.fp8_paged_attention(one.expand(3, 4, 64), c, wide[:, 2:-3], lt), want)
    out, lse = torch.full((3, 4, 64), 7.0, device=DEV), torch.full((3, 4), 7.0, device=DEV)
    got = F.fp8_paged_attention(one.expand(3, 4, 64), c, table, lt, out_dtype=torch.float32, out=out, lse=lse,
                                max_context=0)
    assert got.data_ptr() == out.data_ptr() and not out.any() and (lse == -np.inf).all()
    short = F.fp8_paged_attention(one, c, table[:1, :1], lt[:1])          # one page of five
    assert torch.equal(short, F.fp8_paged_attention(one, c, table[:1], lt[:1], max_context=16))


def test_random_shapes(F):
    """Sizes, layouts, masks and formats drawn together."""
    import random
    rng = random.Random(7)
    for turn in range(40):
        g = W.gen(1000 + turn, DEV)
        H, G, D = rng.choice((1, 2, 3, 5)), rng.choice((1, 2, 3, 4, 7, 8, 16, 18, 33)), 16 * rng.randint(1, 16)
        S, B = rng.choice((16, 32, 128)), rng.choice((1, 2, 5, 17))
        most = rng.choice((20, 200, 2000))
        lens = [rng.randint(0, most) for _ in range(B)]
        pages, table = _book(lens, S, g, room=rng.choice((most, 6000)))
        c = _filled(F, pages, H, S, D, rng.choice(("e5m2", "e4m3")), g)
        q = (rng.choice((0.5, 3.0)) * torch.randn(B, H * G, D, generator=g, device=DEV)).bfloat16()
        print(turn, H, G, D, S, B, most, flush=True)
        _check_attention(F, c, lens, q, table, rng.choice((0, 0, 1, 40, 700)), rng.choice((torch.bfloat16, torch.float32)))


def test_attention_all_empty(F):
    g = W.gen(4, DEV)
    _, table = _book([0, 0, 0], 16, g)
    c = _filled(F, 3, 2, 16, 64, "e5m2", g)
    q = torch.randn(3, 4, 64, generator=g, device=DEV).bfloat16()
    _check_attention(F, c, [0, 0, 0], q, table)
    _check_attention(F, c, [0, -5, 0], q, table, max_context=32)
    out = F.fp8_paged_attention(q[:0], c, table[:0], torch.zeros(0, dtype=torch.int32, device=DEV))
    assert out.shape == (0, 4, 64)


def test_attention_sharp_and_flat_scores(F):
    """Scores so far apart that one token takes all, equal scores, a scale of
    zero and a negative one, maxima that grow along the sequence."""
    g = W.gen(5, DEV)
    n = 900
    pages, table = _book([n], 16, g)
    c = _filled(F, pages, 1, 16, 64, "e5m2", g)
    order = table[0, :-(-n // 16)].long()
    ramp = torch.linspace(0.01, 4.0, order.numel() * 16, device=DEV).view(-1, 16)
    c.k_scales[order, 0] *= ramp
    q = (20 * torch.randn(1, 4, 64, generator=g, device=DEV)).bfloat16()
    for scale in (None, 3.0, 0.0, -0.5):
        _check_attention(F, c, [n], q, table, scale=scale, out_dtype=torch.float32)


@pytest.mark.parametrize("fmt", ["e5m2", "e4m3"])
@pytest.mark.parametrize("max_context", [None, 250])
def test_what_is_not_seen_has_no_effect(F, fmt, max_context):
    """NaN and infinite codes and scales in every place that no sequence sees."""
    g = W.gen(6, DEV)
    lens, window = [5, 37, 250, 0], 20
    pages, table = _book(lens, 32, g)
    c = _filled(F, pages, 2, 32, 128, fmt, g)
    q = torch.randn(4, 8, 128, generator=g, device=DEV).bfloat16()
    lt = torch.tensor(lens, dtype=torch.int32, device=DEV)
    for win in (0, window):
        want = F.fp8_paged_attention(q, c, table, lt, window=win, max_context=max_context)
        seen = torch.zeros(pages, 32, dtype=torch.bool, device=DEV)
        for b, n in enumerate(lens):
            for t in range(max(0, n - win) if win else 0, n):
                seen[table[b, t // 32].long(), t % 32] = True
        dirty = F.KVCache.from_tensors(*(x.clone() for x in (c.k_codes, c.v_codes, c.k_scales, c.v_scales)), fmt)
        bad = ~seen[:, None].expand(pages, 2, 32)
        for codes, scales in ((dirty.k_codes, dirty.k_scales), (dirty.v_codes, dirty.v_scales)):
            codes[bad] = 0x7F                                            # NaN in both formats
            scales[bad] = float("nan")
        assert torch.equal(F.fp8_paged_attention(q, dirty, table, lt, window=win, max_context=max_context), want)
        if fmt == "e5m2":
            dirty.v_codes[bad] = 0x7C                                    # infinity
            dirty.k_codes[bad] = 0xFC
        dirty.k_scales[bad] = float("inf")
        dirty.v_scales[bad] = float("-inf")
        assert torch.equal(F.fp8_paged_attention(q, dirty, table, lt, window=win, max_context=max_context), want)


@pytest.mark.parametrize("max_context", [200, None])         # one workgroup a head; split and joined
def test_nan_among_the_seen(F, max_context):
    """A NaN in one query head, or in the K scale of a seen token, gives NaN there and nowhere else."""
    g = W.gen(8, DEV)
    lens = [150, 200, 37]
    n_cols = 400
    pages, table = _book([16 * n_cols] * 3, 16, g)
    c = _filled(F, pages, 2, 16, 64, "e5m2", g)
    q = torch.randn(3, 8, 64, generator=g, device=DEV).bfloat16()
    lt = torch.tensor(lens, dtype=torch.int32, device=DEV)

    def run():
        lse = torch.empty(3, 8, device=DEV)
        return F.fp8_paged_attention(q, c, table, lt, lse=lse, max_context=max_context), lse

    want, want_l = run()
    assert torch.isfinite(want).all() and torch.isfinite(want_l).all()
    q[1, 5, 3] = float("nan")
    c.k_scales[table[2, 1].long(), 0, 4] = float("nan")           # token 20 of sequence 2, KV head 0
    bad = torch.zeros(3, 8, dtype=torch.bool, device=DEV)
    bad[1, 5] = True
    bad[2, :4] = True
    out, lse = run()
    assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
    assert torch.equal(out[~bad], want[~bad]) and torch.equal(lse[~bad], want_l[~bad])


def test_attention_pages_that_are_none(F):
    """Page ids of seen tokens outside the cache: unspecified rows, no fault, other rows unharmed."""
    g = W.gen(7, DEV)
    lens = [40, 40, 500]
    pages, table = _book(lens, 16, g)
    c = _filled(F, pages, 2, 16, 64, "e5m2", g)
    q = torch.randn(3, 4, 64, generator=g, device=DEV).bfloat16()
    lt = torch.tensor(lens, dtype=torch.int32, device=DEV)
    want = F.fp8_paged_attention(q, c, table, lt)
    bad = table.clone()
    bad[1, 0], bad[1, 1], bad[1, 2] = -3, pages, 2 ** 31 - 1
    got = F.fp8_paged_attention(q, c, bad, lt)
    assert torch.equal(got[[0, 2]], want[[0, 2]])
    # lengths beyond the table are cut to it
    table = table[:, :32]
    cut = torch.tensor([40, 40, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    room = torch.tensor([40, 40, table.shape[1] * 16], dtype=torch.int32, device=DEV)
    assert torch.equal(F.fp8_paged_attention(q, c, table, cut), F.fp8_paged_attention(q, c, table, room))


def test_far_pages(F):
    """Pages beyond 4 GiB of codes: written, read and attended to at the end of a large cache."""
    S, H, D = 4096, 8, 128
    P = 1040
    c = F.KVCache(P, S, H, D, "e5m2", DEV)
    assert c.k_codes.numel() > 1 << 32
    g = W.gen(8, DEV)
    n = 50
    k, v = _rows(n, H, D, g), _rows(n, H, D, g)
    slots = (P - 1) * S + torch.arange(n, device=DEV)
    F.fp8_kv_cache_write(k, v, slots, c)
    table = torch.tensor([[P - 1]], dtype=torch.int32, device=DEV)
    offs = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    kb, vb = F.fp8_kv_cache_read(c, table, offs, n)
    q = torch.randn(1, 16, D, generator=g, device=DEV).bfloat16()
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    got = F.fp8_paged_attention(q, c, table, lens)
    small = F.KVCache(1, 64, H, D, "e5m2", DEV)
    F.fp8_kv_cache_write(k, v, torch.arange(n, device=DEV), small)
    zero = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    ks, vs = F.fp8_kv_cache_read(small, zero, offs, n)
    assert torch.equal(kb, ks) and torch.equal(vb, vs)
    want = F.fp8_paged_attention(q, small, zero, lens, out_dtype=torch.float32)
    assert (got.float() - want).abs().max() <= HB * want.abs().max()


# ---- together ------------------------------------------------------------------


class _Step:
    """A decode step of B sequences: inputs, cache and book."""

    def __init__(self, F, g, B=5, Hq=8, H=2, D=128, S=16, most=600, fmt="e5m2"):
        self.F = F
        self.lens = [int(x) for x in torch.randint(1, most, (B,), generator=g, device=DEV)]
        pages, self.table = _book([most] * B, S, g)
        self.c = _filled(F, pages, H, S, D, fmt, g)
        y = torch.randn(B, (Hq + 2 * H) * D, generator=g, device=DEV).bfloat16()
        self.y = y
        self.q = y[:, :Hq * D].view(B, Hq, D)
        self.k = y[:, Hq * D:(Hq + H) * D].view(B, H, D)
        self.v = y[:, (Hq + H) * D:].view(B, H, D)
        self.tab = _table(D, most)
        self.w = (torch.rand(D, generator=g, device=DEV) + 0.5).bfloat16()
        self.lt = torch.tensor(self.lens, dtype=torch.int32, device=DEV)
        self.S = S
        self.pos, self.slots = torch.empty(B, dtype=torch.int64, device=DEV), torch.empty(B, dtype=torch.int64, device=DEV)
        self.place()

    def place(self):
        """Positions and slots of the newest token for the present lengths."""
        last = self.lt.long() - 1
        self.pos.copy_(last)
        self.slots.copy_(self.table.gather(1, (last // self.S)[:, None])[:, 0] * self.S + last % self.S)

    def run(self, **k):
        return self.F.attention_step(self.q, self.k, self.v, self.tab, self.pos, self.slots, self.c, self.table,
                                     self.lt, self.w, self.w, 1e-6, **k)


@pytest.mark.parametrize("fmt", ["e5m2", "e4m3"])
def test_steps_in_a_row(F, fmt):
    """Several tokens one after the other: each step's output and cache from the parts checked above, and
    against the oracle on the cache as it stands."""
    g = W.gen(12, DEV)
    s = _Step(F, g, fmt=fmt)
    for _ in range(3):
        s.y.copy_(torch.randn(s.y.shape, generator=g, device=DEV).bfloat16())
        got = s.run()
        q2, k2 = F.fp8_qk_norm_rope(s.q, s.k, s.tab, s.pos, s.w, s.w)
        codes, d = A.quantise(_np(k2).astype(np.float32), fmt)
        page, place = s.slots // s.S, s.slots % s.S
        np.testing.assert_array_equal(s.c.k_codes[page, :, place].cpu().numpy(), codes)
        np.testing.assert_array_equal(s.c.k_scales[page, :, place].cpu().numpy(), d)
        out, _ = _check_attention(F, s.c, s.lens, q2, s.table)
        assert torch.equal(out, got)
        s.lens = [n + 1 for n in s.lens]
        s.lt += 1
        s.place()


@pytest.mark.parametrize("B,most", [(5, 100), (2, 2500), (40, 700), (70, 4200)])
def test_step_is_the_two_calls(F, B, most):
    g = W.gen(23, DEV)
    s = _Step(F, g, B=B, most=most)
    for k in (dict(), dict(window=50), dict(out_dtype=torch.float32, scale=0.3), dict(max_context=60)):
        got = s.run(**k)
        codes = s.c.k_codes.clone()
        q = F.fp8_qkv_cache_write(s.q, s.k, s.v, s.tab, s.pos, s.slots, s.c, s.w, s.w, 1e-6)
        assert torch.equal(s.c.k_codes, codes)
        assert torch.equal(F.fp8_paged_attention(q, s.c, s.table, s.lt, **k), got)


def test_a_refused_step_writes_nothing(F):
    s = _Step(F, W.gen(24, DEV), B=3)
    s.c.k_codes.fill_(0x5A)
    for k in (dict(window=-1), dict(scale=float("nan")), dict(max_context=-1), dict(out_dtype=torch.float16)):
        with pytest.raises((ValueError, F.Fp8Error)):
            s.run(**k)
    s.table = s.table[:2]
    with pytest.raises(ValueError):
        s.run()
    torch.cuda.synchronize()
    assert (s.c.k_codes == 0x5A).all()


def test_same_call_same_bits(F):
    g = W.gen(13, DEV)
    s = _Step(F, g, B=9, most=5000)
    first = s.run()
    for _ in range(3):
        assert torch.equal(s.run(), first)


def test_step_in_a_graph(F):
    """Captured, then replayed on other inputs and lengths, with eager work between, against eager results."""
    g = W.gen(14, DEV)
    a, b = _Step(F, g, most=3000), _Step(F, g, B=3, most=2000)
    for s in (a, b):
        s.run()
    torch.cuda.synchronize()
    graphs = []
    for s in (a, b):                                   # two graphs, replayed in turn
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            s.out = s.run()
        graphs.append(gr)
    for turn in range(4):
        for s, gr in zip((a, b), graphs):
            s.y.copy_(torch.randn(s.y.shape, generator=g, device=DEV).bfloat16())
            s.lt.copy_(torch.randint(1, 1900, s.lt.shape, generator=g, device=DEV))
            s.place()
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for s in (a, b):
            replayed = s.out.clone()
            assert torch.equal(s.run(), replayed), turn
            torch.cuda.synchronize()


def test_two_streams_at_once(F):
    g = W.gen(15, DEV)
    steps = [_Step(F, g, most=4000), _Step(F, g, most=4000)]
    want = [s.run() for s in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i].append(steps[i].run())
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(x, want[i]) for x in got[i])
