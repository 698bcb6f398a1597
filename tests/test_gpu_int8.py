"""The quantiser and the products in 8-bit integers on the GPU against the
64-bit oracle, and the expert layer as a whole.

Codes and scales are equal bit for bit.  A product's sum is exact; its fp32
value, the product of the scales and their product are each off by u = 2^-24 at
most, the bias and the rounding follow: |err| <= 3 u |v| + u (|v| + |bias|),
and u |ref| or, for bf16, h |ref| with h = 2^-8.
"""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import moe as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
U, H = 2.0 ** -24, 2.0 ** -8
bf16, f32, i8, i32 = torch.bfloat16, torch.float32, torch.int8, torch.int32
INF = float("inf")


@pytest.fixture(scope="module")
def F():
    import fp8_block_scaled_02_amd as F
    assert torch.cuda.is_available()
    return F


@pytest.fixture
def big():
    """Memory that others do not hold, given back afterwards."""
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def _np(t):
    return t.detach().double().cpu().numpy()


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _rand_codes(shape, g):
    return torch.randint(-128, 128, shape, generator=g, device=DEV, dtype=torch.int32).to(i8)


def _laid_out(codes, fill=77):
    """Codes [M, K] as int8_quant lays them out, the bytes from K on not zero."""
    M, K = codes.shape
    t = torch.full((M, -(-K // 128) * 128), fill, dtype=i8, device=DEV)
    t[:, :K] = codes
    return t[:, :K]


def _scales(n, g):
    return torch.exp2(4 * torch.rand(n, generator=g, device=DEV) - 10)


# ---- the quantiser -----------------------------------------------------------


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (5, 8), (9, 64), (4, 130), (300, 128), (33, 1000), (17, 2048),
                                 (6, 7168), (3, 8200), (2, 16384), (3, 16392), (2, 40000), (2, 40001)])
def test_quant(F, M, K, dtype):
    x = (torch.randn(M, K, generator=_gen(K), device=DEV) * torch.exp2(20 * torch.rand(M, 1, generator=_gen(1), device=DEV) - 10)).to(dtype)
    want = O.quantise(x.float().cpu().numpy())
    c, s = F.int8_quant(x)
    assert c.dtype == i8 and c.shape == (M, K) and (M == 1 or c.stride(0) % 128 == 0)
    assert np.array_equal(c.cpu().numpy(), want[0]) and np.array_equal(s.cpu().numpy(), want[1])
    for pad, at in ((8, 0), (3, 1)):                                   # aligned rows and others, in and out
        wide = torch.zeros(M, K + pad, dtype=dtype, device=DEV)
        wide[:, at:at + K] = x
        codes = torch.full((M, K + pad), 5, dtype=i8, device=DEV)
        got, gs = F.int8_quant(wide[:, at:at + K], codes[:, at:at + K], torch.empty(M, device=DEV))
        assert np.array_equal(got.cpu().numpy(), want[0]) and np.array_equal(gs.cpu().numpy(), want[1])
        assert (codes[:, :at] == 5).all() and (codes[:, at + K:] == 5).all()


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("M,K", [(2100, 8000), (17000, 1003), (140, 130001)])
def test_quant_large(F, M, K, dtype):
    x = torch.randn(M, K, generator=_gen(K), device=DEV).to(dtype)
    want = O.quantise(x.float().cpu().numpy())
    for t in (x, torch.nn.functional.pad(x, (1, 2))[:, 1:K + 1]):
        c, s = F.int8_quant(t)
        assert np.array_equal(c.cpu().numpy(), want[0]) and np.array_equal(s.cpu().numpy(), want[1])


def test_quant_past_32_bits(F, big):
    """Values past 2^31, in rows that would take 2^32 threads together."""
    M, K = (1 << 23) + 5, 4104
    x = torch.empty(M, K, dtype=bf16, device=DEV)
    x.copy_(torch.randn(1, K, generator=_gen(1), device=DEV))
    power = torch.tensor([2.0 ** (i - 5) for i in range(11)], device=DEV)[torch.arange(M, device=DEV) % 11]
    x *= power.to(bf16)[:, None]
    x[M - 2:] = torch.randn(2, K, generator=_gen(2), device=DEV).to(bf16)
    c, s = F.int8_quant(x)
    one, scale = F.int8_quant(x[5:6])                                   # times 1
    assert torch.equal(s[:M - 2], power[:M - 2] * scale)
    for lo in (0, 1_234_567, 1 << 22, M - 1002):
        assert (c[lo:lo + 1000] == one).all()
    want = O.quantise(x[M - 2:].float().cpu().numpy())
    assert np.array_equal(c[M - 2:].cpu().numpy(), want[0]) and np.array_equal(s[M - 2:].cpu().numpy(), want[1])


def test_outputs_hold_no_others_memory(F, big):
    """Scales and weights kept after what came with them is dropped hold their own bytes only, but for small calls."""
    x = torch.zeros(512, 1 << 16, dtype=bf16, device=DEV)
    c, s = F.int8_quant(x)
    assert s.untyped_storage().nbytes() == 2048 and c.untyped_storage().nbytes() == 512 << 16
    r = F.moe_route(torch.zeros(1 << 17, 8, device=DEV), 2)
    assert r.gates.untyped_storage().nbytes() == 1 << 20
    parts = [t for t in (*F.moe_route(torch.zeros(5, 9, device=DEV), 3), *F.int8_quant(x[:3, :200]))]
    for i, a in enumerate(parts):
        for b in parts[:i]:
            assert a.data_ptr() >= b.data_ptr() + b.numel() * b.element_size() or b.data_ptr() >= a.data_ptr() + a.numel() * a.element_size()


def test_quant_at_halves(F):
    """Quotients at and next to a half, for many scales: the whole number
    nearest to the fp32 quotient."""
    g = _gen(2)
    rows = []
    for i in range(512):
        amax = torch.exp2(torch.rand(1, generator=g, device=DEV) * 60 - 30)
        d = amax / torch.full_like(amax, 127.0)
        half = (torch.arange(0, 126, device=DEV) + 0.5) * d
        near = torch.cat((half, torch.nextafter(half, torch.full_like(half, INF)), torch.nextafter(half, torch.zeros_like(half))))
        rows.append(torch.cat((amax, near, -near)))
    x = torch.stack(rows)
    want = O.quantise(x.cpu().numpy())
    c, s = F.int8_quant(x)
    assert np.array_equal(s.cpu().numpy(), want[1]) and np.array_equal(c.cpu().numpy(), want[0])


def test_quant_of_every_bf16_pair_of_some_scales(F):
    """Every bf16 magnitude up to the maximum, for maxima of every fraction and many exponents."""
    top = torch.cat([torch.arange(128, device=DEV) + 128 * e for e in (0, 1, 65, 66, 90, 127, 130, 200, 254)]).to(torch.int16)
    every = torch.arange(0x7F80, device=DEV, dtype=torch.int32)
    for part in top.split(256):
        x = every[None].repeat(part.numel(), 1)
        x = torch.where(x <= part[:, None], x, part[:, None].int())
        x = torch.where(torch.arange(0x7F80, device=DEV) % 2 == 0, x, x | 0x8000)
        x = (x << 16).to(torch.int32).view(f32).to(bf16)
        want = O.quantise(x.float().cpu().numpy())
        c, s = F.int8_quant(x)
        assert np.array_equal(s.cpu().numpy(), want[1]) and np.array_equal(c.cpu().numpy(), want[0])


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("K", [5, 64, 3000, 20000])
def test_quant_special_rows(F, K, dtype):
    x = torch.randn(12, K, generator=_gen(3), device=DEV)
    x[0] = 0.0
    x[1] = -0.0
    x[2, K // 2] = INF
    x[3, K - 1] = -INF
    x[4, 0] = float("nan")
    x[5, K // 3], x[5, 0] = float("nan"), INF
    x[6] *= 1e-38
    x[7] *= 2.0 ** -140                                                # subnormal
    x[8] = 2.0 ** -149
    x[9] = torch.finfo(dtype).max * torch.sign(x[9])
    x[10] *= 2.0 ** -62
    x = x.to(dtype)
    want = O.quantise(x.float().cpu().numpy())
    c, s = F.int8_quant(x)
    assert np.array_equal(s.cpu().numpy(), want[1], equal_nan=True) and np.array_equal(c.cpu().numpy(), want[0])


@pytest.mark.parametrize("G,N,K", [(1, 1, 1), (1, 16, 128), (3, 17, 129), (2, 100, 64), (1, 33, 1480), (5, 48, 256)])
def test_weight_pack(F, G, N, K):
    w = _rand_codes((G, N, K), _gen(N))
    got = F.int8_weight_pack(w)
    want = np.stack([O.packed(m) for m in w.cpu().numpy()])
    assert got.dtype == i8 and np.array_equal(got.cpu().numpy(), want)
    wide = torch.full((G, N + 2, K + 5), 9, dtype=i8, device=DEV)
    wide[:, 1:N + 1, 3:K + 3] = w
    out = torch.empty_like(got)
    assert F.int8_weight_pack(wide[:, 1:N + 1, 3:K + 3], out=out) is out and torch.equal(out, got)
    if G == 1:
        assert torch.equal(F.int8_weight_pack(w[0]), got[0])
    # a matrix shared by every expert
    assert torch.equal(F.int8_weight_pack(w[:1].expand(4, N, K)), got[:1].expand(4, -1, -1))


# ---- the products ------------------------------------------------------------


def _tol(v, bias, ref, out):
    return 3 * U * np.abs(v) + U * (np.abs(v) + np.abs(bias)) + (H if out == bf16 else U) * np.abs(ref)


def _check_gemm(F, M, N, K, out, with_bias, seed=0, a=None, w=None):
    g = _gen(seed)
    a = _rand_codes((M, K), g) if a is None else a
    w = _rand_codes((N, K), g) if w is None else w
    sa, sw = _scales(M, g), _scales(N, g)
    bias = torch.randn(N, generator=g, device=DEV) if with_bias else None
    y = F.int8_gemm(_laid_out(a), sa, F.int8_weight_pack(w), sw, bias, out)
    assert y.dtype == out and y.shape == (M, N)
    v = O.product(a.cpu().numpy(), w.cpu().numpy()) * _np(sa)[:, None] * _np(sw)
    b = _np(bias) if with_bias else np.zeros(N)
    ref = v + b
    assert (np.abs(_np(y) - ref) <= _tol(v, b, ref, out)).all()
    return y


MS = [1, 2, 3, 7, 8, 15, 16, 17, 31, 32, 33, 47, 48, 63, 64, 65, 100, 127, 128, 129, 191, 200, 255, 256, 257, 300, 511, 513]


@pytest.mark.parametrize("M", MS)
def test_gemm_rows(F, M):
    _check_gemm(F, M, 272, 384, bf16, False, M)


@pytest.mark.parametrize("out", [bf16, f32])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (1, 5, 3), (2, 16, 64), (1, 4096, 4096), (5, 17, 65), (16, 1001, 1480), (101, 1001, 1480), (33, 2000, 127),
    (70, 31, 2500), (130, 515, 128), (257, 300, 1000), (300, 1023, 640), (1000, 260, 192), (64, 4097, 700), (3, 2100, 9000),
    (520, 777, 900)])
def test_gemm(F, M, N, K, out, bias):
    _check_gemm(F, M, N, K, out, bias, M + N + K)


@pytest.mark.parametrize("out,bias", [(bf16, False), (f32, True)])
@pytest.mark.parametrize("panels", range(1, 9))
def test_gemm_streamed(F, panels, out, bias):
    """Few rows of outputs so wide that a workgroup has 1 to 8 panels."""
    N = 4096 * panels - 5 * panels
    for M, K in ((1, 64), (16, 200), (17, 1100), (32, 2600)):
        _check_gemm(F, M, N, K, out, bias, panels)


@pytest.mark.parametrize("out,bias", [(bf16, False), (f32, True)])
@pytest.mark.parametrize("M,N", [(250, 16600), (2050, 4101), (4200, 2048), (100, 16400), (65, 20001), (300, 5000),
                                 (900, 1700), (200, 6001)])
def test_gemm_tiles(F, M, N, out, bias):
    """The larger tiles, with one step of K, each number of steps up to the
    ring's length, and some past it."""
    for K in (100, 256, 300, 512, 640, 700, 800, 1000, 1500):
        _check_gemm(F, M, N, K, out, bias, K)


@pytest.mark.parametrize("out,bias", [(bf16, True), (f32, False)])
@pytest.mark.parametrize("M,N", [(17, 64), (33, 130), (101, 1001), (250, 2000), (31, 16384)])
def test_gemm_small_tiles(F, M, N, out, bias):
    """Tiles of 32 x 64, by one group of waves and by two that take the steps
    in turn, with even and odd numbers of steps."""
    for K in (77, 1000, 2047, 2048, 2100, 2200, 2304, 2500, 4000, 8200):
        _check_gemm(F, M, N, K, out, bias, K)


@pytest.mark.parametrize("out", [bf16, f32])
@pytest.mark.parametrize("M,N", [(250, 16602), (2050, 4098), (300, 5002)])
def test_gemm_tiles_into_strided_rows(F, M, N, out):
    K, g = 400, _gen(M)
    a, wp = _laid_out(_rand_codes((M, K), g)), F.int8_weight_pack(_rand_codes((N, K), g))
    sa, sw = _scales(M, g), _scales(N, g)
    want = F.int8_gemm(a, sa, wp, sw, None, out)
    for ld, at in ((N + 1, 1), (N + 6, 0), (N + 30, 8)):
        y = torch.full((M, ld), 4.0, dtype=out, device=DEV)
        F.int8_gemm(a, sa, wp, sw, None, out, y[:, at:at + N])
        assert torch.equal(y[:, at:at + N], want) and (y[:, :at] == 4).all() and (y[:, at + N:] == 4).all()


@pytest.mark.parametrize("M,N", [(70000, 33000), (17, 20_000_000)])
def test_gemm_past_32_bits(F, big, M, N):
    """Results, or weights, past 2^31 bytes: parts are those of the part alone."""
    K, g = 128, _gen(M)
    a, wp = _rand_codes((M, K), g), F.int8_weight_pack(_rand_codes((N, K), g))
    sa, sw = _scales(M, g), _scales(N, g)
    y = F.int8_gemm(a, sa, wp, sw)
    w = wp.view(2, -1, 1024)
    for lo in (0, N // 2 // 16 * 16, N // 16 * 16 - 512):
        part = w[:, lo // 16:lo // 16 + 32].contiguous().view(512, K)
        for m in (0, M // 2, M - 17):
            assert torch.equal(y[m:m + 17, lo:lo + 512], F.int8_gemm(a[m:m + 17], sa[m:m + 17], part, sw[lo:lo + 512]))


def test_grouped_past_32_bits(F, big):
    """Weights of 5 GB, rows of 4 GB: every expert has the same matrix, and
    rows of the same token are equal."""
    E, N, K, T, R = 160, 2048, 16384, 500, 1 << 20
    g = _gen(9)
    w = _rand_codes((N, K), g)
    a = _rand_codes((T, K), g)
    sa, sw = _scales(T, g), _scales(N, g)
    wp = F.int8_weight_pack(w.expand(E, N, K))
    swe = sw.expand(E, N).contiguous()
    index = torch.randint(0, T, (R,), generator=g, device=DEV).int()
    offs = torch.sort(torch.randint(0, R, (E + 1,), generator=g, device=DEV)).values.int()
    offs[0], offs[-1] = 0, R
    want = F.int8_gemm(a, sa, wp[0], sw)
    y = F.int8_grouped_gemm(a, sa, index, offs, wp, swe)
    for lo in range(0, R, 1 << 18):
        assert torch.equal(y[lo:lo + (1 << 18)], want[index[lo:lo + (1 << 18)].long()])
    few = torch.arange(E + 1, device=DEV).int()                         # a row of each expert
    assert torch.equal(F.int8_grouped_gemm(a, sa, index[:E], few, wp, swe), want[index[:E].long()])


@pytest.mark.parametrize("M", [1, 40, 300])
def test_gemm_largest_sums(F, M):
    """Codes of -128 and 127 everywhere at the largest K: sums at the ends of 32 bits."""
    K = 131071
    a = torch.full((M, K), -128, dtype=i8, device=DEV)
    w = torch.full((33, K), -128, dtype=i8, device=DEV)
    w[1::2] = 127
    _check_gemm(F, M, 33, K, f32, False, 3, a, w)


@pytest.mark.parametrize("M,N,K", [(1, 7168, 2048), (32, 4096, 7168), (128, 2048, 1024), (512, 1024, 2048)])
def test_gemm_repeats_itself(F, M, N, K):
    g = _gen(4)
    a, wp = _laid_out(_rand_codes((M, K), g)), F.int8_weight_pack(_rand_codes((N, K), g))
    sa, sw = _scales(M, g), _scales(N, g)
    first = F.int8_gemm(a, sa, wp, sw)
    for _ in range(5):
        assert torch.equal(F.int8_gemm(a, sa, wp, sw), first)


@pytest.mark.parametrize("out", [bf16, f32])
@pytest.mark.parametrize("M", [3, 80, 270])
def test_gemm_strides_and_given_output(F, M, out):
    """Codes as columns of a wider matrix, rows of y apart by any stride, at any
    address, and what lies between left as it was."""
    N, K = 203, 256
    g = _gen(M)
    a, w = _rand_codes((M, K), g), _rand_codes((N, K), g)
    sa, sw = _scales(M, g), _scales(N, g)
    wp = F.int8_weight_pack(w)
    want = F.int8_gemm(a, sa, wp, sw, None, out)
    wide = _rand_codes((M, 3 * K), g)
    wide[:, K:2 * K] = a
    for ld, at in ((N, 0), (N + 1, 1), (N + 5, 0), (N + 53, 16)):
        y = torch.full((M, ld), 4.0, dtype=out, device=DEV)
        v = y[:, at:at + N]
        assert F.int8_gemm(wide[:, K:2 * K], sa, wp, sw, None, out, v) is v
        assert torch.equal(v, want) and (y[:, :at] == 4).all() and (y[:, at + N:] == 4).all()


def test_gemm_rows_that_are_no_numbers(F):
    """A row with a NaN or an infinity gives NaN, and no other row does."""
    x = torch.randn(70, 300, generator=_gen(5), device=DEV)
    x[3, 5], x[40, 299] = float("nan"), INF
    w, sw = F.int8_quant(torch.randn(50, 300, generator=_gen(6), device=DEV))
    y = F.int8_linear(x, F.int8_weight_pack(w), sw)
    bad = torch.isnan(y).all(1)
    assert bad.nonzero()[:, 0].tolist() == [3, 40] and torch.isfinite(y[~bad]).all()


def test_linear_is_its_parts(F):
    for M, N, K, dt in ((1, 260, 500, bf16), (19, 260, 512, f32), (200, 300, 1000, bf16)):
        g = _gen(M)
        x = W.activations(M, K, 3, 50.0, g).to(dt)
        c, sw = F.int8_quant(torch.randn(N, K, generator=g, device=DEV) * 0.02)
        wp = F.int8_weight_pack(c)
        b = torch.randn(N, generator=g, device=DEV)
        a, sa = F.int8_quant(x)
        for out in (bf16, f32):
            assert torch.equal(F.int8_linear(x, wp, sw, b, out), F.int8_gemm(a, sa, wp, sw, b, out))
    assert F.int8_linear(x[:0], wp, sw).shape == (0, 300)


# ---- per expert --------------------------------------------------------------


def _check_grouped(F, T, counts, N, K, out, seed=0, spare=0, direct=False):
    """Rows of each expert as counts says, `spare` rows behind the last one's."""
    g = _gen(seed)
    E, R = len(counts), sum(counts) + spare
    T = R if direct else T
    a, w = _rand_codes((T, K), g), _rand_codes((E, N, K), g)
    sa, sw = _scales(T, g), _scales(E * N, g).view(E, N)
    offs = torch.tensor([0] + list(np.cumsum(counts)), device=DEV).int()
    index = torch.arange(R, device=DEV).int() if direct else torch.randint(0, T, (R,), generator=g, device=DEV).int()
    y = torch.full((R, N), 5.0, dtype=out, device=DEV)
    got = F.int8_grouped_gemm(_laid_out(a), sa, None if direct else index, offs, F.int8_weight_pack(w), sw, out, y)
    assert got is y and (y[R - spare:] == 5).all()
    at = index.cpu().numpy()
    for e, n in enumerate(counts):
        lo = int(offs[e])
        rows = at[lo:lo + n]
        v = O.product(a.cpu().numpy()[rows], w[e].cpu().numpy()) * _np(sa)[rows][:, None] * _np(sw)[e]
        assert (np.abs(_np(y[lo:lo + n]) - v) <= _tol(v, 0, v, out)).all(), (e, n)


@pytest.mark.parametrize("out", [bf16, f32])
@pytest.mark.parametrize("N,K", [(64, 128), (250, 200), (33, 1000)])
@pytest.mark.parametrize("counts", [
    [1], [0, 3, 0], [16, 17, 1, 0, 15, 33], [64, 65, 63, 129, 2], [200, 0, 0, 1, 300], [0, 0, 0], [128, 256, 31, 512],
    [1] * 40, [0] * 300 + [9] + [0] * 723])
def test_grouped(F, counts, N, K, out):
    if len(counts) > 1000:
        N, K = min(N, 64), 128
    _check_grouped(F, 37, counts, N, K, out, sum(counts), spare=6)
    _check_grouped(F, 0, counts, N, K, out, 1, spare=3, direct=True)


@pytest.mark.parametrize("out", [bf16, f32])
@pytest.mark.parametrize("N,K", [(1800, 100), (1793, 700), (1808, 1100), (2048, 512)])
@pytest.mark.parametrize("counts", [
    [1, 31, 32, 33, 64, 65, 127, 128, 129, 160, 161, 200, 300] + [0] * 27, [0] * 19 + [700] + [0] * 20, [0] * 40, [3] * 40,
    [128] * 10 + [0, 1] * 15, [40] * 40, [1000, 0, 17] + [70] * 37])
def test_grouped_tiles(F, counts, N, K, out):
    """Experts and columns enough for tiles: pieces of every kind."""
    _check_grouped(F, 37, counts, N, K, out, sum(counts), spare=40)
    _check_grouped(F, 0, counts, N, K, out, 1, spare=45, direct=True)


def test_grouped_of_many_experts(F):
    rng = np.random.default_rng(3)
    counts = [int(c) for c in np.minimum(rng.zipf(1.5, 1024), 400) * (rng.random(1024) < 0.6)]
    _check_grouped(F, 500, counts, 70, 128, bf16, 3, spare=9)
    _check_grouped(F, 500, [c // 4 for c in counts[:700]], 300, 130, f32, 4, spare=9)


@pytest.mark.parametrize("out", [bf16, f32])
@pytest.mark.parametrize("E,N", [(6, 203), (40, 1803)])
def test_grouped_strides_and_given_output(F, E, N, out):
    g, K, T, R = _gen(N), 256, 60, 333
    a, w = _rand_codes((T, K), g), _rand_codes((E, N, K), g)
    sa, sw = _scales(T, g), _scales(E * N, g).view(E, N)
    index = torch.randint(0, T, (R,), generator=g, device=DEV).int()
    offs = torch.sort(torch.randint(0, R + 1, (E + 1,), generator=g, device=DEV)).values.int()
    offs[0] = 0
    end = int(offs[-1])
    wp = F.int8_weight_pack(w)
    want = F.int8_grouped_gemm(a, sa, index, offs, wp, sw, out)
    wide = _rand_codes((T, 3 * K), g)
    wide[:, K:2 * K] = a
    for ld, at in ((N, 0), (N + 1, 1), (N + 5, 0), (N + 53, 16)):
        y = torch.full((R, ld), 4.0, dtype=out, device=DEV)
        F.int8_grouped_gemm(wide[:, K:2 * K], sa, index, offs, wp, sw, out, y[:, at:at + N])
        assert torch.equal(y[:end, at:at + N], want[:end]) and (y[end:] == 4).all()
        assert (y[:, :at] == 4).all() and (y[:, at + N:] == 4).all()


@pytest.mark.parametrize("seed", range(4))
def test_grouped_skewed(F, seed):
    rng = np.random.default_rng(seed)
    counts = [int(c) for c in np.minimum(rng.zipf(1.3, 24), 700) * (rng.random(24) < 0.8)]
    _check_grouped(F, 200, counts, int(rng.integers(1, 400)), int(rng.integers(1, 900)), bf16, seed, spare=11)


@pytest.mark.parametrize("E,N", [(5, 70), (40, 1800)])
def test_grouped_contract_broken(F, E, N):
    """Offsets and tokens outside their ranges: unspecified rows, no others touched."""
    g = _gen(7)
    T, K, R = 20, 128, 60
    a, wp = _laid_out(_rand_codes((T, K), g)), F.int8_weight_pack(_rand_codes((E, N, K), g))
    sa, sw = _scales(T, g), _scales(E * N, g).view(E, N)
    index = torch.randint(-5, T + 5, (R,), generator=g, device=DEV).int()
    for offs in ([0, 10, 5, 30, 20, 60], [-4, 3, 9, 400, 2 ** 31 - 1, 70], [9, 8, 7, 6, 5, 4], [-2 ** 31] * 6):
        room = torch.full((R + 40, N), 5.0, device=DEV)
        offs = offs + offs[-1:] * (E - 5)
        F.int8_grouped_gemm(a, sa, index, torch.tensor(offs, device=DEV).int(), wp, sw, f32, room[20:20 + R])
        torch.cuda.synchronize()
        assert (room[:20] == 5).all() and (room[20 + R:] == 5).all()
    assert F.int8_grouped_gemm(a, sa, index[:0], torch.zeros(E + 1, device=DEV).int(), wp, sw).shape == (0, N)


# ---- together ----------------------------------------------------------------


@pytest.mark.parametrize("T,E,k,K,N,renorm", [(1, 8, 2, 256, 200, True), (5, 256, 8, 512, 96, True), (70, 12, 3, 300, 129, False),
                                              (600, 16, 4, 256, 256, True)])
@pytest.mark.parametrize("odt", [bf16, f32])
def test_expert_layer(F, T, E, k, K, N, renorm, odt):
    """The layer's call is its parts' calls, and those are the definition."""
    g = _gen(T)
    x = W.activations(T, K, 2, 20.0, g)
    l = torch.randn(T, E, generator=g, device=DEV)
    l[3::7] = -INF
    w = torch.randn(E, N, K, generator=g, device=DEV) * 0.02
    c, sw = F.int8_quant(w.view(E * N, K))
    c, sw = c.reshape(E, N, K), sw.view(E, N)
    wp = F.int8_weight_pack(c)
    out, r = F.int8_moe_forward(x, l, k, wp, sw, renorm, odt)
    r2 = F.moe_route(l, k, renorm)
    assert all(torch.equal(p, q) for p, q in zip(r, r2))
    a, sa = F.int8_quant(x)
    y = F.int8_grouped_gemm(a, sa, r.row_index, r.expert_offsets, wp, sw, odt)
    assert out.dtype == odt and torch.equal(F.moe_combine(y, r.token_rows, r.gates), out)
    oc, os = O.quantise(x.float().cpu().numpy())
    experts = O.choose(_np(l), k)
    gates, dist = O.gates(_np(l), experts, renorm)
    ref, mag = np.zeros((T, N)), np.zeros((T, N))
    for e in range(E):
        v = O.product(oc, c[e].cpu().numpy()) * os[:, None].astype(np.float64) * _np(sw)[e]
        share = (gates * (experts == e)).sum(1)[:, None]
        ref += share * v
        mag += np.abs(share * v)
    # rows rounded to the output's type, products off by 4 u, weights by u (d + 2 n + 8), k sums
    h = H if odt == bf16 else U
    tol = mag * (h + U * (4 + dist.max() + 2 * (k if renorm else E) + 8 + k)) * (1 + h) + h * np.abs(ref)
    assert (np.abs(_np(out) - ref) <= tol).all()
    assert F.int8_moe_forward(x[:0], l[:0], k, wp, sw)[0].shape == (0, N)


def test_the_plan_drives_the_fp8_layer(F):
    """The router's plan in the block-scaled layer, whose combine is this one's."""
    T, E, k, N, K = 150, 20, 4, 256, 512
    g = _gen(21)
    x = torch.randn(T, K, generator=g, device=DEV).to(bf16)
    l = torch.randn(T, E, generator=g, device=DEV)
    l[::10] = -INF
    r = F.moe_route(l, k)
    w = (torch.randn(E * N, K, generator=g, device=DEV) * 0.02).to(bf16)
    wq, ws = F.fp8_weight_quant(w)
    wq, ws = wq.view(E, N, K), ws.view(E, N // 128, K // 128)
    a, sa = F.fp8_act_quant(x)
    # the layer's own combine wants a row for every slot: those of tokens without experts weigh nothing
    y = F.fp8_grouped_gemm(a, sa, r.row_index.clamp(min=0), r.expert_offsets, wq, ws, bf16, torch.zeros(T * k, N, dtype=bf16, device=DEV))
    out = F.moe_combine(y, r.token_rows, r.gates)
    assert torch.equal(out, F.fp8_moe_combine(y, r.token_rows.clamp(min=0), r.gates)) and not out[::10].any()
    live = [t for t in range(T) if t % 10]
    for t in live[::17]:
        for j in range(k):
            e, row = int(r.experts[t, j]), y[r.token_rows[t, j]].float()
            ref = F.fp8_block_gemm(a[t:t + 1], sa[t:t + 1], wq[e], ws[e], f32)[0]
            # either's sums of K products (codes add an eighth to a factor at most), and the row's rounding
            mag = x[t].float().abs() @ w.view(E, N, K)[e].float().abs().T * 1.27
            assert ((row - ref).abs() <= 2 * K * U * mag + H * ref.abs()).all()


def test_a_training_step_of_the_routing(F):
    """Forward and backward through gather, combine and router against torch's
    autograd in 64 bits on the same choice of experts."""
    T, E, k, N = 90, 10, 3, 40
    g = _gen(14)
    l, x, dout = (torch.randn(s, generator=g, device=DEV) for s in ((T, E), (T, N), (T, N)))
    l[::9] = -INF
    scale = 1 + torch.arange(E, device=DEV)                             # an expert is a factor
    r = F.moe_route(l, k)
    rows = F.moe_gather(x, r.token_rows, out=torch.zeros(T * k, N, device=DEV))
    live = int(r.expert_offsets[-1])
    e_of_row = torch.searchsorted(r.expert_offsets[1:].contiguous(), torch.arange(live, device=DEV).int(), right=True)
    f = torch.zeros(T * k, 1, device=DEV)
    f[:live, 0] = scale[e_of_row].float()
    y = rows * f
    out = F.moe_combine(y, r.token_rows, r.gates)
    dy, dg = F.moe_combine_backward(dout, y, r.token_rows, r.gates, dy=torch.zeros_like(y))
    dx = F.moe_gather_backward(dy * f, r.token_rows)
    dl = F.moe_route_backward(dg, l, r.gates, r.experts)
    lx, xx = l.double().cpu().requires_grad_(), x.double().cpu().requires_grad_()
    ex = r.experts.cpu().long()
    keep = (ex >= 0).double()
    z = torch.where(ex >= 0, lx.gather(1, ex.clamp(min=0)), -INF)
    top = z.amax(1, keepdim=True).detach()
    p = torch.exp(z - torch.where(top == -INF, 0.0, top)) * keep
    w = p / p.sum(1, keepdim=True).clamp(min=1e-300)
    ref = (w[..., None] * scale.cpu().double()[ex.clamp(min=0)][..., None] * xx[:, None]).sum(1)
    ref.backward(dout.double().cpu())
    # each result: at most N / 256 + 2 k + 30 roundings of its terms, whose magnitudes sum to at most these
    many = U * (N / 256 + 2 * k + 30)
    big = scale.max().item()
    assert ((out.cpu().double() - ref).abs() <= many * big * x.cpu().double().abs()).all()
    assert ((dx.cpu().double() - xx.grad).abs() <= many * big * dout.cpu().double().abs()).all()
    reach = (dout.abs() * x.abs()).sum(1, keepdim=True).cpu().double() * big
    assert ((dl.cpu().double() - lx.grad).abs() <= 4 * many * reach).all()


def _layer_calls(F, T=33, E=20, k=4, K=256, N=130, seed=15):
    g = _gen(seed)
    x = torch.randn(T, K, generator=g, device=DEV).to(bf16)
    l = torch.randn(T, E, generator=g, device=DEV)
    wp = F.int8_weight_pack(_rand_codes((E, N, K), g))
    sw = _scales(E * N, g).view(E, N)
    wd, swd = F.int8_weight_pack(_rand_codes((N, K), g)), _scales(N, g)
    dout = torch.randn(T, N, generator=g, device=DEV).to(bf16)
    held = torch.zeros(T * k, N, dtype=bf16, device=DEV)

    def run():
        out, r = F.int8_moe_forward(x, l, k, wp, sw)
        y = F.moe_gather(dout, r.token_rows, out=held)
        dy, dg = F.moe_combine_backward(dout, y, r.token_rows, r.gates, dy=torch.zeros_like(held))
        dl = F.moe_route_backward(dg, l, r.gates, r.experts)
        dx = F.moe_gather_backward(dy, r.token_rows)
        z = F.int8_linear(x, wd, swd)
        return [out, *r, y.clone(), dy, dg, dl, dx, z]

    return run, (x, l, dout)


@pytest.mark.parametrize("T", [3, 33, 700])
def test_captured_and_replayed(F, T):
    """All calls in one graph, replayed on changed inputs with eager work between."""
    run, ins = _layer_calls(F, T=T)
    run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = run()
    for i in range(4):
        for j, t in enumerate(ins):
            t.copy_(torch.randn(t.shape, generator=_gen(100 * i + j), device=DEV).to(t.dtype))
        if i == 2:
            ins[1][1::3] = -INF
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        want = run()
        torch.cuda.synchronize()
        for a, b in zip(kept, want):
            assert torch.equal(a, b)


def test_on_two_streams_at_once(F):
    """Two layers' calls on streams of their own give what each gives alone."""
    runs = [_layer_calls(F, T=t, seed=t)[0] for t in (40, 900)]
    want = [r() for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    got = [None, None]
    for _ in range(6):
        for i, (r, s) in enumerate(zip(runs, streams)):
            with torch.cuda.stream(s):
                got[i] = r()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
