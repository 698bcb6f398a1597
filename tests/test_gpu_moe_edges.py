"""Expert routing and the integer layers at the edges of their ranges, on the
GPU against the 64-bit oracle.

Tolerances as where the operators are tested in general: u = 2^-24, a rounding
of fp32; h = 2^-8, one of bf16.
"""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import moe as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
U, H = 2.0 ** -24, 2.0 ** -8
bf16, f32, i8 = torch.bfloat16, torch.float32, torch.int8
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def F():
    import fp8_block_scaled_02_amd as F
    assert torch.cuda.is_available()
    return F


def _np(t):
    return t.detach().double().cpu().numpy()


def _ints(t):
    return t.detach().cpu().numpy()


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


# ---- the expert layer's rows --------------------------------------------------


@pytest.mark.parametrize("T,E,k,K,N,renorm", [(1, 8, 2, 256, 200, True), (7, 256, 8, 512, 1800, True), (70, 12, 3, 300, 129, False),
                                              (600, 16, 8, 256, 256, True)])
def test_layer_rounds_once(F, T, E, k, K, N, renorm):
    """By default the experts' rows keep 32 bits: nothing but the output is
    rounded to bf16.

    A row is off by 3 u (its sum's conversion and two products), a weight by
    u (d + 2 n + 8), the k fused multiply-adds by k u, all of the sum of
    magnitudes; their products are below 2^-10 of that.  Then h |out|."""
    g = _gen(T + N)
    x = W.activations(T, K, 2, 20.0, g)
    l = torch.randn(T, E, generator=g, device=DEV)
    l[3::7] = -INF
    w = torch.randn(E * N, K, generator=g, device=DEV) * 0.02
    c, sw = F.int8_quant(w)
    c, sw = c.reshape(E, N, K), sw.view(E, N)
    out, r = F.int8_moe_forward(x, l, k, F.int8_weight_pack(c), sw, renorm)
    assert out.dtype == bf16
    oc, os = O.quantise(x.float().cpu().numpy())
    experts = O.choose(_np(l), k)
    gates, dist = O.gates(_np(l), experts, renorm)
    ref, mag = np.zeros((T, N)), np.zeros((T, N))
    for e in range(E):
        v = O.product(oc, c[e].cpu().numpy()) * os[:, None].astype(np.float64) * _np(sw)[e]
        share = (gates * (experts == e)).sum(1)[:, None]
        ref += share * v
        mag += np.abs(share * v)
    err = mag * U * (3 + dist.max() + 2 * (k if renorm else E) + 8 + k) * (1 + 2.0 ** -10)
    assert (np.abs(_np(out) - ref) <= err + H * (np.abs(ref) + err)).all()
    # rows of a type that the caller chooses: the parts' calls with it
    a, sa = F.int8_quant(x)
    for rows, odt in ((f32, bf16), (bf16, bf16), (bf16, f32), (f32, f32)):
        y = F.int8_grouped_gemm(a, sa, r.row_index, r.expert_offsets, F.int8_weight_pack(c), sw, rows)
        got, _ = F.int8_moe_forward(x, l, k, F.int8_weight_pack(c), sw, renorm, odt, rows)
        assert got.dtype == odt and torch.equal(got, F.moe_combine(y, r.token_rows, r.gates, odt))
        if (rows, odt) == (f32, bf16):
            assert torch.equal(got, out)


# ---- the router's gradient ------------------------------------------------------


@pytest.mark.parametrize("E", [9, 60, 200, 700])
@pytest.mark.parametrize("dtype", [bf16, f32])
def test_gradient_of_tokens_without_experts(F, E, dtype):
    """Zeros, whatever their logits and the gates' gradient are."""
    T, k = 40, 4
    l = torch.randn(T, E, generator=_gen(E), device=DEV).to(dtype)
    l[::5, E // 2] = NAN
    l[1::5, 0] = INF
    l[2::5] = -INF
    for renorm in (True, False):
        r = F.moe_route(l, k, renorm)
        experts, gates = r.experts.clone(), r.gates.clone()
        experts[:30], gates[:30] = -1, 0.0
        experts[25:30] = E + 5                                                       # ids outside: none either
        d = torch.randn(T, k, generator=_gen(1), device=DEV)
        d[10:20] = NAN
        got = F.moe_route_backward(d, l, gates, experts, renorm)
        assert (got[:30] == 0).all()
        assert torch.equal(got[30:].nan_to_num(7.0), F.moe_route_backward(d, l, r.gates, r.experts, renorm)[30:].nan_to_num(7.0))


class Experts(torch.autograd.Function):
    """Tokens to their experts and back, weighted: a user's training step."""

    @staticmethod
    def forward(ctx, x, logits, scale, k, renorm):
        import fp8_block_scaled_02_amd as F
        r = F.moe_route(logits, k, renorm)
        rows = F.moe_gather(x, r.token_rows, out=x.new_zeros(x.shape[0] * k, x.shape[1]))
        of = torch.searchsorted(r.expert_offsets[1:].contiguous(), torch.arange(rows.shape[0], device=DEV).int(), right=True)
        f = torch.where(of < scale.numel(), scale[of.clamp(max=scale.numel() - 1)], 0.0)[:, None]   # an expert is a factor
        y = rows * f
        ctx.save_for_backward(logits, f, y, r.gates, r.experts, r.token_rows)
        ctx.renorm = renorm
        return F.moe_combine(y, r.token_rows, r.gates)

    @staticmethod
    def backward(ctx, dout):
        import fp8_block_scaled_02_amd as F
        logits, f, y, gates, experts, rows = ctx.saved_tensors
        dy, dg = F.moe_combine_backward(dout.contiguous(), y, rows, gates, dy=torch.zeros_like(y))
        return (F.moe_gather_backward(dy * f, rows), F.moe_route_backward(dg, logits, gates, experts, ctx.renorm), None,
                None, None)


@pytest.mark.parametrize("renorm", [True, False])
def test_in_an_autograd_function(F, renorm):
    """Leaves that require a gradient get the one that the backward calls give."""
    T, E, k, N = 90, 10, 3, 40
    g = _gen(3)
    x, l, w = (torch.randn(s, generator=g, device=DEV) for s in ((T, N), (T, E), (T, N)))
    l[::9] = -INF
    scale = 1.0 + torch.arange(E, device=DEV)
    x.requires_grad_()
    l.requires_grad_()
    out = Experts.apply(x, l, scale, k, renorm)
    (out * w).sum().backward()
    with torch.no_grad():
        r = F.moe_route(l, k, renorm)
        rows = F.moe_gather(x, r.token_rows, out=torch.zeros(T * k, N, device=DEV))
        of = torch.searchsorted(r.expert_offsets[1:].contiguous(), torch.arange(T * k, device=DEV).int(), right=True)
        y = rows * torch.where(of < E, scale[of.clamp(max=E - 1)], 0.0)[:, None]
        assert torch.equal(out, F.moe_combine(y, r.token_rows, r.gates))
        dg = (w[:, None] * y[r.token_rows.clamp(min=0).long()]).double().sum(2) * (r.experts >= 0)
        ref, mag = O.route_backward(_np(dg), np.where(np.isinf(_np(l)), -np.inf, _np(l)), _np(r.gates), _np(r.experts).astype(np.int64), renorm)
    # the weights' gradients are sums of N terms, the logits' of those: (N / 256 + 18) + (2 E + k + 16) and d <= 10 roundings
    reach = np.abs(_np(w)[:, None] * _np(y)[np.maximum(_ints(r.token_rows), 0)]).sum((1, 2))[:, None]
    assert (np.abs(_np(l.grad) - ref) <= U * (N + 18 + 10 + 2 * E + k + 16) * 2 * reach).all()
    # a token's gradient: its weighted factors
    want = (r.gates.double() * torch.where(r.experts >= 0, scale.double()[r.experts.clamp(min=0).long()], 0.0)).sum(1, keepdim=True) * w.double()
    assert ((x.grad.double() - want).abs() <= (k + 3) * U * want.abs()).all()


# ---- the plan in the block-scaled layer ---------------------------------------


@pytest.mark.parametrize("out", [bf16, f32])
@pytest.mark.parametrize("T,k,R,N", [(1, 1, 3, 8), (37, 8, 100, 136), (20, 17, 400, 520), (300, 4, 1300, 1024)])
def test_block_scaled_combine_of_empty_slots(F, T, k, R, N, out):
    g = _gen(N)
    tr = torch.randperm(max(R, T * k), generator=g, device=DEV)[:T * k].view(T, k).int()
    tr[torch.rand(T, k, generator=g, device=DEV) < 0.3] = -1
    tr[::3] = -1
    tr[2::9, 0] = 2 ** 31 - 1
    y = torch.randn(R, N, generator=g, device=DEV).to(bf16)
    y[0] = NAN                                                                       # which no slot names
    tr[tr == 0] = -1
    gates = torch.randn(T, k, generator=g, device=DEV)
    gates[tr < 0] = NAN
    got = F.fp8_moe_combine(y, tr, gates, out)
    assert torch.equal(got, F.moe_combine(y, tr, gates, out)) and not got[::3].any()


@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("T,every", [(3, 2), (150, 3), (700, 5), (40, 1)])
def test_plan_drives_the_block_scaled_layer(F, T, every, packed):
    """The router's plan as it is, with every n-th token padding (with 1: all of
    them, and no row is written), in the grouped product and the whole layer."""
    E, k, N, K = 20, 4, 256, 512
    g = _gen(T)
    x = torch.randn(T, K, generator=g, device=DEV).to(bf16)
    l = torch.randn(T, E, generator=g, device=DEV)
    l[::every] = -INF
    r = F.moe_route(l, k)
    live = int(r.expert_offsets[-1])
    assert live == k * (T - len(range(0, T, every)))
    wq, ws = F.fp8_weight_quant((torch.randn(E * N, K, generator=g, device=DEV) * 0.02).to(bf16))
    wq, ws = wq.view(E, N, K), ws.view(E, N // 128, K // 128)
    w = F.fp8_weight_pack(wq) if packed else wq
    gemm = F.fp8_grouped_gemm_packed if packed else F.fp8_grouped_gemm
    a, sa = F.fp8_act_quant(x)
    y = gemm(a, sa, r.row_index, r.expert_offsets, w, ws, bf16, torch.full((T * k, N), NAN, dtype=bf16, device=DEV))
    assert torch.isfinite(y[:live]).all() and y[live:].isnan().all()
    part = r.row_index[:live].contiguous()                                           # the live rows alone
    if live:
        assert torch.equal(y[:live], gemm(a, sa, part, r.expert_offsets, w, ws, bf16))
    want = F.moe_combine(y, r.token_rows, r.gates)
    assert torch.isfinite(want).all() and not want[::every].any()
    assert torch.equal(F.fp8_moe_combine(y, r.token_rows, r.gates), want)
    del y
    # memory that the layer's rows may come to lie in holds NaN
    torch.full((T * k, N), NAN, dtype=bf16, device=DEV)
    out, y = F.moe_forward(x, r.row_index, r.expert_offsets, r.token_rows, r.gates, w, ws, packed=packed)
    assert torch.equal(out, want)


# ---- scales whose product leaves fp32's range -----------------------------------


def _codes(shape, g):
    return torch.randint(-128, 128, shape, generator=g, device=DEV, dtype=torch.int32).to(i8)


def _near(n, s, g):
    return s * (1 + torch.rand(n, generator=g, device=DEV))


def _scaled(y, v, out):
    """Conversion, the scales' product and the one with the sum: 3 u; where the
    result is subnormal half a step of those, 2^-150, or 2^-134 of bf16's."""
    tol = 3 * U * np.abs(v) * (1 + 2.0 ** -10) + 2.0 ** -149
    if out == bf16:
        tol += H * (np.abs(v) + tol) + 2.0 ** -134
    return (np.abs(_np(y) - v) <= tol).all()


SCALES = [(2.0 ** -75, 2.0 ** -58), (2.0 ** -58, 2.0 ** -75), (2.0 ** -100, 2.0 ** -48), (2.0 ** 100, 2.0 ** -100),
          (2.0 ** -100, 2.0 ** 100), (2.0 ** -135, 2.0 ** 120), (2.0 ** 120, 2.0 ** -135), (-2.0 ** -90, 2.0 ** -50)]


@pytest.mark.parametrize("out", [f32, bf16])
@pytest.mark.parametrize("M,N,K", [(3, 70, 5000), (24, 130, 4096), (100, 300, 6000), (300, 16700, 640), (2050, 4100, 384)])
@pytest.mark.parametrize("sa,sw", SCALES)
def test_products_of_small_and_large_scales(F, M, N, K, sa, sw, out):
    """Values within the range, scales' products below it, and scales of either
    end: every kind of kernel."""
    g = _gen(M + N)
    a, w = _codes((M, K), g), _codes((N, K), g)
    a[0] = 0
    room = torch.zeros(M, -(-K // 128) * 128, dtype=i8, device=DEV)
    room[:, :K] = a
    sa, sw = _near(M, sa, g), _near(N, sw, g)
    v = O.product(a.cpu().numpy(), w.cpu().numpy()) * _np(sa)[:, None] * _np(sw)
    wp = F.int8_weight_pack(w)
    y = F.int8_gemm(room[:, :K], sa, wp, sw, None, out)
    assert _scaled(y, v, out) and not y[0].any()
    # a bias of the values' size: one rounding more, of the sum of both
    bias = torch.randn(N, generator=g, device=DEV) * float(np.abs(v).max())
    ref = v + _np(bias)
    tol = 3 * U * np.abs(v) * (1 + 2.0 ** -10) + U * np.abs(ref) + 2.0 ** -149
    if out == bf16:
        tol += H * (np.abs(ref) + tol) + 2.0 ** -134
    assert (np.abs(_np(F.int8_gemm(room[:, :K], sa, wp, sw, bias, out)) - ref) <= tol * (1 + 2.0 ** -10)).all()


@pytest.mark.parametrize("out", [f32, bf16])
@pytest.mark.parametrize("counts,N", [([5, 0, 40, 3], 130), ([1, 31, 33, 64, 65, 128, 200] + [2] * 33, 1800)])
@pytest.mark.parametrize("sa,sw", SCALES)
def test_grouped_products_of_small_and_large_scales(F, counts, N, sa, sw, out):
    E, R, K = len(counts), sum(counts), 1024
    g = _gen(N)
    a, w = _codes((R, K), g), _codes((E, N, K), g)
    sa, sw = _near(R, sa, g), _near(E * N, sw, g).view(E, N)
    offs = torch.tensor([0] + list(np.cumsum(counts)), device=DEV).int()
    y = F.int8_grouped_gemm(a, sa, None, offs, F.int8_weight_pack(w), sw, out)
    for e in range(E):
        s = slice(int(offs[e]), int(offs[e + 1]))
        v = O.product(a[s].cpu().numpy(), w[e].cpu().numpy()) * _np(sa)[s, None] * _np(sw)[e]
        assert _scaled(y[s], v, out), e


def test_scales_whose_product_overflows(F):
    """A sum of zero stays zero, others are infinite; an infinite or NaN scale gives NaN."""
    g = _gen(1)
    a, w = _codes((40, 256), g), _codes((50, 256), g)
    a[:20] = 0
    for s in (2.0 ** 70, -2.0 ** 100):
        y = F.int8_gemm(a, torch.full((40,), s, device=DEV), F.int8_weight_pack(w), torch.full((50,), 2.0 ** 80, device=DEV))
        assert not y[:20].any() and torch.isinf(y[20:][O.product(a.cpu().numpy()[20:], w.cpu().numpy()) != 0]).all()
    for s in (INF, NAN):
        y = F.int8_gemm(a, torch.full((40,), s, device=DEV), F.int8_weight_pack(w), torch.ones(50, device=DEV))
        assert y[:20].isnan().all()


@pytest.mark.parametrize("M", [5, 90, 300])
def test_scales_of_zero_and_infinity(F, M):
    """Beside the largest and smallest of the other side, with a bias and without."""
    g = _gen(M)
    N, K = 60, 640
    a, w = _codes((M, K), g), _codes((N, K), g)
    w[7] = 0
    a[1:3], w[:2] = 1, -1                                                            # and sums of K with either sign
    a[2] = 0
    a[2, 0] = 1                                                                      # and of one
    sums = torch.from_numpy(O.product(a.cpu().numpy(), w.cpu().numpy())).to(DEV)
    bias = torch.randn(N, generator=g, device=DEV)
    wp = F.int8_weight_pack(w)
    for other in (2.0 ** 127, 2.0 ** 100, 1.0, 2.0 ** -126, 2.0 ** -149):
        for b in (None, bias):
            rest = torch.zeros_like(sums) if b is None else bias.double().expand(M, N)
            zero, inf, most = (torch.full((n,), v, device=DEV) for n, v in ((M, 0.0), (M, INF), (N, other)))
            y = F.int8_gemm(a, zero, wp, most, b, f32)
            assert torch.equal(y.double(), rest)
            y = F.int8_gemm(a, torch.full((M,), other, device=DEV), wp, torch.zeros(N, device=DEV), b, f32)
            assert torch.equal(y.double(), rest)
            want = torch.where(sums == 0, NAN, torch.sign(sums) * INF)
            y = F.int8_gemm(a, inf, wp, most, b, f32).double()
            assert torch.equal(y.isnan(), want.isnan()) and torch.equal(y[~want.isnan()], want[~want.isnan()])


# ---- the weights' gradient ------------------------------------------------------


def _roundings(T, N, ydt, odt, aligned):
    """Of a sum of N products in the combine's gradient: a lane's fused
    multiply-adds (its pieces of C columns, then single ones), six sums over the
    lanes of a wave, and one a wave."""
    C = (8 if bf16 in (ydt, odt) else 4) if aligned else 1
    most = 1024 if T < 1 << 22 else 256
    threads = min(most, max(64, -(-(-(-(N // C) // 2)) // 64) * 64))
    return -(-(N // C) // threads) * C + -(-(N % C) // threads) + 6 + threads // 64


@pytest.mark.parametrize("ydt,odt", [(bf16, bf16), (bf16, f32), (f32, f32), (f32, bf16)])
@pytest.mark.parametrize("N", [8, 24, 520, 1001, 2056, 5000, 7168, 16384, 40000])
def test_gradient_of_the_weights(F, N, ydt, odt):
    T, k = 30, 3
    g = _gen(N)
    y, dout = torch.randn(T * k, N, generator=g, device=DEV).to(ydt), torch.randn(T, N, generator=g, device=DEV).to(odt)
    tr = torch.randperm(T * k, generator=g, device=DEV).view(T, k).int()
    gates = torch.rand(T, k, generator=g, device=DEV)
    terms = _np(y)[_ints(tr)] * _np(dout)[:, None]
    wide = torch.zeros(T * k, N + 3, dtype=ydt, device=DEV)
    wide[:, 1:N + 1] = y
    for v, aligned in ((y, N % 2 == 0 or (ydt, odt) == (f32, f32)), (wide[:, 1:N + 1], ydt == f32 and (odt == f32 or N % 2 == 0))):
        _, dg = F.moe_combine_backward(dout, v, tr, gates)
        n = _roundings(T, N, ydt, odt, aligned)
        assert (np.abs(_np(dg) - terms.sum(2)) <= n * U * (1 + 2.0 ** -10) * np.abs(terms).sum(2)).all()
