"""Expert routing, rows to the experts and back, and their gradients on the
GPU against the 64-bit oracle.

Tolerances (u = 2^-24, a rounding of fp32; h = 2^-8, one of bf16):

* plans: equal.
* weights: a term exp(l - m), d = m - l, is off by d u from the difference and
  2 u from the exponential; the sum of n terms by (n + 2) u and what the d give,
  d exp(-d) <= 1/2 a term; the quotient by u.  So |err| <= g u (d + 2 n + 8),
  n the number of terms, and 2^-148 where a term leaves the normal range.
* the logits' gradient: the weights that are given are exact; the sum over k
  slots is off by (k + 1) u of the terms' sum; p, made again, by the above with
  d up to the largest; three products and sums follow: |err| <=
  mag u (d + 2 E + k + 16) + u |ref|, h |ref| more for bf16, and what 2^-148 of
  a term gives times the largest weight's gradient.
* combine: k fused multiply-adds: k u of the sum of magnitudes, and the
  rounding.  Its gradient: one product, rounded (once more to bf16); sums of N
  products over 256 lanes: chains of N / 256 + 8, then 6 + 4 additions.
"""
import numpy as np
import pytest
import torch

from oracle import moe as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
U, H = 2.0 ** -24, 2.0 ** -8
bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
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


def _ints(t):
    return t.detach().cpu().numpy()


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _strided(t, pad=3, at=1):
    """The same values as columns of a wider tensor."""
    wide = torch.full((t.shape[0], t.shape[1] + pad), 7.0, dtype=t.dtype, device=t.device)
    wide[:, at:at + t.shape[1]] = t
    return wide[:, at:at + t.shape[1]]


def _check_plan(offsets, row_index, token_rows, experts, E):
    want = O.plan(experts, E)
    for got, ref, name in zip((offsets, row_index, token_rows), want, ("expert_offsets", "row_index", "token_rows")):
        assert got.dtype == i32 and np.array_equal(_ints(got), ref), name


def _check_route(r, logits, k, renorm):
    l = _np(logits)
    T, E = l.shape
    experts = O.choose(l, k)
    assert np.array_equal(_ints(r.experts), experts)
    _check_plan(r.expert_offsets, r.row_index, r.token_rows, experts, E)
    ref, dist = O.gates(l, experts, renorm)
    n = k if renorm else E
    got = _np(r.gates)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    ok = np.isnan(ref) | (np.abs(got - ref) <= ref * U * (dist + 2 * n + 8) + 2.0 ** -148)
    assert ok.all(), np.abs(got - ref)[~ok].max()


# ---- the router --------------------------------------------------------------


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("T,E,k", [
    (1, 1, 1), (1, 256, 8), (7, 3, 3), (31, 16, 2), (33, 17, 5), (64, 60, 4), (65, 64, 64), (100, 65, 6), (129, 128, 8),
    (200, 160, 6), (96, 256, 8), (40, 257, 8), (50, 512, 10), (100, 384, 16), (70, 1024, 16), (9, 200, 8), (16, 100, 16), (3, 250, 20), (17, 100, 16), (65, 1000, 33), (33, 1024, 64), (1000, 8, 2)])
def test_route(F, T, E, k, dtype, renorm):
    l = torch.randn(T, E, generator=_gen(T + E), device=DEV).to(dtype)
    _check_route(F.moe_route(l, k, renorm), l, k, renorm)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E", [20, 100, 256, 500, 900])
@pytest.mark.parametrize("k", [6, 16, 20])
def test_route_does_not_depend_on_the_batch(F, E, k, renorm):
    """A token's weights and gradient have the same bits, alone or among others."""
    l = torch.randn(3000, E, generator=_gen(E), device=DEV)
    d = torch.randn(3000, k, generator=_gen(1), device=DEV)
    r = F.moe_route(l, k, renorm)
    dl = F.moe_route_backward(d, l, r.gates, r.experts, renorm)
    for lo, n in ((0, 1), (5, 16), (100, 17), (7, 64), (1000, 65)):
        s = slice(lo, lo + n)
        q = F.moe_route(l[s], k, renorm)
        assert torch.equal(q.gates, r.gates[s]) and torch.equal(q.experts, r.experts[s])
        assert torch.equal(F.moe_route_backward(d[s], l[s], q.gates, q.experts, renorm), dl[s])


@pytest.mark.parametrize("T,E,k", [(8200, 32, 3), (16500, 8, 2)])
def test_route_of_many_tokens(F, T, E, k):
    """Every workgroup of the sort has several rounds of tokens."""
    l = torch.randn(T, E, generator=_gen(5), device=DEV)
    l[::5] = -INF
    _check_route(F.moe_route(l, k), l, k, True)


@pytest.mark.parametrize("E", [9, 64, 256, 700])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_ties_masks_and_no_numbers(F, E, renorm):
    g = _gen(E)
    l = torch.randint(-2, 3, (70, E), generator=g, device=DEV).float()            # many equal ones
    l[1] = -INF                                                                   # padding
    l[2, 3:] = -INF                                                               # fewer than k experts
    l[3] = torch.finfo(f32).min                                                   # the lowest finite value everywhere
    l[4, 1:] = torch.finfo(f32).min
    l[5, 4] = float("nan")
    l[6, ::2] = float("nan")
    l[7, 5] = INF
    l[8] = INF
    l[9] = 0.0
    l[9, 1::2] = -0.0                                                             # equal to 0
    l[10] = torch.finfo(f32).max
    l[11] = 1e-45                                                                 # subnormal: above zero
    l[11, ::3] = 0.0
    l[12] = -1e-45
    l[12, ::3] = 0.0
    l[13] = 1e4 * torch.randn(E, generator=g, device=DEV)
    for k in (1, 6, 9):
        _check_route(F.moe_route(l, k, renorm), l, k, renorm)
    _check_route(F.moe_route(l.bfloat16(), 5, renorm), l.bfloat16(), 5, renorm)


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_route_strided_and_unaligned(F, dtype):
    for T in (50, 300):
        l = _strided(torch.randn(T, 100, generator=_gen(6), device=DEV).to(dtype))
        _check_route(F.moe_route(l, 7), l, 7, True)


def test_route_everything_masked_or_empty(F):
    l = torch.full((100, 20), -INF, device=DEV)
    r = F.moe_route(l, 4)
    assert (r.experts == -1).all() and (r.gates == 0).all() and (r.token_rows == -1).all() and (r.row_index == -1).all()
    assert not r.expert_offsets.any()
    r = F.moe_route(l[:0], 4)
    assert [t.shape for t in r] == [(0, 4), (0, 4), (21,), (0,), (0, 4)] and not r.expert_offsets.any()


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 7, 2), (33, 1024, 64), (70, 300, 3), (1500, 40, 8), (8300, 16, 5)])
def test_sort(F, T, E, k):
    """Ids outside the experts, and experts named twice by a token."""
    e = torch.randint(-3, E + 3, (T, k), generator=_gen(T), device=DEV).int()
    _check_plan(*F.moe_sort(e, E), _ints(e), E)


@pytest.mark.parametrize("T,E,k", [(150000, 300, 4), (40000, 1024, 64), (300001, 5, 1)])
def test_sort_of_many_slots(F, T, E, k):
    """More slots than a workgroup holds at a time; the definition by a stable sort."""
    e = torch.randint(-1, E, (T, k), generator=_gen(T), device=DEV).int()
    offsets, row_index, token_rows = map(_ints, F.moe_sort(e, E))
    flat = _ints(e).ravel()
    kept = np.nonzero(flat >= 0)[0]
    order = kept[np.argsort(flat[kept], kind="stable")]
    assert np.array_equal(offsets, np.concatenate(([0], np.cumsum(np.bincount(flat[kept], minlength=E)))))
    assert np.array_equal(row_index[:len(order)], order // k) and (row_index[len(order):] == -1).all()
    rows = np.full(T * k, -1)
    rows[order] = np.arange(len(order))
    assert np.array_equal(token_rows.ravel(), rows)


def test_sort_extremes(F):
    e = torch.tensor([[2 ** 31 - 1, -2 ** 31, 0]] * 40, device=DEV).int()
    _check_plan(*F.moe_sort(e, 3), _ints(e), 3)
    one = torch.full((3000, 4), 5, device=DEV).int()                              # all rows one expert's
    _check_plan(*F.moe_sort(one, 9), _ints(one), 9)
    offsets, row_index, token_rows = F.moe_sort(one[:0], 9)
    assert not offsets.any() and row_index.shape == (0,) and token_rows.shape == (0, 4)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 5, 5), (40, 16, 2), (33, 60, 4), (50, 128, 8), (65, 256, 8),
                                   (20, 300, 12), (17, 1024, 64), (9000, 100, 4), (8500, 256, 8)])
def test_route_backward(F, T, E, k, dtype, renorm):
    g = _gen(T * E)
    l = (3 * torch.randn(T, E, generator=g, device=DEV)).to(dtype)
    l[::4, E // 2:] = -INF
    l[::7] = -INF
    r = F.moe_route(l, k, renorm)
    d = torch.randn(T, k, generator=g, device=DEV)
    d[r.experts < 0] = float("nan")                                               # not looked at
    got = F.moe_route_backward(d, l, r.gates, r.experts, renorm)
    assert got.dtype == dtype and got.shape == (T, E)
    _check_route_backward(got, d, l, r.gates, r.experts, renorm)
    out = _strided(torch.zeros(T, E, dtype=dtype, device=DEV))
    assert F.moe_route_backward(d, _strided(l), r.gates, r.experts, renorm, out=out) is out
    assert torch.equal(out, got)


def _check_route_backward(got, d, l, gates, experts, renorm):
    ln = _np(l)
    ref, mag = O.route_backward(_np(d), ln, _np(gates), _ints(experts), renorm)
    fin = np.where(ln == -np.inf, np.nan, ln)
    with np.errstate(all="ignore"):
        dist = np.nan_to_num(np.nanmax(fin, 1) - np.nanmin(fin, 1))[:, None]
    E, k = ln.shape[1], experts.shape[1]
    tol = mag * U * (dist + 2 * E + k + 16) + U * np.abs(ref) + 2.0 ** -140
    if got.dtype == bf16:
        tol += H * np.abs(ref)
    assert (np.abs(_np(got) - ref) <= tol).all()


def test_route_backward_of_given_experts(F):
    """An expert named twice gets both terms; ids outside have none."""
    l = torch.randn(30, 12, generator=_gen(8), device=DEV)
    e = torch.randint(-1, 13, (30, 5), generator=_gen(9), device=DEV).int()
    g, d = (torch.rand(30, 5, generator=_gen(s), device=DEV) for s in (10, 11))
    for renorm in (True, False):
        _check_route_backward(F.moe_route_backward(d, l, g, e, renorm), d, l, g, e, renorm)
    assert F.moe_route_backward(d[:0], l[:0], g[:0], e[:0]).shape == (0, 12)


# ---- rows --------------------------------------------------------------------


def _slots(T, k, R, g, empty=True):
    """Rows of [T, k] slots, none named twice, some empty."""
    rows = torch.randperm(max(R, T * k), generator=g, device=DEV)[:T * k].view(T, k).int()
    rows[rows >= R] = -1
    if empty:
        rows[torch.rand(T, k, generator=g, device=DEV) < 0.2] = -1
        rows[::6] = -1
    return rows.contiguous()


SHAPES = [(1, 1, 1, 1), (1, 8, 8, 7168), (3, 2, 9, 8), (5, 3, 15, 1001), (17, 8, 136, 256), (9, 9, 81, 2056),
          (2, 17, 40, 520), (130, 1, 130, 36), (4, 64, 256, 24), (33, 4, 100, 5000)]


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("T,k,R,N", SHAPES)
def test_gather(F, T, k, R, N, dtype):
    g = _gen(T + N)
    x = torch.randn(T, N, generator=g, device=DEV).to(dtype)
    tr = _slots(T, k, R, g)
    held = torch.full((R, N), 3.0, dtype=dtype, device=DEV)
    want = O.gather(_np(x), _ints(tr), _np(held))
    assert F.moe_gather(x, tr, out=held) is held and np.array_equal(_np(held), want)
    for pad, at in ((8, 0), (3, 1)):                                               # aligned and not
        out = _strided(torch.full((R, N), 3.0, dtype=dtype, device=DEV), pad, at)
        F.moe_gather(_strided(x, pad, at), tr, out=out)
        assert np.array_equal(_np(out), want)
    got = F.moe_gather(x, tr, rows=R)
    named = tr[tr >= 0].long()
    assert got.shape == (R, N) and torch.equal(got[named], held[named])


@pytest.mark.parametrize("ydt,odt", [(bf16, bf16), (bf16, f32), (f32, f32), (f32, bf16)])
@pytest.mark.parametrize("T,k,R,N", SHAPES)
def test_combine_and_gradient(F, T, k, R, N, ydt, odt):
    g = _gen(T * N)
    y = torch.randn(R, N, generator=g, device=DEV).to(ydt)
    tr = _slots(T, k, R, g)
    gates = torch.randn(T, k, generator=g, device=DEV)
    named = tr[tr >= 0].long()
    rest = torch.ones(R, dtype=torch.bool, device=DEV)
    rest[named] = False
    y[rest] = float("nan")                                                         # rows without a slot are not read
    gates[tr < 0] = float("nan")                                                   # nor an empty slot's weight
    dout = torch.randn(T, N, generator=g, device=DEV).to(odt)
    h = H if odt == bf16 else U
    for pad, at in ((0, 0), (8, 0), (3, 1)):
        v = _strided(y, pad, at) if pad else y
        d = _strided(dout, pad, at) if pad else dout
        ref, mag = O.combine(_np(y), _ints(tr), _np(gates))
        out = F.moe_combine(v, tr, gates, odt)
        assert out.dtype == odt
        assert (np.abs(_np(out) - ref) <= k * U * mag + h * np.abs(ref)).all()
        given = _strided(torch.zeros(T, N, dtype=odt, device=DEV), 8, 0)
        assert F.moe_combine(v, tr, gates, odt, out=given) is given and torch.equal(given, out)
        # the sum without weights
        ref, mag = O.combine(_np(y), _ints(tr), np.ones((T, k)))
        got = _np(F.moe_gather_backward(v, tr))
        assert (np.abs(got - ref) <= k * U * mag + (H if ydt == bf16 else U) * np.abs(ref)).all()
        # the gradient
        held = torch.full((R, N), 3.0, dtype=ydt, device=DEV)
        rdy, rdg, mag = O.combine_backward(_np(dout), _np(y), _ints(tr), _np(gates), _np(held))
        dy, dg = F.moe_combine_backward(d, v, tr, gates, dy=held)
        assert dy is held
        tol = (H + U if ydt == bf16 else U) * np.abs(rdy)
        assert (np.abs(_np(dy) - rdy) <= tol).all()
        assert (np.abs(_np(dg) - rdg) <= (N / 256 + 18) * U * mag).all()


@pytest.mark.parametrize("T,k,N,dtype", [(4100, 8, 4104, bf16), (4100, 8, 2052, f32), (30000, 3, 1501, bf16), (12000, 3, 2001, f32)])
def test_more_rows_than_a_cache(F, big, T, k, N, dtype):
    g = _gen(N)
    R = T * k
    tr = torch.randperm(R, generator=g, device=DEV).view(T, k).int()
    tr[::5, k // 2] = -1
    x, dout = (torch.randn(T, N, generator=g, device=DEV).to(dtype) for _ in range(2))
    gates = torch.randn(T, k, generator=g, device=DEV)
    held = torch.full((R, N), 3.0, dtype=dtype, device=DEV)
    F.moe_gather(x, tr, out=held)
    token = torch.full((R,), -1, device=DEV)
    slot = token.clone()
    t_of = torch.arange(T, device=DEV)[:, None].expand(T, k)
    live = tr >= 0
    token[tr[live].long()] = t_of[live]
    slot[tr[live].long()] = torch.arange(k, device=DEV).expand(T, k)[live]
    rest = token < 0
    assert torch.equal(held[~rest], x[token[~rest]]) and (held[rest] == 3).all()
    y = torch.randn(R, N, generator=g, device=DEV).to(dtype)
    out, total = F.moe_combine(y, tr, gates), F.moe_gather_backward(y, tr)
    held.fill_(3.0)
    dy, dg = F.moe_combine_backward(dout, y, tr, gates, dy=held)
    assert (dy[rest] == 3).all()
    h = H if dtype == bf16 else U
    for lo in range(0, T, 1000):
        s = tr[lo:lo + 1000].long()
        w = (s >= 0).double()[..., None]
        rows, gt, d = y[s.clamp(min=0)].double() * w, gates[lo:lo + 1000].double()[..., None], dout[lo:lo + 1000].double()
        for got, terms in ((out, rows * gt), (total, rows)):
            ref, mag = terms.sum(1), terms.abs().sum(1)
            assert ((got[lo:lo + 1000].double() - ref).abs() <= k * U * mag + h * ref.abs()).all()
        terms = rows * d[:, None]
        assert ((dg[lo:lo + 1000].double() - terms.sum(2)).abs() <= (N / 256 + 18) * U * terms.abs().sum(2)).all()
        want = gt * d[:, None] * w
        tol = (H + U if dtype == bf16 else U) * want.abs()
        got = torch.where(w > 0, dy[s.clamp(min=0)].double(), 0.0)
        assert ((got - want).abs() <= tol).all()


def test_rows_outside_and_none(F):
    """Rows outside the array count as none; arrays without rows or tokens."""
    tr = torch.tensor([[0, 4, -7], [2 ** 31 - 1, 3, 5]], device=DEV).int()
    y = torch.arange(4.0, device=DEV)[:, None].repeat(1, 16) + 1
    gates = torch.ones(2, 3, device=DEV)
    assert F.moe_combine(y, tr, gates)[:, 0].tolist() == [1.0, 4.0]
    dy, dg = F.moe_combine_backward(torch.ones(2, 16, device=DEV), y, tr, gates, dy=torch.zeros_like(y))
    assert dy[:, 0].tolist() == [1.0, 0.0, 0.0, 1.0] and dg.tolist() == [[16.0, 0.0, 0.0], [0.0, 64.0, 0.0]]
    held = F.moe_gather(torch.ones(2, 16, device=DEV), tr, out=torch.zeros(4, 16, device=DEV))
    assert held[:, 0].tolist() == [1.0, 0.0, 0.0, 1.0]
    assert not F.moe_combine(y[:0], tr, gates).any()
    assert F.moe_combine(y, tr[:0], gates[:0]).shape == (0, 16)
    dy, dg = F.moe_combine_backward(torch.ones(2, 16, device=DEV), y[:0], tr, gates)
    assert dy.shape == (0, 16) and not dg.any()
    assert F.moe_gather(y[:0], tr[:0]).shape == (0, 16)


def test_gradient_against_differences(F):
    """A loss of the whole round trip, in 64 bits, moved along the gradients
    that the kernels give: differences of a function that is linear in y and
    in the weights, and smooth in the logits."""
    T, E, k, N = 40, 12, 3, 64
    g = _gen(12)
    l = torch.randn(T, E, generator=g, device=DEV)
    r = F.moe_route(l, k, False)
    y = torch.randn(T * k, N, generator=g, device=DEV)
    dout = torch.randn(T, N, generator=g, device=DEV)
    dy, dg = F.moe_combine_backward(dout, y, r.token_rows, r.gates)
    dl = F.moe_route_backward(dg, l, r.gates, r.experts, False)
    experts, rows = _ints(r.experts), _ints(r.token_rows)

    def loss(logits, y):
        w, _ = O.gates(logits, experts, False)
        return (O.combine(y, rows, w)[0] * _np(dout)).sum()

    rng = np.random.default_rng(13)
    for a, b, grad in ((1.0, 0.0, dl), (0.0, 1.0, dy)):
        v = rng.standard_normal(grad.shape)
        step = 1e-4
        lo, hi = (loss(_np(l) + a * s * (v if a else 0), _np(y) + b * s * (v if b else 0)) for s in (-step, step))
        want, slope = (hi - lo) / (2 * step), (_np(grad) * v).sum()
        # fp32 roundings of the gradient, at most 2^-18 of its terms (N + E + k of them), and the square of the step
        assert abs(want - slope) <= 2.0 ** -18 * (np.abs(_np(grad)) * np.abs(v)).sum() + 1e-6 * np.abs(_np(dout)).sum()


def test_routing_of_many_tokens_past_32_bits(F, big):
    """Logits past 2^31 values: the choice and the weights of a part are those of the part alone."""
    T, E, k = 9_000_000, 256, 8
    l = torch.empty(T, E, device=DEV)
    l.copy_(torch.rand(1, E, generator=_gen(1), device=DEV))
    for lo in range(0, T, 1_000_000):
        l[lo:lo + 1_000_000] += torch.rand(1_000_000, E, generator=_gen(lo), device=DEV)
    r = F.moe_route(l, k)
    assert int(r.expert_offsets[-1]) == T * k
    named = torch.zeros(T * k, dtype=torch.bool, device=DEV)
    named[r.token_rows.view(-1).long()] = True
    assert named.all()
    assert (r.row_index[r.token_rows.long()] == torch.arange(T, device=DEV)[:, None]).all()
    of_row = torch.empty(T * k, dtype=i32, device=DEV)
    of_row[r.token_rows.view(-1).long()] = r.experts.view(-1)
    assert (of_row[1:] >= of_row[:-1]).all()
    counts = torch.bincount(r.experts.view(-1), minlength=E)
    assert torch.equal(r.expert_offsets[1:].long(), counts.cumsum(0))
    d = torch.rand(T, k, generator=_gen(2), device=DEV)
    dl = F.moe_route_backward(d, l, r.gates, r.experts, False)
    for lo in (0, 4_400_000, 8_388_600, T - 1000):
        part = slice(lo, lo + 1000)
        q = F.moe_route(l[part], k)
        assert torch.equal(q.experts, r.experts[part]) and torch.equal(q.gates, r.gates[part])
        assert torch.equal(F.moe_route_backward(d[part], l[part], q.gates, q.experts, False), dl[part])


def test_more_threads_than_a_launch(F, big):
    """2^23 tokens of rows that would take 576 threads each."""
    T, N, R = (1 << 23) + 3, 1025, 1000
    x = torch.zeros(T, N, dtype=bf16, device=DEV)
    tr = torch.full((T, 1), -1, dtype=i32, device=DEV)
    at = torch.tensor([0, 77, 1 << 21, T - 4, T - 1], device=DEV)
    tr[at, 0] = torch.tensor([5, 999, 0, 3, 4], device=DEV).int()
    x[at] = torch.randn(5, N, generator=_gen(3), device=DEV).to(bf16)
    held = torch.full((R, N), 3.0, dtype=bf16, device=DEV)
    F.moe_gather(x, tr, out=held)
    rows = tr[at, 0].long()
    assert torch.equal(held[rows], x[at]) and int((held == 3).all(1).sum()) == R - 5
    gates = torch.full((T, 1), 2.0, device=DEV)
    dy, dg = F.moe_combine_backward(x, held, tr, gates, dy=torch.full_like(held, 3.0))
    assert torch.equal(dy[rows], 2 * x[at]) and int((dy == 3).all(1).sum()) == R - 5
    assert int((dg != 0).sum()) == 5 and (dg[at, 0] > 0).all()
    F.moe_combine(held, tr, gates, out=x)
    assert torch.equal(x[at], 2 * held[rows]) and not x[:77].any(1)[1:].any() and not x[T - 3:T - 1].any()


def test_many_rows_past_32_bits(F, big):
    """Rows whose values lie past 2^31 elements."""
    N, R = 8192, 300000
    tr = torch.tensor([[R - 1, 7], [0, R - 2]], device=DEV).int()
    y = torch.empty(R, N, dtype=bf16, device=DEV)
    named = [R - 1, 7, 0, R - 2]
    for i, r in enumerate(named):
        y[r] = i + 1
    out = F.moe_combine(y, tr, torch.ones(2, 2, device=DEV))
    assert (out[0] == 3).all() and (out[1] == 7).all()
    F.moe_gather(torch.tensor([[5.0], [6.0]], device=DEV).to(bf16).repeat(1, N), tr, out=y)
    assert [y[r, 77].item() for r in named] == [5.0, 5.0, 6.0, 6.0]
    F.moe_combine_backward(torch.ones(2, N, dtype=bf16, device=DEV), y.clone(), tr, torch.ones(2, 2, device=DEV) * 2, dy=y)
    assert all((y[r] == 2).all() for r in named)
