"""The 64-bit forms of expert routing and of the integer products, pinned by
hand-worked cases, torch and differences (CPU)."""
import numpy as np
import pytest
import torch

from oracle import moe as O

INF = np.inf


def test_plan_by_hand():
    offsets, row_index, token_rows = O.plan(np.array([[2, 0], [-1, 2], [0, 5]]), 4)
    assert offsets.tolist() == [0, 2, 2, 4, 4]
    assert row_index.tolist() == [0, 2, 0, 1, -1, -1]
    assert token_rows.tolist() == [[2, 0], [-1, 3], [1, -1]]


def test_plan_is_the_workloads():
    import workloads as W
    r = W.routing_full(64, 16, 4, 1.0, W.gen(3))
    experts = np.full((64, 4), -1)
    rows = r["token_rows"].numpy()
    for t in range(64):
        experts[t] = r["experts"].numpy()[rows[t]]
    offsets, row_index, token_rows = O.plan(experts, 16)
    assert np.array_equal(offsets, r["offs"].numpy()) and np.array_equal(token_rows, rows)
    assert np.array_equal(row_index, r["row_index"].numpy())


def test_choice_by_hand():
    l = np.array([[1.0, 3.0, 3.0, 2.0], [-INF, 0.0, -0.0, -INF], [np.nan, INF, 1.0, np.nan], [-INF] * 4])
    assert O.choose(l, 3).tolist() == [[1, 2, 3], [1, 2, -1], [0, 3, 1], [-1, -1, -1]]


@pytest.mark.parametrize("renorm", [True, False])
def test_gates_and_their_gradient(renorm):
    """torch's softmax and its autograd, and differences."""
    g = torch.Generator().manual_seed(1)
    l = torch.randn(9, 12, generator=g, dtype=torch.float64)
    l[4] = -INF
    l[5, 2:] = -INF
    e = O.choose(l.numpy(), 3)
    got, _ = O.gates(l.numpy(), e, renorm)
    d = torch.randn(9, 3, generator=g, dtype=torch.float64)
    back, _ = O.route_backward(d.numpy(), l.numpy(), got, e, renorm)
    for t in range(9):
        kept = e[t] >= 0
        if not kept.any():
            assert not got[t].any() and not back[t].any()
            continue
        x = l[t].clone().requires_grad_()
        v = x[torch.tensor(e[t, kept])]
        w = torch.softmax(v, 0) if renorm else torch.softmax(x, 0)[torch.tensor(e[t, kept])]
        assert np.allclose(got[t, kept], w.detach().numpy(), rtol=1e-14, atol=0) and not got[t, ~kept].any()
        (w * d[t, torch.tensor(kept)]).sum().backward()
        assert np.allclose(back[t], x.grad.nan_to_num(0).numpy(), rtol=1e-12, atol=1e-15)
        for i in range(12):                                     # central differences, error of the order of h^2
            if l[t, i] == -INF:
                continue
            f = []
            for h in (1e-5, -1e-5):
                m = l[t].clone().numpy()[None]
                m[0, i] += h
                f.append((O.gates(m, e[t:t + 1], renorm)[0][0] * d[t].numpy()).sum())
            assert abs((f[0] - f[1]) / 2e-5 - back[t, i]) < 1e-8


def test_rows_and_their_gradients():
    rng = np.random.default_rng(2)
    T, k, N, R = 5, 3, 7, 15
    rows = rng.permutation(R)[:T * k].reshape(T, k)
    rows[1, 2], rows[3] = -1, -1
    y, gate, dout = rng.standard_normal((R, N)), rng.standard_normal((T, k)), rng.standard_normal((T, N))
    dy, dg, _ = O.combine_backward(dout, y, rows, gate, np.zeros((R, N)))

    def loss(y, gate):
        return (O.combine(y, rows, gate)[0] * dout).sum()

    for _ in range(40):                                         # linear in each: differences are exact but for rounding
        r, n, t, j = rng.integers(R), rng.integers(N), rng.integers(T), rng.integers(k)
        up, ug = y.copy(), gate.copy()
        up[r, n] += 1.0
        ug[t, j] += 1.0
        assert abs(loss(up, gate) - loss(y, gate) - dy[r, n]) < 1e-12
        assert abs(loss(y, ug) - loss(y, gate) - dg[t, j]) < 1e-12
    x = rng.standard_normal((T, N))
    held = np.full((R, N), 9.0)
    got = O.gather(x, rows, held)
    named = rows[rows >= 0]
    assert all((got[rows[t, j]] == x[t]).all() for t in range(T) for j in range(k) if rows[t, j] >= 0)
    assert (np.delete(got, named, 0) == 9.0).all()
    # the gradient of the gather is the combine with weights of one
    assert np.isclose((got * y)[named].sum(), (O.combine(y, rows, np.ones((T, k)))[0] * x).sum())


def test_quantise_by_hand():
    x = np.array([[127.0, -63.5, 62.5, 0.4], [0, -0.0, 0, 0], [1e-40, -1e-42, 0, 0], [INF, 1, 2, 3], [np.nan, INF, 0, 1],
                  [-254.0, 1.0, 3.0, 253.0]], np.float32)
    c, s = O.quantise(x)
    assert c[0].tolist() == [127, -64, 62, 0] and s[0] == 1.0       # halves go to even
    assert not c[1].any() and s[1] == 1.0
    assert not c[2].any() and s[2] == np.float32(2.0 ** -126)
    assert not c[3].any() and np.isposinf(s[3])
    assert not c[4].any() and np.isnan(s[4])
    assert c[5].tolist() == [-127, 0, 2, 126] and s[5] == 2.0


def test_quantise_against_torch():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(50, 300, generator=g)
    s = x.abs().amax(1) / torch.full((50,), 127.0)
    c, got = O.quantise(x.numpy())
    assert np.array_equal(got, s.numpy()) and np.array_equal(c, torch.round(x / s[:, None]).to(torch.int8).numpy())


def test_product_and_packing():
    rng = np.random.default_rng(4)
    a, w = (rng.integers(-128, 128, s).astype(np.int8) for s in ((5, 200), (37, 200)))
    assert np.array_equal(O.product(a, w), (a.astype(np.int64) @ w.astype(np.int64).T).astype(np.float64))
    p = O.packed(w).reshape(-1)
    assert O.packed(w).shape == (48, 256)
    for n, k in ((0, 0), (36, 199), (17, 63), (16, 64), (5, 130)):
        kc, panel = k // 64, n // 16
        assert p[(kc * 3 + panel) * 1024 + 256 * (k % 64 // 16) + 16 * (n % 16) + k % 16] == w[n, k]
    assert np.count_nonzero(p) == np.count_nonzero(w)
    import oracle                                               # where nothing is filled up: the FP8 weights' layout
    v = rng.integers(0, 256, (128, 256)).astype(np.uint8)
    assert np.array_equal(O.packed(v.view(np.int8)).view(np.uint8).reshape(-1), oracle.weight_pack(v).reshape(-1))
