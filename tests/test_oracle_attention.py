"""The 64-bit attention oracle against sources other than itself: torch's
float8 casts and decoders, the C oracle's KV quantiser, torch's softmax."""
import numpy as np
import pytest
import torch

from oracle import attention as A

FP8 = {"e5m2": torch.float8_e5m2, "e4m3": torch.float8_e4m3fn}


@pytest.mark.parametrize("fmt", ["e5m2", "e4m3"])
def test_code_values(fmt):
    ref = torch.arange(256, dtype=torch.uint8).view(FP8[fmt]).double().numpy()
    np.testing.assert_array_equal(A.code_values(fmt), ref)


@pytest.mark.parametrize("fmt", ["e5m2", "e4m3"])
def test_quantise_is_the_fp32_quotient_and_the_nearest_code(fmt):
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(200, 64, generator=g) * torch.exp2(torch.randint(-30, 30, (200, 1), generator=g).float()))
    x[7] = 0
    x[8, :32] = 0
    x = x.bfloat16().float()
    codes, d = A.quantise(x.numpy(), fmt)
    amax = x.abs().amax(-1)
    dt = torch.where(amax == 0, 1.0, amax / A.FMAX[fmt])
    ct = (x / dt[:, None]).clamp(-A.FMAX[fmt], A.FMAX[fmt]).to(FP8[fmt]).view(torch.uint8)
    np.testing.assert_array_equal(d, dt.numpy())
    np.testing.assert_array_equal(codes, ct.numpy())


def test_quantise_e5m2_is_the_dense_kv_quantiser(orc):
    g = torch.Generator().manual_seed(4)
    x = (torch.randn(64, 128, generator=g) * torch.exp2(16 * torch.rand(64, 1, generator=g) - 8)).bfloat16()
    q, s = orc.kv_quant(x.view(torch.int16).numpy().view(np.uint16))
    codes, d = A.quantise(x.float().numpy(), "e5m2")
    np.testing.assert_array_equal(codes, q)
    np.testing.assert_array_equal(d, s)


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_turns_pairs(interleaved):
    """Rotation keeps each pair's length and adds the angle; positions 0 turn nothing."""
    T, H, D, rot = 5, 3, 48, 32
    rng = np.random.default_rng(0)
    x = rng.standard_normal((T, H, D))
    inv = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    ang = np.arange(9)[:, None] * inv
    tab = np.concatenate((np.cos(ang), np.sin(ang)), 1)
    pos = np.array([0, 3, 8, 1, 2])
    y, mag = A.norm_rope(x, None, 0.0, tab, pos, interleaved)
    np.testing.assert_array_equal(y[0], x[0])
    np.testing.assert_array_equal(y[..., rot:], x[..., rot:])
    ia = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    z = (x[..., ia] + 1j * x[..., ib]) * np.exp(1j * ang[pos])[:, None]
    np.testing.assert_allclose(y[..., ia] + 1j * y[..., ib], z, rtol=1e-12)
    assert (mag * (1 + 1e-12) >= np.abs(y)).all()
    n, _ = A.norm_rope(x, np.ones(D), 0.0, None, None, interleaved)
    np.testing.assert_allclose((n * n).mean(-1), 1.0, rtol=1e-12)


@pytest.mark.parametrize("window", [0, 1, 5, 100])
def test_attention_against_torch(window):
    g = torch.Generator().manual_seed(5)
    Hq, H, D, n = 6, 2, 16, 23
    q = torch.randn(Hq, D, generator=g, dtype=torch.float64)
    k, v = (torch.randn(n, H, D, generator=g, dtype=torch.float64) for _ in range(2))
    out, lse, mag, big = A.attention(q.numpy(), k.numpy(), v.numpy(), 0.25, window)
    lo = max(0, n - window) if window else 0
    s = torch.einsum("hd,nhd->hn", q, k.repeat_interleave(3, 1)[lo:]) * 0.25
    ref = torch.einsum("hn,nhd->hd", s.softmax(-1), v.repeat_interleave(3, 1)[lo:])
    np.testing.assert_allclose(out, ref.numpy(), rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(lse, s.logsumexp(-1).numpy(), rtol=1e-12)
    assert (mag + 1e-13 >= np.abs(out)).all() and (big >= s.abs().amax(-1).numpy() - 1e-12).all()


def test_attention_that_sees_nothing():
    out, lse, mag, _ = A.attention(np.ones((2, 16)), np.ones((0, 1, 16)), np.ones((0, 1, 16)), 1.0)
    assert not out.any() and not mag.any() and (lse == -np.inf).all()


def test_round_bf16():
    x = torch.randn(1000, generator=torch.Generator().manual_seed(6), dtype=torch.float32)
    np.testing.assert_array_equal(A.round_bf16(x.double().numpy()), x.bfloat16().double().numpy())
