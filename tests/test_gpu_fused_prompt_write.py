"""Calls large enough that a row slot walks through several rows (queries, keys and values of its token with the
next row loaded ahead, or four tokens of a head) and that stores are non-temporal, against the same tokens in calls
of a few hundred, which take a slot a row: the same bits."""
import pytest
import torch

import workloads as W
from test_gpu_attention import DEV, F, _check_rope, _expect_written, _assert_cache, _fresh, _rows, _table  # noqa: F401

pytestmark = pytest.mark.gpu


def _same_cache(a, b):
    for x, y in zip((a.k_codes, a.v_codes, a.k_scales, a.v_scales), (b.k_codes, b.v_codes, b.k_scales, b.v_scales)):
        assert torch.equal(x, y)


# 32, 16 and 8 rows at a time for up to 64, 128 and 256 positions; more rows a token than that, so from 1024 tokens
# on a slot takes several
@pytest.mark.parametrize("fmt", ["e5m2", "e4m3"])
@pytest.mark.parametrize("T,Hq,H,D,rot,inter", [(1100, 40, 4, 64, 64, False), (1531, 33, 3, 48, 16, True),
                                                (1024, 64, 8, 128, 128, False), (2500, 12, 3, 128, 48, False),
                                                (1023, 20, 5, 80, 32, True), (2047, 20, 5, 80, 80, False),
                                                (1300, 7, 2, 256, 256, False), (1301, 24, 1, 192, 64, True)])
def test_fused_write_of_a_prompt(F, T, Hq, H, D, rot, inter, fmt):
    g = W.gen(T, DEV)
    y = torch.randn(T, (Hq + 2 * H) * D, generator=g, device=DEV).bfloat16()       # the projection's output
    q, k, v = (y[:, a * D:b * D].view(T, b - a, D) for a, b in ((0, Hq), (Hq, Hq + H), (Hq + H, Hq + 2 * H)))
    tab, pos = _table(rot, 4000), torch.randint(0, 4000, (T,), generator=g, device=DEV)
    qw, kw = (torch.rand(D, generator=g, device=DEV).bfloat16() for _ in range(2))
    pages = -(-T // 32) + 2
    slots = torch.randperm(pages * 32, generator=g, device=DEV)[:T]
    slots[::9] = -1
    slots[5] = pages * 32
    one, two = _fresh(F, pages, H, 32, D, fmt), _fresh(F, pages, H, 32, D, fmt)
    for w in ((qw, kw), (None, kw), (None, None)):
        qo = F.fp8_qkv_cache_write(q, k, v, tab, pos, slots, one, *w, 1e-6, inter)
        k2 = []
        for lo in range(0, T, 300):
            at = slice(lo, lo + 300)
            qc, kc = F.fp8_qk_norm_rope(q[at], k[at], tab, pos[at], *w, 1e-6, inter)
            assert torch.equal(qo[at], qc)
            F.fp8_kv_cache_write(kc, v[at], slots[at], two)
            k2.append(kc)
        _same_cache(one, two)
    # and against the oracle
    _check_rope(qo, q, None, 1e-6, tab, pos, inter)
    _assert_cache(one, _expect_written(one, torch.cat(k2), v, slots))


def test_fused_write_of_a_prompt_over_its_queries(F):
    g = W.gen(2, DEV)
    T, Hq, H, D = 1200, 20, 4, 128
    y = torch.randn(T, (Hq + 2 * H) * D, generator=g, device=DEV).bfloat16()
    q, k, v = (y[:, a * D:b * D].view(T, b - a, D) for a, b in ((0, Hq), (Hq, Hq + H), (Hq + H, Hq + 2 * H)))
    tab, pos = _table(D, 99), torch.randint(0, 99, (T,), generator=g, device=DEV)
    slots = torch.randperm(40 * 32, generator=g, device=DEV)[:T]
    w = torch.rand(D, generator=g, device=DEV).bfloat16()
    one, two = _fresh(F, 40, H, 32, D, "e4m3"), _fresh(F, 40, H, 32, D, "e4m3")
    want = F.fp8_qkv_cache_write(q, k, v, tab, pos, slots, one, w, w)
    rest = y[:, Hq * D:].clone()
    F.fp8_qkv_cache_write(q, k, v, tab, pos, slots, two, w, w, q_out=q)
    assert torch.equal(q, want) and torch.equal(y[:, Hq * D:], rest)
    _same_cache(one, two)


@pytest.mark.parametrize("T,Hq,Hk,D,rot,inter", [(1200, 30, 5, 64, 64, True), (1100, 33, 2, 64, 32, False),
                                                 (1500, 9, 3, 256, 256, False), (1500, 9, 3, 256, 128, True),
                                                 (1030, 20, 4, 128, 128, True), (1100, 10, 3, 160, 160, False)])
def test_large_norm_rope_of_other_widths(F, T, Hq, Hk, D, rot, inter):
    g = W.gen(D + T, DEV)
    q, k = _rows(T, Hq, D, g), _rows(T, Hk, D, g, True)
    tab, pos = _table(rot, 99), torch.randint(0, 99, (T,), generator=g, device=DEV)
    w = torch.rand(D, generator=g, device=DEV).bfloat16()
    qo, ko = F.fp8_qk_norm_rope(q, k, tab, pos, w, w, 1e-6, inter)
    for lo in range(0, T, 500):
        at = slice(lo, lo + 500)
        a, b = F.fp8_qk_norm_rope(q[at], k[at], tab, pos[at], w, w, 1e-6, inter)
        assert torch.equal(qo[at], a) and torch.equal(ko[at], b)
    _check_rope(ko, k, w, 1e-6, tab, pos, inter)


@pytest.mark.parametrize("T,H,D,fmt", [(33011, 8, 64, "e5m2"), (5003, 3, 64, "e4m3"), (45001, 8, 48, "e4m3"),
                                       (70001, 1, 16, "e5m2")])
def test_large_write_of_few_positions(F, T, H, D, fmt):
    """Eight lanes a row, four tokens a slot; the first and third are read past the caches too."""
    g = W.gen(T, DEV)
    k, v = _rows(T, H, D, g), _rows(T, H, D, g, True)
    pages = -(-T // 64) + 1
    slots = torch.randperm(pages * 64, generator=g, device=DEV)[:T]
    slots[::7] = -1
    one, two = _fresh(F, pages, H, 64, D, fmt), _fresh(F, pages, H, 64, D, fmt)
    F.fp8_kv_cache_write(k, v, slots, one)
    for lo in range(0, T, 500):
        F.fp8_kv_cache_write(k[lo:lo + 500], v[lo:lo + 500], slots[lo:lo + 500], two)
    _same_cache(one, two)
