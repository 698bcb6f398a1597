"""The three ways of dealing out fp8_paged_attention's work, each asserted from the workspace it asks for, so that
other rules on sizes cannot leave one untested: the line of all tiles (many regions, wide tables), and whole
regions of eight waves with the most shared memory.  Against the 64-bit oracle, tolerances as in
test_gpu_attention."""
import numpy as np
import pytest
import torch

import workloads as W
from test_gpu_attention import DEV, F, _book, _check_attention, _filled, _Step  # noqa: F401
from test_gpu_attention_weights import dealt

pytestmark = pytest.mark.gpu

ROOM = 6700          # tokens a table has room for: 210 tiles


def _ragged(B, g, longest=(6500, 3333, 2100)):
    """Mostly short sequences, empty ones among them, a few long ones in different places."""
    lens = [int(x) for x in torch.randint(0, 120, (B,), generator=g, device=DEV)]
    for i, n in enumerate(longest):
        lens[(i * B) // 3 + 1] = n
    lens[0], lens[B // 2], lens[-1] = 0, 0, 33
    return lens


def _checked(lens):
    """Sequences to compare: the long ones, the ends, neighbours of both, some of the rest."""
    long = [b for b, n in enumerate(lens) if n > 1000]
    near = {min(max(b + d, 0), len(lens) - 1) for b in long + [0, len(lens) - 1, len(lens) // 2] for d in (-1, 0, 1)}
    return sorted(near | set(range(0, len(lens), 9)))


# 136 regions and more: too many for parts, tables too wide for one workgroup a region
@pytest.mark.parametrize("fmt", ["e5m2", "e4m3"])
@pytest.mark.parametrize("G", [4, 18, 40])
@pytest.mark.parametrize("D", [48, 64, 80, 128, 192, 256])
def test_the_line(F, D, G, fmt):
    g = W.gen(D + G, DEV)
    B, H, S = 69, 2, 32
    lens = _ragged(B, g)
    pages, table = _book(lens, S, g, room=ROOM)
    c = _filled(F, pages, H, S, D, fmt, g)
    q = (2 * torch.randn(B, H * G, D, generator=g, device=DEV)).bfloat16()
    assert dealt(F, c, B, H * G, table.shape[1]) == "line"
    _check_attention(F, c, lens, q, table, out_dtype=torch.float32, check=_checked(lens))
    most = 6400                                                    # a length beyond it
    assert dealt(F, c, B, H * G, table.shape[1], most) == "line"
    _check_attention(F, c, lens, q, table, max_context=most, check=_checked(lens))


@pytest.mark.parametrize("window", [3, 3000, 4500])
@pytest.mark.parametrize("G,D,fmt", [(4, 64, "e4m3"), (3, 128, "e5m2"), (20, 128, "e4m3"), (4, 256, "e5m2"),
                                     (18, 192, "e4m3"), (7, 96, "e5m2")])
def test_windows_on_the_line(F, G, D, fmt, window):
    """Windows as wide as the line needs, and a narrow one over the same book, which whole regions serve."""
    g = W.gen(window + D, DEV)
    B, H, S = 69, 2, 16
    lens = _ragged(B, g, (6500, 3001, 4511))
    pages, table = _book(lens, S, g, room=ROOM)
    c = _filled(F, pages, H, S, D, fmt, g)
    q = torch.randn(B, H * G, D, generator=g, device=DEV).bfloat16()
    qtiles = -(-G // (32 if G > 16 and D <= 128 else 16))
    way = "whole" if window == 3 else "line"
    # (with two query tiles to a KV head, 276 regions, whole ones serve up to 128 tiles)
    if window == 3000 and qtiles == 2:
        way = "whole"
    assert dealt(F, c, B, H * G, table.shape[1], window=window) == way
    _check_attention(F, c, lens, q, table, window, torch.float32, check=_checked(lens))
    _check_attention(F, c, lens, q, table, window, check=_checked(lens))


@pytest.mark.parametrize("B,H", [(300, 1), (66, 5), (1100, 1)])
def test_the_line_of_many_regions(F, B, H):
    """Batches of more than a wave's 64 sequences with pieces that hold many regions, and regions of many pieces."""
    g = W.gen(B, DEV)
    lens = _ragged(B, g, (6001, 5000, 6666))
    pages, table = _book(lens, 16, g, room=ROOM)
    c = _filled(F, pages, H, 16, 64, "e5m2", g)
    q = torch.randn(B, 2 * H, 64, generator=g, device=DEV).bfloat16()
    assert dealt(F, c, B, 2 * H, table.shape[1]) == "line"
    check = [b for b in _checked(lens) if b % 5 == 0 or lens[b] > 1000]
    _check_attention(F, c, lens, q, table, out_dtype=torch.float32, check=check)


@pytest.mark.parametrize("fmt", ["e5m2", "e4m3"])
@pytest.mark.parametrize("window", [0, 4000])
@pytest.mark.parametrize("D,G", [(128, 4), (256, 3), (80, 20)])
def test_what_is_not_seen_on_the_line(F, D, G, window, fmt):
    """NaN and infinite codes and scales in every place that no sequence sees: the same bits."""
    g = W.gen(D, DEV)
    B, H, S = 69, 2, 32
    lens = _ragged(B, g, (6500, 3333, 5001))
    pages, table = _book(lens, S, g, room=ROOM)
    c = _filled(F, pages, H, S, D, fmt, g)
    q = torch.randn(B, H * G, D, generator=g, device=DEV).bfloat16()
    lt = torch.tensor(lens, dtype=torch.int32, device=DEV)
    assert dealt(F, c, B, H * G, table.shape[1], window=window) == "line"
    want = F.fp8_paged_attention(q, c, table, lt, window=window)
    seen = torch.zeros(pages, S, dtype=torch.bool, device=DEV)
    for b, n in enumerate(lens):
        t = torch.arange(max(0, n - window) if window else 0, n, device=DEV)
        seen[table[b, t // S].long(), t % S] = True
    bad = ~seen[:, None].expand(pages, H, S)
    for code, scale in ((0x7F, float("nan")), (0x7C if fmt == "e5m2" else 0xFF, float("inf"))):
        dirty = F.KVCache.from_tensors(*(x.clone() for x in (c.k_codes, c.v_codes, c.k_scales, c.v_scales)), fmt)
        for codes, scales in ((dirty.k_codes, dirty.k_scales), (dirty.v_codes, dirty.v_scales)):
            codes[bad] = code
            scales[bad] = scale
        assert torch.equal(F.fp8_paged_attention(q, dirty, table, lt, window=window), want)


@pytest.mark.parametrize("D,G", [(64, 4), (128, 40), (256, 4)])
def test_nan_among_the_seen_on_the_line(F, D, G):
    """A NaN query head, and NaN scales of seen tokens in a region of many pieces: NaN there and nowhere else."""
    g = W.gen(D + 1, DEV)
    B, H, S = 69, 2, 32
    lens = _ragged(B, g)
    long = lens.index(6500)
    pages, table = _book(lens, S, g, room=ROOM)
    c = _filled(F, pages, H, S, D, "e5m2", g)
    q = torch.randn(B, H * G, D, generator=g, device=DEV).bfloat16()
    lt = torch.tensor(lens, dtype=torch.int32, device=DEV)
    assert dealt(F, c, B, H * G, table.shape[1]) == "line"

    def run():
        lse = torch.empty(B, H * G, device=DEV)
        return F.fp8_paged_attention(q, c, table, lt, lse=lse), lse

    want, want_l = run()
    two = [b for b in range(B) if 40 <= lens[b] < 1000][-1]
    bad = torch.zeros(B, H * G, dtype=torch.bool, device=DEV)
    q[two, 1, 3] = float("nan")
    bad[two, 1] = True
    c.k_scales[table[long, 100].long(), 1, 7] = float("nan")
    bad[long, G:] = True
    out, lse = run()
    assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
    assert torch.equal(out[~bad], want[~bad]) and torch.equal(lse[~bad], want_l[~bad])


def test_the_line_in_a_graph(F):
    """Captured once, replayed on other lengths (long ones moving through the batch, empty ones), eager work between;
    every replay against the eager call and the last against the oracle."""
    g = W.gen(31, DEV)
    B, H, G, D, S = 70, 2, 4, 128, 32
    most = [300] * B
    for b in (3, 35, 69):
        most[b] = 6500
    pages, table = _book(most, S, g, room=ROOM)
    c = _filled(F, pages, H, S, D, "e5m2", g)
    q = torch.randn(B, H * G, D, generator=g, device=DEV).bfloat16()
    lt = torch.tensor(most, dtype=torch.int32, device=DEV)
    assert dealt(F, c, B, H * G, table.shape[1]) == "line"
    F.fp8_paged_attention(q, c, table, lt)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = F.fp8_paged_attention(q, c, table, lt)
    for turn in range(5):
        lens = [int(x) for x in torch.randint(0, 300, (B,), generator=g, device=DEV)]
        for i, b in enumerate((3, 35, 69)):
            lens[b] = (6500, 1, 4097, 0, 250)[(turn + i) % 5]
        lt.copy_(torch.tensor(lens, dtype=torch.int32))
        q.copy_(torch.randn(q.shape, generator=g, device=DEV).bfloat16())
        gr.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(F.fp8_paged_attention(q, c, table, lt), got), turn
        torch.cuda.synchronize()
    full, _ = _check_attention(F, c, lens, q, table, check=[0, 2, 3, 4, 34, 35, 36, 68, 69])
    assert torch.equal(full, got)


def test_steps_on_the_line(F):
    """A decode step with padded rows (no slot, no length) on the line: zeros for them, the rest as the two calls."""
    g = W.gen(32, DEV)
    s = _Step(F, g, B=70, most=6600)
    s.lt[::7] = 0
    s.slots[::7] = -1
    assert dealt(F, s.c, 70, 8, s.table.shape[1]) == "line"
    before = s.c.k_codes.clone()
    got = s.run(out_dtype=torch.float32)
    assert not got[::7].any() and torch.isfinite(got).all()
    changed = (s.c.k_codes != before).flatten(2).any(-1).any(1).nonzero()[:, 0]
    assert set(changed.tolist()) <= set((s.slots[s.slots >= 0] // s.S).tolist())
    q2, _ = F.fp8_qk_norm_rope(s.q, s.k, s.tab, s.pos, s.w, s.w)
    lens = s.lt.tolist()
    out, _ = _check_attention(F, s.c, lens, q2, s.table, out_dtype=torch.float32, check=range(0, 70, 11))
    assert torch.equal(out, got)


@pytest.mark.parametrize("fmt", ["e5m2", "e4m3"])
@pytest.mark.parametrize("D,G,H", [(112, 32, 1), (112, 70, 2), (80, 32, 1), (96, 17, 2), (64, 32, 1), (48, 31, 3),
                                   (192, 16, 2), (208, 40, 1), (144, 9, 1), (240, 16, 1)])
def test_whole_regions_of_eight_waves(F, D, G, H, fmt):
    """Up to 32 rows of 112 positions, or 16 of 240, for each of eight waves: 134 and 137 KB of shared memory."""
    g = W.gen(D + G, DEV)
    lens = [256, 0, 255, 1, 100, 33]
    pages, table = _book(lens, 16, g)
    c = _filled(F, pages, H, 16, D, fmt, g)
    q = torch.randn(len(lens), H * G, D, generator=g, device=DEV).bfloat16()
    assert dealt(F, c, len(lens), H * G, table.shape[1], 256) == "whole"
    _check_attention(F, c, lens, q, table, max_context=256, out_dtype=torch.float32)
    _check_attention(F, c, lens, q, table, max_context=256, window=77)
