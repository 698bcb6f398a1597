"""Outputs that share memory with each other or with what a call reads are refused on the host (no GPU needed:
a call that passes these checks is refused next for lying in host memory); slices of one allocation that lie
apart, however interlaced, are not."""
import ctypes

import pytest
import torch

import fp8_block_scaled_02_amd as F

bf16, f32, i32, i64, u8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8


class _At(F.KVCache):
    """The description of a cache over host tensors, none of which a call gets to touch."""

    def __init__(self, k, v, ks, vs):
        P, H, S, D = k.shape
        self._tensors = k, v, ks, vs
        self._struct = F.attention._CacheStruct(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), k.stride(0),
                                                ks.stride(0), P, S, H, D, F.FMT_E5M2, 0)
        self._ref, self._dev = ctypes.addressof(self._struct), -1


def _cache(P=4, H=2, S=16, D=64):
    return _At(*(torch.zeros(P, H, S, D, dtype=u8) for _ in "kv"), *(torch.zeros(P, H, S) for _ in "kv"))


def _apart(fn, *a, **k):
    with pytest.raises(ValueError, match="on a GPU"):
        fn(*a, **k)


def _not_apart(names, fn, *a, **k):
    with pytest.raises(ValueError, match=f"^{names} must lie apart$"):
        fn(*a, **k)


def test_read_outputs():
    c = _cache()
    table, offs = torch.zeros(2, 4, dtype=i32), torch.zeros(3, dtype=i32)
    buf = torch.zeros(20, 2, 64, dtype=bf16)
    f = F.fp8_kv_cache_read
    _apart(f, c, table, offs, 10, buf[:10], buf[10:])
    _apart(f, c, table, offs, 10, buf[10:], buf[:10])
    _not_apart("k_out and v_out", f, c, table, offs, 10, buf[:10], buf[:10])
    _not_apart("k_out and v_out", f, c, table, offs, 10, buf[:10], buf[1:11])
    _not_apart("k_out and v_out", f, c, table, offs, 10, buf[9:19], buf[:10])
    _apart(f, c, table, offs, 0, buf[:0], buf[:0])
    line = torch.zeros(4096, dtype=i32)
    out = line[64:64 + 640].view(bf16).view(10, 2, 64)
    _not_apart("v_out and block_table", f, c, line[:64 * 40].view(2, -1)[:, 60:64 + 4], offs, 10, None, out)
    _not_apart("k_out and offsets", f, c, table, line[62:65], 10, out, None)
    _apart(f, c, line[:64].view(2, -1), line[704:707], 10, out, None)


def test_read_outputs_in_the_cache():
    c = _cache()
    table, offs = torch.zeros(2, 4, dtype=i32), torch.zeros(3, dtype=i32)
    f = F.fp8_kv_cache_read
    for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales):
        out = t.flatten().view(u8)[:256].view(bf16).view(1, 2, 64)
        _not_apart("v_out and the cache", f, c, table, offs, 1, None, out)
    # the free part of a page's stride
    codes = torch.zeros(4, 2 * 2048 + 256, dtype=u8)
    c = _At(codes[:, :2048].view(4, 2, 16, 64), codes[:, 2048:4096].view(4, 2, 16, 64), c.k_scales, c.v_scales)
    _apart(f, c, table, offs, 1, codes[1, 4096:].view(bf16).view(1, 2, 64))
    _not_apart("k_out and the cache", f, c, table, offs, 1, codes[1, 4080:4336].view(bf16).view(1, 2, 64))


def _projection(T=5, Hq=4, H=2, D=64):
    """q, k, v as slices of one projection's output, and that with room on both sides."""
    n = (Hq + 2 * H) * D
    wide = torch.zeros(T + 2, n, dtype=bf16)
    y = wide[1:T + 1]
    return [y[:, a * D:b * D].view(T, b - a, D) for a, b in ((0, Hq), (Hq, Hq + H), (Hq + H, Hq + 2 * H))], wide


def test_rope_outputs():
    (q, k, v), wide = _projection()
    f = F.fp8_qk_norm_rope
    other = torch.zeros(5, 6, 64, dtype=bf16)
    _apart(f, q, k, q_out=q, k_out=k)                           # in place
    _apart(f, q, k, k_out=v)                                    # over the values: the caller's choice
    _apart(f, q, k, q_out=other[:, :4], k_out=other[:, 4:])
    _not_apart("k_out and q", f, q, k, k_out=q[:, :2])
    _not_apart("q_out and q", f, q, k, q_out=wide.flatten().as_strided(q.shape, q.stride(), q.storage_offset() + 8))
    _not_apart("q_out and q", f, q, k, q_out=wide[:5, :256].view(5, 4, 64))        # a token earlier
    _not_apart("q_out and k", f, torch.zeros_like(q), k, q_out=wide[1:6, 128:384].view(5, 4, 64))
    _not_apart("q_out and k_out", f, q, k, q_out=other[:, :4], k_out=other[:, 3:5])
    same = torch.zeros(5, 2, 64, dtype=bf16)
    _not_apart("q_out and k_out", f, k, v, q_out=same, k_out=same)
    _not_apart("q_out and k", f, k, v, q_out=v)
    tab, pos = torch.zeros(10, 64), torch.zeros(5, dtype=i64)
    _not_apart("k_out and cos_sin", f, q, k, tab, pos, k_out=tab.view(bf16).flatten()[:640].view(5, 2, 64))
    w = torch.zeros(6 * 128, dtype=bf16)
    _not_apart("k_out and q_weight", f, q, k, None, None, w[32:96], k_out=w[64:704].view(5, 2, 64))
    _not_apart("k_out and k_weight", f, q, k, None, None, None, w[640:704], k_out=w[64:704].view(5, 2, 64))
    _apart(f, q, k, None, None, w[:64], w[704:], k_out=w[64:704].view(5, 2, 64))


def test_rope_outputs_head_by_head():
    """q and k of each head side by side, [T, H, 3, D]; heads outside tokens, [3, H, T, D]."""
    f = F.fp8_qk_norm_rope
    y = torch.zeros(5, 4, 3, 64, dtype=bf16)
    q, k = y[:, :, 0], y[:, :, 1]
    _apart(f, q, k, q_out=q, k_out=k)
    _apart(f, q, k, q_out=y[:, :, 2])
    _not_apart("q_out and k", f, q, k, q_out=k)
    z = torch.zeros(4, 3, 5, 64, dtype=bf16)
    q, k = (z[:, i].transpose(0, 1) for i in (0, 1))
    _apart(f, q, k, q_out=q, k_out=k)
    _not_apart("k_out and q", f, q, k, k_out=q)


def test_rope_outputs_drawn():
    """Strided rows in one buffer against a count of the bytes they share: rows that do share some are always
    refused, and rows of one projection that do not are never."""
    import random
    rng, refused, taken = random.Random(3), 0, 0
    buf = torch.zeros(1 << 14, dtype=bf16)
    for _ in range(400):
        T, H, D = rng.randint(1, 4), rng.randint(1, 3), 16 * rng.randint(1, 3)
        h = D + 8 * rng.randint(0, 9)
        t = H * h + 8 * rng.randint(0, 20)
        if rng.random() < 0.3:
            h, t = T * h + 8 * rng.randint(0, 20), h
        shape = (T, H, D)
        if rng.random() < 0.5:
            h2, t2 = h, t
        else:
            h2 = D + 8 * rng.randint(0, 9)
            t2 = H * h2 + 8 * rng.randint(0, 20)
        k = buf.as_strided(shape, (t, h, 1), 8 * rng.randint(0, 60))
        out = buf.as_strided(shape, (t2, h2, 1), 8 * rng.randint(0, 60))
        q = torch.zeros(shape, dtype=bf16)
        buf.zero_()
        k.fill_(1.0)
        shared = bool((out == 1).any())
        with pytest.raises(ValueError) as e:
            F.fp8_qk_norm_rope(q, k, q_out=out)
        if "must lie apart" in str(e.value):
            refused += 1
            one_layout = (t, h) == (t2, h2) and T > 1 and H > 1
            assert shared or not one_layout or _turns_differ(k, out)
        else:
            taken += 1
            assert "on a GPU" in str(e.value) and not shared
    assert refused > 50 and taken > 50


def _turns_differ(a, b):
    """Rows of one layout that neither take turns row by row nor block by block (a token's heads, or a head's tokens)."""
    import math
    d = b.storage_offset() - a.storage_offset()
    (T, H, D), (t, h) = a.shape, a.stride()[:2]
    g = math.gcd(t, h)
    outer, block = (t, (H - 1) * h + D) if t >= h else (h, (T - 1) * t + D)
    return not (D <= d % g <= g - D) and not (block <= d % outer <= outer - block)


def test_fused_write_queries():
    (q, k, v), wide = _projection()
    c = _cache()
    tab, pos, slots = torch.zeros(10, 64), torch.zeros(5, dtype=i64), torch.zeros(5, dtype=i64)
    w = torch.zeros(64, dtype=bf16)

    def f(out, q=q, k=k, v=v, c=c, pos=pos, slots=slots, w=None):
        return F.fp8_qkv_cache_write(q, k, v, tab, pos, slots, c, w, w, q_out=out)

    _apart(f, None)
    _apart(f, q)
    _apart(f, torch.zeros(5, 4, 64, dtype=bf16), w=w)
    _not_apart("q_out and q", f, wide[:5, :256].view(5, 4, 64))
    _not_apart("q_out and k", f, wide[1:6, 256:].view(5, 4, 64))
    _not_apart("q_out and v", f, wide[1:6, 256:].view(5, 4, 64), k=torch.zeros_like(k))
    line = torch.zeros(4096, dtype=i64)
    out = line[16:16 + 320].view(bf16).view(5, 4, 64)
    _not_apart("q_out and positions", f, out, pos=line[12:17])
    _not_apart("q_out and slots", f, out, slots=line[335:340])
    _not_apart("q_out and q_weight", f, out, w=line[:17].view(bf16)[4:68])
    _apart(f, out, pos=line[11:16], slots=line[336:341], w=line[:16].view(bf16))
    _not_apart("q_out and the cache", f, c.v_codes.flatten()[1024:1024 + 2560].view(bf16).view(5, 4, 64))


def test_attention_outputs():
    c = _cache()
    line = torch.zeros(8192, dtype=f32)
    table, lens = torch.zeros(3, 5, dtype=i32), torch.zeros(3, dtype=i32)
    q = torch.zeros(3, 4, 64, dtype=bf16)

    def f(q=q, table=table, lens=lens, **k):
        return F.fp8_paged_attention(q, c, table, lens, **k)

    out = line[64:64 + 384].view(bf16).view(3, 4, 64)
    out32 = line[64:64 + 768].view(3, 4, 64)
    _apart(f, out=out, lse=line[52:64].view(3, 4))
    _apart(f, out=out, lse=line[448:460].view(3, 4))
    _not_apart("out and lse", f, out=out, lse=line[53:65].view(3, 4))
    _not_apart("out and lse", f, out=out32, out_dtype=f32, lse=line[831:843].view(3, 4))
    _not_apart("out and q", f, q=out, out=out)
    _not_apart("out and q", f, q=line[440:440 + 384].view(bf16).view(3, 4, 64), out=out)
    _not_apart("lse and q", f, q=out, lse=line[440:452].view(3, 4))
    _not_apart("out and block_table", f, out=out, table=line[50:65].view(i32).view(3, 5))
    _not_apart("lse and block_table", f, lse=line[60:72].view(3, 4), table=line[50:65].view(i32).view(3, 5))
    _not_apart("out and context_lens", f, out=out, lens=line[447:450].view(i32))
    _not_apart("lse and the cache", f, lse=c.k_scales.flatten()[4:16].view(3, 4))
    _not_apart("out and the cache", f, out=c.k_codes.flatten()[2048:2048 + 1536].view(bf16).view(3, 4, 64))
    y = torch.zeros(3, 8 * 64, dtype=bf16)
    _apart(f, q=y[:, :256].view(3, 4, 64), out=torch.zeros(3, 4, 64, dtype=bf16))


def test_writes_into_a_cache_that_shares_its_places():
    q, k = torch.zeros(3, 4, 64, dtype=bf16), torch.zeros(3, 2, 64, dtype=bf16)
    tab, pos, slots = torch.zeros(10, 64), torch.zeros(3, dtype=i64), torch.zeros(3, dtype=i64)
    bt, lens, offs = torch.zeros(3, 4, dtype=i32), torch.ones(3, dtype=i32), torch.zeros(4, dtype=i32)
    writes = (lambda c: F.fp8_kv_cache_write(k, k, slots, c),
              lambda c: F.fp8_qkv_cache_write(q, k, k, tab, pos, slots, c),
              lambda c: F.attention_step(q, k, k, tab, pos, slots, c, bt, lens))
    codes, scales = torch.zeros(4, 3, 2, 2, 16, 64, dtype=u8), torch.zeros(4, 3, 2, 2, 16)

    def layer(i, j, x=0, y=1):
        return _At(codes[:, i, x], codes[:, j, y], scales[:, i, x], scales[:, j, y])

    packed = torch.zeros(4, 2 * 2048 + 2 * 128, dtype=u8)          # a page: K, V, their scales
    parts = [packed[:, a:a + n] for a, n in ((0, 2048), (2048, 2048), (4096, 128), (4224, 128))]
    parts = [x.view(4, 2, 16, 64) for x in parts[:2]] + [x.view(f32).view(4, 2, 16) for x in parts[2:]]
    flat = codes.flatten()
    shifted = [flat[a:a + 8192].view(4, 2, 16, 64) for a in (0, 8176)]
    for w in writes:
        for good in (layer(0, 0), layer(1, 1), layer(2, 1), _cache(1), _At(*parts)):
            _apart(w, good)
        _not_apart("k_codes and v_codes", w, layer(1, 1, 0, 0))
        _not_apart("k_codes and v_codes", w, _At(*shifted, torch.zeros(4, 2, 16), torch.zeros(4, 2, 16)))
        c = _cache()
        _not_apart("k_scales and v_scales", w, _At(c.k_codes, c.v_codes, c.k_scales, c.k_scales))
        _not_apart("v_codes and k_scales", w,
                   _At(c.k_codes, c.v_codes, c.v_codes.flatten()[:512].view(f32).view(4, 2, 16), c.v_scales))
    one = layer(1, 1, 0, 0)                                        # reading is left alone
    _apart(F.fp8_paged_attention, q, one, bt, lens)
    _apart(F.fp8_kv_cache_read, one, bt, offs, 5)


def test_step_outputs():
    c = _cache()
    q, k = torch.zeros(3, 4, 64, dtype=bf16), torch.zeros(3, 2, 64, dtype=bf16)
    tab, pos, slots = torch.zeros(10, 64), torch.zeros(3, dtype=i64), torch.zeros(3, dtype=i64)
    bt, lens, w = torch.zeros(3, 4, dtype=i32), torch.ones(3, dtype=i32), torch.zeros(64, dtype=bf16)
    out, lse = torch.zeros(3, 4, 64, dtype=bf16), torch.zeros(3, 4)

    def f(q=q, k=k, pos=pos, slots=slots, bt=bt, w=w, **x):
        return F.attention_step(q, k, k, tab, pos, slots, c, bt, lens, w, w, **x)

    _apart(f, out=out, lse=lse)
    _not_apart("out and q", f, q=out, out=out)
    _not_apart("out and k", f, k=out.flatten()[:384].view(3, 2, 64), out=out)
    _not_apart("out and slots", f, slots=out.flatten()[:12].view(i64), out=out)
    _not_apart("out and q_weight", f, w=out.flatten()[64:128], out=out)
    _not_apart("lse and positions", f, pos=lse.flatten()[:6].view(i64), lse=lse)
    _not_apart("lse and cos_sin", f, lse=tab.flatten()[:12].view(3, 4))
    _not_apart("lse and block_table", f, bt=lse.view(i32), lse=lse)
    _not_apart("out and the cache", f, out=c.v_codes.flatten()[:1536].view(bf16).view(3, 4, 64))
    with pytest.raises(ValueError, match="out must be contiguous"):
        f(out=out.float())
    with pytest.raises(ValueError, match="lse must have shape"):
        f(lse=lse[:2])
