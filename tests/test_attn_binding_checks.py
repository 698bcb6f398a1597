"""The attention binding refuses misuse on the host before the library is
called (no GPU needed): layouts and types first, then the device."""
import ctypes

import pytest
import torch

import fp8_block_scaled_02_amd as F

bf16, f32, i32, i64, u8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8


def _raises(match, fn, *a, **k):
    with pytest.raises(ValueError, match=match):
        fn(*a, **k)


def _tensors(P=4, H=2, S=16, D=64):
    return [torch.zeros(P, H, S, D, dtype=u8), torch.zeros(P, H, S, D, dtype=u8), torch.zeros(P, H, S),
            torch.zeros(P, H, S)]


class _HostCache(F.KVCache):
    """A cache on the host, to reach the checks after the cache's own (only its sizes are read there)."""

    def __init__(self):
        self._struct = F.attention._CacheStruct(pages=4, page_size=16, heads=2, head_dim=64, fmt=F.FMT_E5M2)
        self._ref, self._dev = ctypes.addressof(self._struct), -1


def test_cache_layouts():
    make = F.KVCache.from_tensors
    _raises("on a GPU", make, *_tensors())
    _raises("fmt", make, *_tensors(), "e3m4")
    _raises("page_size", make, *_tensors(S=24))
    _raises("page_size", make, *_tensors(S=8))
    _raises("head_dim", make, *_tensors(D=72))
    _raises("head_dim", make, *_tensors(D=272))
    k, v, ks, vs = _tensors()
    _raises("v_codes must be", make, k, v.float(), ks, vs)
    _raises("v_codes must have shape", make, k, v[:3], ks, vs)
    _raises("k_scales must have shape", make, k, v, ks[:, :1], vs)
    _raises("v_scales must be", make, k, v, ks, vs.double())
    _raises("page must be contiguous", make, k, torch.zeros(4, 2, 64, 16, dtype=u8).transpose(2, 3), ks, vs)
    _raises("pages overlap", make, k[:1].expand(4, -1, -1, -1), v, ks, vs)
    _raises("equally far apart", make, torch.zeros(4, 3, 2, 16, 64, dtype=u8)[:, 0], v, ks, vs)
    _raises("one page", make, k[:0], v[:0], ks[:0], vs[:0])
    _raises("on a GPU", F.KVCache, 4, 16, 2, 64, device="cpu")


def test_norm_rope_arguments():
    q, k = torch.zeros(3, 4, 64, dtype=bf16), torch.zeros(3, 2, 64, dtype=bf16)
    tab, pos = torch.zeros(10, 64), torch.zeros(3, dtype=i64)
    f = F.fp8_qk_norm_rope
    _raises("on a GPU", f, q, k, tab, pos)
    _raises("q must be 3-D bf16", f, q.float(), k, tab, pos)
    _raises("k must be 3-D bf16", f, q, k[0], tab, pos)
    _raises("rows contiguous", f, q, torch.zeros(3, 64, 2, dtype=bf16).transpose(1, 2), tab, pos)
    _raises("k must be", f, q, k[:2], tab, pos)
    _raises("go together", f, q, k, tab, None)
    _raises("cos_sin must be", f, q, k, tab.double(), pos)
    _raises("rot_dim", f, q, k, torch.zeros(10, 24), pos)
    _raises("rot_dim", f, q, k, torch.zeros(10, 80), pos)
    _raises("at least one position", f, q, k, tab[:0], pos)
    _raises("positions must be contiguous", f, q, k, tab, pos.int())
    _raises("positions must have shape", f, q, k, tab, pos[:2])
    _raises("q_weight must be contiguous", f, q, k, tab, pos, torch.zeros(64))
    _raises("k_weight must have shape", f, q, k, tab, pos, None, torch.zeros(32, dtype=bf16))
    _raises("q_out must have shape", f, q, k, tab, pos, q_out=torch.zeros(3, 4, 32, dtype=bf16))
    _raises("k_out must be 3-D bf16", f, q, k, tab, pos, k_out=torch.zeros(3, 2, 64))


def test_outputs_lie_apart():
    q, k = torch.zeros(3, 4, 64, dtype=bf16), torch.zeros(3, 2, 64, dtype=bf16)
    f = F.fp8_qk_norm_rope
    line = torch.zeros(4096, dtype=bf16)
    _raises("q_out: rows overlap", f, q, k, q_out=q[:, :1].expand(3, 4, 64))
    _raises("q_out: rows overlap", f, q, k, q_out=q[:1].expand(3, 4, 64))
    _raises("q_out: rows overlap", f, q, k, q_out=line.as_strided((3, 4, 64), (256, 56, 1)))
    _raises("k_out: rows overlap", f, q, k, k_out=line.as_strided((3, 2, 64), (120, 64, 1)))
    for st in ((256, 64), (64, 192), (512, 72), (72, 256)):       # these do not: refused for the host's memory only
        _raises("on a GPU", f, q, k, q_out=line.as_strided((3, 4, 64), (*st, 1)))
    kv = torch.zeros(5, 2, 64, dtype=bf16)
    _raises("apart", F.fp8_kv_cache_read, _HostCache(), torch.zeros(1, 4, dtype=i32), torch.zeros(2, dtype=i32), 5, kv,
            kv)


def test_cache_calls():
    c = _HostCache()
    q, k = torch.zeros(3, 4, 64, dtype=bf16), torch.zeros(3, 2, 64, dtype=bf16)
    slots, tab, pos = torch.zeros(3, dtype=i64), torch.zeros(10, 64), torch.zeros(3, dtype=i64)
    w = F.fp8_kv_cache_write
    _raises("on a GPU", w, k, k, slots, c)
    _raises("k must have shape", w, q, q, slots, c)
    _raises("v must have shape", w, k, k[:2], slots, c)
    _raises("slots must be contiguous", w, k, k, slots.int(), c)
    _raises("slots must have shape", w, k, k, slots[:2], c)
    s = F.fp8_qkv_cache_write
    _raises("on a GPU", s, q, k, k, tab, pos, slots, c)
    _raises("q must be", s, q[:2], k, k, tab, pos, slots, c)
    _raises("q must be", s, q[..., :32], k, k, tab, pos, slots, c)
    _raises("slots must have shape", s, q, k, k, tab, pos, slots[:1], c)
    _raises("go together", s, q, k, k, None, pos, slots, c)
    r = F.fp8_kv_cache_read
    table, offs = torch.zeros(3, 5, dtype=i32), torch.zeros(4, dtype=i32)
    _raises("on a GPU", r, c, table, offs, 7)
    _raises("block_table must be 2-D", r, c, table.long(), offs, 7)
    _raises("block_table must be 2-D", r, c, torch.zeros(5, 3, dtype=i32).t(), offs, 7)
    _raises("offsets must have shape", r, c, table, offs[:3], 7)
    _raises("offsets must be contiguous", r, c, table, offs.long(), 7)
    _raises("k_out must have shape", r, c, table, offs, 7, torch.zeros(6, 2, 64, dtype=bf16))
    _raises("v_out must be contiguous", r, c, table, offs, 7, None, torch.zeros(7, 2, 64))


def test_attention_arguments():
    c = _HostCache()
    q, table, lens = torch.zeros(3, 4, 64, dtype=bf16), torch.zeros(3, 5, dtype=i32), torch.zeros(3, dtype=i32)
    f = F.fp8_paged_attention
    _raises("on a GPU", f, q, c, table, lens)
    _raises("q must be 3-D", f, q.float(), c, table, lens)
    _raises("q must be", f, q[..., :48], c, table, lens)
    _raises("multiple of the cache", f, q[:, :3], c, table, lens)
    _raises("block_table must have", f, q, c, table[:2], lens)
    _raises("context_lens must be", f, q, c, table, lens.long())
    _raises("context_lens must have shape", f, q, c, table, lens[:2])
    _raises("out_dtype", f, q, c, table, lens, out_dtype=torch.float16)
    _raises("out must be contiguous", f, q, c, table, lens, out=torch.zeros(3, 4, 64))
    _raises("out must have shape", f, q, c, table, lens, out=torch.zeros(3, 2, 64, dtype=bf16))
    _raises("max_context must be", f, q, c, table, lens, max_context=-1)
    _raises("max_context must be", f, q, c, table, lens, max_context=(1 << 30) + 1)
    _raises("window must be", f, q, c, table, lens, window=-1)
    with pytest.raises(OverflowError):
        f(q, c, table, lens, window=1 << 64)
    with pytest.raises(TypeError):
        f(q, c, table, lens, window=2.5)
    _raises("must be a tensor", f, q, c, [[0]], lens)
    _raises("lse must have shape", f, q, c, table, lens, lse=torch.zeros(3, 2))


def test_step_arguments():
    """Both halves' checks, the device last."""
    c = _HostCache()
    q, k, v = torch.zeros(3, 4, 64, dtype=bf16), torch.zeros(3, 2, 64, dtype=bf16), torch.zeros(3, 2, 64, dtype=bf16)
    tab, pos, slots = torch.zeros(10, 64), torch.zeros(3, dtype=i64), torch.zeros(3, dtype=i64)
    bt, lens = torch.zeros(3, 4, dtype=i32), torch.ones(3, dtype=i32)
    f = F.attention_step
    _raises("on a GPU", f, q, k, v, tab, pos, slots, c, bt, lens)
    _raises("q must be", f, q[:2], k, v, tab, pos, slots, c, bt, lens)
    _raises("query heads", f, q[:, :3], k, v, tab, pos, slots, c, bt, lens)
    _raises("v must have shape", f, q, k, v[:, :1], tab, pos, slots, c, bt, lens)
    _raises("go together", f, q, k, v, None, pos, slots, c, bt, lens)
    _raises("slots must be", f, q, k, v, tab, pos, slots.int(), c, bt, lens)
    _raises("block_table must have 3 rows", f, q, k, v, tab, pos, slots, c, bt[:2], lens)
    _raises("context_lens must be", f, q, k, v, tab, pos, slots, c, bt, lens.long())
    _raises("window", f, q, k, v, tab, pos, slots, c, bt, lens, window=-1)
    _raises("max_context", f, q, k, v, tab, pos, slots, c, bt, lens, max_context=-1)
    _raises("out_dtype", f, q, k, v, tab, pos, slots, c, bt, lens, out_dtype=torch.float16)
