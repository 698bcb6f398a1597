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
