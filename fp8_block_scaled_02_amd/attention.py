"""Python binding of libfp8attn: the attention side of a decode step on a
paged FP8 key-value cache (C ABI: include/fp8attn.h).

As in the package itself, argument marshalling only: checks, outputs and the
attention's workspace allocated with torch, the current torch stream of the
tensors' device.  There is no fallback: if libfp8attn.so is missing the
functions raise on first use.  Nothing here records a gradient.
"""
import ctypes
import os

import torch

from . import FMT_E4M3, FMT_E5M2, OUT_BF16, OUT_F32, Fp8Error, _need, _shape

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp8attn.so")
MAX_CONTEXT = 1 << 30    # the longest max_context fp8_paged_attention takes

_CACHE_FMT = {"e5m2": FMT_E5M2, "e4m3": FMT_E4M3}

_attn_lib = None


class _CacheStruct(ctypes.Structure):    # fp8b_kv_cache of include/fp8attn.h
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k_codes", "v_codes", "k_scales", "v_scales")] +
                [(n, ctypes.c_int64) for n in ("page_stride", "scale_page_stride", "pages", "page_size", "heads",
                                               "head_dim")] +
                [("fmt", ctypes.c_int32), ("reserved", ctypes.c_int32)])


class _RopeStruct(ctypes.Structure):     # fp8b_rope of include/fp8attn.h
    _fields_ = ([(n, ctypes.c_void_p) for n in ("q_weight", "k_weight", "cos_sin", "positions")] +
                [("max_pos", ctypes.c_int64), ("rot_dim", ctypes.c_int64), ("eps", ctypes.c_float),
                 ("interleaved", ctypes.c_int32)])


def attn_lib():
    """The loaded libfp8attn.so (raises if it has not been built)."""
    global _attn_lib
    if _attn_lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m fp8_block_scaled_02_amd.build` (there is no CPU fallback)")
        L = ctypes.CDLL(LIB_PATH)
        i64, vp, ci = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
        rows = [vp, i64, i64]
        L.fp8b_attn_abi_version.restype = ci
        L.fp8b_attn_abi_version.argtypes = []
        L.fp8_qk_norm_rope.restype = ci
        L.fp8_qk_norm_rope.argtypes = rows + rows + [i64, i64, i64, i64, vp] + rows + rows + [vp]
        L.fp8_kv_cache_write.restype = ci
        L.fp8_kv_cache_write.argtypes = rows + rows + [vp, i64, vp, vp]
        L.fp8_qkv_cache_write.restype = ci
        L.fp8_qkv_cache_write.argtypes = rows + rows + rows + [vp, i64, i64, vp, vp] + rows + [vp]
        L.fp8_kv_cache_read.restype = ci
        L.fp8_kv_cache_read.argtypes = [vp, vp, i64, i64, vp, i64, i64, vp, vp, vp]
        L.fp8_paged_attention_workspace.restype = i64
        L.fp8_paged_attention_workspace.argtypes = [vp, i64, i64, i64, i64, i64]
        L.fp8_paged_attention.restype = ci
        L.fp8_paged_attention.argtypes = rows + [vp, vp, i64, i64, vp, i64, i64, i64, i64, ctypes.c_float, vp, ci, vp,
                                                 vp, vp]
        _attn_lib = L
    return _attn_lib


_bf16, _f32, _i32, _i64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
_contiguous = torch.contiguous_format
_current_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _call(fn, dev, *args):
    """One C call on the current stream of GPU `dev`, which is made current
    for it: a default stream is NULL, which means the current device's."""
    f = getattr(_attn_lib or attn_lib(), fn)
    if dev == _current_device():
        rc = f(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            rc = f(*args, _raw_stream(dev))
    if rc:
        raise Fp8Error(fn, rc)


# The checks below build their messages only when they fail: a decode step on
# a few sequences is bound by the host.


def _on(dev, *ts):
    """Every tensor is on GPU number `dev`: the kernels dereference data_ptr()
    as its memory."""
    if dev < 0:
        raise ValueError("every tensor must be on a GPU (found one on the host)")
    for t in ts:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"every tensor must be on cuda:{dev} (found one on {t.device})")


def _rows(t, name):
    """(address, token stride, head stride) of bf16 [tokens, heads, D]; the
    stride of a dimension of one entry means nothing and is put in order."""
    if t.dtype is not _bf16 or t.ndim != 3:
        raise ValueError(f"{name} must be 3-D bf16 [tokens, heads, head_dim], head rows contiguous")
    T, H, D = t.shape
    st, sh, sd = t.stride()
    if sd != 1 and D != 1:
        raise ValueError(f"{name} must be 3-D bf16 [tokens, heads, head_dim], head rows contiguous")
    if H <= 1:
        sh = D
    return t.data_ptr(), (st if T > 1 else sh * H), sh


def _index(t, dtype, shape, name):
    if t.dtype is not dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype}")
    if t.shape != shape:
        _shape(t, shape, name)


def _out(t, shape, name):
    if t.shape != shape:
        _shape(t, shape, name)
    return t


def _empty_like(t):
    """An uninitialised contiguous tensor (half the host time of torch.empty)."""
    return torch.empty_like(t, memory_format=_contiguous)


class KVCache:
    """A paged key-value cache of one layer in E5M2 or E4M3 codes with one
    fp32 scale per token and head: k_codes, v_codes uint8 [pages, heads,
    page_size, head_dim] and k_scales, v_scales float32 [pages, heads,
    page_size].  Slot s is page s // page_size, place s % page_size.

    KVCache(pages, page_size, heads, head_dim) allocates one (its contents
    are arbitrary until written; what is not read through a length has no
    effect); from_tensors() takes tensors the caller keeps, whose pages may
    lie any distance apart, the same for K and V (one layer of a larger
    allocation, K and V side by side)."""

    def __init__(self, pages, page_size, heads, head_dim, fmt="e5m2", device="cuda"):
        codes = [torch.empty(pages, heads, page_size, head_dim, dtype=torch.uint8, device=device) for _ in range(2)]
        scales = [torch.empty(pages, heads, page_size, dtype=torch.float32, device=device) for _ in range(2)]
        self._take(*codes, *scales, fmt)

    @classmethod
    def from_tensors(cls, k_codes, v_codes, k_scales, v_scales, fmt="e5m2"):
        self = cls.__new__(cls)
        self._take(k_codes, v_codes, k_scales, v_scales, fmt)
        return self

    def _take(self, k_codes, v_codes, k_scales, v_scales, fmt):
        _need(fmt in _CACHE_FMT, "fmt must be 'e5m2' or 'e4m3'")
        _need(k_codes.dim() == 4, "k_codes must be [pages, heads, page_size, head_dim]")
        P, H, S, D = k_codes.shape
        _need(P >= 1 and 1 <= H <= 1024, "a cache has at least one page and 1 to 1024 heads")
        _need(16 <= S <= 4096 and S & (S - 1) == 0, "page_size must be a power of two from 16 to 4096")
        _need(16 <= D <= 256 and D % 16 == 0, "head_dim must be a multiple of 16 from 16 to 256")
        strides = []
        for t, dtype, shape, name in ((k_codes, torch.uint8, (P, H, S, D), "k_codes"),
                                      (v_codes, torch.uint8, (P, H, S, D), "v_codes"),
                                      (k_scales, torch.float32, (P, H, S), "k_scales"),
                                      (v_scales, torch.float32, (P, H, S), "v_scales")):
            _need(t.dtype == dtype, f"{name} must be {dtype}")
            _shape(t, shape, name)
            _need(t[0].is_contiguous(), f"{name}: a page must be contiguous")
            _need(P == 1 or t.stride(0) >= t[0].numel(), f"{name}: pages overlap")
            strides.append(t.stride(0) if P > 1 else t[0].numel())
        _need(strides[0] == strides[1] and strides[2] == strides[3], "K and V pages must lie equally far apart")
        _on(k_codes.get_device(), v_codes, k_scales, v_scales)
        self._tensors = k_codes, v_codes, k_scales, v_scales
        self.pages, self.heads, self.page_size, self.head_dim, self.fmt = P, H, S, D, fmt
        self.device = k_codes.device
        self._dev = k_codes.get_device()
        self._bf16 = torch.empty(0, dtype=torch.bfloat16, device=k_codes.device)    # makes outputs of its kind
        self._struct = _CacheStruct(k_codes.data_ptr(), v_codes.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
                                    strides[0], strides[2], P, S, H, D, _CACHE_FMT[fmt], 0)
        self._ref = ctypes.addressof(self._struct)

    # read-only: the addresses were taken when the cache was made
    k_codes = property(lambda self: self._tensors[0])
    v_codes = property(lambda self: self._tensors[1])
    k_scales = property(lambda self: self._tensors[2])
    v_scales = property(lambda self: self._tensors[3])


def _rope(D, T, cos_sin, positions, q_weight, k_weight, eps, interleaved):
    if (cos_sin is None) != (positions is None):
        raise ValueError("cos_sin and positions go together")
    cs = pos = qw = kw = None
    n = rot = 0
    if cos_sin is not None:
        if cos_sin.dtype is not _f32 or cos_sin.ndim != 2 or not cos_sin.is_contiguous():
            raise ValueError("cos_sin must be contiguous float32 [max_pos, rot_dim]")
        n, rot = cos_sin.shape
        if not 16 <= rot <= D or rot % 16:
            raise ValueError(f"rot_dim must be a multiple of 16 from 16 to {D}")
        if n < 1:
            raise ValueError("cos_sin must hold at least one position")
        _index(positions, _i64, (T,), "positions")
        cs, pos = cos_sin.data_ptr(), positions.data_ptr()
    if q_weight is not None:
        _index(q_weight, _bf16, (D,), "q_weight")
        qw = q_weight.data_ptr()
    if k_weight is not None:
        _index(k_weight, _bf16, (D,), "k_weight")
        kw = k_weight.data_ptr()
    return _RopeStruct(qw, kw, cs, pos, n, rot, eps, bool(interleaved))


def fp8_qk_norm_rope(q, k, cos_sin=None, positions=None, q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                     q_out=None, k_out=None):
    """RMS norm of each query and key head (where its weight is given) and
    rotation by the position, in one pass: q [T, Hq, D] and k [T, Hk, D]
    bf16 with any token and head strides (multiples of 8), cos_sin float32
    [max_pos, rot_dim] (cosines, then sines, of each position), positions
    int64 [T], weights bf16 [D].  Returns (q_out, k_out) bf16; an output may
    be its input."""
    qa, ka = _rows(q, "q"), _rows(k, "k")
    T, Hq, D = q.shape
    Tk, Hk, Dk = k.shape
    if Tk != T or Dk != D:
        raise ValueError(f"k must be [{T}, Hk, {D}]")
    r = _rope(D, T, cos_sin, positions, q_weight, k_weight, eps, interleaved)
    q_out = _empty_like(q) if q_out is None else _out(q_out, q.shape, "q_out")
    k_out = _empty_like(k) if k_out is None else _out(k_out, k.shape, "k_out")
    qo, ko = _rows(q_out, "q_out"), _rows(k_out, "k_out")
    dev = q.get_device()
    _on(dev, k, cos_sin, positions, q_weight, k_weight, q_out, k_out)
    _call("fp8_qk_norm_rope", dev, *qa, *ka, T, Hq, Hk, D, ctypes.addressof(r), *qo, *ko)
    return q_out, k_out


def _kv_rows(k, v, cache):
    ka, va = _rows(k, "k"), _rows(v, "v")
    T = k.shape[0]
    _out(k, (T, cache.heads, cache.head_dim), "k")
    _out(v, k.shape, "v")
    return T, ka, va


def fp8_kv_cache_write(k, v, slots, cache: KVCache):
    """Quantise k, v bf16 [T, heads, D] (any token and head strides that are
    multiples of 8) into the cache at slots int64 [T]; a slot outside the
    cache, such as -1, writes nothing.  Slots should differ: one named twice
    holds either token's row, or a mixture.  Returns the cache."""
    T, ka, va = _kv_rows(k, v, cache)
    _index(slots, _i64, (T,), "slots")
    _on(cache._dev, k, v, slots)
    _call("fp8_kv_cache_write", cache._dev, *ka, *va, slots.data_ptr(), T, cache._ref)
    return cache


def fp8_qkv_cache_write(q, k, v, cos_sin, positions, slots, cache: KVCache, q_weight=None, k_weight=None, eps=1e-6,
                        interleaved=False, q_out=None):
    """fp8_qk_norm_rope and fp8_kv_cache_write in one launch (the same bits):
    returns the queries, normed and rotated; the keys, normed and rotated,
    and the values go to the cache."""
    qa = _rows(q, "q")
    T, ka, va = _kv_rows(k, v, cache)
    Tq, Hq, D = q.shape
    if Tq != T or D != cache.head_dim:
        raise ValueError(f"q must be [{T}, Hq, {cache.head_dim}]")
    r = _rope(D, T, cos_sin, positions, q_weight, k_weight, eps, interleaved)
    _index(slots, _i64, (T,), "slots")
    q_out = _empty_like(q) if q_out is None else _out(q_out, q.shape, "q_out")
    qo = _rows(q_out, "q_out")
    _on(cache._dev, q, k, v, cos_sin, positions, slots, q_weight, k_weight, q_out)
    _call("fp8_qkv_cache_write", cache._dev, *qa, *ka, *va, slots.data_ptr(), T, Hq, ctypes.addressof(r), cache._ref,
          *qo)
    return q_out


def _table(block_table):
    if block_table.dtype is not _i32 or block_table.ndim != 2:
        raise ValueError("block_table must be 2-D int32, rows contiguous")
    B, cols = block_table.shape
    ld, one = block_table.stride()
    if one != 1 and cols != 1:
        raise ValueError("block_table must be 2-D int32, rows contiguous")
    return B, block_table.data_ptr(), (ld if B > 1 else cols), cols


def fp8_kv_cache_read(cache: KVCache, block_table, offsets, rows: int, k_out=None, v_out=None):
    """The cache back as bf16: sequence b's tokens are rows offsets[b] to
    offsets[b + 1] of k_out, v_out [rows, heads, head_dim].  block_table
    int32 [B, cols]: each sequence's pages in order; offsets int32 [B + 1];
    rows from offsets[B] on are left as they were."""
    B, *table = _table(block_table)
    _index(offsets, _i32, (B + 1,), "offsets")
    shape = (rows, cache.heads, cache.head_dim)
    outs = []
    for t, name in ((k_out, "k_out"), (v_out, "v_out")):
        if t is None:
            t = cache._bf16.new_empty(shape)
        _index(t, _bf16, shape, name)
        outs.append(t)
    k_out, v_out = outs
    _on(cache._dev, block_table, offsets, k_out, v_out)
    _call("fp8_kv_cache_read", cache._dev, cache._ref, *table, offsets.data_ptr(), B, rows, k_out.data_ptr(),
          v_out.data_ptr())
    return k_out, v_out


def fp8_paged_attention(q, cache: KVCache, block_table, context_lens, scale=None, window: int = 0,
                        out_dtype=torch.bfloat16, out=None, lse=None, max_context=None):
    """Attention of one new token per sequence over the paged cache: q bf16
    [B, Hq, D] (any strides that are multiples of 8; Hq a multiple of the
    cache's heads), block_table int32 [B, cols], context_lens int32 [B]
    (tokens in the cache, the new one among them; 0 gives a row of zeros).
    scale defaults to D ** -0.5; window > 0 sees only the last `window`
    tokens.  max_context, if given, cuts longer lengths: a tight value saves
    the splitting of short contexts.  Returns out [B, Hq, D] (bf16 or
    fp32); lse, if given (float32 [B, Hq]), receives the log of the sum of
    exponentials, -inf for an empty row."""
    qa = _rows(q, "q")
    shape = q.shape
    B, Hq, D = shape
    if D != cache.head_dim:
        raise ValueError(f"q must be [B, Hq, {cache.head_dim}]")
    if Hq < 1 or Hq % cache.heads:
        raise ValueError(f"query heads must be a multiple of the cache's {cache.heads}")
    Bt, table, ld, cols = _table(block_table)
    if Bt != B:
        raise ValueError(f"block_table must have {B} rows")
    _index(context_lens, _i32, (B,), "context_lens")
    if out_dtype is _bf16:
        od = OUT_BF16
    elif out_dtype is _f32:
        od = OUT_F32
    else:
        raise ValueError("out_dtype must be bfloat16 or float32")
    if out is not None:
        _index(out, out_dtype, shape, "out")
    elif od == OUT_BF16:
        out = _empty_like(q)
    else:
        out = torch.empty(shape, dtype=out_dtype, device=q.device)
    if lse is not None:
        _index(lse, _f32, (B, Hq), "lse")
    if max_context is None:
        max_context = min(cols * cache.page_size, MAX_CONTEXT)
    elif not 0 <= max_context <= MAX_CONTEXT:
        raise ValueError(f"max_context must be from 0 to {MAX_CONTEXT}")
    if not 0 <= window < 1 << 63:
        raise ValueError("window must be 0 or a number of tokens")
    dev = cache._dev
    _on(dev, q, block_table, context_lens, out, lse)
    nbytes = (_attn_lib or attn_lib()).fp8_paged_attention_workspace(cache._ref, B, Hq, cols, max_context, window)
    if nbytes < 0:
        raise Fp8Error("fp8_paged_attention", nbytes)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=q.device) if nbytes else None
    _call("fp8_paged_attention", dev, *qa, cache._ref, table, ld, cols, context_lens.data_ptr(), B, Hq, max_context,
          window, D ** -0.5 if scale is None else scale, out.data_ptr(), od, None if lse is None else lse.data_ptr(),
          None if ws is None else ws.data_ptr())
    return out


def attention_step(q, k, v, cos_sin, positions, slots, cache: KVCache, block_table, context_lens, q_weight=None,
                   k_weight=None, eps=1e-6, interleaved=False, scale=None, window: int = 0, out_dtype=torch.bfloat16,
                   max_context=None):
    """The attention side of one decode step, between the q/k/v projection
    and the output projection: norm and rotate the new token's queries and
    keys, quantise its K and V into the cache, attend.  context_lens counts
    the new token.  Returns out [B, Hq, D]."""
    q = fp8_qkv_cache_write(q, k, v, cos_sin, positions, slots, cache, q_weight, k_weight, eps, interleaved)
    return fp8_paged_attention(q, cache, block_table, context_lens, scale, window, out_dtype,
                               max_context=max_context)
