"""The binding of expert routing and the integer layers refuses misuse on the
host before the library is called (no GPU needed): layouts and types first,
then the device."""
import pytest
import torch

import fp8_block_scaled_02_amd as F

bf16, f32, i32, i8 = torch.bfloat16, torch.float32, torch.int32, torch.int8


def _raises(match, fn, *a, **k):
    with pytest.raises(ValueError, match=match):
        fn(*a, **k)


def test_route():
    l = torch.zeros(4, 16)
    f = F.moe_route
    _raises("on a GPU", f, l, 2)
    _raises("on a GPU", f, l.bfloat16(), 16)
    _raises("bfloat16 or float32", f, l.double(), 2)
    _raises("2-D", f, l[0], 2)
    _raises("rows contiguous", f, torch.zeros(16, 4).t(), 2)
    _raises("rows overlap", f, l[:1].expand(4, 16), 2)
    for k in (0, 17, -1):
        _raises("k must be", f, l, k)
    _raises("k must be", f, torch.zeros(4, 100), 65)
    _raises("1 to 1024 experts", f, torch.zeros(4, 1025), 2)
    _raises("1 to 1024 experts", f, l[:, :0], 1)
    with pytest.raises(TypeError):
        f(l, 2.5)
    with pytest.raises(OverflowError):
        f(l, 1 << 70)


def test_sort():
    e = torch.zeros(4, 2, dtype=i32)
    _raises("on a GPU", F.moe_sort, e, 8)
    _raises("int32", F.moe_sort, e.long(), 8)
    _raises("int32", F.moe_sort, e[0], 8)
    _raises("contiguous", F.moe_sort, torch.zeros(2, 4, dtype=i32).t(), 8)
    _raises("1 to 64 slots", F.moe_sort, e[:, :0], 8)
    _raises("1 to 64 slots", F.moe_sort, torch.zeros(4, 65, dtype=i32), 8)
    for E in (0, 1025):
        _raises("1 to 1024 experts", F.moe_sort, e, E)


def test_route_backward():
    l, g, e = torch.zeros(4, 16), torch.zeros(4, 2), torch.zeros(4, 2, dtype=i32)
    f = F.moe_route_backward
    _raises("on a GPU", f, g.clone(), l, g, e)
    _raises("dgates must have shape", f, g[:3], l, g, e)
    _raises("dgates must be contiguous float32", f, g.bfloat16(), l, g, e)
    _raises("gates must have shape", f, g, l, torch.zeros(4, 3), e)
    _raises("experts must have 4 rows", f, g, l, g, e[:3])
    _raises("out must be float32", f, g, l, g, e, out=l.bfloat16())
    _raises("out must have shape", f, g, l, g, e, out=torch.zeros(4, 8))
    _raises("out and logits must lie apart", f, g, l, g, e, out=l)
    _raises("on a GPU", f, g, l, g, e, out=torch.zeros(4, 32)[:, 16:])


def test_rows():
    x, tr = torch.zeros(4, 32), torch.zeros(4, 2, dtype=i32)
    g = torch.zeros(4, 2)
    f = F.moe_gather
    _raises("on a GPU", f, x, tr)
    _raises("bfloat16 or float32", f, x.half(), tr)
    _raises("token_rows must have 4 rows", f, x, tr[:3])
    _raises("token_rows must be contiguous int32", f, x, tr.long())
    _raises("x must have a column", f, x[:, :0], tr)
    _raises("rows must be", f, x, tr, rows=-1)
    _raises("out must have shape", f, x, tr, rows=8, out=torch.zeros(7, 32))
    _raises("out must be float32", f, x, tr, out=torch.zeros(8, 32, dtype=bf16))
    both = torch.zeros(8, 80)
    _raises("out and x must lie apart", f, both[:4, :32], tr, out=both[:, 16:48])
    _raises("on a GPU", f, both[:4, :32], tr, out=both[:, 32:64])       # columns that take turns are apart
    y = torch.zeros(8, 32)
    c = F.moe_combine
    _raises("on a GPU", c, y, tr, g)
    _raises("gates must be a tensor", c, y, tr, None)
    _raises("gates must have shape", c, y, tr, g[:3])
    _raises("out_dtype", c, y, tr, g, torch.float16)
    _raises("out must be bfloat16", c, y, tr, g, bf16, torch.zeros(4, 32))
    _raises("out must have shape", c, y, tr, g, None, torch.zeros(3, 32))
    _raises("out and y must lie apart", c, y, tr, g, None, y[:4])
    _raises("on a GPU", F.moe_gather_backward, y, tr)
    b = F.moe_combine_backward
    d = torch.zeros(4, 32)
    _raises("on a GPU", b, d, y, tr, g)
    _raises("dout must have shape", b, d[:, :16], y, tr, g)
    _raises("rows overlap", b, d[:1].expand(4, 32), y, tr, g)
    _raises("dy must be float32", b, d, y, tr, g, dy=y.bfloat16())
    _raises("dy and y must lie apart", b, d, y, tr, g, dy=y)
    _raises("dgates must have shape", b, d, y, tr, g, dgates=torch.zeros(4, 3))
    _raises("dgates and gates must lie apart", b, d, y, tr, g, dgates=g)


def test_quant_and_pack():
    x = torch.zeros(4, 100)
    f = F.int8_quant
    _raises("on a GPU", f, x)
    _raises("bfloat16 or float32", f, x.double())
    _raises("2-D", f, x[0])
    _raises("codes must be int8", f, x, torch.zeros(4, 100, dtype=torch.uint8))
    _raises("codes must have shape", f, x, torch.zeros(4, 99, dtype=i8))
    _raises("scales must have shape", f, x, None, torch.zeros(3))
    room = torch.zeros(4, 100)
    _raises("codes and x must lie apart", f, room, room.view(i8)[:, :100])
    w = torch.zeros(3, 20, 100, dtype=i8)
    p = F.int8_weight_pack
    _raises("on a GPU", p, w)
    _raises("on a GPU", p, w[0])
    _raises("must be int8", p, w.to(torch.uint8))
    _raises("must be int8", p, w[0, 0])
    _raises("rows must be contiguous", p, w.transpose(1, 2))
    _raises("at least one matrix", p, w[:0])
    _raises("at least one matrix", p, torch.zeros(1, 131072, dtype=i8))
    _raises("rows overlap", p, w[:, :1].expand(3, 20, 100))
    _raises("out must have shape", p, w, torch.zeros(3, 20, 128, dtype=i8))
    _raises("out must be contiguous int8", p, w, torch.zeros(3, 32, 128))


def _operands(M=4, N=20, K=100, E=None):
    a = torch.zeros(M, 128, dtype=i8)[:, :K]
    lead = () if E is None else (E,)
    return a, torch.zeros(M), torch.zeros(*lead, 32, 128, dtype=i8), torch.zeros(*lead, N)


def test_gemm():
    a, sa, w, sw = _operands()
    f = F.int8_gemm
    _raises("on a GPU", f, a, sa, w, sw)
    _raises("on a GPU", f, a[:1], sa[:1], w, sw)
    _raises("a must be int8", f, a.to(torch.uint8), sa, w, sw)
    _raises("filled up to a multiple of 128", f, torch.zeros(4, 100, dtype=i8), sa, w, sw)
    _raises("multiple of 16", f, torch.zeros(4, 136, dtype=i8)[:, :100], sa, w, sw)
    _raises("last row", f, torch.zeros(1, 100, dtype=i8), sa[:1], w, sw)
    _raises("last row", f, torch.zeros(3 * 128 + 100, dtype=i8).as_strided((4, 100), (128, 1)), sa, w, sw)
    _raises("a_scales must have shape", f, a, sa[:3], w, sw)
    _raises("w_packed must be contiguous int8", f, a, sa, w.float(), sw)
    _raises("w_packed must be contiguous int8", f, a, sa, w[None], sw)
    _raises("20 rows", f, a, sa, w[:16], sw)
    _raises("100 columns", f, a, sa, torch.zeros(32, 256, dtype=i8), sw)
    _raises("w_scales must be", f, a, sa, w, sw.double())
    _raises("w_scales must be", f, a, sa, w, sw[None])
    _raises("bias must have shape", f, a, sa, w, sw, torch.zeros(19))
    _raises("bias must be contiguous float32", f, a, sa, w, sw, sw.bfloat16())
    _raises("out_dtype", f, a, sa, w, sw, None, torch.float16)
    _raises("y must be bfloat16", f, a, sa, w, sw, None, bf16, torch.zeros(4, 20))
    _raises("y must have shape", f, a, sa, w, sw, None, f32, torch.zeros(4, 21))
    b = torch.zeros(20)
    _raises("y and bias must lie apart", f, a[:1], sa[:1], w, sw, b, f32, b[None])
    x = torch.zeros(4, 100)
    _raises("on a GPU", F.int8_linear, x, w, sw)
    _raises("bfloat16 or float32", F.int8_linear, x.half(), w, sw)
    _raises("columns", F.int8_linear, torch.zeros(4, 200), w, sw)
    _raises("out_dtype", F.int8_linear, x, w, sw, None, torch.float16)


def test_grouped():
    a, sa, w, sw = _operands(E=3)
    index, offs = torch.zeros(6, dtype=i32), torch.zeros(4, dtype=i32)
    f = F.int8_grouped_gemm
    _raises("on a GPU", f, a, sa, index, offs, w, sw)
    _raises("on a GPU", f, a, sa, None, offs, w, sw)
    _raises("row_index must be", f, a, sa, index.long(), offs, w, sw)
    _raises("row_index must be", f, a, sa, index.view(2, 3), offs, w, sw)
    _raises("expert_offsets must have shape", f, a, sa, index, offs[:3], w, sw)
    _raises("w_packed must be contiguous int8 .E", f, a, sa, index, offs, w[0], sw)
    _raises("as many experts", f, a, sa, index, offs, w, sw[:2])
    _raises("a must have a row", f, a[:0], sa[:0], index, offs, w, sw)
    _raises("y must have shape", f, a, sa, index, offs, w, sw, bf16, torch.zeros(4, 20, dtype=bf16))
    x, l = torch.zeros(4, 100), torch.zeros(4, 3)
    g = F.int8_moe_forward
    _raises("on a GPU", g, x, l, 2, w, sw)
    _raises("k must be", g, x, l, 4, w, sw)
    _raises("logits must have 4 rows", g, x, l[:3], 2, w, sw)
    _raises("logits must be of 3 experts", g, x, torch.zeros(4, 5), 2, w, sw)
    _raises("must be a tensor", F.moe_gather, x, [[0]])


def test_everything_is_built(tmp_path, monkeypatch):
    """Both libraries of the routing and the integer layers, beside the others."""
    import os

    from fp8_block_scaled_02_amd import build
    for name in ("LIB", "ATTN_LIB", "ATTN_BINDING", "MOE_LIB", "MOE_BINDING"):
        monkeypatch.setattr(build, name, str(tmp_path / os.path.basename(getattr(build, name))))
    monkeypatch.setattr(build.subprocess, "check_call", lambda cmd: open(cmd[cmd.index("-o") + 1], "w").close())
    assert build.build_all() == build.LIB
    assert sorted(os.listdir(tmp_path)) == ["_attn_binding.so", "_moe_binding.so", "libfp8attn.so", "libfp8blk.so",
                                            "libfp8moe.so"]
