"""What the calls of expert routing and the integer layers do not take, refused
on the host before anything is launched (no GPU needed)."""
import pytest
import torch

import fp8_block_scaled_02_amd as F

bf16, f32, i32, i8 = torch.bfloat16, torch.float32, torch.int32, torch.int8


def _raises(match, fn, *a, **k):
    with pytest.raises(ValueError, match=match):
        fn(*a, **k)


def _calls():
    """(call, its arguments, positions of those that may require a gradient)."""
    l, g, e = torch.zeros(4, 16), torch.zeros(4, 2), torch.zeros(4, 2, dtype=i32)
    x, y = torch.zeros(4, 100), torch.zeros(8, 100)
    a = torch.zeros(4, 128, dtype=i8)[:, :100]
    w, sw, b = torch.zeros(32, 128, dtype=i8), torch.zeros(20), torch.zeros(20)
    we, swe, offs = torch.zeros(3, 32, 128, dtype=i8), torch.zeros(3, 20), torch.zeros(4, dtype=i32)
    return [(F.moe_route, [l, 2], [0]), (F.moe_route_backward, [g, l, g, e, True, torch.zeros(4, 16)], [0, 1, 2, 5]),
            (F.moe_gather, [x, e, None, y], [0, 3]), (F.moe_gather_backward, [y, e, x], [0, 2]),
            (F.moe_combine, [y, e, g, None, x], [0, 2, 4]),
            (F.moe_combine_backward, [x, y, e, g, torch.zeros(8, 100), torch.zeros(4, 2)], [0, 1, 3, 4, 5]),
            (F.int8_quant, [x, None, torch.zeros(4)], [0, 2]),
            (F.int8_gemm, [a, torch.zeros(4), w, sw, b, f32, torch.zeros(4, 20)], [1, 3, 4, 6]),
            (F.int8_grouped_gemm, [a, torch.zeros(4), e[:, 0].contiguous(), offs, we, swe, f32, torch.zeros(4, 20)], [1, 5, 7]),
            (F.int8_linear, [x, w, sw, b], [0, 2, 3]), (F.int8_moe_forward, [x, torch.zeros(4, 3), 2, we, swe], [0, 1, 4])]


@pytest.mark.parametrize("i", range(11))
def test_tensors_that_require_a_gradient(i):
    """A gradient that nothing records is not dropped without a word."""
    fn, args, places = _calls()[i]
    _raises("on a GPU", fn, *args)
    for p in places:
        wants = list(args)
        wants[p] = args[p].clone().requires_grad_()
        _raises("requires a gradient", fn, *wants)
        made = list(args)
        made[p] = wants[p] * 1                                      # made from one that does
        _raises("requires a gradient", fn, *made)
        with torch.no_grad():
            _raises("on a GPU", fn, *wants)
        with torch.inference_mode():
            _raises("on a GPU", fn, *wants)
        _raises("on a GPU", fn, *[t.detach() if isinstance(t, torch.Tensor) else t for t in made])


def test_inside_an_autograd_function():
    class Route(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits):
            return F.moe_route(logits, 2).gates

    _raises("on a GPU", Route.apply, torch.zeros(4, 16, requires_grad=True))
