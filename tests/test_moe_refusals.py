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


def _meta(shape, dtype=i8):
    """Sizes alone, of arrays that no machine holds."""
    return torch.empty(shape, dtype=dtype, device="meta")


def test_limits_of_a_whole_layer():
    """A size that any part of int8_linear or int8_moe_forward does not take is
    refused before the first part runs."""
    def layer(T, K, E, k, N):
        F.int8_moe_forward(_meta((T, K), bf16), _meta((T, E), bf16), k, _meta((E, -(-N // 16) * 16, -(-K // 128) * 128)),
                           _meta((E, N), f32))

    _raises("fewer than 2.24", layer, 1 << 22, 16, 8, 4, 16)
    _raises("on a GPU", layer, (1 << 22) - 1, 16, 8, 4, 16)
    _raises("too many codes", layer, 1 << 16, 1 << 16, 8, 2, 16)
    _raises("too many codes", layer, 1 << 23, 400, 8, 1, 16)
    _raises("on a GPU", layer, (1 << 16) - 1, 1 << 16, 8, 2, 16)
    _raises("too many results", layer, 1 << 23, 16, 8, 1, 8193)
    _raises("on a GPU", layer, 1 << 23, 16, 8, 1, 8192)
    _raises("too many weight rows", layer, 8, 16, 1024, 2, (1 << 20) + 1)
    _raises("on a GPU", layer, 8, 16, 1024, 2, 1 << 20)
    _raises("2.25 columns", layer, 8, 16, 1, 1, (1 << 25) + 1)
    _raises("rows_dtype must be", F.int8_moe_forward, _meta((8, 16), bf16), _meta((8, 4)), 2, _meta((4, 16, 128)),
            _meta((4, 16), f32), True, None, torch.float16)

    def linear(M, K, N):
        F.int8_linear(_meta((M, K), bf16), _meta((-(-N // 16) * 16, -(-K // 128) * 128)), _meta((N,), f32))

    _raises("fewer than 2.24", linear, 1 << 24, 16, 16)
    _raises("too many results", linear, 1 << 23, 16, 8193)
    _raises("2.25 columns", linear, 8, 16, (1 << 25) + 1)
    _raises("on a GPU", linear, 1 << 23, 16, 8192)
    _raises("on a GPU", linear, 2048, 16, 1 << 25)


EINVAL, F32, BF16 = -1, 0, 1
GOOD = 1 << 20                                                      # an address, never dereferenced here


def _refuses(f, good, cases):
    """Each case: (position: value, ..., status), the other arguments as in good."""
    for over, want in cases:
        a = list(good)
        for i, v in over.items():
            a[i] = v
        assert f(*a) == want, (over, want)


def test_leading_dimensions_whose_offsets_would_not_fit():
    """Rows times their distance: offsets in bytes stay within 63 bits."""
    L, far = F.moe_lib(), 1 << 40
    T = (1 << 24) - 1                                       # times 2^40 elements: past 2^63 bytes
    good = [GOOD, BF16, 64, 4, 64, 8, 1, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, None]
    _refuses(L.moe_route, good, [({3: T, 2: far}, EINVAL)])
    good = [GOOD, GOOD, F32, 64, GOOD, GOOD, 4, 64, 8, 0, GOOD, 64, None]
    _refuses(L.moe_route_backward, good, [({6: T, 3: far}, EINVAL), ({6: T, 11: far}, EINVAL)])
    good = [GOOD, F32, 64, 4, 64, GOOD, 8, 32, GOOD, 64, None]
    _refuses(L.moe_gather, good, [({3: T, 2: far}, EINVAL), ({7: (1 << 30) - 1, 9: far}, EINVAL)])
    good = [GOOD, F32, 64, 32, 64, GOOD, GOOD, 4, 8, GOOD, BF16, 64, None]
    _refuses(L.moe_combine, good, [({3: (1 << 30) - 1, 2: far}, EINVAL), ({7: T, 11: far}, EINVAL)])
    good = [GOOD, BF16, 64, GOOD, F32, 64, 32, 64, GOOD, GOOD, 4, 8, GOOD, 64, GOOD, None]
    _refuses(L.moe_combine_backward, good, [({10: T, 2: far}, EINVAL), ({6: (1 << 30) - 1, 5: far}, EINVAL),
                                            ({6: (1 << 30) - 1, 13: far}, EINVAL)])
    good = [GOOD, F32, 4, 64, 64, GOOD, 64, GOOD, None]
    _refuses(L.int8_quant, good, [({2: T, 4: far}, EINVAL), ({2: T, 6: far}, EINVAL)])
    good = [GOOD, 2, 64, 64, 64, 4096, GOOD, None]
    _refuses(L.int8_weight_pack, good, [({2: 1 << 25, 4: far}, EINVAL), ({1: 1 << 30, 5: far}, EINVAL)])
    good = [GOOD, 128, GOOD, GOOD, GOOD, None, 4, 64, 100, GOOD, 64, BF16, None]
    _refuses(L.int8_gemm, good, [({6: T, 10: far}, EINVAL)])
    good = [GOOD, 128, GOOD, 4, GOOD, GOOD, 8, 3, GOOD, GOOD, 64, 100, GOOD, 64, F32, None]
    _refuses(L.int8_grouped_gemm, good, [({6: T, 13: far}, EINVAL)])
    # one row has no distance to another
    good = [GOOD, F32, 0, 64, far, GOOD, 64, GOOD, None]
    _refuses(L.int8_quant, good, [({}, 0)])
