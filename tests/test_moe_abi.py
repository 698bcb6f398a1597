"""libfp8moe loads, exports every entry point of include/fp8moe.h, and refuses
bad arguments on the host (no GPU needed: nothing is launched)."""
import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp8moe.h")
ENTRIES = ["fp8b_moe_abi_version", "moe_sort_workspace", "moe_route", "moe_sort", "moe_route_backward", "moe_gather",
           "moe_combine", "moe_combine_backward", "int8_quant", "int8_weight_pack", "int8_gemm", "int8_grouped_gemm"]
OK, EINVAL, EALIGN, EUNSUPPORTED = 0, -1, -2, -3
GOOD, ODD, BYTE = 1 << 20, (1 << 20) + 2, (1 << 20) + 1       # never dereferenced here
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def L():
    from fp8_block_scaled_02_amd import moe
    return moe.moe_lib()


def test_header_and_exports(L, tmp_path):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = re.findall(r"^\s*[a-z_0-9]+\s+\*?\s*([a-z_0-9]+)\s*\(", text, flags=re.M)
    assert sorted(set(names)) == sorted(ENTRIES)
    out = os.popen(f"nm -D --defined-only {L._name}").read()
    assert {ln.split()[-1] for ln in out.splitlines() if " T " in ln} == set(ENTRIES)
    assert L.fp8b_moe_abi_version() == 1
    src = tmp_path / "s.c"
    src.write_text('#include "fp8moe.h"\nint main(void) { return 0; }\n')
    subprocess.check_call(["gcc", "-std=c99", "-pedantic", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
                           "-c", str(src), "-o", str(tmp_path / "s.o")])


def _refuses(f, good, cases):
    """Each case: (position: value, ..., status), against arguments that pass every check before it."""
    for over, want in cases:
        a = list(good)
        for i, v in over.items():
            a[i] = v
        assert f(*a) == want, (over, want)


def test_workspace(L):
    f = L.moe_sort_workspace
    assert f(0, 8, 2) == 0 and f(1, 8, 2) == 0 and f(32, 8, 2) == 0
    assert f(100000, 8, 2) > 0
    for bad in ((-1, 8, 2), (1 << 24, 8, 2), (4, 0, 2), (4, 1025, 2), (4, 8, 0), (4, 80, 65), ((1 << 24) - 1, 64, 17)):
        assert f(*bad) == EINVAL


def test_route(L):
    #       logits dtype ld  T   E  k  ren gates experts offs index rows ws stream
    good = [GOOD, BF16, 64, 4, 64, 8, 1, GOOD, GOOD, GOOD, GOOD, GOOD, None, None]
    _refuses(L.moe_route, good, [
        ({1: 2}, EUNSUPPORTED), ({3: -1}, EINVAL), ({3: 1 << 24}, EINVAL), ({4: 0}, EINVAL), ({4: 1025, 2: 1025}, EINVAL),
        ({5: 0}, EINVAL), ({5: 65, 4: 100, 2: 100}, EINVAL), ({4: 7, 5: 8}, EINVAL), ({2: 63}, EINVAL), ({2: 1 << 41}, EINVAL),
        ({0: None}, EINVAL), ({0: BYTE}, EALIGN), ({1: F32, 0: ODD}, EALIGN)] +
        [({i: None}, EINVAL) for i in range(7, 12)] + [({i: ODD}, EALIGN) for i in range(7, 12)] +
        [({3: 1000, 12: None}, EINVAL), ({3: 1000, 12: GOOD + 8}, EALIGN), ({3: 0, 9: None}, EINVAL)])


def test_sort(L):
    #       experts T  E  k offs index rows ws stream
    good = [GOOD, 4, 64, 8, GOOD, GOOD, GOOD, None, None]
    _refuses(L.moe_sort, good, [
        ({1: -1}, EINVAL), ({1: 1 << 24}, EINVAL), ({2: 0}, EINVAL), ({2: 1025}, EINVAL), ({3: 0}, EINVAL), ({3: 65}, EINVAL),
        ({0: None}, EINVAL), ({0: ODD}, EALIGN), ({4: None}, EINVAL), ({5: None}, EINVAL), ({6: ODD}, EALIGN),
        ({1: 1000}, EINVAL)])


def test_route_backward(L):
    #       dgates logits dtype ld gates experts T E k ren dlogits ld stream
    good = [GOOD, GOOD, F32, 64, GOOD, GOOD, 4, 64, 8, 0, GOOD, 64, None]
    _refuses(L.moe_route_backward, good, [
        ({2: 9}, EUNSUPPORTED), ({6: -1}, EINVAL), ({7: 0}, EINVAL), ({8: 65}, EINVAL), ({3: 60}, EINVAL), ({11: 60}, EINVAL),
        ({0: None}, EINVAL), ({1: None}, EINVAL), ({4: None}, EINVAL), ({5: None}, EINVAL), ({10: None}, EINVAL),
        ({0: ODD}, EALIGN), ({1: ODD}, EALIGN), ({5: BYTE}, EALIGN), ({10: ODD}, EALIGN), ({6: 0, 0: None, 10: None}, OK)])


def test_rows(L):
    #       x dtype ld T N rows k R out ld stream
    good = [GOOD, F32, 64, 4, 64, GOOD, 8, 32, GOOD, 64, None]
    sizes = [({3: -1}, EINVAL), ({3: 1 << 24}, EINVAL), ({4: 0}, EINVAL), ({4: 1 << 30, 2: 1 << 30}, EINVAL), ({6: 0}, EINVAL),
             ({6: 65}, EINVAL), ({7: -1}, EINVAL), ({7: 1 << 30}, EINVAL)]
    _refuses(L.moe_gather, good, sizes + [
        ({1: 5}, EUNSUPPORTED), ({2: 63}, EINVAL), ({9: 63}, EINVAL), ({0: None}, EINVAL), ({5: None}, EINVAL), ({8: None}, EINVAL),
        ({0: ODD}, EALIGN), ({5: ODD}, EALIGN), ({8: ODD}, EALIGN), ({3: 0, 0: None}, OK), ({7: 0, 8: None}, OK)])
    #       y dtype ld R N rows gates T k out dtype ld stream
    good = [GOOD, F32, 64, 32, 64, GOOD, GOOD, 4, 8, GOOD, BF16, 64, None]
    _refuses(L.moe_combine, good, [
        ({1: 5}, EUNSUPPORTED), ({10: 5}, EUNSUPPORTED), ({3: -1}, EINVAL), ({4: 0}, EINVAL), ({7: -1}, EINVAL), ({8: 65}, EINVAL),
        ({2: 63}, EINVAL), ({11: 63}, EINVAL), ({0: None}, EINVAL), ({5: None}, EINVAL), ({9: None}, EINVAL), ({0: ODD}, EALIGN),
        ({6: ODD}, EALIGN), ({9: BYTE}, EALIGN), ({7: 0, 9: None}, OK)])
    #       dout dtype ld y dtype ld R N rows gates T k dy ld dgates stream
    good = [GOOD, BF16, 64, GOOD, F32, 64, 32, 64, GOOD, GOOD, 4, 8, GOOD, 64, GOOD, None]
    _refuses(L.moe_combine_backward, good, [
        ({1: 5}, EUNSUPPORTED), ({4: 5}, EUNSUPPORTED), ({6: -1}, EINVAL), ({7: 0}, EINVAL), ({10: 1 << 24}, EINVAL), ({11: 0}, EINVAL),
        ({2: 63}, EINVAL), ({5: 63}, EINVAL), ({13: 63}, EINVAL), ({0: BYTE}, EALIGN), ({3: ODD}, EALIGN), ({12: ODD}, EALIGN),
        ({14: ODD}, EALIGN), ({10: 0, 14: None}, OK)] + [({i: None}, EINVAL) for i in (0, 3, 8, 9, 12, 14)])


def test_quant_and_pack(L):
    #       x dtype M K ld codes ld scales stream
    good = [GOOD, F32, 4, 64, 64, GOOD, 64, GOOD, None]
    _refuses(L.int8_quant, good, [
        ({1: 2}, EUNSUPPORTED), ({2: -1}, EINVAL), ({2: 1 << 24}, EINVAL), ({3: 0}, EINVAL), ({3: 1 << 30, 4: 1 << 30, 6: 1 << 30}, EINVAL),
        ({4: 63}, EINVAL), ({6: 63}, EINVAL), ({0: None}, EINVAL), ({5: None}, EINVAL), ({7: None}, EINVAL), ({0: ODD}, EALIGN),
        ({7: ODD}, EALIGN), ({2: 0, 0: None}, OK)])
    #       w G N K ld stride out stream
    good = [GOOD, 2, 64, 64, 64, 4096, GOOD, None]
    _refuses(L.int8_weight_pack, good, [
        ({1: 0}, EINVAL), ({2: 0}, EINVAL), ({2: (1 << 25) + 1}, EINVAL), ({3: 0}, EINVAL), ({3: 131072, 4: 131072}, EINVAL),
        ({1: 1 << 46}, EINVAL), ({1: 1 << 33}, EINVAL), ({4: 63}, EINVAL), ({5: -1}, EINVAL), ({0: None}, EINVAL), ({6: None}, EINVAL),
        ({6: GOOD + 8}, EALIGN)])


def test_products(L):
    #       a ld sa w sw bias M N K y ld dtype stream
    good = [GOOD, 128, GOOD, GOOD, GOOD, None, 4, 64, 100, GOOD, 64, BF16, None]
    _refuses(L.int8_gemm, good, [
        ({11: 2}, EUNSUPPORTED), ({6: -1}, EINVAL), ({6: 1 << 24}, EINVAL), ({7: 0}, EINVAL), ({7: (1 << 25) + 1}, EINVAL), ({8: 0}, EINVAL),
        ({8: 131072, 1: 131072}, EINVAL), ({1: 112}, EINVAL), ({1: 1 << 24}, EINVAL), ({1: 136}, EALIGN), ({10: 63}, EINVAL),
        ({0: GOOD + 8}, EALIGN), ({3: GOOD + 8}, EALIGN), ({2: ODD}, EALIGN), ({4: ODD}, EALIGN), ({5: ODD}, EALIGN), ({9: BYTE}, EALIGN),
        ({6: 0, 0: None, 9: None}, OK)] + [({i: None}, EINVAL) for i in (0, 2, 3, 4, 9)])
    #       a ld sa T index offs R E w sw N K y ld dtype stream
    good = [GOOD, 128, GOOD, 4, GOOD, GOOD, 8, 3, GOOD, GOOD, 64, 100, GOOD, 64, F32, None]
    _refuses(L.int8_grouped_gemm, good, [
        ({14: 2}, EUNSUPPORTED), ({3: 0}, EINVAL), ({3: 1 << 24}, EINVAL), ({6: -1}, EINVAL), ({6: 1 << 24}, EINVAL), ({7: 0}, EINVAL),
        ({7: 1025}, EINVAL), ({10: 0}, EINVAL), ({11: 0}, EINVAL), ({4: None}, EINVAL), ({1: 112}, EINVAL), ({1: 136}, EALIGN),
        ({13: 63}, EINVAL), ({4: ODD}, EALIGN), ({5: ODD}, EALIGN), ({12: ODD}, EALIGN), ({6: 0, 0: None, 12: None}, OK),
        ({10: 1 << 25, 11: 131071, 7: 1024, 13: 1 << 25, 1: 131072}, EINVAL)] + [({i: None}, EINVAL) for i in (0, 2, 5, 8, 9, 12)])


def test_largest_products(L):
    """Sizes whose launches or offsets would not fit are refused, whatever the rest is."""
    good = [GOOD, 128, GOOD, GOOD, GOOD, None, 4, 64, 100, GOOD, 64, BF16, None]
    _refuses(L.int8_gemm, good, [({6: 1 << 23, 7: 8193, 10: 8193}, EINVAL), ({6: 4096, 7: 1 << 25, 10: 1 << 25}, EINVAL)])
    good = [GOOD, 128, GOOD, 4, GOOD, GOOD, 8, 3, GOOD, GOOD, 64, 100, GOOD, 64, F32, None]
    _refuses(L.int8_grouped_gemm, good, [
        ({6: 1 << 23, 10: 8193, 13: 8193}, EINVAL),                       # R N
        ({7: 1024, 10: (1 << 20) + 1, 13: 1 << 21}, EINVAL),              # E N
        ({3: 1 << 23, 1: 512}, EINVAL),                                   # T ld
        ({1: 1 << 24}, EINVAL), ({1: 1 << 61, 3: 8}, EINVAL), ({1: -128}, EINVAL)])
    assert L.moe_sort_workspace(1 << 23, 8, 32) == EINVAL and L.moe_sort_workspace(1 << 23, 8, 31) > 0
