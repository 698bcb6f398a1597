"""libfp8attn loads, exports every entry point of include/fp8attn.h, and
refuses bad arguments on the host (no GPU needed: nothing is launched)."""
import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp8attn.h")

ENTRIES = ["fp8b_attn_abi_version", "fp8_qk_norm_rope", "fp8_kv_cache_write", "fp8_qkv_cache_write",
           "fp8_kv_cache_read", "fp8_paged_attention_workspace", "fp8_paged_attention", "fp8_attention_step"]
OK, EINVAL, EALIGN, EUNSUPPORTED = 0, -1, -2, -3
GOOD, ODD = 1 << 20, (1 << 20) + 2       # never dereferenced here


@pytest.fixture(scope="module")
def M():
    from fp8_block_scaled_02_amd import attention
    attention.attn_lib()
    return attention


@pytest.fixture(scope="module")
def L(M):
    return M.attn_lib()


def test_header_and_exports(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = re.findall(r"^\s*[a-z_0-9]+\s*\*?\s*([a-z_0-9]+)\s*\(", text, flags=re.M)
    assert sorted(set(names)) == sorted(ENTRIES)
    out = os.popen(f"nm -D --defined-only {L._name}").read()
    assert {ln.split()[-1] for ln in out.splitlines() if " T " in ln} == set(ENTRIES)
    assert L.fp8b_attn_abi_version() == 1


def test_structs_match_the_header(M, tmp_path):
    """Plain C99, and the binding's structs laid out as the compiler's."""
    lines = []
    for name, cls in (("fp8b_kv_cache", M._CacheStruct), ("fp8b_rope", M._RopeStruct)):
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        lines += [f'printf("%zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    src = tmp_path / "s.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"fp8attn.h\"\nint main(void){" +
                   "".join(lines) + "return 0;}")
    exe = str(tmp_path / "s")
    subprocess.check_call(["gcc", "-std=c99", "-pedantic", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
                           str(src), "-o", exe])
    got = [int(x) for x in subprocess.check_output([exe]).split()]
    want = []
    for cls in (M._CacheStruct, M._RopeStruct):
        want += [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f, _ in cls._fields_]
    assert got == want


def _cache(M, **over):
    c = dict(k_codes=GOOD, v_codes=GOOD, k_scales=GOOD, v_scales=GOOD, page_stride=8 * 16 * 128,
             scale_page_stride=128, pages=10, page_size=16, heads=8, head_dim=128, fmt=1, reserved=0)
    c.update(over)
    return M._CacheStruct(**c)


BAD_CACHES = [
    (dict(fmt=2), EUNSUPPORTED), (dict(pages=0), EINVAL), (dict(pages=1 << 31), EINVAL), (dict(page_size=8), EINVAL),
    (dict(page_size=48), EINVAL), (dict(page_size=8192, page_stride=1 << 30, scale_page_stride=1 << 20), EINVAL),
    (dict(heads=0), EINVAL), (dict(heads=1025), EINVAL), (dict(head_dim=24), EINVAL), (dict(head_dim=272), EINVAL),
    (dict(head_dim=0), EINVAL), (dict(page_stride=8 * 16 * 128 - 16), EINVAL),
    (dict(page_stride=8 * 16 * 128 + 8), EALIGN), (dict(scale_page_stride=124), EINVAL),
    (dict(scale_page_stride=130), EALIGN), (dict(page_stride=1 << 40), EINVAL),
]
BAD_POINTERS = [(dict(k_codes=None), EINVAL), (dict(v_scales=None), EINVAL), (dict(v_codes=ODD), EALIGN),
                (dict(k_scales=GOOD + 4), EALIGN)]


def _with(args, **over):
    a = dict(args)
    a.update(over)
    return list(a.values())


def _byref(s):
    return None if s is None else ctypes.addressof(s)


def test_norm_rope_refusals(M, L):
    f = L.fp8_qk_norm_rope
    rope = M._RopeStruct(GOOD, GOOD, GOOD, GOOD, 4096, 128, 1e-6, 0)
    args = dict(q=GOOD, q_t=1024, q_h=128, k=GOOD, k_t=256, k_h=128, T=4, Hq=8, Hk=2, D=128, rope=_byref(rope),
                qo=GOOD, qo_t=1024, qo_h=128, ko=GOOD, ko_t=256, ko_h=128, s=None)
    for over, rc in [(dict(T=0), OK), (dict(T=-1), EINVAL), (dict(T=1 << 24), EINVAL), (dict(Hq=0, Hk=0), EINVAL),
                     (dict(Hq=-1), EINVAL), (dict(Hk=65537), EINVAL), (dict(D=8), EINVAL), (dict(D=100), EINVAL),
                     (dict(D=512), EINVAL), (dict(rope=None), EINVAL), (dict(q=None), EINVAL), (dict(k=ODD), EALIGN),
                     (dict(q_t=1020), EALIGN), (dict(k_h=-8), EINVAL),
                     (dict(q_h=1 << 30), EINVAL), (dict(k_t=1 << 41), EINVAL), (dict(qo=None), EINVAL),
                     (dict(ko=GOOD + 8), EALIGN), (dict(ko_t=12), EALIGN)]:
        assert f(*_with(args, **over)) == rc, over
    for over, rc in [(dict(rot_dim=8), EINVAL), (dict(rot_dim=144), EINVAL), (dict(rot_dim=-16), EINVAL),
                     (dict(cos_sin=None), EINVAL), (dict(positions=None), EINVAL), (dict(max_pos=0), EINVAL),
                     (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(eps=float("inf")), EINVAL),
                     (dict(q_weight=ODD), EALIGN), (dict(cos_sin=GOOD + 4), EALIGN), (dict(positions=GOOD + 4), EALIGN)]:
        bad = M._RopeStruct.from_buffer_copy(rope)
        for k, v in over.items():
            setattr(bad, k, v)
        assert f(*_with(args, rope=_byref(bad))) == rc, over


def test_cache_write_refusals(M, L):
    good = _cache(M)
    args = dict(k=GOOD, k_t=1024, k_h=128, v=GOOD, v_t=1024, v_h=128, slots=GOOD, T=4, cache=_byref(good), s=None)
    f = L.fp8_kv_cache_write
    for over, rc in [(dict(T=0), OK), (dict(T=-1), EINVAL), (dict(T=1 << 24), EINVAL), (dict(cache=None), EINVAL),
                     (dict(k=None), EINVAL), (dict(v=ODD), EALIGN), (dict(v_h=4), EALIGN), (dict(slots=None), EINVAL),
                     (dict(slots=GOOD + 4), EALIGN)]:
        assert f(*_with(args, **over)) == rc, over
    for over, rc in BAD_CACHES + BAD_POINTERS:
        bad = _cache(M, **over)
        assert f(*_with(args, cache=_byref(bad))) == rc, over


def test_qkv_write_refusals(M, L):
    good = _cache(M)
    rope = M._RopeStruct(None, None, GOOD, GOOD, 4096, 64, 1e-6, 0)
    args = dict(q=GOOD, q_t=4096, q_h=128, k=GOOD, k_t=1024, k_h=128, v=GOOD, v_t=1024, v_h=128, slots=GOOD, T=4,
                Hq=32, rope=_byref(rope), cache=_byref(good), qo=GOOD, qo_t=4096, qo_h=128, s=None)
    f = L.fp8_qkv_cache_write
    for over, rc in [(dict(T=0), OK), (dict(T=-1), EINVAL), (dict(Hq=0), EINVAL), (dict(Hq=65537), EINVAL),
                     (dict(rope=None), EINVAL), (dict(cache=None), EINVAL), (dict(q=None), EINVAL),
                     (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(qo=None), EINVAL), (dict(qo=ODD), EALIGN),
                     (dict(slots=None), EINVAL)]:
        assert f(*_with(args, **over)) == rc, over
    for over, rc in BAD_CACHES + BAD_POINTERS:
        bad = _cache(M, **over)
        assert f(*_with(args, cache=_byref(bad))) == rc, over
    small = _cache(M, head_dim=48)
    assert f(*_with(args, cache=_byref(small))) == EINVAL       # rotates 64 of 48


def test_cache_read_refusals(M, L):
    good = _cache(M)
    args = dict(cache=_byref(good), table=GOOD, ld=7, cols=7, offsets=GOOD, B=3, R=100, k=GOOD, v=GOOD, s=None)
    f = L.fp8_kv_cache_read
    for over, rc in [(dict(R=0), OK), (dict(R=-1), EINVAL), (dict(R=1 << 24), EINVAL), (dict(B=0), EINVAL),
                     (dict(cols=0), EINVAL), (dict(ld=6), EINVAL), (dict(table=None), EINVAL), (dict(table=ODD), EALIGN),
                     (dict(offsets=None), EINVAL), (dict(k=None), EINVAL), (dict(v=GOOD + 8), EALIGN),
                     (dict(cache=None), EINVAL)]:
        assert f(*_with(args, **over)) == rc, over
    for over, rc in BAD_CACHES + BAD_POINTERS:
        bad = _cache(M, **over)
        assert f(*_with(args, cache=_byref(bad))) == rc, over


def test_attention_refusals(M, L):
    good = _cache(M)
    args = dict(q=GOOD, q_b=4096, q_h=128, cache=_byref(good), table=GOOD, ld=1000, cols=1000, lens=GOOD, B=3, Hq=32,
                most=16000, window=0, scale=0.1, out=GOOD, dtype=1, lse=None, ws=GOOD, s=None)
    f = L.fp8_paged_attention
    sizes = [(dict(B=-1), EINVAL), (dict(Hq=0), EINVAL), (dict(Hq=30), EINVAL), (dict(Hq=65544), EINVAL),
             (dict(cols=0), EINVAL), (dict(most=-1), EINVAL), (dict(most=(1 << 30) + 1), EINVAL),
             (dict(window=-1), EINVAL), (dict(cache=None), EINVAL), (dict(B=1 << 19), EINVAL),
             (dict(B=1 << 16, cols=1 << 20, ld=1 << 20, most=1 << 24), EINVAL)]
    for over, rc in sizes + [(dict(B=0), OK), (dict(dtype=2), EUNSUPPORTED), (dict(ld=999), EINVAL),
                             (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL),
                             (dict(q=None), EINVAL), (dict(q=ODD), EALIGN), (dict(q_b=4), EALIGN),
                             (dict(table=None), EINVAL), (dict(lens=None), EINVAL), (dict(lens=ODD), EALIGN),
                             (dict(out=None), EINVAL), (dict(out=GOOD + 4), EALIGN), (dict(lse=ODD), EALIGN),
                             (dict(ws=None), EINVAL), (dict(ws=GOOD + 8), EALIGN)]:
        assert f(*_with(args, **over)) == rc, over
    w = L.fp8_paged_attention_workspace
    keys = ("cache", "B", "Hq", "cols", "most", "window")
    base = {k: args[k] for k in keys}
    for over, rc in sizes:
        over = {k: v for k, v in over.items() if k in keys}
        assert w(*_with(base, **over)) == rc, over
    for over, rc in BAD_CACHES:
        bad = _cache(M, **over)
        assert f(*_with(args, cache=_byref(bad))) == rc, over
        assert w(*_with(base, cache=_byref(bad))) == rc, over
    for over, rc in BAD_POINTERS:
        bad = _cache(M, **over)
        assert f(*_with(args, cache=_byref(bad))) == rc, over


def test_step_refusals(M, L):
    good = _cache(M)
    rope = M._RopeStruct(GOOD, GOOD, GOOD, GOOD, 100, 64, 1e-6, 0)
    args = dict(q=GOOD, q_b=4096, q_h=128, k=GOOD, k_b=1024, k_h=128, v=GOOD, v_b=1024, v_h=128, slots=GOOD, B=3, Hq=32,
                rope=_byref(rope), cache=_byref(good), table=GOOD, ld=1000, cols=1000, lens=GOOD, most=16000, window=0,
                scale=0.1, q_out=GOOD, qo_b=4096, qo_h=128, out=GOOD, dtype=1, lse=None, ws=GOOD, s=None)
    f = L.fp8_attention_step
    bad_rope = M._RopeStruct(GOOD, GOOD, GOOD, GOOD, 100, 136, 1e-6, 0)
    for over, rc in [(dict(B=0), OK), (dict(B=-1), EINVAL), (dict(B=1 << 19), EINVAL), (dict(Hq=30), EINVAL),
                     (dict(cols=0), EINVAL), (dict(ld=999), EINVAL), (dict(most=-1), EINVAL), (dict(window=-1), EINVAL),
                     (dict(scale=float("nan")), EINVAL), (dict(dtype=2), EUNSUPPORTED), (dict(cache=None), EINVAL),
                     (dict(rope=None), EINVAL), (dict(rope=_byref(bad_rope)), EINVAL),
                     (dict(q=None), EINVAL), (dict(k=ODD), EALIGN), (dict(v_h=4), EALIGN), (dict(slots=None), EINVAL),
                     (dict(slots=ODD), EALIGN), (dict(q_out=None), EINVAL), (dict(qo_b=-8), EINVAL),
                     (dict(table=None), EINVAL), (dict(lens=None), EINVAL), (dict(out=None), EINVAL),
                     (dict(out=GOOD + 4), EALIGN), (dict(lse=ODD), EALIGN), (dict(ws=None), EINVAL),
                     (dict(ws=GOOD + 8), EALIGN)]:
        assert f(*_with(args, **over)) == rc, over
    for over, rc in BAD_CACHES + BAD_POINTERS:
        bad = _cache(M, **over)
        assert f(*_with(args, cache=_byref(bad))) == rc, over


def test_workspace_depends_on_what_is_seen(M, L):
    w = L.fp8_paged_attention_workspace
    ref = _byref(c := _cache(M))
    assert c is not None
    assert w(ref, 3, 32, 1000, 64, 0) == 0                       # short contexts are not split
    assert w(ref, 3, 32, 1000, 16000, 8) == 0                    # nor short windows
    assert w(ref, 0, 32, 1000, 16000, 0) == 0
    long = w(ref, 3, 32, 1000, 16000, 0)
    assert long > 0 and long % 4 == 0
    assert w(ref, 300, 32, 1000, 16000, 0) == w(ref, 3000, 32, 1000, 16000, 0)   # bounded
