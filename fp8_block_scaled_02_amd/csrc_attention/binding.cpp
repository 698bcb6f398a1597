// binding.cpp -- the host side of attention.py's calls, as a CPython module
// (_attn_binding): checks, outputs and the workspace from torch's allocator,
// then one C call of libfp8attn.  A decode step on a few sequences is bound by
// the host, and unpacking a call's tensors in Python costs as much as its
// launch.  Host code only; compiled against torch's headers.
//
// Every function takes the stream first (an address; 0: the current device's
// default) and returns its outputs, or the negative status of the C call as an
// int.  A wrong argument raises ValueError before anything is launched.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <exception>
#include <initializer_list>
#include <numeric>
#include <sstream>
#include <string>
#include <utility>

#include "../../include/fp8attn.h"

namespace {

struct Refused {};  // a Python error is set

[[noreturn]] void refuse(const std::string& s) {
  PyErr_SetString(PyExc_ValueError, s.c_str());
  throw Refused();
}

std::string list(at::IntArrayRef s) {
  std::ostringstream o;
  o << '(';
  for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
  o << (s.size() == 1 ? ",)" : ")");
  return o.str();
}

const char* name_of(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kInt: return "torch.int32";
    default: return "torch.int64";
  }
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

void shape(const at::Tensor& t, at::IntArrayRef s, const char* name) {
  if (t.sizes() != s) refuse(std::string(name) + " must have shape " + list(s) + ", not " + list(t.sizes()));
}

// A contiguous tensor of one type and shape; its address.
void* flat(const at::Tensor& t, at::ScalarType type, std::initializer_list<int64_t> s, const char* name) {
  if (t.scalar_type() != type || !t.is_contiguous())
    refuse(std::string(name) + " must be contiguous " + name_of(type));
  shape(t, at::IntArrayRef(s.begin(), s.size()), name);
  return t.data_ptr();
}

// bf16 [tokens, heads, D] with free token and head strides; the stride of a
// dimension of one entry means nothing and is put in order.
struct Rows {
  void* p;
  int64_t t, h, T, H, D;
};
Rows rows(const at::Tensor& t, const char* name) {
  if (t.scalar_type() != at::kBFloat16 || t.dim() != 3 || (t.stride(2) != 1 && t.size(2) != 1))
    refuse(std::string(name) + " must be 3-D bf16 [tokens, heads, head_dim], head rows contiguous");
  Rows r{t.data_ptr(), t.stride(0), t.stride(1), t.size(0), t.size(1), t.size(2)};
  if (r.H <= 1) r.h = r.D;
  if (r.T <= 1) r.t = r.h * r.H;
  return r;
}

// Every tensor is on GPU number `dev`: the kernels dereference its address as
// that GPU's memory.
void on(int64_t dev, std::initializer_list<const at::Tensor*> ts) {
  if (dev < 0) refuse("every tensor must be on a GPU (found one on the host)");
  for (const at::Tensor* t : ts)
    if (t && t->get_device() != dev)
      refuse("every tensor must be on cuda:" + std::to_string(dev) + " (found one on " + t->device().str() + ")");
}

// An optional tensor: NULL for None.
const at::Tensor* maybe(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused();
  return v != 0;
}
void* address(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw Refused();
  return p;
}
const fp8b_kv_cache* cache_of(PyObject* o) { return static_cast<const fp8b_kv_cache*>(address(o)); }

PyObject* status(int64_t rc) { return PyLong_FromLongLong(rc); }

fp8b_rope rope_of(int64_t D, int64_t T, const at::Tensor* cos_sin, const at::Tensor* positions,
                  const at::Tensor* q_weight, const at::Tensor* k_weight, double eps, bool interleaved) {
  if ((cos_sin == nullptr) != (positions == nullptr)) refuse("cos_sin and positions go together");
  fp8b_rope r{};
  r.eps = (float)eps;
  r.interleaved = interleaved;
  if (cos_sin) {
    if (cos_sin->scalar_type() != at::kFloat || cos_sin->dim() != 2 || !cos_sin->is_contiguous())
      refuse("cos_sin must be contiguous float32 [max_pos, rot_dim]");
    r.max_pos = cos_sin->size(0);
    r.rot_dim = cos_sin->size(1);
    if (r.rot_dim < 16 || r.rot_dim > D || r.rot_dim % 16 != 0)
      refuse("rot_dim must be a multiple of 16 from 16 to " + std::to_string(D));
    if (r.max_pos < 1) refuse("cos_sin must hold at least one position");
    r.positions = static_cast<const int64_t*>(flat(*positions, at::kLong, {T}, "positions"));
    r.cos_sin = static_cast<const float*>(cos_sin->data_ptr());
  }
  if (q_weight) r.q_weight = flat(*q_weight, at::kBFloat16, {D}, "q_weight");
  if (k_weight) r.k_weight = flat(*k_weight, at::kBFloat16, {D}, "k_weight");
  return r;
}

// The caller's output, bf16 rows of x's shape that lie apart (tokens outside
// heads or heads outside tokens); NULL for None.
const at::Tensor* given_rows(PyObject* o, const at::Tensor& x, const char* name) {
  const at::Tensor* t = maybe(o, name);
  if (t) {
    shape(*t, x.sizes(), name);
    const Rows r = rows(*t, name);
    const bool apart = (r.h >= r.D && r.t >= (r.H - 1) * r.h + r.D) || (r.t >= r.D && r.h >= (r.T - 1) * r.t + r.D);
    if (!apart && r.T > 0 && r.H > 0) refuse(std::string(name) + ": rows overlap");
  }
  return t;
}

// The bytes of an array: rows of `len` bytes, n[0] x n[1] of them, s[0] and s[1] apart.
struct Area {
  int64_t p, n[2], s[2], len;
  bool empty() const { return n[0] < 1 || n[1] < 1 || len < 1; }
  int64_t end() const { return p + (n[0] - 1) * s[0] + (n[1] - 1) * s[1] + len; }
  int outer() const { return s[0] * (n[0] > 1) >= s[1] * (n[1] > 1) ? 0 : 1; }
};
int64_t number_of(const void* p) { return (int64_t)reinterpret_cast<uintptr_t>(p); }
Area area(const void* p, int64_t bytes) { return {number_of(p), {1, 1}, {0, 0}, bytes}; }
Area area(const at::Tensor& t) { return area(t.data_ptr(), t.numel() * (int64_t)t.element_size()); }  // contiguous

Area area(const Rows& r) { return {number_of(r.p), {r.T, r.H}, {2 * r.t, 2 * r.h}, 2 * r.D}; }

// Blocks of la and lb bytes, delta apart, each repeated at distances that g divides.
bool between(int64_t delta, int64_t g, int64_t la, int64_t lb) {
  if (g == 0) return false;
  const int64_t r = (delta % g + g) % g;
  return r >= la && r + lb <= g;
}
// Whether two arrays have no byte in common: one ends before the other begins,
// or they are slices of one allocation whose rows, or blocks of rows, take
// turns.  (Arrays that are interlaced in another way count as not apart.)
bool apart(const Area& a, const Area& b) {
  if (a.empty() || b.empty() || a.end() <= b.p || b.end() <= a.p) return true;
  int64_t all = 0, outer = 0;
  for (const Area* x : {&a, &b}) {
    for (int i = 0; i < 2; ++i)
      if (x->n[i] > 1) all = std::gcd(all, x->s[i]);
    if (x->n[x->outer()] > 1) outer = std::gcd(outer, x->s[x->outer()]);
  }
  auto block = [](const Area& x) { return x.len + (x.n[1 - x.outer()] - 1) * x.s[1 - x.outer()]; };
  return between(b.p - a.p, all, a.len, b.len) || between(b.p - a.p, outer, block(a), block(b));
}
void keep_apart(const Area& a, const Area& b, const char* x, const char* y) {
  if (!apart(a, b)) refuse(std::string(x) + " and " + y + " must lie apart");
}
void keep_apart(const Area& a, const at::Tensor* b, const char* x, const char* y) {
  if (b) keep_apart(a, area(*b), x, y);
}
// Rows given for an output and the rows it is made from: the same ones, or apart.
void same_or_apart(const Rows& a, const Rows& b, const char* x, const char* y) {
  if (a.p != b.p || a.t != b.t || a.h != b.h) keep_apart(area(a), area(b), x, y);
}
// The arrays of a cache.
struct CacheAreas {
  Area a[4];
  explicit CacheAreas(const fp8b_kv_cache* c) {
    const int64_t rows = c->heads * c->page_size;
    for (int i = 0; i < 2; ++i) {
      a[i] = {number_of(i ? c->v_codes : c->k_codes), {c->pages, 1}, {c->page_stride, 0}, rows * c->head_dim};
      a[2 + i] = {number_of(i ? c->v_scales : c->k_scales), {c->pages, 1}, {4 * c->scale_page_stride, 0}, 4 * rows};
    }
  }
};
// An output and the cache.
void off_cache(const Area& x, const char* name, const fp8b_kv_cache* c) {
  for (const Area& y : CacheAreas(c).a) keep_apart(x, y, name, "the cache");
}
// A cache to be written: the places of K and V, codes and scales.  (One that is only read may share them.)
void writable(const fp8b_kv_cache* c) {
  if (!c->k_codes) return;  // (refused by the call)
  const CacheAreas x(c);
  const char* names[4] = {"k_codes", "v_codes", "k_scales", "v_scales"};
  for (int i = 1; i < 4; ++i)
    for (int j = 0; j < i; ++j) keep_apart(x.a[j], x.a[i], names[j], names[i]);
}

// A C call with other Python threads let in: a launch waits while its queue is full.
struct Unlocked {
  PyThreadState* s = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(s); }
};
template <typename F>
int launch(F f) {
  Unlocked u;
  return f();
}

PyObject* pair(const at::Tensor& s, const at::Tensor& t) {
  PyObject *x = THPVariable_Wrap(s), *y = THPVariable_Wrap(t);
  PyObject* both = x && y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return both;
}

// (stream, q, k, cos_sin, positions, q_weight, k_weight, eps, interleaved, q_out, k_out) -> (q_out, k_out)
PyObject* norm_rope(PyObject* const* a) {
  const at::Tensor &q = tensor(a[1], "q"), &k = tensor(a[2], "k");
  const Rows qr = rows(q, "q"), kr = rows(k, "k");
  if (kr.T != qr.T || kr.D != qr.D)
    refuse("k must be [" + std::to_string(qr.T) + ", Hk, " + std::to_string(qr.D) + "]");
  const at::Tensor *cs = maybe(a[3], "cos_sin"), *pos = maybe(a[4], "positions"), *qw = maybe(a[5], "q_weight"),
                   *kw = maybe(a[6], "k_weight");
  const fp8b_rope r = rope_of(qr.D, qr.T, cs, pos, qw, kw, number(a[7]), truth(a[8]));
  const at::Tensor *gq = given_rows(a[9], q, "q_out"), *gk = given_rows(a[10], k, "k_out");
  const struct {
    const at::Tensor* t;
    const char* name;
    const Rows &own, &other;
    const char *own_name, *other_name;
  } given[2] = {{gq, "q_out", qr, kr, "q", "k"}, {gk, "k_out", kr, qr, "k", "q"}};
  for (const auto& g : given)
    if (g.t) {
      const Rows o = rows(*g.t, g.name);
      same_or_apart(o, g.own, g.name, g.own_name);
      keep_apart(area(o), area(g.other), g.name, g.other_name);
      keep_apart(area(o), cs, g.name, "cos_sin");
      keep_apart(area(o), pos, g.name, "positions");
      keep_apart(area(o), qw, g.name, "q_weight");
      keep_apart(area(o), kw, g.name, "k_weight");
      if (g.t == gq && gk) keep_apart(area(o), area(rows(*gk, "k_out")), g.name, "k_out");
    }
  on(q.get_device(), {&k, cs, pos, qw, kw, gq, gk});
  void* stream = address(a[0]);
  const at::Tensor qo = gq ? *gq : at::empty(q.sizes(), q.options());
  const at::Tensor ko = gk ? *gk : at::empty(k.sizes(), k.options());
  const Rows qor = rows(qo, "q_out"), kor = rows(ko, "k_out");
  const int rc = launch([&] {
    return fp8_qk_norm_rope(qr.p, qr.t, qr.h, kr.p, kr.t, kr.h, qr.T, qr.H, kr.H, qr.D, &r, qor.p, qor.t, qor.h, kor.p,
                            kor.t, kor.h, stream);
  });
  return rc ? status(rc) : pair(qo, ko);
}

void kv_rows(const at::Tensor& k, const at::Tensor& v, const fp8b_kv_cache* c, Rows& kr, Rows& vr) {
  kr = rows(k, "k");
  vr = rows(v, "v");
  shape(k, {kr.T, c->heads, c->head_dim}, "k");
  shape(v, k.sizes(), "v");
}

// (stream, cache, dev, k, v, slots) -> 0
PyObject* cache_write(PyObject* const* a) {
  const fp8b_kv_cache* c = cache_of(a[1]);
  const at::Tensor &k = tensor(a[3], "k"), &v = tensor(a[4], "v"), &slots = tensor(a[5], "slots");
  Rows kr, vr;
  kv_rows(k, v, c, kr, vr);
  writable(c);
  const void* s = flat(slots, at::kLong, {kr.T}, "slots");
  on(integer(a[2]), {&k, &v, &slots});
  void* stream = address(a[0]);
  return status(launch([&] {
    return fp8_kv_cache_write(kr.p, kr.t, kr.h, vr.p, vr.t, vr.h, static_cast<const int64_t*>(s), kr.T, c, stream);
  }));
}

// What a fused write takes, from (q, k, v, cos_sin, positions, slots, q_weight,
// k_weight, eps, interleaved).
struct QkvWrite {
  const at::Tensor &q, &k, &v, &slots;
  const at::Tensor *cs, *pos, *qw, *kw;
  Rows qr, kr, vr;
  fp8b_rope r;
  const int64_t* s;
  QkvWrite(const fp8b_kv_cache* c, PyObject* const* a)
      : q(tensor(a[0], "q")), k(tensor(a[1], "k")), v(tensor(a[2], "v")), slots(tensor(a[5], "slots")),
        cs(maybe(a[3], "cos_sin")), pos(maybe(a[4], "positions")), qw(maybe(a[6], "q_weight")),
        kw(maybe(a[7], "k_weight")), qr(rows(q, "q")) {
    kv_rows(k, v, c, kr, vr);
    writable(c);
    if (qr.T != kr.T || qr.D != c->head_dim)
      refuse("q must be [" + std::to_string(kr.T) + ", Hq, " + std::to_string(c->head_dim) + "]");
    r = rope_of(qr.D, qr.T, cs, pos, qw, kw, number(a[8]), truth(a[9]));
    s = static_cast<const int64_t*>(flat(slots, at::kLong, {qr.T}, "slots"));
  }
  // An output and what is read beside q.
  void keep_off(const Area& x, const char* name) const {
    keep_apart(x, area(kr), name, "k");
    keep_apart(x, area(vr), name, "v");
    keep_apart(x, cs, name, "cos_sin");
    keep_apart(x, pos, name, "positions");
    keep_apart(x, &slots, name, "slots");
    keep_apart(x, qw, name, "q_weight");
    keep_apart(x, kw, name, "k_weight");
  }
  void all_on(int64_t dev) const { on(dev, {&q, &k, &v, cs, pos, &slots, qw, kw}); }
};

// (stream, cache, dev, q, k, v, cos_sin, positions, slots, q_weight, k_weight, eps, interleaved, q_out) -> q_out
PyObject* qkv_write(PyObject* const* a) {
  const fp8b_kv_cache* c = cache_of(a[1]);
  const int64_t dev = integer(a[2]);
  const QkvWrite w(c, a + 3);
  const at::Tensor* gq = given_rows(a[13], w.q, "q_out");
  if (gq) {
    const Rows o = rows(*gq, "q_out");
    const Area x = area(o);
    same_or_apart(o, w.qr, "q_out", "q");
    w.keep_off(x, "q_out");
    off_cache(x, "q_out", c);
  }
  w.all_on(dev);
  on(dev, {gq});
  void* stream = address(a[0]);
  const at::Tensor qo = gq ? *gq : at::empty(w.q.sizes(), w.q.options());
  const Rows o = rows(qo, "q_out");
  const int rc = launch([&] {
    return fp8_qkv_cache_write(w.qr.p, w.qr.t, w.qr.h, w.kr.p, w.kr.t, w.kr.h, w.vr.p, w.vr.t, w.vr.h, w.s, w.qr.T,
                               w.qr.H, &w.r, c, o.p, o.t, o.h, stream);
  });
  return rc ? status(rc) : THPVariable_Wrap(qo);
}

struct Table {
  const int32_t* p;
  int64_t B, ld, cols;
};
Table table_of(const at::Tensor& t) {
  if (t.scalar_type() != at::kInt || t.dim() != 2 || (t.stride(1) != 1 && t.size(1) != 1))
    refuse("block_table must be 2-D int32, rows contiguous");
  const int64_t B = t.size(0), cols = t.size(1);
  return {static_cast<const int32_t*>(t.data_ptr()), B, B > 1 ? t.stride(0) : cols, cols};
}
Area area(const Table& t) { return {number_of(t.p), {t.B, 1}, {4 * t.ld, 0}, 4 * t.cols}; }

// (stream, cache, dev, block_table, offsets, rows, k_out, v_out) -> (k_out, v_out)
PyObject* cache_read(PyObject* const* a) {
  const fp8b_kv_cache* c = cache_of(a[1]);
  const int64_t dev = integer(a[2]), R = integer(a[5]);
  const at::Tensor &bt = tensor(a[3], "block_table"), &offsets = tensor(a[4], "offsets");
  const Table t = table_of(bt);
  const void* offs = flat(offsets, at::kInt, {t.B + 1}, "offsets");
  if (R < 0) refuse("rows must be 0 or more");
  const at::Tensor* given[2] = {maybe(a[6], "k_out"), maybe(a[7], "v_out")};
  const char* names[2] = {"k_out", "v_out"};
  for (int i = 0; i < 2; ++i)
    if (given[i]) flat(*given[i], at::kBFloat16, {R, c->heads, c->head_dim}, names[i]);
  for (int i = 0; i < 2; ++i)
    if (given[i]) {
      const Area o = area(*given[i]);
      if (i == 0 && given[1]) keep_apart(o, area(*given[1]), names[0], names[1]);
      keep_apart(o, area(t), names[i], "block_table");
      keep_apart(o, area(offsets), names[i], "offsets");
      off_cache(o, names[i], c);
    }
  on(dev, {&bt, &offsets, given[0], given[1]});
  void* stream = address(a[0]);
  at::Tensor out[2];
  for (int i = 0; i < 2; ++i)
    out[i] = given[i] ? *given[i] : at::empty({R, c->heads, c->head_dim}, bt.options().dtype(at::kBFloat16));
  void *kp = out[0].data_ptr(), *vp = out[1].data_ptr();
  const int rc = launch([&] {
    return fp8_kv_cache_read(c, t.p, t.ld, t.cols, static_cast<const int32_t*>(offs), t.B, R, kp, vp, stream);
  });
  return rc ? status(rc) : pair(out[0], out[1]);
}

// What an attention takes beside its queries r, from (block_table, context_lens,
// scale, window, fp32) and max_context.
struct Attention {
  const at::Tensor &bt, &lens;
  Table t;
  const int32_t* lp;
  double scale;
  int64_t window, most;
  at::ScalarType type;
  Attention(const fp8b_kv_cache* c, const Rows& r, PyObject* const* a, PyObject* max_context)
      : bt(tensor(a[0], "block_table")), lens(tensor(a[1], "context_lens")) {
    constexpr int64_t kMaxContext = (int64_t)1 << 30;
    if (r.D != c->head_dim) refuse("q must be [B, Hq, " + std::to_string(c->head_dim) + "]");
    if (r.H < 1 || r.H % c->heads != 0)
      refuse("query heads must be a multiple of the cache's " + std::to_string(c->heads));
    t = table_of(bt);
    if (t.B != r.T) refuse("block_table must have " + std::to_string(r.T) + " rows");
    lp = static_cast<const int32_t*>(flat(lens, at::kInt, {r.T}, "context_lens"));
    scale = a[2] == Py_None ? 1.0 / std::sqrt((double)r.D) : number(a[2]);
    window = integer(a[3]);
    type = truth(a[4]) ? at::kFloat : at::kBFloat16;
    most = max_context == Py_None ? std::min(t.cols * c->page_size, kMaxContext) : integer(max_context);
    if (most < 0 || most > kMaxContext) refuse("max_context must be from 0 to " + std::to_string(kMaxContext));
    if (window < 0) refuse("window must be 0 or a number of tokens");
  }
  int dtype() const { return type == at::kFloat ? FP8B_OUT_F32 : FP8B_OUT_BF16; }
};
// Outputs given by the caller, from (out, lse): their checks but the device.
struct Given {
  const at::Tensor *out, *lse;
  float* lse_p;
  Given(const fp8b_kv_cache* c, const Rows& r, const Attention& x, PyObject* const* a)
      : out(maybe(a[0], "out")), lse(maybe(a[1], "lse")) {
    if (out) flat(*out, x.type, {r.T, r.H, r.D}, "out");
    lse_p = lse ? static_cast<float*>(flat(*lse, at::kFloat, {r.T, r.H}, "lse")) : nullptr;
    const std::pair<const at::Tensor*, const char*> outs[2] = {{out, "out"}, {lse, "lse"}};
    for (const auto& [t, name] : outs)
      if (t) {
        const Area o = area(*t);
        if (t == out) keep_apart(o, lse, name, "lse");
        keep_apart(o, area(r), name, "q");
        keep_apart(o, area(x.t), name, "block_table");
        keep_apart(o, &x.lens, name, "context_lens");
        off_cache(o, name, c);
      }
  }
};
// Of `bytes` on the current stream, like the call that uses it.
at::Tensor workspace(int64_t bytes, const at::Tensor& q) {
  return bytes > 0 ? at::empty({bytes}, q.options().dtype(at::kByte)) : at::Tensor();
}

// (stream, cache, dev, q, block_table, context_lens, scale, window, fp32, out, lse, max_context) -> out
PyObject* attention(PyObject* const* a) {
  const fp8b_kv_cache* c = cache_of(a[1]);
  const int64_t dev = integer(a[2]);
  const at::Tensor& q = tensor(a[3], "q");
  const Rows r = rows(q, "q");
  const Attention x(c, r, a + 4, a[11]);
  const Given given(c, r, x, a + 9);
  on(dev, {&q, &x.bt, &x.lens, given.out, given.lse});
  const int64_t bytes = fp8_paged_attention_workspace(c, r.T, r.H, x.t.cols, x.most, x.window);
  if (bytes < 0) return status(bytes);
  void* stream = address(a[0]);
  const at::Tensor out = given.out ? *given.out : at::empty({r.T, r.H, r.D}, q.options().dtype(x.type));
  const at::Tensor ws = workspace(bytes, q);
  void *outp = out.data_ptr(), *wsp = bytes > 0 ? ws.data_ptr() : nullptr;
  const int rc = launch([&] {
    return fp8_paged_attention(r.p, r.t, r.h, c, x.t.p, x.t.ld, x.t.cols, x.lp, r.T, r.H, x.most, x.window,
                               (float)x.scale, outp, x.dtype(), given.lse_p, wsp, stream);
  });
  return rc ? status(rc) : THPVariable_Wrap(out);
}

// (stream, cache, dev, q, k, v, cos_sin, positions, slots, q_weight, k_weight, eps, interleaved, block_table,
// context_lens, scale, window, fp32, max_context, out, lse) -> out
PyObject* step(PyObject* const* a) {
  const fp8b_kv_cache* c = cache_of(a[1]);
  const int64_t dev = integer(a[2]);
  const QkvWrite w(c, a + 3);
  const Rows& r = w.qr;
  const Attention x(c, r, a + 13, a[18]);
  const Given given(c, r, x, a + 19);
  for (const auto& [t, name] : {std::pair{given.out, "out"}, std::pair{given.lse, "lse"}})
    if (t) w.keep_off(area(*t), name);
  w.all_on(dev);
  on(dev, {&x.bt, &x.lens, given.out, given.lse});
  const int64_t bytes = fp8_paged_attention_workspace(c, r.T, r.H, x.t.cols, x.most, x.window);
  if (bytes < 0) return status(bytes);
  void* stream = address(a[0]);
  const at::Tensor qo = at::empty({r.T, r.H, r.D}, w.q.options());
  const at::Tensor out = given.out ? *given.out : at::empty({r.T, r.H, r.D}, w.q.options().dtype(x.type));
  const at::Tensor ws = workspace(bytes, w.q);
  void *qop = qo.data_ptr(), *outp = out.data_ptr(), *wsp = bytes > 0 ? ws.data_ptr() : nullptr;
  const int rc = launch([&] {
    return fp8_attention_step(r.p, r.t, r.h, w.kr.p, w.kr.t, w.kr.h, w.vr.p, w.vr.t, w.vr.h, w.s, r.T, r.H, &w.r, c,
                              x.t.p, x.t.ld, x.t.cols, x.lp, x.most, x.window, (float)x.scale, qop, r.H * r.D, r.D,
                              outp, x.dtype(), given.lse_p, wsp, stream);
  });
  return rc ? status(rc) : THPVariable_Wrap(out);
}

// No C++ exception crosses into Python.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, %zd given", N, n);
    return nullptr;
  }
  try {
    return F(a);
  } catch (const Refused&) {
  } catch (...) {
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<norm_rope, 11>("norm_rope"),   method<cache_write, 6>("cache_write"),
                         method<qkv_write, 14>("qkv_write"),   method<cache_read, 8>("cache_read"),
                         method<attention, 12>("attention"),   method<step, 21>("step"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attn_binding", "Host side of attention.py's calls.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn_binding(void) { return PyModule_Create(&module); }
