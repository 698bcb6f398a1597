// binding.cpp -- the host side of moe.py's calls, as a CPython module
// (_moe_binding): checks, outputs and workspaces from torch's allocator, then
// the C calls of libfp8moe.  The calls of a decode step are bound by the host,
// and unpacking their tensors in Python costs as much as a launch.  Host code
// only; compiled against torch's headers.
//
// Every function takes the stream first (an address; 0: the current device's
// default) and returns its outputs, or the negative status of a C call as an
// int.  A wrong argument raises ValueError before anything is launched.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/core/TensorImpl.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <exception>
#include <initializer_list>
#include <sstream>
#include <string>
#include <utility>
#include <vector>

#include "../../include/fp8moe.h"

namespace {

using at::Tensor;

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
    case at::kBFloat16: return "bfloat16";
    case at::kFloat: return "float32";
    case at::kInt: return "int32";
    default: return "int8";
  }
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
const Tensor* maybe(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }

// No call records a gradient, so none takes a tensor that is to have one: it
// would be lost without a word.
void plain(const Tensor& t, const char* name) {
  if (t.requires_grad() && c10::GradMode::is_enabled())
    refuse(std::string(name) + " requires a gradient, which is not recorded here: call this under torch.no_grad() or in "
           "a torch.autograd.Function, and the backward calls for the gradient");
}

void shape(const Tensor& t, at::IntArrayRef s, const char* name) {
  if (t.sizes() != s) refuse(std::string(name) + " must have shape " + list(s) + ", not " + list(t.sizes()));
}
void shape(const Tensor& t, std::initializer_list<int64_t> s, const char* name) {
  shape(t, at::IntArrayRef(s.begin(), s.size()), name);
}

// A contiguous tensor of one type and shape.
template <typename T>
T* flat(const Tensor& t, at::ScalarType type, std::initializer_list<int64_t> s, const char* name) {
  if (t.scalar_type() != type || !t.is_contiguous()) refuse(std::string(name) + " must be contiguous " + name_of(type));
  shape(t, s, name);
  plain(t, name);
  return static_cast<T*>(t.data_ptr());
}

// A 2-D tensor whose rows are contiguous and lie apart.  The stride of a
// dimension of one entry means nothing: it is put in order.
struct Mat {
  void* p;
  int64_t rows, cols, ld;
  int64_t item;
  int type;  // fp8b_out_dtype
};
Mat mat(const Tensor& t, const char* name) {
  if (t.dim() != 2 || (t.stride(1) != 1 && t.size(1) > 1)) refuse(std::string(name) + " must be 2-D, rows contiguous");
  Mat m{t.data_ptr(), t.size(0), t.size(1), t.stride(0), (int64_t)t.element_size(),
        t.scalar_type() == at::kBFloat16 ? FP8B_OUT_BF16 : FP8B_OUT_F32};
  if (m.rows <= 1) m.ld = m.cols;
  if (m.ld < m.cols) refuse(std::string(name) + ": rows overlap");
  return m;
}
Mat real(const Tensor& t, const char* name) {
  if (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kFloat)
    refuse(std::string(name) + " must be bfloat16 or float32");
  plain(t, name);
  return mat(t, name);
}
Mat real(const Tensor& t, at::ScalarType type, std::initializer_list<int64_t> s, const char* name) {
  if (t.scalar_type() != type) refuse(std::string(name) + " must be " + name_of(type));
  shape(t, s, name);
  plain(t, name);
  return mat(t, name);
}

// Every tensor is on GPU number `dev`: the kernels dereference its address as
// that GPU's memory.
void on(int64_t dev, std::initializer_list<const Tensor*> ts) {
  if (dev < 0) refuse("every tensor must be on a GPU (found one on the host)");
  for (const Tensor* t : ts)
    if (t && t->get_device() != dev)
      refuse("every tensor must be on cuda:" + std::to_string(dev) + " (found one on " + t->device().str() + ")");
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
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
at::ScalarType out_type(PyObject* fp32) { return truth(fp32) ? at::kFloat : at::kBFloat16; }
int type_of(at::ScalarType t) { return t == at::kFloat ? FP8B_OUT_F32 : FP8B_OUT_BF16; }

// The bytes of an array: n rows of `len` bytes, `s` apart.
struct Area {
  int64_t p, n, s, len;
  int64_t end() const { return p + (n - 1) * s + len; }
};
int64_t number_of(const void* p) { return (int64_t)reinterpret_cast<uintptr_t>(p); }
Area area(const Mat& m) { return {number_of(m.p), m.rows, m.ld * m.item, m.cols * m.item}; }
Area area(const Tensor& t) { return {number_of(t.data_ptr()), 1, 0, t.numel() * (int64_t)t.element_size()}; }  // contiguous
// Whether two arrays have no byte in common: one ends before the other begins,
// or they are columns of one allocation, rows equally far apart.
bool apart(const Area& a, const Area& b) {
  if (a.n < 1 || b.n < 1 || a.len < 1 || b.len < 1 || a.end() <= b.p || b.end() <= a.p) return true;
  const int64_t s = a.n > 1 ? a.s : b.s;
  if (s < 1 || (a.n > 1 && b.n > 1 && a.s != b.s)) return false;
  const int64_t d = ((b.p - a.p) % s + s) % s;
  return d >= a.len && d + b.len <= s;
}
void keep_apart(const Area& a, const char* x, std::initializer_list<std::pair<Area, const char*>> others) {
  for (const auto& [b, y] : others)
    if (!apart(a, b)) refuse(std::string(x) + " and " + y + " must lie apart");
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
PyObject* status(int64_t rc) { return PyLong_FromLongLong(rc); }

PyObject* tuple(std::initializer_list<Tensor> ts) {
  PyObject* all = PyTuple_New((Py_ssize_t)ts.size());
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) {
    PyObject* o = all ? THPVariable_Wrap(t) : nullptr;
    if (!o) {
      Py_XDECREF(all);
      return nullptr;
    }
    PyTuple_SET_ITEM(all, i++, o);
  }
  return all;
}

Tensor empty(at::IntArrayRef s, at::ScalarType type, const Tensor& like) {
  return at::empty(s, like.options().dtype(type));
}
int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// A call's outputs.  Small ones share one allocation, each from a 128-byte line
// on: a tensor from the allocator costs the host 1 us, one of these a tenth (a
// decode step's router, five tensors: 8.5 -> 5.9 us of the host).  Larger ones
// have their own, since any part keeps the whole alive.
struct Block {
  static constexpr int64_t kShared = (int64_t)1 << 20;
  const Tensor& like;
  Tensor all;
  int64_t at = 0;
  Block(int64_t bytes, const Tensor& like_) : like(like_) {
    if (bytes > 0 && bytes <= kShared) all = empty({bytes}, at::kByte, like);
  }
  static int64_t room(int64_t bytes) { return up(bytes, 128); }
  // A vector, or rows `ld` elements apart (0: no gaps).
  Tensor take(at::ScalarType type, at::IntArrayRef sizes, int64_t ld = 0) {
    const bool gaps = ld && ld != sizes[1];
    if (!all.defined()) return gaps ? empty({sizes[0], ld}, type, like).narrow(1, 0, sizes[1]) : empty(sizes, type, like);
    const int64_t item = type == at::kChar ? 1 : 4, n = sizes.size() == 1 ? sizes[0] : sizes[0] * (ld ? ld : sizes[1]);
    Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(),
                                                        c10::scalarTypeToTypeMeta(type));
    c10::TensorImpl* impl = t.unsafeGetTensorImpl();
    impl->set_storage_offset(at / item);
    if (gaps)
      impl->set_sizes_and_strides(sizes, {ld, 1});
    else
      impl->set_sizes_contiguous(sizes);
    at += room(n * item);
    return t;
  }
};

template <typename T>
T* ptr(const Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

// ---- the plan ---------------------------------------------------------------

struct Plan {
  Tensor gates, experts, offsets, row_index, token_rows;
};

// The router's call; 0 or its status.
struct Router {
  Mat l;
  int64_t k, ws_bytes;
  Router(const Tensor& logits, int64_t k_) : l(real(logits, "logits")), k(k_) {
    if (l.cols < 1 || l.cols > 1024) refuse("logits must be [T, E] with 1 to 1024 experts");
    if (k < 1 || k > 64 || k > l.cols) refuse("k must be from 1 to 64, and no more than there are experts");
    ws_bytes = moe_sort_workspace(l.rows, l.cols, k);
    if (ws_bytes < 0) refuse("too many tokens: T < 2^24 and T * k < 2^28");
  }
  int run(const Tensor& logits, bool renormalize, void* stream, Plan& p) const {
    const int64_t T = l.rows;
    Block b(4 * Block::room(4 * T * k) + Block::room(4 * (l.cols + 1)), logits);
    p.gates = b.take(at::kFloat, {T, k});
    p.experts = b.take(at::kInt, {T, k});
    p.offsets = b.take(at::kInt, {l.cols + 1});
    p.row_index = b.take(at::kInt, {T * k});
    p.token_rows = b.take(at::kInt, {T, k});
    const Tensor ws = ws_bytes ? empty({ws_bytes}, at::kByte, logits) : Tensor();
    void* wsp = ws_bytes ? ws.data_ptr() : nullptr;
    return launch([&] {
      return moe_route(l.p, l.type, l.ld, T, l.cols, k, renormalize, ptr<float>(p.gates), ptr<int32_t>(p.experts),
                       ptr<int32_t>(p.offsets), ptr<int32_t>(p.row_index), ptr<int32_t>(p.token_rows), wsp, stream);
    });
  }
};

// (stream, logits, k, renormalize) -> (gates, experts, expert_offsets, row_index, token_rows)
PyObject* route(PyObject* const* a) {
  const Tensor& logits = tensor(a[1], "logits");
  const Router r(logits, integer(a[2]));
  const bool renormalize = truth(a[3]);
  on(logits.get_device(), {});
  Plan p;
  const int rc = r.run(logits, renormalize, address(a[0]), p);
  return rc ? status(rc) : tuple({p.gates, p.experts, p.offsets, p.row_index, p.token_rows});
}

// int32 [T, k]
struct Slots {
  int32_t* p;
  int64_t T, k;
};
Slots slots(const Tensor& t, const char* name) {
  if (t.scalar_type() != at::kInt || t.dim() != 2 || !t.is_contiguous())
    refuse(std::string(name) + " must be contiguous int32 [T, k]");
  if (t.size(1) < 1 || t.size(1) > 64) refuse(std::string(name) + " must have 1 to 64 slots a token");
  return {static_cast<int32_t*>(t.data_ptr()), t.size(0), t.size(1)};
}

// (stream, experts, E) -> (expert_offsets, row_index, token_rows)
PyObject* sort(PyObject* const* a) {
  const Tensor& experts = tensor(a[1], "experts");
  const Slots s = slots(experts, "experts");
  const int64_t E = integer(a[2]);
  if (E < 1 || E > 1024) refuse("there must be 1 to 1024 experts");
  const int64_t bytes = moe_sort_workspace(s.T, E, s.k);
  if (bytes < 0) refuse("too many tokens: T < 2^24 and T * k < 2^28");
  on(experts.get_device(), {});
  void* stream = address(a[0]);
  Block b(Block::room(4 * (E + 1)) + 2 * Block::room(4 * s.T * s.k), experts);
  const Tensor offsets = b.take(at::kInt, {E + 1}), row_index = b.take(at::kInt, {s.T * s.k});
  const Tensor token_rows = b.take(at::kInt, {s.T, s.k});
  const Tensor ws = bytes ? empty({bytes}, at::kByte, experts) : Tensor();
  void* wsp = bytes ? ws.data_ptr() : nullptr;
  const int rc = launch([&] {
    return moe_sort(s.p, s.T, E, s.k, ptr<int32_t>(offsets), ptr<int32_t>(row_index), ptr<int32_t>(token_rows), wsp,
                    stream);
  });
  return rc ? status(rc) : tuple({offsets, row_index, token_rows});
}

// (stream, dgates, logits, gates, experts, renormalize, out) -> dlogits
PyObject* route_backward(PyObject* const* a) {
  const Tensor &dgates = tensor(a[1], "dgates"), &logits = tensor(a[2], "logits"), &gates = tensor(a[3], "gates"),
               &experts = tensor(a[4], "experts");
  const Mat l = real(logits, "logits");
  const Slots s = slots(experts, "experts");
  if (l.cols < 1 || l.cols > 1024) refuse("logits must be [T, E] with 1 to 1024 experts");
  if (s.T != l.rows) refuse("experts must have " + std::to_string(l.rows) + " rows");
  const float* dg = flat<float>(dgates, at::kFloat, {s.T, s.k}, "dgates");
  const float* g = flat<float>(gates, at::kFloat, {s.T, s.k}, "gates");
  const bool renormalize = truth(a[5]);
  const Tensor* given = maybe(a[6], "out");
  if (given) {
    const Mat o = real(*given, logits.scalar_type(), {l.rows, l.cols}, "out");
    keep_apart(area(o), "out",
               {{area(dgates), "dgates"}, {area(l), "logits"}, {area(gates), "gates"}, {area(experts), "experts"}});
  }
  on(logits.get_device(), {&dgates, &gates, &experts, given});
  void* stream = address(a[0]);
  const Tensor out = given ? *given : empty({l.rows, l.cols}, logits.scalar_type(), logits);
  const Mat o = mat(out, "out");
  const int rc = launch([&] {
    return moe_route_backward(dg, l.p, l.type, l.ld, g, s.p, s.T, l.cols, s.k, renormalize, o.p, o.ld, stream);
  });
  return rc ? status(rc) : THPVariable_Wrap(out);
}

// ---- rows -------------------------------------------------------------------

// (stream, x, token_rows, rows or None, out) -> rows
PyObject* gather(PyObject* const* a) {
  const Tensor &x = tensor(a[1], "x"), &tr = tensor(a[2], "token_rows");
  const Mat m = real(x, "x");
  const Slots s = slots(tr, "token_rows");
  if (m.cols < 1) refuse("x must have a column");
  if (s.T != m.rows) refuse("token_rows must have " + std::to_string(m.rows) + " rows");
  const Tensor* given = maybe(a[4], "out");
  const int64_t R = a[3] == Py_None ? (given && given->dim() > 0 ? given->size(0) : s.T * s.k) : integer(a[3]);
  if (R < 0) refuse("rows must be 0 or more");
  if (given) {
    const Mat o = real(*given, x.scalar_type(), {R, m.cols}, "out");
    keep_apart(area(o), "out", {{area(m), "x"}, {area(tr), "token_rows"}});
  }
  on(x.get_device(), {&tr, given});
  void* stream = address(a[0]);
  const Tensor out = given ? *given : empty({R, m.cols}, x.scalar_type(), x);
  const Mat o = mat(out, "out");
  const int rc =
      launch([&] { return moe_gather(m.p, m.type, m.ld, m.rows, m.cols, s.p, s.k, R, o.p, o.ld, stream); });
  return rc ? status(rc) : THPVariable_Wrap(out);
}

// (stream, y, token_rows, gates or None, fp32 or None, out) -> out
PyObject* combine(PyObject* const* a) {
  const Tensor &y = tensor(a[1], "y"), &tr = tensor(a[2], "token_rows");
  const Mat m = real(y, "y");
  const Slots s = slots(tr, "token_rows");
  if (m.cols < 1) refuse("y must have a column");
  const Tensor* gates = maybe(a[3], "gates");
  const float* g = gates ? flat<float>(*gates, at::kFloat, {s.T, s.k}, "gates") : nullptr;
  const Tensor* given = maybe(a[5], "out");
  const at::ScalarType type = a[4] == Py_None ? y.scalar_type() : out_type(a[4]);
  if (given) {
    const Area o = area(real(*given, type, {s.T, m.cols}, "out"));
    keep_apart(o, "out", {{area(m), "y"}, {area(tr), "token_rows"}});
    if (gates) keep_apart(o, "out", {{area(*gates), "gates"}});
  }
  on(y.get_device(), {&tr, gates, given});
  void* stream = address(a[0]);
  const Tensor out = given ? *given : empty({s.T, m.cols}, type, y);
  const Mat o = mat(out, "out");
  const int rc = launch([&] {
    return moe_combine(m.p, m.type, m.ld, m.rows, m.cols, s.p, g, s.T, s.k, o.p, o.type, o.ld, stream);
  });
  return rc ? status(rc) : THPVariable_Wrap(out);
}

// (stream, dout, y, token_rows, gates, dy, dgates) -> (dy, dgates)
PyObject* combine_backward(PyObject* const* a) {
  const Tensor &dout = tensor(a[1], "dout"), &y = tensor(a[2], "y"), &tr = tensor(a[3], "token_rows"),
               &gates = tensor(a[4], "gates");
  const Mat m = real(y, "y"), d = real(dout, "dout");
  const Slots s = slots(tr, "token_rows");
  if (m.cols < 1) refuse("y must have a column");
  shape(dout, {s.T, m.cols}, "dout");
  const float* g = flat<float>(gates, at::kFloat, {s.T, s.k}, "gates");
  const Tensor *gy = maybe(a[5], "dy"), *gg = maybe(a[6], "dgates");
  const std::initializer_list<std::pair<Area, const char*>> in = {
      {area(d), "dout"}, {area(m), "y"}, {area(tr), "token_rows"}, {area(gates), "gates"}};
  if (gy) keep_apart(area(real(*gy, y.scalar_type(), {m.rows, m.cols}, "dy")), "dy", in);
  if (gg) {
    flat<float>(*gg, at::kFloat, {s.T, s.k}, "dgates");
    keep_apart(area(*gg), "dgates", in);
    if (gy) keep_apart(area(*gg), "dgates", {{area(mat(*gy, "dy")), "dy"}});
  }
  on(y.get_device(), {&dout, &tr, &gates, gy, gg});
  void* stream = address(a[0]);
  const Tensor dy = gy ? *gy : empty({m.rows, m.cols}, y.scalar_type(), y);
  const Tensor dgates = gg ? *gg : empty({s.T, s.k}, at::kFloat, y);
  const Mat o = mat(dy, "dy");
  const int rc = launch([&] {
    return moe_combine_backward(d.p, d.type, d.ld, m.p, m.type, m.ld, m.rows, m.cols, s.p, g, s.T, s.k, o.p, o.ld,
                                ptr<float>(dgates), stream);
  });
  return rc ? status(rc) : tuple({dy, dgates});
}

// ---- 8-bit integers ---------------------------------------------------------

Mat quant_input(const Tensor& x) {
  const Mat m = real(x, "x");
  if (m.cols < 1) refuse("x must have a column");
  return m;
}

// (stream, x, codes, scales) -> (codes, scales)
PyObject* quant(PyObject* const* a) {
  const Tensor& x = tensor(a[1], "x");
  const Mat m = quant_input(x);
  const Tensor *gc = maybe(a[2], "codes"), *gs = maybe(a[3], "scales");
  if (gc) {
    const Mat o = real(*gc, at::kChar, {m.rows, m.cols}, "codes");
    keep_apart(area(o), "codes", {{area(m), "x"}});
  }
  if (gs) {
    flat<float>(*gs, at::kFloat, {m.rows}, "scales");
    keep_apart(area(*gs), "scales", {{area(m), "x"}});
    if (gc) keep_apart(area(*gs), "scales", {{area(mat(*gc, "codes")), "codes"}});
  }
  on(x.get_device(), {gc, gs});
  void* stream = address(a[0]);
  // new codes have their rows whole 128-byte lines apart, the bytes behind them unwritten
  const int64_t ld = up(m.cols, 128);
  Block b((gc ? 0 : m.rows * ld) + (gs ? 0 : Block::room(4 * m.rows)), x);
  const Tensor codes = gc ? *gc : b.take(at::kChar, {m.rows, m.cols}, ld);
  const Tensor scales = gs ? *gs : b.take(at::kFloat, {m.rows});
  const Mat o = mat(codes, "codes");
  const int rc = launch([&] {
    return int8_quant(m.p, m.type, m.rows, m.cols, m.ld, static_cast<int8_t*>(o.p), o.ld, ptr<float>(scales), stream);
  });
  return rc ? status(rc) : tuple({codes, scales});
}

// (stream, w, out) -> packed
PyObject* pack(PyObject* const* a) {
  const Tensor& w = tensor(a[1], "w");
  if (w.scalar_type() != at::kChar || (w.dim() != 2 && w.dim() != 3)) refuse("w must be int8 [N, K] or [G, N, K]");
  const int64_t d = w.dim() - 2, G = d ? w.size(0) : 1, N = w.size(d), K = w.size(d + 1);
  if (G < 1 || N < 1 || N > (1 << 25) || K < 1 || K > 131071)
    refuse("w must hold at least one matrix of 1 to 2^25 rows of 1 to 131071 codes");
  if (w.stride(d + 1) != 1 && K > 1) refuse("w rows must be contiguous");
  const int64_t ld = N > 1 ? w.stride(d) : K, stride = G > 1 ? w.stride(0) : 0;
  if (ld < K) refuse("w: rows overlap");
  std::vector<int64_t> s(w.sizes().begin(), w.sizes().end());
  s[d] = up(N, 16);
  s[d + 1] = up(K, 128);
  const Tensor* given = maybe(a[2], "out");
  if (given) {
    if (given->scalar_type() != at::kChar || !given->is_contiguous()) refuse("out must be contiguous int8");
    shape(*given, at::IntArrayRef(s), "out");
    keep_apart(area(*given), "out", {{Area{number_of(w.data_ptr()), 1, 0, (G - 1) * stride + (N - 1) * ld + K}, "w"}});
  }
  on(w.get_device(), {given});
  void* stream = address(a[0]);
  const Tensor out = given ? *given : empty(s, at::kChar, w);
  const int rc = launch([&] {
    return int8_weight_pack(ptr<int8_t>(w), G, N, K, ld, stride, ptr<int8_t>(out), stream);
  });
  return rc ? status(rc) : THPVariable_Wrap(out);
}

// Packed weights of `lead` matrices for K columns, and their scales.
struct Weights {
  const Tensor &w, &sw;
  int64_t N;
  Weights(PyObject* wo, PyObject* so, int64_t K, bool experts)
      : w(tensor(wo, "w_packed")), sw(tensor(so, "w_scales")) {
    const int64_t d = experts ? 1 : 0;
    if (w.scalar_type() != at::kChar || w.dim() != 2 + d || !w.is_contiguous())
      refuse(experts ? "w_packed must be contiguous int8 [E, Np, Kp] from int8_weight_pack"
                     : "w_packed must be contiguous int8 [Np, Kp] from int8_weight_pack");
    if (sw.scalar_type() != at::kFloat || sw.dim() != 1 + d || !sw.is_contiguous())
      refuse(experts ? "w_scales must be contiguous float32 [E, N]" : "w_scales must be contiguous float32 [N]");
    plain(sw, "w_scales");
    N = sw.size(d);
    if (experts && sw.size(0) != w.size(0)) refuse("w_scales must be of as many experts as w_packed");
    if (N < 1 || w.size(d) != up(N, 16)) refuse("w_packed must have the " + std::to_string(N) + " rows of w_scales, filled up to a multiple of 16");
    if (K < 1 || K > 131071 || w.size(d + 1) != up(K, 128))
      refuse("w_packed must have the " + std::to_string(K) + " columns of the codes, filled up to a multiple of 128");
  }
};

// Codes whose rows can be read to a multiple of 128 columns.
Mat codes(const Tensor& t, const char* name) {
  if (t.scalar_type() != at::kChar) refuse(std::string(name) + " must be int8");
  Mat m = mat(t, name);
  const int64_t kp = up(m.cols, 128);
  if (m.rows <= 1) m.ld = kp;
  if (m.ld < kp || m.ld % 16 != 0)
    refuse(std::string(name) + ": rows must lie a multiple of 16 bytes apart, filled up to a multiple of 128 columns "
           "(int8_quant lays them out so)");
  const int64_t room = (int64_t)t.storage().nbytes() - t.storage_offset();
  if (m.rows > 0 && (m.rows - 1) * m.ld + kp > room)
    refuse(std::string(name) + ": the last row must be filled up to a multiple of 128 columns too");
  return m;
}

const Tensor* output(PyObject* o, at::ScalarType type, int64_t rows, int64_t N,
                     std::initializer_list<std::pair<Area, const char*>> in) {
  const Tensor* y = maybe(o, "y");
  if (y) keep_apart(area(real(*y, type, {rows, N}, "y")), "y", in);
  return y;
}

// (stream, a, a_scales, w_packed, w_scales, bias, fp32, y) -> y
PyObject* gemm(PyObject* const* a) {
  const Tensor &x = tensor(a[1], "a"), &sa = tensor(a[2], "a_scales");
  const Mat m = codes(x, "a");
  const Weights w(a[3], a[4], m.cols, false);
  const float* sap = flat<float>(sa, at::kFloat, {m.rows}, "a_scales");
  const Tensor* bias = maybe(a[5], "bias");
  const float* bp = bias ? flat<float>(*bias, at::kFloat, {w.N}, "bias") : nullptr;
  const at::ScalarType type = out_type(a[6]);
  const Tensor* given = output(a[7], type, m.rows, w.N,
                               {{area(m), "a"}, {area(sa), "a_scales"}, {area(w.w), "w_packed"}, {area(w.sw), "w_scales"}});
  if (given && bias) keep_apart(area(mat(*given, "y")), "y", {{area(*bias), "bias"}});
  on(x.get_device(), {&sa, &w.w, &w.sw, bias, given});
  void* stream = address(a[0]);
  const Tensor y = given ? *given : empty({m.rows, w.N}, type, x);
  const Mat o = mat(y, "y");
  const int rc = launch([&] {
    return int8_gemm(static_cast<const int8_t*>(m.p), m.ld, sap, ptr<int8_t>(w.w), ptr<float>(w.sw), bp, m.rows, w.N,
                     m.cols, o.p, o.ld, type_of(type), stream);
  });
  return rc ? status(rc) : THPVariable_Wrap(y);
}

// (stream, a, a_scales, row_index or None, expert_offsets, w_packed, w_scales, fp32, y) -> y
PyObject* grouped(PyObject* const* a) {
  const Tensor &x = tensor(a[1], "a"), &sa = tensor(a[2], "a_scales"), &offsets = tensor(a[4], "expert_offsets");
  const Mat m = codes(x, "a");
  const Weights w(a[5], a[6], m.cols, true);
  const int64_t E = w.w.size(0);
  const float* sap = flat<float>(sa, at::kFloat, {m.rows}, "a_scales");
  const Tensor* index = maybe(a[3], "row_index");
  if (index && (index->scalar_type() != at::kInt || index->dim() != 1 || !index->is_contiguous()))
    refuse("row_index must be contiguous int32 [R]");
  const int64_t R = index ? index->size(0) : m.rows;
  if (m.rows < 1 && R > 0) refuse("a must have a row");
  if (E < 1 || E > 1024) refuse("there must be 1 to 1024 experts");
  const int32_t* op = flat<int32_t>(offsets, at::kInt, {E + 1}, "expert_offsets");
  const at::ScalarType type = out_type(a[7]);
  const Tensor* given = output(a[8], type, R, w.N,
                               {{area(m), "a"}, {area(sa), "a_scales"}, {area(offsets), "expert_offsets"},
                                {area(w.w), "w_packed"}, {area(w.sw), "w_scales"}});
  if (given && index) keep_apart(area(mat(*given, "y")), "y", {{area(*index), "row_index"}});
  on(x.get_device(), {&sa, &offsets, &w.w, &w.sw, index, given});
  void* stream = address(a[0]);
  const Tensor y = given ? *given : empty({R, w.N}, type, x);
  const Mat o = mat(y, "y");
  const int rc = launch([&] {
    return int8_grouped_gemm(static_cast<const int8_t*>(m.p), m.ld, sap, std::max<int64_t>(m.rows, 1),
                             index ? ptr<int32_t>(*index) : nullptr, op, R, E, ptr<int8_t>(w.w), ptr<float>(w.sw), w.N,
                             m.cols, o.p, o.ld, type_of(type), stream);
  });
  return rc ? status(rc) : THPVariable_Wrap(y);
}

// The limits of int8_quant and int8_gemm, or of int8_grouped_gemm and what it
// reads and writes, for calls that make more than one of them: all are refused
// before the first is made.
void rows_fit(int64_t M, int64_t R, const Weights& w) {
  if (M >= (1 << 24) || R >= (1 << 24)) refuse("too many rows: fewer than 2^24 are taken");
  if (w.N > (1 << 25)) refuse("w_scales must be of 2^25 columns or fewer");
  if (R * w.N > ((int64_t)1 << 36)) refuse("too many results: rows times columns may be 2^36");
}
void experts_fit(int64_t T, int64_t K, int64_t R, int64_t E, const Weights& w) {
  rows_fit(T, R, w);
  if (T * up(K, 128) >= ((int64_t)1 << 32))
    refuse("too many codes: tokens times columns, filled up to a multiple of 128, must be below 2^32");
  if (E * w.N > ((int64_t)1 << 30)) refuse("too many weight rows: experts times columns may be 2^30");
}

// Room for x's codes and scales, one behind the other.
struct Quantised {
  int64_t ld;
  Tensor both;
  int8_t* c;
  float* s;
  Quantised(const Tensor& x, const Mat& m)
      : ld(up(m.cols, 128)), both(empty({m.rows * (ld + (int64_t)sizeof(float))}, at::kChar, x)), c(ptr<int8_t>(both)),
        s(reinterpret_cast<float*>(c + m.rows * ld)) {}
  int make(const Mat& m, void* stream) const {
    return int8_quant(m.p, m.type, m.rows, m.cols, m.ld, c, ld, s, stream);
  }
};

// (stream, x, w_packed, w_scales, bias, fp32) -> y
PyObject* linear(PyObject* const* a) {
  const Tensor& x = tensor(a[1], "x");
  const Mat m = quant_input(x);
  const Weights w(a[2], a[3], m.cols, false);
  const Tensor* bias = maybe(a[4], "bias");
  const float* bp = bias ? flat<float>(*bias, at::kFloat, {w.N}, "bias") : nullptr;
  const at::ScalarType type = out_type(a[5]);
  rows_fit(m.rows, m.rows, w);
  on(x.get_device(), {&w.w, &w.sw, bias});
  void* stream = address(a[0]);
  const Quantised q(x, m);
  const Tensor y = empty({m.rows, w.N}, type, x);
  void* yp = y.data_ptr();
  const int rc = launch([&] {
    if (const int rc1 = q.make(m, stream)) return rc1;
    return int8_gemm(q.c, q.ld, q.s, ptr<int8_t>(w.w), ptr<float>(w.sw), bp, m.rows, w.N, m.cols, yp, w.N, type_of(type),
                     stream);
  });
  return rc ? status(rc) : THPVariable_Wrap(y);
}

// (stream, x, logits, k, w_packed, w_scales, renormalize, fp32 rows, fp32 output)
//   -> (out, gates, experts, expert_offsets, row_index, token_rows)
PyObject* forward(PyObject* const* a) {
  const Tensor &x = tensor(a[1], "x"), &logits = tensor(a[2], "logits");
  const Mat m = quant_input(x);
  const Router r(logits, integer(a[3]));
  const Weights w(a[4], a[5], m.cols, true);
  if (r.l.rows != m.rows) refuse("logits must have " + std::to_string(m.rows) + " rows");
  if (r.l.cols != w.w.size(0)) refuse("logits must be of " + std::to_string(w.w.size(0)) + " experts");
  const bool renormalize = truth(a[6]);
  const at::ScalarType rows = out_type(a[7]), type = out_type(a[8]);
  const int64_t T = m.rows, k = r.k, R = T * k, E = r.l.cols;
  experts_fit(T, m.cols, R, E, w);
  on(x.get_device(), {&logits, &w.w, &w.sw});
  void* stream = address(a[0]);
  Plan p;
  if (const int rc = r.run(logits, renormalize, stream, p)) return status(rc);
  const Tensor out = empty({T, w.N}, type, x);
  if (T > 0) {
    const Quantised q(x, m);
    // rows of bf16 are rounded once more than the output, for half as many bytes
    // out and back (8 of 256 experts, 7168 -> 2048: 32 tokens 127 us with rows in
    // fp32, 125 in bf16, 4096 tokens 897 and 824); the sum over the slots is in
    // fp32 either way
    const Tensor y = empty({R, w.N}, rows, x);
    void *yp = y.data_ptr(), *op = out.data_ptr();
    const int rc = launch([&] {
      if (const int rc1 = q.make(m, stream)) return rc1;
      if (const int rc1 = int8_grouped_gemm(q.c, q.ld, q.s, T, ptr<int32_t>(p.row_index), ptr<int32_t>(p.offsets), R, E,
                                            ptr<int8_t>(w.w), ptr<float>(w.sw), w.N, m.cols, yp, w.N, type_of(rows),
                                            stream))
        return rc1;
      return moe_combine(yp, type_of(rows), w.N, R, w.N, ptr<int32_t>(p.token_rows), ptr<float>(p.gates), T, k, op,
                         type_of(type), w.N, stream);
    });
    if (rc) return status(rc);
  }
  return tuple({out, p.gates, p.experts, p.offsets, p.row_index, p.token_rows});
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

PyMethodDef methods[] = {method<route, 4>("route"),
                         method<sort, 3>("sort"),
                         method<route_backward, 7>("route_backward"),
                         method<gather, 5>("gather"),
                         method<combine, 6>("combine"),
                         method<combine_backward, 7>("combine_backward"),
                         method<quant, 4>("quant"),
                         method<pack, 3>("pack"),
                         method<gemm, 8>("gemm"),
                         method<grouped, 9>("grouped"),
                         method<linear, 6>("linear"),
                         method<forward, 9>("forward"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_moe_binding", "Host side of moe.py's calls.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__moe_binding(void) { return PyModule_Create(&module); }
