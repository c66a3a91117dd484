// qb_binding.cpp -- the expert layer's calls from Python: checks of the
// tensors' type, device, layout and shape, and the call of the C ABI.
//
// A call of 16 tokens takes the GPU some 4 us.  Marshalled by ctypes it took
// the host 6 to 7.5 (a dozen tensor attributes as Python objects, a dozen
// argument conversions), so a decoding step waited for Python; here the same
// checks read the tensor itself, and a call takes the host 3.5 to 4.  The functions' signatures and defaults are
// qb.py's; this module takes their arguments in order and returns the status.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>
#include <tuple>
#include <type_traits>

#include "../../include/qb.h"

namespace {

using c10::ScalarType;

// An argument that is not what the call takes: becomes a ValueError.
struct Bad {
  std::string what;
};
// A Python error that is already set.
struct Raised {};

const char* type_name(ScalarType t) {
  switch (t) {
    case ScalarType::Float: return "torch.float32";
    case ScalarType::Int: return "torch.int32";
    case ScalarType::Byte: return "torch.uint8";
    case ScalarType::BFloat16: return "torch.bfloat16";
    case ScalarType::Float8_e4m3fn: return "torch.float8_e4m3fn";
    default: return c10::toString(t);
  }
}

std::string shape_name(c10::IntArrayRef s) {
  std::string o = "(";
  for (size_t i = 0; i < s.size(); ++i) o += (i ? ", " : "") + std::to_string(s[i]);
  return o + (s.size() == 1 ? ",)" : ")");
}

// The device of the call's tensors, -1 before the first.
thread_local int device;

// A contiguous GPU tensor of this type, or nullptr for None.
const at::Tensor* tensor_or_none(PyObject* o, ScalarType type, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw Bad{std::string(name) + " must be a GPU tensor"};
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) throw Bad{std::string(name) + " must be a GPU tensor"};
  if (t.scalar_type() != type)
    throw Bad{std::string(name) + " must be " + type_name(type) + ", got " + type_name(t.scalar_type())};
  if (!t.is_contiguous()) throw Bad{std::string(name) + " must be contiguous"};
  const int at = t.device().index();
  if (device >= 0 && at != device)
    throw Bad{std::string(name) + " is on cuda:" + std::to_string(at) + ", another tensor on cuda:" + std::to_string(device)};
  device = at;
  return &t;
}
const at::Tensor& tensor(PyObject* o, ScalarType type, const char* name, int dims) {
  const at::Tensor* t = tensor_or_none(o, type, name);
  if (!t) throw Bad{std::string(name) + " is required"};
  if (t->dim() != dims)
    throw Bad{std::string(name) + " has shape " + shape_name(t->sizes()) + ", expected " + std::to_string(dims) +
              " dimensions"};
  return *t;
}

void check_shape(const at::Tensor& t, const char* name, std::initializer_list<int64_t> shape) {
  const c10::IntArrayRef want(shape);
  if (t.sizes() != want)
    throw Bad{std::string(name) + " has shape " + shape_name(t.sizes()) + ", expected " + shape_name(want)};
}

// An input's address, for T const, or an output's, which gets a storage of
// its own where it shares another tensor's until it is written.
template <class T>
T* address(const at::Tensor& t) {
  if constexpr (std::is_const_v<T>)
    return static_cast<T*>(t.const_data_ptr());
  else
    return static_cast<T*>(t.mutable_data_ptr());
}
// The address of a tensor of this shape, nullptr for None (or a refusal).
template <class T>
T* opt(PyObject* o, ScalarType type, const char* name, std::initializer_list<int64_t> shape) {
  const at::Tensor* t = tensor_or_none(o, type, name);
  if (!t) return nullptr;
  check_shape(*t, name, shape);
  return address<T>(*t);
}
template <class T>
T* req(PyObject* o, ScalarType type, const char* name, std::initializer_list<int64_t> shape) {
  if (o == Py_None) throw Bad{std::string(name) + " is required"};
  return opt<T>(o, type, name, shape);
}

int64_t whole(PyObject* o, const char* name, int64_t low = INT32_MIN, int64_t high = INT32_MAX) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  if (v < low || v > high) throw Bad{std::string(name) + "=" + std::to_string(v) + " is out of range"};
  return v;
}
int narrow(int64_t v, const char* name) {
  if (v > INT32_MAX) throw Bad{std::string(name) + " has " + std::to_string(v) + " entries, at most 2^31 - 1"};
  return int(v);
}

// qb.py's: a stream object, or None for the current one, to its raw handle; refuses one of another device than the tensors'
PyObject* stream_handle;

// The last argument of every call, looked at once the others are sound.
qb_stream_t stream_of(PyObject* o) {
  PyObject* const at = PyLong_FromLong(device);
  if (!at) throw Raised{};
  PyObject* h = PyObject_CallFunctionObjArgs(stream_handle, o, at, nullptr);
  Py_DECREF(at);
  if (!h) throw Raised{};
  void* p = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  if (!p && PyErr_Occurred()) throw Raised{};
  return static_cast<qb_stream_t>(p);
}

struct Workspace {
  void* p;
  int64_t n;
};
Workspace workspace(PyObject* o) {
  const at::Tensor* t = tensor_or_none(o, ScalarType::Byte, "ws");
  return t ? Workspace{address<void>(*t), t->numel()} : Workspace{nullptr, 0};
}

// seq_off [B + 1] and valid [N]
struct Seqs {
  const int32_t* off;
  int B;
  const uint8_t* valid;
};
Seqs sequences(PyObject* off, PyObject* valid, int64_t N) {
  Seqs s{nullptr, 1, opt<const uint8_t>(valid, ScalarType::Byte, "valid", {N})};
  if (off != Py_None) {
    const at::Tensor& t = tensor(off, ScalarType::Int, "seq_off", 1);
    s.off = address<const int32_t>(t);
    s.B = narrow(t.numel() - 1, "seq_off");
  }
  return s;
}

int64_t ld(int64_t n) { return (n + 127) / 128 * 128; }
int64_t sld(int64_t n) { return (n + 511) / 512 * 4; }
int64_t ld4(int64_t n) { return (n + 255) / 256 * 128; }
int64_t sld4(int64_t n) { return (n + 255) / 256 * 8; }

// The library's entry points, set by `connect`.
#define QB_ENTRIES(X) \
  X(qb_balance_forward) X(qb_balance_backward) X(qb_dispatch) X(qb_combine) X(qb_combine_backward) \
  X(qb_fp8_quantize) X(qb_fp8_quantize_cols) X(qb_fp8_quantize_weight) X(qb_fp8_product) X(qb_fp8_weight_grad) \
  X(qb_bf16_product) X(qb_bf16_weight_grad) X(qb_fp4_quantize) X(qb_fp4_quantize_weight) X(qb_fp4_product)
struct Library {
#define X(f) decltype(&::f) f;
  QB_ENTRIES(X)
#undef X
} lib;

constexpr ScalarType F32 = ScalarType::Float, I32 = ScalarType::Int, U8 = ScalarType::Byte,
                     BF16 = ScalarType::BFloat16, F8 = ScalarType::Float8_e4m3fn;

// The arguments of a call are gathered in a braced list, which is looked
// through from left to right: the first wrong one is the one that is named.

// s, b, K, topk, gate, count, weight, loss, ws, coef, seq_off, valid, stream
int balance_forward(PyObject* const* a) {
  const at::Tensor& s = tensor(a[0], F32, "s", 2);
  const int64_t N = s.size(0), E = s.size(1), K = whole(a[2], "K");
  const Seqs q = sequences(a[10], a[11], N);
  const Workspace ws = workspace(a[8]);
  const double coef = PyFloat_AsDouble(a[9]);
  if (coef == -1.0 && PyErr_Occurred()) throw Raised{};
  return std::apply(
      lib.qb_balance_forward,
      std::tuple{address<const float>(s), req<const float>(a[1], F32, "b", {E}), N, narrow(E, "s"), int(K), q.off, q.B,
                 q.valid, float(coef), req<int32_t>(a[3], I32, "topk", {N, K}), opt<float>(a[4], F32, "gate", {N, K}),
                 opt<int32_t>(a[5], I32, "count", {q.B, E}), opt<float>(a[6], F32, "weight", {q.B, E}),
                 opt<float>(a[7], F32, "loss", {1}), ws.p, ws.n, stream_of(a[12])});
}

// s, topk, weight, dloss, dgate, dlogits, seq_off, valid, stream
int balance_backward(PyObject* const* a) {
  const at::Tensor& s = tensor(a[0], F32, "s", 2);
  const int64_t N = s.size(0), E = s.size(1);
  const at::Tensor& topk = tensor(a[1], I32, "topk", 2);
  const int64_t K = topk.size(1);
  check_shape(topk, "topk", {N, K});
  const Seqs q = sequences(a[6], a[7], N);
  return std::apply(
      lib.qb_balance_backward,
      std::tuple{address<const float>(s), address<const int32_t>(topk), N, narrow(E, "s"), narrow(K, "topk"), q.off,
                 q.B, q.valid, opt<const float>(a[2], F32, "weight", {q.B, E}),
                 opt<const float>(a[3], F32, "dloss", {1}), opt<const float>(a[4], F32, "dgate", {N, K}),
                 req<float>(a[5], F32, "dlogits", {N, E}), stream_of(a[8])});
}

// topk, E, align, off, row_src, pos, ws, stream
int dispatch(PyObject* const* a) {
  const at::Tensor& topk = tensor(a[0], I32, "topk", 2);
  const int64_t N = topk.size(0), K = topk.size(1), E = whole(a[1], "E"), align = whole(a[2], "align");
  const at::Tensor& src = tensor(a[4], I32, "row_src", 1);
  const Workspace ws = workspace(a[6]);
  return std::apply(
      lib.qb_dispatch,
      std::tuple{address<const int32_t>(topk), N, narrow(K, "topk"), int(E), int(align),
                 req<int32_t>(a[3], I32, "off", {E + 1}), src.numel(), address<int32_t>(src),
                 req<int32_t>(a[5], I32, "pos", {N, K}), ws.p, ws.n, stream_of(a[7])});
}

// rows, pos, out, gate, stream
int combine(PyObject* const* a) {
  const at::Tensor& rows = tensor(a[0], BF16, "rows", 2);
  const at::Tensor& pos = tensor(a[1], I32, "pos", 2);
  const int64_t N = pos.size(0), K = pos.size(1), H = rows.size(1);
  return std::apply(
      lib.qb_combine,
      std::tuple{address<const uint16_t>(rows), rows.size(0), address<const int32_t>(pos),
                 opt<const float>(a[3], F32, "gate", {N, K}), N, narrow(K, "pos"), narrow(H, "rows"),
                 req<uint16_t>(a[2], BF16, "out", {N, H}), stream_of(a[4])});
}

// dout, rows, pos, row_src, drows, gate, dgate, stream
int combine_backward(PyObject* const* a) {
  const at::Tensor& drows = tensor(a[4], BF16, "drows", 2);
  const at::Tensor& pos = tensor(a[2], I32, "pos", 2);
  const int64_t R = drows.size(0), H = drows.size(1), N = pos.size(0), K = pos.size(1);
  return std::apply(
      lib.qb_combine_backward,
      std::tuple{req<const uint16_t>(a[0], BF16, "dout", {N, H}), opt<const uint16_t>(a[1], BF16, "rows", {R, H}), R,
                 address<const int32_t>(pos), req<const int32_t>(a[3], I32, "row_src", {R}),
                 opt<const float>(a[5], F32, "gate", {N, K}), N, narrow(K, "pos"), narrow(H, "drows"),
                 address<uint16_t>(drows), opt<float>(a[6], F32, "dgate", {N, K}), stream_of(a[7])});
}

// x, xq, xs, row_src, stream; xt and xts in the place of xq and xs for the transpose
int quantize(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], BF16, "x", 2);
  const at::Tensor* src = tensor_or_none(a[3], I32, "row_src");
  const int64_t C = x.size(1), M = src ? src->numel() : x.size(0);
  if (src) check_shape(*src, "row_src", {M});
  return std::apply(
      lib.qb_fp8_quantize,
      std::tuple{address<const uint16_t>(x), x.size(0), src ? address<const int32_t>(*src) : nullptr, M, narrow(C, "x"),
                 req<uint8_t>(a[1], F8, "xq", {M, ld(C)}), req<uint8_t>(a[2], U8, "xs", {M, sld(C)}),
                 stream_of(a[4])});
}
int quantize_cols(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], BF16, "x", 2);
  const at::Tensor* src = tensor_or_none(a[3], I32, "row_src");
  const int64_t C = x.size(1), M = src ? src->numel() : x.size(0);
  if (src) check_shape(*src, "row_src", {M});
  return std::apply(
      lib.qb_fp8_quantize_cols,
      std::tuple{address<const uint16_t>(x), x.size(0), src ? address<const int32_t>(*src) : nullptr, M, narrow(C, "x"),
                 req<uint8_t>(a[1], F8, "xt", {C, ld(M)}), req<uint8_t>(a[2], U8, "xts", {C, sld(M)}),
                 stream_of(a[4])});
}

// A tensor of these dimensions, behind G matrices if `stacked`.
template <class T>
T* stack(PyObject* o, ScalarType type, const char* name, bool stacked, int64_t G, int64_t i, int64_t j) {
  return stacked ? req<T>(o, type, name, {G, i, j}) : req<T>(o, type, name, {i, j});
}

// w, wq, ws, wt, wts, stream
int quantize_weight(PyObject* const* a) {
  const at::Tensor* w = tensor_or_none(a[0], F32, "w");
  if (!w) throw Bad{"w is required"};
  if (w->dim() != 2 && w->dim() != 3) throw Bad{"w must be [N, C] or [G, N, C], got " + shape_name(w->sizes())};
  const bool st = w->dim() == 3;
  const int64_t G = st ? w->size(0) : 1, N = w->size(-2), C = w->size(-1);
  uint8_t* wt = a[3] == Py_None ? nullptr : stack<uint8_t>(a[3], F8, "wt", st, G, C, ld(N));
  uint8_t* wts = a[4] == Py_None ? nullptr : stack<uint8_t>(a[4], U8, "wts", st, G, ld(C) / 128, sld(N));
  return std::apply(
      lib.qb_fp8_quantize_weight,
      std::tuple{address<const float>(*w), narrow(G, "w"), narrow(N, "w"), narrow(C, "w"),
                 stack<uint8_t>(a[1], F8, "wq", st, G, N, ld(C)),
                 stack<uint8_t>(a[2], U8, "ws", st, G, ld(N) / 128, sld(C)), wt, wts, stream_of(a[5])});
}

// off int32 [G + 1], or None for one matrix
struct Offsets {
  const int32_t* off;
  int G;
};
Offsets offsets(PyObject* o) {
  if (o == Py_None) return {nullptr, 1};
  const at::Tensor& t = tensor(o, I32, "off", 1);
  return {address<const int32_t>(t), narrow(t.numel() - 1, "off")};
}

// xq, xs, w, w_scale, y, off, exact, stream
int product(PyObject* const* a) {
  const at::Tensor& xq = tensor(a[0], F8, "xq", 2);
  const Offsets g = offsets(a[5]);
  const bool st = g.off != nullptr;
  const int64_t M = xq.size(0), l = xq.size(1);
  const at::Tensor& w = tensor(a[2], F8, "w", st ? 3 : 2);
  const int64_t N = w.size(-2);
  const int exact = PyObject_IsTrue(a[6]);
  if (exact < 0) throw Raised{};
  return std::apply(
      lib.qb_fp8_product,
      std::tuple{address<const uint8_t>(xq), req<const uint8_t>(a[1], U8, "xs", {M, sld(l)}),
                 stack<const uint8_t>(a[2], F8, "w", st, g.G, N, l),
                 stack<const uint8_t>(a[3], U8, "w_scale", st, g.G, ld(N) / 128, sld(l)), M, narrow(N, "w"),
                 narrow(l, "xq"), g.off, g.G, exact, req<uint16_t>(a[4], BF16, "y", {M, N}), stream_of(a[7])});
}

// dyt, dyts, xt, xts, dw, off, stream
int weight_grad(PyObject* const* a) {
  const at::Tensor& dyt = tensor(a[0], F8, "dyt", 2);
  const at::Tensor& xt = tensor(a[2], F8, "xt", 2);
  const Offsets g = offsets(a[5]);
  const int64_t N = dyt.size(0), l = dyt.size(1), C = xt.size(0);
  check_shape(xt, "xt", {C, l});
  return std::apply(
      lib.qb_fp8_weight_grad,
      std::tuple{address<const uint8_t>(dyt), req<const uint8_t>(a[1], U8, "dyts", {N, sld(l)}),
                 address<const uint8_t>(xt), req<const uint8_t>(a[3], U8, "xts", {C, sld(l)}), l, narrow(N, "dyt"),
                 narrow(C, "xt"), g.off, g.G,
                 stack<float>(a[4], F32, "dw", g.off != nullptr, g.G, N, C), stream_of(a[6])});
}

// row_src int32 [M], or None: the rows as they are
struct Rows {
  const int32_t* src;
  int64_t M;
};
Rows rows_of(PyObject* o, int64_t Mx) {
  const at::Tensor* t = tensor_or_none(o, I32, "row_src");
  if (!t) return {nullptr, Mx};
  if (t->dim() != 1) throw Bad{"row_src has shape " + shape_name(t->sizes()) + ", expected 1 dimensions"};
  return {address<const int32_t>(*t), t->numel()};
}

// x, w, y, off, row_src, transposed, stream
int bf16_product(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], BF16, "x", 2);
  const Offsets g = offsets(a[3]);
  const Rows rows = rows_of(a[4], x.size(0));
  const int transposed = PyObject_IsTrue(a[5]);
  if (transposed < 0) throw Raised{};
  const bool st = g.off != nullptr;
  const int64_t C = x.size(1);
  const at::Tensor& w = tensor(a[1], BF16, "w", st ? 3 : 2);
  const int64_t N = w.size(transposed ? -1 : -2);
  return std::apply(
      lib.qb_bf16_product,
      std::tuple{address<const uint16_t>(x), x.size(0), rows.src, rows.M,
                 stack<const uint16_t>(a[1], BF16, "w", st, g.G, transposed ? C : N, transposed ? N : C),
                 narrow(N, "w"), narrow(C, "x"), g.off, g.G, transposed,
                 req<uint16_t>(a[2], BF16, "y", {rows.M, N}), stream_of(a[6])});
}

// dy, x, dw, off, row_src, ws, stream
int bf16_weight_grad(PyObject* const* a) {
  const at::Tensor& dy = tensor(a[0], BF16, "dy", 2);
  const at::Tensor& x = tensor(a[1], BF16, "x", 2);
  const Offsets g = offsets(a[3]);
  const Rows rows = rows_of(a[4], x.size(0));
  const Workspace ws = workspace(a[5]);
  const int64_t N = dy.size(1), C = x.size(1);
  check_shape(dy, "dy", {rows.M, N});
  return std::apply(
      lib.qb_bf16_weight_grad,
      std::tuple{address<const uint16_t>(dy), address<const uint16_t>(x), x.size(0), rows.src, rows.M, narrow(N, "dy"),
                 narrow(C, "x"), g.off, g.G, stack<float>(a[2], F32, "dw", g.off != nullptr, g.G, N, C), ws.p, ws.n,
                 stream_of(a[6])});
}

// x, xq, xs, row_src, stream
int fp4_quantize(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], BF16, "x", 2);
  const Rows rows = rows_of(a[3], x.size(0));
  const int64_t C = x.size(1);
  return std::apply(
      lib.qb_fp4_quantize,
      std::tuple{address<const uint16_t>(x), x.size(0), rows.src, rows.M, narrow(C, "x"),
                 req<uint8_t>(a[1], U8, "xq", {rows.M, ld4(C)}), req<uint8_t>(a[2], U8, "xs", {rows.M, sld4(C)}),
                 stream_of(a[4])});
}

// w, wq, ws, wt, wts, stream
int fp4_quantize_weight(PyObject* const* a) {
  const at::Tensor* w = tensor_or_none(a[0], F32, "w");
  if (!w) throw Bad{"w is required"};
  if (w->dim() != 2 && w->dim() != 3) throw Bad{"w must be [N, C] or [G, N, C], got " + shape_name(w->sizes())};
  const bool st = w->dim() == 3;
  const int64_t G = st ? w->size(0) : 1, N = w->size(-2), C = w->size(-1);
  uint8_t* wt = a[3] == Py_None ? nullptr : stack<uint8_t>(a[3], U8, "wt", st, G, C, ld4(N));
  uint8_t* wts = a[4] == Py_None ? nullptr : stack<uint8_t>(a[4], U8, "wts", st, G, C, sld4(N));
  return std::apply(
      lib.qb_fp4_quantize_weight,
      std::tuple{address<const float>(*w), narrow(G, "w"), narrow(N, "w"), narrow(C, "w"),
                 stack<uint8_t>(a[1], U8, "wq", st, G, N, ld4(C)), stack<uint8_t>(a[2], U8, "ws", st, G, N, sld4(C)),
                 wt, wts, stream_of(a[5])});
}

// xq, xs, w, w_scale, y, off, stream
int fp4_product(PyObject* const* a) {
  const at::Tensor& xq = tensor(a[0], U8, "xq", 2);
  const Offsets g = offsets(a[5]);
  const bool st = g.off != nullptr;
  const int64_t M = xq.size(0), l = xq.size(1), C = 2 * l;
  check_shape(xq, "xq", {M, ld4(C)});
  const at::Tensor& w = tensor(a[2], U8, "w", st ? 3 : 2);
  const int64_t N = w.size(-2);
  return std::apply(
      lib.qb_fp4_product,
      std::tuple{address<const uint8_t>(xq), req<const uint8_t>(a[1], U8, "xs", {M, sld4(C)}),
                 stack<const uint8_t>(a[2], U8, "w", st, g.G, N, l),
                 stack<const uint8_t>(a[3], U8, "w_scale", st, g.G, N, sld4(C)), M, narrow(N, "w"), narrow(C, "xq"),
                 g.off, g.G, req<uint16_t>(a[4], BF16, "y", {M, N}), stream_of(a[6])});
}

// No C++ exception leaves a call.
template <int (*F)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != N) return PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
  device = -1;
  try {
    return PyLong_FromLong(F(a));
  } catch (const Bad& e) {
    PyErr_SetString(PyExc_ValueError, e.what.c_str());
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// The function that gives a stream's handle, and the entry points' addresses
// in QB_ENTRIES' order.
PyObject* connect(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void** at = reinterpret_cast<void**>(&lib);
  if (--n != Py_ssize_t(sizeof(lib) / sizeof(void*)))
    return PyErr_Format(PyExc_TypeError, "%zu addresses expected, got %zd", sizeof(lib) / sizeof(void*), n);
  Py_INCREF(*a);
  Py_XSETREF(stream_handle, *a++);
  for (Py_ssize_t i = 0; i < n; ++i) {
    at[i] = PyLong_AsVoidPtr(a[i]);
    if (!at[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "NULL entry point");
      return nullptr;
    }
  }
  Py_RETURN_NONE;
}

#define QB_CALL(name, n) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<name, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"connect", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&connect)), METH_FASTCALL, nullptr},
    QB_CALL(balance_forward, 13),
    QB_CALL(balance_backward, 9),
    QB_CALL(dispatch, 8),
    QB_CALL(combine, 5),
    QB_CALL(combine_backward, 8),
    QB_CALL(quantize, 5),
    QB_CALL(quantize_cols, 5),
    QB_CALL(quantize_weight, 6),
    QB_CALL(product, 8),
    QB_CALL(weight_grad, 7),
    QB_CALL(bf16_product, 7),
    QB_CALL(bf16_weight_grad, 7),
    QB_CALL(fp4_quantize, 5),
    QB_CALL(fp4_quantize_weight, 6),
    QB_CALL(fp4_product, 7),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qb_binding", "Calls of libqb's expert layer.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__qb_binding(void) { return PyModule_Create(&module); }
