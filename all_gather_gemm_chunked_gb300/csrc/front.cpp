// front.cpp -- native part of the torch front end of include/ag_moe.h (moe.py, fp8.py):
// checks tensors, allocates outputs, takes the current stream and calls the library.
// A call's host time decides how long a small operator takes: in Python the checks,
// the allocation and the foreign call took 10 to 18 us a call, longer than the kernels.
//
// Wrong tensors raise TypeError or ValueError; a negative code of the library raises
// what the error function given to init() returns.  The tensors of a call, and its plan,
// are on one device, which is current while it allocates and launches.

#include <Python.h>

#include <optional>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include "ag_moe.h"

namespace {

PyObject* g_error = nullptr;  // () -> exception for the library's last error

// Thrown once the Python error is set.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  PyErr_FormatV(type, fmt, ap);
  va_end(ap);
  throw Raised();
}

int64_t check_rc(int64_t rc) {
  if (rc >= 0) return rc;
  PyObject* e = g_error ? PyObject_CallNoArgs(g_error) : nullptr;
  if (e) {
    PyErr_SetObject(reinterpret_cast<PyObject*>(Py_TYPE(e)), e);
    Py_DECREF(e);
  } else if (!PyErr_Occurred()) {
    PyErr_SetString(PyExc_RuntimeError, ag_gemm_last_error_message());
  }
  throw Raised();
}

#define AGG_BEGIN \
  HANDLE_TH_ERRORS try {
#define AGG_END                           \
  }                                       \
  catch (const Raised&) { return nullptr; } \
  END_HANDLE_TH_ERRORS

void check_args(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) raise(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
}

int64_t to_int(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}
int to_int32(PyObject* o, const char* name) {
  const int64_t v = to_int(o);
  if (v != static_cast<int>(v)) raise(PyExc_ValueError, "%s is out of range", name);
  return static_cast<int>(v);
}

ag_moe_plan* to_plan(PyObject* o) {
  if (o == Py_None) raise(PyExc_ValueError, "the plan is closed");
  return reinterpret_cast<ag_moe_plan*>(static_cast<uintptr_t>(to_int(o)));
}

// A call's first tensor.
const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a torch.Tensor", name);
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) raise(PyExc_ValueError, "%s must be on a CUDA device", name);
  return t;
}
// Any other: on the first one's device.
const at::Tensor& tensor(PyObject* o, const char* name, const at::Tensor& first) {
  const at::Tensor& t = tensor(o, name);
  if (t.device() != first.device())
    raise(PyExc_ValueError, "%s is on device %s, the call's first tensor on %s", name, t.device().str().c_str(),
          first.device().str().c_str());
  return t;
}

const char* type_name(at::ScalarType t) { return c10::toString(t); }

int type_code(at::ScalarType t) {
  switch (t) {
    case at::ScalarType::Half: return AG_GEMM_F16;
    case at::ScalarType::BFloat16: return AG_GEMM_BF16;
    case at::ScalarType::Float: return AG_MOE_F32;
    default: return -1;
  }
}
int float_type(const at::Tensor& t, const char* name) {
  const int c = type_code(t.scalar_type());
  if (c < 0)
    raise(PyExc_TypeError, "%s must be float16, bfloat16 or float32, got %s", name, type_name(t.scalar_type()));
  return c;
}
void want_type(const at::Tensor& t, const char* name, at::ScalarType type) {
  if (t.scalar_type() != type)
    raise(PyExc_TypeError, "%s must be %s, got %s", name, type_name(type), type_name(t.scalar_type()));
}

std::string shape_of(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}
void want_shape(const at::Tensor& t, const char* name, at::IntArrayRef shape) {
  if (t.sizes() != shape)
    raise(PyExc_ValueError, "%s must have shape %s, got %s", name, shape_of(shape).c_str(),
          shape_of(t.sizes()).c_str());
}

// Pitch of a matrix with contiguous rows (a column block of a wider one is one).
int64_t pitch(const at::Tensor& t, const char* name, int64_t cols = -1) {
  if (t.dim() != 2 || (cols >= 0 && t.size(1) != cols))
    raise(PyExc_ValueError, "%s must have shape (rows, %s), got %s", name,
          cols < 0 ? "columns" : std::to_string(cols).c_str(), shape_of(t.sizes()).c_str());
  if (t.is_contiguous()) return t.size(1);
  if (t.stride(1) != 1 || t.stride(0) < t.size(1))
    raise(PyExc_ValueError, "%s must have contiguous rows", name);
  return t.stride(0);
}

// Pointer of a contiguous tensor of this type and shape, on the first one's device.
template <typename T = void>
T* plain(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, const at::Tensor& first) {
  const at::Tensor& t = tensor(o, name, first);
  want_type(t, name, type);
  want_shape(t, name, shape);
  if (!t.is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", name);
  return static_cast<T*>(t.data_ptr());
}

at::Tensor make(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
  return at::Tensor(at::detail::empty_cuda(shape, type, like.device(), c10::nullopt));
}

// Tensors that share one allocation, one after the other from 256-byte boundaries (an
// allocation takes about half a microsecond of host time, and as much to give back).
struct Pieces {
  at::Tensor all;
  int64_t used = 0;
  static int64_t room(int64_t bytes) { return (bytes + 255) & ~int64_t{255}; }
  Pieces(int64_t bytes, const at::Tensor& like) : all(make({bytes}, at::ScalarType::Byte, like)) {}
  at::Tensor take(at::IntArrayRef shape, at::ScalarType type) {
    const int64_t size = static_cast<int64_t>(c10::elementSize(type));
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(),
                                                            c10::scalarTypeToTypeMeta(type));
    t.unsafeGetTensorImpl()->set_storage_offset(used / size);
    t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    used += room(t.numel() * size);
    return t;
  }
};

// Makes a tensor's device current for a scope.  (A guard where it is so already takes two
// driver calls to give back what it did not change.)
struct Current {
  std::optional<c10::cuda::CUDAGuard> guard;
  explicit Current(const at::Tensor& t) {
    if (c10::cuda::current_device() != t.device().index()) guard.emplace(t.device());
  }
};

void* stream_of(const at::Tensor& t) {
  return c10::cuda::getCurrentCUDAStream(t.get_device()).stream();
}

PyObject* wrap(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }

template <typename... T>
PyObject* tuple_of(T&&... t) {
  PyObject* r = PyTuple_New(sizeof...(T));
  if (!r) throw Raised();
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(r, i++, wrap(std::move(t))), ...);
  return r;
}

constexpr auto kI32 = at::ScalarType::Int;
constexpr auto kF32 = at::ScalarType::Float;
constexpr auto kE4m3 = at::ScalarType::Float8_e4m3fn;

int64_t blocks(int64_t n) { return (n + AG_MOE_SCALE_BLOCK - 1) / AG_MOE_SCALE_BLOCK; }

// init(error): error() makes the exception for the library's last error.
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  AGG_BEGIN
  check_args(n, 1);
  Py_INCREF(a[0]);
  Py_XDECREF(g_error);
  g_error = a[0];
  Py_RETURN_NONE;
  AGG_END
}

// route(logits, top_k, normalize) -> weights, experts, offsets, order, slots, normalize
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  AGG_BEGIN
  check_args(n, 3);
  const at::Tensor& z = tensor(a[0], "logits");
  const int type = float_type(z, "logits");
  const int64_t ld = pitch(z, "logits"), T = z.size(0), E = z.size(1);
  const int k = to_int32(a[1], "top_k");
  if (E > AG_MOE_MAX_EXPERTS) check_rc(ag_moe_route_workspace(T, AG_MOE_MAX_EXPERTS + 1, k));
  const int64_t size = check_rc(ag_moe_route_workspace(T, static_cast<int>(E), k));
  const Current current(z);
  Pieces pieces(4 * Pieces::room(T * k * 4) + Pieces::room((E + 1) * 4), z);
  at::Tensor w = pieces.take({T, k}, kF32), e = pieces.take({T, k}, kI32), off = pieces.take({E + 1}, kI32),
             order = pieces.take({T * k}, kI32), slots = pieces.take({T, k}, kI32), ws;
  if (size > 0) ws = make({size}, at::ScalarType::Byte, z);
  check_rc(ag_moe_route(T, static_cast<int>(E), k, type, z.data_ptr(), ld, PyObject_IsTrue(a[2]),
                        static_cast<float*>(w.data_ptr()), static_cast<int32_t*>(e.data_ptr()),
                        static_cast<int32_t*>(off.data_ptr()), static_cast<int32_t*>(order.data_ptr()),
                        static_cast<int32_t*>(slots.data_ptr()), size > 0 ? ws.data_ptr() : nullptr,
                        stream_of(z)));
  // (the fields of moe.Routing, which takes the tuple as it is)
  PyObject* r = PyTuple_New(6);
  if (!r) throw Raised();
  Py_ssize_t i = 0;
  for (at::Tensor* t : {&w, &e, &off, &order, &slots}) PyTuple_SET_ITEM(r, i++, wrap(std::move(*t)));
  PyTuple_SET_ITEM(r, i, Py_NewRef(a[2]));
  return r;
  AGG_END
}

// route_backward(logits, weights, experts, dweights, normalize) -> dlogits
PyObject* route_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  AGG_BEGIN
  check_args(n, 5);
  const at::Tensor& z = tensor(a[0], "logits");
  const int type = float_type(z, "logits");
  const int64_t ld = pitch(z, "logits"), T = z.size(0), E = z.size(1);
  const at::Tensor& wt = tensor(a[1], "routing.weights", z);
  const int64_t k = wt.dim() == 2 ? wt.size(1) : 0;
  const float* w = plain<float>(a[1], "routing.weights", kF32, {T, k}, z);
  const int32_t* e = plain<int32_t>(a[2], "routing.experts", kI32, {T, k}, z);
  const float* dw = plain<float>(a[3], "dweights", kF32, {T, k}, z);
  const Current current(z);
  at::Tensor out = make({T, E}, z.scalar_type(), z);
  check_rc(ag_moe_route_backward(T, static_cast<int>(E), static_cast<int>(k), type, z.data_ptr(), ld,
                                 PyObject_IsTrue(a[4]), w, e, dw, out.data_ptr(), stream_of(z)));
  return wrap(out);
  AGG_END
}

// gather(x, order, slots) -> rows
PyObject* gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
  AGG_BEGIN
  check_args(n, 3);
  const at::Tensor& x = tensor(a[0], "x");
  const int type = float_type(x, "x");
  const int64_t ld = pitch(x, "x"), T = x.size(0), H = x.size(1);
  const at::Tensor& slots = tensor(a[2], "routing.slots", x);
  const int64_t k = slots.dim() == 2 ? slots.size(1) : 0;
  const int32_t* order = plain<int32_t>(a[1], "routing.order", kI32, {T * k}, x);
  const Current current(x);
  at::Tensor out = make({T * k, H}, x.scalar_type(), x);
  check_rc(ag_moe_gather(T, static_cast<int>(k), H, type, x.data_ptr(), ld, order, out.data_ptr(), stream_of(x)));
  return wrap(out);
  AGG_END
}

// The layout both directions of combine read: slots, and y with a row for each choice.
struct Choices {
  int64_t T, k;
  const int32_t* slots;
};
Choices choices(PyObject* slots_o, const at::Tensor& y) {
  const at::Tensor& s = tensor(slots_o, "slots", y);
  if (s.dim() != 2) raise(PyExc_ValueError, "slots must have shape (tokens, top_k), got %s", shape_of(s.sizes()).c_str());
  const int64_t T = s.size(0), k = s.size(1);
  if (y.size(0) != T * k)
    raise(PyExc_ValueError, "y must have %lld rows, got %lld", static_cast<long long>(T * k),
          static_cast<long long>(y.size(0)));
  return {T, k, plain<int32_t>(slots_o, "slots", kI32, {T, k}, y)};
}

// combine(y, slots, weights or None) -> out
PyObject* combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
  AGG_BEGIN
  check_args(n, 3);
  const at::Tensor& y = tensor(a[0], "y");
  const int type = float_type(y, "y");
  const int64_t ld = pitch(y, "y"), H = y.size(1);
  const Choices c = choices(a[1], y);
  const float* w = a[2] == Py_None ? nullptr : plain<float>(a[2], "weights", kF32, {c.T, c.k}, y);
  const Current current(y);
  at::Tensor out = make({c.T, H}, y.scalar_type(), y);
  check_rc(ag_moe_combine(c.T, static_cast<int>(c.k), H, type, y.data_ptr(), ld, c.slots, w, out.data_ptr(),
                          stream_of(y)));
  return wrap(out);
  AGG_END
}

// combine_backward(dout, y, slots, weights, offsets or None) -> dy, dweights
PyObject* combine_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  AGG_BEGIN
  check_args(n, 5);
  const at::Tensor &d = tensor(a[0], "dout"), &y = tensor(a[1], "y", d);
  const int type = float_type(y, "y");
  want_type(d, "dout", y.scalar_type());
  const int64_t ld = pitch(y, "y"), H = y.size(1), ldd = pitch(d, "dout", H);
  const Choices c = choices(a[2], y);
  if (d.size(0) != c.T)
    raise(PyExc_ValueError, "dout must have %lld rows, got %lld", static_cast<long long>(c.T),
          static_cast<long long>(d.size(0)));
  const float* w = plain<float>(a[3], "weights", kF32, {c.T, c.k}, y);
  const int32_t* end = nullptr;
  if (a[4] != Py_None) {
    const int64_t m = tensor(a[4], "offsets", y).numel();
    if (m < 1) raise(PyExc_ValueError, "offsets must not be empty");
    end = plain<int32_t>(a[4], "offsets", kI32, {m}, y) + m - 1;
  }
  const Current current(y);
  at::Tensor dy = make({c.T * c.k, H}, y.scalar_type(), y), dw = make({c.T, c.k}, kF32, y);
  check_rc(ag_moe_combine_backward(c.T, static_cast<int>(c.k), H, type, d.data_ptr(), ldd, y.data_ptr(), ld,
                                   c.slots, w, end, dy.data_ptr(), static_cast<float*>(dw.data_ptr()),
                                   stream_of(y)));
  return tuple_of(dy, dw);
  AGG_END
}

// quantize_rows(x, order or None, slots or None) -> codes, scales
PyObject* quantize_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  AGG_BEGIN
  check_args(n, 3);
  const at::Tensor& x = tensor(a[0], "x");
  const int type = float_type(x, "x");
  const int64_t ld = pitch(x, "x"), src = x.size(0), K = x.size(1);
  int64_t rows = src, k = 1;
  const int32_t* order = nullptr;
  if (a[1] != Py_None) {
    const at::Tensor& slots = tensor(a[2], "routing.slots", x);
    k = slots.dim() == 2 ? slots.size(1) : 0;
    rows = src * k;
    order = plain<int32_t>(a[1], "routing.order", kI32, {rows}, x);
  }
  const Current current(x);
  Pieces pieces(Pieces::room(rows * K) + Pieces::room(blocks(K) * rows * 4), x);
  at::Tensor q = pieces.take({rows, K}, kE4m3), s = pieces.take({blocks(K), rows}, kF32);
  check_rc(ag_fp8_quantize_rows(rows, K, type, x.data_ptr(), ld, src, order, static_cast<int>(k), q.data_ptr(),
                                static_cast<float*>(s.data_ptr()), stream_of(x)));
  return tuple_of(q, s);
  AGG_END
}

// quantize_weights(w) -> codes, scales
PyObject* quantize_weights(PyObject*, PyObject* const* a, Py_ssize_t n) {
  AGG_BEGIN
  check_args(n, 1);
  const at::Tensor& w = tensor(a[0], "w");
  const int type = float_type(w, "w");
  if ((w.dim() != 2 && w.dim() != 3) || !w.is_contiguous())
    raise(PyExc_ValueError, "w must be a contiguous (E, K, N) or (K, N) tensor");
  const bool many = w.dim() == 3;
  const int64_t E = many ? w.size(0) : 1, K = w.size(-2), N = w.size(-1);
  const Current current(w);
  at::Tensor q = make({E, N, K}, kE4m3, w), s = make({E, blocks(N), blocks(K)}, kF32, w);
  if (E > AG_MOE_MAX_EXPERTS) raise(PyExc_ValueError, "w has too many experts");
  check_rc(ag_fp8_quantize_weights(static_cast<int>(E), K, N, type, w.data_ptr(), q.data_ptr(),
                                   static_cast<float*>(s.data_ptr()), stream_of(w)));
  if (!many) {
    q = q.squeeze(0);
    s = s.squeeze(0);
  }
  return tuple_of(q, s);
  AGG_END
}

// What a product needs of its plan: (handle, experts, K, N), and its outputs.
struct PlanArgs {
  ag_moe_plan* plan;
  int64_t E, K, N;
};
PlanArgs plan_args(PyObject* const* a) { return {to_plan(a[0]), to_int(a[1]), to_int(a[2]), to_int(a[3])}; }

// A product's first tensor, on its plan's device.
const at::Tensor& tensor(PyObject* o, const char* name, const PlanArgs& p) {
  const at::Tensor& t = tensor(o, name);
  const int64_t device = check_rc(ag_moe_plan_device(p.plan));
  if (t.device().index() != device)
    raise(PyExc_ValueError, "%s is on device %s, the plan on cuda:%d", name, t.device().str().c_str(),
          static_cast<int>(device));
  return t;
}

const int32_t* offsets_of(PyObject* o, int64_t E, const at::Tensor& first) {
  return o == Py_None ? nullptr : plain<int32_t>(o, "offsets", kI32, {E + 1}, first);
}

at::ScalarType dtype_of(PyObject* o) {
  if (!THPDtype_Check(o)) raise(PyExc_TypeError, "out_dtype must be a torch.dtype");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

at::Tensor output(PyObject* o, at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
  if (o == Py_None) return make(shape, type, like);
  const at::Tensor& t = tensor(o, "out", like);
  want_type(t, "out", type);
  want_shape(t, "out", shape);
  return t;
}

// rows_product(handle, E, K, N, dtype, input_gradient, x or dy, offsets, w, out, out_dtype)
PyObject* rows_product(PyObject*, PyObject* const* a, Py_ssize_t n) {
  AGG_BEGIN
  check_args(n, 11);
  const PlanArgs p = plan_args(a);
  const at::ScalarType type = dtype_of(a[4]);
  const bool back = a[5] == Py_True;
  const char* name = back ? "dy" : "x";
  const at::Tensor& x = tensor(a[6], name, p);
  want_type(x, name, type);
  const int64_t ld = pitch(x, name, back ? p.N : p.K), rows = x.size(0), wide = back ? p.K : p.N;
  const int32_t* off = offsets_of(a[7], p.E, x);
  const at::Tensor& w = tensor(a[8], "w", x);
  want_type(w, "w", type);
  want_shape(w, "w", {p.E, p.K, p.N});
  int64_t ldw = p.N, ldw_e = p.K * p.N;
  if (!w.is_contiguous()) {
    if (w.stride(2) != 1) raise(PyExc_ValueError, "w must have contiguous rows");
    ldw = w.stride(1);
    ldw_e = w.stride(0);
  }
  const at::ScalarType ot = a[10] == Py_None ? type : dtype_of(a[10]);
  const Current current(x);
  at::Tensor out = output(a[9], {rows, wide}, ot, x);
  const int64_t ldo = pitch(out, "out");
  check_rc((back ? ag_moe_backward_input : ag_moe_forward)(p.plan, rows, x.data_ptr(), ld, off, w.data_ptr(), ldw,
                                                          ldw_e, out.data_ptr(), ldo, type_code(ot),
                                                          stream_of(x)));
  return wrap(out);
  AGG_END
}

// weight_product(handle, E, K, N, dtype, x, dy, offsets, out, out_dtype)
PyObject* weight_product(PyObject*, PyObject* const* a, Py_ssize_t n) {
  AGG_BEGIN
  check_args(n, 10);
  const PlanArgs p = plan_args(a);
  const at::ScalarType type = dtype_of(a[4]);
  const at::Tensor &x = tensor(a[5], "x", p), &dy = tensor(a[6], "dy", x);
  want_type(x, "x", type);
  want_type(dy, "dy", type);
  const int64_t ldx = pitch(x, "x", p.K), ldd = pitch(dy, "dy", p.N), rows = x.size(0);
  if (dy.size(0) != rows)
    raise(PyExc_ValueError, "x and dy must have the same rows, got %lld and %lld", static_cast<long long>(rows),
          static_cast<long long>(dy.size(0)));
  const int32_t* off = offsets_of(a[7], p.E, x);
  const at::ScalarType ot = dtype_of(a[9]);
  const Current current(x);
  at::Tensor out = output(a[8], {p.E, p.K, p.N}, ot, x);
  if (!out.is_contiguous()) raise(PyExc_ValueError, "out must be contiguous");
  check_rc(ag_moe_backward_weight(p.plan, rows, x.data_ptr(), ldx, dy.data_ptr(), ldd, off, out.data_ptr(),
                                  type_code(ot), stream_of(x)));
  return wrap(out);
  AGG_END
}

// fp8_product(handle, E, K, N, xq, xs, wq, ws, offsets, out, out_dtype)
PyObject* fp8_product(PyObject*, PyObject* const* a, Py_ssize_t n) {
  AGG_BEGIN
  check_args(n, 11);
  const PlanArgs p = plan_args(a);
  const at::Tensor &x = tensor(a[4], "xq", p), &w = tensor(a[6], "wq", x);
  const int64_t rows = x.dim() > 0 ? x.size(0) : 0, kb = blocks(p.K), nb = blocks(p.N);
  const void* xq = plain(a[4], "xq", kE4m3, {rows, p.K}, x);
  const float* xs = plain<float>(a[5], "xs", kF32, {kb, rows}, x);
  const void* wq;
  const float* ws;
  if (p.E == 1 && w.dim() == 2) {
    wq = plain(a[6], "wq", kE4m3, {p.N, p.K}, x);
    ws = plain<float>(a[7], "ws", kF32, {nb, kb}, x);
  } else {
    wq = plain(a[6], "wq", kE4m3, {p.E, p.N, p.K}, x);
    ws = plain<float>(a[7], "ws", kF32, {p.E, nb, kb}, x);
  }
  const int32_t* off = offsets_of(a[8], p.E, x);
  const at::ScalarType ot = dtype_of(a[10]);
  const Current current(x);
  at::Tensor out = output(a[9], {rows, p.N}, ot, x);
  const int64_t ldo = pitch(out, "out");
  check_rc(ag_fp8_forward(p.plan, rows, xq, xs, off, wq, ws, out.data_ptr(), ldo, type_code(ot), stream_of(x)));
  return wrap(out);
  AGG_END
}

#define AGG_METHOD(f) \
  { #f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {AGG_METHOD(init),         AGG_METHOD(route),         AGG_METHOD(route_backward),
                         AGG_METHOD(gather),       AGG_METHOD(combine),       AGG_METHOD(combine_backward),
                         AGG_METHOD(quantize_rows), AGG_METHOD(quantize_weights), AGG_METHOD(rows_product),
                         AGG_METHOD(weight_product), AGG_METHOD(fp8_product),  {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_front", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__front() {
  PyObject* m = PyModule_Create(&module);
  // the torch whose objects it reaches into
  if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) != 0) Py_CLEAR(m);
  return m;
}
