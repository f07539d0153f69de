// Tensor arguments of the row operators, products and the router's
// gradient: a CPython module that checks each torch tensor (device, type,
// shape, contiguity, no gradient to record; ValueError otherwise) and calls the
// C ABI with its address.  The same checks in Python cost 0.4 us a tensor, more than half of
// a small call (nine tensors against a launch of 2.7 us); here about 0.03.
//
// The module holds no library of its own: bind() takes the addresses of the
// entry points of the loaded libmoe355.so.
#include <Python.h>

#include <initializer_list>
#include <string>

#include <c10/core/GradMode.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "moe355.h"

namespace {

struct Entry {
  decltype(&moe_sort_workspace_bytes) sort_ws;
  decltype(&moe_sort_tokens) sort;
  decltype(&moe_sort_tokens_backward) sort_grad;
  decltype(&moe_unsort_combine) unsort;
  decltype(&moe_unsort_combine_backward) unsort_grad;
  decltype(&moe_linear_bytes) linear_bytes;
  decltype(&moe_linear_int4) linear;
  decltype(&moe_expert_linear_int4) expert_linear;
  decltype(&moe_pool_linear_int4) pool_linear;
  decltype(&moe_router_topk_backward) router_grad;
  decltype(&moe_linear) product;
  decltype(&moe_linear_backward) product_grad;
  decltype(&moe_gated) gated;
  decltype(&moe_gated_backward) gated_grad;
  decltype(&moe_quantize_fp8) quantize;
  decltype(&moe_linear_fp8) product_fp8;
} g;

using Shape = std::initializer_list<int64_t>;
constexpr at::ScalarType kF32 = at::kFloat, kI32 = at::kInt, kU8 = at::kByte, kBf16 = at::kBFloat16;

// The error, when thrown, is set already.
struct PyError {};

std::string text(c10::IntArrayRef v) {
  std::string s = "(";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + (v.size() == 1 ? ",)" : ")");
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_ValueError, "%s: a device tensor is wanted", name);
    throw PyError{};
  }
  return THPVariable_Unpack(o);
}

// The calls record nothing for autograd: a tensor whose gradient or tangent
// would be lost without a word is refused.  The backward calls are there for
// torch.autograd.Function, whose forward and backward run without grad mode.
void no_gradient(const at::Tensor& v, const char* name) {
  const bool tangent = v._fw_grad(0).defined();
  if (!tangent && !(v.requires_grad() && c10::GradMode::is_enabled())) return;
  PyErr_Format(PyExc_ValueError, "%s: carries a %s, which this call does not record; detach it, or call under "
               "torch.no_grad() or from a torch.autograd.Function",
               name, tangent ? "forward-mode tangent" : "gradient (requires_grad)");
  throw PyError{};
}

// The address of a contiguous tensor of that type and shape on device dev.
void* need(const at::Tensor& v, const char* name, at::ScalarType type, Shape shape, int dev) {
  const c10::IntArrayRef want(shape.begin(), shape.size());
  if (!v.is_cuda() || v.get_device() != dev || v.scalar_type() != type || v.sizes() != want || !v.is_contiguous()) {
    PyErr_Format(PyExc_ValueError, "%s: a contiguous %s tensor of shape %s on cuda:%d wanted, got %s %s on %s, strides %s",
                 name, c10::toString(type), text(want).c_str(), dev, c10::toString(v.scalar_type()),
                 text(v.sizes()).c_str(), v.device().str().c_str(), text(v.strides()).c_str());
    throw PyError{};
  }
  no_gradient(v, name);
  return v.data_ptr();
}
template <class T>
T* need(PyObject* o, const char* name, at::ScalarType type, Shape shape, int dev) {
  return static_cast<T*>(need(tensor(o, name), name, type, shape, dev));
}
// None passes as null.
template <class T>
T* may(PyObject* o, const char* name, at::ScalarType type, Shape shape, int dev) {
  return o == Py_None ? nullptr : need<T>(o, name, type, shape, dev);
}

// A matrix [rows][cols] whose sizes and type name those of the other arguments.
const at::Tensor& matrix(PyObject* o, const char* name, int* dev, bool rows_type) {
  const at::Tensor& v = tensor(o, name);
  const at::ScalarType t = v.scalar_type();
  if (!v.is_cuda() || v.dim() != 2 || (rows_type && t != kF32 && t != kBf16 && t != at::kHalf)) {
    PyErr_Format(PyExc_ValueError, "%s: a 2-d device tensor%s wanted, got %s %s on %s", name,
                 rows_type ? " of float32, bfloat16 or float16" : "", c10::toString(t), text(v.sizes()).c_str(),
                 v.device().str().c_str());
    throw PyError{};
  }
  *dev = v.get_device();
  return v;
}
int type_code(at::ScalarType t) { return t == kF32 ? MOE_TYPE_F32 : t == kBf16 ? MOE_TYPE_BF16 : MOE_TYPE_F16; }

int size32(int64_t v, const char* name) {
  if (v > INT32_MAX) {
    PyErr_Format(PyExc_ValueError, "%s: %lld is past 2^31 - 1", name, (long long)v);
    throw PyError{};
  }
  return (int)v;
}
int64_t number(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyError{};
  return v;
}
int number32(PyObject* o, const char* name) {
  const int64_t v = number(o);
  if (v < INT32_MIN) return size32(INT64_MAX, name);
  return size32(v, name);
}
void* address(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (p == nullptr && PyErr_Occurred()) throw PyError{};
  return p;
}

// The tensors' device as the current one for the call, and its current stream.
class On {
 public:
  explicit On(int dev) : back_(c10::hip::current_device()) {
    if (back_ == dev)
      back_ = -1;
    else
      c10::hip::set_device((c10::DeviceIndex)dev);
    stream = c10::hip::getCurrentHIPStream((c10::DeviceIndex)dev).stream();
  }
  ~On() {
    if (back_ < 0) return;
    try {
      c10::hip::set_device((c10::DeviceIndex)back_);
    } catch (...) {                             // the next device call reports it
    }
  }
  On(const On&) = delete;
  hipStream_t stream;

 private:
  int back_;
};
uint8_t* workspace(PyObject* o, int dev, size_t* bytes) {
  const at::Tensor& v = tensor(o, "workspace");
  uint8_t* p = static_cast<uint8_t*>(need(v, "workspace", kU8, {v.numel()}, dev));
  *bytes = (size_t)v.numel();
  return p;
}

// One entry point: body(args) gives the status; C++ exceptions stay inside.
template <int N, class F>
PyObject* entry(PyObject* const* a, Py_ssize_t n, F body) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments wanted, got %zd", N, n);
    return nullptr;
  }
  try {
    return PyLong_FromLong(body(a));
  } catch (const PyError&) {
    return nullptr;
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// x, topk_idx, E, x_sorted, offsets, pair_ids, row_of, workspace
PyObject* py_sort(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry<8>(args, n, [](PyObject* const* a) {
    int dev, dev2;
    const at::Tensor& x = matrix(a[0], "x", &dev, true);
    const at::ScalarType t = x.scalar_type();
    const int64_t T = x.size(0), d = x.size(1), k = matrix(a[1], "topk_idx", &dev2, false).size(1), E = number32(a[2], "E");
    size_t nws;
    uint8_t* ws = workspace(a[7], dev, &nws);
    const On on(dev);
    return g.sort(need(x, "x", t, {T, d}, dev), type_code(t), size32(T, "T"), size32(d, "d"),
                  need<int32_t>(a[1], "topk_idx", kI32, {T, k}, dev), size32(k, "k"), (int)E,
                  need<void>(a[3], "x_sorted", t, {T * k, d}, dev), need<int32_t>(a[4], "offsets", kI32, {E + 1}, dev),
                  need<int32_t>(a[5], "pair_ids", kI32, {T * k}, dev), need<int32_t>(a[6], "row_of", kI32, {T, k}, dev),
                  ws, nws, on.stream);
  });
}

// dx_sorted, row_of, dx
PyObject* py_sort_grad(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry<3>(args, n, [](PyObject* const* a) {
    int dev, dev2;
    const at::Tensor& x = matrix(a[0], "dx_sorted", &dev, true);
    const at::Tensor& r = matrix(a[1], "row_of", &dev2, false);
    const at::ScalarType t = x.scalar_type();
    const int64_t T = r.size(0), k = r.size(1), d = x.size(1);
    const On on(dev);
    return g.sort_grad(need(x, "dx_sorted", t, {T * k, d}, dev), type_code(t), size32(T, "T"), size32(k, "k"),
                       size32(d, "d"), static_cast<int32_t*>(need(r, "row_of", kI32, {T, k}, dev)),
                       need<void>(a[2], "out", t, {T, d}, dev), on.stream);
  });
}

// rows, row_of, topk_w, shared_out, shared_gate, y
PyObject* py_unsort(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry<6>(args, n, [](PyObject* const* a) {
    int dev, dev2;
    const at::Tensor& x = matrix(a[0], "rows", &dev, true);
    const at::Tensor& r = matrix(a[1], "row_of", &dev2, false);
    const at::ScalarType t = x.scalar_type();
    const int64_t T = r.size(0), k = r.size(1), d = x.size(1);
    const On on(dev);
    return g.unsort(need(x, "rows", t, {T * k, d}, dev), type_code(t), size32(T, "T"), size32(k, "k"), size32(d, "d"),
                    static_cast<int32_t*>(need(r, "row_of", kI32, {T, k}, dev)),
                    need<float>(a[2], "topk_w", kF32, {T, k}, dev), may<void>(a[3], "shared_out", t, {T, d}, dev),
                    may<float>(a[4], "shared_gate", kF32, {T}, dev), need<void>(a[5], "out", t, {T, d}, dev),
                    on.stream);
  });
}

// dy, rows, row_of, topk_w, shared_out, shared_gate, drows, dtopk_w, dshared_out, dshared_gate
PyObject* py_unsort_grad(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry<10>(args, n, [](PyObject* const* a) {
    int dev, dev2;
    const at::Tensor& x = matrix(a[1], "rows", &dev, true);
    const at::Tensor& r = matrix(a[2], "row_of", &dev2, false);
    const at::ScalarType t = x.scalar_type();
    const int64_t T = r.size(0), k = r.size(1), d = x.size(1);
    const On on(dev);
    return g.unsort_grad(need<void>(a[0], "dy", t, {T, d}, dev), need(x, "rows", t, {T * k, d}, dev), type_code(t),
                         size32(T, "T"), size32(k, "k"), size32(d, "d"),
                         static_cast<int32_t*>(need(r, "row_of", kI32, {T, k}, dev)),
                         need<float>(a[3], "topk_w", kF32, {T, k}, dev), may<void>(a[4], "shared_out", t, {T, d}, dev),
                         may<float>(a[5], "shared_gate", kF32, {T}, dev),
                         need<void>(a[6], "drows", t, {T * k, d}, dev), need<float>(a[7], "dtopk_w", kF32, {T, k}, dev),
                         may<void>(a[8], "dshared_out", t, {T, d}, dev),
                         may<float>(a[9], "dshared_gate", kF32, {T}, dev), on.stream);
  });
}

// packed, x, n_out, group, y
PyObject* py_linear(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry<5>(args, n, [](PyObject* const* a) {
    int dev;
    const at::Tensor& x = matrix(a[1], "x", &dev, false);
    const int64_t T = x.size(0), n_in = x.size(1);
    const moe_linear_shape sh{size32(n_in, "n_in"), number32(a[2], "n_out"), number32(a[3], "group")};
    const On on(dev);
    return g.linear(&sh, need<void>(a[0], "packed", kU8, {(int64_t)g.linear_bytes(&sh)}, dev),
                    static_cast<uint16_t*>(need(x, "x", kBf16, {T, n_in}, dev)), size32(T, "T"),
                    need<float>(a[4], "out", kF32, {T, sh.n_out}, dev), on.stream);
  });
}

// packed, slot_table, x_sorted, offsets, n_out, group, y, error
PyObject* py_expert_linear(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry<8>(args, n, [](PyObject* const* a) {
    int dev, dev2;
    const at::Tensor& x = matrix(a[2], "x_sorted", &dev, false);
    const at::Tensor& w = matrix(a[0], "packed", &dev2, false);
    const int64_t N = x.size(0), n_in = x.size(1), E = tensor(a[3], "offsets").numel() - 1;
    const moe_linear_shape sh{size32(n_in, "n_in"), number32(a[4], "n_out"), number32(a[5], "group")};
    const int64_t bytes = (int64_t)g.linear_bytes(&sh);
    if (w.scalar_type() != kU8 || dev2 != dev || w.stride(1) != 1 || w.size(1) < bytes ||
        (w.size(0) > 1 && w.stride(0) < bytes)) {
      PyErr_Format(PyExc_ValueError, "packed: a uint8 tensor [n_slots, %lld] on cuda:%d wanted, got %s %s on %s",
                   (long long)bytes, dev, c10::toString(w.scalar_type()), text(w.sizes()).c_str(),
                   w.device().str().c_str());
      throw PyError{};
    }
    const size_t stride = w.size(0) > 1 ? (size_t)w.stride(0) : ((size_t)bytes + 3) / 4 * 4;
    const On on(dev);
    return g.expert_linear(&sh, w.data_ptr(), stride, size32(w.size(0), "n_slots"),
                           may<int32_t>(a[1], "slot_table", kI32, {E}, dev), size32(E, "E"),
                           static_cast<uint16_t*>(need(x, "x_sorted", kBf16, {N, n_in}, dev)), size32(N, "N"),
                           need<int32_t>(a[3], "offsets", kI32, {E + 1}, dev),
                           need<float>(a[6], "out", kF32, {N, sh.n_out}, dev),
                           may<int32_t>(a[7], "error", kI32, {1}, dev), on.stream);
  });
}

// pool handle, matrix, n_in, n_out, E, x_sorted, offsets, y
PyObject* py_pool_linear(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry<8>(args, n, [](PyObject* const* a) {
    int dev;
    const at::Tensor& x = matrix(a[5], "x_sorted", &dev, false);
    const int64_t N = x.size(0), n_in = number(a[2]), n_out = number(a[3]), E = number(a[4]);
    const On on(dev);
    return g.pool_linear((const moe_pool*)address(a[0]), number32(a[1], "matrix"),
                         static_cast<uint16_t*>(need(x, "x_sorted", kBf16, {N, n_in}, dev)), size32(N, "N"),
                         need<int32_t>(a[6], "offsets", kI32, {E + 1}, dev),
                         need<float>(a[7], "out", kF32, {N, n_out}, dev), on.stream);
  });
}

// x, w_router, topk_idx, topk_w, shared_gate, dtopk_w, dshared_gate, offsets, pair_ids, dx, dw_router, dlogit_bias,
// workspace
PyObject* py_router_grad(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry<13>(args, n, [](PyObject* const* a) {
    int dev, dev2;
    const at::Tensor& x = matrix(a[0], "x", &dev, false);
    const at::Tensor& W = matrix(a[1], "w_router", &dev2, false);
    const at::Tensor& idx = matrix(a[2], "topk_idx", &dev2, false);
    const int64_t T = x.size(0), d = x.size(1), E = W.size(0) - 1, k = idx.size(1);
    size_t nws;
    uint8_t* ws = workspace(a[12], dev, &nws);
    const On on(dev);
    return g.router_grad(
        static_cast<uint16_t*>(need(x, "x", kBf16, {T, d}, dev)), size32(T, "T"), size32(d, "d"),
        static_cast<float*>(need(W, "w_router", kF32, {E + 1, d}, dev)), size32(E, "E"), size32(k, "k"),
        static_cast<int32_t*>(need(idx, "topk_idx", kI32, {T, k}, dev)), need<float>(a[3], "topk_w", kF32, {T, k}, dev),
        may<float>(a[4], "shared_gate", kF32, {T}, dev), need<float>(a[5], "dtopk_w", kF32, {T, k}, dev),
        may<float>(a[6], "dshared_gate", kF32, {T}, dev), may<int32_t>(a[7], "offsets", kI32, {E + 1}, dev),
        may<int32_t>(a[8], "pair_ids", kI32, {T * k}, dev), may<float>(a[9], "dx", kF32, {T, d}, dev),
        may<float>(a[10], "dw_router", kF32, {E + 1, d}, dev), may<float>(a[11], "dlogit_bias", kF32, {E}, dev), ws, nws,
        on.stream);
  });
}

// Matrices [n_out][n_in] of one type: 2-d, or (with offsets) 3-d [E][n_out][n_in],
// each contiguous, the experts' at any distance.
struct Matrices {
  void* p;
  int E;
  int64_t n_out, n_in;
  size_t stride;                // bytes
};
Matrices matrices(PyObject* o, const char* name, at::ScalarType type, bool experts, int dev) {
  const at::Tensor& v = tensor(o, name);
  const int dim = experts ? 3 : 2;
  if (!v.is_cuda() || v.get_device() != dev || v.scalar_type() != type || v.dim() != dim ||
      (v.size(dim - 1) > 1 && v.stride(dim - 1) != 1) || (v.size(dim - 2) > 1 && v.stride(dim - 2) != v.size(dim - 1)) ||
      (experts && v.size(0) > 1 && v.stride(0) < v.size(1) * v.size(2))) {
    PyErr_Format(PyExc_ValueError, "%s: a %s tensor %s of contiguous matrices on cuda:%d wanted, got %s %s on %s, strides %s",
                 name, c10::toString(type), experts ? "[E, n_out, n_in]" : "[n_out, n_in]", dev,
                 c10::toString(v.scalar_type()), text(v.sizes()).c_str(), v.device().str().c_str(),
                 text(v.strides()).c_str());
    throw PyError{};
  }
  no_gradient(v, name);
  Matrices m{v.data_ptr(), 1, v.size(dim - 2), v.size(dim - 1), 0};
  m.stride = (size_t)(m.n_out * m.n_in) * v.element_size();
  if (experts) {
    m.E = size32(v.size(0), "E");
    if (m.E > 1) m.stride = (size_t)v.stride(0) * v.element_size();
  }
  return m;
}
// m has the sizes of w.
void same(const Matrices& m, const char* name, const Matrices& w) {
  if (m.E == w.E && m.n_out == w.n_out && m.n_in == w.n_in) return;
  PyErr_Format(PyExc_ValueError, "%s: %d matrices of %lld x %lld wanted, got %d of %lld x %lld", name, w.E, (long long)w.n_out,
               (long long)w.n_in, m.E, (long long)m.n_out, (long long)m.n_in);
  throw PyError{};
}
// Matrices of those sizes: an output or a second input; None passes as null.
Matrices like(PyObject* o, const char* name, at::ScalarType type, bool experts, int dev, int E, int64_t n_out, int64_t n_in) {
  if (o == Py_None) return Matrices{nullptr, E, n_out, n_in, 0};
  const Matrices m = matrices(o, name, type, experts, dev);
  same(m, name, Matrices{nullptr, E, n_out, n_in, 0});
  return m;
}
// Matrices that a call uses for an output alone that it does not write (no `use`):
// may be None, with the sizes of the output that it does.
Matrices unless_unused(PyObject* o, const char* name, bool use, const Matrices& sizes, at::ScalarType type, bool experts, int dev) {
  if (o == Py_None && !use) return Matrices{nullptr, sizes.E, sizes.n_out, sizes.n_in, 0};
  return matrices(o, name, type, experts, dev);
}
at::ScalarType type_of(PyObject* o, const char* name) { return tensor(o, name).scalar_type(); }
int32_t* borders(PyObject* o, int E, int dev) { return may<int32_t>(o, "offsets", kI32, {E + 1}, dev); }

// w, x, offsets, y
PyObject* py_product(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry<4>(args, n, [](PyObject* const* a) {
    int dev;
    const at::Tensor& x = matrix(a[1], "x", &dev, true);
    const at::ScalarType t = x.scalar_type(), ty = type_of(a[3], "out");
    const bool experts = a[2] != Py_None;
    const Matrices w = matrices(a[0], "w", t, experts, dev);
    const int64_t N = x.size(0);
    const On on(dev);
    return g.product(w.p, w.stride, w.E, need(x, "x", t, {N, w.n_in}, dev), type_code(t), size32(N, "N"),
                     size32(w.n_in, "n_in"), size32(w.n_out, "n_out"), borders(a[2], w.E, dev),
                     need<void>(a[3], "out", ty == kF32 ? kF32 : t, {N, w.n_out}, dev), type_code(ty == kF32 ? kF32 : t), on.stream);
  });
}

// dy, w, x, offsets, dx, dw (w None without dx, x None without dw)
PyObject* py_product_grad(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry<6>(args, n, [](PyObject* const* a) {
    int dev;
    const at::Tensor& dy = matrix(a[0], "dy", &dev, true);
    const bool for_x = a[4] != Py_None, for_w = a[5] != Py_None, experts = a[3] != Py_None;
    const at::ScalarType t = dy.scalar_type(), td = for_w && type_of(a[5], "dw") == kF32 ? kF32 : t;
    Matrices dw{};
    if (for_w) dw = matrices(a[5], "dw", td, experts, dev);
    const Matrices w = unless_unused(a[1], "w", for_x || !for_w, dw, t, experts, dev);
    if (for_w) same(dw, "dw", w);
    const int64_t N = dy.size(0);
    const On on(dev);
    return g.product_grad(need(dy, "dy", t, {N, w.n_out}, dev), w.p, w.stride, w.E,
                          for_w ? need<void>(a[2], "x", t, {N, w.n_in}, dev) : may<void>(a[2], "x", t, {N, w.n_in}, dev),
                          type_code(t), size32(N, "N"), size32(w.n_in, "n_in"), size32(w.n_out, "n_out"),
                          borders(a[3], w.E, dev), may<void>(a[4], "dx", t, {N, w.n_in}, dev), dw.p, dw.stride,
                          type_code(td), on.stream);
  });
}

// w_gate, w_up, x, offsets, act, h, pre
PyObject* py_gated(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry<7>(args, n, [](PyObject* const* a) {
    int dev;
    const at::Tensor& x = matrix(a[2], "x", &dev, true);
    const at::ScalarType t = x.scalar_type();
    const bool experts = a[3] != Py_None;
    const Matrices wg = matrices(a[0], "w_gate", t, experts, dev);
    const Matrices wu = like(a[1], "w_up", t, experts, dev, wg.E, wg.n_out, wg.n_in);
    const int64_t N = x.size(0), I = wg.n_out;
    const On on(dev);
    return g.gated(wg.p, wg.stride, wu.p, wu.stride, wg.E, need(x, "x", t, {N, wg.n_in}, dev), type_code(t), size32(N, "N"),
                   size32(wg.n_in, "d"), size32(I, "I"), borders(a[3], wg.E, dev), number32(a[4], "act"),
                   need<void>(a[5], "h", t, {N, I}, dev), may<float>(a[6], "pre", kF32, {N, 2 * I}, dev), on.stream);
  });
}

// dh, pre, w_gate, w_up, x, offsets, act, dx, dw_gate, dw_up, workspace (both w
// None without dx, x None without the gradients of matrices)
PyObject* py_gated_grad(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry<11>(args, n, [](PyObject* const* a) {
    int dev;
    const at::Tensor& dh = matrix(a[0], "dh", &dev, true);
    const bool for_x = a[7] != Py_None, for_w = a[8] != Py_None, experts = a[5] != Py_None;
    const at::ScalarType t = dh.scalar_type(), td = for_w && type_of(a[8], "dw_gate") == kF32 ? kF32 : t;
    Matrices dg{};
    if (for_w) dg = matrices(a[8], "dw_gate", td, experts, dev);
    const Matrices wg = unless_unused(a[2], "w_gate", for_x || !for_w, dg, t, experts, dev);
    if (for_w) same(dg, "dw_gate", wg);
    const Matrices wu = unless_unused(a[3], "w_up", for_x || !for_w, dg, t, experts, dev);
    same(wu, "w_up", wg);
    const int64_t N = dh.size(0), I = wg.n_out, d = wg.n_in;
    const Matrices du = like(a[9], "dw_up", td, experts, dev, wg.E, I, d);
    size_t nws;
    uint8_t* ws = workspace(a[10], dev, &nws);
    const On on(dev);
    return g.gated_grad(need(dh, "dh", t, {N, I}, dev), need<float>(a[1], "pre", kF32, {N, 2 * I}, dev), wg.p, wg.stride, wu.p,
                        wu.stride, wg.E, for_w ? need<void>(a[4], "x", t, {N, d}, dev) : may<void>(a[4], "x", t, {N, d}, dev),
                        type_code(t), size32(N, "N"), size32(d, "d"), size32(I, "I"), borders(a[5], wg.E, dev),
                        number32(a[6], "act"), may<void>(a[7], "dx", t, {N, d}, dev), dg.p, dg.stride, du.p, du.stride,
                        type_code(td), ws, nws, on.stream);
  });
}

// x [rows][n] or [count][rows][n], block_rows, codes, scales
PyObject* py_quantize(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry<4>(args, n, [](PyObject* const* a) {
    const at::Tensor& x = tensor(a[0], "x");
    const at::ScalarType t = x.scalar_type();
    if (!x.is_cuda() || (x.dim() != 2 && x.dim() != 3) || (t != kF32 && t != kBf16 && t != at::kHalf)) {
      PyErr_Format(PyExc_ValueError, "x: a 2-d or 3-d device tensor of float32, bfloat16 or float16 wanted, got %s %s on %s",
                   c10::toString(t), text(x.sizes()).c_str(), x.device().str().c_str());
      throw PyError{};
    }
    const int dev = x.get_device();
    const bool batch = x.dim() == 3;
    const int64_t count = batch ? x.size(0) : 1, rows = x.size(-2), cols = x.size(-1);
    const int br = number32(a[1], "block_rows");
    const int64_t rb = br == 128 ? (rows + 127) / 128 : rows, cb = (cols + 127) / 128;
    const On on(dev);
    void *px, *pc, *ps;
    if (batch) {
      px = need(x, "x", t, {count, rows, cols}, dev);
      pc = need<void>(a[2], "codes", at::kFloat8_e4m3fn, {count, rows, cols}, dev);
      ps = need<void>(a[3], "scales", kF32, {count, rb, cb}, dev);
    } else {
      px = need(x, "x", t, {rows, cols}, dev);
      pc = need<void>(a[2], "codes", at::kFloat8_e4m3fn, {rows, cols}, dev);
      ps = need<void>(a[3], "scales", kF32, {rb, cb}, dev);
    }
    return g.quantize(px, type_code(t), size32(count, "count"), size32(rows, "rows"), size32(cols, "n"), br, pc,
                      static_cast<float*>(ps), on.stream);
  });
}

// w, w_scales, x, x_scales, offsets, y
PyObject* py_product_fp8(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry<6>(args, n, [](PyObject* const* a) {
    int dev, dev2;
    const at::Tensor& x = matrix(a[2], "x", &dev, false);
    const at::ScalarType ty = matrix(a[5], "out", &dev2, true).scalar_type();
    const bool experts = a[4] != Py_None;
    const Matrices w = matrices(a[0], "w", at::kFloat8_e4m3fn, experts, dev);
    const int64_t N = x.size(0), rb = (w.n_out + 127) / 128, cb = (w.n_in + 127) / 128;
    const Matrices ws = like(a[1], "w_scales", kF32, experts, dev, w.E, rb, cb);
    if (!ws.p && N > 0) {
      PyErr_SetString(PyExc_ValueError, "w_scales: a device tensor is wanted");
      throw PyError{};
    }
    const On on(dev);
    return g.product_fp8(w.p, w.stride, static_cast<float*>(ws.p), ws.stride / sizeof(float), w.E,
                         need(x, "x", at::kFloat8_e4m3fn, {N, w.n_in}, dev), need<float>(a[3], "x_scales", kF32, {N, cb}, dev),
                         size32(N, "N"), size32(w.n_in, "n_in"), size32(w.n_out, "n_out"), borders(a[4], w.E, dev),
                         need<void>(a[5], "out", ty, {N, w.n_out}, dev), type_code(ty), on.stream);
  });
}

constexpr int kEntries = sizeof(Entry) / sizeof(void*);
PyObject* py_bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry<kEntries>(args, n, [](PyObject* const* a) {
    void** to = reinterpret_cast<void**>(&g);
    for (int i = 0; i < kEntries; ++i) to[i] = address(a[i]);
    return 0;
  });
}
static_assert(sizeof(Entry) == 16 * sizeof(void*), "one address an entry point");

#define METHOD(name, f) {name, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    METHOD("bind", py_bind),           METHOD("sort", py_sort),
    METHOD("sort_grad", py_sort_grad), METHOD("unsort", py_unsort),
    METHOD("unsort_grad", py_unsort_grad), METHOD("linear", py_linear),
    METHOD("expert_linear", py_expert_linear), METHOD("pool_linear", py_pool_linear),
    METHOD("router_grad", py_router_grad), METHOD("product", py_product),
    METHOD("product_grad", py_product_grad), METHOD("gated", py_gated),
    METHOD("gated_grad", py_gated_grad), METHOD("quantize", py_quantize),
    METHOD("product_fp8", py_product_fp8), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_rowops", "Tensor arguments of the row operators.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__rowops() { return PyModule_Create(&module); }
