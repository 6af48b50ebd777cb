// Python entry of the vocabulary operators: checks the tensors of a call, allocates its
// outputs and calls the C ABI on the current stream. It is what vocab.py's functions call;
// the arguments come by position, as that file passes them. A call costs about 4 us of
// host time, most of it the launch; the same checks in Python over ctypes cost 15.
#include <Python.h>
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/record_function.h>
#include <c10/core/GradMode.h>
#include <c10/core/impl/LocalDispatchKeySet.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/embbwd.h"

namespace {

struct Library {
  decltype(&emb_logits_process) logits_process;
  decltype(&emb_distill_forward) distill_forward;
  decltype(&emb_distill_backward) distill_backward;
  decltype(&emb_distill_step) distill_step;
  decltype(&emb_micro_quantize) micro_quantize;
  decltype(&emb_micro_lookup) micro_lookup;
  decltype(&emb_micro_matmul) micro_matmul;
  decltype(&emb_rms_norm_forward) rms_norm_forward;
  decltype(&emb_rms_norm_workspace) rms_norm_workspace;
  decltype(&emb_rms_norm_backward) rms_norm_backward;
  decltype(&emb_dropout) dropout;
  decltype(&emb_cross_entropy_workspace) cross_entropy_workspace;
  decltype(&emb_cross_entropy_forward) cross_entropy_forward;
  decltype(&emb_cross_entropy_backward) cross_entropy_backward;
  decltype(&emb_cross_entropy_step) cross_entropy_step;
} lib;
PyObject* emb_error = nullptr;  // embbwd.EmbError

// A refusal, raised as a Python exception where the entry point returns.
struct Refused {};
template <typename... A>
[[noreturn]] void refuse(const char* format, A... a) {
  PyErr_Format(PyExc_ValueError, format, a...);
  throw Refused{};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse("%s must be a tensor", name);
  return THPVariable_Unpack(o);
}

// A caller's tensor that the call writes to. Autograd's rules for operations in place hold: no
// leaf that takes a gradient (nor a view of one) while gradients are recorded, and a new
// version, so that a backward that saved the old values raises.
const at::Tensor& target(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (c10::GradMode::is_enabled() && t.requires_grad() && (t.is_leaf() || (t.is_view() && t._base().is_leaf())))
    refuse("%s is a leaf (or a view of one) that requires a gradient: it cannot be written in place", name);
  return t;
}
void written(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

int dtype_code(at::ScalarType t) {
  return t == at::kFloat ? EMB_F32 : t == at::kHalf ? EMB_F16 : t == at::kBFloat16 ? EMB_BF16 : -1;
}

// A 2-D CUDA tensor whose rows, if there are any, are contiguous.
struct Matrix {
  at::Tensor t;
  int64_t rows, cols, stride;
  emb_dtype dtype;
  int device;
  Matrix(const at::Tensor& x, const char* name) : t(x) {
    if (x.dim() != 2 || !x.is_cuda()) refuse("%s must be a 2-D CUDA tensor", name);
    const int code = dtype_code(x.scalar_type());
    if (code < 0) refuse("%s must be float32, float16 or bfloat16", name);
    rows = x.size(0), cols = x.size(1), stride = x.stride(0);
    if (rows > 0 && cols > 1 && x.stride(1) != 1) refuse("the rows of %s must be contiguous", name);
    dtype = (emb_dtype)code, device = x.get_device();
  }
  Matrix(PyObject* o, const char* name) : Matrix(tensor(o, name), name) {}
  void* ptr() const { return t.data_ptr(); }
  void wants(int64_t r, int64_t c, int d, const char* name) const {
    if (rows != r || cols != c || device != d) refuse("%s must be a [%lld, %lld] tensor on cuda:%d", name, (long long)r, (long long)c, d);
  }
};

template <typename T>
T* vector(PyObject* o, int device, at::ScalarType type, int64_t n, const char* name) {
  if (o == Py_None) return nullptr;
  const at::Tensor& x = tensor(o, name);
  if (x.scalar_type() != type || !x.is_cuda() || x.get_device() != device || x.numel() != n || !x.is_contiguous())
    refuse("%s must be a contiguous %s tensor of %lld elements on cuda:%d", name, c10::toString(type), (long long)n, device);
  return static_cast<T*>(x.data_ptr());
}

uint32_t* status_word(PyObject* o, int device) {
  if (o == Py_None) return nullptr;
  const at::ScalarType t = tensor(o, "status").scalar_type();
  return vector<uint32_t>(o, device, t == at::kUInt32 ? t : at::kInt, 1, "status");
}

struct Csr {
  const int64_t *ids = nullptr, *offsets = nullptr;
  int64_t n = 0;
  PyObject* values = nullptr;
  Csr(PyObject* o, int device, int64_t B, int parts, const char* name) {
    if (o == Py_None) return;
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != parts) refuse("%s must be a tuple of %d tensors", name, parts);
    n = tensor(PyTuple_GET_ITEM(o, 0), name).numel();
    ids = vector<int64_t>(PyTuple_GET_ITEM(o, 0), device, at::kLong, n, name);
    offsets = vector<int64_t>(PyTuple_GET_ITEM(o, 1), device, at::kLong, B + 1, name);
    if (parts > 2) values = PyTuple_GET_ITEM(o, 2);
  }
};

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  return v;
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return (float)v;
}
int32_t size32(int64_t n, const char* name) {
  if (n > INT32_MAX) refuse("%s has too many rows or columns", name);
  return (int32_t)n;
}
at::ScalarType type_of(PyObject* o) {
  if (!THPDtype_Check(o)) refuse("dtype must be a torch.dtype");
  const at::ScalarType t = reinterpret_cast<THPDtype*>(o)->scalar_type;
  if (dtype_code(t) < 0) refuse("dtype must be float32, float16 or bfloat16");
  return t;
}
// Whether nothing between a call and the allocator has to see an allocation: no dispatch mode or transform, no
// profiler, and no program that wants uninitialised memory filled.
bool unseen() {
  const at::Context& c = at::globalContext();
  return (c10::impl::tls_local_dispatch_key_set().included_ - c10::default_included_set).empty() &&
         !at::getStepCallbacksUnlessEmpty(at::RecordScope::FUNCTION).has_value() &&
         !(c.deterministicAlgorithms() && c.deterministicFillUninitializedMemory());
}
// Then straight from the caching allocator: 0.3 us instead of 0.8 by the dispatcher (a norm of one row 5.0 us of host time instead of 6.5).
at::Tensor empty(at::IntArrayRef size, at::ScalarType type, int device) {
  if (unseen()) return at::Tensor(at::detail::empty_cuda(size, type, at::Device(at::kCUDA, device), std::nullopt));
  return at::empty(size, at::TensorOptions().dtype(type).device(at::kCUDA, device));
}
void* stream(int device) { return c10::cuda::getCurrentCUDAStream(device).stream(); }

// Raises embbwd.EmbError(status, name).
void check(emb_status st, const char* name) {
  if (st == EMB_OK) return;
  if (PyObject* e = PyObject_CallFunction(emb_error, "is", (int)st, name)) {
    PyErr_SetObject(emb_error, e);
    Py_DECREF(e);
  }
  throw Refused{};
}

// Runs an entry point's body: no C++ exception leaves it.
template <typename F>
PyObject* entry(Py_ssize_t given, Py_ssize_t wanted, F body) {
  if (given != wanted) return PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", wanted, given);
  if (!lib.logits_process) return PyErr_Format(PyExc_RuntimeError, "the library is not bound");
  try {
    return body();
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

PyObject* pair(at::Tensor a, at::Tensor b) {
  PyObject *x = THPVariable_Wrap(std::move(a)), *y = THPVariable_Wrap(std::move(b));
  PyObject* r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return r;
}

// logits, prompt, output, repetition, frequency, presence, bias, mask, out, dtype, status
PyObject* process_logits(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 11, [&] {
    const Matrix z(a[0], "logits");
    const int dev = z.device;
    const int32_t B = size32(z.rows, "logits"), V = size32(z.cols, "logits");
    const Csr p(a[1], dev, B, 2, "prompt"), o(a[2], dev, B, 2, "output"), b(a[6], dev, B, 3, "bias");
    const float* values = b.values ? vector<float>(b.values, dev, at::kFloat, b.n, "bias values") : nullptr;
    const float* rep = vector<float>(a[3], dev, at::kFloat, B, "repetition");
    const float* freq = vector<float>(a[4], dev, at::kFloat, B, "frequency");
    const float* pres = vector<float>(a[5], dev, at::kFloat, B, "presence");
    const uint32_t* mask = nullptr;
    int64_t mask_stride = 0;
    if (a[7] != Py_None) {
      const at::Tensor& m = tensor(a[7], "mask");
      if (m.dim() != 2 || (m.scalar_type() != at::kInt && m.scalar_type() != at::kUInt32) || !m.is_cuda() ||
          m.get_device() != dev || m.size(0) != B || m.size(1) < (V + 31) / 32 || (m.size(1) > 1 && m.stride(1) != 1))
        refuse("mask must be an int32 [%d, %d] tensor on cuda:%d", B, (V + 31) / 32, dev);
      mask = static_cast<const uint32_t*>(m.data_ptr()), mask_stride = m.stride(0);
    }
    const at::ScalarType type = a[9] == Py_None ? z.t.scalar_type() : type_of(a[9]);
    const Matrix y(a[8] == Py_None ? empty({B, V}, type, dev) : target(a[8], "out"), "out");
    y.wants(B, V, dev, "out");
    if (a[9] != Py_None && y.t.scalar_type() != type) refuse("out has another type than dtype");
    check(lib.logits_process(dev, z.ptr(), z.dtype, z.stride, B, V, p.ids, p.offsets, p.n, o.ids, o.offsets, o.n, rep,
                             freq, pres, b.ids, b.offsets, values, b.n, mask, mask_stride, y.ptr(), y.dtype, y.stride,
                             status_word(a[10], dev), stream(dev)),
          "emb_logits_process");
    written(y.t);
    return THPVariable_Wrap(y.t);
  });
}

// What the distillation calls share.
struct Rows {
  Matrix z, t;
  const int64_t* ids;
  int32_t N, V, K;
  Rows(PyObject* logits, PyObject* teacher_ids, PyObject* teacher)
      : z(logits, "logits"), t(teacher, "teacher_logits") {
    const at::Tensor& i = tensor(teacher_ids, "teacher_ids");
    if (i.scalar_type() != at::kLong || !i.is_cuda() || i.get_device() != z.device || i.dim() != 2 ||
        i.size(0) != z.rows || t.device != z.device || t.rows != z.rows || i.size(1) != t.cols)
      refuse("teacher_ids (int64) and teacher_logits must be [%lld, K] tensors on cuda:%d", (long long)z.rows, z.device);
    if ((t.cols > 1 && i.stride(1) != 1) || (z.rows > 1 && i.stride(0) != t.stride))
      refuse("teacher_ids and teacher_logits must have contiguous rows and the same row stride");
    ids = static_cast<const int64_t*>(i.data_ptr());
    N = size32(z.rows, "logits"), V = size32(z.cols, "logits"), K = size32(t.cols, "teacher_logits");
  }
  const float* of_rows(PyObject* o, int per_row, const char* name) const {
    return vector<float>(o, z.device, at::kFloat, (int64_t)N * per_row, name);
  }
  // The gradient's tensor: `out`, or a new one. Its rows are contiguous but for what puts them
  // at the same places in 16 bytes as the logits' (a new tensor starts at such a boundary):
  // then the kernels load whole pieces. The logits' own stride may be that of a whole sequence.
  Matrix gradient(PyObject* out) const {
    const int64_t piece = 16 / (int64_t)z.t.element_size();
    const bool alike = N > 1 && z.stride > V && reinterpret_cast<uintptr_t>(z.ptr()) % 16 == 0;
    const int64_t stride = V + (alike ? (z.stride - V) % piece : 0);
    const Matrix g(out == Py_None ? at::empty_strided({N, V}, {stride, 1}, z.t.options()) : target(out, "out"), "out");
    g.wants(N, V, z.device, "out");
    if (g.dtype != z.dtype) refuse("out must have the type of logits");
    return g;
  }
};

// logits, teacher_ids, teacher_logits, temperature, teacher_lse, status
PyObject* distill_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 6, [&] {
    const Rows r(a[0], a[1], a[2]);
    const int dev = r.z.device;
    at::Tensor loss = empty({r.N}, at::kFloat, dev), stats = empty({r.N, 4}, at::kFloat, dev);
    check(lib.distill_forward(dev, r.z.ptr(), r.z.dtype, r.z.stride, r.N, r.V, r.ids, r.t.ptr(), r.t.dtype, r.t.stride,
                              r.K, r.of_rows(a[4], 1, "teacher_lse"), real(a[3]), static_cast<float*>(loss.data_ptr()),
                              static_cast<float*>(stats.data_ptr()), status_word(a[5], dev), stream(dev)),
          "emb_distill_forward");
    return pair(std::move(loss), std::move(stats));
  });
}

// logits, teacher_ids, teacher_logits, stats, row_weight, temperature, out, status
PyObject* distill_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 8, [&] {
    const Rows r(a[0], a[1], a[2]);
    const int dev = r.z.device;
    const Matrix g = r.gradient(a[6]);
    check(lib.distill_backward(dev, r.z.ptr(), r.z.dtype, r.z.stride, r.N, r.V, r.ids, r.t.ptr(), r.t.dtype, r.t.stride,
                               r.K, r.of_rows(a[3], 4, "stats"), r.of_rows(a[4], 1, "row_weight"), real(a[5]), g.ptr(),
                               g.stride, status_word(a[7], dev), stream(dev)),
          "emb_distill_backward");
    written(g.t);
    return THPVariable_Wrap(g.t);
  });
}

// logits, teacher_ids, teacher_logits, row_weight, temperature, teacher_lse, out, status
PyObject* distill_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 8, [&] {
    const Rows r(a[0], a[1], a[2]);
    const int dev = r.z.device;
    const Matrix g = r.gradient(a[6]);
    at::Tensor loss = empty({r.N}, at::kFloat, dev);
    check(lib.distill_step(dev, r.z.ptr(), r.z.dtype, r.z.stride, r.N, r.V, r.ids, r.t.ptr(), r.t.dtype, r.t.stride, r.K,
                           r.of_rows(a[5], 1, "teacher_lse"), r.of_rows(a[3], 1, "row_weight"), real(a[4]),
                           static_cast<float*>(loss.data_ptr()), g.ptr(), g.stride, status_word(a[7], dev), stream(dev)),
          "emb_distill_step");
    written(g.t);
    return pair(std::move(loss), g.t);
  });
}

int64_t row_bytes(int64_t cols, int format) { return (cols + 31) / 32 * (format == EMB_MICRO_MX8 ? 32 : 16); }
int64_t scale_tiles(int64_t cols, int format) { return ((cols + 31) / 32 * (format == EMB_MICRO_NV ? 2 : 1) + 3) / 4; }
// New codes and scales of a microscaled matrix.
void new_micro(int64_t rows, int64_t cols, int format, int device, at::Tensor* codes, at::Tensor* scales) {
  *codes = empty({rows, row_bytes(cols, format)}, at::kByte, device);
  *scales = empty({(rows + 127) / 128, scale_tiles(cols, format), 32, 4, 4}, at::kByte, device);
}

// A microscaled matrix as vocab.py passes it: codes, scales, rows, cols, format, tensor scale.
struct Micro {
  uint8_t *codes, *scales;
  int64_t rows, cols;
  emb_micro_format format;
  float g;
  int device;
  Micro(PyObject* const* a, const char* name) : rows(integer(a[2])), cols(integer(a[3])), g(real(a[5])) {
    format = (emb_micro_format)integer(a[4]);
    const at::Tensor& c = tensor(a[0], name);
    if (!c.is_cuda()) refuse("codes and scales of %s must be contiguous uint8 CUDA tensors on one device", name);
    if (rows < 0 || cols < 1) refuse("%s must have at least one column", name);
    device = c.get_device();
    codes = vector<uint8_t>(a[0], device, at::kByte, rows * row_bytes(cols, format), name);
    scales = vector<uint8_t>(a[1], device, at::kByte, (rows + 127) / 128 * scale_tiles(cols, format) * 512, name);
  }
};

// x, format, tensor_scale, codes, scales (both None: new ones)
PyObject* micro_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 5, [&] {
    const Matrix x(a[0], "x");
    const int format = (int)integer(a[1]), dev = x.device;
    if (x.cols < 1) refuse("x must have at least one column");
    at::Tensor codes, scales;
    if (a[3] == Py_None) {
      new_micro(x.rows, x.cols, format, dev, &codes, &scales);
    } else {
      codes = target(a[3], "out"), scales = target(a[4], "out");
      vector<uint8_t>(a[3], dev, at::kByte, x.rows * row_bytes(x.cols, format), "codes of out");
      vector<uint8_t>(a[4], dev, at::kByte, (x.rows + 127) / 128 * scale_tiles(x.cols, format) * 512, "scales of out");
    }
    check(lib.micro_quantize(dev, x.ptr(), x.dtype, x.stride, x.rows, size32(x.cols, "x"), (emb_micro_format)format,
                             real(a[2]), static_cast<uint8_t*>(codes.data_ptr()),
                             static_cast<uint8_t*>(scales.data_ptr()), stream(dev)),
          "emb_micro_quantize");
    written(codes);
    written(scales);
    return pair(std::move(codes), std::move(scales));
  });
}

// codes, scales, rows, cols, format, tensor_scale, ids, dtype, out, status
PyObject* micro_lookup(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 10, [&] {
    const Micro m(a, "table");
    const int64_t count = a[6] == Py_None ? m.rows : tensor(a[6], "ids").numel();
    const int64_t* ids = vector<int64_t>(a[6], m.device, at::kLong, count, "ids");
    const Matrix y(a[8] == Py_None ? empty({count, m.cols}, type_of(a[7]), m.device) : target(a[8], "out"), "out");
    y.wants(count, m.cols, m.device, "out");
    check(lib.micro_lookup(m.device, m.codes, m.scales, m.rows, size32(m.cols, "table"), m.format, m.g, ids, count, y.ptr(),
                           y.dtype, y.stride, status_word(a[9], m.device), stream(m.device)),
          "emb_micro_lookup");
    written(y.t);
    return THPVariable_Wrap(y.t);
  });
}

// x's and w's six values, dtype, out, status
PyObject* micro_matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 15, [&] {
    const Micro x(a, "x"), w(a + 6, "w");
    if (w.format != x.format || w.cols != x.cols || w.device != x.device)
      refuse("x and w must have the same format, columns and device");
    const int32_t M = size32(x.rows, "x"), N = size32(w.rows, "w");
    const Matrix y(a[13] == Py_None ? empty({M, N}, type_of(a[12]), x.device) : target(a[13], "out"), "out");
    y.wants(M, N, x.device, "out");
    check(lib.micro_matmul(x.device, x.codes, x.scales, x.g, M, w.codes, w.scales, w.g, N, size32(x.cols, "x"), x.format,
                           y.ptr(), y.dtype, y.stride, status_word(a[14], x.device), stream(x.device)),
          "emb_micro_matmul");
    written(y.t);
    return THPVariable_Wrap(y.t);
  });
}

// A matrix beside `like`: its type, shape and device.
Matrix beside(const Matrix& like, PyObject* o, const char* name, bool written_to = false) {
  const Matrix m(written_to ? target(o, name) : tensor(o, name), name);
  m.wants(like.rows, like.cols, like.device, name);
  if (m.dtype != like.dtype) refuse("%s must have the type of the rows", name);
  return m;
}
Matrix new_or(const Matrix& like, PyObject* o, const char* name) {
  return o == Py_None ? Matrix(empty({like.rows, like.cols}, like.t.scalar_type(), like.device), name)
                      : beside(like, o, name, true);
}
// Rows that may be absent.
struct Maybe {
  const void* p = nullptr;
  int64_t stride = 0;
  Maybe(const Matrix& like, PyObject* o, const char* name) {
    if (o == Py_None) return;
    const Matrix m = beside(like, o, name);
    p = m.ptr(), stride = m.stride;
  }
};
// The norm's weights, of a type of their own.
struct Weight {
  void* p = nullptr;
  emb_dtype dtype = EMB_F32;
  at::ScalarType type = at::kFloat;
  Weight(const Matrix& rows, PyObject* o) {
    if (o == Py_None) return;
    type = tensor(o, "weight").scalar_type();
    if (dtype_code(type) < 0) refuse("weight must be float32, float16 or bfloat16");
    dtype = (emb_dtype)dtype_code(type), p = vector<void>(o, rows.device, type, rows.cols, "weight");
  }
};

// x, weight, residual, eps, micro, out, sum_out -> (y, sum, rstd) or ((codes, scales), sum, None). Without a sum
// of its own the sum is x, or None where y has taken x's place.
PyObject* rms_norm_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 7, [&]() -> PyObject* {
    const Matrix x(a[0], "x");
    const int dev = x.device;
    const int32_t D = size32(x.cols, "x");
    if (D < 1) refuse("x must have at least one column");
    const Weight w(x, a[1]);
    const Maybe res(x, a[2], "residual");
    const bool micro = PyObject_IsTrue(a[4]);
    if (micro && a[5] != Py_None) refuse("out is for rows of x's type");
    at::Tensor rstd, codes, scales, y, sum;
    int64_t y_stride = 0, sum_stride = 0;
    if (micro) {
      new_micro(x.rows, x.cols, EMB_MICRO_MX8, dev, &codes, &scales);
    } else {
      const Matrix m = new_or(x, a[5], "out");
      y = m.t, y_stride = m.stride;
      rstd = empty({x.rows}, at::kFloat, dev);  // for the gradient, which codes do not have
    }
    if (a[2] != Py_None || a[6] != Py_None) {  // (rows that are none have no address)
      const Matrix m = new_or(x, a[6], "sum_out");
      sum = m.t, sum_stride = m.stride;
    }
    auto at_of = [](const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
    check(lib.rms_norm_forward(dev, x.ptr(), x.dtype, x.stride, x.rows, D, res.p, res.stride, w.p, w.dtype, real(a[3]),
                               at_of(y), y_stride, static_cast<uint8_t*>(at_of(codes)), static_cast<uint8_t*>(at_of(scales)),
                               at_of(sum), sum_stride, static_cast<float*>(at_of(rstd)), stream(dev)),
          "emb_rms_norm_forward");
    if (y.defined()) written(y);
    if (sum.defined()) written(sum);
    const bool gone = !sum.defined() && y.defined() && x.rows && y.data_ptr() == x.ptr();
    PyObject* first = micro ? pair(std::move(codes), std::move(scales)) : THPVariable_Wrap(std::move(y));
    if (gone) return Py_BuildValue("(NON)", first, Py_None, THPVariable_Wrap(std::move(rstd)));
    if (micro) return Py_BuildValue("(NNO)", first, THPVariable_Wrap(sum.defined() ? sum : x.t), Py_None);
    return Py_BuildValue("(NNN)", first, THPVariable_Wrap(sum.defined() ? sum : x.t), THPVariable_Wrap(std::move(rstd)));
  });
}

// grad, sum, weight, rstd, grad_sum, want_weight, out -> (gradient of the rows, of the weights or None)
PyObject* rms_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 7, [&]() -> PyObject* {
    const Matrix s(a[1], "sum"), g = beside(s, a[0], "grad");
    const int dev = s.device;
    const int32_t D = size32(s.cols, "sum");
    if (D < 1) refuse("sum must have at least one column");
    const Weight w(s, a[2]);
    const float* rstd = vector<float>(a[3], dev, at::kFloat, s.rows, "rstd");
    if (!rstd && s.rows) refuse("rstd must be given");
    const Maybe more(s, a[4], "grad_sum");
    const Matrix out = new_or(s, a[6], "out");
    at::Tensor dw, ws;
    int64_t bytes = 0;
    if (w.p && PyObject_IsTrue(a[5])) {
      bytes = lib.rms_norm_workspace(dev, s.rows, D);
      if (bytes < 0) refuse("sum has too many rows or columns");
      dw = empty({D}, w.type, dev), ws = empty({bytes}, at::kByte, dev);
    }
    check(lib.rms_norm_backward(dev, g.ptr(), s.dtype, g.stride, s.rows, D, s.ptr(), s.stride, w.p, w.dtype, rstd, more.p,
                                more.stride, out.ptr(), out.stride, dw.defined() ? dw.data_ptr() : nullptr,
                                ws.defined() ? ws.data_ptr() : nullptr, bytes, stream(dev)),
          "emb_rms_norm_backward");
    written(out.t);
    if (dw.defined()) return pair(out.t, std::move(dw));
    return Py_BuildValue("(NO)", THPVariable_Wrap(out.t), Py_None);
  });
}

uint64_t word64(PyObject* o, const char* name) {
  const unsigned long long v = PyLong_AsUnsignedLongLong(o);
  if (v == (unsigned long long)-1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse("%s must be an integer of 0 to 2^64 - 1", name);
  }
  return v;
}

// x, p, seed, call (an int or a tensor), residual, out
PyObject* dropout(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 6, [&] {
    const Matrix x(a[0], "x");
    const int dev = x.device;
    if (x.cols < 1) refuse("x must have at least one column");
    const double p = PyFloat_AsDouble(a[1]);
    if (p == -1.0 && PyErr_Occurred()) throw Refused{};
    if (!(p >= 0.0 && p < 1.0)) refuse("p must be at least 0 and below 1");
    const uint64_t seed = word64(a[2], "seed");
    const bool held = THPVariable_Check(a[3]);
    const int64_t* at = held ? vector<int64_t>(a[3], dev, at::kLong, 1, "call") : nullptr;
    const Maybe res(x, a[4], "residual");
    const Matrix y = new_or(x, a[5], "out");
    check(lib.dropout(dev, x.ptr(), x.dtype, x.stride, x.rows, size32(x.cols, "x"), res.p, res.stride, p, seed,
                      held ? 0 : word64(a[3], "call"), at, y.ptr(), y.stride, stream(dev)),
          "emb_dropout");
    written(y.t);
    return THPVariable_Wrap(y.t);
  });
}

// What the cross entropy calls share.
struct Tokens {
  Matrix h, w;
  const int64_t* targets;
  int32_t V, D;
  Tokens(PyObject* hidden, PyObject* table, PyObject* target) : h(hidden, "hidden"), w(table, "table") {
    if (h.dtype == EMB_F32) refuse("hidden must be float16 or bfloat16");
    if (w.dtype != h.dtype) refuse("table must have the type of hidden");
    if (w.cols != h.cols || w.device != h.device || w.rows < 1)
      refuse("table must be a [V, %lld] tensor on cuda:%d", (long long)h.cols, h.device);
    targets = vector<int64_t>(target, h.device, at::kLong, h.rows, "targets");
    if (!targets && h.rows) refuse("targets must be given");
    V = size32(w.rows, "table"), D = size32(h.cols, "hidden");
  }
  const float* of_rows(PyObject* o, const char* name) const { return vector<float>(o, h.device, at::kFloat, h.rows, name); }
  // From the caching allocator, for this call: on the call's stream, in a graph's own pool.
  at::Tensor workspace(bool gradients) const {
    const int64_t n = lib.cross_entropy_workspace(h.device, h.rows, V, D, w.ptr(), w.stride, gradients);
    if (n < 0) refuse("hidden or table has too many rows or columns");
    return empty({n}, at::kByte, h.device);
  }
};
// A gradient like `like`: new, or `out`; none where `want` is false.
struct Gradient {
  at::Tensor t;
  void* p = nullptr;
  int64_t stride = 0;
  Gradient(const Matrix& like, PyObject* want, PyObject* out, const char* name) {
    if (out == Py_None && !PyObject_IsTrue(want)) return;
    const Matrix g(out == Py_None ? empty({like.rows, like.cols}, like.t.scalar_type(), like.device) : target(out, name), name);
    g.wants(like.rows, like.cols, like.device, name);
    if (g.dtype != like.dtype) refuse("%s must have the type of hidden", name);
    t = g.t, p = g.ptr(), stride = g.stride;
  }
  PyObject* wrap() const {
    if (!t.defined()) Py_RETURN_NONE;
    written(t);
    return THPVariable_Wrap(t);
  }
};

// hidden, table, targets, status
PyObject* cross_entropy_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 4, [&] {
    const Tokens x(a[0], a[1], a[2]);
    const int dev = x.h.device;
    at::Tensor loss = empty({x.h.rows}, at::kFloat, dev), lse = empty({x.h.rows}, at::kFloat, dev), ws = x.workspace(false);
    check(lib.cross_entropy_forward(dev, x.h.ptr(), x.h.dtype, x.h.stride, x.h.rows, x.w.ptr(), x.w.stride, x.V, x.D,
                                    x.targets, static_cast<float*>(loss.data_ptr()), static_cast<float*>(lse.data_ptr()),
                                    ws.data_ptr(), ws.numel(), status_word(a[3], dev), stream(dev)),
          "emb_cross_entropy_forward");
    return pair(std::move(loss), std::move(lse));
  });
}

// hidden, table, targets, lse, row_weight, want_hidden, want_table, out_hidden, out_table, status
PyObject* cross_entropy_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 10, [&]() -> PyObject* {
    const Tokens x(a[0], a[1], a[2]);
    const int dev = x.h.device;
    if (a[3] == Py_None) refuse("lse must be given");
    const Gradient h(x.h, a[5], a[7], "out_hidden"), w(x.w, a[6], a[8], "out_table");
    if (!h.t.defined() && !w.t.defined()) refuse("no gradient is asked for");
    const float *lse = x.of_rows(a[3], "lse"), *weight = x.of_rows(a[4], "row_weight");
    uint32_t* const status = status_word(a[9], dev);
    if (x.h.rows > 0 || w.t.defined()) {  // else there is nothing to write, and the hidden states' gradient has no address
      const at::Tensor ws = x.workspace(true);
      check(lib.cross_entropy_backward(dev, x.h.ptr(), x.h.dtype, x.h.stride, x.h.rows, x.w.ptr(), x.w.stride, x.V, x.D,
                                       x.targets, lse, weight, h.p, h.stride, w.p, w.stride, ws.data_ptr(), ws.numel(),
                                       status, stream(dev)),
            "emb_cross_entropy_backward");
    }
    return Py_BuildValue("(NN)", h.wrap(), w.wrap());
  });
}

// hidden, table, targets, row_weight, out_hidden, out_table, status
PyObject* cross_entropy_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 7, [&]() -> PyObject* {
    const Tokens x(a[0], a[1], a[2]);
    const int dev = x.h.device;
    const Gradient h(x.h, Py_True, a[4], "out_hidden"), w(x.w, Py_True, a[5], "out_table");
    at::Tensor loss = empty({x.h.rows}, at::kFloat, dev), ws = x.workspace(true);
    check(lib.cross_entropy_step(dev, x.h.ptr(), x.h.dtype, x.h.stride, x.h.rows, x.w.ptr(), x.w.stride, x.V, x.D,
                                 x.targets, x.of_rows(a[3], "row_weight"), static_cast<float*>(loss.data_ptr()), h.p,
                                 h.stride, w.p, w.stride, ws.data_ptr(), ws.numel(), status_word(a[6], dev), stream(dev)),
          "emb_cross_entropy_step");
    return Py_BuildValue("(NNN)", THPVariable_Wrap(loss), h.wrap(), w.wrap());
  });
}

// EmbError, then the addresses of the library's functions in the order of Library.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr Py_ssize_t count = sizeof(Library) / sizeof(void*);
  void* f[count];
  if (n != count + 1) return PyErr_Format(PyExc_TypeError, "expected %zd arguments", count + 1);
  for (Py_ssize_t i = 0; i < count; ++i)
    if (!(f[i] = PyLong_AsVoidPtr(a[i + 1]))) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "no function");
  Py_INCREF(a[0]);
  Py_XDECREF(emb_error);
  emb_error = a[0];
  memcpy(&lib, f, sizeof lib);
  Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind),           FAST(process_logits), FAST(distill_forward), FAST(distill_backward),
                         FAST(distill_step),   FAST(micro_quantize), FAST(micro_lookup),    FAST(micro_matmul),
                         FAST(rms_norm_forward), FAST(rms_norm_backward), FAST(dropout),
                         FAST(cross_entropy_forward), FAST(cross_entropy_backward), FAST(cross_entropy_step),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_vocab", "Entry of the vocabulary operators (see vocab.py).", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__vocab() { return PyModule_Create(&module); }
