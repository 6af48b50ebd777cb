// Python entry of the vocabulary operators: checks the tensors of a call, allocates its
// outputs and calls the C ABI on the current stream. It is what vocab.py's functions call;
// the arguments come by position, as that file passes them. A call costs about 4 us of
// host time, most of it the launch; the same checks in Python over ctypes cost 15.
#include <Python.h>
#include <ATen/ATen.h>
#include <c10/core/GradMode.h>
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

// A 2-D CUDA tensor whose rows are contiguous.
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
    if (cols > 1 && x.stride(1) != 1) refuse("the rows of %s must be contiguous", name);
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
at::Tensor empty(at::IntArrayRef size, at::ScalarType type, int device) {
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

int64_t row_bytes(int64_t cols) { return (cols + 31) / 32 * 16; }
int64_t scale_tiles(int64_t cols, int format) { return ((cols + 31) / 32 * (format == EMB_MICRO_MX ? 1 : 2) + 3) / 4; }

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
    codes = vector<uint8_t>(a[0], device, at::kByte, rows * row_bytes(cols), name);
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
      codes = empty({x.rows, row_bytes(x.cols)}, at::kByte, dev);
      scales = empty({(x.rows + 127) / 128, scale_tiles(x.cols, format), 32, 4, 4}, at::kByte, dev);
    } else {
      codes = target(a[3], "out"), scales = target(a[4], "out");
      vector<uint8_t>(a[3], dev, at::kByte, x.rows * row_bytes(x.cols), "codes of out");
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

// EmbError, then the addresses of the library's functions in the order of Library.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* f[7];
  if (n != 8) return PyErr_Format(PyExc_TypeError, "expected 8 arguments");
  for (int i = 0; i < 7; ++i)
    if (!(f[i] = PyLong_AsVoidPtr(a[i + 1]))) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "no function");
  Py_INCREF(a[0]);
  Py_XDECREF(emb_error);
  emb_error = a[0];
  lib = {reinterpret_cast<decltype(lib.logits_process)>(f[0]),   reinterpret_cast<decltype(lib.distill_forward)>(f[1]),
         reinterpret_cast<decltype(lib.distill_backward)>(f[2]), reinterpret_cast<decltype(lib.distill_step)>(f[3]),
         reinterpret_cast<decltype(lib.micro_quantize)>(f[4]),   reinterpret_cast<decltype(lib.micro_lookup)>(f[5]),
         reinterpret_cast<decltype(lib.micro_matmul)>(f[6])};
  Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind),           FAST(process_logits), FAST(distill_forward), FAST(distill_backward),
                         FAST(distill_step),   FAST(micro_quantize), FAST(micro_lookup),    FAST(micro_matmul),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_vocab", "Entry of the vocabulary operators (see vocab.py).", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__vocab() { return PyModule_Create(&module); }
