// The calls of ops128.py with nothing unusual about them, marshalled in C++:
// the same checks, output tensors and C entry points in 4 to 6 us a call where
// Python and ctypes take 11 to 17 (a single token's norm runs for 2 us, a few
// tokens' GEMM for 4). Each function returns None for any call that it does not
// take (another device than the current one, a tensor subclass, an argument
// that is refused, an empty tensor): Python then makes the call, or raises. A
// status other than MX_OK comes back as an int. The outputs come from torch's
// CUDA allocator past its dispatcher: dispatch modes do not see them made, and
// torch.utils.deterministic does not fill them.

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

namespace {

using Quantize = int (*)(const void*, int, int64_t, int64_t, int64_t, int, int, void*, int64_t,
                         float*, int64_t, void*, int64_t, float*, int64_t, void*);
using Norm = int (*)(const void*, int64_t, const void*, const void*, int, int64_t, int64_t, float,
                     int, int, void*, void*, void*, int64_t, float*, int64_t, void*);
using NormBwd = int (*)(const void*, const void*, const void*, const void*, int, int64_t, int64_t,
                        float, void*, float*, void*, void*);
using Workspace = int64_t (*)(int64_t, int64_t);
using Gemm = int (*)(const void*, int64_t, const float*, int64_t, int, const void*, int64_t,
                     const float*, int64_t, int, int, int64_t, int64_t, int64_t, int, void*, int*,
                     void*);

Quantize quantize_fn;
Norm norm_fn;
NormBwd norm_bwd_fn;
Workspace workspace_fn;
Gemm gemm_fn;

constexpr int kBlock128 = 1 << 10, kPow2 = 1 << 11;

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// A plain CUDA tensor on the current device (dev: found, or -1 to begin with),
// whose memory holds its values.
const at::Tensor* tensor(PyObject* o, int& dev) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.layout() != at::kStrided || t.is_neg()) return nullptr;
  const int d = t.get_device();
  if (dev < 0) {
    if (d != c10::cuda::current_device()) return nullptr;
    dev = d;
  }
  return d == dev ? &t : nullptr;
}

int dtype_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return 0;
    case at::kHalf: return 1;
    case at::kFloat: return 2;
    default: return -1;
  }
}

// Row pitch of a nonempty [rows, cols] matrix with contiguous rows, else -1.
int64_t matrix_pitch(const at::Tensor& t) {
  if (t.dim() != 2 || t.size(0) == 0 || t.size(1) == 0) return -1;
  if (t.size(1) > 1 && t.stride(1) != 1) return -1;
  if (t.size(0) == 1) return t.size(1);
  return t.stride(0) >= t.size(1) ? t.stride(0) : -1;
}

bool same(const at::Tensor& t, const at::Tensor& like) {
  return t.scalar_type() == like.scalar_type() && t.sizes() == like.sizes() && t.is_contiguous();
}

int64_t codes_pitch(const at::Tensor& t) {
  if (t.scalar_type() != at::kByte || t.dim() != 2) return -1;
  const int64_t rows = t.size(0), cols = t.size(1), need = up(cols, 16);
  if (rows == 0 || cols == 0 || (cols > 1 && t.stride(1) != 1)) return -1;
  const int64_t pitch = rows > 1 ? t.stride(0) : need;
  if (pitch < need || pitch % 16 != 0) return -1;
  return t.storage_offset() + (rows - 1) * pitch + need <= static_cast<int64_t>(t.storage().nbytes())
             ? pitch : -1;
}

int64_t scales_pitch(const at::Tensor& t, int64_t rows, int64_t cols, bool block) {
  const int64_t nb = (cols + 127) / 128;
  if (t.scalar_type() != at::kFloat || t.dim() != 2 || t.size(1) != nb ||
      t.size(0) != (block ? (rows + 127) / 128 : rows))
    return -1;
  if (block) return t.is_contiguous() ? 4 : -1;
  const int64_t need = up(rows, 4), pitch = nb > 1 ? t.stride(1) : need;
  if ((rows > 1 && t.stride(0) != 1) || pitch < need || pitch % 4 != 0) return -1;
  return (t.storage_offset() + (nb - 1) * pitch + need) * 4 <= static_cast<int64_t>(t.storage().nbytes())
             ? pitch : -1;
}

at::Tensor empty(at::IntArrayRef size, at::ScalarType type, int dev) {
  return at::detail::empty_cuda(size, type, c10::Device(c10::kCUDA, static_cast<int8_t>(dev)), std::nullopt);
}

// A new tensor takes other sizes and strides within its storage directly
// (narrow() would cost 1 us).
void as_view(at::Tensor& t, at::IntArrayRef sizes, at::IntArrayRef strides) {
  t.unsafeGetTensorImpl()->set_sizes_and_strides(sizes, strides);
}

at::Tensor new_codes(int64_t rows, int64_t cols, int dev, int64_t& pitch) {
  pitch = up(cols, 16);
  at::Tensor t = empty({rows, pitch}, at::kByte, dev);
  if (pitch != cols) as_view(t, {rows, cols}, {pitch, 1});
  return t;
}

at::Tensor new_scales(int64_t rows, int64_t cols, bool block, int dev, int64_t& pitch) {
  const int64_t nb = (cols + 127) / 128;
  pitch = 4;
  if (block) return empty({(rows + 127) / 128, nb}, at::kFloat, dev);
  pitch = up(rows, 4);
  at::Tensor t = empty({nb, pitch}, at::kFloat, dev);
  as_view(t, {rows, nb}, {1, pitch});
  return t;
}

void* stream(int dev) { return c10::cuda::getCurrentCUDAStream(dev).stream(); }

PyObject* none() { Py_RETURN_NONE; }

// Whether an argument was not the number it should be (Python then says so).
bool bad_number() {
  if (!PyErr_Occurred()) return false;
  PyErr_Clear();
  return true;
}

PyObject* steal(PyObject* tuple, int i, PyObject* o) {
  PyTuple_SET_ITEM(tuple, i, o);
  return tuple;
}

PyObject* none_ref() {
  Py_INCREF(Py_None);
  return Py_None;
}

// C++ exceptions (the allocator's, for one) become Python ones.
template <class F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (...) {
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

// (x, format, block, direction 1 rows | 2 cols, pow2)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5) return none();
  return guarded([&]() -> PyObject* {
    int dev = -1;
    const at::Tensor* x = tensor(a[0], dev);
    if (!x) return none();
    const int64_t ldx = matrix_pitch(*x);
    const int dt = dtype_of(*x);
    if (ldx < 0 || dt < 0) return none();
    const int format = static_cast<int>(PyLong_AsLong(a[1]));
    const bool block = a[2] == Py_True;
    const int way = static_cast<int>(PyLong_AsLong(a[3]));
    if (bad_number()) return none();
    const int64_t rows = x->size(0), cols = x->size(1);
    at::Tensor codes, scales, codes_t, scales_t;
    int64_t ldc = 0, lds = 0, ldct = 0, ldst = 0;
    if (way & 1) {
      codes = new_codes(rows, cols, dev, ldc);
      scales = new_scales(rows, cols, block, dev, lds);
    }
    if (way & 2) {
      codes_t = new_codes(cols, rows, dev, ldct);
      scales_t = new_scales(cols, rows, block, dev, ldst);
    }
    const int st = quantize_fn(
        x->data_ptr(), dt, rows, cols, ldx, format, (block ? kBlock128 : 0) | (a[4] == Py_True ? kPow2 : 0),
        way & 1 ? codes.data_ptr() : nullptr, ldc, way & 1 ? scales.data_ptr<float>() : nullptr, lds,
        way & 2 ? codes_t.data_ptr() : nullptr, ldct, way & 2 ? scales_t.data_ptr<float>() : nullptr,
        ldst, stream(dev));
    if (st != 0) return PyLong_FromLong(st);
    PyObject* r = PyTuple_New(way == 3 ? 4 : 2);
    int i = 0;
    if (way & 1) {
      steal(r, i++, THPVariable_Wrap(std::move(codes)));
      steal(r, i++, THPVariable_Wrap(std::move(scales)));
    }
    if (way & 2) {
      steal(r, i++, THPVariable_Wrap(std::move(codes_t)));
      steal(r, i++, THPVariable_Wrap(std::move(scales_t)));
    }
    return r;
  });
}

// (x, weight, residual or None, eps, format, pow2, return_y)
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 7) return none();
  return guarded([&]() -> PyObject* {
    int dev = -1;
    const at::Tensor* x = tensor(a[0], dev);
    if (!x) return none();
    const at::Tensor* w = tensor(a[1], dev);
    const at::Tensor* res = a[2] == Py_None ? nullptr : tensor(a[2], dev);
    if (!w || (a[2] != Py_None && !res)) return none();
    const int64_t ldx = matrix_pitch(*x);
    const int dt = dtype_of(*x);
    if (ldx < 0 || dt < 0) return none();
    const int64_t rows = x->size(0), cols = x->size(1);
    if (w->scalar_type() != x->scalar_type() || w->dim() != 1 || w->size(0) != cols ||
        !w->is_contiguous())
      return none();
    if (res && !same(*res, *x)) return none();
    const double eps = PyFloat_AsDouble(a[3]);
    const int format = static_cast<int>(PyLong_AsLong(a[4]));
    const bool return_y = a[6] == Py_True;
    if (bad_number()) return none();
    int64_t ldc = 0, lds = 0;
    at::Tensor codes = new_codes(rows, cols, dev, ldc);
    at::Tensor scales = new_scales(rows, cols, false, dev, lds);
    at::Tensor h, y;
    if (res) h = empty({rows, cols}, x->scalar_type(), dev);
    if (return_y) y = empty({rows, cols}, x->scalar_type(), dev);
    const int st = norm_fn(x->data_ptr(), ldx, res ? res->data_ptr() : nullptr, w->data_ptr(), dt, rows,
                           cols, static_cast<float>(eps), format, a[5] == Py_True ? kPow2 : 0,
                           res ? h.data_ptr() : nullptr, return_y ? y.data_ptr() : nullptr,
                           codes.data_ptr(), ldc, scales.data_ptr<float>(), lds, stream(dev));
    if (st != 0) return PyLong_FromLong(st);
    PyObject* r = PyTuple_New(4);
    steal(r, 0, THPVariable_Wrap(std::move(codes)));
    steal(r, 1, THPVariable_Wrap(std::move(scales)));
    steal(r, 2, res ? THPVariable_Wrap(std::move(h)) : none_ref());
    steal(r, 3, return_y ? THPVariable_Wrap(std::move(y)) : none_ref());
    return r;
  });
}

// (grad_y, h, weight, eps, grad_residual or None)
PyObject* norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5) return none();
  return guarded([&]() -> PyObject* {
    int dev = -1;
    const at::Tensor* h = tensor(a[1], dev);
    if (!h) return none();
    const at::Tensor* gy = tensor(a[0], dev);
    const at::Tensor* w = tensor(a[2], dev);
    const at::Tensor* gres = a[4] == Py_None ? nullptr : tensor(a[4], dev);
    if (!gy || !w || (a[4] != Py_None && !gres)) return none();
    const int dt = dtype_of(*h);
    if (dt < 0 || h->dim() != 2 || h->numel() == 0 || !h->is_contiguous()) return none();
    const int64_t rows = h->size(0), cols = h->size(1);
    const double eps = PyFloat_AsDouble(a[3]);
    if (bad_number()) return none();
    if (!same(*gy, *h) || (gres && !same(*gres, *h)) || w->scalar_type() != h->scalar_type() ||
        w->dim() != 1 || w->size(0) != cols || !w->is_contiguous())
      return none();
    at::Tensor gh = empty({rows, cols}, h->scalar_type(), dev);
    at::Tensor gw = empty({cols}, at::kFloat, dev);
    at::Tensor work = empty({workspace_fn(rows, cols)}, at::kByte, dev);
    const int st = norm_bwd_fn(gy->data_ptr(), h->data_ptr(), w->data_ptr(),
                               gres ? gres->data_ptr() : nullptr, dt, rows, cols,
                               static_cast<float>(eps), gh.data_ptr(),
                               gw.data_ptr<float>(), work.data_ptr(), stream(dev));
    if (st != 0) return PyLong_FromLong(st);
    PyObject* r = PyTuple_New(2);
    steal(r, 0, THPVariable_Wrap(std::move(gh)));
    return steal(r, 1, THPVariable_Wrap(std::move(gw)));
  });
}

// (a_codes, a_scales, b_codes, b_scales, a_format, b_format, out_fp32)
PyObject* gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 7) return none();
  return guarded([&]() -> PyObject* {
    int dev = -1;
    const at::Tensor* ac = tensor(a[0], dev);
    if (!ac) return none();
    const at::Tensor* as = tensor(a[1], dev);
    const at::Tensor* bc = tensor(a[2], dev);
    const at::Tensor* bs = tensor(a[3], dev);
    if (!as || !bc || !bs) return none();
    const int64_t lda = codes_pitch(*ac), ldb = codes_pitch(*bc);
    if (lda < 0 || ldb < 0 || ac->size(1) != bc->size(1)) return none();
    const int64_t M = ac->size(0), N = bc->size(0), K = ac->size(1);
    const bool block = bs->dim() == 2 && bs->size(0) == (N + 127) / 128 && (N > 1 || bs->is_contiguous());
    const int64_t ldsa = scales_pitch(*as, M, K, false), ldsb = scales_pitch(*bs, N, K, block);
    if (ldsa < 0 || ldsb < 0) return none();
    const int fa = static_cast<int>(PyLong_AsLong(a[4])), fb = static_cast<int>(PyLong_AsLong(a[5]));
    const bool fp32 = a[6] == Py_True;
    if (bad_number()) return none();
    at::Tensor d = empty({M, N}, fp32 ? at::kFloat : at::kBFloat16, dev);
    const int st = gemm_fn(ac->data_ptr(), lda, as->data_ptr<float>(), ldsa, fa, bc->data_ptr(), ldb,
                           bs->data_ptr<float>(), ldsb, fb, block ? kBlock128 : 0, M, N, K, fp32,
                           d.data_ptr(), nullptr, stream(dev));
    return st != 0 ? PyLong_FromLong(st) : THPVariable_Wrap(std::move(d));
  });
}

// The addresses of mx_quantize128, mx_rms_norm_quant128, mx_rms_norm_bwd,
// mx_rms_norm_bwd_workspace and mx_gemm128.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "bind takes five addresses");
    return nullptr;
  }
  void* p[5];
  for (int i = 0; i < 5; ++i) p[i] = PyLong_AsVoidPtr(a[i]);
  if (PyErr_Occurred()) return nullptr;
  quantize_fn = reinterpret_cast<Quantize>(p[0]);
  norm_fn = reinterpret_cast<Norm>(p[1]);
  norm_bwd_fn = reinterpret_cast<NormBwd>(p[2]);
  workspace_fn = reinterpret_cast<Workspace>(p[3]);
  gemm_fn = reinterpret_cast<Gemm>(p[4]);
  return none();
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(quantize), FAST(norm), FAST(norm_bwd), FAST(gemm), FAST(bind),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast128", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast128(void) { return PyModule_Create(&module); }
