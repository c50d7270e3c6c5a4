// The host side of the 8-bit and log-probability calls for Python, without ctypes: checks, outputs
// and the library's call in one step. A decode call's kernel takes a few microseconds, and the call
// itself was the longer part: quantize_fp8 8.5 us, mm_fp8 9.6, mm_fp8_gated 11.2, token_logprobs 14.6
// through Python's checks, torch.empty and ctypes; here 4.4, 4.2, 4.3 and 6.2, of which the launch is
// 2.5 to 3.
//
// Each function takes exactly what the checks in __init__.py accept and answers None to all else, so
// that they say what is wrong; a status other than FI_OK comes back as a number. Outputs are made
// from the caching allocator of the inputs' device, on its current stream.
#include <Python.h>

#include <algorithm>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fi_nvfp4.h"

namespace {

constexpr int64_t kBlock = 128;  // k (and weight rows) per scale

decltype(&fi_fp8_quantize) quantize_fn, pack_fn;
decltype(&fi_mm_fp8_ex) mm_fn;
decltype(&fi_mm_fp8_gated_ex) gated_fn;
decltype(&fi_token_logprobs) logprobs_fn;

int64_t blocks(int64_t x) { return (x + kBlock - 1) / kBlock; }

// fi_dtype of bf16, f16 and fp32, else -1.
int code_of(at::ScalarType t) {
  return t == at::kBFloat16 ? FI_DTYPE_BF16 : t == at::kHalf ? FI_DTYPE_F16 : t == at::kFloat ? FI_DTYPE_F32 : -1;
}

// The tensor of `o` if it is one of CUDA memory, else null.
const at::Tensor* cuda_tensor(PyObject* o) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.defined() && t.is_cuda() && t.layout() == at::kStrided ? &t : nullptr;
}

const at::Tensor* dense(PyObject* o, at::ScalarType type, int64_t dims) {
  const at::Tensor* t = cuda_tensor(o);
  return t && t->scalar_type() == type && t->dim() == dims && t->is_contiguous() ? t : nullptr;
}

// Codes [r, k] and scales, one per `rows` rows and block of k, all on one device.
struct Operand {
  const at::Tensor *q, *s;
  int64_t r, k;
  bool get(PyObject* codes, PyObject* scale, int64_t rows) {
    q = dense(codes, at::kFloat8_e4m3fn, 2);
    s = q ? dense(scale, at::kFloat, 2) : nullptr;
    if (!s) return false;
    r = q->size(0);
    k = q->size(1);
    return s->size(0) == (r + rows - 1) / rows && s->size(1) == blocks(k) && s->get_device() == q->get_device();
  }
  const uint8_t* codes() const { return static_cast<const uint8_t*>(q->const_data_ptr()); }
  const float* scale() const { return static_cast<const float*>(s->const_data_ptr()); }
};

at::Tensor empty(at::IntArrayRef size, at::ScalarType type, int device) {
  return at::detail::empty_cuda(size, type, at::Device(at::kCUDA, (c10::DeviceIndex)device), std::nullopt);
}

// The output [m, n]: `out` if it is one that fits, a new one of `dtype` (or bf16) if it is None.
bool output(PyObject* out, PyObject* dtype, int64_t m, int64_t n, int device, at::Tensor* t) {
  if (dtype != Py_None && !THPDtype_Check(dtype)) return false;
  const at::ScalarType type = dtype == Py_None ? at::kBFloat16 : reinterpret_cast<THPDtype*>(dtype)->scalar_type;
  if (out == Py_None) {
    if (code_of(type) < 0) return false;
    *t = empty({m, n}, type, device);
    return true;
  }
  const at::Tensor* o = cuda_tensor(out);
  if (!o || code_of(o->scalar_type()) < 0 || (dtype != Py_None && o->scalar_type() != type) || o->dim() != 2 ||
      !o->is_contiguous() || o->size(0) != m || o->size(1) != n || o->get_device() != device)
    return false;
  *t = *o;
  return true;
}

// fn(current stream of `device`), with that device current and without the interpreter's lock.
template <typename F>
int call(int device, F fn) {
  const c10::cuda::OptionalCUDAGuard guard(at::Device(at::kCUDA, (c10::DeviceIndex)device));
  const fi_stream_t stream =
      reinterpret_cast<fi_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream());
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = fn(stream);
  Py_END_ALLOW_THREADS
  return rc;
}

// (x, square, codes, scale): activations or (square) weights to codes and scales, new ones for None.
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const at::Tensor* x = n == 4 ? cuda_tensor(a[0]) : nullptr;
  const int code = x ? code_of(x->scalar_type()) : -1;
  if (code < 0 || x->dim() != 2 || !x->is_contiguous()) Py_RETURN_NONE;
  const bool square = a[1] == Py_True;
  const int64_t rows = x->size(0), k = x->size(1), tall = square ? blocks(rows) : rows;
  const int device = x->get_device();
  at::Tensor q, s;
  if (a[2] == Py_None && a[3] == Py_None) {
    q = empty({rows, k}, at::kFloat8_e4m3fn, device);
    s = empty({tall, blocks(k)}, at::kFloat, device);
  } else {
    const at::Tensor *given = dense(a[2], at::kFloat8_e4m3fn, 2), *scale = dense(a[3], at::kFloat, 2);
    if (!given || !scale || given->size(0) != rows || given->size(1) != k || scale->size(0) != tall ||
        scale->size(1) != blocks(k) || given->get_device() != device || scale->get_device() != device)
      Py_RETURN_NONE;
    q = *given;
    s = *scale;
  }
  const int rc = call(device, [&](fi_stream_t stream) {
    return (square ? pack_fn : quantize_fn)(x->const_data_ptr(), code, rows, k, static_cast<uint8_t*>(q.data_ptr()),
                                            static_cast<float*>(s.data_ptr()), stream);
  });
  if (rc != FI_OK) return PyLong_FromLong(rc);
  PyObject* r = PyTuple_New(2);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(q)));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(s)));
  return r;
  END_HANDLE_TH_ERRORS
}

// An int argument; what no C int holds becomes -1, for the library to refuse.
bool number(PyObject* o, int* v) {
  if (!PyLong_Check(o)) return false;
  int overflow = 0;
  const long x = PyLong_AsLongAndOverflow(o, &overflow);
  *v = overflow || x < 0 || x > 0x7fffffffL ? -1 : (int)x;
  return true;
}

// (Aq, Ascale, Wq, Wscale, out, out_dtype, splits)
PyObject* mm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Operand x, w;
  at::Tensor out;
  int splits;
  if (n != 7 || !number(a[6], &splits) || !x.get(a[0], a[1], 1) || !w.get(a[2], a[3], kBlock) || w.k != x.k ||
      w.q->get_device() != x.q->get_device() || !output(a[4], a[5], x.r, w.r, x.q->get_device(), &out))
    Py_RETURN_NONE;
  const int rc = call(x.q->get_device(), [&](fi_stream_t stream) {
    return mm_fn(x.codes(), x.scale(), w.codes(), w.scale(), out.data_ptr(), code_of(out.scalar_type()), x.r, w.r, x.k,
                 splits, stream);
  });
  return rc != FI_OK ? PyLong_FromLong(rc) : THPVariable_Wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

// (Aq, Ascale, Gq, Gscale, Uq, Uscale, out, out_dtype, splits)
PyObject* gated(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Operand x, g, u;
  at::Tensor out;
  int splits;
  if (n != 9 || !number(a[8], &splits) || !x.get(a[0], a[1], 1) || !g.get(a[2], a[3], kBlock) ||
      !u.get(a[4], a[5], kBlock) || g.k != x.k || u.k != x.k || u.r != g.r || g.q->get_device() != x.q->get_device() || u.q->get_device() != x.q->get_device() ||
      !output(a[6], a[7], x.r, g.r, x.q->get_device(), &out))
    Py_RETURN_NONE;
  const int rc = call(x.q->get_device(), [&](fi_stream_t stream) {
    return gated_fn(x.codes(), x.scale(), g.codes(), g.scale(), u.codes(), u.scale(), out.data_ptr(),
                    code_of(out.scalar_type()), x.r, g.r, x.k, splits, stream);
  });
  return rc != FI_OK ? PyLong_FromLong(rc) : THPVariable_Wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

// (logits, tokens, topk)
PyObject* logprobs(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const at::Tensor* z = n == 3 ? cuda_tensor(a[0]) : nullptr;
  const at::Tensor* tokens = z ? dense(a[1], at::kLong, 1) : nullptr;
  const int code = z ? code_of(z->scalar_type()) : -1;
  int topk;
  if (!tokens || code < 0 || z->dim() != 2 || !number(a[2], &topk)) Py_RETURN_NONE;
  if (topk > FI_LOGPROBS_MAX_TOPK) topk = -1;  // before the outputs are made
  const int64_t rows = z->size(0), vocab = z->size(1), ld = rows <= 1 ? vocab : z->stride(0);
  const int device = z->get_device();
  if ((vocab > 1 && z->stride(1) != 1) || ld < vocab ||
      tokens->size(0) != rows || tokens->get_device() != device)
    Py_RETURN_NONE;
  const int64_t kk = std::min<int64_t>(std::max(topk, 0), vocab);
  at::Tensor lp = empty({rows}, at::kFloat, device), ent = empty({rows}, at::kFloat, device),
             rank = empty({rows}, at::kLong, device), top = empty({rows, kk}, at::kFloat, device),
             ids = empty({rows, kk}, at::kLong, device);
  const int rc = call(device, [&](fi_stream_t stream) {
    return logprobs_fn(z->const_data_ptr(), code, rows, vocab, ld, static_cast<const int64_t*>(tokens->const_data_ptr()),
                       topk, static_cast<float*>(lp.data_ptr()), static_cast<float*>(ent.data_ptr()),
                       static_cast<int64_t*>(rank.data_ptr()), static_cast<float*>(top.data_ptr()),
                       static_cast<int64_t*>(ids.data_ptr()), stream);
  });
  if (rc != FI_OK) return PyLong_FromLong(rc);
  PyObject* r = PyTuple_New(5);
  if (!r) return nullptr;
  at::Tensor* const all[5] = {&lp, &ent, &rank, &top, &ids};
  for (int i = 0; i < 5; ++i) PyTuple_SET_ITEM(r, i, THPVariable_Wrap(std::move(*all[i])));
  return r;
  END_HANDLE_TH_ERRORS
}

// The addresses of fi_fp8_quantize, fi_fp8_pack_weights, fi_mm_fp8_ex, fi_mm_fp8_gated_ex and
// fi_token_logprobs in the library that is loaded.
PyObject* bind(PyObject*, PyObject* args) {
  unsigned long long f[5];
  if (!PyArg_ParseTuple(args, "KKKKK", &f[0], &f[1], &f[2], &f[3], &f[4])) return nullptr;
  quantize_fn = reinterpret_cast<decltype(quantize_fn)>(f[0]);
  pack_fn = reinterpret_cast<decltype(pack_fn)>(f[1]);
  mm_fn = reinterpret_cast<decltype(mm_fn)>(f[2]);
  gated_fn = reinterpret_cast<decltype(gated_fn)>(f[3]);
  logprobs_fn = reinterpret_cast<decltype(logprobs_fn)>(f[4]);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    {"quantize", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(quantize)), METH_FASTCALL, nullptr},
    {"mm", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(mm)), METH_FASTCALL, nullptr},
    {"gated", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(gated)), METH_FASTCALL, nullptr},
    {"logprobs", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(logprobs)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", FI_TORCH_VERSION) != 0) Py_CLEAR(m);
  return m;
}
