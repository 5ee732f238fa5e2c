// pages_torch.cpp - Python binding of the full-attention layers' entry points (module _pages).
//
// A decode step makes these calls once or more a layer, and at their smallest they are a few
// microseconds on the GPU, less than it takes an interpreter to check a call's tensors one
// property at a time.  So checks, outputs and workspaces are made here; pages.py gives the
// calls their names, defaults and documentation.  The kernels and all further checks are
// behind the C ABI (rkv.h), which this file calls like any other user of it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <sstream>
#include <stdexcept>

#include "../../include/rkv.h"

namespace {

PyObject* g_error = nullptr;         // RkvError: (status, message)

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct PythonError {};               // a Python exception is already set

std::string describe(at::ScalarType type, at::IntArrayRef shape) {
  std::ostringstream s;
  s << at::toString(type) << ", shape " << shape;
  return s.str();
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) throw Refused(std::string(what) + " must be a tensor");
  return THPVariable_Unpack(o);
}

// The CUDA device of a call's first tensor.
int device_of(const at::Tensor& t, const char* what) {
  if (!t.is_cuda()) throw Refused(std::string(what) + " must be a CUDA tensor, not on " + t.device().str());
  return t.get_device();
}

void check_dims(const at::Tensor& t, const char* what, int64_t dims) {
  if (t.dim() != dims)
    throw Refused(std::string(what) + " must be a tensor of " + std::to_string(dims) + " dimensions");
}

[[noreturn]] void refuse(const at::Tensor& t, const char* what, const char* kind, at::ScalarType type,
                         at::IntArrayRef shape, int dev) {
  throw Refused(std::string(what) + " must be a " + kind + "tensor of " + describe(type, shape) + " on cuda:" +
                std::to_string(dev) + ", not " + describe(t.scalar_type(), t.sizes()) + " on " + t.device().str());
}

// Address of a contiguous tensor of this type and shape on CUDA device dev.
void* array(PyObject* o, const char* what, at::IntArrayRef shape, int dev, at::ScalarType type = at::kInt) {
  const at::Tensor& t = tensor(o, what);
  if (t.scalar_type() != type || t.sizes() != shape || !t.is_cuda() || t.get_device() != dev || !t.is_contiguous())
    refuse(t, what, "contiguous ", type, shape, dev);
  return t.data_ptr();
}

// The same, or nullptr for None.
void* array_or_none(PyObject* o, const char* what, at::IntArrayRef shape, int dev, at::ScalarType type = at::kInt) {
  return o == Py_None ? nullptr : array(o, what, shape, dev, type);
}

// A [rows, heads, D] tensor of this type and shape on CUDA device dev, whose rows of D start
// on 16 bytes: its address, and its row and head strides.
void* rows_of(const at::Tensor& t, const char* what, at::IntArrayRef shape, int dev, at::ScalarType type,
              int64_t strides[2]) {
  if (t.scalar_type() != type || t.sizes() != shape || !t.is_cuda() || t.get_device() != dev)
    refuse(t, what, "", type, shape, dev);
  // the stride of a single row or head is never used: torch may give any
  strides[0] = shape[0] > 1 ? t.stride(0) : 0;
  strides[1] = shape[1] > 1 ? t.stride(1) : 0;
  const int64_t whole = type == at::kFloat ? 4 : 8;
  if (t.stride(2) != 1 || strides[0] % whole || strides[1] % whole) {
    if (t.numel() != 0) throw Refused(std::string(what) + " needs unit element stride and strides of whole 16 bytes");
    strides[0] = strides[1] = 0;
  }
  return t.data_ptr();
}

double scale_of(PyObject* o, int64_t D) {
  if (o == Py_None) return 1.0 / std::sqrt((double)D);
  const double s = PyFloat_AsDouble(o);
  if (s == -1.0 && PyErr_Occurred()) throw PythonError();
  if (!(std::isfinite(s) && s > 0)) throw Refused("scale must be finite and > 0");
  return s;
}

int32_t int_of(PyObject* o, const char* what) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError();
  if (v < INT32_MIN || v > INT32_MAX) throw Refused(std::string(what) + " is out of range");
  return (int32_t)v;
}

// Makes dev current and finds the stream to launch on: the given torch.cuda.Stream (then also
// the one whose memory outputs and workspaces come from) or dev's current one.
class On {
 public:
  On(int dev, PyObject* stream) : guard_(static_cast<c10::DeviceIndex>(dev)) {
    if (stream == Py_None) {
      raw = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
      return;
    }
    PyObject* ptr = PyObject_GetAttrString(stream, "cuda_stream");
    PyObject* index = PyObject_GetAttrString(stream, "device_index");
    const bool ok = ptr && index;
    if (ok) {
      raw = reinterpret_cast<cudaStream_t>(PyLong_AsVoidPtr(ptr));
      at = (int)PyLong_AsLong(index);
    }
    Py_XDECREF(ptr);
    Py_XDECREF(index);
    if (!ok || PyErr_Occurred()) throw PythonError();
    if (at != dev)
      throw Refused("stream is on cuda:" + std::to_string(at) + ", the call's tensors on cuda:" + std::to_string(dev));
    stream_.emplace(c10::cuda::getStreamFromExternal(raw, static_cast<c10::DeviceIndex>(dev)));
  }
  cudaStream_t raw = nullptr;

 private:
  int at = 0;
  c10::cuda::CUDAGuard guard_;
  std::optional<c10::cuda::CUDAStreamGuard> stream_;
};

at::Tensor make(at::IntArrayRef shape, at::ScalarType type, int dev) {
  return at::detail::empty_cuda(shape, type, c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(dev)), std::nullopt);
}

// n elements of a one-dimensional tensor from `offset`, as a tensor on the same storage.
at::Tensor part(const at::Tensor& base, int64_t offset, int64_t n) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(base.storage()), base.key_set(), base.dtype());
  t.unsafeGetTensorImpl()->set_sizes_contiguous(at::IntArrayRef(&n, 1));
  t.unsafeGetTensorImpl()->set_storage_offset(offset);
  return t;
}

void check(rkv_status st) {
  if (st == RKV_OK) return;
  PyObject* args = Py_BuildValue("(is)", (int)st, rkv_last_error());
  if (args) {
    PyErr_SetObject(g_error, args);
    Py_DECREF(args);
  }
  throw PythonError();
}

rkv_page_table table_of(PyObject* block_table, PyObject* seq_len, int dev) {
  const at::Tensor& t = tensor(block_table, "block_table");
  check_dims(t, "block_table", 2);
  const int64_t B = t.size(0), M = t.size(1);
  rkv_page_table r;
  r.block_table = static_cast<int32_t*>(array(block_table, "block_table", {B, M}, dev));
  r.seq_len = static_cast<int32_t*>(array(seq_len, "seq_len", {B}, dev));
  r.batch = (int32_t)std::min<int64_t>(B, INT32_MAX);
  r.max_blocks = (int32_t)std::min<int64_t>(M, INT32_MAX);
  return r;
}

rkv_pages pages_of(PyObject* k8, PyObject* v8, PyObject* ks, PyObject* vs, int& dev) {
  const at::Tensor& t = tensor(k8, "k8");
  dev = device_of(t, "k8");
  check_dims(t, "k8", 4);
  const int64_t nb = t.size(0), N = t.size(1), P = t.size(2), D = t.size(3);
  rkv_pages r;
  r.k = array(k8, "k8", {nb, N, P, D}, dev, at::kByte);
  r.v = array(v8, "v8", {nb, N, P, D}, dev, at::kByte);
  r.k_scale = static_cast<float*>(array(ks, "k_scale", {nb, N}, dev, at::kFloat));
  r.v_scale = static_cast<float*>(array(vs, "v_scale", {nb, N}, dev, at::kFloat));
  for (int64_t d : {nb, N, P, D})
    if (d > INT32_MAX) throw Refused("k8 is too large");
  r.n_kv_heads = (int32_t)N, r.head_dim = (int32_t)D, r.block_tokens = (int32_t)P, r.num_blocks = (int32_t)nb;
  return r;
}

int32_t* flags_of(PyObject* o, int dev) { return static_cast<int32_t*>(array_or_none(o, "flags", {1}, dev)); }

int64_t length_of(PyObject* o, const char* what) {
  const at::Tensor& t = tensor(o, what);
  check_dims(t, what, 1);
  if (t.size(0) > INT32_MAX) throw Refused(std::string(what) + " is too long");
  return t.size(0);
}

// (new_tokens, seq_len, block_table, free_blocks, n_free, block_tokens, max_rows, seq_len_out,
//  n_free_out, flags, stream) -> (cu_rows, row_seq, row_pos, row_slot)
PyObject* page_plan(PyObject* const* a) {
  const int32_t P = int_of(a[5], "block_tokens"), rows = int_of(a[6], "max_rows");
  if (rows < 0) throw Refused("max_rows must be >= 0");
  const int dev = device_of(tensor(a[2], "block_table"), "block_table");
  rkv_page_table t = table_of(a[2], a[1], dev);
  const int64_t B = t.batch, num = length_of(a[3], "free_blocks");
  const int32_t* nw = static_cast<int32_t*>(array(a[0], "new_tokens", {B}, dev));
  const int32_t* fb = static_cast<int32_t*>(array(a[3], "free_blocks", {num}, dev));
  int32_t* nf = static_cast<int32_t*>(array(a[4], "n_free", {1}, dev));
  int32_t* lo = a[7] == Py_None ? t.seq_len : static_cast<int32_t*>(array(a[7], "seq_len_out", {B}, dev));
  int32_t* no = a[8] == Py_None ? nf : static_cast<int32_t*>(array(a[8], "n_free_out", {1}, dev));
  int32_t* fl = flags_of(a[9], dev);
  const On on(dev, a[10]);
  // one allocation: the offsets, then the three row maps
  const at::Tensor buf = make({B + 1 + 3 * (int64_t)rows}, at::kInt, dev);
  int32_t* p = static_cast<int32_t*>(buf.data_ptr());
  int32_t* r = p + B + 1;
  check(rkv_page_plan(&t, nw, fb, nf, (int32_t)num, P, rows, lo, no, p, r, r + rows, r + 2 * (int64_t)rows, fl, on.raw));
  PyObject* out = PyTuple_New(4);
  if (!out) throw PythonError();
  PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(part(buf, 0, B + 1)));
  for (int i = 0; i < 3; ++i)
    PyTuple_SET_ITEM(out, i + 1, THPVariable_Wrap(part(buf, B + 1 + i * (int64_t)rows, rows)));
  return out;
}

// (finished, seq_len, block_table, free_blocks, n_free, block_tokens, flags, stream)
PyObject* page_release(PyObject* const* a) {
  const int32_t P = int_of(a[5], "block_tokens");
  const int dev = device_of(tensor(a[2], "block_table"), "block_table");
  rkv_page_table t = table_of(a[2], a[1], dev);
  const int64_t num = length_of(a[3], "free_blocks");
  const int32_t* fin = static_cast<int32_t*>(array(a[0], "finished", {t.batch}, dev));
  int32_t* fb = static_cast<int32_t*>(array(a[3], "free_blocks", {num}, dev));
  int32_t* nf = static_cast<int32_t*>(array(a[4], "n_free", {1}, dev));
  int32_t* fl = flags_of(a[6], dev);
  const On on(dev, a[7]);
  check(rkv_page_release(&t, fin, fb, nf, (int32_t)num, P, fl, on.raw));
  Py_RETURN_NONE;
}

// (k, v, k8, v8, k_scale, v_scale, block_table, seq_len, cu_rows, flags, stream)
PyObject* page_append(PyObject* const* a) {
  int dev;
  const rkv_pages pg = pages_of(a[2], a[3], a[4], a[5], dev);
  const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
  check_dims(k, "k", 3);
  if (k.size(0) > INT32_MAX) throw Refused("k has too many rows");
  const at::ScalarType type = k.scalar_type() == at::kFloat ? at::kFloat : at::kBFloat16;
  const int64_t shape[3] = {k.size(0), pg.n_kv_heads, pg.head_dim};
  int64_t ks[2], vs[2];
  const void* kp = rows_of(k, "k", shape, dev, type, ks);
  const void* vp = rows_of(v, "v", shape, dev, type, vs);
  const rkv_page_table t = table_of(a[6], a[7], dev);
  const int32_t* cu = static_cast<int32_t*>(array(a[8], "cu_rows", {(int64_t)t.batch + 1}, dev));
  int32_t* fl = flags_of(a[9], dev);
  const On on(dev, a[10]);
  check(rkv_page_append(&pg, &t, kp, ks, vp, vs, type == at::kFloat ? RKV_F32 : RKV_BF16, (int32_t)shape[0], cu, fl,
                        on.raw));
  Py_RETURN_NONE;
}

// (q, k8, v8, k_scale, v_scale, block_table, seq_len, scale, out, lse, flags, stream) -> out
PyObject* page_attention(PyObject* const* a) {
  int dev;
  const rkv_pages pg = pages_of(a[1], a[2], a[3], a[4], dev);
  const rkv_page_table t = table_of(a[5], a[6], dev);
  const at::Tensor& q = tensor(a[0], "q");
  check_dims(q, "q", 3);
  const int64_t shape[3] = {t.batch, q.size(1), pg.head_dim};
  int64_t qs[2];
  const void* qp = rows_of(q, "q", shape, dev, at::kBFloat16, qs);
  if (shape[1] > INT32_MAX) throw Refused("q has too many heads");
  float* lse = static_cast<float*>(array_or_none(a[9], "lse", {shape[0], shape[1]}, dev, at::kFloat));
  int32_t* fl = flags_of(a[10], dev);
  const double scale = scale_of(a[7], shape[2]);
  void* given = array_or_none(a[8], "out", shape, dev, at::kBFloat16);
  size_t bytes = 0;
  check(rkv_page_attention_workspace(&pg, &t, (int32_t)shape[1], &bytes));
  const On on(dev, a[11]);
  at::Tensor out;
  if (!given) out = make(shape, at::kBFloat16, dev);
  const at::Tensor ws = make({(int64_t)bytes}, at::kByte, dev);
  check(rkv_page_attention(&pg, &t, qp, qs, (int32_t)shape[1], scale, given ? given : out.data_ptr(), lse,
                           ws.data_ptr(), bytes, fl, on.raw));
  if (!given) return THPVariable_Wrap(out);
  Py_INCREF(a[8]);
  return a[8];
}

// (q, k, v, cu_q, cu_k, scale, out, lse, flags, stream) -> out
PyObject* prompt_attention(PyObject* const* a) {
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
  const int dev = device_of(q, "q");
  check_dims(q, "q", 3);
  check_dims(k, "k", 3);
  const int64_t qshape[3] = {q.size(0), q.size(1), q.size(2)}, kshape[3] = {k.size(0), k.size(1), q.size(2)};
  for (int64_t d : {qshape[0], qshape[1], qshape[2], kshape[0], kshape[1]})
    if (d > INT32_MAX) throw Refused("q or k is too large");
  rkv_prompt p;
  p.q = rows_of(q, "q", qshape, dev, at::kBFloat16, p.q_strides);
  p.k = rows_of(k, "k", kshape, dev, at::kBFloat16, p.k_strides);
  p.v = rows_of(v, "v", kshape, dev, at::kBFloat16, p.v_strides);
  const int64_t n_cu = length_of(a[3], "cu_q");
  p.cu_q = static_cast<int32_t*>(array(a[3], "cu_q", {n_cu}, dev));
  p.cu_k = a[4] == Py_None ? p.cu_q : static_cast<int32_t*>(array(a[4], "cu_k", {n_cu}, dev));
  p.lse = static_cast<float*>(array_or_none(a[7], "lse", {qshape[0], qshape[1]}, dev, at::kFloat));
  int32_t* fl = flags_of(a[8], dev);
  p.batch = (int32_t)n_cu - 1;
  p.total_q = (int32_t)qshape[0], p.total_k = (int32_t)kshape[0];
  p.n_q_heads = (int32_t)qshape[1], p.n_kv_heads = (int32_t)kshape[1], p.head_dim = (int32_t)qshape[2];
  p.scale = scale_of(a[5], qshape[2]);
  p.workspace = nullptr;
  p.workspace_bytes = 0;
  const On on(dev, a[9]);
  at::Tensor out, ws;
  if (a[6] == Py_None) {
    out = make(qshape, at::kBFloat16, dev);
    p.out = out.data_ptr();
    p.out_strides[0] = qshape[1] * qshape[2], p.out_strides[1] = qshape[2];
  } else {
    p.out = rows_of(tensor(a[6], "out"), "out", qshape, dev, at::kBFloat16, p.out_strides);
  }
  size_t bytes = 0;
  check(rkv_prompt_attention_workspace(&p, &bytes));
  if (bytes) {
    ws = make({(int64_t)bytes}, at::kByte, dev);
    p.workspace = ws.data_ptr();
    p.workspace_bytes = bytes;
  }
  check(rkv_prompt_attention(&p, fl, on.raw));
  if (a[6] == Py_None) return THPVariable_Wrap(out);
  Py_INCREF(a[6]);
  return a[6];
}

// No C++ exception leaves the module.
template <PyObject* (*kFn)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kArgs) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, not %zd", kArgs, n);
    return nullptr;
  }
  try {
    return kFn(args);
  } catch (const PythonError&) {
    return nullptr;
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XDECREF(g_error);
  g_error = cls;
  Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"page_plan", (PyCFunction)(void (*)(void)) & entry<page_plan, 11>, METH_FASTCALL, nullptr},
    {"page_release", (PyCFunction)(void (*)(void)) & entry<page_release, 8>, METH_FASTCALL, nullptr},
    {"page_append", (PyCFunction)(void (*)(void)) & entry<page_append, 11>, METH_FASTCALL, nullptr},
    {"page_attention", (PyCFunction)(void (*)(void)) & entry<page_attention, 12>, METH_FASTCALL, nullptr},
    {"prompt_attention", (PyCFunction)(void (*)(void)) & entry<prompt_attention, 10>, METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_pages", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pages(void) { return PyModule_Create(&g_module); }
