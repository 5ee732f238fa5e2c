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
#include <cstring>
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

// (q, k, positions, freq, q_weight, k_weight, eps, adjacent, q_out, k_out, stream) -> (q_out, k_out)
PyObject* head_norm_rotate(PyObject* const* a) {
  PyObject *const x[2] = {a[0], a[1]}, *const w[2] = {a[4], a[5]}, *const given[2] = {a[8], a[9]};
  static const char* const names[2][3] = {{"q", "q_weight", "q_out"}, {"k", "k_weight", "k_out"}};
  const int any = x[0] == Py_None;
  if (x[any] == Py_None) throw Refused("q and k are both None");
  const at::Tensor& t = tensor(x[any], names[any][0]);
  const int dev = device_of(t, names[any][0]);
  check_dims(t, names[any][0], 3);
  const at::ScalarType type = t.scalar_type() == at::kFloat ? at::kFloat : at::kBFloat16;
  const int64_t rows = t.size(0), D = t.size(2);
  if (rows > INT32_MAX || D > INT32_MAX) throw Refused(std::string(names[any][0]) + " is too large");
  // outputs' type: that of one that is given, else the inputs'
  at::ScalarType out_type = type;
  for (int i = 0; i < 2; ++i)
    if (given[i] != Py_None) out_type = tensor(given[i], names[i][2]).scalar_type();
  if (out_type != type) out_type = at::kBFloat16;
  const at::Tensor& f = tensor(a[3], "freq");
  check_dims(f, "freq", 1);
  rkv_head_rows r;
  memset(&r, 0, sizeof r);
  const void** in[2] = {&r.q, &r.k};
  void** out[2] = {&r.q_out, &r.k_out};
  const void** weight[2] = {&r.q_weight, &r.k_weight};
  int64_t *strides[2] = {r.q_strides, r.k_strides}, *out_strides[2] = {r.q_out_strides, r.k_out_strides};
  int32_t* heads[2] = {&r.n_q_heads, &r.n_k_heads};
  int64_t shape[2][3] = {{rows, 0, D}, {rows, 0, D}};
  for (int i = 0; i < 2; ++i) {
    if (x[i] == Py_None) {
      if (given[i] != Py_None || w[i] != Py_None) throw Refused(std::string(names[i][0]) + " is None, its output or weight is not");
      continue;
    }
    const at::Tensor& xi = tensor(x[i], names[i][0]);
    check_dims(xi, names[i][0], 3);
    shape[i][1] = xi.size(1);
    if (shape[i][1] > INT32_MAX) throw Refused(std::string(names[i][0]) + " has too many heads");
    *in[i] = rows_of(xi, names[i][0], shape[i], dev, type, strides[i]);
    *heads[i] = (int32_t)shape[i][1];
    *weight[i] = array_or_none(w[i], names[i][1], {D}, dev, type);
    if (given[i] != Py_None) *out[i] = rows_of(tensor(given[i], names[i][2]), names[i][2], shape[i], dev, out_type, out_strides[i]);
  }
  r.positions = static_cast<int32_t*>(array(a[2], "positions", {rows}, dev));
  r.freq = static_cast<double*>(array(a[3], "freq", {f.size(0)}, dev, at::kDouble));
  if (f.size(0) > 1 << 20) throw Refused("freq is too long");
  r.n_rows = (int32_t)rows, r.head_dim = (int32_t)D, r.rotary_dim = 2 * (int32_t)f.size(0);
  r.norm = a[6] != Py_None;
  if (r.norm) {
    r.eps = PyFloat_AsDouble(a[6]);
    if (r.eps == -1.0 && PyErr_Occurred()) throw PythonError();
  }
  r.adjacent = PyObject_IsTrue(a[7]);
  if (r.adjacent < 0) throw PythonError();
  r.dtype = type == at::kFloat ? RKV_F32 : RKV_BF16;
  r.out_dtype = out_type == at::kFloat ? RKV_F32 : RKV_BF16;
  const On on(dev, a[10]);
  at::Tensor made[2];
  for (int i = 0; i < 2; ++i) {
    if (x[i] == Py_None || given[i] != Py_None) continue;
    made[i] = make(shape[i], out_type, dev);
    *out[i] = made[i].data_ptr();
    out_strides[i][0] = shape[i][1] * D, out_strides[i][1] = D;
  }
  check(rkv_head_norm_rotate(&r, on.raw));
  PyObject* both = PyTuple_New(2);
  if (!both) throw PythonError();
  for (int i = 0; i < 2; ++i) {
    PyObject* o = given[i];
    if (made[i].defined()) o = THPVariable_Wrap(made[i]);
    else Py_INCREF(o);
    PyTuple_SET_ITEM(both, i, o);
  }
  return both;
}

// Three int32 tensors of n, n and m elements on one allocation, as a tuple.
PyObject* three(const at::Tensor& buf, int64_t n, int64_t m) {
  PyObject* out = PyTuple_New(3);
  if (!out) throw PythonError();
  for (int i = 0; i < 3; ++i) PyTuple_SET_ITEM(out, i, THPVariable_Wrap(part(buf, i * n, i < 2 ? n : m)));
  return out;
}

// (source, seq_len, block_table, free_blocks, n_free, block_tokens, length, finished, block_table_out,
//  seq_len_out, n_free_out, flags, stream) -> (src, dst, rows)
PyObject* page_fork(PyObject* const* a) {
  const int32_t P = int_of(a[5], "block_tokens");
  const int dev = device_of(tensor(a[2], "block_table"), "block_table");
  const rkv_page_table t = table_of(a[2], a[1], dev);
  const int64_t B = t.batch, num = length_of(a[3], "free_blocks");
  const int32_t* source = static_cast<int32_t*>(array_or_none(a[0], "source", {B}, dev));
  int32_t* fb = static_cast<int32_t*>(array(a[3], "free_blocks", {num}, dev));
  int32_t* nf = static_cast<int32_t*>(array(a[4], "n_free", {1}, dev));
  const int32_t* length = static_cast<int32_t*>(array_or_none(a[6], "length", {B}, dev));
  const int32_t* finished = static_cast<int32_t*>(array_or_none(a[7], "finished", {B}, dev));
  int32_t* to = a[8] == Py_None ? t.block_table : static_cast<int32_t*>(array(a[8], "block_table_out", {B, t.max_blocks}, dev));
  int32_t* lo = a[9] == Py_None ? t.seq_len : static_cast<int32_t*>(array(a[9], "seq_len_out", {B}, dev));
  int32_t* no = a[10] == Py_None ? nf : static_cast<int32_t*>(array(a[10], "n_free_out", {1}, dev));
  int32_t* fl = flags_of(a[11], dev);
  size_t bytes = 0;
  check(rkv_page_fork_workspace(&t, (int32_t)num, P, &bytes));
  const On on(dev, a[12]);
  const at::Tensor buf = make({3 * B}, at::kInt, dev), ws = make({(int64_t)bytes}, at::kByte, dev);
  int32_t* p = static_cast<int32_t*>(buf.data_ptr());
  check(rkv_page_fork(&t, source, length, finished, fb, nf, (int32_t)num, P, to, lo, no, p, p + B, p + 2 * B,
                      ws.data_ptr(), bytes, fl, on.raw));
  return three(buf, B, B);
}

// (seq_len, block_table, free_blocks, n_free, block_tokens, block_table_out, flags, stream) -> (src, dst, count)
PyObject* page_compact(PyObject* const* a) {
  const int32_t P = int_of(a[4], "block_tokens");
  const int dev = device_of(tensor(a[1], "block_table"), "block_table");
  const rkv_page_table t = table_of(a[1], a[0], dev);
  const int64_t num = length_of(a[2], "free_blocks");
  int32_t* fb = static_cast<int32_t*>(array(a[2], "free_blocks", {num}, dev));
  int32_t* nf = static_cast<int32_t*>(array(a[3], "n_free", {1}, dev));
  int32_t* to = a[5] == Py_None ? t.block_table
                                : static_cast<int32_t*>(array(a[5], "block_table_out", {t.batch, t.max_blocks}, dev));
  int32_t* fl = flags_of(a[6], dev);
  size_t bytes = 0;
  check(rkv_page_compact_workspace((int32_t)num, &bytes));
  const On on(dev, a[7]);
  const int64_t n = num / 2;
  const at::Tensor buf = make({2 * n + 1}, at::kInt, dev), ws = make({(int64_t)bytes}, at::kByte, dev);
  int32_t* p = static_cast<int32_t*>(buf.data_ptr());
  check(rkv_page_compact(&t, fb, nf, (int32_t)num, P, to, p, p + n, p + 2 * n, ws.data_ptr(), bytes, fl, on.raw));
  return three(buf, n, 1);
}

// Address of a tensor as array() takes it; of the many tensors of a call that mostly are as asked.
inline void* one_of(PyObject* o, const char* what, at::IntArrayRef shape, int dev, at::ScalarType type) {
  if (THPVariable_Check(o)) {
    const c10::TensorImpl* t = THPVariable_Unpack(o).unsafeGetTensorImpl();
    if (t->dtype() == c10::scalarTypeToTypeMeta(type) && t->sizes() == shape && t->is_cuda() &&
        t->device().index() == dev && t->is_contiguous())
      return THPVariable_Unpack(o).data_ptr();
  }
  return array(o, what, shape, dev, type);
}

// (caches: a list or tuple of (k8, v8, k_scale, v_scale) or of objects whose arrays() are that, src,
//  dst, rows, count, flags, stream)
PyObject* page_copy(PyObject* const* a) {
  if (!PyList_Check(a[0]) && !PyTuple_Check(a[0])) throw Refused("caches must be a list or tuple");
  // arrays() may be any code: what it makes and the caches themselves live until the launch, whatever
  // becomes of the list meanwhile
  struct Held {
    PyObject* o[1 + 128];
    int n = 0;
    PyObject* add(PyObject* x) { return o[n++] = x; }
    ~Held() {
      while (n) Py_DECREF(o[--n]);
    }
  } held;
  PyObject* all = PySequence_Tuple(a[0]);
  if (!all) throw PythonError();
  held.add(all);
  const Py_ssize_t layers = PyTuple_GET_SIZE(all);
  if (layers < 1 || layers > 128) throw Refused("caches must be 1 to 128");
  // (made once: a call's host time is mostly this loop's)
  static PyObject* const arrays = PyUnicode_InternFromString("arrays");
  if (!arrays) throw PythonError();
  rkv_pages pg[128];
  int dev = 0;
  for (Py_ssize_t i = 0; i < layers; ++i) {
    PyObject* l = PyTuple_GET_ITEM(all, i);
    PyObject* made = PyTuple_Check(l) ? nullptr : PyObject_CallMethodNoArgs(l, arrays);
    if (made) {
      l = held.add(made);
    } else if (PyErr_Occurred()) {
      if (!PyErr_ExceptionMatches(PyExc_AttributeError)) throw PythonError();
      PyErr_Clear();
    }
    if (!PyTuple_Check(l) || PyTuple_GET_SIZE(l) != 4) throw Refused("a cache must be (k8, v8, k_scale, v_scale)");
    PyObject* const* t = &PyTuple_GET_ITEM(l, 0);
    if (i == 0) {
      pg[0] = pages_of(t[0], t[1], t[2], t[3], dev);
      continue;
    }
    const int64_t nb = pg[0].num_blocks, N = pg[0].n_kv_heads;
    const int64_t shape[4] = {nb, N, pg[0].block_tokens, pg[0].head_dim};
    pg[i] = pg[0];
    pg[i].k = one_of(t[0], "k8", shape, dev, at::kByte);
    pg[i].v = one_of(t[1], "v8", shape, dev, at::kByte);
    pg[i].k_scale = static_cast<float*>(one_of(t[2], "k_scale", {shape, 2}, dev, at::kFloat));
    pg[i].v_scale = static_cast<float*>(one_of(t[3], "v_scale", {shape, 2}, dev, at::kFloat));
  }
  const int64_t n = length_of(a[1], "src");
  const int32_t* src = static_cast<int32_t*>(array(a[1], "src", {n}, dev));
  const int32_t* dst = static_cast<int32_t*>(array(a[2], "dst", {n}, dev));
  const int32_t* rows = static_cast<int32_t*>(array_or_none(a[3], "rows", {n}, dev));
  const int32_t* count = static_cast<int32_t*>(array_or_none(a[4], "count", {1}, dev));
  int32_t* fl = flags_of(a[5], dev);
  const On on(dev, a[6]);
  check(rkv_page_copy(pg, (int32_t)layers, src, dst, rows, count, (int32_t)n, fl, on.raw));
  Py_RETURN_NONE;
}

// (k8, v8, k_scale, v_scale, block_table, seq_len, max_rows, length, k_out, v_out, flags, stream) -> (k, v, cu_rows)
PyObject* page_gather(PyObject* const* a) {
  int dev;
  const rkv_pages pg = pages_of(a[0], a[1], a[2], a[3], dev);
  const rkv_page_table t = table_of(a[4], a[5], dev);
  PyObject* given[2] = {a[8], a[9]};
  if ((given[0] == Py_None) != (given[1] == Py_None)) throw Refused("k_out and v_out go together");
  const bool fresh = given[0] == Py_None;
  int64_t rows = 0;
  if (a[6] != Py_None) rows = int_of(a[6], "max_rows");
  else if (fresh) throw Refused("max_rows or k_out and v_out must be given");
  if (!fresh) {
    const at::Tensor& k = tensor(given[0], "k_out");
    check_dims(k, "k_out", 3);
    if (k.size(0) > INT32_MAX) throw Refused("k_out has too many rows");
    if (a[6] != Py_None && rows > k.size(0)) throw Refused("k_out has fewer than max_rows rows");
    if (a[6] == Py_None) rows = k.size(0);
  }
  if (rows < 0) throw Refused("max_rows must be >= 0");
  const int32_t* length = static_cast<int32_t*>(array_or_none(a[7], "length", {t.batch}, dev));
  int32_t* fl = flags_of(a[10], dev);
  int64_t strides[2][2];
  void* out[2];
  if (!fresh) {
    static const char* const names[2] = {"k_out", "v_out"};
    const int64_t n = tensor(given[0], names[0]).size(0), shape[3] = {n, pg.n_kv_heads, pg.head_dim};
    for (int i = 0; i < 2; ++i) out[i] = rows_of(tensor(given[i], names[i]), names[i], shape, dev, at::kBFloat16, strides[i]);
  }
  const On on(dev, a[11]);
  at::Tensor made[2];
  if (fresh) {
    for (int i = 0; i < 2; ++i) {
      made[i] = make({rows, pg.n_kv_heads, pg.head_dim}, at::kBFloat16, dev);
      out[i] = made[i].data_ptr();
      strides[i][0] = (int64_t)pg.n_kv_heads * pg.head_dim, strides[i][1] = pg.head_dim;
    }
  }
  const at::Tensor cu = make({(int64_t)t.batch + 1}, at::kInt, dev);
  check(rkv_page_gather(&pg, &t, length, out[0], strides[0], out[1], strides[1], (int32_t)rows,
                        static_cast<int32_t*>(cu.data_ptr()), fl, on.raw));
  PyObject* all = PyTuple_New(3);
  if (!all) throw PythonError();
  for (int i = 0; i < 2; ++i) {
    PyObject* o = given[i];
    if (fresh) o = THPVariable_Wrap(made[i]);
    else Py_INCREF(o);
    PyTuple_SET_ITEM(all, i, o);
  }
  PyTuple_SET_ITEM(all, 2, THPVariable_Wrap(cu));
  return all;
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
    {"head_norm_rotate", (PyCFunction)(void (*)(void)) & entry<head_norm_rotate, 11>, METH_FASTCALL, nullptr},
    {"page_fork", (PyCFunction)(void (*)(void)) & entry<page_fork, 13>, METH_FASTCALL, nullptr},
    {"page_compact", (PyCFunction)(void (*)(void)) & entry<page_compact, 8>, METH_FASTCALL, nullptr},
    {"page_copy", (PyCFunction)(void (*)(void)) & entry<page_copy, 7>, METH_FASTCALL, nullptr},
    {"page_gather", (PyCFunction)(void (*)(void)) & entry<page_gather, 12>, METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_pages", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pages(void) { return PyModule_Create(&g_module); }
