// call.cpp — the Python module decode_attn_call: the common case of the norm, append and
// shared-prefix calls from torch tensors to the C entry points.
//
// A decode step's calls take a few us on the GPU, and their marshalling in Python (attribute reads,
// a ctypes structure, two torch.empty) takes longer on the host of a GB300.  us a call in a loop,
// Python and here: norm and rotation of one token 20 and 7, the append of one 13 and 3, of 32 with
// their queries 27 and 7, a shared-prefix decode of 2 sequences 29 and 12.  A call is
// taken when everything is as the kernels need it: plain tensors of one device, the
// current one, sizes that fit together, for the shared prefix no capture.  Anything
// else is answered with NotImplemented, and the caller's checks in Python name what is wrong or do
// the rest.  An error status of the entry point comes back as an int.
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAStream.h>

#include <utility>

#include "../../include/decode_attn.h"

namespace {

// Entry points of the loaded libdecode_attn.so.
decltype(&decode_attn_qk_norm_rope) norm_rope_fn;
decltype(&decode_attn_append_paged_rope) append_fn;
decltype(&decode_attn_paged_prefix) prefix_fn;
decltype(&decode_attn_paged_prefix_workspace_size) prefix_ws_fn;

struct NotTaken {};  // thrown where the call is not the common case

void need(bool ok) {
  if (!ok) throw NotTaken();
}
const at::Tensor& tensor(PyObject* o) {
  need(THPVariable_CheckExact(o));
  return THPVariable_Unpack(o);
}
int64_t integer(PyObject* o) {
  need(PyLong_Check(o));
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw NotTaken();
  }
  return v;
}
float real(PyObject* o) {
  need(PyFloat_Check(o) || PyLong_Check(o));
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw NotTaken();
  }
  return (float)v;
}
bool truth(PyObject* o) {
  need(PyBool_Check(o));
  return o == Py_True;
}
int32_t i32(int64_t v) {
  need(v >= INT32_MIN && v <= INT32_MAX);
  return (int32_t)v;
}

// Data of a contiguous tensor of this type on device dev; dims < 0: of any.
void* plain(const at::Tensor& t, at::ScalarType type, int dev, int dims) {
  need(t.is_cuda() && t.get_device() == dev && t.scalar_type() == type &&
       (dims < 0 || t.dim() == dims) && t.is_contiguous());
  return t.data_ptr();
}
void* plain_or_null(PyObject* o, at::ScalarType type, int dev, int dims) {
  return o == Py_None ? nullptr : plain(tensor(o), type, dev, dims);
}

// A [tokens, heads, D] view with contiguous rows.
struct Rows {
  const void* p = nullptr;
  int64_t n = 0, h = 0, d = 0, ts = 0, hs = 0;
  Rows() = default;
  Rows(const at::Tensor& t, at::ScalarType type, int dev) {
    need(t.is_cuda() && t.get_device() == dev && t.scalar_type() == type && t.dim() == 3);
    n = t.size(0), h = t.size(1), d = t.size(2);
    need(n > 0 && (t.stride(2) == 1 || d == 1));
    ts = n > 1 ? t.stride(0) : 0;
    hs = h > 1 ? t.stride(1) : 0;
    p = t.data_ptr();
  }
};

// The device of x, which has to be the current one; its stream.
int device(const at::Tensor& x) {
  need(x.is_cuda() && x.get_device() == c10::cuda::current_device());
  return x.get_device();
}
void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(dev).stream(); }

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, int dev) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, dev));
}

da_rope_params rope_params(at::ScalarType type, int64_t d, int dev, PyObject* freqs, PyObject* norm,
                           PyObject* q_weight, PyObject* k_weight, PyObject* weight_offset,
                           PyObject* eps, PyObject* interleaved, const Rows& q, const Rows& k,
                           const Rows& v) {
  da_rope_params r = {};
  need(type == at::kFloat || type == at::kHalf || type == at::kBFloat16);
  r.type = type == at::kFloat ? DA_TYPE_F32 : type == at::kHalf ? DA_TYPE_F16 : DA_TYPE_BF16;
  r.freqs = static_cast<const uint64_t*>(plain_or_null(freqs, at::kLong, dev, 1));
  r.rotary_dim = r.freqs ? i32(2 * tensor(freqs).size(0)) : 0;
  r.interleaved = truth(interleaved);
  r.norm = truth(norm);
  r.eps = real(eps);
  r.weight_offset = real(weight_offset);
  r.q_token_stride = q.ts, r.q_head_stride = q.hs;
  r.k_token_stride = k.ts, r.k_head_stride = k.hs;
  r.v_token_stride = v.ts, r.v_head_stride = v.hs;
  for (PyObject* w : {q_weight, k_weight})
    need(w == Py_None || (r.norm && tensor(w).dim() == 1 && tensor(w).size(0) == d));
  r.q_weight = static_cast<const float*>(plain_or_null(q_weight, at::kFloat, dev, 1));
  r.k_weight = static_cast<const float*>(plain_or_null(k_weight, at::kFloat, dev, 1));
  return r;
}

// An output that the caller gave, or a new one.
struct Output {
  PyObject* given = nullptr;
  at::Tensor made;
  void* p = nullptr;
  Output() = default;
  Output(PyObject* o, at::IntArrayRef shape, at::ScalarType type, int dev) {
    if (o == Py_None) {
      made = empty(shape, type, dev);
      p = made.data_ptr();
      need(p);
    } else {
      need(tensor(o).sizes() == shape);
      p = plain(tensor(o), type, dev, (int)shape.size());
      given = o;
    }
  }
  // None where there is none.
  PyObject* object() {
    if (made.defined()) return THPVariable_Wrap(std::move(made));
    PyObject* o = given ? given : Py_None;
    Py_INCREF(o);
    return o;
  }
};

PyObject* pair(PyObject* a, PyObject* b) {
  PyObject* t = a && b ? PyTuple_New(2) : nullptr;
  if (!t) {
    Py_XDECREF(a);
    Py_XDECREF(b);
    return nullptr;
  }
  PyTuple_SET_ITEM(t, 0, a);
  PyTuple_SET_ITEM(t, 1, b);
  return t;
}

// q, k, positions, freqs, norm, q_weight, k_weight, weight_offset, eps, interleaved, q_out, k_out
PyObject* norm_rope(PyObject* const* a) {
  const bool has_q = a[0] != Py_None, has_k = a[1] != Py_None;
  need(has_q || has_k);
  const at::Tensor& x = tensor(a[has_q ? 0 : 1]);
  const int dev = device(x);
  const at::ScalarType type = x.scalar_type();
  const Rows q = has_q ? Rows(x, type, dev) : Rows();
  const Rows k = has_k ? Rows(tensor(a[1]), type, dev) : Rows();
  const int64_t n = has_q ? q.n : k.n, d = has_q ? q.d : k.d;
  need(!has_k || (k.n == n && k.d == d));
  const auto* pos = static_cast<const int32_t*>(plain_or_null(a[2], at::kInt, dev, 1));
  need(pos ? tensor(a[2]).size(0) == n : a[3] == Py_None);
  const da_rope_params r =
      rope_params(type, d, dev, a[3], a[4], a[5], a[6], a[7], a[8], a[9], q, k, Rows());
  need((has_q || a[10] == Py_None) && (has_k || a[11] == Py_None));
  Output qo, ko;
  if (has_q) qo = Output(a[10], {n, q.h, d}, at::kFloat, dev);
  if (has_k) ko = Output(a[11], {n, k.h, d}, at::kHalf, dev);
  const int st = norm_rope_fn(&r, i32(n), i32(q.h), i32(k.h), i32(d), q.p, k.p, pos,
                              static_cast<float*>(qo.p), static_cast<uint16_t*>(ko.p),
                              stream_of(dev));
  if (st != DA_OK) return PyLong_FromLong(st);
  return pair(qo.object(), ko.object());
}

// k_new, v_new, positions, block_table, k_pool, v_pool, freqs, token_seq, q, norm, q_weight,
// k_weight, weight_offset, eps, interleaved, q_out, dev_status
PyObject* append(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0]);
  const int dev = device(x);
  const at::ScalarType type = x.scalar_type();
  const bool has_q = a[8] != Py_None;
  const Rows k(x, type, dev), v(tensor(a[1]), type, dev);
  const Rows q = has_q ? Rows(tensor(a[8]), type, dev) : Rows();
  need(v.n == k.n && v.h == k.h && v.d == k.d);
  need(has_q ? q.n == k.n && q.d == k.d : a[15] == Py_None);
  const at::Tensor &pos = tensor(a[2]), &table = tensor(a[3]), &kp = tensor(a[4]),
                   &vp = tensor(a[5]);
  const auto* pos_p = static_cast<const int32_t*>(plain(pos, at::kInt, dev, 1));
  const auto* table_p = static_cast<const int32_t*>(plain(table, at::kInt, dev, 2));
  auto* kp_p = static_cast<uint16_t*>(plain(kp, at::kHalf, dev, 4));
  auto* vp_p = static_cast<uint16_t*>(plain(vp, at::kHalf, dev, 4));
  need(vp.sizes() == kp.sizes() && kp.size(2) == k.h && kp.size(3) == k.d && pos.size(0) == k.n);
  const auto* seq = static_cast<const int32_t*>(plain_or_null(a[7], at::kInt, dev, 1));
  need(!seq || tensor(a[7]).size(0) == k.n);
  auto* status = static_cast<int32_t*>(plain_or_null(a[16], at::kInt, dev, -1));
  const da_rope_params r =
      rope_params(type, k.d, dev, a[6], a[9], a[10], a[11], a[12], a[13], a[14], q, k, v);
  da_params p = {};
  p.batch = i32(table.size(0));
  p.num_q_heads = i32(has_q ? q.h : k.h);
  p.num_kv_heads = i32(k.h);
  p.head_dim = i32(k.d);
  p.block_size = i32(kp.size(1));
  p.max_blocks_per_seq = i32(table.size(1));
  p.num_blocks = i32(kp.size(0));
  p.causal = 1;
  Output qo;
  if (has_q) qo = Output(a[15], {q.n, q.h, q.d}, at::kFloat, dev);
  const int st = append_fn(&p, &r, i32(k.n), q.p, k.p, v.p, pos_p, seq, table_p,
                           static_cast<float*>(qo.p), kp_p, vp_p, status, stream_of(dev));
  if (st != DA_OK) return PyLong_FromLong(st);
  return qo.object();
}

// q, k_pool, v_pool, block_table, seq_lens, prefix_len, prefix_table, q_pos, scale, softcap,
// sliding_window, causal, max_seq_len, out, lse, dev_status
PyObject* prefix(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0]);
  const int dev = device(q);
  // captured calls go through Python
  need(c10::cuda::currentStreamCaptureStatusMayInitCtx() == c10::cuda::CaptureStatus::None);
  need(q.dim() == 3 || q.dim() == 4);
  const at::Tensor &kp = tensor(a[1]), &vp = tensor(a[2]), &table = tensor(a[3]),
                   &lens = tensor(a[4]);
  const int64_t B = q.size(0), T = q.dim() == 4 ? q.size(1) : 1, Hq = q.size(-2), D = q.size(-1);
  const auto* qp = static_cast<const float*>(plain(q, at::kFloat, dev, (int)q.dim()));
  const auto* kpp = static_cast<const uint16_t*>(plain(kp, at::kHalf, dev, 4));
  const auto* vpp = static_cast<const uint16_t*>(plain(vp, at::kHalf, dev, 4));
  const auto* tp = static_cast<const int32_t*>(plain(table, at::kInt, dev, 2));
  const auto* lp = static_cast<const int32_t*>(plain(lens, at::kInt, dev, 1));
  const int64_t bs = kp.size(1), len = integer(a[5]);
  need(B > 0 && vp.sizes() == kp.sizes() && kp.size(3) == D && table.size(0) == B &&
       lens.size(0) == B && bs > 0 && len >= 0);
  const auto* pt = a[6] == Py_None
                       ? tp  // its first row
                       : static_cast<const int32_t*>(plain(tensor(a[6]), at::kInt, dev, 1));
  need(a[6] == Py_None || tensor(a[6]).size(0) >= len / bs);
  const auto* pos = static_cast<const int32_t*>(plain_or_null(a[7], at::kInt, dev, 1));
  need(!pos || tensor(a[7]).size(0) == B);
  auto* status = static_cast<int32_t*>(plain_or_null(a[15], at::kInt, dev, -1));
  da_params p = {};
  p.batch = i32(B);
  p.num_q_heads = i32(Hq);
  p.num_kv_heads = i32(kp.size(2));
  p.head_dim = i32(D);
  p.block_size = i32(bs);
  p.max_blocks_per_seq = i32(table.size(1));
  p.num_blocks = i32(kp.size(0));
  p.max_seq_len = i32(integer(a[12]));
  p.scale = real(a[8]);
  p.softcap = real(a[9]);
  p.sliding_window = i32(integer(a[10]));
  p.causal = truth(a[11]);
  const size_t bytes = prefix_ws_fn(&p, i32(T), i32(len));
  need(bytes > 0);
  Output out(a[13], q.sizes(), at::kFloat, dev);
  Output lse(a[14], q.sizes().slice(0, q.dim() - 1), at::kFloat, dev);
  // the call's own, as in Python; its memory goes to the stream's later calls
  const at::Tensor ws = empty({(int64_t)bytes}, at::kByte, dev);
  const int st = prefix_fn(&p, i32(T), i32(len), pt, qp, kpp, vpp, tp, lp, pos,
                           static_cast<float*>(out.p), static_cast<float*>(lse.p), ws.data_ptr(),
                           bytes, status, stream_of(dev));
  if (st != DA_OK) return PyLong_FromLong(st);
  return pair(out.object(), lse.object());
}

template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N || !norm_rope_fn) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments, or bind() was not called");
    return nullptr;
  }
  try {
    return F(args);
  } catch (...) {  // also what torch throws: the caller's own path then says what it is
    PyErr_Clear();
    Py_RETURN_NOTIMPLEMENTED;
  }
}

// Addresses of the four entry points.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "four addresses are needed");
    return nullptr;
  }
  void* f[4];
  for (int i = 0; i < 4; ++i) {
    f[i] = PyLong_AsVoidPtr(args[i]);
    if (!f[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
      return nullptr;
    }
  }
  append_fn = reinterpret_cast<decltype(append_fn)>(f[1]);
  prefix_fn = reinterpret_cast<decltype(prefix_fn)>(f[2]);
  prefix_ws_fn = reinterpret_cast<decltype(prefix_ws_fn)>(f[3]);
  norm_rope_fn = reinterpret_cast<decltype(norm_rope_fn)>(f[0]);
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction method(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"bind", method(bind), METH_FASTCALL, nullptr},
    {"norm_rope", method(entry<norm_rope, 12>), METH_FASTCALL, nullptr},
    {"append", method(entry<append, 17>), METH_FASTCALL, nullptr},
    {"prefix", method(entry<prefix, 16>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "decode_attn_call", nullptr, -1, methods,
                      nullptr,               nullptr,            nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_decode_attn_call() { return PyModule_Create(&module); }
