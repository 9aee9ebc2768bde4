// Python calls of the serving step's operators (norm and rotation, attention of
// trees and over shared prefixes, the cache's pages, a step's tables, sampling): argument checks, output allocation and the
// call of the C entry point of the same name in libmsa.so. A call of these
// takes a few microseconds on the GPU for a decode step, less than checking a
// dozen tensors does in Python, hence a compiled binding: against the same
// checks in Python with ctypes, an append of four tokens (64 query heads, 4 KV
// heads) went from 52 to 21 us, 16 of which are the caller's slicing of its
// inputs; its kernel is 4.0 us.
//
// Arguments come by position from the Python functions that document them.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <optional>
#include <sstream>
#include <string>
#include <vector>

#include "../../include/msa.h"

namespace {

using at::Tensor;
using Shape = std::initializer_list<int64_t>;  // -1: any size

PyObject* g_error = nullptr;  // MSAError(name, status)

[[noreturn]] void bad_value(const std::string& s) {
  TORCH_CHECK_VALUE(false, s);
  __builtin_unreachable();
}
[[noreturn]] void bad_type(const std::string& s) {
  TORCH_CHECK_TYPE(false, s);
  __builtin_unreachable();
}

const Tensor& tensor(const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) bad_type(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

template <class A>
std::string sizes_text(const A& s) {
  std::ostringstream o;
  o << '(';
  for (auto n : s) {
    if (n < 0) o << "any, ";
    else o << n << ", ";
  }
  o << ')';
  return o.str();
}

bool is_16bit(at::ScalarType t) { return t == at::kBFloat16 || t == at::kHalf; }
bool is_kv(at::ScalarType t) { return is_16bit(t) || t == at::kFloat8_e4m3fn || t == at::kByte; }
msa_dtype_t code(at::ScalarType t) {
  return t == at::kBFloat16 ? MSA_BF16 : t == at::kHalf ? MSA_FP16 : MSA_FP8_E4M3;
}

// The place and shape of one tensor argument.
template <class A>
void check_shape(const char* name, const Tensor& t, const A& shape) {
  bool ok = t.dim() == (int64_t)shape.size();
  if (ok) {
    int64_t i = 0;
    for (int64_t n : shape) {
      ok = ok && (n < 0 || t.size(i) == n);
      ++i;
    }
  }
  if (!ok) bad_value(std::string(name) + " must have shape " + sizes_text(shape) + ", got " + sizes_text(t.sizes()));
}
void check_place(const char* name, const Tensor& t, const at::Device* dev) {
  if (!t.is_cuda()) bad_value(std::string(name) + " must be a CUDA tensor");
  if (dev != nullptr && t.device() != *dev) bad_value(std::string(name) + " must be on " + dev->str());
}
[[noreturn]] void wrong_dtype(const char* name, const Tensor& t, const char* want) {
  bad_type(std::string(name) + " must be " + want + ", got " + at::toString(t.scalar_type()));
}
template <class A = Shape>
const Tensor& dense(const char* name, PyObject* o, const at::Device* dev, at::ScalarType dtype, const A& shape) {
  const Tensor& t = tensor(name, o);
  check_place(name, t, dev);
  if (t.scalar_type() != dtype) wrong_dtype(name, t, at::toString(dtype));
  check_shape(name, t, shape);
  if (!t.is_contiguous()) bad_value(std::string(name) + " must be contiguous");
  return t;
}
const Tensor& dense(const char* name, PyObject* o, const at::Device* dev, at::ScalarType dtype, Shape shape) {
  return dense<Shape>(name, o, dev, dtype, shape);
}

// A (tokens, heads, 128) tensor whose heads are contiguous; its token stride.
long long token_stride(const char* name, const Tensor& t) {
  if (t.numel() > 0 && (t.stride(2) != 1 || (t.size(1) > 1 && t.stride(1) != t.size(2))))
    bad_value(std::string(name) + ": each token's heads must be contiguous");
  return t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2);
}
template <class A>
const Tensor& heads(const char* name, PyObject* o, const at::Device* dev, at::ScalarType dtype, const A& shape,
                    long long* stride) {
  const Tensor& t = tensor(name, o);
  check_place(name, t, dev);
  if (t.scalar_type() != dtype) wrong_dtype(name, t, at::toString(dtype));
  check_shape(name, t, shape);
  *stride = token_stride(name, t);
  return t;
}

int as_int(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  if (v > INT32_MAX || v < INT32_MIN) bad_value("an integer argument is out of range");
  return (int)v;
}
float as_float(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return (float)v;
}
int as_flag(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v;
}
int size32(const char* name, int64_t n) {
  if (n > INT32_MAX) bad_value(std::string(name) + ": a size above 2^31 - 1");
  return (int)n;
}

// The device and stream a call runs on. Outputs and workspaces are allocated
// on that stream, which is where the allocator may hand them out again.
class Place {
 public:
  Place(const at::Device& dev, PyObject* stream) : guard_(dev) {
    if (stream == Py_None) {
      stream_ = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
      return;
    }
    PyObject* raw = PyObject_HasAttrString(stream, "cuda_stream") ? PyObject_GetAttrString(stream, "cuda_stream")
                                                                  : Py_NewRef(stream);
    if (raw == nullptr) throw python_error();
    const unsigned long long handle = PyLong_AsUnsignedLongLong(raw);
    Py_DECREF(raw);
    if (PyErr_Occurred()) throw python_error();
    stream_ = reinterpret_cast<cudaStream_t>(handle);
    if (stream_ != c10::cuda::getCurrentCUDAStream(dev.index()).stream())
      under_.emplace(c10::cuda::getStreamFromExternal(stream_, dev.index()));
  }
  cudaStream_t stream() const { return stream_; }

 private:
  c10::cuda::CUDAGuard guard_;
  std::optional<c10::cuda::CUDAStreamGuard> under_;
  cudaStream_t stream_ = nullptr;
};

Tensor fresh(at::IntArrayRef shape, at::ScalarType dtype, const at::Device& dev) {
  return at::empty(shape, at::TensorOptions().dtype(dtype).device(dev));
}
template <class A>
Tensor output(const char* name, PyObject* o, const at::Device& dev, at::ScalarType dtype, const A& shape) {
  if (o == Py_None) return fresh(shape, dtype, dev);
  return dense(name, o, &dev, dtype, shape);
}
Tensor workspace(PyObject* o, const at::Device& dev, size_t need) {
  if (o == Py_None) return fresh({(int64_t)(need < 256 ? 256 : need)}, at::kByte, dev);
  return dense("workspace", o, &dev, at::kByte, {-1});
}

void check(const char* name, msa_status_t st) {
  if (st == MSA_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "si", name, (int)st);
  if (e != nullptr) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw python_error();
}

template <class T>
T* ptr(const Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

PyObject* tuple_of(std::initializer_list<Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (r == nullptr) throw python_error();
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) PyTuple_SET_ITEM(r, i++, t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None));
  return r;
}

void want_args(const char* name, Py_ssize_t got, Py_ssize_t want) {
  if (got != want) bad_type(std::string(name) + ": wrong number of arguments");
}

// ------------------------------------------------------------ norm, rotation
struct Rope {
  const Tensor *q, *k, *wq, *wk, *positions;
  const float* cos_sin = nullptr;
  int most = INT32_MAX, rotary = 0, tokens, hq, hkv;
  long long qs, ks;
  at::Device dev;
  at::ScalarType dtype;
};
Rope rope_args(PyObject* const* a) {  // q, k, q_weight, k_weight, cos_sin, positions
  const Tensor& q = tensor("q", a[0]);
  check_place("q", q, nullptr);
  if (!is_16bit(q.scalar_type())) wrong_dtype("q", q, "bfloat16 or float16");
  check_shape("q", q, Shape{-1, -1, 128});
  Rope r{&q, nullptr, nullptr, nullptr, nullptr, nullptr, INT32_MAX, 0, 0, 0, 0, 0, 0, q.device(), q.scalar_type()};
  r.qs = token_stride("q", q);
  r.k = &heads("k", a[1], &r.dev, r.dtype, Shape{q.size(0), -1, 128}, &r.ks);
  r.wq = &dense("q_weight", a[2], &r.dev, at::kFloat, {128});
  r.wk = &dense("k_weight", a[3], &r.dev, at::kFloat, {128});
  if (a[4] != Py_None) {
    const Tensor& t = dense("cos_sin", a[4], &r.dev, at::kFloat, {-1, -1});
    r.cos_sin = ptr<const float>(t);
    r.most = (int)std::min<int64_t>(t.size(0), INT32_MAX);
    r.rotary = size32("cos_sin", t.size(1));
  }
  r.positions = &dense("positions", a[5], &r.dev, at::kInt, {q.size(0)});
  r.tokens = size32("q", q.size(0)), r.hq = size32("q", q.size(1)), r.hkv = size32("k", r.k->size(1));
  return r;
}

// q, k, q_weight, k_weight, cos_sin, positions, eps, interleaved, q_out, k_out, stream
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want_args("msa_qk_norm_rope", n, 11);
  const Rope r = rope_args(a);
  const Place place(r.dev, a[10]);
  const Tensor qo = output("q_out", a[8], r.dev, r.dtype, r.q->sizes());
  const Tensor ko = output("k_out", a[9], r.dev, r.dtype, r.k->sizes());
  check("msa_qk_norm_rope",
        msa_qk_norm_rope(r.q->data_ptr(), r.qs, r.k->data_ptr(), r.ks, code(r.dtype), ptr<const float>(*r.wq),
                         ptr<const float>(*r.wk), as_float(a[6]), r.cos_sin, r.most, r.rotary, as_flag(a[7]),
                         ptr<const int32_t>(*r.positions), r.tokens, r.hq, r.hkv, 128, qo.data_ptr(), ko.data_ptr(),
                         place.stream()));
  return tuple_of({qo, ko});
  END_HANDLE_TH_ERRORS
}

// q, k, q_weight, k_weight, cos_sin, positions, eps, interleaved, v,
// cu_seqlens_q, k_pool, v_pool, page_table, seqused_k, q_out, stream
PyObject* qk_norm_rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want_args("msa_qk_norm_rope_append", n, 16);
  const Rope r = rope_args(a);
  long long vs;
  const Tensor& v = heads("v", a[8], &r.dev, r.dtype, r.k->sizes(), &vs);
  const Tensor& cu = dense("cu_seqlens_q", a[9], &r.dev, at::kInt, {-1});
  const int64_t batch = cu.size(0) - 1;
  const Tensor& kp = tensor("k_pool", a[10]);
  if (!is_kv(kp.scalar_type())) wrong_dtype("k_pool", kp, "bfloat16, float16 or float8_e4m3fn");
  dense("k_pool", a[10], &r.dev, kp.scalar_type(), {-1, r.hkv, 128, 128});
  const Tensor& vp = dense("v_pool", a[11], &r.dev, kp.scalar_type(), kp.sizes());
  const Tensor& pt = dense("page_table", a[12], &r.dev, at::kInt, {batch < 0 ? 0 : batch, -1});
  const Tensor& used = dense("seqused_k", a[13], &r.dev, at::kInt, {batch < 0 ? 0 : batch});
  const Place place(r.dev, a[15]);
  const Tensor qo = output("q_out", a[14], r.dev, r.dtype, r.q->sizes());
  check("msa_qk_norm_rope_append",
        msa_qk_norm_rope_append(
            r.q->data_ptr(), r.qs, r.k->data_ptr(), r.ks, v.data_ptr(), vs, code(r.dtype), ptr<const float>(*r.wq),
            ptr<const float>(*r.wk), as_float(a[6]), r.cos_sin, r.most, r.rotary, as_flag(a[7]),
            ptr<const int32_t>(*r.positions), ptr<const int32_t>(cu), size32("cu_seqlens_q", batch),
            ptr<const int32_t>(pt), size32("page_table", pt.size(1)), size32("k_pool", kp.size(0)),
            ptr<const int32_t>(used), r.tokens, r.hq, r.hkv, 128, qo.data_ptr(), kp.data_ptr(), vp.data_ptr(),
            code(kp.scalar_type()), place.stream()));
  return THPVariable_Wrap(qo);
  END_HANDLE_TH_ERRORS
}

// q, k, q_weight, k_weight, cos_sin, positions, eps, interleaved, dq_out,
// dk_out, dq, dk, dq_weight, dk_weight, workspace, stream
PyObject* qk_norm_rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want_args("msa_qk_norm_rope_bwd", n, 16);
  const Rope r = rope_args(a);
  const Tensor& dqo = dense("dq_out", a[8], &r.dev, r.dtype, r.q->sizes());
  const Tensor& dko = dense("dk_out", a[9], &r.dev, r.dtype, r.k->sizes());
  const Place place(r.dev, a[15]);
  long long dqs = 128ll * r.hq, dks = 128ll * r.hkv;
  const Tensor dq = a[10] == Py_None ? fresh(r.q->sizes(), r.dtype, r.dev)
                                     : heads("dq", a[10], &r.dev, r.dtype, r.q->sizes(), &dqs);
  const Tensor dk = a[11] == Py_None ? fresh(r.k->sizes(), r.dtype, r.dev)
                                     : heads("dk", a[11], &r.dev, r.dtype, r.k->sizes(), &dks);
  const Tensor dwq = output("dq_weight", a[12], r.dev, at::kFloat, Shape{128});
  const Tensor dwk = output("dk_weight", a[13], r.dev, at::kFloat, Shape{128});
  const Tensor ws = workspace(a[14], r.dev, msa_qk_norm_rope_bwd_workspace_size(r.tokens, r.hq, r.hkv));
  check("msa_qk_norm_rope_bwd",
        msa_qk_norm_rope_bwd(dqo.data_ptr(), dko.data_ptr(), r.q->data_ptr(), r.qs, r.k->data_ptr(), r.ks,
                             code(r.dtype), ptr<const float>(*r.wq), ptr<const float>(*r.wk), as_float(a[6]),
                             r.cos_sin, r.most, r.rotary, as_flag(a[7]), ptr<const int32_t>(*r.positions), r.tokens,
                             r.hq, r.hkv, 128, dq.data_ptr(), dqs, dk.data_ptr(), dks, ptr<float>(dwq), ptr<float>(dwk),
                             ws.data_ptr(), (size_t)ws.numel(), place.stream()));
  return tuple_of({dq, dk, dwq, dwk});
  END_HANDLE_TH_ERRORS
}

// -------------------------------------------------------------- tree attention
// q, k, v, q2k_indices, cu_seqlens_q, tree_mask, page_table, seqused_k,
// max_seqlen_q, softmax_scale (or None), return_softmax_lse, out, lse,
// workspace, stream, prepare: (out, lse or None, workspace, plan or None).
PyObject* tree_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want_args("msa_tree_attention", n, 16);
  const Tensor& q = tensor("q", a[0]);
  check_place("q", q, nullptr);
  if (!is_16bit(q.scalar_type())) wrong_dtype("q", q, "bfloat16 or float16");
  dense("q", a[0], nullptr, q.scalar_type(), {-1, -1, 128});
  const at::Device dev = q.device();
  const Tensor& k = tensor("k", a[1]);
  if (!is_kv(k.scalar_type())) wrong_dtype("k", k, "bfloat16, float16 or float8_e4m3fn");
  dense("k", a[1], &dev, k.scalar_type(), {-1, -1, 128, 128});
  const Tensor& v = dense("v", a[2], &dev, k.scalar_type(), k.sizes());
  const Tensor& lists = dense("q2k_indices", a[3], &dev, at::kInt, {k.size(1), q.size(0), -1});
  const Tensor& cu = dense("cu_seqlens_q", a[4], &dev, at::kInt, {-1});
  const int64_t rows = cu.size(0) > 0 ? cu.size(0) - 1 : 0;
  const Tensor& mask = tensor("tree_mask", a[5]);
  if (mask.scalar_type() != at::kInt && mask.scalar_type() != at::kUInt32) wrong_dtype("tree_mask", mask, "int32 or uint32");
  dense("tree_mask", a[5], &dev, mask.scalar_type(), {q.size(0), -1});
  const Tensor& pt = dense("page_table", a[6], &dev, at::kInt, {rows, -1});
  const Tensor& used = dense("seqused_k", a[7], &dev, at::kInt, {rows});
  const int max_q = as_int(a[8]);
  const float scale = a[9] == Py_None ? 0.f : as_float(a[9]);
  const Place place(dev, a[14]);
  const int total = size32("q", q.size(0)), hq = size32("q", q.size(1)), hkv = size32("k", k.size(1));
  const int topk = size32("q2k_indices", lists.size(2)), words = size32("tree_mask", mask.size(1));
  const int max_pages = size32("page_table", pt.size(1)), pages = size32("k", k.size(0)), batch = size32("cu", rows);
  const msa_dtype_t qt = code(q.scalar_type()), kt = code(k.scalar_type());
  const Tensor out = output("out", a[11], dev, q.scalar_type(), q.sizes());
  Tensor lse;
  if (a[12] != Py_None || as_flag(a[10])) lse = output("lse", a[12], dev, at::kFloat, Shape{total, hq});
  const Tensor ws = workspace(a[13], dev, msa_tree_attention_workspace_size(batch, total, hq, hkv, 128, topk, max_q));
  const bool prepare = as_flag(a[15]);
  msa_attention_plan_t* plan = nullptr;
#define MSA_TREE_CALL                                                                                        \
  q.data_ptr(), qt, k.data_ptr(), v.data_ptr(), kt, ptr<const int32_t>(lists), topk, ptr<const int32_t>(cu), \
      ptr<const uint32_t>(mask), words, ptr<const int32_t>(pt), max_pages, pages, ptr<const int32_t>(used),  \
      batch, total, hq, hkv, 128, max_q, scale, out.data_ptr(), lse.defined() ? ptr<float>(lse) : nullptr,   \
      ws.data_ptr(), (size_t)ws.numel()
  if (prepare) check("msa_tree_attention_prepare", msa_tree_attention_prepare(MSA_TREE_CALL, &plan));
  else if (total > 0) check("msa_tree_attention", msa_tree_attention(MSA_TREE_CALL, place.stream()));
#undef MSA_TREE_CALL
  PyObject* r = tuple_of({out, lse, ws, Tensor()});
  if (prepare) {
    Py_DECREF(PyTuple_GET_ITEM(r, 3));
    PyTuple_SET_ITEM(r, 3, PyLong_FromVoidPtr(plan));
  }
  return r;
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------- attention, shared prefixes
// q, k, v, cu_seqlens_q, page_table, seqused_k, group_rows, cu_groups,
// group_blocks (or None), max_seqlen_q (or None), causal, softmax_scale (or
// None), return_softmax_lse, out, lse, workspace, stream, prepare: (out, lse or
// None, workspace, plan or None).
PyObject* prefix_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want_args("msa_prefix_attention", n, 18);
  const Tensor& q = tensor("q", a[0]);
  check_place("q", q, nullptr);
  if (!is_16bit(q.scalar_type())) wrong_dtype("q", q, "bfloat16 or float16");
  dense("q", a[0], nullptr, q.scalar_type(), {-1, -1, 128});
  const at::Device dev = q.device();
  const Tensor& k = tensor("k", a[1]);
  if (!is_kv(k.scalar_type())) wrong_dtype("k", k, "bfloat16, float16 or float8_e4m3fn");
  dense("k", a[1], &dev, k.scalar_type(), {-1, -1, 128, 128});
  const Tensor& v = dense("v", a[2], &dev, k.scalar_type(), k.sizes());
  const Tensor& cu = dense("cu_seqlens_q", a[3], &dev, at::kInt, {-1});
  const int64_t rows = cu.size(0) > 0 ? cu.size(0) - 1 : 0;
  const Tensor& pt = dense("page_table", a[4], &dev, at::kInt, {rows, -1});
  const Tensor& used = dense("seqused_k", a[5], &dev, at::kInt, {rows});
  const int given = (a[6] != Py_None) + (a[7] != Py_None) + (a[8] != Py_None);
  if (given != 0 && given != 3) bad_value("group_rows, cu_groups and group_blocks go together");
  const int32_t *group_rows = nullptr, *cu_groups = nullptr, *blocks = nullptr;
  if (given) {
    group_rows = ptr<const int32_t>(dense("group_rows", a[6], &dev, at::kInt, {rows}));
    cu_groups = ptr<const int32_t>(dense("cu_groups", a[7], &dev, at::kInt, {rows + 1}));
    blocks = ptr<const int32_t>(dense("group_blocks", a[8], &dev, at::kInt, {rows}));
  }
  const int max_q = a[9] == Py_None ? 0 : as_int(a[9]);
  const int causal = as_flag(a[10]);
  const float scale = a[11] == Py_None ? 0.f : as_float(a[11]);
  const Place place(dev, a[16]);
  const int total = size32("q", q.size(0)), hq = size32("q", q.size(1)), hkv = size32("k", k.size(1));
  const int max_pages = size32("page_table", pt.size(1)), pages = size32("k", k.size(0)), batch = size32("cu", rows);
  const msa_dtype_t qt = code(q.scalar_type()), kt = code(k.scalar_type());
  const Tensor out = output("out", a[13], dev, q.scalar_type(), q.sizes());
  Tensor lse;
  if (a[14] != Py_None || as_flag(a[12])) lse = output("lse", a[14], dev, at::kFloat, Shape{total, hq});
  const Tensor ws = workspace(a[15], dev, msa_prefix_attention_workspace_size(batch, total, hq, hkv, 128, given));
  const bool prepare = as_flag(a[17]);
  msa_attention_plan_t* plan = nullptr;
  // Tensors without tokens have no memory: the workspace stands for them, and is not followed.
  void *qp = total > 0 ? q.data_ptr() : ws.data_ptr(), *op = total > 0 ? out.data_ptr() : ws.data_ptr();
#define MSA_PREFIX_CALL                                                                                          \
  qp, qt, k.data_ptr(), v.data_ptr(), kt, ptr<const int32_t>(cu), ptr<const int32_t>(pt), max_pages,   \
      pages, ptr<const int32_t>(used), group_rows, cu_groups, blocks, batch, total, hq, hkv, 128, max_q, causal, \
      scale, op, lse.defined() ? ptr<float>(lse) : nullptr, ws.data_ptr(), (size_t)ws.numel()
  if (prepare) check("msa_prefix_attention_prepare", msa_prefix_attention_prepare(MSA_PREFIX_CALL, &plan));
  else if (total > 0) check("msa_prefix_attention", msa_prefix_attention(MSA_PREFIX_CALL, place.stream()));
#undef MSA_PREFIX_CALL
  PyObject* r = tuple_of({out, lse, ws, Tensor()});
  if (prepare) {
    Py_DECREF(PyTuple_GET_ITEM(r, 3));
    PyTuple_SET_ITEM(r, 3, PyLong_FromVoidPtr(plan));
  }
  return r;
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------ the cache
// The pools of a cache: a list or tuple of tensors (num_pages, ...) of one
// shape and dtype, or one tensor with a leading dimension over them.
struct Pools {
  std::vector<void*> at;
  int64_t pages = 0, page_bytes = 0, row_bytes = 0, kv_heads = 0;
  std::optional<at::Device> dev;
};
Pools pools_of(PyObject* o, bool rows) {
  Pools p;
  at::IntArrayRef shape;
  int64_t size;
  if (THPVariable_Check(o)) {
    const Tensor& t = THPVariable_Unpack(o);
    check_place("pools", t, nullptr);
    if (t.dim() < 3 || t.size(0) < 1) bad_value("pools must have shape (num_pools, num_pages, ...)");
    int64_t want = 1;
    for (int64_t d = t.dim() - 1; d >= 1; --d) {
      if (t.size(d) > 1 && t.stride(d) != want) bad_value("pools: each pool must be contiguous");
      want *= t.size(d);
    }
    p.dev = t.device();
    size = t.element_size();
    for (int64_t i = 0; i < t.size(0); ++i)
      p.at.push_back(static_cast<char*>(t.data_ptr()) + i * t.stride(0) * size);
    shape = t.sizes().slice(1);
  } else {
    PyObject* list = PySequence_Fast(o, "pools must be tensors");
    if (list == nullptr) throw python_error();
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(list);
    std::vector<Tensor> ts;
    try {
      for (Py_ssize_t i = 0; i < n; ++i) ts.push_back(tensor("pools", PySequence_Fast_GET_ITEM(list, i)));
    } catch (...) {
      Py_DECREF(list);
      throw;
    }
    Py_DECREF(list);
    if (ts.empty() || ts[0].dim() < 2) bad_value("pools must be tensors of shape (num_pages, ...)");
    check_place("pools", ts[0], nullptr);
    p.dev = ts[0].device();
    size = ts[0].element_size();
    shape = ts[0].sizes();
    for (const Tensor& t : ts) {
      check_place("pools", t, &*p.dev);
      if (t.scalar_type() != ts[0].scalar_type()) bad_type("pools must share one dtype");
      check_shape("pools", t, shape);
      if (!t.is_contiguous()) bad_value("pools must be contiguous");
      p.at.push_back(t.data_ptr());
    }
  }
  p.pages = shape[0];
  p.page_bytes = size;
  for (size_t i = 1; i < shape.size(); ++i) p.page_bytes *= shape[i];
  if (rows) {
    if (shape.size() != 4 || shape[2] != 128) bad_value("pools must have shape (num_pages, Hkv, 128, d)");
    p.kv_heads = shape[1];
    p.row_bytes = shape[3] * size;
  }
  return p;
}

struct Table {
  const Tensor *table, *used, *refs;
  int rows, width, pages;
  at::Device dev;
};
Table table_of(PyObject* const* a, const at::Device* dev) {  // page_table, seqused_k, page_refs
  const Tensor& t = dense("page_table", a[0], dev, at::kInt, {-1, -1});
  Table r{&t, nullptr, nullptr, size32("page_table", t.size(0)), size32("page_table", t.size(1)), 0, t.device()};
  r.used = &dense("seqused_k", a[1], &r.dev, at::kInt, {t.size(0)});
  r.refs = &dense("page_refs", a[2], &r.dev, at::kInt, {-1});
  r.pages = size32("page_refs", r.refs->size(0));
  return r;
}

// page_table, seqused_k, page_refs, rows, lengths, status, workspace, stream
PyObject* cache_extend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want_args("msa_cache_extend", n, 8);
  const Table t = table_of(a, nullptr);
  const Tensor& rows = dense("rows", a[3], &t.dev, at::kInt, {-1});
  const Tensor& lengths = dense("lengths", a[4], &t.dev, at::kInt, rows.sizes());
  const Place place(t.dev, a[7]);
  const int count = size32("rows", rows.size(0));
  const Tensor status = output("status", a[5], t.dev, at::kInt, rows.sizes());
  const Tensor ws = workspace(a[6], t.dev, msa_cache_workspace_size(count, t.pages));
  check("msa_cache_extend",
        msa_cache_extend(ptr<int32_t>(*t.table), t.width, t.rows, ptr<int32_t>(*t.used), ptr<int32_t>(*t.refs), t.pages,
                         ptr<const int32_t>(rows), ptr<const int32_t>(lengths), count, ptr<int32_t>(status),
                         ws.data_ptr(), (size_t)ws.numel(), place.stream()));
  return THPVariable_Wrap(status);
  END_HANDLE_TH_ERRORS
}

// page_table, seqused_k, page_refs, pools, src_rows, dst_rows, status, workspace, stream
PyObject* cache_fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want_args("msa_cache_fork", n, 9);
  const Pools p = pools_of(a[3], false);
  const Table t = table_of(a, &*p.dev);
  if (t.pages != p.pages) bad_value("page_refs must have an entry for each page of the pools");
  const Tensor& src = dense("src_rows", a[4], &t.dev, at::kInt, {-1});
  const Tensor& dst = dense("dst_rows", a[5], &t.dev, at::kInt, src.sizes());
  const Place place(t.dev, a[8]);
  const int count = size32("src_rows", src.size(0));
  const Tensor status = output("status", a[6], t.dev, at::kInt, src.sizes());
  const Tensor ws = workspace(a[7], t.dev, msa_cache_workspace_size(count, t.pages));
  check("msa_cache_fork",
        msa_cache_fork(p.at.data(), (int)p.at.size(), p.page_bytes, ptr<int32_t>(*t.table), t.width, t.rows,
                       ptr<int32_t>(*t.used), ptr<int32_t>(*t.refs), t.pages, ptr<const int32_t>(src),
                       ptr<const int32_t>(dst), count, ptr<int32_t>(status), ws.data_ptr(), (size_t)ws.numel(),
                       place.stream()));
  return THPVariable_Wrap(status);
  END_HANDLE_TH_ERRORS
}

// page_table, seqused_k, page_refs, rows, stream
PyObject* cache_free(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want_args("msa_cache_free", n, 5);
  const Table t = table_of(a, nullptr);
  const Tensor& rows = dense("rows", a[3], &t.dev, at::kInt, {-1});
  const Place place(t.dev, a[4]);
  check("msa_cache_free",
        msa_cache_free(ptr<int32_t>(*t.table), t.width, t.rows, ptr<int32_t>(*t.used), ptr<int32_t>(*t.refs), t.pages,
                       ptr<const int32_t>(rows), size32("rows", rows.size(0)), place.stream()));
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// pools, src_pages, dst_pages, stream
PyObject* cache_copy_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want_args("msa_cache_copy_pages", n, 4);
  const Pools p = pools_of(a[0], false);
  const Tensor& src = dense("src_pages", a[1], &*p.dev, at::kInt, {-1});
  const Tensor& dst = dense("dst_pages", a[2], &*p.dev, at::kInt, src.sizes());
  const Place place(*p.dev, a[3]);
  check("msa_cache_copy_pages",
        msa_cache_copy_pages(p.at.data(), (int)p.at.size(), p.page_bytes, size32("pools", p.pages),
                             ptr<const int32_t>(src), ptr<const int32_t>(dst), size32("src_pages", src.size(0)),
                             place.stream()));
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// pools, page_table, seqused_k, cu_seqlens_q, path, path_len, seqused_out, stream
PyObject* cache_accept(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want_args("msa_cache_accept", n, 8);
  const Pools p = pools_of(a[0], true);
  const Tensor& cu = dense("cu_seqlens_q", a[3], &*p.dev, at::kInt, {-1});
  const int64_t rows = cu.size(0) > 0 ? cu.size(0) - 1 : 0;
  const Tensor& pt = dense("page_table", a[1], &*p.dev, at::kInt, {rows, -1});
  const Tensor& used = dense("seqused_k", a[2], &*p.dev, at::kInt, {rows});
  const Tensor& path = dense("path", a[4], &*p.dev, at::kInt, {rows, -1});
  const Tensor& len = dense("path_len", a[5], &*p.dev, at::kInt, {rows});
  const Place place(*p.dev, a[7]);
  const Tensor out = output("seqused_out", a[6], *p.dev, at::kInt, used.sizes());
  check("msa_cache_accept",
        msa_cache_accept(p.at.data(), (int)p.at.size(), size32("pools", p.row_bytes), size32("pools", p.kv_heads),
                         ptr<const int32_t>(pt), size32("page_table", pt.size(1)), size32("pools", p.pages),
                         size32("cu_seqlens_q", rows), ptr<const int32_t>(used), ptr<const int32_t>(cu),
                         ptr<const int32_t>(path), ptr<const int32_t>(len), size32("path", path.size(1)),
                         ptr<int32_t>(out), place.stream()));
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// -------------------------------------------------------------- a step's tables
// page_table, seqused_k, rows, new_lens, total_q, num_pages, out (or None),
// workspace, stream: a tuple of the nine tables.
PyObject* step_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want_args("msa_step_tables", n, 9);
  const Tensor& t = dense("page_table", a[0], nullptr, at::kInt, {-1, -1});
  const at::Device dev = t.device();
  const Tensor& used = dense("seqused_k", a[1], &dev, at::kInt, {t.size(0)});
  const Tensor& rows = dense("rows", a[2], &dev, at::kInt, {-1});
  const Tensor& lens = dense("new_lens", a[3], &dev, at::kInt, rows.sizes());
  const int total = as_int(a[4]), pages = as_int(a[5]);
  if (total < 0) bad_value("total_q must not be negative");
  const int64_t batch = rows.size(0), width = t.size(1);
  const Place place(dev, a[8]);
  PyObject* given[9];
  for (auto& g : given) g = Py_None;
  if (a[6] != Py_None) {
    if (!PyTuple_Check(a[6]) || PyTuple_GET_SIZE(a[6]) != 9) bad_type("out must be what a call returned");
    for (int i = 0; i < 9; ++i) given[i] = PyTuple_GET_ITEM(a[6], i);
  }
  const Tensor cu = output("cu_seqlens_q", given[0], dev, at::kInt, Shape{batch + 1});
  const Tensor used_out = output("seqused_k (out)", given[1], dev, at::kInt, Shape{batch});
  const Tensor table = output("page_table (out)", given[2], dev, at::kInt, Shape{batch, width});
  const Tensor token_rows = output("token_rows", given[3], dev, at::kInt, Shape{total});
  const Tensor positions = output("positions", given[4], dev, at::kInt, Shape{total});
  const Tensor slots = output("slots", given[5], dev, at::kLong, Shape{total});
  const Tensor group_rows = output("group_rows", given[6], dev, at::kInt, Shape{batch});
  const Tensor cu_groups = output("cu_groups", given[7], dev, at::kInt, Shape{batch + 1});
  const Tensor blocks = output("group_blocks", given[8], dev, at::kInt, Shape{batch});
  const int b = size32("rows", batch);
  const Tensor ws = workspace(a[7], dev, msa_step_tables_workspace_size(b));
  check("msa_step_tables",
        msa_step_tables(ptr<const int32_t>(t), size32("page_table", width), size32("page_table", t.size(0)),
                        ptr<const int32_t>(used), pages, ptr<const int32_t>(rows), ptr<const int32_t>(lens), b, total,
                        ptr<int32_t>(cu), ptr<int32_t>(used_out), ptr<int32_t>(table), ptr<int32_t>(token_rows),
                        ptr<int32_t>(positions), static_cast<long long*>(slots.data_ptr()), ptr<int32_t>(group_rows),
                        ptr<int32_t>(cu_groups), ptr<int32_t>(blocks), ws.data_ptr(), (size_t)ws.numel(),
                        place.stream()));
  return tuple_of({cu, used_out, table, token_rows, positions, slots, group_rows, cu_groups, blocks});
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------ tokens and paths
template <class T>
const T* optional_rows(const char* name, PyObject* o, const at::Device& dev, at::ScalarType dtype, int64_t rows) {
  return o == Py_None ? nullptr : ptr<const T>(dense(name, o, &dev, dtype, {rows}));
}

// logits, uniforms, temperature, top_k, top_p, min_p, return_logprobs, tokens,
// logprobs, workspace, stream: (tokens, logprobs or None).
PyObject* sample(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want_args("msa_sample", n, 11);
  const Tensor& x = tensor("logits", a[0]);
  check_place("logits", x, nullptr);
  if (!is_16bit(x.scalar_type()) && x.scalar_type() != at::kFloat) wrong_dtype("logits", x, "bfloat16, float16 or float32");
  check_shape("logits", x, Shape{-1, -1});
  const int64_t rows = x.size(0), vocab = x.size(1);
  if (vocab > 1 && x.stride(1) != 1) bad_value("logits: each row must be contiguous");
  const at::Device dev = x.device();
  const Tensor& u = dense("uniforms", a[1], &dev, at::kFloat, {rows});
  const float* t = optional_rows<float>("temperature", a[2], dev, at::kFloat, rows);
  const int32_t* k = optional_rows<int32_t>("top_k", a[3], dev, at::kInt, rows);
  const float* p = optional_rows<float>("top_p", a[4], dev, at::kFloat, rows);
  const float* m = optional_rows<float>("min_p", a[5], dev, at::kFloat, rows);
  const Place place(dev, a[10]);
  const Tensor tokens = output("tokens", a[7], dev, at::kInt, Shape{rows});
  Tensor logprobs;
  if (a[8] != Py_None || as_flag(a[6])) logprobs = output("logprobs", a[8], dev, at::kFloat, Shape{rows});
  const int count = size32("logits", rows), width = size32("logits", vocab);
  const msa_dtype_t dtype = x.scalar_type() == at::kFloat ? MSA_FP32 : code(x.scalar_type());
  const Tensor ws = workspace(a[9], dev, msa_sample_workspace_size(count, width, dtype));
  check("msa_sample",
        msa_sample(x.data_ptr(), dtype,
                   rows > 1 ? x.stride(0) : vocab, count, width, ptr<const float>(u), t, k, p, m, ptr<int32_t>(tokens),
                   logprobs.defined() ? ptr<float>(logprobs) : nullptr, ws.data_ptr(), (size_t)ws.numel(),
                   place.stream()));
  return tuple_of({tokens, logprobs});
  END_HANDLE_TH_ERRORS
}

// sampled, drafts, tree_mask, cu_seqlens_q, max_path (or None), path, path_len,
// next_tokens, stream: (path, path_len, next_tokens).
PyObject* draft_path(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want_args("msa_draft_path", n, 9);
  const Tensor& sampled = dense("sampled", a[0], nullptr, at::kInt, {-1});
  const at::Device dev = sampled.device();
  const Tensor& drafts = dense("drafts", a[1], &dev, at::kInt, sampled.sizes());
  const Tensor& mask = tensor("tree_mask", a[2]);
  if (mask.scalar_type() != at::kInt && mask.scalar_type() != at::kUInt32) wrong_dtype("tree_mask", mask, "int32 or uint32");
  dense("tree_mask", a[2], &dev, mask.scalar_type(), {sampled.size(0), -1});
  const Tensor& cu = dense("cu_seqlens_q", a[3], &dev, at::kInt, {-1});
  const int64_t batch = cu.size(0) > 0 ? cu.size(0) - 1 : 0;
  const int words = size32("tree_mask", mask.size(1));
  const int most = a[4] == Py_None ? size32("tree_mask", 32 * (int64_t)words) : as_int(a[4]);
  if (most < 1) bad_value("max_path must be at least 1");
  const Place place(dev, a[8]);
  const Tensor path = output("path", a[5], dev, at::kInt, Shape{batch, most});
  const Tensor len = output("path_len", a[6], dev, at::kInt, Shape{batch});
  const Tensor next = output("next_tokens", a[7], dev, at::kInt, Shape{batch});
  check("msa_draft_path",
        msa_draft_path(ptr<const int32_t>(sampled), ptr<const int32_t>(drafts), ptr<const uint32_t>(mask), words,
                       ptr<const int32_t>(cu), size32("cu_seqlens_q", batch), size32("sampled", sampled.size(0)), most,
                       ptr<int32_t>(path), ptr<int32_t>(len), ptr<int32_t>(next), place.stream()));
  return tuple_of({path, len, next});
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_XDECREF(g_error);
  g_error = Py_NewRef(cls);
  Py_RETURN_NONE;
}

#define MSA_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {MSA_METHOD(qk_norm_rope),
                         MSA_METHOD(qk_norm_rope_append),
                         MSA_METHOD(qk_norm_rope_bwd),
                         MSA_METHOD(tree_attention),
                         MSA_METHOD(prefix_attention),
                         MSA_METHOD(cache_extend),
                         MSA_METHOD(cache_fork),
                         MSA_METHOD(cache_free),
                         MSA_METHOD(cache_copy_pages),
                         MSA_METHOD(cache_accept),
                         MSA_METHOD(step_tables),
                         MSA_METHOD(sample),
                         MSA_METHOD(draft_path),
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module_def); }
