// Python module `_ops`: checks and marshals torch tensors for the multi-token operators of
// include/mk.h (ops.py has the documented functions).  A call at batch 1 runs for a few
// microseconds on the GPU; looking at eight tensors from Python takes longer than that.
//
// Every function takes its arguments by position (None where optional), raises ValueError
// for a tensor that does not fit and binding.MkError for a call that the library refuses, and
// runs on the current stream of the tensors' device, which the caller has made current.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/core/GradMode.h>
#include <cuda_runtime_api.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <limits>
#include <string>
#include <vector>

#include "mk.h"

namespace {

PyObject* g_check = nullptr;  // binding._check(rc)

struct Error {};  // a Python exception is set

[[noreturn]] void refuse(const std::string& text) {
  PyErr_SetString(PyExc_ValueError, text.c_str());
  throw Error{};
}

std::string show(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor, not " + Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

const at::Tensor& shaped(PyObject* o, const char* name, int64_t dims) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != dims) refuse(std::string(name) + " has " + std::to_string(t.dim()) + " dimensions, needs " + std::to_string(dims));
  return t;
}

void check(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, int dev) {
  if (t.requires_grad() && c10::GradMode::is_enabled())
    refuse(std::string(name) + " requires a gradient, and this operator has no backward pass");
  if (t._fw_grad(0).defined())  // (forward-mode derivatives have one level, 0)
    refuse(std::string(name) + " carries a forward-mode tangent, and this operator has no derivative");
  if (!t.is_cuda() || t.get_device() != dev)
    refuse(std::string(name) + " must be a CUDA tensor on device " + std::to_string(dev) + ", not on " + t.device().str());
  if (t.scalar_type() != type) refuse(std::string(name) + " must be " + toString(type) + ", not " + toString(t.scalar_type()));
  if (t.sizes() != shape) refuse(std::string(name) + " has shape " + show(t.sizes()) + ", needs " + show(shape));
}

// address of a contiguous operand
template <class T = void>
T* need(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, int dev) {
  check(t, name, type, shape, dev);
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
  return static_cast<T*>(t.data_ptr());
}
template <class T = void>
T* need(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, int dev) {
  return need<T>(tensor(o, name), name, type, shape, dev);
}
template <class T = void>
T* optional(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, int dev) {
  return o == Py_None ? nullptr : need<T>(o, name, type, shape, dev);
}

// address of an operand whose last dimension is contiguous; strides of the others
void* rows(const at::Tensor& t, const char* name, at::IntArrayRef shape, int dev, int64_t* stride, at::ScalarType type = at::kBFloat16) {
  check(t, name, type, shape, dev);
  const int64_t last = t.dim() - 1;
  if (t.stride(last) != 1 && shape[last] != 1) refuse(std::string(name) + ": the last dimension must be contiguous");
  for (int64_t i = 0; i < last; ++i) stride[i] = t.stride(i);
  return t.data_ptr();
}

double number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + " must be a number");
  }
  return v;
}
int32_t whole(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + " must be an integer");
  }
  if (v < std::numeric_limits<int32_t>::min() || v > std::numeric_limits<int32_t>::max())
    refuse(std::string(name) + " does not fit 32 bits");
  return (int32_t)v;
}
// sizes of tensors that go into 32-bit fields
int32_t size32(int64_t v, const char* name) {
  if (v > std::numeric_limits<int32_t>::max()) refuse(std::string(name) + " does not fit 32 bits");
  return (int32_t)v;
}

void* stream(int dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }

PyObject* finish(int rc, PyObject* result) {  // takes `result`
  if (rc == MK_OK) return result;
  Py_XDECREF(result);
  PyObject* r = PyObject_CallFunction(g_check, "i", rc);
  Py_XDECREF(r);
  return nullptr;
}

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }

at::Tensor fresh(at::IntArrayRef shape, const at::Tensor& like, at::ScalarType type, bool zero) {
  const auto o = like.options().dtype(type).requires_grad(false);
  return zero ? at::zeros(shape, o) : at::empty(shape, o);
}

// The cache arguments from a[0] on: k_cache, v_cache (`dims` dimensions), page_table, seq_lens.
mk_paged_kv cache(PyObject* const* a, int64_t dims, int dev) {
  mk_paged_kv c{};
  const at::Tensor& k = shaped(a[0], "k_cache", dims);
  const at::Tensor& t = shaped(a[2], "page_table", 2);
  const auto s = k.sizes();
  if (s[dims - 2] != 16) refuse("k_cache has pages of " + std::to_string(s[dims - 2]) + " tokens, needs 16");
  c.k = need(k, "k_cache", at::kBFloat16, s, dev);
  c.v = need(a[1], "v_cache", at::kBFloat16, s, dev);
  c.page_table = need<int32_t>(t, "page_table", at::kInt, t.sizes(), dev);
  c.seq_lens = need<int32_t>(a[3], "seq_lens", at::kInt, {t.size(0)}, dev);
  c.n_pages = size32(s[dims - 4], "the number of pages");
  c.n_kv_heads = size32(s[dims - 3], "the number of heads");
  c.head_dim = size32(s[dims - 1], "head_dim");
  c.batch = size32(t.size(0), "the batch");
  c.max_pages = size32(t.size(1), "the page table");
  return c;
}

// q, k, v, k_cache, v_cache, page_table, seq_lens, theta, q_gain, k_gain, eps, positions, counts, out, status
PyObject* qk_norm_rope(PyObject* const* a) {
  const at::Tensor& q = shaped(a[0], "q", 4);
  const int dev = (int)q.get_device();
  const mk_paged_kv c = cache(a + 3, 4, dev);
  const int64_t b = c.batch, n = q.size(1), hq = q.size(2), hd = c.head_dim;
  const int64_t qs[4] = {b, n, hq, hd}, ks[4] = {b, n, c.n_kv_heads, hd};
  mk_rope_args r{};
  r.q = rows(q, "q", qs, dev, r.q_stride);
  r.k = rows(tensor(a[1], "k"), "k", ks, dev, r.k_stride);
  r.v = rows(tensor(a[2], "v"), "v", ks, dev, r.v_stride);
  r.q_gain = optional(a[8], "q_gain", at::kBFloat16, {hd}, dev);
  r.k_gain = optional(a[9], "k_gain", at::kBFloat16, {hd}, dev);
  r.positions = optional<int32_t>(a[11], "positions", at::kInt, {b, n}, dev);
  r.counts = optional<int32_t>(a[12], "counts", at::kInt, {b}, dev);
  r.status = optional<int32_t>(a[14], "status", at::kInt, {4}, dev);
  r.theta = number(a[7], "theta");
  r.eps = (float)number(a[10], "eps");
  // (nodes that the kernel leaves alone would be uninitialised memory)
  const at::Tensor out = a[13] == Py_None ? fresh(qs, q, at::kBFloat16, r.counts != nullptr) : tensor(a[13], "out");
  r.q_out = rows(out, "out", qs, dev, r.out_stride);
  r.n_nodes = size32(n, "the number of nodes");
  r.n_q_heads = size32(hq, "the number of heads");
  return finish(n == 0 || b == 0 ? (int)MK_OK : mk_qk_norm_rope(&c, &r, stream(dev)), wrap(out));
}

// q, k_cache, v_cache, page_table, seq_lens, mask, positions, counts, window, scale, out, status
PyObject* tree_attention(PyObject* const* a) {
  const at::Tensor& q = shaped(a[0], "q", 4);
  const int dev = (int)q.get_device();
  const mk_paged_kv c = cache(a + 1, 4, dev);
  const int64_t b = c.batch, n = q.size(1), hq = q.size(2), hd = c.head_dim;
  const int64_t qs[4] = {b, n, hq, hd};
  mk_tree_args r{};
  r.q = rows(q, "q", qs, dev, r.q_stride);
  r.mask = optional<int32_t>(a[5], "mask", at::kInt, {b, n, (n + 31) / 32}, dev);
  r.positions = optional<int32_t>(a[6], "positions", at::kInt, {b, n}, dev);
  r.counts = optional<int32_t>(a[7], "counts", at::kInt, {b}, dev);
  r.status = optional<int32_t>(a[11], "status", at::kInt, {4}, dev);
  r.window = whole(a[8], "window");
  r.scale = a[9] == Py_None ? (float)(1.0 / std::sqrt((double)hd)) : (float)number(a[9], "scale");
  const at::Tensor out = a[10] == Py_None ? fresh(qs, q, at::kBFloat16, r.counts != nullptr) : tensor(a[10], "out");
  r.out = rows(out, "out", qs, dev, r.out_stride);
  r.n_nodes = size32(n, "the number of nodes");
  r.n_q_heads = size32(hq, "the number of heads");
  if (n == 0 || b == 0) return wrap(out);
  int rc = mk_tree_attention_workspace(&c, &r, &r.workspace_bytes);
  if (rc != MK_OK) return finish(rc, nullptr);
  const at::Tensor work = fresh({(int64_t)r.workspace_bytes}, q, at::kByte, false);
  r.workspace = work.data_ptr();
  return finish(mk_tree_attention(&c, &r, stream(dev)), wrap(out));
}

// a list of page numbers: a list or tuple of ints, or what ops._page_ids has made one of
std::vector<int32_t> pages(PyObject* o, const char* name) {
  PyObject* s = PySequence_Fast(o, "a list of page numbers");
  if (!s) throw Error{};
  std::vector<int32_t> v((size_t)PySequence_Fast_GET_SIZE(s));
  for (size_t i = 0; i < v.size(); ++i) {
    PyObject* x = PySequence_Fast_GET_ITEM(s, (Py_ssize_t)i);
    int overflow = 0;
    const long long p = PyLong_Check(x) ? PyLong_AsLongLongAndOverflow(x, &overflow) : -1;
    if (!PyLong_Check(x) || overflow || p < std::numeric_limits<int32_t>::min() || p > std::numeric_limits<int32_t>::max()) {
      Py_DECREF(s);
      refuse(std::string(name) + " must be a list of page numbers of 32 bits");
    }
    v[i] = (int32_t)p;
  }
  Py_DECREF(s);
  return v;
}

// k_cache, v_cache, src, dst
PyObject* copy_pages(PyObject* const* a) {
  const at::Tensor& k = shaped(a[0], "k_cache", 5);
  const int dev = (int)k.get_device();
  const auto s = k.sizes();
  if (s[3] != 16) refuse("k_cache has pages of " + std::to_string(s[3]) + " tokens, needs 16");
  void* kp = need(k, "k_cache", at::kBFloat16, s, dev);
  void* vp = need(a[1], "v_cache", at::kBFloat16, s, dev);
  const std::vector<int32_t> src = pages(a[2], "src"), dst = pages(a[3], "dst");
  if (src.size() != dst.size())
    refuse(std::to_string(src.size()) + " source pages, " + std::to_string(dst.size()) + " destination pages");
  Py_INCREF(Py_None);
  return finish(mk_copy_pages(kp, vp, size32(s[0], "the number of layers"), size32(s[1], "the number of pages"),
                              size32(s[2], "the number of heads"), size32(s[4], "head_dim"), src.data(), dst.data(),
                              size32((int64_t)src.size(), "the number of copies"), stream(dev)),
                Py_None);
}

// k_cache, v_cache, page_table, seq_lens, accepted, out, status
PyObject* commit_nodes(PyObject* const* a) {
  const at::Tensor& k = shaped(a[0], "k_cache", 5);
  const int dev = (int)k.get_device();
  const mk_paged_kv c = cache(a, 5, dev);
  const at::Tensor& acc = shaped(a[4], "accepted", 2);
  const int32_t* accepted = need<int32_t>(acc, "accepted", at::kInt, {c.batch, acc.size(1)}, dev);
  const at::Tensor out = a[5] == Py_None ? fresh({c.batch}, k, at::kInt, false) : tensor(a[5], "out");
  int32_t* lens = need<int32_t>(out, "out", at::kInt, {c.batch}, dev);
  int32_t* status = optional<int32_t>(a[6], "status", at::kInt, {4}, dev);
  if (c.batch == 0) return wrap(out);
  return finish(mk_commit_nodes(&c, size32(k.size(0), "the number of layers"), accepted, size32(acc.size(1), "max_accept"), lens,
                                status, stream(dev)),
                wrap(out));
}

// x, w, offsets, w_up, rows, out, status
PyObject* expert_product(PyObject* const* a) {
  const at::Tensor& x = shaped(a[0], "x", 2);
  const int dev = (int)x.get_device();
  const at::Tensor& w = shaped(a[1], "w", 3);
  const int64_t e = w.size(0), n = w.size(1), k = w.size(2), n_x = x.size(0);
  mk_expert_args r{};
  int64_t stride[1];
  r.x = rows(x, "x", {n_x, k}, dev, stride);
  r.x_stride = n_x > 1 ? stride[0] : k;
  r.w = need(w, "w", at::kBFloat16, {e, n, k}, dev);
  r.w_up = optional(a[3], "w_up", at::kBFloat16, {e, n, k}, dev);
  r.offsets = need<int32_t>(a[2], "offsets", at::kInt, {e + 1}, dev);
  int64_t n_rows = n_x;
  if (a[4] != Py_None) {
    const at::Tensor& named = shaped(a[4], "rows", 1);
    n_rows = named.size(0);
    r.rows = need<int32_t>(named, "rows", at::kInt, {n_rows}, dev);
  }
  const at::Tensor out = a[5] == Py_None ? fresh({n_rows, n}, x, at::kBFloat16, false) : tensor(a[5], "out");
  r.out = rows(out, "out", {n_rows, n}, dev, stride);
  r.out_stride = n_rows > 1 ? stride[0] : n;
  r.status = optional<int32_t>(a[6], "status", at::kInt, {4}, dev);
  r.n_x = size32(n_x, "the number of rows of x");
  r.n_rows = size32(n_rows, "the number of rows");
  r.n_experts = size32(e, "the number of experts");
  r.n = size32(n, "n");
  r.k = size32(k, "k");
  return finish(n_rows == 0 ? (int)MK_OK : mk_expert_product(&r, stream(dev)), wrap(out));
}

// bf16 or float32
bool is_float(const at::Tensor& t, const char* name) {
  if (t.scalar_type() != at::kFloat && t.scalar_type() != at::kBFloat16)
    refuse(std::string(name) + " must be BFloat16 or Float, not " + toString(t.scalar_type()));
  return t.scalar_type() == at::kFloat;
}
// stride of the rows of a matrix (one row has none)
int64_t row_stride(const int64_t* stride, int64_t rows, int64_t width) { return rows > 1 ? stride[0] : width; }

// x, w, bias, activation, residual, out, wide (None: out's type, or bf16), status
PyObject* linear(PyObject* const* a) {
  const at::Tensor& x = shaped(a[0], "x", 2);
  const int dev = (int)x.get_device();
  const at::Tensor& w = shaped(a[1], "w", 2);
  const int64_t m = x.size(0), k = x.size(1), n = w.size(0);
  mk_linear_args r{};
  int64_t stride[1];
  r.x = rows(x, "x", {m, k}, dev, stride);
  r.x_stride = row_stride(stride, m, k);
  r.w = need(w, "w", at::kBFloat16, {n, k}, dev);
  r.bias = optional(a[2], "bias", at::kBFloat16, {n}, dev);
  r.activation = whole(a[3], "activation");
  if (a[4] != Py_None) {
    r.residual = rows(tensor(a[4], "residual"), "residual", {m, n}, dev, stride);
    r.residual_stride = row_stride(stride, m, n);
  }
  at::Tensor out;
  if (a[5] == Py_None) {
    r.out_float = a[6] == Py_True;
    out = fresh({m, n}, x, r.out_float ? at::kFloat : at::kBFloat16, false);
  } else {
    out = shaped(a[5], "out", 2);
    r.out_float = is_float(out, "out");
    if (a[6] != Py_None && (a[6] == Py_True) != (r.out_float != 0)) refuse("out has another dtype than the one asked for");
  }
  r.out = rows(out, "out", {m, n}, dev, stride, r.out_float ? at::kFloat : at::kBFloat16);
  r.out_stride = row_stride(stride, m, n);
  r.status = optional<int32_t>(a[7], "status", at::kInt, {4}, dev);
  r.m = size32(m, "m");
  r.n = size32(n, "n");
  r.k = size32(k, "k");
  return finish(mk_linear(&r, stream(dev)), wrap(out));
}

// x, router, w_gate, w_up, w_down, top_k, residual, ids, weights, out, status
PyObject* moe_layer(PyObject* const* a) {
  const at::Tensor& x = shaped(a[0], "x", 2);
  const int dev = (int)x.get_device();
  const at::Tensor& gate = shaped(a[2], "w_gate", 3);
  const int64_t t = x.size(0), e = gate.size(0), f = gate.size(1), d = gate.size(2);
  mk_moe_args r{};
  int64_t stride[1];
  r.x = rows(x, "x", {t, d}, dev, stride);
  r.x_stride = row_stride(stride, t, d);
  r.router = need(a[1], "router", at::kBFloat16, {e, d}, dev);
  r.w_gate = need(gate, "w_gate", at::kBFloat16, {e, f, d}, dev);
  r.w_up = need(a[3], "w_up", at::kBFloat16, {e, f, d}, dev);
  r.w_down = need(a[4], "w_down", at::kBFloat16, {e, d, f}, dev);
  r.top_k = whole(a[5], "top_k");
  if (a[6] != Py_None) {
    r.residual = rows(tensor(a[6], "residual"), "residual", {t, d}, dev, stride);
    r.residual_stride = row_stride(stride, t, d);
  }
  r.ids = optional<int32_t>(a[7], "ids", at::kInt, {t, r.top_k}, dev);
  r.weights = optional<float>(a[8], "weights", at::kFloat, {t, r.top_k}, dev);
  const at::Tensor out = a[9] == Py_None ? fresh({t, d}, x, at::kBFloat16, false) : tensor(a[9], "out");
  r.out = rows(out, "out", {t, d}, dev, stride);
  r.out_stride = row_stride(stride, t, d);
  r.status = optional<int32_t>(a[10], "status", at::kInt, {4}, dev);
  r.n_tokens = size32(t, "the number of tokens");
  r.d_model = size32(d, "d_model");
  r.d_ff = size32(f, "d_ff");
  r.n_experts = size32(e, "the number of experts");
  const int rc = mk_moe_layer_workspace(&r, &r.workspace_bytes);
  if (rc != MK_OK) return finish(rc, nullptr);
  if (t == 0) return wrap(out);
  const at::Tensor work = fresh({(int64_t)r.workspace_bytes}, x, at::kByte, false);
  r.workspace = work.data_ptr();
  return finish(mk_moe_layer(&r, stream(dev)), wrap(out));
}

// logits, tokens, uniforms, parents, draft_probs, temperature, counts, accepted, next_tokens, status
PyObject* verify_nodes(PyObject* const* a) {
  const at::Tensor& logits = shaped(a[0], "logits", 3);
  const int dev = (int)logits.get_device();
  const int64_t b = logits.size(0), n = logits.size(1), v = logits.size(2);
  mk_verify_args r{};
  r.logits_float = is_float(logits, "logits");
  r.logits = rows(logits, "logits", {b, n, v}, dev, r.logits_stride, r.logits_float ? at::kFloat : at::kBFloat16);
  r.tokens = need<int32_t>(a[1], "tokens", at::kInt, {b, n}, dev);
  r.uniforms = need<float>(a[2], "uniforms", at::kFloat, {b, n}, dev);
  r.parents = optional<int32_t>(a[3], "parents", at::kInt, {b, n}, dev);
  if (a[4] != Py_None)
    r.draft_probs = static_cast<const float*>(rows(tensor(a[4], "draft_probs"), "draft_probs", {b, n, v}, dev, r.draft_stride, at::kFloat));
  r.temperature = optional<float>(a[5], "temperature", at::kFloat, {b}, dev);
  r.counts = optional<int32_t>(a[6], "counts", at::kInt, {b}, dev);
  const at::Tensor accepted = a[7] == Py_None ? fresh({b, n}, logits, at::kInt, false) : tensor(a[7], "accepted");
  const at::Tensor next = a[8] == Py_None ? fresh({b}, logits, at::kInt, false) : tensor(a[8], "next_tokens");
  r.accepted = need<int32_t>(accepted, "accepted", at::kInt, {b, n}, dev);
  r.next_tokens = need<int32_t>(next, "next_tokens", at::kInt, {b}, dev);
  r.status = optional<int32_t>(a[9], "status", at::kInt, {4}, dev);
  r.batch = size32(b, "the batch");
  r.n_nodes = size32(n, "the number of nodes");
  r.vocab = size32(v, "the vocabulary");
  int rc = mk_verify_nodes_workspace(&r, &r.workspace_bytes);
  if (rc == MK_OK && b > 0) {
    const at::Tensor work = fresh({(int64_t)r.workspace_bytes}, logits, at::kByte, false);
    r.workspace = work.data_ptr();
    rc = mk_verify_nodes(&r, stream(dev));
  }
  if (rc != MK_OK) return finish(rc, nullptr);
  PyObject *first = wrap(accepted), *second = wrap(next), *both = first && second ? PyTuple_Pack(2, first, second) : nullptr;
  Py_XDECREF(first);
  Py_XDECREF(second);
  return both;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, %zd given", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Error&) {
    return nullptr;
  } catch (const std::exception& e) {  // an allocation that failed, for one
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// Whether the tensor is on the current device (None: no CUDA tensor).
PyObject* is_here(PyObject*, PyObject* o) {
  if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda()) Py_RETURN_NONE;
  int dev = -1;
  return PyBool_FromLong(cudaGetDevice(&dev) == cudaSuccess && dev == THPVariable_Unpack(o).get_device());
}

PyObject* setup(PyObject*, PyObject* check) {
  Py_INCREF(check);
  Py_XSETREF(g_check, check);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&call<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<qk_norm_rope, 15>("qk_norm_rope"), method<tree_attention, 12>("tree_attention"),
                         method<copy_pages, 4>("copy_pages"),      method<commit_nodes, 7>("commit_nodes"),
                         method<expert_product, 7>("expert_product"), method<linear, 8>("linear"),
                         method<moe_layer, 11>("moe_layer"),       method<verify_nodes, 10>("verify_nodes"), {"is_here", is_here, METH_O, nullptr},
                         {"setup", setup, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops() { return PyModule_Create(&module); }
