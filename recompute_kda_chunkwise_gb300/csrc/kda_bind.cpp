// kda_bind.cpp -- the host side of the Python binding of the operators around
// the delta rule (decode.py, norm.py, rotary.py, attention.py, grads.py): checks
// of the tensors, outputs, and the call of the C entry point (kda_serving.h,
// kda_blocks.h) on the current stream.
//
// These calls take a few microseconds on the GPU. Checking a dozen tensors,
// allocating the outputs and marshalling the arguments in Python took 15 to 27
// on the host; here they take 5 to 7 (with the launch), and the norm's backward,
// with up to six allocations and two launches, 10 to 14. The entry points' addresses come from
// the ctypes loader (init), so this module links to no kernel library of its
// own. Every function either returns its outputs, or the entry point's
// kda_status as an int, or raises ValueError for a tensor that does not fit.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <array>
#include <cmath>
#include <initializer_list>
#include <stdexcept>
#include <string>
#include <vector>

#include "kda_blocks.h"
#include "kda_span.h"

namespace {

using at::Tensor;

struct Entry {
  decltype(&kda_step) step;
  decltype(&kda_gdn2_step) gdn2_step;
  decltype(&kda_block_norm_fwd) norm_fwd;
  decltype(&kda_block_norm_workspace_bytes) norm_bytes;
  decltype(&kda_block_norm_bwd) norm_bwd;
  decltype(&kda_verify_drafts) verify;
  decltype(&kda_paged_append) append;
  decltype(&kda_paged_attention_workspace_bytes) attention_bytes;
  decltype(&kda_paged_attention) attention;
  decltype(&kda_rotary) rotary;
  decltype(&kda_paged_append_rotary) append_rotary;
  decltype(&kda_attention_fwd_workspace_bytes) packed_fwd_bytes;
  decltype(&kda_attention_fwd_fresh) packed_fwd;
  decltype(&kda_attention_bwd_workspace_bytes) packed_bwd_bytes;
  decltype(&kda_attention_bwd_fresh) packed_bwd;
  decltype(&kda_grad_norm_workspace_bytes) norm_of_grads_bytes;
  decltype(&kda_grad_norm) norm_of_grads;
  decltype(&kda_clip_grads) clip;
} g_entry;

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

const char* name_of(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kByte: return "torch.uint8";
    default: return "another dtype";
  }
}

std::string text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

// Argument i as a tensor; None gives an undefined one.
struct Args {
  PyObject* const* v;
  Tensor at(int i, const char* name) const {
    if (!THPVariable_Check(v[i])) throw Refused(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(v[i]);
  }
  Tensor maybe(int i, const char* name) const { return v[i] == Py_None ? Tensor() : at(i, name); }
  double number(int i) const {
    const double x = PyFloat_AsDouble(v[i]);
    if (x == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      throw Refused("a scale or epsilon is not a number");
    }
    return x;
  }
};

// Address of a tensor that the kernels index by `shape`; null for one left out.
void* fit(const Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType dtype, c10::DeviceIndex dev) {
  if (!t.defined()) return nullptr;
  if (t.scalar_type() != dtype || !t.is_cuda() || t.get_device() != dev || t.sizes() != shape || !t.is_contiguous())
    throw Refused(std::string(name) + " must be a contiguous " + name_of(dtype) + " CUDA tensor of shape " + text(shape) +
                  " on the first tensor's device (got " + name_of(t.scalar_type()) + " " + text(t.sizes()) +
                  (t.is_cuda() ? "" : " on the CPU") + (t.is_contiguous() ? ")" : ", strided)"));
  return t.data_ptr();
}
// A size as the entry points take it: one past 32 bits is refused, not cut.
int32_t size32(int64_t n, const char* name) {
  if (n > INT32_MAX) throw Refused(std::string(name) + " " + std::to_string(n) + " is past 32 bits");
  return static_cast<int32_t>(n);
}
void on_cuda(const Tensor& t, const char* name) {
  if (!t.is_cuda()) throw Refused(std::string(name) + " must be a contiguous CUDA tensor");
}
int32_t activation(const Tensor& t, const char* what) {
  if (t.scalar_type() == at::kBFloat16) return KDA_DTYPE_BF16;
  if (t.scalar_type() == at::kFloat) return KDA_DTYPE_F32;
  throw Refused(std::string(what) + " in bfloat16 or float32 (got " + name_of(t.scalar_type()) + " " + text(t.sizes()) + ")");
}
Tensor like(const Tensor& t) { return at::empty(t.sizes(), t.options().requires_grad(false)); }
void* buffer(Tensor& t, size_t bytes, const Tensor& ref) {
  if (!t.defined()) {
    if (bytes == 0) return nullptr;
    t = at::empty({static_cast<int64_t>(bytes)}, ref.options().dtype(at::kByte).requires_grad(false));
  } else if (!t.is_cuda() || t.get_device() != ref.get_device() || !t.is_contiguous() || t.nbytes() < bytes) {
    throw Refused("workspace must be a contiguous CUDA buffer of at least " + std::to_string(bytes) + " bytes");
  }
  return t.data_ptr();
}
void* stream_of(const Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.get_device()).stream(); }
PyObject* wrap(const Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}
int32_t* word(const Tensor& t, c10::DeviceIndex dev) {
  return static_cast<int32_t*>(fit(t, "status", {1}, at::kInt, dev));
}

// A caller's tensor was written behind autograd's back: a graph that saved it has to notice.
void written(const Tensor& t) {
  if (t.defined() && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, const F& f) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", n, want);
    return nullptr;
  }
  try {
    return f();
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {  // allocation
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// q k v g gate0 gate1|None A_log dt_bias cu states index|None commit|None scale lower eps out|None status|None
PyObject* step(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
  return guarded(nargs, 17, [&]() -> PyObject* {
    const Args a{v};
    const Tensor q = a.at(0, "q"), cu = a.at(8, "cu_seqlens"), states = a.at(9, "states");
    if (q.dim() != 3) throw Refused("q must be [S, H, D] (got " + text(q.sizes()) + ")");
    const int32_t code = activation(q, "q must be [S, H, D]");
    if (states.dim() != 4) throw Refused("states must be [slots, H, D, D]");
    const int64_t S = q.size(0), H = q.size(1), D = q.size(2), N = cu.numel() - 1, slots = states.size(0);
    const int32_t num_seqs = size32(N, "the number of sequences of cu_seqlens,"), heads = size32(H, "the number of heads"),
                  head_dim = size32(D, "head_dim");
    on_cuda(q, "q");
    const auto dev = q.get_device();
    const auto dt = q.scalar_type();
    const auto all = q.sizes();
    const bool gdn2 = v[5] != Py_None;
    Tensor out = a.maybe(15, "out");
    kda_problem p{};
    p.total_tokens = S;
    p.num_seqs = num_seqs;
    p.num_heads = heads;
    p.head_dim = head_dim;
    p.dtype = code;
    p.scale = static_cast<float>(a.number(12));
    p.gate_lower_bound = static_cast<float>(a.number(13));
    p.l2_eps = static_cast<float>(a.number(14));
    p.flags = gdn2 ? KDA_FLAG_CHANNEL_GATES : 0;
    p.cu_seqlens = static_cast<const int32_t*>(fit(cu, "cu_seqlens", {N + 1}, at::kInt, dev));
    void* const qp = fit(q, "q", all, dt, dev);
    void* const kp = fit(a.at(1, "k"), "k", all, dt, dev);
    void* const vp = fit(a.at(2, "v"), "v", all, dt, dev);
    void* const gp = fit(a.at(3, "g"), "g", all, dt, dev);
    void* const g0 = gdn2 ? fit(a.at(4, "erase"), "erase", all, dt, dev)
                          : fit(a.at(4, "beta"), "beta", {S, H}, dt, dev);
    void* const g1 = gdn2 ? fit(a.at(5, "write"), "write", all, dt, dev) : nullptr;
    const float* const A = static_cast<float*>(fit(a.at(6, "A_log"), "A_log", {H}, at::kFloat, dev));
    const float* const b = static_cast<float*>(fit(a.at(7, "dt_bias"), "dt_bias", {H, D}, at::kFloat, dev));
    float* const st = static_cast<float*>(fit(states, "states", {slots, H, D, D}, at::kFloat, dev));
    const int32_t* const index = static_cast<int32_t*>(fit(a.maybe(10, "state_index"), "state_index", {N}, at::kInt, dev));
    const int32_t* const commit = static_cast<int32_t*>(fit(a.maybe(11, "commit"), "commit", {N}, at::kInt, dev));
    int32_t* const status = word(a.maybe(16, "status"), dev);
    const c10::cuda::CUDAGuard on(dev);
    if (!out.defined()) out = like(q);
    void* const op = fit(out, "out", all, dt, dev);
    const kda_status r = gdn2 ? g_entry.gdn2_step(&p, qp, kp, vp, gp, g0, g1, A, b, st, slots, index, commit, op, status,
                                                  stream_of(q))
                              : g_entry.step(&p, qp, kp, vp, gp, g0, A, b, st, slots, index, commit, op, status,
                                             stream_of(q));
    return r == KDA_OK ? wrap(out) : PyLong_FromLong(r);
  });
}

kda_norm_problem norm_problem(const Tensor& y, double a, double b, double eps) {
  if (y.dim() < 1) throw Refused("y must be [..., width]");
  kda_norm_problem p{};
  p.dtype = activation(y, "y must be [..., width]");
  p.width = size32(y.size(-1), "width");
  on_cuda(y, "y");
  p.rows = p.width ? y.numel() / p.width : 0;
  p.residual_scale = static_cast<float>(a);
  p.block_scale = static_cast<float>(b);
  p.eps = static_cast<float>(eps);
  return p;
}

// y z|None h|None w_post|None w_pre|None residual_scale block_scale eps h_out|None n|None
PyObject* norm_fwd(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
  return guarded(nargs, 10, [&]() -> PyObject* {
    const Args a{v};
    const Tensor y = a.at(0, "y"), w_pre = a.maybe(4, "w_pre");
    const kda_norm_problem p = norm_problem(y, a.number(5), a.number(6), a.number(7));
    const auto dev = y.get_device();
    const auto dt = y.scalar_type();
    const auto all = y.sizes();
    const std::array<int64_t, 1> wide{y.size(-1)};
    void* const yp = fit(y, "y", all, dt, dev);
    void* const zp = fit(a.maybe(1, "z"), "z", all, dt, dev);
    void* const hp = fit(a.maybe(2, "h"), "h", all, dt, dev);
    const float* const wp = static_cast<float*>(fit(a.maybe(3, "w_post"), "w_post", wide, at::kFloat, dev));
    const float* const wn = static_cast<float*>(fit(w_pre, "w_pre", wide, at::kFloat, dev));
    const c10::cuda::CUDAGuard on(dev);
    Tensor ho = a.maybe(8, "h_out"), n = a.maybe(9, "n");
    if (!ho.defined()) ho = like(y);
    if (!n.defined() && w_pre.defined()) n = like(y);
    const kda_status r = g_entry.norm_fwd(&p, yp, zp, hp, wp, wn, fit(ho, "h_out", all, dt, dev), fit(n, "n", all, dt, dev),
                                          stream_of(y));
    return r == KDA_OK ? Py_BuildValue("(NN)", wrap(ho), wrap(n)) : PyLong_FromLong(r);
  });
}

// y z|None h|None w_post|None w_pre|None dh_out|None dn|None residual_scale block_scale eps workspace|None
PyObject* norm_bwd(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
  return guarded(nargs, 11, [&]() -> PyObject* {
    const Args a{v};
    const Tensor y = a.at(0, "y"), z = a.maybe(1, "z"), h = a.maybe(2, "h"), w_post = a.maybe(3, "w_post"),
                 w_pre = a.maybe(4, "w_pre");
    const kda_norm_problem p = norm_problem(y, a.number(7), a.number(8), a.number(9));
    const auto dev = y.get_device();
    const auto dt = y.scalar_type();
    const auto all = y.sizes();
    const std::array<int64_t, 1> wide{y.size(-1)};
    void* const yp = fit(y, "y", all, dt, dev);
    void* const zp = fit(z, "z", all, dt, dev);
    void* const hp = fit(h, "h", all, dt, dev);
    const float* const wp = static_cast<float*>(fit(w_post, "w_post", wide, at::kFloat, dev));
    const float* const wn = static_cast<float*>(fit(w_pre, "w_pre", wide, at::kFloat, dev));
    void* const gh = fit(a.maybe(5, "dh_out"), "dh_out", all, dt, dev);
    void* const gn = fit(a.maybe(6, "dn"), "dn", all, dt, dev);
    const c10::cuda::CUDAGuard on(dev);
    Tensor ws = a.maybe(10, "workspace");
    void* const wsp = buffer(ws, g_entry.norm_bytes(&p, w_post.defined(), w_pre.defined()), y);
    const Tensor dy = like(y), dz = z.defined() ? like(y) : Tensor(), dh = h.defined() ? like(y) : Tensor(),
                 dwp = w_post.defined() ? like(w_post) : Tensor(), dwn = w_pre.defined() ? like(w_pre) : Tensor();
    auto ptr = [](const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
    const kda_status r = g_entry.norm_bwd(&p, yp, zp, hp, wp, wn, gh, gn, ptr(dy), ptr(dz), ptr(dh),
                                          static_cast<float*>(ptr(dwp)), static_cast<float*>(ptr(dwn)), wsp, stream_of(y));
    return r == KDA_OK ? Py_BuildValue("(NNNNN)", wrap(dy), wrap(dz), wrap(dh), wrap(dwp), wrap(dwn)) : PyLong_FromLong(r);
  });
}

// target draft|None draft_tokens num_drafts|None u noise status|None
PyObject* verify(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
  return guarded(nargs, 7, [&]() -> PyObject* {
    const Args a{v};
    const Tensor target = a.at(0, "target");
    if (target.dim() != 3 || target.size(1) < 1) throw Refused("target must be [N, T + 1, V]");
    const int64_t N = target.size(0), T = target.size(1) - 1, V = target.size(2);
    const int32_t seqs = size32(N, "the number of sequences"), drafts = size32(T, "the number of drafts"),
                  vocab = size32(V, "the vocabulary");
    on_cuda(target, "target");
    const auto dev = target.get_device();
    const float* const tp = static_cast<float*>(fit(target, "target", target.sizes(), at::kFloat, dev));
    const float* const dp = static_cast<float*>(fit(a.maybe(1, "draft"), "draft", {N, T, V}, at::kFloat, dev));
    const int32_t* const xp = static_cast<int32_t*>(fit(a.at(2, "draft_tokens"), "draft_tokens", {N, T}, at::kInt, dev));
    const int32_t* const np = static_cast<int32_t*>(fit(a.maybe(3, "num_drafts"), "num_drafts", {N}, at::kInt, dev));
    const float* const up = static_cast<float*>(fit(a.at(4, "u"), "u", {N, T}, at::kFloat, dev));
    const float* const ep = static_cast<float*>(fit(a.at(5, "noise"), "noise", {N, V}, at::kFloat, dev));
    int32_t* const status = word(a.maybe(6, "status"), dev);
    const c10::cuda::CUDAGuard on(dev);
    const auto ints = target.options().dtype(at::kInt).requires_grad(false);
    const Tensor tokens = at::empty({N, T + 1}, ints), accepted = at::empty({N}, ints);
    const kda_status r = g_entry.verify(seqs, drafts, vocab, tp, dp, xp, np, up, ep, static_cast<int32_t*>(tokens.data_ptr()),
                                        static_cast<int32_t*>(accepted.data_ptr()), status, stream_of(target));
    return r == KDA_OK ? Py_BuildValue("(NN)", wrap(tokens), wrap(accepted)) : PyLong_FromLong(r);
  });
}

struct Paged {
  kda_paged_problem p;
  void *k, *v;
};
// `first`: the new tokens' tensor [S, heads, D], argument `name`; a[i]: k_pages.
Paged paged(const Args& a, int i, const Tensor& first, const char* name, int64_t Hkv, double scale) {
  const int64_t S = first.size(0), Hq = first.size(1), D = first.size(2);
  const Tensor kp = a.at(i, "k_pages"), vp = a.at(i + 1, "v_pages"), table = a.at(i + 2, "page_table"),
               lens = a.at(i + 3, "kv_lens"), cu = a.at(i + 4, "cu_seqlens");
  if (kp.dim() != 4 || table.dim() != 2)
    throw Refused("k_pages must be [pages, page_size, Hkv, D] and page_table [N, max_pages]");
  const int64_t pages = kp.size(0), size = kp.size(1), N = table.size(0), width = table.size(1);
  Paged r{};
  r.p.num_seqs = size32(N, "the number of sequences");
  r.p.num_heads = size32(Hq, "the number of heads");
  r.p.num_kv_heads = size32(Hkv, "the number of key/value heads");
  r.p.head_dim = size32(D, "head_dim");
  r.p.page_size = size32(size, "page_size");
  r.p.max_pages = size32(width, "the width of page_table,");
  on_cuda(first, name);
  const auto dev = first.get_device();
  r.k = fit(kp, "k_pages", {pages, size, Hkv, D}, at::kBFloat16, dev);
  r.v = fit(vp, "v_pages", {pages, size, Hkv, D}, at::kBFloat16, dev);
  r.p.total_tokens = S;
  r.p.num_pages = pages;
  r.p.dtype = KDA_DTYPE_BF16;
  r.p.scale = static_cast<float>(scale);
  r.p.cu_seqlens = static_cast<const int32_t*>(fit(cu, "cu_seqlens", {N + 1}, at::kInt, dev));
  r.p.page_table = static_cast<const int32_t*>(fit(table, "page_table", {N, width}, at::kInt, dev));
  r.p.kv_lens = static_cast<const int32_t*>(fit(lens, "kv_lens", {N}, at::kInt, dev));
  return r;
}

// k v k_pages v_pages page_table kv_lens cu_seqlens status|None
PyObject* append(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
  return guarded(nargs, 8, [&]() -> PyObject* {
    const Args a{v};
    const Tensor k = a.at(0, "k");
    if (k.dim() != 3) throw Refused("k must be [S, Hkv, D] (got " + text(k.sizes()) + ")");
    const Paged g = paged(a, 2, k, "k", k.size(1), 1.0);
    const auto dev = k.get_device();
    void* const kp = fit(k, "k", k.sizes(), at::kBFloat16, dev);
    void* const vp = fit(a.at(1, "v"), "v", k.sizes(), at::kBFloat16, dev);
    int32_t* const status = word(a.maybe(7, "status"), dev);
    const c10::cuda::CUDAGuard on(dev);
    const kda_status r = g_entry.append(&g.p, kp, vp, g.k, g.v, status, stream_of(k));
    if (r != KDA_OK) return PyLong_FromLong(r);
    Py_RETURN_NONE;
  });
}

// q k_pages v_pages page_table kv_lens cu_seqlens scale|None out|None workspace|None
PyObject* attention(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
  return guarded(nargs, 9, [&]() -> PyObject* {
    const Args a{v};
    const Tensor q = a.at(0, "q"), pages = a.at(1, "k_pages");
    if (q.dim() != 3 || pages.dim() != 4)
      throw Refused("q must be [S, Hq, D] and k_pages [pages, page_size, Hkv, D]");
    const double scale = v[6] == Py_None ? 1.0 / std::sqrt(static_cast<double>(q.size(2))) : a.number(6);
    const Paged g = paged(a, 1, q, "q", pages.size(2), scale);
    const auto dev = q.get_device();
    void* const qp = fit(q, "q", q.sizes(), at::kBFloat16, dev);
    const c10::cuda::CUDAGuard on(dev);
    Tensor out = a.maybe(7, "out"), ws = a.maybe(8, "workspace");
    if (!out.defined()) out = like(q);
    void* const op = fit(out, "out", q.sizes(), at::kBFloat16, dev);
    void* const wsp = buffer(ws, g_entry.attention_bytes(&g.p), q);
    const kda_status r = g_entry.attention(&g.p, qp, g.k, g.v, op, wsp, stream_of(q));
    return r == KDA_OK ? wrap(out) : PyLong_FromLong(r);
  });
}

// A tensor [S, heads, D] whose tokens lie a stride apart, heads and channels
// side by side: a slice of a fused projection fits as it is.
struct Rows {
  void* p;
  int64_t stride;
};
Rows rows_of(const Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType dtype, c10::DeviceIndex dev) {
  if (!t.defined()) return {nullptr, 0};
  const bool shaped = t.dim() == 3 && t.sizes() == shape;
  if (!shaped || t.scalar_type() != dtype || !t.is_cuda() || t.get_device() != dev ||
      (t.numel() > 0 && ((t.size(2) > 1 && t.stride(2) != 1) || (t.size(1) > 1 && t.stride(1) != t.size(2)))))
    throw Refused(std::string(name) + " must be a " + name_of(dtype) + " CUDA tensor of shape " + text(shape) +
                  ", contiguous within a token, on the first tensor's device (got " + name_of(t.scalar_type()) + " " +
                  text(t.sizes()) + (t.is_cuda() ? "" : " on the CPU") + (shaped ? ", strided " + text(t.strides()) + ")" : ")"));
  return {t.data_ptr(), t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2)};
}
// Memory of such a tensor, and of one that is contiguous.
kda::Span span(const char* name, const Tensor& t, const Rows& r) {
  if (!t.defined()) return kda::whole(name, nullptr, 0);
  const int64_t elt = t.element_size();
  const int64_t wide = t.size(1) * t.size(2);  // the entry points refuse shorter strides
  return {name, reinterpret_cast<uintptr_t>(r.p), t.size(0), wide * elt, std::max(r.stride, std::max<int64_t>(wide, 1)) * elt};
}
kda::Span span(const char* name, const Tensor& t) {
  return t.defined() ? kda::whole(name, t.data_ptr(), t.nbytes()) : kda::whole(name, nullptr, 0);
}
// What a call writes shares no memory with what else it writes, or reads: kernels
// take both in any order. Output i may lie exactly over one contiguous input, the
// one called over[i]. Outputs that the call itself makes need not be looked at.
void apart(std::initializer_list<kda::Span> outs, std::initializer_list<kda::Span> ins, std::initializer_list<const char*> over = {}) {
  auto own = over.begin();
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    const std::string input = own != over.end() ? *own++ : "";
    for (auto x = o + 1; x != outs.end(); ++x)
      if (kda::meet(*o, *x)) throw Refused(std::string(x->name) + " overlaps " + o->name);
    for (const kda::Span& x : ins)
      if (kda::meet(*o, x) && !(o->at == x.at && (x.rows == 1 || x.step == x.bytes) && input == x.name))
        throw Refused(std::string(o->name) + " overlaps " + x.name);
  }
}

// freqs interleaved magnitude
kda_rotary_problem turn(const Args& a, int i, c10::DeviceIndex dev) {
  kda_rotary_problem p{};
  const Tensor freqs = a.at(i, "frequencies");
  if (freqs.dim() != 1) throw Refused("frequencies must be [rotary_dim / 2]");
  p.rotary_dim = size32(2 * freqs.size(0), "rotary_dim");
  p.freqs = static_cast<const int64_t*>(fit(freqs, "frequencies", freqs.sizes(), at::kLong, dev));
  p.interleaved = a.number(i + 1) != 0;
  p.magnitude = static_cast<float>(a.number(i + 2));
  return p;
}

// freqs interleaved magnitude q k|None inverse positions|None cu_seqlens|None q_out|None k_out|None status|None
PyObject* rotary(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
  return guarded(nargs, 11, [&]() -> PyObject* {
    const Args a{v};
    const Tensor q = a.at(3, "q"), k = a.maybe(4, "k"), pos = a.maybe(6, "positions"), cu = a.maybe(7, "cu_seqlens");
    if (q.dim() != 3 || (k.defined() && k.dim() != 3)) throw Refused("q and k must be [S, heads, D] (q: " + text(q.sizes()) + ")");
    const int32_t code = activation(q, "q must be [S, heads, D]");
    on_cuda(q, "q");
    const auto dev = q.get_device();
    const auto dt = q.scalar_type();
    if (pos.defined() == cu.defined()) throw Refused("one of positions and cu_seqlens has to be given");
    kda_rotary_problem p = turn(a, 0, dev);
    const std::array<int64_t, 3> qs{q.size(0), q.size(1), q.size(2)}, ks{q.size(0), k.defined() ? k.size(1) : 0, q.size(2)};
    p.total_tokens = qs[0];
    p.num_heads = size32(qs[1], "the number of heads");
    p.num_kv_heads = size32(ks[1], "the number of key/value heads");
    p.head_dim = size32(qs[2], "head_dim");
    p.dtype = code;
    p.inverse = a.number(5) != 0;
    if (k.defined() && ks[1] == 0) throw Refused("k has no heads");
    const Rows qr = rows_of(q, "q", qs, dt, dev), kr = rows_of(k, "k", ks, dt, dev);
    p.q_stride = qr.stride;
    p.k_stride = kr.stride;
    p.positions = static_cast<const int32_t*>(fit(pos, "positions", {qs[0]}, at::kInt, dev));
    if (cu.defined()) {
      p.num_seqs = size32(cu.numel() - 1, "the number of sequences of cu_seqlens,");
      p.cu_seqlens = static_cast<const int32_t*>(fit(cu, "cu_seqlens", {cu.numel()}, at::kInt, dev));
    }
    int32_t* const status = word(a.maybe(10, "status"), dev);
    const c10::cuda::CUDAGuard on(dev);
    const Tensor q_given = a.maybe(8, "q_out"), k_given = a.maybe(9, "k_out");
    Tensor qo = q_given, ko = k_given;
    if (!k.defined() && ko.defined()) throw Refused("k_out without k");
    if (!qo.defined()) qo = at::empty(qs, q.options().requires_grad(false));
    if (k.defined() && !ko.defined()) ko = at::empty(ks, q.options().requires_grad(false));
    void *const qop = fit(qo, "q_out", qs, dt, dev), *const kop = fit(ko, "k_out", ks, dt, dev);
    if (q_given.defined() || k_given.defined())
      apart({span("q_out", q_given), span("k_out", k_given)},
            {span("q", q, qr), span("k", k, kr), span("frequencies", a.at(0, "frequencies")), span("positions", pos),
             span("cu_seqlens", cu)}, {"q", "k"});
    p.fresh = (q_given.defined() ? 0 : 1) | (k.defined() && !k_given.defined() ? 2 : 0);
    const kda_status r = g_entry.rotary(&p, qr.p, kr.p, qop, kop, status, stream_of(q));
    if (r != KDA_OK) return PyLong_FromLong(r);
    written(q_given);
    written(k_given);
    return Py_BuildValue("(NN)", wrap(qo), wrap(ko));
  });
}

// freqs interleaved magnitude q|None k v k_pages v_pages page_table kv_lens cu_seqlens q_out|None status|None
PyObject* append_rotary(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
  return guarded(nargs, 13, [&]() -> PyObject* {
    const Args a{v};
    const Tensor q = a.maybe(3, "q"), k = a.at(4, "k");
    if (k.dim() != 3 || (q.defined() && q.dim() != 3)) throw Refused("q and k must be [S, heads, D] (k: " + text(k.sizes()) + ")");
    on_cuda(k, "k");
    const auto dev = k.get_device();
    kda_rotary_problem p = turn(a, 0, dev);
    const Paged g = paged(a, 6, q.defined() ? q : k, q.defined() ? "q" : "k", k.size(1), 1.0);
    const std::array<int64_t, 3> ks{k.size(0), k.size(1), k.size(2)}, qs{ks[0], q.defined() ? q.size(1) : 0, ks[2]};
    const Tensor val = a.at(5, "v"), kp = a.at(6, "k_pages"), vp = a.at(7, "v_pages");
    const Rows qr = rows_of(q, "q", qs, at::kBFloat16, dev), kr = rows_of(k, "k", ks, at::kBFloat16, dev),
               vr = rows_of(val, "v", ks, at::kBFloat16, dev);
    p.q_stride = qr.stride;
    p.k_stride = kr.stride;
    int32_t* const status = word(a.maybe(12, "status"), dev);
    const c10::cuda::CUDAGuard on(dev);
    const Tensor given = a.maybe(11, "q_out");
    Tensor qo = given;
    if (!q.defined() && qo.defined()) throw Refused("q_out without q");
    if (q.defined() && !qo.defined()) qo = at::empty(qs, q.options().requires_grad(false));
    void* const qop = fit(qo, "q_out", qs, at::kBFloat16, dev);
    apart({span("q_out", given), span("k_pages", kp), span("v_pages", vp)},
          {span("q", q, qr), span("k", k, kr), span("v", val, vr), span("frequencies", a.at(0, "frequencies")),
           span("page_table", a.at(8, "page_table")), span("kv_lens", a.at(9, "kv_lens")),
           span("cu_seqlens", a.at(10, "cu_seqlens"))}, {"q"});
    p.fresh = q.defined() && !given.defined() ? 1 : 0;
    const kda_status r = g_entry.append_rotary(&g.p, &p, vr.stride, qr.p, kr.p, vr.p, qop, g.k, g.v, status, stream_of(k));
    if (r != KDA_OK) return PyLong_FromLong(r);
    written(given);
    written(kp);
    written(vp);
    return wrap(qo);
  });
}

struct Packed {
  kda_attention_problem p;
  void *q, *k, *v;
  std::array<int64_t, 3> qs, ks;
};
Packed packed(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& cu, PyObject* scale, double given) {
  if (q.dim() != 3 || k.dim() != 3)
    throw Refused("q must be [S, Hq, D] and k, v [S, Hkv, D] (got " + text(q.sizes()) + ", " + text(k.sizes()) + ")");
  on_cuda(q, "q");
  const auto dev = q.get_device();
  Packed r{};
  r.qs = {q.size(0), q.size(1), q.size(2)};
  r.ks = {q.size(0), k.size(1), q.size(2)};
  r.p.total_tokens = r.qs[0];
  r.p.num_seqs = size32(cu.numel() - 1, "the number of sequences of cu_seqlens,");
  r.p.num_heads = size32(r.qs[1], "the number of heads");
  r.p.num_kv_heads = size32(r.ks[1], "the number of key/value heads");
  r.p.head_dim = size32(r.qs[2], "head_dim");
  r.p.dtype = KDA_DTYPE_BF16;
  r.p.scale = static_cast<float>(scale == Py_None ? 1.0 / std::sqrt(static_cast<double>(r.qs[2])) : given);
  const Rows qr = rows_of(q, "q", r.qs, at::kBFloat16, dev), kr = rows_of(k, "k", r.ks, at::kBFloat16, dev),
             vr = rows_of(v, "v", r.ks, at::kBFloat16, dev);
  r.q = qr.p;
  r.k = kr.p;
  r.v = vr.p;
  r.p.q_stride = qr.stride;
  r.p.k_stride = kr.stride;
  r.p.v_stride = vr.stride;
  r.p.cu_seqlens = static_cast<const int32_t*>(fit(cu, "cu_seqlens", {cu.numel()}, at::kInt, dev));
  return r;
}

// q k v cu_seqlens scale|None out|None workspace|None status|None
PyObject* packed_fwd(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
  return guarded(nargs, 8, [&]() -> PyObject* {
    const Args a{v};
    const Tensor q = a.at(0, "q");
    const Packed g = packed(q, a.at(1, "k"), a.at(2, "v"), a.at(3, "cu_seqlens"), v[4], v[4] == Py_None ? 0 : a.number(4));
    const auto dev = q.get_device();
    const c10::cuda::CUDAGuard on(dev);
    const Tensor given = a.maybe(5, "out");
    Tensor out = given, ws = a.maybe(6, "workspace");
    if (!out.defined()) out = at::empty(g.qs, q.options().requires_grad(false));
    void* const op = fit(out, "out", g.qs, at::kBFloat16, dev);
    const Tensor lse = at::empty({g.qs[1], g.qs[0]}, q.options().dtype(at::kFloat).requires_grad(false));
    const bool own = !ws.defined();
    const size_t bytes = g_entry.packed_fwd_bytes(&g.p);  // of a longer workspace the rest is not touched
    void* const wsp = buffer(ws, bytes, q);
    if (given.defined() || !own) {
      const Tensor k = a.at(1, "k"), val = a.at(2, "v");
      apart({span("out", given), kda::whole("workspace", wsp, own ? 0 : bytes)},
            {span("q", q, {g.q, g.p.q_stride}), span("k", k, {g.k, g.p.k_stride}), span("v", val, {g.v, g.p.v_stride}),
             span("cu_seqlens", a.at(3, "cu_seqlens"))}, {"q"});
    }
    const kda_status r = g_entry.packed_fwd(&g.p, g.q, g.k, g.v, op, static_cast<float*>(lse.data_ptr()), wsp,
                                            given.defined() ? 2 : 3, word(a.maybe(7, "status"), dev), stream_of(q));
    if (r != KDA_OK) return PyLong_FromLong(r);
    written(given);
    return Py_BuildValue("(NN)", wrap(out), wrap(lse));
  });
}

// q k v o lse d_o cu_seqlens scale|None workspace|None status|None
PyObject* packed_bwd(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
  return guarded(nargs, 10, [&]() -> PyObject* {
    const Args a{v};
    const Tensor q = a.at(0, "q");
    const Packed g = packed(q, a.at(1, "k"), a.at(2, "v"), a.at(6, "cu_seqlens"), v[7], v[7] == Py_None ? 0 : a.number(7));
    const auto dev = q.get_device();
    void* const op = fit(a.at(3, "o"), "o", g.qs, at::kBFloat16, dev);
    const float* const lp = static_cast<float*>(fit(a.at(4, "lse"), "lse", {g.qs[1], g.qs[0]}, at::kFloat, dev));
    void* const gp = fit(a.at(5, "d_o"), "d_o", g.qs, at::kBFloat16, dev);
    const c10::cuda::CUDAGuard on(dev);
    Tensor ws = a.maybe(8, "workspace");
    const bool own = !ws.defined();
    const size_t bytes = g_entry.packed_bwd_bytes(&g.p);
    void* const wsp = buffer(ws, bytes, q);
    if (!own) {
      const Tensor k = a.at(1, "k"), val = a.at(2, "v");
      apart({kda::whole("workspace", wsp, bytes)},
            {span("q", q, {g.q, g.p.q_stride}), span("k", k, {g.k, g.p.k_stride}), span("v", val, {g.v, g.p.v_stride}),
             span("o", a.at(3, "o")), span("lse", a.at(4, "lse")), span("d_o", a.at(5, "d_o")),
             span("cu_seqlens", a.at(6, "cu_seqlens"))});
    }
    const auto opts = q.options().requires_grad(false);
    const Tensor dq = at::empty(g.qs, opts), dk = at::empty(g.ks, opts), dv = at::empty(g.ks, opts);
    const kda_status r = g_entry.packed_bwd(&g.p, g.q, g.k, g.v, op, lp, gp, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), wsp, 1,
                                            word(a.maybe(9, "status"), dev), stream_of(q));
    return r == KDA_OK ? Py_BuildValue("(NNN)", wrap(dq), wrap(dk), wrap(dv)) : PyLong_FromLong(r);
  });
}

// Tensors of a list or tuple as the gradient operators take them.
struct Grads {
  std::vector<Tensor> t;
  std::vector<const void*> p;
  std::vector<int64_t> n;
  std::vector<int32_t> dtype;
};
Grads grads_of(PyObject* list, const char* name) {
  if (!PyList_Check(list) && !PyTuple_Check(list)) throw Refused(std::string(name) + " must be a list or tuple of tensors");
  const Py_ssize_t num = PySequence_Fast_GET_SIZE(list);
  PyObject* const* const items = PySequence_Fast_ITEMS(list);
  Grads g;
  g.n.reserve(num);
  g.t.reserve(num);
  g.p.reserve(num);
  g.dtype.reserve(num);
  for (Py_ssize_t i = 0; i < num; ++i) {
    const auto which = [&]() { return std::string(name) + "[" + std::to_string(i) + "]"; };
    if (!THPVariable_Check(items[i])) throw Refused(which() + " must be a tensor");
    const Tensor& t = THPVariable_Unpack(items[i]);
    const bool dense = t.layout() == at::kStrided && (t.is_contiguous() || t.is_non_overlapping_and_dense());
    if (!t.is_cuda() || (i > 0 && t.get_device() != g.t[0].get_device()) || !dense)
      throw Refused(which() + " must be a dense CUDA tensor on the first one's device (got " + text(t.sizes()) +
                    (t.is_cuda() ? ")" : " on the CPU)"));
    const auto dt = t.scalar_type();
    g.dtype.push_back(dt == at::kBFloat16 ? KDA_DTYPE_BF16
                                          : dt == at::kFloat ? KDA_DTYPE_F32 : activation(t, (which() + " must be").c_str()));
    g.p.push_back(t.numel() ? t.data_ptr() : nullptr);
    g.n.push_back(t.numel());
    g.t.push_back(t);
  }
  return g;
}

// An output may be its own gradient's memory and nothing else of the call's.
void no_overlap(const Grads& g, const Grads& o) {
  struct Range {
    uintptr_t at, end;
    bool out;
    size_t i;
  };
  std::vector<Range> r;
  r.reserve(2 * g.t.size());
  for (size_t i = 0; i < g.t.size(); ++i) {
    if (g.n[i] == 0) continue;
    const auto add = [&](const Grads& x, bool out) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(x.p[i]);
      r.push_back({at, at + x.t[i].nbytes(), out, i});
    };
    add(o, true);
    if (g.p[i] != o.p[i]) add(g, false);
  }
  std::sort(r.begin(), r.end(), [](const Range& x, const Range& y) { return x.at < y.at; });
  uintptr_t end = 0, out_end = 0;  // of what came before
  for (const Range& x : r) {
    if (x.at < (x.out ? end : out_end))
      throw Refused((x.out ? "out[" : "grads[") + std::to_string(x.i) + "] overlaps another tensor of the call");
    end = std::max(end, x.end);
    if (x.out) out_end = std::max(out_end, x.end);
  }
}

// grads workspace|None
PyObject* norm_of_grads(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
  return guarded(nargs, 2, [&]() -> PyObject* {
    const Args a{v};
    const Grads g = grads_of(v[0], "grads");
    const auto dev = g.t.empty() ? c10::cuda::current_device() : g.t[0].get_device();
    const c10::cuda::CUDAGuard on(dev);
    const Tensor norm = at::empty({}, at::TensorOptions().dtype(at::kFloat).device(c10::Device(at::kCUDA, dev)));
    const int32_t num = size32(static_cast<int64_t>(g.t.size()), "the number of tensors");
    Tensor ws = a.maybe(1, "workspace");
    void* const wsp = buffer(ws, g_entry.norm_of_grads_bytes(num), norm);
    const kda_status r = g_entry.norm_of_grads(num, g.p.data(), g.n.data(), g.dtype.data(), static_cast<float*>(norm.data_ptr()),
                                               wsp, stream_of(norm));
    return r == KDA_OK ? wrap(norm) : PyLong_FromLong(r);
  });
}

// grads max_norm out|None workspace|None
PyObject* clip(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
  return guarded(nargs, 4, [&]() -> PyObject* {
    const Args a{v};
    const Grads g = grads_of(v[0], "grads");
    const Grads other = v[2] == Py_None ? Grads() : grads_of(v[2], "out");
    const Grads& o = v[2] == Py_None ? g : other;
    if (o.t.size() != g.t.size()) throw Refused("out must have as many tensors as grads");
    for (size_t i = 0; &o != &g && i < g.t.size(); ++i)
      if (o.t[i].sizes() != g.t[i].sizes() || o.t[i].strides() != g.t[i].strides() ||
          o.t[i].get_device() != g.t[i].get_device() || (g.n[i] > 0 && o.p[i] == g.p[i] && o.dtype[i] != g.dtype[i]))
        throw Refused("out[" + std::to_string(i) + "] must have the shape, strides and device of grads[" + std::to_string(i) + "]");
    no_overlap(g, o);
    const auto dev = g.t.empty() ? c10::cuda::current_device() : g.t[0].get_device();
    const c10::cuda::CUDAGuard on(dev);
    const Tensor norm = at::empty({}, at::TensorOptions().dtype(at::kFloat).device(c10::Device(at::kCUDA, dev)));
    const int32_t num = size32(static_cast<int64_t>(g.t.size()), "the number of tensors");
    Tensor ws = a.maybe(3, "workspace");
    void* const wsp = buffer(ws, g_entry.norm_of_grads_bytes(num), norm);
    const kda_status r = g_entry.clip(num, g.p.data(), g.n.data(), g.dtype.data(), const_cast<void* const*>(o.p.data()),
                                      o.dtype.data(), a.number(1), static_cast<float*>(norm.data_ptr()), wsp, stream_of(norm));
    if (r != KDA_OK) return PyLong_FromLong(r);
    for (const Tensor& x : o.t) written(x);
    return wrap(norm);
  });
}

// addresses of the entry points, in the order of Entry
PyObject* init(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
  constexpr Py_ssize_t n = sizeof(Entry) / sizeof(void*);
  return guarded(nargs, n, [&]() -> PyObject* {
    for (Py_ssize_t i = 0; i < n; ++i) {
      void* const p = PyLong_AsVoidPtr(v[i]);
      if (!p) throw Refused("an entry point is missing");
      reinterpret_cast<void**>(&g_entry)[i] = p;
    }
    Py_RETURN_NONE;
  });
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(init),          METHOD(step),       METHOD(norm_fwd),   METHOD(norm_bwd),
                         METHOD(verify),        METHOD(append),     METHOD(attention),  METHOD(rotary),
                         METHOD(append_rotary), METHOD(packed_fwd), METHOD(packed_bwd), METHOD(norm_of_grads),
                         METHOD(clip),          {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kda_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kda_bind() { return PyModule_Create(&module); }
