// kda_bind.cpp -- the host side of the serving operators' Python binding
// (decode.py, norm.py): checks of the tensors, outputs, and the call of the C
// entry point (kda_serving.h) on the current stream.
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

#include <array>
#include <cmath>
#include <initializer_list>
#include <stdexcept>
#include <string>

#include "kda_serving.h"

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
} g_entry;

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

const char* name_of(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kInt: return "torch.int32";
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
PyMethodDef methods[] = {METHOD(init),   METHOD(step),   METHOD(norm_fwd),  METHOD(norm_bwd),
                         METHOD(verify), METHOD(append), METHOD(attention), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kda_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kda_bind() { return PyModule_Create(&module); }
