// Python module _fa_torch: helpers of the paged cache, the rotation and the windowed attention for torch tensors. It
// checks the tensors, allocates what the caller did not give and calls the C
// ABI (by the addresses that bind() is given). A decoding step is a few
// microseconds on the GPU and these calls run between any two of them: the same
// checks in Python with a ctypes call of 27 arguments took 18 us for an
// attention call whose launches take 3.4 us.
//
// Every function returns its result, or an fa_status error code as an int;
// tensors that do not fit raise ValueError.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <stdexcept>
#include <string>

#include "../../include/fa.h"

namespace {

using Plan = int (*)(const int*, const int*, int, int, const int*, int, const int*, int*, int, int*, int*, int*, int,
                     int*, void*);
using Store = int (*)(const void*, const void*, long long, long long, const int*, int, int, int, void*, void*, int, int,
                      int, float, float, void*);
using Bytes = size_t (*)(int, int, int, int, int, int);
using Forward = int (*)(const void*, long long, const void*, const void*, int, float, float, const int*, int,
                        const int*, const int*, void*, float*, int, int, int, int, int, int, int, int, float, int,
                        void*, size_t, void*);
using RopeForward = decltype(&fa_rope_fwd);
using RopeBytes = decltype(&fa_rope_bwd_workspace_bytes);
using RopeBackward = decltype(&fa_rope_bwd);
using Positions = decltype(&fa_paged_positions);
using RopeStore = decltype(&fa_paged_rope_store);
using Window = decltype(&fa_fwd_paged_window);
using WindowForward = decltype(&fa_fwd_window);
using WindowBytes = decltype(&fa_bwd_window_workspace_bytes);
using WindowBackward = decltype(&fa_bwd_window);
Window g_window = nullptr;
WindowForward g_window_forward = nullptr;
WindowBytes g_window_bytes = nullptr;
WindowBackward g_window_backward = nullptr;
RopeForward g_rope = nullptr;
RopeBytes g_rope_bytes = nullptr;
RopeBackward g_rope_backward = nullptr;
Positions g_positions = nullptr;
RopeStore g_rope_store = nullptr;
Plan g_plan = nullptr;
Store g_store = nullptr;
Bytes g_bytes = nullptr;
Forward g_forward = nullptr;

[[noreturn]] void refuse(const std::string& why) { throw std::invalid_argument(why); }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

std::string text(std::initializer_list<int64_t> shape) {
  std::string s = "[";
  for (int64_t n : shape) s += (s.size() > 1 ? ", " : "") + std::to_string(n);
  return s + "]";
}

// A contiguous tensor of this type and shape on this device.
void* contiguous(const at::Tensor& t, const char* name, c10::ScalarType type, std::initializer_list<int64_t> shape,
                 c10::Device device) {
  bool ok = t.scalar_type() == type && t.device() == device && t.dim() == (int64_t)shape.size() && t.is_contiguous();
  int64_t i = 0;
  for (int64_t n : shape) ok = ok && t.size(i++) == n;
  if (!ok)
    refuse(std::string(name) + " must be a contiguous " + c10::toString(type) + " tensor of shape " + text(shape) +
           " on " + device.str());
  return t.data_ptr();
}
int* ints(const at::Tensor& t, const char* name, std::initializer_list<int64_t> shape, c10::Device device) {
  return static_cast<int*>(contiguous(t, name, c10::ScalarType::Int, shape, device));
}

// Sizes as the C ABI takes them.
int size(int64_t n, const char* what) {
  if (n < 0 || n > INT32_MAX) refuse(std::string(what) + " does not fit 32 bits");
  return (int)n;
}
int integer(PyObject* o, const char* what) {
  const long long n = PyLong_AsLongLong(o);
  if (n == -1 && PyErr_Occurred()) throw std::runtime_error("");
  if (n < INT32_MIN || n > INT32_MAX) refuse(std::string(what) + " does not fit 32 bits");
  return (int)n;
}
double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw std::runtime_error("");
  return x;
}
bool truth(PyObject* o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw std::runtime_error("");
  return x != 0;
}

// A packed [T, heads, d] bf16 tensor whose rows of one token are contiguous.
struct Packed {
  void* at;
  int T, heads, d;
  long long stride;
};
Packed packed(const at::Tensor& t, const char* name, c10::Device device) {
  if (t.scalar_type() != c10::ScalarType::BFloat16 || t.device() != device || t.dim() != 3)
    refuse(std::string(name) + " must be a bf16 tensor [T, heads, d] on " + device.str());
  Packed p;
  p.T = size(t.size(0), "T");
  p.heads = size(t.size(1), "heads");
  p.d = size(t.size(2), "d");
  if ((t.stride(2) != 1 && p.d > 1) || (t.stride(1) != p.d && p.heads > 1))
    refuse(std::string("the rows of one token of ") + name + " must be contiguous");
  p.stride = p.T > 1 ? t.stride(0) : (long long)p.heads * p.d;  // one token: its stride is not used
  p.at = t.data_ptr();
  return p;
}

// The cache pair [num_pages, Hkv, page_size, d], bf16 or E4M3 codes.
struct Cache {
  void *k, *v;
  int pages, heads, page, d, fp8;
};
Cache cache(const at::Tensor& k, const at::Tensor& v) {
  const auto type = k.scalar_type();
  Cache c;
  c.fp8 = type != c10::ScalarType::BFloat16;
  if ((c.fp8 && type != c10::ScalarType::Float8_e4m3fn && type != c10::ScalarType::Byte) || k.dim() != 4)
    refuse("the caches must be [num_pages, Hkv, page_size, d] tensors, bf16 or E4M3 codes");
  if (!k.is_cuda() || v.sizes() != k.sizes() || v.scalar_type() != type || v.device() != k.device() ||
      !k.is_contiguous() || !v.is_contiguous())
    refuse("k_cache and v_cache must be contiguous CUDA tensors of one shape, type and device");
  c.pages = size(k.size(0), "num_pages");
  c.heads = size(k.size(1), "Hkv");
  c.page = size(k.size(2), "page_size");
  c.d = size(k.size(3), "d");
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  return c;
}

void* stream_of(c10::Device device) { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }

void count(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) refuse("wrong number of arguments");
}

// Runs a function body: C++ exceptions become Python's.
template <class F>
PyObject* guarded(F body) {
  try {
    return body();
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    constexpr int kFunctions = 13;
    count(n, kFunctions);
    void* p[kFunctions];
    for (int i = 0; i < kFunctions; ++i) {
      p[i] = PyLong_AsVoidPtr(a[i]);
      if (!p[i]) refuse("an address is missing");
    }
    g_plan = reinterpret_cast<Plan>(p[0]);
    g_store = reinterpret_cast<Store>(p[1]);
    g_bytes = reinterpret_cast<Bytes>(p[2]);
    g_forward = reinterpret_cast<Forward>(p[3]);
    g_rope = reinterpret_cast<RopeForward>(p[4]);
    g_rope_bytes = reinterpret_cast<RopeBytes>(p[5]);
    g_rope_backward = reinterpret_cast<RopeBackward>(p[6]);
    g_positions = reinterpret_cast<Positions>(p[7]);
    g_rope_store = reinterpret_cast<RopeStore>(p[8]);
    g_window = reinterpret_cast<Window>(p[9]);
    g_window_forward = reinterpret_cast<WindowForward>(p[10]);
    g_window_bytes = reinterpret_cast<WindowBytes>(p[11]);
    g_window_backward = reinterpret_cast<WindowBackward>(p[12]);
    Py_RETURN_NONE;
  });
}

// plan(ctx_lens, new_lens, block_table, free_pages, page_size, num_tokens, free_head or None, out or None)
PyObject* plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 8);
    const at::Tensor &ctx = tensor(a[0], "ctx_lens"), &fresh = tensor(a[1], "new_lens"),
                     &table = tensor(a[2], "block_table"), &free = tensor(a[3], "free_pages");
    if (!ctx.is_cuda() || ctx.dim() != 1 || table.dim() != 2 || free.dim() != 1)
      refuse("expected CUDA tensors ctx_lens [R], block_table [R, max_pages], free_pages [n]");
    const c10::Device dev = ctx.device();
    const int64_t R = ctx.size(0), width = table.size(1), n_free = free.size(0);
    const int page_size = integer(a[4], "page_size"), T = integer(a[5], "num_tokens");
    if (T < 0) refuse("num_tokens must not be negative");
    const int *pc = ints(ctx, "ctx_lens", {R}, dev), *pn = ints(fresh, "new_lens", {R}, dev),
              *pf = ints(free, "free_pages", {n_free}, dev);
    int* pt = ints(table, "block_table", {R, width}, dev);
    const int* ph = a[6] == Py_None ? nullptr : ints(tensor(a[6], "free_head"), "free_head", {1}, dev);
    const c10::cuda::CUDAGuard guard(dev);
    PyObject* out = a[7];
    if (out == Py_None) {
      const int64_t sizes[4] = {R + 1, R, T, 1};
      out = PyTuple_New(4);
      if (!out) return nullptr;
      for (int i = 0; i < 4; ++i)
        PyTuple_SET_ITEM(out, i, THPVariable_Wrap(at::empty({sizes[i]}, ctx.options())));
    } else {
      if (!PyTuple_Check(out) || PyTuple_GET_SIZE(out) != 4) refuse("out must be a tuple of four tensors");
      Py_INCREF(out);
    }
    int st;
    try {
      int* p[4];
      const char* names[4] = {"query_start", "seq_lens", "slots", "pages_taken"};
      const int64_t sizes[4] = {R + 1, R, T, 1};
      for (int i = 0; i < 4; ++i) p[i] = ints(tensor(PyTuple_GET_ITEM(out, i), names[i]), names[i], {sizes[i]}, dev);
      // an empty list has no address: any valid one will do, since none of its entries is read
      st = g_plan(pc, pn, size(R, "R"), page_size, n_free ? pf : p[3], size(n_free, "free_pages"), ph, pt,
                  size(width, "max_pages"), p[0], p[1], p[2], T, p[3], stream_of(dev));
    } catch (...) {
      Py_DECREF(out);
      throw;
    }
    if (st == 0) return out;
    Py_DECREF(out);
    return PyLong_FromLong(st);
  });
}

// store(k, v, slots, k_cache, v_cache, descale_k, descale_v)
PyObject* store(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 7);
    const at::Tensor& kc = tensor(a[3], "k_cache");
    const Cache c = cache(kc, tensor(a[4], "v_cache"));
    const c10::Device dev = kc.device();
    const Packed k = packed(tensor(a[0], "k"), "k", dev), v = packed(tensor(a[1], "v"), "v", dev);
    if (k.heads != c.heads || v.heads != c.heads || k.d != c.d || v.d != c.d || v.T != k.T)
      refuse("k and v must be [T, " + std::to_string(c.heads) + ", " + std::to_string(c.d) + "], as the caches");
    const int* slots = ints(tensor(a[2], "slots"), "slots", {k.T}, dev);
    const c10::cuda::CUDAGuard guard(dev);
    const int st = g_store(k.at, v.at, k.stride, v.stride, slots, k.T, c.heads, c.d, c.k, c.v, c.pages, c.page, c.fp8,
                           (float)number(a[5]), (float)number(a[6]), stream_of(dev));
    if (st != 0) return PyLong_FromLong(st);
    Py_RETURN_NONE;
  });
}

// forward(q, k_cache, v_cache, block_table, query_start, seq_lens, max_new or None, causal, scale or None, descale_k,
// descale_v, out or None, lse or None, workspace or None, window or None, sinks)
PyObject* forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 16);
    const at::Tensor &tq = tensor(a[0], "q"), &kc = tensor(a[1], "k_cache"), &table = tensor(a[3], "block_table");
    const Cache c = cache(kc, tensor(a[2], "v_cache"));
    const c10::Device dev = kc.device();
    const Packed q = packed(tq, "q", dev);
    if (q.d != c.d || table.dim() != 2)
      refuse("expected q [T, Hq, " + std::to_string(c.d) + "] and block_table [R, max_pages]");
    const int R = size(table.size(0), "R"), width = size(table.size(1), "max_pages");
    const int *pt = ints(table, "block_table", {R, width}, dev),
              *ps = ints(tensor(a[4], "query_start"), "query_start", {(int64_t)R + 1, }, dev),
              *pl = ints(tensor(a[5], "seq_lens"), "seq_lens", {R}, dev);
    const int max_new = a[6] == Py_None ? q.T : integer(a[6], "max_new");
    const double scale = a[8] == Py_None ? 1.0 / std::sqrt((double)c.d) : number(a[8]);
    const bool windowed = a[14] != Py_None, causal = truth(a[7]);
    const int window = windowed ? integer(a[14], "window") : 0, sinks = integer(a[15], "sinks");
    if (windowed && !causal) refuse("a window needs a causal call");
    if (!windowed && sinks != 0) refuse("sinks need a window");
    const c10::cuda::CUDAGuard guard(dev);
    const bool own_o = a[11] == Py_None, own_l = a[12] == Py_None;
    const at::Tensor o = own_o ? at::zeros({q.T, q.heads, q.d}, tq.options()) : tensor(a[11], "out");
    const at::Tensor l = own_l ? at::zeros({q.T, q.heads}, tq.options().dtype(at::kFloat)) : tensor(a[12], "lse");
    void* po = contiguous(o, "out", c10::ScalarType::BFloat16, {q.T, q.heads, q.d}, dev);
    void* plse = contiguous(l, "lse", c10::ScalarType::Float, {q.T, q.heads}, dev);
    const at::Tensor ws = a[13] == Py_None
                              ? at::empty({(int64_t)g_bytes(q.T, R, q.heads, c.heads, c.d, max_new)},
                                          tq.options().dtype(at::kByte))
                              : tensor(a[13], "workspace");
    if (ws.device() != dev || !ws.is_contiguous()) refuse("workspace must be a contiguous tensor on " + dev.str());
    const float fk = (float)number(a[9]), fv = (float)number(a[10]);
    const int st =
        windowed ? g_window(q.at, q.stride, c.k, c.v, c.fp8, fk, fv, pt, width, ps, pl, po, static_cast<float*>(plse), q.T, R,
                            q.heads, c.heads, c.d, c.pages, c.page, max_new, (float)scale, window, sinks, ws.data_ptr(),
                            ws.nbytes(), stream_of(dev))
                 : g_forward(q.at, q.stride, c.k, c.v, c.fp8, fk, fv, pt, width, ps, pl, po, static_cast<float*>(plse), q.T, R,
                             q.heads, c.heads, c.d, c.pages, c.page, max_new, (float)scale, causal, ws.data_ptr(), ws.nbytes(),
                             stream_of(dev));
    if (st != 0) return PyLong_FromLong(st);
    PyObject* r = PyTuple_New(2);
    if (!r) return nullptr;
    if (!own_o) Py_INCREF(a[11]);
    if (!own_l) Py_INCREF(a[12]);
    PyTuple_SET_ITEM(r, 0, own_o ? THPVariable_Wrap(o) : a[11]);
    PyTuple_SET_ITEM(r, 1, own_l ? THPVariable_Wrap(l) : a[12]);
    return r;
  });
}

// ---------------------------------------------------------------- rotation
// Rows [B, H, N, d] of bf16 at any strides, the elements of a row contiguous.
fa_heads heads(const at::Tensor& t, const char* name, c10::Device device) {
  if (t.scalar_type() != c10::ScalarType::BFloat16 || t.device() != device || t.dim() != 4)
    refuse(std::string(name) + " must be a bf16 tensor [B, H, N, d] on " + device.str());
  if (t.stride(3) != 1 && t.size(3) > 1) refuse(std::string("the rows of ") + name + " must be contiguous");
  return {t.data_ptr(), t.stride(0), t.stride(1), t.stride(2)};
}
void same_shape(const at::Tensor& t, const at::Tensor& as, const char* name) {
  if (t.sizes() != as.sizes()) refuse(std::string(name) + " must have the shape " + text({as.size(0), as.size(1), as.size(2), as.size(3)}));
}

// The frequencies, and the norms' weights.
struct Rotation {
  const double* freqs;
  int rotary, fp32 = 0;
  const void *wq = nullptr, *wk = nullptr;
};
Rotation rotation(PyObject* freqs, PyObject* wq, PyObject* wk, int d, c10::Device dev) {
  Rotation r;
  const at::Tensor& f = tensor(freqs, "freqs");
  if (f.dim() != 1) refuse("freqs must be a tensor [rotary / 2]");
  r.rotary = size(2 * f.size(0), "rotary");
  r.freqs = static_cast<const double*>(contiguous(f, "freqs", c10::ScalarType::Double, {f.size(0)}, dev));
  if (wq != Py_None) {
    const at::Tensor& w = tensor(wq, "q_weight");
    r.fp32 = w.scalar_type() == c10::ScalarType::Float;
    r.wq = contiguous(w, "q_weight", r.fp32 ? c10::ScalarType::Float : c10::ScalarType::BFloat16, {d}, dev);
  }
  if (wk != Py_None) {
    const at::Tensor& w = tensor(wk, "k_weight");
    if (wq == Py_None) refuse("k_weight needs q_weight");
    r.wk = contiguous(w, "k_weight", r.fp32 ? c10::ScalarType::Float : c10::ScalarType::BFloat16, {d}, dev);
  }
  return r;
}

struct Places {
  const int* at = nullptr;
  long long stride = 0;
};
Places places(PyObject* o, int64_t B, int64_t N, c10::Device dev) {
  Places p;
  if (o == Py_None) return p;
  const at::Tensor& t = tensor(o, "positions");
  const bool each = t.dim() == 2;
  p.at = each ? ints(t, "positions", {B, N}, dev) : ints(t, "positions", {N}, dev);
  p.stride = each ? N : 0;
  return p;
}

// rope(q, k or None, freqs, positions or None, interleaved, factor, q_weight or None, k_weight or None, eps, out or None)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 10);
    const at::Tensor& q = tensor(a[0], "q");
    if (!q.is_cuda()) refuse("q must be a CUDA tensor");
    const c10::Device dev = q.device();
    const fa_heads hq = heads(q, "q", dev);
    const bool has_k = a[1] != Py_None;
    const at::Tensor& k = has_k ? tensor(a[1], "k") : q;
    const fa_heads hk = heads(k, "k", dev);
    if (k.size(0) != q.size(0) || k.size(2) != q.size(2) || k.size(3) != q.size(3)) refuse("q and k must agree in B, N and d");
    const int B = size(q.size(0), "B"), Hq = size(q.size(1), "Hq"), Hk = has_k ? size(k.size(1), "Hk") : 0,
              N = size(q.size(2), "N"), d = size(q.size(3), "d");
    const Rotation r = rotation(a[2], a[6], a[7], d, dev);
    const Places p = places(a[3], B, N, dev);
    const double factor = number(a[5]), eps = number(a[8]);
    const bool inter = truth(a[4]);
    const c10::cuda::CUDAGuard guard(dev);
    at::Tensor qo, ko;
    if (a[9] == Py_None) {
      qo = at::empty(q.sizes(), q.options());
      if (has_k) ko = at::empty(k.sizes(), k.options());
    } else {
      if (!PyTuple_Check(a[9]) || PyTuple_GET_SIZE(a[9]) != (has_k ? 2 : 1)) refuse("out must be a tuple of the outputs");
      qo = tensor(PyTuple_GET_ITEM(a[9], 0), "q_out");
      same_shape(qo, q, "q_out");
      if (has_k) {
        ko = tensor(PyTuple_GET_ITEM(a[9], 1), "k_out");
        same_shape(ko, k, "k_out");
      }
    }
    const fa_heads oq = heads(qo, "q_out", dev), ok = has_k ? heads(ko, "k_out", dev) : fa_heads{};
    const int st = g_rope(&hq, &hk, &oq, &ok, r.wq, r.wk, r.fp32, (float)eps, r.freqs, r.rotary, inter, (float)factor, p.at,
                          p.stride, B, Hq, Hk, N, d, stream_of(dev));
    if (st != 0) return PyLong_FromLong(st);
    PyObject* out = PyTuple_New(2);
    if (!out) return nullptr;
    PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(qo));
    if (!has_k) Py_INCREF(Py_None);
    PyTuple_SET_ITEM(out, 1, has_k ? THPVariable_Wrap(ko) : Py_None);
    return out;
  });
}

// rope_backward(dq_out, dk_out or None, freqs, positions or None, interleaved, factor, q or None, k or None, q_weight or None,
// k_weight or None, eps)
PyObject* rope_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 11);
    const at::Tensor& gq = tensor(a[0], "dq_out");
    if (!gq.is_cuda()) refuse("dq_out must be a CUDA tensor");
    const c10::Device dev = gq.device();
    const bool has_k = a[1] != Py_None, norm = a[8] != Py_None;
    const at::Tensor& gk = has_k ? tensor(a[1], "dk_out") : gq;
    const fa_heads hgq = heads(gq, "dq_out", dev), hgk = heads(gk, "dk_out", dev);
    if (gk.size(0) != gq.size(0) || gk.size(2) != gq.size(2) || gk.size(3) != gq.size(3))
      refuse("dq_out and dk_out must agree in B, N and d");
    const int B = size(gq.size(0), "B"), Hq = size(gq.size(1), "Hq"), Hk = has_k ? size(gk.size(1), "Hk") : 0,
              N = size(gq.size(2), "N"), d = size(gq.size(3), "d");
    const Rotation r = rotation(a[2], a[8], a[9], d, dev);
    const Places p = places(a[3], B, N, dev);
    fa_heads hq{}, hk{};
    if (norm) {
      if (a[6] == Py_None || (has_k && a[7] == Py_None)) refuse("the gradients of norms need the forward's q and k");
      same_shape(tensor(a[6], "q"), gq, "q");
      hq = heads(tensor(a[6], "q"), "q", dev);
      if (has_k) {
        same_shape(tensor(a[7], "k"), gk, "k");
        hk = heads(tensor(a[7], "k"), "k", dev);
      }
    }
    const bool inter = truth(a[4]);
    const double factor = number(a[5]), eps = number(a[10]);
    const c10::cuda::CUDAGuard guard(dev);
    // token by token, as a projection's output is laid out
    const at::Tensor dq = at::empty({B, N, Hq, d}, gq.options()).transpose(1, 2);
    at::Tensor dk, dwq, dwk, ws;
    if (has_k) dk = at::empty({B, N, Hk, d}, gk.options()).transpose(1, 2);
    if (norm) {
      dwq = at::empty({d}, gq.options().dtype(at::kFloat));
      if (has_k) dwk = at::empty({d}, gq.options().dtype(at::kFloat));
      ws = at::empty({(int64_t)g_rope_bytes(Hq, Hk, d)}, gq.options().dtype(at::kByte));
    }
    const fa_heads odq = heads(dq, "dq", dev), odk = has_k ? heads(dk, "dk", dev) : fa_heads{};
    const int st = g_rope_backward(
        &hgq, &hgk, &hq, &hk, &odq, &odk, r.wq, r.wk, r.fp32, (float)eps, norm ? dwq.data_ptr<float>() : nullptr,
        norm && has_k ? dwk.data_ptr<float>() : nullptr, r.freqs, r.rotary, inter, (float)factor, p.at, p.stride, B, Hq, Hk, N,
        d, norm ? ws.data_ptr() : nullptr, norm ? ws.nbytes() : 0, stream_of(dev));
    if (st != 0) return PyLong_FromLong(st);
    PyObject* out = PyTuple_New(4);
    if (!out) return nullptr;
    const at::Tensor* t[4] = {&dq, &dk, &dwq, &dwk};
    for (int i = 0; i < 4; ++i) {
      if (!t[i]->defined()) Py_INCREF(Py_None);
      PyTuple_SET_ITEM(out, i, t[i]->defined() ? THPVariable_Wrap(*t[i]) : Py_None);
    }
    return out;
  });
}

// positions(query_start, seq_lens, num_tokens, out or None)
PyObject* positions(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 4);
    const at::Tensor& lens = tensor(a[1], "seq_lens");
    if (!lens.is_cuda() || lens.dim() != 1) refuse("seq_lens must be a CUDA tensor [R]");
    const c10::Device dev = lens.device();
    const int64_t R = lens.size(0);
    const int T = integer(a[2], "num_tokens");
    if (T < 0) refuse("num_tokens must not be negative");
    const int *pl = ints(lens, "seq_lens", {R}, dev), *ps = ints(tensor(a[0], "query_start"), "query_start", {R + 1}, dev);
    const c10::cuda::CUDAGuard guard(dev);
    const bool own = a[3] == Py_None;
    const at::Tensor out = own ? at::empty({T}, lens.options()) : tensor(a[3], "out");
    int* po = ints(out, "out", {T}, dev);
    const int st = g_positions(ps, pl, size(R, "R"), po, T, stream_of(dev));
    if (st != 0) return PyLong_FromLong(st);
    if (!own) Py_INCREF(a[3]);
    return own ? THPVariable_Wrap(out) : a[3];
  });
}

// rope_store(q, k, v, slots, positions, freqs, k_cache, v_cache, interleaved, factor, q_weight or None, k_weight or None, eps,
// descale_k, descale_v, out or None)
PyObject* rope_store(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 16);
    const at::Tensor& kc = tensor(a[6], "k_cache");
    const Cache c = cache(kc, tensor(a[7], "v_cache"));
    const c10::Device dev = kc.device();
    const at::Tensor& tq = tensor(a[0], "q");
    const Packed q = packed(tq, "q", dev), k = packed(tensor(a[1], "k"), "k", dev), v = packed(tensor(a[2], "v"), "v", dev);
    if (k.heads != c.heads || v.heads != c.heads || q.d != c.d || k.d != c.d || v.d != c.d || v.T != k.T || q.T != k.T)
      refuse("q must be [T, Hq, " + std::to_string(c.d) + "], k and v [T, " + std::to_string(c.heads) + ", " +
             std::to_string(c.d) + "], as the caches");
    const int *slots = ints(tensor(a[3], "slots"), "slots", {k.T}, dev),
              *pos = ints(tensor(a[4], "positions"), "positions", {k.T}, dev);
    const Rotation r = rotation(a[5], a[10], a[11], c.d, dev);
    const bool inter = truth(a[8]);
    const double factor = number(a[9]), eps = number(a[12]), fk = number(a[13]), fv = number(a[14]);
    const c10::cuda::CUDAGuard guard(dev);
    const bool own = a[15] == Py_None;
    const at::Tensor o = own ? at::zeros({q.T, q.heads, q.d}, tq.options()) : tensor(a[15], "out");
    const Packed po = packed(o, "out", dev);
    if (po.T != q.T || po.heads != q.heads || po.d != q.d) refuse("out must have the shape of q");
    const int st = g_rope_store(q.at, k.at, v.at, q.stride, k.stride, v.stride, slots, pos, r.freqs, r.rotary, inter,
                                (float)factor, r.wq, r.wk, r.fp32, (float)eps, po.at, po.stride, q.T, q.heads, c.heads, c.d,
                                c.k, c.v, c.pages, c.page, c.fp8, (float)fk, (float)fv, stream_of(dev));
    if (st != 0) return PyLong_FromLong(st);
    if (!own) Py_INCREF(a[15]);
    return own ? THPVariable_Wrap(o) : a[15];
  });
}

// ---------------------------------------------------------------- attention in a window
struct WindowSizes {
  int B, Hq, Hkv, Nq, Nk, d;
  c10::Device dev;
};
WindowSizes window_sizes(const at::Tensor& q, const at::Tensor& k, const at::Tensor& v) {
  if (!q.is_cuda() || q.dim() != 4 || k.dim() != 4) refuse("expected CUDA tensors q [B, Hq, Nq, d], k and v [B, Hkv, Nk, d]");
  const c10::Device dev = q.device();
  contiguous(q, "q", c10::ScalarType::BFloat16, {q.size(0), q.size(1), q.size(2), q.size(3)}, dev);
  contiguous(k, "k", c10::ScalarType::BFloat16, {q.size(0), k.size(1), k.size(2), q.size(3)}, dev);
  contiguous(v, "v", c10::ScalarType::BFloat16, {q.size(0), k.size(1), k.size(2), q.size(3)}, dev);
  return {size(q.size(0), "B"), size(q.size(1), "Hq"), size(k.size(1), "Hkv"), size(q.size(2), "Nq"), size(k.size(2), "Nk"),
          size(q.size(3), "d"), dev};
}
int* lengths(PyObject* o, const char* name, const WindowSizes& s) {
  return o == Py_None ? nullptr : ints(tensor(o, name), name, {s.B}, s.dev);
}
double scale_of(PyObject* o, int d) { return o == Py_None ? 1.0 / std::sqrt((double)d) : number(o); }

// window(q, k, v, window, sinks, scale or None, seqlens_q or None, seqlens_k or None)
PyObject* window(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 8);
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const WindowSizes s = window_sizes(q, k, v);
    const int width = integer(a[3], "window"), sinks = integer(a[4], "sinks");
    const double scale = scale_of(a[5], s.d);
    const int *lq = lengths(a[6], "seqlens_q", s), *lk = lengths(a[7], "seqlens_k", s);
    const c10::cuda::CUDAGuard guard(s.dev);
    const at::Tensor o = at::empty(q.sizes(), q.options()), lse = at::empty({s.B, s.Hq, s.Nq}, q.options().dtype(at::kFloat));
    const int st = g_window_forward(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr<float>(), s.B, s.Hq,
                                    s.Hkv, s.Nq, s.Nk, s.d, (float)scale, width, sinks, lq, lk, stream_of(s.dev));
    if (st != 0) return PyLong_FromLong(st);
    PyObject* out = PyTuple_New(2);
    if (!out) return nullptr;
    PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(o));
    PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(lse));
    return out;
  });
}

// window_backward(q, k, v, o, lse, dO, window, sinks, scale or None, seqlens_q or None, seqlens_k or None, workspace or None)
PyObject* window_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 12);
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const WindowSizes s = window_sizes(q, k, v);
    void *o = contiguous(tensor(a[3], "o"), "o", c10::ScalarType::BFloat16, {s.B, s.Hq, s.Nq, s.d}, s.dev),
         *lse = contiguous(tensor(a[4], "lse"), "lse", c10::ScalarType::Float, {s.B, s.Hq, s.Nq}, s.dev),
         *g = contiguous(tensor(a[5], "dO"), "dO", c10::ScalarType::BFloat16, {s.B, s.Hq, s.Nq, s.d}, s.dev);
    const int width = integer(a[6], "window"), sinks = integer(a[7], "sinks");
    const double scale = scale_of(a[8], s.d);
    const int *lq = lengths(a[9], "seqlens_q", s), *lk = lengths(a[10], "seqlens_k", s);
    const c10::cuda::CUDAGuard guard(s.dev);
    const at::Tensor dq = at::empty(q.sizes(), q.options()), dk = at::empty(k.sizes(), q.options()),
                     dv = at::empty(k.sizes(), q.options());
    const at::Tensor ws = a[11] == Py_None
                              ? at::empty({(int64_t)g_window_bytes(s.B, s.Hq, s.Hkv, s.Nq, s.Nk, s.d, width, sinks)},
                                          q.options().dtype(at::kByte))
                              : tensor(a[11], "workspace");
    if (ws.device() != s.dev || !ws.is_contiguous()) refuse("workspace must be a contiguous tensor on " + s.dev.str());
    const int st = g_window_backward(q.data_ptr(), k.data_ptr(), v.data_ptr(), o, static_cast<float*>(lse), g, dq.data_ptr(),
                                     dk.data_ptr(), dv.data_ptr(), s.B, s.Hq, s.Hkv, s.Nq, s.Nk, s.d, (float)scale, width,
                                     sinks, lq, lk, ws.data_ptr(), ws.nbytes(), stream_of(s.dev));
    if (st != 0) return PyLong_FromLong(st);
    PyObject* out = PyTuple_New(3);
    if (!out) return nullptr;
    PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(dq));
    PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(dk));
    PyTuple_SET_ITEM(out, 2, THPVariable_Wrap(dv));
    return out;
  });
}

PyMethodDef g_methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(bind)), METH_FASTCALL, nullptr},
    {"plan", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(plan)), METH_FASTCALL, nullptr},
    {"store", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(store)), METH_FASTCALL, nullptr},
    {"forward", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(forward)), METH_FASTCALL, nullptr},
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(rope)), METH_FASTCALL, nullptr},
    {"rope_backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(rope_backward)), METH_FASTCALL, nullptr},
    {"positions", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(positions)), METH_FASTCALL, nullptr},
    {"window", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(window)), METH_FASTCALL, nullptr},
    {"window_backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(window_backward)), METH_FASTCALL, nullptr},
    {"rope_store", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(rope_store)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_fa_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fa_torch() { return PyModule_Create(&g_module); }
