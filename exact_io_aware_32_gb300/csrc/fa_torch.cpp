// Python module _fa_torch: the paged cache's helpers for torch tensors. It
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

namespace {

using Plan = int (*)(const int*, const int*, int, int, const int*, int, const int*, int*, int, int*, int*, int*, int,
                     int*, void*);
using Store = int (*)(const void*, const void*, long long, long long, const int*, int, int, int, void*, void*, int, int,
                      int, float, float, void*);
using Bytes = size_t (*)(int, int, int, int, int, int);
using Forward = int (*)(const void*, long long, const void*, const void*, int, float, float, const int*, int,
                        const int*, const int*, void*, float*, int, int, int, int, int, int, int, int, float, int,
                        void*, size_t, void*);
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
    count(n, 4);
    void* p[4];
    for (int i = 0; i < 4; ++i) {
      p[i] = PyLong_AsVoidPtr(a[i]);
      if (!p[i]) refuse("an address is missing");
    }
    g_plan = reinterpret_cast<Plan>(p[0]);
    g_store = reinterpret_cast<Store>(p[1]);
    g_bytes = reinterpret_cast<Bytes>(p[2]);
    g_forward = reinterpret_cast<Forward>(p[3]);
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
// descale_v, out or None, lse or None, workspace or None)
PyObject* forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 14);
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
    const int st = g_forward(q.at, q.stride, c.k, c.v, c.fp8, (float)number(a[9]), (float)number(a[10]), pt, width, ps,
                             pl, po, static_cast<float*>(plse), q.T, R, q.heads, c.heads, c.d, c.pages, c.page, max_new,
                             (float)scale, truth(a[7]), ws.data_ptr(), ws.nbytes(), stream_of(dev));
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

PyMethodDef g_methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(bind)), METH_FASTCALL, nullptr},
    {"plan", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(plan)), METH_FASTCALL, nullptr},
    {"store", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(store)), METH_FASTCALL, nullptr},
    {"forward", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(forward)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_fa_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fa_torch() { return PyModule_Create(&g_module); }
