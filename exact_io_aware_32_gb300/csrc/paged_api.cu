// C ABI of the paged key/value cache (declared in include/fa.h): argument
// checks and kernel launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/fa.h"
#include "fa_internal.h"
#include "paged.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// log2 of a page size the kernels take, or -1.
int page_shift(int page_size) {
  for (int s = 4; s <= 8; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

// The cache's shape: its slots and (page, head) pairs are counted in 32 bits.
int check_cache(int num_pages, int page_size, int Hkv, int d) {
  if (num_pages < 1 || Hkv < 1 || d < 1 || page_size < 1) return FA_ERR_INVALID_ARG;
  if ((long long)num_pages * page_size > INT32_MAX || (long long)num_pages * Hkv > INT32_MAX)
    return FA_ERR_INVALID_ARG;
  if (page_shift(page_size) < 0 || (d != 64 && d != 128)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// Token stride of a [T, heads, d] array: rows of one token contiguous, 16-byte aligned, tokens apart.
int check_stride(long long stride, int heads, int d) {
  if (stride < (long long)heads * d || stride >= (1ll << 39)) return FA_ERR_INVALID_ARG;
  return stride % 8 ? FA_ERR_MISALIGNED : FA_OK;
}

bool factor(float x) { return std::isfinite(x) && x > 0.f; }

// SMs that a workspace is made for (the GPU has 152), so that its size does not depend on the device.
constexpr int kMaxSms = 160;

// Requests of a plan: its kernel counts them in 32 bits, a few hundred at a time.
constexpr int kMaxPlanRequests = 1 << 30;

// Keys of the widest table: the kernels add up to four blocks of 128 to a place among the keys, in 32 bits.
constexpr int kMaxKeys = INT32_MAX - 511;

constexpr double kLog2e = 1.4426950408889634074;

int check_paged(int T, int R, int Hq, int Hkv, int d, int max_new) {
  if (T < 1 || R < 1 || Hq < 1 || Hkv < 1 || d < 1 || max_new < 1) return FA_ERR_INVALID_ARG;
  if (Hq % Hkv || (long long)T * Hq > INT32_MAX) return FA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || Hq / Hkv > 128) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

}  // namespace

extern "C" {

int fa_paged_plan(const int* ctx_lens, const int* new_lens, int R, int page_size, const int* free_pages, int n_free,
                  const int* free_head, int* block_table, int max_pages, int* query_start, int* seq_lens, int* slots,
                  int T, int* pages_taken, void* stream) {
  if (!ctx_lens || !new_lens || !free_pages || !block_table || !query_start || !seq_lens || !slots || !pages_taken)
    return FA_ERR_INVALID_ARG;
  if (R < 1 || R > kMaxPlanRequests || T < 1 || n_free < 0 || max_pages < 1 || page_size < 1) return FA_ERR_INVALID_ARG;
  const int shift = page_shift(page_size);
  if (shift < 0) return FA_ERR_UNSUPPORTED;
  if (((long long)max_pages << shift) > INT32_MAX) return FA_ERR_INVALID_ARG;
  for (const void* p : {(const void*)ctx_lens, (const void*)new_lens, (const void*)free_pages, (const void*)free_head,
                        (const void*)block_table, (const void*)query_start, (const void*)seq_lens, (const void*)slots,
                        (const void*)pages_taken})
    if (!aligned(p, 4)) return FA_ERR_MISALIGNED;
  // every block reads all lengths and the free list's head while others write: nothing written may be read elsewhere
  const struct {
    const int* at;
    long long n;
  } arrays[] = {{block_table, (long long)R * max_pages}, {query_start, R + 1ll}, {seq_lens, R}, {slots, T}, {pages_taken, 1},
                {ctx_lens, R}, {new_lens, R}, {free_pages, n_free}, {free_head, free_head ? 1 : 0}};
  for (int i = 0; i < 5; ++i)  // the first five are written
    for (int j = i + 1; j < 9; ++j) {
      const uintptr_t x = reinterpret_cast<uintptr_t>(arrays[i].at), y = reinterpret_cast<uintptr_t>(arrays[j].at);
      if (x < y + arrays[j].n * sizeof(int) && y < x + arrays[i].n * sizeof(int)) return FA_ERR_INVALID_ARG;
    }
  fa::PlanArgs a;
  std::memset(&a, 0, sizeof(a));
  int sms = 0;
  if (const int st = fa::device_facts(&sms, &a.status)) return st;
  a.ctx_lens = ctx_lens;
  a.new_lens = new_lens;
  a.free_pages = free_pages;
  a.free_head = free_head;
  a.block_table = block_table;
  a.query_start = query_start;
  a.seq_lens = seq_lens;
  a.slots = slots;
  a.pages_taken = pages_taken;
  a.R = R;
  a.T = T;
  a.n_free = n_free;
  a.max_pages = max_pages;
  a.page_shift = shift;
  return fa::launch_plan(a, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

int fa_paged_store(const void* k, const void* v, long long k_stride, long long v_stride, const int* slots, int T,
                   int Hkv, int d, void* k_cache, void* v_cache, int num_pages, int page_size, int fp8,
                   float descale_k, float descale_v, void* stream) {
  if (!k || !v || !slots || !k_cache || !v_cache || T < 1) return FA_ERR_INVALID_ARG;
  int st = check_cache(num_pages, page_size, Hkv, d);
  if (st != FA_OK) return st;
  if (fp8 && (!factor(descale_k) || !factor(descale_v))) return FA_ERR_INVALID_ARG;
  if ((st = check_stride(k_stride, Hkv, d)) != FA_OK || (st = check_stride(v_stride, Hkv, d)) != FA_OK) return st;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(slots, 4))
    return FA_ERR_MISALIGNED;
  fa::StoreArgs a;
  std::memset(&a, 0, sizeof(a));
  int sms = 0;
  if ((st = fa::device_facts(&sms, &a.status)) != FA_OK) return st;
  a.k = k;
  a.v = v;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.slots = slots;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.T = T;
  a.Hkv = Hkv;
  a.d = d;
  a.num_pages = num_pages;
  a.page_shift = page_shift(page_size);
  a.fp8 = fp8 ? 1 : 0;
  a.descale_k = descale_k;
  a.descale_v = descale_v;
  return fa::launch_store(a, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

size_t fa_fwd_paged_workspace_bytes(int T, int R, int Hq, int Hkv, int d, int max_new) {
  if (check_paged(T, R, Hq, Hkv, d, max_new) != FA_OK) return 0;
  size_t most = 0;
  for (int fp8 = 0; fp8 < 2; ++fp8) {  // one size for both kinds of cache
    fa::PagedPlan p[2];
    const int n = fa::plan_paged(T, R, Hq, Hkv, d, fp8, max_new, 16, INT32_MAX, 0, 0, kMaxSms, p);  // (any table width)
    for (int i = 0; i < n; ++i) most = std::max(most, p[i].bytes());
  }
  return most;
}

}  // extern "C"

namespace {

// Both forms of the attention; window 0: none.
int fwd_paged(const void* q, long long q_stride, const void* k_cache, const void* v_cache, int fp8, float descale_k,
              float descale_v, const int* block_table, int max_pages, const int* query_start, const int* seq_lens, void* o,
              float* lse, int T, int R, int Hq, int Hkv, int d, int num_pages, int page_size, int max_new, float scale,
              int causal, int window, int sinks, void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !k_cache || !v_cache || !block_table || !query_start || !seq_lens || !o || !lse) return FA_ERR_INVALID_ARG;
  int st = check_paged(T, R, Hq, Hkv, d, max_new);
  if (st == FA_OK) st = check_cache(num_pages, page_size, Hkv, d);
  if (st != FA_OK) return st;
  if (max_pages < 1 || (long long)max_pages * page_size > kMaxKeys || !factor(scale)) return FA_ERR_INVALID_ARG;
  if (fp8 && (!factor(descale_k) || !factor(descale_v))) return FA_ERR_INVALID_ARG;
  const float scale_log2 = (float)((double)scale * (fp8 ? (double)descale_k : 1.0) * kLog2e);
  if (!factor(scale_log2)) return FA_ERR_INVALID_ARG;  // over- or underflow
  if ((st = check_stride(q_stride, Hq, d)) != FA_OK) return st;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(o, 16) || !aligned(lse, 16) ||
      !aligned(block_table, 4) || !aligned(query_start, 4) || !aligned(seq_lens, 4))
    return FA_ERR_MISALIGNED;
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < fa_fwd_paged_workspace_bytes(T, R, Hq, Hkv, d, max_new))
    return FA_ERR_WORKSPACE;
  // places in the row of tiles are 32-bit numbers of key blocks (paged_work.cuh)
  const int max_keys = max_pages * page_size;
  fa::PagedPlan p[2];
  // (a window or sinks past every key there can be are the widest that make a difference)
  window = std::min(window, max_keys);
  sinks = std::min(sinks, max_keys);
  int n = fa::plan_paged(T, R, Hq, Hkv, d, fp8 ? 1 : 0, max_new, page_size, max_keys, window, sinks, kMaxSms, p);
  for (int i = 0; i < n; ++i)
    if (fa::most_blocks(T, R, Hkv, p[i].tpt, max_keys) >= (double)INT32_MAX) return FA_ERR_INVALID_ARG;
  fa::PagedArgs a;
  std::memset(&a, 0, sizeof(a));
  int sms = 0;
  if ((st = fa::device_facts(&sms, &a.status)) != FA_OK) return st;
  a.q = q;
  a.q_stride = q_stride;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.block_table = block_table;
  a.query_start = query_start;
  a.seq_lens = seq_lens;
  a.o = o;
  a.lse = lse;
  a.T = T;
  a.R = R;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.num_pages = num_pages;
  a.page_shift = page_shift(page_size);
  a.max_pages = max_pages;
  a.causal = causal ? 1 : 0;
  a.fp8 = fp8 ? 1 : 0;
  a.scale_log2 = scale_log2;
  a.o_scale = fp8 ? descale_v : 1.0f;
  a.max_keys = max_keys;
  a.window = window;
  a.sinks = sinks;
  a.test_fault = fa::take_test_fault();
  n = fa::plan_paged(T, R, Hq, Hkv, d, a.fp8, max_new, page_size, a.max_keys, window, sinks, std::min(sms, kMaxSms), p);
  for (int i = 0; i < n; ++i) {
    a.most = (int)fa::most_blocks(T, R, Hkv, p[i].tpt, max_keys);
    if (fa::launch_paged(a, p[i], workspace, static_cast<cudaStream_t>(stream)) != cudaSuccess) return FA_ERR_LAUNCH;
  }
  return FA_OK;
}

}  // namespace

extern "C" {

int fa_fwd_paged(const void* q, long long q_stride, const void* k_cache, const void* v_cache, int fp8,
                 float descale_k, float descale_v, const int* block_table, int max_pages, const int* query_start,
                 const int* seq_lens, void* o, float* lse, int T, int R, int Hq, int Hkv, int d, int num_pages,
                 int page_size, int max_new, float scale, int causal, void* workspace, size_t workspace_bytes,
                 void* stream) {
  return fwd_paged(q, q_stride, k_cache, v_cache, fp8, descale_k, descale_v, block_table, max_pages, query_start, seq_lens, o,
                   lse, T, R, Hq, Hkv, d, num_pages, page_size, max_new, scale, causal, 0, 0, workspace, workspace_bytes,
                   stream);
}

int fa_fwd_paged_window(const void* q, long long q_stride, const void* k_cache, const void* v_cache, int fp8,
                        float descale_k, float descale_v, const int* block_table, int max_pages, const int* query_start,
                        const int* seq_lens, void* o, float* lse, int T, int R, int Hq, int Hkv, int d, int num_pages,
                        int page_size, int max_new, float scale, int window, int sinks, void* workspace,
                        size_t workspace_bytes, void* stream) {
  if (window < 1 || sinks < 0) return FA_ERR_INVALID_ARG;
  return fwd_paged(q, q_stride, k_cache, v_cache, fp8, descale_k, descale_v, block_table, max_pages, query_start, seq_lens, o,
                   lse, T, R, Hq, Hkv, d, num_pages, page_size, max_new, scale, 1, window, sinks, workspace, workspace_bytes,
                   stream);
}

}  // extern "C"
