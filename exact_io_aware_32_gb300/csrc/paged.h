// Internal interface of the paged key/value cache's kernels (paged_api.cu calls
// the launchers of paged_cache.cu and paged_fwd.cu).
#pragma once
#include <cuda_runtime.h>
#include <cstddef>

namespace fa {

struct PlanArgs {
  const int *ctx_lens, *new_lens;       // [R]
  const int *free_pages, *free_head;    // [n_free]; [1] or NULL
  int *block_table;                     // [R][max_pages]
  int *query_start, *seq_lens, *slots;  // [R + 1], [R], [T]
  int *pages_taken;                     // [1]
  unsigned int* status;
  int R, T, n_free, max_pages, page_shift;  // page_size = 1 << page_shift
  int group;                                // requests per CTA (set by launch_plan)
};

struct StoreArgs {
  const void *k, *v;  // bf16 [T][Hkv][d]
  long long k_stride, v_stride;
  const int* slots;
  void *k_cache, *v_cache;
  unsigned int* status;
  int T, Hkv, d, num_pages, page_shift, fp8;
  float descale_k, descale_v;
};

struct PagedArgs {
  const void* q;  // bf16 [T][Hq][d], q_stride elements between tokens
  long long q_stride;
  const void *k_cache, *v_cache;
  const int *block_table, *query_start, *seq_lens;
  void* o;
  float* lse;
  unsigned int* status;
  int T, R, Hq, Hkv, d, num_pages, page_shift, max_pages, causal, fp8;
  float scale_log2;  // scale * log2(e), times the key factor
  float o_scale;     // the value factor
};

cudaError_t launch_plan(const PlanArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_store(const StoreArgs& a, cudaStream_t stream);
cudaError_t launch_paged(const PagedArgs& a, int num_sms, cudaStream_t stream);

}  // namespace fa
