// Attention of new tokens over the paged cache: one warp per (packed row, query
// head), the keys one after another with a running maximum and sum.
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "fa_internal.h"
#include "paged.h"

namespace fa {
namespace {

template <int V, bool FP8>
__device__ __forceinline__ void load_row(const void* cache, long long at, float (&x)[V]) {
  if constexpr (FP8) {
    const __nv_fp8_e4m3* p = static_cast<const __nv_fp8_e4m3*>(cache) + at;
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = (float)p[i];
  } else {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(cache) + at;
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = __bfloat162float(p[i]);
  }
}

template <int D, bool FP8>
__global__ void __launch_bounds__(128) fa_fwd_paged_kernel(const __grid_constant__ PagedArgs a) {
  constexpr int V = D / 32;
  const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int t = (int)(w / a.Hq), h = (int)(w - (long long)t * a.Hq), hk = h / (a.Hq / a.Hkv);
  if (w == 0)  // one warp reports what is out of range in the lengths
    for (int r = lane; r < a.R; r += 32) {
      const int s0 = a.query_start[r], s1 = a.query_start[r + 1];
      if (s0 < 0 || s1 < s0 || s1 > a.T) atomicOr(a.status, kStatusBadLength);
    }
  if (t >= a.T) return;
  int lo = 0, hi = a.R;  // the last request that starts at or before row t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.query_start[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int r = lo, start = max(a.query_start[r], 0), n = min(a.query_start[r + 1], a.T) - start;
  if (t < start || t >= start + n) return;
  const long long cap = (long long)a.max_pages << a.page_shift;
  const int asked = a.seq_lens[r];
  const int len = (int)min((long long)max(asked, 0), cap);
  if (len != asked && lane == 0) atomicOr(a.status, kStatusBadLength);
  const int see = a.causal ? min(len, len - n + (t - start) + 1) : len;
  float q[V], acc[V], m = -INFINITY, l = 0.f;
  load_row<V, false>(a.q, t * a.q_stride + (long long)h * D + lane * V, q);
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  const int mask = (1 << a.page_shift) - 1;
  for (int j = 0; j < see; ++j) {
    const int page = a.block_table[(long long)r * a.max_pages + (j >> a.page_shift)];
    const bool ok = page >= 0 && page < a.num_pages;
    if (!ok && lane == 0) atomicOr(a.status, kStatusBadLength);
    const long long at = ((((long long)(ok ? page : 0) * a.Hkv + hk) << a.page_shift) + (j & mask)) * D + lane * V;
    float k[V], v[V], s = 0.f;
    load_row<V, FP8>(a.k_cache, at, k);
    load_row<V, FP8>(a.v_cache, at, v);
#pragma unroll
    for (int i = 0; i < V; ++i) s += ok ? q[i] * k[i] : 0.f;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= a.scale_log2;
    const float m_new = fmaxf(m, s), alpha = exp2f(m - m_new), p = exp2f(s - m_new);
    m = m_new;
    l = l * alpha + p;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = acc[i] * alpha + (ok ? p * v[i] : 0.f);
  }
  const float inv = l > 0.f ? a.o_scale / l : 0.f;
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.o) + ((long long)t * a.Hq + h) * D + lane * V;
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = __float2bfloat16_rn(acc[i] * inv);
  if (lane == 0) a.lse[(long long)t * a.Hq + h] = l > 0.f ? (m + log2f(l)) * 0.693147180559945309f : -INFINITY;
}

}  // namespace

cudaError_t launch_paged(const PagedArgs& a, int, cudaStream_t stream) {
  const unsigned grid = (unsigned)(((long long)a.T * a.Hq + 3) / 4);
  if (a.d == 64)
    (a.fp8 ? fa_fwd_paged_kernel<64, true> : fa_fwd_paged_kernel<64, false>)<<<grid, 128, 0, stream>>>(a);
  else
    (a.fp8 ? fa_fwd_paged_kernel<128, true> : fa_fwd_paged_kernel<128, false>)<<<grid, 128, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace fa
