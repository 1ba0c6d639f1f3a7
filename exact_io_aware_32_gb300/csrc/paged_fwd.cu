// Host side of the paged attention (which kernel, how many CTAs, tensor maps) and
// the kernel that joins tiles cut between CTAs.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "fa_internal.h"
#include "paged.h"
#include "paged_work.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

using paged::Parts;

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Joins the parts of one cut tile: with m = max_z lse_z, o = sum_z 2^(lse_z - m) o_z
// / sum_z 2^(lse_z - m). The CTA that opened the tile names it; the parts after
// its own are the leading pieces of the CTAs that follow, in order, up to the one
// that ends the tile: a fixed order, so the same bits every time. A block of
// kJoinWarps warps takes kJoinWarps / W rows of a tile, W warps per row, each
// every W-th part with kAhead parts' loads in flight. A part's O is read beside
// its logsumexp, not after it: bound by latency, not by the few bytes.
constexpr int kJoinWarps = 8;
template <int D, int W>
__global__ void __launch_bounds__(32 * kJoinWarps) fa_paged_join_kernel(const __grid_constant__ PagedArgs a,
                                                                        int rows_per_tile) {
  constexpr int V = D / 32, kAhead = W > 1 ? 8 : 4;
  using Vec = typename std::conditional<V == 4, float4, float2>::type;
  __shared__ float s_acc[W > 1 ? kJoinWarps : 1][D];
  __shared__ float2 s_ml[W > 1 ? kJoinWarps : 1];
  const int c = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % W;
  ptx::grid_wait();
  const Parts mine = static_cast<const Parts*>(a.parts)[c];
  if (!mine.open) return;
  const int G = a.Hq / a.Hkv, rows1 = a.tpt1 * G;
  const int i = (int)blockIdx.y * (kJoinWarps / W) + warp / W;  // half * rows1 + token * G + head
  const int half = i / rows1, rr = i - half * rows1, tk = rr / G, row = half * 128 + rr;
  const int tok = mine.tok + half * a.tpt1 + tk;
  const bool valid = half * a.tpt1 < a.tpt && tok < mine.n;
  float m = -INFINITY, tot = 0.f, acc[V];
#pragma unroll
  for (int k = 0; k < V; ++k) acc[k] = 0.f;
  if (valid)
    for (int z0 = c + sub; z0 <= mine.end; z0 += kAhead * W) {
      float l[kAhead];
      Vec x[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int z = z0 + u * W;
        const long long slot = ((long long)z * 2 + (z == c ? 1 : 0)) * rows_per_tile + row;
        l[u] = z <= mine.end ? a.part_lse[slot] : -INFINITY;
        x[u] = z <= mine.end ? reinterpret_cast<const Vec*>(a.part_o + slot * D)[lane] : Vec{};
      }
      float m_new = m;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) m_new = fmaxf(m_new, l[u]);
      if (m_new == -INFINITY) continue;
      const float back = exp2f(m - m_new);
      tot *= back;
#pragma unroll
      for (int k = 0; k < V; ++k) acc[k] *= back;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const float w = exp2f(l[u] - m_new);
        tot += w;
        const float* xs = reinterpret_cast<const float*>(&x[u]);
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] += w > 0.f ? w * xs[k] : 0.f;  // (a part without keys wrote no O)
      }
      m = m_new;
    }
  if constexpr (W > 1) {
#pragma unroll
    for (int k = 0; k < V; ++k) s_acc[warp][lane * V + k] = acc[k];
    if (lane == 0) s_ml[warp] = make_float2(m, tot);
    __syncthreads();
    if (sub != 0) return;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < W; ++w) top = fmaxf(top, s_ml[warp + w].x);
    tot = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float2 s = s_ml[warp + w];
      const float f = s.y > 0.f ? exp2f(s.x - top) : 0.f;
      tot += f * s.y;
#pragma unroll
      for (int k = 0; k < V; ++k) acc[k] += f * s_acc[warp + w][lane * V + k];
    }
    m = top;
  }
  if (!valid) return;
  const float inv = tot > 0.f ? 1.f / tot : 0.f;
  const long long out = (long long)(mine.start + tok) * a.Hq + mine.h * G + (rr - tk * G);
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.o) + (out * D + lane * V) * 2);
#pragma unroll
  for (int k = 0; k < V / 2; ++k) dst[k] = ptx::pack_bf16x2(acc[2 * k] * inv, acc[2 * k + 1] * inv);
  if (lane == 0) a.lse[out] = tot > 0.f ? (m + log2f(tot)) * 0.693147180559945309417f : -INFINITY;
}

template <int D>
cudaError_t launch_join(const PagedArgs& a, const PagedPlan& p, cudaStream_t stream) {
  // a block per row where tiles have few rows and maybe a part on every SM, else a warp per row
  const int rows = p.tpt * (a.Hq / a.Hkv), w = p.few ? kJoinWarps : 1;
  const dim3 grid((unsigned)p.ctas, (unsigned)((rows * w + kJoinWarps - 1) / kJoinWarps));
  auto kern = p.few ? fa_paged_join_kernel<D, kJoinWarps> : fa_paged_join_kernel<D, 1>;
  return launch_dependent(kern, grid, 32 * kJoinWarps, 0, stream, a, p.rows);
}

}  // namespace

cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (done.load(std::memory_order_acquire) >> dev & 1u) return cudaSuccess;  // (device_facts has checked dev < 64)
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(1ull << dev, std::memory_order_release);
  return e;
}

PagedPlan plan_paged(int Hq, int Hkv, int d, int fp8, int max_new, int num_sms) {
  const int G = Hq / Hkv;
  PagedPlan p;
  // at most 32 rows a tile: the decoding kernel
  p.few = (long long)G * max_new <= 32;
  const int halves = p.few || (d == 64 && !fp8) ? 1 : 2;
  p.rows = p.few ? 32 : 128 * halves;
  p.tpt1 = std::min(max_new, (p.few ? 32 : 128) / G);
  p.tpt = halves * p.tpt1;
  p.ctas = num_sms * (!p.few && halves == 1 ? 2 : 1);
  p.parts_bytes = align256(sizeof(Parts) * p.ctas);
  p.o_bytes = align256((size_t)p.ctas * 2 * p.rows * d * sizeof(float));
  p.lse_bytes = align256((size_t)p.ctas * 2 * p.rows * sizeof(float));
  return p;
}

cudaError_t launch_paged(PagedArgs a, const PagedPlan& p, cudaStream_t stream) {
  const unsigned long long d = a.d, ps = 1ull << a.page_shift;
  const unsigned per = (unsigned)std::min(ps, 128ull);
  const unsigned long long heads = (unsigned long long)a.num_pages * a.Hkv;
  bool ok = true;
  for (int i = 0; i < 2; ++i) {
    CUtensorMap* m = i ? &a.tm_v : &a.tm_k;
    const void* base = i ? a.v_cache : a.k_cache;
    if (a.fp8) {
      const unsigned long long dims[3] = {d, ps, heads}, strides[2] = {d, ps * d};
      const unsigned box[3] = {(unsigned)d, per, 1u};
      ok = ok && encode_map(m, base, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, dims, strides, box, i ? 0 : a.d);
    } else {
      const unsigned long long dims[5] = {64, 8, d / 64, ps / 8, heads}, strides[4] = {d * 2, 128, d * 16, ps * d * 2};
      const unsigned box[5] = {64u, 8u, (unsigned)d / 64u, per / 8u, 1u};
      ok = ok && encode_map(m, base, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, dims, strides, box, 128);
    }
  }
  const unsigned long long q_dims[3] = {d, (unsigned long long)a.Hq, (unsigned long long)a.T};
  const unsigned long long q_strides[2] = {d * 2, (unsigned long long)a.q_stride * 2};
  const unsigned q_box[3] = {64u, (unsigned)(a.Hq / a.Hkv), (unsigned)p.tpt1};
  ok = ok && encode_map(&a.tm_q, a.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, q_dims, q_strides, q_box, 128);
  if (!ok) return cudaErrorInvalidValue;
  a.tpt = p.tpt;
  a.tpt1 = p.tpt1;
  cudaError_t e = p.few ? launch_paged_few(a, p.ctas, stream) : launch_paged_chunk(a, p.ctas, stream);
  if (e != cudaSuccess) return e;
  return a.d == 64 ? launch_join<64>(a, p, stream) : launch_join<128>(a, p, stream);
}

}  // namespace fa
