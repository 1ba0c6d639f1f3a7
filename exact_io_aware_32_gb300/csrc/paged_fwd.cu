// Host side of the paged attention (which kernel, how many CTAs, tensor maps) and
// the kernel that joins tiles cut between CTAs.
#include <algorithm>
#include <cstdint>

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
// that ends the tile: a fixed order, so the same bits every time. W warps per
// row, each taking every W-th part with kAhead parts' loads in flight: a tile of
// one long request can have a part on every SM.
constexpr int kJoinWarps = 16;
template <int D, int W>
__global__ void __launch_bounds__(32 * kJoinWarps) fa_paged_join_kernel(const __grid_constant__ PagedArgs a,
                                                                        int rows_per_tile) {
  constexpr int V = D / 32, kAhead = 4;
  __shared__ float s_acc[kJoinWarps][D];
  __shared__ float s_tot[kJoinWarps];
  const Parts* parts = static_cast<const Parts*>(a.parts);
  const int c = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % W;
  const Parts mine = parts[c];
  if (!mine.open) return;
  const int G = a.Hq / a.Hkv, row = (int)blockIdx.y * (kJoinWarps / W) + warp / W;
  // row = half * 128 + token * G + head (halves of tpt1 tokens)
  const int half = row >> 7, rr = row & 127, tk = rr / G;
  const int tok = mine.tok + half * a.tpt1 + tk;
  const bool valid = tk < a.tpt1 && tok < mine.n;
  if (__syncthreads_or(valid) == 0) return;
  // the CTA that ends the tile: the first after c whose leading piece says so
  int end = -1;
  for (int z0 = c + 1; z0 < (int)gridDim.x; z0 += 32) {
    const int z = z0 + lane;
    const bool ends = z < (int)gridDim.x && parts[z].lead && parts[z].lead_ends;
    const unsigned b = __ballot_sync(0xffffffffu, ends);
    if (b) {
      end = z0 + __ffs((int)b) - 1;
      break;
    }
  }
  auto slot = [&](int z) { return ((long long)z * 2 + (z == c ? 1 : 0)) * rows_per_tile + row; };
  float m = -INFINITY;
  if (valid)
    for (int z = c + lane; z <= end; z += 32) m = fmaxf(m, a.part_lse[slot(z)]);
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
  float acc[V], tot = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  if (m != -INFINITY)
    for (int z0 = c + sub; z0 <= end; z0 += kAhead * W) {
      float w[kAhead], x[kAhead][V];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int z = z0 + u * W;
        const float lz = z <= end ? a.part_lse[slot(z)] : -INFINITY;
        w[u] = exp2f(lz - m);
#pragma unroll
        for (int i = 0; i < V; ++i) x[u][i] = 0.f;
        if (lz != -INFINITY) {  // else that part saw no key of this row and wrote no O
          const float* oz = a.part_o + slot(z) * D + lane * V;
#pragma unroll
          for (int i = 0; i < V; ++i) x[u][i] = oz[i];
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        tot += w[u];
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] += w[u] * x[u][i];
      }
    }
  if constexpr (W > 1) {
#pragma unroll
    for (int i = 0; i < V; ++i) s_acc[warp][lane * V + i] = acc[i];
    if (lane == 0) s_tot[warp] = tot;
    __syncthreads();
    if (sub != 0) return;
#pragma unroll
    for (int w = 1; w < W; ++w) {
      tot += s_tot[warp + w];
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += s_acc[warp + w][lane * V + i];
    }
  }
  if (!valid) return;
  const float inv = tot > 0.f ? 1.f / tot : 0.f;
  const long long out = (long long)(mine.start + tok) * a.Hq + mine.h * G + (rr - tk * G);
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.o) + (out * D + lane * V) * 2);
#pragma unroll
  for (int i = 0; i < V / 2; ++i) dst[i] = ptx::pack_bf16x2(acc[2 * i] * inv, acc[2 * i + 1] * inv);
  if (lane == 0) a.lse[out] = tot > 0.f ? (m + log2f(tot)) * 0.693147180559945309417f : -INFINITY;
}

template <int D>
void launch_join(const PagedArgs& a, const PagedPlan& p, cudaStream_t stream) {
  // four warps per row where tiles have few rows and many parts, else one
  const int w = p.few ? 4 : 1;
  const dim3 grid((unsigned)p.ctas, (unsigned)(p.rows * w / kJoinWarps));
  auto kern = p.few ? fa_paged_join_kernel<D, 4> : fa_paged_join_kernel<D, 1>;
  kern<<<grid, 32 * kJoinWarps, 0, stream>>>(a, p.rows);
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
  if (a.d == 64)
    launch_join<64>(a, p, stream);
  else
    launch_join<128>(a, p, stream);
  return cudaGetLastError();
}

}  // namespace fa
