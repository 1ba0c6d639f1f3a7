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
// that ends the tile: a fixed order, so the same bits every time. One warp per
// row, grid.y over the tile's rows.
template <int D>
__global__ void __launch_bounds__(128) fa_paged_join_kernel(const __grid_constant__ PagedArgs a, int rows_per_tile) {
  constexpr int V = D / 32;
  const Parts* parts = static_cast<const Parts*>(a.parts);
  const int c = blockIdx.x, lane = threadIdx.x & 31;
  const Parts mine = parts[c];
  if (!mine.open) return;
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
  if (end < 0) return;
  const int G = a.Hq / a.Hkv;
  const int row = (int)blockIdx.y * 4 + (threadIdx.x >> 5);
  // row = half * 128 + token * G + head (halves of tpt1 tokens)
  const int half = row >> 7, rr = row & 127, tk = rr / G;
  const int tok = mine.tok + half * a.tpt1 + tk;
  if (tk >= a.tpt1 || tok >= mine.n) return;
  auto slot = [&](int z) { return ((long long)z * 2 + (z == c ? 1 : 0)) * rows_per_tile + row; };
  float m = -INFINITY;
  for (int z = c + lane; z <= end; z += 32) m = fmaxf(m, a.part_lse[slot(z)]);
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
  float acc[V], tot = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  if (m != -INFINITY)
#pragma unroll 4
    for (int z = c; z <= end; ++z) {
      const float lz = a.part_lse[slot(z)];
      const float w = exp2f(lz - m);
      tot += w;
      if (lz == -INFINITY) continue;  // that part saw no key of this row and wrote no O
      const float* oz = a.part_o + slot(z) * D + lane * V;
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += w * oz[i];
    }
  const float inv = tot > 0.f ? 1.f / tot : 0.f;
  const long long out = (long long)(mine.start + tok) * a.Hq + mine.h * G + (rr - tk * G);
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.o) + (out * D + lane * V) * 2);
#pragma unroll
  for (int i = 0; i < V / 2; ++i) dst[i] = ptx::pack_bf16x2(acc[2 * i] * inv, acc[2 * i + 1] * inv);
  if (lane == 0) a.lse[out] = tot > 0.f ? (m + log2f(tot)) * 0.693147180559945309417f : -INFINITY;
}

}  // namespace

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
  const unsigned long long d = a.d, elem = a.fp8 ? 1 : 2, ps = 1ull << a.page_shift;
  const unsigned per = (unsigned)std::min(ps, 128ull);
  const CUtensorMapDataType type = a.fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const unsigned long long kv_dims[3] = {d, ps, (unsigned long long)a.num_pages * a.Hkv};
  const unsigned long long kv_strides[2] = {d * elem, ps * d * elem};
  const unsigned kv_box[3] = {a.fp8 ? (unsigned)d : 64u, per, 1u};
  const unsigned long long q_dims[3] = {d, (unsigned long long)a.Hq, (unsigned long long)a.T};
  const unsigned long long q_strides[2] = {d * 2, (unsigned long long)a.q_stride * 2};
  const unsigned q_box[3] = {64u, (unsigned)(a.Hq / a.Hkv), (unsigned)p.tpt1};
  if (!encode_map3(&a.tm_q, a.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, q_dims, q_strides, q_box, true) ||
      !encode_map3(&a.tm_k, a.k_cache, type, kv_dims, kv_strides, kv_box, !a.fp8) ||
      !encode_map3(&a.tm_v, a.v_cache, type, kv_dims, kv_strides, kv_box, !a.fp8))
    return cudaErrorInvalidValue;
  a.tpt = p.tpt;
  a.tpt1 = p.tpt1;
  cudaError_t e = p.few ? launch_paged_few(a, p.ctas, stream) : launch_paged_chunk(a, p.ctas, stream);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)p.ctas, (unsigned)(p.rows / 4));
  if (a.d == 64)
    fa_paged_join_kernel<64><<<grid, 128, 0, stream>>>(a, p.rows);
  else
    fa_paged_join_kernel<128><<<grid, 128, 0, stream>>>(a, p.rows);
  return cudaGetLastError();
}

}  // namespace fa
