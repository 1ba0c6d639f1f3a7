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

// Joining the parts of a cut tile: with m = max_z lse_z, o = sum_z 2^(lse_z - m) o_z
// / sum_z 2^(lse_z - m). The CTA that opened the tile names it; the parts after
// its own are the leading pieces of the CTAs that follow, in order, up to the one
// that ends the tile: a fixed order, so the same bits every time. A part's O is
// read beside its logsumexp, not after it (one that saw no key of the row wrote
// none: weight 0, its O not looked at).
constexpr int kJoinWarps = 8;

template <int V>
struct Joined {  // of one row, V columns per lane
  float m, tot, acc[V];
  __device__ __forceinline__ void clear() {
    m = -INFINITY;
    tot = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.f;
  }
  __device__ __forceinline__ void add(float l, const float* x) {  // a part: its logsumexp and O / l
    if (l == -INFINITY) return;
    const float m_new = fmaxf(m, l), back = exp2f(m - m_new), w = exp2f(l - m_new);
    tot = tot * back + w;
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = acc[k] * back + w * x[k];
    m = m_new;
  }
};

template <int D>
__device__ __forceinline__ void write_row(const PagedArgs& a, long long out, const Joined<D / 32>& s, int lane) {
  constexpr int V = D / 32;
  const float inv = s.tot == 0.f ? 0.f : 1.f / s.tot;  // (a NaN goes on to the result)
  uint32_t w[V / 2];
#pragma unroll
  for (int k = 0; k < V / 2; ++k) w[k] = ptx::pack_bf16x2(s.acc[2 * k] * inv, s.acc[2 * k + 1] * inv);
  uint8_t* dst = static_cast<uint8_t*>(a.o) + (out * D + lane * V) * 2;
  if constexpr (V == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t*>(dst) = w[0];
  if (lane == 0) a.lse[out] = s.tot != 0.f ? (s.m + log2f(s.tot)) * 0.693147180559945309417f : -INFINITY;
}

// Few rows (decoding): one long request's tile can have a part on every SM, so a
// block takes one row, each warp every kJoinWarps-th part, eight in flight.
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) fa_paged_join_few_kernel(const __grid_constant__ PagedArgs a) {
  constexpr int V = D / 32, kAhead = 8;
  using Vec = typename std::conditional<V == 4, float4, float2>::type;
  __shared__ float s_acc[kJoinWarps][D];
  __shared__ float2 s_ml[kJoinWarps];
  const int c = blockIdx.x, row = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  ptx::grid_wait();
  const Parts mine = static_cast<const Parts*>(a.parts)[c];
  if (!mine.open) return;
  const int G = a.Hq / a.Hkv, tk = row / G, tok = mine.tok + tk;
  if (tok >= mine.n) return;
  Joined<V> s;
  s.clear();
  for (int z0 = c + warp; z0 <= mine.end; z0 += kAhead * kJoinWarps) {
    float l[kAhead];
    Vec x[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int z = z0 + u * kJoinWarps;
      const long long slot = ((long long)z * 2 + (z == c ? 1 : 0)) * 32 + row;
      l[u] = z <= mine.end ? a.part_lse[slot] : -INFINITY;
      x[u] = z <= mine.end ? reinterpret_cast<const Vec*>(a.part_o + slot * D)[lane] : Vec{};
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) s.add(l[u], reinterpret_cast<const float*>(&x[u]));
  }
#pragma unroll
  for (int k = 0; k < V; ++k) s_acc[warp][lane * V + k] = s.acc[k];
  if (lane == 0) s_ml[warp] = make_float2(s.m, s.tot);
  __syncthreads();
  if (warp != 0) return;
  float top = -INFINITY;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, s_ml[w].x);
  s.clear();
  s.m = top;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    const float2 ml = s_ml[w];
    const float f = ml.y != 0.f ? exp2f(ml.x - top) : 0.f;
    s.tot += f * ml.y;
#pragma unroll
    for (int k = 0; k < V; ++k) s.acc[k] += f * s_acc[w][lane * V + k];
  }
  write_row<D>(a, (long long)(mine.start + tok) * a.Hq + mine.h * G + (row - tk * G), s, lane);
}

// Tiles of 128 or 256 rows, mostly of two parts: a warp per two rows. (Three chunks
// of 1024 tokens, 32 heads of 128, whole call: a warp per row 243 us, per two rows
// 236 us, per four 238 us, four with three parts in flight 240 us.)
constexpr int kJoinRows = 2;
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) fa_paged_join_chunk_kernel(const __grid_constant__ PagedArgs a,
                                                                              int rows_per_tile) {
  constexpr int V = D / 32, kRows = kJoinRows, kAhead = 2;
  using Vec = typename std::conditional<V == 4, float4, float2>::type;
  const int c = blockIdx.x, lane = threadIdx.x & 31;
  const int row0 = ((int)blockIdx.y * kJoinWarps + (threadIdx.x >> 5)) * kRows;  // half * 128 + token * G + head
  ptx::grid_wait();
  const Parts mine = static_cast<const Parts*>(a.parts)[c];
  if (!mine.open) return;
  const int G = a.Hq / a.Hkv, half = row0 >> 7, r0 = row0 & 127, tk0 = r0 / G;
  const int tok0 = mine.tok + half * a.tpt1;
  const int rows = min(a.tpt1, mine.n - tok0) * G - r0;  // of this half from r0 on
  if (rows <= 0) return;
  Joined<V> s[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) s[i].clear();
  for (int z0 = c; z0 <= mine.end; z0 += kAhead) {
    float l[kAhead][kRows];
    Vec x[kAhead][kRows];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int z = z0 + u;
      const long long slot = ((long long)z * 2 + (z == c ? 1 : 0)) * rows_per_tile + row0;
      const float* lp = a.part_lse + slot;
      const Vec* xp = reinterpret_cast<const Vec*>(a.part_o + slot * D) + lane;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const bool there = i < rows && z <= mine.end;
        l[u][i] = there ? lp[i] : -INFINITY;
        x[u][i] = there ? xp[i * 32] : Vec{};
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int i = 0; i < kRows; ++i) s[i].add(l[u][i], reinterpret_cast<const float*>(&x[u][i]));
  }
  int tk = tk0, h = r0 - tk0 * G;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (i < rows) write_row<D>(a, (long long)(mine.start + tok0 + tk) * a.Hq + mine.h * G + h, s[i], lane);
    if (++h == G) {
      h = 0;
      ++tk;
    }
  }
}

template <int D>
cudaError_t launch_join(const PagedArgs& a, const PagedPlan& p, cudaStream_t stream) {
  if (p.few)
    return launch_dependent(fa_paged_join_few_kernel<D>, dim3((unsigned)p.ctas, (unsigned)(p.tpt * (a.Hq / a.Hkv))),
                            32 * kJoinWarps, 0, stream, a);
  return launch_dependent(fa_paged_join_chunk_kernel<D>, dim3((unsigned)p.ctas, (unsigned)(p.rows / (kJoinRows * kJoinWarps))),
                          32 * kJoinWarps, 0, stream, a, p.rows);
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

namespace {
// Tables for no more than 8 blocks a request: nothing is cut, and there is no join to launch. Measured with 32 heads over 8
// of 128, cut and whole: 16 requests of up to 300 keys 13.0 and 10.0 us, of up to 1000 15.2 and 12.4 us, 256 of up to 1000
// 87.4 and 84.7 us (E4M3 93.9 and 93.5 us); at 16 blocks 4 requests of up to 1500 keys 12.0 and 13.5 us.
constexpr int kWholeBlocks = 8;

PagedPlan plan_kernel(bool few, int G, int d, int fp8, int max_new, int max_keys, int num_sms) {
  PagedPlan p;
  p.few = few;
  const int halves = few || (d == 64 && !fp8) ? 1 : 2;
  p.rows = few ? 32 : 128 * halves;
  p.tpt1 = std::min(max_new, (few ? 32 : 128) / G);
  p.tpt = halves * p.tpt1;
  // Cutting a tile of the chunk kernel costs two more epilogues and a join: short tiles stay whole and parts have at least
  // four blocks (eight prompts of up to 1024 tokens, 12 heads of 64, when it was chosen: 44 us with every cut, 35 us). The
  // decoding kernel's parts are a few rows: there only a call without any cut is worth it.
  const int blocks = (max_keys >> 7) + (max_keys % 128 != 0);  // of the longest request there can be
  p.whole = few && blocks > kWholeBlocks ? 0 : kWholeBlocks;
  p.join = blocks > p.whole;
  p.snap = few ? 0 : 4;
  p.n_min = 0;
  p.n_max = INT32_MAX;
  p.ctas = num_sms * (!few && halves == 1 ? 2 : 1);
  p.parts_bytes = align256(sizeof(Parts) * p.ctas);
  p.o_bytes = align256((size_t)p.ctas * 2 * p.rows * d * sizeof(float));
  p.lse_bytes = align256((size_t)p.ctas * 2 * p.rows * sizeof(float));
  return p;
}
}  // namespace

int plan_paged(int T, int R, int Hq, int Hkv, int d, int fp8, int max_new, int max_keys, int num_sms,
               PagedPlan (&p)[2]) {
  const int G = Hq / Hkv;
  // no request has more than 32 rows per key head: the decoding kernel alone
  if ((long long)G * max_new <= 32) {
    p[0] = plan_kernel(true, G, d, fp8, max_new, max_keys, num_sms);
    return 1;
  }
  p[0] = plan_kernel(false, G, d, fp8, max_new, max_keys, num_sms);
  // Requests of mostly far fewer tokens than the largest: decoding requests beside chunks of prompts. A tile of 128 rows
  // for a few takes the chunk kernel 3000 cycles per key block and the decoding kernel a third of that, but a second
  // kernel with its join costs 20 us, so each takes its requests only where there may be many keys. Measured with one
  // chunk of 777 tokens beside R requests of one token and up to n keys, d = 128, chunk kernel alone and both:
  //   R = 128, n = 8192, 32 heads over 8   E4M3 452 and 300 us, bf16 451 and 409 us
  //   R = 128, n = 4096, 32 heads over 8        287 and 191 us,      242 and 237 us
  //   R = 64,  n = 8192, 16 heads over 4        158 and 136 us,      144 and 159 us
  //   R = 64,  n = 4096, 16 heads over 4        100 and 101 us,       88 and 106 us
  const long long keys = (long long)R * max_keys * Hkv;
  if (G <= 32 && (long long)T * 2 < (long long)R * max_new && keys >= (fp8 ? 1500000ll : 4000000ll)) {
    const int most = 32 / G;
    p[1] = p[0];
    p[1].n_min = most + 1;
    p[0] = plan_kernel(true, G, d, fp8, most, max_keys, num_sms);
    p[0].n_max = most;
    return 2;
  }
  return 1;
}

cudaError_t launch_paged(PagedArgs a, const PagedPlan& p, void* workspace, cudaStream_t stream) {
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
  a.n_min = p.n_min;
  a.n_max = p.n_max;
  a.whole = p.whole;
  a.snap = p.snap;
  a.tpt = p.tpt;
  a.tpt1 = p.tpt1;
  char* w = static_cast<char*>(workspace);
  a.parts = w;
  a.part_o = reinterpret_cast<float*>(w + p.parts_bytes);
  a.part_lse = reinterpret_cast<float*>(w + p.parts_bytes + p.o_bytes);
  cudaError_t e = p.few ? launch_paged_few(a, p.ctas, stream) : launch_paged_chunk(a, p.ctas, stream);
  if (e != cudaSuccess || !p.join) return e;
  return a.d == 64 ? launch_join<64>(a, p, stream) : launch_join<128>(a, p, stream);
}

}  // namespace fa
