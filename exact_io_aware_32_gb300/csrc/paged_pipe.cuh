// Parts that the two paged attention kernels share: a key block's copies out of
// its pages, E4M3 codes to bf16 operands, and the values past a request's end.
#pragma once
#include <cstdint>

#include "paged.h"
#include "paged_work.cuh"
#include "ptx.cuh"

namespace fa {
namespace paged {

using namespace fa::ptx;

constexpr float kLn2 = 0.693147180559945309417f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units: how far the exponent reference may lag the row maximum

// Pages of key block jj of a piece that hold keys (one copy each, by lane l).
__device__ __forceinline__ int block_pages(const PagedArgs& a, const Request& q, int jj) {
  const int rows = min(128, q.len - jj * 128), per = min(1 << a.page_shift, 128);
  return (rows + per - 1) / per;
}
// The page that lane 'lane' copies for key block jj (its block_table entry), or -1 past the block's pages.
__device__ __forceinline__ int lane_page(const PagedArgs& a, const Piece& p, int jj, int lane) {
  if (lane >= block_pages(a, p.q, jj)) return -1;
  return __ldg(a.block_table + (long long)p.r * a.max_pages + ((jj * 128) >> a.page_shift) + lane);
}

// A 16-bit key or value tile in shared memory: groups of 8 rows, in each its
// 64-column panels (8 rows x 128 bytes, 128-byte swizzle) one after another.
template <int D>
struct Tile {
  static constexpr int kPanels = D / 64, kGroup = 1024 * kPanels, kBytes = 16 * kGroup;
  // Byte offset of 16-byte chunk c of row r, as the swizzle places it.
  static __device__ __forceinline__ uint32_t chunk(int r, int c) {
    return (uint32_t)((r >> 3) * kGroup + (c >> 3) * 1024 + (r & 7) * 128 + (((c & 7) ^ (r & 7)) << 4));
  }
  // Matrix descriptors: keys K-major (k-steps of 16 columns), values MN-major (k-steps of 16 rows).
  static __device__ __forceinline__ uint64_t desc_k(const uint8_t* p) { return sdesc_sw128(smem_u32(p), 16, kGroup); }
  static __device__ __forceinline__ uint64_t desc_v(const uint8_t* p) { return sdesc_sw128(smem_u32(p), 1024, kGroup); }
  static __host__ __device__ constexpr uint32_t step_k(int kk) { return (uint32_t)((kk >> 2) * 1024 + (kk & 3) * 32) >> 4; }
  static __host__ __device__ constexpr uint32_t step_v(int kk) { return (uint32_t)(kk * 2 * kGroup) >> 4; }
};

// Copies key block jj of one cache into a 128-row tile: a page per lane, all on
// one barrier. One copy per page, not one per panel: with pages of 16 tokens
// the number of copies sets the pace (decoding, 64 requests, d = 128: 184 us
// with a copy per panel, against 163 us with pages of 32). A page outside the
// cache reads as zeros: its copy lies past the tensor map's end.
template <int D, bool FP8>
__device__ __forceinline__ void load_block(const PagedArgs& a, const Piece& p, int jj, int page, int lane,
                                           const CUtensorMap* tm, uint8_t* dst, uint64_t* bar) {
  const int n = block_pages(a, p.q, jj), per = min(1 << a.page_shift, 128);
  if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(n * per * D * (FP8 ? 1 : 2)));
  __syncwarp();
  if (lane < n) {
    const bool ok = page >= 0 && page < a.num_pages;
    const int z = ok ? page * a.Hkv + p.h : a.num_pages * a.Hkv;
    const int y = (jj * 128) & ((1 << a.page_shift) - 1) & ~127;  // a 256-token page's second half
    if constexpr (FP8)
      tma_load_3d(dst + lane * per * D, tm, bar, 0, y, z);
    else
      tma_load_5d(dst + lane * per * D * 2, tm, bar, 0, 0, 0, y >> 3, z);
    if (!ok) atomicOr(a.status, kStatusBadLength);
  }
  __syncwarp();
}

// Zeros the rows of a bf16 value tile from 'row' on (past the request's last
// key): whatever the cache or an earlier block left there, even NaN, must meet
// its zero weights as a number. By one warp, before its products are issued.
template <int D>
__device__ __forceinline__ void zero_rows_from(uint8_t* tile, int row, int lane) {
  const uint32_t base = smem_u32(tile);
  for (int i = row * (D / 8) + lane; i < 128 * (D / 8); i += 32)
    st_shared_v4(base + Tile<D>::chunk(i / (D / 8), i % (D / 8)), 0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  __syncwarp();
}

// ---------------------------------------------------------------- E4M3 caches
// Both products take f16 operands there: every code is an f16 value, so one
// conversion instruction makes two operands. (bf16 has no such instruction: by
// integer steps on the bits, the converters took 3.5 us a block of the
// decoding kernel, 595 us for 48 requests of up to 16384 keys, d = 128.) Q goes
// from bf16 to f16 with each row scaled by the power of two that brings its
// largest magnitude into [1, 2), undone in the row's softmax scale; what that
// loses are elements below 2^-24 of the row's largest. P keeps 11 bits instead
// of 8, times 2^kPBias so that weights down to 2^-32 do not vanish (P stays
// below 2^(kRescaleThreshold + kPBias) = 2^15).
constexpr float kPBias = 7.0f;

// Two codes (the low 16 bits) to f16, exactly, NaN among them.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t c) {
  uint32_t r;
  asm("{\n .reg .b16 x, y;\n mov.b32 {x, y}, %1;\n cvt.rn.f16x2.e4m3x2 %0, x;\n}\n" : "=r"(r) : "r"(c));
  return r;
}

// A 128 x D tile of codes (rows of D bytes) to an f16 tile, by the 128 threads
// of the converters; rows from 'rows' on become zero. A thread takes 16 codes,
// two chunks; threads of odd panels store theirs in the other order, so that
// the eight threads of a quarter warp write to different banks.
template <int D>
__device__ __forceinline__ void convert_tile(const uint8_t* src, uint8_t* dst, int rows, int tid) {
  constexpr int kPairs = D / 16;
  const uint32_t base = smem_u32(dst);
  const int c = tid % kPairs, r0 = tid / kPairs;
  const bool odd = (c >> 2) & 1;
  const uint32_t first = base + Tile<D>::chunk(r0, 2 * c + (odd ? 1 : 0));
  const uint32_t second = base + Tile<D>::chunk(r0, 2 * c + (odd ? 0 : 1));
#pragma unroll
  for (int it = 0; it < kPairs; ++it) {  // row r0 + it * 128 / kPairs: a multiple of 8 rows on, the same swizzle
    const uint4 w = *reinterpret_cast<const uint4*>(src + (it * 128 + tid) * 16);
    uint32_t x[4] = {odd ? w.z : w.x, odd ? w.w : w.y, odd ? w.x : w.z, odd ? w.y : w.w};
    if (rows < 128 && r0 + it * (128 / kPairs) >= rows) x[0] = x[1] = x[2] = x[3] = 0u;  // code 0 is zero
    constexpr uint32_t kStep = 16 / kPairs * Tile<D>::kGroup;
    st_shared_v4(first + it * kStep, e4m3x2_to_f16(x[0]), e4m3x2_to_f16(x[0] >> 16), e4m3x2_to_f16(x[1]),
                 e4m3x2_to_f16(x[1] >> 16));
    st_shared_v4(second + it * kStep, e4m3x2_to_f16(x[2]), e4m3x2_to_f16(x[2] >> 16), e4m3x2_to_f16(x[3]),
                 e4m3x2_to_f16(x[3] >> 16));
  }
}

// Q rows in a [panel][128 rows][128 bytes] swizzled tile from bf16 to scaled f16
// in place, by the converters' 128 threads, four per row: rows [0, 32 * groups),
// and with COPIES rows 0 - 31 also to the other three row quarters. ex[row] gets
// the biased exponent of the power of two that the softmax has to put back.
template <int D, bool COPIES>
__device__ __forceinline__ void convert_q(uint8_t* q, uint8_t* ex, int groups, int tid) {
  constexpr int kChunks = D / 8 / 4;  // 16-byte chunks per thread
  for (int g = 0; g < groups; ++g) {
    const int row = g * 32 + (tid >> 2), part = tid & 3;
    uint4 x[kChunks];
    uint32_t at[kChunks], big = 0;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = part * kChunks + i;
      at[i] = (uint32_t)((c >> 3) * 16384 + row * 128 + (((c & 7) ^ (row & 7)) << 4));
      x[i] = *reinterpret_cast<const uint4*>(q + at[i]);
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) big = max(big, max(w[k] & 0x7FFFu, (w[k] >> 16) & 0x7FFFu));
    }
    big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
    big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
    const uint32_t e = min(max(big >> 7, 1u), 253u);  // exponent of the row's largest magnitude
    const float f = __uint_as_float((254u - e) << 23);
    if (part == 0) ex[row] = (uint8_t)e;
    const uint32_t base = smem_u32(q);
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        o[k] = pack_f16x2(__uint_as_float(w[k] << 16) * f, __uint_as_float(w[k] & 0xffff0000u) * f);
#pragma unroll
      for (int n = 0; n < (COPIES ? 4 : 1); ++n) st_shared_v4(base + at[i] + n * 4096, o[0], o[1], o[2], o[3]);
    }
  }
}

// The converters' hand-over of shared memory that they wrote to the products:
// one arrival per warp (barriers count kConvArrivals).
constexpr uint32_t kConvArrivals = 4;
__device__ __forceinline__ void conv_arrive(uint64_t* full, uint64_t* empty, int lane) {
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    mbar_arrive(full);
    if (empty) mbar_arrive(empty);
  }
}

// 32 bytes to global memory in one instruction (a whole sector per lane).
__device__ __forceinline__ void st_global_v8(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// The same to an address that may be only 16-byte aligned.
__device__ __forceinline__ void st_global_32(void* p, const uint32_t (&v)[8], bool aligned32) {
  if (aligned32) {
    st_global_v8(p, v);
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// The part descriptor of this CTA, kept up by one thread as it walks the pieces.
__device__ __forceinline__ void note_piece(Parts& s, const Piece& p) {
  if (p.jb > 0) {
    s.lead = 1;
    s.lead_ends = p.je == p.nb;
  } else if (p.je < p.nb) {
    s.open = 1;
    s.start = p.q.start;
    s.n = p.q.n;
    s.tok = p.tok;
    s.h = p.h;
  }
}

}  // namespace paged
}  // namespace fa
