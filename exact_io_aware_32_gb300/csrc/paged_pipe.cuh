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

// Copies key block jj of one cache into a 128-row tile: a page per lane (two
// 64-column panels at bf16 d = 128), all on one barrier. A page outside the
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
    if constexpr (FP8) {
      tma_load_3d(dst + lane * per * D, tm, bar, 0, y, z);
    } else {
#pragma unroll
      for (int pn = 0; pn < D / 64; ++pn) tma_load_3d(dst + pn * 16384 + lane * per * 128, tm, bar, pn * 64, y, z);
    }
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
  for (int i = row * 8 + lane; i < 128 * 8; i += 32)
#pragma unroll
    for (int pn = 0; pn < D / 64; ++pn) st_shared_v4(base + pn * 16384 + i * 16, 0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  __syncwarp();
}

// Four E4M3 codes to two pairs of bf16 (exact). A code's exponent and mantissa
// bits moved to the top of bf16's mantissa and the bottom of its exponent are
// the value times 2^-120 (bias 7 against 127), subnormal codes among them, as
// bf16 has subnormals too; one exact product restores the scale. NaN (all
// seven bits set) would come out as 480.
__device__ __forceinline__ void e4m3x4_to_bf16(uint32_t c, uint32_t& lo, uint32_t& hi) {
  const uint32_t x0 = __byte_perm(c, 0u, 0x1404), x1 = __byte_perm(c, 0u, 0x3424);  // bytes in the high halves
  const uint32_t y0 = (x0 & 0x80008000u) | ((x0 & 0x7F007F00u) >> 4);
  const uint32_t y1 = (x1 & 0x80008000u) | ((x1 & 0x7F007F00u) >> 4);
  constexpr uint32_t k2p120 = 0x7B807B80u;  // 2^120 twice
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(y0), "r"(k2p120));
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(y1), "r"(k2p120));
  if ((((c & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0u) {
    if ((c & 0x7Fu) == 0x7Fu) lo |= 0x00007FFFu;
    if ((c & 0x7F00u) == 0x7F00u) lo |= 0x7FFF0000u;
    if ((c & 0x7F0000u) == 0x7F0000u) hi |= 0x00007FFFu;
    if ((c & 0x7F000000u) == 0x7F000000u) hi |= 0x7FFF0000u;
  }
}

// A 128 x D tile of codes (rows of D bytes) to the swizzled bf16 panels that
// the products read, by 128 threads; rows from 'rows' on become zero. Eight
// neighbouring threads write the eight 16-byte chunks of one 128-byte row, so
// a quarter warp's stores touch every bank once.
template <int D>
__device__ __forceinline__ void convert_tile(const uint8_t* src, uint8_t* dst, int rows, int tid) {
  constexpr int kChunks = D / 8;
  const uint32_t base = smem_u32(dst);
#pragma unroll 4
  for (int i = tid; i < 128 * kChunks; i += 128) {
    const int row = i / kChunks, c = i % kChunks;
    const uint2 w = *reinterpret_cast<const uint2*>(src + i * 8);
    uint32_t o[4];
    e4m3x4_to_bf16(w.x, o[0], o[1]);
    e4m3x4_to_bf16(w.y, o[2], o[3]);
    if (row >= rows) o[0] = o[1] = o[2] = o[3] = 0u;
    st_shared_v4(base + (c >> 3) * 16384 + row * 128 + (((c & 7) ^ (row & 7)) << 4), o[0], o[1], o[2], o[3]);
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
