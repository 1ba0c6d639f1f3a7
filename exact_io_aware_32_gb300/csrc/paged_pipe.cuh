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

// A request's block table as one warp reads it: 32 entries in the lanes'
// registers and the next 32 on their way, so that no key block waits for a load
// from the table (one block ahead, each took 950 cycles to issue).
struct Pages {
  int base, now, next;  // entries base + lane and base + 32 + lane
  __device__ __forceinline__ int entry(const PagedArgs& a, const Piece& p, int i) const {
    return i <= (p.q.len - 1) >> a.page_shift ? a.block_table[(long long)p.r * a.max_pages + i] : -1;
  }
  __device__ __forceinline__ void begin(const PagedArgs& a, const Piece& p, int lane) {
    base = ((p.jb * 128) >> a.page_shift) & ~31;
    now = entry(a, p, base + lane);
    next = entry(a, p, base + 32 + lane);
  }
  // The page that this lane copies for key block jj (blocks in order; a block's pages lie in one window).
  __device__ __forceinline__ int of(const PagedArgs& a, const Piece& p, int jj, int lane) {
    const int first = (jj * 128) >> a.page_shift;
    if (first - base >= 32) {
      base += 32;
      now = next;
      next = entry(a, p, base + 32 + lane);
    }
    return __shfl_sync(0xffffffffu, now, (first + lane) & 31);
  }
};

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
// cache reads as zeros: its copy lies past the tensor map's end. (A copy may
// complete before lane 0 has said how many bytes are to come: the phase waits
// for that arrival.)
template <int D, bool FP8>
__device__ __forceinline__ void load_block(const PagedArgs& a, const Piece& p, int jj, int page, int lane,
                                           const CUtensorMap* tm, uint8_t* dst, uint64_t* bar) {
  const int shift = min(a.page_shift, 7), rows = min(128, p.q.len - jj * 128);
  const int n = (rows + (1 << shift) - 1) >> shift;  // pages with keys
  if (lane < n) {
    constexpr int kRow = D * (FP8 ? 1 : 2);
    if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)((n << shift) * kRow));
    const bool ok = (unsigned)page < (unsigned)a.num_pages;
    const int z = (ok ? page : a.num_pages) * a.Hkv + (ok ? p.h : 0);
    const int y = (jj * 128) & ((1 << a.page_shift) - 1) & ~127;  // a 256-token page's second half
    if constexpr (FP8)
      tma_load_3d(dst + (lane << shift) * kRow, tm, bar, 0, y, z);
    else
      tma_load_5d(dst + (lane << shift) * kRow, tm, bar, 0, 0, 0, y >> 3, z);
    if (!ok) atomicOr(a.status, kStatusBadLength);
  }
  __syncwarp();
}

// 16-key steps of P V for a block with 'keys' keys left in its request: the rest of a last block is not multiplied.
__device__ __forceinline__ int pv_steps(int keys) { return min(8, (keys + 15) >> 4); }

// O += P V of 'steps' 16-key steps by the elected lane: all eight in straight code, since a condition on each costs the
// issuing warp time that it does not have.
template <int D>
__device__ __forceinline__ void issue_pv_steps(uint32_t d_o, uint32_t a_p, uint64_t dv, uint32_t idesc, int steps,
                                               bool first) {
  if (steps == 8) {
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)  // P columns [8 kk, 8 kk + 8), V rows [16 kk, 16 kk + 16)
      mma_ts(d_o, a_p + kk * 8, dv + Tile<D>::step_v(kk), idesc, (!first || kk > 0) ? 1u : 0u);
  } else {
#pragma unroll 1
    for (int kk = 0; kk < steps; ++kk)
      mma_ts(d_o, a_p + kk * 8, dv + Tile<D>::step_v(kk), idesc, (!first || kk > 0) ? 1u : 0u);
  }
}

// Zeros rows [row, end) of a value tile, those past the request's last key that
// its last step still multiplies: whatever the cache or an earlier block left there, even
// NaN, must meet its zero weights as a number. By one warp, before the products are issued.
template <int D>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int row, int end, int lane) {
  const uint32_t base = smem_u32(tile);
  for (int i = row * (D / 8) + lane; i < end * (D / 8); i += 32)
    st_shared_v4(base + Tile<D>::chunk(i / (D / 8), i % (D / 8)), 0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  __syncwarp();
}

// With bf16 caches P enters O += P V as bf16, since one tcgen05.mma takes both 16-bit operands of one type: half a step
// of each weight, 2^-8 at most, which leaves o a relative RMS error of 0.0020 to 0.0024 where rounding o alone leaves
// 0.0017. The weights' sum is taken before that rounding, in fp32.
// ---------------------------------------------------------------- E4M3 caches
// Keys stay codes: S = Q K^T on 8-bit operands (kind::f8f6f4), with Q as two of
// them, hi + lo. A bf16 value has 8 significant bits; hi takes the upper
// four, lo the lower four, so hi + lo = q exactly unless a part falls below
// E4M3's normal range. Each row of Q is first scaled by the power of two that
// brings its largest magnitude into [128, 256) (undone in the row's softmax
// scale), so what is lost stays below 2^-16 of that magnitude. Two 8-bit products take as long as one 16-bit product.
// Values become f16 operands, one conversion instruction for two of them, by
// warps between the copy and the product; P enters that product as f16: 11 bits, times
// 2^kPBias so that weights down to 2^-32 do not vanish (P stays below
// 2^(kRescaleThreshold + kPBias) = 2^15). In two E4M3 parts P would lose every
// weight below 2^-10.
// Measured, decoding 48 requests of up to 16384 keys at d = 128: both caches to
// bf16 by integer steps on the bits 595 us, both to f16 211 us.
constexpr float kPBias = 7.0f;

// Two codes (the low 16 bits) to f16, exactly, NaN among them.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t c) {
  uint32_t r;
  asm("{\n .reg .b16 x, y;\n mov.b32 {x, y}, %1;\n cvt.rn.f16x2.e4m3x2 %0, x;\n}\n" : "=r"(r) : "r"(c));
  return r;
}

// A 128 x D tile of value codes (rows of D bytes) to an f16 tile, by NT threads;
// of the rows from 'rows' on those that pv_steps still multiplies become zero. A thread takes 8 codes, one 16-byte chunk, at
// a time: sixteen threads read 128 neighbouring bytes and a quarter warp writes
// the eight chunks of one 128-byte row, so neither meets a bank twice.
template <int D, int NT>
__device__ __forceinline__ void convert_tile(const uint8_t* src, uint8_t* dst, int rows, int tid) {
  constexpr int kChunks = D / 8, kRows = NT / kChunks;  // chunks per row, rows per step
  static_assert(kRows % 4 == 0, "two steps must keep the swizzle");
  const int c = tid % kChunks, r0 = tid / kChunks;
  const uint32_t base = smem_u32(dst);
  // where this thread's chunk of the steps' rows lies: the swizzle goes by row % 8
  const uint32_t even = base + Tile<D>::chunk(r0, c), odd = base + Tile<D>::chunk(r0 + kRows, c);
  auto convert = [&](int it) {
    uint2 w = *reinterpret_cast<const uint2*>(src + (it * NT + tid) * 8);
    if (rows < 128 && r0 + it * kRows >= rows) w = make_uint2(0u, 0u);  // code 0 is zero
    const uint32_t at = (it & 1) ? odd + (it >> 1) * (2 * kRows / 8) * Tile<D>::kGroup
                                 : even + (it >> 1) * (2 * kRows / 8) * Tile<D>::kGroup;
    st_shared_v4(at, e4m3x2_to_f16(w.x), e4m3x2_to_f16(w.x >> 16), e4m3x2_to_f16(w.y), e4m3x2_to_f16(w.y >> 16));
  };
  if (rows >= 128) {
#pragma unroll 8
    for (int it = 0; it < 128 / kRows; ++it) convert(it);
  } else {
#pragma unroll 1
    for (int it = 0; it * kRows < pv_steps(rows) * 16; ++it) convert(it);
  }
}

// hi and lo codes of two values (the low half of each result): hi is the value cut to four significant bits, lo the rest.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const float hx = __uint_as_float(__float_as_uint(x) & 0xFFF00000u), hy = __uint_as_float(__float_as_uint(y) & 0xFFF00000u);
  asm("{\n .reg .b16 c, z;\n cvt.rn.satfinite.e4m3x2.f32 c, %2, %1;\n mov.b16 z, 0;\n mov.b32 %0, {c, z};\n}\n"
      : "=r"(hi)
      : "f"(hx), "f"(hy));
  asm("{\n .reg .b16 c, z;\n cvt.rn.satfinite.e4m3x2.f32 c, %2, %1;\n mov.b16 z, 0;\n mov.b32 %0, {c, z};\n}\n"
      : "=r"(lo)
      : "f"(x - hx), "f"(y - hy));
}

// Rows 0 - 31 of Q, a [panel][32 rows][128 bytes] swizzled tile, from 64 bf16 to
// 64 hi and 64 lo codes per 128-byte row, four times (a row quarter each) into a
// [panel][128 rows][128 bytes] one, by 256 threads, eight neighbours per row.
// ex[row] gets the biased exponent e of the row's largest magnitude: the row was
// scaled by 2^(134 - e).
template <int D>
__device__ __forceinline__ void convert_q(const uint8_t* raw, uint8_t* q, uint8_t* ex, int tid) {
  constexpr int kPanels = D / 64;
  const int part = tid & 7, row = tid >> 3;
  auto at = [&](int c) { return (uint32_t)(row * 128 + ((c ^ (row & 7)) << 4)); };
  uint32_t w[kPanels][4], big = 0;  // chunk 'part' of each panel
#pragma unroll
  for (int pn = 0; pn < kPanels; ++pn) {
    const uint4 x = *reinterpret_cast<const uint4*>(raw + pn * 4096 + at(part));
    w[pn][0] = x.x;
    w[pn][1] = x.y;
    w[pn][2] = x.z;
    w[pn][3] = x.w;
#pragma unroll
    for (int k = 0; k < 4; ++k) big = max(big, max(w[pn][k] & 0x7FFFu, (w[pn][k] >> 16) & 0x7FFFu));
  }
#pragma unroll
  for (int s = 1; s < 8; s <<= 1) big = max(big, __shfl_xor_sync(0xffffffffu, big, s));
  const uint32_t e = min(max(big >> 7, 8u), 254u);
  const float f = __uint_as_float((261u - e) << 23);
  if (part == 0) ex[row] = (uint8_t)e;
  uint8_t* dst = q + at(part >> 1) + (part & 1) * 8;  // hi codes; lo codes four chunks on
  const int lo_at = (int)at(4 + (part >> 1)) - (int)at(part >> 1);
#pragma unroll
  for (int pn = 0; pn < kPanels; ++pn) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      split2(__uint_as_float(w[pn][k] << 16) * f, __uint_as_float(w[pn][k] & 0xffff0000u) * f, h[k], l[k]);
    const uint2 hi = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
    const uint2 lo = make_uint2(l[0] | (l[1] << 16), l[2] | (l[3] << 16));
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      *reinterpret_cast<uint2*>(dst + pn * 16384 + n * 4096) = hi;
      *reinterpret_cast<uint2*>(dst + pn * 16384 + n * 4096 + lo_at) = lo;
    }
  }
}
// The same for one row by one thread (neighbouring lanes take neighbouring rows); returns e.
template <int D>
__device__ __forceinline__ uint32_t convert_row(uint8_t* q, int row) {
  constexpr int kPanels = D / 64;
  const uint32_t base = smem_u32(q);
  auto at = [&](int pn, int c) { return (uint32_t)(pn * 16384 + row * 128 + ((c ^ (row & 7)) << 4)); };
  uint32_t w[kPanels][32], big = 0;
#pragma unroll
  for (int pn = 0; pn < kPanels; ++pn)
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const uint4 x = *reinterpret_cast<const uint4*>(q + at(pn, c));
      w[pn][4 * c] = x.x;
      w[pn][4 * c + 1] = x.y;
      w[pn][4 * c + 2] = x.z;
      w[pn][4 * c + 3] = x.w;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        big = max(big, max(w[pn][4 * c + k] & 0x7FFFu, (w[pn][4 * c + k] >> 16) & 0x7FFFu));
    }
  const uint32_t e = min(max(big >> 7, 8u), 254u);
  const float f = __uint_as_float((261u - e) << 23);
#pragma unroll
  for (int pn = 0; pn < kPanels; ++pn)
#pragma unroll
    for (int c = 0; c < 4; ++c) {  // 16 values: a chunk of hi and one of lo
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t x = w[pn][8 * c + 2 * k], y = w[pn][8 * c + 2 * k + 1];
        uint32_t h0, l0, h1, l1;
        split2(__uint_as_float(x << 16) * f, __uint_as_float(x & 0xffff0000u) * f, h0, l0);
        split2(__uint_as_float(y << 16) * f, __uint_as_float(y & 0xffff0000u) * f, h1, l1);
        hi[k] = h0 | (h1 << 16);
        lo[k] = l0 | (l1 << 16);
      }
      st_shared_v4(base + at(pn, c), hi[0], hi[1], hi[2], hi[3]);
      st_shared_v4(base + at(pn, 4 + c), lo[0], lo[1], lo[2], lo[3]);
    }
  return e;
}
// What the softmax multiplies its scale by for a row whose exponent is e.
__device__ __forceinline__ float unscale(uint32_t e) { return __uint_as_float((e - 7u) << 23); }

// S = Q K^T of one 128 x 128 block by the elected lane: Q and K both K-major, at
// bf16 from the panels' 32-byte k-steps; with E4M3 caches hi and lo codes of Q
// (64 bytes each of a panel's rows) against the same key columns.
template <int D, bool FP8>
__device__ __forceinline__ uint64_t desc_keys(const uint8_t* p) {
  if constexpr (!FP8) return Tile<D>::desc_k(p);
  if constexpr (D == 128) return sdesc_sw128(smem_u32(p), 16, 1024);
  return sdesc_sw64(smem_u32(p), 16, 512);
}
template <int D, bool FP8>
__device__ __forceinline__ void issue_qk(uint32_t d_s, uint64_t dq, uint64_t dk) {
  if constexpr (FP8) {
    constexpr uint32_t kId = idesc_e4m3(128, 128, false, false);
#pragma unroll
    for (int pn = 0; pn < D / 64; ++pn)
#pragma unroll
      for (int i = 0; i < 4; ++i)  // hi, hi, lo, lo
        mma_ss_f8(d_s, dq + ((pn * 16384 + i * 32) >> 4), dk + ((pn * 64 + (i & 1) * 32) >> 4), kId,
                  pn > 0 || i > 0);
  } else {
    constexpr uint32_t kId = idesc_bf16(128, 128, false, false);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
      mma_ss(d_s, dq + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4), dk + Tile<D>::step_k(kk), kId, kk > 0);
  }
}

// The converters' hand-over of shared memory that they wrote to the products:
// one arrival per warp.
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

// The pieces of a CTA's range, worked out by its loading warp and told to the
// other warps: a step of the walk takes about 1000 cycles, most of them waiting
// for instructions that run once per tile, and stood in every role's chain.
constexpr int kRing = 4;
struct alignas(16) PieceRing {
  int4 at[kRing][3];
  uint64_t full[kRing], empty[kRing];
  __device__ __forceinline__ void init(int readers) {  // readers: warps
    for (int s = 0; s < kRing; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], readers);
    }
  }
  // The n-th piece (more: not the end), with two numbers of the caller's.
  __device__ __forceinline__ bool tell(int n, const Piece& p, bool more, int x, int y, int lane, volatile int* abort_flag) {
    const int s = n % kRing;
    if (!warp_wait(&empty[s], ((n / kRing) & 1) ^ 1, abort_flag)) return false;
    if (lane == 0) {
      at[s][0] = make_int4(p.q.start, p.q.n, p.q.len, more);
      at[s][1] = make_int4(p.h, p.tok, p.jb, p.je);
      at[s][2] = make_int4(p.nb, p.r, x, y);
      mbar_arrive(&full[s]);
    }
    __syncwarp();
    return true;
  }
};
// A reading warp's place in the ring: for (bool more = in.next(p); more; more = in.next(p)).
struct PieceReader {
  PieceRing& ring;
  volatile int* abort_flag;
  int lane, n = 0, x = 0, y = 0;
  bool ok = true;
  __device__ __forceinline__ PieceReader(PieceRing& ring_, volatile int* flag, int lane_)
      : ring(ring_), abort_flag(flag), lane(lane_) {}
  __device__ __forceinline__ bool next(Piece& p) {  // false: the end, or (ok) the wait ran out
    const int s = n % kRing;
    if (!(ok = warp_wait(&ring.full[s], (n / kRing) & 1, abort_flag))) return false;
    ++n;
    const int4 u = ring.at[s][0], v = ring.at[s][1], w = ring.at[s][2];
    __syncwarp();
    if (lane == 0) mbar_arrive(&ring.empty[s]);
    p.q = {u.x, u.y, u.z};
    p.h = v.x;
    p.tok = v.y;
    p.jb = v.z;
    p.je = v.w;
    p.nb = w.x;
    p.r = w.y;
    x = w.z;
    y = w.w;
    return u.w != 0;
  }
};

// The part descriptor of this CTA, kept up by one thread as it walks the pieces.
__device__ __forceinline__ void note_piece(const PagedArgs& a, Parts& s, const Piece& p, const Walk& walk,
                                           int per) {
  if (p.jb > 0) {
    s.lead = 1;
    s.lead_ends = p.je == p.nb;
  } else if (p.je < p.nb) {
    s.open = 1;
    s.end = walk.ender(a, per, p);
    s.start = p.q.start;
    s.n = p.q.n;
    s.tok = p.tok;
    s.h = p.h;
  }
}

}  // namespace paged
}  // namespace fa
