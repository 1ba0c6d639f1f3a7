// Rotation of queries and keys by their positions, with the norm of each head in
// the same pass, on sm_103a: forward, backward, and on the way into the paged cache.
//
//   z = x rstd w, rstd = (mean(x^2) + eps)^(-1/2)      (norms; else z = x)
//   pair i of z, (a, b):  y = factor (a cos t - b sin t, b cos t + a sin t), t = position * freqs[i]
// and backward, with R the rotation:
//   g = factor R(-t) dy,  dw = sum over rows g o x rstd,
//   dx = rstd (u - xh mean(u o xh)),  u = w o g, xh = x rstd.
//
// Everything is a pass over the rows, bound by HBM where there are many and by
// latency where there are few; the norms add enough instructions to stay behind it
// (16384 tokens of 32 + 8 heads of 128: 55 us forward, 6.1 TB/s; with norms 58 us,
// 5.7 TB/s, and backward, where three passes move, 87 us, 5.8 TB/s). A thread holds
// 16 elements of a row, those of eight whole pairs, in two 16-byte chunks: D / 16
// lanes a row. A warp takes one token and a slice of its heads, so that its lanes
// make each angle once for all of them.
//
// Angles: a position times a frequency may be millions of radians, of which fp32
// keeps no fraction of a turn. The frequency is taken in turns as a 64-bit
// fraction, 2^64 a turn, so that its product with the position modulo 2^64 is
// the place in the turn (an integer multiplication; the fraction's rounding,
// 2^-64 of a turn a position, is all that is lost), of which the upper 32 bits go to sincospi.
#include <algorithm>
#include <atomic>
#include <cstdint>

#include <cuda_bf16.h>

#include "fa_internal.h"
#include "paged.h"
#include "ptx.cuh"
#include "quant.cuh"
#include "rope.h"

namespace fa {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

enum Mode { kForward, kBackward, kStore };

// A lane's place in its row: where its two chunks of 8 elements begin, each beside its neighbours' (so that a load or store of
// a row's lanes is of whole sectors). Neighbours make pairs in any chunk; halves apart, the second chunk is the first one's.
struct Place {
  int a, b;
};
template <int D, bool INTER>
__device__ __forceinline__ Place place(int part, int rot) {
  const int half = INTER ? D / 2 : rot / 2, past = part - rot / 16;
  if (INTER || past < 0) return {8 * part, half + 8 * part};
  return {rot + 8 * past, rot + (D - rot) / 2 + 8 * past};  // not rotated
}

struct Raw {
  uint4 a, b;
};
// Rows on their way, DEPTH steps ahead, T tensors a step: copied past the registers into a thread's own slots of shared
// memory, so that the registers are free for the work. A slot is filled again a step after it was read, when what was read
// of it has been used. 16384 tokens of 32 + 8 heads of 128 with norms, forward and backward: 162.9 us with the rows in
// registers, 142 to 143 us with 2 steps ahead, 149 us with 3 (of an SM's shared memory more is a ring, and less a cache).
constexpr int kAhead = 2;
template <int DEPTH, int T>
struct Ring {
  static constexpr int kSlots = DEPTH + 1, kBytes = kSlots * T * 2 * kThreads * 16;
  uint32_t at;  // this thread's first slot
  uint32_t fill, take;
  __device__ __forceinline__ explicit Ring(const void* smem) : at(ptx::smem_u32(smem) + threadIdx.x * 16), fill(0), take(0) {}
  __device__ __forceinline__ static uint32_t next(uint32_t i) { return i + 1 == kSlots ? 0 : i + 1; }
  // Tensor t of the step to come: the row's two chunks, or (there is no row) zeros.
  __device__ __forceinline__ void load(int t, const __nv_bfloat16* row, const Place& p, bool there) {
    const uint32_t to = at + (fill * T + t) * (2 * kThreads * 16);
    const int bytes = there ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(row + p.a), "r"(bytes) : "memory");
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + kThreads * 16), "l"(row + p.b), "r"(bytes) : "memory");
  }
  // The step's loads are under way ('step': there is one, else nothing was loaded).
  __device__ __forceinline__ void loaded(bool step) {
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (step) fill = next(fill);
  }
  // The oldest of DEPTH steps that are on their way has come.
  __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory"); }
  __device__ __forceinline__ Raw get(int t) const {
    const uint32_t from = at + (take * T + t) * (2 * kThreads * 16);
    Raw r;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.a.x), "=r"(r.a.y), "=r"(r.a.z), "=r"(r.a.w) : "r"(from) : "memory");
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.b.x), "=r"(r.b.y), "=r"(r.b.z), "=r"(r.b.w) : "r"(from + kThreads * 16) : "memory");
    return r;
  }
  __device__ __forceinline__ void taken() { take = next(take); }
};
// A lane's 16 elements in fp32: of pairs 2 i and 2 i + 1 the first elements in a[i], the second in b[i], so that the work on
// them is packed, two at an instruction.
struct Row {
  float2 a[4], b[4];
};
// INTER: a word is a pair, else the chunks' elements stand side by side.
template <bool INTER>
__device__ __forceinline__ Row unpack(const Raw& r) {
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
  float lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo[i] = __uint_as_float(w[i] << 16);
    hi[i] = __uint_as_float(w[i] & 0xffff0000u);
  }
  Row x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x.a[i] = INTER ? make_float2(lo[2 * i], lo[2 * i + 1]) : make_float2(lo[i], hi[i]);
    x.b[i] = INTER ? make_float2(hi[2 * i], hi[2 * i + 1]) : make_float2(lo[4 + i], hi[4 + i]);
  }
  return x;
}
// The elements in the order of the row's two chunks.
template <bool INTER>
__device__ __forceinline__ void in_order(const Row& x, float (&y)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[INTER ? 4 * i : 2 * i] = x.a[i].x;
    y[INTER ? 4 * i + 2 : 2 * i + 1] = x.a[i].y;
    y[INTER ? 4 * i + 1 : 8 + 2 * i] = x.b[i].x;
    y[INTER ? 4 * i + 3 : 9 + 2 * i] = x.b[i].y;
  }
}
template <bool INTER>
__device__ __forceinline__ void store_row(__nv_bfloat16* row, const Place& p, const Row& x) {
  float y[16];
  in_order<INTER>(x, y);
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = ptx::pack_bf16x2(y[2 * i], y[2 * i + 1]);
  *reinterpret_cast<uint4*>(row + p.a) = make_uint4(w[0], w[1], w[2], w[3]);
  *reinterpret_cast<uint4*>(row + p.b) = make_uint4(w[4], w[5], w[6], w[7]);
}

// Cosines and sines of a lane's pairs, as a Row's.
struct Turn {
  float2 c[4], s[4];
};
// (Chunks are rotated wholly or not at all, and those from rot on are left out: turned by cosine 1 and sine 0 their infinities
// and NaN would reach the elements that stand where their pairs would. Halves apart, both of a lane's chunks are alike.
// Whole heads, the same test for all lanes, cost nothing; without that test the backward with norms took 83.9 us, with it 83.3.)
template <int D, bool INTER>
__device__ __forceinline__ void rotate(Row& x, const Turn& t, const Place& p, int rot) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (rot != D && (INTER && i >= 2 ? p.b : p.a) >= rot) continue;
    const float2 a = x.a[i], bs = ptx::fmul2(x.b[i], t.s[i]);
    x.b[i] = ptx::ffma2(a, t.s[i], ptx::fmul2(x.b[i], t.c[i]));
    x.a[i] = make_float2(fmaf(a.x, t.c[i].x, -bs.x), fmaf(a.y, t.c[i].y, -bs.y));
  }
}

// Frequencies as fractions of a turn, 2^64 a turn: the 53 bits of |f| times 128 bits of 1 / 2 pi, 2^-130 k, moved to where the
// fraction's 64 bits are; off by 2^-64 of a turn up to 2^54 radians. (A product of doubles loses up to 1.6 2^-53 of f, at a
// position of 2^31 2^-24 of a turn for one radian each and in proportion for more; with 1 / 2 pi as a sum of two doubles nothing
// is lost either, but one token of 32 + 8 heads then takes 3.0 us, and 2.7 so.)
__device__ __forceinline__ unsigned long long turns(double f) {
  constexpr unsigned long long kHigh = 0xa2f9836e4e441529ull, kLow = 0xfc2757d1f534ddc0ull;
  const unsigned long long bits = (unsigned long long)__double_as_longlong(f);
  const int e = (int)(bits >> 52) & 0x7ff;
  const unsigned long long m = (bits & 0xfffffffffffffull) | (e ? 1ull << 52 : 0ull);
  const unsigned long long low = __umul64hi(m, kLow), mid = m * kHigh + low, high = __umul64hi(m, kHigh) + (mid < low);
  const int s = 1077 - max(e, 1);  // how far the 128 bits high, mid stand above the fraction's last
  unsigned long long t = 0;
  if (s >= 0 && s < 64) t = mid >> s | high << 1 << (63 - s);
  if (s >= 64 && s < 128) t = high >> (s - 64);
  return bits >> 63 ? 0ull - t : t;
}

// Cosines and sines of the tokens that a warp has at a time, in its part of shared memory: made by its lanes in turn, four
// pairs' halves of every lane side by side (no bank twice), as place() deals them out.
template <int D>
struct Angles {
  float4 at[D / 2 * 32 / (D / 16) / 2];  // two pairs' cosines, then their sines; D / 2 pairs a token, up to 32 / (D / 16) tokens
};
// Where a token is: number n of sequence b. on(): so many tokens later.
struct Token {
  int b, n;
  __device__ __forceinline__ Token on(int more, int N) const {
    Token t = {b, n + more};
    while (t.n >= N) {
      t.n -= N;
      ++t.b;
    }
    return t;
  }
};
template <int D, bool INTER>
__device__ __forceinline__ void make_angles(const RopeArgs& a, const unsigned long long* turn, Angles<D>& to, int tokens,
                                            const Token& first, int lane, float sign) {
  constexpr int kLanes = D / 16;
  __syncwarp();  // the angles before have been read
  for (int i = lane; i < tokens * (D / 2); i += 32) {
    const int which = i / (D / 2), pair = i % (D / 2);
    if (pair >= a.rot / 2) continue;
    const Token at_token = first.on(which, a.N);
    const int position = !a.pos ? at_token.n : at_token.b < a.B ? a.pos[at_token.b * a.pos_b + at_token.n] : 0;
    const unsigned long long t = (unsigned long long)(long long)position * turn[pair];
    float2 cs;
    sincospif((float)(int)(t >> 32) * 0x1p-31f, &cs.y, &cs.x);
    cs.x *= a.factor;
    cs.y *= sign * a.factor;
    const int part = INTER ? pair % (D / 4) / 4 : pair / 8, own = INTER ? pair / (D / 4) * 4 + pair % 4 : pair % 8;
    float* at = reinterpret_cast<float*>(&to.at[which * (D / 4) + own / 2 * kLanes + part]) + own % 2;
    at[0] = cs.x;
    at[2] = cs.y;
  }
  __syncwarp();
}
template <int D>
__device__ __forceinline__ Turn take_angles(const Angles<D>& from, int which, int part) {
  Turn t;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = from.at[which * (D / 4) + i * (D / 16) + part];
    t.c[i] = make_float2(v.x, v.y);
    t.s[i] = make_float2(v.z, v.w);
  }
  return t;
}

// The weights of a part in shared memory, a[i] and b[i] of every lane side by side (no bank twice), as place() deals them out.
template <int D, bool INTER>
__device__ __forceinline__ void stage_weights(const RopeArgs& a, const void* w, float4* to) {
  constexpr int kLanes = D / 16;
  for (int i = threadIdx.x; i < D; i += kThreads) {
    const int part = i / 16, e = i % 16;
    const Place p = place<D, INTER>(part, a.rot);
    const int at = e < 8 ? p.a + e : p.b + e - 8;
    const float x = a.w_fp32 ? static_cast<const float*>(w)[at] : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[at]);
    const int pair = INTER ? e / 2 : e % 8, second = INTER ? e % 2 : e / 8;
    reinterpret_cast<float*>(to + (pair / 2) * kLanes + part)[2 * second + pair % 2] = x;
  }
}
template <int D>
__device__ __forceinline__ void times_weights(Row& x, const float4* w, int part) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = w[i * (D / 16) + part];
    x.a[i] = ptx::fmul2(x.a[i], make_float2(v.x, v.y));
    x.b[i] = ptx::fmul2(x.b[i], make_float2(v.z, v.w));
  }
}
__device__ __forceinline__ void times(Row& x, float f) {
  const float2 ff = make_float2(f, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x.a[i] = ptx::fmul2(x.a[i], ff);
    x.b[i] = ptx::fmul2(x.b[i], ff);
  }
}
// This lane's part of the rows' product.
__device__ __forceinline__ float dot(const Row& x, const Row& y) {
  float2 a = ptx::fmul2(x.a[0], y.a[0]), b = ptx::fmul2(x.b[0], y.b[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    a = ptx::ffma2(x.a[i], y.a[i], a);
    b = ptx::ffma2(x.b[i], y.b[i], b);
  }
  a = ptx::fadd2(a, b);
  return a.x + a.y;
}

// Sum over the lanes of a row.
template <int D>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int s = 1; s < D / 16; s <<= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
  return x;
}

template <int D>
__device__ __forceinline__ float inverse_deviation(const Row& x, float eps) {
  return rsqrtf(fmaf(row_sum<D>(dot(x, x)), 1.f / D, eps));
}

// Sixteen codes of a lane's row into a cache page. (Factors far from 1 with the values' scale: without it 1 / f may be infinite,
// and zero times that is no zero, or subnormal and short of bits. Keys are made smaller before their rotation, where the
// largest would overflow, and larger after it, where infinities would meet.)
template <bool INTER>
__device__ __forceinline__ void store_codes(uint8_t* row, const Place& p, Row& y, const Factor& f) {
  if (f.scale > 1.f) times(y, f.scale);
  float x[16];
  in_order<INTER>(y, x);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = e4m3x4(x[4 * i] * f.inv, x[4 * i + 1] * f.inv, x[4 * i + 2] * f.inv, x[4 * i + 3] * f.inv);
  *reinterpret_cast<uint2*>(row + p.a) = make_uint2(w[0], w[1]);
  *reinterpret_cast<uint2*>(row + p.b) = make_uint2(w[2], w[3]);
}

// What a warp has at a time: 'tokens' tokens' slice of heads, a step of which is one row for each of its groups of kLanes
// lanes. Several tokens only where a part has fewer heads than the warp has groups; then there is one step.
struct Unit {
  Token first, token;  // the first, and this lane's group's
  int h, h1;           // the group's first head, the slice's end
  int steps;
  bool there;
};
// (64-bit division takes far longer)
__device__ __forceinline__ long long divide(long long x, int y) {
  return x <= 0xFFFFFFFFll ? (long long)((unsigned)x / (unsigned)y) : x / y;
}
__device__ __forceinline__ Unit unit(const RopeArgs& a, int kind, long long i, int group) {
  Unit u;
  const int many = a.tokens[kind], heads = a.part[kind].heads, slices = a.slices[kind];
  const long long of = slices == 1 ? i : divide(i, slices), first = of * many;
  const int h0 = (int)(i - of * slices) * a.slice_heads[kind];
  u.first.b = (int)divide(first, a.N);
  u.first.n = (int)(first - (long long)u.first.b * a.N);
  const int share = a.groups[kind];  // groups of a token
  u.token = u.first.on(many > 1 ? group / share : 0, a.N);
  u.there = u.token.b < a.B;
  if (!u.there) u.token = {a.B - 1, a.N - 1};
  u.h1 = min(heads, h0 + a.slice_heads[kind]);
  u.h = h0 + (many > 1 ? group % share : group);
  u.steps = (u.h1 - h0 + share - 1) / share;
  if (!u.there) u.h1 = 0;
  return u;
}

// Forward and store: units of the queries first, then the keys (and the values).
constexpr int fwd_ctas_per_sm(bool norm, Mode mode) { return norm || mode == kStore ? 3 : 4; }
template <int D, bool NORM, bool INTER, Mode MODE>
__global__ void __launch_bounds__(kThreads, fwd_ctas_per_sm(NORM, MODE)) fa_rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes;  // lanes of a row, rows a warp has at a time
  __shared__ unsigned long long turn[D / 2];
  __shared__ float4 weights[NORM ? 2 : 1][NORM ? D / 4 : 1];
  __shared__ Angles<D> angles[kWarps];
  extern __shared__ __align__(16) unsigned char ring_at[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = lane / kLanes, part_of = lane % kLanes;
  ptx::grid_release();
  ptx::grid_wait();
  for (int i = threadIdx.x; i < a.rot / 2; i += kThreads) turn[i] = turns(a.freqs[i]);
  if constexpr (NORM) {
    stage_weights<D, INTER>(a, a.part[0].w, weights[0]);
    if (a.part[1].heads) stage_weights<D, INTER>(a, a.part[1].w, weights[1]);
  }
  __syncthreads();
  Ring<kAhead, 1> ring(ring_at);
  const Factor key_factor = factor_of(MODE == kStore && a.fp8 ? a.descale_k : 1.f);
  const long long first_k = a.units[0], first_v = first_k + a.units[1];
  const long long units = MODE == kStore ? first_v + a.units[1] : first_v;
  for (long long i = (long long)blockIdx.x * kWarps + warp; i < units; i += (long long)gridDim.x * kWarps) {
    const bool value = MODE == kStore && i >= first_v;
    const int kind = i >= first_k ? 1 : 0;
    Unit u = unit(a, kind, i - (value ? first_v : kind ? first_k : 0), group);
    const RopePart& part = a.part[kind];
    long long place_in_cache = 0;
    if constexpr (MODE == kStore) {  // rows without a slot have no heads
      const int slot = u.there ? a.slots[u.token.n] : -1;
      if (slot < 0) u.h1 = 0;
      if (kind) {
        const int page = slot >> a.page_shift;
        if (slot >= 0 && page >= a.num_pages) {
          u.h1 = 0;
          if (part_of == 0) atomicOr(a.status, kStatusBadLength);
        }
        place_in_cache = (((long long)page * part.heads) << a.page_shift) + (slot & ((1 << a.page_shift) - 1));
      }
    }
    const Place p = value ? place<D, true>(part_of, 0) : place<D, INTER>(part_of, a.rot);
    const RopeView& src = value ? a.v : part.in;
    int h = u.h;
    const int step = a.groups[kind];
    const __nv_bfloat16* row = static_cast<const __nv_bfloat16*>(src.at) + (u.token.b * src.b + u.token.n * src.n);
    auto load = [&](int k, int ahead) {  // for step k, 'ahead' steps on
      if (k < u.steps) {
        const bool there = h + ahead * step < u.h1;
        ring.load(0, row + (there ? (h + ahead * step) * src.h : 0), p, there);
      }
      ring.loaded(k < u.steps);
    };
#pragma unroll
    for (int k = 0; k < kAhead; ++k) load(k, k);
    if (MODE == kStore && value) {
      for (int k = 0; k < u.steps; ++k, h += step) {
        ring.wait();
        const Raw raw = ring.get(0);
        ring.taken();
        load(k + kAhead, kAhead);
        if (h >= u.h1) continue;
        const long long at = (place_in_cache + ((long long)h << a.page_shift)) * D;
        if (a.fp8) {
          const Factor f = factor_of(a.descale_v);
          uint8_t* dst = static_cast<uint8_t*>(a.v_cache) + at;
          *reinterpret_cast<uint2*>(dst + p.a) = make_uint2(quantise4(raw.a.x, raw.a.y, f), quantise4(raw.a.z, raw.a.w, f));
          *reinterpret_cast<uint2*>(dst + p.b) = make_uint2(quantise4(raw.b.x, raw.b.y, f), quantise4(raw.b.z, raw.b.w, f));
        } else {
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.v_cache) + at;
          *reinterpret_cast<uint4*>(dst + p.a) = raw.a;
          *reinterpret_cast<uint4*>(dst + p.b) = raw.b;
        }
      }
      continue;
    }
    make_angles<D, INTER>(a, turn, angles[warp], a.tokens[kind], u.first, lane, 1.f);
    const Turn t = take_angles<D>(angles[warp], a.tokens[kind] > 1 ? group / step : 0, part_of);
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(part.out.at) + (u.token.b * part.out.b + u.token.n * part.out.n);
    for (int k = 0; k < u.steps; ++k, h += step) {  // (uniform: the sums of a row are a warp's work)
      ring.wait();
      Row x = unpack<INTER>(ring.get(0));
      ring.taken();
      load(k + kAhead, kAhead);
      if (NORM) {
        const float r = inverse_deviation<D>(x, a.eps);
        times_weights<D>(x, weights[kind], part_of);
        times(x, r);
      }
      if (MODE == kStore && kind && key_factor.scale < 1.f) times(x, key_factor.scale);
      rotate<D, INTER>(x, t, p, a.rot);
      if (h >= u.h1) continue;
      if (MODE == kStore && kind) {
        const long long at = (place_in_cache + ((long long)h << a.page_shift)) * D;
        if (a.fp8)
          store_codes<INTER>(static_cast<uint8_t*>(a.k_cache) + at, p, x, key_factor);
        else
          store_row<INTER>(static_cast<__nv_bfloat16*>(a.k_cache) + at, p, x);
      } else {
        store_row<INTER>(out + h * part.out.h, p, x);
      }
    }
  }
}

// Backward: the CTAs of a part take its units in turn, a warp one at a time, so that a lane adds up the weights'
// gradients of its 16 elements in registers; the sums of a CTA go to the workspace, and a second kernel adds those up in
// order (no atomics: repeated calls give the same bits).
constexpr int kMaxSms = 160;
// (Without norms 3 and 4 of them, 16384 tokens of 32 + 8 heads of 128 and 32768 of 64: 53.0 and 57.1 us, 65.9 and 58.3 us.)
constexpr int bwd_ctas_per_sm(bool norm, int d) { return norm ? 2 : d == 64 ? 4 : 3; }
template <int D, bool NORM, bool INTER>
__global__ void __launch_bounds__(kThreads, bwd_ctas_per_sm(NORM, D)) fa_rope_bwd_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int kLanes = D / 16;
  __shared__ unsigned long long turn[D / 2];
  __shared__ float sums[NORM ? kWarps : 1][D];
  __shared__ float4 weights[NORM ? D / 4 : 1];
  __shared__ Angles<D> angles[kWarps];
  extern __shared__ __align__(16) unsigned char ring_at[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = lane / kLanes, part_of = lane % kLanes;
  ptx::grid_release();
  ptx::grid_wait();
  const int kind = (int)blockIdx.x >= a.ctas[0] ? 1 : 0;
  const RopePart& part = a.part[kind];
  for (int i = threadIdx.x; i < a.rot / 2; i += kThreads) turn[i] = turns(a.freqs[i]);
  if constexpr (NORM) stage_weights<D, INTER>(a, part.w, weights);
  __syncthreads();
  Ring<kAhead, NORM ? 2 : 1> ring(ring_at);
  const int cta = (int)blockIdx.x - (kind ? a.ctas[0] : 0), step = a.groups[kind];
  const Place p = place<D, INTER>(part_of, a.rot);
  Row dw;
#pragma unroll
  for (int e = 0; e < 4; ++e) dw.a[e] = dw.b[e] = make_float2(0.f, 0.f);
  for (long long i = (long long)cta * kWarps + warp; i < a.units[kind]; i += (long long)a.ctas[kind] * kWarps) {
    const Unit u = unit(a, kind, i, group);
    int h = u.h;
    const __nv_bfloat16 *in = static_cast<const __nv_bfloat16*>(part.in.at) + (u.token.b * part.in.b + u.token.n * part.in.n),
                        *in_x = static_cast<const __nv_bfloat16*>(part.x.at) + (u.token.b * part.x.b + u.token.n * part.x.n);
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(part.out.at) + (u.token.b * part.out.b + u.token.n * part.out.n);
    auto load = [&](int k, int ahead) {
      if (k < u.steps) {
        const bool there = h + ahead * step < u.h1;
        const int hh = there ? h + ahead * step : 0;
        ring.load(0, in + hh * part.in.h, p, there);
        if (NORM) ring.load(NORM ? 1 : 0, in_x + hh * part.x.h, p, there);
      }
      ring.loaded(k < u.steps);
    };
#pragma unroll
    for (int k = 0; k < kAhead; ++k) load(k, k);
    make_angles<D, INTER>(a, turn, angles[warp], a.tokens[kind], u.first, lane, -1.f);
    const Turn t = take_angles<D>(angles[warp], a.tokens[kind] > 1 ? group / step : 0, part_of);
    for (int k = 0; k < u.steps; ++k, h += step) {
      ring.wait();
      Row g = unpack<INTER>(ring.get(0)), x;
      if (NORM) x = unpack<INTER>(ring.get(NORM ? 1 : 0));
      ring.taken();
      load(k + kAhead, kAhead);
      const bool live = h < u.h1;
      rotate<D, INTER>(g, t, p, a.rot);
      if (NORM) {
        const float all = inverse_deviation<D>(x, a.eps);  // (sums over lanes: every lane takes part)
        const float r = live ? all : 0.f;  // no row: zeros, which add nothing to dw, whatever eps
        times(x, r);  // the normed row before its weights
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          dw.a[e] = ptx::ffma2(g.a[e], x.a[e], dw.a[e]);
          dw.b[e] = ptx::ffma2(g.b[e], x.b[e], dw.b[e]);
        }
        times_weights<D>(g, weights, part_of);
        const float mean = row_sum<D>(dot(g, x)) * (1.f / D);
        const float2 m = make_float2(-mean, -mean);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          g.a[e] = ptx::ffma2(x.a[e], m, g.a[e]);
          g.b[e] = ptx::ffma2(x.b[e], m, g.b[e]);
        }
        times(g, r);
      }
      if (live) store_row<INTER>(out + h * part.out.h, p, g);
    }
  }
  if constexpr (NORM) {
    float sum[16];
    in_order<INTER>(dw, sum);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
#pragma unroll
      for (int s = kLanes; s < 32; s <<= 1) sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], s);
      if (group == 0) sums[warp][(e < 8 ? p.a : p.b - 8) + e] = sum[e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < D; i += kThreads) {
      float t = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) t += sums[k][i];
      a.dw_part[(long long)blockIdx.x * D + i] = t;
    }
  }
}

// The CTAs' sums of one part's weights: a block per 32 elements, its warps every kSumWarps-th CTA.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(32 * kSumWarps) fa_rope_dw_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ float sums[kSumWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, kind = blockIdx.y, e = blockIdx.x * 32 + lane;
  ptx::grid_wait();
  const int first = kind ? a.ctas[0] : 0, last = first + a.ctas[kind];
  float t = 0.f;
#pragma unroll 8
  for (int c = first + warp; c < last; c += kSumWarps) t += a.dw_part[(long long)c * a.d + e];
  sums[warp][lane] = t;
  __syncthreads();
  if (warp) return;
#pragma unroll
  for (int k = 1; k < kSumWarps; ++k) t += sums[k][lane];
  if (a.part[kind].heads) a.dw[kind][e] = t;
}

// Positions of packed tokens: token t of request r, the last of whose n rows has its last key, stands at
// seq_lens[r] - n + its number. A thread finds its row's request among the starts (in shared memory where they fit).
constexpr int kStarts = 4096;
__global__ void __launch_bounds__(kThreads) fa_paged_positions_kernel(const __grid_constant__ PositionsArgs a) {
  __shared__ int starts[kStarts];
  ptx::grid_release();
  ptx::grid_wait();
  const bool fits = a.R < kStarts;
  if (fits) {
    for (int i = threadIdx.x; i <= a.R; i += kThreads) starts[i] = a.query_start[i];
    __syncthreads();
  }
  const int* start = fits ? starts : a.query_start;
  const long long t = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (t >= a.T) return;
  int lo = 0, hi = a.R;  // the last request that begins at or before row t
  while (hi - lo > 1) {
    const int mid = lo + ((hi - lo) >> 1);
    if (start[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  const int s0 = min(max(start[lo], 0), a.T), s1 = min(start[lo + 1], a.T);
  const long long at = (long long)a.seq_lens[lo] - s1 + t;
  a.positions[t] = s0 <= t && t < s1 ? (int)max(at, -1ll) : -1;
}

// Units of each part. Where a part's heads are fewer than a warp's groups of lanes, a warp takes several tokens, a power of
// two groups each; else all heads of a token where the tokens alone fill the GPU, and fewer the fewer tokens there are.
void make_units(RopeArgs& a, int groups, int num_sms) {
  const long long want = (long long)num_sms * 32;  // warps
  const long long tokens = (long long)a.B * a.N;
  int steps = 0;  // of a warp, for all heads of a token
  for (const RopePart& p : a.part) steps += (p.heads + groups - 1) / groups;
  for (int k = 0; k < 2; ++k) {
    const int heads = a.part[k].heads;
    a.tokens[k] = a.slices[k] = 1;
    a.groups[k] = groups;
    a.slice_heads[k] = heads;
    a.units[k] = 0;
    if (!heads) continue;
    if (heads < groups) {
      int share = 1;
      while (share < heads) share *= 2;
      a.groups[k] = share;
      a.tokens[k] = groups / share;
    } else {
      const long long per = std::max(1ll, std::min<long long>(steps, tokens * steps / want));  // steps of a warp
      const int mine = (heads + groups - 1) / groups;
      a.slice_heads[k] = (int)per * groups;
      a.slices[k] = (int)((mine + per - 1) / per);
    }
    a.units[k] = (tokens + a.tokens[k] - 1) / a.tokens[k] * a.slices[k];
  }
}

template <int D, Mode MODE>
cudaError_t launch_forward(const RopeArgs& args, bool norm, bool inter, int num_sms, cudaStream_t stream) {
  RopeArgs a = args;
  make_units(a, 32 / (D / 16), num_sms);
  const long long units = a.units[0] + (MODE == kStore ? 2 : 1) * a.units[1];
  // As many CTAs as run at once, or twice that where their warps have five units each and more, the units in turn: the
  // frequencies and weights are staged once for all. Once, twice and a warp a unit, for 16384 tokens of 32 + 8 heads of 128:
  // without norms 64.2, 55.5 and 54.2 us, with norms 63.3, 58.4 and 61.0 us; the store of 15523 tokens to E4M3 70.0, 68.3 and
  // 74.7 us; with four units a warp, norms of 8008 tokens of 12 + 12 heads of 64, 13.5, 15.0 and 15.7 us.
  const long long once = (long long)num_sms * fwd_ctas_per_sm(norm, MODE);
  const long long resident = units >= 5 * once * kWarps ? 2 * once : once;
  const unsigned ctas = (unsigned)std::min<long long>((units + kWarps - 1) / kWarps, resident);
  auto kern = norm ? (inter ? fa_rope_kernel<D, true, true, MODE> : fa_rope_kernel<D, true, false, MODE>)
                   : (inter ? fa_rope_kernel<D, false, true, MODE> : fa_rope_kernel<D, false, false, MODE>);
  constexpr int kBytes = Ring<kAhead, 1>::kBytes;
  static std::atomic<unsigned long long> known[4];  // devices that know the kernels' shared memory
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), kBytes, known[2 * norm + inter]);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(ctas), kThreads, kBytes, stream, a);
}

// CTAs of the backward for each part, in the ratio of the steps that they have to take.
void backward_ctas(RopeArgs& a, int groups, bool norm, int num_sms) {
  make_units(a, groups, num_sms);
  double steps[2];
  for (int k = 0; k < 2; ++k)
    steps[k] = (double)a.units[k] * ((std::min(a.part[k].heads, a.slice_heads[k]) + a.groups[k] - 1) / a.groups[k] + 0.5 + 0.5 * a.tokens[k]);
  const int all = std::min(num_sms, kMaxSms) * bwd_ctas_per_sm(norm, a.d);
  for (int k = 0; k < 2; ++k) {
    const int most = std::max(1, (int)(all * steps[k] / (steps[0] + steps[1]) + 0.5));
    a.ctas[k] = (int)std::min<long long>((a.units[k] + kWarps - 1) / kWarps, most);
  }
}

template <int D>
cudaError_t launch_backward(const RopeArgs& args, bool norm, bool inter, int num_sms, cudaStream_t stream) {
  RopeArgs a = args;
  backward_ctas(a, 32 / (D / 16), norm, num_sms);
  auto kern = norm ? (inter ? fa_rope_bwd_kernel<D, true, true> : fa_rope_bwd_kernel<D, true, false>)
                   : (inter ? fa_rope_bwd_kernel<D, false, true> : fa_rope_bwd_kernel<D, false, false>);
  const int bytes = norm ? Ring<kAhead, 2>::kBytes : Ring<kAhead, 1>::kBytes;
  static std::atomic<unsigned long long> known[4];
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), bytes, known[2 * norm + inter]);
  if (e != cudaSuccess) return e;
  e = launch_dependent(kern, dim3((unsigned)(a.ctas[0] + a.ctas[1])), kThreads, bytes, stream, a);
  if (e != cudaSuccess || !norm) return e;
  return launch_dependent(fa_rope_dw_kernel, dim3(D / 32, 2u), 32 * kSumWarps, 0, stream, a);
}

}  // namespace

size_t rope_bwd_bytes(int Hq, int Hk, int d) {
  return Hq + Hk > 0 ? (size_t)(kMaxSms * bwd_ctas_per_sm(true, d) + 2) * d * sizeof(float) : 0;
}

cudaError_t launch_rope_fwd(RopeArgs a, bool norm, bool inter, int num_sms, cudaStream_t stream) {
  return a.d == 64 ? launch_forward<64, kForward>(a, norm, inter, num_sms, stream)
                   : launch_forward<128, kForward>(a, norm, inter, num_sms, stream);
}
cudaError_t launch_rope_store(RopeArgs a, bool norm, bool inter, int num_sms, cudaStream_t stream) {
  return a.d == 64 ? launch_forward<64, kStore>(a, norm, inter, num_sms, stream)
                   : launch_forward<128, kStore>(a, norm, inter, num_sms, stream);
}
cudaError_t launch_rope_bwd(RopeArgs a, bool norm, bool inter, int num_sms, cudaStream_t stream) {
  return a.d == 64 ? launch_backward<64>(a, norm, inter, num_sms, stream) : launch_backward<128>(a, norm, inter, num_sms, stream);
}
cudaError_t launch_positions(const PositionsArgs& a, cudaStream_t stream) {
  return launch_dependent(fa_paged_positions_kernel, dim3((unsigned)(((long long)a.T + kThreads - 1) / kThreads)), kThreads, 0,
                          stream, a);
}

}  // namespace fa
