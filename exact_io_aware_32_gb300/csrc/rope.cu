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
// latency where there are few. A thread holds 16 elements of a row, those of
// eight whole pairs, in two 16-byte chunks: D / 16 lanes a row. A warp takes one
// token and a slice of its heads, so that the eight angles of a lane serve all of them.
//
// Angles: a position times a frequency may be millions of radians, of which fp32
// keeps no fraction of a turn. The frequency is taken in turns as a 64-bit
// fraction, 2^64 a turn, so that its product with the position modulo 2^64 is
// the exact place in the turn (an integer multiplication; the frequency's own
// rounding, 2^-53 of it, is all that is lost), of which the upper 32 bits go to sincospi.
#include <algorithm>
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

// A lane's place in its row: where its two chunks of 8 elements begin, and its first pair (< 0: not rotated).
struct Place {
  int a, b, pair;
};
template <bool INTER>
__device__ __forceinline__ Place place(int part, int rot) {
  if (INTER || 16 * part >= rot) return {16 * part, 16 * part + 8, 16 * part < rot ? 8 * part : -1};
  return {8 * part, rot / 2 + 8 * part, 8 * part};
}

struct Raw {
  uint4 a, b;
};
__device__ __forceinline__ Raw load_row(const RopeView& v, long long at, const Place& p) {
  const __nv_bfloat16* row = static_cast<const __nv_bfloat16*>(v.at) + at;
  return {*reinterpret_cast<const uint4*>(row + p.a), *reinterpret_cast<const uint4*>(row + p.b)};
}
__device__ __forceinline__ void unpack(const Raw& r, float (&x)[16]) {
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store_row(const RopeView& v, long long at, const Place& p, const float (&x)[16]) {
  __nv_bfloat16* row = static_cast<__nv_bfloat16*>(v.at) + at;
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = ptx::pack_bf16x2(x[2 * i], x[2 * i + 1]);
  *reinterpret_cast<uint4*>(row + p.a) = make_uint4(w[0], w[1], w[2], w[3]);
  *reinterpret_cast<uint4*>(row + p.b) = make_uint4(w[4], w[5], w[6], w[7]);
}

// The pairs of a lane's 16 elements: neighbours, or the two chunks' elements side by side.
template <bool INTER>
__device__ __forceinline__ void rotate(float (&x)[16], const float (&c)[8], const float (&s)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float &a = x[INTER ? 2 * i : i], &b = x[INTER ? 2 * i + 1 : 8 + i];
    const float a0 = a;
    a = fmaf(a0, c[i], -b * s[i]);
    b = fmaf(b, c[i], a0 * s[i]);
  }
}

// Frequencies as fractions of a turn, 2^64 a turn.
__device__ __forceinline__ unsigned long long turns(double f) {
  const double x = f * 0.15915494309189533577;
  return __double2ull_rn((x - floor(x)) * 18446744073709551616.0);
}

__device__ __forceinline__ void angles(const RopeArgs& a, const unsigned long long* turn, const Place& p, int position,
                                       float sign, float (&c)[8], float (&s)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    c[i] = 1.f;
    s[i] = 0.f;
  }
  if (p.pair < 0) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const unsigned long long t = (unsigned long long)(long long)position * turn[p.pair + i];
    sincospif((float)(int)(t >> 32) * 0x1p-31f, &s[i], &c[i]);
    c[i] *= a.factor;
    s[i] *= sign * a.factor;
  }
}

__device__ __forceinline__ void load_weights(const RopeArgs& a, const void* w, const Place& p, float (&x)[16]) {
  if (a.w_fp32) {
    const float* f = static_cast<const float*>(w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = f[p.a + i];
      x[8 + i] = f[p.b + i];
    }
  } else {
    unpack(load_row(RopeView{const_cast<void*>(w), 0, 0, 0}, 0, p), x);
  }
}

// Sum over the lanes of a row.
template <int D>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int s = 1; s < D / 16; s <<= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
  return x;
}

template <int D>
__device__ __forceinline__ float inverse_deviation(const float (&x)[16], float eps) {
  float q[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 16; ++i) q[i & 1] = fmaf(x[i], x[i], q[i & 1]);
  return rsqrtf(fmaf(row_sum<D>(q[0] + q[1]), 1.f / D, eps));
}

// Sixteen codes of a lane's row into a cache page.
__device__ __forceinline__ void store_codes(uint8_t* row, const Place& p, const float (&x)[16], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = e4m3x4(x[4 * i] * inv, x[4 * i + 1] * inv, x[4 * i + 2] * inv, x[4 * i + 3] * inv);
  *reinterpret_cast<uint2*>(row + p.a) = make_uint2(w[0], w[1]);
  *reinterpret_cast<uint2*>(row + p.b) = make_uint2(w[2], w[3]);
}

// Forward and store: units (token, slice of heads), a warp each; of the queries first, then the keys (and the values).
template <int D, bool NORM, bool INTER, Mode MODE>
__global__ void __launch_bounds__(kThreads) fa_rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes;  // lanes of a row, rows a warp has at a time
  __shared__ unsigned long long turn[D / 2];
  const int lane = threadIdx.x & 31, row = lane / kLanes;
  ptx::grid_release();
  ptx::grid_wait();
  for (int i = threadIdx.x; i < a.rot / 2; i += kThreads) turn[i] = turns(a.freqs[i]);
  __syncthreads();
  const long long tokens = (long long)a.B * a.N;
  const long long first_k = tokens * a.slices[0], first_v = first_k + tokens * a.slices[1];
  const long long units = MODE == kStore ? first_v + tokens * a.slices[1] : first_v;
  for (long long u = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); u < units; u += (long long)gridDim.x * kWarps) {
    const bool value = MODE == kStore && u >= first_v;
    const int kind = u >= first_k ? 1 : 0;
    const long long i = u - (value ? first_v : kind ? first_k : 0);
    const RopePart& part = a.part[kind];
    const int slices = a.slices[kind];
    const long long token = i / slices;
    const int h0 = (int)(i - token * slices) * a.slice_heads[kind], h1 = min(part.heads, h0 + a.slice_heads[kind]);
    const int b = (int)(token / a.N), n = (int)(token - (long long)b * a.N);
    int slot = 0;
    if constexpr (MODE == kStore) {
      slot = a.slots[n];
      if (slot < 0) continue;
      if (kind && slot >> a.page_shift >= a.num_pages) {
        if (lane == 0) atomicOr(a.status, kStatusBadLength);
        continue;
      }
    }
    const Place p = value ? place<true>(lane % kLanes, 0) : place<INTER>(lane % kLanes, a.rot);
    const RopeView& src = value ? a.v : part.in;
    const long long from = b * src.b + n * src.n;
    int h = h0 + row;
    Raw next{};
    if (h < h1) next = load_row(src, from + h * src.h, p);
    float c[8], s[8], w[16];
    if (!value) {
      if (NORM) load_weights(a, part.w, p, w);
      angles(a, turn, p, a.pos ? a.pos[b * a.pos_b + n] : n, 1.f, c, s);
    }
    for (int k = h0; k < h1; k += kRows, h += kRows) {  // (uniform: the sums of a row are a warp's work)
      const Raw raw = next;
      if (h + kRows < h1) next = load_row(src, from + (h + kRows) * src.h, p);
      if (MODE == kStore && kind) {
        const long long at = ((((long long)(slot >> a.page_shift) * part.heads + h) << a.page_shift) +
                              (slot & ((1 << a.page_shift) - 1))) * D;
        if (value) {
          if (h >= h1) continue;
          if (a.fp8) {
            const Factor f = factor_of(a.descale_v);
            *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.v_cache) + at + p.a) =
                make_uint4(quantise4(raw.a.x, raw.a.y, f), quantise4(raw.a.z, raw.a.w, f), quantise4(raw.b.x, raw.b.y, f),
                           quantise4(raw.b.z, raw.b.w, f));
          } else {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.v_cache) + at + p.a);
            dst[0] = raw.a;
            dst[1] = raw.b;
          }
          continue;
        }
        float x[16];
        unpack(raw, x);
        if (NORM) {
          const float r = inverse_deviation<D>(x, a.eps);
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] *= r * w[e];
        }
        rotate<INTER>(x, c, s);
        if (h >= h1) continue;
        if (a.fp8)
          store_codes(static_cast<uint8_t*>(a.k_cache) + at, p, x, 1.f / a.descale_k);
        else
          store_row(RopeView{a.k_cache, 0, 0, 0}, at, p, x);
      } else {
        float x[16];
        unpack(raw, x);
        if (NORM) {
          const float r = inverse_deviation<D>(x, a.eps);
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] *= r * w[e];
        }
        rotate<INTER>(x, c, s);
        if (h < h1) store_row(part.out, b * part.out.b + n * part.out.n + h * part.out.h, p, x);
      }
    }
  }
}

// Backward: the CTAs of a part take its tokens in turn, a warp a token at a time, so that a lane adds up the weights'
// gradients of its 16 elements in registers; the sums of a CTA go to the workspace, and a second kernel adds those up in
// order (no atomics: repeated calls give the same bits).
template <int D, bool NORM, bool INTER>
__global__ void __launch_bounds__(kThreads) fa_rope_bwd_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes;
  __shared__ unsigned long long turn[D / 2];
  __shared__ float sums[NORM ? kWarps : 1][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = lane / kLanes;
  ptx::grid_release();
  ptx::grid_wait();
  for (int i = threadIdx.x; i < a.rot / 2; i += kThreads) turn[i] = turns(a.freqs[i]);
  __syncthreads();
  const int kind = (int)blockIdx.x >= a.ctas[0] ? 1 : 0;
  const RopePart& part = a.part[kind];
  const int cta = (int)blockIdx.x - (kind ? a.ctas[0] : 0), slices = a.slices[kind];
  const long long units = (long long)a.B * a.N * slices;
  const Place p = place<INTER>(lane % kLanes, a.rot);
  float w[16], dw[16];
  if (NORM) load_weights(a, part.w, p, w);
#pragma unroll
  for (int e = 0; e < 16; ++e) dw[e] = 0.f;
  for (long long u = (long long)cta * kWarps + warp; u < units; u += (long long)a.ctas[kind] * kWarps) {
    const long long token = u / slices;
    const int h0 = (int)(u - token * slices) * a.slice_heads[kind], h1 = min(part.heads, h0 + a.slice_heads[kind]);
    const int b = (int)(token / a.N), n = (int)(token - (long long)b * a.N);
    const long long from = b * part.in.b + n * part.in.n, x_from = b * part.x.b + n * part.x.n;
    int h = h0 + row;
    Raw next{}, next_x{};
    if (h < h1) {
      next = load_row(part.in, from + h * part.in.h, p);
      if (NORM) next_x = load_row(part.x, x_from + h * part.x.h, p);
    }
    float c[8], s[8];
    angles(a, turn, p, a.pos ? a.pos[b * a.pos_b + n] : n, -1.f, c, s);
    for (int k = h0; k < h1; k += kRows, h += kRows) {
      const Raw raw = next, raw_x = next_x;
      if (h + kRows < h1) {
        next = load_row(part.in, from + (h + kRows) * part.in.h, p);
        if (NORM) next_x = load_row(part.x, x_from + (h + kRows) * part.x.h, p);
      }
      float g[16];
      unpack(raw, g);
      rotate<INTER>(g, c, s);
      if (NORM) {
        float x[16];
        unpack(raw_x, x);
        const float r = inverse_deviation<D>(x, a.eps);
        float m[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          x[e] *= r;  // the normed row before its weights
          if (h < h1) dw[e] = fmaf(g[e], x[e], dw[e]);
          g[e] *= w[e];
          m[e & 1] = fmaf(g[e], x[e], m[e & 1]);
        }
        const float mean = row_sum<D>(m[0] + m[1]) * (1.f / D);
#pragma unroll
        for (int e = 0; e < 16; ++e) g[e] = r * fmaf(-x[e], mean, g[e]);
      }
      if (h < h1) store_row(part.out, b * part.out.b + n * part.out.n + h * part.out.h, p, g);
    }
  }
  if constexpr (NORM) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
#pragma unroll
      for (int s = kLanes; s < 32; s <<= 1) dw[e] += __shfl_xor_sync(0xffffffffu, dw[e], s);
      if (row == 0) sums[warp][(e < 8 ? p.a : p.b - 8) + e] = dw[e];
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

// The CTAs' sums of one part's weights: a block per 32 elements, its warps every kWarps-th CTA.
__global__ void __launch_bounds__(kThreads) fa_rope_dw_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ float sums[kWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, kind = blockIdx.y, e = blockIdx.x * 32 + lane;
  ptx::grid_wait();
  const int first = kind ? a.ctas[0] : 0, last = first + a.ctas[kind];
  float t = 0.f;
#pragma unroll 4
  for (int c = first + warp; c < last; c += kWarps) t += a.dw_part[(long long)c * a.d + e];
  sums[warp][lane] = t;
  __syncthreads();
  if (warp) return;
#pragma unroll
  for (int k = 1; k < kWarps; ++k) t += sums[k][lane];
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

// Warps that share a token's heads, and how many heads each takes: all of them where the tokens alone fill the GPU, fewer
// the fewer tokens there are.
void slice(RopeArgs& a, int rows, int num_sms) {
  const long long want = (long long)num_sms * 32;  // warps
  const long long tokens = (long long)a.B * a.N;
  const int steps = (a.part[0].heads + rows - 1) / rows + (a.part[1].heads + rows - 1) / rows;  // of a warp, for a token
  for (int k = 0; k < 2; ++k) {
    const int mine = (a.part[k].heads + rows - 1) / rows;
    long long per = std::max(1ll, std::min<long long>(steps, tokens * steps / want));  // steps of a warp
    a.slice_heads[k] = (int)per * rows;
    a.slices[k] = mine ? (int)((mine + per - 1) / per) : 0;
  }
}

template <int D, Mode MODE>
cudaError_t launch_forward(const RopeArgs& args, bool norm, bool inter, int num_sms, cudaStream_t stream) {
  RopeArgs a = args;
  slice(a, 32 / (D / 16), num_sms);
  const long long units = (long long)a.B * a.N * (a.slices[0] + (MODE == kStore ? 2 : 1) * a.slices[1]);
  const unsigned ctas = (unsigned)std::min<long long>((units + kWarps - 1) / kWarps, 1 << 20);
  auto kern = norm ? (inter ? fa_rope_kernel<D, true, true, MODE> : fa_rope_kernel<D, true, false, MODE>)
                   : (inter ? fa_rope_kernel<D, false, true, MODE> : fa_rope_kernel<D, false, false, MODE>);
  return launch_dependent(kern, dim3(ctas), kThreads, 0, stream, a);
}

// CTAs of the backward for each part, in the ratio of their heads.
constexpr int kMaxSms = 160, kBwdCtasPerSm = 4;
void backward_ctas(RopeArgs& a, int rows, int num_sms) {
  slice(a, rows, num_sms);
  const int H = a.part[0].heads + a.part[1].heads, all = std::min(num_sms, kMaxSms) * kBwdCtasPerSm;
  for (int k = 0; k < 2; ++k) {
    const long long units = (long long)a.B * a.N * a.slices[k];
    const long long most = std::max(1ll, (long long)all * a.part[k].heads / H);
    a.ctas[k] = a.part[k].heads ? (int)std::min<long long>((units + kWarps - 1) / kWarps, most) : 0;
  }
}

template <int D>
cudaError_t launch_backward(const RopeArgs& args, bool norm, bool inter, int num_sms, cudaStream_t stream) {
  RopeArgs a = args;
  backward_ctas(a, 32 / (D / 16), num_sms);
  auto kern = norm ? (inter ? fa_rope_bwd_kernel<D, true, true> : fa_rope_bwd_kernel<D, true, false>)
                   : (inter ? fa_rope_bwd_kernel<D, false, true> : fa_rope_bwd_kernel<D, false, false>);
  const cudaError_t e = launch_dependent(kern, dim3((unsigned)(a.ctas[0] + a.ctas[1])), kThreads, 0, stream, a);
  if (e != cudaSuccess || !norm) return e;
  return launch_dependent(fa_rope_dw_kernel, dim3(D / 32, 2u), kThreads, 0, stream, a);
}

}  // namespace

size_t rope_bwd_bytes(int Hq, int Hk, int d) {
  return Hq + Hk > 0 ? (size_t)(kMaxSms * kBwdCtasPerSm + 2) * d * sizeof(float) : 0;
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
