// The paged cache's bookkeeping: planning a step (block tables, slots) and
// storing new keys and values.
#include <algorithm>
#include <cstdint>

#include <cuda_bf16.h>

#include "fa_internal.h"
#include "paged.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kPlanThreads = 256;

// One request's lengths as the plan takes them.
struct Need {
  long long rows;         // new tokens (packed rows)
  long long ctx, len;     // tokens before and after, cut to the table's width
  int held, pages;        // pages before, pages to take
  bool bad;
};

__device__ __forceinline__ Need need_of(const PlanArgs& a, int r) {
  Need n;
  const int c = a.ctx_lens[r], w = a.new_lens[r];
  const long long cap = (long long)a.max_pages << a.page_shift;
  n.rows = max(w, 0);
  n.ctx = max(c, 0);
  n.len = n.ctx + n.rows;
  n.bad = c < 0 || w < 0 || n.len > cap;
  n.len = min(n.len, cap);
  n.ctx = min(n.ctx, cap);
  const int up = (1 << a.page_shift) - 1;
  n.held = (int)((n.ctx + up) >> a.page_shift);
  n.pages = (int)((n.len + up) >> a.page_shift) - n.held;
  return n;
}

__device__ __forceinline__ long long warp_scan(long long x, int lane) {  // inclusive
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, s);
    if (lane >= s) x += y;
  }
  return x;
}

// Prefix sums over the requests give each its packed rows and its pages; every
// CTA (a group of requests by a slice of their tokens) adds up the requests
// before its own, so one launch does it without a pass between CTAs: R lengths
// are a few KB that L2 serves to all of them, and the call is bound by latency.
__global__ void __launch_bounds__(kPlanThreads) fa_paged_plan_kernel(const __grid_constant__ PlanArgs a) {
  constexpr int kWarps = kPlanThreads / 32;
  __shared__ long long s_sum[2][kWarps];
  __shared__ long long s_row[kPlanThreads], s_page[kPlanThreads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int slices = gridDim.y, slice = blockIdx.y;
  const int r0 = blockIdx.x * a.group, r1 = min(a.R, r0 + a.group);
  ptx::grid_release();
  ptx::grid_wait();
  const int told = a.free_head ? *a.free_head : 0, head = max(told, 0);
  const long long avail = max(a.n_free - head, 0);

  // rows and pages of the requests before this group
  long long rows = 0, pages = 0;
  for (int r = tid; r < r0; r += kPlanThreads) {
    const Need n = need_of(a, r);
    rows += n.rows;
    pages += n.pages;
  }
  rows = warp_scan(rows, lane);
  pages = warp_scan(pages, lane);
  if (lane == 31) {
    s_sum[0][warp] = rows;
    s_sum[1][warp] = pages;
  }
  __syncthreads();
  rows = pages = 0;
  for (int w = 0; w < kWarps; ++w) {
    rows += s_sum[0][w];
    pages += s_sum[1][w];
  }

  for (int c0 = r0; c0 < r1; c0 += kPlanThreads) {  // up to kPlanThreads requests at a time
    const int r = c0 + tid;
    Need n{};
    if (r < r1) n = need_of(a, r);
    const long long ir = warp_scan(n.rows, lane), ip = warp_scan(n.pages, lane);
    __syncthreads();  // the sums of the pass before have been read
    if (lane == 31) {
      s_sum[0][warp] = ir;
      s_sum[1][warp] = ip;
    }
    __syncthreads();
    long long row = rows + ir - n.rows, page = pages + ip - n.pages;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) {
        row += s_sum[0][w];
        page += s_sum[1][w];
      }
      rows += s_sum[0][w];
      pages += s_sum[1][w];
    }
    s_row[tid] = row;
    s_page[tid] = page;
    if (r < r1 && slice == 0) {
      a.query_start[r] = (int)min(row, (long long)a.T);
      a.seq_lens[r] = (int)min(n.len, n.ctx + max((long long)a.T - row, 0ll));  // tokens that have no row are not there
      if (n.bad || row + n.rows > a.T) atomicOr(a.status, kStatusBadLength);
    }
    __syncthreads();
    for (int i = warp; i < min(kPlanThreads, r1 - c0); i += kWarps) {  // one warp per request
      const Need m = need_of(a, c0 + i);
      const long long first_row = s_row[i], first_page = s_page[i];
      int* tab = a.block_table + (long long)(c0 + i) * a.max_pages;
      auto fresh = [&](long long x) { return first_page + x < avail ? a.free_pages[head + first_page + x] : -1; };
      for (int x = slice * 32 + lane; x < m.pages; x += 32 * slices) {
        const int page = fresh(x);
        tab[m.held + x] = page;
        if (page < 0) atomicOr(a.status, first_page + x >= avail ? kStatusNoPages : kStatusBadLength);
      }
      const long long n_rows = min(m.rows, (long long)a.T - first_row);
      for (long long x = slice * 32 + lane; x < n_rows; x += 32 * slices) {
        const long long pos = m.ctx + x;
        const long long pi = pos >> a.page_shift;
        int slot = -1;
        if (pi < a.max_pages) {
          const long long pg = pi < m.held ? tab[pi] : fresh(pi - m.held);
          const long long at = (pg << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
          if (pg >= 0 && at <= INT32_MAX)
            slot = (int)at;
          else if (pi < m.held || pg >= 0)
            atomicOr(a.status, kStatusBadLength);
        }
        a.slots[first_row + x] = slot;
      }
    }
  }
  if (r1 == a.R) {  // the last group knows the totals
    if (slice == 0 && tid == 0) {
      a.query_start[a.R] = (int)min(rows, (long long)a.T);
      *a.pages_taken = (int)min(pages, avail);
      if (told < 0) atomicOr(a.status, kStatusBadLength);
    }
    for (long long t = rows + slice * kPlanThreads + tid; t < a.T; t += (long long)kPlanThreads * slices)
      a.slots[t] = -1;
  }
}

// x / f for an E4M3 code, rounded once: the quotient rounded to odd (24 bits, the
// last one set when something was cut off) rounds to the code's 4 bits as the
// exact quotient would, ties among them. q = x / f to within one last place by
// one correction of x * (1 / f); the remainder x - q f is exact and its sign
// says on which side of q the quotient lies: an odd neighbour of q (or q, if
// odd) on that side has no tie between it and the quotient.
__device__ __forceinline__ float quotient_odd(float x, float f, float inv) {
  const float q0 = x * inv;
  const float q = fmaf(fmaf(-q0, f, x), inv, q0);
  const float r = fmaf(-q, f, x);
  const uint32_t b = __float_as_uint(q);
  const uint32_t odd = (b - ((b ^ __float_as_uint(r)) >> 31)) | 1u;  // towards zero when r's sign is the other one
  const float y = r != 0.f ? __uint_as_float(odd) : q;
  return fabsf(q0) < 512.f ? y : q0;  // past the largest code, infinite or NaN: as it is
}

// Four values to E4M3 codes, nearest even, +-448 beyond, NaN for NaN.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n .reg .b16 lo, hi;\n cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
      " mov.b32 %0, {lo, hi};\n}\n"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// Factors far from 1, where the remainder or 1 / f would leave the normal range: f and the values are first multiplied by
// a power of two, 2^120 or 2^-110. f, subnormal or not, stays exact so. A value that overflows is 2^100 factors or more,
// the largest code; one that is rounded is below 2^-100 factors, code zero.
struct Factor {
  float f, inv, scale;
};
__device__ __forceinline__ Factor factor_of(float f) {
  const float scale = f <= 0x1p-100f ? 0x1p120f : f >= 0x1p100f ? 0x1p-110f : 1.0f;
  return {f * scale, 1.0f / (f * scale), scale};
}

// Four bf16 values as codes, each quotient rounded to odd first.
__device__ __noinline__ uint32_t quantise4_exact(uint32_t lo, uint32_t hi, float f, float inv, float scale) {
  float x[4] = {__uint_as_float(lo << 16), __uint_as_float(lo & 0xffff0000u), __uint_as_float(hi << 16),
                __uint_as_float(hi & 0xffff0000u)};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = quotient_odd(x[i] * scale, f, inv);
  return e4m3x4(x[0], x[1], x[2], x[3]);
}

// The same. x * (1 / f) is within two last places of the quotient, so its code is the quotient's unless a tie of two
// codes lies that near: the 20 bits that a normal code drops within two of 0x80000. Those, and values below the normal
// codes, whose ties lie elsewhere, go the exact way. (All values that way: 27 us for 15523 tokens of 8 heads of 128,
// bound by its 14 instructions a value; a correctly truncated division for each: 58 us.)
__device__ __forceinline__ uint32_t quantise4(uint32_t lo, uint32_t hi, const Factor& s) {
  const float x[4] = {__uint_as_float(lo << 16), __uint_as_float(lo & 0xffff0000u), __uint_as_float(hi << 16),
                      __uint_as_float(hi & 0xffff0000u)};
  float q[4];
  bool exact = s.scale != 1.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    q[i] = x[i] * s.inv;
    exact |= ((__float_as_uint(q[i]) - 0x7FFFEu) & 0xFFFFFu) <= 4u || fabsf(q[i]) < 0x1p-6f;
  }
  return exact ? quantise4_exact(lo, hi, s.f, s.inv, s.scale) : e4m3x4(q[0], q[1], q[2], q[3]);
}

// 32 bytes of a row (16 elements) at a time per thread; keys in grid.y 0, values
// in 1. Neighbouring threads take neighbouring pieces of one token, so reads and
// writes are whole rows of a head. LOOP: a thread takes several pieces, the next
// on its way while one is converted (E4M3 only: the conversion is what a load
// can hide behind). 15523 tokens of 8 heads of 128 to E4M3: a piece per thread
// 20.3 us, a loop over three, four or six blocks per SM 20.4, 18.5 and 19.0 us
// (5.2 TB/s); bf16 21.2 us (6.0 TB/s), in a loop 22 to 27 us.
constexpr int kStoreBlocks = 4;  // per SM, of keys and of values each, in a loop
constexpr int kStoreLoop = 3;    // pieces per thread from which on it pays (4000 tokens: 5.7 and 6.1 us, 8000 alike)
template <bool FP8, bool LOOP>
__global__ void __launch_bounds__(256) fa_paged_store_kernel(const __grid_constant__ StoreArgs a) {
  const unsigned row_shift = a.d == 64 ? 2u : 3u, per_token = (unsigned)a.Hkv << row_shift;  // pieces of a row, of a token
  const bool value = blockIdx.y != 0;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  Factor f{};
  if constexpr (FP8) f = factor_of(value ? a.descale_v : a.descale_k);
  ptx::grid_release();
  ptx::grid_wait();
  long long t = i <= 0xFFFFFFFFll ? (unsigned)i / per_token : i / per_token;  // (64-bit division takes far longer)
  if (t >= a.T) return;
  unsigned x = (unsigned)(i - t * per_token);
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(value ? a.v : a.k);
  uint8_t* cache = static_cast<uint8_t*>(value ? a.v_cache : a.k_cache);
  int slot;
  uint4 w0, w1;
  auto load = [&] {
    const uint4* s = reinterpret_cast<const uint4*>(src + t * (value ? a.v_stride : a.k_stride) + (long long)x * 16);
    slot = a.slots[t];
    w0 = s[0];
    w1 = s[1];
  };
  auto store = [&](int slot, uint4 w0, uint4 w1, unsigned x) {
    if (slot < 0) return;
    const int page = slot >> a.page_shift;
    if (page >= a.num_pages) {
      atomicOr(a.status, kStatusBadLength);
      return;
    }
    const unsigned h = x >> row_shift, c = x & ((1u << row_shift) - 1u);
    const long long row = (((long long)page * a.Hkv + h) << a.page_shift) + (slot & ((1 << a.page_shift) - 1));
    const long long at = row * a.d + c * 16;
    if constexpr (FP8) {
      *reinterpret_cast<uint4*>(cache + at) = make_uint4(quantise4(w0.x, w0.y, f), quantise4(w0.z, w0.w, f),
                                                         quantise4(w1.x, w1.y, f), quantise4(w1.z, w1.w, f));
    } else {
      uint4* d = reinterpret_cast<uint4*>(cache + at * 2);
      d[0] = w0;
      d[1] = w1;
    }
  };
  load();
  if constexpr (LOOP) {
    for (;;) {
      const int slot_now = slot;
      const uint4 u0 = w0, u1 = w1;
      const unsigned x_now = x;
      t += a.step_tokens;
      x += (unsigned)a.step_pieces;
      if (x >= per_token) {
        x -= per_token;
        ++t;
      }
      const bool more = t < a.T;
      if (more) load();
      store(slot_now, u0, u1, x_now);
      if (!more) return;
    }
  } else {
    store(slot, w0, w1, x);
  }
}

}  // namespace

cudaError_t launch_plan(const PlanArgs& args, int num_sms, cudaStream_t stream) {
  PlanArgs a = args;
  // a warp per request where there are few, and several slices of the tokens
  // where the rows outnumber the requests by far
  const int groups = std::max(1, std::min((a.R + 7) / 8, 2 * num_sms));
  a.group = (a.R + groups - 1) / groups;
  const int n = (a.R + a.group - 1) / a.group;
  const int slices = std::max(1, std::min(2 * num_sms / n, (a.T / a.R + 255) / 256));
  return launch_dependent(fa_paged_plan_kernel, dim3((unsigned)n, (unsigned)slices), kPlanThreads, 0, stream, a);
}

cudaError_t launch_store(const StoreArgs& args, int num_sms, cudaStream_t stream) {
  StoreArgs a = args;
  const int per_token = a.Hkv * (a.d / 16), resident = kStoreBlocks * num_sms;
  const long long blocks = ((long long)a.T * per_token + 255) / 256;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  const bool loop = a.fp8 && blocks > kStoreLoop * resident;
  a.step_tokens = resident * 256 / per_token;  // from one piece of a thread to its next
  a.step_pieces = resident * 256 % per_token;
  return launch_dependent(!a.fp8 ? fa_paged_store_kernel<false, false>
                          : loop ? fa_paged_store_kernel<true, true>
                                 : fa_paged_store_kernel<true, false>,
                          dim3(loop ? (unsigned)resident : (unsigned)blocks, 2u), 256, 0, stream, a);
}

}  // namespace fa
