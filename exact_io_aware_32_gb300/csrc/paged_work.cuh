// How the work of one paged attention call is cut up, on the device, from the
// requests' lengths.
//
// A tile is the new tokens [i tpt, (i + 1) tpt) of one request with the query
// heads of one key head; it streams the 128-key blocks its last token sees.
// The tiles stand in a row (request, key head, token tile), each as long as
// the keys it sees plus a fixed part for its prologue and epilogue, and the
// row is cut into one equal range per CTA. So a decoding batch of any lengths
// and a long prompt alike end at about the same time on every SM. A cut inside a tile falls on a
// block border; the parts of a cut tile are joined by a second kernel. Every
// CTA works out its own range from prefix sums over the requests (a few KB
// that all read through L2), so no kernel has to run before.
#pragma once
#include <cstdint>

#include "fa_internal.h"
#include "paged.h"
#include "ptx.cuh"

namespace fa {
namespace paged {

// Fixed part of a tile, in keys: what a CTA spends between two tiles (the last products, the epilogue, the next tile's Q
// and first product) is about the time of two key blocks. Without it a CTA whose range holds a hundred requests of one
// token each took 320 us beside others of 20.
constexpr int kTileCost = 256;
constexpr long long kMinRange = 256;    // the shortest range worth a CTA: two blocks

struct Request {
  int start, n, len;  // packed rows [start, start + n), keys [0, len)
};

// What memory says of request r.
struct RawRequest {
  int s0, s1, l;
};
__device__ __forceinline__ RawRequest load_request(const PagedArgs& a, int r) {
  return {__ldg(a.query_start + r), __ldg(a.query_start + r + 1), __ldg(a.seq_lens + r)};
}
// The request as the call takes it; bad: something was out of range.
__device__ __forceinline__ Request request(const PagedArgs& a, const RawRequest& raw, bool& bad) {
  Request q;
  const int s0 = raw.s0, s1 = raw.s1, l = raw.l;
  q.start = min(max(s0, 0), a.T);
  q.n = min(max(s1, q.start), a.T) - q.start;
  q.len = min(max(l, 0), a.max_keys);
  bad = q.start != s0 || q.start + q.n != s1 || q.len != l;
  if (q.n < a.n_min || q.n > a.n_max) q.n = 0;  // the other kernel's
  return q;
}

__device__ __forceinline__ Request request(const PagedArgs& a, int r, bool& bad) {
  return request(a, load_request(a, r), bad);
}

// Keys that the tokens before 'upto' (of the request's n) see.
__device__ __forceinline__ int keys_seen(const PagedArgs& a, const Request& q, int upto) {
  return a.causal ? max(q.len - q.n + min(upto, q.n), 0) : q.len;
}

// Length of tile i in the row of tiles, without its fixed part.
__device__ __forceinline__ long long tile_keys(const PagedArgs& a, const Request& q, int i) {
  return a.causal ? (long long)max(q.len - q.n, 0) + min((long long)q.n, (long long)(i + 1) * a.tpt) : q.len;
}
// The same summed over tiles 0 .. i - 1 of a request of nt tiles.
__device__ __forceinline__ long long keys_before(const PagedArgs& a, const Request& q, int i, int nt) {
  if (!a.causal) return (long long)i * q.len;
  const long long whole = min(i, nt - 1);  // tiles of tpt tokens; the last one may have fewer
  return (long long)i * max(q.len - q.n, 0) + a.tpt * (whole * (whole + 1) / 2) + (i == nt ? q.n : 0);
}

// A part of a tile for this CTA: key blocks [jb, je) of nb.
struct Piece {
  Request q;
  int r, h, tok;  // request, key head, first token
  int jb, je, nb;
  __device__ __forceinline__ bool whole() const { return jb == 0 && je == nb; }
};

struct Range {
  long long p0, p1;    // this CTA's range of the row of tiles
  long long per;       // length of a range
  long long pos, len;  // the tile that holds p0: where it begins, and its length
  int i, nt;           // its number of its request's nt tiles
  int some, use;       // whether the range holds anything, and whether that tile's part of it is a piece
  Piece first;         // that part
};

// a / b for non-negative a, in 32 bits where that is enough (64-bit division takes several times as long).
__device__ __forceinline__ long long divide(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (unsigned)a / (unsigned)b;
  return a / b;
}

// Where a cut x keys past a tile's fixed part falls: the nearest block border, or the tile's end where fewer than a.snap
// blocks would be left on that side.
__device__ __forceinline__ int border(const PagedArgs& a, long long x, int nb) {
  const long long b = (x - kTileCost + 64) >> 7;
  return b < a.snap ? 0 : b > nb - a.snap ? nb : (int)b;
}

// The part of tile i of request q, at pos and len long, that lies in [p0, p1): p.jb, p.je, p.nb; whether it is a piece.
// A tile of at most a.whole blocks is not cut but goes to the CTA that holds its middle (one that sees no key: its
// beginning).
__device__ __forceinline__ bool cut(const PagedArgs& a, const Request& q, int i, long long pos, long long len, long long p0,
                                    long long p1, Piece& p) {
  p.q = q;
  p.tok = i * a.tpt;
  p.nb = (keys_seen(a, q, p.tok + a.tpt) + 127) >> 7;
  if (p.nb <= a.whole) {
    p.jb = 0;
    p.je = p.nb;
    const long long at = p.nb ? pos + (len >> 1) : pos;
    return p0 <= at && at < p1;
  }
  p.jb = p0 <= pos ? 0 : border(a, p0 - pos, p.nb);
  p.je = p1 >= pos + len ? p.nb : border(a, p1 - pos, p.nb);
  return p.jb < p.je;
}

// This CTA's range, by all NT threads of the block. What was set up in shared
// memory before is there after. Up to 32 * kWarpRequests requests are one warp's
// work, the others wait: every instruction here counts once per warp that runs
// it, and all warps working it out took 1500 cycles more.
constexpr int kWarpRequests = 8;
template <int NT>
__device__ __forceinline__ void find_range(const PagedArgs& a, Range& out, long long (&s_sum)[2][NT / 32]) {
  constexpr int kWarps = NT / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool alone = a.R <= 32 * kWarpRequests;  // by the first warp
  ptx::grid_wait();  // nothing before this has read or written what other kernels do
  ptx::grid_release();
  if (!alone || warp == 0) {
    const int threads = alone ? 32 : NT;
    const int seg = (a.R + threads - 1) / threads, r0 = min(a.R, tid * seg), r1 = min(a.R, r0 + seg);
    long long keys = 0, tiles = 0;  // of this thread's requests
    bool any_bad = false;
    Request first{};
    for (int r = r0; r < r1; ++r) {
      bool bad;
      const Request q = request(a, r, bad);
      if (r == r0) first = q;
      any_bad |= bad;
      const int nt = (q.n + a.tpt - 1) / a.tpt;
      keys += a.Hkv * keys_before(a, q, nt, nt);
      tiles += (long long)a.Hkv * nt;
    }
    if (any_bad && blockIdx.x == 0) atomicOr(a.status, kStatusBadLength);
    long long ik = keys, it = tiles;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, ik, s), y = __shfl_up_sync(0xffffffffu, it, s);
      if (lane >= s) {
        ik += x;
        it += y;
      }
    }
    long long all_k = __shfl_sync(0xffffffffu, ik, 31), all_t = __shfl_sync(0xffffffffu, it, 31);
    long long k0 = ik - keys, t0 = it - tiles;
    if (!alone) {
      if (lane == 31) {
        s_sum[0][warp] = ik;
        s_sum[1][warp] = it;
      }
      __syncthreads();
      all_k = all_t = 0;
#pragma unroll 1
      for (int w = 0; w < kWarps; ++w) {
        const long long x = s_sum[0][w], y = s_sum[1][w];
        if (w < warp) {
          k0 += x;
          t0 += y;
        }
        all_k += x;
        all_t += y;
      }
    }
    const long long ctas = gridDim.x;
    const long long total = all_k + kTileCost * all_t;
    const long long per = max(kMinRange, divide(total + ctas - 1, ctas));
    const long long p0 = per * blockIdx.x, p1 = min(total, p0 + per);
    if (tid == 0 && p0 >= total) out.some = 0;
    long long pos = k0 + kTileCost * t0;
    if (p0 < total && pos <= p0 && p0 < pos + keys + kTileCost * tiles) {  // one thread holds p0
      Request q = first;
      for (int r = r0;;) {
        const int nt = (q.n + a.tpt - 1) / a.tpt;
        const long long head = keys_before(a, q, nt, nt) + (long long)kTileCost * nt;
        if (p0 >= pos + a.Hkv * head) {
          pos += a.Hkv * head;
          bool bad;
          q = request(a, ++r, bad);
          continue;
        }
        const int h = (int)divide(p0 - pos, head);
        pos += h * head;
        int lo = 0, hi = nt;  // the last tile that begins at or before p0
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (keys_before(a, q, mid, nt) + (long long)kTileCost * mid <= p0 - pos)
            lo = mid;
          else
            hi = mid;
        }
        pos += keys_before(a, q, lo, nt) + (long long)kTileCost * lo;
        Range g;
        g.p0 = p0;
        g.p1 = p1;
        g.per = per;
        g.pos = pos;
        g.len = tile_keys(a, q, lo) + kTileCost;
        g.i = lo;
        g.nt = nt;
        g.some = 1;
        g.use = cut(a, q, lo, pos, g.len, p0, p1, g.first);
        g.first.r = r;
        g.first.h = h;
        out = g;
        break;
      }
    }
  }
  __syncthreads();
}

// Walks a range's pieces in order; every warp role walks the same ones:
// for (bool more = walk.begin(a, range, p); more; more = walk.step(a, p)).
struct Walk {
  Request q;
  RawRequest next;           // the request after q, loaded ahead and not looked at before it is needed
  long long p0, p1, pos;     // pos: where the next tile begins
  long long last, last_len;  // the tile of the last step
  int r, h, i, nt;
  bool first;  // the range's first tile has not been left yet

  __device__ __forceinline__ void ahead(const PagedArgs& a) { next = load_request(a, min(r + 1, a.R - 1)); }
  __device__ __forceinline__ void advance(const PagedArgs& a, long long len) {
    last = pos;
    last_len = len;
    pos += len;
    if (++i < nt) return;
    i = 0;
    if (++h < a.Hkv) return;
    h = 0;
    do {
      if (++r >= a.R) {
        p1 = pos;  // past the last request
        return;
      }
      bool bad;
      q = request(a, next, bad);
      ahead(a);
    } while (q.n == 0);
    nt = (q.n + a.tpt - 1) / a.tpt;
  }
  __device__ __forceinline__ bool begin(const PagedArgs& a, const Range& g, Piece& p) {
    p = g.first;
    p0 = g.p0;
    p1 = g.p1;
    pos = last = g.pos;
    last_len = g.len;
    q = p.q;
    r = p.r;
    h = p.h;
    i = g.i;
    nt = g.nt;
    first = true;
    return g.use ? true : step(a, p);
  }
  __device__ __forceinline__ bool step(const PagedArgs& a, Piece& p) {
    if (first) {  // put off until here: the first piece's copies do not wait for it
      first = false;
      ahead(a);
      advance(a, last_len);
    }
    while (pos < p1) {
      const long long len = tile_keys(a, q, i) + kTileCost;
      p.r = r;
      p.h = h;
      const bool use = cut(a, q, i, pos, len, p0, p1, p);
      advance(a, len);
      if (use) return true;
    }
    return false;
  }
  // The CTA that ends the tile of the last step, which this one opened: the last
  // whose range begins inside the tile and, its cut rounded to a block, before its last block's end.
  __device__ __forceinline__ int ender(const PagedArgs& a, long long per, const Piece& p) const {
    long long z = divide(last + last_len - 1, per);
    while (border(a, z * per - last, p.nb) >= p.nb) --z;
    return (int)z;
  }
};

// What a CTA tells the joining kernel: whether its first piece continues a tile
// that CTAs before it began (lead) and ends it, and whether its last piece
// begins a tile that later CTAs end (open), with that tile.
struct Parts {
  int lead, lead_ends, open;
  int end;               // the CTA that ends the open tile
  int start, n, tok, h;  // the open tile: its request's rows, first token, key head
};

}  // namespace paged
}  // namespace fa
