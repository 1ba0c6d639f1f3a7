// How the work of one paged attention call is cut up, on the device, from the
// requests' lengths.
//
// A tile is the new tokens [i tpt, (i + 1) tpt) of one request with the query
// heads of one key head; it streams the 128-key blocks its last token sees.
// The tiles stand in a row (request, key head, token tile), each as long as
// the blocks it streams plus a fixed part for its prologue and epilogue, and
// the row is cut into one equal range per CTA. So a decoding batch of any lengths
// and a long prompt alike end at about the same time on every SM. A cut inside a
// tile falls on a block border; the parts of a cut tile are joined by a second
// kernel. (Tiles of at most a.whole blocks stay whole, and loads are as uneven as
// they are: eight prompts of up to 1024 tokens, 12 heads of 64, leave the fullest
// of 304 CTAs 19 blocks of work for 12 on average.) Every CTA works out its own
// range from prefix sums over the requests (a few KB that all read through L2),
// so no kernel has to run before. Places in the row are blocks in 32 bits (the
// host refuses calls of 2^31 blocks), since this is latency that every call
// pays: in 64 bits, by keys, the first copy went out 2500 cycles later. What the
// host counts holds for requests that share no rows; the sum here saturates, and
// a row of tiles longer than that is not walked.
#pragma once
#include <cstdint>

#include "fa_internal.h"
#include "paged.h"
#include "ptx.cuh"

namespace fa {
namespace paged {

// Fixed part of a tile, in blocks: what a CTA spends between two tiles (the last products, the epilogue, the next tile's
// Q and first product) is about the time of two key blocks. Without it a CTA whose range holds a hundred requests of one
// token each took 320 us beside others of 20.
constexpr int kTileCost = 2;
constexpr int kMinRange = 2;  // the shortest range worth a CTA

struct Request {
  int start, n, len;  // packed rows [start, start + n), keys [0, len)
};

// What memory says of request r.
struct RawRequest {
  int s0, s1, l;
};
__device__ __forceinline__ RawRequest load_request(const PagedArgs& a, int r) {
  return {a.query_start[r], a.query_start[r + 1], a.seq_lens[r]};
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
__host__ __device__ __forceinline__ int keys_seen(const PagedArgs& a, const Request& q, int upto) {
  return a.causal ? max(q.len - q.n + min(upto, q.n), 0) : q.len;
}

// Length of the first i of a request's nt tiles (for one key head): the keys that their last tokens see, summed and then
// taken as blocks, and the fixed parts. Where the first tokens see no key it counts more than they see, up to the request's
// keys for each tile. (Exact sums, with a division for such requests, cost the others too: one short request 10.2 us,
// with this 9.9 us.)
__host__ __device__ __forceinline__ int tiles_len(const PagedArgs& a, const Request& q, int i, int nt) {
  long long keys = (long long)i * q.len;
  if (a.causal) {
    const int whole = min(i, nt - 1);  // tiles of tpt tokens; the last one may have fewer
    const long long seen =
        (long long)i * max(q.len - q.n, 0) + (long long)whole * (whole + 1) / 2 * a.tpt + (i == nt ? q.n : 0);
    keys = min(keys, seen);  // (the sum is the smaller one unless the first tokens see no key)
  }
  return (int)(keys >> 7) + kTileCost * i;
}
// (two lengths or sums of them; INT_MAX: too many to count)
__host__ __device__ __forceinline__ int add_len(int x, int y) {
  return (int)min((unsigned)x + (unsigned)y, 0x7FFFFFFFu);
}
__host__ __device__ __forceinline__ int tiles_of(const PagedArgs& a, const Request& q) { return (q.n + a.tpt - 1) / a.tpt; }

// A part of a tile for this CTA: key blocks [jb, je) of nb.
struct Piece {
  Request q;
  int r, h, tok;  // request, key head, first token
  int jb, je, nb;
  __device__ __forceinline__ bool whole() const { return jb == 0 && je == nb; }
};

struct Range {
  int p0, p1;     // this CTA's range of the row of tiles
  int per;        // length of a range
  int head, len;  // the tile that holds p0: where its request's tiles of its key head begin; its length
  int pos;        // where it begins
  int i, nt;      // its number of those nt tiles
  int some, use;  // whether the range holds anything, and whether that tile's part of it is a piece
  Piece first;    // that part
};

// Where a cut x blocks past a tile's beginning falls: a block border, or the tile's end where fewer than a.snap blocks
// would be left on that side.
__device__ __forceinline__ int border(const PagedArgs& a, int x, int nb) {
  const int b = x - kTileCost;
  return b < a.snap || b < 0 ? 0 : b > nb - a.snap ? nb : b;
}

// The part of tile i of request q, at pos and len long, that lies in [p0, p1): p.jb, p.je, p.nb; whether it is a piece.
// A tile of at most a.whole blocks is not cut but goes to the CTA that holds its middle (one that sees no key: its
// beginning).
__device__ __forceinline__ bool cut(const PagedArgs& a, const Request& q, int i, int pos, int len, int p0, int p1,
                                    Piece& p) {
  p.q = q;
  p.tok = i * a.tpt;
  p.nb = (keys_seen(a, q, p.tok + a.tpt) + 127) >> 7;
  if (p.nb <= a.whole) {
    p.jb = 0;
    p.je = p.nb;
    const int at = p.nb ? pos + (len >> 1) : pos;
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
__device__ __forceinline__ void find_range(const PagedArgs& a, Range& out, int (&s_sum)[NT / 32]) {
  constexpr int kWarps = NT / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool alone = a.R <= 32 * kWarpRequests;  // by the first warp
  ptx::grid_wait();  // nothing before this has read or written what other kernels do
  ptx::grid_release();
  if (!alone || warp == 0) {
    const int threads = alone ? 32 : NT;
    const int seg = (a.R + threads - 1) / threads, r0 = min(a.R, tid * seg), r1 = min(a.R, r0 + seg);
    int mine = 0;  // length of this thread's requests
    bool any_bad = false;
    Request first{};
    for (int r = r0; r < r1; ++r) {
      bool bad;
      const Request q = request(a, r, bad);
      if (r == r0) first = q;
      any_bad |= bad;
      const int nt = tiles_of(a, q);
      if (nt) mine = add_len(mine, a.Hkv * tiles_len(a, q, nt, nt));
    }
    int upto = mine;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, s);
      if (lane >= s) upto = add_len(upto, x);
    }
    int total = __shfl_sync(0xffffffffu, upto, 31), pos = upto - mine;
    if (!alone) {
      if (lane == 31) s_sum[warp] = upto;
      __syncthreads();
      total = 0;
#pragma unroll 1
      for (int w = 0; w < kWarps; ++w) {
        const int x = s_sum[w];
        if (w < warp) pos = add_len(pos, x);
        total = add_len(total, x);
      }
    }
    if (total > a.most) {  // requests that share rows: nobody's range holds anything
      total = 0;
      any_bad = true;
    }
    if (any_bad && blockIdx.x == 0) atomicOr(a.status, kStatusBadLength);
    const int ctas = (int)gridDim.x, per = max(kMinRange, (int)(((unsigned)total + ctas - 1) / (unsigned)ctas));
    const long long at = (long long)per * blockIdx.x;
    const int p0 = (int)min(at, (long long)total), p1 = (int)min(at + per, (long long)total);
    if (tid == 0 && p0 >= total) out.some = 0;
    if (p0 < total && pos <= p0 && p0 < pos + mine) {  // one thread holds p0
      Request q = first;
      for (int r = r0;;) {
        const int nt = tiles_of(a, q), head = nt ? tiles_len(a, q, nt, nt) : 0;
        if (p0 >= pos + a.Hkv * head) {
          pos += a.Hkv * head;
          bool bad;
          q = request(a, ++r, bad);
          continue;
        }
        const int h = a.Hkv == 1 ? 0 : (int)((unsigned)(p0 - pos) / (unsigned)head);
        pos += h * head;
        int lo = 0, hi = nt;  // the last tile that begins at or before p0
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (tiles_len(a, q, mid, nt) <= p0 - pos)
            lo = mid;
          else
            hi = mid;
        }
        Range g;
        g.p0 = p0;
        g.p1 = p1;
        g.per = per;
        g.head = pos;
        g.pos = pos + tiles_len(a, q, lo, nt);
        g.len = pos + tiles_len(a, q, lo + 1, nt) - g.pos;
        g.i = lo;
        g.nt = nt;
        g.some = 1;
        g.use = cut(a, q, lo, g.pos, g.len, p0, p1, g.first);
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
  RawRequest next;         // the request after q, loaded ahead and not looked at before it is needed
  int p0, p1, head, pos;   // head: where the tiles of this key head begin; pos: the next tile
  int last, last_len;      // the tile of the last step
  int r, h, i, nt;
  bool first;  // the range's first tile has not been left yet

  __device__ __forceinline__ void ahead(const PagedArgs& a) { next = load_request(a, min(r + 1, a.R - 1)); }
  __device__ __forceinline__ void advance(const PagedArgs& a, int len) {
    last = pos;
    last_len = len;
    pos += len;
    if (++i < nt) return;
    i = 0;
    head = pos;
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
    nt = tiles_of(a, q);
  }
  __device__ __forceinline__ void begin(const Range& g) {
    const Piece& p = g.first;
    p0 = g.p0;
    p1 = g.p1;
    head = g.head;
    pos = last = g.pos;
    last_len = g.len;
    q = p.q;
    r = p.r;
    h = p.h;
    i = g.i;
    nt = g.nt;
    first = true;
  }
  __device__ __forceinline__ bool begin(const PagedArgs& a, const Range& g, Piece& p) {
    begin(g);
    p = g.first;
    return g.use ? true : step(a, p);
  }
  // kOne: most requests are one tile per key head.
  template <bool kOne = false>
  __device__ __forceinline__ bool step(const PagedArgs& a, Piece& p) {
    if (first) {  // put off until here: the first piece's copies do not wait for it
      first = false;
      ahead(a);
      advance(a, last_len);
    }
    while (pos < p1) {
      const bool again = kOne && nt == 1 && p.r == r;  // the same tile of the next key head
      const int len = again ? last_len : head + tiles_len(a, q, i + 1, nt) - pos;
      p.r = r;
      p.h = h;
      bool use = true;
      if (again && p0 <= pos && pos + len <= p1) {
        p.jb = 0;
        p.je = p.nb;
      } else {
        use = cut(a, q, i, pos, len, p0, p1, p);
      }
      advance(a, len);
      if (use) return true;
    }
    return false;
  }
  // The CTA that ends the tile of the last step, which this one opened: the last
  // whose range begins inside the tile and, its cut taken to a border, before its last block's end.
  __device__ __forceinline__ int ender(const PagedArgs& a, int per, const Piece& p) const {
    int z = (int)((unsigned)(last + last_len - 1) / (unsigned)per);
    while (border(a, z * per - last, p.nb) >= p.nb) --z;
    return z;
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
