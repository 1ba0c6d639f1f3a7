// Forward attention with a sliding window and a few first keys that stay visible
// (sinks), grouped heads, on sm_103a.
//
// Row i of a sequence stands at p = i + sk - sq and sees key j iff j <= p and
// (p - j < window or j < sinks). Per 128-row tile that leaves the key blocks of
// its rows' windows, and before them the blocks of the sinks: a tile of any
// text length streams (window + 127) / 128 + 1 blocks or so, five or nine where
// the causal forward streams hundreds. What a tile costs besides (its Q, the first S,
// reading O out) counts accordingly, so the CTAs are persistent as in fa_fwd_persist.cu:
// the rings and barriers count on across tiles, and the next tile's loads and
// first products run beside this one's epilogue. S = Q K^T, the softmax with one TMEM lane per row
// and O += P V with P from TMEM are those of fa_fwd.cu.
//
// d = 128: a CTA has two tiles at a time, which share the key blocks: two query heads
// of one key head on the same rows (or, without grouped heads, two
// neighbouring row blocks, whose bands differ by a block at either end: each
// skips the one that it does not see). d = 64: one tile per CTA and two CTAs per
// SM, P in TMEM columns of its own.
//
// Every block but those where a window begins or ends (and a sink block beyond its sinks) is
// unmasked: its row maximum comes with the TMEM load.
//
// Bound by a block's chain of S, softmax and P V (about 2950 cycles for the blocks of
// two tiles, 2048 of them products) and, where windows are short, by what a tile costs besides: 16384
// tokens, 32 heads over 8 of 128, window 4096, 4 sinks 669 us in a CUDA graph, 1440 TFLOP/s of the
// pairs seen, 693 to 730 us as calls one after another; 4 x 4096 tokens, window 512, 150 to 169 us from
// run to run (860 to 760 TFLOP/s; of the blocks' keys a fifth is hidden), with 4 sinks 160 to 163 us;
// 8 x 4096 at d = 64 198 to 213 us (650 to 605). Issuing both tiles' first S of the next item before this one's last
// products cost more than it gave (158 and 162 us, window 4096 692 and 721 us): what stands
// in the MMA warp's way delays every block.
//
// P enters P V as bf16, as in fa_fwd.cu: the product takes both operands in V's type, and a
// second one with P's remainder would add 1024 cycles to a block of two tiles. The errors of
// a row's weights are independent, so o is off by 0.0021 to 0.0022 (relative RMS) where its own rounding to
// bf16 leaves 0.0016. Scores, maxima, sums and O are fp32.
//
// Warp roles: a softmax warpgroup per tile, the TMA warp, the MMA warp; two tiles: a warp that stores O.
#include <algorithm>

#include "fa_internal.h"
#include "paged.h"
#include "ptx.cuh"

namespace fa {
namespace {

using namespace fa::ptx;

constexpr float kLn2 = 0.693147180559945309417f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units, as in fa_fwd.cu

template <int D_>
struct WCfg {
  static constexpr int D = D_;
  static constexpr int kTiles = D == 64 ? 1 : 2;
  static constexpr int kCtasPerSm = 3 - kTiles;
  static constexpr int kPanels = D / 64, kPanelBytes = 128 * 128, kTileBytes = kPanels * kPanelBytes;
  // V is read last, so it gets the deeper ring; with two tiles its third place is where their O are staged in turn
  static constexpr int kKStages = 2, kVStages = kTiles == 2 ? 2 : 3;
  // Q: a slot per tile, or two for one tile, so that the next one's is there when this one ends (each also stages its tile's O)
  static constexpr int kOffQ = 0, kOffK = 2 * kTileBytes, kOffV = kOffK + kKStages * kTileBytes;
  static constexpr int kOffO = kOffV + kVStages * kTileBytes, kOffBar = kOffO + (kTiles == 2 ? kTileBytes : 0);
  // No alignment slack (two CTAs share an SM's 228 KB): the kernel checks that shared memory starts on 1024 bytes.
  static constexpr int kSmemBytes = kOffBar + 640;
  static_assert(kSmemBytes <= 232448 && (kCtasPerSm == 1 || 2 * (kSmemBytes + 1024) <= 233472), "shared memory");
  static constexpr uint32_t kTmemCols = kTiles == 2 ? 512u : 256u;
  // S (fp32, 128 columns), P (bf16 pairs, 64 columns: over S, or in columns of its own) and O (fp32, D columns) of tile t
  __host__ __device__ static constexpr uint32_t col_s(int t) { return (uint32_t)t * 128u; }
  __host__ __device__ static constexpr uint32_t col_p(int t) { return kTiles == 2 ? col_s(t) : 128u; }
  __host__ __device__ static constexpr uint32_t col_o(int t) { return kTiles == 2 ? 256u + (uint32_t)t * D : 192u; }
  // two tiles: a warp that stores their staged O (one tile: the TMA warp does)
  static constexpr int kWarpTma = 4 * kTiles, kWarpMma = 4 * kTiles + 1, kWarpStore = 4 * kTiles + 2;
  static constexpr int kThreads = 128 * kTiles + 64 + (kTiles == 2 ? 32 : 0);
};

struct WBars {
  uint64_t q_full[2][2], q_free[2];  // by tile (q_full: and its items in turn); one tile: q_full by its items in turn
  uint64_t k_full[2], k_empty[2], v_full[3], v_empty[3];
  uint64_t s_full[2], p_full[2], o_done[2], o_free[2];  // (one tile: o_done follows every P V)
  uint64_t s_free;                                      // one tile: S is in registers
  // two tiles: a panel of O has been staged; tile t may stage a panel (the O staged there before has been read by its store);
  // one tile: O has been staged in its Q's slot
  uint64_t o_staged[2], o_place[2][2];
  uint64_t teardown;
  uint64_t item_full[4], item_empty[4];
  int4 items[4][4];
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(WBars) <= 640, "barriers exceed their shared memory");

// The last sinks' block costs as much as any other, six blocks instead of five with a window of 512, unless it is known to
// be thin: with at most kThin sinks in it only so many keys are loaded, columns of S and keys of P V worked on.
constexpr int kThin = kThinRows;

// What a CTA works on at a time: up to two tiles of 128 rows of one key head, and the key blocks that they stream:
// block j of the first 'sunk' ones, then block j + skip.
struct Item {
  int bhk;              // batch and key head; < 0: past the last item
  int head[2], row[2];  // query head, first row
  int nb[2];            // blocks up to the last one that the tile sees (0: padding rows, or no tile)
  int sunk, skip;
  int miss;             // a block that the second tile does not see (its window begins one later)
  int thin;             // a block of which only the first 32 keys, sinks, can be seen
  int sq, off;
  bool there[2];        // the tile has rows of the array
  __device__ __forceinline__ int at(int j) const { return j < sunk ? j : j + skip; }
  __device__ __forceinline__ bool uses(int t, int j) const { return j < nb[t] && (t == 0 || j != miss); }
};

// The i-th item of this CTA. Items are dealt in rounds of one per CTA, odd rounds in reverse: a head's later rows, with whole
// windows, first.
template <int kTiles>
__device__ __forceinline__ Item item(const WindowArgs& a, int i) {
  Item x;
  const int ctas = (int)gridDim.x, c = (int)blockIdx.x;
  const long long L = (long long)i * ctas + ((i & 1) ? ctas - 1 - c : c);
  x.bhk = -1;
  if (L >= a.items) return x;
  const int per = a.items_per_head, G = a.group, tiles = G * ((a.Nq + 127) / 128);
  x.bhk = (int)L / per;
  const int u0 = kTiles * (per - 1 - ((int)L - x.bhk * per));
  int sk;
  seq_lens(a.seqlens_q, a.seqlens_k, x.bhk / a.Hkv, a.Nq, a.Nk, true, x.sq, sk);
  x.off = sk - x.sq;
  int low[2] = {0, 0};
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int u = u0 + t, blk = u / G;
    x.there[t] = t < kTiles && u < tiles;
    x.head[t] = x.bhk * G + u - blk * G;
    x.row[t] = blk * 128;
    low[t] = max(x.row[t] + x.off - a.window + 1, 0) >> 7;
    x.nb[t] = x.there[t] && x.row[t] < x.sq ? ((min(x.row[t] + 127, x.sq - 1) + x.off) >> 7) + 1 : 0;
  }
  const int sunk = (a.sinks + 127) >> 7;  // blocks that hold sinks
  x.sunk = min(sunk, low[0]);
  x.skip = low[0] - x.sunk;
  x.miss = low[1] > low[0] && low[0] >= sunk ? x.sunk : -1;
  x.thin = x.sunk == sunk && sunk > 0 && a.sinks - 128 * (sunk - 1) <= kThin ? sunk - 1 : -1;
#pragma unroll
  for (int t = 0; t < 2; ++t) x.nb[t] = max(x.nb[t] - x.skip, 0);
  return x;
}

// The items of a CTA, worked out by its loading warp and told to the others (a step's divisions took every softmax thread
// 1400 cycles between two items).
constexpr int kItemRing = 4;
__device__ __forceinline__ bool tell(WBars& bars, int n, const Item& x, int lane, volatile int* abort_flag) {
  const int s = n % kItemRing;
  if (!warp_wait(&bars.item_empty[s], ((n / kItemRing) & 1) ^ 1, abort_flag)) return false;
  if (lane == 0) {
    bars.items[s][0] = make_int4(x.bhk, x.head[0], x.head[1], x.row[0]);
    bars.items[s][1] = make_int4(x.row[1], x.nb[0], x.nb[1], x.sunk);
    bars.items[s][2] = make_int4(x.skip, x.miss, x.thin, x.sq);
    bars.items[s][3] = make_int4(x.off, x.there[0], x.there[1], 0);
    mbar_arrive(&bars.item_full[s]);
  }
  __syncwarp();
  return true;
}
// The n-th item; past the last one, and when the wait runs out, bhk < 0.
__device__ __forceinline__ Item hear(WBars& bars, int n, int lane, volatile int* abort_flag) {
  const int s = n % kItemRing;
  Item x;
  x.bhk = -1;
  if (!warp_wait(&bars.item_full[s], (n / kItemRing) & 1, abort_flag)) return x;
  const int4 a = bars.items[s][0], b = bars.items[s][1], c = bars.items[s][2], d = bars.items[s][3];
  __syncwarp();
  if (lane == 0) mbar_arrive(&bars.item_empty[s]);
  x.bhk = a.x;
  x.head[0] = a.y;
  x.head[1] = a.z;
  x.row[0] = a.w;
  x.row[1] = b.x;
  x.nb[0] = b.y;
  x.nb[1] = b.z;
  x.sunk = b.w;
  x.skip = c.x;
  x.miss = c.y;
  x.thin = c.z;
  x.sq = c.w;
  x.off = d.x;
  x.there[0] = d.y != 0;
  x.there[1] = d.z != 0;
  return x;
}

template <int D>
__global__ void __launch_bounds__(WCfg<D>::kThreads, WCfg<D>::kCtasPerSm)
    fa_fwd_window_kernel(const __grid_constant__ WindowArgs a) {
  using C = WCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw;
  if (smem_u32(smem) & 1023u) {  // uniform over the CTA: every thread leaves before any barrier
    if (threadIdx.x == 0) atomicOr(a.status, 16u);
    return;
  }
  WBars& bars = *reinterpret_cast<WBars*>(smem + C::kOffBar);
  volatile int* abort_flag = &bars.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == C::kWarpTma && elect_one()) {
    tma_prefetch_desc(&a.tm_q);
    tma_prefetch_desc(&a.tm_k);
    tma_prefetch_desc(&a.tm_v);
  }
  if (threadIdx.x == 0) {
    bars.abort = 0;
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars.q_full[s][0], 1);
      mbar_init(&bars.q_full[s][1], 1);
      mbar_init(&bars.q_free[s], 1);
      mbar_init(&bars.s_full[s], 1);
      mbar_init(&bars.p_full[s], 128);
      mbar_init(&bars.o_done[s], 1);
      mbar_init(&bars.o_free[s], 128);
    }
    for (int s = 0; s < C::kKStages; ++s) {
      mbar_init(&bars.k_full[s], 1);
      mbar_init(&bars.k_empty[s], 1);
    }
    for (int s = 0; s < C::kVStages; ++s) {
      mbar_init(&bars.v_full[s], 1);
      mbar_init(&bars.v_empty[s], 1);
    }
    mbar_init(&bars.s_free, 128);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars.o_staged[s], 128);
      mbar_init(&bars.o_place[s][0], 1);
      mbar_init(&bars.o_place[s][1], 1);
    }
    for (int s = 0; s < kItemRing; ++s) {
      mbar_init(&bars.item_full[s], 1);
      mbar_init(&bars.item_empty[s], 4 * C::kTiles + (C::kTiles == 2 ? 2 : 1));  // softmax, MMA and store warps
    }
    mbar_init(&bars.teardown, 1);
    fence_mbar_init();
  }
  if (warp == C::kWarpMma) {
    tmem_alloc(&bars.tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;
  grid_release();
  grid_wait();  // nothing before this has read or written what other kernels do
  if (a.seqlens_q || a.seqlens_k)  // the CTAs check the lengths among themselves
    for (int b = blockIdx.x * C::kThreads + threadIdx.x; b < a.B; b += gridDim.x * C::kThreads) {
      int sq, sk;
      if (seq_lens(a.seqlens_q, a.seqlens_k, b, a.Nq, a.Nk, true, sq, sk)) atomicOr(a.status, kStatusBadLength);
    }

  if (warp == C::kWarpTma) {
    // ------------------------------------------------------------ TMA producer
    int g = 0, nk = 0, nv = 0, nq[2] = {0, 0};  // key blocks, and loads issued
    bool ok = true;
    // test hook: without the first Q tile, the MMA warp's first wait expires
    bool withhold = a.test_fault == 1;
    int rows[2] = {0, 0}, heads[2] = {0, 0}, stored = 0;  // one tile: of the last two items, and those whose O has been stored
    auto store_o = [&]() -> bool {  // of the item 'stored', from its Q's slot
      const int s = stored & 1;
      if (!warp_wait(&bars.o_staged[s], (stored >> 1) & 1, abort_flag)) return false;
      if (elect_one()) {
        if (!*abort_flag) {
          tma_store_3d(&a.tm_o, smem + C::kOffQ + s * C::kTileBytes, 0, s ? rows[1] : rows[0], s ? heads[1] : heads[0]);
          bulk_commit();
        }
        bulk_wait_read0();
      }
      __syncwarp();
      ++stored;
      return true;
    };
    auto load_q = [&](int t, int row, int head) -> bool {
      const int s = C::kTiles == 2 ? t : nq[t] & 1;  // the slot: tile t's own, or the two in turn
      if (C::kTiles == 2) {
        if (!warp_wait(&bars.q_free[s], (nq[t] & 1) ^ 1, abort_flag)) return false;
      } else {
        if (nq[0] >= 2 && !store_o()) return false;
        if (s) {
          rows[1] = row;
          heads[1] = head;
        } else {
          rows[0] = row;
          heads[0] = head;
        }
      }
      if (!withhold) {
        if (elect_one()) {
          uint64_t* bar = &bars.q_full[t][nq[t] & 1];
          mbar_arrive_expect_tx(bar, C::kTileBytes);
          for (int pn = 0; pn < C::kPanels; ++pn)
            tma_load_3d(smem + C::kOffQ + s * C::kTileBytes + pn * C::kPanelBytes, &a.tm_q, bar, pn * 64, row, head);
        }
        __syncwarp();
        ++nq[t];
      }
      withhold = false;
      return true;
    };
    auto load = [&](const CUtensorMap* tm, uint8_t* dst, uint64_t* bar, int row, int head, bool thin) {
      if (elect_one()) {
        mbar_arrive_expect_tx(bar, thin ? C::kTileBytes * kThin / 128 : C::kTileBytes);
        for (int pn = 0; pn < C::kPanels; ++pn) tma_load_3d(dst + pn * C::kPanelBytes, tm, bar, pn * 64, row, head);
      }
      __syncwarp();
    };
    for (int i = 0; ok; ++i) {
      const Item x = item<C::kTiles>(a, i);
      if (!(ok = tell(bars, i, x, lane, abort_flag)) || x.bhk < 0) break;
      const int n = max(x.nb[0], x.nb[1]);
      if (x.nb[0] > 0 && !(ok = load_q(0, x.row[0], x.head[0]))) break;
      for (int j = 0; j < n; ++j, ++g) {
        const int ks = g % C::kKStages, vs = g % C::kVStages, row = x.at(j) * 128;
        if (!(ok = warp_wait(&bars.k_empty[ks], ((g / C::kKStages) & 1) ^ 1, abort_flag))) break;
        const bool thin = j == x.thin;
        load(thin ? &a.tm_k_thin : &a.tm_k, smem + C::kOffK + ks * C::kTileBytes, &bars.k_full[ks], row, x.bhk, thin);
        nk = g + 1;
        if (C::kTiles == 2 && j == 0 && x.nb[1] > 0 && !(ok = load_q(1, x.row[1], x.head[1]))) break;
        if (!(ok = warp_wait(&bars.v_empty[vs], ((g / C::kVStages) & 1) ^ 1, abort_flag))) break;
        load(thin ? &a.tm_v_thin : &a.tm_v, smem + C::kOffV + vs * C::kTileBytes, &bars.v_full[vs], row, x.bhk, thin);
        nv = g + 1;
      }
    }
    if (C::kTiles == 1)
      while (ok && stored < nq[0]) ok = store_o();
    // Let every issued copy land before the CTA can exit (an earlier load's slot was refilled only after its reader
    // completed, so it has landed).
    for (int t = 0; t < C::kTiles; ++t)
      for (int last = max(0, nq[t] - 2); last < nq[t]; ++last) mbar_wait_drain(&bars.q_full[t][last & 1], (last >> 1) & 1);
    for (int s = max(0, nk - C::kKStages); s < nk; ++s)
      mbar_wait_drain(&bars.k_full[s % C::kKStages], (s / C::kKStages) & 1);
    for (int s = max(0, nv - C::kVStages); s < nv; ++s)
      mbar_wait_drain(&bars.v_full[s % C::kVStages], (s / C::kVStages) & 1);
  } else if (warp == C::kWarpMma) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t kIdS = idesc_bf16(128, 128, false, false);  // Q, K both K-major
    constexpr uint32_t kIdThin = idesc_bf16(128, kThin, false, false);
    constexpr uint32_t kIdO = idesc_bf16(128, D, false, true);     // P from TMEM, V MN-major
    const uint64_t dq0 = sdesc_sw128(smem_u32(smem + C::kOffQ), 16, 1024);
    const uint64_t dk0 = sdesc_sw128(smem_u32(smem + C::kOffK), 16, 1024);
    const uint64_t dv0 = sdesc_sw128(smem_u32(smem + C::kOffV), C::kPanelBytes, 1024);
    auto issue_s = [&](int t, int qs, int ks, bool thin, bool last) {  // by the elected lane
      const uint32_t id = thin ? kIdThin : kIdS;
      const uint32_t qo = (uint32_t)(qs * C::kTileBytes) >> 4, ko = (uint32_t)(ks * C::kTileBytes) >> 4;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {  // each k-step reads 32 bytes of every row
        const uint32_t o = ((kk >> 2) * C::kPanelBytes + (kk & 3) * 32) >> 4;
        mma_ss(tmem + C::col_s(t), dq0 + qo + o, dk0 + ko + o, id, kk > 0);
      }
      mma_commit(&bars.s_full[t]);
      // the tile's last product to read Q (one tile: its slot is free once O, staged there, has been stored)
      if (C::kTiles == 2 && last) mma_commit(&bars.q_free[qs]);
    };
    auto issue_pv = [&](int t, int vs, bool thin, bool first) {
      const uint32_t vo = (uint32_t)(vs * C::kTileBytes) >> 4;
#pragma unroll
      for (int kk = 0; kk < kThin / 16; ++kk)  // P columns [8 kk, 8 kk + 8), V rows [16 kk, 16 kk + 16)
        mma_ts(tmem + C::col_o(t), tmem + C::col_p(t) + kk * 8, dv0 + vo + kk * ((16 * 128) >> 4), kIdO,
               (!first || kk > 0) ? 1u : 0u);
      if (thin) return;
#pragma unroll
      for (int kk = kThin / 16; kk < 8; ++kk)
        mma_ts(tmem + C::col_o(t), tmem + C::col_p(t) + kk * 8, dv0 + vo + kk * ((16 * 128) >> 4), kIdO,
               (!first || kk > 0) ? 1u : 0u);
    };
    int g = 0, nq[2] = {0, 0}, np[2] = {0, 0};  // key blocks; items and P blocks of each tile so far
    bool ok = true;
    for (int i = 0; ok; ++i) {
      const Item x = hear(bars, i, lane, abort_flag);
      if (x.bhk < 0) break;
      const int n = max(x.nb[0], x.nb[1]);
      if (n == 0) continue;
      // S of the first block
      ok = warp_wait(&bars.k_full[g % C::kKStages], (g / C::kKStages) & 1, abort_flag);
      if (C::kTiles == 1 && ok) ok = warp_wait(&bars.s_free, (g & 1) ^ 1, abort_flag);
      for (int t = 0; t < C::kTiles && ok; ++t)
        if (x.nb[t] > 0) {
          if (!(ok = warp_wait(&bars.q_full[t][nq[t] & 1], (nq[t] >> 1) & 1, abort_flag))) break;
          tc_fence_after();
          if (x.uses(t, 0)) {
            if (elect_one()) issue_s(t, C::kTiles == 2 ? t : nq[0] & 1, g % C::kKStages, x.thin == 0, x.nb[t] == 1);
            __syncwarp();
          }
        }
      if (!ok) break;
      if (elect_one()) mma_commit(&bars.k_empty[g % C::kKStages]);
      __syncwarp();
      if constexpr (C::kTiles == 2) {
        // Per key block j and tile t: O_t += P_t V_j, then at once S_t for block j + 1 (its columns are P_t's, which the
        // products of one thread have read by then, as they execute in issue order).
        bool begun[2] = {false, false};  // whether O_t holds anything of this item
        for (int j = 0; j < n; ++j, ++g) {
          const int s = g % C::kVStages;
          const uint32_t ph = (g / C::kVStages) & 1;
          const int v_last = x.uses(1, j) ? 1 : 0;  // the tile whose PV reads V_j last
          const int jn = j + 1, sn = (g + 1) % C::kKStages;
          const bool k_next = jn < n, u0 = x.uses(0, j);
          ok = warp_wait3(&bars.v_full[s], ph, u0 ? &bars.p_full[0] : &bars.v_full[s], u0 ? (np[0] & 1) : ph,
                          k_next ? &bars.k_full[sn] : &bars.v_full[s], k_next ? ((g + 1) / C::kKStages) & 1 : ph, abort_flag);
          if (!ok) break;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (x.uses(t, j)) {
              if (t == 1 && !(ok = warp_wait(&bars.p_full[1], np[1] & 1, abort_flag))) break;
              // an item's first PV overwrites O: the tile before has been read out
              if (!begun[t] && !(ok = warp_wait(&bars.o_free[t], (nq[t] & 1) ^ 1, abort_flag))) break;
              tc_fence_after();
              if (elect_one()) {
                issue_pv(t, s, j == x.thin, !begun[t]);
                if (j == x.nb[t] - 1) mma_commit(&bars.o_done[t]);
                if (t == v_last) mma_commit(&bars.v_empty[s]);
              }
              __syncwarp();
              begun[t] = true;
              ++np[t];
            }
            if (x.uses(t, jn)) {
              if (elect_one()) issue_s(t, t, sn, jn == x.thin, jn == x.nb[t] - 1);
              __syncwarp();
            }
          }
          if (!ok) break;
          if (k_next) {
            if (elect_one()) mma_commit(&bars.k_empty[sn]);
            __syncwarp();
          }
        }
      } else {
        // Per key block: S of the tile's next block as soon as the softmax has this one's in registers, then O += P V.
        for (int j = 0; j < n; ++j, ++g) {
          if (j + 1 < n) {
            const int sn = (g + 1) % C::kKStages;
            ok = warp_wait2(&bars.s_free, g & 1, &bars.k_full[sn], ((g + 1) / C::kKStages) & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              issue_s(0, nq[0] & 1, sn, j + 1 == x.thin, j + 2 == n);
              mma_commit(&bars.k_empty[sn]);
            }
            __syncwarp();
          }
          const int s = g % C::kVStages;
          ok = warp_wait2(&bars.p_full[0], g & 1, &bars.v_full[s], (g / C::kVStages) & 1, abort_flag);
          if (ok && j == 0) ok = warp_wait(&bars.o_free[0], (nq[0] & 1) ^ 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            issue_pv(0, s, j == x.thin, j == 0);
            mma_commit(&bars.o_done[0]);
            mma_commit(&bars.v_empty[s]);
          }
          __syncwarp();
        }
      }
      for (int t = 0; t < 2; ++t) nq[t] += x.nb[t] > 0;
    }
    if (elect_one()) mma_commit(&bars.teardown);
    __syncwarp();
    mbar_wait_drain(&bars.teardown, 0);
  } else if (C::kTiles == 2 && warp == C::kWarpStore) {
    // ------------------------------------------------------------ stores of staged O, a panel at a time
    // Both tiles stage in one place, in the items' order. It is given to them by this warp, which knows that order and waits
    // for the reads before, over a barrier of each tile's own: a tile waits for each of its phases in turn. (One barrier for
    // both, told after every read, would be waited for by parity two phases on by a tile that staged two O ago, and the
    // phase of that O still open looks like the one after it complete.)
    int n = 0;  // O stored so far
    bool ok = true;
    for (int i = 0; ok; ++i) {
      const Item x = hear(bars, i, lane, abort_flag);
      if (x.bhk < 0) break;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (x.nb[t] == 0) continue;
        if (elect_one()) {
          bulk_wait_read1();  // the first panel has been read; the writes finish on their own
          mbar_arrive(&bars.o_place[t][0]);
          bulk_wait_read0();
          mbar_arrive(&bars.o_place[t][1]);
        }
        __syncwarp();
#pragma unroll
        for (int pn = 0; pn < C::kPanels; ++pn) {
          if (!(ok = warp_wait(&bars.o_staged[pn], n & 1, abort_flag))) break;
          if (elect_one()) {
            tma_store_3d(&a.tm_o, smem + C::kOffO + pn * C::kPanelBytes, pn * 64, x.row[t], x.head[t]);
            bulk_commit();
          }
          __syncwarp();
        }
        if (!ok) break;
        ++n;
      }
    }
    if (elect_one()) bulk_wait_read0();
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax + epilogue
    const int t = warp >> 2;
    const int r = (warp & 3) * 32 + lane;  // row within the tile = TMEM lane
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lane_off + C::col_s(t);
    const uint32_t t_p = tmem + lane_off + C::col_p(t);
    const uint32_t t_o = tmem + lane_off + C::col_o(t);
    const float sl2 = a.scale_log2;
    int np = 0, nq = 0;  // blocks and items of this tile so far
    bool ok = true;
    for (int i = 0; ok; ++i) {
      const Item x = hear(bars, i, lane, abort_flag);
      if (x.bhk < 0) break;
      if (!(t ? x.there[1] : x.there[0])) continue;
      const int row0 = t ? x.row[1] : x.row[0], row = row0 + r, p = row + x.off;  // p: the row's position
      const int nb = t ? x.nb[1] : x.nb[0], head = t ? x.head[1] : x.head[0], miss = t ? x.miss : -1;
      const int p_last = row0 + 127 + x.off;
      float m_ref = -INFINITY;  // exponent reference, log2 units of scaled scores
      float l_sum = 0.f;        // sum of 2^(s * sl2 - m_ref) over the keys seen so far
      bool begun = false;       // whether O holds anything
      for (int j = 0; j < nb; ++j) {
        if (j == miss) continue;
        ok = __all_sync(0xffffffffu, mbar_wait(&bars.s_full[t], np & 1, abort_flag));
        if (!ok) break;
        tc_fence_after();
        // S_t, with the maximum of each 32 columns from the load itself
        uint32_t sr[4][32];
        float cmax[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32_max(t_s + c * 32, sr[c], cmax[c]);
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_wait(sr[c], cmax[c]);
        if constexpr (C::kTiles == 1) {
          tc_fence_before();
          mbar_arrive(&bars.s_free);  // S is in registers: the next block's S may overwrite it
        }
        const bool thin = j == x.thin;
        // Masked: blocks that reach past the first row's position (keys past sk are past every row's) and those with keys
        // behind the last row's window that are not all sinks.
        const int kv0 = x.at(j) * 128;
        float mx = fmax3(fmax3(cmax[0], cmax[1], cmax[2]), cmax[3], -INFINITY);
        if (thin) {  // the sinks alone, which every row sees
          const uint32_t keep = first_bits(a.sinks - kv0);
          float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int q = 0; q < 32; ++q) {
            if (!(keep >> q & 1u)) sr[0][q] = __float_as_uint(-INFINITY);
            m[q & 3] = fmaxf(m[q & 3], __uint_as_float(sr[0][q]));
          }
          mx = fmaxf(fmax3(m[0], m[1], m[2]), m[3]);
        } else if (kv0 + 127 > row0 + x.off || (p_last - kv0 >= a.window && kv0 + 128 > a.sinks)) {
          // column c iff c <= lim and (c > out or c < sunk)
          const int lim = p - kv0, out = lim - a.window, sunk = a.sinks - kv0;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t keep = first_bits(lim + 1 - 32 * c) & ~(first_bits(out + 1 - 32 * c) & ~first_bits(sunk - 32 * c));
#pragma unroll
            for (int q = 0; q < 32; ++q)
              if (!(keep >> q & 1u)) sr[c][q] = __float_as_uint(-INFINITY);
          }
          float mxc[8];  // row maximum over eight chains of 16 scores, then a tree
#pragma unroll
          for (int q = 0; q < 8; ++q)
            mxc[q] = fmaxf(__uint_as_float(sr[0][2 * q]), __uint_as_float(sr[0][2 * q + 1]));
#pragma unroll
          for (int c = 16; c < 128; c += 16)
#pragma unroll
            for (int q = 0; q < 8; ++q)
              mxc[q] = fmax3(mxc[q], __uint_as_float(sr[c >> 5][(c & 31) + 2 * q]),
                             __uint_as_float(sr[c >> 5][(c & 31) + 2 * q + 1]));
          mx = fmax3(fmax3(mxc[0], mxc[1], mxc[2]), fmax3(mxc[3], mxc[4], mxc[5]), fmaxf(mxc[6], mxc[7]));
        }
        float alpha = 1.f;
        const float m_new = fmaxf(m_ref, mx * sl2);
        const bool move = m_new > m_ref + kRescaleThreshold;
        if (move) {
          alpha = ex2(m_ref - m_new);
          m_ref = m_new;
        }
        const bool rescale = __any_sync(0xffffffffu, move && begun);
        float2 sum4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const float m_use = m_ref == -INFINITY ? 0.f : m_ref;  // a row that has seen no key yet: P = 0
        const float2 scale2 = make_float2(sl2, sl2), shift2 = make_float2(-m_use, -m_use);
        auto chunk = [&](int ch) {  // P of 32 keys as bf16 pairs, packed in place (pair c / 2 into word c / 2, already read)
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float2 y =
                ffma2(make_float2(__uint_as_float(sr[ch][c]), __uint_as_float(sr[ch][c + 1])), scale2, shift2);
            const float2 e = make_float2(ex2(y.x), ex2(y.y));
            sum4[(c >> 1) & 3] = fadd2(sum4[(c >> 1) & 3], e);
            sr[ch][c >> 1] = pack_bf16x2(e.x, e.y);
          }
        };
        auto store = [&](int ch) {
          uint32_t pk[16];
#pragma unroll
          for (int q = 0; q < 16; ++q) pk[q] = sr[ch][q];
          tmem_st16(t_p + 16 * ch, pk);
        };
        chunk(0);
        if constexpr (C::kTiles == 2) {
          store(0);
          if (!thin) chunk(1);
        } else {
          // P and O are free once the P V before this one has completed (an item's first block: the epilogue waited)
          if (!thin) chunk(1);
          if (begun) {
            ok = __all_sync(0xffffffffu, mbar_wait(&bars.o_done[0], (np - 1) & 1, abort_flag));
            if (!ok) break;
            tc_fence_after();
          }
          store(0);
        }
        if (!thin) {
          store(1);
          chunk(2);
          store(2);
          chunk(3);
          store(3);
        }
        const float2 sum = fadd2(fadd2(sum4[0], sum4[1]), fadd2(sum4[2], sum4[3]));
        l_sum = l_sum * alpha + (sum.x + sum.y);
        if (rescale) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld32(t_o + c, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int q = 0; q < 32; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * alpha);
            tmem_st32(t_o + c, o);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bars.p_full[t]);
        begun = true;
        ++np;
      }
      if (ok && nb > 0) ok = mbar_wait(&bars.o_done[t], (C::kTiles == 2 ? nq : np - 1) & 1, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const bool valid = row < a.Nq, real = row < x.sq;  // a padding row: o = 0
      const long long at = (long long)head * a.Nq + row;
      if (nb > 0) {
        // O, normalised, as bf16 into the staging place (rows of 128 swizzled bytes a panel), a panel at a time
        tc_fence_after();
        const float inv = 1.f / l_sum;
#pragma unroll 1
        for (int pn = 0; pn < C::kPanels; ++pn) {
          uint8_t* stage = smem + (C::kTiles == 2 ? C::kOffO : C::kOffQ + (nq & 1) * C::kTileBytes) + pn * C::kPanelBytes;
          if (C::kTiles == 2) {
            ok = __all_sync(0xffffffffu, mbar_wait(&bars.o_place[t][pn], nq & 1, abort_flag));
            if (!ok) break;
          }
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
            uint32_t o[32];
            tmem_ld32(t_o + pn * 64 + c, o);
            tmem_ld_wait(o);
            if (c == 32 && pn + 1 == C::kPanels) {
              tc_fence_before();
              mbar_arrive(&bars.o_free[t]);  // O is in registers: the next item may accumulate there
            }
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) {
              uint32_t w[4];
#pragma unroll
              for (int q = 0; q < 4; ++q)
                w[q] = real ? pack_bf16x2(__uint_as_float(o[8 * q4 + 2 * q]) * inv, __uint_as_float(o[8 * q4 + 2 * q + 1]) * inv)
                            : 0u;
              st_shared_v4(smem_u32(stage + r * 128 + (((c / 8 + q4) ^ (r & 7)) << 4)), w[0], w[1], w[2], w[3]);
            }
          }
          fence_proxy_async_smem();
          mbar_arrive(&bars.o_staged[C::kTiles == 2 ? pn : nq & 1]);
        }
        if (!ok) break;
        ++nq;
      } else if (valid) {
        uint4* orow = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.o) + at * (D * 2));
        for (int c = 0; c < D / 8; ++c) orow[c] = make_uint4(0u, 0u, 0u, 0u);
      }
      if (valid) a.lse[at] = real ? (m_ref + log2f(l_sum)) * kLn2 : -INFINITY;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kWarpMma) tmem_dealloc(tmem, C::kTmemCols);
  if (threadIdx.x == 0 && bars.abort) atomicOr(a.status, 1u);
}

template <int D>
cudaError_t launch(WindowArgs a, int num_sms, cudaStream_t stream) {
  using C = WCfg<D>;
  const int tiles = a.group * ((a.Nq + 127) / 128);
  a.items_per_head = (tiles + C::kTiles - 1) / C::kTiles;
  a.items = (long long)a.B * a.Hkv * a.items_per_head;
  static std::atomic<unsigned long long> done;  // devices (a bit each) that know the kernel's shared memory
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(fa_fwd_window_kernel<D>), C::kSmemBytes, done);
  if (e != cudaSuccess) return e;
  const unsigned ctas = (unsigned)std::min<long long>(a.items, (long long)num_sms * C::kCtasPerSm);
  return launch_dependent(fa_fwd_window_kernel<D>, dim3(ctas), C::kThreads, C::kSmemBytes, stream, a);
}

}  // namespace

cudaError_t launch_fwd_window(const WindowArgs& a, int num_sms, cudaStream_t stream) {
  return a.d == 64 ? launch<64>(a, num_sms, stream) : launch<128>(a, num_sms, stream);
}

}  // namespace fa
