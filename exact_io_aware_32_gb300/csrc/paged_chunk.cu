// Attention of chunks of new tokens over the paged cache, on sm_103a.
//
// The blocked loop of fa_fwd.cu (S = Q K^T on tcgen05 into TMEM, softmax with a
// running maximum and one TMEM lane per query row, O += P V with P read back
// from TMEM) with three things of its own:
//   - a tile's 128 rows are the new tokens of one request times the query heads
//     that share a key head (row = token * G + head), so grouped heads read
//     each key and value once; one TMA box of 64 x G x tokens fetches them;
//   - a key block's copies come from its pages, one per lane of the loading
//     warp, each at the page that the block table names;
//   - the CTAs are persistent and each runs its range of the row of tiles
//     (paged_work.cuh); the rings and barriers count on across tiles, so the
//     next tile's loads and first products overlap this one's epilogue.
// Rows of O go from registers to global memory, 32 bytes per store: packed
// tokens of neighbouring requests make a tile's rows no rectangle that a
// tensor store could write.
//
// Warp roles: a softmax warpgroup per 128-row half, the TMA warp, the MMA warp,
// and with E4M3 caches two warps that turn value codes into f16 operands (TMA ->
// ring of codes -> converters -> V ring); Q's rows become their two 8-bit parts by
// the softmax threads that own them (by the converters that took 5500 cycles a half).
#include "paged_pipe.cuh"

namespace fa {
namespace {

using namespace fa::ptx;
using namespace fa::paged;

template <int D_, bool FP8_>
struct CCfg {
  static constexpr int D = D_;
  static constexpr bool FP8 = FP8_;
  // At d = 64 bf16 one 128-row tile per CTA and two CTAs per SM, as in fa_fwd.cu;
  // otherwise two halves of 128 rows that share the key blocks.
  static constexpr int kTiles = D == 64 && !FP8 ? 1 : 2;
  static constexpr int kCtasPerSm = 3 - kTiles;
  static constexpr int kPanels = D / 64;
  static constexpr int kTileBytes = kPanels * 16384;  // 128 rows, 16-bit
  static constexpr int kCodeBytes = 128 * D;          // 128 rows of codes
  static constexpr int kKBytes = FP8 ? kCodeBytes : kTileBytes;  // a key block: codes stay codes
  static constexpr int kKStages = FP8 ? 3 : 2, kVStages = (FP8 && D == 128) || kTiles == 1 ? 2 : 3;
  static constexpr int kCStages = FP8 ? 3 : 0;  // value codes on their way to f16
  // Q tiles: one per half, or two for one half, so that the next tile's is there when this one ends
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + 2 * kTileBytes;
  static constexpr int kOffV = kOffK + kKStages * kKBytes;
  static constexpr int kOffC = kOffV + kVStages * kTileBytes;
  static constexpr int kOffBar = kOffC + kCStages * kCodeBytes;
  static constexpr int kSmemBytes = kOffBar + 1024 + 1024;  // barriers, alignment slack
  static_assert(kSmemBytes <= 232448 && (kCtasPerSm == 1 || 2 * (kSmemBytes + 1024) <= 233472), "shared memory");
  static constexpr uint32_t kTmemCols = kTiles == 2 ? 512u : 256u;
  __host__ __device__ static constexpr uint32_t col_s(int t) { return (uint32_t)t * 128u; }
  // P lies over the first 64 columns of its S; with one half in columns of its own, so that S of the next block can be
  // made during the softmax
  __host__ __device__ static constexpr uint32_t col_p(int t) { return kTiles == 2 ? col_s(t) : 128u; }
  __host__ __device__ static constexpr uint32_t col_o(int t) { return kTiles == 2 ? 256u + (uint32_t)t * D : 192u; }
  static constexpr int kWarpTma = 4 * kTiles, kWarpMma = 4 * kTiles + 1;
  // With FP8 two converter warps: more than 384 threads leave a softmax thread, which holds 128 scores, no more than 128
  // registers. (Four of them and a warp for the values' copies, with S loaded twice: chunks of prompts at d = 128 333 us;
  // with S held once and spilled 433 us.)
  static constexpr int kWarpConv = 4 * kTiles + 2, kConvWarps = 2;
  static constexpr int kThreads = 128 * kTiles + 64 + (FP8 ? 32 * kConvWarps : 0);
};

struct CBars {
  uint64_t q_raw[2], q_full[2][2], q_free[2];  // by half (q_full: and tile in turn); E4M3 caches: Q as loaded, as converted
  uint64_t k_full[3], k_empty[3], v_full[3], v_empty[3], c_full[3], c_empty[3];
  uint64_t s_full[2], p_full[2], o_done[2], o_free[2];  // (one half: o_done follows every P V)
  uint64_t s_free;                                      // one half: S is in registers
  uint64_t teardown;
  PieceRing ring;
  uint32_t tmem_base;
  int abort;
  Range range;
  int sums[16];
};
static_assert(sizeof(CBars) <= 1024, "barriers exceed their shared memory");

// Key blocks that each 128-row half sees of a piece (nb[t] from p.jb on).
template <int kTiles, bool WIN>
__device__ __forceinline__ void half_blocks(const PagedArgs& a, const Piece& p, int (&nb)[2]) {
  const int gap = WIN ? band_of(a, p.q, p.tok).gap : 0;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int tok = p.tok + t * a.tpt1;
    const int blocks = t < kTiles && tok < p.q.n ? (max(keys_seen(a, p.q, tok + a.tpt1) - gap, 0) + 127) >> 7 : 0;
    nb[t] = max(0, min(blocks, p.je) - p.jb);
  }
}

// WIN (with CAUSAL): a token sees its last a.window keys and the first a.sinks; keys are counted without a tile's gap (Band),
// which is that of both halves (the second's window begins a block later at most once in 128 / tpt1 tiles).
template <int D, bool FP8, bool CAUSAL, bool WIN = false>
__global__ void __launch_bounds__(CCfg<D, FP8>::kThreads, CCfg<D, FP8>::kCtasPerSm)
    fa_paged_chunk_kernel(const __grid_constant__ PagedArgs a) {
  using C = CCfg<D, FP8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  CBars& bars = *reinterpret_cast<CBars*>(smem + C::kOffBar);
  volatile int* abort_flag = &bars.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // Everything that does not depend on the lengths first; the range's barriers cover it.
  if (warp == C::kWarpTma && elect_one()) {
    tma_prefetch_desc(&a.tm_q);
    tma_prefetch_desc(&a.tm_k);
    tma_prefetch_desc(&a.tm_v);
  }
  if (threadIdx.x == 32) {
    bars.abort = 0;
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars.q_raw[s], 1);
      mbar_init(&bars.q_full[s][0], FP8 ? 4 : 1);
      mbar_init(&bars.q_full[s][1], FP8 ? 4 : 1);
      mbar_init(&bars.q_free[s], 1);
      mbar_init(&bars.s_full[s], 1);
      mbar_init(&bars.p_full[s], 128);
      mbar_init(&bars.o_done[s], 1);
      mbar_init(&bars.o_free[s], 128);
    }
    for (int s = 0; s < 3; ++s) {
      mbar_init(&bars.k_full[s], 1);
      mbar_init(&bars.k_empty[s], 1);
      mbar_init(&bars.v_full[s], FP8 ? C::kConvWarps : 1);
      mbar_init(&bars.v_empty[s], 1);
      mbar_init(&bars.c_full[s], 1);
      mbar_init(&bars.c_empty[s], C::kConvWarps);
    }
    mbar_init(&bars.s_free, 128);
    mbar_init(&bars.teardown, 1);
    bars.ring.init(4 * C::kTiles + 1 + (FP8 ? C::kConvWarps : 0));  // softmax, MMA and converter warps
    fence_mbar_init();
  }
  if (warp == C::kWarpMma) {
    tmem_alloc(&bars.tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  find_range<C::kThreads, WIN>(a, bars.range, reinterpret_cast<int(&)[C::kThreads / 32]>(bars.sums));
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;
  if (!bars.range.some) {  // uniform: nothing has been issued
    if (warp == C::kWarpMma) tmem_dealloc(tmem, C::kTmemCols);
    if (threadIdx.x == 0) static_cast<Parts*>(a.parts)[blockIdx.x] = Parts{};
    return;
  }
  PieceReader in(bars.ring, abort_flag, lane);
  Piece p = bars.range.first;
  const bool first = bars.range.use;  // the first piece is there already
  int blocks[2];                      // key blocks that each half sees of it
  half_blocks<C::kTiles, WIN>(a, p, blocks);
  auto next_piece = [&] {
    const bool there = in.next(p);
    blocks[0] = in.x;
    blocks[1] = in.y;
    return there;
  };

  if (warp == C::kWarpTma) {
    // ------------------------------------------------------------ TMA producer
    const uint32_t q_bytes = (uint32_t)(a.Hq / a.Hkv * a.tpt1 * D * 2);
    constexpr int kS = FP8 ? C::kCStages : C::kVStages;  // values, or their codes
    uint64_t *v_full = FP8 ? bars.c_full : bars.v_full, *v_empty = FP8 ? bars.c_empty : bars.v_empty;
    Parts parts{};
    int g = 0, nk = 0, nv = 0, nq[2] = {0, 0};  // key blocks, and loads issued
    bool ok = true;
    // test hook: without the first Q tile, the MMA warp's first wait expires
    bool withhold = a.test_fault == 1;
    auto load_q = [&](int t) {
      // the slot and its uses so far: half t's own, or the two in turn
      const int s = C::kTiles == 2 ? t : nq[t] & 1, use = C::kTiles == 2 ? nq[t] : nq[t] >> 1;
      if (!(ok = warp_wait(&bars.q_free[s], (use & 1) ^ 1, abort_flag))) return;
      if (!withhold) {
        if (elect_one()) {
          uint64_t* bar = FP8 ? &bars.q_raw[t] : &bars.q_full[t][nq[t] & 1];
          mbar_arrive_expect_tx(bar, q_bytes);
          for (int pn = 0; pn < C::kPanels; ++pn)
            tma_load_3d(smem + C::kOffQ + s * C::kTileBytes + pn * 16384, &a.tm_q, bar, pn * 64,
                        p.h * (a.Hq / a.Hkv), p.q.start + p.tok + t * a.tpt1);
        }
        __syncwarp();
        ++nq[t];
      }
      withhold = false;
    };
    Walk<WIN> walk;
    walk.begin(bars.range);
    Piece next = p;
    int next_nb[2] = {blocks[0], blocks[1]}, told = 0;
    bool more = true;
    auto step = [&] {  // works out the next piece and tells the others
      more = walk.step(a, next);
      half_blocks<C::kTiles, WIN>(a, next, next_nb);
      ok = bars.ring.tell(told++, next, more, next_nb[0], next_nb[1], lane, abort_flag);
    };
    if (!first) step();
    while (ok && more) {
      p = next;
      blocks[0] = next_nb[0];
      blocks[1] = next_nb[1];
      note_piece(a, parts, p, walk, bars.range.per);
      const int nbm = max(blocks[0], blocks[1]);
      Pages<WIN> pages;
      Band band{};
      if (WIN) band = band_of(a, p.q, p.tok);
      if (nbm > 0) pages.begin(a, p, band, lane);
      if (blocks[0] > 0) load_q(0);
      for (int j = 0; ok && j < max(nbm, 1); ++j) {
        if (nbm > 0) {
          const int jj = p.jb + j, page_now = pages.of(a, p, jj, lane);
          const int sk = g % C::kKStages;
          if (!(ok = warp_wait(&bars.k_empty[sk], ((g / C::kKStages) & 1) ^ 1, abort_flag))) break;
          load_block<D, FP8, WIN>(a, p, jj, page_now, lane, &a.tm_k, smem + C::kOffK + sk * C::kKBytes, &bars.k_full[sk],
                                  p.q.len - band.gap, band.low);
          nk = g + 1;
          if (C::kTiles == 2 && j == 0 && blocks[1] > 0) {
            load_q(1);
            if (!ok) break;
          }
          const int sv = g % kS;
          if (!(ok = warp_wait(&v_empty[sv], ((g / kS) & 1) ^ 1, abort_flag))) break;
          load_block<D, FP8, WIN>(a, p, jj, page_now, lane, &a.tm_v,
                                  smem + (FP8 ? C::kOffC + sv * C::kCodeBytes : C::kOffV + sv * C::kTileBytes), &v_full[sv],
                                  p.q.len - band.gap, band.low);
          nv = ++g;
        }
        if (j == 0) step();  // while those are on their way
      }
    }
    if (lane == 0) static_cast<Parts*>(a.parts)[blockIdx.x] = parts;
    // Let every issued copy land before the CTA can exit (an earlier load's slot
    // was refilled only after its reader completed, so it has landed).
    for (int t = 0; t < C::kTiles; ++t)
      for (int last = max(0, nq[t] - (C::kTiles == 2 ? 1 : 2)); last < nq[t]; ++last) {
        mbar_wait_drain(FP8 ? &bars.q_raw[t] : &bars.q_full[t][last & 1], FP8 ? last & 1 : (last >> 1) & 1);
      }
    for (int x = max(0, nk - C::kKStages); x < nk; ++x)
      mbar_wait_drain(&bars.k_full[x % C::kKStages], (x / C::kKStages) & 1);
    for (int x = max(0, nv - kS); x < nv; ++x) mbar_wait_drain(&v_full[x % kS], (x / kS) & 1);
  } else if (warp == C::kWarpMma) {
    // ------------------------------------------------------------ MMA issuer
    // P from TMEM, V MN-major
    constexpr uint32_t kIdO = FP8 ? idesc_f16(128, D, false, true) : idesc_bf16(128, D, false, true);
    const uint64_t dq0 = sdesc_sw128(smem_u32(smem + C::kOffQ), 16, 1024);
    const uint64_t dk0 = desc_keys<D, FP8>(smem + C::kOffK), dv0 = Tile<D>::desc_v(smem + C::kOffV);
    // by the elected lane: S of half t from Q slot qs and key slot st
    auto issue_s = [&](int t, int qs, int st, bool last) {
      issue_qk<D, FP8>(tmem + C::col_s(t), dq0 + ((uint32_t)(qs * C::kTileBytes) >> 4),
                       dk0 + ((uint32_t)(st * C::kKBytes) >> 4));
      mma_commit(&bars.s_full[t]);
      if (last) mma_commit(&bars.q_free[qs]);  // the tile's last product to read Q
    };
    auto issue_pv = [&](int t, int st, int steps, bool first) {
      issue_pv_steps<D>(tmem + C::col_o(t), tmem + C::col_p(t), dv0 + ((uint32_t)(st * C::kTileBytes) >> 4), kIdO, steps,
                        first);
    };
    int g = 0, nq[2] = {0, 0}, np[2] = {0, 0};  // key blocks; tiles and P blocks of each half so far
    bool ok = true;
    for (bool more = first || next_piece(); ok && more; more = next_piece()) {
      const int nbm = max(blocks[0], blocks[1]);
      Band band{};
      if (WIN) band = band_of(a, p.q, p.tok);
      if (nbm > 0) {
        // S of the first block
        ok = warp_wait(&bars.k_full[g % C::kKStages], (g / C::kKStages) & 1, abort_flag);
        if (C::kTiles == 1 && ok) ok = warp_wait(&bars.s_free, (g & 1) ^ 1, abort_flag);
        for (int t = 0; t < C::kTiles && ok; ++t)
          if (blocks[t] > 0) {
            if (!(ok = warp_wait(&bars.q_full[t][nq[t] & 1], (nq[t] >> 1) & 1, abort_flag))) break;
            tc_fence_after();
            if (elect_one()) issue_s(t, C::kTiles == 2 ? t : nq[0] & 1, g % C::kKStages, blocks[t] == 1);
            __syncwarp();
          }
        if (!ok) break;
        if (elect_one()) mma_commit(&bars.k_empty[g % C::kKStages]);
        __syncwarp();
      }
      if constexpr (C::kTiles == 2) {
        // Per key block j and half t: O_t += P_t V_j, then at once S_t for block j + 1 (its columns are P_t's, which the
        // products of one thread have read by then, as they execute in issue order).
        for (int j = 0; j < nbm; ++j, ++g) {
          const int s = g % C::kVStages;
          const uint32_t ph = (g / C::kVStages) & 1;
          const int v_last = j < blocks[1] ? 1 : 0;  // the half whose PV reads V_j last
          const int jn = j + 1, sn = (g + 1) % C::kKStages;
          const bool k_next = jn < nbm;
          ok = warp_wait3(&bars.v_full[s], ph, j < blocks[0] ? &bars.p_full[0] : &bars.v_full[s],
                          j < blocks[0] ? (np[0] & 1) : ph, k_next ? &bars.k_full[sn] : &bars.v_full[s],
                          k_next ? ((g + 1) / C::kKStages) & 1 : ph, abort_flag);
          if (!ok) break;
          const int keys = p.q.len - band.gap - (p.jb + j) * 128, steps = pv_steps(keys);
          if (!FP8 && keys < steps * 16) zero_rows<D>(smem + C::kOffV + s * C::kTileBytes, keys, steps * 16, lane);
          for (int t = 0; t < 2; ++t) {
            if (j < blocks[t]) {
              if (t == 1 && !(ok = warp_wait(&bars.p_full[1], np[1] & 1, abort_flag))) break;
              // a tile's first PV overwrites O: the tile before has been read out
              if (j == 0 && !(ok = warp_wait(&bars.o_free[t], (nq[t] & 1) ^ 1, abort_flag))) break;
              tc_fence_after();
              if (elect_one()) {
                issue_pv(t, s, steps, j == 0);
                if (j == blocks[t] - 1) mma_commit(&bars.o_done[t]);
                if (t == v_last) mma_commit(&bars.v_empty[s]);
              }
              __syncwarp();
              ++np[t];
            }
            if (jn < blocks[t]) {
              if (elect_one()) issue_s(t, t, sn, jn == blocks[t] - 1);
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
        for (int j = 0; j < nbm; ++j, ++g) {
          if (j + 1 < nbm) {
            const int sn = (g + 1) % C::kKStages;
            ok = warp_wait2(&bars.s_free, g & 1, &bars.k_full[sn], ((g + 1) / C::kKStages) & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              issue_s(0, nq[0] & 1, sn, j + 2 == nbm);
              mma_commit(&bars.k_empty[sn]);
            }
            __syncwarp();
          }
          const int s = g % C::kVStages;
          ok = warp_wait2(&bars.p_full[0], g & 1, &bars.v_full[s], (g / C::kVStages) & 1, abort_flag);
          if (ok && j == 0) ok = warp_wait(&bars.o_free[0], (nq[0] & 1) ^ 1, abort_flag);
          if (!ok) break;
          const int keys = p.q.len - band.gap - (p.jb + j) * 128, steps = pv_steps(keys);
          if (keys < steps * 16) zero_rows<D>(smem + C::kOffV + s * C::kTileBytes, keys, steps * 16, lane);
          tc_fence_after();
          if (elect_one()) {
            issue_pv(0, s, steps, j == 0);
            mma_commit(&bars.o_done[0]);
            mma_commit(&bars.v_empty[s]);
          }
          __syncwarp();
        }
      }
      for (int t = 0; t < 2; ++t) nq[t] += blocks[t] > 0;
    }
    if (elect_one()) mma_commit(&bars.teardown);
    __syncwarp();
    mbar_wait_drain(&bars.teardown, 0);
  } else if (FP8 && warp >= C::kWarpConv) {
    // ------------------------------------------------------------ converters
    const int tid = threadIdx.x - C::kWarpConv * 32;
    constexpr int kCS = FP8 ? C::kCStages : 1;
    int g = 0;
    bool ok = true;
    for (bool more = first || next_piece(); ok && more; more = next_piece()) {
      const int nbm = max(blocks[0], blocks[1]);
      Band band{};
      if (WIN) band = band_of(a, p.q, p.tok);
      for (int j = 0; ok && j < nbm; ++j, ++g) {
        const int vs = g % C::kVStages, cs = g % kCS;
        ok = warp_wait2(&bars.c_full[cs], (g / kCS) & 1, &bars.v_empty[vs], ((g / C::kVStages) & 1) ^ 1, abort_flag);
        if (!ok) break;
        convert_tile<D, 32 * C::kConvWarps>(smem + C::kOffC + cs * C::kCodeBytes, smem + C::kOffV + vs * C::kTileBytes,
                                            p.q.len - band.gap - (p.jb + j) * 128, tid);
        conv_arrive(&bars.v_full[vs], &bars.c_empty[cs], lane);
      }
    }
  } else if (warp < 4 * C::kTiles) {
    // ------------------------------------------------------------ softmax + epilogue
    const int t = warp >> 2;
    const int r = (warp & 3) * 32 + lane;  // row within the half = TMEM lane
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lane_off + C::col_s(t);
    const uint32_t t_p = tmem + lane_off + C::col_p(t);
    const uint32_t t_o = tmem + lane_off + C::col_o(t);
    constexpr float kBias = FP8 ? kPBias : 0.f;
    const int G = a.Hq / a.Hkv, rt = r / G, rh = r - rt * G;  // this row's token within the half, and head
    const bool o32 = (reinterpret_cast<uintptr_t>(a.o) & 31u) == 0;
    int np = 0, nq = 0;  // blocks and tiles of this half so far
    bool ok = true;
    for (bool more = first || next_piece(); ok && more; more = next_piece()) {
      const int nb = t ? blocks[1] : blocks[0];
      const int tok0 = p.tok + t * a.tpt1, tok = tok0 + rt;
      Band band{};
      if (WIN) band = band_of(a, p.q, p.tok);
      const int len = p.q.len - band.gap, off = len - p.q.n;  // causal: token i sees keys 0 .. i + off
      const bool valid = rt < a.tpt1 && tok < p.q.n;
      // window: the last key that is behind the window of this half's last token
      const int out_last = WIN ? min(tok0 + a.tpt1, p.q.n) - 1 + off - band.wide : 0;
      float sl2 = a.scale_log2;
      if (FP8 && nb > 0) {  // this thread's row of Q to its two 8-bit parts
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bars.q_raw[t], nq & 1, abort_flag)))) break;
        sl2 *= unscale(convert_row<D>(smem + C::kOffQ + t * C::kTileBytes, r));
        conv_arrive(&bars.q_full[t][nq & 1], nullptr, lane);
      }
      float m_ref = -INFINITY;  // exponent reference, log2 units of scaled scores
      float l_sum = 0.f;        // sum of 2^(s * sl2 - m_ref) over the keys seen so far
      for (int j = 0; j < nb; ++j, ++np) {
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
        float mx = fmax3(fmax3(cmax[0], cmax[1], cmax[2]), cmax[3], -INFINITY);
        // only blocks that reach past the first row's last key, or past the request's, need masking
        const int kv0 = (p.jb + j) * 128;
        if ((CAUSAL && kv0 + 127 > tok0 + off) || kv0 + 128 > len || (WIN && kv0 <= out_last && kv0 + 128 > a.sinks)) {
          const int lim = (CAUSAL ? min(tok + off, len - 1) : len - 1) - kv0;  // keep column c iff c <= lim
          const int out = lim - band.wide, sunk = a.sinks - kv0;  // window: hidden too are columns up to 'out', from 'sunk' on
          if constexpr (WIN) {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              const uint32_t keep =
                  first_bits(lim + 1 - 32 * h) & ~(first_bits(out + 1 - 32 * h) & ~first_bits(sunk - 32 * h));
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!(keep >> c & 1u)) sr[h][c] = __float_as_uint(-INFINITY);
            }
          } else {
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if (c > lim) sr[c >> 5][c & 31] = __float_as_uint(-INFINITY);
          }
          float mxc[8];  // row maximum over eight chains of 16 scores, then a tree
#pragma unroll
          for (int i = 0; i < 8; ++i)
            mxc[i] = fmaxf(__uint_as_float(sr[0][2 * i]), __uint_as_float(sr[0][2 * i + 1]));
#pragma unroll
          for (int c = 16; c < 128; c += 16)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              mxc[i] = fmax3(mxc[i], __uint_as_float(sr[c >> 5][(c & 31) + 2 * i]),
                             __uint_as_float(sr[c >> 5][(c & 31) + 2 * i + 1]));
          mx = fmax3(fmax3(mxc[0], mxc[1], mxc[2]), fmax3(mxc[3], mxc[4], mxc[5]), fmaxf(mxc[6], mxc[7]));
        }
        float alpha = 1.f;
        const float m_new = fmaxf(m_ref, mx * sl2);
        const bool move = m_new > m_ref + kRescaleThreshold;
        if (move) {
          alpha = ex2(m_ref - m_new);
          m_ref = m_new;
        }
        const bool rescale = __any_sync(0xffffffffu, move && j > 0);
        float2 sum4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const float m_use = (m_ref == -INFINITY ? 0.f : m_ref) - kBias;  // a row that has seen no key yet: P = 0
        const float2 scale2 = make_float2(sl2, sl2), shift2 = make_float2(-m_use, -m_use);
        auto chunk = [&](int ch) {  // P of 32 keys as 16-bit pairs, packed in place (pair c / 2 into word c / 2, already read)
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float2 x =
                ffma2(make_float2(__uint_as_float(sr[ch][c]), __uint_as_float(sr[ch][c + 1])), scale2, shift2);
            const float2 e = make_float2(ex2(x.x), ex2(x.y));
            sum4[(c >> 1) & 3] = fadd2(sum4[(c >> 1) & 3], e);
            sr[ch][c >> 1] = FP8 ? pack_f16x2(e.x, e.y) : pack_bf16x2(e.x, e.y);
          }
        };
        auto store = [&](int ch) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) pk[i] = sr[ch][i];
          tmem_st16(t_p + 16 * ch, pk);
        };
        chunk(0);
        if constexpr (C::kTiles == 2) {
          store(0);
          chunk(1);
        } else {
          // P and O are free once the P V before this one has completed (a tile's first block: the epilogue waited)
          chunk(1);
          if (j > 0) {
            ok = __all_sync(0xffffffffu, mbar_wait(&bars.o_done[0], (np - 1) & 1, abort_flag));
            if (!ok) break;
            tc_fence_after();
          }
          store(0);
        }
        store(1);
        chunk(2);
        store(2);
        chunk(3);
        store(3);
        const float2 sum = fadd2(fadd2(sum4[0], sum4[1]), fadd2(sum4[2], sum4[3]));
        l_sum = l_sum * alpha + (sum.x + sum.y);
        if (rescale) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld32(t_o + c, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st32(t_o + c, o);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bars.p_full[t]);
      }
      if (ok && nb > 0) ok = mbar_wait(&bars.o_done[t], (C::kTiles == 2 ? nq : np - 1) & 1, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const bool seen = l_sum != 0.f;  // (a NaN sum goes on to the result)
      const float lse2 = seen ? m_ref - kBias + log2f(l_sum) : -INFINITY;
      const float inv = seen ? a.o_scale / l_sum : 0.f;
      if (p.whole()) {
        const long long row = ((long long)(p.q.start + tok) * a.Hq) + p.h * G + rh;
        uint8_t* orow = static_cast<uint8_t*>(a.o) + row * (D * 2);
        if (nb > 0) {
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld32(t_o + c, o);
            tmem_ld_wait(o);
            if (valid) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  // a row that has seen no key: 0, whatever its products made
                  const float x = __uint_as_float(o[16 * h + 2 * i]), y = __uint_as_float(o[16 * h + 2 * i + 1]);
                  w[i] = seen ? pack_bf16x2(x * inv, y * inv) : 0u;
                }
                st_global_32(orow + c * 2 + h * 32, w, o32);
              }
            }
          }
        } else if (valid) {
          const uint32_t zero[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
          for (int c = 0; c < D; c += 16) st_global_32(orow + c * 2, zero, o32);
        }
        if (valid) a.lse[row] = seen ? lse2 * kLn2 : -INFINITY;
      } else {
        // this part's O / l and logsumexp, fp32, for the join
        const long long prow =
            ((long long)blockIdx.x * 2 + (p.jb == 0 ? 1 : 0)) * (128 * C::kTiles) + t * 128 + r;
        if (nb > 0) {
          tc_fence_after();
          uint8_t* orow = reinterpret_cast<uint8_t*>(a.part_o + prow * D);
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld32(t_o + c, o);
            tmem_ld_wait(o);
            if (valid && seen)
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                uint32_t w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(__uint_as_float(o[8 * h + i]) * inv);
                st_global_v8(orow + c * 4 + h * 32, w);
              }
          }
        }
        if (valid) a.part_lse[prow] = lse2;
      }
      if (nb > 0) {
        tc_fence_before();
        mbar_arrive(&bars.o_free[t]);
        ++nq;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kWarpMma) tmem_dealloc(tmem, C::kTmemCols);
  if (threadIdx.x == 0 && bars.abort) atomicOr(a.status, 1u);
}

template <int D, bool FP8>
cudaError_t launch(const PagedArgs& a, int ctas, cudaStream_t stream) {
  using C = CCfg<D, FP8>;
  auto kern = a.window   ? fa_paged_chunk_kernel<D, FP8, true, true>
              : a.causal ? fa_paged_chunk_kernel<D, FP8, true>
                         : fa_paged_chunk_kernel<D, FP8, false>;
  static std::atomic<unsigned long long> done[3];  // devices (a bit each) that know the kernel's shared memory
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), C::kSmemBytes, done[a.window ? 2 : a.causal]);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3((unsigned)ctas), C::kThreads, C::kSmemBytes, stream, a);
}

}  // namespace

cudaError_t launch_paged_chunk(const PagedArgs& a, int ctas, cudaStream_t stream) {
  if (a.d == 64) return a.fp8 ? launch<64, true>(a, ctas, stream) : launch<64, false>(a, ctas, stream);
  return a.fp8 ? launch<128, true>(a, ctas, stream) : launch<128, false>(a, ctas, stream);
}

}  // namespace fa
