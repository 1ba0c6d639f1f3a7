// Attention of few new tokens (decoding) over the paged cache, on sm_103a: tiles
// of at most 32 rows (new tokens x query heads of one key head).
//
// Such a call is bound by reading the cache: a key block of 128 keys costs 64 KB
// at bf16 d = 128, 1.47 us of an SM's share of the bandwidth, while one 128-row
// tile's chain (S, softmax, P V) takes about 1.3 us when a thread works through
// all 128 scores of its row. Here the tile's 32 rows stand four times in the
// 128-row Q operand, so that S comes out once per TMEM lane quarter and warp w
// takes only keys [32 w, 32 w + 32) of every block: a quarter of the softmax
// chain, with a running maximum and sum of its own, as if the keys were split
// among four. P of warp w is zero outside its 32 columns (written once), so row
// 32 w + r of O sums over warp w's keys, and the four quarters are joined
// through shared memory when the tile ends. The products cost what they cost
// with 32 rows, since tcgen05 takes 128 anyway.
//
// TMEM: S twice and P twice (S of the next block is made while the softmax works
// on this one, P of the next is written while this one's product runs), O.
// Persistent CTAs over ranges of the row of tiles (paged_work.cuh), rings and
// barriers counting on across tiles.
//
// Warp roles: 0-3 softmax and epilogue; 4 walks the range and tells the others its
// pieces; two warps copy keys, every other block each, and two values; one issues P V
// and owns TMEM, one copies Q and issues Q K^T; with E4M3 caches eight converter warps
// (value codes to f16, Q to its two parts; by four of them 7% slower where tiles are
// short). A block of pages of 16 tokens takes its copying warp 1150 cycles and a step
// of the walk 1200 to 2200: at d = 64, where a block is 760 cycles of HBM, one
// warp for the keys and the walk set the pace.
//
// Measured, d = 128, 8 key heads, 32 query heads: 64 requests of up to 8192 keys
// 157 us, 6.6 TB/s of keys and values (bound by them); 48 of up to 16384, E4M3
// caches, 140 us (the tensor cores, which take 128 rows, and the bytes about alike;
// at d = 64 with pages of 16 tokens 107 us, 126 with one copying warp for keys and one for values);
// 256 requests of up to 1000 keys, bf16 and E4M3, 94 and 91 us, of up to 100 keys 37 and 48 us
// (bound by a tile's chain: its first S, softmax, last product, join).
// Where a page has 32 tokens and more the second copying warps gain nothing and cost up to 0.5%, in
// the E4M3 case 1%: the 48 requests, calls one after another, 142.4 and 144.3 us; the 64 at d = 64 with pages of 64
// tokens 91.8 and 92.2 us.
// Under a window of 1024 with 4 sinks 64 requests of 8192 keys 50 us, 5.2 TB/s of what they see.
#include "paged_pipe.cuh"

namespace fa {
namespace {

using namespace fa::ptx;
using namespace fa::paged;

template <int D_, bool FP8_>
struct FCfg {
  static constexpr int D = D_;
  static constexpr int kPanels = D / 64;
  static constexpr int kTileBytes = kPanels * 16384;  // 128 rows, 16-bit
  static constexpr int kCodeBytes = 128 * D;          // 128 rows of codes
  static constexpr int kKBytes = FP8_ ? kCodeBytes : kTileBytes;  // a key block: codes stay codes
  static constexpr int kKStages = FP8_ ? (D == 64 ? 6 : 4) : (D == 64 ? 4 : 2);
  static constexpr int kVStages = FP8_ ? (D == 64 ? 3 : 2) : (D == 64 ? 4 : 3);
  static constexpr int kCStages = FP8_ ? (D == 64 ? 6 : 3) : 0;  // value codes on their way to f16
  static constexpr int kOffQ = 0, kOffRaw = kOffQ + kTileBytes;  // E4M3 caches: the next tile's 32 rows as loaded
  static constexpr int kOffK = kOffRaw + (FP8_ ? 32 * D * 2 : 0);
  static constexpr int kOffV = kOffK + kKStages * kKBytes;
  static constexpr int kOffC = kOffV + kVStages * kTileBytes;
  // the quarters' O of kJoinRows rows at a time, rows padded by 16 bytes against bank conflicts; (m, l) of all rows
  static constexpr int kJoinRows = (D == 64 ? 16 : 8) / (FP8_ ? 2 : 1), kJoinStride = D + 4;
  static constexpr int kOffJoin = kOffC + kCStages * kCodeBytes;
  static constexpr int kOffBar = kOffJoin + 4 * kJoinRows * kJoinStride * 4 + 4 * 32 * 8;
  static constexpr int kSmemBytes = kOffBar + 768 + 1024;  // barriers, alignment slack
  static_assert(kSmemBytes <= 232448, "shared memory");
  static constexpr uint32_t kColS = 0, kColP = 256, kColO = 384, kTmemCols = 512;  // S and P twice
  static constexpr int kWarpWalk = 4, kWarpTmaK = 5, kWarpTmaV = 7, kWarpPv = 9, kWarpQk = 10, kWarpConv = 11, kConvWarps = 8;
  static constexpr int kThreads = 32 * (kWarpConv + (FP8_ ? kConvWarps : 0));
};

struct FBars {
  // q_full of tile n is q_full[n % 3]: with E4M3 caches the softmax waits for it too, and reads the exponents, maybe only
  // after the next two tiles' Q are there (S runs two blocks ahead of it, and a tile may be one block)
  uint64_t q_raw, q_full[3], q_free;  // E4M3 caches: Q as loaded, as converted
  uint64_t k_full[6], k_empty[6], v_full[4], v_empty[4], c_full[6], c_empty[6];
  uint64_t s_full[2], s_free[2], p_full[2], pv_done[2], o_free;
  uint64_t teardown[2];
  PieceRing ring;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(FBars) <= 672, "barriers exceed their shared memory");

// WIN (with CAUSAL): a token sees its last a.window keys and the first a.sinks; keys are counted without a tile's gap (Band).
template <int D, bool FP8, bool CAUSAL, bool WIN = false>
__global__ void __launch_bounds__(FCfg<D, FP8>::kThreads, 1) fa_paged_few_kernel(const __grid_constant__ PagedArgs a) {
  using C = FCfg<D, FP8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  FBars& bars = *reinterpret_cast<FBars*>(smem + C::kOffBar);
  volatile int* abort_flag = &bars.abort;
  // in the join's place, which is not in use yet: the range and its sums; behind the barriers: the exponents of Q's row
  // scales (E4M3 caches), of this tile and the two before
  Range& range = *reinterpret_cast<Range*>(smem + C::kOffJoin);
  auto& sums = *reinterpret_cast<int(*)[C::kThreads / 32]>(smem + C::kOffJoin + 256);
  auto& q_ex = *reinterpret_cast<uint8_t(*)[3][32]>(smem + C::kOffBar + 672);
  static_assert(sizeof(Range) <= 256, "the sums follow the range");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.Hq / a.Hkv;

  // Everything that does not depend on the lengths first; the range's barriers cover it.
  if (warp == C::kWarpTmaK && elect_one()) {
    tma_prefetch_desc(&a.tm_q);
    tma_prefetch_desc(&a.tm_k);
    tma_prefetch_desc(&a.tm_v);
  }
  if (threadIdx.x == 32) {
    bars.abort = 0;
    mbar_init(&bars.q_raw, 1);
    for (int s = 0; s < 3; ++s) mbar_init(&bars.q_full[s], FP8 ? C::kConvWarps : 1);
    mbar_init(&bars.q_free, 1);
    for (int s = 0; s < 6; ++s) {
      mbar_init(&bars.k_full[s], 1);
      mbar_init(&bars.k_empty[s], 1);
      mbar_init(&bars.c_full[s], 1);
      mbar_init(&bars.c_empty[s], C::kConvWarps);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&bars.v_full[s], FP8 ? C::kConvWarps : 1);
      mbar_init(&bars.v_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars.s_full[s], 1);
      mbar_init(&bars.s_free[s], 128);
      mbar_init(&bars.p_full[s], 128);
      mbar_init(&bars.pv_done[s], 1);
      mbar_init(&bars.teardown[s], 1);
    }
    mbar_init(&bars.o_free, 128);
    bars.ring.init(10 + (FP8 ? C::kConvWarps : 0));  // four softmax warps, two for K, two for V, Q K^T, P V, converters
    fence_mbar_init();
  }
  // rows of Q that no copy fills (G that does not divide 32, short tiles) are zeros, not leftovers
  for (int i = threadIdx.x; i < (C::kOffK - C::kOffQ) / 16; i += C::kThreads)
    st_shared_v4(smem_u32(smem + C::kOffQ) + i * 16, 0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  if (warp == C::kWarpPv) {
    tmem_alloc(&bars.tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  find_range<C::kThreads, WIN>(a, range, sums);
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;
  if (!range.some) {  // uniform: nothing has been issued
    if (warp == C::kWarpPv) tmem_dealloc(tmem, C::kTmemCols);
    if (threadIdx.x == 0) static_cast<Parts*>(a.parts)[blockIdx.x] = Parts{};
    return;
  }
  PieceReader in(bars.ring, abort_flag, lane);
  Piece p = range.first;
  const bool first = range.use;  // the first piece is there already
  Walk<WIN> walk;
  if (warp == C::kWarpWalk) walk.begin(range);
  const int per = range.per;
  __syncthreads();  // all have read the range: the join may write there
  if (warp == C::kWarpWalk) {
    // ------------------------------------------------------------ the walk, for all
    Parts parts{};
    int n = 0;  // pieces told
    bool more = true, ok = true;
    if (!first) {
      more = walk.template step<true>(a, p);
      ok = bars.ring.tell(n++, p, more, 0, 0, lane, abort_flag);
    }
    while (ok && more) {
      note_piece(a, parts, p, walk, per);
      more = walk.template step<true>(a, p);
      ok = bars.ring.tell(n++, p, more, 0, 0, lane, abort_flag);
    }
    if (lane == 0) static_cast<Parts*>(a.parts)[blockIdx.x] = parts;
  } else if (warp >= C::kWarpTmaK && warp < C::kWarpPv) {
    // ------------------------------------------------------------ keys, values: every other block each
    const bool value = warp >= C::kWarpTmaV;
    const int mine = (warp - C::kWarpTmaK) & 1;
    const int stages = !value ? C::kKStages : FP8 ? C::kCStages : C::kVStages;
    const int bytes = !value ? C::kKBytes : FP8 ? C::kCodeBytes : C::kTileBytes;
    uint8_t* ring = smem + (!value ? C::kOffK : FP8 ? C::kOffC : C::kOffV);
    uint64_t *full = !value ? bars.k_full : FP8 ? bars.c_full : bars.v_full,
             *empty = !value ? bars.k_empty : FP8 ? bars.c_empty : bars.v_empty;
    const CUtensorMap* tm = value ? &a.tm_v : &a.tm_k;
    int g = 0, last = 0;  // key blocks; the end of those that this warp has copied
    bool ok = true;
    for (bool more = first || in.next(p); ok && more; more = in.next(p)) {
      if (p.jb == p.je) continue;
      Pages<WIN> pages;
      Band band{};
      if (WIN) band = band_of(a, p.q, p.tok);
      pages.begin(a, p, band, lane);
      for (int jj = p.jb; jj < p.je; ++jj, ++g) {
        const int page_now = pages.of(a, p, jj, lane), s = g % stages;
        if ((g & 1) != mine) continue;
        if (!(ok = warp_wait(&empty[s], ((g / stages) & 1) ^ 1, abort_flag))) break;
        load_block<D, FP8, WIN>(a, p, jj, page_now, lane, tm, ring + s * bytes, &full[s], p.q.len - band.gap, band.low);
        last = g + 1;
      }
    }
    // Let every issued copy land before the CTA can exit: those of the run's last blocks. (A place that the other warp has filled
    // since is another phase, and was filled only after this warp's copy had been read.)
    for (int x = max(0, (ok ? g : last) - stages); x < last; ++x)
      if ((x & 1) == mine) mbar_wait_drain(&full[x % stages], (x / stages) & 1);
  } else if (warp == C::kWarpQk) {
    // ------------------------------------------------------------ S = Q K^T, up to two blocks ahead of the softmax
    const uint64_t dq = sdesc_sw128(smem_u32(smem + C::kOffQ), 16, 1024);
    const uint64_t dk = desc_keys<D, FP8>(smem + C::kOffK);
    // Q is copied by this warp too: at bf16 four times into the operand, as soon as the tile before has been read; with
    // E4M3 caches once into a place of its own, as soon as the converters have made the tile before's four from there, so
    // that it is there when they come to this tile's.
    const bool withhold = a.test_fault == 1;  // test hook: without its Q the wait below expires
    int g = 0, n = 0, nq = 0;                 // key blocks, tiles, copies of Q issued
    auto load_q = [&](const Piece& x) {
      constexpr int kCopies = FP8 ? 1 : 4, kPanelBytes = FP8 ? 4096 : 16384;
      if (withhold) return;
      uint64_t* bar = FP8 ? &bars.q_raw : &bars.q_full[nq % 3];
      if (elect_one()) {
        mbar_arrive_expect_tx(bar, (uint32_t)(kCopies * G * a.tpt * D * 2));
        for (int w = 0; w < kCopies; ++w)
          for (int pn = 0; pn < C::kPanels; ++pn)
            tma_load_3d(smem + (FP8 ? C::kOffRaw : C::kOffQ) + pn * kPanelBytes + w * 4096, &a.tm_q, bar, pn * 64, x.h * G,
                        x.q.start + x.tok);
      }
      __syncwarp();
      ++nq;
    };
    // It looks one piece ahead and no further before this one's products are issued: the loading warp may wait for the
    // softmax, which waits for them, before it tells the piece after that.
    bool ok = true, asked = false;  // asked: for p's Q (E4M3 caches)
    Piece next;
    for (bool more = first || in.next(p), more_next; ok && more; p = next, more = more_next) {
      if (p.jb == p.je) {
        more_next = in.next(next);
        asked = false;
        continue;
      }
      if (!FP8 && !(ok = warp_wait(&bars.q_free, (n & 1) ^ 1, abort_flag))) break;
      if (!asked) load_q(p);
      more_next = in.next(next);
      if (!(ok = warp_wait(&bars.q_full[n % 3], (n / 3) & 1, abort_flag))) break;
      asked = FP8 && more_next && next.jb < next.je;
      if (asked) load_q(next);
      ++n;
      for (int jj = p.jb; jj < p.je; ++jj, ++g) {
        const int s = g % C::kKStages, b = g & 1;
        ok = warp_wait2(&bars.k_full[s], (g / C::kKStages) & 1, &bars.s_free[b], ((g >> 1) & 1) ^ 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          issue_qk<D, FP8>(tmem + C::kColS + b * 128, dq, dk + ((uint32_t)(s * C::kKBytes) >> 4));
          mma_commit(&bars.s_full[b]);
          mma_commit(&bars.k_empty[s]);
          if (jj + 1 == p.je) mma_commit(&bars.q_free);  // the tile's last product to read Q
        }
        __syncwarp();
      }
    }
    // a copy of Q still on its way after an abort lands before the CTA can exit
    if (nq > n) mbar_wait_drain(FP8 ? &bars.q_raw : &bars.q_full[n % 3], FP8 ? (nq - 1) & 1 : (n / 3) & 1);
    if (elect_one()) mma_commit(&bars.teardown[0]);
    __syncwarp();
    mbar_wait_drain(&bars.teardown[0], 0);
  } else if (warp == C::kWarpPv) {
    // ------------------------------------------------------------ O += P V
    constexpr uint32_t kIdO = FP8 ? idesc_f16(128, D, false, true) : idesc_bf16(128, D, false, true);  // V MN-major
    const uint64_t dv = Tile<D>::desc_v(smem + C::kOffV);
    int g = 0, n = 0;  // key blocks, tiles
    bool ok = true;
    for (bool more = first || in.next(p); ok && more; more = in.next(p)) {
      if (p.jb == p.je) continue;
      Band band{};
      if (WIN) band = band_of(a, p.q, p.tok);
      for (int jj = p.jb; jj < p.je; ++jj, ++g) {
        const int s = g % C::kVStages, b = g & 1;
        if (!(ok = warp_wait2(&bars.v_full[s], (g / C::kVStages) & 1, &bars.p_full[b], (g >> 1) & 1, abort_flag))) break;
        // a tile's first P V overwrites O: the tile before has been read out
        if (jj == p.jb && !(ok = warp_wait(&bars.o_free, (n & 1) ^ 1, abort_flag))) break;
        const int keys = p.q.len - band.gap - jj * 128, steps = pv_steps(keys);
        if (!FP8 && keys < steps * 16) zero_rows<D>(smem + C::kOffV + s * C::kTileBytes, keys, steps * 16, lane);
        tc_fence_after();
        if (elect_one()) {
          const uint32_t vo = (uint32_t)(s * C::kTileBytes) >> 4;
          issue_pv_steps<D>(tmem + C::kColO, tmem + C::kColP + b * 64, dv + vo, kIdO, steps, jj == p.jb);
          mma_commit(&bars.pv_done[b]);
          mma_commit(&bars.v_empty[s]);
        }
        __syncwarp();
      }
      ++n;
    }
    if (elect_one()) mma_commit(&bars.teardown[1]);
    __syncwarp();
    mbar_wait_drain(&bars.teardown[1], 0);
  } else if (FP8 && warp >= C::kWarpConv) {
    // ------------------------------------------------------------ converters
    const int tid = threadIdx.x - C::kWarpConv * 32;
    constexpr int kCS = FP8 ? C::kCStages : 1;
    int g = 0, n = 0;
    bool ok = true;
    for (bool more = first || in.next(p); ok && more; more = in.next(p)) {
      if (p.je > p.jb) {
        if (!(ok = warp_wait2(&bars.q_raw, n & 1, &bars.q_free, (n & 1) ^ 1, abort_flag))) break;
        convert_q<D>(smem + C::kOffRaw, smem + C::kOffQ, q_ex[n % 3], tid);
        conv_arrive(&bars.q_full[n % 3], nullptr, lane);
        ++n;
      }
      Band band{};
      if (WIN) band = band_of(a, p.q, p.tok);
      for (int j = p.jb; j < p.je; ++j, ++g) {
        const int vs = g % C::kVStages, cs = g % kCS;
        ok = warp_wait2(&bars.c_full[cs], (g / kCS) & 1, &bars.v_empty[vs], ((g / C::kVStages) & 1) ^ 1, abort_flag);
        if (!ok) break;
        convert_tile<D, 32 * C::kConvWarps>(smem + C::kOffC + cs * C::kCodeBytes, smem + C::kOffV + vs * C::kTileBytes,
                                            p.q.len - band.gap - j * 128, tid);
        conv_arrive(&bars.v_full[vs], &bars.c_empty[cs], lane);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax + epilogue
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    const uint32_t t_s = tmem + lane_off + C::kColS + warp * 32;  // this warp's rows and keys
    const uint32_t t_p = tmem + lane_off + C::kColP;
    const uint32_t t_o = tmem + lane_off + C::kColO;
    constexpr float kBias = FP8 ? kPBias : 0.f;
    const int rt = lane / G;  // this row's token within the tile
    float* join = reinterpret_cast<float*>(smem + C::kOffJoin);
    float2* stats = reinterpret_cast<float2*>(join + 4 * C::kJoinRows * C::kJoinStride);  // (m, l) by quarter and row
    {
      const uint32_t zero[16] = {};
#pragma unroll
      for (int c = 0; c < 8; ++c) tmem_st16(t_p + c * 16, zero);  // both P outside this warp's columns stay 0
      tmem_st_wait();
    }
    int g = 0, n = 0;
    bool more = first || in.next(p), ok = first || named_bar_and(1, 128, in.ok);
    while (ok && more) {
      const int nb = p.je - p.jb;
      float sl2 = a.scale_log2;
      if (FP8 && nb > 0) {  // (their place is written again three tiles on, after this warp has read the first S of this one)
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bars.q_full[n % 3], (n / 3) & 1, abort_flag)))) sl2 = 0.f;
        sl2 *= unscale(q_ex[n % 3][lane]);
        ++n;
      }
      Band band{};
      if (WIN) band = band_of(a, p.q, p.tok);
      const int len = p.q.len - band.gap, off = len - p.q.n;  // causal: token i sees keys 0 .. i + off
      const int lim_row = (CAUSAL ? min(p.tok + rt + off, len - 1) : len - 1) - warp * 32;
      const int lim_first = (CAUSAL ? min(p.tok + off, len - 1) : len - 1) - warp * 32;
      const int rows = min(a.tpt, p.q.n - p.tok) * G;
      // window: the last key, of this warp's, that is behind the last token's
      const int out_last = WIN ? min(p.tok + a.tpt, p.q.n) - 1 + off - band.wide - warp * 32 : 0;
      float m_ref = -INFINITY;  // exponent reference, log2 units of scaled scores
      float l_sum = 0.f;        // sum of 2^(s * sl2 - m_ref) over this warp's keys so far
      for (int j = 0; ok && j < nb; ++j, ++g) {
        const int b = g & 1;
        // S, and with it the place of this block's P: free once the P V two blocks back has completed
        ok = warp_wait2(&bars.s_full[b], (g >> 1) & 1, &bars.pv_done[b], ((g >> 1) & 1) ^ 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        uint32_t sr[32];
        float mx;
        tmem_ld32_max(t_s + b * 128, sr, mx);
        tmem_ld_wait(sr, mx);
        tc_fence_before();
        mbar_arrive(&bars.s_free[b]);  // S is in registers: the block after the next may overwrite it
        const int kv0 = (p.jb + j) * 128;
        if (kv0 + 31 > lim_first || (WIN && kv0 <= out_last)) {  // some row does not see all of these keys
          const int lim = lim_row - kv0;
          const int out = lim - band.wide, sunk = a.sinks - warp * 32 - kv0;  // hidden too: keys up to 'out', from 'sunk' on
          mx = -INFINITY;
          const uint32_t keep = WIN ? first_bits(lim + 1) & ~(first_bits(out + 1) & ~first_bits(sunk)) : 0u;
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            if (WIN ? !(keep >> c & 1u) : c > lim) sr[c] = __float_as_uint(-INFINITY);
            mx = fmaxf(mx, __uint_as_float(sr[c]));
          }
        }
        float alpha = 1.f;
        const float m_new = fmaxf(m_ref, mx * sl2);
        const bool move = m_new > m_ref + kRescaleThreshold;
        if (move) {
          alpha = ex2(m_ref - m_new);
          m_ref = m_new;
        }
        const bool rescale = __any_sync(0xffffffffu, move && j > 0);
        const float m_use = (m_ref == -INFINITY ? 0.f : m_ref) - kBias;  // a row that has seen no key yet: P = 0
        const float2 scale2 = make_float2(sl2, sl2), shift2 = make_float2(-m_use, -m_use);
        float2 sum2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        uint32_t pk[16];
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          const float2 x = ffma2(make_float2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), scale2, shift2);
          const float2 e = make_float2(ex2(x.x), ex2(x.y));
          sum2[(c >> 1) & 1] = fadd2(sum2[(c >> 1) & 1], e);
          pk[c >> 1] = FP8 ? pack_f16x2(e.x, e.y) : pack_bf16x2(e.x, e.y);
        }
        const float2 sum = fadd2(sum2[0], sum2[1]);
        l_sum = l_sum * alpha + (sum.x + sum.y);
        tmem_st16(t_p + b * 64 + 16 * warp, pk);
        if (rescale) {  // O, once the last P V has completed
          if (!(ok = warp_wait(&bars.pv_done[b ^ 1], ((g - 1) >> 1) & 1, abort_flag))) break;
          tc_fence_after();
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
        mbar_arrive(&bars.p_full[b]);
      }
      const bool whole = p.whole();
      const long long row0 = (long long)(p.q.start + p.tok) * a.Hq + p.h * G;  // row r: token r / G, head r % G
      const long long part0 = ((long long)blockIdx.x * 2 + (p.jb == 0 ? 1 : 0)) * 32;
      if (ok) {
        more = in.next(p);
        ok = in.ok;
      }
      // ---- the tile's four quarters joined: o = sum_w 2^(m_w - m) O_w / sum_w 2^(m_w - m) l_w
      if (ok && nb > 0) ok = mbar_wait(&bars.pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!named_bar_and(1, 128, ok)) {  // the four warps agree whether to go on, and have read the join before
        ok = false;
        break;
      }
      stats[warp * 32 + lane] = make_float2(m_ref, l_sum);
      if (nb > 0) tc_fence_after();
      for (int r0 = 0; r0 < rows; r0 += C::kJoinRows) {  // kJoinRows rows at a time
        const int mine = lane - r0;
        const bool writes = mine >= 0 && mine < C::kJoinRows;
        const uint32_t dst = smem_u32(join + (warp * C::kJoinRows + mine) * C::kJoinStride);
        if (nb > 0) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld32(t_o + c, o);
            tmem_ld_wait(o);
            if (writes)
#pragma unroll
              for (int i = 0; i < 32; i += 4) st_shared_v4(dst + (c + i) * 4, o[i], o[i + 1], o[i + 2], o[i + 3]);
          }
          if (r0 + C::kJoinRows >= rows) {
            tc_fence_before();
            mbar_arrive(&bars.o_free);  // O has been read: the next tile may accumulate there
          }
        }
        named_bar_sync(1, 128);
        const int count = min(C::kJoinRows, rows - r0);
        for (int i = threadIdx.x; i < count * (D / 4); i += 128) {  // a row's four columns each
          const int rr = i / (D / 4), c = (i % (D / 4)) * 4, r = r0 + rr;
          float2 ml[4];
          float m = -INFINITY, l = 0.f;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            ml[w] = stats[w * 32 + r];
            m = fmaxf(m, ml[w].x);
          }
          float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            if (ml[w].y == 0.f) continue;  // that warp saw no key of this row (a NaN sum goes on to the result)
            const float f = ex2(ml[w].x - m);
            const float4 x = *reinterpret_cast<const float4*>(join + (w * C::kJoinRows + rr) * C::kJoinStride + c);
            l += f * ml[w].y;
            s.x += f * x.x;
            s.y += f * x.y;
            s.z += f * x.z;
            s.w += f * x.w;
          }
          const bool seen = l != 0.f;
          const float inv = seen ? a.o_scale / l : 0.f, lse2 = seen ? m - kBias + log2f(l) : -INFINITY;
          s = make_float4(s.x * inv, s.y * inv, s.z * inv, s.w * inv);
          if (whole) {
            const int tk = r / G;
            const long long row = row0 + (long long)tk * a.Hq + (r - tk * G);
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.o) + (row * D + c) * 2) =
                make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
            if (c == 0) a.lse[row] = seen ? lse2 * kLn2 : -INFINITY;
          } else {
            *reinterpret_cast<float4*>(a.part_o + (part0 + r) * D + c) = s;
            if (c == 0) a.part_lse[part0 + r] = lse2;
          }
        }
        if (r0 + C::kJoinRows < rows) named_bar_sync(1, 128);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kWarpPv) tmem_dealloc(tmem, C::kTmemCols);
  if (threadIdx.x == 0 && bars.abort) atomicOr(a.status, 1u);
}

template <int D, bool FP8>
cudaError_t launch(const PagedArgs& a, int ctas, cudaStream_t stream) {
  using C = FCfg<D, FP8>;
  auto kern = a.window   ? fa_paged_few_kernel<D, FP8, true, true>
              : a.causal ? fa_paged_few_kernel<D, FP8, true>
                         : fa_paged_few_kernel<D, FP8, false>;
  static std::atomic<unsigned long long> done[3];  // devices (a bit each) that know the kernel's shared memory
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), C::kSmemBytes, done[a.window ? 2 : a.causal]);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3((unsigned)ctas), C::kThreads, C::kSmemBytes, stream, a);
}

}  // namespace

cudaError_t launch_paged_few(const PagedArgs& a, int ctas, cudaStream_t stream) {
  if (a.d == 64) return a.fp8 ? launch<64, true>(a, ctas, stream) : launch<64, false>(a, ctas, stream);
  return a.fp8 ? launch<128, true>(a, ctas, stream) : launch<128, false>(a, ctas, stream);
}

}  // namespace fa
