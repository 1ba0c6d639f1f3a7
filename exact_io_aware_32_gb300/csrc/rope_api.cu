// C ABI of the rotation of queries and keys (declared in include/fa.h): argument
// checks and kernel launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <utility>

#include "../../include/fa.h"
#include "fa_internal.h"
#include "paged.h"
#include "rope.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool factor(float x) { return std::isfinite(x) && x > 0.f; }

constexpr long long kMaxStride = 1ll << 39;

// Rows [B][H][N][d]: 16-byte aligned pieces; those of an output share no memory with one another.
int check_rows(const fa_heads* x, int B, int H, int N, int d, bool out) {
  if (!x || !x->data) return FA_ERR_INVALID_ARG;
  const long long s[3] = {x->stride_b, x->stride_h, x->stride_n};
  std::pair<long long, int> dim[3] = {{s[0], B}, {s[1], H}, {s[2], N}};
  for (long long v : s)
    if (v < 0 || v >= kMaxStride) return FA_ERR_INVALID_ARG;
  if (out) {
    std::sort(dim, dim + 3);
    long long extent = d;
    for (const auto& p : dim) {
      if (p.second == 1) continue;
      if (p.first < extent) return FA_ERR_INVALID_ARG;
      extent += p.first * (p.second - 1);
    }
  }
  if (!aligned(x->data, 16)) return FA_ERR_MISALIGNED;
  for (const auto& p : dim)
    if (p.second > 1 && p.first % 8) return FA_ERR_MISALIGNED;
  return FA_OK;
}

int check_rotation(int d, const double* freqs, int rotary, float factor_, const int* positions) {
  if (rotary < 0 || rotary > d || !std::isfinite(factor_) || (rotary && !freqs)) return FA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || rotary % 16) return FA_ERR_UNSUPPORTED;
  return aligned(freqs, 8) && aligned(positions, 4) ? FA_OK : FA_ERR_MISALIGNED;
}

// Both weights or neither (a part that is not there has none).
int check_norm(const void* wq, const void* wk, int Hk, float eps) {
  if (!wq && !wk) return FA_OK;
  if (!wq || (Hk > 0) != (wk != nullptr) || !(eps >= 0.f) || !std::isfinite(eps)) return FA_ERR_INVALID_ARG;
  return aligned(wq, 16) && aligned(wk, 16) ? FA_OK : FA_ERR_MISALIGNED;
}

int check_sizes(int B, int Hq, int Hk, int N) {
  return B < 1 || Hq < 1 || Hk < 0 || N < 1 || (long long)Hq + Hk > INT32_MAX / 2 ||
                 (long long)B * N > (1ll << 40) / (Hq + Hk)
             ? FA_ERR_INVALID_ARG
             : FA_OK;
}

fa::RopeView view(const fa_heads* x) { return {x->data, x->stride_b, x->stride_h, x->stride_n}; }

void common(fa::RopeArgs& a, const void* wq, const void* wk, int w_fp32, float eps, const double* freqs, int rotary,
            float factor_, const int* positions, long long positions_stride, int B, int Hq, int Hk, int N, int d) {
  std::memset(&a, 0, sizeof(a));
  a.part[0].w = wq;
  a.part[1].w = wk;
  a.part[0].heads = Hq;
  a.part[1].heads = Hk;
  a.freqs = freqs;
  a.pos = positions;
  a.pos_b = positions_stride;
  a.B = B;
  a.N = N;
  a.d = d;
  a.rot = rotary;
  a.w_fp32 = w_fp32 ? 1 : 0;
  a.factor = factor_;
  a.eps = eps;
}

int done(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_LAUNCH; }

}  // namespace

extern "C" {

int fa_rope_fwd(const fa_heads* q, const fa_heads* k, const fa_heads* q_out, const fa_heads* k_out, const void* q_weight,
                const void* k_weight, int weights_fp32, float eps, const double* freqs, int rotary, int interleaved,
                float factor_, const int* positions, long long positions_stride, int B, int Hq, int Hk, int N, int d,
                void* stream) {
  int st = check_sizes(B, Hq, Hk, N);
  if (st == FA_OK) st = check_rotation(d, freqs, rotary, factor_, positions);
  if (st == FA_OK) st = check_norm(q_weight, k_weight, Hk, eps);
  if (st == FA_OK) st = check_rows(q, B, Hq, N, d, false);
  if (st == FA_OK) st = check_rows(q_out, B, Hq, N, d, true);
  if (st == FA_OK && Hk) st = check_rows(k, B, Hk, N, d, false);
  if (st == FA_OK && Hk) st = check_rows(k_out, B, Hk, N, d, true);
  if (st != FA_OK) return st;
  if (positions_stride < 0 || positions_stride >= kMaxStride) return FA_ERR_INVALID_ARG;
  fa::RopeArgs a;
  common(a, q_weight, k_weight, weights_fp32, eps, freqs, rotary, factor_, positions, positions_stride, B, Hq, Hk, N, d);
  int sms = 0;
  if ((st = fa::device_facts(&sms, &a.status)) != FA_OK) return st;
  a.part[0].in = view(q);
  a.part[0].out = view(q_out);
  if (Hk) {
    a.part[1].in = view(k);
    a.part[1].out = view(k_out);
  }
  return done(fa::launch_rope_fwd(a, q_weight != nullptr, interleaved != 0, sms, static_cast<cudaStream_t>(stream)));
}

size_t fa_rope_bwd_workspace_bytes(int Hq, int Hk, int d) {
  return Hq < 1 || Hk < 0 || (d != 64 && d != 128) ? 0 : fa::rope_bwd_bytes(Hq, Hk, d);
}

int fa_rope_bwd(const fa_heads* dq_out, const fa_heads* dk_out, const fa_heads* q, const fa_heads* k, const fa_heads* dq,
                const fa_heads* dk, const void* q_weight, const void* k_weight, int weights_fp32, float eps,
                float* dq_weight, float* dk_weight, const double* freqs, int rotary, int interleaved, float factor_,
                const int* positions, long long positions_stride, int B, int Hq, int Hk, int N, int d, void* workspace,
                size_t workspace_bytes, void* stream) {
  const bool norm = q_weight != nullptr;
  int st = check_sizes(B, Hq, Hk, N);
  if (st == FA_OK) st = check_rotation(d, freqs, rotary, factor_, positions);
  if (st == FA_OK) st = check_norm(q_weight, k_weight, Hk, eps);
  if (st == FA_OK) st = check_rows(dq_out, B, Hq, N, d, false);
  if (st == FA_OK) st = check_rows(dq, B, Hq, N, d, true);
  if (st == FA_OK && norm) st = check_rows(q, B, Hq, N, d, false);
  if (st == FA_OK && Hk) st = check_rows(dk_out, B, Hk, N, d, false);
  if (st == FA_OK && Hk) st = check_rows(dk, B, Hk, N, d, true);
  if (st == FA_OK && Hk && norm) st = check_rows(k, B, Hk, N, d, false);
  if (st != FA_OK) return st;
  if (positions_stride < 0 || positions_stride >= kMaxStride || (norm && (!dq_weight || (Hk && !dk_weight))))
    return FA_ERR_INVALID_ARG;
  if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4)) return FA_ERR_MISALIGNED;
  if (norm && (!workspace || !aligned(workspace, 16) || workspace_bytes < fa_rope_bwd_workspace_bytes(Hq, Hk, d)))
    return FA_ERR_WORKSPACE;
  fa::RopeArgs a;
  common(a, q_weight, k_weight, weights_fp32, eps, freqs, rotary, factor_, positions, positions_stride, B, Hq, Hk, N, d);
  int sms = 0;
  if ((st = fa::device_facts(&sms, &a.status)) != FA_OK) return st;
  a.part[0].in = view(dq_out);
  a.part[0].out = view(dq);
  if (norm) a.part[0].x = view(q);
  if (Hk) {
    a.part[1].in = view(dk_out);
    a.part[1].out = view(dk);
    if (norm) a.part[1].x = view(k);
  }
  a.dw_part = static_cast<float*>(workspace);
  a.dw[0] = dq_weight;
  a.dw[1] = dk_weight;
  return done(fa::launch_rope_bwd(a, norm, interleaved != 0, sms, static_cast<cudaStream_t>(stream)));
}

int fa_paged_positions(const int* query_start, const int* seq_lens, int R, int* positions, int T, void* stream) {
  if (!query_start || !seq_lens || !positions || R < 1 || T < 1) return FA_ERR_INVALID_ARG;
  if (!aligned(query_start, 4) || !aligned(seq_lens, 4) || !aligned(positions, 4)) return FA_ERR_MISALIGNED;
  fa::PositionsArgs a{query_start, seq_lens, positions, R, T};
  int sms = 0;
  unsigned int* status = nullptr;
  if (const int st = fa::device_facts(&sms, &status)) return st;
  return done(fa::launch_positions(a, static_cast<cudaStream_t>(stream)));
}

int fa_paged_rope_store(const void* q, const void* k, const void* v, long long q_stride, long long k_stride,
                        long long v_stride, const int* slots, const int* positions, const double* freqs, int rotary,
                        int interleaved, float factor_, const void* q_weight, const void* k_weight, int weights_fp32,
                        float eps, void* q_out, long long q_out_stride, int T, int Hq, int Hkv, int d, void* k_cache,
                        void* v_cache, int num_pages, int page_size, int fp8, float descale_k, float descale_v,
                        void* stream) {
  if (!k || !v || !slots || !positions || !k_cache || !v_cache || Hkv < 1 || num_pages < 1 || page_size < 1)
    return FA_ERR_INVALID_ARG;
  const fa_heads hq{const_cast<void*>(q), 0, d, q_stride}, ho{q_out, 0, d, q_out_stride},
      hk{const_cast<void*>(k), 0, d, k_stride}, hv{const_cast<void*>(v), 0, d, v_stride};
  int st = check_sizes(1, Hq, Hkv, T);
  if (st == FA_OK) st = check_rotation(d, freqs, rotary, factor_, positions);
  if (st == FA_OK) st = check_norm(q_weight, k_weight, Hkv, eps);
  for (const auto& x : {std::make_pair(q_stride, Hq), std::make_pair(q_out_stride, Hq), std::make_pair(k_stride, Hkv),
                        std::make_pair(v_stride, Hkv)})
    if (st == FA_OK && x.first < (long long)x.second * d) st = FA_ERR_INVALID_ARG;
  if (st == FA_OK) st = check_rows(&hq, 1, Hq, T, d, false);
  if (st == FA_OK) st = check_rows(&ho, 1, Hq, T, d, true);
  if (st == FA_OK) st = check_rows(&hk, 1, Hkv, T, d, false);
  if (st == FA_OK) st = check_rows(&hv, 1, Hkv, T, d, false);
  if (st != FA_OK) return st;
  if ((long long)num_pages * page_size > INT32_MAX || (long long)num_pages * Hkv > INT32_MAX) return FA_ERR_INVALID_ARG;
  int shift = 4;
  while (shift <= 8 && page_size != 1 << shift) ++shift;
  if (shift > 8) return FA_ERR_UNSUPPORTED;
  if (fp8 && (!factor(descale_k) || !factor(descale_v))) return FA_ERR_INVALID_ARG;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(slots, 4)) return FA_ERR_MISALIGNED;
  fa::RopeArgs a;
  common(a, q_weight, k_weight, weights_fp32, eps, freqs, rotary, factor_, positions, 0, 1, Hq, Hkv, T, d);
  int sms = 0;
  if ((st = fa::device_facts(&sms, &a.status)) != FA_OK) return st;
  a.part[0].in = view(&hq);
  a.part[0].out = view(&ho);
  a.part[1].in = view(&hk);
  a.v = view(&hv);
  a.slots = slots;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.num_pages = num_pages;
  a.page_shift = shift;
  a.fp8 = fp8 ? 1 : 0;
  a.descale_k = descale_k;
  a.descale_v = descale_v;
  return done(fa::launch_rope_store(a, q_weight != nullptr, interleaved != 0, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
