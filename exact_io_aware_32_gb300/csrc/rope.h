// Internal interface of the rotation kernels (rope_api.cu calls the launchers of rope.cu).
#pragma once
#include <cuda_runtime.h>
#include <cstddef>

namespace fa {

// Rows [B][H][N][d] of bf16 at any strides (in elements), d innermost.
struct RopeView {
  void* at;
  long long b, h, n;
};

// One of queries and keys.
struct RopePart {
  RopeView in, x, out;  // in: what is rotated (forward: the rows, backward: the gradient); x: backward with norms: the rows
  const void* w;        // norm weights [d], or NULL
  int heads;            // 0: there is none
};

struct RopeArgs {
  RopePart part[2];      // queries, keys
  const double* freqs;   // [rot / 2], radians a position
  const int* pos;        // position of token n of sequence b at pos[b * pos_b + n]; NULL: n
  long long pos_b;
  int B, N, d, rot, w_fp32;
  float factor, eps;
  float* dw_part;        // backward with norms: fp32 [CTAs][d], the CTAs of queries first
  float* dw[2];          // [d]
  // set by the launcher: CTAs of each part (backward); tokens that a warp has at a time, its groups of lanes that share one,
  // slices of a token's heads, heads of each; units (slices of so many tokens)
  int ctas[2], tokens[2], groups[2], slices[2], slice_heads[2];
  long long units[2];
  // the store (B = 1, N tokens): row t of the keys and values goes to slots[t], nothing of a row with a negative one anywhere
  const int* slots;
  RopeView v;
  void *k_cache, *v_cache;
  unsigned int* status;
  int num_pages, page_shift, fp8;
  float descale_k, descale_v;
};

struct PositionsArgs {
  const int *query_start, *seq_lens;  // [R + 1], [R]
  int* positions;                     // [T]
  int R, T;
};

// Bytes of a backward's partial sums (norms), for any device.
size_t rope_bwd_bytes(int Hq, int Hk, int d);
cudaError_t launch_rope_fwd(RopeArgs a, bool norm, bool interleaved, int num_sms, cudaStream_t stream);
cudaError_t launch_rope_bwd(RopeArgs a, bool norm, bool interleaved, int num_sms, cudaStream_t stream);
cudaError_t launch_rope_store(RopeArgs a, bool norm, bool interleaved, int num_sms, cudaStream_t stream);
cudaError_t launch_positions(const PositionsArgs& a, cudaStream_t stream);

}  // namespace fa
