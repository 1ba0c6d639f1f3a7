// Internal interface of the paged key/value cache's kernels (paged_api.cu calls
// the launchers of paged_cache.cu and paged_fwd.cu).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cstddef>

namespace fa {

struct PlanArgs {
  const int *ctx_lens, *new_lens;       // [R]
  const int *free_pages, *free_head;    // [n_free]; [1] or NULL
  int *block_table;                     // [R][max_pages]
  int *query_start, *seq_lens, *slots;  // [R + 1], [R], [T]
  int *pages_taken;                     // [1]
  unsigned int* status;
  int R, T, n_free, max_pages, page_shift;  // page_size = 1 << page_shift
  int group;                                // requests per CTA (set by launch_plan)
};

struct StoreArgs {
  const void *k, *v;  // bf16 [T][Hkv][d]
  long long k_stride, v_stride;
  const int* slots;
  void *k_cache, *v_cache;
  unsigned int* status;
  int T, Hkv, d, num_pages, page_shift, fp8;
  float descale_k, descale_v;
  int step_tokens, step_pieces;  // set by launch_store
};

struct PagedArgs {
  const void* q;  // bf16 [T][Hq][d], q_stride elements between tokens
  long long q_stride;
  const void *k_cache, *v_cache;
  const int *block_table, *query_start, *seq_lens;
  void* o;
  float* lse;
  unsigned int* status;
  int T, R, Hq, Hkv, d, num_pages, page_shift, max_pages, causal, fp8;
  float scale_log2;  // scale * log2(e), times the key factor
  float o_scale;     // the value factor
  int max_keys;      // max_pages pages of keys
  // set by launch_paged
  CUtensorMap tm_q;         // bf16 [T][Hq][d], box 64 x (Hq / Hkv) x tokens of a 128-row (32-row) tile, 128B swizzle
  // A page's rows of one head, up to 128 of them, per copy. bf16: seen as [page, head][row / 8][panel][row % 8][64
  // columns] with 128B swizzle, so that one copy brings every 64-column panel. E4M3: [page, head][row][d], keys
  // swizzled over their d-byte rows, values not.
  CUtensorMap tm_k, tm_v;
  int n_min, n_max;         // new tokens of the requests to take
  int most;                 // length of the row of tiles, at most (most_blocks)
  int whole, snap;          // key blocks of a tile that is not cut; of the smallest part of one that is
  int tpt;                  // tokens per tile
  int tpt1;                 // tokens per 128-row half of a tile (two halves at d = 128)
  void* parts;              // Parts per CTA, then the cut tiles' results, in the caller's workspace
  float* part_o;            // fp32 [CTA][2][rows][d]: O / l of a leading (0) and an opening (1) piece
  float* part_lse;          // fp32 [CTA][2][rows]: their logsumexps in log2 units
  int test_fault;           // as in FwdArgs
};

// How one kernel of a call is laid out (see plan_paged).
struct PagedPlan {
  bool few;          // the kernel for at most 32 rows per tile
  int ctas;          // persistent CTAs
  int rows;          // rows of a tile
  int tpt, tpt1, whole, snap;
  bool join;         // whether any tile may be cut
  int n_min, n_max;  // the requests that are this kernel's: those with so many new tokens
  size_t parts_bytes, o_bytes, lse_bytes;  // of the workspace, each a multiple of 256
  size_t bytes() const { return parts_bytes + o_bytes + lse_bytes; }
};

// The length of a kernel's row of tiles in key blocks (paged_work.cuh), at most: requests that share no rows have T / tpt + R
// tiles per key head, each with the table's key blocks and its fixed part, rounded up.
inline double most_blocks(int T, int R, int Hkv, int tpt, int max_keys) {
  return ((double)T / tpt + R) * Hkv * (max_keys / 128.0 + 4.0);
}

// Launches a kernel that begins with grid_wait (ptx.cuh) once its own set-up is done, so that the set-up and the launch
// itself overlap the end of the kernel before it in the stream.
template <class Args, class... More>
cudaError_t launch_dependent(void (*kernel)(Args, More...), dim3 grid, int threads, int smem, cudaStream_t stream,
                             const Args& args, const More&... more) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3((unsigned)threads);
  c.dynamicSmemBytes = (size_t)smem;
  c.stream = stream;
  c.attrs = &attr;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, args, more...);
}

cudaError_t launch_plan(const PlanArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_store(const StoreArgs& a, int num_sms, cudaStream_t stream);
// The kernels of a call (1 or 2) in p[]; each may use the whole workspace, one after the other.
int plan_paged(int T, int R, int Hq, int Hkv, int d, int fp8, int max_new, int max_keys, int num_sms,
               PagedPlan (&p)[2]);
// Encodes the tensor maps, gives the kernel its parts of the workspace and launches it with its join;
// cudaErrorInvalidValue if the encoding fails.
cudaError_t launch_paged(PagedArgs a, const PagedPlan& p, void* workspace, cudaStream_t stream);
// The two kernels (paged_few.cu, paged_chunk.cu) and the join of cut tiles.
cudaError_t launch_paged_few(const PagedArgs& a, int ctas, cudaStream_t stream);
cudaError_t launch_paged_chunk(const PagedArgs& a, int ctas, cudaStream_t stream);
// Tensor map (sizes, strides in bytes and box, innermost first); swizzle: bytes (128 or 64), or 0 for none.
bool encode_map(CUtensorMap* m, const void* base, CUtensorMapDataType type, int rank, const unsigned long long* dims,
                const unsigned long long* strides, const unsigned* box, int swizzle);
// Allows the kernel its dynamic shared memory on the current device, once per device ('done' has a bit for each:
// the attribute costs a microsecond, as long as a short call's whole kernel).
cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<unsigned long long>& done);
// Takes the fault that fa_test_arm_fault armed (0: none).
int take_test_fault();

}  // namespace fa
