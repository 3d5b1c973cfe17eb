// Differential attention: parameters shared by its entry points and kernels.
#pragma once

#include <cuda.h>

#include "decode_kernel.cuh"
#include "pa_internal.h"

namespace pa {

constexpr uint32_t kDiffMagic = 0x46444150u;  // "PADF", header word 0 of a one-token plan

// A pair of KV heads as the planner sees it: one KV head with 2G rows (both
// queries of its G heads) and values of 2D dims.
constexpr int kDiffWarps = 4;          // warps sharing one task's pages
static_assert(kDiffWarps == kWarpsPerCta, "the planner deals short tasks to as many warps of a CTA");
// Up to this many splits the last task of a pair joins them in the split kernel, beyond
// it a kernel of its own does.  The former is the shorter of many groups (40 sequences
// of 3 splits, 4 pairs: 17.3 against 22.1 us; 10 of 4: 14.6 against 17.2) and few splits
// (one sequence, 16 pairs, 2 splits: 11.3 against 11.8; 4: 12.2 both), the latter of single
// sequences with more (8: 13.4 against 12.2; 4 pairs, 76: 38.6 against 27.6).
constexpr int kDiffMergeSplits = 8;
// Automatic plans cut no split shorter than this many pages: 384 KB where the
// (sequence, pair)s alone give each SM a task (batch of 48 short sequences, 16 pairs:
// 17.8 us, cut at half of that 21.2), two pages a warp where they do not (4096
// tokens, 4 pairs: 10.3 us; 13.1 with four pages, 11.1 with one; 1000 tokens: 10.5, 11.7
// and 9.0).
constexpr int kDiffShortChunkPages = 8;
PA_HD constexpr int diff_min_chunk(int head_dim) { return head_dim == 64 ? 48 : 24; }
// Page tiles of a warp in flight (K or V of one page and pair: 64 D bytes), and
// the CTAs an SM holds with them.
constexpr int kDiffStages = 3;
PA_HD constexpr int diff_ctas_per_sm(int head_dim) { return head_dim == 64 ? 4 : 2; }
// Pages of each warp of the first CTAs that L2 is asked for while the kernel ahead
// still runs (one: long context 27.6 us, batch of 48 short ones 18.2; none: 29.1 and
// 20.6; two: 27.0 and 18.3).
constexpr int kDiffPrefetchPages = 1;

// What turns the two maps of a head into its output.
struct DiffEpilogue {
  const float* lambda;  // [H]
  const float* weight;  // [2D], or null: ones
  float eps;            // 0: no normalisation
  float factor;
};

struct DiffDecodeParams {
  SplitParams s;    // num_kv_heads counts pairs, the partials hold 2G rows of 2D values;
                    // fuse_merge 0: launch_diff_merge joins them
  // A partial's row is o, its values over its sum of weights; m, the reference of the
  // weights (in s.part_lse; NaN: the split gave up); and l, their sum, here.  m and l stay
  // apart: in m + log2(l), with scores of 10^5 the roundings of m are parts of a unit, and
  // splits with as large scores were weighted wrong.  m = -inf: no token, l = 0.
  float* part_sum;
  DiffEpilogue e;
};

// The workspace: the decode layout, then the partials' sums.
inline size_t diff_workspace_bytes(const Layout& l, int split_items, int rows) {
  return l.total + align_sz(4 * (size_t)split_items * rows, 256);
}

struct DiffPrefillParams {
  const void* q;
  void* out;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* ws;  // the uploaded multi-token plan
  const int32_t* cu;  // its row offsets
  int32_t* status;
  DiffEpilogue e;
  float qscale;       // scale * log2(e)
  int32_t batch, num_q_heads, num_kv_heads, max_pages, num_pages, num_tiles, total_q;
  uint64_t wait_ns;
  CUtensorMap tmap_k, tmap_v;
};

cudaError_t launch_diff_decode(const DiffDecodeParams& p, int head_dim, int group, int dtype, int grid,
                               cudaStream_t stream);
// Joins the split (sequence, pair)s of a one-token call, a CTA for each head.
cudaError_t launch_diff_merge(const DiffDecodeParams& p, int head_dim, int group, int dtype,
                              cudaStream_t stream);
cudaError_t launch_diff_decode_d64(const DiffDecodeParams& p, int group, int dtype, int grid,
                                   cudaStream_t stream);
cudaError_t launch_diff_decode_d128(const DiffDecodeParams& p, int group, int dtype, int grid,
                                    cudaStream_t stream);
cudaError_t launch_diff_prefill(const DiffPrefillParams& p, int head_dim, int group, int dtype,
                                cudaStream_t stream);

}  // namespace pa
