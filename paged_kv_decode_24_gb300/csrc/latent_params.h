// Parameter blocks and launchers of the latent attention kernels.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "latent.h"

namespace pa {

// cuTensorMapEncodeTiled; nullptr where the driver has none (latent.cu)
PFN_cuTensorMapEncodeTiled_v12000 latent_map_encoder();

// Rows between packed tensors and pages (append and gather).
struct LatentRowsParams {
  const void* c;  // append: latents; gather: unused
  const void* r;  // append: rotary keys
  void* rows;     // gather: packed rows
  void* pages;
  const int32_t* block_table;
  const int32_t* ws;  // the uploaded plan
  int32_t* status;
  int64_t c_stride, r_stride;
  int32_t batch, total, max_pages, num_pages, page_size;
};

cudaError_t launch_latent_append(const LatentRowsParams& p, cudaStream_t stream);
cudaError_t launch_latent_gather(const LatentRowsParams& p, cudaStream_t stream);

// Absorbed attention.
struct LatentParams {
  CUtensorMap pages_map;  // the pool, in the boxes of the plan's kernel
  const void* q;
  void* out;
  const int32_t* block_table;
  const int32_t* ws;
  const int32_t* ranges;
  const LatentSegment* segments;
  const LatentMerge* merges;
  float* part_lse;
  float* part_o;
  int32_t* status;
  uint64_t wait_ns;
  float qscale;  // scale x log2(e)
  int32_t batch, heads, max_pages, num_pages, page_size;
  int32_t num_ranges, num_segments, num_merges, num_slots, total_q, rows;
};

// pages_map is the launchers' to fill: each kernel has boxes of its own.
cudaError_t launch_latent_mma(const LatentParams& p, const pa_latent_shape_t& shape, const void* pages,
                              cudaStream_t stream);
cudaError_t launch_latent_solo(const LatentParams& p, const pa_latent_shape_t& shape,
                               const void* pages, cudaStream_t stream);
cudaError_t launch_latent_pair(const LatentParams& p, const pa_latent_shape_t& shape,
                               const void* pages, cudaStream_t stream);
cudaError_t launch_latent_merge(const LatentParams& p, int dtype, cudaStream_t stream);

// Expanded attention.
struct LatentPrefillParams {
  const void* q;
  const void* k;
  const void* k_rope;
  const void* v;
  void* out;
  const int32_t* ws;
  const LatentTile* tiles;
  int32_t* status;
  int64_t k_token, k_head, kr_token, v_token, v_head;  // strides, elements
  uint64_t wait_ns;
  float qscale;
  int32_t batch, heads, num_tiles, total_q, total_k;
  bool k_token_major, v_token_major;  // set by the launcher: tokens are further apart than heads
};

cudaError_t launch_latent_prefill(const LatentPrefillParams& p, int head_dim, int dtype,
                                  cudaStream_t stream);

}  // namespace pa
