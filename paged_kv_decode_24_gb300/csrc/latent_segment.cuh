// The device's check of a piece of the absorbed work list.
#pragma once

#include "latent_params.h"

namespace pa {

// A segment of this call's plan whose rows and tokens are its sequence's.
__device__ __forceinline__ bool latent_segment_ok(const LatentParams& p, const LatentSegment& s,
                                                  int rows) {
  if (s.b < 0 || s.b >= p.batch || s.nrows < 1 || s.nrows > rows || s.row0 < 0 ||
      s.slot >= p.num_slots || s.tok0 < 0 || s.tok0 % kLatentStage != 0 || s.tok1 <= s.tok0)
    return false;
  const int cq = p.cu_q[s.b], qn = p.cu_q[s.b + 1] - cq, len = p.cu_k[s.b + 1] - p.cu_k[s.b];
  return cq >= 0 && p.cu_q[s.b + 1] <= p.total_q &&
         (int64_t)s.row0 + s.nrows <= (int64_t)qn * p.heads && qn <= len && s.tok1 <= len &&
         (int64_t)len <= (int64_t)p.max_pages * p.page_size;
}

}  // namespace pa
