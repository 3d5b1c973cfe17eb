// The device's check of a piece of the absorbed work list.
#pragma once

#include "latent_params.h"

namespace pa {

// A piece whose rows and tokens lie within this call's tensors.
__device__ __forceinline__ bool latent_segment_ok(const LatentParams& p, const LatentSegment& s,
                                                  int rows) {
  return s.b >= 0 && s.b < p.batch && s.nrows >= 1 && s.nrows <= rows && s.row0 >= 0 &&
         s.packed0 >= 0 && (int64_t)s.packed0 + s.nrows <= (int64_t)p.total_q * p.heads &&
         s.slot < p.num_slots && s.tok0 >= 0 && s.tok0 % kLatentStage == 0 && s.tok1 > s.tok0 &&
         (int64_t)s.tok1 <= (int64_t)p.max_pages * p.page_size && s.pos0 >= 0;
}

// The workspace holds a plan of this call's sizes.  It is written by the
// upload alone, which the programmatic launch does not overlap, so it may be
// read before the wait for the kernel ahead.
__device__ __forceinline__ bool latent_planned(const LatentParams& p, int rows) {
  const int4 h0 = reinterpret_cast<const int4*>(p.ws)[0], h1 = reinterpret_cast<const int4*>(p.ws)[1];
  const int4 h2 = reinterpret_cast<const int4*>(p.ws)[2];
  return h0.x == (int)kLatentMagic && h0.y == p.batch && h0.z == p.total_q &&
         h1.z == PA_LATENT_ABSORBED && h1.w == rows && h2.x == p.num_ranges &&
         h2.y == p.num_segments && h2.z == p.num_merges && h2.w == p.num_slots;
}

// The pieces [first, last) of one range, or none where the workspace does
// not hold this call's plan.
__device__ __forceinline__ bool latent_range(const LatentParams& p, int rows, int range, int& first,
                                             int& last) {
  first = p.ranges[range];
  last = min(p.ranges[range + 1], p.num_segments);
  const bool ok = latent_planned(p, rows) && first >= 0;
  if (!ok) first = last = 0;
  return ok;
}

}  // namespace pa
