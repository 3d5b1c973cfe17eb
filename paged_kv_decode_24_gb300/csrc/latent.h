// Latent attention: constants, plan layout and kernel parameters shared by
// the planner, the entry points and the kernels.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "pa_internal.h"

namespace pa {

constexpr int kLatent = 512;                  // latent values of a cached row (also the values)
constexpr int kRope = 64;                     // rotary key values
constexpr int kLatentRow = kLatent + kRope;   // elements of a cached row
constexpr int kLatentStage = 64;              // tokens of a stage of 16- and 64-row tiles:
                                              // their pieces are cut at its multiples
constexpr int kLatentStagePair = 128;         // the same of 128-row tiles
constexpr int kLatentBlock = 16;              // tokens of one page copy (divides every page size)
constexpr int kLatentRowsMma = 16;            // rows of a tile: the mma.sync kernel
constexpr int kLatentRowsSolo = 64;           // rows of a tile: the tcgen05 kernel on one SM
constexpr int kLatentRowsPair = 128;          // rows of a tile: the tcgen05 kernel on SM pairs
constexpr int kLatentRowsExpanded = 256;      // query tokens of an expanded tile
constexpr uint32_t kLatentMagic = 0x564b414cu;  // "LAKV"

// A piece of the absorbed work list: rows row0 .. row0 + nrows - 1 of
// sequence b (row = query token x heads + head), packed rows packed0 .. of
// [T * H], over tokens [tok0, tok1).  The sequence's first query token sits
// at position pos0.  slot < 0: writes out; else its partial result goes to
// that slot.  A piece holds all that a kernel has to know, so that it is one
// load away from its work.
struct LatentSegment {
  int32_t b, row0, nrows, tok0, tok1, slot, packed0, pos0;
};

// A tile cut into several pieces: its partials are in slots slot0 ..
// slot0 + n - 1, its rows are rows row0 .. of the packed [T * H] rows.
struct LatentMerge {
  int32_t slot0, n, row0, nrows;
};

// An expanded tile: ntok query tokens of one head, from packed row q0; the
// first sits at position pos0 of its sequence, whose tokens are packed from
// k0.
struct LatentTile {
  int32_t head, ntok, q0, pos0, k0, pad0, pad1, pad2;
};

// Blob = header (16 x int32) | cu_q [B+1] | cu_k [B+1] | then for
//   absorbed: first segment of each range [ranges + 1] | segments | merges
//   expanded: tiles
// header: [0] magic [1] B [2] T [3] Tk [4,5] plan_id [6] form [7] rows
//         [8] ranges [9] segments [10] merges [11] slots.
// The partials (fp32 lse [slot][rows], fp32 o [slot][rows][512]) follow it.
struct LatentLayout {
  size_t cu_q, cu_k, ranges, work, merges, blob_bytes, lse, o, total;
};

inline LatentLayout latent_layout(int batch, int form, int rows, int ranges, int segments,
                                  int merges, int slots) {
  LatentLayout l{};
  l.cu_q = 64;
  l.cu_k = l.cu_q + 4 * ((size_t)batch + 1);
  l.ranges = align_sz(l.cu_k + 4 * ((size_t)batch + 1), 16);
  if (form == PA_LATENT_ABSORBED) {
    l.work = align_sz(l.ranges + 4 * ((size_t)ranges + 1), 16);
    l.merges = l.work + sizeof(LatentSegment) * (size_t)segments;
    l.blob_bytes = l.merges + sizeof(LatentMerge) * (size_t)merges;
  } else {
    l.work = l.ranges;
    l.merges = l.work + sizeof(LatentTile) * (size_t)ranges;
    l.blob_bytes = l.merges;
  }
  l.lse = align_sz(l.blob_bytes, 256);
  l.o = align_sz(l.lse + 4 * (size_t)slots * (size_t)rows, 256);
  l.total = align_sz(l.o + 4 * (size_t)slots * (size_t)rows * kLatent, 256);
  return l;
}

pa_status_t check_latent_shape(const pa_latent_shape_t* s);

}  // namespace pa
