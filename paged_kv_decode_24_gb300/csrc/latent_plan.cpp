// Host-side planner of the latent attention calls.
//
// Absorbed form.  A tile is up to `rows` consecutive query rows of one
// sequence (its tokens x heads, which lie next to each other in q and out);
// its work is the stages of 64 or 128 tokens its last row sees.  The GPU runs
// one CTA (or CTA pair) per SM (pair of SMs), each of which takes one range of
// the list of all tiles' stages: the list is cut into ranges of equal work,
// wherever that falls, so that the CTAs end together whatever the lengths.
// A tile that a cut falls into becomes several pieces, whose partial results
// are merged.  A piece costs its stages and a fixed part (queries in, output
// out), kPieceStages16 or 128; a cut that would leave a piece of less than
// kMinPiece stages is moved to the tile's edge.  Few tiles may be cut one by one
// instead (piece_stages).
//
// Expanded form.  A tile is up to 256 query tokens of one head, or up to 128
// where that is estimated to end sooner (few tiles), the longest first, so that
// the short ones fill the tail of the grid.
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <atomic>
#include <functional>
#include <queue>
#include <vector>

#include "latent.h"

namespace pa {

pa_status_t check_latent_shape(const pa_latent_shape_t* s) {
  if (!s) return PA_ERR_INVALID_ARG;
  if (s->batch < 0 || s->num_heads <= 0 || s->head_dim <= 0 || s->latent_dim <= 0 ||
      s->rope_dim <= 0 || s->page_size <= 0 || s->max_pages_per_seq <= 0 || s->num_pages <= 0)
    return PA_ERR_INVALID_ARG;
  if (s->num_heads > 128 || (s->head_dim != 64 && s->head_dim != 128) ||
      s->latent_dim != kLatent || s->rope_dim != kRope)
    return PA_ERR_UNSUPPORTED;
  if (s->page_size != 16 && s->page_size != 32 && s->page_size != 64 && s->page_size != 128)
    return PA_ERR_UNSUPPORTED;
  if (s->dtype != PA_DTYPE_F16 && s->dtype != PA_DTYPE_BF16) return PA_ERR_UNSUPPORTED;
  if ((int64_t)s->max_pages_per_seq * s->page_size > INT32_MAX) return PA_ERR_INVALID_ARG;
  return PA_OK;
}

namespace {

std::atomic<uint64_t> g_latent_ids{1};

// Fixed cost of a piece, in stages: measured 2 to 2.8 of the 128-row kernel's
// 2 us, about 1 of the 16-row kernel's 1.7 us (batch of 64 with 16 heads 64.6 us
// with 1, 66.5 with 2).  The 64-row kernel's calls take the same within 2 % with
// 1, 2 and 3.
constexpr int kPieceStages16 = 1, kPieceStages128 = 2;
constexpr int kMinPiece = 1;     // stages of the shortest piece a cut leaves
constexpr int kMinRange = 1;     // stages a range is worth launching a CTA for

// What a batch's time has beside the stages of its longest range, in hundredths
// of a stage: each piece (its partials out and in again) and the merge, by the
// kernel of 16, 64 and 128 rows.  From calls of 1 to 16 sequences of 64 to 2048
// tokens, with stages of 1.85, 1.45 and 1.5 us.
struct PieceTimes {
  int64_t piece, merge;
};
constexpr PieceTimes kTimes16 = {1, 130}, kTimes64 = {4, 290}, kTimes128 = {7, 270};

// Expanded tiles: their start and output, and a stage of a tile of more than 128
// query tokens and of fewer, in 0.05 us (contexts of 4096 and 8192 tokens, 32
// heads: one tile of 256 takes 71 and 137 us, two of 128 side by side 56 and
// 106).
constexpr int kExpandedFixed = 100, kExpandedWhole = 41, kExpandedHalf = 32;
constexpr int kExpandedFew = 2;  // whole tiles for each SM up to which halves are considered

struct Work {
  std::vector<int32_t> ranges;
  std::vector<LatentSegment> segments;
  std::vector<LatentMerge> merges;
  std::vector<LatentTile> tiles;
  int64_t slots = 0;
};

// One tile's pieces: cuts (in stages, ascending, first 0 and last the tile's
// stages) become segments; several of them a merge.
struct AbsorbedTile {
  int32_t b, row0, nrows, span;  // span: tokens its last row sees
};

// Where every tile has a CTA of its own, tiles may also be cut one by one: into
// pieces of up to `longest` stages, one a CTA.  This returns the length with
// the least time, 0 where ranges of equal work take less: those keep every CTA
// busy to the end, but most CTAs then have two pieces to write.  Whole and cut
// tiles, us: 8 sequences of 256 tokens with 64 heads 10.9 and 13.1; of 1024 with
// 16 heads 33.4, and 9.4 in pieces of one stage (equal ranges 10.7); 16 of 1024
// with 64 heads 30.5, and 16.7 in pieces of four (equal ranges 22).
int64_t piece_stages(const std::vector<int64_t>& stages, int rows, int64_t workers,
                     int64_t piece_cost, int64_t equal_ranges, int64_t equal_quota) {
  const PieceTimes& t = rows == kLatentRowsMma    ? kTimes16
                        : rows == kLatentRowsSolo ? kTimes64
                                                  : kTimes128;
  const int64_t tiles = (int64_t)stages.size();
  if (tiles > workers) return 0;
  const int64_t longest = *std::max_element(stages.begin(), stages.end());
  int64_t best = 100 * (equal_quota - piece_cost) + t.piece * (tiles + equal_ranges) + t.merge;
  int64_t found = 0, last = 0;
  for (int64_t k = 1; k <= std::min(workers, longest); ++k) {
    const int64_t n = (longest + k - 1) / k;
    if (n == last) continue;
    last = n;
    int64_t pieces = 0;
    for (int64_t x : stages) pieces += (x + n - 1) / n;
    if (pieces > workers) break;
    const int64_t time = 100 * n + t.piece * pieces + (pieces > tiles ? t.merge : 0);
    if (time <= best) {
      best = time;
      found = n;
    }
  }
  return found;
}

void absorbed_work(const pa_latent_shape_t& s, const int32_t* lens, const int32_t* qs,
                   const std::vector<int32_t>& cu_q, int rows, int workers, int forced, Work* w) {
  const int64_t stage = rows == kLatentRowsPair ? kLatentStagePair : kLatentStage;
  const int64_t piece_cost = rows == kLatentRowsPair ? kPieceStages128 : kPieceStages16;
  auto stages_of = [&](int64_t tokens) { return (tokens + stage - 1) / stage; };
  std::vector<AbsorbedTile> tiles;
  std::vector<int64_t> stages;
  int64_t total = 0;
  for (int b = 0; b < s.batch; ++b) {
    const int64_t all = (int64_t)qs[b] * s.num_heads;
    for (int64_t r = 0; r < all; r += rows) {
      const int n = (int)std::min<int64_t>(rows, all - r);
      const int32_t last = (int32_t)((r + n - 1) / s.num_heads);  // query token of its last row
      const int32_t span = lens[b] - qs[b] + last + 1;
      tiles.push_back({b, (int32_t)r, n, span});
      stages.push_back(stages_of(span));
      total += stages.back() + piece_cost;
    }
  }
  if (tiles.empty()) {
    w->ranges.push_back(0);
    return;
  }
  const int64_t by_work = std::max<int64_t>(1, total / (kMinRange + piece_cost));
  const int64_t ranges = std::min<int64_t>(workers, by_work);
  // each range gets an equal share of what is left when it is opened, where
  // every range but the last is expected to end in a cut, a piece more
  auto share = [&](int64_t open) { return (total + piece_cost * (open - 1) + open - 1) / open; };
  int64_t quota = share(ranges);
  const int64_t each = forced ? 0 : piece_stages(stages, rows, workers, piece_cost, ranges, quota);
  int64_t left = quota;  // of the range that is being filled
  w->ranges.push_back(0);
  auto close = [&] {
    if (w->ranges.back() != (int32_t)w->segments.size())
      w->ranges.push_back((int32_t)w->segments.size());
    const int64_t open = std::max<int64_t>(1, ranges - ((int64_t)w->ranges.size() - 1));
    left = quota = share(open);
  };
  for (const AbsorbedTile& t : tiles) {
    const int64_t n = stages_of(t.span);
    const size_t first = w->segments.size();
    int64_t at = 0, piece = 0;
    while (at < n) {
      int64_t take = n - at;
      if (forced > 0 || each > 0) {
        const int64_t parts = forced > 0 ? std::min<int64_t>(forced, n) : (n + each - 1) / each;
        ++piece;
        take = n * piece / parts - at;
        close();
      } else if (take + piece_cost > left) {
        if (left < kMinPiece + piece_cost && left < quota) {  // nothing worth starting
          close();
          continue;
        }
        take = std::min<int64_t>(take, std::max<int64_t>(left - piece_cost, kMinPiece));
        if (n - at - take < kMinPiece) take = n - at;
      }
      const int32_t tok1 = (int32_t)std::min<int64_t>((at + take) * stage, t.span);
      w->segments.push_back({t.b, t.row0, t.nrows, (int32_t)(at * stage), tok1, -1,
                             (int32_t)((int64_t)cu_q[(size_t)t.b] * s.num_heads + t.row0),
                             lens[t.b] - qs[t.b]});
      at += take;
      left -= take + piece_cost;
      total -= take + (at == n ? piece_cost : 0);
      if (forced == 0 && each == 0 && left <= 0) close();
    }
    const size_t pieces = w->segments.size() - first;
    if (pieces > 1) {
      w->merges.push_back({(int32_t)w->slots, (int32_t)pieces, w->segments[first].packed0, t.nrows});
      for (size_t i = first; i < w->segments.size(); ++i)
        w->segments[i].slot = (int32_t)w->slots++;
    }
  }
  if (w->ranges.back() != (int32_t)w->segments.size())
    w->ranges.push_back((int32_t)w->segments.size());
}

struct Sized {
  LatentTile t;
  int64_t stages, cost;
};

// The tiles of up to `rows` query tokens, those with most stages first.  (By
// their cost, which puts short whole tiles before long halves, six chunks of 513
// tokens take 170 us, this way 158: a chunk's tiles that run together share
// its keys and values in L2.)
std::vector<Sized> expanded_tiles(const pa_latent_shape_t& s, const int32_t* lens, const int32_t* qs,
                                  const std::vector<int32_t>& cu_q, const std::vector<int32_t>& cu_k,
                                  int rows) {
  std::vector<Sized> all;
  for (int b = 0; b < s.batch; ++b)
    for (int32_t t0 = 0; t0 < qs[b]; t0 += rows) {
      const int32_t n = std::min(rows, qs[b] - t0), pos0 = lens[b] - qs[b] + t0;
      const int64_t stages = ((int64_t)pos0 + n + 127) / 128;
      const int64_t cost =
          kExpandedFixed + stages * (n > kLatentRowsExpanded / 2 ? kExpandedWhole : kExpandedHalf);
      for (int h = 0; h < s.num_heads; ++h)
        all.push_back({{h, n, cu_q[(size_t)b] + t0, pos0, cu_k[(size_t)b], 0, 0, 0}, stages, cost});
    }
  std::stable_sort(all.begin(), all.end(),
                   [](const Sized& x, const Sized& y) { return x.stages > y.stages; });
  return all;
}

// When the last of `workers` CTAs ends that take the tiles in this order.
int64_t expanded_end(const std::vector<Sized>& tiles, int workers) {
  std::priority_queue<int64_t, std::vector<int64_t>, std::greater<int64_t>> ends;
  int64_t last = 0;
  for (const Sized& x : tiles) {
    int64_t end = x.cost;
    if ((int64_t)ends.size() == workers) {
      end += ends.top();
      ends.pop();
    }
    ends.push(end);
    last = std::max(last, end);
  }
  return last;
}

void expanded_work(const pa_latent_shape_t& s, const int32_t* lens, const int32_t* qs,
                   const std::vector<int32_t>& cu_q, const std::vector<int32_t>& cu_k, int rows,
                   int workers, Work* w) {
  std::vector<Sized> tiles = expanded_tiles(s, lens, qs, cu_q, cu_k, rows ? rows : kLatentRowsExpanded);
  if (!rows && (int64_t)tiles.size() <= (int64_t)kExpandedFew * workers) {
    std::vector<Sized> halves = expanded_tiles(s, lens, qs, cu_q, cu_k, kLatentRowsExpanded / 2);
    if (expanded_end(halves, workers) * 100 <= expanded_end(tiles, workers) * 95) tiles.swap(halves);
  }
  for (const Sized& x : tiles) w->tiles.push_back(x.t);
}

}  // namespace
}  // namespace pa

extern "C" pa_status_t pa_latent_plan(const pa_latent_shape_t* shape, const int32_t* seq_lens_host,
                                      const int32_t* q_lens_host, int32_t num_sms, int32_t form,
                                      const pa_latent_options_t* options,
                                      pa_latent_plan_t* plan_out) try {
  using namespace pa;
  if (!plan_out) return PA_ERR_INVALID_ARG;
  memset(plan_out, 0, sizeof(*plan_out));
  const pa_status_t st = check_latent_shape(shape);
  if (st != PA_OK) return st;
  const pa_latent_options_t o = options ? *options : pa_latent_options_t{};
  const bool absorbed = form == PA_LATENT_ABSORBED;
  if ((!absorbed && form != PA_LATENT_EXPANDED) || num_sms <= 0 || o.forced_splits < 0 ||
      o.rows_per_tile < 0)
    return PA_ERR_INVALID_ARG;
  if (absorbed ? (o.rows_per_tile != 0 && o.rows_per_tile != kLatentRowsMma &&
                  o.rows_per_tile != kLatentRowsSolo && o.rows_per_tile != kLatentRowsPair)
               : (o.rows_per_tile != 0 && o.rows_per_tile != kLatentRowsExpanded / 2 &&
                  o.rows_per_tile != kLatentRowsExpanded) || o.forced_splits != 0)
    return PA_ERR_INVALID_ARG;
  const int B = shape->batch;
  if (B > 0 && (!seq_lens_host || !q_lens_host)) return PA_ERR_INVALID_ARG;

  std::vector<int32_t> cu_q((size_t)B + 1, 0), cu_k((size_t)B + 1, 0);
  for (int b = 0; b < B; ++b) {
    const int32_t len = seq_lens_host[b], q = q_lens_host[b];
    if (q < 0 || q > len || (int64_t)len > (int64_t)shape->max_pages_per_seq * shape->page_size)
      return PA_ERR_INVALID_ARG;
    // the packed rows are indexed with 32 bits, heads included; the kernels look
    // a few stages past the last token
    if (((int64_t)cu_q[(size_t)b] + q) * shape->num_heads > INT32_MAX ||
        (int64_t)cu_k[(size_t)b] + len > INT32_MAX - 65536)
      return PA_ERR_INVALID_ARG;
    cu_q[(size_t)b + 1] = cu_q[(size_t)b] + q;
    cu_k[(size_t)b + 1] = cu_k[(size_t)b] + len;
  }
  Work w;
  int rows = kLatentRowsExpanded;
  if (absorbed) {
    // The kernel with the least empty rows for the sequence with most of them: all
    // rows of a tile share one pass over its tokens, so a second tile reads the
    // cache again.  Batches of 64 sequences of 500 to 8001 tokens, in us with
    // tiles of 16, 64 and 128 rows: 32 rows a sequence 117, 65.7, 71.6; 64 rows
    // 225, 72, 77; 80 rows 279, 122, 78.  (Short calls differ by less: four
    // sequences of 200 to 600 tokens with 40 rows 10.4, 11.2, 14.1.)
    int64_t most = 0;  // query rows of one sequence
    for (int b = 0; b < B; ++b)
      most = std::max(most, (int64_t)q_lens_host[b] * shape->num_heads);
    rows = o.rows_per_tile             ? o.rows_per_tile
           : most <= kLatentRowsMma  ? kLatentRowsMma
           : most <= kLatentRowsSolo ? kLatentRowsSolo
                                     : kLatentRowsPair;
  }
  if (absorbed)
    absorbed_work(*shape, seq_lens_host, q_lens_host, cu_q, rows,
                  rows == kLatentRowsPair ? std::max(1, num_sms / 2) : num_sms, o.forced_splits, &w);
  else
    expanded_work(*shape, seq_lens_host, q_lens_host, cu_q, cu_k, o.rows_per_tile, num_sms, &w);
  const size_t ranges = absorbed ? w.ranges.size() - 1 : w.tiles.size();
  if (ranges > (size_t)INT32_MAX || w.segments.size() > (size_t)INT32_MAX ||
      w.slots > INT32_MAX / rows)
    return PA_ERR_INVALID_ARG;
  const LatentLayout lay = latent_layout(B, form, rows, (int)ranges, (int)w.segments.size(),
                                         (int)w.merges.size(), (int)w.slots);
  char* blob = (char*)calloc(1, lay.blob_bytes);
  if (!blob) return PA_ERR_NO_MEMORY;
  const uint64_t id = g_latent_ids.fetch_add(1);
  const int32_t header[16] = {(int32_t)kLatentMagic, B, cu_q[(size_t)B], cu_k[(size_t)B],
                              (int32_t)(id & 0xffffffffu), (int32_t)(id >> 32), form, rows,
                              (int32_t)ranges, (int32_t)w.segments.size(),
                              (int32_t)w.merges.size(), (int32_t)w.slots};
  memcpy(blob, header, sizeof(header));
  memcpy(blob + lay.cu_q, cu_q.data(), 4 * cu_q.size());
  memcpy(blob + lay.cu_k, cu_k.data(), 4 * cu_k.size());
  if (absorbed) {
    memcpy(blob + lay.ranges, w.ranges.data(), 4 * w.ranges.size());
    if (!w.segments.empty())
      memcpy(blob + lay.work, w.segments.data(), sizeof(LatentSegment) * w.segments.size());
    if (!w.merges.empty())
      memcpy(blob + lay.merges, w.merges.data(), sizeof(LatentMerge) * w.merges.size());
  } else if (!w.tiles.empty()) {
    memcpy(blob + lay.work, w.tiles.data(), sizeof(LatentTile) * w.tiles.size());
  }
  plan_out->shape = *shape;
  plan_out->form = form;
  plan_out->rows_per_tile = rows;
  plan_out->num_ranges = (int32_t)ranges;
  plan_out->num_segments = (int32_t)w.segments.size();
  plan_out->num_merges = (int32_t)w.merges.size();
  plan_out->num_slots = (int32_t)w.slots;
  plan_out->total_q = cu_q[(size_t)B];
  plan_out->total_k = cu_k[(size_t)B];
  plan_out->owns_blob = 1;
  plan_out->plan_id = id;
  plan_out->blob_bytes = lay.blob_bytes;
  plan_out->workspace_bytes = lay.total;
  plan_out->host_blob = blob;
  plan_out->wait_limit_ns = o.wait_limit_ns;
  return PA_OK;
} catch (...) {  // the only exceptions here are failed allocations
  return PA_ERR_NO_MEMORY;
}

extern "C" void pa_latent_plan_free(pa_latent_plan_t* plan) {
  if (!plan) return;
  if (plan->owns_blob && plan->host_blob) free(plan->host_blob);
  plan->host_blob = nullptr;
  plan->blob_bytes = 0;
}
