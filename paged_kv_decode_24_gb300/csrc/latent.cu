// Latent attention: the entry points, and the kernels that move rows.
#include <math.h>

#include <mutex>

#include "device_common.cuh"
#include "latent_params.h"
#include "latent_launch.cuh"

namespace pa {

PFN_cuTensorMapEncodeTiled_v12000 latent_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    else
      (void)cudaGetLastError();
  });
  return fn;
}

namespace {

constexpr int kRowChunks = kLatentRow / 8;    // 16-byte chunks of a row
constexpr int kCChunks = kLatent / 8;         // of its latent

// The sequence of packed row r: the largest b with cu[b] <= r (the last of
// equal ones, so sequences without rows are passed over).  The warp's lanes
// probe 32 places at once.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int batch, int r, int lane) {
  int lo = 0, n = batch;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lo + lane * step;
    const unsigned below = __ballot_sync(kFull, lane * step < n && cu[at] <= r);
    const int k = 31 - __clz(below | 1u);
    n = min(step, n - k * step);
    lo += k * step;
  }
  return lo;
}

// Two consecutive packed rows per warp and turn: 144 chunks of 16 bytes, up to
// five a lane, in flight at once behind one look-up of the rows' places (lane
// u looks up row u).  Both directions only move bytes.  Measured against the
// copy bandwidth: contexts of 292 MB read back at 90 to 93 %, prompts of 125 MB
// written at 85 % (one row per warp 83 and 85 %, four 89 and 67 %: the lanes'
// registers then leave too few warps), with up to 16 blocks an SM (8: 90 and
// 83 %).
constexpr int kWarpRows = 2;
constexpr int kRowBlocks = 152 * 16;

template <bool APPEND>
__global__ void __launch_bounds__(256) latent_rows_kernel(const LatentRowsParams p) {
  constexpr int CHUNKS = (kWarpRows * kRowChunks + 31) / 32;  // of a lane
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int32_t* cu_q = p.ws + 16;
  const int32_t* cu_k = cu_q + p.batch + 1;
  const int32_t* cu = APPEND ? cu_q : cu_k;
  // the plan is written by the upload alone: it may be read before the wait
  const bool planned = p.ws[0] == (int)kLatentMagic && p.ws[1] == p.batch && p.ws[APPEND ? 2 : 3] == p.total;
  const int64_t turns = ((int64_t)p.total + kWarpRows - 1) / kWarpRows;
  const int64_t step = (int64_t)gridDim.x * (blockDim.x >> 5);
  int64_t turn = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  pdl_wait_primary();
  if (!planned) {
    if (threadIdx.x == 0) set_status(p.status, PA_DEV_PLAN_MISMATCH);
    return;
  }
  for (; turn < turns; turn += step) {
    const int r0 = (int)(turn * kWarpRows);
    int b = sequence_of(cu, p.batch, r0, lane);
    // lane u: where row r0 + u is cached, -1 for a bad page or past the end
    int64_t at = -1;
    if (lane < kWarpRows && r0 + lane < p.total) {
      const int r = r0 + lane;
      while (r >= cu[b + 1]) ++b;
      int t = r - cu[b];
      if (APPEND) t += cu_k[b + 1] - cu_k[b] - (cu_q[b + 1] - cu_q[b]);
      const int j = t / p.page_size;
      const int page = j < p.max_pages ? p.block_table[(int64_t)b * p.max_pages + j] : -1;
      if (page >= 0 && page < p.num_pages)
        at = ((int64_t)page * p.page_size + t % p.page_size) * kRowChunks;
      else
        set_status(p.status, PA_DEV_BAD_PAGE);
    }
    uint4 v[CHUNKS];
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      const int c = lane + 32 * i, u = c / kRowChunks, ch = c % kRowChunks;
      const int64_t cached = __shfl_sync(kFull, at, u);
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (cached < 0 || u >= kWarpRows) continue;
      if (!APPEND)
        v[i] = static_cast<const uint4*>(p.pages)[cached + ch];
      else if (ch < kCChunks)
        v[i] = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.c) +
                                              (r0 + u) * p.c_stride)[ch];
      else
        v[i] = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.r) +
                                              (r0 + u) * p.r_stride)[ch - kCChunks];
    }
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      const int c = lane + 32 * i, u = c / kRowChunks, ch = c % kRowChunks;
      const int64_t cached = __shfl_sync(kFull, at, u);
      if (u >= kWarpRows) continue;
      if (APPEND) {
        if (cached >= 0) static_cast<uint4*>(p.pages)[cached + ch] = v[i];
      } else if (r0 + u < p.total) {
        static_cast<uint4*>(p.rows)[(int64_t)(r0 + u) * kRowChunks + ch] = v[i];
      }
    }
  }
}

template <bool APPEND>
cudaError_t launch_rows(const LatentRowsParams& p, cudaStream_t stream) {
  static std::atomic<unsigned long long> configured{0};
  const int64_t blocks = ((int64_t)p.total + 8 * kWarpRows - 1) / (8 * kWarpRows);
  const int grid = (int)(blocks < kRowBlocks ? blocks : kRowBlocks);
  return launch_latent(latent_rows_kernel<APPEND>, 0, configured, grid, 256, stream, p);
}

}  // namespace

cudaError_t launch_latent_append(const LatentRowsParams& p, cudaStream_t stream) {
  return launch_rows<true>(p, stream);
}
cudaError_t launch_latent_gather(const LatentRowsParams& p, cudaStream_t stream) {
  return launch_rows<false>(p, stream);
}

namespace {

bool aligned(const void* p, uintptr_t a) { return p && ((uintptr_t)p % a) == 0; }

pa_status_t cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return PA_OK;
  (void)cudaGetLastError();  // clear a launch error so that later calls report their own
  return PA_ERR_CUDA;
}

// What every call checks first: the shape, the plan against it, and the workspace.
// form < 0: a plan of either form serves.
pa_status_t check_latent_call(const pa_latent_shape_t* s, const pa_latent_plan_t* plan, int form,
                              const void* workspace, size_t workspace_bytes) {
  const pa_status_t st = check_latent_shape(s);
  if (st != PA_OK) return st;
  if (!plan) return PA_ERR_INVALID_ARG;
  const pa_latent_shape_t& a = plan->shape;
  if (a.batch != s->batch || a.num_heads != s->num_heads || a.head_dim != s->head_dim ||
      a.latent_dim != s->latent_dim || a.rope_dim != s->rope_dim || a.page_size != s->page_size ||
      a.max_pages_per_seq != s->max_pages_per_seq)
    return PA_ERR_PLAN;
  if ((plan->form != PA_LATENT_ABSORBED && plan->form != PA_LATENT_EXPANDED) ||
      (form >= 0 && plan->form != form))
    return PA_ERR_PLAN;
  const int rows = plan->rows_per_tile;
  const bool absorbed_rows =
      rows == kLatentRowsMma || rows == kLatentRowsSolo || rows == kLatentRowsPair;
  if (plan->form == PA_LATENT_ABSORBED ? !absorbed_rows : rows != kLatentRowsExpanded)
    return PA_ERR_PLAN;
  if (plan->num_ranges < 0 || plan->num_segments < 0 || plan->num_merges < 0 ||
      plan->num_slots < 0 || plan->total_q < 0 || plan->total_k < 0)
    return PA_ERR_PLAN;
  const LatentLayout l = latent_layout(s->batch, plan->form, plan->rows_per_tile, plan->num_ranges,
                                       plan->num_segments, plan->num_merges, plan->num_slots);
  if (plan->workspace_bytes != l.total) return PA_ERR_PLAN;
  if (s->batch == 0) return PA_OK;
  if (!aligned(workspace, 16)) return PA_ERR_INVALID_ARG;
  if (workspace_bytes < plan->workspace_bytes) return PA_ERR_WORKSPACE;
  return PA_OK;
}

// The scale of scores in log2 units; infinite where it leaves fp32.
float log2_scale(float scale) { return (float)((double)scale * 1.4426950408889634); }

// Strides in elements: multiples of 16 bytes below 2^40 bytes.
bool stride_ok(int64_t stride, int width) {
  return stride >= width && stride % 8 == 0 && stride < (int64_t)1 << 39;
}

// Tokens and heads of D values whose strides keep them apart, tokens outside
// heads or heads outside tokens.
bool planes_ok(int64_t token, int64_t head, int64_t tokens, int64_t heads, int d) {
  if (!stride_ok(token, 8) || !stride_ok(head, 8)) return false;
  const bool token_major = token >= head;
  const int64_t inner = token_major ? head : token, outer = token_major ? token : head;
  const int64_t n_inner = token_major ? heads : tokens, n_outer = token_major ? tokens : heads;
  // inner < 2^39 and n_inner < 2^31: compared by division
  if (n_inner > 1 && inner < d) return false;
  return n_outer <= 1 || (outer >= d && (n_inner <= 1 || (outer - d) / inner >= n_inner - 1));
}

LatentRowsParams rows_params(const pa_latent_shape_t* s, const int32_t* block_table,
                             const void* pages, const void* workspace, int32_t* dev_status,
                             int32_t total) {
  LatentRowsParams p{};
  p.pages = const_cast<void*>(pages);
  p.block_table = block_table;
  p.ws = static_cast<const int32_t*>(workspace);
  p.status = dev_status;
  p.batch = s->batch;
  p.total = total;
  p.max_pages = s->max_pages_per_seq;
  p.num_pages = s->num_pages;
  p.page_size = s->page_size;
  return p;
}

}  // namespace
}  // namespace pa

extern "C" pa_status_t pa_latent_plan_upload(const pa_latent_plan_t* plan, void* workspace,
                                             size_t workspace_bytes, void* stream) {
  using namespace pa;
  if (!plan || !plan->host_blob || !aligned(workspace, 16)) return PA_ERR_INVALID_ARG;
  if (workspace_bytes < plan->workspace_bytes || workspace_bytes < plan->blob_bytes)
    return PA_ERR_WORKSPACE;
  return cuda_status(cudaMemcpyAsync(workspace, plan->host_blob, plan->blob_bytes,
                                     cudaMemcpyHostToDevice, (cudaStream_t)stream));
}

extern "C" pa_status_t pa_latent_append(const pa_latent_shape_t* shape,
                                        const pa_latent_plan_t* plan, const void* c_new,
                                        int64_t c_stride, const void* r_new, int64_t r_stride,
                                        void* pages, const int32_t* block_table,
                                        const void* workspace, size_t workspace_bytes,
                                        int32_t* dev_status, void* stream) {
  using namespace pa;
  const pa_status_t st = check_latent_call(shape, plan, -1, workspace, workspace_bytes);
  if (st != PA_OK) return st;
  if (shape->batch == 0 || plan->total_q == 0) return PA_OK;
  if (!aligned(c_new, 16) || !aligned(r_new, 16) || !aligned(pages, 16) ||
      !aligned(block_table, 4) || !aligned(dev_status, 4))
    return PA_ERR_INVALID_ARG;
  if (!stride_ok(c_stride, kLatent) || !stride_ok(r_stride, kRope)) return PA_ERR_INVALID_ARG;
  LatentRowsParams p = rows_params(shape, block_table, pages, workspace, dev_status, plan->total_q);
  p.c = c_new;
  p.r = r_new;
  p.c_stride = c_stride;
  p.r_stride = r_stride;
  return cuda_status(launch_latent_append(p, (cudaStream_t)stream));
}

extern "C" pa_status_t pa_latent_gather(const pa_latent_shape_t* shape,
                                        const pa_latent_plan_t* plan, const void* pages,
                                        const int32_t* block_table, void* rows,
                                        const void* workspace, size_t workspace_bytes,
                                        int32_t* dev_status, void* stream) {
  using namespace pa;
  const pa_status_t st = check_latent_call(shape, plan, -1, workspace, workspace_bytes);
  if (st != PA_OK) return st;
  if (shape->batch == 0 || plan->total_k == 0) return PA_OK;
  if (!aligned(rows, 16) || !aligned(pages, 16) || !aligned(block_table, 4) ||
      !aligned(dev_status, 4))
    return PA_ERR_INVALID_ARG;
  LatentRowsParams p = rows_params(shape, block_table, pages, workspace, dev_status, plan->total_k);
  p.rows = rows;
  return cuda_status(launch_latent_gather(p, (cudaStream_t)stream));
}

extern "C" pa_status_t pa_latent_attention(const pa_latent_shape_t* shape,
                                           const pa_latent_plan_t* plan, const void* q,
                                           const void* pages, const int32_t* block_table,
                                           float scale, void* out, void* workspace,
                                           size_t workspace_bytes, int32_t* dev_status,
                                           void* stream) {
  using namespace pa;
  const pa_status_t st =
      check_latent_call(shape, plan, PA_LATENT_ABSORBED, workspace, workspace_bytes);
  if (st != PA_OK) return st;
  if (shape->batch == 0 || plan->total_q == 0) return PA_OK;
  if (!aligned(q, 16) || !aligned(pages, 16) || !aligned(out, 16) || !aligned(block_table, 4) ||
      !aligned(dev_status, 4))
    return PA_ERR_INVALID_ARG;
  const float qscale = log2_scale(scale);
  if (!(scale > 0.f) || !isfinite(qscale)) return PA_ERR_INVALID_ARG;
  if (plan->num_ranges < 1 || plan->num_segments < plan->num_ranges) return PA_ERR_PLAN;
  LatentParams p{};
  const LatentLayout l = latent_layout(shape->batch, plan->form, plan->rows_per_tile,
                                       plan->num_ranges, plan->num_segments, plan->num_merges,
                                       plan->num_slots);
  char* ws = static_cast<char*>(workspace);
  p.q = q;
  p.out = out;
  p.block_table = block_table;
  p.ws = reinterpret_cast<const int32_t*>(ws);
  p.ranges = reinterpret_cast<const int32_t*>(ws + l.ranges);
  p.segments = reinterpret_cast<const LatentSegment*>(ws + l.work);
  p.merges = reinterpret_cast<const LatentMerge*>(ws + l.merges);
  p.part_lse = reinterpret_cast<float*>(ws + l.lse);
  p.part_o = reinterpret_cast<float*>(ws + l.o);
  p.status = dev_status;
  p.wait_ns = wait_limit_or_default(plan->wait_limit_ns);
  p.qscale = qscale;
  p.batch = shape->batch;
  p.heads = shape->num_heads;
  p.max_pages = shape->max_pages_per_seq;
  p.num_pages = shape->num_pages;
  p.page_size = shape->page_size;
  p.num_ranges = plan->num_ranges;
  p.num_segments = plan->num_segments;
  p.num_merges = plan->num_merges;
  p.num_slots = plan->num_slots;
  p.total_q = plan->total_q;
  p.rows = plan->rows_per_tile;
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = plan->rows_per_tile == kLatentRowsPair   ? launch_latent_pair(p, *shape, pages, s)
                  : plan->rows_per_tile == kLatentRowsSolo ? launch_latent_solo(p, *shape, pages, s)
                                                           : launch_latent_mma(p, *shape, pages, s);
  if (e == cudaSuccess && p.num_merges > 0) e = launch_latent_merge(p, shape->dtype, s);
  return cuda_status(e);
}

extern "C" pa_status_t pa_latent_prefill(const pa_latent_shape_t* shape,
                                         const pa_latent_plan_t* plan, const void* q,
                                         const void* k, int64_t k_token_stride,
                                         int64_t k_head_stride, const void* k_rope,
                                         int64_t kr_stride, const void* v, int64_t v_token_stride,
                                         int64_t v_head_stride, float scale, void* out,
                                         void* workspace, size_t workspace_bytes,
                                         int32_t* dev_status, void* stream) {
  using namespace pa;
  const pa_status_t st =
      check_latent_call(shape, plan, PA_LATENT_EXPANDED, workspace, workspace_bytes);
  if (st != PA_OK) return st;
  if (shape->batch == 0 || plan->total_q == 0) return PA_OK;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(k_rope, 16) || !aligned(v, 16) ||
      !aligned(out, 16) || !aligned(dev_status, 4))
    return PA_ERR_INVALID_ARG;
  const float qscale = log2_scale(scale);
  if (!(scale > 0.f) || !isfinite(qscale)) return PA_ERR_INVALID_ARG;
  if (!planes_ok(k_token_stride, k_head_stride, plan->total_k, shape->num_heads, shape->head_dim) ||
      !planes_ok(v_token_stride, v_head_stride, plan->total_k, shape->num_heads, shape->head_dim) ||
      !stride_ok(kr_stride, kRope))
    return PA_ERR_INVALID_ARG;
  LatentPrefillParams p{};
  const LatentLayout l = latent_layout(shape->batch, plan->form, plan->rows_per_tile,
                                       plan->num_ranges, 0, 0, 0);
  char* ws = static_cast<char*>(workspace);
  p.q = q;
  p.k = k;
  p.k_rope = k_rope;
  p.v = v;
  p.out = out;
  p.ws = reinterpret_cast<const int32_t*>(ws);
  p.tiles = reinterpret_cast<const LatentTile*>(ws + l.work);
  p.status = dev_status;
  p.k_token = k_token_stride;
  p.k_head = k_head_stride;
  p.kr_token = kr_stride;
  p.v_token = v_token_stride;
  p.v_head = v_head_stride;
  p.wait_ns = wait_limit_or_default(plan->wait_limit_ns);
  p.qscale = qscale;
  p.batch = shape->batch;
  p.heads = shape->num_heads;
  p.num_tiles = plan->num_ranges;
  p.total_q = plan->total_q;
  p.total_k = plan->total_k;
  return cuda_status(
      launch_latent_prefill(p, shape->head_dim, shape->dtype, (cudaStream_t)stream));
}
