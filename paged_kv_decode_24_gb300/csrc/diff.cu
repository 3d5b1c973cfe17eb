// Differential attention: the planner's entry point and the calls.
#include <math.h>
#include <stdlib.h>
#include <string.h>

#include <new>

#include "diff.h"
#include "latent_launch.cuh"
#include "latent_params.h"

namespace pa {

cudaError_t launch_diff_decode(const DiffDecodeParams& p, int head_dim, int group, int dtype, int grid,
                               cudaStream_t stream) {
  return head_dim == 64 ? launch_diff_decode_d64(p, group, dtype, grid, stream)
                        : launch_diff_decode_d128(p, group, dtype, grid, stream);
}

namespace {

bool aligned(const void* p, uintptr_t a) { return p && ((uintptr_t)p % a) == 0; }

pa_status_t cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return PA_OK;
  (void)cudaGetLastError();  // clear a launch error so that later calls report their own
  return PA_ERR_CUDA;
}

pa_status_t check_diff_shape(const pa_shape_t* s) {
  const pa_status_t st = check_shape(s);
  if (st != PA_OK) return st;
  return s->num_kv_heads % 2 == 0 ? PA_OK : PA_ERR_UNSUPPORTED;
}

// What the kernel's tasks see: a KV head for each pair, its 2G queries as rows
// and values of 2D dims.
pa_shape_t pair_shape(const pa_shape_t& s) {
  pa_shape_t p = s;
  p.num_kv_heads = s.num_kv_heads / 2;
  p.head_dim = 2 * s.head_dim;
  return p;
}

pa_status_t check_weights(const pa_diff_t* d, float scale, float* qscale, DiffEpilogue* e) {
  if (!d || !aligned(d->lambda, 4) || (d->norm_weight && !aligned(d->norm_weight, 16)))
    return PA_ERR_INVALID_ARG;
  if (!(d->norm_eps >= 0.f) || !isfinite(d->norm_eps) || !isfinite(d->factor)) return PA_ERR_INVALID_ARG;
  *qscale = (float)((double)scale * 1.4426950408889634);  // log2(e)
  if (!(scale > 0.f) || !isfinite(*qscale)) return PA_ERR_INVALID_ARG;
  *e = DiffEpilogue{d->lambda, d->norm_weight, d->norm_eps, d->factor};
  return PA_OK;
}

// A pool [P][Hkv][16][D] of 16-bit elements as a 4-D tensor, innermost
// first, with boxes of 64 elements x 16 rows x `heads` and the 128-byte swizzle.
bool encode_pool(CUtensorMap* map, const void* pool, const pa_shape_t& s, int heads) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = latent_map_encoder();
  if (!enc) return false;
  const cuuint64_t row = (cuuint64_t)s.head_dim * 2;
  cuuint64_t dims[4] = {(cuuint64_t)s.head_dim, (cuuint64_t)kPageSize, (cuuint64_t)s.num_kv_heads,
                        (cuuint64_t)s.num_pages};
  cuuint64_t strides[3] = {row, row * kPageSize, row * kPageSize * s.num_kv_heads};
  cuuint32_t box[4] = {64, (cuuint32_t)kPageSize, (cuuint32_t)heads, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUtensorMapDataType ty = s.dtype == PA_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                         : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return enc(map, ty, 4, const_cast<void*>(pool), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace pa

extern "C" pa_status_t pa_diff_plan(const pa_shape_t* shape, const int32_t* seq_lens_host,
                                    int32_t num_sms, const pa_diff_options_t* options,
                                    pa_diff_plan_t* plan_out) {
  using namespace pa;
  if (!plan_out) return PA_ERR_INVALID_ARG;
  memset(plan_out, 0, sizeof(*plan_out));
  pa_status_t st = check_diff_shape(shape);
  if (st != PA_OK) return st;
  const pa_diff_options_t o = options ? *options : pa_diff_options_t{};
  if (num_sms <= 0 || o.forced_splits < 0 || o.min_chunk_pages < 0) return PA_ERR_INVALID_ARG;
  const pa_shape_t pairs = pair_shape(*shape);
  const bool filled = (int64_t)shape->batch * (shape->num_kv_heads / 2) >= num_sms;
  const PlanGeometry geo{kDiffMagic, diff_ctas_per_sm(shape->head_dim),
                         filled ? diff_min_chunk(shape->head_dim) : kDiffShortChunkPages, true};
  pa_plan_options_t po{};
  po.min_chunk_pages = o.min_chunk_pages;
  pa_plan_t plan{};
  try {
    st = plan_tasks(&pairs, geo, seq_lens_host, num_sms, o.forced_splits, po, nullptr, 0, true, &plan);
  } catch (const std::bad_alloc&) {
    st = PA_ERR_NO_MEMORY;
  }
  if (st != PA_OK) return st;
  plan_out->shape = *shape;
  plan_out->num_work_items = plan.num_work_items;
  plan_out->num_groups = plan.num_groups;
  plan_out->num_split_items = plan.num_split_items;
  plan_out->max_splits = plan.max_splits;
  plan_out->num_ctas = plan.num_ctas;
  plan_out->num_shared_ctas = plan.num_shared_ctas;
  plan_out->owns_blob = 1;
  plan_out->plan_id = plan.plan_id;
  plan_out->blob_bytes = plan.blob_bytes;
  const int rows = 2 * (shape->num_q_heads / shape->num_kv_heads);
  plan_out->workspace_bytes = diff_workspace_bytes(
      layout(plan.num_work_items, plan.num_groups, plan.num_split_items, rows, pairs.head_dim),
      plan.num_split_items, rows);
  plan_out->host_blob = plan.host_blob;
  plan_out->wait_limit_ns = o.wait_limit_ns;
  return PA_OK;
}

extern "C" void pa_diff_plan_free(pa_diff_plan_t* plan) {
  if (!plan) return;
  if (plan->owns_blob) free(plan->host_blob);
  plan->owns_blob = 0;
  plan->host_blob = nullptr;
  plan->blob_bytes = 0;
}

extern "C" pa_status_t pa_diff_plan_upload(const pa_diff_plan_t* plan, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  using namespace pa;
  if (!plan || !plan->host_blob || plan->blob_bytes == 0 || !aligned(workspace, 256))
    return PA_ERR_INVALID_ARG;
  if (workspace_bytes < plan->workspace_bytes || workspace_bytes < plan->blob_bytes) return PA_ERR_WORKSPACE;
  return cuda_status(cudaMemcpyAsync(workspace, plan->host_blob, plan->blob_bytes,
                                     cudaMemcpyHostToDevice, (cudaStream_t)stream));
}

extern "C" pa_status_t pa_diff_attention(const pa_shape_t* shape, const pa_diff_plan_t* plan,
                                         const pa_diff_t* diff, const void* q, const void* k_pages,
                                         const void* v_pages, const int32_t* block_table,
                                         const int32_t* seq_lens, float scale, void* out,
                                         void* workspace, size_t workspace_bytes,
                                         int32_t* dev_status, void* stream) {
  using namespace pa;
  pa_status_t st = check_diff_shape(shape);
  if (st != PA_OK) return st;
  if (!plan) return PA_ERR_INVALID_ARG;
  if (!same_plan_shape(plan->shape, *shape)) return PA_ERR_PLAN;
  DiffDecodeParams p{};
  st = check_weights(diff, scale, &p.s.qscale, &p.e);
  if (st != PA_OK) return st;
  if (shape->batch == 0) return PA_OK;
  if (plan->num_work_items <= 0 || plan->num_groups < 0 || plan->num_split_items < 0 || plan->num_ctas <= 0 ||
      plan->num_shared_ctas < 0 || plan->num_shared_ctas > plan->num_ctas)
    return PA_ERR_PLAN;
  const int G = shape->num_q_heads / shape->num_kv_heads, D = shape->head_dim;
  const Layout lay = layout(plan->num_work_items, plan->num_groups, plan->num_split_items, 2 * G, 2 * D);
  if (plan->workspace_bytes != diff_workspace_bytes(lay, plan->num_split_items, 2 * G)) return PA_ERR_PLAN;
  if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(out, 16) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(dev_status, 4) ||
      !aligned(workspace, 256))
    return PA_ERR_INVALID_ARG;
  if (workspace_bytes < plan->workspace_bytes) return PA_ERR_WORKSPACE;
  char* ws = (char*)workspace;
  SplitParams& s = p.s;
  s.q = q;
  s.k_pages = k_pages;
  s.v_pages = v_pages;
  s.block_table = block_table;
  s.seq_lens = seq_lens;
  s.out = out;
  s.ws_header = (const int32_t*)ws;
  s.items = (const int4*)(ws + lay.items_off);
  s.item_slots = (const int2*)(ws + lay.slots_off);
  s.groups = (const int4*)(ws + lay.groups_off);
  s.counters = (int*)(ws + lay.counters_off);
  s.part_lse = (float*)(ws + lay.lse_off);
  s.part_o = (float*)(ws + lay.o_off);
  p.part_sum = (float*)(ws + lay.total);
  s.status = dev_status;
  s.batch = shape->batch;
  s.num_q_heads = shape->num_q_heads;
  s.num_kv_heads = shape->num_kv_heads / 2;
  s.max_pages = shape->max_pages_per_seq;
  s.num_pages = shape->num_pages;
  s.num_items = plan->num_work_items;
  s.num_groups = plan->num_groups;
  s.num_split_items = plan->num_split_items;
  s.num_ctas = plan->num_ctas;
  s.num_shared = plan->num_shared_ctas;
  s.wait_ns = wait_limit_or_default(plan->wait_limit_ns);
  s.fuse_merge = plan->max_splits <= kDiffMergeSplits;
  s.pf_pages = kDiffPrefetchPages;
  s.pf_ctas = sm_count() * diff_ctas_per_sm(D);  // those that may start before the kernel ahead ends
  if (!encode_pool(&s.tmap_k, k_pages, *shape, 2) || !encode_pool(&s.tmap_v, v_pages, *shape, 2))
    return PA_ERR_CUDA;
  cudaError_t e = launch_diff_decode(p, D, G, shape->dtype, plan->num_ctas, (cudaStream_t)stream);
  if (e == cudaSuccess && !s.fuse_merge && s.num_groups > 0)
    e = launch_diff_merge(p, D, G, shape->dtype, (cudaStream_t)stream);
  return cuda_status(e);
}

extern "C" pa_status_t pa_diff_prefill(const pa_shape_t* shape, const pa_prefill_plan_t* plan,
                                       const pa_diff_t* diff, const void* q, const void* k_pages,
                                       const void* v_pages, const int32_t* block_table,
                                       const int32_t* seq_lens, float scale, void* out,
                                       void* workspace, size_t workspace_bytes,
                                       int32_t* dev_status, void* stream) {
  using namespace pa;
  pa_status_t st = check_diff_shape(shape);
  if (st != PA_OK) return st;
  st = check_prefill_call(shape, plan, workspace, workspace_bytes);
  if (st != PA_OK) return st;
  // the plan's tiles come in twos, one for each KV head of a pair
  if (plan->rows_per_tile != kPrefillRowsTc5 || plan->num_tiles % 2 != 0) return PA_ERR_PLAN;
  DiffPrefillParams p{};
  st = check_weights(diff, scale, &p.qscale, &p.e);
  if (st != PA_OK) return st;
  if (shape->batch == 0 || plan->num_tiles == 0) return PA_OK;
  const PrefillLayout lay = prefill_layout(plan->num_tiles, shape->batch);
  if (plan->workspace_bytes != lay.blob_bytes) return PA_ERR_PLAN;
  if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(out, 16) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(dev_status, 4))
    return PA_ERR_INVALID_ARG;
  p.q = q;
  p.out = out;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.ws = (const int32_t*)workspace;
  p.cu = (const int32_t*)((const char*)workspace + lay.cu_off);
  p.status = dev_status;
  p.batch = shape->batch;
  p.num_q_heads = shape->num_q_heads;
  p.num_kv_heads = shape->num_kv_heads;
  p.max_pages = shape->max_pages_per_seq;
  p.num_pages = shape->num_pages;
  p.num_tiles = plan->num_tiles;
  p.total_q = plan->total_q;
  p.wait_ns = wait_limit_or_default(plan->wait_limit_ns);
  if (!encode_pool(&p.tmap_k, k_pages, *shape, 1) || !encode_pool(&p.tmap_v, v_pages, *shape, 2))
    return PA_ERR_CUDA;
  const int G = shape->num_q_heads / shape->num_kv_heads;
  return cuda_status(launch_diff_prefill(p, shape->head_dim, G, shape->dtype, (cudaStream_t)stream));
}
