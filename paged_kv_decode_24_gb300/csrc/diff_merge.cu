// Differential one-token attention: the join of split sequences as a kernel of
// its own, for plans with many splits.
//
// A head's output is the difference of two rows, each joined from ns partials
// (o_s, m_s, l_s): with M = max_s m_s, w_s = 2^(m_s - M) l_s,
//   row = sum_s w_s o_s / sum_s w_s.
// Two rows of 2D fp32 values a split and head have to be read: with one SM doing it
// for all heads of a pair (the last task of the pair in the split kernel), 76
// splits of four heads of 128 are 620 KB through one SM.  Here a CTA joins one head,
// its threads a sixteenth of the splits each: sixteen lanes of splits by VD / 4 groups
// of four dims.  Bound by a launch, and by three dependent reads (plan, sums, values):
// 5 to 6 us of the 28.5 of a context of 32,768 tokens (76 splits of 4 pairs of 128).  64
// registers a thread, all of an SM's: none of its CTAs starts beside the split kernel's.
#include <math.h>

#include <atomic>

#include "diff_decode.cuh"
#include "latent_launch.cuh"

namespace pa {

namespace {

constexpr int kLanes = 16;  // threads that share a group of four dims

template <typename T, int D>
__global__ void __launch_bounds__(2 * D / 4 * kLanes) diff_merge_kernel(const __grid_constant__ DiffDecodeParams dp,
                                                                        int group_size) {
  constexpr int VD = 2 * D, QUADS = VD / 4, THREADS = QUADS * kLanes;
  const SplitParams& p = dp.s;
  __shared__ float weight[2][kMaxSplits];
  __shared__ float norm[2];  // 1 / sum of the weights
  __shared__ int missing;    // a split gave up
  __shared__ float4 part[kLanes][2][QUADS];
  const int gi = blockIdx.x / group_size, h = blockIdx.x % group_size;
  // the plan is written by the upload alone: it may be read before the wait
  const int4 hdr = *reinterpret_cast<const int4*>(p.ws_header);
  const int2 hdr_ctas = *reinterpret_cast<const int2*>(p.ws_header + 8);
  const int4 grp = gi < p.num_groups ? p.groups[gi] : make_int4(0, 0, 0, 0);  // {seq, pair, splits, first slot}
  if (threadIdx.x == 0) missing = 0;
  pdl_launch_dependents();
  pdl_wait_primary();  // the partials are there
  const int ns = grp.z, off = grp.w, R = 2 * group_size;
  // (The split kernel's own checks of the plan: where it refuses one, nothing is joined.)
  if (hdr.x != (int)kDiffMagic || hdr.y != p.num_items || hdr.z != p.num_groups || hdr.w != p.num_split_items ||
      hdr_ctas.x != p.num_ctas || hdr_ctas.y != p.num_shared || gi >= p.num_groups || ns < 1 ||
      ns > kMaxSplits || off < 0 || off + ns > p.num_split_items || grp.x < 0 || grp.x >= p.batch || grp.y < 0 ||
      grp.y >= p.num_kv_heads) {
    if (threadIdx.x == 0) set_status(p.status, PA_DEV_PLAN_MISMATCH);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = threadIdx.x % QUADS, sl = threadIdx.x / QUADS;
  const float* o = p.part_o + ((size_t)off * R + h) * VD + 4 * quad;
  constexpr int BATCH = 4;
  float4 x[2][BATCH];
  auto load = [&](int s0) {
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const int s = s0 + u * kLanes;
#pragma unroll
      for (int m = 0; m < 2; ++m)
        x[m][u] = s < ns ? __ldcg(reinterpret_cast<const float4*>(o + ((size_t)s * R + m * group_size) * VD))
                         : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  load(sl);  // on their way while the weights are made
  __syncthreads();
  if (warp < 2) {  // a map each: the splits' weights
    const size_t first = (size_t)off * R + warp * group_size + h;
    // the lane's own sums, where the joined values will be
    float* sum = reinterpret_cast<float*>(part) + warp * kMaxSplits;
    float top = -INFINITY;
    bool lost = false;
#pragma unroll 4
    for (int s = lane; s < ns; s += 32) {
      const float v = __ldcg(p.part_lse + first + (size_t)s * R);
      weight[warp][s] = v;
      sum[s] = __ldcg(dp.part_sum + first + (size_t)s * R);
      lost = lost || isnan(v);
      top = fmaxf(top, v);
    }
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, m));
    float z = 0.f;
    for (int s = lane; s < ns; s += 32) {
      const float w = diff_split_weight(weight[warp][s], sum[s], top);
      weight[warp][s] = w;
      z += w;
    }
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) z += __shfl_xor_sync(kFull, z, m);
    if (lane == 0) norm[warp] = z == 0.f ? 0.f : 1.f / z;
    if (lost) missing = 1;
  }
  __syncthreads();
  if (missing) return;  // a split gave up: the head's output stays unwritten
  float4 acc[2];
  acc[0] = acc[1] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = sl; s0 < ns; s0 += kLanes * BATCH) {
    if (s0 != sl) load(s0);
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const int s = s0 + u * kLanes;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const float w = s < ns ? weight[m][s] : 0.f;
        acc[m].x = fmaf(w, x[m][u].x, acc[m].x);
        acc[m].y = fmaf(w, x[m][u].y, acc[m].y);
        acc[m].z = fmaf(w, x[m][u].z, acc[m].z);
        acc[m].w = fmaf(w, x[m][u].w, acc[m].w);
      }
    }
  }
  part[sl][0][quad] = acc[0];
  part[sl][1][quad] = acc[1];
  __syncthreads();
  if (warp > 0) return;
  float4 r[2][VD / 128];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int i = 0; i < VD / 128; ++i) {
      float4 v = part[0][m][32 * i + lane];
#pragma unroll
      for (int k = 1; k < kLanes; ++k) {
        const float4 y = part[k][m][32 * i + lane];
        v = make_float4(v.x + y.x, v.y + y.y, v.z + y.z, v.w + y.w);
      }
      r[m][i] = make_float4(v.x * norm[m], v.y * norm[m], v.z * norm[m], v.w * norm[m]);
    }
  const size_t head = (size_t)grp.y * group_size + h;
  diff_write_head<T, VD>(dp.e, __ldg(dp.e.lambda + head), r[0], r[1], lane,
                         static_cast<T*>(p.out) + ((size_t)grp.x * p.num_kv_heads * group_size + head) * VD);
  static_assert(THREADS >= 64, "a warp for each map");
  static_assert(2 * kMaxSplits * sizeof(float) <= sizeof(part), "the sums fit where the values go");
}

template <typename T, int D>
cudaError_t launch_t(const DiffDecodeParams& p, int group, cudaStream_t stream) {
  static std::atomic<unsigned long long> configured{0};
  return launch_latent(diff_merge_kernel<T, D>, 0, configured, p.s.num_groups * group, 2 * D / 4 * kLanes, stream,
                       p, group);
}

}  // namespace

cudaError_t launch_diff_merge(const DiffDecodeParams& p, int head_dim, int group, int dtype,
                              cudaStream_t stream) {
  const bool bf = dtype == PA_DTYPE_BF16;
  if (head_dim == 64) return bf ? launch_t<__nv_bfloat16, 64>(p, group, stream) : launch_t<__half, 64>(p, group, stream);
  return bf ? launch_t<__nv_bfloat16, 128>(p, group, stream) : launch_t<__half, 128>(p, group, stream);
}

}  // namespace pa
