// Expanded latent attention of prompts (mma.sync): keys of D + 64 dims whose
// last 64 are shared by the heads, values of D dims, causal.
//
// A CTA owns 64 query tokens of one head, 16 per warp, with q in registers.
// Stages of 64 tokens' keys and values are staged in shared memory; scores,
// online softmax and output stay in registers.
#include <math.h>

#include "decode_tc.cuh"
#include "device_common.cuh"
#include "elem.cuh"
#include "latent_params.h"
#include "split_launch.cuh"

namespace pa {

namespace {

constexpr int kTok = 64;

template <int D>
struct PrefillLayout1 {
  static constexpr int KP = (D + kRope) * 2 + 16;  // bytes per key row (padded: conflict-free ldmatrix)
  static constexpr int VP = D * 2 + 16;
  static constexpr int K = 0;
  static constexpr int V = K + kTok * KP;
  static constexpr int BYTES = V + kTok * VP;
};

template <typename T, int D>
__global__ void __launch_bounds__(128)
    latent_prefill_kernel(const __grid_constant__ LatentPrefillParams p) {
  using L = PrefillLayout1<D>;
  constexpr int DK = D + kRope;
  extern __shared__ __align__(16) unsigned char sm[];
  const uint32_t sbase = smem_u32(sm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  pdl_launch_dependents();
  pdl_wait_primary();
  const int4 h0 = reinterpret_cast<const int4*>(p.ws)[0];
  if (h0.x != (int)kLatentMagic || h0.y != p.batch || h0.z != p.total_q || h0.w != p.total_k ||
      p.ws[6] != PA_LATENT_EXPANDED || p.ws[7] != kLatentRowsExpanded || p.ws[8] != p.num_tiles) {
    if (threadIdx.x == 0) set_status(p.status, PA_DEV_PLAN_MISMATCH);
    return;
  }
  const LatentTile tile = p.tiles[blockIdx.x];
  int cq = 0, qn = 0, ck = 0, len = 0;
  bool bad = tile.b < 0 || tile.b >= p.batch || tile.head < 0 || tile.head >= p.heads || tile.tok0 < 0 ||
             tile.ntok < 1 || tile.ntok > kLatentRowsExpanded;
  if (!bad) {
    cq = p.cu_q[tile.b];
    qn = p.cu_q[tile.b + 1] - cq;
    ck = p.cu_k[tile.b];
    len = p.cu_k[tile.b + 1] - ck;
    bad = cq < 0 || ck < 0 || cq + qn > p.total_q || ck + len > p.total_k || qn > len ||
          tile.tok0 + tile.ntok > qn;
  }
  if (bad) {
    if (threadIdx.x == 0) set_status(p.status, PA_DEV_PLAN_MISMATCH);
    return;
  }
  const int pos0 = len - qn + tile.tok0;
  const int span = pos0 + tile.ntok;
  const int row0 = 16 * warp + g;
  uint32_t qa[DK / 16][4];
  const T* q = static_cast<const T*>(p.q) + ((int64_t)(cq + tile.tok0) * p.heads + tile.head) * DK + 2 * t4;
#pragma unroll
  for (int ks = 0; ks < DK / 16; ++ks)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int row = row0 + (c & 1) * 8;
      qa[ks][c] = row < tile.ntok ? __ldg(reinterpret_cast<const unsigned int*>(
                                        q + (int64_t)row * p.heads * DK + ks * 16 + (c >> 1) * 8))
                                  : 0u;
    }
  float o[D / 8][4];
#pragma unroll
  for (int n = 0; n < D / 8; ++n)
#pragma unroll
    for (int c = 0; c < 4; ++c) o[n][c] = 0.f;
  float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
  const int lim[2] = {row0 < tile.ntok ? pos0 + row0 : -1,
                      row0 + 8 < tile.ntok ? pos0 + row0 + 8 : -1};
  const T* kp = static_cast<const T*>(p.k) + ck * p.k_token + tile.head * p.k_head;
  const T* vp = static_cast<const T*>(p.v) + ck * p.v_token + tile.head * p.v_head;
  const T* rp = static_cast<const T*>(p.k_rope) + ck * p.kr_token;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);

  for (int t0 = 0; t0 < span; t0 += kTok) {
    __syncthreads();
    for (int i = threadIdx.x; i < kTok * (DK / 8); i += 128) {  // rows past the span become zeros
      const int t = i / (DK / 8), c = i % (DK / 8);
      uint4 v = zero;
      if (t0 + t < span)
        v = c < D / 8 ? *reinterpret_cast<const uint4*>(kp + (t0 + t) * p.k_token + c * 8)
                      : *reinterpret_cast<const uint4*>(rp + (t0 + t) * p.kr_token + c * 8 - D);
      *reinterpret_cast<uint4*>(sm + L::K + t * L::KP + c * 16) = v;
    }
    for (int i = threadIdx.x; i < kTok * (D / 8); i += 128) {
      const int t = i / (D / 8), c = i % (D / 8);
      *reinterpret_cast<uint4*>(sm + L::V + t * L::VP + c * 16) =
          t0 + t < span ? *reinterpret_cast<const uint4*>(vp + (t0 + t) * p.v_token + c * 8) : zero;
    }
    __syncthreads();
    float sc[kTok / 8][4];
#pragma unroll
    for (int n = 0; n < kTok / 8; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c) sc[n][c] = 0.f;
    const int krow = (lane & 7) + ((lane >> 4) & 1) * 8, kch = (lane >> 3) & 1;
#pragma unroll
    for (int ks = 0; ks < DK / 16; ++ks)
#pragma unroll
      for (int n = 0; n < kTok / 16; ++n) {
        uint32_t r0, r1, r2, r3;
        ldsm_x4(sbase + L::K + (n * 16 + krow) * L::KP + (ks * 2 + kch) * 16, r0, r1, r2, r3);
        mma_16816<T>(sc[2 * n], qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], r0, r1);
        mma_16816<T>(sc[2 * n + 1], qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], r2, r3);
      }
    uint32_t ph[kTok / 16][4], pl[kTok / 16][4];
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      float mx = -INFINITY;
#pragma unroll
      for (int n = 0; n < kTok / 8; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float& x = sc[n][2 * hh + c];
          x = t0 + n * 8 + 2 * t4 + c <= lim[hh] ? x * p.qscale : -INFINITY;
          mx = fmaxf(mx, x);
        }
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
      const float m_new = fmaxf(m_run[hh], mx);
      const float ref = m_new == -INFINITY ? 0.f : m_new;
      const float al = ex2(m_run[hh] - ref);
      float ps = 0.f;
#pragma unroll
      for (int n = 0; n < kTok / 8; ++n) {
        const float2 w = make_float2(ex2(sc[n][2 * hh] - ref), ex2(sc[n][2 * hh + 1] - ref));
        ps += w.x + w.y;
        // the A fragment of 16 tokens: (row, low 8), (row + 8, low 8), (row, high 8), (row + 8, high 8)
        split_hi_lo<T>(w, ph[n / 2][hh + 2 * (n & 1)], pl[n / 2][hh + 2 * (n & 1)]);
      }
      ps += __shfl_xor_sync(kFull, ps, 1);
      ps += __shfl_xor_sync(kFull, ps, 2);
      l_run[hh] = l_run[hh] * al + ps;
      m_run[hh] = m_new;
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        o[n][2 * hh] *= al;
        o[n][2 * hh + 1] *= al;
      }
    }
    const int vrow = (lane & 7) + ((lane >> 3) & 1) * 8, vch = lane >> 4;
#pragma unroll
    for (int u = 0; u < kTok / 16; ++u)
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        uint32_t r0, r1, r2, r3;
        ldsm_x4_t(sbase + L::V + (u * 16 + vrow) * L::VP + (d * 2 + vch) * 16, r0, r1, r2, r3);
        mma_16816<T>(o[2 * d], ph[u][0], ph[u][1], ph[u][2], ph[u][3], r0, r1);
        mma_16816<T>(o[2 * d + 1], ph[u][0], ph[u][1], ph[u][2], ph[u][3], r2, r3);
        mma_16816<T>(o[2 * d], pl[u][0], pl[u][1], pl[u][2], pl[u][3], r0, r1);
        mma_16816<T>(o[2 * d + 1], pl[u][0], pl[u][1], pl[u][2], pl[u][3], r2, r3);
      }
  }
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    const int row = row0 + 8 * hh;
    if (row >= tile.ntok) continue;
    const float inv = 1.f / l_run[hh];  // every row sees its own token
    T* out = static_cast<T*>(p.out) + ((int64_t)(cq + tile.tok0 + row) * p.heads + tile.head) * D + 2 * t4;
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
      *reinterpret_cast<uint32_t*>(out + 8 * n) = Elem<T>::from_f2(o[n][2 * hh] * inv, o[n][2 * hh + 1] * inv);
  }
}

template <typename T, int D>
cudaError_t launch_t(const LatentPrefillParams& p, cudaStream_t stream) {
  static std::atomic<unsigned long long> configured{0};
  return launch_pdl(latent_prefill_kernel<T, D>, PrefillLayout1<D>::BYTES, configured, p, p.num_tiles, 128,
                    stream);
}

}  // namespace

cudaError_t launch_latent_prefill(const LatentPrefillParams& p, int head_dim, int dtype,
                                  cudaStream_t stream) {
  const bool bf = dtype == PA_DTYPE_BF16;
  if (head_dim == 64) return bf ? launch_t<__nv_bfloat16, 64>(p, stream) : launch_t<__half, 64>(p, stream);
  return bf ? launch_t<__nv_bfloat16, 128>(p, stream) : launch_t<__half, 128>(p, stream);
}

}  // namespace pa
