// Expanded latent attention of prompts on tcgen05: keys of D + 64 dims whose
// last 64 (the rotary part) are shared by the heads, values of D dims, causal.
//
//   s[i][t] = q_i . [k_th ; r_t],  o_i = sum_t 2^(s qscale - m_i) v_th / sum_t 2^(s qscale - m_i)
//
// The work is 2 (2D + 64) operations per visible pair and head over data that
// the tiles share through L2: it is bound by the tensor cores, then by the
// exponentials.  A CTA (one per SM) owns 256 query tokens of one head as two
// tiles of 128 rows, so that the softmax of one tile runs while the tensor
// cores work on the other.
//   warps 0-3: softmax and output of tile 0 (thread = row = TMEM lane)
//   warps 4-7: the same of tile 1
//   warp 8:    issues the MMAs
//   warp 9:    copies q, then stages of 128 tokens' keys and values
// TMEM (512 columns): S0, S1 (128 each), O0, O1 (128 each).  The weights
// P_t take S_t's place, two 16-bit weights a column: the A operand of P V.
// Shared memory (128-byte swizzle): q 2 x [DK/64][128 rows][128 B], two key
// stages [DK/64][128 tokens][128 B], one value stage [D/64][128 tokens][128 B].
//
// Per stage j and tile t:
//   S_t(j) = q_t K(j)^T             DK/16 MMAs, M = N = 128
//   softmax in registers, P_t(j) over S_t(j)
//   O_t += P_t(j) V(j)              8 MMAs, N = D
//   S_t(j+1) once P V(j) of the tile is done, which reads the same columns
// in the order PV_0, S_0, PV_1, S_1.  The weights are rounded to the element
// type once: the product's time is what a second part of them would cost
// again, and the error stays below that of rounding the result.  For fp16
// they carry a factor 2^7, so that small weights stay normal numbers.  The
// running maximum is raised only when a row's grows by more than 2^8
// (p <= 2^8, 2^15 with the factor), which keeps O's rescaling rare.
//
// Value rows past the tile's last visible token (a neighbour's rows, which
// may hold anything) become zeros before P V reads them.  Every wait is
// bounded; a CTA that gave up writes nothing.
#include <math.h>

#include "latent_params.h"
#include "latent_tc5.cuh"
#include "split_launch.cuh"

namespace pa {

namespace {

constexpr int kRows = 128;                  // query rows of a tile (TMEM lanes)
constexpr int kTokens = 128;                // tokens of a stage
constexpr int kPrefillThreads = 10 * 32;
constexpr float kLazyLog2 = 8.f;            // the maximum is raised when it grows by more than 2^8
static_assert(kLatentRowsExpanded == 2 * kRows, "a CTA has two tiles");

template <int D>
struct XLayout {
  static constexpr int DK = D + kRope;
  static constexpr int BOX = kTokens * 128;             // 16 KB: 64 dims of 128 rows
  static constexpr int QTILE = DK / 64 * BOX;
  static constexpr int KSTAGE = DK / 64 * BOX;
  static constexpr int VSTAGE = D / 64 * BOX;
  static constexpr int NK = 2;
  static constexpr int Q = 0;
  static constexpr int K = Q + 2 * QTILE;
  static constexpr int V = K + NK * KSTAGE;
  static constexpr int BARS = V + VSTAGE;
  // mbarriers
  static constexpr int Q_FULL = BARS;
  static constexpr int K_FULL = Q_FULL + 8;             // NK
  static constexpr int K_FREE = K_FULL + 8 * NK;        // NK
  static constexpr int V_FULL = K_FREE + 8 * NK;
  static constexpr int V_FREE = V_FULL + 8;
  static constexpr int S_DONE = V_FREE + 8;             // one per tile, as the next two
  static constexpr int P_READY = S_DONE + 16;
  static constexpr int PV_DONE = P_READY + 16;
  static constexpr int DRAIN = PV_DONE + 16;
  static constexpr int TMEM_SLOT = DRAIN + 8;
  static constexpr int FLAG = TMEM_SLOT + 8;
  static constexpr int BYTES = FLAG + 8 + 1024;
};
static_assert(XLayout<128>::BYTES <= kMaxCtaSmem, "stages do not fit in shared memory");

struct XMaps {
  CUtensorMap q, k, kr, v;
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                            int c2, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy)
      : "memory");
}

template <typename T, int D>
__global__ void __launch_bounds__(kPrefillThreads, 1)
    latent_prefill_kernel(const __grid_constant__ LatentPrefillParams p,
                          const __grid_constant__ XMaps maps) {
  using L = XLayout<D>;
  constexpr int DK = L::DK;
  extern __shared__ unsigned char smem_dyn[];
  unsigned char* base = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(base);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* flag = reinterpret_cast<int*>(base + L::FLAG);

  if (threadIdx.x == 0) {
    *flag = 0;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.q)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.kr)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.v)) : "memory");
    mbar_init(sb + L::Q_FULL, 1);
    for (int s = 0; s < L::NK; ++s) {
      mbar_init(sb + L::K_FULL + 8 * s, 1);
      mbar_init(sb + L::K_FREE + 8 * s, 1);
    }
    mbar_init(sb + L::V_FULL, 1);
    mbar_init(sb + L::V_FREE, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(sb + L::S_DONE + 8 * t, 1);
      mbar_init(sb + L::P_READY + 8 * t, 4);
      mbar_init(sb + L::PV_DONE + 8 * t, 1);
    }
    mbar_init(sb + L::DRAIN, 1);
    fence_barrier_init();
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     sb + L::TMEM_SLOT)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc5::fence_before();
  __syncthreads();
  tc5::fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(base + L::TMEM_SLOT);
  pdl_launch_dependents();
  pdl_wait_primary();

  const int4 h0 = reinterpret_cast<const int4*>(p.ws)[0];
  bool bad = h0.x != (int)kLatentMagic || h0.y != p.batch || h0.z != p.total_q || h0.w != p.total_k ||
             p.ws[6] != PA_LATENT_EXPANDED || p.ws[7] != kLatentRowsExpanded || p.ws[8] != p.num_tiles;
  LatentTile tile{};
  int cq = 0, qn = 0, ck = 0, len = 0;
  if (!bad) {
    tile = p.tiles[blockIdx.x];
    bad = tile.b < 0 || tile.b >= p.batch || tile.head < 0 || tile.head >= p.heads || tile.tok0 < 0 ||
          tile.ntok < 1 || tile.ntok > kLatentRowsExpanded;
  }
  if (!bad) {
    cq = p.cu_q[tile.b];
    qn = p.cu_q[tile.b + 1] - cq;
    ck = p.cu_k[tile.b];
    len = p.cu_k[tile.b + 1] - ck;
    bad = cq < 0 || ck < 0 || qn > len || tile.tok0 + tile.ntok > qn || cq + qn > p.total_q ||
          ck + len > p.total_k;
  }
  if (bad && threadIdx.x == 0) set_status(p.status, PA_DEV_PLAN_MISMATCH);
  const int pos0 = len - qn + tile.tok0;  // position of the first row
  // stages of each tile (0: it has no rows)
  const int n0 = bad ? 0 : (pos0 + min(tile.ntok, kRows) + kTokens - 1) / kTokens;
  const int n1 = bad || tile.ntok <= kRows ? 0 : (pos0 + tile.ntok + kTokens - 1) / kTokens;
  const int n = max(n0, n1);
  const int span = pos0 + tile.ntok;

  if (warp == 9) {
    // ================= copies =================
    if (lane == 0 && n > 0) {
      const uint64_t keep = tc5::l2_evict_normal_policy(), once = l2_evict_first_policy();
      const int tiles = n1 > 0 ? 2 : 1;
      mbar_arrive_expect_tx(sb + L::Q_FULL, (uint32_t)(tiles * L::QTILE));
      for (int t = 0; t < tiles; ++t)
        for (int b = 0; b < DK / 64; ++b)
          tma_load_3d(sb + L::Q + t * L::QTILE + b * L::BOX, &maps.q, b * 64, tile.head,
                      cq + tile.tok0 + t * kRows, sb + L::Q_FULL, once);
      int j = 0, jv = 0;
      bool good = true;
      for (; j < n; ++j) {
        const int s = j % L::NK, tok = ck + j * kTokens;
        good = j < L::NK || mbar_wait_bounded_sleep(sb + L::K_FREE + 8 * s,
                                                    (uint32_t)((j / L::NK - 1) & 1), p.wait_ns);
        if (!good) break;
        const uint32_t kb = sb + L::K + s * L::KSTAGE, kf = sb + L::K_FULL + 8 * s;
        mbar_arrive_expect_tx(kf, L::KSTAGE);
        for (int b = 0; b < D / 64; ++b)
          tma_load_3d(kb + b * L::BOX, &maps.k, b * 64, p.k_token_major ? tile.head : tok,
                      p.k_token_major ? tok : tile.head, kf, keep);
        tma_load_3d(kb + D / 64 * L::BOX, &maps.kr, 0, tok, 0, kf, keep);
        good = j < 1 || mbar_wait_bounded_sleep(sb + L::V_FREE, (uint32_t)((j - 1) & 1), p.wait_ns);
        if (!good) break;
        mbar_arrive_expect_tx(sb + L::V_FULL, L::VSTAGE);
        for (int b = 0; b < D / 64; ++b)
          tma_load_3d(sb + L::V + b * L::BOX, &maps.v, b * 64, p.v_token_major ? tile.head : tok,
                      p.v_token_major ? tok : tile.head, sb + L::V_FULL, keep);
        ++jv;
      }
      if (!good) {
        set_status(p.status, PA_DEV_TIMEOUT);
        *flag = 1;
        ++j;  // the stage whose keys were issued (or an older phase, complete already)
      }
      // copies in flight land before the CTA exits
      mbar_wait_bounded_sleep(sb + L::Q_FULL, 0u, kDrainWaitNs);
      for (int i = j < L::NK ? 0 : j - L::NK; i < j && i < n; ++i)
        if (i < jv || !good)
          mbar_wait_bounded_sleep(sb + L::K_FULL + 8 * (i % L::NK), (uint32_t)((i / L::NK) & 1),
                                  kDrainWaitNs);
      if (jv > 0) mbar_wait_bounded_sleep(sb + L::V_FULL, (uint32_t)((jv - 1) & 1), kDrainWaitNs);
    }
    __syncwarp();
  } else if (warp == 8) {
    // ================= MMAs =================
    if (n > 0) {
      const uint32_t idesc_s = tc5::instr_desc<T>(kRows, kTokens, false);
      const uint32_t idesc_o = tc5::instr_desc<T>(kRows, D, true);
      const uint64_t q_desc = tc5::smem_desc(sb + L::Q, 16, 1024), k_desc = tc5::smem_desc(sb + L::K, 16, 1024);
      const uint64_t v_desc = tc5::smem_desc(sb + L::V, L::BOX, 1024);
      auto issue_s = [&](int t, int j) {
        if (tc5::elect_one()) {
          tc5::fence_after();
          const uint64_t qb = tc5::desc_at(q_desc, t * L::QTILE);
          const uint64_t kb = tc5::desc_at(k_desc, (j % L::NK) * L::KSTAGE);
#pragma unroll
          for (int k = 0; k < DK / 16; ++k)
            tc5::mma1(tmem + t * kTokens, tc5::desc_at(qb, (k >> 2) * L::BOX + (k & 3) * 32),
                      tc5::desc_at(kb, (k >> 2) * L::BOX + (k & 3) * 32), idesc_s, k > 0 ? 1u : 0u);
          tc5::commit(sb + L::S_DONE + 8 * t);
        }
        __syncwarp();
      };
      auto wait = [&](int bar, uint32_t parity) {
        return __all_sync(kFull, mbar_wait_bounded(sb + bar, parity, p.wait_ns)) != 0;
      };
      bool good = wait(L::Q_FULL, 0u) && wait(L::K_FULL, 0u);
      if (good) {
        if (n0 > 0) issue_s(0, 0);
        if (n1 > 0) issue_s(1, 0);
        if (tc5::elect_one()) tc5::commit(sb + L::K_FREE);
      }
      for (int j = 0; j < n && good; ++j) {
        bool have_v = false;
        const bool next = j + 1 < n;
        bool have_k = false;
        for (int t = 0; t < 2 && good; ++t) {
          const int nt = t ? n1 : n0;
          if (j < nt) {
            good = wait(L::P_READY + 8 * t, (uint32_t)(j & 1));
            if (good && !have_v) {
              good = wait(L::V_FULL, (uint32_t)(j & 1));
              have_v = true;
              const int valid = span - j * kTokens;  // rows of the stage that some row sees
              if (good && valid < kTokens) {
                for (int i = lane; i < (kTokens - valid) * 8 * (D / 64); i += 32) {
                  const int b = i / ((kTokens - valid) * 8), c = i % ((kTokens - valid) * 8);
                  *reinterpret_cast<uint4*>(base + L::V + b * L::BOX + valid * 128 + c * 16) =
                      make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();  // the tensor core reads them (async proxy)
                __syncwarp();
              }
            }
            if (!good) break;
            if (tc5::elect_one()) {
              tc5::fence_after();
#pragma unroll
              for (int k = 0; k < kTokens / 16; ++k)
                tc5::mma1_tmem(tmem + 2 * kTokens + t * D, tmem + t * kTokens + 8 * k,
                               tc5::desc_at(v_desc, k * 2048), idesc_o, j > 0 || k > 0 ? 1u : 0u);
              tc5::commit(sb + L::PV_DONE + 8 * t);
              if (t == (n1 > j ? 1 : 0)) tc5::commit(sb + L::V_FREE);
            }
            __syncwarp();
          }
          if (j + 1 < nt) {
            if (!have_k) good = wait(L::K_FULL + 8 * ((j + 1) % L::NK), (uint32_t)(((j + 1) / L::NK) & 1));
            have_k = true;
            // P V(j) reads P_t from the columns that S_t(j + 1) overwrites
            good = good && wait(L::PV_DONE + 8 * t, (uint32_t)(j & 1));
            if (!good) break;
            issue_s(t, j + 1);
          }
        }
        if (good && next && tc5::elect_one()) tc5::commit(sb + L::K_FREE + 8 * ((j + 1) % L::NK));
      }
      if (!good && lane == 0) {
        set_status(p.status, PA_DEV_TIMEOUT);
        *flag = 1;
      }
      // every MMA issued finishes before TMEM is freed
      __syncwarp();
      if (tc5::elect_one()) {
        tc5::commit(sb + L::DRAIN);
        mbar_wait_bounded_sleep(sb + L::DRAIN, 0u, kDrainWaitNs);
      }
      __syncwarp();
    }
  } else {
    // ================= softmax and output =================
    const int t = warp >> 2;
    const int row = threadIdx.x & 127;                 // of the tile
    const int nt = t ? n1 : n0;
    const bool ok = !bad && t * kRows + row < tile.ntok;
    const int qpos = ok ? pos0 + t * kRows + row : -1;  // last visible token
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t t_s = tmem + t * kTokens + lane_off, t_o = tmem + 2 * kTokens + t * D + lane_off;
    constexpr float kBias = std::is_same<T, __half>::value ? 7.f : 0.f;
    float m_run = -INFINITY, l_run = 0.f;
    bool good = true;
    for (int j = 0; j < nt; ++j) {
      good = __all_sync(kFull, mbar_wait_bounded_sleep(sb + L::S_DONE + 8 * t, (uint32_t)(j & 1), p.wait_ns));
      if (!good) break;
      tc5::fence_after();
      float sv[kTokens];
#pragma unroll
      for (int c = 0; c < kTokens; c += 32) tc5::ld32(t_s + (uint32_t)c, sv + c);
      tc5::wait_ld();
      const int lim = qpos - j * kTokens;  // last visible column of the stage
      if (!__all_sync(kFull, lim >= kTokens - 1)) {
#pragma unroll
        for (int c = 0; c < kTokens; ++c) sv[c] = c <= lim ? sv[c] : -INFINITY;
      }
      float mx4[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
      for (int c = 4; c < kTokens; ++c) mx4[c & 3] = fmaxf(mx4[c & 3], sv[c]);
      const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * p.qscale;
      float al = 1.f;
      bool resc = false;
      if (mx > m_run + kLazyLog2) {
        al = ex2(m_run - mx);  // 0 when the row had no weight yet
        resc = m_run != -INFINITY;
        m_run = mx;
      }
      const float nm = m_run == -INFINITY ? -INFINITY : kBias - m_run;  // no token yet: weights 0
      const float2 qs2 = make_float2(p.qscale, p.qscale), nm2 = make_float2(nm, nm);
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int c0 = 0; c0 < kTokens; c0 += 32) {
        uint32_t pk[16];
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          const float2 x = ffma2(make_float2(sv[c0 + c], sv[c0 + c + 1]), qs2, nm2);
          const float2 w = make_float2(ex2(x.x), ex2(x.y));
          sum[(c >> 1) & 1] = fadd2(sum[(c >> 1) & 1], w);
          pk[c >> 1] = Elem<T>::from_f2(w.x, w.y);
        }
        tc5::st16u(t_s + (uint32_t)(c0 / 2), pk);
      }
      const float2 s2 = fadd2(sum[0], sum[1]);
      l_run = l_run * al + (s2.x + s2.y);
      // S(j) was issued after P V(j - 1) was done, so O may be rescaled now
      if (j > 0 && __any_sync(kFull, resc)) {
        const float f = resc ? al : 1.f;
#pragma unroll
        for (int c = 0; c < D; c += 16) {
          float ov[16];
          tc5::ld16(t_o + (uint32_t)c, ov);
          tc5::wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) ov[i] *= f;
          tc5::st16(t_o + (uint32_t)c, ov);
        }
      }
      tc5::wait_st();
      tc5::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(sb + L::P_READY + 8 * t);
    }
    if (nt > 0 && good) {
      good = __all_sync(kFull, mbar_wait_bounded_sleep(sb + L::PV_DONE + 8 * t, (uint32_t)((nt - 1) & 1),
                                                       p.wait_ns));
      if (good) {
        tc5::fence_after();
        const float inv = l_run > 0.f || l_run != l_run ? 1.f / l_run : 0.f;
        T* out = static_cast<T*>(p.out) +
                 ((int64_t)(cq + tile.tok0 + t * kRows + row) * p.heads + tile.head) * D;
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          float ov[32];
          tc5::ld32(t_o + (uint32_t)c, ov);
          tc5::wait_ld();
          if (ok) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              uint4 w;
              w.x = Elem<T>::from_f2(ov[i] * inv, ov[i + 1] * inv);
              w.y = Elem<T>::from_f2(ov[i + 2] * inv, ov[i + 3] * inv);
              w.z = Elem<T>::from_f2(ov[i + 4] * inv, ov[i + 5] * inv);
              w.w = Elem<T>::from_f2(ov[i + 6] * inv, ov[i + 7] * inv);
              *reinterpret_cast<uint4*>(out + c + i) = w;
            }
          }
        }
      }
    }
    if (!good && lane == 0) set_status(p.status, PA_DEV_TIMEOUT);
  }

  tc5::fence_before();
  __syncthreads();
  if (warp == 8) {
    tc5::fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// Rows [outer][inner] of `width` dense elements, as a 3-D map with boxes of
// 64 elements by 128 tokens of one head.  token_major: tokens are the outer
// dimension.
bool encode_rows(CUtensorMap* map, const void* ptr, int dtype, int width, int64_t tokens,
                 int64_t token_stride, int64_t heads, int64_t head_stride, bool token_major) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t nt = (cuuint64_t)tokens, nh = (cuuint64_t)heads;
  cuuint64_t dims[3] = {(cuuint64_t)width, token_major ? nh : nt, token_major ? nt : nh};
  cuuint64_t strides[2] = {(cuuint64_t)(token_major ? head_stride : token_stride) * 2,
                           (cuuint64_t)(token_major ? token_stride : head_stride) * 2};
  cuuint32_t box[3] = {64, token_major ? 1u : (cuuint32_t)kTokens, token_major ? (cuuint32_t)kTokens : 1u};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapDataType ty = dtype == PA_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                       : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return enc(map, ty, 3, const_cast<void*>(ptr), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D>
cudaError_t launch_t(const LatentPrefillParams& p, const XMaps& maps, cudaStream_t stream) {
  static std::atomic<unsigned long long> configured{0};
  return launch_pdl(latent_prefill_kernel<T, D>, XLayout<D>::BYTES, configured, p, p.num_tiles,
                    kPrefillThreads, stream, maps);
}

}  // namespace

cudaError_t launch_latent_prefill(const LatentPrefillParams& params, int head_dim, int dtype,
                                  cudaStream_t stream) {
  LatentPrefillParams p = params;
  const int64_t dk = head_dim + kRope;
  // the outer dimension of a map is the one with the larger stride
  p.k_token_major = p.k_token >= p.k_head;
  p.v_token_major = p.v_token >= p.v_head;
  XMaps maps{};
  if (!encode_rows(&maps.q, p.q, dtype, (int)dk, p.total_q, p.heads * dk, p.heads, dk, true) ||
      !encode_rows(&maps.k, p.k, dtype, head_dim, p.total_k, p.k_token, p.heads, p.k_head,
                   p.k_token_major) ||
      !encode_rows(&maps.kr, p.k_rope, dtype, kRope, p.total_k, p.kr_token, 1,
                   p.kr_token * p.total_k, false) ||
      !encode_rows(&maps.v, p.v, dtype, head_dim, p.total_k, p.v_token, p.heads, p.v_head,
                   p.v_token_major))
    return cudaErrorInvalidValue;
  const bool bf = dtype == PA_DTYPE_BF16;
  if (head_dim == 64)
    return bf ? launch_t<__nv_bfloat16, 64>(p, maps, stream) : launch_t<__half, 64>(p, maps, stream);
  return bf ? launch_t<__nv_bfloat16, 128>(p, maps, stream) : launch_t<__half, 128>(p, maps, stream);
}

}  // namespace pa
