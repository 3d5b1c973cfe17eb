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
//   warp 8:    issues the MMAs;  warp 9: copies q and keys;  warp 10: copies values
// TMEM (512 columns): S0, S1 (128 each), O0, O1 (128 each).  The weights
// P_t take S_t's place, two 16-bit weights a column: the A operand of P V.
// Shared memory (128-byte swizzle): q 2 x [DK/64][128 rows][128 B] takes
// almost half.  The rest is two rings of four 16 KB units each:
// keys [128 tokens][128 B] of 64 dims, DK/64 of them a stage, and values
// [D/64][64 tokens][128 B] of half a stage.  That is two stages of values and
// one and a third of keys at D = 128 (with two of keys and one of values each
// product waited 0.5 us of a stage's 2.1 for the values).
//
// Per stage j of 128 tokens and tile t:
//   S_t(j) = q_t K(j)^T             DK/16 MMAs, M = N = 128
//   softmax in registers, P_t(j) over S_t(j), in two halves of 64 tokens
//   O_t += P_t(j) V(j)              4 MMAs, N = D, as each half is written
//   S_t(j+1) once P V(j) of the tile is done, which reads the same columns
// in the order PV_0, PV_1, S_0, S_1.  The weights are rounded to the element
// type once: the product's time is what a second part of them would cost
// again, and the error stays below that of rounding the result.  For fp16
// they carry a factor 2^7, so that small weights stay normal numbers.  The
// running maximum is raised only when a row's grows by more than 2^8
// (p <= 2^8, 2^15 with the factor), which keeps O's rescaling rare.
//
// Value rows past the tile's last visible token (a neighbour's rows, which
// may hold anything) become zeros before P V reads them.  Every wait is
// bounded; a CTA that gave up writes nothing.
//
// Measured: a prompt of 8192 tokens with 32 heads of 128, 515 to 535 us, 1300 TFLOP/s
// of visible pairs (77 % of what cuBLAS sustains under the power cap); a stage
// takes 2.05 us where few CTAs run, 2.3 on all SMs (clocks under the cap).  A
// tile of 128 tokens or fewer takes 1.6 us a stage: nothing overlaps its
// softmax.  (So whole tiles where there are enough of them, see the planner.)  Six chunks of 513 tokens behind up to 5700 with 16 heads of 128:
// 161 us, a fifth of it the tiles of the 513th tokens, the rest uneven ends.
#include <math.h>

#include "latent_params.h"
#include "latent_tc5.cuh"
#include "latent_launch.cuh"

namespace pa {

namespace {

constexpr int kRows = 128;                  // query rows of a tile (TMEM lanes)
constexpr int kTokens = 128;                // tokens of a stage
constexpr int kPrefillThreads = 11 * 32;
constexpr float kLazyLog2 = 8.f;            // the maximum is raised when it grows by more than 2^8
static_assert(kLatentRowsExpanded == 2 * kRows, "a CTA has two tiles");

template <int D>
struct XLayout {
  static constexpr int DK = D + kRope;
  static constexpr int KB = DK / 64;                    // key units of a stage
  static constexpr int BOX = kTokens * 128;             // 16 KB: 64 dims of 128 rows
  static constexpr int QTILE = KB * BOX;
  static constexpr int VBOX = kTokens / 2 * 128;        // 8 KB: 64 dims of 64 tokens
  static constexpr int VUNIT = D / 64 * VBOX;
  static constexpr int NK = 4;                          // units of the key ring
  static constexpr int NV = 4;                          // units of the value ring
  static constexpr int Q = 0;
  static constexpr int K = Q + 2 * QTILE;
  static constexpr int V = K + NK * BOX;
  static constexpr int BARS = V + NV * VUNIT;
  // mbarriers
  static constexpr int Q_FULL = BARS;
  static constexpr int K_FULL = Q_FULL + 8;             // stages j & 1
  static constexpr int V_FULL = K_FULL + 16;            // stages j & 1
  // [tile][j & 1]: a copy thread that looks at stage j's late may find that of
  // stage j + 1 complete too, but never that of stage j + 2
  static constexpr int S_DONE = V_FULL + 16;
  static constexpr int PV_DONE = S_DONE + 32;
  static constexpr int V_CLEAR = PV_DONE + 32;          // the last stage's rows
  static constexpr int P_READY = V_CLEAR + 8;           // two halves per tile
  static constexpr int DRAIN = P_READY + 32;
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
  extern __shared__ unsigned char smem_dyn[];
  unsigned char* base = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(base);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* flag = reinterpret_cast<int*>(base + L::FLAG);

  // The plan is written by the upload alone, which the programmatic launch
  // does not overlap: it may be read before the wait for the kernel ahead.
  const int4 h0 = reinterpret_cast<const int4*>(p.ws)[0], h1 = reinterpret_cast<const int4*>(p.ws)[1];
  const LatentTile tile = p.tiles[blockIdx.x];
  const int pos0 = tile.pos0;  // position of the first row
  const int span = pos0 + tile.ntok;
  const bool bad = h0.x != (int)kLatentMagic || h0.y != p.batch || h0.z != p.total_q ||
                   h0.w != p.total_k || h1.z != PA_LATENT_EXPANDED || h1.w != kLatentRowsExpanded ||
                   p.ws[8] != p.num_tiles || tile.head < 0 || tile.head >= p.heads || tile.ntok < 1 ||
                   tile.ntok > kLatentRowsExpanded || tile.q0 < 0 || tile.q0 > p.total_q - tile.ntok ||
                   pos0 < 0 || tile.k0 < 0 || (int64_t)tile.k0 + pos0 + tile.ntok > p.total_k;
  // stages of each tile (0: it has no rows)
  const int n0 = bad ? 0 : (pos0 + min(tile.ntok, kRows) + kTokens - 1) / kTokens;
  const int n1 = bad || tile.ntok <= kRows ? 0 : (span + kTokens - 1) / kTokens;
  const int n = max(n0, n1);
  if (threadIdx.x == 0) {
    *flag = 0;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.q)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.kr)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.v)) : "memory");
    for (int b = L::Q_FULL; b < L::P_READY; b += 8) mbar_init(sb + b, 1);
    for (int b = L::P_READY; b < L::DRAIN; b += 8) mbar_init(sb + b, 4);
    mbar_init(sb + L::DRAIN, 1);
    fence_barrier_init();
  }
  if (warp == 8) {
    __syncwarp();
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
  if (bad && threadIdx.x == 0) set_status(p.status, PA_DEV_PLAN_MISMATCH);

  if (warp == 9 || warp == 10) {
    // ================= copies =================
    const int valid = span - (n - 1) * kTokens;  // rows of the last stage that some row sees
    if (lane == 0 && n > 0) {
      const bool keys = warp == 9;
      const uint64_t keep = tc5::l2_evict_normal_policy(), once = l2_evict_first_policy();
      const int per = keys ? L::KB : 2, ring = keys ? L::NK : L::NV;  // units of a stage, of the ring
      // The last tile of a stage has read its keys once its scores are done, and
      // its values once its product is: no barriers of their own for the free units.
      const uint32_t done = sb + (keys ? L::S_DONE : L::PV_DONE);
      const uint32_t full = sb + (keys ? L::K_FULL : L::V_FULL);
      if (keys) {
        const int tiles = n1 > 0 ? 2 : 1;
        mbar_arrive_expect_tx(sb + L::Q_FULL, (uint32_t)(tiles * L::QTILE));
        for (int t = 0; t < tiles; ++t)
          for (int b = 0; b < L::KB; ++b)
            tma_load_3d(sb + L::Q + t * L::QTILE + b * L::BOX, &maps.q, b * 64, tile.head,
                        tile.q0 + t * kRows, sb + L::Q_FULL, once);
      }
      bool good = true;
      int j = 0, freed = 0;  // stages issued, stages known to be free
      for (int u = 0; j < n && good; ++j) {
        const uint32_t bar = full + 8 * (j & 1);
        for (int x = 0; x < per; ++x, ++u) {
          // the unit's slot was last used by unit u - ring, of stage (u - ring) / per
          for (; freed * per < u - ring + 1; ++freed) {
            good = mbar_wait_bounded_sleep(done + (n1 > freed ? 16 : 0) + 8 * (freed & 1),
                                           (uint32_t)((freed >> 1) & 1), p.wait_ns);
            if (!good) break;
          }
          if (!good) break;
          const int slot = u % ring, tok = tile.k0 + j * kTokens + (keys ? 0 : x * (kTokens / 2));
          if (x == 0) mbar_arrive_expect_tx(bar, (uint32_t)(keys ? L::KB * L::BOX : 2 * L::VUNIT));
          if (keys) {
            if (x < D / 64)
              tma_load_3d(sb + L::K + slot * L::BOX, &maps.k, x * 64, p.k_token_major ? tile.head : tok,
                          p.k_token_major ? tok : tile.head, bar, keep);
            else
              tma_load_3d(sb + L::K + slot * L::BOX, &maps.kr, 0, tok, 0, bar, keep);
          } else {
            for (int b = 0; b < D / 64; ++b)
              tma_load_3d(sb + L::V + slot * L::VUNIT + b * L::VBOX, &maps.v, b * 64,
                          p.v_token_major ? tile.head : tok, p.v_token_major ? tok : tile.head, bar, keep);
          }
        }
      }
      // rows to clear: the last stage's copies land before the zeros are written
      if (good && !keys && valid < kTokens)
        good = mbar_wait_bounded_sleep(full + 8 * ((n - 1) & 1), (uint32_t)(((n - 1) >> 1) & 1), p.wait_ns);
      if (!good) {
        set_status(p.status, PA_DEV_TIMEOUT);
        *flag = 1;
      }
      // copies in flight land before the CTA exits: those of every stage that is not
      // known to be free, in order, since a barrier's parity tells a stage only from
      // the next one on the same barrier
      if (keys) mbar_wait_bounded_sleep(sb + L::Q_FULL, 0u, kDrainWaitNs);
      for (int i = freed; i < j; ++i)
        mbar_wait_bounded_sleep(full + 8 * (i & 1), (uint32_t)((i >> 1) & 1), kDrainWaitNs);
    }
    __syncwarp();
    // Rows of the last stage that no row of the tile sees become zeros (the
    // copies have landed, and no product reads them before).  A CTA that gave up
    // leaves them and V_CLEAR alone: the product is not formed.
    // (One vote decides for the warp: another warp may set the flag while it is read.)
    if (warp == 10 && n > 0 && valid < kTokens && __all_sync(kFull, *flag == 0)) {
      for (int h = 0; h < 2; ++h) {
        const int v0 = min(64, max(0, valid - h * 64)), chunks = (64 - v0) * 8;
        unsigned char* unit = base + L::V + (2 * (n - 1) + h) % L::NV * L::VUNIT;
        for (int i = lane; i < chunks * (D / 64); i += 32)
          *reinterpret_cast<uint4*>(unit + (i / chunks) * L::VBOX + v0 * 128 + (i % chunks) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();  // the tensor core reads them (async proxy)
      __syncwarp();
      if (lane == 0) mbar_arrive(sb + L::V_CLEAR);
    }
  } else if (warp == 8) {
    // ================= MMAs (one thread) =================
    if (n > 0 && tc5::elect_one()) {
      const uint32_t idesc_s = tc5::instr_desc<T>(kRows, kTokens, false);
      const uint32_t idesc_o = tc5::instr_desc<T>(kRows, D, true);
      const uint64_t q_desc = tc5::smem_desc(sb + L::Q, 16, 1024), k_desc = tc5::smem_desc(sb + L::K, 16, 1024);
      const uint64_t v_desc = tc5::smem_desc(sb + L::V, L::VBOX, 1024);
      auto wait = [&](int bar, uint32_t parity) { return mbar_wait_bounded(sb + bar, parity, p.wait_ns); };
      auto scores = [&](int t, int j) {  // S_t(j)
        tc5::fence_after();
        const uint64_t qb = tc5::desc_at(q_desc, t * L::QTILE);
#pragma unroll
        for (int b = 0; b < L::KB; ++b) {
          const uint64_t kb = tc5::desc_at(k_desc, (j * L::KB + b) % L::NK * L::BOX);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc5::mma1(tmem + t * kTokens, tc5::desc_at(qb, b * L::BOX + k * 32), tc5::desc_at(kb, k * 32),
                      idesc_s, b > 0 || k > 0 ? 1u : 0u);
        }
        tc5::commit(sb + L::S_DONE + 16 * t + 8 * (j & 1));
      };
      bool good = wait(L::Q_FULL, 0u) && wait(L::K_FULL, 0u);
      if (good && n0 > 0) scores(0, 0);
      if (good && n1 > 0) scores(1, 0);
      for (int j = 0; j < n && good; ++j) {
        const int valid = span - j * kTokens;  // rows of the stage that some row sees
        bool have_v = false, have_k = false;
        // both products first: with S_0(j+1) between them each product waited for
        // the tile's other one (prompt of 8192: 552 against 522 us)
        for (int t = 0; t < 2 && good; ++t) {
          const int nt = t ? n1 : n0;
          if (j < nt) {
            if (!have_v)
              good = wait(L::V_FULL + 8 * (j & 1), (uint32_t)((j >> 1) & 1)) &&
                     (valid >= kTokens || wait(L::V_CLEAR, 0u));  // rows to clear: once they are
            have_v = true;
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // halves of 64 tokens
              good = good && wait(L::P_READY + 16 * t + 8 * h, (uint32_t)(j & 1));
              if (!good) break;
              tc5::fence_after();
              const uint64_t vb = tc5::desc_at(v_desc, (2 * j + h) % L::NV * L::VUNIT);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                tc5::mma1_tmem(tmem + 2 * kTokens + t * D, tmem + t * kTokens + 32 * h + 8 * k,
                               tc5::desc_at(vb, k * 2048), idesc_o, j > 0 || h > 0 || k > 0 ? 1u : 0u);
            }
            if (!good) break;
            tc5::commit(sb + L::PV_DONE + 16 * t + 8 * (j & 1));
          }
        }
        for (int t = 0; t < 2 && good; ++t) {
          const int nt = t ? n1 : n0;
          if (j + 1 < nt) {
            if (!have_k) good = wait(L::K_FULL + 8 * ((j + 1) & 1), (uint32_t)(((j + 1) >> 1) & 1));
            have_k = true;
            // P V(j) reads P_t from the columns that S_t(j + 1) overwrites
            good = good && wait(L::PV_DONE + 16 * t + 8 * (j & 1), (uint32_t)((j >> 1) & 1));
            if (good) scores(t, j + 1);
          }
        }
      }
      if (!good) {
        set_status(p.status, PA_DEV_TIMEOUT);
        *flag = 1;
      }
      // every MMA issued finishes before TMEM is freed
      tc5::commit(sb + L::DRAIN);
      mbar_wait_bounded_sleep(sb + L::DRAIN, 0u, kDrainWaitNs);
    }
    __syncwarp();
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
    bool beyond = false;  // some row of the warp has scores beyond the fused product's range
    for (int j = 0; j < nt; ++j) {
      good = __all_sync(kFull, mbar_wait_bounded_sleep(sb + L::S_DONE + 16 * t + 8 * (j & 1),
                                                       (uint32_t)((j >> 1) & 1), p.wait_ns));
      if (!good) break;
      tc5::fence_after();
      float sv[kTokens];
      __syncwarp();  // the wait's lanes meet: tensor memory is for a whole warp
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
      bool resc = false, raised = false;
      if (mx > m_run + kLazyLog2) {
        raised = true;
        al = ex2(m_run - mx);  // 0 when the row had no weight yet
        resc = m_run != -INFINITY;
        m_run = mx;
      }
      // S(j) was issued after P V(j - 1) was done, so O may be rescaled now
      if (__any_sync(kFull, raised)) {
        beyond = beyond_fused(m_run);
        const float f = resc ? al : 1.f;
        if (j > 0) {
          __syncwarp();  // rows whose maximum rose have branched
#pragma unroll 2
          for (int c = 0; c < D; c += 16) {
            float ov[16];
            tc5::ld16(t_o + (uint32_t)c, ov);
            tc5::wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) ov[i] *= f;
            tc5::st16(t_o + (uint32_t)c, ov);
          }
        }
      }
      const float nm = m_run == -INFINITY ? -INFINITY : kBias - m_run;  // no token yet: weights 0
      const float2 qs2 = make_float2(p.qscale, p.qscale), nm2 = make_float2(nm, nm);
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      auto hand_over = [&](int h) {  // half h of the weights is written
        tc5::wait_st();
        tc5::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sb + L::P_READY + 16 * t + 8 * h);
      };
      if (!beyond) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          __syncwarp();  // lanes may have branched, and what follows is for a whole warp
#pragma unroll
          for (int c0 = 64 * h; c0 < 64 * h + 64; c0 += 32) {
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
          hand_over(h);
        }
      } else {  // from the scores in tensor memory again, which P has not reached yet
#pragma unroll 1
        for (int c0 = 0; c0 < kTokens; c0 += 32) {
          uint32_t pk[16];
          const int seen = qpos - j * kTokens - c0;
#pragma unroll
          for (int b = 0; b < 32; b += 16) {
            __syncwarp();
            float x[16];
            tc5::ld16(t_s + (uint32_t)(c0 + b), x);
            tc5::wait_ld();
#pragma unroll
            for (int c = 0; c < 16; ++c) x[c] = b + c <= seen ? x[c] : -INFINITY;
            rounded_differences(x, p.qscale, m_run);
#pragma unroll
            for (int c = 0; c < 16; c += 2) {
              const float2 w = make_float2(ex2(x[c] + kBias), ex2(x[c + 1] + kBias));
              sum[0] = fadd2(sum[0], w);
              pk[(b + c) >> 1] = Elem<T>::from_f2(w.x, w.y);
            }
          }
          tc5::st16u(t_s + (uint32_t)(c0 / 2), pk);
          if (c0 % 64 == 32) hand_over(c0 / 64);
        }
      }
      const float2 s2 = fadd2(sum[0], sum[1]);
      l_run = l_run * al + (s2.x + s2.y);
    }
    if (nt > 0 && good) {
      good = __all_sync(kFull, mbar_wait_bounded_sleep(sb + L::PV_DONE + 16 * t + 8 * ((nt - 1) & 1),
                                                       (uint32_t)(((nt - 1) >> 1) & 1),
                                                       p.wait_ns));
      if (good) {
        tc5::fence_after();
        const float inv = l_run > 0.f || l_run != l_run ? 1.f / l_run : 0.f;
        T* out = static_cast<T*>(p.out) +
                 ((int64_t)(tile.q0 + t * kRows + row) * p.heads + tile.head) * D;
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          __syncwarp();  // the rows that are written have branched
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
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// Rows [outer][inner] of `width` dense elements, as a 3-D map with boxes of
// 64 elements by `box_tokens` tokens of one head.  token_major: tokens are
// the outer dimension.
bool encode_rows(CUtensorMap* map, const void* ptr, int dtype, int box_tokens, int width,
                 int64_t tokens, int64_t token_stride, int64_t heads, int64_t head_stride,
                 bool token_major) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = latent_map_encoder();
  if (!enc) return false;
  const cuuint64_t nt = (cuuint64_t)tokens, nh = (cuuint64_t)heads;
  cuuint64_t dims[3] = {(cuuint64_t)width, token_major ? nh : nt, token_major ? nt : nh};
  cuuint64_t strides[2] = {(cuuint64_t)(token_major ? head_stride : token_stride) * 2,
                           (cuuint64_t)(token_major ? token_stride : head_stride) * 2};
  cuuint32_t box[3] = {64, token_major ? 1u : (cuuint32_t)box_tokens,
                       token_major ? (cuuint32_t)box_tokens : 1u};
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
  return launch_latent(latent_prefill_kernel<T, D>, XLayout<D>::BYTES, configured, p.num_tiles,
                       kPrefillThreads, stream, p, maps);
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
  if (!encode_rows(&maps.q, p.q, dtype, kRows, (int)dk, p.total_q, p.heads * dk, p.heads, dk, true) ||
      !encode_rows(&maps.k, p.k, dtype, kTokens, head_dim, p.total_k, p.k_token, p.heads, p.k_head,
                   p.k_token_major) ||
      !encode_rows(&maps.kr, p.k_rope, dtype, kTokens, kRope, p.total_k, p.kr_token, 1,
                   p.kr_token * p.total_k, false) ||
      !encode_rows(&maps.v, p.v, dtype, kTokens / 2, head_dim, p.total_k, p.v_token, p.heads, p.v_head,
                   p.v_token_major))
    return cudaErrorInvalidValue;
  const bool bf = dtype == PA_DTYPE_BF16;
  if (head_dim == 64)
    return bf ? launch_t<__nv_bfloat16, 64>(p, maps, stream) : launch_t<__half, 64>(p, maps, stream);
  return bf ? launch_t<__nv_bfloat16, 128>(p, maps, stream) : launch_t<__half, 128>(p, maps, stream);
}

}  // namespace pa
