// Absorbed latent attention for tiles of 17 to 64 query rows (tcgen05, one
// SM per tile).
//
//   s[i][t] = q_i . [c_t ; r_t],  o_i = sum_t 2^(s qscale - m_i) c_t / sum_t 2^(s qscale - m_i)
//
// With at most 64 rows a cached byte feeds 121 operations or less where the
// card does 280, so HBM bounds the work with room to spare and a pair of SMs
// per tile would only halve what each keeps in flight.  The
// weight-stationary MMA (tcgen05.mma.ws) with M = 64 spreads 64 rows over all
// 128 lanes, the second half of the columns in lanes 64-127: O takes 256
// columns and S 32, as on a pair of SMs.  (Measured: 33 clocks for 64 x 64 x
// 16, 81 for 64 x 256 x 16, so a stage of 64 tokens takes 1.0 us of the 1.65
// us that its bytes take at the copy bandwidth.)
// One CTA holds all 576 dims of a stage's 64 tokens once: keys of the scores
// (K-major) and values of the product (MN-major) are the same bytes.
// Shared memory (128-byte swizzle): q [9 boxes][64 rows][128 B], two stages
// [9 boxes of 64 dims][64 tokens][128 B], P [64 rows][128 B].
//   warps 0-3: softmax and output.  Thread (warp, lane) owns row
//              32 (warp % 2) + lane: tokens 0-31 of the stage in warps 0-1,
//              32-63 in warps 2-3; the two threads of a row exchange maxima
//   warp 4:    one thread issues the MMAs
//   warp 5:    copies, clears rows
// Per stage j: S(j+1) = q K^T into one of two TMEM buffers, if its tokens have
// landed; softmax(j); the product over dims 0-255, which frees boxes 0-3 for
// stage j+2, then over 256-511, which frees the rest.  Weights, masks,
// cleared rows, bounded waits: as in latent_pair.cu.
//
// Measured, merge included: 64 sequences of 500 to 8001 tokens, 322 MB, with 32
// heads 66.9 us (71 % of the copy bandwidth; 71.6 on pairs of SMs, 117 with
// 16-row tiles), with 64 heads 72.6 us (77 on pairs).  21 sequences of 200 to 6003
// tokens, three new tokens each, 20 heads: 30.0 us for 11.7 us of bytes: the
// start about 5, eight stages 12, a piece's output (128 KB of fp32 per CTA at
// what one SM writes to L2) 3.5, the merge and its launch the rest.
#include <math.h>

#include "latent_segment.cuh"
#include "latent_tc5.cuh"
#include "latent_launch.cuh"

namespace pa {

namespace {

constexpr int kSoloTokens = 64;        // tokens of a stage
constexpr int kSoloThreads = 6 * 32;
constexpr float kSoloLazyLog2 = 8.f;   // the maximum is raised when it grows by more than 2^8
static_assert(kLatentRowsSolo == 64 && kLatentStage == kSoloTokens, "plan and kernel");

struct SoloLayout {
  static constexpr int BOX = 64 * 128;                    // 8 KB: 64 dims of 64 rows or tokens
  static constexpr int STAGE = 9 * BOX;
  static constexpr int Q = 0;
  static constexpr int K = Q + 9 * BOX;                   // two stages
  static constexpr int P = K + 2 * STAGE;
  static constexpr int BARS = P + BOX;
  // mbarriers; [buffer] where there are two
  static constexpr int Q_FULL = BARS;
  static constexpr int Q_FREE = Q_FULL + 8;
  static constexpr int K_FULL = Q_FREE + 8;               // [buffer][group]: boxes 0-3, 4-8
  static constexpr int K_FREE = K_FULL + 32;              // [buffer]: boxes 0-3 read by the product
  static constexpr int S_DONE = K_FREE + 16;              // [buffer]
  static constexpr int PV_DONE = S_DONE + 16;             // [buffer]
  static constexpr int CLEARED = PV_DONE + 16;            // [buffer]: a stage's rows are cleared
  static constexpr int DRAIN = CLEARED + 16;
  static constexpr int P_READY = DRAIN + 8;
  static constexpr int CLEAR = P_READY + 8;               // [buffer] flags: the stage has rows to clear
  static constexpr int TMEM_SLOT = CLEAR + 8;
  static constexpr int XMAX = align_up(TMEM_SLOT + 8, 16);  // [2][128] floats: row maxima, sums
  static constexpr int BYTES = XMAX + 2 * 128 * 4 + 1024;
};
static_assert(SoloLayout::BYTES <= kMaxCtaSmem, "stages do not fit in shared memory");

// D (+)= A B, weight-stationary.
__device__ __forceinline__ void mma_ws(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.ws.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tma_load_box(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2,
                                             uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void tma_load_rows(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                              uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar), "l"(policy)
      : "memory");
}

template <typename T>
__global__ void __launch_bounds__(kSoloThreads, 1)
    latent_solo_kernel(const __grid_constant__ LatentParams p, const __grid_constant__ CUtensorMap q_map) {
  using L = SoloLayout;
  extern __shared__ unsigned char smem_dyn[];
  unsigned char* base = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(base);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int first, last;
  const bool planned = latent_range(p, kLatentRowsSolo, (int)blockIdx.x, first, last);

  if (threadIdx.x == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.pages_map)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&q_map)) : "memory");
    for (int b = L::Q_FULL; b < L::P_READY; b += 8) mbar_init(sb + b, 1);
    mbar_init(sb + L::P_READY, 4);
    fence_barrier_init();
  }
  if (warp == 4) {
    __syncwarp();
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     sb + L::TMEM_SLOT)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  LatentSegment s{};
  if (first < last) s = p.segments[first];
  tc5::fence_before();
  __syncthreads();
  tc5::fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(base + L::TMEM_SLOT);
  const uint32_t t_o = tmem, t_s = tmem + 256;  // O 256 columns, S two buffers of 32
  pdl_launch_dependents();
  pdl_wait_primary();
  if (!planned && threadIdx.x == 0) set_status(p.status, PA_DEV_PLAN_MISMATCH);

  auto usable = [&](const LatentSegment& s) {  // the same answer in every warp
    return latent_segment_ok(p, s, kLatentRowsSolo);
  };
  auto stages_of = [](const LatentSegment& s) {
    return (s.tok1 - s.tok0 + kSoloTokens - 1) / kSoloTokens;
  };

  if (warp == 5) {
    // ================= copies =================
    // Stages are counted over all segments: stage c uses buffer c & 1 for the
    // (c >> 1)-th time.
    int c = 0, qc = 0;
    int issued = 0;  // after giving up: groups of stage c whose copies are under way
    bool good = true;
    const uint64_t once = l2_evict_first_policy();
    const int box = p.page_size < 64 ? p.page_size : 64;  // tokens of one copy
    const int copies = kSoloTokens / box;                 // of a stage
    for (int i = first; i < last && good; ++i) {
      if (i > first) s = p.segments[i];
      if (!usable(s)) continue;
      const int32_t* table = p.block_table + (int64_t)s.b * p.max_pages;
      const int n = stages_of(s);
      // lane u: the page of tokens u * box .. of a stage, a stage ahead of its use
      const int lane_end = lane < copies ? s.tok1 : 0;
      int next = table_entry(table, p.page_size, s.tok0 + lane * box, lane_end);
      good = qc == 0 || tc5::warp_wait(sb + L::Q_FREE, (uint32_t)((qc - 1) & 1), p.wait_ns);
      if (!good) break;
      if (lane == 0) mbar_arrive_expect_tx(sb + L::Q_FULL, 9 * L::BOX);
      __syncwarp();
      if (lane < 9)
        tma_load_rows(sb + L::Q + lane * L::BOX, &q_map, lane * 64, s.packed0, sb + L::Q_FULL, once);
      ++qc;
      for (int j = 0; j < n && good; ++j, ++c) {
        const int buf = c & 1, tok = s.tok0 + j * kSoloTokens + lane * box;
        int page = next;
        next = table_entry(table, p.page_size, tok + kSoloTokens, lane_end);
        if (page >= p.num_pages) page = -1;
        if (tok < lane_end && page < 0) set_status(p.status, PA_DEV_BAD_PAGE);
        const unsigned have = __ballot_sync(kFull, page >= 0);
        const unsigned missing = __ballot_sync(kFull, tok < lane_end && page < 0);
        const int row = tok % p.page_size;
        const int valid = min(kSoloTokens, s.tok1 - s.tok0 - j * kSoloTokens);
        const bool clear = missing != 0 || valid % kLatentBlock != 0;
        const uint32_t kb = sb + L::K + buf * L::STAGE;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          good = c < 2 || tc5::warp_wait(sb + (g ? L::PV_DONE : L::K_FREE) + 8 * buf,
                                         (uint32_t)(((c >> 1) - 1) & 1), p.wait_ns);
          if (!good) {
            issued = g;
            break;
          }
          const uint32_t full = sb + L::K_FULL + 16 * buf + 8 * g;
          if (lane == 0) {
            const uint32_t bytes = (uint32_t)(__popc(have) * box * 128 * (g ? 5 : 4));
            if (g == 0) *reinterpret_cast<volatile int*>(base + L::CLEAR + 4 * buf) = clear;
            if (bytes) mbar_arrive_expect_tx(full, bytes);
            else mbar_arrive(full);
          }
          __syncwarp();
          if (page >= 0)
#pragma unroll
            for (int b = 4 * g; b < (g ? 9 : 4); ++b)
              tma_load_box(kb + b * L::BOX + lane * box * 128, &p.pages_map, b * 64, row, page, full, once);
          __syncwarp();
        }
        if (!good) break;
        if (clear) {  // the rest of the last 16 tokens, and the tokens of bad pages
          for (int g = 0; g < 2 && good; ++g)
            good = tc5::warp_wait(sb + L::K_FULL + 16 * buf + 8 * g, (uint32_t)((c >> 1) & 1), p.wait_ns);
          if (!good) {
            issued = 2;
            break;
          }
          __syncwarp();
          for (int at = 0; at < valid; at += kLatentBlock) {
            const int from = missing >> (at / box) & 1 ? 0 : valid - at, rows = kLatentBlock - from;
            for (int x = lane; x < rows * 8 * 8; x += 32) {  // the eight boxes of values
              const int b = x / (rows * 8), k = x % (rows * 8);
              *reinterpret_cast<uint4*>(base + L::K + buf * L::STAGE + b * L::BOX + (at + from) * 128 +
                                        k * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          fence_proxy_async_smem();  // the tensor core reads them (async proxy)
          __syncwarp();
          if (lane == 0) mbar_arrive(sb + L::CLEARED + 8 * buf);
        }
      }
    }
    if (!good && lane == 0) set_status(p.status, PA_DEV_TIMEOUT);
    // copies in flight land before the CTA ends: each group's last use of stage c's
    // buffer, where stage c itself was begun if the warp gave up, and stage c - 1
    for (int g = 0; g < 2; ++g) {
      const int u = c - (g < issued ? 0 : 2);
      if (u >= 0)
        tc5::warp_wait(sb + L::K_FULL + 16 * (u & 1) + 8 * g, (uint32_t)((u >> 1) & 1), kDrainWaitNs);
      if (c > 0)
        tc5::warp_wait(sb + L::K_FULL + 16 * ((c - 1) & 1) + 8 * g, (uint32_t)(((c - 1) >> 1) & 1), kDrainWaitNs);
    }
    if (qc > 0) tc5::warp_wait(sb + L::Q_FULL, (uint32_t)((qc - 1) & 1), kDrainWaitNs);
  } else if (warp == 4) {
    // ================= MMAs (one thread) =================
    if (tc5::elect_one()) {
      const uint32_t idesc_s = tc5::instr_desc<T>(64, kSoloTokens, false);
      const uint32_t idesc_o = tc5::instr_desc<T>(64, 256, true);
      const uint64_t q_desc = tc5::smem_desc(sb + L::Q, 16, 1024), k_desc = tc5::smem_desc(sb + L::K, 16, 1024);
      const uint64_t p_desc = tc5::smem_desc(sb + L::P, 16, 1024);
      const uint64_t v_desc = tc5::smem_desc(sb + L::K, L::BOX, 1024);
      bool good = true;
      int c = 0, qc = 0;           // stages, segments
      int cleared[2] = {0, 0};     // stages with rows to clear, by buffer
      auto wait = [&](int bar, int count) {
        return mbar_wait_bounded(sb + bar, (uint32_t)(count & 1), p.wait_ns);
      };
      auto landed = [&](int cs) {
        const uint32_t bar = sb + L::K_FULL + 16 * (cs & 1);
        return mbar_test_wait(bar, (uint32_t)((cs >> 1) & 1)) && mbar_test_wait(bar + 8, (uint32_t)((cs >> 1) & 1));
      };
      auto scores = [&](int cs, bool last_of_segment) {  // S of stage number cs
        const int buf = cs & 1;
        const uint64_t kd = tc5::desc_at(k_desc, buf * L::STAGE);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          if (!wait(L::K_FULL + 16 * buf + 8 * g, cs >> 1)) return false;
          tc5::fence_after();
#pragma unroll
          for (int k = 16 * g; k < (g ? 36 : 16); ++k)
            mma_ws(t_s + (uint32_t)(32 * buf), tc5::desc_at(q_desc, (k >> 2) * L::BOX + (k & 3) * 32),
                   tc5::desc_at(kd, (k >> 2) * L::BOX + (k & 3) * 32), idesc_s, k > 0 ? 1u : 0u);
        }
        tc5::commit(sb + L::S_DONE + 8 * buf);
        if (last_of_segment) tc5::commit(sb + L::Q_FREE);
        return true;
      };
      for (int i = first; i < last && good; ++i) {
        if (i > first) s = p.segments[i];
        if (!usable(s)) continue;
        const int n = stages_of(s);
        good = wait(L::Q_FULL, qc) && scores(c, n == 1);
        for (int j = 0; j < n && good; ++j) {
          const int cs = c + j, buf = cs & 1;
          const int valid = min(kSoloTokens, s.tok1 - s.tok0 - j * kSoloTokens);
          // S(j+1) goes ahead of the product of stage j if its tokens land before the
          // weights are ready; else the product goes first, which frees its buffer
          bool ahead = j + 1 == n;
          const uint64_t t0 = global_timer_ns();
          while (!mbar_test_wait(sb + L::P_READY, (uint32_t)(cs & 1))) {
            if (!ahead && landed(cs + 1)) {
              good = scores(cs + 1, j + 2 == n);
              ahead = true;
              if (!good) break;
            }
            if (global_timer_ns() - t0 > p.wait_ns) {
              good = false;
              break;
            }
          }
          if (good && *reinterpret_cast<volatile int*>(base + L::CLEAR + 4 * buf))
            good = wait(L::CLEARED + 8 * buf, buf ? cleared[1]++ : cleared[0]++);
          if (!good) break;
          tc5::fence_after();
          const uint64_t vd = tc5::desc_at(v_desc, buf * L::STAGE);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k * 16 < valid)
                mma_ws(t_o + (uint32_t)(128 * h), tc5::desc_at(p_desc, k * 32),
                       tc5::desc_at(vd, 4 * h * L::BOX + k * 2048), idesc_o, j > 0 || k > 0 ? 1u : 0u);
            tc5::commit(sb + (h ? L::PV_DONE : L::K_FREE) + 8 * buf);
          }
          if (!ahead) good = scores(cs + 1, j + 2 == n);
        }
        c += n;
        ++qc;
      }
      if (!good) set_status(p.status, PA_DEV_TIMEOUT);
      // every MMA issued finishes before TMEM is freed
      tc5::commit(sb + L::DRAIN);
      mbar_wait_bounded_sleep(sb + L::DRAIN, 0u, kDrainWaitNs);
    }
    __syncwarp();
  } else {
    // ================= softmax and output =================
    const int row = (warp & 1) * 32 + lane;        // of the tile
    const int half = warp >> 1;                    // tokens 32 half .. of a stage; the same part of O
    const uint32_t lane_off = (uint32_t)(32 * warp) << 16;
    volatile float* xmax = reinterpret_cast<float*>(base + L::XMAX);  // [2 uses][2 halves][64 rows]
    constexpr float kBias = std::is_same<T, __half>::value ? 7.f : 0.f;
    bool good = true;  // after a wait that gave up, a warp only keeps its place in the pair barriers
    int c = 0;
    auto wait = [&](int bar, uint32_t parity) {
      if (good) good = tc5::warp_wait(sb + bar, parity, p.wait_ns);
    };
    for (int i = first; i < last; ++i) {
      if (i > first) s = p.segments[i];
      if (!usable(s)) {
        if (threadIdx.x == 0) set_status(p.status, PA_DEV_PLAN_MISMATCH);
        continue;
      }
      const int32_t* table = p.block_table + (int64_t)s.b * p.max_pages;
      const int n = stages_of(s);
      const int lim0 = row < s.nrows ? s.pos0 + (s.row0 + row) / p.heads : -1;  // last visible token
      const bool idle = (warp & 1) * 32 >= s.nrows;  // no row of the warp's is real
      float m_run = -INFINITY, l_run = 0.f;
      int nph[2];  // pages of the thread's 32 tokens, a stage ahead
      auto load_pages = [&](int j) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int tok = s.tok0 + j * kSoloTokens + half * 32 + u * 16;
          nph[u] = table_entry(table, p.page_size, tok, idle ? 0 : s.tok1);
        }
      };
      load_pages(0);
      for (int j = 0; j < n; ++j) {
        const int cs = c + j;
        if (!idle) {
          bool ok_page[2];
          bool all_ok = true;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            ok_page[u] = nph[u] >= 0 && nph[u] < p.num_pages;
            all_ok = all_ok && ok_page[u];
          }
          if (j + 1 < n) load_pages(j + 1);
          wait(L::S_DONE + 8 * (cs & 1), (uint32_t)((cs >> 1) & 1));
          tc5::fence_after();
          float sv[32];
          __syncwarp();  // the wait's lanes meet: tensor memory is for a whole warp
          tc5::ld32(t_s + (uint32_t)(32 * (cs & 1)) + lane_off, sv);
          tc5::wait_ld();
          const int tok = s.tok0 + j * kSoloTokens + half * 32;
          const int lim = min(lim0, s.tok1 - 1) - tok;  // last visible column
          if (!__all_sync(kFull, all_ok && lim >= 31)) {
#pragma unroll
            for (int x = 0; x < 32; ++x) sv[x] = ok_page[x / 16] && x <= lim ? sv[x] : -INFINITY;
          }
          float mx4[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
          for (int x = 4; x < 32; ++x) mx4[x & 3] = fmaxf(mx4[x & 3], sv[x]);
          float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * p.qscale;
          // the maximum over both halves; two uses in turn, so one barrier a stage
          volatile float* xm = xmax + (cs & 1) * 128;
          xm[half * 64 + row] = mx;
          row_pair_barrier(warp);
          mx = fmaxf(mx, xm[(half ^ 1) * 64 + row]);
          float al = 1.f;
          bool resc = false;
          if (mx > m_run + kSoloLazyLog2) {
            al = ex2(m_run - mx);  // 0 when the row had no weight yet
            resc = m_run != -INFINITY;
            m_run = mx;
          }
          float nm = m_run == -INFINITY ? -INFINITY : kBias - m_run;  // no token yet: weights 0
          float qs = p.qscale;
          if (beyond_fused(m_run)) {
            rounded_differences(sv, qs, m_run);
            qs = 1.f;
            if (m_run != -INFINITY) nm = kBias;
          }
          const float2 qs2 = make_float2(qs, qs), nm2 = make_float2(nm, nm);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          uint32_t pk[16];
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            const float2 e = ffma2(make_float2(sv[x], sv[x + 1]), qs2, nm2);
            const float2 w = make_float2(ex2(e.x), ex2(e.y));
            sum[(x >> 1) & 1] = fadd2(sum[(x >> 1) & 1], w);
            pk[x >> 1] = Elem<T>::from_f2(w.x, w.y);
          }
          const float2 s2 = fadd2(sum[0], sum[1]);
          l_run = l_run * al + (s2.x + s2.y);
          // P and O are free once the product before is done
          if (cs > 0) wait(L::PV_DONE + 8 * ((cs - 1) & 1), (uint32_t)(((cs - 1) >> 1) & 1));
          tc5::fence_after();
          unsigned char* pr = base + L::P + row * 128;
#pragma unroll
          for (int x = 0; x < 4; ++x)
            *reinterpret_cast<uint4*>(pr + (((4 * half + x) ^ (row & 7)) << 4)) =
                make_uint4(pk[4 * x], pk[4 * x + 1], pk[4 * x + 2], pk[4 * x + 3]);
          if (j > 0 && __any_sync(kFull, resc)) {
            const float f = resc ? al : 1.f;
            __syncwarp();  // rows whose maximum rose have branched
#pragma unroll 4
            for (int x = 0; x < 256; x += 16) {
              float ov[16];
              tc5::ld16(t_o + (uint32_t)x + lane_off, ov);
              tc5::wait_ld();
#pragma unroll
              for (int y = 0; y < 16; ++y) ov[y] *= f;
              tc5::st16(t_o + (uint32_t)x + lane_off, ov);
            }
            tc5::wait_st();
          }
          fence_proxy_async_smem();  // the tensor core reads P (async proxy)
          tc5::fence_before();
        } else if (cs > 0) {
          wait(L::PV_DONE + 8 * ((cs - 1) & 1), (uint32_t)(((cs - 1) >> 1) & 1));
        }
        __syncwarp();
        if (good && lane == 0) mbar_arrive(sb + L::P_READY);
      }
      c += n;
      wait(L::PV_DONE + 8 * ((c - 1) & 1), (uint32_t)(((c - 1) >> 1) & 1));
      if (!idle) {
        // the row's sum over both halves, and whether both warps got here in order
        volatile float* xs = xmax + (c & 1) * 128;
        xs[half * 64 + row] = good ? l_run : -1.f;
        row_pair_barrier(warp);
        const float other = xs[(half ^ 1) * 64 + row];
        const bool whole = good && !(other < 0.f);
        const float l = l_run + other;
        const float inv = l > 0.f || l != l ? 1.f / l : 0.f;  // a NaN sum stays NaN
        const bool mine = row < s.nrows;
        const int64_t grow = (int64_t)s.packed0 + row;
        const int64_t at = (int64_t)s.slot * p.rows + row;
        const bool whole32 =
            ((reinterpret_cast<uintptr_t>(p.out) | reinterpret_cast<uintptr_t>(p.part_o)) & 31) == 0;
        if (whole) {
          tc5::fence_after();
#pragma unroll 2
          for (int x = 0; x < 256; x += 32) {
            __syncwarp();  // the rows that are written have branched
            float ov[32];
            tc5::ld16(t_o + (uint32_t)x + lane_off, ov);
            tc5::ld16(t_o + (uint32_t)x + 16u + lane_off, ov + 16);
            tc5::wait_ld();
            const int dim = (x >> 7) * 256 + half * 128 + (x & 127);
            // a thread's row is its own: 32 bytes a store, a whole sector each
            if (mine && s.slot < 0) {
              T* out = static_cast<T*>(p.out) + grow * kLatent + dim;
#pragma unroll
              for (int y = 0; y < 32; y += 16) {
                uint32_t w[8];
#pragma unroll
                for (int z = 0; z < 8; ++z)
                  w[z] = Elem<T>::from_f2(ov[y + 2 * z] * inv, ov[y + 2 * z + 1] * inv);
                store32(out + y, w, whole32);
              }
            } else if (mine) {
              float* po = p.part_o + at * kLatent + dim;
#pragma unroll
              for (int y = 0; y < 32; y += 8) {
                uint32_t w[8];
#pragma unroll
                for (int z = 0; z < 8; ++z) w[z] = __float_as_uint(ov[y + z] * inv);
                store32(po + y, w, whole32);
              }
            }
          }
        }
        if (mine && s.slot >= 0 && half == 0)
          // a row that was not written keeps its whole tile's row unwritten
          p.part_lse[at] = !whole ? INFINITY : l > 0.f || l != l ? m_run + lg2(l) - kBias : -INFINITY;
        if (!whole && lane == 0) set_status(p.status, PA_DEV_TIMEOUT);
        tc5::fence_before();  // O is read before the next segment's first product
        row_pair_barrier(warp);
      }
    }
    if (!good && lane == 0) set_status(p.status, PA_DEV_TIMEOUT);
  }

  tc5::fence_before();
  __syncthreads();
  if (warp == 4) {
    tc5::fence_after();
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

template <typename T>
cudaError_t launch_t(const LatentParams& p, const CUtensorMap& q_map, cudaStream_t stream) {
  static std::atomic<unsigned long long> configured{0};
  return launch_latent(latent_solo_kernel<T>, SoloLayout::BYTES, configured, p.num_ranges, kSoloThreads,
                       stream, p, q_map);
}

}  // namespace

cudaError_t launch_latent_solo(const LatentParams& params, const pa_latent_shape_t& shape,
                               const void* pages, cudaStream_t stream) {
  LatentParams p = params;
  CUtensorMap q_map;
  if (!encode_latent_q(&q_map, p, shape.dtype) ||
      !encode_latent_boxes(&p.pages_map, pages, shape, shape.page_size < 64 ? shape.page_size : 64))
    return cudaErrorInvalidValue;
  if (shape.dtype == PA_DTYPE_BF16) return launch_t<__nv_bfloat16>(p, q_map, stream);
  return launch_t<__half>(p, q_map, stream);
}

}  // namespace pa
