// Absorbed latent attention for tiles of 65 to 128 query rows, on pairs of
// SMs (tcgen05 with cta_group::2).
//
//   s[i][t] = q_i . [c_t ; r_t],  o_i = sum_t 2^(s qscale - m_i) c_t / sum_t 2^(s qscale - m_i)
//
// With 128 rows a cached row of 1152 bytes feeds 2 x 128 x 1088 operations,
// 242 a byte: the card does 280 a byte, so HBM bounds the work and the tensor
// cores have to run at more than three quarters of their rate under it.  What
// makes that hard is the output: 128 rows x 512 values of fp32 would fill one
// SM's TMEM.  A pair of SMs shares the tile instead: each CTA keeps 64 rows
// (M = 128 over the pair puts 64 rows in 128 lanes, the second half of the
// columns in lanes 64-127), so O takes 256 columns and S 64, and each MMA
// reads half of its B operand from either SM.  Per stage of 128 tokens a CTA
// holds
//   K [9 boxes of 64 dims][64 tokens][128 B]   its half of the stage's tokens
//   V [2 groups of 64 tokens][4 boxes][64 tokens][128 B]   its half of the 512 values
// of which K is refilled in three groups of boxes and V in two groups of
// tokens, each as soon as the MMAs that read it are done.
//   warps 0-3: softmax and output.  Thread (warp, lane) owns row
//              32 (warp % 2) + lane of the CTA's 64: tokens 0-63 of the stage
//              in warps 0-1, 64-127 in warps 2-3; the two threads of a row
//              exchange their maxima through shared memory.
//   warp 4:    in the pair's first CTA one thread issues the MMAs of both
//   warp 5:    copies K;  warp 6: copies q and V, clears value rows
// Per stage j: S(j+1) = q K^T into one of two TMEM buffers; softmax(j);
// O += P(j) V(j), P from shared memory [2 boxes of 64 tokens][64 rows][128 B].
// The weights are rounded to the element type once (fp16: times 2^7, so that
// small ones stay normal): a second part would cost the product again, and
// the error stays below that of rounding the result.
//
// Value rows of tokens past the piece's end or of a bad page become zeros
// before they are used (their weight is 0, but they may hold anything).
// Every wait is bounded; a CTA that gave up keeps its place in the barriers
// between its own warps, writes nothing, and meets the other CTA at the end.
//
// Measured: a stage of 128 tokens takes 2.05 us on all pairs at once, in which
// each CTA receives 139 KB: 68 KB/us of the 82 that copies alone reach from L2
// on every SM at once.  That, not HBM (1.65 us) or the MMAs (1.15 us), bounds
// the steady state.  32 sequences of 700 to 8191 tokens with 128 heads (176 MB
// in all): 51.8 us, merge included; two of 40001 and 65537 in pages of 16 tokens:
// 43 us; 64 sequences of 500 to 8001 with 80 heads 78 us (64-row tiles 122).
// A piece costs about two stages beside its own: the queries in, and 128 KB of
// fp32 or 64 KB of results out of each CTA.
// Tried and not kept: prefetching the next stages into L2 (0 to 8 % slower),
// one copy group per box (60 against 52 us), 24 KB copies of three boxes
// (53.5), output through shared memory in whole lines (47.1 against 45.4 us of
// kernel).
#include <math.h>

#include "latent_segment.cuh"
#include "latent_tc5.cuh"
#include "latent_launch.cuh"

namespace pa {

namespace {

constexpr int kPairRows = 64;          // rows of one CTA
constexpr int kPairTokens = 128;       // tokens of a stage
constexpr int kPairThreads = 7 * 32;
constexpr float kPairLazyLog2 = 8.f;   // the maximum is raised when it grows by more than 2^8
static_assert(kLatentRowsPair == 2 * kPairRows && kLatentStagePair == kPairTokens, "plan and kernel");

struct PLayout {
  static constexpr int QBOX = kPairRows * 128;            // 8 KB
  static constexpr int KBOX = kPairTokens / 2 * 128;      // 8 KB
  static constexpr int VBOX = 64 * 128;                   // 8 KB
  static constexpr int VGROUP = 4 * VBOX;                 // 64 tokens of the CTA's 256 values
  static constexpr int NG = 3, NV = 2;                    // groups of K boxes, of V tokens
  static constexpr int BPG = 9 / NG;                      // boxes of a K group
  static constexpr int Q = 0;
  static constexpr int K = Q + 9 * QBOX;
  static constexpr int V = K + 9 * KBOX;
  static constexpr int P = V + NV * VGROUP;
  static constexpr int PBOX = kPairRows * 128;
  static constexpr int BARS = P + 2 * PBOX;
  // mbarriers that the MMAs arrive on, in both CTAs
  static constexpr int Q_FREE = BARS;
  static constexpr int K_FREE = Q_FREE + 8;               // NG - 1 (S_DONE frees the last group)
  static constexpr int V_FREE = K_FREE + 8 * (NG - 1);    // NV - 1 (PV_DONE frees the last group)
  static constexpr int S_DONE = V_FREE + 8 * (NV - 1);    // 2
  static constexpr int PV_DONE = S_DONE + 16;
  static constexpr int DRAIN = PV_DONE + 8;
  // in the first CTA: the copies of both have landed
  static constexpr int Q_FULL = DRAIN + 8;
  static constexpr int K_FULL = Q_FULL + 8;               // NG
  static constexpr int V_FULL = K_FULL + 8 * NG;          // NV
  // values with rows to clear: landed in the second CTA (there), cleared in
  // both (in the first CTA)
  static constexpr int V_HERE = V_FULL + 8 * NV;          // NV
  static constexpr int V_CLEAR = V_HERE + 8 * NV;         // NV
  // in the first CTA: the weights of both are written
  static constexpr int P_READY = V_CLEAR + 8 * NV;
  static constexpr int CLEAR = P_READY + 8;               // NV flags: this use has rows to clear
  static constexpr int TMEM_SLOT = CLEAR + 4 * NV;
  static constexpr int XMAX = align_up(TMEM_SLOT + 8, 16);  // [2][128] floats: row maxima, sums
  static constexpr int BYTES = XMAX + 2 * 128 * 4 + 1024;
};
static_assert(PLayout::BYTES <= kMaxCtaSmem, "stages do not fit in shared memory");

__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();  // the barrier is for converged warps
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

// Arrive on the first CTA's barrier at this offset of its shared memory.
// What the arrival announces (weights, cleared values) lies in the arriving
// CTA's shared memory and is read there by its own tensor core, so it is
// fence.proxy.async before the arrival that makes it visible, and neither side
// needs a cluster-wide fence (measured at 0.7 us each, on the path of every
// stage).
__device__ __forceinline__ void arrive_first_cta(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .b32 ra;\n\t"
      "mapa.shared::cluster.u32 ra, %0, 0;\n\t"
      "mbarrier.arrive.shared::cluster.b64 _, [ra];\n\t}" ::"r"(bar)
      : "memory");
}

// The address of this offset of the first CTA's shared memory.
__device__ __forceinline__ uint32_t in_first_cta(uint32_t addr) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}

// TMA copies into this CTA whose barrier may be the other CTA's.
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                                 int c2, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2.L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                                 uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2.L2::cache_hint [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar), "l"(policy)
      : "memory");
}

template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    latent_pair_kernel(const __grid_constant__ LatentParams p,
                       const __grid_constant__ CUtensorMap q_map) {
  using L = PLayout;
  extern __shared__ unsigned char smem_dyn[];
  unsigned char* base = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(base);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cta_rank();
  int first, last;
  const bool planned = latent_range(p, kLatentRowsPair, (int)(blockIdx.x >> 1), first, last);

  if (threadIdx.x == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.pages_map)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&q_map)) : "memory");
    for (int b = L::Q_FREE; b < L::V_CLEAR; b += 8) mbar_init(sb + b, 1);
    for (int b = L::V_CLEAR; b < L::P_READY; b += 8) mbar_init(sb + b, 2);
    mbar_init(sb + L::P_READY, 8);
    fence_barrier_init();
  }
  if (warp == 4) {
    __syncwarp();
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     sb + L::TMEM_SLOT)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  LatentSegment s{};
  if (first < last) s = p.segments[first];
  tc5::fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before either is arrived on
  tc5::fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(base + L::TMEM_SLOT);
  const uint32_t t_o = tmem, t_s = tmem + 256;  // O 256 columns, S two buffers of 64
  pdl_launch_dependents();
  pdl_wait_primary();
  if (!planned && threadIdx.x == 0) set_status(p.status, PA_DEV_PLAN_MISMATCH);

  auto usable = [&](const LatentSegment& s) {  // the same answer in every warp of both CTAs
    return latent_segment_ok(p, s, kLatentRowsPair);
  };
  auto stages_of = [](const LatentSegment& s) {
    return (s.tok1 - s.tok0 + kPairTokens - 1) / kPairTokens;
  };

  if (warp == 5 || warp == 6) {
    // ================= copies =================
    // Stages are counted over all segments: use c of a buffer has parity
    // c & 1.  The copies of both CTAs complete on the first CTA's barriers,
    // whose own copy warps announce the bytes of both.
    const bool keys = warp == 5;
    int c = 0, qc = 0;
    int g = 0;           // after giving up: the group it happened at,
    bool begun = false;  // and whether that one's copies are under way
    bool good = true;
    const uint64_t once = l2_evict_first_policy(), keep = tc5::l2_evict_normal_policy();
    const int box = p.page_size < 64 ? p.page_size : 64;  // tokens of one copy
    const int copies = kPairTokens / box;                 // of a stage
    const int per = 64 / box;                             // of a group
    const int groups = keys ? L::NG : L::NV;
    int clears = 0;                                       // uses of V_HERE, a bit a group: parities
    // use c of group g has been read
    auto wait_free = [&](int g, int c, uint64_t limit) {
      if (g < groups - 1)
        return tc5::warp_wait(sb + (keys ? L::K_FREE : L::V_FREE) + 8 * g, (uint32_t)(c & 1), limit);
      return keys ? tc5::warp_wait(sb + L::S_DONE + 8 * (c & 1), (uint32_t)((c >> 1) & 1), limit)
                  : tc5::warp_wait(sb + L::PV_DONE, (uint32_t)(c & 1), limit);
    };
    const uint32_t full0 = in_first_cta(sb + (keys ? L::K_FULL : L::V_FULL));
    for (int i = first; i < last && good; ++i) {
      if (i > first) s = p.segments[i];
      if (!usable(s)) continue;
      const int32_t* table = p.block_table + (int64_t)s.b * p.max_pages;
      if (!keys) {  // q: the CTA's 64 rows, by the warp whose own copies are needed later
        good = qc == 0 || tc5::warp_wait(sb + L::Q_FREE, (uint32_t)((qc - 1) & 1), p.wait_ns);
        if (!good) break;
        if (rank == 0 && lane == 0) mbar_arrive_expect_tx(sb + L::Q_FULL, 2 * 9 * L::QBOX);
        if (lane < 9)
          tma_load_2d_pair(sb + L::Q + lane * L::QBOX, &q_map, lane * 64, s.packed0 + rank * kPairRows,
                           in_first_cta(sb + L::Q_FULL), once);
        ++qc;
      }
      const int n = stages_of(s);
      // lane u: the page of tokens u * box .. of a stage, a stage ahead of its use
      int next = table_entry(table, p.page_size, s.tok0 + lane * box, lane < copies ? s.tok1 : 0);
      for (int j = 0; j < n && good; ++j, ++c) {
        const int tok = s.tok0 + j * kPairTokens + lane * box;
        const bool wanted = lane < copies && tok < s.tok1;
        int page = next;
        next = table_entry(table, p.page_size, tok + kPairTokens, lane < copies ? s.tok1 : 0);
        if (page >= p.num_pages) page = -1;
        if (wanted && page < 0) set_status(p.status, PA_DEV_BAD_PAGE);
        const unsigned have = __ballot_sync(kFull, page >= 0);
        const unsigned missing = __ballot_sync(kFull, wanted && page < 0);
        const int row = tok % p.page_size;
        const int valid = min(kPairTokens, s.tok1 - s.tok0 - j * kPairTokens);
        for (g = 0; g < groups; ++g) {
          good = c == 0 || wait_free(g, c - 1, p.wait_ns);
          if (!good) break;
          // One lane a copy
          if (keys) {  // boxes of the CTA's half of the tokens
            if (rank == 0 && lane == 0) {
              const uint32_t bytes = (uint32_t)(__popc(have) * box * 128 * L::BPG);
              if (bytes) mbar_arrive_expect_tx(sb + L::K_FULL + 8 * g, bytes);
              else mbar_arrive(sb + L::K_FULL + 8 * g);
            }
            const int u = lane - rank * per;
            if (page >= 0 && u >= 0 && u < per)
#pragma unroll
              for (int b = L::BPG * g; b < L::BPG * (g + 1); ++b)
                tma_load_3d_pair(sb + L::K + b * L::KBOX + u * box * 128, &p.pages_map, b * 64, row, page,
                                 full0 + 8 * g, keep);
          } else {     // four boxes, the CTA's half of the values, of 64 tokens
            const unsigned mask = ((1u << per) - 1u) << (g * per);
            // rows to clear: the second CTA's copies complete on its own barrier
            const bool clear = (missing & mask) != 0 || (valid % kLatentBlock != 0 && (valid - 1) / 64 == g);
            const uint32_t bytes = (uint32_t)(__popc(have & mask) * box * 128 * 4);
            const bool here = rank != 0 && clear;
            if (lane == 0 && (rank == 0 || clear)) {
              const uint32_t bar = sb + (here ? L::V_HERE : L::V_FULL) + 8 * g;
              *reinterpret_cast<volatile int*>(base + L::CLEAR + 4 * g) = clear;
              if (bytes) mbar_arrive_expect_tx(bar, rank == 0 && !clear ? 2 * bytes : bytes);
              else mbar_arrive(bar);
            }
            __syncwarp();
            const int u = lane - g * per;
            const uint32_t bar = here ? sb + L::V_HERE + 8 * g : full0 + 8 * g;
            if (page >= 0 && u >= 0 && u < per)
#pragma unroll
              for (int b = 0; b < 4; ++b)
                tma_load_3d_pair(sb + L::V + g * L::VGROUP + b * L::VBOX + u * box * 128, &p.pages_map,
                                 ((b >> 1) * 4 + rank * 2 + (b & 1)) * 64, row, page, bar, keep);
            if (clear) {  // the rest of the last 16 tokens, and the tokens of bad pages
              const uint32_t landed = sb + (rank == 0 ? L::V_FULL : L::V_HERE) + 8 * g;
              const uint32_t parity = (uint32_t)((rank == 0 ? c : clears >> g) & 1);
              good = tc5::warp_wait(landed, parity, p.wait_ns);
              clears ^= 1 << g;
              if (!good) {
                tc5::warp_wait(landed, parity, kDrainWaitNs);
                begun = true;
                break;
              }
              __syncwarp();
              for (int v = 0; v < 4; ++v) {
                const int at = g * 64 + v * kLatentBlock;  // first token of the block
                if (at >= valid) break;
                const int from = missing >> (at / box) & 1 ? 0 : valid - at, rows = kLatentBlock - from;
                for (int x = lane; x < rows * 8 * 4; x += 32) {
                  const int b = x / (rows * 8), k = x % (rows * 8);
                  *reinterpret_cast<uint4*>(base + L::V + g * L::VGROUP + b * L::VBOX +
                                            (v * kLatentBlock + from) * 128 + k * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
              }
              fence_proxy_async_smem();  // the tensor core reads them (async proxy)
              __syncwarp();
              if (lane == 0) arrive_first_cta(sb + L::V_CLEAR + 8 * g);
            }
          }
          __syncwarp();
        }
      }
    }
    if (good) {
      // every copy has been read, and with it every arrival that the MMAs send
      // here has come, before the CTA ends
      if (c > 0)
        for (int g = 0; g < groups; ++g) wait_free(g, c - 1, kDrainWaitNs);
      if (qc > 0) tc5::warp_wait(sb + L::Q_FREE, (uint32_t)((qc - 1) & 1), kDrainWaitNs);
    } else {
      if (lane == 0) set_status(p.status, PA_DEV_TIMEOUT);
      // What is under way lands before the CTAs meet at the end: each group's last
      // use, in the stage at which the warp gave up (c - 1: it is counted) or the
      // one before.  The first CTA's barriers count the copies of both (the
      // arrivals of the MMAs come before that of DRAIN).  A count of groups kept
      // as they are issued made two long contexts in pages of 16 tokens 44.4 us
      // instead of 42.9.
      if (rank == 0) {
        const int issued = g + (begun ? 1 : 0);
        for (int x = 0; x < groups; ++x) {
          const int u = c - 1 - (x < issued ? 0 : 1);
          if (u >= 0)
            tc5::warp_wait(sb + (keys ? L::K_FULL : L::V_FULL) + 8 * x, (uint32_t)(u & 1), kDrainWaitNs);
        }
        if (!keys && qc > 0) tc5::warp_wait(sb + L::Q_FULL, (uint32_t)((qc - 1) & 1), kDrainWaitNs);
      }
    }
    __syncwarp();
  } else if (warp == 4) {
    // ================= MMAs (one thread of the first CTA) =================
    if (rank == 0 && tc5::elect_one()) {
      const uint32_t idesc_s = tc5::instr_desc<T>(128, kPairTokens, false);
      const uint32_t idesc_o = tc5::instr_desc<T>(128, 256, true);
      const uint64_t q_desc = tc5::smem_desc(sb + L::Q, 16, 1024), k_desc = tc5::smem_desc(sb + L::K, 16, 1024);
      const uint64_t p_desc = tc5::smem_desc(sb + L::P, 16, 1024);
      const uint64_t v_desc = tc5::smem_desc(sb + L::V, L::VBOX, 1024);
      bool good = true;
      int c = 0, qc = 0;             // stages, segments
      int cleared[L::NV] = {0, 0};   // uses of each value group with rows to clear
      auto wait = [&](int bar, int count) {
        return mbar_wait_bounded(sb + bar, (uint32_t)(count & 1), p.wait_ns);
      };
      // S of stage number cs
      auto scores = [&](int cs, bool last_of_segment) {
#pragma unroll
        for (int g = 0; g < L::NG; ++g) {
          if (!wait(L::K_FULL + 8 * g, cs)) return false;
          tc5::fence_after();
#pragma unroll
          for (int k = 4 * L::BPG * g; k < 4 * L::BPG * (g + 1); ++k)
            tc5::mma2(t_s + (uint32_t)(64 * (cs & 1)),
                      tc5::desc_at(q_desc, (k >> 2) * L::QBOX + (k & 3) * 32),
                      tc5::desc_at(k_desc, (k >> 2) * L::KBOX + (k & 3) * 32), idesc_s, k > 0 ? 1u : 0u);
          if (g < L::NG - 1) tc5::commit2(sb + L::K_FREE + 8 * g);
        }
        tc5::commit2(sb + L::S_DONE + 8 * (cs & 1));
        if (last_of_segment) tc5::commit2(sb + L::Q_FREE);
        return true;
      };
      for (int i = first; i < last && good; ++i) {
        if (i > first) s = p.segments[i];
        if (!usable(s)) continue;
        const int n = stages_of(s);
        good = wait(L::Q_FULL, qc) && scores(c, n == 1);
        for (int j = 0; j < n && good; ++j) {
          const int valid = min(kPairTokens, s.tok1 - s.tok0 - j * kPairTokens);
          if (j + 1 < n) good = scores(c + j + 1, j + 2 == n);
          good = good && wait(L::P_READY, c + j);
          if (!good) break;
#pragma unroll
          for (int g = 0; g < L::NV; ++g) {
            good = wait(L::V_FULL + 8 * g, c + j);
            if (good && *reinterpret_cast<volatile int*>(base + L::CLEAR + 4 * g))
              good = wait(L::V_CLEAR + 8 * g, cleared[g]++);
            if (!good) break;
            tc5::fence_after();
#pragma unroll
            for (int k = 4 * g; k < 4 * g + 4; ++k)
              if (k * 16 < valid) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  tc5::mma2(t_o + (uint32_t)(128 * h),
                            tc5::desc_at(p_desc, (k >> 2) * L::PBOX + (k & 3) * 32),
                            tc5::desc_at(v_desc, g * L::VGROUP + 2 * h * L::VBOX + (k & 3) * 2048), idesc_o,
                            j > 0 || k > 0 ? 1u : 0u);
              }
            if (g < L::NV - 1) tc5::commit2(sb + L::V_FREE + 8 * g);
          }
          if (good) tc5::commit2(sb + L::PV_DONE);
        }
        c += n;
        ++qc;
      }
      if (!good) set_status(p.status, PA_DEV_TIMEOUT);
      // every MMA issued has finished before either CTA goes on
      tc5::commit2(sb + L::DRAIN);
    }
    __syncwarp();
    if (rank == 0) tc5::warp_wait(sb + L::DRAIN, 0u, kDrainWaitNs);
  } else {
    // ================= softmax and output =================
    const int row = (warp & 1) * 32 + lane;        // of the CTA's 64
    const int half = warp >> 1;                    // tokens 64 half .. of a stage; the same part of O
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
        if (threadIdx.x == 0 && rank == 0) set_status(p.status, PA_DEV_PLAN_MISMATCH);
        continue;
      }
      const int32_t* table = p.block_table + (int64_t)s.b * p.max_pages;
      const int n = stages_of(s);
      const int trow = rank * kPairRows + row;     // of the tile
      const int lim0 = trow < s.nrows ? s.pos0 + (s.row0 + trow) / p.heads : -1;  // last visible token
      const bool idle = rank * kPairRows + (warp & 1) * 32 >= s.nrows;  // no row of the warp's is real
      float m_run = -INFINITY, l_run = 0.f;
      int nph[4];  // pages of the thread's 64 tokens, a stage ahead
      auto load_pages = [&](int j) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int tok = s.tok0 + j * kPairTokens + half * 64 + u * 16;
          nph[u] = table_entry(table, p.page_size, tok, idle ? 0 : s.tok1);
        }
      };
      load_pages(0);
      for (int j = 0; j < n; ++j) {
        const int cs = c + j;
        if (!idle) {
          bool ok_page[4];
          bool all_ok = true;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            ok_page[u] = nph[u] >= 0 && nph[u] < p.num_pages;
            all_ok = all_ok && ok_page[u];
          }
          if (j + 1 < n) load_pages(j + 1);
          wait(L::S_DONE + 8 * (cs & 1), (uint32_t)((cs >> 1) & 1));
          tc5::fence_after();
          float sv[64];
          __syncwarp();  // the wait's lanes meet: tensor memory is for a whole warp
#pragma unroll
          for (int x = 0; x < 64; x += 16) tc5::ld16(t_s + (uint32_t)(64 * (cs & 1) + x) + lane_off, sv + x);
          tc5::wait_ld();
          const int tok = s.tok0 + j * kPairTokens + half * 64;
          const int lim = min(lim0, s.tok1 - 1) - tok;  // last visible column
          if (!__all_sync(kFull, all_ok && lim >= 63)) {
#pragma unroll
            for (int x = 0; x < 64; ++x) sv[x] = ok_page[x / 16] && x <= lim ? sv[x] : -INFINITY;
          }
          float mx4[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
          for (int x = 4; x < 64; ++x) mx4[x & 3] = fmaxf(mx4[x & 3], sv[x]);
          float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * p.qscale;
          // the maximum over both halves; two uses in turn, so one barrier a stage
          volatile float* xm = xmax + (cs & 1) * 128;
          xm[half * 64 + row] = mx;
          row_pair_barrier(warp);
          mx = fmaxf(mx, xm[(half ^ 1) * 64 + row]);
          float al = 1.f;
          bool resc = false;
          if (mx > m_run + kPairLazyLog2) {
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
          uint32_t pk[32];
#pragma unroll
          for (int x = 0; x < 64; x += 2) {
            const float2 e = ffma2(make_float2(sv[x], sv[x + 1]), qs2, nm2);
            const float2 w = make_float2(ex2(e.x), ex2(e.y));
            sum[(x >> 1) & 1] = fadd2(sum[(x >> 1) & 1], w);
            pk[x >> 1] = Elem<T>::from_f2(w.x, w.y);
          }
          const float2 s2 = fadd2(sum[0], sum[1]);
          l_run = l_run * al + (s2.x + s2.y);
          // P and O are free once the product before is done
          if (cs > 0) wait(L::PV_DONE, (uint32_t)((cs - 1) & 1));
          tc5::fence_after();
          unsigned char* pr = base + L::P + half * L::PBOX + row * 128;
#pragma unroll
          for (int x = 0; x < 8; ++x)
            *reinterpret_cast<uint4*>(pr + ((x ^ (row & 7)) << 4)) =
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
          wait(L::PV_DONE, (uint32_t)((cs - 1) & 1));
        }
        __syncwarp();
        if (good && lane == 0) arrive_first_cta(sb + L::P_READY);
      }
      c += n;
      wait(L::PV_DONE, (uint32_t)((c - 1) & 1));
      if (!idle) {
        // the row's sum over both halves, and whether both warps got here in order
        volatile float* xs = xmax + (c & 1) * 128;
        xs[half * 64 + row] = good ? l_run : -1.f;
        row_pair_barrier(warp);
        const float other = xs[(half ^ 1) * 64 + row];
        const bool whole = good && !(other < 0.f);
        const float l = l_run + other;
        const float inv = l > 0.f || l != l ? 1.f / l : 0.f;  // a NaN sum stays NaN
        const bool mine = trow < s.nrows;
        const int64_t grow = (int64_t)s.packed0 + trow;
        const int64_t at = (int64_t)s.slot * p.rows + trow;
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
  cluster_sync();  // the first CTA has committed its last products and seen them end
  if (warp == 4) {
    // the commit's arrival here: counted from the barrier, so that the limit holds
    // whatever the range took
    if (rank != 0) tc5::warp_wait(sb + L::DRAIN, 0u, kDrainWaitNs);
    tc5::fence_after();
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
  cluster_sync();
}

template <typename T>
cudaError_t launch_t(const LatentParams& p, const CUtensorMap& q_map, cudaStream_t stream) {
  static std::atomic<unsigned long long> configured{0};
  return launch_latent(latent_pair_kernel<T>, PLayout::BYTES, configured, 2 * p.num_ranges, kPairThreads,
                       stream, p, q_map);
}

}  // namespace

cudaError_t launch_latent_pair(const LatentParams& params, const pa_latent_shape_t& shape,
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
