// Absorbed latent attention for tiles of up to 16 query rows (mma.sync), and
// the merge of tiles that were cut.
//
// For a tile of 16 rows (tokens x heads of one sequence) over its cached
// rows z_t = [c_t ; r_t]:
//   s[i][t] = q_i . z_t,  p = 2^(s * qscale - m),  o_i = sum_t p[i][t] c_t / sum_t p[i][t]
// with the running maximum m of an online softmax.  Every cached byte is
// read once for up to 16 rows and feeds 1088 multiply-adds per row and
// token, far below what the tensor cores do in the time its bytes take, so
// the kernel is built to keep HBM busy.
//
// One CTA per SM.  Warp 8 copies: a ring of 11 blocks of 16 tokens (18 KB
// each, one TMA copy) holds about 200 KB, so that some 130 KB are in flight
// while 64 tokens are worked on.  A block lands as [16 tokens][9 x 128 B]
// with the 128-byte swizzle over the 128-byte lines, line = 9 token + box:
// eight tokens of one box differ in line % 8, so every ldmatrix is free of
// bank conflicts.
// Warps 0-7 work on stages of 64 tokens:
//   scores: warp w takes a quarter of the 576 dims (w % 4) of 32 tokens
//     (w / 4), its part of q held in 36 registers per lane; the four parts are
//     added through shared memory
//   softmax: warp w takes rows 2w and 2w + 1
//   output: warp w takes 64 of the 512 values, over all 64 tokens
// The weights p go to the second product as hi + lo parts of the element
// type (elem.cuh): the tensor cores have the time, and the result then
// differs from fp32 weights by its own rounding only.
//
// Measured: 64 sequences of 500 to 8001 tokens with 16 heads (320 MB) 64.6 us,
// merge included, 73 % of the copy bandwidth; in its steady state a stage of 64
// tokens takes 1.7 us on every SM at once, 95 % of it.  The rest is the start,
// the last pieces' output and the merge, about 10 us.  One sequence of 1000
// tokens: 8.6 us.
#include <math.h>

#include "decode_tc.cuh"
#include "device_common.cuh"
#include "elem.cuh"
#include "latent_segment.cuh"
#include "latent_launch.cuh"

namespace pa {

namespace {

constexpr int kWorkWarps = 8;
// Warps of the merge in all up to which a warp may have as few as two pieces of a
// row, and three (about 7 and 20 an SM).
constexpr int kMergeFewWarps = 1100, kMergeMostWarps = 3040;
PA_HD constexpr int kMergeWarps(int warps_per_row) { return warps_per_row < 4 ? 4 : warps_per_row; }
constexpr int kMmaThreads = (kWorkWarps + 1) * 32;

struct MmaLayout {
  static constexpr int SLOTS = 11;
  static constexpr int SLOT = kLatentBlock * kLatentRow * 2;  // 18 KB, a multiple of 1024
  static constexpr int RED_PITCH = 68;                        // floats per row of partial scores
  static constexpr int RED = SLOTS * SLOT;                    // [4 quarters][16 rows][pitch]
  static constexpr int P_PITCH = 144;                         // bytes per row of 64 weights
  static constexpr int P_HI = RED + 4 * 16 * RED_PITCH * 4;
  static constexpr int P_LO = P_HI + 16 * P_PITCH;
  static constexpr int ALPHA = P_LO + 16 * P_PITCH;           // [16] rescale factors
  static constexpr int SUM = ALPHA + 64;                      // [16] row sums
  static constexpr int MAX = SUM + 64;                        // [16] row maxima (log2 units)
  static constexpr int FULL = MAX + 64;                       // mbarriers: a block has landed
  static constexpr int FREE = FULL + 8 * SLOTS;               // every warp is done with a block
  static constexpr int VALID = FREE + 8 * SLOTS;              // the block's page index was good
  static constexpr int FLAG = VALID + 4 * SLOTS;              // a working warp's wait gave up
  static constexpr int BYTES = align_up(FLAG + 4, 16) + 1024;
};
static_assert(MmaLayout::BYTES <= kMaxCtaSmem, "ring does not fit in shared memory");

__device__ __forceinline__ void work_barrier() {
  __syncwarp();  // the barrier is for converged warps
  asm volatile("bar.sync 1, %0;" ::"n"(kWorkWarps * 32) : "memory");
}

// Address of 16-byte chunk `chunk` (0..71) of token `row` of a block.
__device__ __forceinline__ uint32_t block_chunk(uint32_t block, int row, int chunk) {
  const int line = row * (kLatentRow / 64) + (chunk >> 3);
  return block + (uint32_t)(line * 128 + (((chunk ^ line) & 7) << 4));
}

template <typename T>
__global__ void __launch_bounds__(kMmaThreads, 1)
    latent_mma_kernel(const __grid_constant__ LatentParams p) {
  using L = MmaLayout;
  extern __shared__ unsigned char smem_dyn[];
  unsigned char* base = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(base);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* flag = reinterpret_cast<int*>(base + L::FLAG);
  volatile int* valid = reinterpret_cast<int*>(base + L::VALID);

  int first, last;
  const bool planned = latent_range(p, kLatentRowsMma, (int)blockIdx.x, first, last);
  if (threadIdx.x == 0) {
    *flag = 0;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.pages_map)) : "memory");
    for (int s = 0; s < L::SLOTS; ++s) {
      mbar_init(sbase + L::FULL + 8 * s, 1);
      mbar_init(sbase + L::FREE + 8 * s, kWorkWarps);
    }
    fence_barrier_init();
  }
  LatentSegment s{};
  if (first < last) s = p.segments[first];
  __syncthreads();
  pdl_launch_dependents();
  pdl_wait_primary();
  if (!planned && threadIdx.x == 0) set_status(p.status, PA_DEV_PLAN_MISMATCH);

  if (warp == kWorkWarps) {
    // ================= copies =================
    const uint64_t policy = l2_evict_first_policy();
    int k = 0;  // blocks issued
    bool good = true;
    for (int i = first; i < last && good; ++i) {
      if (i > first) s = p.segments[i];
      if (!latent_segment_ok(p, s, kLatentRowsMma)) continue;  // the working warps report it
      const int32_t* table = p.block_table + (int64_t)s.b * p.max_pages;
      const int blocks = (s.tok1 - s.tok0 + kLatentBlock - 1) / kLatentBlock;
      int entry = -1;
      for (int j = 0; j < blocks; ++j) {
        if ((j & 31) == 0) {
          const int t = s.tok0 + (j + lane) * kLatentBlock;
          entry = j + lane < blocks ? table[t / p.page_size] : -1;
        }
        const int page = __shfl_sync(kFull, entry, j & 31);
        const int slot = k % L::SLOTS;
        if (lane == 0) {
          good = k < L::SLOTS || mbar_wait_bounded_sleep(sbase + L::FREE + 8 * slot,
                                                         (uint32_t)((k / L::SLOTS - 1) & 1), p.wait_ns);
          if (good) {
            const bool ok = page >= 0 && page < p.num_pages;
            valid[slot] = ok;
            const uint32_t bar = sbase + L::FULL + 8 * slot;
            if (ok) {
              mbar_arrive_expect_tx(bar, L::SLOT);
              tma_load_4d(sbase + slot * L::SLOT, &p.pages_map, 0, 0,
                          (s.tok0 + j * kLatentBlock) % p.page_size, page, bar, policy);
            } else {
              set_status(p.status, PA_DEV_BAD_PAGE);
              mbar_arrive(bar);
            }
          }
        }
        good = __shfl_sync(kFull, good, 0);
        if (!good) break;
        ++k;
      }
    }
    if (lane == 0) {
      if (!good) set_status(p.status, PA_DEV_TIMEOUT);  // the working warps' waits run out too
      // copies in flight land before the CTA exits
      for (int j = k < L::SLOTS ? 0 : k - L::SLOTS; j < k; ++j)
        mbar_wait_bounded_sleep(sbase + L::FULL + 8 * (j % L::SLOTS), (uint32_t)((j / L::SLOTS) & 1),
                                kDrainWaitNs);
    }
    return;
  }

  // ================= work =================
  const int g = lane >> 2, t4 = lane & 3;
  const int quarter = warp & 3, half = warp >> 2;
  float* red = reinterpret_cast<float*>(base + L::RED);
  volatile float* alpha_s = reinterpret_cast<float*>(base + L::ALPHA);
  volatile float* sum_s = reinterpret_cast<float*>(base + L::SUM);
  volatile float* max_s = reinterpret_cast<float*>(base + L::MAX);
  const int srow = 2 * warp + (lane >> 4), scol = (lane & 15) * 4;  // this lane's softmax row, tokens
  int k = 0;         // blocks consumed
  bool good = true;  // after a wait that gave up, a warp only keeps its place in the barriers
  for (int i = first; i < last; ++i) {
    if (i > first) s = p.segments[i];
    if (!latent_segment_ok(p, s, kLatentRowsMma)) {  // the same for every warp
      if (threadIdx.x == 0) set_status(p.status, PA_DEV_PLAN_MISMATCH);
      continue;
    }
    const int64_t grow = s.packed0;  // packed row of tile row 0

    // this warp's quarter of q: nine A fragments of 16 dims
    uint32_t qa[9][4];
    const T* q = static_cast<const T*>(p.q) + grow * kLatentRow + quarter * 144 + 2 * t4;
#pragma unroll
    for (int ks = 0; ks < 9; ++ks)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int row = g + (c & 1) * 8;
        qa[ks][c] = row < s.nrows ? __ldg(reinterpret_cast<const unsigned int*>(
                                        q + (int64_t)row * kLatentRow + ks * 16 + (c >> 1) * 8))
                                  : 0u;
      }
    // last token that this lane's softmax row sees
    const int lim = srow < s.nrows ? s.pos0 + (s.row0 + srow) / p.heads : -1;
    float m_run = -INFINITY, l_run = 0.f;
    float o[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[n][c] = 0.f;

    for (int t0 = s.tok0; t0 < s.tok1; t0 += kLatentStage) {
      const int blocks = min(kLatentStage / kLatentBlock, (s.tok1 - t0 + kLatentBlock - 1) / kLatentBlock);
      // lane u waits for block u; a block counts if its page was good
      bool landed = true, usable = false;
      if (lane < blocks) {
        const int slot = (k + lane) % L::SLOTS;
        landed = good && mbar_wait_bounded(sbase + L::FULL + 8 * slot,
                                           (uint32_t)(((k + lane) / L::SLOTS) & 1), p.wait_ns);
        usable = landed && valid[slot];
      }
      good = __all_sync(kFull, landed);
      const unsigned ok_blocks = good ? __ballot_sync(kFull, usable) : 0u;
      __syncwarp();
      uint32_t blk[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) blk[u] = sbase + (uint32_t)((k + u) % L::SLOTS) * L::SLOT;
      if (!good) *flag = 1;

      // ---- scores of 32 tokens over a quarter of the dims
#pragma unroll
      for (int u2 = 0; u2 < 2; ++u2) {
        const int u = 2 * half + u2;
        float sc[2][4] = {};
        if (ok_blocks >> u & 1) {
          const int row = (lane & 7) + ((lane >> 4) & 1) * 8;
          const uint32_t b0 = half ? blk[2 + u2] : blk[u2];
#pragma unroll
          for (int ks = 0; ks < 9; ++ks) {
            uint32_t r0, r1, r2, r3;
            ldsm_x4(block_chunk(b0, row, (quarter * 9 + ks) * 2 + ((lane >> 3) & 1)), r0, r1, r2, r3);
            mma_16816<T>(sc[0], qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], r0, r1);
            mma_16816<T>(sc[1], qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], r2, r3);
          }
        }
        float* dst = red + (quarter * 16 + g) * L::RED_PITCH + u * 16 + 2 * t4;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          *reinterpret_cast<float2*>(dst + 8 * n) = make_float2(sc[n][0], sc[n][1]);
          *reinterpret_cast<float2*>(dst + 8 * L::RED_PITCH + 8 * n) = make_float2(sc[n][2], sc[n][3]);
        }
      }
      work_barrier();

      // ---- softmax of two rows per warp, four tokens per lane
      {
        float x[4] = {};
#pragma unroll
        for (int qt = 0; qt < 4; ++qt) {
          const float4 v = *reinterpret_cast<const float4*>(red + (qt * 16 + srow) * L::RED_PITCH + scol);
          x[0] += v.x;
          x[1] += v.y;
          x[2] += v.z;
          x[3] += v.w;
        }
        const bool okb = ok_blocks >> (scol / kLatentBlock) & 1;
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int t = t0 + scol + c;
          x[c] = okb && t <= lim && t < s.tok1 ? x[c] * p.qscale : -INFINITY;
          mx = fmaxf(mx, x[c]);
        }
#pragma unroll
        for (int w = 8; w >= 1; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, w));
        const float m_new = fmaxf(m_run, mx);
        const float m_ref = m_new == -INFINITY ? 0.f : m_new;  // a row with no token yet: all weights 0
        const float al = ex2(m_run - m_ref);
        const float2 p0 = make_float2(ex2(x[0] - m_ref), ex2(x[1] - m_ref));
        const float2 p1 = make_float2(ex2(x[2] - m_ref), ex2(x[3] - m_ref));
        float ps = (p0.x + p0.y) + (p1.x + p1.y);
#pragma unroll
        for (int w = 8; w >= 1; w >>= 1) ps += __shfl_xor_sync(kFull, ps, w);
        l_run = l_run * al + ps;
        m_run = m_new;
        uint2 hi, lo;
        split_hi_lo<T>(p0, hi.x, lo.x);
        split_hi_lo<T>(p1, hi.y, lo.y);
        *reinterpret_cast<uint2*>(base + L::P_HI + srow * L::P_PITCH + scol * 2) = hi;
        *reinterpret_cast<uint2*>(base + L::P_LO + srow * L::P_PITCH + scol * 2) = lo;
        if ((lane & 15) == 0) alpha_s[srow] = al;
      }
      // rows past the last token (their weight is 0, but they may hold
      // anything, NaN too) become zeros; the scores have read them
      const int tail = s.tok1 - t0 - (blocks - 1) * kLatentBlock;  // tokens of the last block
      if (tail < kLatentBlock && good) {
        unsigned char* b = base + ((k + blocks - 1) % L::SLOTS) * L::SLOT;
        const int lines = kLatentRow / 64 * 8;  // 16-byte chunks per row
        for (int c = tail * lines + (int)threadIdx.x; c < kLatentBlock * lines; c += kWorkWarps * 32)
          *reinterpret_cast<uint4*>(b + c * 16) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();  // a later copy (async proxy) writes them again
      }
      work_barrier();

      // ---- o = o * alpha + p c, 64 values per warp
      const float a0 = alpha_s[g], a1 = alpha_s[g + 8];
      if (__any_sync(kFull, a0 != 1.f || a1 != 1.f)) {
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          o[n][0] *= a0;
          o[n][1] *= a0;
          o[n][2] *= a1;
          o[n][3] *= a1;
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (!(ok_blocks >> u & 1)) continue;
        const int row = (lane & 7) + ((lane >> 3) & 1) * 8;
        const uint32_t pa = (uint32_t)(row * L::P_PITCH + (u * 2 + (lane >> 4)) * 16);
        uint32_t h[4], l[4];
        ldsm_x4(sbase + L::P_HI + pa, h[0], h[1], h[2], h[3]);
        ldsm_x4(sbase + L::P_LO + pa, l[0], l[1], l[2], l[3]);
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          uint32_t r0, r1, r2, r3;
          ldsm_x4_t(block_chunk(blk[u], row, warp * 8 + d * 2 + (lane >> 4)), r0, r1, r2, r3);
          mma_16816<T>(o[2 * d], h[0], h[1], h[2], h[3], r0, r1);
          mma_16816<T>(o[2 * d + 1], h[0], h[1], h[2], h[3], r2, r3);
          mma_16816<T>(o[2 * d], l[0], l[1], l[2], l[3], r0, r1);
          mma_16816<T>(o[2 * d + 1], l[0], l[1], l[2], l[3], r2, r3);
        }
      }
      __syncwarp();
      if (good && lane < blocks) mbar_arrive(sbase + L::FREE + 8 * ((k + lane) % L::SLOTS));
      k += blocks;
    }

    if ((lane & 15) == 0) {
      sum_s[srow] = l_run;
      max_s[srow] = m_run;
    }
    work_barrier();
    if (*flag == 0) {
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int row = g + 8 * hh;
        if (row >= s.nrows) continue;
        const float l = sum_s[row];
        const float inv = l > 0.f || l != l ? 1.f / l : 0.f;  // a NaN sum stays NaN
        const int dim = warp * 64 + 2 * t4;
        if (s.slot < 0) {
          T* out = static_cast<T*>(p.out) + (grow + row) * kLatent + dim;
#pragma unroll
          for (int n = 0; n < 8; ++n)
            *reinterpret_cast<uint32_t*>(out + 8 * n) =
                Elem<T>::from_f2(o[n][2 * hh] * inv, o[n][2 * hh + 1] * inv);
        } else {
          const int64_t at = (int64_t)s.slot * p.rows + row;
          float* po = p.part_o + at * kLatent + dim;
#pragma unroll
          for (int n = 0; n < 8; ++n)
            *reinterpret_cast<float2*>(po + 8 * n) =
                make_float2(o[n][2 * hh] * inv, o[n][2 * hh + 1] * inv);
          if (warp == 0 && t4 == 0)
            p.part_lse[at] = l > 0.f || l != l ? max_s[row] + lg2(l) : -INFINITY;
        }
      }
    } else {
      if (threadIdx.x == 0) set_status(p.status, PA_DEV_TIMEOUT);
      if (s.slot >= 0 && (int)threadIdx.x < s.nrows)  // the merge leaves these rows unwritten
        p.part_lse[(int64_t)s.slot * p.rows + threadIdx.x] = INFINITY;
    }
    work_barrier();  // the statistics are read before the next segment writes them
  }
}

// Merge the rows of the tiles that were cut: out = sum_s w_s o_s / sum_s w_s,
// w_s = 2^(lse_s - max lse).  Pieces in a fixed order, so the sum is the same
// on every call.  A piece whose waits gave up left an lse of +infinity, which
// no piece that completed has: its rows stay unwritten.
// The partials come from L2, where they were written a moment before: the time
// is that of a launch and of a row's loads, one behind the other.
// WARPS warps share a row's pieces, each covering all 512 values: as many as
// leave each a few pieces and run at once.  Measured, whole calls: 1280 rows of 7
// pieces (64-row tiles) 31.7 us with one warp a row, 29.9 with two, 30.5 with
// four; 512 rows of 8 pieces 14.8 with two, 16.2 with four, 17.1 with eight; 128
// rows of 16 pieces 10.0 with four, 9.4 with eight; 64 rows of 152 pieces 26.6
// with four, 23.6 with eight; 1024 rows of 4 pieces 14.7 with one, 15.9 with two.
// A merge by the last piece of a tile to end, inside the first kernel, was
// slower (batch of 64, 16 heads: 69.6 against 64.5 us): its reads began when
// everything else was over, on one SM a tile.
template <typename T, int WARPS>
__global__ void __launch_bounds__(kMergeWarps(WARPS) * 32)
    latent_merge_kernel(const __grid_constant__ LatentParams p) {
  constexpr int ROWS = kMergeWarps(WARPS) / WARPS;  // rows of a block
  constexpr int BATCH = 4;                          // pieces in flight
  __shared__ float4 acc_s[kMergeWarps(WARPS)][WARPS > 1 ? kLatent / 4 : 1];
  __shared__ float sum_s[kMergeWarps(WARPS)];
  const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
  const int part = warp % WARPS;
  const bool planned = latent_planned(p, p.rows);
  const int which = (int)blockIdx.x * ROWS + warp / WARPS;  // row of all tiles' rows
  const LatentMerge m = p.merges[which / p.rows];           // p.rows is a multiple of ROWS
  const int row = which % p.rows;
  pdl_launch_dependents();
  pdl_wait_primary();
  if (!planned) return;  // reported already; the same in the whole grid
  const bool ok = row < m.nrows && m.slot0 >= 0 && m.n >= 1 && (int64_t)m.slot0 + m.n <= p.num_slots &&
                  m.row0 >= 0 && (int64_t)m.row0 + m.nrows <= (int64_t)p.total_q * p.heads;
  const int n = ok ? m.n : 0;
  const float* lse = p.part_lse + (int64_t)m.slot0 * p.rows + row;
  const float4* o =
      reinterpret_cast<const float4*>(p.part_o + ((int64_t)m.slot0 * p.rows + row) * kLatent) + lane;
  const int64_t step = (int64_t)p.rows * (kLatent / 4);
  float4 v[BATCH][4];
  auto load = [&](int s0) {
#pragma unroll
    for (int b = 0; b < BATCH; ++b)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        v[b][c] = s0 + b * WARPS < n ? __ldcg(o + (int64_t)(s0 + b * WARPS) * step + 32 * c)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  load(part);  // in flight while the weights are found
  float mx = -INFINITY;
  for (int s = lane; s < n; s += 32) mx = fmaxf(mx, __ldcg(lse + (int64_t)s * p.rows));
#pragma unroll
  for (int w = 16; w >= 1; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, w));
  const bool whole = ok && mx != INFINITY;  // the same in every warp of the row
  const float ref = mx == -INFINITY ? 0.f : mx;
  float4 acc[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  for (int s0 = part; s0 < n; s0 += BATCH * WARPS) {
    if (s0 >= WARPS) load(s0);
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      const int s = s0 + b * WARPS;
      if (s >= n) break;
      const float w = ex2(__ldcg(lse + (int64_t)s * p.rows) - ref);
      sum += w;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        acc[c].x += w * v[b][c].x;
        acc[c].y += w * v[b][c].y;
        acc[c].z += w * v[b][c].z;
        acc[c].w += w * v[b][c].w;
      }
    }
  }
  if (WARPS > 1) {
#pragma unroll
    for (int c = 0; c < 4; ++c) acc_s[warp][lane + 32 * c] = acc[c];
    if (lane == 0) sum_s[warp] = sum;
    __syncthreads();
    if (part > 0) return;
#pragma unroll 1
    for (int g = warp + 1; g < warp + WARPS; ++g) {
      sum += sum_s[g];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float4 x = acc_s[g][lane + 32 * c];
        acc[c].x += x.x;
        acc[c].y += x.y;
        acc[c].z += x.z;
        acc[c].w += x.w;
      }
    }
  }
  if (!whole) return;
  const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
  uint2* out = reinterpret_cast<uint2*>(static_cast<T*>(p.out) + ((int64_t)m.row0 + row) * kLatent) + lane;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    out[32 * c] = make_uint2(Elem<T>::from_f2(acc[c].x * inv, acc[c].y * inv),
                             Elem<T>::from_f2(acc[c].z * inv, acc[c].w * inv));
}

// The pool [P][S][576] with boxes of 16 whole rows, 128-byte swizzle over
// their 128-byte lines.
bool encode_latent_map(CUtensorMap* map, const void* pages, const pa_latent_shape_t& s) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = latent_map_encoder();
  if (!enc) return false;
  const cuuint64_t row = kLatentRow * 2;
  cuuint64_t dims[4] = {64, kLatentRow / 64, (cuuint64_t)s.page_size, (cuuint64_t)s.num_pages};
  cuuint64_t strides[3] = {128, row, row * s.page_size};
  cuuint32_t box[4] = {64, kLatentRow / 64, kLatentBlock, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUtensorMapDataType ty = s.dtype == PA_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                         : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return enc(map, ty, 4, const_cast<void*>(pages), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T>
cudaError_t launch_mma_t(const LatentParams& p, cudaStream_t stream) {
  static std::atomic<unsigned long long> configured{0};
  return launch_latent(latent_mma_kernel<T>, MmaLayout::BYTES, configured, p.num_ranges, kMmaThreads,
                       stream, p);
}

template <typename T, int WARPS>
cudaError_t launch_merge_t(const LatentParams& p, cudaStream_t stream) {
  static std::atomic<unsigned long long> configured{0};
  constexpr int ROWS = kMergeWarps(WARPS) / WARPS;
  const int64_t rows = (int64_t)p.num_merges * p.rows;
  return launch_latent(latent_merge_kernel<T, WARPS>, 0, configured, (int)(rows / ROWS),
                       kMergeWarps(WARPS) * 32, stream, p);
}

template <typename T>
cudaError_t launch_merge_any(const LatentParams& p, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.num_merges * p.rows, pieces = p.num_slots / p.num_merges;
  int warps = 8;
  while (warps > 1 && !(rows * warps <= kMergeFewWarps && pieces >= 2 * warps) &&
         !(rows * warps <= kMergeMostWarps && pieces >= 3 * warps))
    warps /= 2;
  if (warps == 1) return launch_merge_t<T, 1>(p, stream);
  if (warps == 2) return launch_merge_t<T, 2>(p, stream);
  if (warps == 4) return launch_merge_t<T, 4>(p, stream);
  return launch_merge_t<T, 8>(p, stream);
}

}  // namespace

cudaError_t launch_latent_mma(const LatentParams& params, const pa_latent_shape_t& shape,
                              const void* pages, cudaStream_t stream) {
  LatentParams p = params;
  if (!encode_latent_map(&p.pages_map, pages, shape)) return cudaErrorInvalidValue;
  if (shape.dtype == PA_DTYPE_BF16) return launch_mma_t<__nv_bfloat16>(p, stream);
  return launch_mma_t<__half>(p, stream);
}

cudaError_t launch_latent_merge(const LatentParams& p, int dtype, cudaStream_t stream) {
  if (dtype == PA_DTYPE_BF16) return launch_merge_any<__nv_bfloat16>(p, stream);
  return launch_merge_any<__half>(p, stream);
}

}  // namespace pa
