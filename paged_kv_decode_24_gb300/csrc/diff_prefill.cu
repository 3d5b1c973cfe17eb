// Differential attention of several new tokens a sequence on tcgen05, causal,
// over the paged cache, in two passes over the keys:
//
//   pass 1:  m_k = max_t s_k[t],  l_k = sum_t 2^(s_k[t] - m_k)     (k = 1, 2)
//   pass 2:  o = sum_t (2^(s_1[t] - m_1) / l_1 - lambda 2^(s_2[t] - m_2) / l_2) V[t]
//   out = factor w o / sqrt(mean(o^2) + eps)
//
// With both maps' sums known, their difference is formed as one weight before
// it meets the values.  That is as many operations as two products with the
// values (12 D a head and visible pair: 4 D of scores twice, 4 D of values, with
// values twice as wide as keys), but one weight is rounded where there were two,
// one accumulator of 2D columns is left of two (with D = 128 two do not fit in
// tensor memory), and it is never rescaled.  It costs every exponential twice.
// A weight is kept in two parts of the element type, what rounding left of the
// first being the second: rounded once, the outputs of long prompts were 1.35 to
// 1.4 times as far from the 64-bit ones as those of fp32 weights.
// The tiles are those of the multi-token plan, 128 rows (128 / G query tokens
// times the G heads of a KV head), of which the plan lists two for each pair of
// KV heads.  A CTA (one per SM) takes both as one:
//   16 row warps: softmax and output, thread = row = TMEM lane, four warps to the
//              same 32 rows: in pass 1 half of the columns of one map each, in
//              pass 2 a share of the tokens, at the end a quarter of the columns.
//              (Two warps to 32 rows, with twice the columns each, left the
//              exponentials' latencies open: 4100 tokens, 32 heads of 64, 176 us.)
//   2 warps:   one thread issues the MMAs of the scores, one those with the values
//   2 warps:   one thread copies keys, one values
// Shared memory (128-byte swizzle): q 2 x [D/64][128 rows][128 B]; a ring of key
// stages, [2 maps][D/64][tokens][128 B]; a ring of value stages,
// [pages][D/64][2 heads][16 tokens][128 B].  A stage is 128 tokens with D = 64,
// 64 with D = 128.
// TMEM (512 columns): pass 1 has score buffers of both maps' stages in all of
// them (D = 128: in three quarters, and q); in pass 2 a buffer is 2 x 64 columns, and
// O takes the last 2D.  The weights take the place of the first map's scores, each
// warp's over its own columns, two 16-bit weights a column.
//
// Pass 2, 64 tokens at a time, B buffers:
//   S_2(i), S_1(i) = q_k K_k(i)^T     D/16 MMAs each, M = 128, N = 64
//   weights in registers, written over S_1(i)
//   O += P(i) V(i)                    8 MMAs, N = 2D: both parts of the weights
//   S_2(i + B), then, once P V(i) is done, S_1(i + B)
// Value rows past the tile's last visible token and of bad pages (which may
// hold anything) become zeros before P V reads them.  Every wait is bounded; a
// CTA that gave up writes nothing.
//
// Measured: a prompt of 8192 tokens with 32 query heads of 128 (16 heads), 762 to 780 us,
// 1070 TFLOP/s of the formula's operations (12 D a visible pair), 1430 with those of the
// weights' second parts (4 D more), of the 1705 that a library product reaches under the
// power cap; the tensor cores and the thread that feeds them bound it, in pass 2 with
// 64-token score tiles that read q from shared memory at two thirds of their rate.  4100
// tokens, 32 query heads of 64: 151 us, 684 TFLOP/s (912): neither the tensor cores (42 % of
// the clocks) nor the exponentials (40 %, each taken twice), but the waits and hand-overs
// between them.  Weights rounded once took 620 and 143 us; the steps' figures below were
// taken with those.
#include <math.h>

#include "diff.h"
#include "latent_launch.cuh"
#include "latent_tc5.cuh"

namespace pa {

namespace {

constexpr int kRows = 128;    // rows of a tile (TMEM lanes)
constexpr int kTokens = 64;   // tokens of a buffer in pass 2
constexpr int kRowWarps = 16;  // four to each 32 rows: with two the exponentials' latencies showed
constexpr int kDiffPrefillThreads = (kRowWarps + 4) * 32;
// Beyond this a row's reference point is too coarse in fp32 to hold log2 of the
// sum as well (2^-14 of a weight at 2^10): the factor is multiplied instead.
constexpr float kFoldedLog2 = 1024.f;
// A stage's sum of weights, relative to the row's reference, up to which that
// reference stays.
constexpr float kLateSum = 128.f;

template <int D>
struct DPLayout {
  // Tokens of a stage of copies, and of a score buffer in pass 1.  Waits and loops
  // take each of the CTA's threads 500 to 700 clocks a stage with nothing to do in it,
  // as long as the work on 64 tokens with D = 64, so those stages have 128; with
  // D = 128 such stages leave no room for a second one.
  static constexpr int KT = D == 64 ? 128 : 64;
  static constexpr int PAGES = KT / kPageSize;
  static constexpr int PARTS = KT / kTokens;            // buffers of pass 2 in a stage
  static constexpr int KB = D / 64;                     // boxes of 64 dims
  static constexpr int QBOX = kRows * 128;              // 16 KB: 64 dims of 128 rows
  static constexpr int QMAP = KB * QBOX;
  static constexpr int KBOX = KT * 128;                 // 64 dims of a stage's tokens
  static constexpr int KSTAGE = 2 * KB * KBOX;
  static constexpr int VPAGE = 2 * KB * kPageSize * 128;
  static constexpr int VSTAGE = PAGES * VPAGE;
  static constexpr int NK = 3;                          // key stages
  static constexpr int NV = D == 64 ? 3 : 2;            // value stages
  // With D = 128 pass 1 reads q from tensor memory too, in the columns that a fourth
  // buffer would take: with 64 tokens a product, reading both operands from shared memory
  // takes half as long again as the product (658 -> 635 us, prompt of 8192 tokens).
  static constexpr bool QT = D == 128;
  static constexpr int NB1 = QT ? 3 : 512 / (2 * KT);   // score buffers of pass 1
  [[maybe_unused]] static constexpr int QCOL = 512 - D;  // q's first column in pass 1: 2 maps x D / 2
  static constexpr int NB = D == 64 ? 3 : 2;            // score buffers of pass 2
  // In pass 1 with D = 128, half of the row warps take every other buffer, all columns of
  // a map each (635 -> 620 us); with D = 64 a buffer has twice the tokens already.
  static constexpr int TURNS1 = D == 128 ? 2 : 1;
  // With three buffers, half of the row warps take every other one, 32 columns each, and
  // a warp's waits and hand-overs are half as many; with two, the next product would
  // wait for the longer way through a buffer (658 against 692 us, prompt of 8192 tokens),
  // and all warps take 16 columns of each.
  static constexpr int TURNS = NB > 2 ? 2 : 1;
  static constexpr int MINE = 16 * TURNS;               // columns of a warp
  static constexpr int O = 4 * 128 - 2 * D;             // O's first column
  static_assert(NB * 128 <= O, "O follows the buffers");
  static constexpr int Q = 0;
  static constexpr int K = Q + 2 * QMAP;
  static constexpr int V = K + NK * KSTAGE;
  static constexpr int BARS = V + NV * VSTAGE;
  // mbarriers
  static constexpr int K_FULL = BARS;
  static constexpr int K_FREE = K_FULL + 8 * NK;
  static constexpr int V_FULL = K_FREE + 8 * NK;
  static constexpr int V_FREE = V_FULL + 8 * NV;
  static constexpr int S1_DONE = V_FREE + 8 * NV;       // pass 1: scores are there
  static constexpr int S2_DONE = S1_DONE + 8 * NB1;     // pass 2
  static constexpr int PV_DONE = S2_DONE + 8 * NB;
  static constexpr int V_CLEAR = PV_DONE + 8 * NB;      // the last stage's rows
  static constexpr int DRAIN = V_CLEAR + 8;             // of the scores' thread, of the products'
  static constexpr int S1_READ = DRAIN + 16;            // by the row warps: pass 1's scores were read
  static constexpr int P_READY = S1_READ + 8 * NB1;     // by the row warps of the buffer
  static constexpr int Q_READY = P_READY + 8 * NB;      // by the row warps
  static constexpr int TMEM_SLOT = Q_READY + 8;
  static constexpr int FLAG = TMEM_SLOT + 8;            // this CTA gave up
  static constexpr int MISSING = FLAG + 4;              // a page of the span does not exist
  static constexpr int MOVED = MISSING + 4;             // score products issued so far
  static constexpr int BYTES = MOVED + 4 + 1024;
  // once every product of the CTA is done, output rows where q was ([row warp][32
  // rows][D / 2 dims]), and where keys were
  static constexpr int SQ = K;                          // [quarter of the columns][row] sums of squares
  static constexpr int WN = SQ + 4 * kRows * 4;         // [2D] weights of the norm
  static_assert(kRowWarps * 32 * D <= 2 * QMAP, "output rows take q's place");
};
static_assert(DPLayout<128>::BYTES <= kMaxCtaSmem, "stages do not fit in shared memory");
static_assert(DPLayout<64>::BYTES <= kMaxCtaSmem, "stages do not fit in shared memory");

__device__ __forceinline__ void row_warps_barrier() {
  __syncwarp();
  asm volatile("bar.sync 1, %0;" ::"n"(kRowWarps * 32) : "memory");
}

// Two fp32 values in a register pair.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pack(float a, float b) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack(Pair v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair exp2_of(Pair v) {
  const float2 x = unpack(v);
  return pack(ex2(x.x), ex2(x.y));
}

// Loads from tensor memory that are on their way while something else runs: what
// they return may be used behind land(), which waits for all of them.
__device__ __forceinline__ void ld16_late(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void land(float (&a)[16], float (&b)[16]) {
  tc5::wait_ld();
  // the values come into being here, as far as the compiler may order their uses
  asm volatile("" : "+f"(a[0]), "+f"(a[1]), "+f"(a[2]), "+f"(a[3]), "+f"(a[4]), "+f"(a[5]), "+f"(a[6]), "+f"(a[7]),
               "+f"(a[8]), "+f"(a[9]), "+f"(a[10]), "+f"(a[11]), "+f"(a[12]), "+f"(a[13]), "+f"(a[14]), "+f"(a[15]));
  asm volatile("" : "+f"(b[0]), "+f"(b[1]), "+f"(b[2]), "+f"(b[3]), "+f"(b[4]), "+f"(b[5]), "+f"(b[6]), "+f"(b[7]),
               "+f"(b[8]), "+f"(b[9]), "+f"(b[10]), "+f"(b[11]), "+f"(b[12]), "+f"(b[13]), "+f"(b[14]), "+f"(b[15]));
}

__device__ __forceinline__ void st8u(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Two columns of this thread's TMEM lane written, four read.
__device__ __forceinline__ void st2(uint32_t taddr, float a, float b) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(taddr),
               "r"(__float_as_uint(a)), "r"(__float_as_uint(b))
               : "memory");
}
__device__ __forceinline__ float4 ld4(uint32_t taddr) {
  uint32_t r[4];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr));
  return make_float4(__uint_as_float(r[0]), __uint_as_float(r[1]), __uint_as_float(r[2]),
                     __uint_as_float(r[3]));
}

template <typename T, int D, int G>
__global__ void __launch_bounds__(kDiffPrefillThreads, 1)
    diff_prefill_kernel(const __grid_constant__ DiffPrefillParams p) {
  using L = DPLayout<D>;
  extern __shared__ unsigned char smem_dyn[];
  unsigned char* base = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(base);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* flag = reinterpret_cast<int*>(base + L::FLAG);
  volatile int* missing = reinterpret_cast<int*>(base + L::MISSING);
  volatile int* moved = reinterpret_cast<int*>(base + L::MOVED);

  // The plan is written by the upload alone, which the programmatic launch
  // does not overlap: it may be read before the wait for the kernel ahead.
  const int4 hdr = *reinterpret_cast<const int4*>(p.ws);
  const int4 tile = reinterpret_cast<const int4*>(p.ws + 16)[2 * blockIdx.x];
  const int4 twin = reinterpret_cast<const int4*>(p.ws + 16)[2 * blockIdx.x + 1];
  if (threadIdx.x == 0) {
    *flag = 0;
    *missing = 0;
    *moved = 0;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tmap_k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tmap_v)) : "memory");
    for (int b = L::K_FULL; b < L::S1_READ; b += 8) mbar_init(sb + b, 1);
    for (int b = L::S1_READ; b < L::TMEM_SLOT; b += 8)
      mbar_init(sb + b, b >= L::Q_READY ? kRowWarps : kRowWarps / (b >= L::P_READY ? L::TURNS : L::TURNS1));
    fence_barrier_init();
  }
  if (warp == kRowWarps) {
    __syncwarp();
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     sb + L::TMEM_SLOT)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  const int b = tile.x, pair = tile.y >> 1, tok0 = tile.z, ntok = tile.w;
  bool bad = hdr.x != (int)kPrefillMagic || hdr.y != p.num_tiles || hdr.z != p.batch || hdr.w != p.total_q ||
             b < 0 || b >= p.batch || tile.y < 0 || (tile.y & 1) || tile.y + 1 >= p.num_kv_heads || tok0 < 0 ||
             ntok < 1 || ntok > kRows / G || twin.x != b || twin.y != tile.y + 1 || twin.z != tok0 ||
             twin.w != ntok;
  int cu0 = 0, qn = 0;
  if (!bad) {
    cu0 = p.cu[b];
    const int end = p.cu[b + 1];
    qn = end - cu0;
    bad = cu0 < 0 || end > p.total_q || qn < tok0 + ntok;
  }
  pdl_launch_dependents();
  pdl_wait_primary();

  // What needs no length is on its way while the length is read.
  constexpr int KT = L::KT, kPages = L::PAGES;
  const int len = bad ? 0 : p.seq_lens[b];
  const int32_t* table = p.block_table + (size_t)(bad ? 0 : b) * p.max_pages;
  int first_entry = -1;  // copy warps: entry `lane` of the sequence's pages
  if (warp >= kRowWarps + 2 && !bad && lane < kPages && lane < p.max_pages) first_entry = __ldg(table + lane);
  // row warps: group; pass 1: map, and half of the columns
  const int g = warp >> 2, m = g & 1, h = g >> 1;
  const int row = 32 * (warp & 3) + lane;
  const int tt = row / G;                       // the row's query token within the tile
  const int head = pair * G + row % G;          // and its head
  // Half of the rows of q_m that the warp has, read in whole lines: 16-byte chunk
  // c % CH of row c / CH, c = lane, lane + 32, ... (Each lane reading its own row cost
  // 10,000 clocks with D = 128, in 4096 pieces of lines.  620 -> 586 us, prompt of
  // 8192 tokens, with the output's rows written so too; one of 4100, D = 64: 153 -> 149.)
  constexpr int CH = D / 16;
  uint4 w0[CH];
  float lambda = 0.f;
  if (warp < kRowWarps) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int r = 32 * (warp & 3) + (c * 32 + lane) / CH;
      const T* src = static_cast<const T*>(p.q) +
                     ((size_t)(cu0 + tok0 + r / G) * p.num_q_heads + 2 * (pair * G + r % G) + m) * D +
                     (h * CH + lane % CH) * 8;
      w0[c] = !bad && r / G < ntok ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0u, 0u, 0u, 0u);
    }
    if (!bad && tt < ntok) lambda = __ldg(p.e.lambda + head);
  }
  tc5::fence_before();
  __syncthreads();
  tc5::fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(base + L::TMEM_SLOT);

  int span = 0, pos0 = 0;
  if (!bad && len >= qn && len <= p.max_pages * kPageSize) {
    pos0 = len - qn + tok0;  // position of the first query
    span = pos0 + ntok;      // tokens that some row sees
  } else {
    if (threadIdx.x == 0)
      set_status(p.status, len > p.max_pages * kPageSize ? PA_DEV_BAD_SEQ_LEN : PA_DEV_PLAN_MISMATCH);
    bad = true;
  }
  const int n = (span + KT - 1) / KT;                   // stages (0: nothing to do)
  const int parts = (span + kTokens - 1) / kTokens;     // buffers of pass 2
  // The first value slot to be read again and the first weights come after all of pass 1,
  // which takes as long as the context is: such a wait's limit counts from the last score
  // product that was issued, so that every limit is one of a stage, in both passes.
  auto while_moving = [&](auto&& wait) {
    for (int seen = *moved; !wait();) {
      const int now = *moved;
      if (now == seen) return false;
      seen = now;
    }
    return true;
  };
  const int npages = (span + kPageSize - 1) / kPageSize;

  if (warp >= kRowWarps + 2) {
    // ================= copies =================
    const bool keys = warp == kRowWarps + 2;
    const int valid = span - (n - 1) * KT;  // rows of the last stage that some row sees
    int nxt[kPages];  // block-table entries of the next stage, loaded a stage ahead of their use
#pragma unroll
    for (int u = 0; u < kPages; ++u) {
      const int entry = __shfl_sync(kFull, first_entry, u);
      nxt[u] = u < npages ? entry : -1;
    }
    // The elected lane's code has to be short: a copy that the compiler does not
    // know to be one thread's, or that waits for its own branch, takes it 100 clocks.
    if (n > 0 && tc5::elect_one()) {
      const uint64_t keep = tc5::l2_evict_normal_policy();
      auto load_entries = [&](int i) {
        const int32_t* entry = table + i * kPages;
        const int there = npages - i * kPages;
#pragma unroll
        for (int u = 0; u < kPages; ++u) {
          nxt[u] = -1;
          if (u < there) asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(nxt[u]) : "l"(entry + u));
        }
      };
      // the entries of the next stage, and whether all its pages exist
      auto take_entries = [&](int (&phys)[kPages], int& there) {
        there = 0;
#pragma unroll
        for (int u = 0; u < kPages; ++u) {
          phys[u] = (unsigned)nxt[u] < (unsigned)p.num_pages ? nxt[u] : -1;
          there += phys[u] >= 0;
        }
        return there == kPages;
      };
      auto page_of = [&](const int (&phys)[kPages], int u) {
        int page = -1;
#pragma unroll
        for (int v = 0; v < kPages; ++v) page = u == v ? phys[v] : page;
        return page;
      };
      bool good = true;
      int slot = 0, issued = 0;
      uint32_t phase = 1;  // of the slot's last use
      if (keys) {
        const int total = 2 * n;  // the keys pass twice
        for (int i = 0; issued < total; ++issued) {
          int phys[kPages], there;
          const bool all = take_entries(phys, there);
          if (!all && there < min(kPages, npages - i * kPages)) set_status(p.status, PA_DEV_BAD_PAGE);
          i = i + 1 < n ? i + 1 : 0;
          load_entries(i);
          if (issued >= L::NK) {
            good = mbar_wait_bounded_sleep(sb + L::K_FREE + 8 * slot, phase, p.wait_ns);
            if (!good) break;
          }
          const uint32_t bar = sb + L::K_FULL + 8 * slot;
          const uint32_t dst = sb + L::K + slot * L::KSTAGE;
          if (all) {
            mbar_arrive_expect_tx(bar, (uint32_t)L::KSTAGE);
#pragma unroll
            for (int x = 0; x < 2 * L::KB; ++x)  // map x / KB, box x % KB
#pragma unroll
              for (int u = 0; u < kPages; ++u)
                tma_load_4d(dst + x * L::KBOX + u * kPageSize * 128, &p.tmap_k, x % L::KB * 64, 0,
                            2 * pair + x / L::KB, phys[u], bar, keep);
          } else {
            if (there > 0)
              mbar_arrive_expect_tx(bar, (uint32_t)(there * 2 * kPageSize * D * 2));
            else
              mbar_arrive(bar);
#pragma unroll 1
            for (int u = 0; u < kPages; ++u) {
              const int page = page_of(phys, u);
              if (page < 0) continue;
              for (int x = 0; x < 2 * L::KB; ++x)
                tma_load_4d(dst + x * L::KBOX + u * kPageSize * 128, &p.tmap_k, x % L::KB * 64, 0,
                            2 * pair + x / L::KB, page, bar, keep);
            }
          }
          if (++slot == L::NK) slot = 0, phase ^= 1;
        }
      } else {
        for (; issued < n; ++issued) {
          int phys[kPages], there;
          const bool all = take_entries(phys, there);
          if (issued + 1 < n) load_entries(issued + 1);
          if (issued >= L::NV) {
            good = while_moving([&]() { return mbar_wait_bounded_sleep(sb + L::V_FREE + 8 * slot, phase, p.wait_ns); });
            if (!good) break;
          }
          const uint32_t bar = sb + L::V_FULL + 8 * slot;
          const uint32_t dst = sb + L::V + slot * L::VSTAGE;
          if (all) {
            mbar_arrive_expect_tx(bar, (uint32_t)L::VSTAGE);
#pragma unroll
            for (int u = 0; u < kPages; ++u)
#pragma unroll
              for (int x = 0; x < L::KB; ++x)  // 64 dims of both heads
                tma_load_4d(dst + u * L::VPAGE + x * 2 * kPageSize * 128, &p.tmap_v, x * 64, 0, 2 * pair, phys[u],
                            bar, keep);
          } else {
            // a page that does not exist becomes zeros; pages past the span are cleared
            // with the last stage's other rows
#pragma unroll 1
            for (int u = 0; u < kPages && issued * kPages + u < npages; ++u) {
              if (page_of(phys, u) >= 0) continue;
              for (int at = 0; at < L::VPAGE; at += 16)
                *reinterpret_cast<uint4*>(base + L::V + slot * L::VSTAGE + u * L::VPAGE + at) =
                    make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();  // the tensor core reads them (async proxy)
            if (there > 0)
              mbar_arrive_expect_tx(bar, (uint32_t)(there * L::VPAGE));
            else
              mbar_arrive(bar);
#pragma unroll 1
            for (int u = 0; u < kPages; ++u) {
              const int page = page_of(phys, u);
              if (page < 0) continue;
              for (int x = 0; x < L::KB; ++x)
                tma_load_4d(dst + u * L::VPAGE + x * 2 * kPageSize * 128, &p.tmap_v, x * 64, 0, 2 * pair, page, bar,
                            keep);
            }
          }
          if (++slot == L::NV) slot = 0, phase ^= 1;
        }
        // rows to clear: the last stage's copies land before the zeros are written
        if (good && valid < KT)
          good = mbar_wait_bounded_sleep(sb + L::V_FULL + 8 * ((n - 1) % L::NV), (uint32_t)(((n - 1) / L::NV) & 1),
                                         p.wait_ns);
      }
      if (!good) {
        set_status(p.status, PA_DEV_TIMEOUT);
        *flag = 1;
      }
      // copies in flight land before the CTA exits: the last stage issued into each
      // slot (the one before it in the slot was read)
      const int ring = keys ? L::NK : L::NV;
      for (int c = max(0, issued - ring); c < issued; ++c)
        mbar_wait_bounded_sleep(sb + (keys ? L::K_FULL : L::V_FULL) + 8 * (c % ring), (uint32_t)((c / ring) & 1),
                                kDrainWaitNs);
    }
    __syncwarp();
    // Rows of the last stage that no row of the tile sees become zeros (the
    // copies have landed, and no product reads them before).  A CTA that gave up
    // leaves them and V_CLEAR alone: the product is not formed.
    // (One vote decides for the warp: another warp may set the flag while it is read.)
    if (!keys && n > 0 && valid < KT && __all_sync(kFull, *flag == 0)) {
      unsigned char* stage = base + L::V + (n - 1) % L::NV * L::VSTAGE;
      const int rows = KT - valid;
      for (int i = lane; i < rows * 2 * L::KB * 8; i += 32) {
        const int r = valid + i / (2 * L::KB * 8), at = i % (2 * L::KB * 8);
        *reinterpret_cast<uint4*>(stage + r / kPageSize * L::VPAGE + at / 8 * (kPageSize * 128) +
                                  r % kPageSize * 128 + at % 8 * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();  // the tensor core reads them (async proxy)
      __syncwarp();
      if (lane == 0) mbar_arrive(sb + L::V_CLEAR);
    }
  } else if (warp >= kRowWarps) {
    // ================= MMAs: one thread for the scores, one for the products ===========
    // (A stage's waits and loop take a thread 100 to 200 clocks each, with their
    // barriers long complete: one thread for both was behind its tensor core.)
    if (n > 0 && tc5::elect_one()) {
      const uint64_t q_desc = tc5::smem_desc(sb + L::Q, 16, 1024), k_desc = tc5::smem_desc(sb + L::K, 16, 1024);
      const uint64_t v_desc = tc5::smem_desc(sb + L::V, kPageSize * 128, 1024);
      auto wait = [&](int bar, uint32_t parity) {
        return mbar_test_wait(sb + bar, parity) || mbar_wait_bounded(sb + bar, parity, p.wait_ns);
      };
      bool good = true;
      if (warp == kRowWarps) {
        const uint32_t idesc1 = tc5::instr_desc<T>(kRows, KT, false);
        const uint32_t idesc2 = tc5::instr_desc<T>(kRows, kTokens, false);
        int ks = 0;
        uint32_t kphase = 0;
        // scores of map m and the tokens from `part` on of the key slot
        auto scores = [&](int m, uint32_t idesc, uint32_t column, int part) {
          const uint64_t qb = tc5::desc_at(q_desc, m * L::QMAP);
          const uint64_t kb = tc5::desc_at(k_desc, ks * L::KSTAGE + m * L::KB * L::KBOX + part * kTokens * 128);
#pragma unroll
          for (int x = 0; x < L::KB; ++x)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc5::mma1(tmem + column, tc5::desc_at(qb, x * L::QBOX + k * 32),
                        tc5::desc_at(kb, x * L::KBOX + k * 32), idesc, x > 0 || k > 0 ? 1u : 0u);
        };
        auto read_keys = [&]() {  // the key slot's last scores are on their way
          tc5::commit(sb + L::K_FREE + 8 * ks);
          if (++ks == L::NK) ks = 0, kphase ^= 1;
        };
        good = wait(L::Q_READY, 0u);
        tc5::fence_after();
        for (int i = 0; i < n && good; ++i) {  // pass 1
          const int at = i % L::NB1;
          good = (i < L::NB1 || wait(L::S1_READ + 8 * at, (uint32_t)((i / L::NB1 - 1) & 1))) &&
                 wait(L::K_FULL + 8 * ks, kphase);
          if (!good) break;
          tc5::fence_after();
          if constexpr (L::QT) {
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              const uint64_t kb = tc5::desc_at(k_desc, ks * L::KSTAGE + m * L::KB * L::KBOX);
#pragma unroll
              for (int x = 0; x < L::KB; ++x)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  tc5::mma1_tmem(tmem + at * 2 * KT + m * KT, tmem + L::QCOL + m * (D / 2) + x * 32 + k * 8,
                                 tc5::desc_at(kb, x * L::KBOX + k * 32), idesc1, x > 0 || k > 0 ? 1u : 0u);
            }
          } else {
            scores(0, idesc1, at * 2 * KT, 0);
            scores(1, idesc1, at * 2 * KT + KT, 0);
          }
          tc5::commit(sb + L::S1_DONE + 8 * at);
          *moved = i + 1;
          read_keys();
        }
        int at = 0, part = 0;
        uint32_t phase = 1;  // of the buffer's last use
        for (int i = 0; i < parts && good; ++i) {  // pass 2
          // the second map's scores overwrite what was read before P was written, the
          // first map's overwrite P; the first ones those of pass 1.  (With three
          // buffers the product is long done, and one wait less is shorter.)
          if (i < L::NB) {
            const int b1 = i * 128 / (2 * KT), uses = (n - b1 + L::NB1 - 1) / L::NB1;
            good = uses < 1 || wait(L::S1_READ + 8 * b1, (uint32_t)((uses - 1) & 1));
          } else {
            good = wait((L::NB > 2 ? L::PV_DONE : L::P_READY) + 8 * at, phase);
          }
          good = good && (part > 0 || wait(L::K_FULL + 8 * ks, kphase));
          if (!good) break;
          tc5::fence_after();
          scores(1, idesc2, at * 128 + kTokens, part);
          if (i >= L::NB && L::NB == 2) {
            good = wait(L::PV_DONE + 8 * at, phase);
            if (!good) break;
            tc5::fence_after();
          }
          scores(0, idesc2, at * 128, part);
          tc5::commit(sb + L::S2_DONE + 8 * at);
          *moved = n + i + 1;
          if (++part == L::PARTS || i == parts - 1) {
            part = 0;
            read_keys();
          }
          if (++at == L::NB) at = 0, phase ^= 1;
        }
      } else {
        const uint32_t idesc = tc5::instr_desc<T>(kRows, 2 * D, true);
        int at = 0, vs = 0, part = 0;
        uint32_t phase = 0, vphase = 0;
        // where a warp of MINE columns puts the (high parts of the) weights of tokens 16 k ..
        auto column_of = [](int k) { return (uint32_t)(16 * k / L::MINE * L::MINE + 16 * k % L::MINE / 2); };
        for (int i = 0; i < parts && good; ++i) {
          if (part == 0)
            good = wait(L::V_FULL + 8 * vs, vphase) &&
                   (i + L::PARTS < parts || span % KT == 0 || wait(L::V_CLEAR, 0u));  // rows to clear: once they are
          good = good && while_moving([&]() { return wait(L::P_READY + 8 * at, phase); });
          if (!good) break;
          tc5::fence_after();
          const uint64_t vb = tc5::desc_at(v_desc, vs * L::VSTAGE + part * (kTokens / kPageSize) * L::VPAGE);
          const uint32_t t_p = tmem + (uint32_t)at * 128;
#pragma unroll
          for (int k = 0; k < kTokens / kPageSize; ++k)
            tc5::mma1_tmem(tmem + L::O, t_p + column_of(k), tc5::desc_at(vb, k * L::VPAGE), idesc,
                           i > 0 || k > 0 ? 1u : 0u);
#pragma unroll
          for (int k = 0; k < kTokens / kPageSize; ++k)  // the second parts
            tc5::mma1_tmem(tmem + L::O, t_p + column_of(k) + L::MINE / 2, tc5::desc_at(vb, k * L::VPAGE), idesc, 1u);
          tc5::commit(sb + L::PV_DONE + 8 * at);
          if (++part == L::PARTS) {
            part = 0;
            tc5::commit(sb + L::V_FREE + 8 * vs);
            if (++vs == L::NV) vs = 0, vphase ^= 1;
          }
          if (++at == L::NB) at = 0, phase ^= 1;
        }
      }
      if (!good) {
        set_status(p.status, PA_DEV_TIMEOUT);
        *flag = 1;
      }
      // every MMA that this thread issued finishes before TMEM is freed
      tc5::commit(sb + L::DRAIN + 8 * (warp - kRowWarps));
      mbar_wait_bounded_sleep(sb + L::DRAIN + 8 * (warp - kRowWarps), 0u, kDrainWaitNs);
    }
    __syncwarp();
  } else {
    // ================= softmax and output =================
    const bool ok = !bad && tt < ntok;
    // last visible token; rows that are not there see all of zero queries' scores
    const int qpos = ok ? pos0 + tt : span - 1;
    const uint32_t t_row = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    // log2 of a factor of the weights, which are at most 2 in size without it.  fp16's
    // smallest step is 2^-24: beside a token that takes nearly all of both maps, the others'
    // weights keep the two parts' bits down to 2^-17 of it, and 2^-39 of it at least.
    constexpr float kBias = std::is_same<T, __half>::value ? 14.f : 0.f;

    // q into shared memory (zeros where there is none): K-major, 16-byte chunk c of a
    // row's 128-byte box at chunk c ^ (row % 8).
    {
      auto place = [&](int r, int c) {  // chunk c of the warp's half of row r
        const int chunk = h * CH + c;
        return reinterpret_cast<uint4*>(base + L::Q + m * L::QMAP + (chunk >> 3) * L::QBOX + r * 128 +
                                        (((chunk & 7) ^ (r & 7)) << 4));
      };
#pragma unroll
      for (int c = 0; c < CH; ++c) *place(32 * (warp & 3) + (c * 32 + lane) / CH, lane % CH) = w0[c];
      fence_proxy_async_smem();  // the tensor core reads it (async proxy)
      __syncwarp();
      if constexpr (L::QT) {  // and into tensor memory, for pass 1
        uint4 w[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) w[c] = *place(row, c);
        __syncwarp();
        const uint32_t column = t_row + (uint32_t)(L::QCOL + m * (D / 2) + h * (D / 4));
        tc5::st16u(column, reinterpret_cast<const uint32_t*>(w));
        tc5::st16u(column + 16, reinterpret_cast<const uint32_t*>(w) + 16);
        tc5::wait_st();
        tc5::fence_before();
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(sb + L::Q_READY);
    }
    // Pages of the span that do not exist: looked for once, and masked only then.
    for (int i = threadIdx.x; i < npages; i += kRowWarps * 32) {
      const int entry = __ldg(table + i);
      if (entry < 0 || entry >= p.num_pages) *missing = 1;
    }
    row_warps_barrier();
    const bool holes = __any_sync(kFull, *missing != 0);
    auto page_there = [&](int token) {
      const int i = token / kPageSize;
      const int entry = i < npages ? __ldg(table + i) : -1;
      return entry >= 0 && entry < p.num_pages;
    };
    const bool idle = __all_sync(kFull, !ok);  // no row of the warp: its weights feed rows that are not written
    float qscale = p.qscale;
    const Pair qs2 = pack(qscale, qscale);
    // stages, and buffers of pass 2, that every row of the tile sees whole: no masks
    const int whole1 = holes ? 0 : min(n, (pos0 + 1) / KT), whole = holes ? 0 : min(parts, (pos0 + 1) / kTokens);
    bool good = true;
    auto wait_all = [&](uint32_t bar, uint32_t parity) {
      return __all_sync(kFull, mbar_wait_bounded_sleep(bar, parity, p.wait_ns)) != 0;
    };
    auto minus = [](float ref) { return ref == -INFINITY ? -INFINITY : -ref; };  // no token yet: weights 0

    // ---- pass 1: a reference point of the row's scores of map m in half of the
    // columns, and their sum relative to it.  The reference is a maximum, but an
    // old one will do while the sum shows that no score is far above it (kLateSum).
    constexpr int MINE = KT / 2 * L::TURNS1;  // columns of a stage
    const int col1 = L::TURNS1 == 2 ? 0 : h * MINE;
    float m_run = -INFINITY, l_run = 0.f;
    bool beyond = false;   // some row of the warp has scores beyond the fused product's range
    bool settled = false;  // every row of the warp has a reference, none is beyond
    // the weights of 16 columns relative to a reference, added to four running sums
    auto accumulate = [&](Pair (&sum)[4], const float (&a)[16], Pair minus_ref) {
#pragma unroll
      for (int c = 0; c < 16; c += 2)
        sum[(c >> 1) & 3] = add2(sum[(c >> 1) & 3], exp2_of(fma2(pack(a[c], a[c + 1]), qs2, minus_ref)));
    };
    auto total_of = [&](const Pair (&sum)[4]) {
      const float2 s2 = unpack(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
      return s2.x + s2.y;
    };
    auto raise = [&](float (&a)[16], float (&b)[16]) {  // with the reference raised to the columns' maximum
      float top4[4] = {a[0], a[1], a[2], a[3]};
#pragma unroll
      for (int c = 4; c < 16; ++c) top4[c & 3] = fmaxf(top4[c & 3], a[c]);
#pragma unroll
      for (int c = 0; c < 16; ++c) top4[c & 3] = fmaxf(top4[c & 3], b[c]);
      const float mx = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3])) * qscale;
      const float top = fmaxf(m_run, mx);
      if (m_run != -INFINITY) l_run *= ex2(m_run - top);
      m_run = top;
      beyond = beyond_fused(m_run);
      settled = !beyond && __all_sync(kFull, m_run != -INFINITY);
      if (beyond) {
        rounded_differences(a, qscale, m_run);
        rounded_differences(b, qscale, m_run);
#pragma unroll
        for (int c = 0; c < 16; ++c) l_run += ex2(a[c]) + ex2(b[c]);
      } else {
        Pair sum[4] = {0, 0, 0, 0};  // zeros
        const float nm = minus(m_run);
        accumulate(sum, a, pack(nm, nm));
        accumulate(sum, b, pack(nm, nm));
        l_run += total_of(sum);
      }
    };
    uint32_t phase = 0;
    int at = L::TURNS1 == 2 ? h : 0;
    for (int i = at; i < n; i += L::TURNS1) {
      good = wait_all(sb + L::S1_DONE + 8 * at, phase);
      if (!good) break;
      if (!idle) {
        tc5::fence_after();
        const uint32_t columns = t_row + (uint32_t)(at * 2 * KT + m * KT + col1);
        float a[16], b[16];
        bool stays = false;
        if (i < whole1 && settled) {
          const float nm = minus(m_run);
          const Pair nm2 = pack(nm, nm);
          Pair sum[4] = {0, 0, 0, 0};
#pragma unroll
          for (int c = 0; c < MINE; c += 32) {
            __syncwarp();
            ld16_late(columns + (uint32_t)c, a);
            ld16_late(columns + (uint32_t)(c + 16), b);
            land(a, b);
            accumulate(sum, a, nm2);
            accumulate(sum, b, nm2);
          }
          const float sum_all = total_of(sum);
          stays = __all_sync(kFull, sum_all <= kLateSum) != 0;
          if (stays) l_run += sum_all;
        }
        if (!stays) {
          const int first = i * KT + col1, lim = qpos - first;  // last visible column
#pragma unroll 1
          for (int c = 0; c < MINE; c += 32) {
            if (!__any_sync(kFull, ok && lim >= c)) break;  // no row sees these or later ones
            __syncwarp();
            ld16_late(columns + (uint32_t)c, a);
            ld16_late(columns + (uint32_t)(c + 16), b);
            land(a, b);
            if (holes || !__all_sync(kFull, lim >= c + 31)) {
              const bool there_a = !holes || page_there(first + c), there_b = !holes || page_there(first + c + 16);
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                a[k] = there_a && c + k <= lim ? a[k] : -INFINITY;
                b[k] = there_b && c + 16 + k <= lim ? b[k] : -INFINITY;
              }
            }
            if (settled) {
              const float nm = minus(m_run);
              Pair sum[4] = {0, 0, 0, 0};
              accumulate(sum, a, pack(nm, nm));
              accumulate(sum, b, pack(nm, nm));
              const float sum_all = total_of(sum);
              if (__all_sync(kFull, sum_all <= kLateSum)) {
                l_run += sum_all;
                continue;
              }
            }
            raise(a, b);
          }
        }
        tc5::fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(sb + L::S1_READ + 8 * at);
      at += L::TURNS1;
      if (at >= L::NB1) at -= L::NB1, phase ^= 1;
    }
    if (!good && lane == 0) {
      set_status(p.status, PA_DEV_TIMEOUT);
      *flag = 1;
    }
    // The four warps of a row exchange what they found through the columns that O
    // will take, once all have read pass 1's scores from them.
    row_warps_barrier();
    tc5::fence_after();
    st2(t_row + (uint32_t)(L::O + 2 * g), m_run, l_run);
    tc5::wait_st();
    tc5::fence_before();
    row_warps_barrier();
    tc5::fence_after();
    const float4 low = ld4(t_row + (uint32_t)L::O), high = ld4(t_row + (uint32_t)(L::O + 4));
    tc5::wait_ld();
    tc5::fence_before();
    row_warps_barrier();  // the first product, which writes O, waits for some of the warps only
    auto joined = [&](float ma, float la, float mb, float lb) {  // {reference, sum} of both halves
      const float ref = fmaxf(ma, mb);
      if (ref == -INFINITY) return make_float2(ref, la + lb);  // 0, or NaN
      return make_float2(ref, la * ex2(ma - ref) + lb * ex2(mb - ref));
    };
    const float2 st1 = joined(low.x, low.y, high.x, high.y), st2v = joined(low.z, low.w, high.z, high.w);

    // ---- pass 2: weights f (2^(s_1 - m_1) / l_1 - lambda 2^(s_2 - m_2) / l_2), f = 1 / max(1, |lambda|)
    // (The other quotients within 2 units in the last place: 8.7 -> 8.4 us, 3 prompts of up to 130 tokens.)
    const float c1 = st1.y > 0.f || st1.y != st1.y ? __fdividef(1.f, st1.y) : 0.f;
    const float c2 = st2v.y > 0.f || st2v.y != st2v.y ? __fdividef(fabsf(lambda), st2v.y) : 0.f;
    const float most = fmaxf(1.f, fabsf(lambda)), f = 1.f / most;
    const float sgn = lambda < 0.f ? 1.f : -1.f;
    const bool far = __any_sync(kFull, (fabsf(st1.x) > kFoldedLog2 && st1.x != -INFINITY) ||
                                           (fabsf(st2v.x) > kFoldedLog2 && st2v.x != -INFINITY)) != 0;
    const float nc1 = st1.x == -INFINITY ? -INFINITY : kBias + lg2(c1 * f) - st1.x;
    const float nc2 = st2v.x == -INFINITY ? -INFINITY : kBias + lg2(c2 * f) - st2v.x;
    const Pair n1 = pack(nc1, nc1), n2 = pack(nc2, nc2), sg = pack(sgn, sgn), minus1 = pack(-1.f, -1.f);
    at = L::TURNS == 2 ? h : 0;
    phase = 0;
    const int mine = L::MINE * (L::TURNS == 2 ? m : g);  // the warp's first column
    for (int i = at; i < parts && good; i += L::TURNS) {
      good = wait_all(sb + L::S2_DONE + 8 * at, phase);
      if (!good) break;
      if (!idle) {
        tc5::fence_after();
        const uint32_t columns = t_row + (uint32_t)(at * 128 + mine);  // of map 1
        float s1[16], s2[16];
        Pair d[8];
        uint32_t w[8];
        auto load = [&](int c) {
          __syncwarp();
          ld16_late(columns + (uint32_t)c, s1);
          ld16_late(columns + (uint32_t)(c + kTokens), s2);
        };
        auto weights = [&](int c) {
          if (i >= whole) {
            const int first = i * kTokens + mine + c, lim = qpos - first;  // last visible column of the 16
            const bool there = !holes || page_there(first);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const bool seen = there && k <= lim;
              s1[k] = seen ? s1[k] : -INFINITY;
              s2[k] = seen ? s2[k] : -INFINITY;
            }
          }
          if (!far) {
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              const Pair x = exp2_of(fma2(pack(s1[k], s1[k + 1]), qs2, n1));
              const Pair y = exp2_of(fma2(pack(s2[k], s2[k + 1]), qs2, n2));
              d[k >> 1] = fma2(y, sg, x);
            }
          } else {
            const bool beyond1 = beyond_fused(st1.x), beyond2 = beyond_fused(st2v.x);
            if (beyond1) rounded_differences(s1, qscale, st1.x);
            if (beyond2) rounded_differences(s2, qscale, st2v.x);
            const float r1 = minus(st1.x), r2 = minus(st2v.x), up = exp2f(kBias);
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              float e[2];
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const float x = beyond1 ? s1[k + u] : fmaf(s1[k + u], qscale, r1);
                const float y = beyond2 ? s2[k + u] : fmaf(s2[k + u], qscale, r2);
                e[u] = fmaf(sgn * c2 * f * up, ex2(y), c1 * f * up * ex2(x));
              }
              d[k >> 1] = pack(e[0], e[1]);
            }
          }
        };
        // the weights of 16 columns over the scores of the warp's own, which were all read
        auto put = [&](int half) {
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float2 df = unpack(d[c]);
            w[c] = Elem<T>::from_f2(df.x, df.y);
          }
          __syncwarp();  // lanes may have branched, and what follows is for a whole warp
          st8u(columns + (uint32_t)(8 * half), w);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float2 hi = Elem<T>::to_f2(w[c]);
            const float2 rest = unpack(fma2(pack(hi.x, hi.y), minus1, d[c]));  // exact
            w[c] = Elem<T>::from_f2(rest.x, rest.y);
          }
          __syncwarp();
          st8u(columns + (uint32_t)(L::MINE / 2 + 8 * half), w);
        };
        load(0);
        __syncwarp();
        land(s1, s2);
        weights(0);
        if (L::TURNS == 2) {
          load(16);
          __syncwarp();
          land(s1, s2);
          put(0);
          weights(16);
          put(1);
        } else {
          put(0);
        }
        __syncwarp();
        tc5::wait_st();
        tc5::fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(sb + L::P_READY + 8 * at);
      at += L::TURNS;
      if (at >= L::NB) at -= L::NB, phase ^= 1;
    }

    // ---- output: the four warps of a row take a quarter of the columns each
    // (A parity tells the last product only from the one before it in its buffer: that
    // one is done once some warp has seen the last scores, so all meet here first.)
    float norm_weight = 1.f;
    if (threadIdx.x < 2 * D && p.e.weight != nullptr) norm_weight = __ldg(p.e.weight + threadIdx.x);
    row_warps_barrier();
    if (n > 0 && good)
      good = wait_all(sb + L::PV_DONE + 8 * ((parts - 1) % L::NB), (uint32_t)(((parts - 1) / L::NB) & 1));
    if (!good && lane == 0) {
      set_status(p.status, PA_DEV_TIMEOUT);
      *flag = 1;
    }
    tc5::fence_after();
    const float inv = exp2f(-kBias) * most;
    const uint32_t t_o = t_row + (uint32_t)(L::O + D / 2 * g);
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < D / 2; c += 32) {
      float a[16], b[16];
      __syncwarp();
      ld16_late(t_o + (uint32_t)c, a);
      ld16_late(t_o + (uint32_t)(c + 16), b);
      land(a, b);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        sum = fmaf(a[i] * inv, a[i] * inv, sum);
        sum = fmaf(b[i] * inv, b[i] * inv, sum);
      }
    }
    float* sq = reinterpret_cast<float*>(base + L::SQ);
    sq[g * kRows + row] = sum;
    float* wn = reinterpret_cast<float*>(base + L::WN);
    if (threadIdx.x < 2 * D) wn[threadIdx.x] = norm_weight;
    row_warps_barrier();
    float gain = p.e.factor * inv;
    if (p.e.eps > 0.f)
      gain *= rsqrtf(((sq[row] + sq[kRows + row]) + (sq[2 * kRows + row] + sq[3 * kRows + row])) * (1.f / (2 * D)) +
                     p.e.eps);
    const bool write = __all_sync(kFull, n > 0 && *flag == 0);
    // Column 64 k + j of O holds dim j of box k / 2 of head k % 2: a warp's D / 2 columns
    // are neighbours, from dim d0 on.  Through shared memory, for whole lines: rows of CH
    // chunks, chunk c of a row at another place of its 128 bytes than those of the seven
    // rows around it.
    const int col = D / 2 * g, d0 = (col / 64 % 2) * D + col / 128 * 64 + col % 64;
    unsigned char* stage = base + L::Q + warp * (32 * D);
    auto spot = [&](int r, int c) {
      const int at = D == 128 ? c ^ (r & 7) : (c ^ ((r >> 1) & 3));
      return reinterpret_cast<uint4*>(stage + r * D + at * 16);
    };
#pragma unroll
    for (int c = 0; c < D / 2; c += 16) {
      float o[16];
      __syncwarp();
      tc5::ld16(t_o + (uint32_t)c, o);
      tc5::wait_ld();
#pragma unroll
      for (int i = 0; i < 16; i += 8) {
        const float4 wa = *reinterpret_cast<const float4*>(wn + d0 + c + i);
        const float4 wb = *reinterpret_cast<const float4*>(wn + d0 + c + i + 4);
        uint4 v;
        v.x = Elem<T>::from_f2(o[i] * gain * wa.x, o[i + 1] * gain * wa.y);
        v.y = Elem<T>::from_f2(o[i + 2] * gain * wa.z, o[i + 3] * gain * wa.w);
        v.z = Elem<T>::from_f2(o[i + 4] * gain * wb.x, o[i + 5] * gain * wb.y);
        v.w = Elem<T>::from_f2(o[i + 6] * gain * wb.z, o[i + 7] * gain * wb.w);
        *spot(lane, (c + i) / 8) = v;
      }
    }
    __syncwarp();
    if (write && !bad) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int r = (c * 32 + lane) / CH, rt = (32 * (warp & 3) + r) / G, rh = (32 * (warp & 3) + r) % G;
        if (rt < ntok)
          *reinterpret_cast<uint4*>(static_cast<T*>(p.out) +
                                    ((size_t)(cu0 + tok0 + rt) * (p.num_q_heads / 2) + pair * G + rh) * (2 * D) + d0 +
                                    lane % CH * 8) = *spot(r, lane % CH);
      }
    }
  }

  tc5::fence_before();
  __syncthreads();
  if (warp == kRowWarps) {
    tc5::fence_after();
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

template <typename T, int D, int G>
cudaError_t launch_t(const DiffPrefillParams& p, cudaStream_t stream) {
  static std::atomic<unsigned long long> configured{0};
  return launch_latent(diff_prefill_kernel<T, D, G>, DPLayout<D>::BYTES, configured, p.num_tiles / 2,
                       kDiffPrefillThreads, stream, p);
}

template <typename T, int D>
cudaError_t launch_g(const DiffPrefillParams& p, int group, cudaStream_t stream) {
  switch (group) {
    case 1: return launch_t<T, D, 1>(p, stream);
    case 2: return launch_t<T, D, 2>(p, stream);
    case 4: return launch_t<T, D, 4>(p, stream);
    case 8: return launch_t<T, D, 8>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_diff_prefill(const DiffPrefillParams& p, int head_dim, int group, int dtype,
                                cudaStream_t stream) {
  const bool bf = dtype == PA_DTYPE_BF16;
  if (head_dim == 64)
    return bf ? launch_g<__nv_bfloat16, 64>(p, group, stream) : launch_g<__half, 64>(p, group, stream);
  return bf ? launch_g<__nv_bfloat16, 128>(p, group, stream) : launch_g<__half, 128>(p, group, stream);
}

}  // namespace pa
