// Differential attention of one new token of every sequence:
//
//   o_h = sum_t (P1[t] - lambda_h P2[t]) V[t],   P_m = softmax(scale q_m K_m^T),
//   out_h = factor w o_h / sqrt(mean(o_h^2) + eps),
//
// over the pages of a pair of KV heads: K_1, K_2 are the two heads' keys, a
// value is the two heads' value rows side by side (2D dims).  12 D operations
// a head and token against 8 D bytes that the G heads of a pair share: bound
// by the cache's bytes.
//
// The two maps differ only in their sums, so a task keeps one online softmax
// with 2G rows: row m G + h is map m of head h.  Every page's keys and values
// are read once for all of them, and the difference and the norm are taken
// when a row's sums are complete: by the task itself, or by the last split of
// the pair to finish.  Tasks, CTA shapes, splits and the mma.sync products
// with the weights in two parts (hi + lo) are those of decode_tc.cuh (see
// there for the fragments).  What differs:
//  - A tile is the keys (or values) of one page for both heads of the pair,
//    two neighbouring [16][D] blocks of the pool: boxes of 64 dims x 16 rows
//    x 2 heads, [D/64][2][16 rows][128 B] in shared memory.
//  - With G <= 4 the eight columns of a product hold both maps, map 0 in
//    columns 0-3 and map 1 in 4-7.  S^T of the two key tiles is formed for all
//    eight and each column takes its own map's; the values then need one
//    product for both maps.  With G = 8 each map has a column tile.
//
// Measured: 160 sequences of 128 to 2048 tokens, 32 query heads over 8 KV heads of 128
// (718 MB), 103 to 104 us, the measured copy bandwidth, with DRAM traffic within 1 % of
// the bytes; 48 of 5 to 563, 32 over 32 of 64 (111 MB), 18.9 us, 87 %; one of 32,768 (134 MB),
// 28.5 us: about 23 in this kernel (87 %), the rest in the join of 76 splits.
// Registers: 221 with head_dim 128 and G up to 4, 255 with G = 8; 128 and less with
// head_dim 64 (G = 8 spills 68 bytes).
#pragma once

#include <type_traits>

#include "decode_tc.cuh"
#include "diff.h"
#include "elem.cuh"

namespace pa {

template <int D, int NW, int NSH>
struct DiffLayout {
  static constexpr int TILE = 2 * kPageSize * D * 2;  // a multiple of 4096
  static constexpr int RING = NSH * TILE;             // per warp
  static constexpr int RINGS = NW * RING;
  static constexpr int BARS = 0;                      // NSH mbarriers
  static constexpr int PAGES = align_up(8 * NSH, 16); // NSH page ids
  static constexpr int EXTRA = align_up(PAGES + 4 * NSH, 16);
  static constexpr int FLAG = RINGS + NW * EXTRA;
  static constexpr int BYTES = FLAG + 16 + 1024;      // + slack to align the base to 1024
};

// Weights are 2^(s - m + kDiffBias), m the row's running maximum.  In fp16 both parts of
// a weight have their smallest step at 2^-24: of a largest weight of 1, one 2^-20 of it
// was off by up to 3 %, and beside a first token that takes nearly all of both maps such
// weights are what the difference is made of.  With a largest weight of 2^15 (below
// fp16's 65,504) they keep the two parts' bits down to 2^-18 of it and 2^-40 of it at least.
// The factor is in the sums as well, and leaves with them.
template <typename T>
constexpr float kDiffBias = std::is_same<T, __half>::value ? 15.f : 0.f;

// A token that is left out (s = -inf) has weight 0 under any maximum, that of no token
// (-inf) too, under which a score that is not a number stays one.
template <typename T>
__device__ __forceinline__ float diff_weight(float s, float m) {
  float x = s - m;
  if constexpr (kDiffBias<T> != 0.f) x += kDiffBias<T>;
  return s == -INFINITY ? 0.f : ex2(x);
}

// Lane's share of head dims: chunk i holds dims 128 i + 4 lane .. + 3.  The
// order of the sum of squares is the same wherever a head is finished.
template <typename T, int VD>
__device__ __forceinline__ void diff_write_head(const DiffEpilogue& e, float lambda, const float4* a,
                                                const float4* b, int lane, T* dst) {
  constexpr int N = VD / 128;
  float4 o[N];
  float sq = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    o[i].x = fmaf(-lambda, b[i].x, a[i].x);
    o[i].y = fmaf(-lambda, b[i].y, a[i].y);
    o[i].z = fmaf(-lambda, b[i].z, a[i].z);
    o[i].w = fmaf(-lambda, b[i].w, a[i].w);
    sq = fmaf(o[i].x, o[i].x, sq);
    sq = fmaf(o[i].y, o[i].y, sq);
    sq = fmaf(o[i].z, o[i].z, sq);
    sq = fmaf(o[i].w, o[i].w, sq);
  }
  float f = e.factor;
  if (e.eps > 0.f) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) sq += __shfl_xor_sync(kFull, sq, m);
    f *= rsqrtf(sq * (1.f / VD) + e.eps);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int d = 128 * i + 4 * lane;
    float4 w = make_float4(1.f, 1.f, 1.f, 1.f);
    if (e.weight != nullptr) w = __ldg(reinterpret_cast<const float4*>(e.weight + d));
    uint2 v;
    v.x = Elem<T>::from_f2(o[i].x * f * w.x, o[i].y * f * w.y);
    v.y = Elem<T>::from_f2(o[i].z * f * w.z, o[i].w * f * w.w);
    *reinterpret_cast<uint2*>(dst + d) = v;
  }
}

// What a split's row counts for beside others, relative to the reference M of them all.
// (m = -inf: no token, and l is 0, or NaN where scores were.)
__device__ __forceinline__ float diff_split_weight(float m, float l, float M) {
  return m == -INFINITY ? l : ex2(m - M) * l;
}

// Dims d0 .. d0+3 of a row over all splits of the target, in their order, NB at once.
template <int VD, int NB>
__device__ __forceinline__ float4 diff_merge_chunk(const MergeTarget& t, const float* part_sum, int row, int d0) {
  const int ns = t.grp.z;
  const size_t first = (size_t)t.grp.w * t.G + row;
  float m = -INFINITY, z = 0.f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < ns; s0 += NB) {
    float r[NB], l[NB];
    float4 x[NB];
#pragma unroll
    for (int u = 0; u < NB; ++u) {
      r[u] = -INFINITY;
      l[u] = 0.f;
      x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s0 + u < ns) {
        const size_t at = first + (size_t)(s0 + u) * t.G;
        r[u] = __ldcg(t.lse + at);
        l[u] = __ldcg(part_sum + at);
        x[u] = __ldcg(reinterpret_cast<const float4*>(t.o + at * VD + d0));
      }
    }
    float M = m;
#pragma unroll
    for (int u = 0; u < NB; ++u) M = fmaxf(M, r[u]);
    const float sc = m == -INFINITY ? 1.f : ex2(m - M);  // nothing but zeros (or NaN) so far: as it is
    z *= sc;
    a.x *= sc;
    a.y *= sc;
    a.z *= sc;
    a.w *= sc;
#pragma unroll
    for (int u = 0; u < NB; ++u) {
      const float w = diff_split_weight(r[u], l[u], M);
      z += w;
      a.x = fmaf(w, x[u].x, a.x);
      a.y = fmaf(w, x[u].y, a.y);
      a.z = fmaf(w, x[u].z, a.z);
      a.w = fmaf(w, x[u].w, a.w);
    }
    m = M;
  }
  if (z == 0.f) return make_float4(0.f, 0.f, 0.f, 0.f);
  return make_float4(a.x / z, a.y / z, a.z / z, a.w / z);
}

// The heads first, first + stride, ... of a pair whose partials are complete,
// a warp each.
template <typename T, int D, int G>
__device__ __forceinline__ void diff_merge_heads(const DiffDecodeParams& p, const MergeTarget& t, int first,
                                                 int stride, int lane) {
  constexpr int VD = 2 * D, N = VD / 128;
  for (int h = first; h < G; h += stride) {
    float4 r[2][N];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int i = 0; i < N; ++i)
        r[m][i] = t.grp.z <= kMergeBatchSmall
                      ? diff_merge_chunk<VD, kMergeBatchSmall>(t, p.part_sum, m * G + h, 128 * i + 4 * lane)
                      : diff_merge_chunk<VD, kDiffMergeSplits>(t, p.part_sum, m * G + h, 128 * i + 4 * lane);
    const size_t head = (size_t)t.grp.y * G + h;
    diff_write_head<T, VD>(p.e, __ldg(p.e.lambda + head), r[0], r[1], lane,
                           static_cast<T*>(p.s.out) +
                               ((size_t)t.grp.x * p.s.num_kv_heads * G + head) * VD);
  }
}

template <typename T, int D, int G, int NW, int NSH, int CTAS>
__global__ void __launch_bounds__(NW * 32, CTAS)
    diff_decode_kernel(const __grid_constant__ DiffDecodeParams dp) {
  static_assert(G <= 8, "the mma tile holds at most 8 query heads");
  using L = DiffLayout<D, NW, NSH>;
  constexpr int VD = 2 * D;
  constexpr int KSTEPS = D / 16;
  constexpr int VTILES = VD / 16;
  constexpr int BOXES = D / 64;
  constexpr int NT = G <= 4 ? 1 : 2;  // column tiles of the products
  constexpr int R = 2 * G;            // rows of a pair
  const SplitParams& p = dp.s;
  extern __shared__ unsigned char smem_dyn[];
  unsigned char* base = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int g = lane >> 2;
  const int t = lane & 3;
  const uint32_t ring = smem_u32(base) + warp * L::RING;
  unsigned char* extra = base + L::RINGS + warp * L::EXTRA;
  const uint32_t bars = smem_u32(extra) + L::BARS;
  int* page_ids = reinterpret_cast<int*>(extra + L::PAGES);
  int* cta_failed = reinterpret_cast<int*>(base + L::FLAG);
  int* cta_last = cta_failed + 1;

  if ((int)blockIdx.x >= p.num_ctas) return;  // whole CTA
  // Plan data is written only by the upload (a copy, which the programmatic
  // launch does not overlap): it may be read before the wait.
  const int4 hdr = *reinterpret_cast<const int4*>(p.ws_header);
  const int2 hdr_ctas = *reinterpret_cast<const int2*>(p.ws_header + 8);
  const bool coop = (int)blockIdx.x < p.num_shared;  // CTA-uniform
  const int first = coop ? (int)blockIdx.x : p.num_shared + ((int)blockIdx.x - p.num_shared) * NW;
  const int count = coop ? 1 : min(NW, p.num_items - first);
  const int task = coop ? first : (warp < count ? first + warp : -1);
  int4 it = make_int4(0, 0, 0, 0);
  int2 sg = make_int2(-1, -1);  // {partial slot, group}
  int4 grp = make_int4(-1, -1, 0, 0);
  if (task >= 0 && task < p.num_items) {
    it = p.items[task];
    sg = p.item_slots[task];
    if (sg.y >= 0 && sg.y < p.num_groups) grp = p.groups[sg.y];
  }
  const int slot = sg.x;
  if (task >= 0 && task < p.num_items && (int)blockIdx.x < p.pf_ctas) {
    const int phys = prefetch_page_of_lane<NW>(p, it, coop, warp, lane);
    if (phys >= 0) {
      const size_t off = ((size_t)phys * p.num_kv_heads + ((uint32_t)it.y & kItemHeadMask)) *
                         (2 * kPageSize * D);
      prefetch_l2_bulk(static_cast<const T*>(p.k_pages) + off, L::TILE);
      prefetch_l2_bulk(static_cast<const T*>(p.v_pages) + off, L::TILE);
    }
  }
  if (threadIdx.x == 0) {
    *cta_failed = 0;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tmap_k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tmap_v)) : "memory");
  }
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < NSH; ++s) mbar_init(bars + 8 * s, 1);
    fence_barrier_init();
  }
  __syncthreads();

  pdl_launch_dependents();
  pdl_wait_primary();  // everything the kernels ahead wrote is visible from here on

  if (hdr.x != (int)kDiffMagic || hdr.y != p.num_items || hdr.z != p.num_groups ||
      hdr.w != p.num_split_items || hdr_ctas.x != p.num_ctas || hdr_ctas.y != p.num_shared ||
      count < 1 || first < 0 || first + count > p.num_items) {
    if (threadIdx.x == 0) set_status(p.status, PA_DEV_PLAN_MISMATCH);
    return;  // CTA-uniform
  }
  if (task < 0) return;  // idle warp of a partial bundle; bundles never sync the CTA
  const int b = it.x;
  const uint32_t hw = (uint32_t)it.y;
  const int pair = (int)(hw & kItemHeadMask);
  const bool is_split = (hw & kItemSplit) != 0;
  const bool is_last = (hw & kItemLast) != 0;
  const int pg0 = it.z, pg1 = it.w;
  const bool slot_ok = is_split && split_slot_ok(p, sg, grp, b, pair);
  if (b < 0 || b >= p.batch || pair >= p.num_kv_heads || pg0 < 0 || pg1 < pg0 || pg1 > p.max_pages ||
      slot_ok != is_split) {
    if (lane == 0) set_status(p.status, PA_DEV_PLAN_MISMATCH);
    if (slot_ok && (!coop || warp == 0)) mark_split_missing(p.part_lse, slot, R, lane);
    return;  // all warps of a shared task see the same task
  }
  const int Lmax = p.max_pages * kPageSize;
  int seq_len = p.seq_lens[b];
  if (seq_len < 0 || seq_len > Lmax) {
    if (lane == 0) set_status(p.status, PA_DEV_BAD_SEQ_LEN);
    seq_len = min(max(seq_len, 0), Lmax);
  }
  if (is_last && seq_len > pg1 * kPageSize && lane == 0) set_status(p.status, PA_DEV_PLAN_MISMATCH);
  const int npg = pg1 - pg0;
  const int pstart = coop ? warp : 0;
  const int pstride = coop ? NW : 1;
  const int npk = coop ? (warp < npg ? (npg - warp + NW - 1) / NW : 0) : npg;

  const int32_t* bt_row = p.block_table + (size_t)b * p.max_pages + pg0;
  const uint64_t policy = l2_evict_first_policy();
  int bt_cur = lane < npg ? __ldg(bt_row + lane) : -1;
  int bt_nxt = 32 + lane < npg ? __ldg(bt_row + 32 + lane) : -1;
  int bt_w = 0;

  // Issue tile hi of this warp (keys of its page hi/2 for even hi, values for
  // odd hi) into stage hi % NSH; warp-collective, lane 0 issues.
  auto issue = [&](int hi) {
    const int j = pstart + (hi >> 1) * pstride;
    if ((j >> 5) != bt_w) {  // j grows by at most NW <= 32 between calls
      ++bt_w;
      bt_cur = bt_nxt;
      const int idx = 32 * (bt_w + 1) + lane;
      bt_nxt = idx < npg ? __ldg(bt_row + idx) : -1;
    }
    int phys = __shfl_sync(kFull, bt_cur, j & 31);
    if (lane == 0) {
      const int s = hi % NSH;
      const uint32_t bar = bars + 8 * s;
      if ((pg0 + j) * kPageSize >= seq_len) {
        phys = -1;
      } else if (phys < 0 || phys >= p.num_pages) {
        if ((hi & 1) == 0) set_status(p.status, PA_DEV_BAD_PAGE);
        phys = -1;
      }
      page_ids[s] = phys;
      fence_proxy_async_smem();
      if (phys >= 0) {
        const CUtensorMap* map = (hi & 1) ? &p.tmap_v : &p.tmap_k;
        mbar_arrive_expect_tx(bar, L::TILE);
#pragma unroll
        for (int bx = 0; bx < BOXES; ++bx)
          tma_load_4d(ring + s * L::TILE + bx * 4096, map, bx * 64, 0, 2 * pair, phys, bar, policy);
      } else {
        mbar_arrive(bar);
      }
    }
  };

  const int nhalf = 2 * npk;
  const int npre = nhalf < NSH ? nhalf : NSH;
  for (int hi = 0; hi < npre; ++hi) issue(hi);

  // Q^T fragments (B operand of S^T = K Q^T): column g, rows = dims.  Query
  // 2h + m of the pair is map m of head h; columns without a head are zero.
  uint32_t qb[NT][KSTEPS][2];
  {
    const T* q0 = static_cast<const T*>(p.q) +
                  ((size_t)b * p.num_kv_heads + pair) * (size_t)(R * D);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int head = NT == 1 ? (g & 3) : g, map = NT == 1 ? (g >> 2) : n;
      const T* qrow = q0 + (size_t)(2 * head + map) * D;
#pragma unroll
      for (int kk = 0; kk < KSTEPS; ++kk) {
        if (head < G) {
          qb[n][kk][0] = __ldg(reinterpret_cast<const unsigned int*>(qrow + kk * 16 + 2 * t));
          qb[n][kk][1] = __ldg(reinterpret_cast<const unsigned int*>(qrow + kk * 16 + 2 * t + 8));
        } else {
          qb[n][kk][0] = qb[n][kk][1] = 0u;
        }
      }
    }
  }

  // Online softmax state of columns 2t and 2t+1 of each column tile, and this
  // lane's share of their running sums.
  float m_run[NT][2], l_part[NT][2];
  float o[VTILES][NT][4];  // O^T: dims 16*mt + g (+8), columns 2t, 2t+1
#pragma unroll
  for (int n = 0; n < NT; ++n) m_run[n][0] = m_run[n][1] = -INFINITY, l_part[n][0] = l_part[n][1] = 0.f;
#pragma unroll
  for (int mt = 0; mt < VTILES; ++mt)
#pragma unroll
    for (int n = 0; n < NT; ++n) o[mt][n][0] = o[mt][n][1] = o[mt][n][2] = o[mt][n][3] = 0.f;
  const float qs = p.qscale;
  // lanes whose P^T entries this lane needs (decode_tc.cuh)
  const int src1 = (2 * t) * 4 + (g >> 1);
  const int src2 = (2 * t + 1) * 4 + (g >> 1);
  const unsigned int perm = (g & 1) ? 0x7632u : 0x5410u;

  bool failed = false;
  int hfail = 0;
  for (int k = 0; k < npk; ++k) {
    const int hk = 2 * k;
    const int sk = hk % NSH;
    if (!__all_sync(kFull, mbar_wait_bounded(bars + 8 * sk, (hk / NSH) & 1, p.wait_ns))) {
      failed = true;
      hfail = hk;
      break;
    }
    const int phys = page_ids[sk];
    const int j = pstart + k * pstride;
    const int nvalid = phys < 0 ? 0 : min(kPageSize, seq_len - (pg0 + j) * kPageSize);
    const uint32_t ktile = ring + sk * L::TILE;

    uint32_t pb_hi[NT][2], pb_lo[NT][2];
    float al[NT][2];
    bool rescale = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      pb_hi[n][0] = pb_hi[n][1] = pb_lo[n][0] = pb_lo[n][1] = 0u;
      al[n][0] = al[n][1] = 1.f;
    }
    if (nvalid > 0) {
      // ---- S^T = K_m . Q^T for both key tiles
      float c[2][4];
#pragma unroll
      for (int m = 0; m < 2; ++m) c[m][0] = c[m][1] = c[m][2] = c[m][3] = 0.f;
      const int kr = (lane & 7) + 8 * ((lane >> 3) & 1);  // token row this lane addresses
#pragma unroll
      for (int kk = 0; kk < KSTEPS; ++kk) {
        const uint32_t at = ktile + (kk >> 2) * 4096 + swz(kr, (kk & 3) * 2 + (lane >> 4));
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          uint32_t a0, a1, a2, a3;
          ldsm_x4(at + m * 2048, a0, a1, a2, a3);
          mma_16816<T>(c[m], a0, a1, a2, a3, qb[NT == 1 ? 0 : m][kk][0], qb[NT == 1 ? 0 : m][kk][1]);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float s[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = (NT == 1 ? (t < 2 ? c[0][i] : c[1][i]) : c[n][i]) * qs;
        if (g >= nvalid) s[0] = s[1] = -INFINITY;
        if (g + 8 >= nvalid) s[2] = s[3] = -INFINITY;
        // ---- online softmax for columns 2t (s0, s2) and 2t+1 (s1, s3)
        float mA = fmaxf(s[0], s[2]), mB = fmaxf(s[1], s[3]);
#pragma unroll
        for (int m = 4; m <= 16; m <<= 1) {
          mA = fmaxf(mA, __shfl_xor_sync(kFull, mA, m));
          mB = fmaxf(mB, __shfl_xor_sync(kFull, mB, m));
        }
        const float nA = fmaxf(m_run[n][0], mA), nB = fmaxf(m_run[n][1], mB);
        al[n][0] = nA == -INFINITY ? 1.f : ex2(m_run[n][0] - nA);
        al[n][1] = nB == -INFINITY ? 1.f : ex2(m_run[n][1] - nB);
        const float p0 = diff_weight<T>(s[0], nA), p2 = diff_weight<T>(s[2], nA);
        const float p1 = diff_weight<T>(s[1], nB), p3 = diff_weight<T>(s[3], nB);
        l_part[n][0] = l_part[n][0] * al[n][0] + (p0 + p2);
        l_part[n][1] = l_part[n][1] * al[n][1] + (p1 + p3);
        m_run[n][0] = nA;
        m_run[n][1] = nB;
        rescale = rescale || al[n][0] != 1.f || al[n][1] != 1.f;
        // ---- P^T into B fragments, hi and lo parts in the element type
        const uint32_t h01 = Elem<T>::from_f2(p0, p1);  // token g: columns 2t, 2t+1
        const uint32_t h23 = Elem<T>::from_f2(p2, p3);  // token g+8
        const float2 f01 = Elem<T>::to_f2(h01), f23 = Elem<T>::to_f2(h23);
        const uint32_t l01 = Elem<T>::from_f2(p0 - f01.x, p1 - f01.y);
        const uint32_t l23 = Elem<T>::from_f2(p2 - f23.x, p3 - f23.y);
        pb_hi[n][0] = __byte_perm(__shfl_sync(kFull, h01, src1), __shfl_sync(kFull, h01, src2), perm);
        pb_hi[n][1] = __byte_perm(__shfl_sync(kFull, h23, src1), __shfl_sync(kFull, h23, src2), perm);
        pb_lo[n][0] = __byte_perm(__shfl_sync(kFull, l01, src1), __shfl_sync(kFull, l01, src2), perm);
        pb_lo[n][1] = __byte_perm(__shfl_sync(kFull, l23, src1), __shfl_sync(kFull, l23, src2), perm);
      }
      rescale = __any_sync(kFull, rescale);
    }
    // the key stage is free: refill it
    __syncwarp();
    if (hk + NSH < nhalf) issue(hk + NSH);

    const int hv = hk + 1;
    const int sv = hv % NSH;
    if (!__all_sync(kFull, mbar_wait_bounded(bars + 8 * sv, (hv / NSH) & 1, p.wait_ns))) {
      failed = true;
      hfail = hv;
      break;
    }
    const uint32_t vtile = ring + sv * L::TILE;
    if (nvalid > 0) {
      if (rescale) {
#pragma unroll
        for (int mt = 0; mt < VTILES; ++mt)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            o[mt][n][0] *= al[n][0];
            o[mt][n][1] *= al[n][1];
            o[mt][n][2] *= al[n][0];
            o[mt][n][3] *= al[n][1];
          }
      }
      // ---- O^T += V^T . P^T (hi and lo)
      // masks for tokens 2t, 2t+1 and 2t+8, 2t+9 (zero the rows past nvalid)
      const uint32_t mk0 = (2 * t < nvalid ? 0x0000ffffu : 0u) | (2 * t + 1 < nvalid ? 0xffff0000u : 0u);
      const uint32_t mk8 =
          (2 * t + 8 < nvalid ? 0x0000ffffu : 0u) | (2 * t + 9 < nvalid ? 0xffff0000u : 0u);
      const int q4 = lane >> 3;
      const int vr = (q4 >> 1) * 8 + (lane & 7);  // token row this lane addresses
#pragma unroll
      for (int mt = 0; mt < VTILES; ++mt) {
        constexpr int PER = D / 16;  // m-tiles of one head's values
        const int head = mt / PER, box = (mt % PER) >> 2, chunk = (mt & 3) * 2 + (q4 & 1);
        uint32_t a0, a1, a2, a3;
        ldsm_x4_t(vtile + box * 4096 + head * 2048 + swz(vr, chunk), a0, a1, a2, a3);
        if (nvalid < kPageSize) {
          a0 &= mk0;
          a1 &= mk0;
          a2 &= mk8;
          a3 &= mk8;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_16816<T>(o[mt][n], a0, a1, a2, a3, pb_hi[n][0], pb_hi[n][1]);
          mma_16816<T>(o[mt][n], a0, a1, a2, a3, pb_lo[n][0], pb_lo[n][1]);
        }
      }
    }
    __syncwarp();
    if (hv + NSH < nhalf) issue(hv + NSH);
  }

  if (failed) {
    // A copy did not land in time.  Report it and let the copies already
    // issued finish (bounded).  The task writes nothing.
    if (lane == 0) {
      set_status(p.status, PA_DEV_TIMEOUT);
      const int last = min(nhalf, hfail + NSH);
      for (int h = hfail; h < last; ++h)
        mbar_wait_bounded(bars + 8 * (h % NSH), (h / NSH) & 1, kDrainWaitNs);
      *cta_failed = 1;
    }
    __syncwarp();
  } else if (lane == 0) {
#pragma unroll
    for (int s = 0; s < NSH; ++s) mbar_inval(bars + 8 * s);
  }

  // full running sums: add the shares of the 8 lanes of t
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 4; m <= 16; m <<= 1) {
      l_part[n][0] += __shfl_xor_sync(kFull, l_part[n][0], m);
      l_part[n][1] += __shfl_xor_sync(kFull, l_part[n][1], m);
    }

  // the row of column i (0, 1) of column tile n, or -1
  auto row_of = [&](int n, int i) {
    const int col = 2 * t + i;
    const int head = NT == 1 ? (col & 3) : col, map = NT == 1 ? (col >> 2) : n;
    return head < G ? map * G + head : -1;
  };
  T* const out = static_cast<T*>(p.out) + ((size_t)b * p.num_kv_heads + pair) * (size_t)(G * VD);
  const float* const lambda = dp.e.lambda + (size_t)pair * G;

  if (!coop) {
    // ---- a task of its own: normalise into this warp's (now free) ring
    if (failed) {
      if (is_split) mark_split_missing(p.part_lse, slot, R, lane);
      return;
    }
    float* stage = reinterpret_cast<float*>(base + warp * L::RING);  // [R][VD]
    static_assert(R * VD * 4 <= L::RING, "a warp's rows fit in its ring");
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = row_of(n, i);
        if (row < 0) continue;
        const float inv = l_part[n][i] > 0.f || l_part[n][i] != l_part[n][i] ? 1.f / l_part[n][i] : 0.f;
#pragma unroll
        for (int mt = 0; mt < VTILES; ++mt) {
          stage[row * VD + 16 * mt + g] = o[mt][n][i] * inv;
          stage[row * VD + 16 * mt + g + 8] = o[mt][n][2 + i] * inv;
        }
        if (is_split && g == 0) {
          p.part_lse[(size_t)slot * R + row] = m_run[n][i];
          dp.part_sum[(size_t)slot * R + row] = l_part[n][i];
        }
      }
    __syncwarp();
    if (!is_split) {
      for (int h = 0; h < G; ++h) {
        float4 r[2][VD / 128];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int i = 0; i < VD / 128; ++i)
            r[m][i] = *reinterpret_cast<const float4*>(stage + (m * G + h) * VD + 128 * i + 4 * lane);
        diff_write_head<T, VD>(dp.e, __ldg(lambda + h), r[0], r[1], lane, out + (size_t)h * VD);
      }
    } else {
      float* dst = p.part_o + (size_t)slot * R * VD;
      for (int i = lane * 4; i < R * VD; i += 128)
        *reinterpret_cast<float4*>(dst + i) = *reinterpret_cast<const float4*>(stage + i);
      if (!p.fuse_merge) return;
      const MergeTarget mt = merge_target(p, sg.y, grp, R);
      __syncwarp();
      int last = 0;
      if (lane == 0) last = atom_add_acq_rel_gpu(mt.counter, 1) == grp.z - 1;
      last = __shfl_sync(kFull, last, 0);
      if (!last) return;
      __syncwarp();
      diff_merge_heads<T, D, G>(dp, mt, 0, 1, lane);
      if (lane == 0) *mt.counter = 0;
    }
    return;
  }

  // ---- shared task: merge the NW warp states in shared memory (rings are free)
  __syncthreads();
  if (*cta_failed) {
    if (is_split && warp == 0) mark_split_missing(p.part_lse, slot, R, lane);
    return;
  }
  float* st = reinterpret_cast<float*>(base);  // [NW][2R + R*VD]
  constexpr int SLOT = 2 * R + R * VD;
  static_assert(NW * SLOT * 4 <= L::RINGS, "the warps' states fit in the rings");
  float* mine = st + warp * SLOT;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = row_of(n, i);
      if (row < 0) continue;
      if (g == 0) {
        mine[row] = m_run[n][i];
        mine[R + row] = l_part[n][i];
      }
#pragma unroll
      for (int mt = 0; mt < VTILES; ++mt) {
        mine[2 * R + row * VD + 16 * mt + g] = o[mt][n][i];
        mine[2 * R + row * VD + 16 * mt + g + 8] = o[mt][n][2 + i];
      }
    }
  __syncthreads();

  // four dims of a row over the warps, normalised; the row's reference and sum
  auto merged = [&](int row, int d, float& M, float& Z) {
    M = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, st[w * SLOT + row]);
    Z = 0.f;
    float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      // 0 for an empty warp (m = -inf), unless all are: zeros, or NaN, then
      const float sc = M == -INFINITY ? 1.f : ex2(st[w * SLOT + row] - M);
      const float4 x = *reinterpret_cast<const float4*>(st + w * SLOT + 2 * R + row * VD + d);
      Z = fmaf(st[w * SLOT + R + row], sc, Z);
      r.x = fmaf(x.x, sc, r.x);
      r.y = fmaf(x.y, sc, r.y);
      r.z = fmaf(x.z, sc, r.z);
      r.w = fmaf(x.w, sc, r.w);
    }
    const float inv = Z > 0.f || Z != Z ? 1.f / Z : 0.f;
    return make_float4(r.x * inv, r.y * inv, r.z * inv, r.w * inv);
  };
  float ref, total;
  if (!is_split) {
    for (int h = warp; h < G; h += NW) {
      float4 r[2][VD / 128];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < VD / 128; ++i) r[m][i] = merged(m * G + h, 128 * i + 4 * lane, ref, total);
      diff_write_head<T, VD>(dp.e, __ldg(lambda + h), r[0], r[1], lane, out + (size_t)h * VD);
    }
    return;
  }
  for (int idx = threadIdx.x; idx < R * VD / 4; idx += NW * 32) {
    const int row = idx / (VD / 4), d = idx % (VD / 4) * 4;
    const float4 r = merged(row, d, ref, total);
    *reinterpret_cast<float4*>(p.part_o + ((size_t)slot * R + row) * VD + d) = r;
    if (d == 0) {
      p.part_lse[(size_t)slot * R + row] = ref;
      dp.part_sum[(size_t)slot * R + row] = total;
    }
  }
  if (!p.fuse_merge) return;
  const MergeTarget mt = merge_target(p, sg.y, grp, R);
  __syncthreads();
  if (threadIdx.x == 0) *cta_last = atom_add_acq_rel_gpu(mt.counter, 1) == grp.z - 1;
  __syncthreads();
  if (!*cta_last) return;
  diff_merge_heads<T, D, G>(dp, mt, warp, NW, lane);
  if (threadIdx.x == 0) *mt.counter = 0;
}

}  // namespace pa
