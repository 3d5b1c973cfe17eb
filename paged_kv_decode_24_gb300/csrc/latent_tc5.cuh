// tcgen05 helpers of the latent attention kernels.
//
// The MMA warp elects its issuing lane with elect.sync, so the compiler knows
// that one thread runs the issue blocks and keeps descriptors in uniform
// registers; descriptors are a base plus constants.
#pragma once

#include "latent_params.h"
#include "prefill_tc5.cuh"

namespace pa {
namespace tc5 {

// True in one lane of the (converged) warp, always the same one.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e != 0;
}

// A descriptor `bytes` further on (within shared memory: no carry out of the address field).
__device__ __forceinline__ uint64_t desc_at(uint64_t base, uint32_t bytes) {
  return base + (uint64_t)(bytes >> 4);
}

// D (+)= A B, one CTA.
__device__ __forceinline__ void mma1(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                     uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The same with A from TMEM.
__device__ __forceinline__ void mma1_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// D (+)= A B over a pair of CTAs, each with half of A's rows and of B's.
__device__ __forceinline__ void mma2(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                     uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The barrier at this offset in both CTAs, once every MMA issued so far is done.
__device__ __forceinline__ void commit2(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}

// 32 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void ld32(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// A bounded wait of the whole warp.  Every lane polls: with one lane polling
// and a shuffle behind it the wake-up took longer (prompt 8192 x 32 heads 585
// against 542 us, batch of 32 with 128 heads 68 against 60 us).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  return __all_sync(kFull, mbar_wait_bounded_sleep(bar, parity, limit_ns)) != 0;
}

}  // namespace tc5

// Weights are 2^(s qscale - m) in one fused multiply-add, with m the rounded
// product of a maximal score.  The fused product is exact, so the exponent keeps
// what m lost in its rounding, up to half of m's last place, the same for the
// whole row: no error of the weights until it reaches many units, beyond
// |m| = 2^24, where it would overflow or empty them.  A warp that has a row
// beyond 2^23 therefore takes the product rounded as m was: its scores become
// s qscale - m, to be used with a factor of 1 and m = 0.
constexpr float kFusedLog2 = 8388608.f;

__device__ __forceinline__ bool beyond_fused(float m) {
  return __any_sync(kFull, fabsf(m) > kFusedLog2 && m != -INFINITY) != 0;
}

template <int N>
__device__ __forceinline__ void rounded_differences(float (&s)[N], float qscale, float m) {
  const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = __fsub_rn(__fmul_rn(s[i], qscale), ref);
}

// The page of token tok, -1 from `end` on.  A volatile load, which stays where
// it is written: a stage ahead of its use.
__device__ __forceinline__ int table_entry(const int32_t* table, int page_size, int tok, int end) {
  int page = -1;
  if (tok < end) asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(page) : "l"(table + tok / page_size));
  return page;
}

// 32 bytes to a 16-byte aligned address; `whole`: it is 32-byte aligned.
__device__ __forceinline__ void store32(void* dst, const uint32_t* w, bool whole) {
  if (whole) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

__device__ __forceinline__ void row_pair_barrier(int warp) {  // the two warps that share 32 rows
  __syncwarp();  // the barrier is for converged warps
  asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp & 1)) : "memory");
}

// q as [T * H][576], with boxes of 64 rows by 64 dims.
inline bool encode_latent_q(CUtensorMap* map, const LatentParams& p, int dtype) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = latent_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {kLatentRow, (cuuint64_t)p.total_q * (cuuint64_t)p.heads};
  cuuint64_t strides[1] = {kLatentRow * 2};
  cuuint32_t box[2] = {64, kLatentRowsSolo};
  cuuint32_t estr[2] = {1, 1};
  const CUtensorMapDataType ty = dtype == PA_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                       : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return enc(map, ty, 2, const_cast<void*>(p.q), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The pool [P][S][576] with boxes of `tokens` tokens by 64 dims.  (With the
// row split into a dimension of nine boxes the copies run 12 % slower.)
inline bool encode_latent_boxes(CUtensorMap* map, const void* pages, const pa_latent_shape_t& s, int tokens) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = latent_map_encoder();
  if (!enc) return false;
  const cuuint64_t row = kLatentRow * 2;
  cuuint64_t dims[3] = {kLatentRow, (cuuint64_t)s.page_size, (cuuint64_t)s.num_pages};
  cuuint64_t strides[2] = {row, row * s.page_size};
  cuuint32_t box[3] = {64, (cuuint32_t)tokens, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapDataType ty = s.dtype == PA_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                         : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return enc(map, ty, 3, const_cast<void*>(pages), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace pa
