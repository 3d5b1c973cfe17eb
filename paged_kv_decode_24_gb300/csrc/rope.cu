// Rotary append: the step's query rows rotated, its key rows rotated into
// their pages and its value rows copied there, in one launch.
//
//   x[a]' = x[a] c - x[b] s,   x[b]' = x[b] c + x[a] s
//
// Every row is read once and written once, with six operations a pair: bound
// by the bytes of the rows, and by a launch where there are few.
// A lane owns one unit of 16 values of a row, two 16-byte words: units of the
// rotated part hold both halves of eight pairs, so a pair never crosses lanes
// (values i .. i+7 and i + R/2 .. i + R/2 + 7, or 16 neighbours when pairs
// are neighbours).  D/16 lanes make a row, a warp 32 / (D/16) rows at once,
// all of one token: the token's place is looked up once a warp, and its
// cosines and sines stay in registers over the rows.
//
// Measured: 24 prompts with 54,358 tokens, 32 query and 8 KV heads of 128,
// 213.5 us, 93 % of the measured copy bandwidth; one token of 160 sequences,
// the same heads, 3.6 us, of one sequence 3.4 (a launch).  Prompts of 54,939 tokens
// into an INT8 cache 277 us, into an FP8 one 268 (1269 MB, 4.6 and 4.7 TB/s; 213 into a
// 16-bit one): the codes' divisions, with half of the issue slots taken.
#include <math.h>

#include <atomic>

#include "device_common.cuh"
#include "elem.cuh"
#include "latent_launch.cuh"
#include "pa_internal.h"
#include "quant_common.cuh"

namespace pa {

namespace {

constexpr int kCode16 = 2;  // a cache of 16-bit elements (after kCodeInt8 and kCodeE4m3)
constexpr int kRopeThreads = 128;

struct RopeParams {
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  void* k_pages;
  void* v_pages;
  float* k_scales;
  float* v_scales;
  const float* table;
  const int32_t* positions;  // or null
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* ws;  // the uploaded multi-token plan, or null: one token a sequence
  const int32_t* cu;  // its row offsets
  int32_t* status;
  int64_t q_stride, k_stride, v_stride;
  int32_t batch, rows, num_tiles, num_q_heads, num_kv_heads, max_pages, num_pages;
  int32_t rotary, interleaved, num_positions;
  int32_t turns, parts;  // groups of rows a warp takes, warps of a token
};

// The sequence of packed row r: the largest b with cu[b] <= r (the last of
// equal ones, so sequences without rows are passed over).  The warp's lanes
// probe 32 places at once.
__device__ __forceinline__ int sequence_of_row(const int32_t* cu, int batch, int r, int lane) {
  int lo = 0, n = batch;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const unsigned below = __ballot_sync(kFull, lane * step < n && cu[lo + lane * step] <= r);
    const int k = 31 - __clz(below | 1u);
    n = min(step, n - k * step);
    lo += k * step;
  }
  return lo;
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& raw, float* x) {
  float2 f[4];
  elem8_to_float2x4<T>(raw, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = f[i].x;
    x[2 * i + 1] = f[i].y;
  }
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float* x) {
  uint4 r;
  r.x = Elem<T>::from_f2(x[0], x[1]);
  r.y = Elem<T>::from_f2(x[2], x[3]);
  r.z = Elem<T>::from_f2(x[4], x[5]);
  r.w = Elem<T>::from_f2(x[6], x[7]);
  return r;
}

// Eight codes, low byte first, by the rules of quant_common.cuh.
template <int FMT>
__device__ __forceinline__ uint2 codes8(const float* x, float scale) {
  uint32_t w[2] = {0u, 0u};
  if (scale > 0.f) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float a = __fdiv_rn(x[i], scale), b = __fdiv_rn(x[i + 1], scale);
      uint32_t two;
      if constexpr (FMT == kCodeE4m3) {
        two = f2_to_e4m3x2(a, b);
      } else {
        const int ca = min(127, max(-127, __float2int_rn(a)));
        const int cb = min(127, max(-127, __float2int_rn(b)));
        two = (uint32_t)(ca & 0xff) | (uint32_t)(cb & 0xff) << 8;
      }
      w[i >> 2] |= two << (8 * (i & 3));
    }
  }
  return make_uint2(w[0], w[1]);
}

template <typename T, int D, int FMT>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const __grid_constant__ RopeParams p) {
  constexpr int UNITS = D / 16;       // lanes of a row
  constexpr int ROWS = 32 / UNITS;    // rows of a warp at once
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const int64_t row64 = w / p.parts;
  if (row64 >= p.rows) return;  // whole warp
  const int row = (int)row64, part = (int)(w % p.parts);

  // The plan is written by the upload alone, which the programmatic launch
  // does not overlap: it may be read before the wait for the kernel ahead.
  int b = row, back = 1, fresh = 1;  // the row's sequence, its token from the end, new tokens
  bool bad = false;
  if (p.ws != nullptr) {
    const int4 hdr = *reinterpret_cast<const int4*>(p.ws);
    bad = hdr.x != (int)kPrefillMagic || hdr.y != p.num_tiles || hdr.z != p.batch || hdr.w != p.rows;
    if (!bad) {
      b = sequence_of_row(p.cu, p.batch, row, lane);
      const int end = p.cu[b + 1];
      back = end - row;
      fresh = end - p.cu[b];
      bad = back < 1 || back > fresh;
    }
  }
  pdl_wait_primary();
  if (bad) {
    if (lane == 0) set_status(p.status, PA_DEV_PLAN_MISMATCH);
    return;
  }
  const int len = p.seq_lens[b], longest = p.max_pages * kPageSize;
  if (len < 0 || len > longest) {
    if (lane == 0) set_status(p.status, PA_DEV_BAD_SEQ_LEN);
    return;
  }
  if (p.ws == nullptr && len == 0) return;
  if (len < fresh) {
    if (lane == 0) set_status(p.status, PA_DEV_PLAN_MISMATCH);
    return;
  }
  const int pos = len - back;
  const int turn = p.positions != nullptr ? p.positions[row] : pos;
  if (turn < 0 || turn >= p.num_positions) {
    if (lane == 0) set_status(p.status, PA_DEV_BAD_POSITION);
    return;
  }
  const int page = p.block_table[(size_t)b * p.max_pages + pos / kPageSize];
  const bool page_ok = page >= 0 && page < p.num_pages;
  if (!page_ok && lane == 0) set_status(p.status, PA_DEV_BAD_PAGE);

  const int u = lane % UNITS, sub = lane / UNITS;
  const int half = p.rotary / 2;
  const bool rotated = 16 * u < p.rotary;
  const bool split = rotated && !p.interleaved;  // the unit's words lie R/2 apart
  const int o0 = split ? 8 * u : 16 * u, o1 = split ? half + 8 * u : 16 * u + 8;
  float c[8], s[8];
  if (rotated) {
    const float4* t = reinterpret_cast<const float4*>(p.table + (size_t)turn * p.rotary + 8 * u);
    const float4* t2 = reinterpret_cast<const float4*>(p.table + (size_t)turn * p.rotary + half + 8 * u);
    const float4 a = __ldg(t), d = __ldg(t + 1), e = __ldg(t2), f = __ldg(t2 + 1);
    c[0] = a.x, c[1] = a.y, c[2] = a.z, c[3] = a.w, c[4] = d.x, c[5] = d.y, c[6] = d.z, c[7] = d.w;
    s[0] = e.x, s[1] = e.y, s[2] = e.z, s[3] = e.w, s[4] = f.x, s[5] = f.y, s[6] = f.z, s[7] = f.w;
  }
  const int nq = p.q != nullptr ? p.num_q_heads : 0;
  const int total = nq + 2 * p.num_kv_heads;  // rows of the token
  const int first = part * p.turns * ROWS;
#pragma unroll 2
  for (int it = 0; it < p.turns; ++it) {
    const int r = first + it * ROWS + sub;
    const bool on = r < total;
    const int kind = r < nq ? 0 : r < nq + p.num_kv_heads ? 1 : 2;  // q, k, v
    const int h = r - (kind == 0 ? 0 : kind == 1 ? nq : nq + p.num_kv_heads);
    uint4 w0 = make_uint4(0u, 0u, 0u, 0u), w1 = w0;
    if (on) {
      const T* src = kind == 0   ? static_cast<const T*>(p.q) + row * p.q_stride
                     : kind == 1 ? static_cast<const T*>(p.k) + row * p.k_stride
                                 : static_cast<const T*>(p.v) + row * p.v_stride;
      src += (size_t)h * D;
      const bool apart = split && kind != 2;
      w0 = *reinterpret_cast<const uint4*>(src + (apart ? o0 : 16 * u));
      w1 = *reinterpret_cast<const uint4*>(src + (apart ? o1 : 16 * u + 8));
    }
    float x[16];  // the rotated values in fp32, words 0 and 1
    const bool eight = FMT != kCode16 && kind != 0;
    if (kind != 2 || eight) {
      unpack8<T>(w0, x);
      unpack8<T>(w1, x + 8);
    }
    if (kind != 2 && rotated) {
      if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float a = x[2 * i], d = x[2 * i + 1];
          x[2 * i] = fmaf(a, c[i], -(d * s[i]));
          x[2 * i + 1] = fmaf(d, c[i], a * s[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float a = x[i], d = x[8 + i];
          x[i] = fmaf(a, c[i], -(d * s[i]));
          x[8 + i] = fmaf(d, c[i], a * s[i]);
        }
      }
      if (!eight) {
        w0 = pack8<T>(x);
        w1 = pack8<T>(x + 8);
      }
    }
    const int e0 = kind == 2 ? 16 * u : o0, e1 = kind == 2 ? 16 * u + 8 : o1;
    const size_t slot = ((size_t)(page_ok ? page : 0) * p.num_kv_heads + (kind == 0 ? 0 : h)) * kPageSize +
                        pos % kPageSize;
    if constexpr (FMT != kCode16) {
      float top = 0.f;
      if (eight) {
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(x[i]));
      }
      __syncwarp();
#pragma unroll
      for (int m = UNITS / 2; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, m));
      if (on && eight && page_ok) {
        const float scale = __fdiv_rn(top, FMT == kCodeE4m3 ? 448.f : 127.f);
        uint8_t* dst = static_cast<uint8_t*>(kind == 1 ? p.k_pages : p.v_pages) + slot * D;
        *reinterpret_cast<uint2*>(dst + e0) = codes8<FMT>(x, scale);
        *reinterpret_cast<uint2*>(dst + e1) = codes8<FMT>(x + 8, scale);
        if (u == 0) (kind == 1 ? p.k_scales : p.v_scales)[slot] = scale;
      }
      if (eight) continue;
    }
    if (!on) continue;
    T* dst;
    if (kind == 0)
      dst = static_cast<T*>(p.q_out) + ((size_t)row * p.num_q_heads + h) * D;
    else if (page_ok)
      dst = static_cast<T*>(kind == 1 ? p.k_pages : p.v_pages) + slot * D;
    else
      continue;
    *reinterpret_cast<uint4*>(dst + e0) = w0;
    *reinterpret_cast<uint4*>(dst + e1) = w1;
  }
}

template <typename T, int D, int FMT>
cudaError_t launch_t(const RopeParams& p, int grid, cudaStream_t stream) {
  static std::atomic<unsigned long long> configured{0};
  return launch_latent(rope_append_kernel<T, D, FMT>, 0, configured, grid, kRopeThreads, stream, p);
}

cudaError_t launch_rope(RopeParams& p, int head_dim, int dtype, int kv_kind, cudaStream_t stream) {
  const int rows = 32 / (head_dim / 16);  // of a warp at once
  const int total = (p.q != nullptr ? p.num_q_heads : 0) + 2 * p.num_kv_heads;
  const int groups = (total + rows - 1) / rows;
  // A warp takes as many of its token's row groups as leave every SM 32 warps.
  const int64_t warps = (int64_t)p.rows * groups;
  const int sms = sm_count();
  int64_t turns = warps / ((sms > 0 ? sms : 1) * 32);
  turns = turns < 1 ? 1 : turns > groups ? groups : turns;
  p.turns = (int)turns;
  p.parts = (groups + p.turns - 1) / p.turns;
  const int64_t grid = ((int64_t)p.rows * p.parts + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  const int g = (int)grid;
  if (kv_kind == PA_KV_INT8)
    return head_dim == 64 ? launch_t<__half, 64, kCodeInt8>(p, g, stream)
                          : launch_t<__half, 128, kCodeInt8>(p, g, stream);
  if (kv_kind == PA_KV_FP8)
    return head_dim == 64 ? launch_t<__half, 64, kCodeE4m3>(p, g, stream)
                          : launch_t<__half, 128, kCodeE4m3>(p, g, stream);
  if (dtype == PA_DTYPE_BF16)
    return head_dim == 64 ? launch_t<__nv_bfloat16, 64, kCode16>(p, g, stream)
                          : launch_t<__nv_bfloat16, 128, kCode16>(p, g, stream);
  return head_dim == 64 ? launch_t<__half, 64, kCode16>(p, g, stream)
                        : launch_t<__half, 128, kCode16>(p, g, stream);
}

bool aligned(const void* p, uintptr_t a) { return p && ((uintptr_t)p % a) == 0; }

// Tokens of `width` values `stride` apart: multiples of 16 bytes below 2^40.
bool stride_ok(int64_t stride, int64_t width) {
  return stride >= width && stride % 8 == 0 && stride < (int64_t)1 << 39;
}

// Whether `rows` tokens of `width` 16-bit values, `stride` apart from p on, share
// a byte's range with the dense ones from q on.
bool ranges_meet(const void* p, int64_t stride, int64_t width, const void* q, int64_t dense, int64_t rows) {
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  const uintptr_t a_end = a + 2 * (uintptr_t)((rows - 1) * stride + width);
  const uintptr_t b_end = b + 2 * (uintptr_t)(rows * dense);
  return a < b_end && b < a_end;
}

// What both calls check and launch; `rows` tokens, the plan (plan_bytes) already in p.ws.
pa_status_t rope_impl(const pa_shape_t* s, const pa_rope_t* rope, RopeParams& p, int64_t rows,
                      size_t plan_bytes, int32_t* dev_status, void* stream) {
  if (!rope) return PA_ERR_INVALID_ARG;
  if (rope->rotary_dim < 16 || rope->rotary_dim > s->head_dim || rope->rotary_dim % 16 != 0)
    return PA_ERR_UNSUPPORTED;
  if ((rope->interleaved != 0 && rope->interleaved != 1) || rope->num_positions < 1)
    return PA_ERR_INVALID_ARG;
  if (rope->kv_kind != PA_KV_16BIT && rope->kv_kind != PA_KV_INT8 && rope->kv_kind != PA_KV_FP8)
    return PA_ERR_INVALID_ARG;
  const bool eight = rope->kv_kind != PA_KV_16BIT;
  if (eight && s->dtype != PA_DTYPE_F16) return PA_ERR_UNSUPPORTED;
  if (rows == 0) return PA_OK;
  if (!aligned(p.k, 16) || !aligned(p.v, 16) || !aligned(p.k_pages, 16) || !aligned(p.v_pages, 16) ||
      !aligned(rope->table, 16) || !aligned(p.block_table, 4) || !aligned(p.seq_lens, 4) ||
      !aligned(dev_status, 4) || (p.positions && !aligned(p.positions, 4)))
    return PA_ERR_INVALID_ARG;
  if (eight ? !aligned(p.k_scales, 16) || !aligned(p.v_scales, 16) : p.k_scales || p.v_scales)
    return PA_ERR_INVALID_ARG;
  const int64_t wq = (int64_t)s->num_q_heads * s->head_dim, wk = (int64_t)s->num_kv_heads * s->head_dim;
  if (!stride_ok(p.k_stride, wk) || !stride_ok(p.v_stride, wk)) return PA_ERR_INVALID_ARG;
  if (p.q || p.q_out) {
    if (!aligned(p.q, 16) || !aligned(p.q_out, 16) || !stride_ok(p.q_stride, wq)) return PA_ERR_INVALID_ARG;
    const bool in_place = p.q == p.q_out && (p.q_stride == wq || rows == 1);
    if ((!in_place && ranges_meet(p.q, p.q_stride, wq, p.q_out, wq, rows)) ||
        ranges_meet(p.k, p.k_stride, wk, p.q_out, wq, rows) ||
        ranges_meet(p.v, p.v_stride, wk, p.q_out, wq, rows))
      return PA_ERR_INVALID_ARG;
    auto meets = [&](const void* a, uintptr_t bytes) {
      return a && (uintptr_t)a < (uintptr_t)p.q_out + 2 * (uintptr_t)(rows * wq) && (uintptr_t)p.q_out < (uintptr_t)a + bytes;
    };
    const uintptr_t slots = (uintptr_t)s->num_pages * s->num_kv_heads * kPageSize;
    const uintptr_t pool = slots * s->head_dim * (eight ? 1 : 2);
    if (meets(rope->table, 4 * (uintptr_t)rope->num_positions * rope->rotary_dim) || meets(p.positions, 4 * rows) ||
        meets(p.block_table, 4 * (uintptr_t)s->batch * s->max_pages_per_seq) ||
        meets(p.seq_lens, 4 * (uintptr_t)s->batch) || meets(p.ws, plan_bytes) || meets(dev_status, 4) ||
        meets(p.k_pages, pool) || meets(p.v_pages, pool) || meets(p.k_scales, 4 * slots) ||
        meets(p.v_scales, 4 * slots))
      return PA_ERR_INVALID_ARG;
  }
  p.table = rope->table;
  p.status = dev_status;
  p.batch = s->batch;
  p.rows = (int32_t)rows;
  p.num_q_heads = s->num_q_heads;
  p.num_kv_heads = s->num_kv_heads;
  p.max_pages = s->max_pages_per_seq;
  p.num_pages = s->num_pages;
  p.rotary = rope->rotary_dim;
  p.interleaved = rope->interleaved;
  p.num_positions = rope->num_positions;
  const cudaError_t e = launch_rope(p, s->head_dim, s->dtype, rope->kv_kind, (cudaStream_t)stream);
  if (e == cudaSuccess) return PA_OK;
  (void)cudaGetLastError();  // clear a launch error so that later calls report their own
  return PA_ERR_CUDA;
}

}  // namespace
}  // namespace pa

extern "C" pa_status_t pa_rope_append(const pa_shape_t* shape, const pa_rope_t* rope, const void* q,
                                      int64_t q_stride, const void* k_new, int64_t k_stride,
                                      const void* v_new, int64_t v_stride,
                                      const int32_t* positions, void* q_out, void* k_pages,
                                      void* v_pages, float* k_scales, float* v_scales,
                                      const int32_t* block_table, const int32_t* seq_lens,
                                      int32_t* dev_status, void* stream) {
  using namespace pa;
  const pa_status_t st = check_shape(shape);
  if (st != PA_OK) return st;
  RopeParams p{};
  p.q = q, p.k = k_new, p.v = v_new, p.q_out = q_out;
  p.q_stride = q_stride, p.k_stride = k_stride, p.v_stride = v_stride;
  p.k_pages = k_pages, p.v_pages = v_pages, p.k_scales = k_scales, p.v_scales = v_scales;
  p.positions = positions, p.block_table = block_table, p.seq_lens = seq_lens;
  return rope_impl(shape, rope, p, shape->batch, 0, dev_status, stream);
}

extern "C" pa_status_t pa_rope_append_tokens(
    const pa_shape_t* shape, const pa_prefill_plan_t* plan, const pa_rope_t* rope, const void* q,
    int64_t q_stride, const void* k_new, int64_t k_stride, const void* v_new, int64_t v_stride,
    const int32_t* positions, void* q_out, void* k_pages, void* v_pages, float* k_scales,
    float* v_scales, const int32_t* block_table, const int32_t* seq_lens, const void* workspace,
    size_t workspace_bytes, int32_t* dev_status, void* stream) {
  using namespace pa;
  const pa_status_t st = check_prefill_call(shape, plan, workspace, workspace_bytes);
  if (st != PA_OK) return st;
  RopeParams p{};
  p.q = q, p.k = k_new, p.v = v_new, p.q_out = q_out;
  p.q_stride = q_stride, p.k_stride = k_stride, p.v_stride = v_stride;
  p.k_pages = k_pages, p.v_pages = v_pages, p.k_scales = k_scales, p.v_scales = v_scales;
  p.positions = positions, p.block_table = block_table, p.seq_lens = seq_lens;
  p.num_tiles = plan->num_tiles;
  p.ws = static_cast<const int32_t*>(workspace);
  p.cu = reinterpret_cast<const int32_t*>(static_cast<const char*>(workspace) +
                                          prefill_layout(plan->num_tiles, shape->batch).cu_off);
  return rope_impl(shape, rope, p, shape->batch == 0 ? 0 : plan->total_q, plan->workspace_bytes, dev_status, stream);
}
