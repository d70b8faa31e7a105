// kda_attn.cuh -- arguments and small device helpers shared by the softmax
// attention kernels: attention over packed rows (kda_attn.cu), the 8-bit paged
// cache (kda_cache.cu) and attention over it (kda_cache_attn.cu).
//
// Score of a visible (query i, key j) pair, in this order:
//   x = scale * q_i . k_j;  x = cap * tanh(x / cap) if cap > 0;  x -= slope_h * |p_i - p_j|
// The kernels hold scores in units of log2 (x * log2 e), so that a softmax
// weight is one ex2.  Sums, maxima and accumulators are fp32.
#pragma once

#include <cuda_fp16.h>

#include "kda.h"
#include "kda_common.cuh"

namespace kda {

constexpr float kLog2e = 1.4426950408889634f;
// SMs of a GB300.  What a call of the cache is cut into follows from it, and a workspace's
// size from that, so it is not asked of the device.
constexpr int kSMs = 152;

// Attention over packed rows.
struct AttnArgs {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  __nv_bfloat16* out;
  const int32_t* cu;      // [N + 1] or null: N equal sequences
  const int32_t* prefix;  // [N], KDA_MASK_PREFIX only
  const float* slopes;    // [H] or null
  int64_t T;
  int H, Hk, N;
  int mask;
  float scale, cap;
};

// A cache and the sequences in it.
struct CacheArgs {
  uint8_t* k;      // e4m3 [pages, Hk, page, 128]
  uint8_t* v;
  float* ks;       // [pages, Hk]
  float* vs;
  int32_t* pos;    // [pages, Hk, page]
  float* weight;   // [pages, Hk, page]
  const int32_t* table;  // [N, width]
  const int32_t* lens;   // [N]
  int pages, page, lg;   // page == 1 << lg
  int Hk, N, width;
};

// cap * tanh(x / cap) * log2 e from one exponential and one reciprocal:
// tanh(y) = 1 - 2 / (1 + e^(2 y)).  x is scale * q . k; c1 = 2 log2 e / cap, c2 = cap log2 e.
// The absolute error is a few 2^-24 of cap log2 e (what an exponent can take),
// which tanh.approx (2^-11 of the result) does not reach.  For caps up to kCapSmall:
// there that moves a weight by 1.5e-5 at most, a thirtieth of its fp16 rounding.
constexpr float kCapSmall = 128.0f;
__device__ __forceinline__ float cap_log2(float x, float c1, float c2) {
  return fmaf(-2.0f * c2, rcp_approx(1.0f + ex2_approx(x * c1)), c2);
}

// The same to a few 2^-24 of the score itself, for larger caps, where that difference
// would cancel: tanh(y) = y (t0 + t1 y^2 + t2 y^4 + t3 y^6) for |y| <= 0.35, fitted for
// the least relative error (3.3e-8; 1.5e-7 with its roundings), and the form above
// beyond, where it is off by 4.5e-7 of the result at most.  per_cap = 1 / cap.
constexpr float kTanhNear = 0.35f;
__device__ constexpr float kTanhRel[4] = {0.99999994f, -0.333324254f, 0.132958218f, -0.0489584431f};
__device__ __forceinline__ float tanh_ratio(float y2) {  // tanh(y) / y
  return fmaf(y2, fmaf(y2, fmaf(y2, kTanhRel[3], kTanhRel[2]), kTanhRel[1]), kTanhRel[0]);
}
__device__ __forceinline__ float cap_log2_large(float x, float per_cap, float c1, float c2) {
  const float y = x * per_cap;
  return fabsf(y) <= kTanhNear ? x * kLog2e * tanh_ratio(y * y) : cap_log2(x, c1, c2);
}

// c1 of cap_log2 for scores that `scale` is still to be multiplied with; finite for the
// smallest caps too, so that a score of 0 stays 0.
__device__ __forceinline__ float cap_exponent(float scale, float cap) {
  const float c1 = scale * (2.0f * kLog2e / cap);
  return fminf(fmaxf(c1, -3e38f), 3e38f);
}

// The cached tokens of sequence n: lens[n], or what its table row can hold (or
// 0) and a latched KDA_ERR_INVALID_ARG if it is outside that, so that no later
// index leaves the tables.
__device__ __forceinline__ int checked_len(const CacheArgs& c, int64_t len, int* err) {
  const int64_t most = static_cast<int64_t>(c.width) << c.lg;
  if (len >= 0 && len <= most) return static_cast<int>(len);
  atomicCAS(err, 0, static_cast<int>(KDA_ERR_INVALID_ARG));
  return static_cast<int>(len < 0 ? 0 : most);
}
__device__ __forceinline__ int cached_len(const CacheArgs& c, int n, int* err) {
  return checked_len(c, __ldg(c.lens + n), err);
}

// Page id of page j of sequence n, or -1 (and a latched KDA_ERR_INVALID_ARG)
// if the table holds none of the pool's pages there.
__device__ __forceinline__ int page_id(const CacheArgs& c, int n, int j, int* err) {
  const int p = __ldg(c.table + static_cast<int64_t>(n) * c.width + j);
  if (p < 0 || p >= c.pages) {
    atomicCAS(err, 0, static_cast<int>(KDA_ERR_INVALID_ARG));
    return -1;
  }
  return p;
}

// Two e4m3 codes -> two fp16 values (exact; the NaN code gives NaN).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
  return r;
}

// Two fp32 -> two e4m3 codes (round to nearest even; lo in the low byte).
__device__ __forceinline__ uint16_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The last n in [0, N) with first(n) <= s, for a function that does not decrease
// (for another, as a malformed cu_seqlens gives, any n: first(n) may be over s);
// 0 if there is none.  All lanes of a warp call it with the same arguments; each
// round tries 32 places, so a thousand sequences take two dependent loads.
template <class F>
__device__ __forceinline__ int warp_search(int N, int64_t s, F first) {
  int lo = 0, hi = N - 1;
  const int lane = threadIdx.x & 31;
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const int64_t at = lo + static_cast<int64_t>(lane + 1) * step;
    const bool below = at <= hi && first(static_cast<int>(at)) <= s;
    const int took = __popc(__ballot_sync(0xffffffffu, below)) * step;
    lo = lo + took < hi ? lo + took : hi;
    hi = hi < lo + step - 1 ? hi : lo + step - 1;
  }
  return lo;
}

// Sequence of slot s where sequence n owns the slots from floor(bos_n / unit) +
// extra * n on.  All lanes of a warp call it.
__device__ __forceinline__ int seq_of_slot(const int32_t* cu, int64_t T, int N, int unit, int extra,
                                           int64_t s) {
  const int64_t per = cu ? 0 : T / N;
  return warp_search(N, s, [&](int n) -> int64_t {
    int64_t bos = cu ? __ldg(cu + n) : n * per;
    bos = bos < 0 ? 0 : (bos > T ? T : bos);
    return bos / unit + static_cast<int64_t>(extra) * n;
  });
}

cudaError_t launch_attn(const AttnArgs& a, int sm_count, int* err, cudaStream_t stream);
cudaError_t launch_cache_append(const CacheArgs& c, const void* k, const void* v,
                                const int32_t* positions, const int32_t* cu, int64_t T, int* err,
                                cudaStream_t stream);
cudaError_t launch_cache_evict(const CacheArgs& c, const int32_t* dst, int dst_width, int budget,
                               int recent, int32_t* new_lens, int32_t* kept, int* err,
                               cudaStream_t stream);

// Queries over a cache.
struct CacheAttnArgs {
  CacheArgs c;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  const int32_t* cu;         // of the query rows
  const int32_t* positions;  // [T] or null
  const float* slopes;       // [H] or null
  int64_t T;
  int H;
  float scale, cap;
  int accumulate;
};
size_t cache_attn_workspace(int64_t T, int H, int Hk, int N, bool cu, int64_t max_len, bool accumulate);
cudaError_t launch_cache_attn(const CacheAttnArgs& a, void* ws, int* err, cudaStream_t stream);

}  // namespace kda
