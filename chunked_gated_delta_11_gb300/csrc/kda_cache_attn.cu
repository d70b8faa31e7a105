// kda_cache_attn.cu -- attention of a few new tokens per sequence over the
// 8-bit paged cache (kda_cache_attn), and the weights it accumulates.
#include "kda_attn.cuh"

namespace kda {
namespace {

// Position of query token i of `cnt` of sequence n, for the slots of KV head hk:
// given, or counted back from the newest slot.
__device__ __forceinline__ int query_pos(const CacheAttnArgs& a, int n, int hk, int64_t bos, int i,
                                         int cnt, int len, int* err) {
  if (a.positions) return __ldg(a.positions + bos + i);
  if (len == 0) return 0;
  const int pid = page_id(a.c, n, (len - 1) >> a.c.lg, err);
  if (pid < 0) return 0;
  const int64_t b = static_cast<int64_t>(pid) * a.c.Hk + hk;
  return a.c.pos[b * a.c.page + ((len - 1) & (a.c.page - 1))] - (cnt - 1 - i);
}

__device__ __forceinline__ float4 decode4(uint32_t codes) {
  const uint32_t lo = e4m3x2_to_f16x2(static_cast<uint16_t>(codes));
  const uint32_t hi = e4m3x2_to_f16x2(static_cast<uint16_t>(codes >> 16));
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return make_float4(a.x, a.y, b.x, b.y);
}

__device__ __forceinline__ void load_q(const CacheAttnArgs& a, int64_t t, int h, int l, float (&q)[4]) {
  const __nv_bfloat16* p = a.q + (t * a.H + h) * kDim + l * 4;
  for (int i = 0; i < 4; ++i) q[i] = __bfloat162float(p[i]);
}

// Score of the warp's query against slot row r of block b, in log2 units.
__device__ __forceinline__ float score(const CacheAttnArgs& a, const float (&q)[4], int64_t b, int64_t r, int l,
                                       float slope, int gap) {
  const float4 k = decode4(*reinterpret_cast<const uint32_t*>(a.c.k + r * kDim + l * 4));
  float x = q[0] * k.x + q[1] * k.y + q[2] * k.z + q[3] * k.w;
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
  x *= a.c.ks[b] * a.scale;
  x = a.cap > 0.f ? cap_log2(x, 2.f * kLog2e / a.cap, a.cap * kLog2e) : x * kLog2e;
  return x - slope * static_cast<float>(gap);
}

// One warp per (query token, head): the output row, and the log2 of the softmax
// denominator into lse[t * H + h].
__global__ void __launch_bounds__(32) row_kernel(CacheAttnArgs a, float* __restrict__ lse, int* err) {
  const int l = threadIdx.x, h = blockIdx.y;
  const int64_t t = blockIdx.x;
  int n;
  if (a.cu) {
    int lo = 0, hi = a.c.N - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(a.cu + mid) <= t) lo = mid;
      else hi = mid - 1;
    }
    n = lo;
  } else {
    n = static_cast<int>(t / (a.T / a.c.N));
  }
  int64_t bos, eos;
  seq_bounds(a.cu, a.T, a.c.N, n, bos, eos);
  if (t < bos || t >= eos) return;
  const int hk = h / (a.H / a.c.Hk);
  const int len = cached_len(a.c, n, err);
  const int qp = query_pos(a, n, hk, bos, static_cast<int>(t - bos), static_cast<int>(eos - bos), len, err);
  float q[4];
  load_q(a, t, h, l, q);
  const float slope = a.slopes ? __ldg(a.slopes + h) * kLog2e : 0.f;
  float m = -INFINITY, sum = 0.f;
  float o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < len; ++i) {
    const int pid = page_id(a.c, n, i >> a.c.lg, err);
    if (pid < 0) continue;
    const int64_t b = static_cast<int64_t>(pid) * a.c.Hk + hk;
    const int64_t r = b * a.c.page + (i & (a.c.page - 1));
    const int gap = qp - a.c.pos[r];
    if (gap < 0) continue;
    const float x = score(a, q, b, r, l, slope, gap);
    const float4 v = decode4(*reinterpret_cast<const uint32_t*>(a.c.v + r * kDim + l * 4));
    const float mn = fmaxf(m, x), f = ex2_approx(m - mn), p = ex2_approx(x - mn);
    const float pv = p * a.c.vs[b];
    sum = sum * f + p;
    o[0] = o[0] * f + pv * v.x;
    o[1] = o[1] * f + pv * v.y;
    o[2] = o[2] * f + pv * v.z;
    o[3] = o[3] * f + pv * v.w;
    m = mn;
  }
  const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
  *reinterpret_cast<uint2*>(a.out + (t * a.H + h) * kDim + l * 4) =
      make_uint2(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv));
  if (lse && l == 0) lse[t * a.H + h] = m + log2f(sum);
}

// One warp per (slot, sequence, KV head): the weights of the slot, summed over
// the query rows of the head in order and added to the cache once.
__global__ void __launch_bounds__(32) weight_kernel(CacheAttnArgs a, const float* __restrict__ lse, int* err) {
  const int l = threadIdx.x, hk = blockIdx.y % a.c.Hk, n = blockIdx.y / a.c.Hk;
  const int len = cached_len(a.c, n, err), i = blockIdx.x;
  if (i >= len) return;
  int64_t bos, eos;
  seq_bounds(a.cu, a.T, a.c.N, n, bos, eos);
  const int pid = page_id(a.c, n, i >> a.c.lg, err);
  if (pid < 0) return;
  const int64_t b = static_cast<int64_t>(pid) * a.c.Hk + hk;
  const int64_t r = b * a.c.page + (i & (a.c.page - 1));
  const int group = a.H / a.c.Hk;
  float w = 0.f;
  for (int64_t t = bos; t < eos; ++t) {
    const int gap = query_pos(a, n, hk, bos, static_cast<int>(t - bos), static_cast<int>(eos - bos), len, err) - a.c.pos[r];
    if (gap < 0) continue;
    for (int h = hk * group; h < (hk + 1) * group; ++h) {
      float q[4];
      load_q(a, t, h, l, q);
      w += ex2_approx(score(a, q, b, r, l, a.slopes ? __ldg(a.slopes + h) * kLog2e : 0.f, gap) - lse[t * a.H + h]);
    }
  }
  if (l == 0) a.c.weight[r] += w;
}

}  // namespace

size_t cache_attn_workspace(int64_t T, int H, int Hk, int N, int64_t max_len, bool accumulate) {
  (void)Hk;
  (void)N;
  (void)max_len;
  return accumulate ? static_cast<size_t>(T) * H * 4 : 0;
}

cudaError_t launch_cache_attn(const CacheAttnArgs& a, void* ws, int sm_count, int* err,
                              cudaStream_t stream) {
  (void)sm_count;
  float* lse = static_cast<float*>(ws);
  row_kernel<<<dim3(static_cast<unsigned>(a.T), a.H), 32, 0, stream>>>(a, lse, err);
  if (a.accumulate)
    weight_kernel<<<dim3(static_cast<unsigned>(a.c.width) << a.c.lg, a.c.N * a.c.Hk), 32, 0, stream>>>(a, lse, err);
  return cudaGetLastError();
}

}  // namespace kda
