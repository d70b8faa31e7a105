// kda_attn.cu -- softmax attention over packed rows (kda_attn_fwd).
//
// One warp per (token, head): the four channels of a lane in registers, the
// visible keys one after the other with a running maximum and sum.
#include "kda_attn.cuh"

namespace kda {
namespace {

__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 b = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xffff0000u),
                     __uint_as_float(b.y << 16), __uint_as_float(b.y & 0xffff0000u));
}

__global__ void __launch_bounds__(128) attn_kernel(AttnArgs a) {
  const int l = threadIdx.x & 31;
  const int h = blockIdx.y;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (t >= a.T) return;
  int64_t bos = 0, eos = 0;
  int n = 0;
  if (a.cu) {
    int lo = 0, hi = a.N - 1;  // last sequence that starts at or before t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(a.cu + mid) <= t) lo = mid;
      else hi = mid - 1;
    }
    n = lo;
  } else {
    n = static_cast<int>(t / (a.T / a.N));
  }
  seq_bounds(a.cu, a.T, a.N, n, bos, eos);
  if (t < bos || t >= eos) return;
  int64_t end = eos;
  if (a.mask != KDA_MASK_FULL) {
    end = t + 1;
    if (a.mask == KDA_MASK_PREFIX) {
      const int64_t p = bos + __ldg(a.prefix + n);
      end = p > end ? (p < eos ? p : eos) : end;
    }
  }
  const int64_t row = (t * a.H + h) * kDim + l * 4;
  const float4 q = load4(a.q + row);
  const float slope = a.slopes ? __ldg(a.slopes + h) * kLog2e : 0.f;
  const int hk = h / (a.H / a.Hk);
  float m = -INFINITY, sum = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int64_t j = bos; j < end; ++j) {
    const int64_t at = (j * a.Hk + hk) * kDim + l * 4;
    const float4 k = load4(a.k + at), v = load4(a.v + at);
    float x = q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
    x *= a.scale;
    x = a.cap > 0.f ? cap_log2(x, 2.f * kLog2e / a.cap, a.cap * kLog2e) : x * kLog2e;
    x -= slope * fabsf(static_cast<float>(t - j));
    const float mn = fmaxf(m, x), r = ex2_approx(m - mn), p = ex2_approx(x - mn);
    sum = sum * r + p;
    o.x = o.x * r + p * v.x;
    o.y = o.y * r + p * v.y;
    o.z = o.z * r + p * v.z;
    o.w = o.w * r + p * v.w;
    m = mn;
  }
  const float inv = 1.f / sum;
  *reinterpret_cast<uint2*>(a.out + row) =
      make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
}

}  // namespace

cudaError_t launch_attn(const AttnArgs& a, int sm_count, int* err, cudaStream_t stream) {
  (void)sm_count;
  (void)err;
  attn_kernel<<<dim3(static_cast<unsigned>((a.T + 3) / 4), a.H), 128, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace kda
