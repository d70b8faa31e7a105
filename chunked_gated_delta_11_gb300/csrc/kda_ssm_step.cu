// kda_ssm_step.cu -- the state-space recurrence token by token (kda_ssm_step):
//
//   d = softplus(dt + dt_bias),  M = e^(A d) M + d x B^T,  y = M C + skip x,
//
// per sequence and head, with M [P, S] in registers.  A step of one token moves the
// state in and out and computes little, so the bytes of the state bound it.  A CTA has one
// (sequence, head); 16 bytes of a state row to a lane, LR lanes to a row, so every
// access of a warp is whole lines, and a thread's whole share of the state is under way at
// once.  States, products and sums are fp32.
#include "kda_layers.cuh"

namespace kda {

namespace {

// 32 to 64 state values a thread
constexpr int step_threads(int P, int S) { return P * S > 8192 ? 256 : 128; }

template <int P, int S, bool BF16>
__global__ void __launch_bounds__(step_threads(P, S))
step_kernel(SsmArgs a) {
  constexpr int ST_THREADS = step_threads(P, S);
  constexpr int VEC = BF16 ? 8 : 4;          // state values of 16 bytes
  constexpr int LR = S / VEC;                // lanes of a row
  constexpr int RW = 32 / LR;                // rows of a warp's access
  constexpr int NR = P / (RW * (ST_THREADS / 32));  // accesses
  static_assert(LR <= 32 && NR >= 1, "tile");
  grid_dep_wait();
  grid_dep_launch();
  const int h = blockIdx.x % a.H, n = blockIdx.x / a.H;
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  const int row0 = w * RW * NR + l / LR, col = (l % LR) * VEC;  // rows row0 + i * RW
  int64_t bos, eos;
  seq_bounds(a.cu, a.T, a.N, n, bos, eos);
  const int64_t base = (static_cast<int64_t>(n) * a.H + h) * (P * S) + row0 * S + col;
  float m[NR][VEC];
  if (a.init) {
    uint4 raw[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i)
      raw[i] = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.init) + (base + i * RW * S) * (BF16 ? 2 : 4));
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        m[i][e] = BF16 ? __uint_as_float(e & 1 ? u[e >> 1] & 0xffff0000u : u[e >> 1] << 16) : __uint_as_float(u[e & 3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) m[i][e] = 0.f;
  }
  const int g = h / (a.H / a.G);
  const float A = __ldg(a.A + h), bias = a.dt_bias ? __ldg(a.dt_bias + h) : 0.f, skip = a.skip ? __ldg(a.skip + h) : 0.f;
  for (int64_t t = bos; t < eos; ++t) {
    const float d = softplus(__bfloat162float(a.dt[t * a.dt_stride + h]) + bias);
    const float keep = expf(A * d);
    float b[VEC], c[VEC];
    const __nv_bfloat16* bp = a.B + t * a.b_stride + g * S + col;
    const __nv_bfloat16* cp = a.C + t * a.c_stride + g * S + col;
#pragma unroll
    for (int e = 0; e < VEC; e += 4) {
      const uint2 rb = *reinterpret_cast<const uint2*>(bp + e), rc = *reinterpret_cast<const uint2*>(cp + e);
      const uint32_t ub[2] = {rb.x, rb.y}, uc[2] = {rc.x, rc.y};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        b[e + 2 * k] = __uint_as_float(ub[k] << 16);
        b[e + 2 * k + 1] = __uint_as_float(ub[k] & 0xffff0000u);
        c[e + 2 * k] = __uint_as_float(uc[k] << 16);
        c[e + 2 * k + 1] = __uint_as_float(uc[k] & 0xffff0000u);
      }
    }
    float x[NR], y[NR];
    const __nv_bfloat16* xp = a.x + t * a.x_stride + h * P + row0;
#pragma unroll
    for (int i = 0; i < NR; ++i) x[i] = __bfloat162float(xp[i * RW]);
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const float dx = d * x[i];
      y[i] = 0.f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        m[i][e] = fmaf(m[i][e], keep, dx * b[e]);
        y[i] = fmaf(m[i][e], c[e], y[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) {
#pragma unroll
      for (int o = LR / 2; o > 0; o >>= 1) y[i] += __shfl_xor_sync(0xffffffffu, y[i], o);
      if (l % LR == 0) a.out[(t * a.H + h) * P + row0 + i * RW] = __float2bfloat16_rn(fmaf(skip, x[i], y[i]));
    }
  }
  if (!a.fin) return;
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    uint32_t u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) u[k] = BF16 ? pack_bf16(m[i][(2 * k) % VEC], m[i][(2 * k + 1) % VEC]) : __float_as_uint(m[i][k]);
    *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.fin) + (base + i * RW * S) * (BF16 ? 2 : 4)) =
        make_uint4(u[0], u[1], u[2], u[3]);
  }
}

template <int P, int S>
cudaError_t launch(const SsmArgs& a, cudaStream_t stream) {
  const unsigned ctas = static_cast<unsigned>(a.N) * static_cast<unsigned>(a.H);
  const dim3 threads(step_threads(P, S));
  return a.bf16_state ? launch_pdl(step_kernel<P, S, true>, dim3(ctas), threads, 0, stream, a)
                      : launch_pdl(step_kernel<P, S, false>, dim3(ctas), threads, 0, stream, a);
}

}  // namespace

cudaError_t launch_ssm_step(const SsmArgs& a, int P, int S, cudaStream_t stream) {
  if (P == 64) return S == 64 ? launch<64, 64>(a, stream) : launch<64, 128>(a, stream);
  return S == 64 ? launch<128, 64>(a, stream) : launch<128, 128>(a, stream);
}

}  // namespace kda
