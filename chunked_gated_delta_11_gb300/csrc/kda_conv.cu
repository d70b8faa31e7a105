// kda_conv.cu -- the short causal convolution before a recurrent layer (kda_conv_fwd):
//
//   y[t, c] = act(bias[c] + sum_{j < W} w[c, j] x[t - W + 1 + j, c]),  act(y) = y sigmoid(y) or y,
//
// where the W - 1 rows before a sequence's first come from its state, and its last W - 1
// rows are the next state.  Products and sums are fp32, the output is rounded once.
//
// A thread has 8 channels (one 16-byte access a row) and walks down a strip of rows with
// the last W - 1 of them in registers, so that a row is read once but for the W - 1 before
// a strip.  A sequence's first W - 1 rows and its two states are a block's of their own
// (a head block): it reads the old state before it writes the new one, so that the two may
// be the same buffer, and a step of one token a sequence is such blocks alone.
#include "kda_attn.cuh"
#include "kda_layers.cuh"

namespace kda {

namespace {

constexpr int CV_THREADS = 128;
constexpr int CV_CHANNELS = CV_THREADS * 8;
constexpr int CV_AHEAD = 8;  // rows under way in a thread

__device__ __forceinline__ void widen(const uint4& r, float (&f)[8]) {
  const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

// The taps and the bias of a thread's 8 channels.
template <int W>
struct Taps {
  float w[8][W], b[8];
  __device__ __forceinline__ void load(const ConvArgs& a, int c) {
#pragma unroll
    for (int k = 0; k < W; ++k) {  // 8 W values, 16 bytes at a time
      float f[8];
      widen(__ldg(reinterpret_cast<const uint4*>(a.w + static_cast<int64_t>(c) * W) + k), f);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[(8 * k + e) / W][(8 * k + e) % W] = f[e];
    }
    if (a.bias) {
      widen(__ldg(reinterpret_cast<const uint4*>(a.bias + c)), b);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) b[e] = 0.f;
    }
  }
  // rows: the W rows that end with the output's own
  __device__ __forceinline__ uint4 output(const uint4 (&rows)[W], bool silu) const {
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = b[e];
#pragma unroll
    for (int j = 0; j < W; ++j) {
      float f[8];
      widen(rows[j], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = fmaf(w[e][j], f[e], y[e]);
    }
    if (silu) {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= sigmoid_fast(y[e]);
    }
    return make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
  }
};

// Rows of a thread's channels, from the input or a state.
__device__ __forceinline__ uint4 row_of(const __nv_bfloat16* base, int64_t stride, int64_t row, int c) {
  return __ldg(reinterpret_cast<const uint4*>(base + row * stride + c));
}

template <int W>
__global__ void __launch_bounds__(CV_THREADS)
conv_kernel(ConvArgs a, int heads, int strip) {
  grid_dep_wait();
  grid_dep_launch();
  const int c = (blockIdx.y * CV_THREADS + threadIdx.x) * 8;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  if (static_cast<int>(blockIdx.x) < heads) {
    const int n = blockIdx.x;
    int64_t bos, eos;
    seq_bounds(a.cu, a.T, a.N, n, bos, eos);
    if (c >= a.C) return;
    const int64_t len = eos - bos, at = static_cast<int64_t>(n) * (W - 1);
    uint4 rows[2 * (W - 1)];  // the old state, then the first rows
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {
      // not the read-only path: the state may be written further down
      rows[r] = a.init ? *reinterpret_cast<const uint4*>(a.init + (at + r) * a.C + c) : zero;
      rows[W - 1 + r] = r < len ? row_of(a.x, a.x_stride, bos + r, c) : zero;
    }
    Taps<W> taps;
    taps.load(a, c);
    if (a.fin) {
#pragma unroll
      for (int r = 0; r < W - 1; ++r) {
        uint4 last = zero;
        if (len >= W - 1) {
          last = row_of(a.x, a.x_stride, eos - (W - 1) + r, c);
        } else {
#pragma unroll
          for (int k = 0; k < 2 * (W - 1); ++k)
            if (k == len + r) last = rows[k];
        }
        *reinterpret_cast<uint4*>(a.fin + (at + r) * a.C + c) = last;
      }
    }
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {
      uint4 in[W];
#pragma unroll
      for (int j = 0; j < W; ++j) in[j] = rows[r + j];
      if (r < len) *reinterpret_cast<uint4*>(a.out + (bos + r) * a.C + c) = taps.output(in, a.silu);
    }
    return;
  }
  const int64_t t0 = static_cast<int64_t>(blockIdx.x - heads) * strip;
  const int64_t t1 = t0 + strip < a.T ? t0 + strip : a.T;
  // the sequence of the strip's first row; cu_seqlens need not cover all rows
  int n = seq_of_slot(a.cu, a.T, a.N, 1, 0, t0);
  int64_t bos, eos;
  seq_bounds(a.cu, a.T, a.N, n, bos, eos);
  if (c >= a.C) return;
  Taps<W> taps;
  bool loaded = false;
  for (int64_t t = t0; t < t1;) {
    while (t >= eos && n + 1 < a.N) seq_bounds(a.cu, a.T, a.N, ++n, bos, eos);
    if (t >= eos) return;  // rows behind the last sequence stay as they are
    // this sequence's rows of the strip, but for its first W - 1
    const int64_t end = eos < t1 ? eos : t1;
    t = t > bos + (W - 1) ? t : bos + (W - 1);
    if (t >= end) {
      t = end;
      continue;
    }
    if (!loaded) taps.load(a, c);
    loaded = true;
    uint4 rows[W - 1 + CV_AHEAD];
#pragma unroll
    for (int r = 0; r < W - 1; ++r) rows[r] = row_of(a.x, a.x_stride, t - (W - 1) + r, c);
    for (; t < end; t += CV_AHEAD) {
#pragma unroll
      for (int r = 0; r < CV_AHEAD; ++r)
        if (t + r < end) rows[W - 1 + r] = row_of(a.x, a.x_stride, t + r, c);
#pragma unroll
      for (int r = 0; r < CV_AHEAD; ++r) {
        uint4 in[W];
#pragma unroll
        for (int j = 0; j < W; ++j) in[j] = rows[r + j];
        if (t + r < end) *reinterpret_cast<uint4*>(a.out + (t + r) * a.C + c) = taps.output(in, a.silu);
      }
#pragma unroll
      for (int r = 0; r < W - 1; ++r) rows[r] = rows[CV_AHEAD + r];
    }
    t = end;
  }
}

template <int W>
cudaError_t launch(const ConvArgs& a, int sm_count, cudaStream_t stream) {
  const int64_t blocks_c = (a.C + CV_CHANNELS - 1) / CV_CHANNELS;
  // strips of 32 rows (3 rows read twice in 32), or of 8 where that leaves the SMs idle
  const int strip = (a.T + 31) / 32 * blocks_c >= 4 * sm_count ? 32 : 8;
  const int64_t blocks = a.N + (a.T + strip - 1) / strip;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_pdl(conv_kernel<W>, dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(blocks_c)),
                    dim3(CV_THREADS), 0, stream, a, a.N, strip);
}

}  // namespace

cudaError_t launch_conv(const ConvArgs& a, int W, int sm_count, cudaStream_t stream) {
  switch (W) {
    case 2: return launch<2>(a, sm_count, stream);
    case 3: return launch<3>(a, sm_count, stream);
    default: return launch<4>(a, sm_count, stream);
  }
}

}  // namespace kda
