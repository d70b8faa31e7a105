// kda_conv.cu -- the short causal convolution before a recurrent layer (kda_conv_fwd):
//
//   y[t, c] = act(bias[c] + sum_{j < W} w[c, j] x[t - W + 1 + j, c]),  act(y) = y sigmoid(y) or y,
//
// where the W - 1 rows before a sequence's first come from its state, and its last W - 1
// rows are the next state.  Products and sums are fp32, the output is rounded once.
//
// A thread has 4 channels (8 bytes a row, whole lines a warp) and walks down a strip of rows
// with the last W - 1 of them in registers, 8 rows under way at a time, so that a row is
// read once but for the W - 1 before a strip.  (With 8 channels a thread the weights and the
// rows took 166 registers, and too few rows were under way: 209 us for the rows below.)  A
// sequence's first W - 1 rows and its two states are a block's of their own (a head block):
// it reads the old state before it writes the new one, so that the two may be the same
// buffer, and a step of one token a sequence is such blocks alone.
#include "kda_attn.cuh"
#include "kda_layers.cuh"
#include "kda_tc.cuh"

namespace kda {

namespace {

constexpr int CV_THREADS = 128;
constexpr int CV_VEC = 4;                        // channels of a thread
constexpr int CV_CHANNELS = CV_THREADS * CV_VEC;
constexpr int CV_AHEAD = 8;                      // rows under way in a thread

// Four channels of a row, in pairs.
struct Row {
  f2 lo, hi;
};
__device__ __forceinline__ Row widen(uint2 r) {
  return {pair(r.x << 16, r.x & 0xffff0000u), pair(r.y << 16, r.y & 0xffff0000u)};
}

__device__ __forceinline__ uint2 row_of(const __nv_bfloat16* base, int64_t stride, int64_t row, int c) {
  return __ldg(reinterpret_cast<const uint2*>(base + row * stride + c));
}

__device__ __forceinline__ uint32_t silu_pair(f2 y, bool silu) {
  float a, b;
  unpair(y, a, b);
  if (silu) {
    a *= sigmoid_fast(a);
    b *= sigmoid_fast(b);
  }
  return pack_bf16(a, b);
}

// The taps and the bias of a thread's channels.
template <int W>
struct Taps {
  Row w[W], b;
  __device__ __forceinline__ void load(const ConvArgs& a, int c) {
    float f[CV_VEC][W];
#pragma unroll
    for (int k = 0; k < W; ++k) {  // 4 W values, 8 bytes at a time
      const uint2 u = __ldg(reinterpret_cast<const uint2*>(a.w + static_cast<int64_t>(c) * W) + k);
      const uint32_t x[2] = {u.x, u.y};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        f[(4 * k + e) / W][(4 * k + e) % W] = __uint_as_float(e & 1 ? x[e >> 1] & 0xffff0000u : x[e >> 1] << 16);
    }
#pragma unroll
    for (int j = 0; j < W; ++j) w[j] = {pair(f[0][j], f[1][j]), pair(f[2][j], f[3][j])};
    b = a.bias ? widen(__ldg(reinterpret_cast<const uint2*>(a.bias + c))) : Row{0ull, 0ull};
  }
  // rows: the W rows that end with the output's own
  __device__ __forceinline__ uint2 output(const Row (&rows)[W], bool silu) const {
    Row y = b;
#pragma unroll
    for (int j = 0; j < W; ++j) y = {fma2(w[j].lo, rows[j].lo, y.lo), fma2(w[j].hi, rows[j].hi, y.hi)};
    return make_uint2(silu_pair(y.lo, silu), silu_pair(y.hi, silu));
  }
};

template <int W>
__global__ void __launch_bounds__(CV_THREADS, 8)
conv_kernel(ConvArgs a, int heads, int strip) {
  grid_dep_wait();
  grid_dep_launch();
  int c = (blockIdx.y * CV_THREADS + threadIdx.x) * CV_VEC;
  if (static_cast<int>(blockIdx.x) < heads) {
    const int n = blockIdx.x;
    int64_t bos, eos;
    seq_bounds(a.cu, a.T, a.N, n, bos, eos);
    if (c >= a.C) return;
    const int64_t len = eos - bos, at = static_cast<int64_t>(n) * (W - 1);
    const uint2 zero = make_uint2(0, 0);
    uint2 rows[2 * (W - 1)];  // the old state, then the first rows
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {
      // not the read-only path: the state may be written further down
      rows[r] = a.init ? *reinterpret_cast<const uint2*>(a.init + (at + r) * a.C + c) : zero;
      rows[W - 1 + r] = r < len ? row_of(a.x, a.x_stride, bos + r, c) : zero;
    }
    Taps<W> taps;
    taps.load(a, c);
    if (a.fin) {
#pragma unroll
      for (int r = 0; r < W - 1; ++r) {
        uint2 last = zero;
        if (len >= W - 1) {
          last = row_of(a.x, a.x_stride, eos - (W - 1) + r, c);
        } else {
#pragma unroll
          for (int k = 0; k < 2 * (W - 1); ++k)
            if (k == len + r) last = rows[k];
        }
        *reinterpret_cast<uint2*>(a.fin + (at + r) * a.C + c) = last;
      }
    }
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {
      Row in[W];
#pragma unroll
      for (int j = 0; j < W; ++j) in[j] = widen(rows[r + j]);
      if (r < len) *reinterpret_cast<uint2*>(a.out + (bos + r) * a.C + c) = taps.output(in, a.silu);
    }
    return;
  }
  const int64_t t0 = static_cast<int64_t>(blockIdx.x - heads) * strip;
  const int64_t t1 = t0 + strip < a.T ? t0 + strip : a.T;
  // the sequence of the strip's first row; cu_seqlens need not cover all rows
  int n = seq_of_slot(a.cu, a.T, a.N, 1, 0, t0);
  int64_t bos, eos;
  seq_bounds(a.cu, a.T, a.N, n, bos, eos);
  // (threads behind the last channel write its values once more: whole warps look for sequences)
  c = c < a.C ? c : a.C - CV_VEC;
  Taps<W> taps;
  bool loaded = false;
  for (int64_t t = t0; t < t1;) {
    if (t >= eos && n + 1 < a.N) seq_bounds(a.cu, a.T, a.N, ++n, bos, eos);
    if (t >= eos && n + 1 < a.N) {  // empty ones between
      const int at = seq_of_slot(a.cu, a.T, a.N, 1, 0, t);
      n = at > n ? at : n + 1;
      seq_bounds(a.cu, a.T, a.N, n, bos, eos);
      if (t >= eos && n + 1 < a.N) continue;  // (a malformed cu_seqlens)
    }
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
    Row in[W];  // the rows before, then the current one
#pragma unroll
    for (int r = 0; r < W - 1; ++r) in[r] = widen(row_of(a.x, a.x_stride, t - (W - 1) + r, c));
    const __nv_bfloat16* x = a.x + t * a.x_stride + c;
    __nv_bfloat16* out = a.out + t * a.C + c;
    for (int left = static_cast<int>(end - t); left > 0; left -= CV_AHEAD) {
      uint2 raw[CV_AHEAD];
#pragma unroll
      for (int r = 0; r < CV_AHEAD; ++r) {
        raw[r] = make_uint2(0, 0);
        if (r < left) raw[r] = __ldg(reinterpret_cast<const uint2*>(x + r * a.x_stride));
      }
#pragma unroll
      for (int r = 0; r < CV_AHEAD; ++r) {
        in[W - 1] = widen(raw[r]);
        const uint2 y = taps.output(in, a.silu);
        if (r < left) *reinterpret_cast<uint2*>(out + static_cast<int64_t>(r) * a.C) = y;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) in[j] = in[j + 1];
      }
      x += CV_AHEAD * a.x_stride;
      out += static_cast<int64_t>(CV_AHEAD) * a.C;
    }
    t = end;
  }
}

template <int W>
cudaError_t launch(const ConvArgs& a, int sm_count, cudaStream_t stream) {
  const int64_t blocks_c = (a.C + CV_CHANNELS - 1) / CV_CHANNELS;
  // strips of 64 rows (3 rows read twice in 64), or of 8 where that leaves the SMs idle
  const int strip = (a.T + 63) / 64 * blocks_c >= 4 * sm_count ? 64 : 8;
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
