// kda_layers.cuh -- arguments of the recurrent layers' other operators (the short
// causal convolution and the state-space recurrence) and of the page tables of the
// attention layers' cache.
#pragma once

#include "kda.h"
#include "kda_common.cuh"

namespace kda {

// Causal convolution over packed rows.
struct ConvArgs {
  const __nv_bfloat16* x;     // [T, C], rows x_stride apart
  const __nv_bfloat16* w;     // [C, W]
  const __nv_bfloat16* bias;  // [C] or null
  const __nv_bfloat16* init;  // [N, W - 1, C] or null
  __nv_bfloat16* out;         // [T, C]
  __nv_bfloat16* fin;         // [N, W - 1, C] or null
  const int32_t* cu;
  int64_t T, x_stride;
  int C, N;
  int silu;
};
cudaError_t launch_conv(const ConvArgs& a, int W, int sm_count, cudaStream_t stream);

// State-space recurrence over packed rows.  P channels a head, S values a channel's state.
struct SsmArgs {
  const __nv_bfloat16* x;   // [T, H, P]
  const __nv_bfloat16* dt;  // [T, H]
  const __nv_bfloat16* B;   // [T, G, S]
  const __nv_bfloat16* C;   // [T, G, S]
  const float* A;           // [H]
  const float* skip;        // [H] or null
  const float* dt_bias;     // [H] or null
  const void* init;         // [N, H, P, S] or null
  void* fin;                // [N, H, P, S] or null
  __nv_bfloat16* out;       // [T, H, P]
  const int32_t* cu;
  int64_t T, x_stride, dt_stride, b_stride, c_stride;  // elements between tokens
  int H, G, N;
  int bf16_state;
};
cudaError_t launch_ssm_step(const SsmArgs& a, int P, int S, cudaStream_t stream);
size_t ssm_workspace(int64_t T, int H, int G, int N, int P, int S);
cudaError_t launch_ssm_fwd(const SsmArgs& a, int P, int S, void* ws, int* err, cudaStream_t stream);

// log(1 + e^v), the step size of a token; no branch, so that several are under way at once
__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.f) + log1pf(__expf(-fabsf(v))); }

// Pages of a cache: what sequences take and give back.
struct PagesArgs {
  int32_t* table;        // [N, width]
  const int32_t* lens;   // [N]
  const int32_t* other;  // [N]: new rows (reserve), slots to keep or null (release)
  int32_t* free_pages;   // [pages]
  const int32_t* free_count;
  int32_t* new_free_count;
  int32_t* new_lens;     // [N]
  int32_t* cu;           // [N + 1]
  int64_t* slots;        // [T] or null
  int64_t T;
  int width, lg, N, pages;
};
constexpr int kPagesMaxN = 16384;
cudaError_t launch_reserve(const PagesArgs& a, int* err, cudaStream_t stream);
cudaError_t launch_release(const PagesArgs& a, int* err, cudaStream_t stream);

}  // namespace kda
