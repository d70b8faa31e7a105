// kda_layers_api.cu -- host side of the short convolution, the state-space recurrence and
// the cache's page tables (include/kda.h): argument checks and launches.
#include <cstdint>

#include "kda_layers.cuh"
#include "kda_workspace.cuh"

namespace kda {

kda_status device_info_for_attn(int* sm_count, int** err);

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kMaxElems = static_cast<int64_t>(1) << 40;
constexpr int64_t kMaxSpan = static_cast<int64_t>(1) << 60;  // elements between a tensor's ends

kda_status check_packing(int64_t T, int32_t N, const int32_t* cu) {
  if (T < 0 || T >= (static_cast<int64_t>(1) << 31) || N <= 0) return KDA_ERR_INVALID_ARG;
  if (!cu && T % N != 0) return KDA_ERR_INVALID_ARG;
  return aligned(cu, 4) ? KDA_OK : KDA_ERR_INVALID_ARG;
}

// T rows of `row` elements, `stride` apart (0: one after the other).
bool good_stride(int64_t& stride, int64_t T, int64_t row, int64_t unit) {
  if (stride == 0) stride = row;
  return stride >= row && stride <= kMaxElems && T <= kMaxSpan / stride && stride % unit == 0;
}

// Bytes [p, p + bytes) and [q, q + more) have some in common.
bool overlap(const void* p, int64_t bytes, const void* q, int64_t more) {
  if (!p || !q || bytes <= 0 || more <= 0) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + static_cast<uintptr_t>(more) && b < a + static_cast<uintptr_t>(bytes);
}

// Written arrays lie apart from the others (and from one another), but for those pairs that may be one.
struct Range {
  const void* at;
  int64_t bytes;
};
bool apart(const Range& w, const Range* others, int n) {
  for (int i = 0; i < n; ++i)
    if (overlap(w.at, w.bytes, others[i].at, others[i].bytes)) return false;
  return true;
}

int64_t span(int64_t T, int64_t stride, int64_t row) { return T > 0 ? ((T - 1) * stride + row) * 2 : 0; }

// A state that is updated in place, or two that lie apart.
bool good_states(const void* init, const void* fin, int64_t bytes) {
  return aligned(init, 16) && aligned(fin, 16) && (init == fin || !overlap(init, bytes, fin, bytes));
}

constexpr int64_t kMaxMapStride = static_cast<int64_t>(1) << 39;  // elements of 2 bytes between a tensor map's rows
constexpr int64_t kSsmMaxT = (static_cast<int64_t>(1) << 31) - 128;  // a chunk's end is an int32 too

kda_status check_ssm_sizes(int64_t T, int32_t H, int32_t G, int32_t N, int32_t P, int32_t S) {
  if ((P != 64 && P != 128) || (S != 64 && S != 128)) return KDA_ERR_UNSUPPORTED;
  if (H <= 0 || G <= 0 || H % G != 0 || H > 65535) return KDA_ERR_INVALID_ARG;
  if (T < 0 || T >= (static_cast<int64_t>(1) << 31) || N <= 0) return KDA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(N) * H > 0x7fffffLL) return KDA_ERR_INVALID_ARG;
  if (T > kMaxElems / (static_cast<int64_t>(H) * P)) return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

kda_status check_ssm(const kda_ssm_options* o, const void* x, const void* dt, const float* A, const void* B,
                     const void* C, const void* init, const int32_t* cu, int64_t T, int32_t H, int32_t G, int32_t N,
                     int32_t P, int32_t S, void* out, void* fin, const void* ws, int64_t need, SsmArgs& a) {
  if (!o) return KDA_ERR_INVALID_ARG;
  kda_status s = check_ssm_sizes(T, H, G, N, P, S);
  if (s == KDA_OK) s = check_packing(T, N, cu);
  if (s != KDA_OK) return s;
  if (o->state_dtype != KDA_STATE_F32 && o->state_dtype != KDA_STATE_BF16) return KDA_ERR_INVALID_ARG;
  a = SsmArgs{};
  a.x_stride = o->x_stride;
  a.dt_stride = o->dt_stride;
  a.b_stride = o->b_stride;
  a.c_stride = o->c_stride;
  const int64_t row = static_cast<int64_t>(H) * P, wide = static_cast<int64_t>(G) * S;
  if (!good_stride(a.x_stride, T, row, 8) || !good_stride(a.dt_stride, T, H, 1) ||
      !good_stride(a.b_stride, T, wide, 8) || !good_stride(a.c_stride, T, wide, 8))
    return KDA_ERR_INVALID_ARG;
  if (!A || !aligned(A, 4) || !aligned(o->skip, 4) || !aligned(o->dt_bias, 4)) return KDA_ERR_INVALID_ARG;
  const int64_t state = static_cast<int64_t>(N) * H * P * S * (o->state_dtype == KDA_STATE_BF16 ? 2 : 4);
  if (!good_states(init, fin, state)) return KDA_ERR_INVALID_ARG;
  if (T > 0) {
    if (!x || !dt || !B || !C || !out) return KDA_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(dt, 2) || !aligned(B, 16) || !aligned(C, 16) || !aligned(out, 16))
      return KDA_ERR_INVALID_ARG;
  }
  // inputs, then the initial state and what is written (also the workspace: need == 0 where there is none)
  const Range all[] = {{x, span(T, a.x_stride, row)}, {dt, span(T, a.dt_stride, H)}, {B, span(T, a.b_stride, wide)},
                       {C, span(T, a.c_stride, wide)}, {A, H * 4LL}, {o->skip, H * 4LL}, {o->dt_bias, H * 4LL},
                       {cu, (N + 1LL) * 4}, {init, state}, {fin, state}, {out, T * row * 2}};
  if (!apart(all[9], all, 8) || !apart(all[10], all, 10) || !apart({ws, need}, all, 11)) return KDA_ERR_INVALID_ARG;
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.dt = static_cast<const __nv_bfloat16*>(dt);
  a.B = static_cast<const __nv_bfloat16*>(B);
  a.C = static_cast<const __nv_bfloat16*>(C);
  a.A = A;
  a.skip = o->skip;
  a.dt_bias = o->dt_bias;
  a.init = init;
  a.fin = fin;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.cu = cu;
  a.T = T;
  a.H = H;
  a.G = G;
  a.N = N;
  a.bf16_state = o->state_dtype == KDA_STATE_BF16;
  return KDA_OK;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status kda_conv_fwd(const kda_conv_options* opts, const void* x, const void* weight,
                                   const void* bias, const void* initial_state,
                                   const int32_t* cu_seqlens, int64_t T_total, int32_t C, int32_t W,
                                   int32_t N, void* out, void* final_state, void* stream) {
  if (!opts) return KDA_ERR_INVALID_ARG;
  if (W < 2 || W > 4 || C % 8 != 0) return KDA_ERR_UNSUPPORTED;
  if (C <= 0) return KDA_ERR_INVALID_ARG;
  kda_status s = check_packing(T_total, N, cu_seqlens);
  if (s != KDA_OK) return s;
  if (T_total > kMaxElems / C || N > kMaxElems / C) return KDA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(C) > 65535LL * 512) return KDA_ERR_INVALID_ARG;  // blocks of 512 channels
  if (static_cast<int64_t>(N) + T_total / 8 + 1 > 0x7fffffffLL) return KDA_ERR_INVALID_ARG;
  int64_t stride = opts->x_stride;
  if (!good_stride(stride, T_total, C, 8)) return KDA_ERR_INVALID_ARG;
  if (!weight || !aligned(weight, 16) || !aligned(bias, 16)) return KDA_ERR_INVALID_ARG;
  const int64_t state = static_cast<int64_t>(N) * (W - 1) * C * 2, bytes = T_total * C * 2;
  if (!good_states(initial_state, final_state, state)) return KDA_ERR_INVALID_ARG;
  if (T_total > 0 && (!x || !out || !aligned(x, 16) || !aligned(out, 16))) return KDA_ERR_INVALID_ARG;
  const Range all[] = {{x, span(T_total, stride, C)}, {weight, C * 2LL * W}, {bias, C * 2LL}, {cu_seqlens, (N + 1LL) * 4},
                       {initial_state, state}, {final_state, state}, {out, bytes}};
  if (!apart(all[5], all, 4) || !apart(all[6], all, 6)) return KDA_ERR_INVALID_ARG;
  int sms = 0, *err = nullptr;
  if ((s = device_info_for_attn(&sms, &err)) != KDA_OK) return s;
  ConvArgs a{};
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.w = static_cast<const __nv_bfloat16*>(weight);
  a.bias = static_cast<const __nv_bfloat16*>(bias);
  a.init = static_cast<const __nv_bfloat16*>(initial_state);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.fin = static_cast<__nv_bfloat16*>(final_state);
  a.cu = cu_seqlens;
  a.T = T_total;
  a.x_stride = stride;
  a.C = C;
  a.N = N;
  a.silu = opts->silu != 0;
  return launch_conv(a, W, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

extern "C" kda_status kda_ssm_step(const kda_ssm_options* opts, const void* x, const void* dt,
                                   const float* A, const void* B, const void* C,
                                   const void* initial_state, const int32_t* cu_seqlens,
                                   int64_t T_total, int32_t H, int32_t G, int32_t N, int32_t P,
                                   int32_t S, void* out, void* final_state, void* stream) {
  SsmArgs a;
  const kda_status s = check_ssm(opts, x, dt, A, B, C, initial_state, cu_seqlens, T_total, H, G, N, P, S, out,
                                 final_state, nullptr, 0, a);
  if (s != KDA_OK) return s;
  return launch_ssm_step(a, P, S, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

extern "C" size_t kda_ssm_workspace_size(int64_t T_total, int32_t H, int32_t G, int32_t N, int32_t P, int32_t S) {
  if (check_ssm_sizes(T_total, H, G, N, P, S) != KDA_OK || T_total >= kSsmMaxT) return 0;
  return ssm_workspace(T_total, H, G, N, P, S);
}

extern "C" kda_status kda_ssm_fwd(const kda_ssm_options* opts, const void* x, const void* dt, const float* A,
                                  const void* B, const void* C, const void* initial_state,
                                  const int32_t* cu_seqlens, int64_t T_total, int32_t H, int32_t G,
                                  int32_t N, int32_t P, int32_t S, void* out, void* final_state,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  SsmArgs a;
  const size_t need = kda_ssm_workspace_size(T_total, H, G, N, P, S);
  if (workspace && (!aligned(workspace, 16) || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
  kda_status s = check_ssm(opts, x, dt, A, B, C, initial_state, cu_seqlens, T_total, H, G, N, P, S, out, final_state,
                           workspace, static_cast<int64_t>(need), a);
  if (s != KDA_OK) return s;
  if (T_total >= kSsmMaxT) return KDA_ERR_INVALID_ARG;
  if (a.x_stride >= kMaxMapStride || a.b_stride >= kMaxMapStride || a.c_stride >= kMaxMapStride) return KDA_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  int sms = 0, *err = nullptr;
  if ((s = device_info_for_attn(&sms, &err)) != KDA_OK) return s;
  Workspace ws(workspace, workspace_bytes, need, st);
  if (!ws.ok()) return KDA_ERR_WORKSPACE;
  return launch_ssm_fwd(a, P, S, ws.get(), err, st) == cudaSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

namespace {

// What kda_cache_reserve and kda_cache_release have in common.
kda_status check_pages(const int32_t* table, int32_t width, const int32_t* lens, const int32_t* free_pages,
                       const int32_t* free_count, int32_t pages, int32_t page_size, int32_t N,
                       const int32_t* new_free_count) {
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) return KDA_ERR_UNSUPPORTED;
  if (N > kPagesMaxN) return KDA_ERR_UNSUPPORTED;
  if (width <= 0 || N <= 0 || pages < 0) return KDA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(width) * page_size > 0x7fffff00LL) return KDA_ERR_INVALID_ARG;
  if (!table || !lens || (pages > 0 && !free_pages) || !free_count || !new_free_count) return KDA_ERR_INVALID_ARG;
  if (!aligned(table, 4) || !aligned(lens, 4) || !aligned(free_pages, 4) || !aligned(free_count, 4) ||
      !aligned(new_free_count, 4))
    return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

int log2_of(int32_t page_size) { return page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7; }

}  // namespace

extern "C" kda_status kda_cache_reserve(int32_t* block_table, int32_t table_width, const int32_t* lens,
                                        const int32_t* new_rows, const int32_t* free_pages,
                                        const int32_t* free_count, int32_t pages, int32_t page_size,
                                        int64_t T_total, int32_t N, int32_t* new_lens,
                                        int32_t* cu_seqlens, int64_t* slots, int32_t* new_free_count,
                                        void* stream) {
  kda_status s = check_pages(block_table, table_width, lens, free_pages, free_count, pages, page_size, N, new_free_count);
  if (s != KDA_OK) return s;
  if (T_total < 0 || T_total > 0x7fffffffLL) return KDA_ERR_INVALID_ARG;
  if (!new_rows || !new_lens || !cu_seqlens || !aligned(new_rows, 4) || !aligned(new_lens, 4) || !aligned(cu_seqlens, 4) ||
      !aligned(slots, 16))
    return KDA_ERR_INVALID_ARG;
  const int64_t n4 = static_cast<int64_t>(N) * 4;
  const Range table{block_table, n4 * table_width}, old{lens, n4}, add{new_rows, n4}, list{free_pages, pages * 4LL},
      count{free_count, 4}, fresh{new_lens, n4}, sums{cu_seqlens, n4 + 4}, places{slots, T_total * 8}, left{new_free_count, 4};
  const Range in_table[] = {old, add, list, count, fresh, sums, places, left};
  const Range in_fresh[] = {add, list, count, sums, places, left, new_lens == lens ? Range{} : old};
  const Range in_sums[] = {old, add, list, count, places, left};
  const Range in_places[] = {old, add, list, count, left};
  const Range in_left[] = {old, add, list, new_free_count == free_count ? Range{} : count};
  if (!apart(table, in_table, 8) || !apart(fresh, in_fresh, 7) || !apart(sums, in_sums, 6) || !apart(places, in_places, 5) ||
      !apart(left, in_left, 4))
    return KDA_ERR_INVALID_ARG;
  int sms = 0, *err = nullptr;
  if ((s = device_info_for_attn(&sms, &err)) != KDA_OK) return s;
  PagesArgs a{};
  a.table = block_table;
  a.lens = lens;
  a.other = new_rows;
  a.free_pages = const_cast<int32_t*>(free_pages);
  a.free_count = free_count;
  a.new_free_count = new_free_count;
  a.new_lens = new_lens;
  a.cu = cu_seqlens;
  a.slots = slots;
  a.T = T_total;
  a.width = table_width;
  a.lg = log2_of(page_size);
  a.N = N;
  a.pages = pages;
  return launch_reserve(a, err, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

extern "C" kda_status kda_cache_release(const int32_t* block_table, int32_t table_width, const int32_t* lens,
                                        const int32_t* keep, int32_t* free_pages, const int32_t* free_count,
                                        int32_t pages, int32_t page_size, int32_t N,
                                        int32_t* new_free_count, void* stream) {
  kda_status s = check_pages(block_table, table_width, lens, free_pages, free_count, pages, page_size, N, new_free_count);
  if (s != KDA_OK) return s;
  if (!aligned(keep, 4)) return KDA_ERR_INVALID_ARG;
  const int64_t n4 = static_cast<int64_t>(N) * 4;
  const Range table{block_table, n4 * table_width}, old{lens, n4}, kept{keep, n4}, list{free_pages, pages * 4LL},
      count{free_count, 4}, left{new_free_count, 4};
  const Range in_list[] = {table, old, kept, count, left};
  const Range in_left[] = {table, old, kept, new_free_count == free_count ? Range{} : count};
  if (!apart(list, in_list, 5) || !apart(left, in_left, 4)) return KDA_ERR_INVALID_ARG;
  int sms = 0, *err = nullptr;
  if ((s = device_info_for_attn(&sms, &err)) != KDA_OK) return s;
  PagesArgs a{};
  a.table = const_cast<int32_t*>(block_table);
  a.lens = lens;
  a.other = keep;
  a.free_pages = free_pages;
  a.free_count = free_count;
  a.new_free_count = new_free_count;
  a.width = table_width;
  a.lg = log2_of(page_size);
  a.N = N;
  a.pages = pages;
  return launch_release(a, err, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}
