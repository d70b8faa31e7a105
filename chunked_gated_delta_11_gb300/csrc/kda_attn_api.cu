// kda_attn_api.cu -- host side of the softmax-attention entry points
// (include/kda.h): argument checks, workspace sizes and launches.
#include <cmath>
#include <cstdint>

#include "kda_attn.cuh"
#include "kda_workspace.cuh"

namespace kda {

kda_status device_info_for_attn(int* sm_count, int** err);

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kMaxElems = static_cast<int64_t>(1) << 40;

kda_status check_rows(int64_t T, int32_t H, int32_t Hk, int32_t N, int32_t D, const int32_t* cu) {
  if (D != KDA_HEAD_DIM) return KDA_ERR_UNSUPPORTED;
  if (T < 0 || H <= 0 || Hk <= 0 || N <= 0 || H % Hk != 0) return KDA_ERR_INVALID_ARG;
  if (H > 65535 || T >= (static_cast<int64_t>(1) << 31)) return KDA_ERR_INVALID_ARG;
  if (T > kMaxElems / (static_cast<int64_t>(H) * D)) return KDA_ERR_INVALID_ARG;
  if (!cu && T % N != 0) return KDA_ERR_INVALID_ARG;
  if (cu && !aligned(cu, 4)) return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

bool good_scores(float scale, float cap, const float* slopes) {
  return std::isfinite(scale) && std::isfinite(cap) && cap >= 0.0f && aligned(slopes, 4);
}

kda_status check_cache(const kda_cache* c) {
  if (!c) return KDA_ERR_INVALID_ARG;
  if (c->D != KDA_HEAD_DIM) return KDA_ERR_UNSUPPORTED;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return KDA_ERR_UNSUPPORTED;
  if (c->pages <= 0 || c->Hk <= 0 || c->Hk > 65535) return KDA_ERR_INVALID_ARG;
  // rows of the pool are int32
  if (static_cast<int64_t>(c->pages) * c->Hk > 0x7fffffffLL / c->page_size) return KDA_ERR_INVALID_ARG;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->pos || !c->weight)
    return KDA_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) ||
      !aligned(c->v_scale, 4) || !aligned(c->pos, 16) || !aligned(c->weight, 16))
    return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

kda_status check_table(const kda_cache* c, const int32_t* table, int32_t width,
                       const int32_t* lens, int32_t N) {
  if (!table || !lens || !aligned(table, 4) || !aligned(lens, 4)) return KDA_ERR_INVALID_ARG;
  if (width <= 0 || N <= 0) return KDA_ERR_INVALID_ARG;
  // slots of a sequence and (sequence, head) units are int32
  if (static_cast<int64_t>(width) * c->page_size > 0x7fffff00LL) return KDA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(N) * c->Hk > 0x7fffffLL) return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

CacheArgs cache_args(const kda_cache* c, const int32_t* table, int32_t width, const int32_t* lens,
                     int32_t N) {
  CacheArgs a{};
  a.k = static_cast<uint8_t*>(c->k);
  a.v = static_cast<uint8_t*>(c->v);
  a.ks = c->k_scale;
  a.vs = c->v_scale;
  a.pos = c->pos;
  a.weight = c->weight;
  a.table = table;
  a.lens = lens;
  a.pages = c->pages;
  a.page = c->page_size;
  a.lg = c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7;
  a.Hk = c->Hk;
  a.N = N;
  a.width = width;
  return a;
}

// The larger need of the two ways to give the sequences (cu_seqlens or equal shares).
size_t cached_need(const kda_cache* c, int64_t T, int H, int N, int64_t max_len, bool accumulate) {
  const size_t a = cache_attn_workspace(T, H, c->Hk, N, true, max_len, accumulate);
  const size_t b = T % N == 0 ? cache_attn_workspace(T, H, c->Hk, N, false, max_len, accumulate) : 0;
  return a > b ? a : b;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status kda_attn_fwd(const kda_attn_options* opts, const void* q, const void* k,
                                   const void* v, float scale, const int32_t* cu_seqlens,
                                   int64_t T_total, int32_t H, int32_t Hk, int32_t N, int32_t D,
                                   void* out, void* stream) {
  if (!opts) return KDA_ERR_INVALID_ARG;
  if (opts->mask < KDA_MASK_FULL || opts->mask > KDA_MASK_PREFIX) return KDA_ERR_INVALID_ARG;
  if ((opts->mask == KDA_MASK_PREFIX) != (opts->prefix_lens != nullptr)) return KDA_ERR_INVALID_ARG;
  if (!aligned(opts->prefix_lens, 4)) return KDA_ERR_INVALID_ARG;
  kda_status s = check_rows(T_total, H, Hk, N, D, cu_seqlens);
  if (s != KDA_OK) return s;
  if (!good_scores(scale, opts->cap, opts->slopes)) return KDA_ERR_INVALID_ARG;
  if (T_total == 0) return KDA_OK;
  if (!q || !k || !v || !out) return KDA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16))
    return KDA_ERR_INVALID_ARG;
  int sms = 0, *err = nullptr;
  if ((s = device_info_for_attn(&sms, &err)) != KDA_OK) return s;
  AttnArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.cu = cu_seqlens;
  a.prefix = opts->prefix_lens;
  a.slopes = opts->slopes;
  a.T = T_total;
  a.H = H;
  a.Hk = Hk;
  a.N = N;
  a.mask = opts->mask;
  a.scale = scale;
  a.cap = opts->cap;
  return launch_attn(a, sms, err, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK
                                                                                    : KDA_ERR_LAUNCH;
}

extern "C" kda_status kda_cache_append(const kda_cache* cache, const void* k, const void* v,
                                       const int32_t* block_table, int32_t table_width,
                                       const int32_t* lens, const int32_t* positions,
                                       const int32_t* cu_seqlens, int64_t T_total, int32_t N,
                                       void* stream) {
  kda_status s = check_cache(cache);
  if (s != KDA_OK) return s;
  if ((s = check_table(cache, block_table, table_width, lens, N)) != KDA_OK) return s;
  if ((s = check_rows(T_total, cache->Hk, cache->Hk, N, cache->D, cu_seqlens)) != KDA_OK) return s;
  if (!aligned(positions, 4)) return KDA_ERR_INVALID_ARG;
  if (T_total == 0) return KDA_OK;
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return KDA_ERR_INVALID_ARG;
  int sms = 0, *err = nullptr;
  if ((s = device_info_for_attn(&sms, &err)) != KDA_OK) return s;
  const CacheArgs c = cache_args(cache, block_table, table_width, lens, N);
  return launch_cache_append(c, k, v, positions, cu_seqlens, T_total, err,
                             static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? KDA_OK
             : KDA_ERR_LAUNCH;
}

extern "C" size_t kda_cache_attn_workspace_size(const kda_cache* cache, int64_t T_total, int32_t H,
                                                int32_t N, int32_t table_width,
                                                int32_t accumulate) {
  if (check_cache(cache) != KDA_OK || table_width <= 0) return 0;
  if (check_rows(T_total, H, cache->Hk, N, cache->D, reinterpret_cast<const int32_t*>(4)) != KDA_OK)
    return 0;
  const int64_t max_len = static_cast<int64_t>(table_width) * cache->page_size;
  if (max_len > 0x7fffff00LL || T_total > 0x7fffffffLL / H) return 0;
  if (T_total == 0) return 0;
  const size_t need = cached_need(cache, T_total, H, N, max_len, accumulate != 0);
  return need == SIZE_MAX ? 0 : need;
}

extern "C" kda_status kda_cache_attn(const kda_cache_attn_options* opts, const kda_cache* cache,
                                     const void* q, float scale, const int32_t* block_table,
                                     int32_t table_width, const int32_t* lens,
                                     const int32_t* cu_seqlens, int64_t T_total, int32_t H,
                                     int32_t N, void* out, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  if (!opts) return KDA_ERR_INVALID_ARG;
  kda_status s = check_cache(cache);
  if (s != KDA_OK) return s;
  if ((s = check_table(cache, block_table, table_width, lens, N)) != KDA_OK) return s;
  if ((s = check_rows(T_total, H, cache->Hk, N, cache->D, cu_seqlens)) != KDA_OK) return s;
  if (!good_scores(scale, opts->cap, opts->slopes) || !aligned(opts->positions, 4))
    return KDA_ERR_INVALID_ARG;
  if (T_total > 0x7fffffffLL / H) return KDA_ERR_INVALID_ARG;  // (token, head) rows are int32
  if (T_total == 0) return KDA_OK;
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16)) return KDA_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const size_t need = cached_need(cache, T_total, H, N,
                                  static_cast<int64_t>(table_width) * cache->page_size,
                                  opts->accumulate != 0);
  if (need == SIZE_MAX) return KDA_ERR_WORKSPACE;  // no device has as much
  if (workspace && (!aligned(workspace, 16) || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
  int sms = 0, *err = nullptr;
  if ((s = device_info_for_attn(&sms, &err)) != KDA_OK) return s;
  Workspace ws(workspace, workspace_bytes, need, st);
  if (!ws.ok()) return KDA_ERR_WORKSPACE;
  CacheAttnArgs a{};
  a.c = cache_args(cache, block_table, table_width, lens, N);
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.cu = cu_seqlens;
  a.positions = opts->positions;
  a.slopes = opts->slopes;
  a.T = T_total;
  a.H = H;
  a.scale = scale;
  a.cap = opts->cap;
  a.accumulate = opts->accumulate != 0;
  return launch_cache_attn(a, ws.get(), err, st) == cudaSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

extern "C" size_t kda_cache_evict_workspace_size(const kda_cache* cache, int32_t N,
                                                 int32_t budget) {
  if (check_cache(cache) != KDA_OK || N <= 0 || budget <= 0) return 0;
  if (static_cast<int64_t>(N) * cache->Hk > 0x7fffffLL) return 0;
  const int64_t bytes = static_cast<int64_t>(N) * cache->Hk * budget * 4;
  return static_cast<size_t>((bytes + 255) & ~static_cast<int64_t>(255));
}

extern "C" kda_status kda_cache_evict(const kda_cache* cache, const int32_t* block_table,
                                      int32_t table_width, const int32_t* lens,
                                      const int32_t* dst_table, int32_t dst_width, int32_t budget,
                                      int32_t recent, int32_t N, int32_t* new_lens,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  kda_status s = check_cache(cache);
  if (s != KDA_OK) return s;
  if ((s = check_table(cache, block_table, table_width, lens, N)) != KDA_OK) return s;
  if (!dst_table || !aligned(dst_table, 4) || dst_width <= 0) return KDA_ERR_INVALID_ARG;
  if (!new_lens || !aligned(new_lens, 4)) return KDA_ERR_INVALID_ARG;
  if (new_lens != lens && new_lens < lens + N && lens < new_lens + N) return KDA_ERR_INVALID_ARG;
  if (budget <= 0 || recent < 0 || recent > budget) return KDA_ERR_INVALID_ARG;
  // a budget beyond the table keeps everything, as one of the table's slots does
  const int32_t slots = table_width * cache->page_size;
  budget = budget < slots ? budget : slots;
  recent = recent < budget ? recent : budget;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const size_t need = kda_cache_evict_workspace_size(cache, N, budget);
  if (workspace && (!aligned(workspace, 16) || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
  int sms = 0, *err = nullptr;
  if ((s = device_info_for_attn(&sms, &err)) != KDA_OK) return s;
  Workspace ws(workspace, workspace_bytes, need, st);
  if (!ws.ok()) return KDA_ERR_WORKSPACE;
  const CacheArgs c = cache_args(cache, block_table, table_width, lens, N);
  return launch_cache_evict(c, dst_table, dst_width, budget, recent, new_lens,
                            static_cast<int32_t*>(ws.get()), err, st) == cudaSuccess
             ? KDA_OK
             : KDA_ERR_LAUNCH;
}
