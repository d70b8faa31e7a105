// kda_cache.cu -- writing the 8-bit paged key/value cache: append and evict.
//
// A page holds `page` token slots of every KV head; the slots of one (page,
// head) are one block of page x 128 e4m3 codes with one fp32 scale, for keys
// and for values each.  The value of a code is code * scale.
//
// append: a block's scale is 2^e, e the smallest exponent in [-64, 120] with
//   amax <= 448 * 2^e over the finite new values of the block, and at least
//   what the block's older rows had.  Powers of two make the division exact, so
//   a value is rounded once, and re-rounding older rows when the scale grows
//   loses only what drops below the smallest code.  A non-finite value becomes
//   the NaN code and stays out of the scale: it spoils its own row only.
// evict: per (sequence, head), the newest `recent` slots stay, and of the
//   others the budget - recent of largest weight (ties: the lowest slot), in
//   their old order, packed into other pages.  A packed block's scale is the
//   largest block scale among its rows, so no value can overflow.
//
// Both are bound by memory: append reads 2 bytes and writes 1 per element,
// evict reads one weight per slot and moves 2 x 128 codes per kept slot.
// Measured (GB300, replayed from a graph): append of 32 ragged prompts (62,700
// tokens, 8 heads) 67 us = 5.8 TB/s, of 256 single tokens 3.8 us; eviction of 64
// ragged sequences to 4096 slots 37 us for the selection and 171 us for the packing,
// 5.6 TB/s of rows of 128 bytes that lie anywhere; of one sequence 11 us.
#include "kda_attn.cuh"

namespace kda {
namespace {

constexpr int kScaleMin = -64, kScaleMax = 120;

// exponent e of the block scale for a largest magnitude `amax` (finite, >= 0)
__device__ __forceinline__ float block_scale(float amax) {
  const uint32_t b = __float_as_uint(amax);
  // amax = m 2^x, 1 <= m < 2: 448 = 1.75 * 2^8
  int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = e < kScaleMin ? kScaleMin : (e > kScaleMax ? kScaleMax : e);
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

__device__ __forceinline__ float finite_or_nan(float x) {
  return fabsf(x) < INFINITY ? x : __uint_as_float(0x7fffffffu);
}

// largest finite magnitude of 2 bf16 values, and their codes
__device__ __forceinline__ float amax2(uint32_t w) {
  const float lo = fabsf(__uint_as_float(w << 16)), hi = fabsf(__uint_as_float(w & 0xffff0000u));
  return fmaxf(lo < INFINITY ? lo : 0.f, hi < INFINITY ? hi : 0.f);
}
// CHECK: non-finite values become NaN.
template <bool CHECK = true>
__device__ __forceinline__ uint32_t encode2(uint32_t w, float inv) {
  const float lo = __uint_as_float(w << 16), hi = __uint_as_float(w & 0xffff0000u);
  return f32x2_to_e4m3x2((CHECK ? finite_or_nan(lo) : lo) * inv, (CHECK ? finite_or_nan(hi) : hi) * inv);
}
// The larger magnitudes, two bf16 at a time as integers (their order is the same).
__device__ __forceinline__ uint32_t larger2(uint32_t m, const uint4& x) {
  m = __vmaxu2(m, x.x & 0x7fff7fffu);
  m = __vmaxu2(m, x.y & 0x7fff7fffu);
  m = __vmaxu2(m, x.z & 0x7fff7fffu);
  return __vmaxu2(m, x.w & 0x7fff7fffu);
}
__device__ __forceinline__ float amax8(const uint4& x) {
  return fmaxf(fmaxf(amax2(x.x), amax2(x.y)), fmaxf(amax2(x.z), amax2(x.w)));
}
template <bool CHECK>
__device__ __forceinline__ uint2 encode8(const uint4& x, float inv) {
  return make_uint2(encode2<CHECK>(x.x, inv) | (encode2<CHECK>(x.y, inv) << 16),
                    encode2<CHECK>(x.z, inv) | (encode2<CHECK>(x.w, inv) << 16));
}

// 4 codes times `ratio`, rounded to codes again
__device__ __forceinline__ uint32_t rescale4(uint32_t codes, float ratio) {
  uint32_t r[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t h = e4m3x2_to_f16x2(static_cast<uint16_t>(codes >> (16 * i)));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    r[i] = f32x2_to_e4m3x2(f.x * ratio, f.y * ratio);
  }
  return r[0] | (r[1] << 16);
}

__device__ __forceinline__ uint4 rescale16(const uint4& x, float ratio) {
  return make_uint4(rescale4(x.x, ratio), rescale4(x.y, ratio), rescale4(x.z, ratio), rescale4(x.w, ratio));
}

// A page that gets rows: its id, its rows [lo, hi) that are new, the sequence slot
// of its row 0, and the input row that goes to row lo.
struct Touched {
  int pid, lo, hi;
  int64_t first, row0;
};

// Page slot s of the list in which sequence n owns the slots from floor(bos_n /
// page) + 2 n on (r new rows touch at most floor(r / page) + 2 pages).  False if
// there is no such page.  The same for all threads of a warp.
template <int PAGE>
__device__ __forceinline__ bool touched_page(const CacheArgs& c, const int32_t* cu, int64_t T,
                                             int64_t s, int* err, Touched& p) {
  const int n = seq_of_slot(cu, T, c.N, PAGE, 2, s);
  int64_t bos, eos;
  seq_bounds(cu, T, c.N, n, bos, eos);
  const int64_t len = cached_len(c, n, err), most = static_cast<int64_t>(c.width) * PAGE;
  const int64_t fresh = eos - bos;
  int64_t end = len + fresh;
  if (end > most) {
    atomicCAS(err, 0, static_cast<int>(KDA_ERR_INVALID_ARG));
    end = most;
  }
  const int64_t ahead = s - (bos / PAGE + 2 * static_cast<int64_t>(n));
  const int64_t pj = len / PAGE + ahead;
  p.first = pj * PAGE;
  // (a malformed cu_seqlens can give a slot before its sequence's first; behind a negative
  // length, which cached_len reports, there is no place)
  if (fresh == 0 || ahead < 0 || p.first >= end || __ldg(c.lens + n) < 0) return false;
  p.pid = page_id(c, n, static_cast<int>(pj), err);
  p.lo = static_cast<int>(len > p.first ? len - p.first : 0);
  p.hi = static_cast<int>(end - p.first < PAGE ? end - p.first : PAGE);
  p.row0 = bos + p.first + p.lo - len;
  return p.pid >= 0;
}

// A CTA per (page that gets rows, KV head) for its keys and one for its values: what
// bounds it is the latency of lookups, rows, maximum and codes one after the other, and
// with one of the two a thread's rows are few enough registers for 6 CTAs per SM (both in
// one CTA, 4 per SM: 84 us where this takes 67).  A row is 16 threads of 8 elements; the
// new rows stay in registers between the maximum and the codes.
template <int PAGE>
__global__ void __launch_bounds__(256)
append_kernel(CacheArgs c, const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v,
              const int32_t* __restrict__ positions, const int32_t* __restrict__ cu, int64_t T,
              int* __restrict__ err) {
  constexpr int PASSES = PAGE / 16;
  __shared__ uint32_t red[8];
  grid_dep_wait();
  grid_dep_launch();
  const int t = threadIdx.x, sub = t & 15, row0 = t >> 4, h = blockIdx.y;
  const bool values = blockIdx.z;
  Touched pg;
  if (!touched_page<PAGE>(c, cu, T, blockIdx.x, err, pg)) return;
  const int lo = pg.lo, hi = pg.hi;
  const int64_t block = static_cast<int64_t>(pg.pid) * c.Hk + h;
  const __nv_bfloat16* from = (values ? v : k) + (pg.row0 * c.Hk + h) * kDim + sub * 8;
  float* scale = (values ? c.vs : c.ks) + block;

  uint4 x[PASSES];
  uint32_t m = 0u;  // largest magnitudes, two bf16 at a time as integers
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int r = p * 16 + row0;
    x[p] = make_uint4(0, 0, 0, 0);
    if (r >= lo && r < hi) x[p] = *reinterpret_cast<const uint4*>(from + static_cast<int64_t>(r - lo) * c.Hk * kDim);
  }
#pragma unroll
  for (int p = 0; p < PASSES; ++p) m = larger2(m, x[p]);
  m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
  if ((t & 31) == 0) red[t >> 5] = m;
  const float old = lo > 0 ? *scale : 0.f;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, red[i]);
  const bool finite = m < 0x7f80u;  // the same for the CTA
  if (!finite) {
    // infinities or NaN among the rows: the largest finite value, after all
    float most = 0.f;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) most = fmaxf(most, amax8(x[p]));
    __syncthreads();
    const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
    if ((t & 31) == 0) red[t >> 5] = bits >> 16;
    __syncthreads();
    m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, red[i]);
  }
  const float s = fmaxf(block_scale(__uint_as_float(m << 16)), old), inv = 1.0f / s;
  uint8_t* to = (values ? c.v : c.k) + block * (PAGE * kDim) + sub * 8;
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int r = p * 16 + row0;
    if (r >= lo && r < hi) {
      *reinterpret_cast<uint2*>(to + r * kDim) = finite ? encode8<false>(x[p], inv) : encode8<true>(x[p], inv);
    } else if (r < lo && s != old) {
      uint2* at = reinterpret_cast<uint2*>(to + r * kDim);
      const uint2 y = *at;
      *at = make_uint2(rescale4(y.x, old * inv), rescale4(y.y, old * inv));
    }
  }
  if (!values && t >= lo && t < hi) {
    c.pos[block * PAGE + t] = positions ? __ldg(positions + pg.row0 + t - lo) : static_cast<int32_t>(pg.first + t);
    c.weight[block * PAGE + t] = 0.f;
  }
  // the old scale was read before the barrier above
  if (t == 0) *scale = s;
}

// The same for few new rows (serving steps): a warp per (page, KV head), 8 heads
// of a page per CTA.  A lane has 4 channels of a row; rows are read twice.
template <int PAGE>
__global__ void __launch_bounds__(256)
append_few_kernel(CacheArgs c, const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v,
                  const int32_t* __restrict__ positions, const int32_t* __restrict__ cu, int64_t T,
                  int* __restrict__ err) {
  grid_dep_wait();
  grid_dep_launch();
  const int l = threadIdx.x & 31, h = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (h >= c.Hk) return;
  Touched p;
  if (!touched_page<PAGE>(c, cu, T, blockIdx.x, err, p)) return;
  const int64_t block = static_cast<int64_t>(p.pid) * c.Hk + h;
  const float oldk = p.lo > 0 ? c.ks[block] : 0.f, oldv = p.lo > 0 ? c.vs[block] : 0.f;
  const int64_t at0 = (p.row0 * c.Hk + h) * kDim + l * 4, step = static_cast<int64_t>(c.Hk) * kDim;
  const int rows = p.hi - p.lo;
  float mk = 0.f, mv = 0.f;
  for (int i = 0; i < rows; ++i) {
    const uint2 x = *reinterpret_cast<const uint2*>(k + at0 + i * step);
    const uint2 y = *reinterpret_cast<const uint2*>(v + at0 + i * step);
    mk = fmaxf(mk, fmaxf(amax2(x.x), amax2(x.y)));
    mv = fmaxf(mv, fmaxf(amax2(y.x), amax2(y.y)));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, o));
    mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, o));
  }
  const float sk = fmaxf(block_scale(mk), oldk), sv = fmaxf(block_scale(mv), oldv);
  const float ik = 1.0f / sk, iv = 1.0f / sv;
  uint8_t* dk = c.k + block * (PAGE * kDim);
  uint8_t* dv = c.v + block * (PAGE * kDim);
  for (int i = 0; i < rows; ++i) {
    const uint2 x = *reinterpret_cast<const uint2*>(k + at0 + i * step);
    const uint2 y = *reinterpret_cast<const uint2*>(v + at0 + i * step);
    *reinterpret_cast<uint32_t*>(dk + (p.lo + i) * kDim + l * 4) = encode2(x.x, ik) | (encode2(x.y, ik) << 16);
    *reinterpret_cast<uint32_t*>(dv + (p.lo + i) * kDim + l * 4) = encode2(y.x, iv) | (encode2(y.y, iv) << 16);
  }
  // older rows under a grown scale, 16 codes a lane
  auto again = [&](uint8_t* d, float ratio) {
    for (int e = l; e < p.lo * 8; e += 32) {
      uint4* q = reinterpret_cast<uint4*>(d) + e;
      *q = rescale16(*q, ratio);
    }
  };
  if (p.lo > 0 && sk != oldk) again(dk, oldk * ik);
  if (p.lo > 0 && sv != oldv) again(dv, oldv * iv);
  for (int i = l; i < rows; i += 32) {
    c.pos[block * PAGE + p.lo + i] = positions ? __ldg(positions + p.row0 + i) : static_cast<int32_t>(p.first + p.lo + i);
    c.weight[block * PAGE + p.lo + i] = 0.f;
  }
  if (l == 0) {
    c.ks[block] = sk;
    c.vs[block] = sv;
  }
}

// Order-preserving integer key of a weight; NaN above everything, -0 equal to 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t b = __float_as_uint(w + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

constexpr int SEL_THREADS = 512;
constexpr int SEL_BINS = 2048;
constexpr int SEL_KEYS = 32768;  // keys that a CTA can hold
constexpr int SEL_SMEM = SEL_KEYS * 4;
constexpr int SEL_MAX_CLUSTER = 8;
constexpr int SEL_GROUPS = SEL_BINS / 32;
static_assert(SEL_GROUPS * SEL_MAX_CLUSTER == SEL_THREADS, "one word of the cluster's sums a thread");

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// Word at `local` (this CTA's shared memory) in the CTA of `rank`.
__device__ __forceinline__ uint32_t cluster_load(const uint32_t* local, unsigned rank) {
  uint32_t at, x;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(local)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(at));
  return x;
}

__device__ __forceinline__ uint32_t sum8(uint32_t x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  x += __shfl_xor_sync(0xffffffffu, x, 2);
  return x + __shfl_xor_sync(0xffffffffu, x, 4);
}
// One warp: `a` and `b` are the counts of digits top - 2 lane and top - 2 lane - 1;
// finds the digit with the need-th slot from the top, and which of the digit's it is.
__device__ __forceinline__ void pick_digit(uint32_t a, uint32_t b, uint32_t need, int top, uint32_t* pick) {
  const int l = threadIdx.x & 31;
  uint32_t sum = a + b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, sum, o);
    if (l >= o) sum += x;
  }
  const uint32_t above = sum - a - b;
  if (above < need && need <= above + a) {
    pick[0] = top - 2 * l;
    pick[1] = need - above;
  } else if (above + a < need && need <= sum) {
    pick[0] = top - 2 * l - 1;
    pick[1] = need - above - a;
  }
}

// The rows (block * page + slot in it, -1: bad page) of the kept slots of one
// (sequence, head), in order, into kept[unit * budget]: a
// radix selection finds the key of the last slot to be kept (three passes of 11,
// 11 and 10 bits), then one ordered pass writes the slots.  A cluster of CTAs
// shares a unit, each with a stretch of its slots, whose keys stay in shared
// memory (the first SEL_KEYS of them; the rest are read again); the histograms
// and counts are summed through distributed shared memory.  What bounds it is the
// latency of the passes, so few long sequences get the largest cluster.
__global__ void __launch_bounds__(SEL_THREADS, 2)
select_kernel(CacheArgs c, int budget, int recent, int cluster, int32_t* __restrict__ kept,
              int* __restrict__ err) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ uint32_t hist[2][SEL_BINS];  // alternate, so that a pass can be cleared while others read the last
  __shared__ uint32_t coarse[2][SEL_GROUPS];  // sums of 32 bins of each
  __shared__ uint32_t totals[SEL_GROUPS];     // over the cluster
  __shared__ uint32_t warp_n[32];
  __shared__ uint32_t pick[2];   // digit chosen, how many of its slots are still to be kept
  __shared__ uint32_t count[2];  // this CTA's slots above and at the last key
  grid_dep_wait();
  grid_dep_launch();
  const int t = threadIdx.x, l = t & 31, w = t >> 5;
  const int unit = blockIdx.x / static_cast<unsigned>(cluster);
  const unsigned rank = cluster > 1 ? cluster_rank() : 0u;
  const int n = unit / c.Hk, h = unit - n * c.Hk;
  const int len = cached_len(c, n, err);
  int32_t* list = kept + static_cast<int64_t>(unit) * budget;
  auto row_of = [&](int slot) -> int {
    const int pid = page_id(c, n, slot >> c.lg, err);
    return pid < 0 ? -1 : ((pid * c.Hk + h) << c.lg) + (slot & (c.page - 1));
  };
  // the newest, or everything (the same for the whole cluster)
  const int old = len <= budget ? 0 : len - recent, want = len <= budget ? 0 : budget - recent;
  for (int i = rank * SEL_THREADS + t; i < len - old; i += cluster * SEL_THREADS) list[want + i] = row_of(old + i);
  if (want == 0) return;
  const int share = ((old + cluster - 1) / cluster + 3) & ~3;
  const int begin = old < static_cast<int>(rank) * share ? old : static_cast<int>(rank) * share;
  const int mine = old - begin < share ? old - begin : share;
  // keys of the 4 slots from i on (a multiple of 4: one page; those past `mine` are
  // the page's own, and not used)
  auto read4 = [&](int i) -> uint4 {
    const int pid = page_id(c, n, (begin + i) >> c.lg, err);
    if (pid < 0) return make_uint4(0u, 0u, 0u, 0u);
    const float4 x = __ldg(reinterpret_cast<const float4*>(
        c.weight + (static_cast<int64_t>(pid) * c.Hk + h) * c.page + ((begin + i) & (c.page - 1))));
    return make_uint4(weight_key(x.x), weight_key(x.y), weight_key(x.z), weight_key(x.w));
  };
  auto keys4 = [&](int i) -> uint4 { return i < SEL_KEYS ? *reinterpret_cast<const uint4*>(keys + i) : read4(i); };
  for (int i = t; i < 2 * SEL_BINS; i += SEL_THREADS) (&hist[0][0])[i] = 0;
  // 4 groups of 4 slots a thread at a time: table entries, then weights, then keys
  for (int i0 = 4 * t; i0 < mine && i0 < SEL_KEYS; i0 += 16 * SEL_THREADS) {
    int id[4];
    float4 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + j * 4 * SEL_THREADS;
      id[j] = i < mine && i < SEL_KEYS ? __ldg(c.table + static_cast<int64_t>(n) * c.width + ((begin + i) >> c.lg)) : -1;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + j * 4 * SEL_THREADS;
      if (id[j] >= 0 && id[j] < c.pages)
        x[j] = __ldg(reinterpret_cast<const float4*>(
            c.weight + (static_cast<int64_t>(id[j]) * c.Hk + h) * c.page + ((begin + i) & (c.page - 1))));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + j * 4 * SEL_THREADS;
      if (i >= mine || i >= SEL_KEYS) continue;
      const bool good = id[j] >= 0 && id[j] < c.pages;
      if (!good) atomicCAS(err, 0, static_cast<int>(KDA_ERR_INVALID_ARG));
      *reinterpret_cast<uint4*>(keys + i) =
          good ? make_uint4(weight_key(x[j].x), weight_key(x[j].y), weight_key(x[j].z), weight_key(x[j].w)) : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  if (t < 2) count[t] = 0;
  __syncthreads();
  uint32_t last = 0, need = static_cast<uint32_t>(want);
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int bins = pass == 2 ? 1024 : 2048;
    uint32_t* hs = hist[pass & 1];
    const uint32_t mask = pass == 0 ? 0u : 0xffffffffu << (shift + (pass == 1 ? 11 : 10));
    for (int i = 4 * t; i < mine; i += 4 * SEL_THREADS) {
      const uint4 k = keys4(i);
      const uint32_t key[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e < mine && (key[e] & mask) == last) atomicAdd(&hs[(key[e] >> shift) & (bins - 1)], 1u);
    }
    __syncthreads();
    // The digit of the last kept slot in two steps, groups of 32 bins and then the
    // group's own: of the other CTAs' histograms (all of them would be 57 KB) only 64
    // sums and 32 bins are read, one word a thread.
    uint32_t* cs = coarse[pass & 1];
#pragma unroll
    for (int i = 0; i < SEL_GROUPS * 32 / SEL_THREADS; ++i) {
      const int g = w * (SEL_GROUPS * 32 / SEL_THREADS) + i;
      const uint32_t x = __reduce_add_sync(0xffffffffu, hs[g * 32 + l]);
      if (l == 0) cs[g] = x;
    }
    __syncthreads();
    if (cluster > 1) cluster_sync_all();
    // lanes t & 7 of group SEL_GROUPS - 1 - t / 8: the CTAs
    const unsigned r = t & 7;
    uint32_t x = r == rank ? cs[SEL_GROUPS - 1 - (t >> 3)]
                 : r < static_cast<unsigned>(cluster) ? cluster_load(&cs[SEL_GROUPS - 1 - (t >> 3)], r) : 0u;
    x = sum8(x);
    if (r == 0) totals[t >> 3] = x;
    __syncthreads();
    if (w == 0) pick_digit(totals[2 * l], totals[2 * l + 1], need, SEL_GROUPS - 1, pick);
    __syncthreads();
    const int group = pick[0] * 32;
    const uint32_t rest = pick[1];
    x = 0u;
    if (t < 256) {
      const uint32_t* at = &hs[group + 31 - (t >> 3)];
      x = r == rank ? *at : r < static_cast<unsigned>(cluster) ? cluster_load(at, r) : 0u;
    }
    x = sum8(x);
    __syncthreads();
    if (r == 0 && t < 256) totals[t >> 3] = x;
    __syncthreads();
    if (w == 0) pick_digit(l < 16 ? totals[2 * l] : 0u, l < 16 ? totals[2 * l + 1] : 0u, rest, 31, pick);
    __syncthreads();
    last |= static_cast<uint32_t>(group) << shift;
    last |= pick[0] << shift;
    need = pick[1];
    // the last pass uses hist[0] again: the others read it before this pass's barrier
    if (pass == 1)
      for (int i = t; i < SEL_BINS; i += SEL_THREADS) hist[0][i] = 0;
    __syncthreads();
  }
  // keep the slots with key > last, and the first `need` with key == last
  uint32_t above0 = 0, ties0 = 0;  // in the stretches of lower ranks
  if (cluster > 1) {
    uint32_t g = 0, e = 0;
    for (int i = 4 * t; i < mine; i += 4 * SEL_THREADS) {
      const uint4 k = keys4(i);
      const uint32_t key[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        g += i + j < mine && key[j] > last;
        e += i + j < mine && key[j] == last;
      }
    }
    g = __reduce_add_sync(0xffffffffu, g);
    e = __reduce_add_sync(0xffffffffu, e);
    if (l == 0) {
      atomicAdd(&count[0], g);
      atomicAdd(&count[1], e);
    }
    __syncthreads();
    cluster_sync_all();
    uint32_t theirs[SEL_MAX_CLUSTER - 1][2];
#pragma unroll
    for (unsigned r = 0; r < SEL_MAX_CLUSTER - 1; ++r)
#pragma unroll
      for (int i = 0; i < 2; ++i) theirs[r][i] = r < rank ? cluster_load(&count[i], r) : 0u;
#pragma unroll
    for (unsigned r = 0; r < SEL_MAX_CLUSTER - 1; ++r) {
      above0 += theirs[r][0];
      ties0 += theirs[r][1];
    }
    cluster_sync_all();  // nobody leaves while its counts are read
  }
  // 4 slots a thread; (slots above, ties) of a stretch packed as 16 + 16 bits
  uint32_t ties = ties0, base = above0;  // before the stretch: ties met, slots above
  for (int i0 = 0; i0 < mine; i0 += 4 * SEL_THREADS) {
    const int i = i0 + 4 * t;
    uint32_t above4 = 0, tie4 = 0, own = 0;
    if (i < mine) {
      const uint4 k = keys4(i);
      const uint32_t key[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        above4 |= (i + j < mine && key[j] > last ? 1u : 0u) << j;
        tie4 |= (i + j < mine && key[j] == last ? 1u : 0u) << j;
      }
      own = (__popc(above4) << 16) | __popc(tie4);
    }
    uint32_t sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, sum, o);
      if (l >= o) sum += x;
    }
    if (l == 31) warp_n[w] = sum;
    __syncthreads();
    uint32_t all = l < SEL_THREADS / 32 ? warp_n[l] : 0u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, all, o);
      if (l >= o) all += x;
    }
    const uint32_t total = __shfl_sync(0xffffffffu, all, 31);
    const uint32_t before = (w ? __shfl_sync(0xffffffffu, all, w - 1) : 0u) + sum - own;
    uint32_t g = base + (before >> 16), e = ties + (before & 0xffffu);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool gt = above4 >> j & 1u, eq = tie4 >> j & 1u;
      if (gt || (eq && e < need)) list[g + (e < need ? e : need)] = row_of(begin + i + j);
      g += gt;
      e += eq;
    }
    base += total >> 16;
    ties += total & 0xffffu;
    __syncthreads();
  }
}

// A warp per (destination page, sequence, head), 4 pages of a unit per CTA: gathers
// the page's rows, 8 lanes a row, 4 groups of 4 rows under way at a time.  What
// bounds it is how many bytes are in flight, so the chain of lookups before the
// rows (length, kept row) is short and shared by a whole page.  SPLIT = 4: the 4
// warps share a page, for calls with fewer pages than warps that fit the GPU.  64 registers
// a thread for 32 warps per SM: pages of 64 and 128 spill some (316 and 672 bytes loaded).
template <int PAGE, int SPLIT>
__global__ void __launch_bounds__(128, 8)
pack_kernel(CacheArgs c, const int32_t* __restrict__ dst, int dst_width, int budget,
            const int32_t* __restrict__ kept, int32_t* new_lens, int* __restrict__ err) {
  constexpr int LOOKS = (PAGE + 31) / 32;  // rows a lane looks up: lane, lane + 32, ..
  constexpr int GROUPS = PAGE / 4 / SPLIT;  // of 4 rows: the warp's part, + SPLIT, ..
  constexpr int BATCH = GROUPS < 4 ? GROUPS : 4;
  grid_dep_wait();
  grid_dep_launch();
  const int l = threadIdx.x & 31, unit = blockIdx.x;
  const int n = unit / static_cast<unsigned>(c.Hk), h = unit - n * c.Hk;
  const int len = checked_len(c, c.lens[n], err), now = len < budget ? len : budget;
  const int w = threadIdx.x >> 5, part = SPLIT == 1 ? 0 : w;
  const int step = gridDim.y * (4 / SPLIT);
  for (int j = blockIdx.y * (4 / SPLIT) + (SPLIT == 1 ? w : 0); static_cast<int64_t>(j) * PAGE < now; j += step) {
    const int first = j * PAGE;
    const int rows = now - first < PAGE ? now - first : PAGE;
    int from[LOOKS];  // source row (block * PAGE + row), -1: none
#pragma unroll
    for (int i = 0; i < LOOKS; ++i) {
      const int r = l + 32 * i;
      from[i] = r < rows ? __ldg(kept + static_cast<int64_t>(unit) * budget + first + r) : -1;
    }
    const int dp = j < dst_width ? __ldg(dst + static_cast<int64_t>(n) * dst_width + j) : -1;
    if (dp < 0 || dp >= c.pages) {
      if (l == 0) atomicCAS(err, 0, static_cast<int>(KDA_ERR_INVALID_ARG));
      continue;
    }
    const int64_t block = static_cast<int64_t>(dp) * c.Hk + h;
    float fk[LOOKS], fv[LOOKS], mk = 0.f, mv = 0.f;
#pragma unroll
    for (int i = 0; i < LOOKS; ++i) {
      fk[i] = from[i] < 0 ? 0.f : c.ks[from[i] / PAGE];
      fv[i] = from[i] < 0 ? 0.f : c.vs[from[i] / PAGE];
      mk = fmaxf(mk, fk[i]);
      mv = fmaxf(mv, fv[i]);
    }
    const uint8_t* ck = c.k + (l & 7) * 16;
    const uint8_t* cv = c.v + (l & 7) * 16;
#pragma unroll
    for (int g0 = 0; g0 < GROUPS; g0 += BATCH) {
      if (g0 * SPLIT * 4 >= rows) break;
      uint4 a[BATCH], b[BATCH];
      int sr[BATCH];
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const int r = 4 * ((g0 + i) * SPLIT + part) + (l >> 3);  // looked up by lane r & 31
        sr[i] = __shfl_sync(0xffffffffu, from[4 * (g0 + i) * SPLIT / 32], r & 31);
        if (sr[i] >= 0) {
          a[i] = *reinterpret_cast<const uint4*>(ck + static_cast<int64_t>(sr[i]) * kDim);
          b[i] = *reinterpret_cast<const uint4*>(cv + static_cast<int64_t>(sr[i]) * kDim);
        }
      }
      if (g0 == 0) {
        // the maxima are not negative: their order is that of their bits
        mk = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mk)));
        mv = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mv)));
#pragma unroll
        for (int i = 0; i < LOOKS; ++i) {
          fk[i] = fk[i] == mk ? 1.f : fk[i] / mk;
          fv[i] = fv[i] == mv ? 1.f : fv[i] / mv;
        }
      }
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const int r = 4 * ((g0 + i) * SPLIT + part) + (l >> 3);
        const float rk = __shfl_sync(0xffffffffu, fk[4 * (g0 + i) * SPLIT / 32], r & 31);
        const float rv = __shfl_sync(0xffffffffu, fv[4 * (g0 + i) * SPLIT / 32], r & 31);
        if (sr[i] < 0) continue;
        if (rk != 1.f) a[i] = rescale16(a[i], rk);
        if (rv != 1.f) b[i] = rescale16(b[i], rv);
        const int64_t to = (block * PAGE + r) * kDim + (l & 7) * 16;
        *reinterpret_cast<uint4*>(c.k + to) = a[i];
        *reinterpret_cast<uint4*>(c.v + to) = b[i];
      }
    }
#pragma unroll
    for (int i = 0; i < LOOKS; ++i) {
      if (from[i] < 0 || part != 0) continue;
      c.pos[block * PAGE + l + 32 * i] = c.pos[from[i]];
      c.weight[block * PAGE + l + 32 * i] = c.weight[from[i]];
    }
    if (l == 0 && part == 0) {
      c.ks[block] = mk;
      c.vs[block] = mv;
    }
  }
  // new_lens may be lens: here, where every reader comes to the same `now` from either value
  // (the selection, whose CTAs would not, is over)
  if (h == 0 && blockIdx.y == 0 && threadIdx.x == 0) new_lens[n] = now;
}

template <int PAGE>
cudaError_t launch_pack(const CacheArgs& c, const int32_t* dst, int dst_width, int budget,
                        const int32_t* kept, int32_t* new_lens, int* err, cudaStream_t stream) {
  // pages that the kept rows can need, whatever the destination table's width
  const int64_t most = static_cast<int64_t>(c.width) << c.lg;
  const int64_t rows = budget < most ? budget : most;
  const int64_t pages = (rows + PAGE - 1) / PAGE;
  const unsigned units = static_cast<unsigned>(c.N) * static_cast<unsigned>(c.Hk);
  const bool split = pages * units < kSMs * 24;  // of the 32 warps (64 registers) that an SM holds
  const int64_t y = split ? pages : (pages + 3) / 4;
  return launch_pdl(split ? pack_kernel<PAGE, 4> : pack_kernel<PAGE, 1>,
                    dim3(units, static_cast<unsigned>(y < 65535 ? y : 65535)), dim3(128), 0, stream, c, dst, dst_width,
                    budget, kept, new_lens, err);
}

template <int PAGE>
cudaError_t append_page(const CacheArgs& c, const void* k, const void* v, const int32_t* positions,
                        const int32_t* cu, int64_t T, int* err, cudaStream_t stream) {
  const int64_t slots = T / PAGE + 2 * static_cast<int64_t>(c.N);
  if (slots > 0x7fffffffLL) return cudaErrorInvalidValue;
  // A few rows per sequence leave most of a CTA's threads idle: a warp does them (8 heads; 256
  // sequences of 1 row 3.9 us, of 4 rows 5.5 us, with a CTA each 25 us; where all of it fits
  // the GPU at once a warp's rows take longer: 8 sequences of 4 rows 3.6 and 2.6 us).
  const bool few = T <= 4 * static_cast<int64_t>(c.N);
  const dim3 grid(static_cast<unsigned>(slots), static_cast<unsigned>(few ? (c.Hk + 7) / 8 : c.Hk), few ? 1 : 2);
  return launch_pdl(few ? append_few_kernel<PAGE> : append_kernel<PAGE>, grid, dim3(256), 0, stream, c,
                    static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v), positions, cu,
                    T, err);
}

}  // namespace

cudaError_t launch_cache_append(const CacheArgs& c, const void* k, const void* v,
                                const int32_t* positions, const int32_t* cu, int64_t T, int* err,
                                cudaStream_t stream) {
  switch (c.page) {
    case 16: return append_page<16>(c, k, v, positions, cu, T, err, stream);
    case 32: return append_page<32>(c, k, v, positions, cu, T, err, stream);
    case 64: return append_page<64>(c, k, v, positions, cu, T, err, stream);
    default: return append_page<128>(c, k, v, positions, cu, T, err, stream);
  }
}

cudaError_t launch_cache_evict(const CacheArgs& c, const int32_t* dst, int dst_width, int budget,
                               int recent, int32_t* new_lens, int32_t* kept, int* err,
                               cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(select_kernel), SEL_SMEM, done);
  if (e != cudaSuccess) return e;
  const unsigned units = static_cast<unsigned>(c.N) * static_cast<unsigned>(c.Hk);
  const int64_t most = static_cast<int64_t>(c.width) << c.lg;
  // CTAs per unit: up to 8 while that leaves SMs idle and gives each 2048 slots
  int cluster = 1;
  while (cluster < SEL_MAX_CLUSTER && units * 2u * cluster <= 2u * kSMs && most > 4096LL * cluster) cluster *= 2;
  const int64_t share = ((most + cluster - 1) / cluster + 3) & ~3LL;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(units * cluster);
  cfg.blockDim = dim3(SEL_THREADS);
  cfg.dynamicSmemBytes = static_cast<size_t>(share < SEL_KEYS ? share : SEL_KEYS) * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if ((e = cudaLaunchKernelEx(&cfg, select_kernel, c, budget, recent, cluster, kept, err)) != cudaSuccess)
    return e;
  switch (c.page) {
    case 16: return launch_pack<16>(c, dst, dst_width, budget, kept, new_lens, err, stream);
    case 32: return launch_pack<32>(c, dst, dst_width, budget, kept, new_lens, err, stream);
    case 64: return launch_pack<64>(c, dst, dst_width, budget, kept, new_lens, err, stream);
    default: return launch_pack<128>(c, dst, dst_width, budget, kept, new_lens, err, stream);
  }
}

}  // namespace kda
