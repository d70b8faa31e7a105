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

// largest finite magnitude of 8 bf16 values
__device__ __forceinline__ float amax8(const uint4& x) {
  float m = 0.f;
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = fabsf(__uint_as_float(w[i] << 16));
    const float hi = fabsf(__uint_as_float(w[i] & 0xffff0000u));
    // fmaxf drops NaN; infinities are left out here
    m = fmaxf(m, lo < INFINITY ? lo : 0.f);
    m = fmaxf(m, hi < INFINITY ? hi : 0.f);
  }
  return m;
}

__device__ __forceinline__ float finite_or_nan(float x) {
  return fabsf(x) < INFINITY ? x : __uint_as_float(0x7fffffffu);
}

// 8 bf16 values -> 8 codes of value * inv
__device__ __forceinline__ uint2 encode8(const uint4& x, float inv) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t r[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t c[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float lo = finite_or_nan(__uint_as_float(w[2 * i + j] << 16));
      const float hi = finite_or_nan(__uint_as_float(w[2 * i + j] & 0xffff0000u));
      c[j] = f32x2_to_e4m3x2(lo * inv, hi * inv);
    }
    r[i] = c[0] | (c[1] << 16);
  }
  return make_uint2(r[0], r[1]);
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

// One CTA per (page that gets rows, KV head).  Its page is slot blockIdx.x of
// the list in which sequence n owns the slots from floor(bos_n / page) + 2 n on:
// n new rows touch at most floor(n / page) + 2 pages.  A row is 16 threads of 8
// elements; the new rows stay in registers between the maximum and the codes.
template <int PAGE>
__global__ void __launch_bounds__(256)
append_kernel(CacheArgs c, const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v,
              const int32_t* __restrict__ positions, const int32_t* __restrict__ cu, int64_t T,
              int* __restrict__ err) {
  constexpr int PASSES = PAGE / 16;
  __shared__ float red[2][8];
  const int t = threadIdx.x, sub = t & 15, row0 = t >> 4, h = blockIdx.y;
  const int64_t slot = blockIdx.x;
  const int n = seq_of_slot(cu, T, c.N, PAGE, 2, slot);
  int64_t bos, eos;
  seq_bounds(cu, T, c.N, n, bos, eos);
  const int64_t len = cached_len(c, n, err), most = static_cast<int64_t>(c.width) * PAGE;
  const int64_t fresh = eos - bos;
  int64_t end = len + fresh;
  if (end > most) {
    if (t == 0) atomicCAS(err, 0, static_cast<int>(KDA_ERR_INVALID_ARG));
    end = most;
  }
  const int64_t pj = len / PAGE + (slot - (bos / PAGE + 2 * static_cast<int64_t>(n)));
  if (fresh == 0 || pj * PAGE >= end) return;
  const int pid = page_id(c, n, static_cast<int>(pj), err);
  if (pid < 0) return;
  const int64_t first = pj * PAGE;  // sequence slot of the page's row 0
  const int lo = static_cast<int>(len > first ? len - first : 0);
  const int hi = static_cast<int>(end - first < PAGE ? end - first : PAGE);
  const int64_t block = static_cast<int64_t>(pid) * c.Hk + h;

  uint4 xk[PASSES], xv[PASSES];
  float mk = 0.f, mv = 0.f;
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int r = p * 16 + row0;
    xk[p] = xv[p] = make_uint4(0, 0, 0, 0);
    if (r >= lo && r < hi) {
      const int64_t at = ((bos + first + r - len) * c.Hk + h) * kDim + sub * 8;
      xk[p] = *reinterpret_cast<const uint4*>(k + at);
      xv[p] = *reinterpret_cast<const uint4*>(v + at);
      mk = fmaxf(mk, amax8(xk[p]));
      mv = fmaxf(mv, amax8(xv[p]));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, o));
    mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, o));
  }
  if ((t & 31) == 0) {
    red[0][t >> 5] = mk;
    red[1][t >> 5] = mv;
  }
  const float oldk = lo > 0 ? c.ks[block] : 0.f, oldv = lo > 0 ? c.vs[block] : 0.f;
  __syncthreads();
  mk = mv = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    mk = fmaxf(mk, red[0][i]);
    mv = fmaxf(mv, red[1][i]);
  }
  const float sk = fmaxf(block_scale(mk), oldk), sv = fmaxf(block_scale(mv), oldv);
  const float ik = 1.0f / sk, iv = 1.0f / sv;
  uint8_t* dk = c.k + block * (PAGE * kDim) + sub * 8;
  uint8_t* dv = c.v + block * (PAGE * kDim) + sub * 8;
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int r = p * 16 + row0;
    if (r >= lo && r < hi) {
      *reinterpret_cast<uint2*>(dk + r * kDim) = encode8(xk[p], ik);
      *reinterpret_cast<uint2*>(dv + r * kDim) = encode8(xv[p], iv);
    } else if (r < lo) {
      if (sk != oldk) {
        uint2* at = reinterpret_cast<uint2*>(dk + r * kDim);
        const uint2 x = *at;
        *at = make_uint2(rescale4(x.x, oldk * ik), rescale4(x.y, oldk * ik));
      }
      if (sv != oldv) {
        uint2* at = reinterpret_cast<uint2*>(dv + r * kDim);
        const uint2 x = *at;
        *at = make_uint2(rescale4(x.x, oldv * iv), rescale4(x.y, oldv * iv));
      }
    }
  }
  if (t >= lo && t < hi) {
    const int64_t row = first + t - len;
    c.pos[block * PAGE + t] = positions ? __ldg(positions + bos + row) : static_cast<int32_t>(first + t);
    c.weight[block * PAGE + t] = 0.f;
  }
  // the old scales were read before the barrier above
  if (t == 0) {
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

constexpr int SEL_THREADS = 1024;

// The kept slots of one (sequence, head), in order, into kept[unit * budget].
// A radix selection finds the key of the last slot to be kept (four passes of 8
// bits over the weights), then one ordered pass writes the slots.
__global__ void __launch_bounds__(SEL_THREADS)
select_kernel(CacheArgs c, int budget, int recent, int32_t* __restrict__ new_lens,
              int32_t* __restrict__ kept, int* __restrict__ err) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t warp_n[2][32];
  __shared__ uint32_t pick[2];  // digit chosen, how many of its slots are still to be kept
  const int t = threadIdx.x, l = t & 31, w = t >> 5;
  const int n = blockIdx.x / c.Hk, h = blockIdx.x - n * c.Hk;
  const int len = cached_len(c, n, err);
  if (h == 0 && t == 0) new_lens[n] = len < budget ? len : budget;
  if (len <= budget) return;  // everything stays, in place: no list
  const int old = len - recent, want = budget - recent;
  int32_t* list = kept + static_cast<int64_t>(blockIdx.x) * budget;
  for (int i = t; i < recent; i += SEL_THREADS) list[want + i] = old + i;
  if (want == 0) return;
  auto key_at = [&](int i) -> uint32_t {
    const int pid = page_id(c, n, i >> c.lg, err);
    if (pid < 0) return 0u;
    return weight_key(__ldg(c.weight + (static_cast<int64_t>(pid) * c.Hk + h) * c.page + (i & (c.page - 1))));
  };
  uint32_t prefix = 0, need = static_cast<uint32_t>(want);
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (t < 256) hist[t] = 0;
    __syncthreads();
    const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
    for (int i = t; i < old; i += SEL_THREADS) {
      const uint32_t key = key_at(i);
      if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (t == 0) {
      uint32_t left = need;
      int d = 255;
      while (d > 0 && hist[d] < left) left -= hist[d--];
      pick[0] = static_cast<uint32_t>(d);
      pick[1] = left;
    }
    __syncthreads();
    prefix |= pick[0] << shift;
    need = pick[1];
    __syncthreads();
  }
  // keep key > prefix, and the first `need` slots with key == prefix
  uint32_t base = 0, ties = 0;
  for (int i0 = 0; i0 < old; i0 += SEL_THREADS) {
    const int i = i0 + t;
    const uint32_t key = i < old ? key_at(i) : 0u;
    const bool eq = i < old && key == prefix, gt = i < old && key > prefix;
    const uint32_t be = __ballot_sync(0xffffffffu, eq), bg = __ballot_sync(0xffffffffu, gt);
    if (l == 0) {
      warp_n[0][w] = __popc(be);
      warp_n[1][w] = __popc(bg);
    }
    __syncthreads();
    uint32_t e = warp_n[0][l], g = warp_n[1][l];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t a = __shfl_up_sync(0xffffffffu, e, o), b = __shfl_up_sync(0xffffffffu, g, o);
      if (l >= o) {
        e += a;
        g += b;
      }
    }
    const uint32_t etot = __shfl_sync(0xffffffffu, e, 31), gtot = __shfl_sync(0xffffffffu, g, 31);
    const uint32_t ew = __shfl_sync(0xffffffffu, e, (w + 31) & 31), gw = __shfl_sync(0xffffffffu, g, (w + 31) & 31);
    const uint32_t below = (1u << l) - 1u;
    const uint32_t er = ties + (w ? ew : 0u) + __popc(be & below);    // ties before this slot
    const uint32_t gr = (w ? gw : 0u) + __popc(bg & below);
    const uint32_t eq_kept = er < need ? er : need;
    const uint32_t ties0 = ties < need ? ties : need;
    if (gt || (eq && er < need)) list[base + gr + (eq_kept - ties0)] = i;
    const uint32_t ties1 = ties + etot < need ? ties + etot : need;
    base += gtot + (ties1 - ties0);
    ties += etot;
    __syncthreads();
  }
}

// One CTA per (destination page, sequence, head), the page along grid.y: gathers
// the page's rows.  A row is 8 threads of 16 codes.
__global__ void __launch_bounds__(256)
pack_kernel(CacheArgs c, const int32_t* __restrict__ dst, int dst_width, int budget,
            const int32_t* __restrict__ kept, int* __restrict__ err) {
  __shared__ int64_t src[128];  // source row (block * page + row), -1: bad page
  __shared__ float sks[128], svs[128];
  const int t = threadIdx.x, unit = blockIdx.x;
  const int n = unit / c.Hk, h = unit - n * c.Hk;
  const int len = cached_len(c, n, err), now = len < budget ? len : budget;
  for (int j = blockIdx.y; (static_cast<int64_t>(j) << c.lg) < now; j += gridDim.y) {
    const int first = j << c.lg;
    const int rows = now - first < c.page ? now - first : c.page;
    const int dp = j < dst_width ? __ldg(dst + static_cast<int64_t>(n) * dst_width + j) : -1;
    if (dp < 0 || dp >= c.pages) {
      if (t == 0) atomicCAS(err, 0, static_cast<int>(KDA_ERR_INVALID_ARG));
      continue;
    }
    const int64_t block = static_cast<int64_t>(dp) * c.Hk + h;
    __syncthreads();  // the last page's rows are no longer read
    if (t < rows) {
      const int i = len <= budget ? first + t : kept[static_cast<int64_t>(unit) * budget + first + t];
      const int pid = page_id(c, n, i >> c.lg, err);
      src[t] = -1;
      sks[t] = svs[t] = 0.f;
      if (pid >= 0) {
        const int64_t b = static_cast<int64_t>(pid) * c.Hk + h;
        const int64_t r = b * c.page + (i & (c.page - 1));
        src[t] = r;
        sks[t] = c.ks[b];
        svs[t] = c.vs[b];
        c.pos[block * c.page + t] = c.pos[r];
        c.weight[block * c.page + t] = c.weight[r];
      }
    }
    __syncthreads();
    float mk = 0.f, mv = 0.f;
    for (int r = 0; r < rows; ++r) {
      mk = fmaxf(mk, sks[r]);
      mv = fmaxf(mv, svs[r]);
    }
    const int sub = (t & 7) * 16;
    for (int r = t >> 3; r < rows; r += 32) {
      if (src[r] < 0) continue;
      const uint4 a = *reinterpret_cast<const uint4*>(c.k + src[r] * kDim + sub);
      const uint4 b = *reinterpret_cast<const uint4*>(c.v + src[r] * kDim + sub);
      const float fk = mk > 0.f ? sks[r] / mk : 1.f, fv = mv > 0.f ? svs[r] / mv : 1.f;
      uint4* ok = reinterpret_cast<uint4*>(c.k + (block * c.page + r) * kDim + sub);
      uint4* ov = reinterpret_cast<uint4*>(c.v + (block * c.page + r) * kDim + sub);
      *ok = fk == 1.f ? a : make_uint4(rescale4(a.x, fk), rescale4(a.y, fk), rescale4(a.z, fk), rescale4(a.w, fk));
      *ov = fv == 1.f ? b : make_uint4(rescale4(b.x, fv), rescale4(b.y, fv), rescale4(b.z, fv), rescale4(b.w, fv));
    }
    if (t == 0) {
      c.ks[block] = mk;
      c.vs[block] = mv;
    }
  }
}

}  // namespace

cudaError_t launch_cache_append(const CacheArgs& c, const void* k, const void* v,
                                const int32_t* positions, const int32_t* cu, int64_t T, int* err,
                                cudaStream_t stream) {
  const int64_t slots = T / c.page + 2 * static_cast<int64_t>(c.N);
  if (slots > 0x7fffffffLL) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(slots), static_cast<unsigned>(c.Hk));
  const auto* kk = static_cast<const __nv_bfloat16*>(k);
  const auto* vv = static_cast<const __nv_bfloat16*>(v);
  switch (c.page) {
    case 16: append_kernel<16><<<grid, 256, 0, stream>>>(c, kk, vv, positions, cu, T, err); break;
    case 32: append_kernel<32><<<grid, 256, 0, stream>>>(c, kk, vv, positions, cu, T, err); break;
    case 64: append_kernel<64><<<grid, 256, 0, stream>>>(c, kk, vv, positions, cu, T, err); break;
    default: append_kernel<128><<<grid, 256, 0, stream>>>(c, kk, vv, positions, cu, T, err); break;
  }
  return cudaGetLastError();
}

cudaError_t launch_cache_evict(const CacheArgs& c, const int32_t* dst, int dst_width, int budget,
                               int recent, int32_t* new_lens, int32_t* kept, int* err,
                               cudaStream_t stream) {
  const unsigned units = static_cast<unsigned>(c.N) * static_cast<unsigned>(c.Hk);
  select_kernel<<<units, SEL_THREADS, 0, stream>>>(c, budget, recent, new_lens, kept, err);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // pages that the kept rows can need, whatever the destination table's width
  const int64_t most = static_cast<int64_t>(c.width) << c.lg;
  const int64_t rows = budget < most ? budget : most;
  const unsigned pages = static_cast<unsigned>((rows + c.page - 1) >> c.lg);
  pack_kernel<<<dim3(units, pages < 65535u ? pages : 65535u), 256, 0, stream>>>(c, dst, dst_width, budget, kept, err);
  return cudaGetLastError();
}

}  // namespace kda
