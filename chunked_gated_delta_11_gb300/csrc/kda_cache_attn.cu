// kda_cache_attn.cu -- attention of a few new tokens per sequence over the
// 8-bit paged cache (kda_cache_attn), and the weights it accumulates.
//
// Bound by the cache's bytes (256 per token and KV head), so the kernel is a
// stream over them with the arithmetic kept beside it:
//
// Work.  A unit is (sequence, KV head, tile of 8 NT query rows); a row is a
//   (token, head of the group).  Its slots are cut into chunks, one CTA each (4
//   warps, a quarter of the chunk each), and joined afterwards.
// Loads.  cp.async, 16 bytes a lane, into a ring of the warp's own: no warp waits
//   for another.  A stage is 32 slots; its keys are refilled as soon as they are
//   in registers, its values at the end, so three quarters of the ring is in
//   flight.  Slots past the end arrive as zeros, so what they hold reaches nothing.
// Products.  e4m3 codes are exact in fp16, so both products run on fp16
//   mma.m16n8k16 with fp32 sums, the slots as its M side (S^T = K Q^T) and then
//   its K side (O^T = V^T P^T): 8 query rows fill the N side, where rows as M
//   would leave half of it empty.  The contraction order is free, so a lane's 16
//   consecutive channels of a key row are its operand as they lie in memory, and
//   16 consecutive channels of 4 value rows the other's.  Queries are scaled by a
//   power of two to [2^14, 2^15) (exact in fp16 but for channels below 2^-38 of
//   the row's largest); P^T goes from accumulator to operand by movmatrix.
// Softmax.  Block scales: x = acc * (k_scale * scale / fq); the value scale joins
//   the exponent, p' = 2^(x + log2 v_scale - m) with m within 2^6 of the running
//   maximum of x + log2 v_scale, so p' <= 2^6 whatever the scales are and its fp16
//   rounding (2^-11 of the value at most) is the only one before the output's; the
//   denominator sums p' / v_scale, or (scales far apart, whose p' may leave fp32's range
//   where their weights do not) 2^(x - m) itself.
//
// Measured (GB300, replayed from a graph): one sequence of 131072 slots, 8 KV heads
// of 4 rows, capped and biased, 57 us = 4.8 TB/s (the cap's instructions and one
// round of chunks); 256 sequences (498,000 slots) with weights 190 us = 5.4 TB/s and 33 us for the
// join; one of 4096 slots 8.6 us, two launches' worth.  32 sequences x 4 tokens (32
// rows per KV head) 132 us = 2.2 TB/s: 8 warps per SM with 255 registers each, which
// neither the copies nor the products keep busy.
#include "kda_attn.cuh"

namespace kda {
namespace {

constexpr int CA_WARPS = 4;
constexpr int CA_STEP = 32;                          // slots of a warp's stage
constexpr int CA_STAGE_BYTES = 16 * 512 + 128 + 16;  // 16 pieces per lane, positions, scales
constexpr int CA_PIECE = 18, CA_ROW = 8 * CA_PIECE;  // floats: a warp's output rows in shared memory
constexpr int ca_wchunk(bool share) { return share ? 128 : 512; }  // slots per CTA of the weight sums

// 8 rows: 3 CTAs per SM, two stages each.  16 and 32 rows (more registers): 2
// CTAs, three stages.  32 rows keep the queries' operand words in shared memory.
constexpr int ca_stages(int nt) { return nt == 1 ? 2 : 3; }
constexpr int ca_ctas(int nt) { return nt == 1 ? 3 : 2; }
constexpr int ca_qbytes(int nt) { return nt == 4 ? nt * 16 * 32 * 4 : 0; }
constexpr int ca_smem(int nt) {
  const int ring = CA_WARPS * ca_stages(nt) * CA_STAGE_BYTES;
  const int join = CA_WARPS * 8 * nt * (CA_ROW * 4 + 8);
  return ca_qbytes(nt) + (ring > join ? ring : join);
}

// How a call is cut.  Row tiles of the sequences: without cu_seqlens each has the
// same number `per_tiles`; with it sequence n owns the tile slots from
// floor(bos_n group / rows) + n on, T group / rows + N in all.
struct CachePlan {
  int nt;         // query rows per tile / 8
  int n;          // sequences
  int per;        // tokens per sequence (0: cu_seqlens)
  int per_tiles;
  int64_t tiles;  // tile slots
  int chunk, splits;  // slots per chunk, chunks of the longest possible sequence
  int64_t max_len;
  int ctas;        // > 0: that many CTAs share a list of the chunks that exist (plan_kernel)
  int weight_per;  // CTAs of the weight sums per (sequence, KV head)
  bool share;      // whose warps share the rows of 128 slots, instead of taking 128 slots each
};

__device__ __forceinline__ void cp16(void* dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4(void* dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(there ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Four e4m3 codes -> two words of two fp16 values (exact).
__device__ __forceinline__ void unpack4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Power of two that takes a largest magnitude to [2^14, 2^15): 1 for 0 (and
// non-finite rows, whose results are not finite either).
__device__ __forceinline__ float query_factor(float amax) {
  const int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
  if (!(amax > 0.f) || e > 127) return 1.f;
  const int f = 14 - e;
  return __uint_as_float(static_cast<uint32_t>((f > 100 ? 100 : f) + 127) << 23);
}

// A denominator may be as large as 1 / v_scale, so that times 2^d it may count where 2^d
// is below fp32's range: factors between references are taken as the square of their
// root, which holds for d down to -252.
__device__ __forceinline__ float root_factor(float from, float to) { return ex2_approx(0.5f * (from - to)); }
constexpr float kScaleNormal = 1.17549435e-38f;  // 2^-126: blocks of smaller scales are not seen
constexpr float kScaleWide = 1.8446744e19f;      // 2^64: value scales that are far apart

// Query tokens of sequence n.
__device__ __forceinline__ void tokens_of(const CacheAttnArgs& a, const CachePlan& p, int n,
                                          int64_t& bos, int& cnt) {
  if (a.cu) {
    int64_t eos;
    clamp_seq_bounds(__ldg(a.cu + n), __ldg(a.cu + n + 1), a.T, bos, eos);
    cnt = static_cast<int>(eos - bos);
  } else {
    bos = static_cast<int64_t>(n) * p.per;
    cnt = p.per;
  }
}

// First tile slot of sequence n.
__device__ __forceinline__ int64_t first_tile(const CacheAttnArgs& a, const CachePlan& p, int n,
                                              int64_t bos) {
  return a.cu ? bos * static_cast<unsigned>(a.H / a.c.Hk) / (8u * p.nt) + n
              : static_cast<int64_t>(n) * p.per_tiles;
}

// Sequence, its tokens, and the tile (which may be past its last) of tile slot s.
__device__ __forceinline__ void tile_of(const CacheAttnArgs& a, const CachePlan& p, int s, int& n,
                                        int64_t& bos, int& cnt, int& tile) {
  if (a.cu) {
    n = warp_search(a.c.N, s, [&](int i) -> int64_t {
      const int64_t c = __ldg(a.cu + i);
      return first_tile(a, p, i, c < 0 ? 0 : (c > a.T ? a.T : c));
    });
  } else {
    n = static_cast<unsigned>(s) / static_cast<unsigned>(p.per_tiles);
  }
  tokens_of(a, p, n, bos, cnt);
  tile = static_cast<int>(s - first_tile(a, p, n, bos));
}

// A warp's view of its stretch [begin, end) of a sequence's slots.
struct Stretch {
  const CacheArgs& c;
  int n, hk, end;
  int window;  // first table column that the lanes hold
  int ids;     // this lane's page id (-1: none)
  int* err;
  int pid[2], left[2];  // of the located slots: pages, and how many of each 16 exist (may be more)
  int64_t row[2];
  bool whole;

  __device__ Stretch(const CacheArgs& cc, int n_, int hk_, int end_, int* e)
      : c(cc), n(n_), hk(hk_), end(end_), window(-64), ids(-1), err(e) {}

  __device__ int page_of(int slot) {  // slot < end, the same for all lanes
    const int j = slot >> c.lg;
    if (j < window || j >= window + 32) {
      window = j;
      const int col = j + (threadIdx.x & 31);
      ids = (static_cast<int64_t>(col) << c.lg) < end ? page_id(c, n, col, err) : -1;
    }
    return __shfl_sync(0xffffffffu, ids, j - window);
  }

  // Finds the slots [t0, t0 + 32): their two blocks, or block 0 and nothing left.
  __device__ __forceinline__ void locate(int t0) {
    pid[0] = page_of(t0);
    pid[1] = c.lg > 4 || t0 + 16 >= end ? pid[0] : page_of(t0 + 16);
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      left[st] = pid[st] < 0 ? 0 : end - t0 - 16 * st;
      const int64_t block = static_cast<int64_t>(pid[st] < 0 ? 0 : pid[st]) * c.Hk + hk;
      row[st] = block * c.page + ((t0 + 16 * st) & (c.page - 1));
    }
    whole = left[0] >= 32 && left[1] >= 16;
  }

  // Issues the copies of the located slots into `stage`: the keys (with the
  // positions and both scales), or the values.  For the keys a lane copies what it
  // reads itself, rows g and g + 8, channels 16 q .. and 64 + 16 q ..: four lanes
  // take 64 bytes of a row.  Value rows are read by lanes with the rows across the
  // four, so they are copied whole, 8 lanes a row, and their 16-byte pieces stored
  // in the order c ^ (row & 6), where reads of 8 lanes meet no bank conflict.
  template <bool VALUES>
  __device__ __forceinline__ void issue(uint8_t* stage) {
    const int l = threadIdx.x & 31;
    const int r0 = VALUES ? l >> 3 : l >> 2, c0 = VALUES ? l & 7 : l & 3;
    const uint8_t* from = (VALUES ? c.v : c.k) + r0 * kDim + c0 * 16;
    uint8_t* mine = VALUES ? stage + 4096 + r0 * kDim : stage + l * 16;
    auto at = [&](int st, int i) {
      return from + (st ? row[1] : row[0]) * kDim + (VALUES ? 4 * i * kDim : 8 * (i >> 1) * kDim + (i & 1) * 64);
    };
    auto to = [&](int st, int i) {  // rows r0 + 4 i: (r & 6) is r0 & 2 and 4 (i & 1)
      return VALUES ? mine + (st * 16 + 4 * i) * kDim + ((c0 ^ (r0 & 2)) ^ (4 * (i & 1))) * 16 : mine + (st * 4 + i) * 512;
    };
    if (whole) {
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int i = 0; i < 4; ++i) cp16(to(st, i), at(st, i));
    } else {
#pragma unroll 1
      for (int st = 0; st < 2; ++st)
#pragma unroll 1
        for (int i = 0; i < 4; ++i)
          cp16(to(st, i), at(st, i), r0 + (VALUES ? 4 * i : 8 * (i >> 1)) < (st ? left[1] : left[0]));
    }
    if (VALUES) return;
    const int half = l >> 4;
    const int64_t mine_row = half ? row[1] : row[0];
    const int mine_left = half ? left[1] : left[0];
    cp4(stage + 8192 + l * 4, c.pos + mine_row + (l & 15), (l & 15) < mine_left);
    if ((l & 15) < 2) cp4(stage + 8320 + half * 8 + (l & 1) * 4, (l & 1 ? c.vs : c.ks) + (mine_row >> c.lg), mine_left > 0);
  }
};

// Chunks of a sequence of `len` slots.
__device__ __forceinline__ int chunks_of(const CachePlan& p, int len) {
  return len > p.chunk ? (len + p.chunk - 1) / p.chunk : 1;
}

// first[n]: (tile, chunk) pairs of the sequences before n, n = 0 .. N.  One CTA.
// Sequences of a malformed cu_seqlens may overlap: the sums are held to the number of
// places, so that the list stays one.
constexpr int PLAN_THREADS = 1024;
__global__ void __launch_bounds__(PLAN_THREADS)
plan_kernel(CacheAttnArgs a, CachePlan plan, int32_t* __restrict__ first, int* err) {
  __shared__ long long sums[32];
  grid_dep_wait();
  grid_dep_launch();
  const int t = threadIdx.x, l = t & 31, w = t >> 5;
  const long long places = plan.tiles * plan.splits;
  long long carry = 0;
  for (int n0 = 0; n0 < a.c.N; n0 += PLAN_THREADS) {
    const int n = n0 + t;
    long long own = 0;
    if (n < a.c.N) {
      int64_t bos;
      int cnt;
      tokens_of(a, plan, n, bos, cnt);
      const int rt = 8 * plan.nt;
      own = (static_cast<int64_t>(cnt) * (a.H / a.c.Hk) + rt - 1) / rt * chunks_of(plan, cached_len(a.c, n, err));
    }
    long long sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, sum, o);
      if (l >= o) sum += x;
    }
    if (l == 31) sums[w] = sum;
    __syncthreads();
    long long before = sums[l];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, before, o);
      if (l >= o) before += x;
    }
    const long long total = __shfl_sync(0xffffffffu, before, 31);
    before = w ? __shfl_sync(0xffffffffu, before, w - 1) : 0;
    const long long at = carry + before + sum - own;
    if (n < a.c.N) first[n] = static_cast<int32_t>(at < places ? at : places);
    carry += total;
    __syncthreads();
  }
  if (t == 0) first[a.c.N] = static_cast<int32_t>(carry < places ? carry : places);
}

// A CTA takes the chunk that its grid place says, or (LIST, plan.ctas)
// every so manieth of the list of those that exist: a table much wider than the
// sequences would otherwise leave most of the grid with nothing to do.
template <int NT, bool CAP, bool LIST>
__global__ void __launch_bounds__(CA_WARPS * 32, ca_ctas(NT))
cache_attn_kernel(CacheAttnArgs a, CachePlan plan, const int32_t* __restrict__ list,
                  float* __restrict__ part_o, float2* __restrict__ part_ml,
                  float* __restrict__ scores, int* err) {
  constexpr int RT = 8 * NT, STAGES = ca_stages(NT);
  constexpr bool QSMEM = NT == 4;
  extern __shared__ __align__(16) uint8_t smem[];
  grid_dep_wait();
  grid_dep_launch();
  const int l = threadIdx.x & 31, w = threadIdx.x >> 5, g = l >> 2, q = l & 3;
  const unsigned group = a.H / a.c.Hk;
  // without a list there is one turn (a loop's registers cost the 32-row tile 9 %)
  const unsigned items = LIST ? static_cast<unsigned>(__ldg(list + a.c.N)) * a.c.Hk : blockIdx.x + 1;
  for (unsigned item = blockIdx.x; LIST ? item < items : item == blockIdx.x; item = LIST ? item + gridDim.x : items) {
    int n, cnt, tile, chunk, hk;
    int64_t bos;
    if (LIST) {
      const int j = item / static_cast<unsigned>(a.c.Hk);
      hk = item - j * a.c.Hk;
      n = warp_search(a.c.N, j, [&](int i) -> int64_t { return __ldg(list + i); });
      tokens_of(a, plan, n, bos, cnt);
      const int chunks = chunks_of(plan, cached_len(a.c, n, err)), rest = j - __ldg(list + n);
      if (rest < 0) continue;
      tile = rest / chunks;
      chunk = rest - tile * chunks;
    } else {
      const int slot = item / static_cast<unsigned>(a.c.Hk);
      hk = item - slot * a.c.Hk;
      chunk = blockIdx.y;
      tile_of(a, plan, slot, n, bos, cnt, tile);
    }
    // where the tile's partial rows go (worked out where it is used: registers)
    auto unit = [&]() -> int64_t {
      return LIST ? (first_tile(a, plan, n, bos) + tile) * a.c.Hk + hk : static_cast<int64_t>(item);
    };
    const int64_t left_rows = static_cast<int64_t>(cnt) * group - static_cast<int64_t>(tile) * RT;
    if (tile < 0 || left_rows <= 0) continue;  // (a malformed cu_seqlens can give the former)
    const int rows = left_rows < RT ? static_cast<int>(left_rows) : RT;  // of this tile
    const unsigned row0 = static_cast<unsigned>(tile) * RT;               // its first (token, head) row
    const int len = cached_len(a.c, n, err);
    // the sequence's chunks are equal, in steps of 128 slots, and so are the warps' shares
    const int chunks = chunks_of(plan, len);
    if (chunk >= chunks) continue;
    constexpr int WHOLE = CA_WARPS * CA_STEP;
    const int size = ((len + chunks - 1) / chunks + WHOLE - 1) / WHOLE * WHOLE;
    const int begin = len < chunk * size ? len : chunk * size;
    const int end = len - begin < size ? len : begin + size;

    // the warp's quarter of the chunk; its first copies go out first
    const int quarter = (end - begin + WHOLE - 1) / WHOLE * CA_STEP;
    const int wb = begin + w * quarter;
    const int we = end < wb + quarter ? end : wb + quarter;
    const int steps = we > wb ? (we - wb + CA_STEP - 1) / CA_STEP : 0;
    uint8_t* ring = smem + ca_qbytes(NT) + w * (STAGES * CA_STAGE_BYTES);
    // Without given positions the queries are the newest tokens.  That slot's page is looked up
    // beside the first of the chunk's own, its position beside the queries.
    const bool by_newest = !a.positions && len > 0;
    const int newest_page = by_newest ? __ldg(a.c.table + static_cast<int64_t>(n) * a.c.width + ((len - 1) >> a.c.lg)) : -1;
    Stretch src(a.c, n, hk, we, err);
#pragma unroll
    for (int i = 0; i < STAGES; ++i) {
      if (i < steps) {
        src.locate(wb + i * CA_STEP);
        src.issue<false>(ring + i * CA_STAGE_BYTES);
      }
      cp_commit();
      if (i < steps) src.issue<true>(ring + i * CA_STAGE_BYTES);
      cp_commit();
    }

    // query rows 8 t + g as operand words, channels as the keys' bytes
    uint32_t qf[QSMEM ? 1 : NT][16];
    uint32_t* qs = reinterpret_cast<uint32_t*>(smem);  // QSMEM: [t][word pair][lane][2]
    float mul[NT][2], slope[NT][2], m[NT][2], sum[NT][2];
    int qpos[NT][2];
    int qleast = 0x7fffffff;  // least position of the tile's queries
    int newest = 0;  // for a bad page too, which the chunk that has it reports
    if (newest_page >= 0 && newest_page < a.c.pages)
      newest = a.c.pos[(static_cast<int64_t>(newest_page) * a.c.Hk + hk) * a.c.page + ((len - 1) & (a.c.page - 1))];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = 8 * t + g;
      uint4 x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = make_uint4(0, 0, 0, 0);
      if (r < rows) {
        const unsigned rr = row0 + r, tok = rr / group;
        const int64_t at = ((bos + tok) * a.H + hk * group + (rr - tok * group)) * kDim + q * 16;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[i] = *reinterpret_cast<const uint4*>(a.q + at + (i >> 1) * 64 + (i & 1) * 8);
      }
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t ws[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          top = fmaxf(top, fmaxf(fabsf(__uint_as_float(ws[j] << 16)), fabsf(__uint_as_float(ws[j] & 0xffff0000u))));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float f = query_factor(top), inv = 1.f / f;
      if (!QSMEM || w == t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t ws[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t v = pack_f16(__uint_as_float(ws[j] << 16) * f, __uint_as_float(ws[j] & 0xffff0000u) * f);
            if (QSMEM) qs[((t * 8 + i * 2 + (j >> 1)) * 32 + l) * 2 + (j & 1)] = v;
            else qf[QSMEM ? 0 : t][i * 4 + j] = v;
          }
        }
      }
      // what the lane's columns (query rows 8 t + 2 q + e) need
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int c = 8 * t + 2 * q + e;
        mul[t][e] = __shfl_sync(0xffffffffu, inv, (2 * q + e) * 4) * a.scale * (CAP ? 1.f : kLog2e);
        slope[t][e] = 0.f;
        qpos[t][e] = -1;
        if (c < rows) {
          const unsigned rr = row0 + c, tok = rr / group;
          qpos[t][e] = a.positions ? __ldg(a.positions + bos + tok) : newest - (cnt - 1 - static_cast<int>(tok));
          qleast = qleast < qpos[t][e] ? qleast : qpos[t][e];
          if (a.slopes) slope[t][e] = __ldg(a.slopes + hk * group + (rr - tok * group)) * kLog2e;
        }
        m[t][e] = -INFINITY;
        sum[t][e] = 0.f;
      }
    }
    float o[NT][8][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][i][e] = 0.f;
    qleast = min(qleast, __shfl_xor_sync(0xffffffffu, qleast, 1));
    qleast = min(qleast, __shfl_xor_sync(0xffffffffu, qleast, 2));
    float qfar[NT][2];  // positions relative to that
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) qfar[t][e] = static_cast<float>(qpos[t][e] - qleast);
    if (QSMEM) __syncthreads();
    const float c1 = CAP ? cap_exponent(1.f, a.cap) : 0.f, c2 = CAP ? a.cap * kLog2e : 0.f;
    const bool large = CAP && a.cap > kCapSmall;
    const float per_cap = large ? 1.f / a.cap : 0.f;

    float* srow = scores ? scores + unit() * RT * plan.max_len : nullptr;
    float vs_most = 0.f, vs_least = INFINITY;  // v_scale so far
    int buf = 0;
    for (int it = 0; it < steps; ++it) {
      // one group for the keys and one for the values of each stage: 2 STAGES - 1
      // younger ones may be in flight
      cp_wait<2 * STAGES - 1>();
      __syncwarp();  // positions and scales come from other lanes
      uint8_t* stage = ring + buf * CA_STAGE_BYTES;
      buf = buf + 1 == STAGES ? 0 : buf + 1;
      const uint8_t* mine = stage + l * 16;
      const int t0 = wb + it * CA_STEP;

      float s[2][NT][4];
      float s2[2][4];  // NT = 1: the second half of the channels, for two shorter chains
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s2[st][e] = 0.f;
#pragma unroll
          for (int t = 0; t < NT; ++t) s[st][t][e] = 0.f;
        }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint4 kk[2][2];
#pragma unroll
        for (int st = 0; st < 2; ++st) {
          kk[st][0] = *reinterpret_cast<const uint4*>(mine + (st * 4 + half) * 512);
          kk[st][1] = *reinterpret_cast<const uint4*>(mine + (st * 4 + 2 + half) * 512);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t af[2][4];
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            const uint32_t r0[4] = {kk[st][0].x, kk[st][0].y, kk[st][0].z, kk[st][0].w};
            const uint32_t r1[4] = {kk[st][1].x, kk[st][1].y, kk[st][1].z, kk[st][1].w};
            unpack4(r0[j], af[st][0], af[st][2]);
            unpack4(r1[j], af[st][1], af[st][3]);
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            uint2 b;
            if (QSMEM) b = *reinterpret_cast<const uint2*>(qs + ((t * 8 + half * 4 + j) * 32 + l) * 2);
            else b = make_uint2(qf[QSMEM ? 0 : t][half * 8 + 2 * j], qf[QSMEM ? 0 : t][half * 8 + 2 * j + 1]);
#pragma unroll
            for (int st = 0; st < 2; ++st)
              mma_f16(NT == 1 && half ? s2[st] : s[st][t], af[st][0], af[st][1], af[st][2], af[st][3], b.x, b.y);
          }
        }
      }
      if (NT == 1) {
#pragma unroll
        for (int st = 0; st < 2; ++st)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[st][0][e] += s2[st][e];
      }
      // scores in log2 units, plus log2 v_scale
      float lvs[2], ivs[2], ksc[2];
      bool page_ok[2];
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        const float2 sc = *reinterpret_cast<const float2*>(stage + 8320 + st * 8);
        page_ok[st] = sc.y >= kScaleNormal;
        ksc[st] = sc.x;
        lvs[st] = page_ok[st] ? __log2f(sc.y) : 0.f;
        ivs[st] = page_ok[st] ? ex2_approx(-lvs[st]) : 0.f;  // undoes what the exponent adds
        vs_most = fmaxf(vs_most, sc.y);
        vs_least = page_ok[st] ? fminf(vs_least, sc.y) : vs_least;
      }
      const bool wide = vs_least * kScaleWide < vs_most;  // the same for the warp
#pragma unroll
      for (int st = 0; st < 2; ++st) ivs[st] = wide ? 0.f : ivs[st];
      // whole stages of visible slots (almost all) need no selection
      bool whole = t0 + CA_STEP <= we && page_ok[0] && page_ok[1];
      const int pl = *reinterpret_cast<const int*>(stage + 8192 + l * 4);
      whole = __all_sync(0xffffffffu, whole && pl <= qleast);
      // the keys have been read by every lane: refill them while the rest goes on
      __syncwarp();
      if (it + STAGES < steps) {
        src.locate(t0 + STAGES * CA_STEP);
        src.issue<false>(stage);
      }
      cp_commit();
      const bool bias = a.slopes != nullptr;
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float f = mul[t][e] * ksc[st];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float& x = s[st][t][2 * r + e];
              x = !CAP ? fmaf(x, f, lvs[st]) : (large ? cap_log2_large(x * f, per_cap, c1, c2) : cap_log2(x * f, c1, c2)) + lvs[st];
            }
          }
      if (bias) {
        const float far = static_cast<float>(pl - qleast);
#pragma unroll
        for (int st = 0; st < 2; ++st)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float p = __shfl_sync(0xffffffffu, far, 16 * st + 8 * r + g);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                s[st][t][2 * r + e] = fmaf(-slope[t][e], qfar[t][e] - p, s[st][t][2 * r + e]);
          }
      }
      if (!whole) {
#pragma unroll
        for (int st = 0; st < 2; ++st)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int p = __shfl_sync(0xffffffffu, pl, 16 * st + 8 * r + g);
            const bool there = t0 + 16 * st + 8 * r + g < we && page_ok[st];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (!there || p > qpos[t][e]) s[st][t][2 * r + e] = -INFINITY;
          }
      }
      if (srow) {
#pragma unroll
        for (int st = 0; st < 2; ++st)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int tok = t0 + 16 * st + 8 * r + g;
            if (tok < we) {
#pragma unroll
              for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (8 * t + 2 * q + e < rows)
                    srow[(8 * t + 2 * q + e) * plan.max_len + tok] = s[st][t][2 * r + e] - lvs[st];
            }
          }
      }
      // running maximum
      uint32_t pf[2][NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float mx[2], f[2], h[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          mx[e] = fmaxf(fmaxf(s[0][t][e], s[0][t][2 + e]), fmaxf(s[1][t][e], s[1][t][2 + e]));
        // the reference moves only when the maximum outgrows it by 2^6: p' stays in
        // fp16's range, and its rounding below 2^-25 of the largest weight
        if (__any_sync(0xffffffffu, mx[0] > m[t][0] + 6.f || mx[1] > m[t][1] + 6.f)) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 4));
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 8));
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 16));
            const bool grow = mx[e] > m[t][e] + 6.f;
            h[e] = grow ? root_factor(m[t][e], mx[e]) : 1.f;
            f[e] = h[e] * h[e];
            sum[t][e] = sum[t][e] * h[e] * h[e];
            if (grow) m[t][e] = mx[e];
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            o[t][i][0] *= f[0];
            o[t][i][1] *= f[1];
            o[t][i][2] *= f[0];
            o[t][i][3] *= f[1];
          }
        }
        const float ref0 = m[t][0] == -INFINITY ? 0.f : m[t][0], ref1 = m[t][1] == -INFINITY ? 0.f : m[t][1];
        if (wide) {  // the exponentials of the plain scores; p' adds nothing then
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            if (!page_ok[st]) continue;
            sum[t][0] += ex2_approx(s[st][t][0] - lvs[st] - ref0) + ex2_approx(s[st][t][2] - lvs[st] - ref0);
            sum[t][1] += ex2_approx(s[st][t][1] - lvs[st] - ref1) + ex2_approx(s[st][t][3] - lvs[st] - ref1);
          }
        }
#pragma unroll
        for (int st = 0; st < 2; ++st) {
          const float p0 = ex2_approx(s[st][t][0] - ref0), p1 = ex2_approx(s[st][t][1] - ref1);
          const float p2 = ex2_approx(s[st][t][2] - ref0), p3 = ex2_approx(s[st][t][3] - ref1);
          sum[t][0] = fmaf(p0 + p2, ivs[st], sum[t][0]);
          sum[t][1] = fmaf(p1 + p3, ivs[st], sum[t][1]);
          pf[st][t][0] = transpose8x8(pack_f16(p0, p1));
          pf[st][t][1] = transpose8x8(pack_f16(p2, p3));
        }
      }
      cp_wait<2 * STAGES - 1>();
      __syncwarp();
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        uint32_t v[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 2 * q + (i & 1) + 8 * (i >> 1);  // r & 6 = 2 q
          const uint4 x = *reinterpret_cast<const uint4*>(stage + 4096 + (st * 16 + r) * kDim + ((g ^ (2 * q)) * 16));
          v[i][0] = x.x;
          v[i][1] = x.y;
          v[i][2] = x.z;
          v[i][3] = x.w;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // channels 4 j .. 4 j + 3 of the lane's 16
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            // bytes 2 half, 2 half + 1 of the rows' words, interleaved
            const uint32_t x = __byte_perm(v[0][j], v[1][j], half ? 0x7362 : 0x5140);
            const uint32_t y = __byte_perm(v[2][j], v[3][j], half ? 0x7362 : 0x5140);
            uint32_t a0, a1, a2, a3;
            unpack4(x, a0, a1);
            unpack4(y, a2, a3);
#pragma unroll
            for (int t = 0; t < NT; ++t)
              mma_f16(o[t][2 * j + half], a0, a1, a2, a3, pf[st][t][0], pf[st][t][1]);
          }
        }
      }
      __syncwarp();
      if (it + STAGES < steps) src.issue<true>(stage);
      cp_commit();
    }

    // join the warps: the ring is done with.  Channel 16 g + 2 i + b of a row is at
    // i * CA_PIECE + 2 g + b (no worse than 2-way bank conflicts either way).
    cp_wait<0>();
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sum[t][e] += __shfl_xor_sync(0xffffffffu, sum[t][e], 4);
        sum[t][e] += __shfl_xor_sync(0xffffffffu, sum[t][e], 8);
        sum[t][e] += __shfl_xor_sync(0xffffffffu, sum[t][e], 16);
      }
    __syncthreads();
    float* so = reinterpret_cast<float*>(smem + ca_qbytes(NT));          // [warp][row][CA_ROW]
    float2* sml = reinterpret_cast<float2*>(so + CA_WARPS * RT * CA_ROW);  // [warp][row]
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * t + 2 * q + e;
        if (g == 0) sml[w * RT + r] = make_float2(m[t][e], sum[t][e]);
        float* dst = so + (w * RT + r) * CA_ROW + g * 2;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<float2*>(dst + i * CA_PIECE) = make_float2(o[t][i][e], o[t][i][2 + e]);
      }
    }
    __syncthreads();
    const bool direct = part_o == nullptr;
    for (int r = w; r < rows; r += CA_WARPS) {
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < CA_WARPS; ++i) top = fmaxf(top, sml[i * RT + r].x);
      const float ref = top == -INFINITY ? 0.f : top;
      float tot = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < CA_WARPS; ++i) {
        const float2 ml = sml[i * RT + r];
        const float h = root_factor(ml.x, ref), f = h * h;
        const float* at = so + (i * RT + r) * CA_ROW + (l & 3) * (2 * CA_PIECE) + (l >> 2) * 2;
        const float2 x = *reinterpret_cast<const float2*>(at);
        const float2 y = *reinterpret_cast<const float2*>(at + CA_PIECE);
        tot = fmaf(ml.y * h, h, tot);
        acc.x = fmaf(x.x, f, acc.x);
        acc.y = fmaf(x.y, f, acc.y);
        acc.z = fmaf(y.x, f, acc.z);
        acc.w = fmaf(y.y, f, acc.w);
      }
      const unsigned rr = row0 + r, tok = rr / group;
      if (direct) {
        const float inv = tot == 0.f ? 0.f : 1.f / tot;
        const int64_t at = ((bos + tok) * a.H + hk * group + (rr - tok * group)) * kDim + l * 4;
        *reinterpret_cast<uint2*>(a.out + at) =
            make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
      } else {
        const int64_t at = (unit() * plan.splits + chunk) * RT + r;
        *reinterpret_cast<float4*>(part_o + at * kDim + l * 4) = acc;
        if (l == 0) part_ml[at] = make_float2(top, tot);
      }
    }
    if (LIST) __syncthreads();  // the next item's copies go where the rows were
  }
}

// Adds the weights of ca_wchunk(SHARE) slots from `first` on; all threads of a CTA of
// 128.  Rows in order, 8 of them under way at a time; SHARE: a quarter of every tile's
// per warp, their loads under way while the denominators are worked out, and the warps'
// sums in order.
template <bool SHARE>
__device__ __forceinline__ void add_weights(const CacheAttnArgs& a, const CachePlan& plan,
                                            const float2* __restrict__ part_ml,
                                            const float* __restrict__ scores, float* lse, float (*so)[kDim], int n,
                                            int hk, int len, int first, int* err) {
  const int l = threadIdx.x & 31, w = threadIdx.x >> 5;
  const unsigned group = a.H / a.c.Hk, rt = 8 * plan.nt;
  const int most = SHARE ? rt / 4 : 8, mine = SHARE ? w * most : 0;  // the warp's rows of a tile
  int64_t bos;
  int cnt;
  tokens_of(a, plan, n, bos, cnt);
  const int64_t rows = static_cast<int64_t>(cnt) * group;
  const int chunks = chunks_of(plan, len);
  const int64_t slot = first_tile(a, plan, n, bos);
  const int tok = first + (SHARE ? l : threadIdx.x) * 4;  // the thread's 4 slots, of one page
  const int at = tok < len ? tok : (len - 1) & ~3;  // past the length: reads the last, drops it
  const int pid = tok < len ? page_id(a.c, n, tok >> a.c.lg, err) : -1;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int64_t r0 = 0; r0 < rows; r0 += rt) {
    const int64_t unit = (slot + r0 / rt) * a.c.Hk + hk;
    const int here = rows - r0 < rt ? static_cast<int>(rows - r0) : static_cast<int>(rt);
    const float* row = scores + unit * rt * plan.max_len + at;
    float4 x[8];
    auto load = [&](int r) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x[i] = i < most && r + i < here ? *reinterpret_cast<const float4*>(row + (r + i) * plan.max_len)
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    if (SHARE) load(mine);
    __syncthreads();
    {
      // denominators: row threadIdx / 4, its chunks over 4 lanes
      const int r = threadIdx.x >> 2;
      float top = -INFINITY, tot = 0.f;
      if (r < here) {
        for (int c0 = l & 3; c0 < chunks; c0 += 4) {
          const float2 ml = part_ml[(unit * plan.splits + c0) * rt + r];
          const float mn = fmaxf(top, ml.x), ref = mn == -INFINITY ? 0.f : mn;
          const float h0 = root_factor(top, ref), h1 = root_factor(ml.x, ref);
          tot = tot * h0 * h0 + ml.y * h1 * h1;
          top = mn;
        }
      }
      float all = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, 2));
      const float h = root_factor(top, all == -INFINITY ? 0.f : all);
      tot = tot * h * h;
      tot += __shfl_xor_sync(0xffffffffu, tot, 1);
      tot += __shfl_xor_sync(0xffffffffu, tot, 2);
      // nothing seen: every score of the row is -inf and gives 0 against 0; rows that
      // are not there give 0 against infinity
      if ((l & 3) == 0) lse[r] = r >= here ? INFINITY : all == -INFINITY ? 0.f : all + log2f(tot);
    }
    __syncthreads();
    for (int r = mine; r < (SHARE ? mine + 1 : here); r += 8) {
      if (!SHARE) load(r);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = i < most ? lse[r + i] : INFINITY;
        sum.x += ex2_approx(x[i].x - d);
        sum.y += ex2_approx(x[i].y - d);
        sum.z += ex2_approx(x[i].z - d);
        sum.w += ex2_approx(x[i].w - d);
      }
    }
  }
  if (SHARE) {
    __syncthreads();  // (the last chunk's sums have been read)
    *reinterpret_cast<float4*>(&so[w][l * 4]) = sum;
    __syncthreads();
    if (w > 0) return;
    sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(&so[i][l * 4]);
      sum.x += x.x;
      sum.y += x.y;
      sum.z += x.z;
      sum.w += x.w;
    }
  }
  if (pid < 0) return;
  float4* to = reinterpret_cast<float4*>(a.c.weight + (static_cast<int64_t>(pid) * a.c.Hk + hk) * a.c.page +
                                         (tok & (a.c.page - 1)));
  float4 x = *to;
  x.x += sum.x;  // the scores of slots past the length were never written
  if (tok + 1 < len) x.y += sum.y;
  if (tok + 2 < len) x.z += sum.z;
  if (tok + 3 < len) x.w += sum.w;
  *to = x;
}

// Joins the chunks.  The first CTAs take output rows: 4 each, a warp a row, or
// (plan.splits > 16) one each, 4 warps over its chunks; always in a fixed order.
// With `scores` the other CTAs add the weights of some slots of a (sequence, KV head)
// each, the rows in a fixed order; a row's denominator they work out again from the
// chunks' pairs.
template <bool SHARE>
__global__ void __launch_bounds__(128)
join_kernel(CacheAttnArgs a, CachePlan plan, unsigned row_ctas, const float* __restrict__ part_o,
            const float2* __restrict__ part_ml, const float* __restrict__ scores, int* err) {
  __shared__ float so[4][kDim];
  __shared__ float2 sml[4];
  __shared__ float lse[32];
  grid_dep_wait();
  grid_dep_launch();
  const int l = threadIdx.x & 31, w = threadIdx.x >> 5;
  const unsigned group = a.H / a.c.Hk, rt = 8 * plan.nt;
  if (blockIdx.x < row_ctas) {
    const bool spread = plan.splits > 16;
    const unsigned row = spread ? blockIdx.x : blockIdx.x * 4 + w;
    const int t = row / static_cast<unsigned>(a.H);
    const int h = row - t * a.H, hk = h / group;
    if (t >= a.T) return;  // a whole warp, or the whole CTA
    int n = 0;
    if (a.cu) {
      n = warp_search(a.c.N, t, [&](int i) -> int64_t { return __ldg(a.cu + i); });
    } else {
      n = static_cast<unsigned>(t) / static_cast<unsigned>(plan.per);
    }
    int64_t bos;
    int cnt;
    tokens_of(a, plan, n, bos, cnt);
    if (t < bos || t >= bos + cnt) return;
    const int len = cached_len(a.c, n, err);
    const int chunks = chunks_of(plan, len);
    const unsigned rr = static_cast<unsigned>(t - bos) * group + (h - hk * group);
    const int64_t unit = (first_tile(a, plan, n, bos) + rr / rt) * a.c.Hk + hk;
    const int64_t base = unit * plan.splits * rt + rr % rt;
    const int stride = spread ? 4 : 1;
    float top = -INFINITY, tot = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c0 = spread ? w : 0; c0 < chunks; c0 += 4 * stride) {
      float2 ml[4];
      float4 x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ml[i] = make_float2(-INFINITY, 0.f);
        x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c0 + stride * i < chunks) {
          const int64_t at = base + static_cast<int64_t>(c0 + stride * i) * rt;
          ml[i] = part_ml[at];
          x[i] = *reinterpret_cast<const float4*>(part_o + at * kDim + l * 4);
        }
      }
      const float mn = fmaxf(fmaxf(fmaxf(top, ml[0].x), ml[1].x), fmaxf(ml[2].x, ml[3].x));
      const float ref = mn == -INFINITY ? 0.f : mn;
      const float h = root_factor(top, ref), f = h * h;
      top = mn;
      tot = tot * h * h;
      acc.x *= f;
      acc.y *= f;
      acc.z *= f;
      acc.w *= f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float r = root_factor(ml[i].x, ref), e = r * r;
        tot = fmaf(ml[i].y * r, r, tot);
        acc.x = fmaf(x[i].x, e, acc.x);
        acc.y = fmaf(x[i].y, e, acc.y);
        acc.z = fmaf(x[i].z, e, acc.z);
        acc.w = fmaf(x[i].w, e, acc.w);
      }
    }
    if (spread) {
      *reinterpret_cast<float4*>(&so[w][l * 4]) = acc;
      if (l == 0) sml[w] = make_float2(top, tot);
      __syncthreads();
      if (w != 0) return;
      top = fmaxf(fmaxf(sml[0].x, sml[1].x), fmaxf(sml[2].x, sml[3].x));
      const float ref = top == -INFINITY ? 0.f : top;
      tot = 0.f;
      acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float r = root_factor(sml[i].x, ref), e = r * r;
        const float4 x = *reinterpret_cast<const float4*>(&so[i][l * 4]);
        tot = fmaf(sml[i].y * r, r, tot);
        acc.x = fmaf(x.x, e, acc.x);
        acc.y = fmaf(x.y, e, acc.y);
        acc.z = fmaf(x.z, e, acc.z);
        acc.w = fmaf(x.w, e, acc.w);
      }
    }
    const float inv = tot == 0.f ? 0.f : 1.f / tot;
    *reinterpret_cast<uint2*>(a.out + static_cast<int64_t>(row) * kDim + l * 4) =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    return;
  }
  const unsigned b = static_cast<unsigned>(blockIdx.x - row_ctas);
  const unsigned pair = b / plan.weight_per;
  const int n = pair / static_cast<unsigned>(a.c.Hk), hk = pair - n * a.c.Hk;
  const int len = cached_len(a.c, n, err);
  const int64_t wide = ca_wchunk(SHARE);
  for (int64_t first = (b - pair * plan.weight_per) * wide; first < len; first += plan.weight_per * wide)
    add_weights<SHARE>(a, plan, part_ml, scores, lse, so, n, hk, len, static_cast<int>(first), err);
}

// Tile heights of 8, 16 and 32 rows by the rows of an average sequence: the cache
// is read once per tile, and a lane keeps 4 accumulators per row.
CachePlan make_plan(int64_t T, int H, int Hk, int N, bool cu, int64_t max_len) {
  CachePlan p{};
  const int64_t group = H / Hk, rows = T * group;
  p.nt = rows <= 8 * static_cast<int64_t>(N) ? 1 : rows <= 16 * static_cast<int64_t>(N) ? 2 : 4;
  const int64_t rt = 8 * p.nt;
  p.n = N;
  p.per = cu ? 0 : static_cast<int>(T / N);
  p.per_tiles = cu ? 0 : static_cast<int>((p.per * group + rt - 1) / rt);
  p.tiles = cu ? rows / rt + N : static_cast<int64_t>(N) * p.per_tiles;
  p.max_len = max_len;
  // One sequence: the chunks fill the GPU once, evenly.  More of them are ragged:
  // chunks of at most 2048 slots (or a sixteenth of the longest) keep the last ones
  // short.
  const int64_t slots = ca_ctas(p.nt) * kSMs;
  const int64_t tiles = (rows + rt - 1) / rt;
  const int64_t units = (tiles > N ? tiles : N) * Hk;
  int64_t chunk = (max_len * units + slots - 1) / slots;
  const int64_t most = max_len / 16 > 2048 ? max_len / 16 : 2048;
  if (N > 1 && chunk > most) chunk = most;
  const int64_t step = CA_WARPS * CA_STEP;
  chunk = (chunk + step - 1) / step * step;
  const int64_t least = (max_len + 65534) / 65535;  // grid.y
  if (chunk < least) chunk = (least + step - 1) / step * step;
  p.chunk = static_cast<int>(chunk);
  p.splits = static_cast<int>((max_len + chunk - 1) / chunk);
  // A CTA that finds no chunk at its place costs about half a microsecond of one of the
  // `slots`; the list costs a launch and the overlap of one CTA's end with the next one's
  // start.  They meet at about 30 rounds of places (8 KV heads of 4 rows, slots in the
  // sequences and in the table, microseconds without and with the list: 256 x 1024 in 4096, 9
  // rounds, 95 and 103; 64 x 2000 in 32768, 18 rounds, 59 and 63; 256 x 1024 in 16384, 36
  // rounds, 108 and 104; in 131072, 72 rounds, 128 and 104; 256 x 100 in 16384, 46 and 33).
  p.ctas = p.splits > 1 && p.tiles * Hk * p.splits > 32 * slots ? static_cast<int>(slots) : 0;
  // Weight sums: a warp has 128 slots and all rows, unless that leaves SMs idle and there
  // are rows to share (84 short sequences with 72 rows each: 47 us, shared 32 us; one of
  // 40,000 slots with 12 rows: 41 us, shared 48 us).
  const int64_t pairs = static_cast<int64_t>(N) * Hk;
  p.share = p.nt > 1 && pairs * ((max_len + ca_wchunk(false) - 1) / ca_wchunk(false)) < 2 * kSMs;
  const int64_t ranges = (max_len + ca_wchunk(p.share) - 1) / ca_wchunk(p.share);
  const int64_t fill = (32768 + pairs - 1) / pairs;
  p.weight_per = static_cast<int>(ranges < fill ? ranges : fill);
  return p;
}

// Places in the workspace; total is SIZE_MAX for more than any device has.
struct CacheScratch {
  size_t list, ml, scores, total;
};

CacheScratch scratch_of(const CachePlan& p, int Hk, bool accumulate) {
  CacheScratch s{};
  const size_t rows = static_cast<size_t>(p.tiles) * Hk * 8 * p.nt;
  if (p.splits > 1 || accumulate) {
    if (static_cast<double>(rows) * (p.splits * (kDim * 4.0 + 8.0) + (accumulate ? p.max_len * 4.0 : 0.0)) > 1e14) {
      s.total = SIZE_MAX;
      return s;
    }
    s.ml = rows * p.splits * kDim * 4;
    s.scores = s.ml + rows * p.splits * 8;
    s.list = s.scores + (accumulate ? rows * static_cast<size_t>(p.max_len) * 4 : 0);
    s.total = s.list + (p.ctas ? (static_cast<size_t>(p.n) + 1) * 4 : 0);
  }
  return s;
}

template <int NT, bool CAP, bool LIST>
cudaError_t launch_one(const CacheAttnArgs& a, const CachePlan& p, const int32_t* list, float* o,
                       float2* ml, float* scores, int* err, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  auto* kernel = cache_attn_kernel<NT, CAP, LIST>;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), ca_smem(NT), done);
  if (e != cudaSuccess) return e;
  const dim3 grid = p.ctas ? dim3(static_cast<unsigned>(p.ctas))
                           : dim3(static_cast<unsigned>(p.tiles * a.c.Hk), static_cast<unsigned>(p.splits));
  return launch_pdl(kernel, grid, dim3(CA_WARPS * 32), ca_smem(NT), stream, a, p, list, o, ml, scores, err);
}

template <int NT>
cudaError_t launch_variant(bool cap, const CacheAttnArgs& a, const CachePlan& p, const int32_t* list,
                           float* o, float2* ml, float* scores, int* err, cudaStream_t stream) {
  auto one = p.ctas ? cap ? launch_one<NT, true, true> : launch_one<NT, false, true>
                    : cap ? launch_one<NT, true, false> : launch_one<NT, false, false>;
  return one(a, p, list, o, ml, scores, err, stream);
}

}  // namespace

size_t cache_attn_workspace(int64_t T, int H, int Hk, int N, bool cu, int64_t max_len, bool accumulate) {
  return scratch_of(make_plan(T, H, Hk, N, cu, max_len), Hk, accumulate).total;
}

cudaError_t launch_cache_attn(const CacheAttnArgs& a, void* ws, int* err, cudaStream_t stream) {
  const int64_t max_len = static_cast<int64_t>(a.c.width) << a.c.lg;
  const CachePlan p = make_plan(a.T, a.H, a.c.Hk, a.c.N, a.cu != nullptr, max_len);
  if (p.tiles * a.c.Hk > 0x7fffffffLL / p.splits) return cudaErrorInvalidValue;
  const CacheScratch s = scratch_of(p, a.c.Hk, a.accumulate != 0);
  float *o = nullptr, *scores = nullptr;
  float2* ml = nullptr;
  int32_t* list = nullptr;
  cudaError_t e = cudaSuccess;
  if (s.total) {
    o = static_cast<float*>(ws);
    ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + s.ml);
    if (a.accumulate) scores = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + s.scores);
    if (p.ctas) {
      list = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + s.list);
      e = launch_pdl(plan_kernel, dim3(1), dim3(PLAN_THREADS), 0, stream, a, p, list, err);
      if (e != cudaSuccess) return e;
    }
  }
  const bool cap = a.cap > 0.f;
  e = p.nt == 1   ? launch_variant<1>(cap, a, p, list, o, ml, scores, err, stream)
      : p.nt == 2 ? launch_variant<2>(cap, a, p, list, o, ml, scores, err, stream)
                  : launch_variant<4>(cap, a, p, list, o, ml, scores, err, stream);
  if (e != cudaSuccess || !s.total) return e;
  const int64_t weights = a.accumulate ? static_cast<int64_t>(p.weight_per) * a.c.N * a.c.Hk : 0;
  const int64_t rows = a.T * a.H, row_ctas = p.splits > 16 ? rows : (rows + 3) / 4;
  const int64_t blocks = row_ctas + weights;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_pdl(p.share ? join_kernel<true> : join_kernel<false>, dim3(static_cast<unsigned>(blocks)), dim3(128), 0, stream, a, p,
                    static_cast<unsigned>(row_ctas), static_cast<const float*>(o),
                    static_cast<const float2*>(ml), static_cast<const float*>(scores), err);
}

}  // namespace kda
