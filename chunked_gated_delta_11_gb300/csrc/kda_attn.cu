// kda_attn.cu -- softmax attention over packed rows (kda_attn_fwd) on tcgen05.
//
// A CTA takes (256 query rows of a sequence, head), and then others, 12 warps:
//   warps 0-3, 4-7  the softmax of query tiles 0 and 1 (128 rows each, one thread
//                   a row, tensor-memory lane = row)
//   warp 8          TMA: the two query tiles once, then key and value tiles of
//                   128 rows through two stages each; finds the next piece of work
//   warp 9          the MMAs, issued by one lane (warps 10, 11 fill the warpgroup)
// Per key tile j and query tile t:  S = Q_t K_j^T (A, B in shared memory) into
// tensor memory; the row's thread reads it, takes the running maximum and sum,
// and writes P = 2^(S - m) in bf16 over S; O_t += P V_j (A in tensor memory, B =
// V in its own row order, an MN-major operand).  The two query tiles alternate:
// while the tensor core works for one, the softmax of the other runs.
// Tensor memory: S0 | S1 | O0 | O1, 128 columns each, all 512.
//
// Softmax.  m moves only when a row's maximum may grow by more than 2^16 over it (P
// then stays below 2^16, in bf16's range, and the sum in fp32), so O is rarely
// rescaled; a row thread rescales its own row of O in tensor memory.  P is
// rounded to bf16 (2^-8 of the value at most, as the output once more), the type
// the product takes; its sum is taken in fp32 before that rounding.
//
// Masks.  Every row sees a prefix of its sequence's keys: all of them, up to
// itself, or up to max(itself, prefix_len).  Tiles past a query tile's last
// visible key are skipped, and only tiles that cross a row's limit select.
// Nothing that a row does not see shows in its bits: its reference comes from visible
// scores, and what a warp decides for its 32 rows together changes no arithmetic.
// Rows of V past the sequence's end (another sequence's, whatever they hold)
// are overwritten with zeros in shared memory before the product.
//
// More work.  A CTA that has started asks for the place of one that has not (in the
// order of the grid, so long rows first), and its warps go on from one piece to the
// next by themselves: the next keys and queries are under way during the last
// products, and no barrier or tensor memory is set up again.  Causal documents of
// 256 rows: 71 us as a CTA each, 51 us so (8192 rows, 32 heads); of 1024: 96, 88 us.
//
// Little work.  With fewer pieces than half the SMs a cluster of CTAs shares each piece's
// key tiles; the parts are joined through distributed shared memory, every CTA joining
// some of the channels.
//
// Output.  A row's thread holds all of it; written from there, every store of a warp
// would be 16 bytes of 32 rows (5000 cycles for the 256 rows).  A warp passes half of
// its channels at a time through 4 KB of its own and stores whole lines (3000).
//
// Measured (GB300, replayed from a graph, warm): 8192 tokens causal with bias, 64
// query and 8 KV heads, 712 us = 1.54 PFLOP/s of visible products; the two query
// tiles' chains set it (softmax 1100-1300 cycles a tile, its two products 1024, the
// hand-overs between them about 600, against 2048 cycles of products for both), and
// the products' operands take most of what shared memory can deliver.  8 x 1024
// capped, 32 heads: 98 us; a piece's first tile, with its limits and no reference
// yet, took 4800 cycles where a later one takes 1700 (with a second maximum, over hidden
// scores, that it no longer has), its output 3000.  One sequence of 64 tokens: 6.0 us,
// two launches' worth.
#include <type_traits>

#include "kda_attn.cuh"
#include "kda_tc.cuh"
#include "kda_tma.cuh"

namespace kda {

namespace {

constexpr int AT_ROWS = 128;                   // rows of a query or key tile
constexpr int AT_TILE = AT_ROWS * kDim * 2;    // bytes of a tile (two boxes of 64 channels)
constexpr int AT_BOX = AT_TILE / 2;
constexpr int AT_THREADS = 384;
// three warpgroups of 168 registers a thread at launch; the softmax ones (a row of
// 128 scores in registers) take from the third: 2 x 224 + 56 = 3 x 168
constexpr int AT_REGS_SOFTMAX = 224, AT_REGS_ISSUE = 56;
constexpr int AT_Q = 0, AT_K = 2 * AT_TILE, AT_V = 4 * AT_TILE, AT_CTL = 6 * AT_TILE;
constexpr int AT_OUT_WARP = 32 * 128;          // 32 rows, 64 channels: staging of a warp's output
constexpr int AT_OUT = AT_CTL + 512;
constexpr int AT_SMEM = AT_OUT + 8 * AT_OUT_WARP + 1024;
// What a CTA does: one piece of work; that and others' (more pieces than SMs); or a share
// of the key tiles of one, a cluster of CTAs to a piece (few pieces)
enum { AT_ONE, AT_MORE, AT_SHARE };
constexpr int AT_MAX_SHARES = 8;
constexpr float AT_GROW = 16.0f;               // how far a maximum may outgrow the reference
constexpr float AT_HEAD = 40.0f;               // and how far above it the reference of a row starts that its first tile hides keys from

struct AttnMaps {
  CUtensorMap q, k, v;
};

// What a CTA works on at a time: 256 rows from i0 on of a sequence, and a head.
struct AttnItem {
  int64_t bos;
  int len, prefix;  // len < 0: nothing more
  int i0, h;
  float slope;
};

struct AttnCtl {
  uint64_t q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_full[2], drained;
  uint64_t taken, item_full[2], item_empty[2];
  alignas(16) uint8_t took[16];  // what asking for another CTA's place gave
  AttnItem first, item[2];
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(AttnCtl) <= 512, "control block");
constexpr int AT_READERS = 9;  // of an item: 8 softmax warps and the issuing lane

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float row_max(const uint32_t (&s)[4][32]) {
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int e = 0; e < 32; e += 2)
      m[(e >> 1) & 3] = max3(m[(e >> 1) & 3], __uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]));
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}
// tanh(y) = y (c0 + c1 y^2 + c2 y^4 + c3 y^6) for |y| <= 0.7, fitted for the least
// maximum error: 2.1e-6, which moves a capped score by 3.9e-4 (in units of log2) at
// a cap of 128 and so a weight by a fourteenth of its bf16 rounding.  Five
// multiply-adds a score, where an exponential and a reciprocal take 12 cycles of a
// special-function unit that a tile's weights keep busy already.  For caps up to
// kCapSmall; larger ones take kTanhRel, up to kTanhNear.
constexpr float kTanhMost = 0.7f;
__device__ constexpr float kTanh[4] = {0.999972696f, -0.332557463f, 0.127291387f, -0.0357217971f};

// What a query tile of a sequence sees.
struct TileView {
  int len, prefix, mask;
  // keys that row i (of the sequence) sees: the first limit(i)
  __device__ __forceinline__ int limit(int i) const {
    if (mask == KDA_MASK_FULL) return len;
    const int own = i + 1 > prefix ? i + 1 : prefix;
    return own < len ? own : len;
  }
  // key tiles of the 128 rows from i0 on; 0 past the sequence's end
  __device__ __forceinline__ int tiles(int i0) const {
    if (i0 >= len) return 0;
    const int last = i0 + AT_ROWS < len ? i0 + AT_ROWS - 1 : len - 1;
    return (limit(last) + AT_ROWS - 1) / AT_ROWS;
  }
};

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// What the CTA of `rank` has at the place of this CTA's `local`.
__device__ __forceinline__ uint32_t cluster_place(const void* local, unsigned rank) {
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(local)), "r"(rank));
  return at;
}
__device__ __forceinline__ float2 cluster_read2(const void* local, unsigned rank) {
  float2 x;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(x.x), "=f"(x.y) : "r"(cluster_place(local, rank)));
  return x;
}
__device__ __forceinline__ float4 cluster_read4(const void* local, unsigned rank) {
  float4 x;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
               : "r"(cluster_place(local, rank)));
  return x;
}

// Asks for the place of a CTA of this grid that has not started (one lane).  The
// answer is 16 bytes in ctl->took, counted by ctl->taken.
__device__ __forceinline__ void ask_place(AttnCtl* ctl) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the last answer has been read
  mbar_arrive_expect_tx(&ctl->taken, 16);
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
          smem_u32(ctl->took)),
      "r"(smem_u32(&ctl->taken))
      : "memory");
}

// The answer: that CTA's place, which is now this one's to do; false if there was none
// (it must not be asked for again then).
__device__ __forceinline__ bool place_taken(AttnCtl* ctl, uint32_t& place) {
  uint32_t yes;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}\n"
      : "=r"(yes), "=r"(place)
      : "r"(smem_u32(ctl->took))
      : "memory");
  return yes != 0;
}

template <bool CAP, bool BIAS, int MODE>
__global__ void __launch_bounds__(AT_THREADS, 1)
attn_kernel(const __grid_constant__ AttnMaps maps, AttnArgs a, int64_t slots, int shares, int* err) {
  constexpr bool MORE = MODE == AT_MORE, SHARE = MODE == AT_SHARE;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  AttnCtl* ctl = reinterpret_cast<AttnCtl*>(smem + AT_CTL);
  grid_dep_wait();
  grid_dep_launch();
  const int tid = threadIdx.x, w = tid >> 5, l = tid & 31;
  // The item at a place of the grid (len 0: none).  Long causal rows come last in a
  // sequence: start from the last slot.
  auto item_at = [&](uint32_t place) -> AttnItem {
    AttnItem it;
    it.h = place % a.H;
    const int64_t slot = slots - 1 - place / a.H;
    const int n = seq_of_slot(a.cu, a.T, a.N, 2 * AT_ROWS, 1, slot);
    int64_t eos;
    seq_bounds(a.cu, a.T, a.N, n, it.bos, eos);
    const int64_t first = (slot - (it.bos / (2 * AT_ROWS) + n)) * (2 * AT_ROWS);
    const bool there = first >= 0 && first < eos - it.bos;  // (a malformed cu_seqlens can give less)
    it.len = there ? static_cast<int>(eos - it.bos) : 0;
    it.i0 = there ? static_cast<int>(first) : 0;
    const int p = there && a.mask == KDA_MASK_PREFIX ? __ldg(a.prefix + n) : 0;
    it.prefix = p < 0 ? 0 : (p < it.len ? p : it.len);
    it.slope = BIAS && a.slopes ? __ldg(a.slopes + it.h) * kLog2e : 0.f;
    return it;
  };
  const int rank = SHARE ? static_cast<int>(cluster_rank()) : 0;
  // The key tiles that this CTA takes of an item, last ones first: nj of them, the first
  // being tile top - 1, and the last n0 and n1 of them for the two query tiles.
  struct Tiles {
    int nj, top, n0, n1;
  };
  auto tiles_of = [&](const AttnItem& it) -> Tiles {
    const TileView view{it.len, it.prefix, a.mask};
    const int n0 = view.tiles(it.i0), n1 = view.tiles(it.i0 + AT_ROWS);
    const int nj = n0 > n1 ? n0 : n1;
    if (!SHARE) return {nj, nj, n0, n1};
    const int from = nj * rank / shares, to = nj * (rank + 1) / shares;
    auto part = [&](int nt) {
      const int begin = nj - nt > from ? nj - nt : from;
      return to > begin ? to - begin : 0;
    };
    return {to - from, nj - from, part(n0), part(n1)};
  };
  // The m-th item after the CTA's own, for its readers; false at the end.
  auto next_item = [&](AttnItem& it, int m) -> bool {
    if (!wait_for(&ctl->item_full[m & 1], (m >> 1) & 1, ctl, err)) return false;
    it = ctl->item[m & 1];
    return true;
  };

  if (tid == 0) {
    mbar_init(&ctl->q_full, 1);
    mbar_init(&ctl->drained, 1);
    mbar_init(&ctl->taken, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->k_full[i], 1);
      mbar_init(&ctl->k_empty[i], 1);
      mbar_init(&ctl->v_full[i], 1);
      mbar_init(&ctl->v_empty[i], 1);
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->p_full[i], AT_ROWS);
      mbar_init(&ctl->o_full[i], 1);
      mbar_init(&ctl->item_full[i], 1);
      mbar_init(&ctl->item_empty[i], AT_READERS);
    }
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (w == 8) {
    const AttnItem it = item_at(SHARE ? blockIdx.x / static_cast<unsigned>(shares) : blockIdx.x);
    if (l == 0) ctl->first = it;
  }
  if (w == 9) {
    tmem_alloc(&ctl->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;

  if (w >= 8) {
    regs_give<AT_REGS_ISSUE>();
    if (w == 8) {
      auto tile = [&](int off, const CUtensorMap* map, int head, int64_t tok, uint64_t* bar) {
        tma_box(smem + off, map, 0, head, static_cast<int>(tok), bar);
        tma_box(smem + off + AT_BOX, map, 64, head, static_cast<int>(tok), bar);
      };
      AttnItem it = ctl->first;
      bool ok = true, asked = false;
      int asks = 0;    // answers awaited so far
      int first = 0;   // key tiles of the items before
      int ks = 0, vs = 0, qs = 0;  // tiles issued, over all items
      for (int m = 0;; ++m) {
        if (l == 0) {
          if (MORE) ask_place(ctl);
          const Tiles tiles = tiles_of(it);
          const int nj = tiles.nj, n1 = tiles.n1, end = first + nj, hk = it.h / (a.H / a.Hk);
          auto key_row = [&](int g) { return it.bos + static_cast<int64_t>(tiles.top - 1 - (g - first)) * AT_ROWS; };
          auto load_k = [&]() -> bool {
            if (ks >= 2 && !wait_for(&ctl->k_empty[ks & 1], ((ks >> 1) - 1) & 1, ctl, err)) return false;
            mbar_arrive_expect_tx(&ctl->k_full[ks & 1], AT_TILE);
            tile(AT_K + (ks & 1) * AT_TILE, &maps.k, hk, key_row(ks), &ctl->k_full[ks & 1]);
            ++ks;
            return true;
          };
          if (nj > 0) {
            ok = load_k();
            // the queries' place is free once the last product with them is done
            if (ok && first > 0) ok = wait_for(&ctl->k_empty[(first - 1) & 1], ((first - 1) >> 1) & 1, ctl, err);
            if (ok) {
              mbar_arrive_expect_tx(&ctl->q_full, n1 > 0 ? 2 * AT_TILE : AT_TILE);
              tile(AT_Q, &maps.q, it.h, it.bos + it.i0, &ctl->q_full);
              if (n1 > 0) tile(AT_Q + AT_TILE, &maps.q, it.h, it.bos + it.i0 + AT_ROWS, &ctl->q_full);
              ++qs;
            }
          }
          while (ok && vs < end) {
            if (vs >= 2) ok = wait_for(&ctl->v_empty[vs & 1], ((vs >> 1) - 1) & 1, ctl, err);
            if (!ok) break;
            mbar_arrive_expect_tx(&ctl->v_full[vs & 1], AT_TILE);
            tile(AT_V + (vs & 1) * AT_TILE, &maps.v, hk, key_row(vs), &ctl->v_full[vs & 1]);
            ++vs;
            if (ks < end) ok = load_k();
          }
          first = end;
        }
        if (!MORE) break;
        asked = true;
        // the next item: the place of a CTA that has not started yet
        uint32_t place;
        while (true) {
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          ok = warp_wait(&ctl->taken, asks & 1, ctl, err);
          if (!ok) break;
          ++asks;
          asked = false;
          if (!place_taken(ctl, place)) {
            it.len = -1;
            break;
          }
          it = item_at(place);
          if (it.len > 0) break;
          __syncwarp();
          if (l == 0) ask_place(ctl);
          asked = true;
        }
        __syncwarp();
        if (!ok) break;
        if (l == 0) {
          if (m >= 2) ok = wait_for(&ctl->item_empty[m & 1], ((m >> 1) - 1) & 1, ctl, err);
          if (ok) {
            ctl->item[m & 1] = it;
            mbar_arrive(&ctl->item_full[m & 1]);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok || it.len < 0) break;
      }
      // after a wait that ran out, copies may be in flight: let them land first
      if (l == 0 && !ok) {
        if (asked) mbar_wait(&ctl->taken, asks & 1);
        if (qs > 0) mbar_wait(&ctl->q_full, (qs - 1) & 1);
        for (int i = ks > 2 ? ks - 2 : 0; i < ks; ++i) mbar_wait(&ctl->k_full[i & 1], (i >> 1) & 1);
        for (int i = vs > 2 ? vs - 2 : 0; i < vs; ++i) mbar_wait(&ctl->v_full[i & 1], (i >> 1) & 1);
      }
      __syncwarp();
    } else if (w == 9) {
      const uint32_t sb = smem_u32(smem);
      constexpr uint32_t id_s = make_idesc(1, AT_ROWS, AT_ROWS);
      constexpr uint32_t id_o = make_idesc(1, AT_ROWS, kDim) | (1u << 16);  // B is MN-major
      // One lane issues.  Descriptors are stepped by constants (stage and tile are
      // template values): worked out from the loop's variables they take the lane
      // twice as long as the products themselves.
      const bool one = elect_one();
      const uint64_t qk_desc = make_sdesc(sb, 16, 1024, 2), v_desc = make_sdesc(sb + AT_V, AT_BOX, 1024, 2);
      const uint32_t qk_lo = static_cast<uint32_t>(qk_desc), v_lo = static_cast<uint32_t>(v_desc);
      const uint32_t desc_hi = static_cast<uint32_t>(qk_desc >> 32);  // the same for both
      auto issue_s = [&](auto tile, auto stage) {
        constexpr uint32_t q = (AT_Q + tile.value * AT_TILE) >> 4, k = (AT_K + stage.value * AT_TILE) >> 4;
        constexpr uint32_t B = AT_BOX >> 4;
        const uint32_t d = tmem + tile.value * 128;
        mma_ss_step<q, k>(d, qk_lo, qk_lo, desc_hi, id_s, 0);
        mma_ss_step<q + 2, k + 2>(d, qk_lo, qk_lo, desc_hi, id_s, 1);
        mma_ss_step<q + 4, k + 4>(d, qk_lo, qk_lo, desc_hi, id_s, 1);
        mma_ss_step<q + 6, k + 6>(d, qk_lo, qk_lo, desc_hi, id_s, 1);
        mma_ss_step<q + B, k + B>(d, qk_lo, qk_lo, desc_hi, id_s, 1);
        mma_ss_step<q + B + 2, k + B + 2>(d, qk_lo, qk_lo, desc_hi, id_s, 1);
        mma_ss_step<q + B + 4, k + B + 4>(d, qk_lo, qk_lo, desc_hi, id_s, 1);
        mma_ss_step<q + B + 6, k + B + 6>(d, qk_lo, qk_lo, desc_hi, id_s, 1);
      };
      // 16 keys a step: two groups of 8 rows of 128 bytes; channels 64.. one box further
      auto issue_o = [&](auto tile, auto stage, bool add, int steps) {
        constexpr uint32_t p = tile.value * 128, v = stage.value * (AT_TILE >> 4);
        const uint32_t o = tmem + 256 + p;
        mma_ts_step<p, v>(o, tmem, v_lo, desc_hi, id_o, add);
        if (steps > 1) mma_ts_step<p + 8, v + 128>(o, tmem, v_lo, desc_hi, id_o, 1);
        if (steps > 2) mma_ts_step<p + 16, v + 256>(o, tmem, v_lo, desc_hi, id_o, 1);
        if (steps > 3) mma_ts_step<p + 24, v + 384>(o, tmem, v_lo, desc_hi, id_o, 1);
        if (steps > 4) mma_ts_step<p + 32, v + 512>(o, tmem, v_lo, desc_hi, id_o, 1);
        if (steps > 5) mma_ts_step<p + 40, v + 640>(o, tmem, v_lo, desc_hi, id_o, 1);
        if (steps > 6) mma_ts_step<p + 48, v + 768>(o, tmem, v_lo, desc_hi, id_o, 1);
        if (steps > 7) mma_ts_step<p + 56, v + 896>(o, tmem, v_lo, desc_hi, id_o, 1);
      };
      using N0 = std::integral_constant<uint32_t, 0>;
      using N1 = std::integral_constant<uint32_t, 1>;
      if (one) {
        AttnItem it = ctl->first;
        int first = 0;             // key tiles of the items before
        int rows0 = 0, rows1 = 0;  // the same of query tiles 0 and 1
        for (int m = 0, items = 0;; ++m) {
          const Tiles tiles = tiles_of(it);
          const int nj = tiles.nj, n0 = tiles.n0, n1 = tiles.n1;
          // Step j: the weights times key tile nj - 1 - j's values, in stage `stage`, and the
          // next tile's scores (before step 0 those only).  A query tile that sees fewer key
          // tiles joins in at step nj - nt.  False once a wait has run out.
          auto body = [&](int j, auto stage, auto next) -> bool {
            constexpr uint32_t st = stage.value;
            const int g = first + j;
            int steps = AT_ROWS / 16;
            if (j >= 0) {
              if (!wait_for(&ctl->v_full[st], (g >> 1) & 1, ctl, err)) return false;
              if (j == 0) {
                // the sequence's last keys: zeros in the rows between their end and the last step's
                const int left = it.len - (tiles.top - 1) * AT_ROWS;
                steps = left >= AT_ROWS ? AT_ROWS / 16 : (left + 15) / 16;
                if (left < steps * 16) {
                  for (int r = left; r < steps * 16; ++r)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                      *reinterpret_cast<uint4*>(smem + AT_V + st * AT_TILE + (e & 8 ? AT_BOX : 0) + r * 128 + (e & 7) * 16) = make_uint4(0, 0, 0, 0);
                  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
              }
            }
            if (j + 1 < nj && !wait_for(&ctl->k_full[next.value], ((g + 1) >> 1) & 1, ctl, err)) return false;
            auto tile = [&](auto which, int nt, int rows) -> bool {
              constexpr uint32_t t = which.value;
              const int mine = j - (nj - nt);  // the query tile's own step
              if (mine >= 0) {
                if (!wait_for(&ctl->p_full[t], (rows + mine) & 1, ctl, err)) return false;
                tc_fence_after();
                issue_o(which, stage, mine > 0, steps);
                if (j + 1 == nj) tc_commit(&ctl->o_full[t]);
              }
              // the tensor core runs these in order: S may follow into the columns P is read from
              if (j + 1 < nj && mine + 1 >= 0) {
                issue_s(which, next);
                tc_commit(&ctl->s_full[t]);
              }
              return true;
            };
            if (!tile(N0{}, n0, rows0) || (n1 > 0 && !tile(N1{}, n1, rows1))) return false;
            if (j >= 0) tc_commit(&ctl->v_empty[st]);
            if (j + 1 < nj) tc_commit(&ctl->k_empty[next.value]);
            return true;
          };
          bool ok = true;
          if (nj > 0) {
            ok = wait_for(&ctl->q_full, items & 1, ctl, err);
            ++items;
            for (int j = -1; ok && j < nj; ++j) ok = (first + j) & 1 ? body(j, N1{}, N0{}) : body(j, N0{}, N1{});
          }
          first += nj;
          rows0 += n0;
          rows1 += n1;
          if (!MORE || !ok || !next_item(it, m)) break;
          mbar_arrive(&ctl->item_empty[m & 1]);
          if (it.len < 0) break;
        }
        // nothing may be running in tensor memory when it is freed
        tc_commit(&ctl->drained);
        mbar_wait(&ctl->drained, 0);
      }
      __syncwarp();
    }
    if (SHARE) {
      __syncwarp();
      cluster_sync_all();
      cluster_sync_all();
    }
  } else {
    regs_take<AT_REGS_SOFTMAX>();
    const int t = w >> 2;
    const uint32_t lane = static_cast<uint32_t>((w & 3) * 32) << 16;
    const uint32_t S = tmem + t * 128 + lane, O = tmem + 256 + t * 128 + lane;
    const float c1 = a.scale * kLog2e;
    const float cap2 = CAP ? a.cap * kLog2e : 0.f, per_cap = CAP ? a.scale / a.cap : 0.f;
    const float e1 = CAP ? cap_exponent(a.scale, a.cap) : 0.f;
    const bool large = CAP && a.cap > kCapSmall;
    const float tanh_most = large ? kTanhNear : kTanhMost;
    // multipliers of the one-pass scores: s (k0 + k1 s^2 + k2 s^4 + k3 s^6), or s k0
    const float pc2 = per_cap * per_cap;
    const float w0 = CAP ? (large ? kTanhRel[0] : kTanh[0]) * c1 : c1, w1 = (large ? kTanhRel[1] : kTanh[1]) * c1 * pc2,
                w2 = (large ? kTanhRel[2] : kTanh[2]) * c1 * pc2 * pc2,
                w3 = (large ? kTanhRel[3] : kTanh[3]) * c1 * pc2 * pc2 * pc2;
    const f2 k0 = pair(w0, w0), k1 = pair(w1, w1), k2 = pair(w2, w2), k3 = pair(w3, w3);
    // a positive scale; with a cap, powers of scale / cap that fp32 holds
    const bool usual = c1 > 0.f && (!CAP || (per_cap > 1e-5f && per_cap < 1e5f));
    AttnItem it = ctl->first;
    int tiles = 0, items = 0;  // key tiles, and items with any, so far
    for (int m = 0;; ++m) {
      const TileView view{it.len, it.prefix, a.mask};
      const int i0 = it.i0, all = view.tiles(i0 + t * AT_ROWS);
      int nt = all, high = all;  // key tiles, and the one above the first
      if (SHARE) {
        const Tiles part = tiles_of(it);
        nt = t == 0 ? part.n0 : part.n1;
        high = part.top < all ? part.top : all;
      }
      const int i = i0 + t * AT_ROWS + (tid & 127);  // row of the sequence
      const int limit = view.limit(i);
      const int tile_lo = view.limit(i0 + t * AT_ROWS);  // least limit of the tile's rows
      const float slope = it.slope;
      float ref = -INFINITY, sum = 0.f;
      bool ok = true;
      for (int j = 0; j < nt; ++j) {
        ok = warp_wait(&ctl->s_full[t], (tiles + j) & 1, ctl, err);
        if (!ok) break;
        tc_fence_after();
        const int j0 = (high - 1 - j) * AT_ROWS;
        const int lo = i0 + t * AT_ROWS - j0;  // first row less first column
        // Without a cap the row's 128 scores stay in registers.  With one the usual tile
        // takes them 64 at a time in a loop that stays rolled: unrolled, its code
        // outgrows the instruction caches that the SM's warps share.
        uint32_t s[4][32];
        auto load = [&]() {
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(S + c * 32, s[c]);
          tmem_wait_ld();
        };
        if (!CAP) load();
        f2 parts[2] = {0ull, 0ull};
        // weights of a pair of scores, into their sum and a word of P
        auto weigh = [&](f2 x, f2& acc) -> uint32_t {
          float p0, p1;
          unpair(x, p0, p1);
          p0 = ex2_approx(p0);
          p1 = ex2_approx(p1);
          acc = add2(acc, pair(p0, p1));
          return pack_bf16(p0, p1);
        };
        // The row's reference becomes `top` where it grows: what it has so far follows.
        auto move_ref = [&](bool grow, float top) {
          if (!__any_sync(0xffffffffu, grow)) return;
          const float now = grow ? top : ref;
          const float f = grow ? ex2_approx(ref - now) : 1.f;
          sum *= f;
          ref = now;
          if (j == 0) return;
          // the products of the tiles before are complete (S came after them)
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            tmem_ld32(O + c * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32(O + c * 32, o);
          }
        };
        // The usual tile: no row's limit in it, a bias linear in the column.  From products to
        // weights in one pass, with the largest product found on the way; if that shows that
        // a row's reference had to move, or that the polynomial does not hold somewhere, the
        // warp does the tile again.  What a row gets is the same bits either way unless its
        // own reference moves: the other rows of its warp, which may be another sequence's
        // or see later keys, do not show in it.
        if (j > 0 && j0 + AT_ROWS <= tile_lo && usual && (!BIAS || lo >= AT_ROWS - 1 || lo + AT_ROWS - 1 <= 0)) {
          const float step = lo >= 0 ? slope : -slope;
          const float base = BIAS ? -step * static_cast<float>(i - j0) : 0.f;
          const f2 up = pair(2.f * step, 2.f * step);
          float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          auto under_cap = [&](f2 xx) -> f2 {
            const f2 u = mul2(xx, xx);
            return fma2(u, fma2(u, fma2(u, k3, k2), k1), k0);
          };
          // what the score of column col, and of the next, is off by
          auto offset = [&](float col, float less) -> f2 {
            const float off0 = fmaf(step, col, base - less);
            return pair(off0, off0 + step);
          };
          // weights of 32 columns from column col on
          auto columns = [&](const uint32_t (&x)[32], uint32_t* pk, float col, float less) {
            f2 off = offset(col, less);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float x0 = __uint_as_float(x[e]), x1 = __uint_as_float(x[e + 1]);
              float& mx = m[(e >> 1) & 3];
              mx = CAP ? fmaxf(fmaxf(mx, fabsf(x0)), fabsf(x1)) : max3(mx, x0, x1);
              const f2 xx = pair(x0, x1);
              pk[e >> 1] = weigh(fma2(xx, CAP ? under_cap(xx) : k0, off), parts[(e >> 1) & 1]);
              if (BIAS) off = add2(off, up);
            }
          };
          uint32_t pk[32], first[32];  // CAP: P is written at the end, over scores still needed if it fails
          if (CAP) {
#pragma unroll
            for (int e = 0; e < 32; ++e) pk[e] = 0u;
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
#pragma unroll
              for (int e = 0; e < 32; ++e) first[e] = pk[e];
              tmem_ld32(S + half * 64, s[0]);
              tmem_ld32(S + half * 64 + 32, s[1]);
              tmem_wait_ld();
              columns(s[0], pk, 64.f * half, ref);
              columns(s[1], pk + 16, 64.f * half + 32.f, ref);
            }
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t p16[16];
              columns(s[c], p16, 32.f * c, ref);
              tmem_st16(S + c * 16, p16);
            }
          }
          const float most = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
          // tanh(y) <= y: c1 is the slope of the capped score at 0 too
          const float bound = most * c1 + base + (BIAS ? fmaxf(step * (AT_ROWS - 1.f), 0.f) : 0.f);
          const bool stays = bound <= ref + AT_GROW && ref > -INFINITY;
          if (__all_sync(0xffffffffu, stays && (!CAP || most * per_cap <= tanh_most))) {
            if (CAP) {
              tmem_st32(S, first);
              tmem_st32(S + 32, pk);
            }
          } else if (!CAP) {
            float top = most * c1;
            if (BIAS) {
              float t[2] = {-INFINITY, -INFINITY};
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                f2 off = offset(32.f * c, 0.f);
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                  float x0, x1;
                  unpair(fma2(pair(s[c][e], s[c][e + 1]), k0, off), x0, x1);
                  t[(e >> 1) & 1] = max3(t[(e >> 1) & 1], x0, x1);
                  off = add2(off, up);
                }
              }
              top = fmaxf(t[0], t[1]);
            }
            move_ref(!stays && top > ref, top);
            parts[0] = parts[1] = 0ull;
            const float less = ref == -INFINITY ? 0.f : ref;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t p16[16];
              columns(s[c], p16, 32.f * c, less);
              tmem_st16(S + c * 16, p16);
            }
          } else {
            // scores of a pair with their offsets: the polynomial where it holds, else the exact form
            auto score = [&](const uint32_t& a0, const uint32_t& a1, f2 off) -> f2 {
              const float x0 = __uint_as_float(a0), x1 = __uint_as_float(a1);
              const f2 xx = pair(x0, x1);
              float s0, s1, off0, off1;
              unpair(fma2(xx, under_cap(xx), off), s0, s1);
              unpair(off, off0, off1);
              s0 = fabsf(x0) * per_cap <= tanh_most ? s0 : cap_log2(x0, e1, cap2) + off0;
              s1 = fabsf(x1) * per_cap <= tanh_most ? s1 : cap_log2(x1, e1, cap2) + off1;
              return pair(s0, s1);
            };
            float top = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              tmem_ld32(S + c * 32, s[0]);
              tmem_wait_ld();
              f2 off = offset(32.f * c, 0.f);
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                float x0, x1;
                unpair(score(s[0][e], s[0][e + 1], off), x0, x1);
                top = max3(top, x0, x1);
                if (BIAS) off = add2(off, up);
              }
            }
            move_ref(!stays && top > ref, top);
            parts[0] = parts[1] = 0ull;
            const float less = ref == -INFINITY ? 0.f : ref;
            // P goes over scores that have been read
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t p16[16];
              tmem_ld32(S + c * 32, s[0]);
              tmem_wait_ld();
              f2 off = offset(32.f * c, less);
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                p16[e >> 1] = weigh(score(s[0][e], s[0][e + 1], off), parts[(e >> 1) & 1]);
                if (BIAS) off = add2(off, up);
              }
              tmem_st16(S + c * 16, p16);
            }
          }
        } else {
          if (CAP) load();
          // scores in log2 units
          if (CAP) {
            float m[2] = {0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int e = 0; e < 32; e += 2)
                m[(e >> 1) & 1] = fmaxf(fmaxf(m[(e >> 1) & 1], fabsf(__uint_as_float(s[c][e]))), fabsf(__uint_as_float(s[c][e + 1])));
            // the polynomial, and the exact form where that does not hold for a score
            const bool small = __all_sync(0xffffffffu, usual && fmaxf(m[0], m[1]) * per_cap <= tanh_most);
            if (usual) {
#pragma unroll
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                  const f2 x = pair(s[c][e], s[c][e + 1]), u = mul2(x, x);
                  unpair(mul2(x, fma2(u, fma2(u, fma2(u, k3, k2), k1), k0)), s[c][e], s[c][e + 1]);
                }
            }
            if (!small) {
              const float limit_y = usual ? tanh_most : large ? kTanhNear : -1.f;
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                uint32_t raw[32];
                tmem_ld32(S + c * 32, raw);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                  const float x = __uint_as_float(raw[e]), y = x * per_cap;
                  const float near = usual ? __uint_as_float(s[c][e]) : x * c1 * tanh_ratio(y * y);
                  s[c][e] = __float_as_uint(fabsf(y) <= limit_y ? near : cap_log2(x, e1, cap2));
                }
              }
            }
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int e = 0; e < 32; ++e) s[c][e] = __float_as_uint(__uint_as_float(s[c][e]) * c1);
          }
          if (BIAS) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                s[c][e] = __float_as_uint(fmaf(-slope, fabsf(static_cast<float>(i - j0 - (c * 32 + e))), __uint_as_float(s[c][e])));
          }
          // -inf where the row does not see
          const bool crossed = j0 + AT_ROWS > tile_lo;
          if (crossed) {
            const int left = limit - j0;
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (c * 32 + e >= left) s[c][e] = 0xff800000u;
          }
          // A row that sees few keys of its first tile would move its reference again in the
          // next: it starts that much higher, which costs no accuracy.
          float top = row_max(s);
          if (crossed && ref == -INFINITY) top += AT_HEAD;
          move_ref(top > ref, top);  // ref = -inf: any finite maximum
          // nothing seen yet: every weight is 0
          const float sub = ref == -INFINITY ? 0.f : ref;
          const f2 off = pair(-sub, -sub);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              pk[e >> 1] = weigh(add2(pair(s[c][e], s[c][e + 1]), off), parts[(e >> 1) & 1]);
            tmem_st16(S + c * 16, pk);
          }
        }
        float s0, s1;
        unpair(add2(parts[0], parts[1]), s0, s1);
        sum += s0 + s1;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&ctl->p_full[t]);
      }
      if (SHARE) {
        if (ok && nt > 0) ok = warp_wait(&ctl->o_full[t], 0, ctl, err);
        tc_fence_after();
        // Both tiles' products are complete in all of the CTA: the queries' place takes
        // the rows' references and sums, the keys' and values' their outputs, column
        // groups of 4 by rows.
        named_bar(1, 256);
        const int row = tid & 127;
        uint8_t* stats = smem + AT_Q + (t * AT_ROWS + row) * 8;
        uint8_t* mine = smem + AT_K + t * 2 * AT_TILE + row * 16;
        *reinterpret_cast<float2*>(stats) = make_float2(ok && nt > 0 ? ref : -INFINITY, sum);
        if (ok && nt > 0) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            tmem_ld32(O + c * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<uint4*>(mine + (c * 8 + e) * (AT_ROWS * 16)) = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
        cluster_sync_all();
        // Every CTA joins a share of the channels, the others' parts in order.
        float2 ml[AT_MAX_SHARES];
        float top = -INFINITY, tot = 0.f;
#pragma unroll
        for (int p = 0; p < AT_MAX_SHARES; ++p) {
          ml[p] = make_float2(-INFINITY, 0.f);
          if (p < shares) ml[p] = cluster_read2(stats, p);
          top = fmaxf(top, ml[p].x);
        }
#pragma unroll
        for (int p = 0; p < AT_MAX_SHARES; ++p) {
          ml[p].x = ml[p].x == -INFINITY ? 0.f : ex2_approx(ml[p].x - top);
          tot = fmaf(ml[p].y, ml[p].x, tot);
        }
        const float inv = 1.f / tot;
        const int rows = view.len - (i - l);
        uint8_t* out = smem + AT_OUT + w * AT_OUT_WARP;
        __nv_bfloat16* dst = a.out + ((it.bos + (i - l)) * a.H + it.h) * kDim + (l & 1) * 8;
        for (int c = rank; c < kDim / 16; c += shares) {  // 16 channels
          float4 acc[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int p = 0; p < shares; ++p) {
            float f = 0.f;
#pragma unroll
            for (int x = 0; x < AT_MAX_SHARES; ++x) f = x == p ? ml[x].x : f;
            if (f == 0.f) continue;  // (what a part without a tile left is not its own)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 x = cluster_read4(mine + (c * 4 + e) * (AT_ROWS * 16), p);
              acc[e].x = fmaf(x.x, f, acc[e].x);
              acc[e].y = fmaf(x.y, f, acc[e].y);
              acc[e].z = fmaf(x.z, f, acc[e].z);
              acc[e].w = fmaf(x.w, f, acc[e].w);
            }
          }
#pragma unroll
          for (int e = 0; e < 4; e += 2)
            *reinterpret_cast<uint4*>(out + l * 32 + (((e >> 1) ^ ((l >> 2) & 1)) << 4)) =
                make_uint4(pack_bf16(acc[e].x * inv, acc[e].y * inv), pack_bf16(acc[e].z * inv, acc[e].w * inv),
                           pack_bf16(acc[e + 1].x * inv, acc[e + 1].y * inv), pack_bf16(acc[e + 1].z * inv, acc[e + 1].w * inv));
          __syncwarp();
#pragma unroll
          for (int r = l >> 1; r < 32; r += 16)
            if (r < rows)
              *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(r) * a.H * kDim + c * 16) =
                  *reinterpret_cast<const uint4*>(out + r * 32 + (((l & 1) ^ ((r >> 2) & 1)) << 4));
          __syncwarp();
        }
        cluster_sync_all();  // nobody leaves while its rows are read
      } else if (ok && nt > 0) {
        ok = warp_wait(&ctl->o_full[t], items & 1, ctl, err);  // the last product
        tc_fence_after();
        if (ok) {
          const float inv = 1.f / sum;
          // Rows go out through the warp's own shared memory, half of their channels at a
          // time: a thread's own stores would each be 16 bytes of another row.
          uint8_t* mine = smem + AT_OUT + w * AT_OUT_WARP;
          const int rows = view.len - (i - l);  // of the warp's 32, those there
          __nv_bfloat16* dst = a.out + ((it.bos + (i - l)) * a.H + it.h) * kDim;
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t o[32];
              tmem_ld32(O + half * 64 + c * 32, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t p[4];
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  p[x] = pack_bf16(__uint_as_float(o[e * 8 + 2 * x]) * inv, __uint_as_float(o[e * 8 + 2 * x + 1]) * inv);
                *reinterpret_cast<uint4*>(mine + l * 128 + (((c * 4 + e) ^ (l & 7)) << 4)) = make_uint4(p[0], p[1], p[2], p[3]);
              }
            }
            __syncwarp();
#pragma unroll
            for (int r = l >> 3; r < 32; r += 4)
              if (r < rows)
                *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(r) * a.H * kDim + half * 64 + (l & 7) * 8) =
                    *reinterpret_cast<const uint4*>(mine + r * 128 + (((l & 7) ^ (r & 7)) << 4));
            __syncwarp();
          }
        }
      }
      tiles += nt;
      items += nt > 0;
      // the next item may write P once this one's rows are out of tensor memory
      tc_fence_before();
      if (!MORE) break;
      if (!__all_sync(0xffffffffu, ok && next_item(it, m))) break;
      __syncwarp();
      if (l == 0) mbar_arrive(&ctl->item_empty[m & 1]);
      if (it.len < 0) break;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (w == 9) tmem_dealloc(tmem, 512);
}

template <bool CAP, bool BIAS, int MODE>
cudaError_t launch_one(const AttnMaps& maps, const AttnArgs& a, int64_t slots, int shares, int* err,
                       cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  auto* kernel = attn_kernel<CAP, BIAS, MODE>;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), AT_SMEM, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(slots * a.H * shares));
  cfg.blockDim = dim3(AT_THREADS);
  cfg.dynamicSmemBytes = AT_SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = shares;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = MODE == AT_SHARE ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, maps, a, slots, shares, err);
}

template <int MODE>
cudaError_t launch_mode(const AttnMaps& maps, const AttnArgs& a, int64_t slots, int shares, int* err,
                        cudaStream_t stream) {
  // the plain kernel takes its maximum before the scale, which has to be positive for that
  const bool bias = a.slopes || !(a.scale > 0.f), cap = a.cap > 0.f;
  auto one = cap ? bias ? launch_one<true, true, MODE> : launch_one<true, false, MODE>
                 : bias ? launch_one<false, true, MODE> : launch_one<false, false, MODE>;
  return one(maps, a, slots, shares, err, stream);
}

}  // namespace

cudaError_t launch_attn(const AttnArgs& a, int sm_count, int* err, cudaStream_t stream) {
  AttnMaps maps;
  cudaError_t e = make_tile_map(&maps.q, a.q, a.T, a.H, AT_ROWS);
  if (e == cudaSuccess) e = make_tile_map(&maps.k, a.k, a.T, a.Hk, AT_ROWS);
  if (e == cudaSuccess) e = make_tile_map(&maps.v, a.v, a.T, a.Hk, AT_ROWS);
  if (e != cudaSuccess) return e;
  // sequence n owns the slots of 256 rows from floor(bos_n / 256) + n on
  const int64_t slots = a.cu ? a.T / (2 * AT_ROWS) + a.N
                             : (a.T - a.T / a.N) / (2 * AT_ROWS) + a.N - 1 + (a.T / a.N + 2 * AT_ROWS - 1) / (2 * AT_ROWS);
  if (slots * a.H > 0x7fffffffLL) return cudaErrorInvalidValue;
  const int64_t pieces = slots * a.H;
  // A CTA asks for others' work only where some have to wait for a place: asking and its
  // hand-overs cost the smallest calls 0.8 us (64 tokens: 6.9 us against 6.1 us).
  if (pieces > sm_count) return launch_mode<AT_MORE>(maps, a, slots, 1, err, stream);
  // Few pieces: a cluster to each, as large as idle SMs allow, where its CTAs have two key
  // tiles each and that is worth 3 us of joining (4 heads x 2048 tokens: 26.9 us, shared
  // 16.6 us; 2 x 1024: 15.7 and 12.7 us; 8 x 512: 10.2 and 11.6 us).
  const int64_t tiles = (a.T / a.N + AT_ROWS - 1) / AT_ROWS;
  int64_t shares = pieces > 0 ? sm_count / pieces : 1;
  shares = shares < tiles / 2 ? shares : tiles / 2;
  shares = tiles < 6 ? 1 : shares < AT_MAX_SHARES ? shares : AT_MAX_SHARES;
  return shares > 1 ? launch_mode<AT_SHARE>(maps, a, slots, static_cast<int>(shares), err, stream)
                    : launch_mode<AT_ONE>(maps, a, slots, 1, err, stream);
}

}  // namespace kda
