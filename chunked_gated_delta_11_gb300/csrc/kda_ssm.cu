// kda_ssm.cu -- the state-space recurrence over prompts (kda_ssm_fwd) on tcgen05.
//
// A chunk of 128 tokens at a time.  With d the step sizes and l_i the sum of A d up to
// token i of the chunk (log of the decay since its start), Q its last token:
//
//   Y_i = e^{l_i} M C_i + sum_{j <= i} e^{l_i - l_j} d_j (C_i . B_j) x_j + skip x_i
//   M'  = e^{l_Q} M + sum_j (e^{l_Q - l_j} d_j x_j) B_j^T
//
// A CTA has 128 channels of one sequence (or of a piece of one): two heads of 64 that share
// B and C, or one of 128.  28 warps:
//   warps 0-3    weights: S = C B^T (one thread a row) times e^{l_i - l_j} d_j, per head, in bf16
//                over S in tensor memory
//   warps 4-7    the state, a thread a channel: M' from M and the chunk's sum
//   warps 8-15   the weighted rows x' = e^{l_Q - l_j} d_j x_j, transposed into tensor memory, as
//                the left operand of M' += x'^T B: groups of 32 tokens, each four warps' every other
//   warps 16-23  outputs: e^{l_i} M C_i + skip x_i in tensor memory, then the finished rows, four
//                warps 64 channels
//   warp 24      TMA;  warp 25  the products;  warps 26, 27  step sizes and decays
// Tensor memory: S and P | Y | a chunk's sum x'^T B, 128 columns each, x' (two places of a group), 96,
// and 32 columns of M.
// M is fp32: 64 columns in the state warps' registers, the others (of 128) in tensor and shared memory.
// A chunk's products add up from zero, and their sum comes to M in one rounded fma.  An accumulator
// is cut off, not rounded, at each of a chunk's 24 products: added to M itself they drew it toward
// zero, by 4.2e-5 over 8192 tokens without decay and 2.1e-4 over 32,768.  As it is, M is off by 5e-7
// of its norm however long the sequence.
// (M as bf16 upper halves, which the copy is anyway, and lower ones beside them: 263 us for 16 other
// prompts that take 195; 252 with the output warps at half of the columns.)
// The loops are kept short (rolled, and one copy of what two products share): unrolled,
// the roles' code outgrew the instruction caches (37 % of fetches missed, 9300 cycles a chunk).
//
// Roundings.  x' enters the product with B as the sum of three bf16 numbers, which hold all 24
// bits, so that a state in fp32 is one.  (Fewer where the caller takes the state in bf16 or not at all
// gained 3 %, but the outputs of a call then depended on that.)  P and the copy of M that the outputs
// see are rounded to bf16 once (2^-8 of the value at most, as the output): their error against 64 bits is
// 1.7e-3 to 2.4e-3, where rounding the outputs alone gives 1.66e-3.
// A second addend of P has no columns left in tensor memory, one of the copy no room in shared memory.
//
// Measured (GB300; heads of 64, states of 128 in fp32): 16 ragged prompts, 33,600 tokens, 64 heads,
// 245 us, about 6400 cycles and 12,300 warp instructions a chunk.  The products themselves are 3100
// cycles; one lane issues them in order, at 75 to 100 each, because their operands take most of what
// shared memory delivers beside what the roles read and write there (5300 of 128 bytes a
// chunk), and the order S, M C, x'^T B, P x waits for each role once.  Tried and slower, while the
// same prompts took 235: two lanes that issue the outputs' and the state's products side by side (291
// us), rolled issue loops (247 to 260), 16-token places of x' (266), half of x' before M C (244); no
// faster: eight warps for the weights or for the state.
#include <type_traits>

#include "kda_attn.cuh"
#include "kda_layers.cuh"
#include "kda_tc.cuh"
#include "kda_tma.cuh"

namespace kda {

namespace {

constexpr int SS_TOK = 128;              // tokens of a chunk, channels of a CTA
constexpr int SS_BOX = SS_TOK * 128;     // bytes of 64 elements of 128 rows
constexpr int SS_THREADS = 896;
// seven warpgroups of 72 registers a thread at launch: 88 + 112 + 2 x 64 + 2 x 64 + 48 = 7 x 72
// (PRE: 72 + 112 + 4 x 64 + 56)
constexpr int SS_REGS_WEIGHTS = 88, SS_REGS_STATE = 112, SS_REGS_ROWS = 64, SS_REGS_OUT = 64, SS_REGS_ISSUE = 48;
constexpr uint32_t SS_SP = 0, SS_Y = 128, SS_D = 256, SS_XP = 384, SS_M = 480;  // columns
constexpr int SS_GROUP = 32;             // tokens of a place of x'
constexpr int SS_TERMS = 3;              // addends of x', 16 columns each
constexpr float SS_LEAST = -128.f;       // log2 of the strongest decay that a token counts for

// Steps and decays of a chunk's tokens for one head, in units of log2.  All are sums of A d over the
// tokens in question, and not differences of longer sums, but for those inside 32 tokens.  So
// that such a difference keeps its bits, a token counts for SS_LEAST at most: less than the least
// float is left of anything behind it either way.
struct SsmPrep {
  float2 ld[SS_TOK];  // sum of A d up to the token in its block of 32; its step size, 0 behind the sequence's end
  float w[SS_TOK];   // e^{l_Q - l_j} d_j
  float e[SS_TOK];   // e^{l_i}, l_i from the chunk's start
  float cf[192];     // e^{l_b - l_j} d_j, b the last token before rows 32, 64, 96 (32, 64, 96 of them)
  float keep, pad[3];  // e^{l_Q}
};

struct SsmItem {
  int64_t tok;   // first token
  int len;       // tokens; < 0: nothing to do
  int n, k;      // sequence, piece
  int last;      // its last piece
};

struct SsmCtl {
  uint64_t x_full[2], x_empty[2], b_full[2], b_empty[2], c_full, c_empty, prep_full[2], prep_empty[2];
  uint64_t s_full, p_full, yoff_full, y_scaled, y_full, y_empty, xp_full[4], xp_empty[4], zeroed, start_full, start_read, drained;
  // a chunk's sum is there; M's copy for the next chunk is there and the sum has been read (PRE: two sums in turn)
  uint64_t d_full[2], h_full[2];
  SsmItem item;
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(SsmCtl) <= 512, "control block");

struct SsmMaps {
  CUtensorMap x, b, c, out, init, fin;
};

template <int S>
struct SsmSmem {
  static constexpr int SB = S / 64;
  static constexpr int X = 0, B = 4 * SS_BOX, C = B + 2 * SB * SS_BOX, H = C + SB * SS_BOX;
  static constexpr int M = H + SB * SS_BOX;  // M's last 32 columns of 128, 128 bytes a channel
  static constexpr int PREP = M + (SB - 1) * SS_BOX;
  // PRE: the state so far, fp32, over C and H
  static constexpr int SUM = C;
  static constexpr int CTL = PREP + 4 * static_cast<int>(sizeof(SsmPrep));
  static constexpr int BYTES = CTL + 512 + 1024;
  // A state on its way in or out, 32 rows of 128 bytes at a time: in, over the second places of B and
  // x, which the second chunk's rows wait for; out, over both places of B.
  static constexpr int STATE_BOX = 32 * 128;
  static __device__ __forceinline__ int state_in(int box) {
    return box < SB * 4 ? B + SB * SS_BOX + box * STATE_BOX : X + 2 * SS_BOX + (box - SB * 4) * STATE_BOX;
  }
  static __device__ __forceinline__ int state_out(int box) { return B + box * STATE_BOX; }
};
static_assert(SsmSmem<128>::BYTES <= 227 * 1024, "shared memory");

// A piece's state from zero and its decay, as kept between the two kernels of a split
// pass: [slot][unit][S / 4][128 channels] float4, then [slot][unit][2].
struct SsmParts {
  float* m;
  float* keep;
  const void* init;  // initial states, where the pass does not write
};

__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Four 8 x 8 matrices of bf16, each transposed; a lane's address is a row's.
__device__ __forceinline__ void ldmatrix_t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}

// 16 lanes x 16 columns in the layout that transposed matrices have: r[2 j] and r[2 j + 1] are column
// 4 j + l % 4 of lanes l / 4 and l / 4 + 8.
__device__ __forceinline__ void tmem_st_16x128(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// 16 lanes x 32 columns of 32 bits: r[4 j] and r[4 j + 1] are columns 8 j + 2 (l % 4) and the next of lane l / 4,
// r[4 j + 2] and r[4 j + 3] those of lane l / 4 + 8.
__device__ __forceinline__ void tmem_ld_16x256(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// 32 rows of 64 channels from shared memory, and the wait until they have been read.
__device__ __forceinline__ void tma_store_box(const CUtensorMap* map, int x, int t, const void* src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(t), "r"(smem_u32(src))
               : "memory");
}
__device__ __forceinline__ void tma_prefetch_box(const CUtensorMap* map, int x, int t) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(t)
               : "memory");
}
__device__ __forceinline__ void tma_stores_read() {
  asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
}

// Columns of the weights of 32 keys, block jb of head hh: where the block of S was that they come from.
__device__ __forceinline__ uint32_t weights_at(int hh, int jb) { return SS_SP + 32 * jb + 16 * hh; }

// v - h for a bf16 h.
__device__ __forceinline__ float minus_bf16(float v, uint16_t h) {
  float r;
  asm("fma.rn.f32.bf16 %0, %1, %2, %3;" : "=f"(r) : "h"(h), "h"(static_cast<uint16_t>(0xbf80)), "f"(v));
  return r;
}

// 2^s, s <= 0, to half a step where it is near 1 and counts in many chunks, and to two steps of
// itself where it is not (1 + expm1 would leave nothing of 2^-24 there).
__device__ __forceinline__ float decay_of(float s) { return s > -0.5f ? 1.f + expm1f(s * 0.693147181f) : exp2f(s); }

// One arrival a warp, after all its lanes.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// PRE: only the state that each piece but a sequence's last adds, walking from its last
// chunk to its first, with weights that reach to the piece's end: the chunks' sums, two in turn
// in tensor memory, add up in shared memory.  The output warps join in with x' there, each four with
// a group and a place of its own (8192 tokens, 64 heads, four pieces: 45 us with two places).
template <int P, int S, bool PRE>
__global__ void __launch_bounds__(SS_THREADS, 1)
ssm_kernel(const __grid_constant__ SsmMaps maps, SsmArgs a, SsmParts parts, int64_t piece, int units, bool ranked, int* err) {
  using L = SsmSmem<S>;
  constexpr int HU = SS_TOK / P;  // heads of a unit
  constexpr int SB = L::SB;
  constexpr int SIDES = PRE ? 4 : 2;                // warpgroups of x', and its places
  constexpr uint32_t XP0 = PRE ? SS_SP : SS_XP;     // their columns
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  SsmCtl* ctl = reinterpret_cast<SsmCtl*>(smem + L::CTL);
  SsmPrep* prep = reinterpret_cast<SsmPrep*>(smem + L::PREP);  // [stage][head]
  grid_dep_wait();
  grid_dep_launch();
  const int tid = threadIdx.x, w = tid >> 5, l = tid & 31;
  const int unit = blockIdx.x % units;
  const int64_t slot = blockIdx.x / units;
  const int per_group = a.H / a.G, upg = (per_group + HU - 1) / HU;
  const int g = unit / upg, hu = (unit % upg) * HU, h0 = g * per_group + hu;
  const int nh = per_group - hu < HU ? per_group - hu : HU;  // heads that exist

  if (tid == 0) {
    constexpr int users = PRE ? 16 : 24;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->x_full[i], 1);
      mbar_init(&ctl->x_empty[i], PRE ? 16 : 9);
      mbar_init(&ctl->b_full[i], 1);
      mbar_init(&ctl->b_empty[i], 1);
      mbar_init(&ctl->prep_full[i], HU);
      mbar_init(&ctl->prep_empty[i], users);
    }
    mbar_init(&ctl->c_full, 1);
    mbar_init(&ctl->c_empty, 1);
    mbar_init(&ctl->s_full, 1);
    mbar_init(&ctl->p_full, 4);
    mbar_init(&ctl->yoff_full, 1);
    mbar_init(&ctl->y_scaled, 8);
    mbar_init(&ctl->y_full, 1);
    mbar_init(&ctl->y_empty, 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->d_full[i], 1);
      mbar_init(&ctl->h_full[i], 4);
    }
    for (int i = 0; i < SIDES; ++i) {
      mbar_init(&ctl->xp_full[i], 4);
      mbar_init(&ctl->xp_empty[i], 1);
    }
    mbar_init(&ctl->zeroed, 4);
    mbar_init(&ctl->start_full, 1);
    mbar_init(&ctl->start_read, 4);
    mbar_init(&ctl->drained, 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  // Sequence n owns the slots from floor(bos_n / piece) + n on, one for each of its pieces; whole
  // ones come in the order of their lengths, the longest first.
  const int whole = ranked ? seq_by_rank(a.cu, a.N, static_cast<int>(slot), reinterpret_cast<int*>(smem)) : 0;
  if (w == 24) {
    const int n = ranked ? whole : seq_of_slot(a.cu, a.T, a.N, static_cast<int>(piece), 1, slot);
    int64_t bos, eos;
    seq_bounds(a.cu, a.T, a.N, n, bos, eos);
    const int64_t k = ranked ? 0 : slot - (bos / piece + n), first = k * piece;
    const bool there = k >= 0 && (k == 0 || first < eos - bos);  // (a malformed cu_seqlens can give less)
    const int64_t left = eos - bos - first;
    SsmItem it;
    it.tok = bos + first;
    it.len = there ? static_cast<int>(left < piece ? left : piece) : -1;
    it.n = n;
    it.k = static_cast<int>(k);
    it.last = left <= piece;
    if (PRE && it.last) it.len = -1;
    if (l == 0) ctl->item = it;
  }
  if (w == 26 && l < 6) {
    const CUtensorMap* map = &maps.x + l;
    // (without rows there are no maps of rows, without states none of states)
    const bool used = l < 4 ? a.T > 0 && (l < 2 || !PRE) : !PRE && (l == 4 ? parts.init : a.fin) != nullptr;
    if (used) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
  }
  if (w == 25) {
    tmem_alloc(&ctl->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  const SsmItem it = ctl->item;
  const int nc = it.len > 0 ? (it.len + SS_TOK - 1) / SS_TOK : 0;
  const int64_t part = slot * units + unit;
  // the state that the piece starts from: bytes of a value and of a channel's row, first row
  const int state_size = a.bf16_state ? 2 : 4, state_row = S * state_size;
  const int64_t state_first = (static_cast<int64_t>(it.n) * a.H + h0) * P;
  const bool start = !PRE && parts.init != nullptr && it.len >= 0;
  // the c-th chunk that is worked on, and its tokens
  auto chunk = [&](int c) { return PRE ? nc - 1 - c : c; };
  auto tokens = [&](int c) {
    const int left = it.len - chunk(c) * SS_TOK;
    return left < SS_TOK ? left : SS_TOK;
  };

  if (w >= 24) {
    regs_give<PRE ? 56 : SS_REGS_ISSUE>();
    if (w == 24) {
      if (l == 0) {
        bool ok = true;
        int c = 0, cs = 0;
        if (start) {
          const int rows = nh * P / 32, boxes = rows * (state_row / 128);
          mbar_arrive_expect_tx(&ctl->start_full, boxes * L::STATE_BOX);
          for (int b = 0; b < boxes; ++b)
            tma_box2(smem + L::state_in(b), &maps.init, b / rows * (128 / state_size),
                     static_cast<int>(state_first) + b % rows * 32, &ctl->start_full);
        }
        for (; ok && c < nc; ++c) {
          const int st = c & 1, row = static_cast<int>(it.tok + chunk(c) * SS_TOK);
          const int boxes = P == 64 ? nh : 2;
          // in the order in which their places become free
          if (c >= 2) ok = wait_for(&ctl->b_empty[st], ((c >> 1) - 1) & 1, ctl, err);
          if (c == 1 && start) ok = wait_for(&ctl->start_read, 0, ctl, err);
          if (!ok) break;
          mbar_arrive_expect_tx(&ctl->b_full[st], SB * SS_BOX);
          for (int b = 0; b < SB; ++b)
            tma_box2(smem + L::B + (SB * st + b) * SS_BOX, &maps.b, g * S + b * 64, row, &ctl->b_full[st]);
          if (c + 1 < nc) {  // the next rows come to L2 meanwhile
            const int next = static_cast<int>(it.tok + chunk(c + 1) * SS_TOK);
            for (int b = 0; b < boxes; ++b) tma_prefetch_box(&maps.x, h0 * P + b * 64, next);
          }
          if (c >= 2) ok = wait_for(&ctl->x_empty[st], ((c >> 1) - 1) & 1, ctl, err);
          if (!ok) {
            mbar_wait(&ctl->b_full[st], (c >> 1) & 1);
            break;
          }
          mbar_arrive_expect_tx(&ctl->x_full[st], boxes * SS_BOX);
          for (int b = 0; b < boxes; ++b)
            tma_box2(smem + L::X + (2 * st + b) * SS_BOX, &maps.x, h0 * P + b * 64, row, &ctl->x_full[st]);
          if (!PRE) {
            if (c >= 1) ok = wait_for(&ctl->c_empty, (c - 1) & 1, ctl, err);
            if (!ok) {
              mbar_wait(&ctl->x_full[st], (c >> 1) & 1);
              mbar_wait(&ctl->b_full[st], (c >> 1) & 1);
              break;
            }
            mbar_arrive_expect_tx(&ctl->c_full, SB * SS_BOX);
            for (int b = 0; b < SB; ++b)
              tma_box2(smem + L::C + b * SS_BOX, &maps.c, g * S + b * 64, row, &ctl->c_full);
            ++cs;
          }
        }
        // copies that may be in flight after a wait that ran out land first
        if (start) mbar_wait(&ctl->start_full, 0);
        if (*reinterpret_cast<volatile int*>(&ctl->abort) || !ok) {
          for (int i = c > 2 ? c - 2 : 0; i < c; ++i) {
            mbar_wait(&ctl->x_full[i & 1], (i >> 1) & 1);
            mbar_wait(&ctl->b_full[i & 1], (i >> 1) & 1);
          }
          if (cs > 0) mbar_wait(&ctl->c_full, (cs - 1) & 1);
        }
      }
      __syncwarp();
    } else if (w == 25) {
      if (elect_one()) {
        const uint32_t sb = smem_u32(smem);
        constexpr uint32_t id_s = make_idesc(1, SS_TOK, SS_TOK);
        constexpr uint32_t id_m = make_idesc(1, SS_TOK, S) | (1u << 16);  // B is MN-major
        constexpr uint32_t id_y = make_idesc(1, SS_TOK, P) | (1u << 16);
        const uint64_t rows_desc = make_sdesc(sb, 16, 1024, 2), cols_desc = make_sdesc(sb, SS_BOX, 1024, 2);
        const uint32_t hi = static_cast<uint32_t>(rows_desc >> 32);  // the same for both
        const uint32_t rows_lo = static_cast<uint32_t>(rows_desc), cols_lo = static_cast<uint32_t>(cols_desc);
        constexpr uint32_t BX = SS_BOX >> 4, C0 = L::C >> 4;
        bool ok = true;
        for (int c = 0; c < nc; ++c) {
          const uint32_t st = c & 1;
          const int len = tokens(c);
          const uint32_t b_stage = (L::B >> 4) + st * SB * BX, x_stage = (L::X >> 4) + st * 2 * BX;
          ok = wait_for(&ctl->b_full[st], (c >> 1) & 1, ctl, err);
          if (!ok) break;
          if (!PRE) {
            // C with the rows of B, then with those of the state's copy.  S goes into the columns that the
            // products of the chunk before read P from, and waits until they have ended: products of another
            // shape and accumulator are not ordered by being issued first.
#pragma unroll 1
            for (int of_m = 0; of_m < 2; ++of_m) {
              ok = wait_for(of_m ? &ctl->h_full[0] : &ctl->c_full, c & 1, ctl, err);
              if (ok && c > 0) ok = wait_for(of_m ? &ctl->y_empty : &ctl->y_full, (c - 1) & 1, ctl, err);
              if (!ok) break;
              tc_fence_after();
              const uint32_t d = tmem + (of_m ? SS_Y : SS_SP), b_lo = rows_lo + (of_m ? L::H >> 4 : b_stage);
              mma_ss_step<C0, 0>(d, rows_lo, b_lo, hi, id_s, 0);
              mma_ss_step<C0 + 2, 2>(d, rows_lo, b_lo, hi, id_s, 1);
              mma_ss_step<C0 + 4, 4>(d, rows_lo, b_lo, hi, id_s, 1);
              mma_ss_step<C0 + 6, 6>(d, rows_lo, b_lo, hi, id_s, 1);
              if constexpr (SB == 2) {
                mma_ss_step<C0 + BX, BX>(d, rows_lo, b_lo, hi, id_s, 1);
                mma_ss_step<C0 + BX + 2, BX + 2>(d, rows_lo, b_lo, hi, id_s, 1);
                mma_ss_step<C0 + BX + 4, BX + 4>(d, rows_lo, b_lo, hi, id_s, 1);
                mma_ss_step<C0 + BX + 6, BX + 6>(d, rows_lo, b_lo, hi, id_s, 1);
              }
              tc_commit(of_m ? &ctl->yoff_full : &ctl->s_full);
            }
            if (!ok) break;
            tc_commit(&ctl->c_empty);
          }
          // the chunk's sum: into what the state warps have read (before M's copy was there, or two chunks ago)
          const uint32_t sum = tmem + SS_D + (PRE ? st * 128 : 0);
          if (PRE && c >= 2) ok = wait_for(&ctl->h_full[st], ((c >> 1) - 1) & 1, ctl, err);
          if (!ok) break;
          const int groups = (len + SS_GROUP - 1) / SS_GROUP;
          for (int q = 0; q < groups; ++q) {
            const int place = q % SIDES;  // a whole chunk uses each 4 / SIDES times
            ok = wait_for(&ctl->xp_full[place], (PRE ? c : q >> 1) & 1, ctl, err);
            if (!ok) break;
            tc_fence_after();
            const uint32_t x = tmem + XP0 + place * 48, b_lo = cols_lo + b_stage + q * 256;
            mma_ts_step<0, 0>(sum, x, b_lo, hi, id_m, q > 0);
            mma_ts_step<8, 128>(sum, x, b_lo, hi, id_m, 1);
            mma_ts_step<16, 0>(sum, x, b_lo, hi, id_m, 1);
            mma_ts_step<24, 128>(sum, x, b_lo, hi, id_m, 1);
            mma_ts_step<32, 0>(sum, x, b_lo, hi, id_m, 1);
            mma_ts_step<40, 128>(sum, x, b_lo, hi, id_m, 1);
            tc_commit(&ctl->xp_empty[place]);
          }
          if (!ok) break;
          tc_commit(&ctl->b_empty[st]);
          tc_commit(&ctl->d_full[PRE ? st : 0]);
          if (!PRE) {
            ok = wait_for(&ctl->p_full, c & 1, ctl, err) && wait_for(&ctl->y_scaled, c & 1, ctl, err);
            if (!ok) break;
            tc_fence_after();
            const int steps = (len + 15) / 16;
#pragma unroll 1
            for (int hh = 0; hh < nh; ++hh) {
              const uint32_t d = tmem + SS_Y + hh * 64, p = tmem + weights_at(hh, 0);
              const uint32_t x_lo = cols_lo + x_stage + hh * BX;
              mma_ts_step<0, 0>(d, p, x_lo, hi, id_y, 1);
              if (steps > 1) mma_ts_step<8, 128>(d, p, x_lo, hi, id_y, 1);
              if (steps > 2) mma_ts_step<32, 256>(d, p, x_lo, hi, id_y, 1);
              if (steps > 3) mma_ts_step<40, 384>(d, p, x_lo, hi, id_y, 1);
              if (steps > 4) mma_ts_step<64, 512>(d, p, x_lo, hi, id_y, 1);
              if (steps > 5) mma_ts_step<72, 640>(d, p, x_lo, hi, id_y, 1);
              if (steps > 6) mma_ts_step<96, 768>(d, p, x_lo, hi, id_y, 1);
              if (steps > 7) mma_ts_step<104, 896>(d, p, x_lo, hi, id_y, 1);
            }
            tc_commit(&ctl->y_full);
            tc_commit(&ctl->x_empty[st]);
          }
        }
        // nothing may be running in tensor memory when it is freed
        tc_commit(&ctl->drained);
        mbar_wait(&ctl->drained, 0);
      }
      __syncwarp();
    } else {
      // Step sizes and decays of one head, four tokens to a lane.
      const int hh = w - 26;
      if (hh < HU) {
        const bool there = hh < nh;
        const int h = h0 + (there ? hh : 0);
        const float rate = __ldg(a.A + h) * kLog2e, bias = a.dt_bias ? __ldg(a.dt_bias + h) : 0.f;
        float tail = 0.f;  // of the chunks behind (PRE)
        // raw step sizes are loaded a chunk ahead
        __nv_bfloat16 raw[4], next[4];
        auto load = [&](int c, __nv_bfloat16 (&to)[4]) {
          const __nv_bfloat16* dt = a.dt + (it.tok + chunk(c) * SS_TOK) * a.dt_stride + h;
          const int len = tokens(c);
#pragma unroll
          for (int e = 0; e < 4; ++e) to[e] = there && 4 * l + e < len ? dt[(4 * l + e) * a.dt_stride] : __nv_bfloat16{};
        };
        if (nc > 0) load(0, next);
        for (int c = 0; c < nc; ++c) {
          const int st = c & 1, len = tokens(c);
#pragma unroll
          for (int e = 0; e < 4; ++e) raw[e] = next[e];
          if (c + 1 < nc) load(c + 1, next);
          float d[4], s[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool in = there && 4 * l + e < len;
            d[e] = in ? softplus(__bfloat162float(raw[e]) + bias) : 0.f;
            s[e] = in ? rate * d[e] : 0.f;
            if (s[e] < SS_LEAST) s[e] = SS_LEAST;  // (a NaN stays one)
          }
          // sums up to a token from its block's start, and behind it to the block's end
          float pre[4], suf[4];
          pre[0] = s[0];
          suf[3] = 0.f;
#pragma unroll
          for (int e = 1; e < 4; ++e) {
            pre[e] = pre[e - 1] + s[e];
            suf[3 - e] = suf[4 - e] + s[4 - e];
          }
          const int seat = l & 7;  // eight lanes a block
          float upto = pre[3], from = pre[3];
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) {
            const float x = __shfl_up_sync(0xffffffffu, upto, o), y = __shfl_down_sync(0xffffffffu, from, o);
            if (seat >= o) upto += x;
            if (seat + o < 8) from += y;
          }
          float block[4];  // sums of whole blocks
#pragma unroll
          for (int b = 0; b < 4; ++b) block[b] = __shfl_sync(0xffffffffu, from, 8 * b);
          const float lo = __shfl_up_sync(0xffffffffu, upto, 1), hi = __shfl_down_sync(0xffffffffu, from, 1);
          const float before = seat == 0 ? 0.f : lo, behind = seat == 7 ? 0.f : hi;
          const int mine = l >> 3;
          float first = 0.f, last = tail;  // blocks before and behind the lane's
#pragma unroll
          for (int b = 0; b < 3; ++b) first += b < mine ? block[b] : 0.f;
#pragma unroll
          for (int b = 3; b > 0; --b) last += b > mine ? block[b] : 0.f;
          if (c >= 2 && !warp_wait(&ctl->prep_empty[st], ((c >> 1) - 1) & 1, ctl, err)) break;
          SsmPrep& o = prep[st * 2 + hh];
          float ll[4], ww[4], ee[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            ll[e] = before + pre[e];
            ww[e] = ex2_approx(suf[e] + behind + last) * d[e];
            ee[e] = ex2_approx(first + ll[e]);
          }
          *reinterpret_cast<float4*>(o.w + 4 * l) = make_float4(ww[0], ww[1], ww[2], ww[3]);
          if (!PRE) {
            *reinterpret_cast<float4*>(o.ld + 4 * l) = make_float4(ll[0], d[0], ll[1], d[1]);
            *reinterpret_cast<float4*>(o.ld + 4 * l + 2) = make_float4(ll[2], d[2], ll[3], d[3]);
            *reinterpret_cast<float4*>(o.e + 4 * l) = make_float4(ee[0], ee[1], ee[2], ee[3]);
            float between = 0.f;  // blocks between the lane's and block b
#pragma unroll
            for (int b = 1; b < 4; ++b) {
              if (b - 1 > mine) between += block[b - 1];
              if (b > mine) {
                float f[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] = ex2_approx(suf[e] + behind + between) * d[e];
                *reinterpret_cast<float4*>(o.cf + 16 * b * (b - 1) + 4 * l) = make_float4(f[0], f[1], f[2], f[3]);
              }
            }
          }
          const float all = (block[0] + block[1]) + (block[2] + block[3]);
          if (PRE) tail += all;
          if (l == 0) o.keep = decay_of(all);
          warp_arrive(&ctl->prep_full[st]);
        }
        if (PRE && l == 0 && nc > 0) parts.keep[part * 2 + hh] = decay_of(tail);
      }
      __syncwarp();
    }
  } else if (w < 4) {
    if (!PRE) regs_take<SS_REGS_WEIGHTS>();
    const uint32_t SP = tmem + SS_SP + (static_cast<uint32_t>(w * 32) << 16);
    const int i = w * 32 + l;
    for (int c = 0; !PRE && c < nc; ++c) {
      const int st = c & 1;
      if (!warp_wait(&ctl->prep_full[st], (c >> 1) & 1, ctl, err)) break;
      if (!warp_wait(&ctl->s_full, c & 1, ctl, err)) break;
      tc_fence_after();
      const SsmPrep* pr = prep + st * 2;
      // A lane has columns 8 j + 2 (l % 4) and the next of rows l / 4, + 8, + 16 and + 24: two factors of
      // 8 columns to load, not eight.
      uint32_t s[2][16];
      auto load = [&](int jb) {
        tmem_ld_16x256(SP + jb * 32, s[0]);
        tmem_ld_16x256(SP + jb * 32 + (16u << 16), s[1]);
        tmem_wait_ld();
      };
      const int row = w * 32 + (l >> 2), col = 2 * (l & 3);
      // Blocks of 32 columns before the row's own: e^{l_i - l_b} (e^{l_b - l_j} d_j), two factors
      // that stay below 1.
      float ri[HU][4];
#pragma unroll
      for (int hh = 0; hh < HU; ++hh)
#pragma unroll
        for (int k = 0; k < 4; ++k) ri[hh][k] = ex2_approx(pr[hh].ld[row + 8 * k].x);
#pragma unroll 1
      for (int jb = 0; jb < w; ++jb) {
        load(jb);
#pragma unroll
        for (int hh = 0; hh < HU; ++hh) {
          const float* cf = pr[hh].cf + 16 * w * (w - 1) + jb * 32 + col;
          uint32_t p[2][8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = *reinterpret_cast<const float2*>(cf + 8 * j);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float x0, x1;
              unpair(mul2(pair(s[k >> 1][4 * j + 2 * (k & 1)], s[k >> 1][4 * j + 2 * (k & 1) + 1]),
                          mul2(pair(f.x, f.y), pair(ri[hh][k], ri[hh][k]))),
                     x0, x1);
              p[k >> 1][2 * j + (k & 1)] = pack_bf16(x0, x1);
            }
          }
          tmem_st_16x128(SP + weights_at(hh, jb), p[0]);
          tmem_st_16x128(SP + weights_at(hh, jb) + (16u << 16), p[1]);
        }
      }
      // its own block, the last one of S that it needs
      load(w);
      const int ahead = (l >> 2) - col;  // the lane's first row less its first column
#pragma unroll 1
      for (int hh = 0; hh < HU; ++hh) {
        float li[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) li[k] = pr[hh].ld[row + 8 * k].x;
        const float2* ldj = pr[hh].ld + w * 32 + col;
        uint32_t p[2][8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 f = *reinterpret_cast<const float4*>(ldj + 8 * j);  // of two columns
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t word = 0u;
            if (j <= k) {  // (others are behind the diagonal in every lane)
              // Chosen, not multiplied: S behind the diagonal can hold another sequence's rows, whatever those are.
              // d is a factor and not part of the exponent: a token's own weight is d whatever l is.
              float x0, x1;
              unpair(mul2(pair(s[k >> 1][4 * j + 2 * (k & 1)], s[k >> 1][4 * j + 2 * (k & 1) + 1]),
                          mul2(pair(ex2_approx(li[k] - f.x), ex2_approx(li[k] - f.z)), pair(f.y, f.w))),
                     x0, x1);
              word = pack_bf16(8 * (j - k) <= ahead ? x0 : 0.f, 8 * (j - k) + 1 <= ahead ? x1 : 0.f);
            }
            p[k >> 1][2 * j + (k & 1)] = word;
          }
        }
        tmem_st_16x128(SP + weights_at(hh, w), p[0]);
        tmem_st_16x128(SP + weights_at(hh, w) + (16u << 16), p[1]);
      }
      // and none behind it
#pragma unroll 1
      for (int jb = w + 1; jb < 4; ++jb) {
        uint32_t none[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) none[e] = 0u;
#pragma unroll
        for (int hh = 0; hh < HU; ++hh) tmem_st16(SP + weights_at(hh, jb), none);
      }
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(&ctl->p_full);
      warp_arrive(&ctl->prep_empty[st]);
    }
  } else if (w < 8) {
    regs_take<SS_REGS_STATE>();
    const int r = tid & 127, hh = r / P;  // channel of the unit, its head
    const bool there = hh < nh;
    const uint32_t lanes = static_cast<uint32_t>((w & 3) * 32) << 16;
    const uint32_t D = tmem + SS_D + lanes, M = tmem + SS_M + lanes;
    bool ok = true;
    if (PRE) {
      float4* sum = reinterpret_cast<float4*>(smem + L::SUM) + r;
      float4* dst = reinterpret_cast<float4*>(parts.m) + part * (S / 4) * SS_TOK + r;
      for (int c = 0; ok && c < nc; ++c) {
        ok = warp_wait(&ctl->d_full[c & 1], (c >> 1) & 1, ctl, err);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int cb = 0; cb < S / 32; ++cb) {
          uint32_t d[32];
          tmem_ld32(D + (c & 1) * 128 + cb * 32, d);
          tmem_wait_ld();
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            float4 v = make_float4(__uint_as_float(d[4 * q]), __uint_as_float(d[4 * q + 1]), __uint_as_float(d[4 * q + 2]),
                                   __uint_as_float(d[4 * q + 3]));
            const int at = (cb * 8 + q) * SS_TOK;
            if (c > 0) {
              const float4 u = sum[at];
              v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
            }
            if (c + 1 < nc) sum[at] = v;
            else dst[at] = v;
          }
        }
        tc_fence_before();
        warp_arrive(&ctl->h_full[c & 1]);
      }
    } else if (it.len >= 0) {
      if (start) ok = warp_wait(&ctl->start_full, 0, ctl, err);
      // column `at` (in 16 bytes) of the channel's row of the state that comes in
      auto piece16 = [&](int at) -> uint4 {
        return *reinterpret_cast<const uint4*>(smem + L::state_in((at >> 3) * (nh * P / 32) + (r >> 5)) + l * 128 +
                                               (((at & 7) ^ (l & 7)) << 4));
      };
#pragma unroll 1
      for (int cb = 0; cb < S / 32; ++cb) {
        float m[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) m[e] = 0.f;
        if (start && ok && there) {
          if (a.bf16_state) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint4 x = piece16(cb * 4 + q);
              const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                m[8 * q + 2 * e] = __uint_as_float(u[e] << 16);
                m[8 * q + 2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
              }
            }
          } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const uint4 x = piece16(cb * 8 + q);
              m[4 * q] = __uint_as_float(x.x);
              m[4 * q + 1] = __uint_as_float(x.y);
              m[4 * q + 2] = __uint_as_float(x.z);
              m[4 * q + 3] = __uint_as_float(x.w);
            }
          }
        }
        for (int j = 0; j < it.k; ++j) {
          const int64_t p = (slot - it.k + j) * units + unit;
          const float keep = there ? parts.keep[p * 2 + hh] : 0.f;
          const float4* src = reinterpret_cast<const float4*>(parts.m) + (p * (S / 4) + cb * 8) * SS_TOK + r;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const float4 x = src[q * SS_TOK];
            m[4 * q] = fmaf(m[4 * q], keep, x.x);
            m[4 * q + 1] = fmaf(m[4 * q + 1], keep, x.y);
            m[4 * q + 2] = fmaf(m[4 * q + 2], keep, x.z);
            m[4 * q + 3] = fmaf(m[4 * q + 3], keep, x.w);
          }
        }
        uint32_t u[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(m[e]);
        tmem_st32(D + cb * 32, u);
      }
      tmem_wait_st();
      warp_arrive(&ctl->start_read);
      // Sixteen columns of M each: h < 4 in registers, 4 and 5 in tensor memory, 6 and 7 in shared memory.
      uint32_t m[64];
      auto held = [&](int h, int q) { return reinterpret_cast<uint4*>(smem + L::M + r * 128 + (((4 * (h & 1) + q) ^ (r & 7)) << 4)); };
      auto fetch = [&](int h, uint32_t (&v)[16]) {
        if (h < 4) {
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = m[(16 * h + e) & 63];
        } else if (h < 6) {
          tmem_ld16(M + 16 * (h - 4), v);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint4 x = *held(h, q);
            v[4 * q] = x.x;
            v[4 * q + 1] = x.y;
            v[4 * q + 2] = x.z;
            v[4 * q + 3] = x.w;
          }
        }
      };
      auto store = [&](int h, const uint32_t (&v)[16]) {
        if (h < 4) {
#pragma unroll
          for (int e = 0; e < 16; ++e) m[(16 * h + e) & 63] = v[e];
        } else if (h < 6) {
          tmem_st16(M + 16 * (h - 4), v);
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) *held(h, q) = make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        }
      };
      {
        uint32_t none[16];  // -0: what is added to it stays
#pragma unroll
        for (int e = 0; e < 16; ++e) none[e] = 0x80000000u;
#pragma unroll
        for (int h = 0; h < S / 16; ++h) store(h, none);
        tmem_wait_st();
      }
      // M becomes keep M + the sum in tensor memory: the state that the piece starts from, then chunk after
      // chunk; the last one's M is the state at the end.
      const bool wanted = it.last && a.fin != nullptr;
      for (int c = -1; ok && c < nc; ++c) {
        const int st = c & 1;
        float keep = 1.f;
        if (c >= 0) {
          if (c + 1 == nc && !wanted) break;
          ok = warp_wait(&ctl->prep_full[st], (c >> 1) & 1, ctl, err) && warp_wait(&ctl->d_full[0], c & 1, ctl, err);
          if (!ok) break;
          tc_fence_after();
          keep = prep[st * 2 + hh].keep;
        }
        const f2 keeps = pair(keep, keep);
        uint32_t d[2][16];
        tmem_ld16(D, d[0]);
#pragma unroll
        for (int h = 0; h < S / 16; ++h) {
          uint32_t v[16];
          fetch(h, v);
          tmem_wait_ld();
          if (h + 1 < S / 16) tmem_ld16(D + 16 * (h + 1), d[(h + 1) & 1]);
#pragma unroll
          for (int e = 0; e < 16; e += 2)
            unpair(fma2(pair(v[e], v[e + 1]), keeps, pair(d[h & 1][e], d[h & 1][e + 1])), v[e], v[e + 1]);
          store(h, v);
          uint8_t* dst = smem + L::H + (h >> 2) * SS_BOX + r * 128;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              p[e] = pack_bf16(__uint_as_float(v[8 * q + 2 * e]), __uint_as_float(v[8 * q + 2 * e + 1]));
            *reinterpret_cast<uint4*>(dst + ((((h & 3) * 2 + q) ^ (r & 7)) << 4)) = make_uint4(p[0], p[1], p[2], p[3]);
          }
        }
        tmem_wait_st();
        if (c + 1 < nc) {
          fence_async();
          tc_fence_before();
          warp_arrive(&ctl->h_full[0]);
          if (c >= 0) warp_arrive(&ctl->prep_empty[st]);
        }
      }
      if (ok && nc == 0 && start) ok = warp_wait(&ctl->start_read, 0, ctl, err);  // (it goes out over where it came in)
      if (ok && wanted && there) {
        // out through shared memory, by TMA
        auto out16 = [&](int at) -> uint4* {
          return reinterpret_cast<uint4*>(smem + L::state_out((at >> 3) * (nh * P / 32) + (r >> 5)) + l * 128 +
                                          (((at & 7) ^ (l & 7)) << 4));
        };
#pragma unroll
        for (int h = 0; h < S / 16; ++h) {
          uint32_t v[16];
          fetch(h, v);
          if (a.bf16_state) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint32_t p[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                p[e] = pack_bf16(__uint_as_float(v[8 * q + 2 * e]), __uint_as_float(v[8 * q + 2 * e + 1]));
              *out16(2 * h + q) = make_uint4(p[0], p[1], p[2], p[3]);
            }
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) *out16(4 * h + q) = make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
          }
        }
        fence_async();
        __syncwarp();
        if (l == 0) {
          for (int b = 0; b < state_row / 128; ++b)
            tma_store_box(&maps.fin, b * (128 / state_size), static_cast<int>(state_first) + r,
                          smem + L::state_out(b * (nh * P / 32) + (r >> 5)));
          tma_stores_read();
        }
        __syncwarp();
      }
    }
  } else if (w < 8 + 4 * SIDES) {
    regs_give<SS_REGS_ROWS>();
    const int place = (w - 8) >> 2, wq = w & 3;
    const int r = tid & 127, hh = r / P;
    const uint32_t XP = tmem + XP0 + place * 48 + (static_cast<uint32_t>(wq * 32) << 16);
    // where a lane's row of an 8 x 8 matrix lies, for the warp's first and second 16 channels
    uint32_t at[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int channel = wq * 32 + q * 16 + ((l >> 3) & 1) * 8, token = (l >> 4) * 8 + (l & 7);
      at[q] = (channel >> 6) * SS_BOX + token * 128 + ((((channel & 63) >> 3) ^ (l & 7)) << 4);
    }
    int used = 0;  // groups so far
    for (int c = 0; c < nc; ++c) {
      const int st = c & 1, len = tokens(c);
      if (!warp_wait(&ctl->x_full[st], (c >> 1) & 1, ctl, err)) break;
      uint8_t* x = smem + L::X + 2 * st * SS_BOX;
      if (len < SS_TOK) {
        // rows behind the sequence's end (another's, whatever they hold) take no part in a product
        if (place == 0) {
          if (!warp_wait(&ctl->b_full[st], (c >> 1) & 1, ctl, err)) break;
          if (r >= len) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              *reinterpret_cast<uint4*>(x + (e >> 3) * SS_BOX + r * 128 + (e & 7) * 16) = make_uint4(0, 0, 0, 0);
            uint8_t* b = smem + L::B + SB * st * SS_BOX;
#pragma unroll
            for (int e = 0; e < 8 * SB; ++e)
              *reinterpret_cast<uint4*>(b + (e >> 3) * SS_BOX + r * 128 + (e & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_async();
          warp_arrive(&ctl->zeroed);  // one chunk of a piece at most
        }
        if (!warp_wait(&ctl->zeroed, 0, ctl, err)) break;
      }
      if (!warp_wait(&ctl->prep_full[st], (c >> 1) & 1, ctl, err)) break;
      const float* weight = prep[st * 2 + hh].w + 2 * (l & 3);
      const uint32_t from = smem_u32(x);
      const int groups = (len + SS_GROUP - 1) / SS_GROUP;
      bool ok = true;
#pragma unroll 1
      for (int q = place; q < groups; q += SIDES, ++used) {
        // Transposed on the way into registers: of 16 channels at a time, a lane has tokens 8 j + 2
        // (l % 4) and the next of channels l / 4 and l / 4 + 8.
        uint32_t raw[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) ldmatrix_t(raw[k], from + (q * SS_GROUP + (k >> 1) * 16) * 128 + at[k & 1]);
        float v[2][16];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = *reinterpret_cast<const float2*>(weight + q * SS_GROUP + 8 * j);
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t u = raw[2 * (j >> 1) + k][2 * (j & 1) + e];
              unpair(mul2(pair(u << 16, u & 0xffff0000u), pair(f.x, f.y)), v[k][4 * j + 2 * e], v[k][4 * j + 2 * e + 1]);
            }
        }
        if (used > 0 && !(ok = warp_wait(&ctl->xp_empty[place], (used - 1) & 1, ctl, err))) break;
        tc_fence_after();
        // One bf16 addend after the other, each of what the ones before leave: three hold all 24 bits.
        // (Rolled: unrolled, 16 prompts took 200 us instead of 185.)
#pragma unroll 1
        for (int t = 0; t < SS_TERMS; ++t) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t p[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              p[e] = pack_bf16(v[k][2 * e], v[k][2 * e + 1]);
              v[k][2 * e] = minus_bf16(v[k][2 * e], static_cast<uint16_t>(p[e]));
              v[k][2 * e + 1] = minus_bf16(v[k][2 * e + 1], static_cast<uint16_t>(p[e] >> 16));
            }
            tmem_st_16x128(XP + t * 16 + (static_cast<uint32_t>(k * 16) << 16), p);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(&ctl->xp_full[place]);
      }
      if (!ok) break;
      warp_arrive(&ctl->prep_empty[st]);
      if (PRE) warp_arrive(&ctl->x_empty[st]);
    }
  } else {
    regs_give<SS_REGS_OUT>();
    const int i = tid & 127, side = (w - 16) >> 2;  // row; 64 channels
    const int hh = side * 64 / P;                   // their head
    const bool there = hh < nh;
    const uint32_t Y = tmem + SS_Y + side * 64 + (static_cast<uint32_t>((w & 3) * 32) << 16);
    const float sk = !PRE && a.skip && there ? __ldg(a.skip + h0 + hh) : 0.f;
    const f2 skip = pair(sk, sk);
    for (int c = 0; !PRE && c < nc; ++c) {
      const int st = c & 1, len = tokens(c);
      if (!warp_wait(&ctl->prep_full[st], (c >> 1) & 1, ctl, err)) break;
      if (!warp_wait(&ctl->x_full[st], (c >> 1) & 1, ctl, err)) break;
      if (!warp_wait(&ctl->yoff_full, c & 1, ctl, err)) break;
      tc_fence_after();
      // what the tokens of the chunk add comes on top of e^{l_i} M C_i + skip x_i
      uint8_t* x = smem + L::X + (2 * st + side) * SS_BOX;
      uint8_t* row = x + i * 128;
      const float ei = prep[st * 2 + hh].e[i];
      const f2 f = pair(ei, ei);
#pragma unroll 1
      for (int cb = 0; cb < 2; ++cb) {
        uint32_t y[32];
        tmem_ld32(Y + cb * 32, y);
        tmem_wait_ld();
        if (a.skip) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint4 v = *reinterpret_cast<const uint4*>(row + (((cb * 4 + q) ^ (i & 7)) << 4));
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              unpair(fma2(pair(y[8 * q + 2 * k], y[8 * q + 2 * k + 1]), f, mul2(pair(u[k] << 16, u[k] & 0xffff0000u), skip)),
                     y[8 * q + 2 * k], y[8 * q + 2 * k + 1]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 32; k += 2) unpair(mul2(pair(y[k], y[k + 1]), f), y[k], y[k + 1]);
        }
        tmem_st32(Y + cb * 32, y);
      }
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(&ctl->y_scaled);
      warp_arrive(&ctl->prep_empty[st]);
      if (!warp_wait(&ctl->y_full, c & 1, ctl, err)) break;
      tc_fence_after();
      // The rows take the place of x's, which no product reads any more, and leave from there: 32
      // at a time by TMA, or those of them that are the sequence's own.
#pragma unroll 1
      for (int cb = 0; cb < 2; ++cb) {
        uint32_t y[32];
        tmem_ld32(Y + cb * 32, y);
        tmem_wait_ld();
        if (cb == 1) {
          tc_fence_before();
          warp_arrive(&ctl->y_empty);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t p[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            p[k] = pack_bf16(__uint_as_float(y[8 * q + 2 * k]), __uint_as_float(y[8 * q + 2 * k + 1]));
          *reinterpret_cast<uint4*>(row + (((cb * 4 + q) ^ (i & 7)) << 4)) = make_uint4(p[0], p[1], p[2], p[3]);
        }
      }
      const int rows = len - (i - l);  // of the warp's 32, those there
      const int64_t tok = it.tok + c * SS_TOK + (i - l);
      const uint8_t* first = x + (i - l) * 128;
      fence_async();
      __syncwarp();
      if (there && rows >= 32) {
        if (l == 0) {
          tma_store_box(&maps.out, h0 * P + side * 64, static_cast<int>(tok), first);
          tma_stores_read();
        }
      } else if (there) {
        __nv_bfloat16* dst = a.out + (tok * a.H + h0) * P + side * 64 + (l & 7) * 8;
        for (int q = l >> 3; q < rows; q += 4)
          *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(q) * a.H * P) =
              *reinterpret_cast<const uint4*>(first + q * 128 + (((l & 7) ^ (q & 7)) << 4));
      }
      warp_arrive(&ctl->x_empty[st]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (w == 25) tmem_dealloc(tmem, 512);
}

int units_of(int H, int G, int P) {
  const int per_group = H / G, heads = SS_TOK / P;
  return G * ((per_group + heads - 1) / heads);
}

// How a call is cut: pieces of `piece` tokens (beyond T: sequences stay whole).
struct Plan {
  int64_t piece, slots;
  int units;
  bool split;
  size_t part_bytes, keep_bytes, state_bytes;  // of the workspace
  size_t bytes() const { return split ? part_bytes + keep_bytes + state_bytes : 0; }
};

// Sequences are cut where whole ones would leave SMs without work.  A piece's state from
// zero takes about half of what the piece itself does, each kernel a few chunks' time to
// start and to end, and each piece before one half a chunk's (its state is read); the number
// of pieces is the one of least time under that count.  Whole and cut, in us (heads of 64,
// states of 128): 8192 tokens, 64 heads 190 and 99 (4 pieces; 5 take a second round: 126);
// 16384 tokens, 8 heads 368 and 65 (16); 2048 tokens, 16 heads 51 and 29 (8); 1024 tokens, 64
// heads 29 and 26 (4); four sequences of 2048 tokens, 64 heads 60 and 125 (5, not taken).
Plan plan_of(int64_t T, int H, int G, int N, int P, int S) {
  Plan p{};
  p.units = units_of(H, G, P);
  p.piece = (T / SS_TOK + 1) * SS_TOK;  // (T is below 2^31 - 128)
  p.slots = N;
  const int64_t ctas = static_cast<int64_t>(N) * p.units, chunks = (T / N + SS_TOK - 1) / SS_TOK;
  if (ctas >= kSMs || chunks < 4) return p;
  constexpr int64_t kEnds = 4;  // of half a chunk's time
  int64_t best = 2 * chunks, k_best = 1;
  for (int64_t k = 2; k <= 32 && 2 * k <= chunks; ++k) {
    const int64_t each = (chunks + k - 1) / k;
    const int64_t main = (ctas * k + kSMs - 1) / kSMs * (2 * each + kEnds) + k;
    const int64_t pre = (ctas * (k - 1) + kSMs - 1) / kSMs * (each + kEnds);
    if (main + pre - kEnds < best) {
      best = main + pre - kEnds;
      k_best = k;
    }
  }
  if (k_best == 1) return p;
  p.split = true;
  p.piece = (chunks + k_best - 1) / k_best * SS_TOK;
  p.slots = T / p.piece + N;
  const auto round = [](size_t b) { return (b + 255) & ~static_cast<size_t>(255); };
  p.part_bytes = round(static_cast<size_t>(p.slots) * p.units * SS_TOK * S * 4);
  p.keep_bytes = round(static_cast<size_t>(p.slots) * p.units * 8);
  p.state_bytes = round(static_cast<size_t>(N) * H * P * S * 4);
  return p;
}

template <int P, int S, bool PRE>
cudaError_t launch_one(const SsmMaps& maps, const SsmArgs& a, const SsmParts& parts, const Plan& plan, int* err,
                       cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  auto* kernel = ssm_kernel<P, S, PRE>;
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), SsmSmem<S>::BYTES, done);
  if (e != cudaSuccess) return e;
  const bool ranked = !plan.split && a.cu && a.N > 1 && a.N <= kOrderMaxN;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(plan.slots * plan.units)), dim3(SS_THREADS), SsmSmem<S>::BYTES, stream,
                    maps, a, parts, plan.piece, plan.units, ranked, err);
}

template <int P, int S>
cudaError_t launch(const SsmArgs& a, const Plan& plan, void* ws, int* err, cudaStream_t stream) {
  SsmMaps maps{};
  if (a.T > 0) {
    const int64_t row = static_cast<int64_t>(a.H) * P, wide = static_cast<int64_t>(a.G) * S;
    cudaError_t e = make_matrix_map(&maps.x, a.x, a.T, row, a.x_stride, SS_TOK);
    if (e == cudaSuccess) e = make_matrix_map(&maps.b, a.B, a.T, wide, a.b_stride, SS_TOK);
    if (e == cudaSuccess) e = make_matrix_map(&maps.c, a.C, a.T, wide, a.c_stride, SS_TOK);
    if (e == cudaSuccess) e = make_matrix_map(&maps.out, a.out, a.T, row, row, 32);
    if (e != cudaSuccess) return e;
  }
  SsmParts parts{nullptr, nullptr, a.init};
  const auto state_map = [&](CUtensorMap* map, const void* at) {
    return at ? make_state_map(map, at, static_cast<int64_t>(a.N) * a.H * P, S, a.bf16_state) : cudaSuccess;
  };
  if (plan.split) {
    uint8_t* at = static_cast<uint8_t*>(ws);
    parts.m = reinterpret_cast<float*>(at);
    parts.keep = reinterpret_cast<float*>(at + plan.part_bytes);
    if (a.init && a.init == a.fin) {
      // every piece reads the initial state, and the last may write it before the others have
      void* copy = at + plan.part_bytes + plan.keep_bytes;
      const size_t bytes = static_cast<size_t>(a.N) * a.H * P * S * (a.bf16_state ? 2 : 4);
      const cudaError_t e = cudaMemcpyAsync(copy, a.init, bytes, cudaMemcpyDeviceToDevice, stream);
      if (e != cudaSuccess) return e;
      parts.init = copy;
    }
    const cudaError_t e = launch_one<P, S, true>(maps, a, parts, plan, err, stream);
    if (e != cudaSuccess) return e;
  }
  cudaError_t e = state_map(&maps.init, parts.init);
  if (e == cudaSuccess) e = state_map(&maps.fin, a.fin);
  if (e != cudaSuccess) return e;
  return launch_one<P, S, false>(maps, a, parts, plan, err, stream);
}

}  // namespace

size_t ssm_workspace(int64_t T, int H, int G, int N, int P, int S) { return plan_of(T, H, G, N, P, S).bytes(); }

cudaError_t launch_ssm_fwd(const SsmArgs& a, int P, int S, void* ws, int* err, cudaStream_t stream) {
  const Plan plan = plan_of(a.T, a.H, a.G, a.N, P, S);
  if (plan.slots * plan.units > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (P == 64) return S == 64 ? launch<64, 64>(a, plan, ws, err, stream) : launch<64, 128>(a, plan, ws, err, stream);
  return S == 64 ? launch<128, 64>(a, plan, ws, err, stream) : launch<128, 128>(a, plan, ws, err, stream);
}

}  // namespace kda
