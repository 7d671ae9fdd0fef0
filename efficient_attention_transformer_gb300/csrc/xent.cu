// Softmax cross entropy of the logits X W^T over a vocabulary, with the
// gradients of X [N, d] and W [V, d]:
//   l = x W^T     loss = log sum_v exp(l_v) - l_y
//   dX_i = g (sum_v p_iv W_v - W_y)      dW_v = g sum_i (p_iv - [v = y_i]) x_i
//
// Tokens without a label cost nothing: xent_gather_kernel first copies the
// others' rows behind one another (their number stays on the device, and the
// kernels behind it take their tile counts from there).  The rows are then
// taken in pieces, so that no more than a piece's [tokens, V] is held at any
// time, and the logits themselves are never stored.
//
// The logits are formed once, 6 N d V operations in all: the product's
// epilogue needs the row's normaliser for p = exp(l - lse), which is known
// only after the last word, so it writes E = exp(l - ref) with a reference
// that is known before the product, the label's logit t (a dot product a row,
// in the gather).  E rounded to bf16 keeps its relative precision whatever
// its size, and sum_v p_v >= p_y makes sum_v E >= 1: nothing that counts is
// lost below.  Above, a (row, 128 words) whose largest l exceeds t by 40
// takes that largest l as its reference instead, writes it beside its sum,
// and xent_rows_kernel rescales such rows' E to the row's largest reference
// afterwards.  The rest is linear:
//   Zx = sum_{v != y} E_v, Z = E_y + Zx, loss = log Z + ref - t
//        (log1p(Zx) where the reference is t: exact for sure predictions),
//   E_y := -Zx (p_y - 1 = -Zx / Z without cancellation),
//   dX_i = (g / Z_i) sum_v E_iv W_v         (scaled when the parts are joined)
//   dW_v = sum_i E_iv (g / Z_i) x_i         (x scaled and rounded once)
// Roundings with bf16 io: E, the scaled x, and the results, to bf16.  The
// label's term outweighs the others, so its E's rounding is taken out again:
// in dX as a multiple of the label's row of W, in dW by the row's factor
// (which puts that half step on the other words' terms there).
//
// All three products run on the 2-SM tcgen05 tiles of the layer's projection
// (256 x 256 of a CTA pair, 64-deep k-blocks by TMA into a 6-stage ring, two
// TMEM accumulators, 8 epilogue warps a CTA).  Every extent may be ragged:
// what is behind an edge is zero (TMA's fill, or padding) and stores are
// clipped.
//
// fp32 io runs on the same tiles.  An fp32 value is the sum of three bf16
// ones, x = x1 + x2 + x3 (8 + 8 + 8 bits), kept side by side, and a product
// of two such sums is taken as the six products that matter, x1 w1, x1 w2,
// x2 w1, x2 w2, x1 w3, x3 w1: what is left out is below 2^-24 of a term, as
// an fp32 product's rounding is.  The small products come first, so that the
// accumulator's own rounding meets few large partial sums.  Six passes at the
// bf16 rate are four times the fp32 units' (1931 / 6 against 80 TFLOP/s).
//
// A few tokens without gradients (xent_few_kernel) only read W: dot products
// on the CUDA cores.
//
// Measured (bf16, V 50257, loss and both gradients), back to back under the
// power cap: 8192 tokens of d 768 1.27 ms at 1440 MHz, 429 us of it up to the
// rows' sums, 424 for dX and 414 for dW; 16384 tokens of d 1024, a tenth
// without label, 2.92 ms at 1410 MHz, 997, 952 and 974.  The tensor pipe
// bounds them.
#include <cuda_bf16.h>

#include <atomic>

#include "flash_gau_internal.h"
#include "packed_f32.cuh"
#include "sm103_ptx.cuh"
#include "tma_host.h"

namespace flashgau {
namespace {

using namespace ptx;

constexpr int BM = 128, BN = 256, BK = 64, STAGES = 6;
constexpr int A_BYTES = BM * BK * 2;
constexpr int BOX_BYTES = 64 * 64 * 2;
constexpr int STAGE_BYTES = A_BYTES + BN / 2 * BK * 2;
constexpr int ACC_COLS = 256, TMEM_COLS = 2 * ACC_COLS;
constexpr int EPI_WARPS = 8, NUM_THREADS = 32 * (2 + EPI_WARPS);
constexpr int STG_BYTES = 32 * 128;
constexpr int TILE_BYTES = STAGES * STAGE_BYTES + EPI_WARPS * STG_BYTES;
constexpr int SMEM_BYTES = TILE_BYTES + 1024 + 256;
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory of one CTA");
constexpr uint16_t kPair = 0x3, kLeader = 0x1;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kRaise = 40.0f * kLog2e;  // how far above the label's logit E is kept to it

// kLoss: the logits' product, sums only; kProbs: sums and E; kDX: E W as
// fp32 parts; kDW: E^T X', stored in bf16, or in fp32, or added to fp32
// (kLoss3, kProbs3: of fp32 io, E as three terms)
enum Epi { kLoss, kProbs, kLoss3, kProbs3, kDX, kDW };
constexpr bool is_logits3(int epi) { return epi == kLoss3 || epi == kProbs3; }
constexpr bool is_logits(int epi) { return epi == kLoss || epi == kProbs || is_logits3(epi); }

// fp32 io adds up a tile's logits over several works (see kFp32Blocks): an
// epilogue thread's 128 of them, 64 in registers and 64 in shared memory, in
// the place of the ring's last two stages, or without stores of its last one
// and of the stores' staging.
constexpr int kSumColumns = 64;
constexpr int stages_of(int epi) {
  return epi == kProbs3 ? STAGES - 2 : epi == kLoss3 ? STAGES - 1 : STAGES;
}
static_assert(EPI_WARPS * kSumColumns * 32 * sizeof(float) == 2 * STAGE_BYTES &&
                  EPI_WARPS * STG_BYTES == STAGE_BYTES,
              "sums of the logits");

constexpr int kTerms = 3, kProducts = 6;  // of an fp32 value; of two

struct Params {
  // M rows of the result, N columns, K deep.  The side that tokens are on is
  // what *live leaves of `rows` from `first` on.
  int M, N, K;
  const int *live;
  long long first;
  int rows;
  int products;            // 1, or kProducts with operands' terms side by side
  int a_term, b_term;      // columns from one term of an operand to the next
  const float *ref;        // the label's logit in units of ln 2
  const int *labels;
  float2 *part;            // [N / 128, rounded up][rows] (reference, sum without the label)
  int e_term;              // kProbs: columns between E's terms
  int fp32;                // kDW: fp32 result
  int add;                 // kDW: add to the fp32 result
  int *status;
};

// which terms of A and B a product takes, the small ones first
__device__ __forceinline__ void terms_of(const Params &p, int product, int &a, int &b) {
  if (p.products == 1) {
    a = b = 0;
    return;
  }
  constexpr uint32_t kA = 0x001102u, kB = 0x010120u;  // product k: hex digit k
  a = (int)(kA >> (4 * product) & 15u);
  b = (int)(kB >> (4 * product) & 15u);
}

// dX's sum over the words is long and its tiles are few, so what does not fill
// a round of them is dealt out by k-blocks.  `nt` pairs (one for each 256
// columns) form a group.  Each group takes whole row pairs as long as there is
// one for every group, all at the same words, whose rows of W they share in
// L2; the sums of the row pairs left are laid end to end and cut into runs of
// `run` k-blocks, one a group.  A row pair that groups share has a part from
// each, at index row pair + group (each step along the runs raises one or the
// other, so no two parts meet); a whole one is the part of its own index.
struct DxPlan {
  int row_pairs, nt, groups;
  int rounds;   // of whole row pairs
  int steps;    // k-blocks of a row pair
  int run;
  int runs;     // groups that have one
  __host__ __device__ int first_left() const { return rounds * groups; }
};
__host__ __device__ inline DxPlan dx_plan(int rows, int d, int V, int products, int pairs) {
  DxPlan q;
  q.row_pairs = (rows + 2 * BM - 1) / (2 * BM);
  q.nt = (d + BN - 1) / BN;
  q.steps = products * ((V + BK - 1) / BK);
  q.groups = pairs / q.nt > 0 ? pairs / q.nt : 1;
  q.rounds = q.row_pairs / q.groups;
  const int total = (q.row_pairs - q.first_left()) * q.steps;  // under 2^7 * 2^19
  q.run = (total + q.groups - 1) / q.groups;
  if (q.run < 8) q.run = 8;
  q.runs = (total + q.run - 1) / q.run;
  return q;
}
constexpr int kPlanPairs = kXentPlanSms / 2;

struct Smem {
  uint64_t full[STAGES], empty[STAGES];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  volatile int abort_flag;
};

__device__ __forceinline__ void raise_timeout(Smem *sm, int *status) {
  sm->abort_flag = 1;
  atomicExch(status, FLASH_GAU_ETIMEOUT);
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// A piece of work of one pair: the product of k-blocks k0 .. k1 for 256 rows
// and nsz columns.
struct Work {
  int rp, n0, nsz;
  int k0, k1;
  int part;   // kDX: where the result goes
  bool add;   // it adds to what the work before has left there
  bool last;  // of this product, or share of one
};
// The tensor cores cut off what an accumulator cannot hold at each step, so
// a long sum comes out short, by 6e-8 of itself a k-block (fp32 io, 1400
// k-blocks: 8e-5).  With fp32 io the large product of a sum is therefore
// taken in works of few k-blocks, which add up in memory (gradients) or in
// the epilogue's registers (logits); the five small products before it lose
// nothing that counts and go into its first
// (1001 tokens, 8003 words, d = 520, errors of dX and dW: 16 k-blocks 1.4e-6
// and 1.1e-6 in 201 us, 8 0.8e-6 and 0.6e-6 in 219 us, 4 0.4e-6 and 0.3e-6 in
// 280 us, each 10 less with W's terms written by the gather's launch; the
// logits in works of 8 too, whose error grows with d otherwise, 2% more).
constexpr int kFp32Blocks = 8;

// The works of one pair, in order.  Every role of the kernel walks the same.
template <int EPI>
struct Walk {
  const Params &p;
  int M, row_pairs, n_tiles, step;
  int steps;     // k-blocks of a whole product
  int large;     // the first k-block of a work's limit (see kFp32Blocks)
  unsigned u;    // next tile (kDX: unit, a group's columns)
  int pos, end;  // k-blocks of what is under way
  int rp, n0, part;
  // kDX
  int round, run_pos, run_end;
  DxPlan dx;
  __device__ Walk(const Params &params) : p(params) {
    const long long left = *reinterpret_cast<const volatile int *>(p.live) - p.first;
    const int tokens = left < 0 ? 0 : left < p.rows ? (int)left : p.rows;
    u = blockIdx.x / 2;
    step = gridDim.x / 2;
    pos = end = 0;
    M = EPI == kDW ? p.M : tokens;
    n_tiles = (p.N + BN - 1) / BN;
    row_pairs = (M + 2 * BM - 1) / (2 * BM);
    const int K = EPI == kDW ? tokens : p.K;
    steps = p.products * ((K + BK - 1) / BK);
    large = p.products == 1 ? 0x7fffffff : steps / p.products * (p.products - 1);
    if (EPI == kDX) {
      dx = dx_plan(tokens, p.N, p.K, p.products, kPlanPairs);
      round = run_pos = run_end = 0;
      start_unit();
    }
  }
  __device__ void start_unit() {
    const int g = (int)(u / dx.nt);
    n0 = (int)(u % dx.nt) * BN;
    round = 0;
    run_pos = g * dx.run;
    run_end = min(run_pos + dx.run, (dx.row_pairs - dx.first_left()) * dx.steps);
    part = g;
  }
  // the next row pair, or share of one
  __device__ bool advance_dx() {
    for (;;) {
      if (u >= (unsigned)(dx.groups * dx.nt)) return false;
      const int g = (int)(u / dx.nt);
      if (round < dx.rounds) {
        rp = part = round++ * dx.groups + g;
        pos = 0;
        end = dx.steps;
        return true;
      }
      if (run_pos < run_end) {
        const int q = run_pos / dx.steps;
        rp = dx.first_left() + q;
        part = rp + g;
        pos = run_pos - q * dx.steps;
        end = min(dx.steps, pos + run_end - run_pos);
        run_pos += end - pos;
        return true;
      }
      u += step;
      start_unit();
    }
  }
  __device__ bool next(Work &w) {
    w.add = EPI == kDW && p.add;
    if (pos == end) {
      if (EPI == kDX) {
        if (!advance_dx()) return false;
      } else {
        if (u >= (unsigned)row_pairs * n_tiles) return false;
        if (EPI == kDW) {
          n0 = (int)(u % n_tiles) * BN;
          rp = (int)(u / n_tiles);
        } else {
          // rows fastest: the pairs share a tile of W while X stays in L2
          rp = (int)(u % row_pairs);
          n0 = (int)(u / row_pairs) * BN;
        }
        pos = 0;
        end = steps;
        u += step;
      }
    } else {
      w.add = true;
    }
    w.rp = rp;
    w.n0 = n0;
    w.part = part;
    w.k0 = pos;
    w.k1 = end;
    if (end > large) w.k1 = min(end, max(pos, large) + kFp32Blocks);
    pos = w.k1;
    w.last = pos == end;
    // a multiple of 128: each CTA holds whole 64-column boxes; the logits'
    // sums are kept by 128 words, so their tiles are never narrower
    w.nsz = is_logits(EPI) ? BN : min(BN, (p.N - n0 + 127) / 128 * 128);
    return true;
  }
  // k-block s of a product: which term pair, and the depth in it
  __device__ void locate(int s, int &product, int &k) const {
    const unsigned per = (unsigned)(EPI == kDX ? dx.steps : steps) / p.products;
    product = p.products == 1 ? 0 : (int)((unsigned)s / per);
    k = (int)((unsigned)s - product * per) * BK;
  }
};

// Stores one 32-row x 128-byte box from a warp's staging buffer.
struct Stager {
  uint8_t *buf;
  int lane;
  __device__ void begin() {
    if (lane == 0) tma_store_wait_read<0>();
    __syncwarp();
  }
  __device__ void put(int c, uint4 w) { *reinterpret_cast<uint4 *>(buf + sw128_offset(lane, c)) = w; }
  __device__ void finish(const CUtensorMap *tm, int x, int y, bool add) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (add) tma_reduce_add_2d(tm, smem_u32(buf), x, y);
      else tma_store_2d(tm, smem_u32(buf), x, y);
      tma_store_commit();
    }
  }
};

// 32 values as bf16 into columns 8 c0 .. of this lane's row of a box
__device__ __forceinline__ void put32(Stager &st, int c0, const float (&e)[32]) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    st.put(c0 + q, make_uint4(pack_bf16(e[8 * q], e[8 * q + 1]), pack_bf16(e[8 * q + 2], e[8 * q + 3]),
                              pack_bf16(e[8 * q + 4], e[8 * q + 5]),
                              pack_bf16(e[8 * q + 6], e[8 * q + 7])));
}

template <int EPI>
__global__ void __launch_bounds__(NUM_THREADS, 1)
xent_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const __grid_constant__ CUtensorMap tmC, const Params p) {
  constexpr bool A_MN = EPI == kDW;                     // E read by columns
  constexpr bool B_KM = is_logits(EPI);                 // W read by rows
  constexpr int kStages = stages_of(EPI);
  extern __shared__ uint8_t smem_raw[];
  uint8_t *tiles = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Smem *sm = reinterpret_cast<Smem *>(tiles + TILE_BYTES);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = (int)cluster_ctarank();
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&sm->full[i]), 1);
      mbar_init(smem_u32(&sm->empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sm->acc_full[i]), 1);
      mbar_init(smem_u32(&sm->acc_empty[i]), 2 * EPI_WARPS);
    }
    mbar_init(smem_u32(&sm->drain), 1);
    sm->abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&sm->tmem_base), TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  griddep_wait();
  const uint32_t tmem_base = sm->tmem_base;
  Walk<EPI> walk(p);
  Work x;

  if (warp == 0) {
    // ------------------------------------------------ TMA producer (both)
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      while (!sm->abort_flag && walk.next(x)) {
        const int m0 = (x.rp * 2 + rank) * BM, half = x.nsz / 2, hboxes = half / 64;
        for (int s = x.k0; s < x.k1; ++s) {
          int product, k, ta, tb;
          walk.locate(s, product, k);
          terms_of(p, product, ta, tb);
          ta *= p.a_term;
          tb *= p.b_term;
          if (!mbar_wait(smem_u32(&sm->empty[stage]), phase ^ 1, &sm->abort_flag)) {
            raise_timeout(sm, p.status);
            break;
          }
          const uint32_t full_own = smem_u32(&sm->full[stage]);
          const uint32_t full_leader = mapa_shared(full_own, 0);
          uint8_t *sA = tiles + stage * STAGE_BYTES;
          uint8_t *sB = sA + A_BYTES;
          // a K-major B box is always 128 rows
          const uint32_t b_bytes = B_KM ? 2 * BOX_BYTES : hboxes * BOX_BYTES;
          if (leader) mbar_arrive_expect_tx(full_own, 2 * (A_BYTES + b_bytes));
          if (A_MN) {
            tma_load_2d_pair(smem_u32(sA), &tmA, full_leader, ta + m0, k);
            tma_load_2d_pair(smem_u32(sA + BOX_BYTES), &tmA, full_leader, ta + m0 + 64, k);
          } else {
            tma_load_2d_pair(smem_u32(sA), &tmA, full_leader, ta + k, m0);
          }
          if (B_KM) {
            tma_load_2d_pair(smem_u32(sB), &tmB, full_leader, tb + k, x.n0 + rank * half);
          } else {
            for (int j = 0; j < hboxes; ++j)
              tma_load_2d_pair(smem_u32(sB + j * BOX_BYTES), &tmB, full_leader,
                               tb + x.n0 + rank * half + j * 64, k);
          }
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer (leader)
    if (leader && elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      int local = 0;
      Work following;
      bool more = walk.next(x);
      for (; more && !sm->abort_flag; ++local, x = following) {
        const int acc = local & 1;
        if (!mbar_wait(smem_u32(&sm->acc_empty[acc]), ((local >> 1) & 1) ^ 1, &sm->abort_flag)) {
          raise_timeout(sm, p.status);
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * ACC_COLS;
        const uint32_t idesc = idesc_bf16_f32(2 * BM, x.nsz, A_MN ? 1 : 0, B_KM ? 0 : 1);
        bool ok = true;
        for (int s = x.k0; s < x.k1; ++s) {
          if (!mbar_wait(smem_u32(&sm->full[stage]), phase, &sm->abort_flag)) {
            raise_timeout(sm, p.status);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sA = smem_u32(tiles + stage * STAGE_BYTES);
          const uint64_t da = A_MN ? sw128_desc(sA, BOX_BYTES, 1024) : sw128_desc(sA, 16, 1024);
          const uint64_t db = B_KM ? sw128_desc(sA + A_BYTES, 16, 1024)
                                   : sw128_desc(sA + A_BYTES, BOX_BYTES, 1024);
#pragma unroll
          for (int k = 0; k < BK / 16; ++k)
            mma_f16_ss_pair(d_tmem, desc_advance(da, k * (A_MN ? 2048 : 32)),
                            desc_advance(db, k * (B_KM ? 32 : 2048)), idesc,
                            s != x.k0 || k != 0);
          mma_commit_pair_mc(smem_u32(&sm->empty[stage]), kPair);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
          // found while the tensor cores work, not between two works
          if (s == x.k0) more = walk.next(following);
        }
        if (!ok) break;
        mma_commit_pair_mc(smem_u32(&sm->acc_full[acc]), kPair);
        if (x.k0 == x.k1) more = walk.next(following);
      }
      mma_commit_pair_mc(smem_u32(&sm->drain), kLeader);
      if (!mbar_wait(smem_u32(&sm->drain), 0)) raise_timeout(sm, p.status);
    }
  } else {
    // -------------------------------------------------- epilogue (both)
    const int quarter = warp & 3;
    const int half = (warp - 2) >> 2;
    Stager st{tiles + STAGES * STAGE_BYTES + (warp - 2) * STG_BYTES, lane};
    int local = 0;
    // fp32 io: this row's 128 logits, a work's share added to those before;
    // column c of the second 64 at far[32 c]
    float near[is_logits3(EPI) ? 2 : 1][32];
    float *const far = reinterpret_cast<float *>(tiles + kStages * STAGE_BYTES) +
                       (warp - 2) * kSumColumns * 32 + lane;
    for (; !sm->abort_flag && walk.next(x); ++local) {
      const int acc = local & 1;
      const int row0 = (x.rp * 2 + rank) * BM + quarter * 32, row = row0 + lane;
      const int c_begin = half * (x.nsz / 2), c_end = c_begin + x.nsz / 2;
      const bool live = row < walk.M;
      // this row's scalars, before the wait
      float ref = 0.f;
      int label = -1;
      if constexpr (is_logits(EPI)) {
        if (live) {
          ref = p.ref[row];
          label = p.labels[row];
        }
      }
      if (!mbar_wait(smem_u32(&sm->acc_full[acc]), (local >> 1) & 1, &sm->abort_flag)) {
        raise_timeout(sm, p.status);
        break;
      }
      tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16) + acc * ACC_COLS;
      auto drained = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&sm->acc_empty[acc]), 0));
      };
      if constexpr (is_logits(EPI)) {
        const bool whole = x.n0 + c_end <= p.N;  // every column is a word
        // the largest logit of this row's 128 words
        float top = -INFINITY;
        auto largest = [&](int c, const auto &l) {
          if (whole) {
#pragma unroll
            for (int j = 0; j < 32; ++j) top = fmaxf(top, l(j));
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (x.n0 + c + j < p.N) top = fmaxf(top, l(j));
          }
        };
        if constexpr (is_logits3(EPI)) {
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            uint32_t v[32];
            tmem_ld32(taddr + c_begin + 32 * h, v);
            tmem_ld_wait();
            if (h == 3) drained();
            auto sums = [&](int j) -> float & { return h < 2 ? near[h & 1][j] : far[32 * (32 * (h - 2) + j)]; };
            float l[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              l[j] = __uint_as_float(v[j]);
              if (x.add) l[j] += sums(j);
              sums(j) = l[j];
            }
            if (x.last) largest(c_begin + 32 * h, [&](int j) { return l[j]; });
          }
          if (!x.last) continue;
        } else {
          for (int c0 = c_begin; c0 < c_end; c0 += 32) {
            uint32_t v[32];
            tmem_ld32(taddr + c0, v);
            tmem_ld_wait();
            largest(c0, [&](int j) { return __uint_as_float(v[j]); });
          }
        }
        top *= kLog2e;
        if (top > ref + kRaise) ref = top;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        // 32 exponentials of this row from column c on, summed up; fp32 io: in
        // their logits' place
        auto exps = [&](int c, float (&e)[32]) {
          if constexpr (!is_logits3(EPI)) {
            uint32_t v[32];
            tmem_ld32(taddr + c, v);
            tmem_ld_wait();
            if (c + 32 >= c_end) drained();
#pragma unroll
            for (int j = 0; j < 32; ++j) e[j] = __uint_as_float(v[j]);
          }
          const int col = x.n0 + c;
#pragma unroll
          for (int j = 0; j < 32; ++j) e[j] = exp2_approx(fmaf(e[j], kLog2e, -ref));
          if (!whole) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (col + j >= p.N) e[j] = 0.f;
          }
          // the label's own term stays out of the sum, exactly
          if ((unsigned)(label - col) < 32u) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (label - col == j) e[j] = 0.f;
          }
          if (label < 0) {  // no token: whatever the row holds
#pragma unroll
            for (int j = 0; j < 32; ++j) e[j] = 0.f;
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) sum[j & 3] += e[j];
        };
        // Boxes wholly behind an edge are not stored; rows behind the last one
        // are, as zeros: the products that follow read whole tiles.
        if constexpr (is_logits3(EPI)) {
#pragma unroll 1
          for (int c0 = c_begin; c0 < c_end; c0 += 64) {
            if (c0 > c_begin) {
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                near[0][j] = far[32 * j];
                near[1][j] = far[32 * (32 + j)];
              }
            }
            exps(c0, near[0]);
            exps(c0 + 32, near[1]);
            const bool stored = EPI == kProbs3 && x.n0 + c0 < p.N;
            for (int term = 0; stored && term < kTerms; ++term) {
              st.begin();
              put32(st, 0, near[0]);
              put32(st, 4, near[1]);
              st.finish(&tmC, term * p.e_term + x.n0 + c0, row0, false);
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                near[0][j] -= __bfloat162float(__float2bfloat16_rn(near[0][j]));
                near[1][j] -= __bfloat162float(__float2bfloat16_rn(near[1][j]));
              }
            }
          }
        } else {
          for (int c0 = c_begin; c0 < c_end; c0 += 64) {
            const bool stored = EPI == kProbs && x.n0 + c0 < p.N;
            if (stored) st.begin();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float e[32];
              exps(c0 + 32 * h, e);
              if (stored) put32(st, 4 * h, e);
            }
            if (stored) st.finish(&tmC, x.n0 + c0, row0, false);
          }
        }
        if (live && x.n0 + c_begin < p.N)
          p.part[(size_t)((x.n0 + c_begin) / 128) * p.rows + row] =
              make_float2(ref, (sum[0] + sum[1]) + (sum[2] + sum[3]));
      } else {
        // kDX: parts of 256 rows; nothing but zeros where there are no tokens
        const int out_row = EPI == kDX ? x.part * 2 * BM + row0 - x.rp * 2 * BM : row0;
        const bool none = x.k1 == x.k0;
        if (p.products > 1) {
          // sums in memory: the work before is there before this one adds
          if (lane == 0) tma_store_wait<0>();
          __syncwarp();
        }
        for (int c0 = c_begin; c0 < c_end; c0 += 64) {
          uint32_t a[32], b[32];
          tmem_ld32(taddr + c0, a);
          tmem_ld32(taddr + c0 + 32, b);
          tmem_ld_wait();
          if (c0 + 64 >= c_end) drained();
          if ((EPI == kDW && row0 >= p.M) || x.n0 + c0 >= p.N) continue;
          if (none) {
#pragma unroll
            for (int j = 0; j < 32; ++j) a[j] = b[j] = 0;
          }
          if (EPI == kDX || p.fp32) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t *v = h == 0 ? a : b;
              if (x.n0 + c0 + 32 * h >= p.N) break;
              st.begin();
#pragma unroll
              for (int q = 0; q < 8; ++q)
                st.put(q, make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]));
              st.finish(&tmC, x.n0 + c0 + 32 * h, out_row, x.add);
            }
          } else {
            st.begin();
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const uint32_t *v = q < 4 ? &a[8 * q] : &b[8 * (q - 4)];
              st.put(q, make_uint4(pack_bf16(__uint_as_float(v[0]), __uint_as_float(v[1])),
                                   pack_bf16(__uint_as_float(v[2]), __uint_as_float(v[3])),
                                   pack_bf16(__uint_as_float(v[4]), __uint_as_float(v[5])),
                                   pack_bf16(__uint_as_float(v[6]), __uint_as_float(v[7]))));
            }
            st.finish(&tmC, x.n0 + c0, out_row, false);
          }
        }
      }
    }
    if (lane == 0) tma_store_wait<0>();
    __syncwarp();
  }

  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

template <int EPI>
cudaError_t launch_gemm(const CUtensorMap &a, const CUtensorMap &b, const CUtensorMap &c,
                        const Params &p, long long works, int num_sms, cudaStream_t stream) {
  static std::atomic<int> max_pairs[64];
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  auto kernel = xent_gemm_kernel<EPI>;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.blockDim = dim3(NUM_THREADS);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  int pairs = max_pairs[dev].load(std::memory_order_acquire);
  if (pairs == 0) {
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (err != cudaSuccess) return err;
    int n = 0;
    cfg.gridDim = dim3(2 * (num_sms / 2));
    err = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
    if (err != cudaSuccess) return err;
    pairs = n > 0 ? n : 1;
    max_pairs[dev].store(pairs, std::memory_order_release);
  }
  cfg.gridDim = dim3(2 * (int)(works < pairs ? works : pairs));
  return cudaLaunchKernelEx(&cfg, kernel, a, b, c, p);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}


__device__ __forceinline__ bool is_word(int y, int V) { return y >= 0 && y < V; }

// An fp32 value as the sum of three bf16 ones, each the rounding of what the
// ones before leave.
__device__ __forceinline__ void split3(float x, float (&t)[kTerms]) {
#pragma unroll
  for (int k = 0; k < kTerms; ++k) {
    t[k] = __bfloat162float(__float2bfloat16_rn(x));
    x -= t[k];
  }
}
// A row of d fp32 values times `f` as three rows of `term` bf16 ones side by
// side, zeros behind d; one warp.
__device__ __forceinline__ void split_row(const float *x, int d, float f, __nv_bfloat16 *out, int term,
                                          int lane) {
  for (int k = 2 * lane; k < term; k += 64) {
    float a[kTerms], b[kTerms];
    split3(k < d ? x[k] * f : 0.f, a);
    split3(k + 1 < d ? x[k + 1] * f : 0.f, b);
#pragma unroll
    for (int t = 0; t < kTerms; ++t)
      *reinterpret_cast<uint32_t *>(out + t * term + k) = pack_bf16(a[t], b[t]);
  }
}

template <typename T>
struct GatherArgs {
  const T *X, *W;
  const int *labels;
  long long N;
  int d, V, mean, block_rows;
  float scale;
  XentLayout L;
  float *loss, *lse;
  T *dX;
  int copy;    // there is one piece: its rows are copied here
  int blocks;  // of the rows; fp32: the others take W's terms
};

// A row of X as the products read it; one warp.
__device__ __forceinline__ void copy_row(const __nv_bfloat16 *x, int d, __nv_bfloat16 *out, int,
                                         int lane) {
  for (int k = 8 * lane; k < d; k += 256)
    *reinterpret_cast<uint4 *>(out + k) = *reinterpret_cast<const uint4 *>(x + k);
}
__device__ __forceinline__ void copy_row(const float *x, int d, __nv_bfloat16 *out, int term, int lane) {
  split_row(x, d, 1.f, out, term, lane);
}
// zeros behind the last row, to the end of its k-block: dW's sum over the
// tokens reads it whole
__device__ __forceinline__ void zero_tail(__nv_bfloat16 *Xc, long long rows, long long width) {
  const long long end = (rows + BK - 1) / BK * BK * width;
  for (long long i = rows * width + threadIdx.x; i < end; i += 256) Xc[i] = __float2bfloat16_rn(0.f);
}

// The rows of X with a label, one behind another (as three terms for fp32),
// with their labels, where they came from and their reference, the label's
// logit; zeros in the outputs of the other rows.  A block finds where its
// rows go by counting the labels before them, so the order is the tokens'.
// The last block leaves the number of rows, the gradients' factor, a cleared
// status word and a tile's worth of rows without a label behind the last one.
// With fp32 io the blocks behind these write W as three terms, a warp a row
// (in a launch of its own that took 9 us at 8003 x 520).  Latency bounds
// it: labels, a row and its word's row one after another (4096 x 768 bf16:
// 9 us; 16384 x 1024: 21).
template <typename T>
__global__ void __launch_bounds__(256) xent_gather_kernel(const GatherArgs<T> a) {
  __shared__ int counts[8];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = a.d;
  if constexpr (sizeof(T) == 4) {
    if (blockIdx.x >= (unsigned)a.blocks) {
      const int v = (int)(blockIdx.x - a.blocks) * 8 + warp;
      if (v < a.V)
        split_row(a.W + (size_t)v * d, d, 1.f,
                  static_cast<__nv_bfloat16 *>(a.L.Ws) + (size_t)v * kTerms * a.L.term, a.L.term, lane);
      return;
    }
  }
  const long long row0 = (long long)blockIdx.x * a.block_rows;
  const long long end = min(row0 + a.block_rows, a.N);
  int n = 0;
#pragma unroll 8
  for (long long i = threadIdx.x; i < row0; i += 256) n += is_word(__ldg(a.labels + i), a.V);
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0) counts[warp] = n;
  __syncthreads();
  long long base = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) base += counts[k];
  const long long width = (long long)(sizeof(T) == 4 ? kTerms : 1) * a.L.term;
  for (long long r0 = row0; r0 < end; r0 += 8) {
    const int y8 = lane < 8 && r0 + lane < end ? a.labels[r0 + lane] : -1;
    const unsigned mask = __ballot_sync(0xffffffffu, is_word(y8, a.V));
    const int y = __shfl_sync(0xffffffffu, y8, warp);
    const long long row = r0 + warp, c = base + __popc(mask & ((1u << warp) - 1));
    base += __popc(mask);
    if (row >= end) continue;
    const T *x = a.X + row * d;
    if (mask >> warp & 1) {
      const T *w = a.W + (size_t)y * d;
      float s = 0.f;
      if constexpr (sizeof(T) == 2) {
        for (int k = 8 * lane; k < d; k += 256) {
          const uint4 u = *reinterpret_cast<const uint4 *>(x + k);
          const uint4 v = __ldg(reinterpret_cast<const uint4 *>(w + k));
          const uint32_t au[4] = {u.x, u.y, u.z, u.w}, bu[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&au[q]));
            const float2 g = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&bu[q]));
            s = fmaf(f.x, g.x, fmaf(f.y, g.y, s));
          }
        }
      } else {
        for (int k = lane; k < d; k += 32) s = fmaf(x[k], __ldg(w + k), s);
      }
      if (a.copy) copy_row(x, d, static_cast<__nv_bfloat16 *>(a.L.Xc) + c * width, a.L.term, lane);
      s = warp_sum(s);
      if (lane == 0) {
        a.L.ref[c] = s * kLog2e;
        a.L.labels[c] = y;
        a.L.index[c] = (int)row;
      }
    } else {
      if (lane == 0) {
        a.loss[row] = 0.f;
        if (a.lse) a.lse[row] = 0.f;
      }
      if (a.dX)
        for (int k = lane; k < d; k += 32) a.dX[row * d + k] = T(0.f);
    }
  }
  if (blockIdx.x != (unsigned)a.blocks - 1) return;
  // base is the number of labels now
  const long long tile = (base + 2 * BM - 1) / (2 * BM) * (2 * BM);
  for (long long c = base + threadIdx.x; c < tile; c += 256) a.L.labels[c] = -1;
  if (a.copy) zero_tail(static_cast<__nv_bfloat16 *>(a.L.Xc), base, width);
  if (threadIdx.x == 0) {
    *a.L.status = FLASH_GAU_OK;
    *a.L.live = (int)base;
    *a.L.done = 0;
    *a.L.factor = a.mean ? a.scale / (float)(base > 0 ? base : 1) : a.scale;
  }
}

// The rows of one piece of several; a warp a row.
template <typename T>
__global__ void __launch_bounds__(256)
xent_copy_kernel(const T *__restrict__ X, int d, const XentLayout L, long long first, int rows) {
  griddep_wait();
  const long long left = *L.live - first;
  const int tokens = left < 0 ? 0 : left < rows ? (int)left : rows;
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5);
  const long long width = (long long)(sizeof(T) == 4 ? kTerms : 1) * L.term;
  __nv_bfloat16 *Xc = static_cast<__nv_bfloat16 *>(L.Xc);
  if (row < tokens)
    copy_row(X + (long long)L.index[first + row] * d, d, Xc + row * width, L.term, threadIdx.x & 31);
  if (blockIdx.x == 0) zero_tail(Xc, tokens, width);
}

struct RowArgs {
  XentLayout L;
  long long first, N;  // this piece's first row; all tokens
  int rows, V, d;
  int parts;
  int grad, scaled;    // E is there; dW wants scaled rows
  int blocks;          // of every piece's launch
  const void *X;       // fp32: the tokens' rows
  float *loss, *lse, *total;
};

// (reference, sum) of two parts of a row; whether the references differ
__device__ __forceinline__ bool join_parts(float &top, float &sum, float ref, float s) {
  if (ref == top) {
    sum += s;
    return false;
  }
  const float t = fmaxf(top, ref);
  // a reference of minus infinity has no terms below it
  sum = (top == t ? sum : sum * exp2f(top - t)) + (ref == t ? s : s * exp2f(ref - t));
  top = t;
  return true;
}

// log Z - t of a row (times ln 2 where it is in logs of two): sum is of the
// other words relative to 2^top, t2 the label's logit
__device__ __forceinline__ float row_loss(float top, float sum, float t2, float *z) {
  if (top == t2) {
    // an infinite logit makes both NaN, as inf - inf does
    *z = 1.0f + sum + 0.f * t2;
    return log1pf(sum) + 0.f * t2;
  }
  *z = exp2f(t2 - top) + sum;
  return logf(*z) + (top - t2) * kLn2;
}
// and its log sum exp: from the loss only where that is relative to the
// label's logit, which may be minus infinity elsewhere
__device__ __forceinline__ float row_lse(float top, float t2, float z, float loss) {
  return top == t2 ? fmaf(t2, kLn2, loss) : fmaf(top, kLn2, logf(z));
}

// A row's E from its parts' references to the row's, by the whole block, but
// for the label's.  Only rows with a logit 40 above the label's need it
// (where all of 1000 rows of 50000 words do the kernel takes 61 us; 607 with
// a warp a row and part by part).
template <int TERMS>
__device__ __forceinline__ void rescale_row(const RowArgs &a, int row, float top) {
  constexpr int U = TERMS == 1 ? 4 : 2;  // loads under way
  const long long ld = a.L.ldE;          // a multiple of 64
  __nv_bfloat16 *E = static_cast<__nv_bfloat16 *>(a.L.E) + (size_t)row * TERMS * ld;
  const int label = a.L.labels[a.first + row], n = (int)(ld / 8);
  for (int v0 = threadIdx.x; v0 < n; v0 += 256 * U) {
    uint4 w[U][TERMS];
    float from[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = v0 + 256 * u;
      from[u] = v < n ? a.L.part[(size_t)(v / 16) * a.rows + row].x : top;
#pragma unroll
      for (int t = 0; t < TERMS; ++t)
        if (v < n) w[u][t] = *reinterpret_cast<const uint4 *>(E + t * ld + 8 * v);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (from[u] == top) continue;
      const int c = 8 * (v0 + 256 * u);
      // in two factors: E goes up to 2^58, and what is left of it may be a
      // normal number where the factor alone is none
      const float by = from[u] - top, f = exp2f(fmaxf(by, -126.f)), g = exp2f(fminf(by + 126.f, 0.f));
      float e[8] = {};
#pragma unroll
      for (int t = TERMS - 1; t >= 0; --t) {
        const uint32_t x[4] = {w[u][t].x, w[u][t].y, w[u][t].z, w[u][t].w};
#pragma unroll
        for (int q = 0; q < 8; ++q)
          e[q] += __uint_as_float(q & 1 ? x[q / 2] & 0xffff0000u : x[q / 2] << 16);
      }
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (c + q != label) e[q] = e[q] * f * g;
#pragma unroll
      for (int t = 0; t < TERMS; ++t) {
        *reinterpret_cast<uint4 *>(E + t * ld + c) =
            make_uint4(pack_bf16(e[0], e[1]), pack_bf16(e[2], e[3]), pack_bf16(e[4], e[5]),
                       pack_bf16(e[6], e[7]));
#pragma unroll
        for (int q = 0; q < 8; ++q) e[q] -= __bfloat162float(__float2bfloat16_rn(e[q]));
      }
    }
  }
}

// Eight rows a block.  First 32 threads a row join the parts of its sum, then
// a warp a row writes the loss, and with gradients the row's factor, the
// label's E, the scaled row of X, and where a part took another reference
// than the row's its E again.  The last block of all adds the losses up.
// (V 50257: 18 us at 4096 x 768 bf16, 37 at 16384 x 1024; 393 parts a row, read
// with 32 threads and eight loads in flight each.)
template <typename T>
__global__ void __launch_bounds__(256) xent_rows_kernel(const RowArgs a) {
  __shared__ float2 joined[8][33];
  __shared__ int differ[8], last;
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row0 = blockIdx.x * 8, row = row0 + warp;  // this warp's row, later
  // everything that does not wait for the number of rows is asked for first
  // (the buffers hold a.rows rows; what is behind the last one is not used)
  const int safe = row < a.rows ? row : a.rows - 1;
  const float ref = a.L.ref[a.first + safe], factor = *a.L.factor;
  const int label = a.L.labels[a.first + safe], token = a.L.index[a.first + safe];
  const int r = threadIdx.x & 7, part_row = row0 + r < a.rows ? row0 + r : a.rows - 1;
  const float part_ref = a.L.ref[a.first + part_row];
  const long long left = *a.L.live - a.first;
  const int tokens = left < 0 ? 0 : left < a.rows ? (int)left : a.rows;
  if (row0 < tokens) {
    if (threadIdx.x < 8) differ[threadIdx.x] = 0;
    __syncthreads();
    {
      float top = part_ref, sum = 0.f;
      bool mixed = false;
      if (row0 + r < tokens) {
        const float2 *part = a.L.part + part_row;
#pragma unroll 8
        for (int k = threadIdx.x >> 3; k < a.parts; k += 32) {
          const float2 v = part[(size_t)k * a.rows];
          mixed |= join_parts(top, sum, v.x, v.y);
        }
      }
      joined[r][threadIdx.x >> 3] = make_float2(top, sum);
      if (mixed) differ[r] = 1;
    }
    __syncthreads();
    if (row < tokens) {
      const float2 own = joined[warp][lane];
      float top = own.x, sum = own.y;
      bool mixed = differ[warp];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float r = __shfl_xor_sync(0xffffffffu, top, o);
        const float s = __shfl_xor_sync(0xffffffffu, sum, o);
        mixed |= join_parts(top, sum, r, s);
      }
      mixed = __any_sync(0xffffffffu, mixed);
      float z;
      const float loss = row_loss(top, sum, ref, &z);
      float scale = factor / z;  // of dX, then of the scaled row
      const int terms = sizeof(T) == 4 ? kTerms : 1;
      __nv_bfloat16 *E = static_cast<__nv_bfloat16 *>(a.L.E) + (size_t)row * terms * a.L.ldE;
      if (lane == 0) {
        a.loss[token] = loss;
        if (a.lse) a.lse[token] = row_lse(top, ref, z, loss);
      }
      if (a.grad) {
        if constexpr (sizeof(T) == 2) {
          const __nv_bfloat16 e = __float2bfloat16_rn(-sum);
          const bool rounded = sum > 0.f && sum < INFINITY;
          if (lane == 0) {
            E[label] = e;
            a.L.row_scale[row] = scale;
            a.L.left[row] = rounded ? -sum - __bfloat162float(e) : 0.f;
          }
          if (rounded) scale *= sum / -__bfloat162float(e);
        } else {
          float t[kTerms];
          split3(-sum, t);
          if (lane < kTerms)
            E[lane * a.L.ldE + label] =
                __float2bfloat16_rn(lane == 0 ? t[0] : lane == 1 ? t[1] : t[2]);
          if (lane == 0) a.L.row_scale[row] = scale;
        }
        if (a.scaled) {
          __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.L.Xc) + (size_t)row * terms * a.L.term;
          if constexpr (sizeof(T) == 2) {
            for (int k = 8 * lane; k < a.d; k += 256) {
              const uint4 w = *reinterpret_cast<const uint4 *>(o + k);
              uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u[q]));
                u[q] = pack_bf16(f.x * scale, f.y * scale);
              }
              *reinterpret_cast<uint4 *>(o + k) = make_uint4(u[0], u[1], u[2], u[3]);
            }
          } else {
            split_row(static_cast<const float *>(a.X) + (size_t)token * a.d, a.d, scale, o, a.L.term,
                      lane);
          }
        }
        if (lane == 0) {
          differ[warp] = mixed;
          joined[warp][32].x = top;
        }
      }
    } else if (lane == 0) {
      differ[warp] = 0;
    }
    if (a.grad) {
      __syncthreads();
      for (int k = 0; k < 8; ++k)
        if (differ[k]) rescale_row<sizeof(T) == 4 ? kTerms : 1>(a, row0 + k, joined[k][32].x);
    }
  }
  // total, by whichever block comes last (lane 0 wrote the loss)
  if (lane == 0) __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(a.L.done, 1) == a.blocks - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  for (long long i = threadIdx.x; i < a.N; i += 1024)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + 256 * k < a.N) s[k] += __ldcg(a.loss + i + 256 * k);
  const float v = warp_sum((s[0] + s[1]) + (s[2] + s[3]));
  if (lane == 0) joined[0][warp].x = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    float t = 0.f;
    for (int k = 0; k < 8; ++k) t += joined[0][k].x;
    *a.total = factor * t;
  }
}

__device__ __forceinline__ void store_as(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_as(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// dX from the parts of its sum, in the groups' order, with what the label's
// term has lost (bf16), times the row's factor, to where the row came from;
// four columns a thread (4096 x 768 bf16: 15 us).
template <typename T>
__global__ void __launch_bounds__(256)
xent_join_kernel(const XentLayout L, long long first, int rows, int d, int V, int products,
                 const T *__restrict__ W, T *__restrict__ out) {
  __shared__ DxPlan q;
  griddep_wait();
  const long long left = *L.live - first;
  const int tokens = left < 0 ? 0 : left < rows ? (int)left : rows;
  const int quads = (d + 3) / 4;
  const long long i = blockIdx.x * 256LL + threadIdx.x;
  if (blockIdx.x * 256LL >= (long long)tokens * quads) return;
  if (threadIdx.x == 0) q = dx_plan(tokens, d, V, products, kPlanPairs);
  __syncthreads();
  const int row = (int)(i / quads), c = (int)(i % quads) * 4;
  if (row >= tokens) return;
  const int rp = row / (2 * BM);
  int g0 = 0, n = 1;
  if (rp >= q.first_left()) {
    const int at = (rp - q.first_left()) * q.steps;
    g0 = at / q.run;
    n = (at + q.steps - 1) / q.run - g0 + 1;
  }
  const long long step = 2LL * BM * L.ld_part;
  const float *p = L.dx_part + (rp + g0) * step + (long long)(row - rp * 2 * BM) * L.ld_part + c;
  const float f = L.row_scale[row];
  float4 s = __ldcs(reinterpret_cast<const float4 *>(p));
#pragma unroll 8
  for (int k = 1; k < n; ++k) {
    const float4 v = __ldcs(reinterpret_cast<const float4 *>(p + k * step));
    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
  }
  T *o = out + (size_t)L.index[first + row] * d + c;
  if constexpr (sizeof(T) == 2) {  // d is a multiple of 8
    const float lost = L.left[row];
    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(W + (size_t)L.labels[first + row] * d + c));
    s.x = fmaf(lost, __uint_as_float(w.x << 16), s.x);
    s.y = fmaf(lost, __uint_as_float(w.x & 0xffff0000u), s.y);
    s.z = fmaf(lost, __uint_as_float(w.y << 16), s.z);
    s.w = fmaf(lost, __uint_as_float(w.y & 0xffff0000u), s.w);
    *reinterpret_cast<uint2 *>(o) =
        make_uint2(pack_bf16(s.x * f, s.y * f), pack_bf16(s.z * f, s.w * f));
  } else {
    const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c + k < d) o[k] = v[k] * f;
  }
}

// dW from its fp32 sum, rows of `ld` values
template <typename T>
__global__ void __launch_bounds__(256)
xent_finish_kernel(const float *__restrict__ in, int ld, int V, int d, T *__restrict__ out) {
  griddep_wait();
  const int quads = (d + 3) / 4;
  const long long i = blockIdx.x * 256LL + threadIdx.x;
  if (i >= (long long)V * quads) return;
  const long long row = i / quads;
  const int c = (int)(i % quads) * 4;
  const float4 s = *reinterpret_cast<const float4 *>(in + row * ld + c);
  const float v[4] = {s.x, s.y, s.z, s.w};
  T *o = out + row * d + c;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (c + k < d) store_as(o + k, v[k]);
}

// ---- a few tokens, no gradients -------------------------------------------
// W is read once and nothing else counts (50257 x 768 bf16: 77 MB, 11.4 us at
// the copy rate).  A warp takes four words at a time, 16 bytes of each a lane,
// against the tokens' x in shared memory; the 4 NT sums over the warp leave
// each lane one token and word of its own, whose running maximum and sum it
// keeps, and xent_few_join_kernel joins the blocks'.  Back to back in a graph,
// W from memory: one token 17 us, two 19, four 23; fp32 29, 31 and 31, eight
// 40.  By the tensor cores: bf16 30 to 31 whatever the tokens, fp32 169 (W has
// to be split there), and 12 for 5 at 3000 x 256.  So bf16 takes this way up to four
// tokens (eight: 36 us), fp32 up to eight.
constexpr int kFewTokens = 8, kFewTokensBf16 = 4;

struct FewArgs {
  const void *X, *W;
  const int *labels;
  int N, d, V, mean;
  float scale;
  float2 *part;    // [kFewTokens][blocks]
  float *target;   // [kFewTokens] the label's logit in units of ln 2
  int blocks;
  int *status;
  float *loss, *lse, *total;
};

__device__ __forceinline__ void add_logit(float &top, float &sum, float l) {
  if (l > top) {
    sum = fmaf(sum, exp2_approx(top - l), 1.f);  // top minus infinity: sum is zero
    top = l;
  } else {
    // (l - top is NaN where one of them is, or where both are infinite)
    sum += l == -INFINITY ? 0.f : exp2_approx(l - top);
  }
}

// R values of every lane summed over the warp, halving what a lane holds with
// each exchange: lane i is left with the sum of value i / (32 / R).
template <int R>
__device__ __forceinline__ float warp_sums(float (&v)[R], int lane) {
  int o = 16;
#pragma unroll
  for (int half = R / 2; half > 0; half /= 2, o /= 2) {
    const bool upper = lane & o;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float keep = upper ? v[i + half] : v[i], give = upper ? v[i] : v[i + half];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
#pragma unroll
  for (int k = 16 / R; k > 0; k /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], k);
  return v[0];
}

// (blocks an SM and the unrolling by time: 50257 x 768 bf16, two tokens: 19 us
// for 23 without the bound, four: 23 for 29 with a tighter one; fp32, eight:
// 40 for 64)
template <typename T, int NT>
__global__ void __launch_bounds__(256, NT <= 2 ? 4 : 2) xent_few_kernel(const FewArgs a) {
  extern __shared__ __align__(16) float xs[];  // [NT][d]
  __shared__ float2 mine[8][NT];
  griddep_wait();
  constexpr int W16 = 16 / sizeof(T);  // values of 16 bytes
  constexpr int kSame = 8 / NT;        // lanes that are left with the same sum
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = a.d;
  const T *X = static_cast<const T *>(a.X), *W = static_cast<const T *>(a.W);
  for (int i = threadIdx.x; i < NT * d; i += 256) xs[i] = i < a.N * d ? (float)X[i] : 0.f;
  __syncthreads();
  // this lane's token and which of the four words, of what the sums leave it
  const int n_own = lane / kSame / 4, j_own = lane / kSame % 4;
  const int label = n_own < a.N ? a.labels[n_own] : -1;
  float top = -INFINITY, sum = 0.f;
  for (int w0 = (blockIdx.x * 8 + warp) * 4; w0 < a.V; w0 += gridDim.x * 32) {
    f2 acc[NT][4] = {};
#pragma unroll (NT <= 4 ? 2 : 1)
    for (int k = W16 * lane; k < d; k += 32 * W16) {
      f2 w[4][W16 / 2];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(W + (size_t)min(w0 + j, a.V - 1) * d + k));
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int q = 0; q < W16 / 2; ++q) {
          if constexpr (sizeof(T) == 2)
            w[j][q] = pair(__uint_as_float(u[q] << 16), __uint_as_float(u[q] & 0xffff0000u));
          else
            w[j][q] = pair(__uint_as_float(u[2 * q]), __uint_as_float(u[2 * q + 1]));
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int q = 0; q < W16; q += 4) {
          const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(xs + n * d + k + q);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[n][j] = fma2(w[j][q / 2 + 1], x.y, fma2(w[j][q / 2], x.x, acc[n][j]));
        }
    }
    float v[4 * NT];
#pragma unroll
    for (int r = 0; r < 4 * NT; ++r) {
      const float2 t = split(acc[r / 4][r % 4]);
      v[r] = t.x + t.y;
    }
    const float l = warp_sums(v, lane) * kLog2e;
    const int word = w0 + j_own;
    if (word == label) {
      if (lane % kSame == 0) a.target[n_own] = l;
    } else if (word < a.V) {
      add_logit(top, sum, l);
    }
  }
  // the four words' lanes of a token
#pragma unroll
  for (int o = kSame; o <= 2 * kSame; o *= 2) {
    const float t = __shfl_xor_sync(0xffffffffu, top, o), s = __shfl_xor_sync(0xffffffffu, sum, o);
    join_parts(top, sum, t, s);
  }
  if (lane % (4 * kSame) == 0) mine[warp][n_own] = make_float2(top, sum);
  __syncthreads();
  if (threadIdx.x < NT) {
    float2 v = mine[0][threadIdx.x];
    for (int k = 1; k < 8; ++k) join_parts(v.x, v.y, mine[k][threadIdx.x].x, mine[k][threadIdx.x].y);
    a.part[(size_t)threadIdx.x * gridDim.x + blockIdx.x] = v;
  }
}

// The blocks' parts of each token joined by 256 / NT threads, its loss, and
// the total; one block.
template <int NT>
__global__ void __launch_bounds__(256) xent_few_join_kernel(const FewArgs a) {
  __shared__ float2 mine[8][NT];
  __shared__ float losses[kFewTokens];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kShare = 256 / NT, kWarps = kShare / 32;
  {
    const int n = threadIdx.x / kShare;
    float t = -INFINITY, s = 0.f;
    float2 v[4];
    for (int k0 = threadIdx.x % kShare; k0 < a.blocks; k0 += 4 * kShare) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int k = k0 + q * kShare;
        v[q] = k < a.blocks ? a.part[(size_t)n * a.blocks + k] : make_float2(-INFINITY, 0.f);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) join_parts(t, s, v[q].x, v[q].y);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float r = __shfl_xor_sync(0xffffffffu, t, o);
      const float u = __shfl_xor_sync(0xffffffffu, s, o);
      join_parts(t, s, r, u);
    }
    if (lane == 0) mine[warp % kWarps][n] = make_float2(t, s);
  }
  __syncthreads();
  if (threadIdx.x < a.N) {
    const int n = threadIdx.x, y = a.labels[n];
    float loss = 0.f, lse = 0.f;
    if (is_word(y, a.V)) {
      float t = mine[0][n].x, s = mine[0][n].y;
      for (int k = 1; k < kWarps; ++k) join_parts(t, s, mine[k][n].x, mine[k][n].y);
      const float t2 = a.target[n];
      if (t <= t2) {  // relative to the label: log1p keeps a small loss's digits
        s = t == t2 ? s : s * exp2f(t - t2);
        t = t2;
      }
      float z;
      loss = row_loss(t, s, t2, &z);
      lse = row_lse(t, t2, z, loss);
    }
    losses[n] = loss;
    a.loss[n] = loss;
    if (a.lse) a.lse[n] = lse;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.f;
    int n = 0;
    for (int k = 0; k < a.N; ++k) {
      s += losses[k];
      n += is_word(a.labels[k], a.V);
    }
    *a.total = (a.mean ? a.scale / (float)(n > 0 ? n : 1) : a.scale) * s;
    *a.status = FLASH_GAU_OK;
  }
}

Params gemm_params(int M, int N, int K, const XentLayout &L, long long first, int rows, int products) {
  Params p = {};
  p.M = M;
  p.N = N;
  p.K = K;
  p.live = L.live;
  p.first = first;
  p.rows = rows;
  p.products = products;
  p.status = L.status;
  return p;
}

template <typename T>
cudaError_t run_few(const XentProblem &q) {
  FewArgs a = {};
  a.X = q.X;
  a.W = q.W;
  a.labels = q.labels;
  a.N = (int)q.N;
  a.d = q.d;
  a.V = q.V;
  a.mean = q.mean;
  a.scale = q.scale;
  a.part = q.L.part;
  a.target = q.L.ref;
  a.status = q.L.status;
  a.loss = q.loss;
  a.lse = q.lse;
  a.total = q.total;
  const int need = (q.V + 31) / 32;
  a.blocks = need < kXentFewBlocks ? need : kXentFewBlocks;
  const dim3 grid(a.blocks), block(256);
  auto go = [&](auto kernel, auto join, int nt) {
    const size_t smem = (size_t)nt * q.d * sizeof(float);
    // 48 KB are there unasked, for the tokens and the kernel's own array together
    if (smem + 8 * nt * sizeof(float2) > 48 * 1024) {
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 kXentFewSmem);
      if (e != cudaSuccess) return e;
    }
    const cudaError_t e = launch_pdl(kernel, grid, block, smem, q.stream, a);
    return e != cudaSuccess ? e : launch_pdl(join, dim3(1), block, 0, q.stream, a);
  };
  if (q.N == 1) return go(xent_few_kernel<T, 1>, xent_few_join_kernel<1>, 1);
  if (q.N == 2) return go(xent_few_kernel<T, 2>, xent_few_join_kernel<2>, 2);
  if constexpr (sizeof(T) == 4)
    if (q.N > 4) return go(xent_few_kernel<T, 8>, xent_few_join_kernel<8>, 8);
  return go(xent_few_kernel<T, 4>, xent_few_join_kernel<4>, 4);
}

template <typename T>
cudaError_t run(const XentProblem &q) {
  constexpr bool bf16 = sizeof(T) == 2;
  constexpr int products = bf16 ? 1 : kProducts, terms = bf16 ? 1 : kTerms;
  const XentLayout &L = q.L;
  const bool grad = q.dX || q.dW;
  cudaError_t err;
  GatherArgs<T> g = {};
  g.X = static_cast<const T *>(q.X);
  g.W = static_cast<const T *>(q.W);
  g.labels = q.labels;
  g.N = q.N;
  g.d = q.d;
  g.V = q.V;
  g.mean = q.mean;
  g.scale = q.scale;
  // every block counts the labels before it: at most 2048 of them
  g.block_rows = (int)(8 * ((q.N + 8 * 2048 - 1) / (8 * 2048)));
  g.L = L;
  g.loss = q.loss;
  g.lse = q.lse;
  g.dX = static_cast<T *>(q.dX);
  g.copy = L.piece >= q.N;
  g.blocks = (int)((q.N + g.block_rows - 1) / g.block_rows);
  const unsigned blocks = (unsigned)(g.blocks + (bf16 ? 0 : (q.V + 7) / 8));
  if ((err = launch_pdl(xent_gather_kernel<T>, dim3(blocks), dim3(256), 0, q.stream, g)) != cudaSuccess)
    return err;
  const void *W = bf16 ? q.W : L.Ws;
  // an operand's columns: d of the bf16 one (TMA fills what is behind with
  // zeros), or three padded terms
  const uint64_t width = bf16 ? (uint64_t)q.d : (uint64_t)terms * L.term;
  CUtensorMap tW, tWn;
  if ((err = make_tmap_bf16_2d(&tW, W, q.V, width, width, BN / 2, BK)) != cudaSuccess) return err;
  if ((err = make_tmap_bf16_2d(&tWn, W, q.V, width, width, BK, 64)) != cudaSuccess) return err;
  long long row_blocks = 0;
  for (long long n0 = 0; n0 < q.N; n0 += L.piece)
    row_blocks += ((q.N - n0 < L.piece ? q.N - n0 : L.piece) + 7) / 8;
  for (long long n0 = 0; n0 < q.N; n0 += L.piece) {
    const int rows = (int)(q.N - n0 < L.piece ? q.N - n0 : L.piece);
    const int whole = (rows + 2 * BM - 1) / (2 * BM) * (2 * BM);  // rows of the buffers
    const void *x = L.Xc;
    if (!g.copy) {
      err = launch_pdl(xent_copy_kernel<T>, dim3((rows + 7) / 8), dim3(256), 0, q.stream, g.X, q.d, L,
                       n0, rows);
      if (err != cudaSuccess) return err;
    }
    const uint64_t cols = (uint64_t)terms * L.ldE;
    CUtensorMap tX, tE = tW;
    if ((err = make_tmap_bf16_2d(&tX, x, whole, width, width, BM, BK)) != cudaSuccess) return err;
    if (grad && (err = make_tmap_bf16_2d(&tE, L.E, whole, cols, cols, 32, 64)) != cudaSuccess)
      return err;
    Params p = gemm_params(rows, q.V, q.d, L, n0, rows, products);
    p.a_term = p.b_term = L.term;
    p.ref = L.ref + n0;
    p.labels = L.labels + n0;
    p.part = L.part;
    p.e_term = (int)L.ldE;
    const long long works = (long long)(whole / (2 * BM)) * ((q.V + BN - 1) / BN);
    // fp32 without E: one work a tile needs no sums, and the whole ring is
    // there (9 x 512 x 50257: 112 us, 119 with four stages of it; gradients,
    // 1001 x 520 x 8003, alike)
    if (grad) err = launch_gemm<bf16 ? kProbs : kProbs3>(tX, tW, tE, p, works, q.num_sms, q.stream);
    else if (bf16 || q.d <= kFp32Blocks * BK)
      err = launch_gemm<kLoss>(tX, tW, tE, p, works, q.num_sms, q.stream);
    else err = launch_gemm<kLoss3>(tX, tW, tE, p, works, q.num_sms, q.stream);
    if (err != cudaSuccess) return err;
    RowArgs r = {};
    r.L = L;
    r.first = n0;
    r.N = q.N;
    r.rows = rows;
    r.V = q.V;
    r.d = q.d;
    r.parts = (q.V + 127) / 128;
    r.grad = grad;
    r.scaled = q.dW != nullptr;
    r.blocks = (int)row_blocks;
    r.X = q.X;
    r.loss = q.loss;
    r.lse = q.lse;
    r.total = q.total;
    err = launch_pdl(xent_rows_kernel<T>, dim3((rows + 7) / 8), dim3(256), 0, q.stream, r);
    if (err != cudaSuccess) return err;
    if (q.dX) {
      CUtensorMap tEa, tO;
      if ((err = make_tmap_bf16_2d(&tEa, L.E, whole, cols, cols, BM, BK)) != cudaSuccess) return err;
      err = make_tmap_f32_2d(&tO, L.dx_part, xent_dx_part_rows(rows, q.d), L.ld_part, L.ld_part, 32, 32);
      if (err != cudaSuccess) return err;
      Params g2 = gemm_params(rows, q.d, q.V, L, n0, rows, products);
      g2.a_term = (int)L.ldE;
      g2.b_term = L.term;
      if ((err = launch_gemm<kDX>(tEa, tWn, tO, g2, kPlanPairs, q.num_sms, q.stream)) != cudaSuccess)
        return err;
      const long long quads = (long long)rows * ((q.d + 3) / 4);
      err = launch_pdl(xent_join_kernel<T>, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0,
                       q.stream, L, n0, rows, q.d, q.V, products, g.W, static_cast<T *>(q.dX));
      if (err != cudaSuccess) return err;
    }
    if (q.dW) {
      CUtensorMap tEt, tXs, tO;
      if ((err = make_tmap_bf16_2d(&tEt, L.E, whole, cols, cols, BK, 64)) != cudaSuccess) return err;
      if ((err = make_tmap_bf16_2d(&tXs, x, whole, width, width, BK, 64)) != cudaSuccess) return err;
      if (L.dw_sum) err = make_tmap_f32_2d(&tO, L.dw_sum, q.V, q.d, L.ld_dw, 32, 32);
      else if (bf16) err = make_tmap_bf16_2d(&tO, q.dW, q.V, q.d, q.d, 32, 64);
      else err = make_tmap_f32_2d(&tO, q.dW, q.V, q.d, q.d, 32, 32);
      if (err != cudaSuccess) return err;
      Params g3 = gemm_params(q.V, q.d, rows, L, n0, rows, products);
      g3.a_term = (int)L.ldE;
      g3.b_term = L.term;
      g3.fp32 = !bf16 || L.dw_sum;
      g3.add = n0 > 0;
      const long long tiles = (long long)((q.V + 2 * BM - 1) / (2 * BM)) * ((q.d + BN - 1) / BN);
      if ((err = launch_gemm<kDW>(tEt, tXs, tO, g3, tiles, q.num_sms, q.stream)) != cudaSuccess)
        return err;
    }
  }
  if (q.dW && L.dw_sum) {
    const long long quads = (long long)q.V * ((q.d + 3) / 4);
    return launch_pdl(xent_finish_kernel<T>, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0,
                      q.stream, L.dw_sum, L.ld_dw, q.V, q.d, static_cast<T *>(q.dW));
  }
  return cudaSuccess;
}

}  // namespace

size_t xent_dx_part_rows(long long rows, int d) {
  const DxPlan q = dx_plan((int)rows, d, 1, 1, kPlanPairs);
  return (size_t)(q.row_pairs + q.groups) * 2 * BM;
}

bool xent_few(long long N, int d, int dtype, bool grad) {
  const bool bf16 = dtype == FLASH_GAU_BF16;
  const int io = bf16 ? 2 : 4;
  const long long tokens = N <= 2 ? N : N <= 4 ? 4 : 8;
  return !grad && N <= (bf16 ? kFewTokensBf16 : kFewTokens) && (long long)d * io % 16 == 0 &&
         tokens * d * (long long)sizeof(float) <= kXentFewSmem;
}

cudaError_t xent(const XentProblem &q, int dtype) {
  const bool few = xent_few(q.N, q.d, dtype, q.dX || q.dW);
  if (dtype == FLASH_GAU_BF16) return few ? run_few<__nv_bfloat16>(q) : run<__nv_bfloat16>(q);
  return few ? run_few<float>(q) : run<float>(q);
}

}  // namespace flashgau
