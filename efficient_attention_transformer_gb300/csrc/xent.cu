// Softmax cross entropy of the logits X W^T over a vocabulary, with the
// gradients of X [N, d] and W [V, d], bf16 operands, fp32 accumulation:
//   l = x W^T     loss = log sum_v exp(l_v) - l_y
//   dX_i = g (sum_v p_iv W_v - W_y)      dW_v = g sum_i (p_iv - [v = y_i]) x_i
// The tokens are taken in pieces (xent_plan), so that no more than a piece's
// [Nc, V] is held at any time, and the logits themselves are never stored.
//
// The logits are formed once, 6 N d V operations in all: the product's
// epilogue needs the row's normaliser for p = exp(l - lse), which is known
// only after the last word, so it writes E = exp(l - ref) with a reference
// that is known before the product, the label's logit t (a dot product a row,
// xent_target_kernel).  E rounded to bf16 keeps its relative precision
// whatever its size, and sum_v p_v >= p_y makes sum_v E >= 1: nothing that
// counts is lost below.  Above, a (row, 128 words) whose largest l exceeds t
// by 40 takes that largest l as its reference instead, writes it beside its
// sum, and xent_rows_kernel rescales such rows' E to the row's largest
// reference afterwards.  The rest is linear:
//   Zx = sum_{v != y} E_v, Z = E_y + Zx, loss = log Z + ref - t
//        (log1p(Zx) where the reference is t: exact for sure predictions),
//   E_y := -Zx (p_y - 1 = -Zx / Z without cancellation),
//   dX_i = (g / Z_i) sum_v E_iv W_v         (scaled in the epilogue)
//   dW_v = sum_i E_iv (g / Z_i) x_i         (x scaled and rounded once)
// Roundings to bf16: E, the scaled x, and the results.  The label's term
// outweighs the others, so the row's factor takes its E's rounding out again
// (and puts that half step on the other words' terms).
//
// All three products run on the 2-SM tcgen05 tiles of the layer's projection
// (256 x 256 of a CTA pair, 64-deep k-blocks by TMA into a 6-stage ring, two
// TMEM accumulators, 8 epilogue warps a CTA).  Every extent may be ragged:
// TMA fills what is behind an edge with zeros and clips stores.
#include <cuda_bf16.h>

#include "flash_gau_internal.h"
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

// kLoss: the logits' product, sums only; kProbs: sums and E; kDX: E W with
// scaled rows, or fp32 parts of a split sum; kDW: E^T X', stored in bf16, or
// in fp32, or added to fp32
enum Epi { kLoss, kProbs, kDX, kDW };

struct Params {
  int M, N, K;  // of the product; the logits' N is V
  int row_pairs, n_tiles, splits, kb_split, total;
  int rows_first;  // row pairs walk fastest (the logits), else columns
  const float *ref;     // [M] the label's logit in units of ln 2
  const int *labels;    // [M]
  float2 *part;         // [N / 128, rounded up][M] (reference, sum without the label)
  const float *scale;   // [M] kDX without splits: factors of the rows
  int fp32;             // kDX / kDW: fp32 result
  int add;              // kDW: add to the fp32 result
  int part_rows;        // kDX with splits: rows between parts
  int *status;
};

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

struct Tile {
  int rp, n0, nsz, kb0, kb1, split;
};
__device__ __forceinline__ Tile tile_of(const Params &p, int t) {
  Tile x;
  const int tiles = p.row_pairs * p.n_tiles;
  x.split = t / tiles;
  const int u = t - x.split * tiles;
  int nt;
  if (p.rows_first) {
    x.rp = u % p.row_pairs;
    nt = u / p.row_pairs;
  } else {
    nt = u % p.n_tiles;
    x.rp = u / p.n_tiles;
  }
  x.n0 = nt * BN;
  // a multiple of 128: each CTA holds whole 64-column boxes; the logits'
  // sums are kept by 128 words, so their tiles are never narrower
  x.nsz = p.rows_first ? BN : min(BN, (p.N - x.n0 + 127) / 128 * 128);
  x.kb0 = x.split * p.kb_split;
  x.kb1 = min((p.K + BK - 1) / BK, x.kb0 + p.kb_split);
  return x;
}

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

template <int EPI>
__global__ void __launch_bounds__(NUM_THREADS, 1)
xent_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const __grid_constant__ CUtensorMap tmC, const Params p) {
  constexpr bool A_MN = EPI == kDW;                     // E read by columns
  constexpr bool B_KM = EPI == kLoss || EPI == kProbs;  // W read by rows
  extern __shared__ uint8_t smem_raw[];
  uint8_t *tiles = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Smem *sm = reinterpret_cast<Smem *>(tiles + TILE_BYTES);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = (int)cluster_ctarank();
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
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
  const int first = blockIdx.x / 2, step = gridDim.x / 2;

  if (warp == 0) {
    // ------------------------------------------------ TMA producer (both)
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      for (int t = first; t < p.total && !sm->abort_flag; t += step) {
        const Tile x = tile_of(p, t);
        const int m0 = (x.rp * 2 + rank) * BM, half = x.nsz / 2, hboxes = half / 64;
        for (int kb = x.kb0; kb < x.kb1; ++kb) {
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
            tma_load_2d_pair(smem_u32(sA), &tmA, full_leader, m0, kb * BK);
            tma_load_2d_pair(smem_u32(sA + BOX_BYTES), &tmA, full_leader, m0 + 64, kb * BK);
          } else {
            tma_load_2d_pair(smem_u32(sA), &tmA, full_leader, kb * BK, m0);
          }
          if (B_KM) {
            tma_load_2d_pair(smem_u32(sB), &tmB, full_leader, kb * BK, x.n0 + rank * half);
          } else {
            for (int j = 0; j < hboxes; ++j)
              tma_load_2d_pair(smem_u32(sB + j * BOX_BYTES), &tmB, full_leader,
                               x.n0 + rank * half + j * 64, kb * BK);
          }
          if (++stage == STAGES) {
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
      for (int t = first; t < p.total && !sm->abort_flag; t += step, ++local) {
        const Tile x = tile_of(p, t);
        const int acc = local & 1;
        if (!mbar_wait(smem_u32(&sm->acc_empty[acc]), ((local >> 1) & 1) ^ 1, &sm->abort_flag)) {
          raise_timeout(sm, p.status);
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * ACC_COLS;
        const uint32_t idesc = idesc_bf16_f32(2 * BM, x.nsz, A_MN ? 1 : 0, B_KM ? 0 : 1);
        bool ok = true;
        for (int kb = x.kb0; kb < x.kb1; ++kb) {
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
                            kb != x.kb0 || k != 0);
          mma_commit_pair_mc(smem_u32(&sm->empty[stage]), kPair);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        mma_commit_pair_mc(smem_u32(&sm->acc_full[acc]), kPair);
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
    for (int t = first; t < p.total && !sm->abort_flag; t += step, ++local) {
      const Tile x = tile_of(p, t);
      const int acc = local & 1;
      const int row0 = (x.rp * 2 + rank) * BM + quarter * 32, row = row0 + lane;
      const int c_begin = half * (x.nsz / 2), c_end = c_begin + x.nsz / 2;
      const bool live = row < p.M;
      // this row's scalars, before the wait
      float ref = 0.f, scale = 0.f;
      int label = -1;
      if constexpr (EPI == kLoss || EPI == kProbs) {
        if (live) {
          ref = p.ref[row];
          label = p.labels[row];
          if (label >= p.N) label = -1;
        }
      }
      if constexpr (EPI == kDX)
        if (!p.fp32 && live) scale = p.scale[row];
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
      if constexpr (EPI == kLoss || EPI == kProbs) {
        const bool whole = x.n0 + c_end <= p.N;  // every column is a word
        // the largest logit of this row's 128 words
        float top = -INFINITY;
        for (int c0 = c_begin; c0 < c_end; c0 += 32) {
          uint32_t v[32];
          tmem_ld32(taddr + c0, v);
          tmem_ld_wait();
          if (whole) {
#pragma unroll
            for (int j = 0; j < 32; ++j) top = fmaxf(top, __uint_as_float(v[j]));
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (x.n0 + c0 + j < p.N) top = fmaxf(top, __uint_as_float(v[j]));
          }
        }
        top *= kLog2e;
        if (top > ref + kRaise) ref = top;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        for (int c0 = c_begin; c0 < c_end; c0 += 64) {
          if (EPI == kProbs) st.begin();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t v[32];
            tmem_ld32(taddr + c0 + 32 * h, v);
            tmem_ld_wait();
            if (c0 + 64 >= c_end && h == 1) drained();
            const int col = x.n0 + c0 + 32 * h;
            float e[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) e[j] = exp2_approx(fmaf(__uint_as_float(v[j]), kLog2e, -ref));
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
            if (label < 0) {  // whatever the row holds
#pragma unroll
              for (int j = 0; j < 32; ++j) e[j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) sum[j & 3] += e[j];
            if (EPI == kProbs) {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                st.put(4 * h + q, make_uint4(pack_bf16(e[8 * q], e[8 * q + 1]),
                                             pack_bf16(e[8 * q + 2], e[8 * q + 3]),
                                             pack_bf16(e[8 * q + 4], e[8 * q + 5]),
                                             pack_bf16(e[8 * q + 6], e[8 * q + 7])));
            }
          }
          // boxes wholly behind an edge are not stored
          if (EPI == kProbs && row0 < p.M && x.n0 + c0 < p.N)
            st.finish(&tmC, x.n0 + c0, row0, false);
        }
        if (live && x.n0 + c_begin < p.N)
          p.part[(size_t)((x.n0 + c_begin) / 128) * p.M + row] =
              make_float2(ref, (sum[0] + sum[1]) + (sum[2] + sum[3]));
      } else {
        const int out_row = row0 + (EPI == kDX ? x.split * p.part_rows : 0);
        for (int c0 = c_begin; c0 < c_end; c0 += 64) {
          uint32_t a[32], b[32];
          tmem_ld32(taddr + c0, a);
          tmem_ld32(taddr + c0 + 32, b);
          tmem_ld_wait();
          if (c0 + 64 >= c_end) drained();
          if (row0 >= p.M || x.n0 + c0 >= p.N) continue;
          if (p.fp32) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t *v = h == 0 ? a : b;
              if (x.n0 + c0 + 32 * h >= p.N) break;
              st.begin();
#pragma unroll
              for (int q = 0; q < 8; ++q)
                st.put(q, make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]));
              st.finish(&tmC, x.n0 + c0 + 32 * h, out_row, EPI == kDW && p.add);
            }
          } else {
            st.begin();
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const uint32_t *v = q < 4 ? &a[8 * q] : &b[8 * (q - 4)];
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                float lo = __uint_as_float(v[2 * k]), hi = __uint_as_float(v[2 * k + 1]);
                if (EPI == kDX) {
                  lo *= scale;
                  hi *= scale;
                }
                w[k] = pack_bf16(lo, hi);
              }
              st.put(q, make_uint4(w[0], w[1], w[2], w[3]));
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
                        const Params &p, int num_sms, cudaStream_t stream) {
  static int max_pairs[64];
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
  if (max_pairs[dev] == 0) {
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (err != cudaSuccess) return err;
    int n = 0;
    cfg.gridDim = dim3(2 * (num_sms / 2));
    err = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
    if (err != cudaSuccess) return err;
    max_pairs[dev] = n > 0 ? n : 1;
  }
  cfg.gridDim = dim3(2 * (p.total < max_pairs[dev] ? p.total : max_pairs[dev]));
  return cudaLaunchKernelEx(&cfg, kernel, a, b, c, p);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ int label_of(const int *labels, long long i, int V) {
  const int y = labels[i];
  return y >= 0 && y < V ? y : -1;
}

// One warp a row: ref = log2(e) x . W_y, 0 for rows without a label.  The
// launch's last block instead counts the labels of all N tokens and writes
// the factor g of the gradients (count != null).
__global__ void __launch_bounds__(256)
xent_target_kernel(const __nv_bfloat16 *__restrict__ X, const __nv_bfloat16 *__restrict__ W,
                   const int *__restrict__ labels, int rows, int d, int V, float *__restrict__ ref,
                   const int *__restrict__ all_labels, long long N, int mean, float scale,
                   float *__restrict__ factor) {
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (factor && blockIdx.x == gridDim.x - 1) {
    __shared__ int counts[8];
    int n = 0;
    for (long long i = threadIdx.x; i < N; i += blockDim.x) n += label_of(all_labels, i, V) >= 0;
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) counts[warp] = n;
    __syncthreads();
    if (threadIdx.x == 0) {
      n = 0;
      for (int k = 0; k < 8; ++k) n += counts[k];
      *factor = mean ? scale / (float)(n > 0 ? n : 1) : scale;
    }
    return;
  }
  const int row = blockIdx.x * 8 + warp;
  if (row >= rows) return;
  const int y = label_of(labels, row, V);
  float s = 0.f;
  if (y >= 0) {
    const uint4 *x = reinterpret_cast<const uint4 *>(X + (size_t)row * d);
    const uint4 *w = reinterpret_cast<const uint4 *>(W + (size_t)y * d);
    for (int k = lane; k < d / 8; k += 32) {
      const uint4 a = __ldg(x + k), b = __ldg(w + k);
      const uint32_t au[4] = {a.x, a.y, a.z, a.w}, bu[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&au[q]));
        const float2 g = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&bu[q]));
        s = fmaf(f.x, g.x, fmaf(f.y, g.y, s));
      }
    }
    s = warp_sum(s);
  }
  if (lane == 0) ref[row] = s * kLog2e;
}

struct RowArgs {
  const float *ref;
  const int *labels;
  const float2 *part;
  int parts, rows, V, d;
  float *loss, *lse;           // of this piece's rows; lse may be null
  const float *factor;
  __nv_bfloat16 *E;            // null: no gradients
  long long ldE;
  float *scale;                // g / Z
  const __nv_bfloat16 *X;
  __nv_bfloat16 *Xs;           // (g / Z) x, or null
};

// 32 rows a block: joins the parts of each row's sum (a lane a row, the
// parts dealt to 8 warps), writes the loss, and with gradients the row's
// factor, the label's E, the scaled row of X, and where a part took another
// reference than the row's its E again.
__global__ void __launch_bounds__(256) xent_rows_kernel(const RowArgs a) {
  __shared__ float2 joined[8][32];
  __shared__ float row_ref[32], row_scale[32];
  __shared__ int row_mixed[32];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row0 = blockIdx.x * 32, row = row0 + lane;
  const bool live = row < a.rows;
  const float ref = live ? a.ref[row] : 0.f;
  float top = ref, sum = 0.f;
  int mixed = 0;
  auto join = [&](float2 v) {
    if (v.x == top) {
      sum += v.y;
    } else {
      mixed = 1;
      const float t = fmaxf(top, v.x);
      // a reference of minus infinity has no terms below it
      sum = (top == t ? sum : sum * exp2f(top - t)) + (v.x == t ? v.y : v.y * exp2f(v.x - t));
      top = t;
    }
  };
  if (live)
    for (int k = warp; k < a.parts; k += 8) join(a.part[(size_t)k * a.rows + row]);
  joined[warp][lane] = make_float2(top, sum);
  if (warp == 0) row_mixed[lane] = 0;
  __syncthreads();
  if (mixed) row_mixed[lane] = 1;
  if (warp == 0) {
    for (int k = 1; k < 8; ++k) join(joined[k][lane]);
    const int label = live ? label_of(a.labels, row, a.V) : -1;
    float loss = 0.f, scale = 0.f;
    if (label >= 0) {
      if (top == ref) {
        // an infinite logit makes both NaN, as inf - inf does
        loss = log1pf(sum) + 0.f * ref;
        scale = *a.factor / (1.0f + sum) + 0.f * ref;
      } else {
        const float z = exp2f(ref - top) + sum;
        loss = logf(z) + (top - ref) * kLn2;
        scale = *a.factor / z;
      }
    }
    if (live) {
      a.loss[row] = loss;
      if (a.lse) a.lse[row] = label >= 0 ? fmaf(ref, kLn2, loss) : 0.f;
      if (a.E) {
        if (label >= 0) {
          const __nv_bfloat16 own = __float2bfloat16_rn(-sum);
          a.E[(size_t)row * a.ldE + label] = own;
          // its rounding goes into the row's factor
          if (sum > 0.f && sum < INFINITY) scale *= sum / -__bfloat162float(own);
        }
        a.scale[row] = scale;
      }
    }
    row_ref[lane] = top;
    row_scale[lane] = scale;
    if (mixed) row_mixed[lane] = 1;
  }
  if (!a.E) return;
  __syncthreads();
  for (int k = warp; k < 32 && row0 + k < a.rows; k += 8) {
    const int r = row0 + k, label = label_of(a.labels, r, a.V);
    if (a.Xs) {
      const uint4 *x = reinterpret_cast<const uint4 *>(a.X + (size_t)r * a.d);
      uint4 *o = reinterpret_cast<uint4 *>(a.Xs + (size_t)r * a.d);
      const float s = row_scale[k];
      for (int j = lane; j < a.d / 8; j += 32) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (label >= 0) {
          w = __ldg(x + j);
          uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u[q]));
            u[q] = pack_bf16(f.x * s, f.y * s);
          }
          w = make_uint4(u[0], u[1], u[2], u[3]);
        }
        o[j] = w;
      }
    }
    if (row_mixed[k] && label >= 0) {
      for (int j = 0; j < a.parts; ++j) {
        const float from = a.part[(size_t)j * a.rows + r].x;
        if (from == row_ref[k]) continue;
        const float f = exp2f(from - row_ref[k]);
        for (int c = 128 * j + lane; c < min(128 * j + 128, a.V); c += 32)
          if (c != label) {
            __nv_bfloat16 *e = a.E + (size_t)r * a.ldE + c;
            *e = __float2bfloat16_rn(__bfloat162float(*e) * f);
          }
      }
    }
  }
}

// dX from the fp32 parts of its split sum, in the parts' order.
__global__ void __launch_bounds__(256)
xent_join_kernel(const float *__restrict__ part, long long stride, int splits,
                 const float *__restrict__ scale, int rows, int d, __nv_bfloat16 *__restrict__ out) {
  griddep_wait();
  const long long i = (blockIdx.x * 256LL + threadIdx.x) * 4;
  if (i >= (long long)rows * d) return;
  float4 s = *reinterpret_cast<const float4 *>(part + i);
  for (int k = 1; k < splits; ++k) {
    const float4 v = *reinterpret_cast<const float4 *>(part + k * stride + i);
    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
  }
  const float f = scale[i / d];
  *reinterpret_cast<uint2 *>(out + i) =
      make_uint2(pack_bf16(s.x * f, s.y * f), pack_bf16(s.z * f, s.w * f));
}

__global__ void __launch_bounds__(256)
xent_round_kernel(const float *__restrict__ in, long long n, __nv_bfloat16 *__restrict__ out) {
  griddep_wait();
  const long long i = (blockIdx.x * 256LL + threadIdx.x) * 8;
  if (i >= n) return;
  const float4 a = *reinterpret_cast<const float4 *>(in + i);
  const float4 b = *reinterpret_cast<const float4 *>(in + i + 4);
  *reinterpret_cast<uint4 *>(out + i) = make_uint4(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w),
                                                   pack_bf16(b.x, b.y), pack_bf16(b.z, b.w));
}

// total = factor * sum of the losses, in a fixed order
__global__ void __launch_bounds__(1024)
xent_total_kernel(const float *__restrict__ loss, long long N, const float *__restrict__ factor,
                  float *__restrict__ total) {
  __shared__ float buf[32];
  griddep_wait();
  float s = 0.f;
  for (long long i = threadIdx.x; i < N; i += 1024) s += loss[i];
  s = warp_sum(s);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x < 32) {
    s = warp_sum(buf[threadIdx.x]);
    if (threadIdx.x == 0) *total = *factor * s;
  }
}

Params gemm_params(int M, int N, int K, int *status) {
  Params p = {};
  p.M = M;
  p.N = N;
  p.K = K;
  p.row_pairs = (M + 2 * BM - 1) / (2 * BM);
  p.n_tiles = (N + BN - 1) / BN;
  p.splits = 1;
  p.kb_split = (K + BK - 1) / BK;
  p.total = p.row_pairs * p.n_tiles;
  p.status = status;
  return p;
}

}  // namespace

// Splits of dX's sum over the words: the count with the least estimated time,
// the rounds of tiles over the pairs times a split's k-blocks (0.33 us a
// k-block of a 256 x 256 tile at the measured bf16 rate), plus for more than
// one the fp32 parts, written and read again at about 5 TB/s.
int xent_dx_splits(int rows, int d, int V) {
  const int tiles = ((rows + 2 * BM - 1) / (2 * BM)) * ((d + BN - 1) / BN);
  const int pairs = kXentPlanSms / 2, kblocks = (V + BK - 1) / BK;
  int best_n = 1;
  double best = 0.0;
  for (int s = 1; s <= 32 && (s == 1 || kblocks / s >= 8); ++s) {
    const int kb = (kblocks + s - 1) / s, n = (kblocks + kb - 1) / kb;
    const long long rounds = ((long long)tiles * n + pairs - 1) / pairs;
    const double cost = 0.33 * (double)rounds * kb +
                        (n > 1 ? n * (double)rows * d * 8 / 5e6 + 4.0 : 0.0);
    if (s == 1 || cost < best) {
      best = cost;
      best_n = n;
    }
  }
  return best_n;
}

cudaError_t xent_bf16(const XentProblem &q) {
  const XentLayout &L = q.L;
  cudaError_t err = cudaMemsetAsync(L.status, 0, sizeof(int), q.stream);
  if (err != cudaSuccess) return err;
  const bool grad = q.dX || q.dW;
  const __nv_bfloat16 *X = static_cast<const __nv_bfloat16 *>(q.X);
  const __nv_bfloat16 *W = static_cast<const __nv_bfloat16 *>(q.W);
  CUtensorMap tW, tWn;
  if ((err = make_tmap_bf16_2d(&tW, W, q.V, q.d, q.d, BN / 2, BK)) != cudaSuccess) return err;
  if ((err = make_tmap_bf16_2d(&tWn, W, q.V, q.d, q.d, BK, 64)) != cudaSuccess) return err;
  const bool pieces = L.piece < q.N;
  for (long long n0 = 0; n0 < q.N; n0 += L.piece) {
    const int rows = (int)(q.N - n0 < L.piece ? q.N - n0 : L.piece);
    const __nv_bfloat16 *x = X + n0 * q.d;
    const int *labels = q.labels + n0;
    float *factor = n0 == 0 ? L.factor : nullptr;
    err = launch_pdl(xent_target_kernel, dim3((rows + 7) / 8 + (factor ? 1 : 0)), dim3(256), 0,
                     q.stream, x, W, labels, rows, q.d, q.V, L.ref, q.labels, q.N, q.mean, q.scale,
                     factor);
    if (err != cudaSuccess) return err;
    CUtensorMap tX, tE = tW;
    if ((err = make_tmap_bf16_2d(&tX, x, rows, q.d, q.d, BM, BK)) != cudaSuccess) return err;
    if (grad && (err = make_tmap_bf16_2d(&tE, L.E, rows, q.V, L.ldE, 32, 64)) != cudaSuccess)
      return err;
    Params p = gemm_params(rows, q.V, q.d, L.status);
    p.rows_first = 1;
    p.ref = L.ref;
    p.labels = labels;
    p.part = L.part;
    err = grad ? launch_gemm<kProbs>(tX, tW, tE, p, q.num_sms, q.stream)
               : launch_gemm<kLoss>(tX, tW, tE, p, q.num_sms, q.stream);
    if (err != cudaSuccess) return err;
    RowArgs r = {};
    r.ref = L.ref;
    r.labels = labels;
    r.part = L.part;
    r.parts = (q.V + 127) / 128;
    r.rows = rows;
    r.V = q.V;
    r.d = q.d;
    r.loss = q.loss + n0;
    r.lse = q.lse ? q.lse + n0 : nullptr;
    r.factor = L.factor;
    r.E = grad ? static_cast<__nv_bfloat16 *>(L.E) : nullptr;
    r.ldE = L.ldE;
    r.scale = L.row_scale;
    r.X = x;
    r.Xs = q.dW ? static_cast<__nv_bfloat16 *>(L.Xs) : nullptr;
    err = launch_pdl(xent_rows_kernel, dim3((rows + 31) / 32), dim3(256), 0, q.stream, r);
    if (err != cudaSuccess) return err;
    if (q.dX) {
      __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(q.dX) + n0 * q.d;
      CUtensorMap tEa, tO;
      if ((err = make_tmap_bf16_2d(&tEa, L.E, rows, q.V, L.ldE, BM, BK)) != cudaSuccess) return err;
      Params g = gemm_params(rows, q.d, q.V, L.status);
      const int splits = xent_dx_splits(rows, q.d, q.V);
      g.kb_split = (g.kb_split + splits - 1) / splits;
      g.splits = splits;
      g.total *= splits;
      g.scale = L.row_scale;
      g.fp32 = splits > 1;
      g.part_rows = (rows + 31) / 32 * 32;
      if (splits > 1)
        err = make_tmap_f32_2d(&tO, L.dx_part, (uint64_t)splits * g.part_rows, q.d, q.d, 32, 32);
      else
        err = make_tmap_bf16_2d(&tO, out, rows, q.d, q.d, 32, 64);
      if (err != cudaSuccess) return err;
      if ((err = launch_gemm<kDX>(tEa, tWn, tO, g, q.num_sms, q.stream)) != cudaSuccess) return err;
      if (splits > 1) {
        const long long quads = (long long)rows * q.d / 4;
        err = launch_pdl(xent_join_kernel, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0,
                         q.stream, L.dx_part, (long long)g.part_rows * q.d, splits, L.row_scale,
                         rows, q.d, out);
        if (err != cudaSuccess) return err;
      }
    }
    if (q.dW) {
      CUtensorMap tEt, tXs, tO;
      if ((err = make_tmap_bf16_2d(&tEt, L.E, rows, q.V, L.ldE, BK, 64)) != cudaSuccess) return err;
      if ((err = make_tmap_bf16_2d(&tXs, L.Xs, rows, q.d, q.d, BK, 64)) != cudaSuccess) return err;
      if (pieces) err = make_tmap_f32_2d(&tO, L.dw_sum, q.V, q.d, q.d, 32, 32);
      else err = make_tmap_bf16_2d(&tO, q.dW, q.V, q.d, q.d, 32, 64);
      if (err != cudaSuccess) return err;
      Params g = gemm_params(q.V, q.d, rows, L.status);
      g.fp32 = pieces;
      g.add = n0 > 0;
      if ((err = launch_gemm<kDW>(tEt, tXs, tO, g, q.num_sms, q.stream)) != cudaSuccess) return err;
    }
  }
  if (q.dW && pieces) {
    const long long n = (long long)q.V * q.d;
    err = launch_pdl(xent_round_kernel, dim3((unsigned)((n / 8 + 255) / 256)), dim3(256), 0,
                     q.stream, L.dw_sum, n, static_cast<__nv_bfloat16 *>(q.dW));
    if (err != cudaSuccess) return err;
  }
  return xent_total(q);
}

cudaError_t xent_total(const XentProblem &q) {
  return launch_pdl(xent_total_kernel, dim3(1), dim3(1024), 0, q.stream, q.loss, q.N, q.L.factor,
                    q.total);
}

}  // namespace flashgau
