// Activation checkpoints in 8 bits (checkpoint_rows.cuh): the kernels over rows on
// vectors' boundaries, a LayerNorm's gradients with copies ahead, the join of the
// blocks' sums, and the choice between them.  Rows that are not on boundaries
// have a file of their own (checkpoint_odd.cu), so that both compile at once.
#include "checkpoint_rows.cuh"

namespace flashgau {
namespace {

__device__ __forceinline__ void copy16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(dst)), "l"(src)
               : "memory");
}
template <int BYTES>
__device__ __forceinline__ void copy_few(void *dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(ptx::smem_u32(dst)), "l"(src),
               "n"(BYTES)
               : "memory");
}

__device__ __forceinline__ Eight widen(const uint4 *p, int step, const float *) {
  const ulonglong2 *q = reinterpret_cast<const ulonglong2 *>(p);
  const ulonglong2 v[2] = {q[0], q[step]};
  return {{v[0].x, v[0].y, v[1].x, v[1].y}};
}
__device__ __forceinline__ Eight widen(const uint4 *p, int, const __nv_bfloat16 *) {
  const uint4 w = *p;
  return {{unpack_bf16(w.x), unpack_bf16(w.y), unpack_bf16(w.z), unpack_bf16(w.w)}};
}

// Shared memory of a step: for each of a thread's NC runs of 8 columns dn, dr,
// codes and the scale, the threads' side by side.
constexpr int ring_run(int io, int threads) { return threads * (2 * 8 * io + 8 + 4); }
// steps under way: as many as fit, up to four
constexpr int ring_steps(int io, int runs, int threads) {
  const int n = 200 * 1024 / (runs * ring_run(io, threads));
  return n < 4 ? n : 4;
}
template <typename T, int NC, int THREADS>
struct Ring {
  static constexpr int kPieces = sizeof(T) * 8 / 16;  // 16-byte pieces of a run
  static constexpr int kRun = ring_run(sizeof(T), THREADS);
  static constexpr int kStep = NC * kRun;
  static constexpr int kSteps = ring_steps(sizeof(T), NC, THREADS);
  static constexpr int kBytes = kSteps * kStep;
  char *at;
  __device__ uint4 *dn(int k) const { return reinterpret_cast<uint4 *>(at + k * kRun) + threadIdx.x; }
  __device__ uint4 *dr(int k) const { return dn(k) + kPieces * THREADS; }
  __device__ uint2 *codes(int k) const {
    return reinterpret_cast<uint2 *>(at + k * kRun + 32 * kPieces * THREADS) + threadIdx.x;
  }
  __device__ float *scale(int k) const {
    return reinterpret_cast<float *>(at + k * kRun + (32 * kPieces + 8) * THREADS) + threadIdx.x;
  }
};

template <typename T, int NC, int WARPS, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) ring_backward_kernel(const CheckpointArgs a) {
  using R = Ring<T, NC, THREADS>;
  constexpr int kRows = THREADS / 32 / WARPS;
  extern __shared__ __align__(16) char shared[];
  __shared__ float part[kRows * 2 * WARPS];
  const int t = threadIdx.x % (32 * WARPS), group = threadIdx.x / (32 * WARPS);
  RowSum<WARPS> row_sum{part + group * 2 * WARPS, group};
  float s1;
  Eight sg[NC] = {}, sb[NC] = {};
  ptx::griddep_wait();
  auto fetch = [&](long long m, int turn) {
    const R r{shared + turn * R::kStep};
    if (m < a.M) {
      const long long at = m * a.d;
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        const int c = (k * 32 * WARPS + t) * 8;
        if (c >= a.d) continue;
#pragma unroll
        for (int v = 0; v < R::kPieces; ++v) {
          constexpr int kElements = 16 / sizeof(T);
          copy16(r.dn(k) + v * THREADS, static_cast<const T *>(a.dn) + at + c + v * kElements);
          if (a.dr)
            copy16(r.dr(k) + v * THREADS, static_cast<const T *>(a.dr) + at + c + v * kElements);
        }
        copy_few<8>(r.codes(k), a.codes + at + c);
        copy_few<4>(r.scale(k), a.scales + m * a.groups + c / kGroup);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const long long step = (long long)gridDim.x * kRows;
  long long m = (long long)blockIdx.x * kRows + group;
#pragma unroll
  for (int i = 0; i < R::kSteps - 1; ++i) fetch(m + i * step, i);
  // a LayerNorm's g, behind the steps
  float *gains = reinterpret_cast<float *>(shared + R::kBytes);
  for (int c = threadIdx.x; c < a.d; c += THREADS) gains[c] = a.norm_g[c];
  __syncthreads();
  const Eight none = {{0, 0, 0, 0}};
  const RowAt one(0, 1, a.d);
  for (int turn = 0; m < a.M; m += step, turn = turn + 1 == R::kSteps ? 0 : turn + 1) {
    fetch(m + (R::kSteps - 1) * step, turn ? turn - 1 : R::kSteps - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(R::kSteps - 1) : "memory");
    const R r{shared + turn * R::kStep};
    Eight x[NC], w[NC];
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      x[k] = w[k] = none;
      if ((k * 32 * WARPS + t) * 8 < a.d) {
        x[k] = times_scale(*r.codes(k), *r.scale(k));
        w[k] = widen(r.dn(k), THREADS, static_cast<const T *>(nullptr));
      }
    }
    row_gradient<true, NC, WARPS>(a, x, w, sg, sb, s1, t, row_sum, [&](int k) {
      return load8<true>(gains, one, (k * 32 * WARPS + t) * 8, a.d);
    });
    const RowAt row(m, a.M, a.d);
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = (k * 32 * WARPS + t) * 8;
      if (c >= a.d) continue;
      if (a.dr) {
        const Eight v = widen(r.dr(k), THREADS, static_cast<const T *>(nullptr));
#pragma unroll
        for (int q = 0; q < 4; ++q) w[k].v[q] = add2(w[k].v[q], v.v[q]);
      }
      store8<true>(static_cast<T *>(a.dh), row, c, a.d, w[k]);
    }
  }
  if (!a.part) return;
  // the block's sums: every group's in shared memory, then column by column
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  float *cols = reinterpret_cast<float *>(shared);
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const int c = (k * 32 * WARPS + t) * 8;
    if (c >= a.d) continue;
    store8<true>(cols, RowAt(2 * group, 2 * kRows, a.d), c, a.d, sg[k]);
    store8<true>(cols, RowAt(2 * group + 1, 2 * kRows, a.d), c, a.d, sb[k]);
  }
  __syncthreads();
  float *to = a.part + (long long)blockIdx.x * 2 * a.d;
  for (int c = threadIdx.x; c < 2 * a.d; c += THREADS) {
    float v = cols[c];
#pragma unroll
    for (int g = 1; g < kRows; ++g) v += cols[(long long)g * 2 * a.d + c];
    to[c] = v;
  }
}

// Adds the blocks' sums up: 32 columns a block, its 32 warps taking every 32nd
// block's row, then the 32 in order.
__global__ void __launch_bounds__(1024)
join_columns_kernel(const float *__restrict__ part, int blocks, int d, float *__restrict__ dg,
                    float *__restrict__ db) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
  ptx::griddep_wait();
  float v = 0.f;
  if (c < 2 * d)
#pragma unroll 5
    for (int b = w; b < blocks; b += 32) v += part[(long long)b * 2 * d + c];
  s[lane][w] = v;
  __syncthreads();
  const float all = warp_sum(s[w][lane]);  // warp w's column
  const int mine = blockIdx.x * 32 + w;
  float *to = mine < d ? dg : db;
  if (lane == 0 && mine < 2 * d && to) to[mine < d ? mine : mine - d] = all;
}
// ScaleNorm's one g: n sums of both signs that nearly cancel, so what each
// addition cuts off is added up beside it.
__global__ void __launch_bounds__(1024)
join_scalar_kernel(const float *__restrict__ part, int n, float *__restrict__ dg) {
  __shared__ float2 s[32];
  ptx::griddep_wait();
  float2 v = make_float2(0.f, 0.f);
  auto add = [&](float x, float left) {
    const float t = v.x + x, b = t - v.x;
    v.y += (v.x - (t - b)) + (x - b) + left;
    v.x = t;
  };
  auto warp = [&] {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      add(__shfl_xor_sync(kAll, v.x, o), __shfl_xor_sync(kAll, v.y, o));
  };
  for (int k = threadIdx.x; k < n; k += 1024) add(part[k], 0.f);
  warp();
  if (threadIdx.x % 32 == 0) s[threadIdx.x / 32] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    v = s[threadIdx.x];
    warp();
    if (threadIdx.x == 0) *dg = v.x + v.y;
  }
}

// The form with copies ahead, one block an SM.  Returns the blocks' number and
// their warps.
struct Grid {
  int blocks, warps;
};
template <typename T, int NC, int WARPS>
cudaError_t launch_ring(const CheckpointArgs &a, int num_sms, cudaStream_t stream, Grid *g) {
  // as many as the column sums' registers leave, and three steps' memory where a
  // row's warps allow
  constexpr int kMost = NC < 3 ? 512 : NC == 3 ? 384 : 256, kIo = sizeof(T);
  constexpr int kThreads = ring_steps(kIo, NC, kMost) >= 3               ? kMost
                           : kMost > 384 && ring_steps(kIo, NC, 384) >= 3 ? 384
                           : ring_steps(kIo, NC, 256) >= 3 || WARPS == 8 ? 256
                           : WARPS == 4                                  ? 128
                                                                         : 192;
  constexpr int kRows = kThreads / 32 / WARPS;
  constexpr auto kernel = ring_backward_kernel<T, NC, WARPS, kThreads>;
  // the steps and a LayerNorm's g, then the groups' column sums; d is at most kD
  constexpr size_t kD = NC * WARPS * 256, kSteps = Ring<T, NC, kThreads>::kBytes;
  constexpr size_t kSums = kRows * 2 * kD * sizeof(float), kAll = kSteps + kD * sizeof(float);
  constexpr size_t kMostShared = kSums > kAll ? kSums : kAll;
  const cudaError_t err = allow_shared<kernel>(kMostShared);
  if (err != cudaSuccess) return err;
  const size_t sums = (size_t)kRows * 2 * a.d * sizeof(float);
  const size_t steps = kSteps + a.d * sizeof(float), smem = sums > steps ? sums : steps;
  const long long all = (a.M + kRows - 1) / kRows;
  g->blocks = (int)(all < num_sms ? all : num_sms);
  if (g->blocks > kCheckpointBlocks) g->blocks = kCheckpointBlocks;
  g->warps = kThreads / 32;
  return launch_pdl(kernel, dim3(g->blocks), dim3(kThreads), smem, stream, a);
}
template <typename T>
cudaError_t dispatch_ring(const CheckpointArgs &a, int num_sms, cudaStream_t stream, Grid *g) {
  if (a.d <= 256) return launch_ring<T, 1, 1>(a, num_sms, stream, g);
  if (a.d <= 512) return launch_ring<T, 2, 1>(a, num_sms, stream, g);
  if (a.d <= 768) return launch_ring<T, 3, 1>(a, num_sms, stream, g);
  if (a.d <= 1024) return launch_ring<T, 4, 1>(a, num_sms, stream, g);
  if (a.d <= 2048) return launch_ring<T, 2, 4>(a, num_sms, stream, g);
  if (a.d <= 4096) return launch_ring<T, 4, 4>(a, num_sms, stream, g);
  return launch_ring<T, 4, 8>(a, num_sms, stream, g);
}

bool on(const void *p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

CheckpointArgs finish(CheckpointArgs a) {
  a.groups = (a.d + kGroup - 1) / kGroup;
  a.vec = a.d % 8 == 0 && on(a.codes, 8);
  for (const void *p : {a.h, a.y, a.dr, a.dn, (const void *)a.r, (const void *)a.n,
                        (const void *)a.dh, (const void *)a.norm_g, (const void *)a.norm_b})
    a.vec = a.vec && on(p, 16);
  return a;
}

cudaError_t all_rows(int what, const CheckpointArgs &a, int dtype, unsigned most_blocks,
                     cudaStream_t stream) {
  return a.vec ? rows<true>(what, a, dtype, most_blocks, stream)
               : checkpoint_rows_odd(what, a, dtype, most_blocks, stream);
}

}  // namespace

cudaError_t checkpoint_pack(const CheckpointArgs &a, int dtype, cudaStream_t stream) {
  return all_rows(kCheckpointPack, finish(a), dtype, 0, stream);
}

cudaError_t checkpoint_restore(const CheckpointArgs &a, int dtype, cudaStream_t stream) {
  return all_rows(kCheckpointRestore, finish(a), dtype, 0, stream);
}

size_t checkpoint_part_bytes(int d) {
  const size_t columns = (size_t)kCheckpointBlocks * 2 * d, warps = kCheckpointScaleBlocks * 8;
  return (columns > warps ? columns : warps) * sizeof(float);
}

cudaError_t checkpoint_backward(const CheckpointArgs &args, float *dg, float *db, int dtype,
                                int num_sms, cudaStream_t stream) {
  CheckpointArgs a = finish(args);
  if (!dg && !db) a.part = nullptr;
  Grid g;
  cudaError_t err;
  const bool layer = a.norm == FLASH_GAU_NORM_LAYER;
  if (a.vec && layer) {
    err = dtype == FLASH_GAU_BF16 ? dispatch_ring<__nv_bfloat16>(a, num_sms, stream, &g)
                                  : dispatch_ring<float>(a, num_sms, stream, &g);
  } else {
    const unsigned most = layer ? kCheckpointBlocks : kCheckpointScaleBlocks;
    err = all_rows(kCheckpointBackward, a, dtype, most, stream);
    const int warps = checkpoint_row_warps(a.d), rows = warps == 1 ? 4 : 1;
    const long long all = (a.M + rows - 1) / rows;
    g = {(int)(all < most ? all : most), warps > 4 ? warps : 4};
  }
  if (err != cudaSuccess || !a.part) return err;
  if (layer)
    return launch_pdl(join_columns_kernel, dim3((2 * a.d + 31) / 32), dim3(1024), 0, stream,
                      a.part, g.blocks, a.d, dg, db);
  return launch_pdl(join_scalar_kernel, dim3(1), dim3(1024), 0, stream, a.part,
                    g.blocks * g.warps, dg);
}

}  // namespace flashgau
