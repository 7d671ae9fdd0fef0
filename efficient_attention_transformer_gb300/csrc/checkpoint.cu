// Activation checkpoints in 8 bits (checkpoint_rows.cuh): the kernels over rows of
// whole vectors, the join of the blocks' sums, and the choice between the forms.
// The other forms have a file of their own (checkpoint_odd.cu), so that both
// compile at once.
#include "checkpoint_rows.cuh"

namespace flashgau {
namespace {

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
// addition cuts off is added up beside it (of an infinite sum nothing is: infinity
// less itself is no number).
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
    if (threadIdx.x == 0) *dg = isfinite(v.x) ? v.x + v.y : v.x;
  }
}

bool on(const void *p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

CheckpointArgs finish(CheckpointArgs a) {
  a.groups = (a.d + kGroup - 1) / kGroup;
  bool bounds = on(a.codes, 8);
  for (const void *p : {a.h, a.y, a.dr, a.dn, (const void *)a.r, (const void *)a.n,
                        (const void *)a.dh, (const void *)a.norm_g, (const void *)a.norm_b})
    bounds = bounds && on(p, 16);
  // as blocks a row can begin seven columns into its first vector
  a.form = !bounds ? kElements
           : a.d % 8 == 0 ? kVectors
           : a.d + 7 <= kCheckpointMaxD ? kBlocks
                                        : kElements;
  a.width = a.form == kBlocks ? a.d + 7 : a.d;
  return a;
}

cudaError_t all_rows(int what, const CheckpointArgs &a, int dtype, int num_sms,
                     cudaStream_t stream, CheckpointGrid *g) {
  return a.form == kVectors ? rows<kVectors>(what, a, dtype, num_sms, stream, g)
                            : checkpoint_rows_odd(what, a, dtype, num_sms, stream, g);
}

}  // namespace

cudaError_t checkpoint_pack(const CheckpointArgs &a, int dtype, cudaStream_t stream) {
  return all_rows(kCheckpointPack, finish(a), dtype, 0, stream, nullptr);
}

cudaError_t checkpoint_restore(const CheckpointArgs &a, int dtype, cudaStream_t stream) {
  return all_rows(kCheckpointRestore, finish(a), dtype, 0, stream, nullptr);
}

size_t checkpoint_part_bytes(int d) {
  const size_t columns = (size_t)kCheckpointBlocks * 2 * d, warps = kCheckpointScaleBlocks * 8;
  return (columns > warps ? columns : warps) * sizeof(float);
}

cudaError_t checkpoint_backward(const CheckpointArgs &args, float *dg, float *db, int dtype,
                                int num_sms, cudaStream_t stream) {
  CheckpointArgs a = finish(args);
  if (!dg && !db) a.part = nullptr;
  CheckpointGrid g;
  const cudaError_t err = all_rows(kCheckpointBackward, a, dtype, num_sms, stream, &g);
  if (err != cudaSuccess || !a.part) return err;
  if (a.norm == FLASH_GAU_NORM_LAYER)
    return launch_pdl(join_columns_kernel, dim3((2 * a.d + 31) / 32), dim3(1024), 0, stream,
                      a.part, g.blocks, a.d, dg, db);
  return launch_pdl(join_scalar_kernel, dim3(1), dim3(1024), 0, stream, a.part,
                    g.blocks * g.warps, dg);
}

}  // namespace flashgau
