// The layer's relative position table from learned values by buckets of
// distance, and the gradient of those values:
//   relpos[h][C-1 + o] = table[h][bucket(o)]
//   dtable[h][b] = sum over r and all o with bucket(o) = b of drelpos[r][h][C-1 + o]
// where o is a key's offset from its query.  A direction has n buckets, near =
// n / 2: distances below `near` have one each, distance t from there on is in
//   near + floor(log(t / near) / log(far / near) (n - near)),  at most n - 1.
//
// The buckets of a direction are runs of distances, so a list of where each
// run starts says everything.  The host makes it from the definition in whole
// numbers and the kernels take it in their parameters: no table of buckets in
// memory, no logarithm on the device, and a gradient that is a sum over a run
// rather than a scatter, so nothing is added atomically and a call repeats bit
// for bit.  Its sums are fp32, eight values behind one another, then as many of
// those as there are, then a bucket's in 32 lanes: off by 1e-7 (2-norm) at six
// layers, as a result that fp32 rounds; at thousands of layers by up to R / 8
// roundings.
//
// Both move a few MB at most (64 tables of 8191 offsets: 2.1 MB out, six
// layers' gradients 12.6 MB in, 2.2 us at the copy rate), so launch and
// latency bound them: 3.8 and 8.4 us, 1.8 and 3.4 for 12 tables of 511.
#include <cooperative_groups.h>
#include <math.h>

#include "flash_gau_internal.h"

namespace flashgau {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kGradThreads = 512;
constexpr int kMaxCluster = 8;
constexpr int kEach = 2;  // offsets a thread: a cluster of eight takes 8192
constexpr int kRun = 8;   // rows of drelpos under way at once, and in one fp32 sum

struct Starts {
  int n;       // buckets of a direction
  int ahead;   // offsets above zero have buckets n .. 2n-1 of their own
  int start[kBucketMax];  // first distance of each bucket, rising; C or more: of none
};

// Whether (t / near)^m >= (far / near)^i, in whole numbers: t^m near^i against
// far^i near^m, at most 20 bits times 2 * 128 factors each.
struct Whole {
  uint32_t w[176];
  int len;
  void set(uint32_t x) {
    w[0] = x;
    len = 1;
  }
  void times(uint32_t x, int power) {
    for (; power > 0; --power) {
      uint64_t carry = 0;
      for (int k = 0; k < len; ++k) {
        carry += (uint64_t)w[k] * x;
        w[k] = (uint32_t)carry;
        carry >>= 32;
      }
      if (carry) w[len++] = (uint32_t)carry;
    }
  }
  bool at_least(const Whole &o) const {
    if (len != o.len) return len > o.len;
    for (int k = len - 1; k >= 0; --k)
      if (w[k] != o.w[k]) return w[k] > o.w[k];
    return true;
  }
};
bool reaches(uint32_t t, uint32_t near, uint32_t far, int i, int m) {
  Whole a, b;
  a.set(1);
  b.set(1);
  a.times(t, m);
  a.times(near, i);
  b.times(far, i);
  b.times(near, m);
  return a.at_least(b);
}

Starts make_starts(const BucketProblem &q) {
  Starts s;
  s.ahead = !q.causal;
  s.n = q.causal ? q.buckets : q.buckets / 2;
  const int near = s.n / 2, rest = s.n - near;
  const double ratio = (double)q.far / near;
  for (int b = 0; b < s.n; ++b) {
    if (b <= near) {
      s.start[b] = b;
      continue;
    }
    // the smallest t with t >= near ratio^((b - near) / rest); where that is
    // next to a whole number, the whole number itself decides.  x is off by less
    // than 4e-15 of itself: the exponent's rounding times log(ratio) <= 14, a
    // rounding of ratio and of the product, and pow's.  Distances end at C - 1,
    // so the starts behind are anything above (to look at all of 128 of them up
    // to 2^20 took the host half a millisecond).
    const double x = near * pow(ratio, (double)(b - near) / rest), r = nearbyint(x);
    if (x > q.C + 1.0) {
      for (; b < s.n; ++b) s.start[b] = q.C + 1 > near ? q.C + 1 : near;
      break;
    }
    if (fabs(x - r) > 1e-12 * x)
      s.start[b] = (int)ceil(x);
    else
      s.start[b] = (int)r + !reaches((uint32_t)r, near, q.far, b - near, rest);
  }
  return s;
}

// the last bucket of a direction that starts at or before distance t
__device__ __forceinline__ int bucket_of(const int *start, int n, int t) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (start[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads)
bucket_bias_kernel(const Starts s, const float *__restrict__ table, int buckets, int C,
                   float *__restrict__ relpos) {
  __shared__ int start[kBucketMax];
  __shared__ float value[kBucketMax];
  const int h = blockIdx.y, rows = 2 * C - 1;
  for (int b = threadIdx.x; b < buckets; b += kThreads) {
    if (b < s.n) start[b] = s.start[b];
    value[b] = table[(long long)h * buckets + b];
  }
  __syncthreads();
  for (int k = blockIdx.x * kThreads + threadIdx.x; k < rows; k += gridDim.x * kThreads) {
    const int o = k - (C - 1);
    const int t = o <= 0 ? -o : s.ahead ? o : 0;
    const int b = bucket_of(start, s.n, t) + (o > 0 && s.ahead ? s.n : 0);
    relpos[(long long)h * rows + k] = value[b];
  }
}

// A cluster takes one table; its blocks take runs of offsets, add up the R
// rows of each into shared memory, then each warp the runs of some buckets, and
// the first block joins the blocks' sums in their order.
__global__ void __launch_bounds__(kGradThreads)
bucket_bias_grad_kernel(const Starts s, const float *__restrict__ drelpos, int R, int H,
                        int buckets, int C, int slice, float *__restrict__ dtable) {
  __shared__ float column[kEach * kGradThreads];
  __shared__ float sum[kBucketMax];
  const cg::cluster_group cluster = cg::this_cluster();
  const int h = blockIdx.y, rows = 2 * C - 1, tid = threadIdx.x;
  const int k0 = (int)cluster.block_rank() * slice, k1 = min(rows, k0 + slice);
  const float *src = drelpos + (long long)h * rows + k0 + tid;
  const long long step = (long long)H * rows;
  float total[kEach] = {};
  for (int r0 = 0; r0 < R; r0 += kRun) {
    float x[kEach][kRun];
#pragma unroll
    for (int j = 0; j < kEach; ++j)
#pragma unroll
      for (int r = 0; r < kRun; ++r)
        x[j][r] = k0 + tid + j * kGradThreads < k1 && r0 + r < R
                      ? src[j * kGradThreads + (r0 + r) * step]
                      : 0.f;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      float part = x[j][0];
#pragma unroll
      for (int r = 1; r < kRun; ++r) part += x[j][r];
      total[j] += part;
    }
  }
#pragma unroll
  for (int j = 0; j < kEach; ++j) column[tid + j * kGradThreads] = total[j];
  __syncthreads();
  for (int b = tid / 32; b < buckets; b += kGradThreads / 32) {
    const bool past = b < s.n;
    const int i = past ? b : b - s.n;
    // distances [t0, t1) of this bucket, then its offsets' places [lo, hi)
    const int t0 = s.start[i], t1 = i + 1 < s.n ? min(s.start[i + 1], C) : C;
    int lo = past ? C - t1 : C - 1 + max(t0, 1), hi = past ? C - t0 : C - 1 + t1;
    if (past && i == 0 && !s.ahead) hi = rows;  // offsets above zero count as distance 0
    lo = max(lo, k0);
    hi = min(hi, k1);
    float v = 0.f;
    for (int k = lo + tid % 32; k < hi; k += 32) v += column[k - k0];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (tid % 32 == 0) sum[b] = v;
  }
  cluster.sync();
  if (cluster.block_rank() == 0) {
    const int blocks = (int)cluster.num_blocks();
    for (int b = tid; b < buckets; b += kGradThreads) {
      float x[kMaxCluster];
#pragma unroll
      for (int j = 0; j < kMaxCluster; ++j)
        x[j] = j < blocks ? cluster.map_shared_rank(sum, j)[b] : 0.f;
      float v = x[0];
#pragma unroll
      for (int j = 1; j < kMaxCluster; ++j) v += x[j];
      dtable[(long long)h * buckets + b] = v;
    }
  }
  cluster.sync();  // the others' shared memory is read until here
}

}  // namespace

cudaError_t bucket_bias(const BucketProblem &q, const float *table, float *relpos) {
  const int rows = 2 * q.C - 1;
  // an offset a thread where there are few, four blocks an SM where there are many
  const int most = q.H < 608 ? 608 / q.H : 1, blocks = (rows + kThreads - 1) / kThreads;
  bucket_bias_kernel<<<dim3(blocks < most ? blocks : most, q.H), kThreads, 0, q.stream>>>(
      make_starts(q), table, q.buckets, q.C, relpos);
  return cudaGetLastError();
}

cudaError_t bucket_bias_grad(const BucketProblem &q, const float *drelpos, int R, float *dtable) {
  const int rows = 2 * q.C - 1;
  int blocks = 1;
  while (blocks < kMaxCluster && rows > blocks * kThreads) blocks *= 2;  // 256 offsets a block
  const int slice = (rows + blocks - 1) / blocks;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, q.H);
  cfg.blockDim = dim3(kGradThreads);
  cfg.stream = q.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = blocks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, bucket_bias_grad_kernel, make_starts(q), drelpos, R, q.H,
                            q.buckets, q.C, slice, dtable);
}

}  // namespace flashgau
