// Softmax cross entropy over a vocabulary with fp32 operands: the products
// run in fp32 on the CUDA cores, a piece of tokens at a time.  The piece's
// logits are written once, turned in place into the gradients' weights
// g (p - [v = y]) by one block a row, and read by the two products
//   dX = P W        dW (+)= P^T X
//
// Products: 128 x 128 tiles of 256 threads, 8 x 8 results a thread as packed
// pairs (fma.rn.f32x2), 16-deep slices double-buffered in shared memory, the
// next slice's global loads in flight during the current one's products.
// They are bound by the fp32 units (80 TFLOP/s).  Operands are read as they
// are stored, either index running fastest; what is behind an edge is zero.
#include "flash_gau_internal.h"
#include "sm103_ptx.cuh"

namespace flashgau {
namespace {

using ptx::griddep_wait;

constexpr int TM = 128, TN = 128, TK = 16, PITCH = 132;

// An operand [rows, K] (A's M or B's N rows): element (r, k) at r * ld + k
// (KC), or at k * ld + r.  mask: labels of its k (rows of another matrix);
// a k without a label in [0, V) reads as zero whatever is stored there.
struct Operand {
  const float *p;
  long long ld;
  int rows;
  int vec;  // 16-byte loads: base and ld allow them
  const int *mask;
  int V;
};

template <bool KC>
struct Loader {
  float v[2][4];
  __device__ __forceinline__ void load(const Operand &o, int r0, int k0, int k_end) {
    const int tid = threadIdx.x;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = r0 + (KC ? (tid >> 2) + 64 * i : (tid & 31) * 4);
      const int k = k0 + (KC ? (tid & 3) * 4 : (tid >> 5) + 8 * i);
      const float *p = o.p + (KC ? r * o.ld + k : k * o.ld + r);
      const bool row_ok = KC ? r < o.rows : k < k_end;
      const int left = KC ? k_end - k : o.rows - r;  // along the fast index
      bool live = row_ok && left > 0;
      if (!KC && live && o.mask) {
        const int y = o.mask[k];
        live = y >= 0 && y < o.V;
      }
      if (live && o.vec && left >= 4) {
        const float4 t = *reinterpret_cast<const float4 *>(p);
        v[i][0] = t.x; v[i][1] = t.y; v[i][2] = t.z; v[i][3] = t.w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][j] = live && j < left ? p[j] : 0.f;
      }
    }
  }
  __device__ __forceinline__ void store(float (*s)[PITCH]) const {
    const int tid = threadIdx.x;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (KC) {
#pragma unroll
        for (int j = 0; j < 4; ++j) s[(tid & 3) * 4 + j][(tid >> 2) + 64 * i] = v[i][j];
      } else {
        *reinterpret_cast<float4 *>(&s[(tid >> 5) + 8 * i][(tid & 31) * 4]) =
            make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
      }
    }
  }
};

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ void fma2(uint64_t &c, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(a), "l"(b));
}

struct Out {
  float *p;
  long long ld, split_stride;
  int add, vec;
};

// C[z] (+)= A B^T over the z-th range of K; grid (N tiles, M tiles, splits).
template <bool A_KC, bool B_KC>
__global__ void __launch_bounds__(256, 2)
xent_f32_gemm(int M, int N, int K, int k_split, Operand a, Operand b, Out c) {
  __shared__ __align__(16) float As[2][TK][PITCH], Bs[2][TK][PITCH];
  griddep_wait();
  const int m0 = blockIdx.y * TM, n0 = blockIdx.x * TN;
  const int k_begin = blockIdx.z * k_split, k_end = min(K, k_begin + k_split);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  uint64_t acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0;
  Loader<A_KC> la;
  Loader<B_KC> lb;
  la.load(a, m0, k_begin, k_end);
  lb.load(b, n0, k_begin, k_end);
  la.store(As[0]);
  lb.store(Bs[0]);
  __syncthreads();
  int buf = 0;
  for (int k0 = k_begin; k0 < k_end; k0 += TK, buf ^= 1) {
    const bool more = k0 + TK < k_end;
    if (more) {
      la.load(a, m0, k0 + TK, k_end);
      lb.load(b, n0, k0 + TK, k_end);
    }
#pragma unroll
    for (int k = 0; k < TK; ++k) {
      const float4 a0 = *reinterpret_cast<const float4 *>(&As[buf][k][ty * 4]);
      const float4 a1 = *reinterpret_cast<const float4 *>(&As[buf][k][64 + ty * 4]);
      const ulonglong2 b0 = *reinterpret_cast<const ulonglong2 *>(&Bs[buf][k][tx * 4]);
      const ulonglong2 b1 = *reinterpret_cast<const ulonglong2 *>(&Bs[buf][k][64 + tx * 4]);
      const float av[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint64_t aa = pack2(av[i], av[i]);
        fma2(acc[i][0], aa, b0.x);
        fma2(acc[i][1], aa, b0.y);
        fma2(acc[i][2], aa, b1.x);
        fma2(acc[i][3], aa, b1.y);
      }
    }
    if (more) {
      la.store(As[buf ^ 1]);
      lb.store(Bs[buf ^ 1]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int m = m0 + (i < 4 ? ty * 4 + i : 64 + ty * 4 + i - 4);
    if (m >= M) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int n = n0 + 64 * h + tx * 4;
      const float2 lo = unpack2(acc[i][2 * h]), hi = unpack2(acc[i][2 * h + 1]);
      float v[4] = {lo.x, lo.y, hi.x, hi.y};
      float *p = c.p + blockIdx.z * c.split_stride + m * c.ld + n;
      if (c.vec && n + 4 <= N) {
        float4 t = make_float4(v[0], v[1], v[2], v[3]);
        if (c.add) {
          const float4 o = *reinterpret_cast<const float4 *>(p);
          t.x += o.x; t.y += o.y; t.z += o.z; t.w += o.w;
        }
        *reinterpret_cast<float4 *>(p) = t;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n + j < N) p[j] = c.add ? p[j] + v[j] : v[j];
      }
    }
  }
}

__device__ __forceinline__ float block_max(float v, float *buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  v = buf[0];
  for (int k = 1; k < 8; ++k) v = fmaxf(v, buf[k]);
  __syncthreads();
  return v;
}
__device__ __forceinline__ float block_sum(float v, float *buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  for (int k = 0; k < 8; ++k) v += buf[k];
  __syncthreads();
  return v;
}

// One block a row of logits l: the loss, and with gradients P = g (p - [v =
// y]) in place, the label's entry as minus the others' sum.
__global__ void __launch_bounds__(256)
xent_f32_rows(float *__restrict__ P, long long ld, int V, const int *__restrict__ labels,
              const float *__restrict__ factor, float *__restrict__ loss, float *__restrict__ lse,
              int grad) {
  __shared__ float buf[8];
  griddep_wait();
  const int row = blockIdx.x, y = labels[row];
  float *l = P + row * ld;
  if (y < 0 || y >= V) {
    if (threadIdx.x == 0) {
      loss[row] = 0.f;
      if (lse) lse[row] = 0.f;
    }
    if (grad)
      for (int c = threadIdx.x; c < V; c += 256) l[c] = 0.f;
    return;
  }
  float top = -INFINITY;
  for (int c = threadIdx.x; c < V; c += 256) top = fmaxf(top, l[c]);
  top = block_max(top, buf);
  const float t = l[y];
  float sum = 0.f;
  for (int c = threadIdx.x; c < V; c += 256)
    if (c != y) sum += expf(l[c] - top);
  sum = block_sum(sum, buf);
  // the label's term apart: exact where it is nearly everything
  const float own = expf(t - top);
  const float z = own + sum;
  if (threadIdx.x == 0) {
    const float v = t == top ? log1pf(sum) : logf(z) + (top - t);
    loss[row] = v;
    if (lse) lse[row] = t + v;
  }
  if (!grad) return;
  const float f = *factor / z;
  for (int c = threadIdx.x; c < V; c += 256) l[c] = c == y ? -sum * f : expf(l[c] - top) * f;
}

// the factor g of the gradients from the count of labels
__global__ void __launch_bounds__(1024)
xent_f32_factor(const int *__restrict__ labels, long long N, int V, int mean, float scale,
                float *__restrict__ factor) {
  __shared__ int buf[32];
  griddep_wait();
  int n = 0;
  for (long long i = threadIdx.x; i < N; i += 1024) n += labels[i] >= 0 && labels[i] < V;
  n = __reduce_add_sync(0xffffffffu, n);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = n;
  __syncthreads();
  if (threadIdx.x == 0) {
    n = 0;
    for (int k = 0; k < 32; ++k) n += buf[k];
    *factor = mean ? scale / (float)(n > 0 ? n : 1) : scale;
  }
}

__global__ void __launch_bounds__(256)
xent_f32_join(const float *__restrict__ part, long long n, int splits, float *__restrict__ out) {
  griddep_wait();
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < n; i += gridDim.x * 256LL) {
    float s = part[i];
    for (int k = 1; k < splits; ++k) s += part[k * n + i];
    out[i] = s;
  }
}

bool vec4(const float *p, long long ld) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 4 == 0;
}
Operand operand(const float *p, long long ld, int rows) { return {p, ld, rows, vec4(p, ld), nullptr, 0}; }

template <bool A_KC, bool B_KC>
cudaError_t gemm(int M, int N, int K, int splits, const Operand &a, const Operand &b, Out c,
                 cudaStream_t stream) {
  int k_split = (K + splits - 1) / splits;
  k_split = (k_split + TK - 1) / TK * TK;
  c.vec = vec4(c.p, c.ld) && c.split_stride % 4 == 0;
  const dim3 grid((N + TN - 1) / TN, (M + TM - 1) / TM, splits);
  return launch_pdl(xent_f32_gemm<A_KC, B_KC>, grid, dim3(256), 0, stream, M, N, K, k_split, a, b, c);
}

}  // namespace

// Splits of dX's sum over the words: enough thread blocks for two a SM, of at
// least 512 words each.
int xent_f32_dx_splits(int rows, int d, int V) {
  const int tiles = ((rows + TM - 1) / TM) * ((d + TN - 1) / TN);
  int s = (2 * kXentPlanSms + tiles - 1) / tiles;
  if (s > V / 512) s = V / 512;
  return s < 1 ? 1 : (s > 16 ? 16 : s);
}

cudaError_t xent_f32(const XentProblem &q) {
  const XentLayout &L = q.L;
  cudaError_t err = cudaMemsetAsync(L.status, 0, sizeof(int), q.stream);
  if (err != cudaSuccess) return err;
  const bool grad = q.dX || q.dW;
  const float *X = static_cast<const float *>(q.X), *W = static_cast<const float *>(q.W);
  float *P = static_cast<float *>(L.E);
  err = launch_pdl(xent_f32_factor, dim3(1), dim3(1024), 0, q.stream, q.labels, q.N, q.V, q.mean,
                   q.scale, L.factor);
  for (long long n0 = 0; err == cudaSuccess && n0 < q.N; n0 += L.piece) {
    const int rows = (int)(q.N - n0 < L.piece ? q.N - n0 : L.piece);
    const float *x = X + n0 * q.d;
    const int *labels = q.labels + n0;
    err = gemm<true, true>(rows, q.V, q.d, 1, operand(x, q.d, rows), operand(W, q.d, q.V),
                           Out{P, L.ldE, 0, 0, 0}, q.stream);
    if (err != cudaSuccess) return err;
    err = launch_pdl(xent_f32_rows, dim3(rows), dim3(256), 0, q.stream, P, L.ldE, q.V, labels,
                     L.factor, q.loss + n0, q.lse ? q.lse + n0 : nullptr, grad ? 1 : 0);
    if (err != cudaSuccess) return err;
    if (q.dX) {
      float *out = static_cast<float *>(q.dX) + n0 * q.d;
      const int splits = xent_f32_dx_splits(rows, q.d, q.V);
      const long long n = (long long)rows * q.d;
      err = gemm<true, false>(rows, q.d, q.V, splits, operand(P, L.ldE, rows), operand(W, q.d, q.d),
                              Out{splits > 1 ? L.dx_part : out, q.d, n, 0, 0}, q.stream);
      if (err == cudaSuccess && splits > 1) {
        const long long blocks = (n + 255) / 256;
        err = launch_pdl(xent_f32_join, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256),
                         0, q.stream, L.dx_part, n, splits, out);
      }
      if (err != cudaSuccess) return err;
    }
    if (q.dW) {
      Operand b = operand(x, q.d, q.d);
      b.mask = labels;
      b.V = q.V;
      err = gemm<false, false>(q.V, q.d, rows, 1, operand(P, L.ldE, q.V), b,
                               Out{static_cast<float *>(q.dW), q.d, 0, n0 > 0, 0}, q.stream);
      if (err != cudaSuccess) return err;
    }
  }
  if (err != cudaSuccess) return err;
  return xent_total(q);
}

}  // namespace flashgau
