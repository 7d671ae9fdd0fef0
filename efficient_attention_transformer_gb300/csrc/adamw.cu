// One AdamW step over a list of tensors, and the values of 8-bit moments.
//
//   g' = grad_scale g
//   m' = beta1 m + (1 - beta1) g'         v' = beta2 v + (1 - beta2) g' g'
//   p' = (1 - lr wd) p - lr / (1 - beta1^t) m' / (sqrt(v') / sqrt(1 - beta2^t) + eps)
//
// 8-bit moments: every 256 consecutive elements of a tensor (its last block
// may be short) share two fp32 scales.  m is held as s_m c |c|, c in -127 ..
// 127, and sqrt(v) as s_v c^2, c in 0 .. 255: squaring the code makes the
// steps fine near zero (the smallest nonzero value is 2^-14 of the block's
// largest |m|, 2^-16 of its largest sqrt(v)) while one step at the top stays
// under 1.6% (0.8%).  A nonzero v keeps a code of at least 1, so that the
// update's denominator does not lose it.  A block whose largest value is
// below 2^-60 is held as zeros, and one with a value that is not finite
// decodes to values that are not finite.  The update itself uses the fresh
// fp32 moments.  Moments and codes take one correctly rounded fp32
// operation at a time (no contraction), so that the codes next to a rounding
// border do not depend on the compiler.
//
// The work is memory traffic: 28 bytes a parameter with fp32 moments (p, m, v
// in and out, g in), 16 with 8-bit ones, 2 more for a bf16 copy.  The list
// goes into the kernel's parameters, so that a step is one launch (per 384
// tensors), needs no workspace and can be captured; a block takes 2048
// elements of one tensor, a warp 256 of them as two runs of 128, four
// consecutive elements a lane (16-byte accesses).
#include <cuda_bf16.h>
#include <math.h>

#include "flash_gau_internal.h"
#include "sm103_ptx.cuh"

namespace flashgau {
namespace {

constexpr int kThreads = 256;
constexpr int kBlock = 256;                    // elements that share a scale
constexpr int kChunk = kThreads / 32 * kBlock;  // elements of a thread block

struct Entry {
  float *p;
  __nv_bfloat16 *copy;
  const void *g;
  void *m, *v;
  float *m_scale, *v_scale;
  long long n;
  float decay;    // 1 - lr * weight_decay
  int first;      // first thread block of the tensor in this launch
  int g_bf16, vec;  // vec: every pointer aligned for four elements at a time
};

template <int CAP>
struct List {
  Entry e[CAP];
  int count;
  float step_size, beta1, omb1, beta2, omb2, inv_c2, eps;
  const float *grad_scale;
};

// the tensor of this thread block: the last entry whose first block is not
// behind it
template <int CAP>
__device__ __forceinline__ int find(const List<CAP> &l, int b) {
  int lo = 0, hi = l.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (l.e[mid].first <= b) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Four elements at i of an fp32 array, of which `n` are inside.
__device__ __forceinline__ void load4(const float *a, long long i, int n, int vec, float (&x)[4]) {
  if (vec && n == 4) {
    const float4 t = *reinterpret_cast<const float4 *>(a + i);
    x[0] = t.x; x[1] = t.y; x[2] = t.z; x[3] = t.w;
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] = q < n ? a[i + q] : 0.f;
  }
}
__device__ __forceinline__ void load4(const __nv_bfloat16 *a, long long i, int n, int vec,
                                      float (&x)[4]) {
  if (vec && n == 4) {
    const uint2 t = *reinterpret_cast<const uint2 *>(a + i);
    const float2 u = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&t.x));
    const float2 w = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&t.y));
    x[0] = u.x; x[1] = u.y; x[2] = w.x; x[3] = w.y;
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] = q < n ? __bfloat162float(a[i + q]) : 0.f;
  }
}
__device__ __forceinline__ void store4(float *a, long long i, int n, int vec, const float (&x)[4]) {
  if (vec && n == 4) {
    *reinterpret_cast<float4 *>(a + i) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q < n) a[i + q] = x[q];
  }
}
__device__ __forceinline__ void store4(__nv_bfloat16 *a, long long i, int n, int vec,
                                       const float (&x)[4]) {
  if (vec && n == 4) {
    const __nv_bfloat162 u = __floats2bfloat162_rn(x[0], x[1]), w = __floats2bfloat162_rn(x[2], x[3]);
    uint2 t;
    t.x = *reinterpret_cast<const uint32_t *>(&u);
    t.y = *reinterpret_cast<const uint32_t *>(&w);
    *reinterpret_cast<uint2 *>(a + i) = t;
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q < n) a[i + q] = __float2bfloat16_rn(x[q]);
  }
}
// Four codes as one word (byte q: element q).
__device__ __forceinline__ uint32_t load_codes(const void *a, long long i, int n, int vec) {
  const uint8_t *c = static_cast<const uint8_t *>(a) + i;
  if (vec && n == 4) return *reinterpret_cast<const uint32_t *>(c);
  uint32_t w = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (q < n) w |= (uint32_t)c[q] << (8 * q);
  return w;
}
__device__ __forceinline__ void store_codes(void *a, long long i, int n, int vec, uint32_t w) {
  uint8_t *c = static_cast<uint8_t *>(a) + i;
  if (vec && n == 4) {
    *reinterpret_cast<uint32_t *>(c) = w;
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q < n) c[q] = (uint8_t)(w >> (8 * q));
  }
}

__device__ __forceinline__ float decode_m(uint32_t w, int q, float scale) {
  const int c = (int8_t)(w >> (8 * q));
  return __fmul_rn((float)(c * abs(c)), scale);
}
__device__ __forceinline__ float decode_root(uint32_t w, int q, float scale) {
  const int c = (int)((w >> (8 * q)) & 255u);
  return __fmul_rn((float)(c * c), scale);
}

// A block's scale and its inverse from the largest magnitude (as bits: a
// value that is not finite is larger than any finite one).
template <int TOP>
__device__ __forceinline__ void block_scale(uint32_t bits, float *scale, float *inv) {
  const float big = __uint_as_float(bits);
  const bool live = !(big < 0x1p-60f);
  *scale = live ? __fmul_rn(big, 1.0f / (TOP * TOP)) : 0.f;
  *inv = live ? __fmul_rn(__frcp_rn(big), (float)(TOP * TOP)) : 0.f;
}

template <int BITS, int CAP>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ List<CAP> l) {
  ptx::griddep_wait();
  const Entry &e = l.e[find(l, blockIdx.x)];
  const int lane = threadIdx.x & 31;
  const long long blk = (long long)(blockIdx.x - e.first) * (kChunk / kBlock) + (threadIdx.x >> 5);
  const long long i0 = blk * kBlock + 4 * lane;
  if (blk * kBlock >= e.n) return;
  const float gs = l.grad_scale ? *l.grad_scale : 1.f;
  int n[2];
  float p[2][4], g[2][4], m[2][4], v[2][4];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const long long i = i0 + 128 * j, left = e.n - i;
    n[j] = left >= 4 ? 4 : (left > 0 ? (int)left : 0);
    load4(e.p, i, n[j], e.vec, p[j]);
    if (e.g_bf16) load4(static_cast<const __nv_bfloat16 *>(e.g), i, n[j], e.vec, g[j]);
    else load4(static_cast<const float *>(e.g), i, n[j], e.vec, g[j]);
    if constexpr (BITS == 32) {
      load4(static_cast<const float *>(e.m), i, n[j], e.vec, m[j]);
      load4(static_cast<const float *>(e.v), i, n[j], e.vec, v[j]);
    }
  }
  if constexpr (BITS == 8) {
    const float ms = e.m_scale[blk], vs = e.v_scale[blk];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t mc = load_codes(e.m, i0 + 128 * j, n[j], e.vec);
      const uint32_t vc = load_codes(e.v, i0 + 128 * j, n[j], e.vec);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        m[j][q] = decode_m(mc, q, ms);
        const float r = decode_root(vc, q, vs);
        v[j][q] = __fmul_rn(r, r);
      }
    }
  }
  float root[2][4];
  uint32_t mmax = 0, rmax = 0;
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float gg = l.grad_scale ? __fmul_rn(g[j][q], gs) : g[j][q];
      m[j][q] = __fadd_rn(__fmul_rn(m[j][q], l.beta1), __fmul_rn(gg, l.omb1));
      v[j][q] = __fadd_rn(__fmul_rn(v[j][q], l.beta2), __fmul_rn(__fmul_rn(gg, l.omb2), gg));
      root[j][q] = __fsqrt_rn(v[j][q]);
      p[j][q] = p[j][q] * e.decay - l.step_size * m[j][q] / fmaf(root[j][q], l.inv_c2, l.eps);
      if (BITS == 8) {
        mmax = max(mmax, __float_as_uint(m[j][q]) & 0x7fffffffu);
        rmax = max(rmax, __float_as_uint(root[j][q]) & 0x7fffffffu);
      }
    }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const long long i = i0 + 128 * j;
    store4(e.p, i, n[j], e.vec, p[j]);
    if (e.copy) store4(e.copy, i, n[j], e.vec, p[j]);
    if constexpr (BITS == 32) {
      store4(static_cast<float *>(e.m), i, n[j], e.vec, m[j]);
      store4(static_cast<float *>(e.v), i, n[j], e.vec, v[j]);
    }
  }
  if constexpr (BITS == 8) {
    // elements behind the tensor's end are zeros throughout
    mmax = __reduce_max_sync(0xffffffffu, mmax);
    rmax = __reduce_max_sync(0xffffffffu, rmax);
    float ms, mi, vs, vi;
    block_scale<127>(mmax, &ms, &mi);
    block_scale<255>(rmax, &vs, &vi);
    if (lane == 0) {
      e.m_scale[blk] = ms;
      e.v_scale[blk] = vs;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t mw = 0, vw = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        int c = min(__float2int_rn(__fsqrt_rn(__fmul_rn(fabsf(m[j][q]), mi))), 127);
        if (m[j][q] < 0.f) c = -c;
        mw |= (uint32_t)(c & 255) << (8 * q);
        int r = min(__float2int_rn(__fsqrt_rn(__fmul_rn(root[j][q], vi))), 255);
        if (r == 0 && root[j][q] > 0.f && vs != 0.f) r = 1;
        vw |= (uint32_t)r << (8 * q);
      }
      store_codes(e.m, i0 + 128 * j, n[j], e.vec, mw);
      store_codes(e.v, i0 + 128 * j, n[j], e.vec, vw);
    }
  }
}

// m and v of 8-bit moments as fp32: `p` holds m's values, `copy` v's.
template <int CAP>
__global__ void __launch_bounds__(kThreads) moments_kernel(const __grid_constant__ List<CAP> l) {
  ptx::griddep_wait();
  const Entry &e = l.e[find(l, blockIdx.x)];
  const int lane = threadIdx.x & 31;
  const long long blk = (long long)(blockIdx.x - e.first) * (kChunk / kBlock) + (threadIdx.x >> 5);
  if (blk * kBlock >= e.n) return;
  const float ms = e.m_scale[blk], vs = e.v_scale[blk];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const long long i = blk * kBlock + 4 * lane + 128 * j, left = e.n - i;
    const int n = left >= 4 ? 4 : (left > 0 ? (int)left : 0);
    const uint32_t mc = load_codes(e.m, i, n, e.vec), vc = load_codes(e.v, i, n, e.vec);
    float m[4], v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      m[q] = decode_m(mc, q, ms);
      const float r = decode_root(vc, q, vs);
      v[q] = __fmul_rn(r, r);
    }
    store4(e.p, i, n, e.vec, m);
    store4(reinterpret_cast<float *>(e.copy), i, n, e.vec, v);
  }
}

bool aligned(const void *p, unsigned bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

template <int CAP, typename Kernel, typename Fill>
cudaError_t run(Kernel kernel, const AdamwProblem &q, Fill fill) {
  List<CAP> l;
  l.step_size = (float)(q.lr / (1.0 - pow(q.beta1, (double)q.step)));
  l.beta1 = (float)q.beta1;
  l.omb1 = (float)(1.0 - q.beta1);
  l.beta2 = (float)q.beta2;
  l.omb2 = (float)(1.0 - q.beta2);
  l.inv_c2 = (float)(1.0 / sqrt(1.0 - pow(q.beta2, (double)q.step)));
  l.eps = (float)q.eps;
  l.grad_scale = q.grad_scale;
  for (int k = 0; k < q.n_tensors;) {
    l.count = 0;
    long long blocks = 0;
    // as many tensors as fit the list and the grid
    for (; k < q.n_tensors && l.count < CAP; ++k) {
      const flash_gau_adamw_tensor &t = q.tensors[k];
      if (t.n == 0) continue;
      const long long b = (t.n + kChunk - 1) / kChunk;
      if (l.count && blocks + b > 0x7fffffffLL) break;
      Entry &e = l.e[l.count++];
      fill(k, e);
      e.n = t.n;
      e.first = (int)blocks;
      blocks += b;
    }
    if (!l.count) break;
    const cudaError_t err =
        launch_pdl(kernel, dim3((unsigned)blocks), dim3(kThreads), 0, q.stream, l);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

// short lists keep the launch's parameters small
constexpr int kSmall = 16, kLarge = 384;

}  // namespace

cudaError_t adamw_step(const AdamwProblem &q) {
  auto fill = [&](int k, Entry &e) {
    const flash_gau_adamw_tensor &t = q.tensors[k];
    e.p = t.p;
    e.copy = static_cast<__nv_bfloat16 *>(t.copy);
    e.g = t.g;
    e.m = t.m;
    e.v = t.v;
    e.m_scale = t.m_scale;
    e.v_scale = t.v_scale;
    e.decay = (float)(1.0 - q.lr * (double)t.weight_decay);
    e.g_bf16 = t.g_dtype == FLASH_GAU_BF16;
    const unsigned state = q.state_bits == 8 ? 4 : 16;
    e.vec = aligned(t.p, 16) && aligned(t.copy, 8) && aligned(t.g, e.g_bf16 ? 8 : 16) &&
            aligned(t.m, state) && aligned(t.v, state);
  };
  if (q.n_tensors <= kSmall)
    return q.state_bits == 8 ? run<kSmall>(adamw_kernel<8, kSmall>, q, fill)
                             : run<kSmall>(adamw_kernel<32, kSmall>, q, fill);
  return q.state_bits == 8 ? run<kLarge>(adamw_kernel<8, kLarge>, q, fill)
                           : run<kLarge>(adamw_kernel<32, kLarge>, q, fill);
}

cudaError_t adamw_moments(const AdamwProblem &q, float *const *m_out, float *const *v_out) {
  auto fill = [&](int k, Entry &e) {
    const flash_gau_adamw_tensor &t = q.tensors[k];
    e = {};
    e.p = m_out[k];
    e.copy = reinterpret_cast<__nv_bfloat16 *>(v_out[k]);
    e.m = t.m;
    e.v = t.v;
    e.m_scale = t.m_scale;
    e.v_scale = t.v_scale;
    e.vec = aligned(e.p, 16) && aligned(e.copy, 16) && aligned(t.m, 4) && aligned(t.v, 4);
  };
  return q.n_tensors <= kSmall ? run<kSmall>(moments_kernel<kSmall>, q, fill)
                               : run<kLarge>(moments_kernel<kLarge>, q, fill);
}

}  // namespace flashgau
