// The residual stream around a block: the block's output, normalised, gated
// and scaled, is added to the stream, and the next block's pre-norm is taken
// in the same pass,
//   r = h + scale * gate * post(y)        n = norm(r)
// and its gradients.  post and norm are the flash_block norms:
//   LayerNorm  (x - mean) / sqrt(var + eps) * g + b     (biased variance)
//   ScaleNorm  g x / max(|x|, eps)                      (g a single scalar)
//
// Backward, with u the normalised row without its parameters, i = 1 / spread
// and w = g * (gradient of the norm's output):
//   LayerNorm  dx = i (w - mean(w) - u mean(w u))
//   ScaleNorm  dx = i (w - u sum(w u)), the second term only where |x| > eps
//   dh = dr + dx_norm(dn; r)      dgate = dh * post(y) * scale
//   dy = dx_post(dh * scale * gate; y)
// and the column sums over the rows for the parameters.
//
// Both directions only move rows (at d = 768, bf16: 5 rows in and out
// forward with a gate, 8 backward), so the aim is to read each value once
// from memory with many rows in flight.
//
// Forward, one warp a row in registers: 256 columns a step of the warp (16
// bytes a lane), no block-wide step at all.  16384 x 768 bf16 with every
// option takes 26 us, 4.8 TB/s (a persistent form with the next row's loads
// under way 23 for 23 there and 10 for 8.5 us at 4096 rows, by itself).  Rows
// wider than 2048 columns, or not on 16-byte boundaries, take a form with
// eight columns a thread and a block a row.
//
// Backward, rows of up to 2048 columns on 16-byte boundaries: one to four
// warps a row, see residual_norm_grad_rows_kernel (16384 x 768 bf16 with every
// option 44 us with the join of the column sums, 63 by tiles).  Others, a
// tile of rows (about 44 KB, four blocks an SM) is brought into shared memory by
// asynchronous copies.  First one warp a row takes the row's sums;
// means come first and squares around them second (no difference of large
// squares), and the sums that dx needs ride along, three passes over shared
// memory in all.  Then the threads turn by 90 degrees: each keeps four
// columns for the whole launch, forms the outputs of the tile's rows from
// the rows' sums, and adds up the parameters' gradients in registers.
#include <cuda_bf16.h>

#include <atomic>
#include <type_traits>

#include "flash_gau_internal.h"
#include "packed_f32.cuh"
#include "sm103_ptx.cuh"

namespace flashgau {
namespace {

constexpr unsigned kAll = 0xffffffffu;

struct Args {
  const void *h, *y, *gate;  // backward: h is the stored r; y may be null there
                             // where nothing needs its values
  const void *dr, *dn;
  void *r, *n;               // forward outputs
  void *dh, *dy, *dgate;     // backward outputs
  const float *norm_g, *norm_b, *post_g, *post_b, *scale;
  float *part;               // backward: [parts][kSums][d] column sums
  float *scalar_part;        // backward: [2][blocks][kMaxWarps], ScaleNorm's g
  long long M;
  int d, norm, post;
  float eps;
  int rows, subsets;         // backward: rows of a tile, threads that share a column
};

// the column sums, in the workspace's order
enum { kNormG = 0, kNormB = 1, kPostG = 2, kPostB = 3, kScale = 4, kSums = 5 };
constexpr int kMaxWarps = 16;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack_bf16(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// 1 / spread of a row from its sum of squares around the mean (LayerNorm) or
// around zero (ScaleNorm).  The hardware's reciprocal square root (off by at
// most 2 units in the last place): exact division and root cost a row more
// instructions than its sums do.
__device__ __forceinline__ float inv_layer(float m2, float inv_d, float eps) {
  return rsqrtf(fmaf(m2, inv_d, eps));
}
// at most inv_eps = 1 / eps, and not a number where m2 is not (a minimum alone
// would leave such a row's other values finite)
__device__ __forceinline__ float inv_scale(float m2, float inv_eps) {
  const float r = rsqrtf(m2);
  return r > inv_eps ? inv_eps : r;
}
__device__ __forceinline__ float inv_spread(float m2, int kind, float inv_d, float eps) {
  return kind == FLASH_GAU_NORM_LAYER ? inv_layer(m2, inv_d, eps) : inv_scale(m2, 1.0f / eps);
}
// ScaleNorm: whether |x| > eps, where the gradient has its second term
__device__ __forceinline__ bool longer(float m2, float eps) { return m2 > eps * eps; }

// ---------------------------------------------------------------- forward --
// Eight columns of a row a lane: chunk k covers columns 256 k .. 256 k + 255,
// as 8 consecutive bf16 or two runs of 4 fp32.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 w;
  static __device__ int column(int k, int lane, int q) { return 256 * k + 8 * lane + q; }
  __device__ void load(const __nv_bfloat16 *row, int k, int lane, int d) {
    const int c = column(k, lane, 0);
    w = c < d ? *reinterpret_cast<const uint4 *>(row + c) : make_uint4(0, 0, 0, 0);
  }
  __device__ float get(int q) const {
    const uint32_t v = q < 2 ? w.x : q < 4 ? w.y : q < 6 ? w.z : w.w;
    const float2 f = unpack_bf16(v);
    return (q & 1) ? f.y : f.x;
  }
  static __device__ void store(__nv_bfloat16 *row, int k, int lane, int d, const float (&x)[8]) {
    const int c = column(k, lane, 0);
    if (c < d)
      *reinterpret_cast<uint4 *>(row + c) =
          make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                     pack_bf16(x[6], x[7]));
  }
};
template <>
struct Eight<float> {
  float4 a, b;
  static __device__ int column(int k, int lane, int q) {
    return 256 * k + 4 * lane + (q & 3) + (q < 4 ? 0 : 128);
  }
  __device__ void load(const float *row, int k, int lane, int d) {
    const int c0 = column(k, lane, 0), c1 = column(k, lane, 4);
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    a = c0 < d ? *reinterpret_cast<const float4 *>(row + c0) : zero;
    b = c1 < d ? *reinterpret_cast<const float4 *>(row + c1) : zero;
  }
  __device__ float get(int q) const {
    const float4 &v = q < 4 ? a : b;
    return (q & 3) == 0 ? v.x : (q & 3) == 1 ? v.y : (q & 3) == 2 ? v.z : v.w;
  }
  static __device__ void store(float *row, int k, int lane, int d, const float (&x)[8]) {
    const int c0 = column(k, lane, 0), c1 = column(k, lane, 4);
    if (c0 < d) *reinterpret_cast<float4 *>(row + c0) = make_float4(x[0], x[1], x[2], x[3]);
    if (c1 < d) *reinterpret_cast<float4 *>(row + c1) = make_float4(x[4], x[5], x[6], x[7]);
  }
};

// a parameter's values in a lane's columns of chunk k; columns behind the row
// read as zero, so that their results are never stored anyway
template <typename T>
__device__ __forceinline__ void load_param(const float *p, int k, int lane, int d, float (&x)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = Eight<T>::column(k, lane, 4 * h);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < d) v = __ldg(reinterpret_cast<const float4 *>(p + c));
    x[4 * h] = v.x; x[4 * h + 1] = v.y; x[4 * h + 2] = v.z; x[4 * h + 3] = v.w;
  }
}

// (mean, 1 / spread) of a row of NC chunks in registers
template <typename T, int NC, typename Get>
__device__ __forceinline__ float2 row_stat(Get get, int kind, int lane, int d, float eps) {
  float mean = 0.f;
  if (kind == FLASH_GAU_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int q = 0; q < 8; ++q) s += get(k, q);  // zeros behind the row
    mean = warp_sum(s) / (float)d;
  }
  float m2 = 0.f;
#pragma unroll
  for (int k = 0; k < NC; ++k)
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float c = Eight<T>::column(k, lane, q) < d ? get(k, q) - mean : 0.f;
      m2 = fmaf(c, c, m2);
    }
  return make_float2(mean, inv_spread(warp_sum(m2), kind, 1.0f / (float)d, eps));
}

template <typename T, int NC>
__global__ void __launch_bounds__(128) residual_norm_kernel(const Args a) {
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31, d = a.d;
  const long long row = blockIdx.x * (long long)(blockDim.x >> 5) + (threadIdx.x >> 5);
  if (row >= a.M) return;
  Eight<T> h[NC], y[NC], gt[NC];
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    h[k].load(static_cast<const T *>(a.h) + row * d, k, lane, d);
    if (a.y) y[k].load(static_cast<const T *>(a.y) + row * d, k, lane, d);
    if (a.gate) gt[k].load(static_cast<const T *>(a.gate) + row * d, k, lane, d);
  }
  float r[NC][8];
  if (a.y) {
    const bool layer = a.post == FLASH_GAU_NORM_LAYER;
    float2 st = make_float2(0.f, 1.f);
    if (a.post)
      st = row_stat<T, NC>([&](int k, int q) { return y[k].get(q); }, a.post, lane, d, a.eps);
    if (a.post == FLASH_GAU_NORM_SCALE) st.y *= __ldg(a.post_g);
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      float g[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) r[k][q] = (y[k].get(q) - st.x) * st.y;
      if (layer) {
        load_param<T>(a.post_g, k, lane, d, g);
#pragma unroll
        for (int q = 0; q < 8; ++q) r[k][q] *= g[q];
        if (a.post_b) {
          load_param<T>(a.post_b, k, lane, d, g);
#pragma unroll
          for (int q = 0; q < 8; ++q) r[k][q] += g[q];
        }
      }
      if (a.gate) {
#pragma unroll
        for (int q = 0; q < 8; ++q) r[k][q] *= gt[k].get(q);
      }
      if (a.scale) {
        load_param<T>(a.scale, k, lane, d, g);
#pragma unroll
        for (int q = 0; q < 8; ++q) r[k][q] *= g[q];
      }
#pragma unroll
      for (int q = 0; q < 8; ++q)
        r[k][q] = Eight<T>::column(k, lane, q) < d ? r[k][q] + h[k].get(q) : 0.f;
    }
  } else {
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int q = 0; q < 8; ++q) r[k][q] = h[k].get(q);
  }
  if (a.r) {
#pragma unroll
    for (int k = 0; k < NC; ++k) Eight<T>::store(static_cast<T *>(a.r) + row * d, k, lane, d, r[k]);
  }
  if (!a.norm) return;
  float2 st = row_stat<T, NC>([&](int k, int q) { return r[k][q]; }, a.norm, lane, d, a.eps);
  const bool layer = a.norm == FLASH_GAU_NORM_LAYER;
  if (!layer) st.y *= __ldg(a.norm_g);
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    float g[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) r[k][q] = (r[k][q] - st.x) * st.y;
    if (layer) {
      load_param<T>(a.norm_g, k, lane, d, g);
#pragma unroll
      for (int q = 0; q < 8; ++q) r[k][q] *= g[q];
      if (a.norm_b) {
        load_param<T>(a.norm_b, k, lane, d, g);
#pragma unroll
        for (int q = 0; q < 8; ++q) r[k][q] += g[q];
      }
    }
    Eight<T>::store(static_cast<T *>(a.n) + row * d, k, lane, d, r[k]);
  }
}

// Any width and alignment: a thread has eight columns of a row in registers,
// consecutive ones (VEC: rows and arrays on 16-byte boundaries; two runs of
// four fp32) or one from every `threads`; up to 256 columns are a warp's, and
// four rows a block, wider ones a block's (16384 x 767 bf16 66 us, 3000 x 4096
// 54 in either type).  A warp a row that read the row again for each sum took
// 120 us at 16384 x 767 bf16, and 268 at 3000 x 4096 bf16.
template <typename T, bool VEC>
__global__ void __launch_bounds__(1024) residual_norm_any_kernel(const Args a) {
  __shared__ float shared_sums[2][32];
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = a.d;
  const bool alone = d <= 256;  // a warp a row
  const int t = alone ? lane : threadIdx.x, threads = alone ? 32 : blockDim.x;
  const int at_once = alone ? blockDim.x / 32 : 1;
  auto column = [&](int q) {
    if (!VEC) return t + threads * q;
    return sizeof(T) == 2 ? 8 * t + q : 4 * t + (q & 3) + (q < 4 ? 0 : 4 * threads);
  };
  auto load = [&](const auto *row, float (&x)[8]) {
    using E = std::remove_const_t<std::remove_pointer_t<decltype(row)>>;
    if constexpr (VEC && sizeof(E) == 2) {
      const uint4 w = t * 8 < d ? *reinterpret_cast<const uint4 *>(row + 8 * t) : make_uint4(0, 0, 0, 0);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 f = unpack_bf16(u[q]);
        x[2 * q] = f.x;
        x[2 * q + 1] = f.y;
      }
    } else if constexpr (VEC) {
#pragma unroll
      for (int q = 0; q < 8; q += 4) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (column(q) < d) v = *reinterpret_cast<const float4 *>(row + column(q));
        x[q] = v.x; x[q + 1] = v.y; x[q + 2] = v.z; x[q + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] = column(q) < d ? to_f(row[column(q)]) : 0.f;
    }
  };
  auto store = [&](T *row, const float (&x)[8]) {
    if constexpr (VEC && sizeof(T) == 2) {
      if (8 * t < d)
        *reinterpret_cast<uint4 *>(row + 8 * t) = make_uint4(
            pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    } else if constexpr (VEC) {
#pragma unroll
      for (int q = 0; q < 8; q += 4)
        if (column(q) < d)
          *reinterpret_cast<float4 *>(row + column(q)) =
              make_float4(x[q], x[q + 1], x[q + 2], x[q + 3]);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (column(q) < d) row[column(q)] = (T)x[q];
    }
  };
  int flip = 0;
  auto row_sum = [&](float v) {
    v = warp_sum(v);
    if (alone) return v;
    if (lane == 0) shared_sums[flip][warp] = v;
    __syncthreads();
    v = warp_sum(lane < threads / 32 ? shared_sums[flip][lane] : 0.f);
    flip ^= 1;  // written again only after the next barrier: everyone has read it
    return v;
  };
  const float inv_d = 1.0f / (float)d;
  // x becomes its normalised row with parameters, zeros behind it
  auto normalise = [&](float (&x)[8], int kind, const float *g, const float *b) {
    const bool layer = kind == FLASH_GAU_NORM_LAYER;
    float mean = 0.f, m2 = 0.f;
    if (layer) {
      float s = 0.f;
#pragma unroll
      for (int q = 0; q < 8; ++q) s += x[q];
      mean = row_sum(s) / (float)d;
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      x[q] = column(q) < d ? x[q] - mean : 0.f;
      m2 = fmaf(x[q], x[q], m2);
    }
    const float inv = inv_spread(row_sum(m2), kind, inv_d, a.eps) * (layer ? 1.f : __ldg(g));
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] *= inv;
    if (!layer) return;
    float w[8];
    load(g, w);
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] *= w[q];
    if (!b) return;
    load(b, w);
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] += w[q];
  };
  for (long long row = blockIdx.x * (long long)at_once + (alone ? warp : 0); row < a.M;
       row += gridDim.x * (long long)at_once) {
    const long long off = row * d;
    float h[8], r[8], w[8];
    load(static_cast<const T *>(a.h) + off, h);
    if (a.y) {
      load(static_cast<const T *>(a.y) + off, r);
      if (a.gate) load(static_cast<const T *>(a.gate) + off, w);
      if (a.post) normalise(r, a.post, a.post_g, a.post_b);
      if (a.gate) {
#pragma unroll
        for (int q = 0; q < 8; ++q) r[q] *= w[q];
      }
      if (a.scale) {
        load(a.scale, w);
#pragma unroll
        for (int q = 0; q < 8; ++q) r[q] *= w[q];
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) r[q] = column(q) < d ? r[q] + h[q] : 0.f;
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) r[q] = h[q];
    }
    if (a.r) store(static_cast<T *>(a.r) + off, r);
    if (!a.norm) continue;
    normalise(r, a.norm, a.norm_g, a.norm_b);
    store(static_cast<T *>(a.n) + off, r);
  }
}

// --------------------------------------------------------------- backward --
// The backward keeps neither instruction issue (55% of the cycles) nor memory
// (201 MB in 43 us at 16384 x 768) busy all the time: its registers leave a
// quarter of the warps.  Half of what it issues is arithmetic on pairs
// (packed_f32.cuh).
// Four columns of a row: consecutive ones from c on (VEC; 8 bytes of bf16,
// 16 of fp32), or c, c + stride, c + 2 stride, c + 3 stride, zeros behind d.
struct F4 {
  f2 a, b;
};
template <bool VEC>
__device__ __forceinline__ F4 load4(const float *row, int c, int stride, int d) {
  if (VEC) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(row + c);
    return {v.x, v.y};
  }
  float x[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) x[q] = c + q * stride < d ? row[c + q * stride] : 0.f;
  return {pair(x[0], x[1]), pair(x[2], x[3])};
}
template <bool VEC>
__device__ __forceinline__ F4 load4(const __nv_bfloat16 *row, int c, int stride, int d) {
  if (VEC) {
    const uint2 v = *reinterpret_cast<const uint2 *>(row + c);
    const float2 a = unpack_bf16(v.x), b = unpack_bf16(v.y);
    return {pair(a.x, a.y), pair(b.x, b.y)};
  }
  float x[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    x[q] = c + q * stride < d ? __bfloat162float(row[c + q * stride]) : 0.f;
  return {pair(x[0], x[1]), pair(x[2], x[3])};
}
template <bool VEC>
__device__ __forceinline__ void store4(float *row, int c, int stride, int d, const F4 &x) {
  if (VEC) {
    *reinterpret_cast<ulonglong2 *>(row + c) = make_ulonglong2(x.a, x.b);
    return;
  }
  const float2 a = split(x.a), b = split(x.b);
  const float v[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (c + q * stride < d) row[c + q * stride] = v[q];
}
template <bool VEC>
__device__ __forceinline__ void store4(__nv_bfloat16 *row, int c, int stride, int d, const F4 &x) {
  const float2 a = split(x.a), b = split(x.b);
  if (VEC) {
    *reinterpret_cast<uint2 *>(row + c) = make_uint2(pack_bf16(a.x, a.y), pack_bf16(b.x, b.y));
    return;
  }
  const float v[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (c + q * stride < d) row[c + q * stride] = __float2bfloat16_rn(v[q]);
}
// x + m, but zero behind d (element-wise columns; others are inside)
template <bool VEC>
__device__ __forceinline__ F4 shift4(const F4 &x, f2 m, int c, int stride, int d) {
  F4 r = {add2(x.a, m), add2(x.b, m)};
  if (!VEC) {
    const float2 a = split(r.a), b = split(r.b);
    r.a = pair(c < d ? a.x : 0.f, c + stride < d ? a.y : 0.f);
    r.b = pair(c + 2 * stride < d ? b.x : 0.f, c + 3 * stride < d ? b.y : 0.f);
  }
  return r;
}

// 16 bytes from global into shared memory without passing through registers
__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(dst)), "l"(src)
               : "memory");
}
// this thread's copies have landed
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
}

// A row's sums as the second half needs them: u = x i + m (m = -mean i), and
// dx = i (w + a + u b).
struct __align__(16) RowSums {
  float inv_r, m_r, a_r, b_r, inv_y, m_y, a_y, b_y;
};

// The tile in shared memory: rows of r, dn, dr, y and gate where there are
// such, and the column factors of w (ng) and of dy (kp = scale post_g).
template <typename T>
struct TileRows {
  const T *x, *dn, *dr, *y, *gate;
  const float *ng, *kp;
};

// The sums of row k of a tile, by one warp, columns c = 4 lane + 128 j (VEC,
// conflict-free) or lane + 128 j + 32 q; the row is read again for each sum.
template <typename T, bool VEC>
__device__ __forceinline__ RowSums row_sums(const Args &a, const TileRows<T> &t, int k, int lane) {
  const int d = a.d, c0 = VEC ? 4 * lane : lane;
  const float inv_d = 1.0f / (float)d;
  const bool norm_layer = a.norm == FLASH_GAU_NORM_LAYER, post_layer = a.post == FLASH_GAU_NORM_LAYER;
  const size_t at = (size_t)k * d;
  const T *x = t.x + at, *dn = t.dn + at, *dr = t.dr + at, *y = t.y + at, *gt = t.gate + at;
  RowSums s = {1.f, 0.f, 0.f, 0.f, 1.f, 0.f, 0.f, 0.f};
  float mean_r = 0.f, mean_y = 0.f;
  if (norm_layer) {
    f2 v = 0;
    for (int c = c0; c < d; c += 128) {
      const F4 e = load4<VEC>(x, c, 32, d);
      v = add2(v, add2(e.a, e.b));
    }
    mean_r = warp_sum(sum(v)) * inv_d;
  }
  if (post_layer) {
    f2 v = 0;
    for (int c = c0; c < d; c += 128) {
      const F4 e = load4<VEC>(y, c, 32, d);
      v = add2(v, add2(e.a, e.b));
    }
    mean_y = warp_sum(sum(v)) * inv_d;
  }
  float ub = 0.f;
  if (a.norm) {
    f2 m2 = 0, sw = 0, swx = 0;
    const f2 shift = both(-mean_r);
    for (int c = c0; c < d; c += 128) {
      const F4 e = shift4<VEC>(load4<VEC>(x, c, 32, d), shift, c, 32, d);
      const F4 g = load4<VEC>(dn, c, 32, d), w = load4<VEC>(t.ng, c, 32, d);
      const f2 wa = mul2(w.a, g.a), wb = mul2(w.b, g.b);
      m2 = fma2(e.a, e.a, fma2(e.b, e.b, m2));
      sw = add2(sw, add2(wa, wb));
      swx = fma2(wa, e.a, fma2(wb, e.b, swx));
    }
    const float q = warp_sum(sum(m2));
    s.inv_r = inv_spread(q, a.norm, inv_d, a.eps);
    s.m_r = -mean_r * s.inv_r;
    const float swu = warp_sum(sum(swx)) * s.inv_r;
    if (norm_layer) {
      s.a_r = -warp_sum(sum(sw)) * inv_d;
      s.b_r = -swu * inv_d;
    } else {
      s.b_r = longer(q, a.eps) ? -swu : 0.f;
    }
    ub = s.inv_r * s.b_r;
  }
  if (!a.post) return s;
  f2 m2 = 0, sg = 0, sgy = 0;
  const f2 inv_r = both(s.inv_r), a_r = both(s.a_r), ubb = both(ub), shift_y = both(-mean_y),
           shift_r = both(-mean_r);
  for (int c = c0; c < d; c += 128) {
    F4 dh = {0, 0};
    if (a.dr) dh = load4<VEC>(dr, c, 32, d);
    if (a.norm) {
      const F4 e = shift4<VEC>(load4<VEC>(x, c, 32, d), shift_r, c, 32, d);
      const F4 g = load4<VEC>(dn, c, 32, d), w = load4<VEC>(t.ng, c, 32, d);
      dh.a = fma2(inv_r, fma2(e.a, ubb, fma2(w.a, g.a, a_r)), dh.a);
      dh.b = fma2(inv_r, fma2(e.b, ubb, fma2(w.b, g.b, a_r)), dh.b);
    }
    F4 w = load4<VEC>(t.kp, c, 32, d);  // zero behind the row
    if (a.gate) {
      const F4 g = load4<VEC>(gt, c, 32, d);
      w.a = mul2(w.a, g.a);
      w.b = mul2(w.b, g.b);
    }
    const F4 e = shift4<VEC>(load4<VEC>(y, c, 32, d), shift_y, c, 32, d);
    const f2 fa = mul2(dh.a, w.a), fb = mul2(dh.b, w.b);
    m2 = fma2(e.a, e.a, fma2(e.b, e.b, m2));
    sg = add2(sg, add2(fa, fb));
    sgy = fma2(fa, e.a, fma2(fb, e.b, sgy));
  }
  const float q = warp_sum(sum(m2));
  s.inv_y = inv_spread(q, a.post, inv_d, a.eps);
  s.m_y = -mean_y * s.inv_y;
  const float sgu = warp_sum(sum(sgy)) * s.inv_y;
  if (post_layer) {
    s.a_y = -warp_sum(sum(sg)) * inv_d;
    s.b_y = -sgu * inv_d;
  } else {
    s.b_y = longer(q, a.eps) ? -sgu : 0.f;
  }
  return s;
}

// bytes from one array of a tile to the next
template <typename T, bool VEC>
__host__ __device__ inline size_t tile_pitch(long long rows, int d) {
  return ((size_t)rows * d * sizeof(T) + 15) / 16 * 16 + (VEC ? 0 : 16);
}

template <typename T, bool VEC, int NG, int MAXT, int BLOCKS>
__global__ void __launch_bounds__(MAXT, BLOCKS) residual_norm_grad_kernel(const Args a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int t = threadIdx.x, threads = blockDim.x, lane = t & 31, warp = t >> 5, d = a.d;
  const int warps = threads >> 5;
  const bool norm_layer = a.norm == FLASH_GAU_NORM_LAYER, post_layer = a.post == FLASH_GAU_NORM_LAYER;
  // the rows' sums, w's and dy's column factors, then the tile's arrays
  RowSums *sums = reinterpret_cast<RowSums *>(smem);
  const int dp = (d + 3) / 4 * 4;
  float *ng = reinterpret_cast<float *>(sums + a.rows), *kp = ng + dp;
  const size_t pitch = tile_pitch<T, VEC>(a.rows, d);
  const T *src[5] = {static_cast<const T *>(a.norm ? a.h : nullptr), static_cast<const T *>(a.dn),
                     static_cast<const T *>(a.dr), static_cast<const T *>(a.y),
                     static_cast<const T *>(a.gate)};
  T *tile[5];
  uint8_t *at = reinterpret_cast<uint8_t *>(kp + dp);
#pragma unroll
  for (int k = 0; k < 5; ++k) {
    tile[k] = reinterpret_cast<T *>(at);
    if (src[k]) at += pitch;
  }
  ptx::griddep_wait();
  for (int c = t; c < d; c += threads) {
    ng[c] = a.norm ? a.norm_g[norm_layer ? c : 0] : 1.f;
    kp[c] = (a.post ? a.post_g[post_layer ? c : 0] : 1.f) * (a.scale ? a.scale[c] : 1.f);
  }
  __syncthreads();
  // this thread's columns: groups of four, and which share of a tile's rows
  const int per = (d + 3) / 4;
  const int stride = NG == 1 ? per : threads;  // threads that have columns of their own
  const int sub = t / stride, own = t % stride;
  const bool active = sub < a.subsets;
  auto column = [&](int g) { return VEC ? 4 * (own + g * threads) : own + 4 * g * threads; };
  F4 acc[kSums][NG];
#pragma unroll
  for (int s = 0; s < kSums; ++s)
#pragma unroll
    for (int g = 0; g < NG; ++g) acc[s][g] = {0, 0};
  for (long long row0 = (long long)blockIdx.x * a.rows; row0 < a.M;
       row0 += (long long)gridDim.x * a.rows) {
    const int rows = (int)(a.M - row0 < a.rows ? a.M - row0 : a.rows);
    const int n = rows * d;
    const T *in_tile[5];
#pragma unroll
    for (int k = 0; k < 5; ++k) {
      in_tile[k] = tile[k];
      if (!src[k]) continue;
      const T *from = src[k] + row0 * d;
      // a tile's rows are one run of memory; it stands as far behind a 16-byte
      // boundary in shared memory as there, so that all but its ends moves 16
      // bytes at a time
      constexpr int W = 16 / sizeof(T);
      const int skew = VEC ? 0 : (int)(reinterpret_cast<uintptr_t>(from) % 16 / sizeof(T));
      T *to = tile[k] + skew;
      in_tile[k] = to;
      const int head = min((W - skew) % W, n), whole = head + (n - head) / W * W;
      for (int i = head + t * W; i < whole; i += threads * W) cp_async16(to + i, from + i);
      if (t < head) to[t] = from[t];
      for (int i = whole + t; i < n; i += threads) to[i] = from[i];
    }
    const TileRows<T> rows_in = {in_tile[0], in_tile[1], in_tile[2], in_tile[3], in_tile[4], ng, kp};
    cp_async_wait();
    __syncthreads();
    // ---- one warp a row: its sums
    for (int k = warp; k < rows; k += warps) {
      const RowSums s = row_sums<T, VEC>(a, rows_in, k, lane);
      if (lane == 0) sums[k] = s;
    }
    __syncthreads();
    // ---- four columns a thread and group: outputs and column sums
    if (active) {
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const int c = column(g);
        if (c >= d) continue;
        // the columns' parameters, read again for each tile: registers are
        // better spent on more blocks
        const F4 gn = load4<VEC>(ng, c, stride, d);
        float x[3][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int cq = VEC ? c + q : c + q * stride;
          const bool in = cq < d;
          x[0][q] = in ? (a.post ? __ldg(a.post_g + (post_layer ? cq : 0)) : 1.f) : 0.f;
          x[1][q] = in && post_layer && a.post_b ? __ldg(a.post_b + cq) : 0.f;
          x[2][q] = in ? (a.scale ? __ldg(a.scale + cq) : 1.f) : 0.f;
        }
        const F4 pg = {pair(x[0][0], x[0][1]), pair(x[0][2], x[0][3])};
        const F4 pb = {pair(x[1][0], x[1][1]), pair(x[1][2], x[1][3])};
        const F4 sc = {pair(x[2][0], x[2][1]), pair(x[2][2], x[2][3])};
        for (int k = sub; k < rows; k += a.subsets) {
          const RowSums s = sums[k];
          const int in = k * d;
          const long long out = (row0 + k) * d;
          F4 dh = {0, 0};
          if (a.dr) dh = load4<VEC>(rows_in.dr + in, c, stride, d);
          if (a.norm) {
            const F4 x = load4<VEC>(rows_in.x + in, c, stride, d);
            const F4 e = load4<VEC>(rows_in.dn + in, c, stride, d);
            const f2 i = both(s.inv_r), m = both(s.m_r), ar = both(s.a_r), br = both(s.b_r);
            const f2 ua = fma2(x.a, i, m), ub = fma2(x.b, i, m);
            dh.a = fma2(i, fma2(ua, br, fma2(e.a, gn.a, ar)), dh.a);
            dh.b = fma2(i, fma2(ub, br, fma2(e.b, gn.b, ar)), dh.b);
            acc[kNormG][g].a = fma2(e.a, ua, acc[kNormG][g].a);
            acc[kNormG][g].b = fma2(e.b, ub, acc[kNormG][g].b);
            acc[kNormB][g].a = add2(e.a, acc[kNormB][g].a);
            acc[kNormB][g].b = add2(e.b, acc[kNormB][g].b);
          }
          store4<VEC>(static_cast<T *>(a.dh) + out, c, stride, d, dh);
          if (!a.dy) continue;
          F4 y = {0, 0};
          if (a.y) y = load4<VEC>(rows_in.y + in, c, stride, d);
          const f2 i = both(s.inv_y), m = both(s.m_y), ay = both(s.a_y), by = both(s.b_y);
          const f2 ua = fma2(y.a, i, m), ub = fma2(y.b, i, m);
          // p = dh post(y); dp = dh scale gate
          const f2 pa = mul2(dh.a, fma2(ua, pg.a, pb.a));
          const f2 pb2 = mul2(dh.b, fma2(ub, pg.b, pb.b));
          f2 dpa = mul2(dh.a, sc.a), dpb = mul2(dh.b, sc.b);
          if (a.gate) {
            const F4 gv = load4<VEC>(rows_in.gate + in, c, stride, d);
            if (a.dgate)
              store4<VEC>(static_cast<T *>(a.dgate) + out, c, stride, d,
                          F4{mul2(pa, sc.a), mul2(pb2, sc.b)});
            acc[kScale][g].a = fma2(pa, gv.a, acc[kScale][g].a);
            acc[kScale][g].b = fma2(pb2, gv.b, acc[kScale][g].b);
            dpa = mul2(dpa, gv.a);
            dpb = mul2(dpb, gv.b);
          } else {
            acc[kScale][g].a = add2(pa, acc[kScale][g].a);
            acc[kScale][g].b = add2(pb2, acc[kScale][g].b);
          }
          acc[kPostG][g].a = fma2(dpa, ua, acc[kPostG][g].a);
          acc[kPostG][g].b = fma2(dpb, ub, acc[kPostG][g].b);
          acc[kPostB][g].a = add2(dpa, acc[kPostB][g].a);
          acc[kPostB][g].b = add2(dpb, acc[kPostB][g].b);
          // without a norm dy is dp: y, which may hold anything, has no part in it
          F4 dy = {dpa, dpb};
          if (a.post)
            dy = {mul2(i, fma2(ua, by, fma2(dpa, pg.a, ay))),
                  mul2(i, fma2(ub, by, fma2(dpb, pg.b, ay)))};
          store4<VEC>(static_cast<T *>(a.dy) + out, c, stride, d, dy);
        }
      }
    }
    __syncthreads();
  }
  // this thread's column sums, and the warps' sums for a ScaleNorm's g
  if (active) {
    float *part = a.part + ((long long)blockIdx.x * a.subsets + sub) * kSums * d;
#pragma unroll
    for (int s = 0; s < kSums; ++s)
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const float2 v = split(acc[s][g].a), w = split(acc[s][g].b);
        const float x[4] = {v.x, v.y, w.x, w.y};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c = VEC ? column(g) + q : column(g) + q * stride;
          if (c < d) part[s * (long long)d + c] = x[q];
        }
      }
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    f2 v = 0;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const F4 &x = acc[s ? kPostG : kNormG][g];
      v = add2(v, add2(x.a, x.b));
    }
    const float w = warp_sum(sum(v));
    if (lane == 0) a.scalar_part[((long long)s * gridDim.x + blockIdx.x) * kMaxWarps + warp] = w;
  }
}

// ---- rows of up to 2048 columns, on 16-byte boundaries
// WPR warps a row from its loads to its outputs, each a run of 128 NJ
// columns: the row's values stay in registers, the column sums of a lane's
// columns too, for the whole launch, and the next rows are on their way into
// the warp's own part of shared memory meanwhile.  Row sums pass between a row's
// warps through shared memory, one named barrier of theirs each.
//
// What a row costs in instructions beside its columns' arithmetic decides the
// time, so nothing in the loops over columns asks about the call's options:
// an array that is not there is a row of zeros (the gate: ones) written to
// shared memory once, columns behind d are zeros there, a missing norm is
// one whose row scalars change nothing, and the two norms differ in their
// row scalars alone.  Only what would hold registers is a template argument,
// the column sums: NORM_COL, of a LayerNorm's parameters; PS, behind the
// addition (0 none, 1 the scale's, 2 the scale's and a LayerNorm's).  A
// ScaleNorm's g takes one sum a lane.
constexpr int kRowWarps = 4;
// rows of a warp in shared memory: the one it works on and those on their
// way, about as many bytes of either type
template <typename T>
__host__ __device__ constexpr int row_slots() { return sizeof(T) == 2 ? 3 : 2; }
template <bool B>
using Is = std::integral_constant<bool, B>;

template <typename T, int WPR, int NJ, bool NORM_COL, int PS>
__global__ void __launch_bounds__(32 * kRowWarps, NJ * (NORM_COL * 2 + PS + (PS == 2)) <= 9 ? 4 : 3)
residual_norm_grad_rows_kernel(const Args a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float4 shared_sums[2][kRowWarps];
  constexpr int kWidth = 128 * NJ;       // columns of a warp
  constexpr int kRow = kWidth * WPR;     // and of a row, d and what is behind it
  constexpr int kSlot = 5 * kWidth;      // r, dn, dr, y, gate
  constexpr int kSlots = row_slots<T>();
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, d = a.d;
  const int first = kWidth * (warp % WPR), c0 = first + 4 * lane;
  const bool norm_layer = a.norm == FLASH_GAU_NORM_LAYER, post_layer = a.post == FLASH_GAU_NORM_LAYER;
  const float inv_d = 1.0f / (float)d, inv_eps = 1.0f / a.eps;
  // the columns' parameters, then the slots of rows of each warp
  float *ng = reinterpret_cast<float *>(smem), *sc = ng + kRow, *pg = sc + kRow, *pb = pg + kRow;
  T *const ring = reinterpret_cast<T *>(pb + (PS == 2 ? kRow : 0)) + warp * kSlots * kSlot;
  const T *src[5] = {static_cast<const T *>(a.norm ? a.h : nullptr), static_cast<const T *>(a.dn),
                     static_cast<const T *>(a.dr), static_cast<const T *>(a.y),
                     static_cast<const T *>(a.gate)};
  constexpr int kRowsAtOnce = kRowWarps / WPR;
  const long long step = (long long)gridDim.x * kRowsAtOnce;
  const long long row_first = (long long)blockIdx.x * kRowsAtOnce + warp / WPR;
  constexpr int W = 16 / sizeof(T);
  auto fetch = [&](long long row, int s) {
    if (row < a.M) {
      const long long off = row * d + first + lane * W;
      T *to = ring + s * kSlot + lane * W;
#pragma unroll
      for (int k = 0; k < 5; ++k) {
        if (!src[k]) continue;
#pragma unroll
        for (int j = 0; j < (kWidth + 32 * W - 1) / (32 * W); ++j) {
          const int c = (lane + 32 * j) * W;
          if (c < kWidth && first + c < d)
            cp_async16(to + k * kWidth + 32 * j * W, src[k] + off + 32 * j * W);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // zeros and ones, 16 bytes at a time
  const uint32_t ones = a.gate ? 0u : sizeof(T) == 2 ? 0x3f803f80u : 0x3f800000u;
  for (int i = lane * W; i < kSlots * kSlot; i += 32 * W) {
    const uint32_t v = i % kSlot >= 4 * kWidth ? ones : 0u;
    *reinterpret_cast<uint4 *>(ring + i) = make_uint4(v, v, v, v);
  }
  __syncwarp();
  ptx::griddep_wait();
#pragma unroll
  for (int k = 0; k < kSlots - 1; ++k) fetch(row_first + k * step, k);
  for (int c = t; c < kRow; c += 32 * kRowWarps) {
    const bool in = c < d;
    ng[c] = in && a.norm ? a.norm_g[norm_layer ? c : 0] : 0.f;
    sc[c] = !in ? 0.f : a.scale ? a.scale[c] : 1.f;
    pg[c] = !in ? 0.f : a.post ? a.post_g[post_layer ? c : 0] : 1.f;
    if (PS == 2) pb[c] = in && a.post_b ? a.post_b[c] : 0.f;
  }
  __syncthreads();
  F4 acc_ng[NORM_COL ? NJ : 1], acc_nb[NORM_COL ? NJ : 1], acc_sc[PS ? NJ : 1];
  F4 acc_pg[PS == 2 ? NJ : 1], acc_pb[PS == 2 ? NJ : 1];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    if (NORM_COL || j == 0) acc_ng[j] = acc_nb[j] = {0, 0};
    if (PS || j == 0) acc_sc[j] = {0, 0};
    if (PS == 2 || j == 0) acc_pg[j] = acc_pb[j] = {0, 0};
  }
  // sums of the row from its warps' sums, in the warps' order
  int flip = 0;
  auto row_sum = [&](float x, float y, auto with_z, float z) {
    float4 r = make_float4(warp_sum(x), warp_sum(y), 0.f, 0.f);
    if constexpr (decltype(with_z)::value) r.z = warp_sum(z);
    if constexpr (WPR > 1) {
      const int of = warp / WPR * WPR;
      if (lane == 0) shared_sums[flip][warp] = r;
      asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / WPR), "r"(32 * WPR) : "memory");
      r = shared_sums[flip][of];
#pragma unroll
      for (int w = 1; w < WPR; ++w) {
        const float4 v = shared_sums[flip][of + w];
        r.x += v.x;
        r.y += v.y;
        r.z += v.z;
      }
      flip ^= 1;  // written again only after the next barrier: everyone has read it
    }
    return r;
  };
  // added to a column of the row to take its mean off: zero behind the row
  auto shift_of = [&](int j, f2 minus_mean) { return c0 + 128 * j < d ? minus_mean : f2(0); };
  int s = 0;
  for (long long row = row_first; row < a.M; row += step) {
    fetch(row + (kSlots - 1) * step, s == 0 ? kSlots - 1 : s - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 1) : "memory");
    __syncwarp();
    const T *in = ring + s * kSlot + 4 * lane;
    const float *ngc = ng + c0, *scc = sc + c0, *pgc = pg + c0, *pbc = pb + c0;
    const long long out = row * d + c0;
    F4 x[NJ], y[NJ], dh[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      x[j] = load4<true>(in + 128 * j, 0, 0, d);
      y[j] = load4<true>(in + 3 * kWidth + 128 * j, 0, 0, d);
    }
    float mean_r = 0.f, mean_y = 0.f;
    if (NORM_COL || PS == 2) {
      f2 v = 0, vy = 0;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        v = add2(v, add2(x[j].a, x[j].b));
        vy = add2(vy, add2(y[j].a, y[j].b));
      }
      const float4 r = row_sum(sum(v), sum(vy), Is<false>(), 0.f);
      mean_r = norm_layer ? r.x * inv_d : 0.f;
      mean_y = post_layer ? r.y * inv_d : 0.f;
      const f2 mr = both(-mean_r), my = both(-mean_y);
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const f2 xs = shift_of(j, mr), ys = shift_of(j, my);
        x[j] = {add2(x[j].a, xs), add2(x[j].b, xs)};
        y[j] = {add2(y[j].a, ys), add2(y[j].b, ys)};
      }
    }
    float inv_r, a_r = 0.f, b_r;
    {
      f2 m2 = 0, sw = 0, swx = 0;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const F4 g = load4<true>(in + kWidth + 128 * j, 0, 0, d), w = load4<true>(ngc + 128 * j, 0, 0, d);
        dh[j] = {mul2(w.a, g.a), mul2(w.b, g.b)};
        m2 = fma2(x[j].a, x[j].a, fma2(x[j].b, x[j].b, m2));
        if (NORM_COL) sw = add2(sw, add2(dh[j].a, dh[j].b));
        swx = fma2(dh[j].a, x[j].a, fma2(dh[j].b, x[j].b, swx));
      }
      const float4 q = row_sum(sum(m2), sum(swx), Is<NORM_COL>(), sum(sw));
      if (NORM_COL) {
        inv_r = inv_layer(q.x, inv_d, a.eps);
        a_r = -q.z * inv_d;
        b_r = -q.y * inv_r * inv_d;
      } else {
        inv_r = inv_scale(q.x, inv_eps);
        b_r = longer(q.x, a.eps) ? -q.y * inv_r : 0.f;
      }
    }
    // dh = dr + i (w + a + u b), and the sums that dy needs
    const f2 ir = both(inv_r), ar = both(a_r), br = both(b_r);
    f2 m2 = 0, sg = 0, sgy = 0;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const F4 r = load4<true>(in + 2 * kWidth + 128 * j, 0, 0, d);
      const F4 g = load4<true>(in + kWidth + 128 * j, 0, 0, d);
      const f2 ua = mul2(x[j].a, ir), ub = mul2(x[j].b, ir);
      F4 &n = acc_ng[NORM_COL ? j : 0], &nb = acc_nb[NORM_COL ? j : 0];
      n = {fma2(g.a, ua, n.a), fma2(g.b, ub, n.b)};
      if (NORM_COL) nb = {add2(nb.a, g.a), add2(nb.b, g.b)};
      dh[j] = {fma2(ir, fma2(ua, br, add2(dh[j].a, ar)), r.a),
               fma2(ir, fma2(ub, br, add2(dh[j].b, ar)), r.b)};
      if (c0 + 128 * j < d) store4<true>(static_cast<T *>(a.dh) + out + 128 * j, 0, 0, d, dh[j]);
      // dp = dh scale gate stays in x's place
      const F4 w = load4<true>(scc + 128 * j, 0, 0, d), p = load4<true>(pgc + 128 * j, 0, 0, d);
      const F4 gt = load4<true>(in + 4 * kWidth + 128 * j, 0, 0, d);
      x[j] = {mul2(mul2(dh[j].a, w.a), gt.a), mul2(mul2(dh[j].b, w.b), gt.b)};
      const f2 fa = mul2(x[j].a, p.a), fb = mul2(x[j].b, p.b);
      m2 = fma2(y[j].a, y[j].a, fma2(y[j].b, y[j].b, m2));
      if (PS == 2) sg = add2(sg, add2(fa, fb));
      sgy = fma2(fa, y[j].a, fma2(fb, y[j].b, sgy));
    }
    if (a.dy) {
      float inv_y = 1.f, a_y = 0.f, b_y = 0.f;
      if (a.post) {
        const float4 q = row_sum(sum(m2), sum(sgy), Is<PS == 2>(), sum(sg));
        if (PS == 2) {
          inv_y = inv_layer(q.x, inv_d, a.eps);
          a_y = -q.z * inv_d;
          b_y = -q.y * inv_y * inv_d;
        } else {
          inv_y = inv_scale(q.x, inv_eps);
          b_y = longer(q.x, a.eps) ? -q.y * inv_y : 0.f;
        }
      }
      const f2 iy = both(inv_y), ay = both(a_y), by = both(b_y);
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const F4 u = {mul2(y[j].a, iy), mul2(y[j].b, iy)};
        const F4 g = load4<true>(pgc + 128 * j, 0, 0, d), w = load4<true>(scc + 128 * j, 0, 0, d);
        const F4 gt = load4<true>(in + 4 * kWidth + 128 * j, 0, 0, d);
        F4 p;  // dh post(y)
        if (PS == 2) {
          const F4 b = load4<true>(pbc + 128 * j, 0, 0, d);
          p = {mul2(dh[j].a, fma2(u.a, g.a, b.a)), mul2(dh[j].b, fma2(u.b, g.b, b.b))};
        } else {
          p = {mul2(dh[j].a, mul2(u.a, g.a)), mul2(dh[j].b, mul2(u.b, g.b))};
        }
        F4 &as = acc_sc[PS ? j : 0], &ag = acc_pg[PS == 2 ? j : 0], &ab = acc_pb[PS == 2 ? j : 0];
        if (PS) as = {fma2(p.a, gt.a, as.a), fma2(p.b, gt.b, as.b)};
        ag = {fma2(x[j].a, u.a, ag.a), fma2(x[j].b, u.b, ag.b)};
        if (PS == 2) ab = {add2(ab.a, x[j].a), add2(ab.b, x[j].b)};
        F4 dy = {mul2(iy, fma2(u.a, by, fma2(x[j].a, g.a, ay))),
                 mul2(iy, fma2(u.b, by, fma2(x[j].b, g.b, ay)))};
        // without a norm dy is dp: y, which may hold anything, has no part in it
        if (PS != 2 && !a.post) dy = x[j];
        if (c0 + 128 * j < d) {
          store4<true>(static_cast<T *>(a.dy) + out + 128 * j, 0, 0, d, dy);
          if (a.dgate)
            store4<true>(static_cast<T *>(a.dgate) + out + 128 * j, 0, 0, d,
                         F4{mul2(p.a, w.a), mul2(p.b, w.b)});
        }
      }
    }
    __syncwarp();  // the slot is read before it is filled again
    s = s + 1 == kSlots ? 0 : s + 1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  // the block's column sums, its rows' warps in order
  float *buf = reinterpret_cast<float *>(smem);  // [rows at once][kRow], over the parameters and rows
  float *part = a.part + (long long)blockIdx.x * kSums * d;
  auto gather = [&](int which, const F4 *acc) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NJ; ++j) store4<true>(buf + warp / WPR * kRow + c0 + 128 * j, 0, 0, d, acc[j]);
    __syncthreads();
    for (int c = t; c < d; c += 32 * kRowWarps) {
      float v = buf[c];
#pragma unroll
      for (int w = 1; w < kRowsAtOnce; ++w) v += buf[w * kRow + c];
      part[which * (long long)d + c] = v;
    }
  };
  if constexpr (NORM_COL) {
    gather(kNormG, acc_ng);
    gather(kNormB, acc_nb);
  }
  if constexpr (PS > 0) gather(kScale, acc_sc);
  if constexpr (PS == 2) {
    gather(kPostG, acc_pg);
    gather(kPostB, acc_pb);
  }
  // a ScaleNorm's g: one value a warp
  float *scalar = a.scalar_part + (long long)blockIdx.x * kMaxWarps + warp;
  if constexpr (!NORM_COL) {
    const float v = warp_sum(sum(add2(acc_ng[0].a, acc_ng[0].b)));
    if (lane == 0) scalar[0] = v;
  }
  if constexpr (PS != 2) {
    const float v = warp_sum(sum(add2(acc_pg[0].a, acc_pg[0].b)));
    if (lane == 0) scalar[(long long)gridDim.x * kMaxWarps] = v;
  }
}

struct SumArgs {
  const float *part, *scalar_part;
  float *out[kSums];    // null: not wanted
  int scalar[kSums];    // a ScaleNorm's g: one value
  int parts, blocks, warps, d;
};

// A sum with what its roundings have left out (Knuth's two-sum; nothing of a sum
// that is not finite, infinity less itself being no number).
struct Exact {
  float sum, left;
  __device__ float all() const { return isfinite(sum) ? sum + left : sum; }
  __device__ void add(float x, float x_left) {
    const float t = sum + x, b = t - sum;
    left += x_left + ((sum - (t - b)) + (x - b));
    sum = t;
  }
  __device__ void join_warp() {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float x = __shfl_xor_sync(kAll, sum, o), e = __shfl_xor_sync(kAll, left, o);
      add(x, e);
    }
  }
};

constexpr int kAtOnce = 10;  // loads under way: half of what 608 blocks leave a thread

// Sums the parts in a fixed order: a thread block takes 32 columns of one
// kind (blockIdx.y), 32 threads a column.  A ScaleNorm's g gathers terms of
// either sign from the whole [M, d], which cancel, so the roundings of its
// last sums are kept (2000 x 513 fp32, ten inputs: relative error 1.8e-7 ->
// 1.3e-7 in the middle; in fp64, whose units are few here, 10 us more).
__global__ void __launch_bounds__(1024) sum_parts_kernel(const SumArgs a) {
  ptx::griddep_wait();
  const int s = blockIdx.y;
  if (!a.out[s] || (a.scalar[s] && blockIdx.x)) return;
  const int lane = threadIdx.x & 31, sub = threadIdx.x >> 5;
  if (a.scalar[s]) {
    __shared__ Exact sums[32];
    const float *p = a.scalar_part + (s == kPostG ? (long long)a.blocks * kMaxWarps : 0);
    Exact v = {0.f, 0.f};
    if (lane < a.warps)
      for (int b0 = sub; b0 < a.blocks; b0 += 32 * kAtOnce) {
        float x[kAtOnce];
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q) {
          const int b = b0 + 32 * q;
          x[q] = b < a.blocks ? p[(long long)b * kMaxWarps + lane] : 0.f;
        }
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q) v.add(x[q], 0.f);
      }
    v.join_warp();
    if (lane == 0) sums[sub] = v;
    __syncthreads();
    if (sub == 0) {
      v = sums[lane];
      v.join_warp();
      if (lane == 0) a.out[s][0] = v.all();
    }
    return;
  }
  __shared__ float buf[32][33];
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < a.d) {
    const float *p = a.part + (long long)s * a.d + c;
    const long long step = (long long)kSums * a.d;
    for (int b0 = sub; b0 < a.parts; b0 += 32 * kAtOnce) {
      float x[kAtOnce];
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q) {
        const int b = b0 + 32 * q;
        x[q] = b < a.parts ? p[b * step] : 0.f;
      }
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q) v += x[q];
    }
  }
  buf[lane][sub] = v;
  __syncthreads();
  // warp w joins column w
  v = warp_sum(buf[sub][lane]);
  if (lane == 0 && blockIdx.x * 32 + sub < a.d) a.out[s][blockIdx.x * 32 + sub] = v;
}

bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// the accesses of 16 bytes that rows allow
bool vectors(const Args &a, int io) {
  bool vec = (long long)a.d * io % 16 == 0;
  for (const void *p : {a.h, a.y, a.gate, a.dr, a.dn, (const void *)a.r, (const void *)a.n,
                        (const void *)a.dh, (const void *)a.dy, (const void *)a.dgate})
    vec = vec && aligned16(p);
  return vec;
}

template <typename T>
cudaError_t forward(const Args &a, cudaStream_t stream) {
  // a warp a row: few rows go to as many SMs as there are
  const int warps = a.M <= kResidualMaxBlocks ? 1 : 4;
  const dim3 grid((unsigned)((a.M + warps - 1) / warps)), block(32 * warps);
  const int chunks = (a.d + 255) / 256;
  const bool params = aligned16(a.norm_g) && aligned16(a.norm_b) && aligned16(a.post_g) &&
                      aligned16(a.post_b) && aligned16(a.scale);
  const bool vec = vectors(a, sizeof(T)) && params;
  if (!vec || chunks > 8) {
    const unsigned threads = a.d <= 256 ? 128 : (unsigned)((a.d + 255) / 256 * 32);
    const long long rows = a.d <= 256 ? (a.M + 3) / 4 : a.M;
    const dim3 any((unsigned)(rows < 0x7fffffff ? rows : 0x7fffffff)), of(threads);
    return vec ? launch_pdl(residual_norm_any_kernel<T, true>, any, of, 0, stream, a)
               : launch_pdl(residual_norm_any_kernel<T, false>, any, of, 0, stream, a);
  }
  switch (chunks) {
    case 1: return launch_pdl(residual_norm_kernel<T, 1>, grid, block, 0, stream, a);
    case 2: return launch_pdl(residual_norm_kernel<T, 2>, grid, block, 0, stream, a);
    case 3: return launch_pdl(residual_norm_kernel<T, 3>, grid, block, 0, stream, a);
    case 4: return launch_pdl(residual_norm_kernel<T, 4>, grid, block, 0, stream, a);
    case 5:
    case 6: return launch_pdl(residual_norm_kernel<T, 6>, grid, block, 0, stream, a);
    default: return launch_pdl(residual_norm_kernel<T, 8>, grid, block, 0, stream, a);
  }
}

// The backward's shape: four columns a thread (a group), up to 256 threads
// with up to four groups each, 512 above 4096 columns; narrow rows share a
// block of 128 threads among `subsets` rows.
struct Shape {
  int groups, threads, subsets;
};
Shape shape_of(int d) {
  const int per = (d + 3) / 4;
  Shape s;
  s.groups = per <= 256 ? 1 : per <= 512 ? 2 : 4;
  const int t = ((per + s.groups - 1) / s.groups + 31) / 32 * 32;
  s.threads = t < 128 ? 128 : t;
  s.subsets = s.groups == 1 ? s.threads / per : 1;
  return s;
}

template <typename T, bool VEC, int NG, int MAXT, int BLOCKS>
cudaError_t launch_grad(const Args &a, const Shape &s, int blocks, size_t smem, cudaStream_t stream) {
  auto kernel = residual_norm_grad_kernel<T, VEC, NG, MAXT, BLOCKS>;
  static std::atomic<int> allowed[64];  // per device
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!allowed[dev].load(std::memory_order_acquire)) {
    // the most that any call asks for
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kGradSmemMax);
    if (err != cudaSuccess) return err;
    allowed[dev].store(1, std::memory_order_release);
  }
  return launch_pdl(kernel, dim3(blocks), dim3(s.threads), smem, stream, a);
}

template <typename T, bool VEC>
cudaError_t backward(Args &a, int num_sms, int *blocks_out, cudaStream_t stream) {
  const Shape s = shape_of(a.d);
  int arrays = 0;
  for (const void *p : {a.norm ? a.h : nullptr, a.dn, a.dr, a.y, a.gate}) arrays += p != nullptr;
  const size_t row = (size_t)arrays * a.d * sizeof(T);
  // rows of a tile: one for each warp while four blocks fit an SM, more of
  // narrow rows, and of wide ones half as many as warps where that fits at all
  const int warps = s.threads / 32;
  long long rows = (44 * 1024) / (long long)(row ? row : 1);
  if (rows > 4 * warps) rows = 4 * warps;
  if (rows > warps) rows = rows / warps * warps;
  const long long few = (warps + 1) / 2;
  if (rows < few) rows = few * (long long)row <= 160 * 1024 ? few : (160 * 1024) / (long long)row;
  if (rows < 1) rows = 1;
  // few rows in all: spread them over the blocks that fit the SMs
  const long long even = (a.M + 4LL * num_sms - 1) / (4LL * num_sms);
  if (rows > even) rows = even;
  // rows of odd widths: up to as many as leave every tile on 16-byte boundaries
  // (16384 x 767: 128 us for 141 in bf16, 146 for 188 in fp32)
  const long long unit = 16 / (int)sizeof(T);
  if (!VEC && rows >= unit / 2 && (rows + unit - 1) / unit * unit * (long long)row <= 160 * 1024)
    rows = (rows + unit - 1) / unit * unit;
  a.rows = (int)rows;
  a.subsets = s.subsets;
  const size_t smem = tile_pitch<T, VEC>(rows, a.d) * arrays + (size_t)((a.d + 3) / 4 * 4) * 8 + rows * sizeof(RowSums);
  const long long tiles = (a.M + rows - 1) / rows;
  long long per_sm = (long long)(224 * 1024 / (smem + 1024));
  if (per_sm > 2048 / s.threads) per_sm = 2048 / s.threads;
  if (per_sm < 1) per_sm = 1;
  if (per_sm > 4) per_sm = 4;
  long long blocks = per_sm * num_sms;
  if (blocks > kResidualMaxBlocks) blocks = kResidualMaxBlocks;
  if (blocks > tiles) blocks = tiles;
  *blocks_out = (int)blocks;
  a.scalar_part = a.part + (long long)blocks * s.subsets * kSums * a.d;
  const int n = (int)blocks;
  if (s.groups == 1) return launch_grad<T, VEC, 1, 256, 2>(a, s, n, smem, stream);
  if (s.groups == 2) return launch_grad<T, VEC, 2, 256, 1>(a, s, n, smem, stream);
  if (s.threads <= 256) return launch_grad<T, VEC, 4, 256, 1>(a, s, n, smem, stream);
  return launch_grad<T, VEC, 4, 512, 1>(a, s, n, smem, stream);
}

template <typename T, int WPR, int NJ, bool NORM_COL, int PS>
cudaError_t launch_rows(Args &a, int num_sms, int *blocks_out, cudaStream_t stream) {
  auto kernel = residual_norm_grad_rows_kernel<T, WPR, NJ, NORM_COL, PS>;
  // as the kernel lays it out; the column sums' exchange is no larger
  constexpr size_t row = 128 * NJ * WPR;
  constexpr size_t smem =
      (PS == 2 ? 4 : 3) * row * sizeof(float) + kRowWarps * row_slots<T>() * 5 * 128 * NJ * sizeof(T);
  static_assert(kRowWarps / WPR * row * sizeof(float) <= smem, "exchange of the column sums");
  static std::atomic<int> fit[64];  // per device: blocks that fit an SM
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int per_sm = fit[dev].load(std::memory_order_acquire);
  if (!per_sm) {
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess) return err;
    err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, 32 * kRowWarps, smem);
    if (err != cudaSuccess) return err;
    if (per_sm < 1) per_sm = 1;
    fit[dev].store(per_sm, std::memory_order_release);
  }
  long long blocks = (long long)num_sms * per_sm;
  if (blocks > kResidualMaxBlocks) blocks = kResidualMaxBlocks;
  const long long need = (a.M + kRowWarps / WPR - 1) / (kRowWarps / WPR);
  if (blocks > need) blocks = need;
  *blocks_out = (int)blocks;
  a.subsets = 1;
  a.scalar_part = a.part + (long long)blocks * kSums * a.d;
  return launch_pdl(kernel, dim3((unsigned)blocks), dim3(32 * kRowWarps), smem, stream, a);
}

template <typename T, int WPR, int NJ>
cudaError_t rows_by_sums(Args &a, int num_sms, int *blocks, cudaStream_t stream) {
  const bool col = a.norm == FLASH_GAU_NORM_LAYER;
  const int ps = a.post == FLASH_GAU_NORM_LAYER ? 2 : a.scale ? 1 : 0;
  switch (ps + (col ? 3 : 0)) {
    case 0: return launch_rows<T, WPR, NJ, false, 0>(a, num_sms, blocks, stream);
    case 1: return launch_rows<T, WPR, NJ, false, 1>(a, num_sms, blocks, stream);
    case 2: return launch_rows<T, WPR, NJ, false, 2>(a, num_sms, blocks, stream);
    case 3: return launch_rows<T, WPR, NJ, true, 0>(a, num_sms, blocks, stream);
    case 4: return launch_rows<T, WPR, NJ, true, 1>(a, num_sms, blocks, stream);
    default: return launch_rows<T, WPR, NJ, true, 2>(a, num_sms, blocks, stream);
  }
}

// rows on 16-byte boundaries of up to 2048 columns: up to 512 columns a warp,
// fewer where that leaves registers for more warps
template <typename T>
cudaError_t backward_vec(Args &a, int num_sms, int *blocks, cudaStream_t stream) {
  if (a.d <= 256) return rows_by_sums<T, 1, 2>(a, num_sms, blocks, stream);
  if (a.d <= 512) return rows_by_sums<T, 2, 2>(a, num_sms, blocks, stream);
  if (a.d <= 768) return rows_by_sums<T, 2, 3>(a, num_sms, blocks, stream);
  if (a.d <= 1024) return rows_by_sums<T, 2, 4>(a, num_sms, blocks, stream);
  if (a.d <= 2048) return rows_by_sums<T, 4, 4>(a, num_sms, blocks, stream);
  return backward<T, true>(a, num_sms, blocks, stream);
}

Args args_of(const ResidualProblem &q) {
  Args a = {};
  a.gate = q.o.gate;
  a.norm_g = q.o.norm_g;
  a.norm_b = q.o.norm_b;
  a.post_g = q.o.post_g;
  a.post_b = q.o.post_b;
  a.scale = q.o.scale;
  a.norm = q.o.norm;
  a.post = q.o.post;
  a.eps = q.o.eps;
  a.M = q.M;
  a.d = q.d;
  a.y = q.y;
  return a;
}

}  // namespace

size_t residual_norm_part_bytes(long long M, int d) {
  const size_t blocks = (size_t)(M < kResidualMaxBlocks ? M : kResidualMaxBlocks);
  return (blocks * shape_of(d).subsets * kSums * d + 2 * blocks * kMaxWarps) * sizeof(float);
}

cudaError_t residual_norm(const ResidualProblem &q, const void *h, void *r, void *n) {
  Args a = args_of(q);
  a.h = h;
  a.r = r;
  a.n = n;
  return q.dtype == FLASH_GAU_BF16 ? forward<__nv_bfloat16>(a, q.stream)
                                   : forward<float>(a, q.stream);
}

cudaError_t residual_norm_grad(const ResidualProblem &q, const void *dr, const void *dn,
                               const void *r, const flash_gau_residual_grads &g, void *workspace) {
  Args a = args_of(q);
  a.h = r;
  a.dr = dr;
  a.dn = dn;
  a.dh = g.dh;
  a.dy = g.dy;
  a.dgate = g.dgate;
  a.part = static_cast<float *>(workspace);
  if (!a.post && !a.gate && !a.scale) a.y = nullptr;  // nothing needs its values
  int blocks = 0;
  cudaError_t err;
  if (q.dtype == FLASH_GAU_BF16)
    err = vectors(a, 2) ? backward_vec<__nv_bfloat16>(a, q.num_sms, &blocks, q.stream)
                        : backward<__nv_bfloat16, false>(a, q.num_sms, &blocks, q.stream);
  else
    err = vectors(a, 4) ? backward_vec<float>(a, q.num_sms, &blocks, q.stream)
                        : backward<float, false>(a, q.num_sms, &blocks, q.stream);
  if (err != cudaSuccess) return err;
  SumArgs s = {};
  s.part = a.part;
  s.scalar_part = a.scalar_part;
  s.parts = blocks * a.subsets;
  s.blocks = blocks;
  s.warps = a.rows ? shape_of(q.d).threads / 32 : kRowWarps;
  s.d = q.d;
  s.out[kNormG] = a.norm ? g.dnorm_g : nullptr;
  s.out[kNormB] = a.norm == FLASH_GAU_NORM_LAYER ? g.dnorm_b : nullptr;
  s.out[kPostG] = a.post ? g.dpost_g : nullptr;
  s.out[kPostB] = a.post == FLASH_GAU_NORM_LAYER ? g.dpost_b : nullptr;
  s.out[kScale] = a.scale ? g.dscale : nullptr;
  s.scalar[kNormG] = a.norm == FLASH_GAU_NORM_SCALE;
  s.scalar[kPostG] = a.post == FLASH_GAU_NORM_SCALE;
  bool any = false;
  for (const float *p : s.out) any = any || p;
  if (!any) return cudaSuccess;
  return launch_pdl(sum_parts_kernel, dim3((q.d + 31) / 32, kSums), dim3(1024), 0, q.stream, s);
}

}  // namespace flashgau
