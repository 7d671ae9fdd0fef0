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
// bytes a lane), no block-wide step at all.  Rows wider than 2048 columns, or
// not on 16-byte boundaries, take a plain form that reads the row again from
// L1 for each of its sums.
//
// Backward, a tile of rows (about 44 KB, four blocks an SM) is brought into
// shared memory by asynchronous copies.  First one warp a row takes the row's sums;
// means come first and squares around them second (no difference of large
// squares), and the sums that dx needs ride along, three passes over shared
// memory in all.  Then the threads turn by 90 degrees: each keeps four
// columns for the whole launch, forms the outputs of the tile's rows from
// the rows' sums, and adds up the parameters' gradients in registers.
#include <cuda_bf16.h>

#include "flash_gau_internal.h"
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
// around zero (ScaleNorm)
__device__ __forceinline__ float inv_spread(float m2, int kind, int d, float eps) {
  return kind == FLASH_GAU_NORM_LAYER ? 1.0f / sqrtf(m2 / (float)d + eps)
                                      : 1.0f / fmaxf(sqrtf(m2), eps);
}

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
    if (c < d) {  // 4-byte alignment is all that is asked of parameters
      v.x = __ldg(p + c);
      v.y = __ldg(p + c + 1);
      v.z = __ldg(p + c + 2);
      v.w = __ldg(p + c + 3);
    }
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
  return make_float2(mean, inv_spread(warp_sum(m2), kind, d, eps));
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

// Any width and alignment: one warp a row, element by element, the row read
// again for each sum.  Outputs are written last, each after the same
// element's inputs, so they may be the inputs' arrays.
template <typename T>
__global__ void __launch_bounds__(128) residual_norm_any_kernel(const Args a) {
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31, d = a.d;
  const long long row = blockIdx.x * (long long)(blockDim.x >> 5) + (threadIdx.x >> 5);
  if (row >= a.M) return;
  const T *h = static_cast<const T *>(a.h) + row * d;
  const T *y = a.y ? static_cast<const T *>(a.y) + row * d : nullptr;
  const T *gate = a.gate ? static_cast<const T *>(a.gate) + row * d : nullptr;
  auto stat = [&](auto get, int kind) {
    float mean = 0.f, m2 = 0.f;
    if (kind == FLASH_GAU_NORM_LAYER) {
      float s = 0.f;
      for (int c = lane; c < d; c += 32) s += get(c);
      mean = warp_sum(s) / (float)d;
    }
    for (int c = lane; c < d; c += 32) {
      const float v = get(c) - mean;
      m2 = fmaf(v, v, m2);
    }
    return make_float2(mean, inv_spread(warp_sum(m2), kind, d, a.eps));
  };
  auto affine = [&](float u, int kind, const float *g, const float *b, int c) {
    if (kind == FLASH_GAU_NORM_LAYER) return fmaf(u, g[c], b ? b[c] : 0.f);
    return kind == FLASH_GAU_NORM_SCALE ? u * g[0] : u;
  };
  float2 sy = make_float2(0.f, 1.f);
  if (y && a.post) sy = stat([&](int c) { return to_f(y[c]); }, a.post);
  auto r = [&](int c) {
    if (!y) return to_f(h[c]);
    float v = affine((to_f(y[c]) - sy.x) * sy.y, a.post, a.post_g, a.post_b, c);
    if (gate) v *= to_f(gate[c]);
    if (a.scale) v *= a.scale[c];
    return to_f(h[c]) + v;
  };
  float2 sr = make_float2(0.f, 1.f);
  if (a.norm) sr = stat(r, a.norm);
  for (int c = lane; c < d; c += 32) {
    const float v = r(c);
    const float n = affine((v - sr.x) * sr.y, a.norm, a.norm_g, a.norm_b, c);
    if (a.r) static_cast<T *>(a.r)[row * d + c] = (T)v;
    if (a.norm) static_cast<T *>(a.n)[row * d + c] = (T)n;
  }
}

// --------------------------------------------------------------- backward --
// Four columns of a row: consecutive ones from c on (VEC; 8 bytes of bf16,
// 16 of fp32), or c, c + stride, c + 2 stride, c + 3 stride, zeros behind d.
template <bool VEC>
__device__ __forceinline__ void load4(const float *row, int c, int stride, int d, float (&x)[4]) {
  if (VEC) {
    const float4 v = *reinterpret_cast<const float4 *>(row + c);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] = c + q * stride < d ? row[c + q * stride] : 0.f;
  }
}
template <bool VEC>
__device__ __forceinline__ void load4(const __nv_bfloat16 *row, int c, int stride, int d,
                                      float (&x)[4]) {
  if (VEC) {
    const uint2 v = *reinterpret_cast<const uint2 *>(row + c);
    const float2 a = unpack_bf16(v.x), b = unpack_bf16(v.y);
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      x[q] = c + q * stride < d ? __bfloat162float(row[c + q * stride]) : 0.f;
  }
}
template <bool VEC>
__device__ __forceinline__ void store4(float *row, int c, int stride, int d, const float (&x)[4]) {
  if (VEC) {
    *reinterpret_cast<float4 *>(row + c) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (c + q * stride < d) row[c + q * stride] = x[q];
  }
}
template <bool VEC>
__device__ __forceinline__ void store4(__nv_bfloat16 *row, int c, int stride, int d,
                                       const float (&x)[4]) {
  if (VEC) {
    *reinterpret_cast<uint2 *>(row + c) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (c + q * stride < d) row[c + q * stride] = __float2bfloat16_rn(x[q]);
  }
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

// A row's sums as the second half needs them: u = (x - mean) i, and
// dx = i (w - a - u b).
struct RowSums {
  float mean_r, inv_r, a_r, b_r, mean_y, inv_y, a_y, b_y;
};

template <typename T, bool VEC, int NG, int MAXT>
__global__ void __launch_bounds__(MAXT) residual_norm_grad_kernel(const Args a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int t = threadIdx.x, threads = blockDim.x, lane = t & 31, warp = t >> 5, d = a.d;
  const int warps = threads >> 5;
  const bool norm_layer = a.norm == FLASH_GAU_NORM_LAYER, post_layer = a.post == FLASH_GAU_NORM_LAYER;
  // the tile's arrays, then w's and dy's column factors, then the rows' sums
  const size_t array = (size_t)a.rows * d * sizeof(T), pitch = (array + 15) / 16 * 16;
  const T *src[5] = {static_cast<const T *>(a.norm ? a.h : nullptr), static_cast<const T *>(a.dn),
                     static_cast<const T *>(a.dr), static_cast<const T *>(a.y),
                     static_cast<const T *>(a.gate)};
  T *tile[5];
  uint8_t *at = smem;
#pragma unroll
  for (int k = 0; k < 5; ++k) {
    tile[k] = reinterpret_cast<T *>(at);
    if (src[k]) at += pitch;
  }
  T *const tx = tile[0], *const tdn = tile[1], *const tdr = tile[2], *const ty = tile[3],
           *const tg = tile[4];
  const int dp = (d + 3) / 4 * 4;
  float *ng = reinterpret_cast<float *>(at), *kp = ng + dp;
  RowSums *sums = reinterpret_cast<RowSums *>(kp + dp);
  ptx::griddep_wait();
  for (int c = t; c < d; c += threads) {
    ng[c] = a.norm ? a.norm_g[norm_layer ? c : 0] : 1.f;
    kp[c] = (a.post ? a.post_g[post_layer ? c : 0] : 1.f) * (a.scale ? a.scale[c] : 1.f);
  }
  __syncthreads();
  // this thread's columns: group g of four, and which share of a tile's rows
  const int per = (d + 3) / 4;
  const int lanes = NG == 1 ? per : threads;  // threads that have columns of their own
  const int sub = t / lanes, own = t % lanes;
  const bool active = sub < a.subsets;
  const int stride = lanes;  // element-wise: between a group's columns
  auto column = [&](int g) { return VEC ? 4 * (own + g * threads) : own + 4 * g * threads; };
  float pg[NG][4], pb[NG][4], sc[NG][4], gn[NG][4], acc[kSums][NG][4];
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = VEC ? column(g) + q : column(g) + q * stride;
      const bool in = active && c < d;
      gn[g][q] = in ? ng[c] : 0.f;
      sc[g][q] = in ? (a.scale ? a.scale[c] : 1.f) : 0.f;
      pg[g][q] = in ? (a.post ? a.post_g[post_layer ? c : 0] : 1.f) : 0.f;
      pb[g][q] = in && post_layer && a.post_b ? a.post_b[c] : 0.f;
#pragma unroll
      for (int s = 0; s < kSums; ++s) acc[s][g][q] = 0.f;
    }
  const float inv_d = 1.0f / (float)d;
  for (long long row0 = (long long)blockIdx.x * a.rows; row0 < a.M;
       row0 += (long long)gridDim.x * a.rows) {
    const int rows = (int)(a.M - row0 < a.rows ? a.M - row0 : a.rows);
    const int n = rows * d;
#pragma unroll
    for (int k = 0; k < 5; ++k) {
      if (!src[k]) continue;
      const T *from = src[k] + row0 * d;
      if (VEC) {
        constexpr int W = 16 / sizeof(T);
        for (int i = t * W; i < n; i += threads * W) cp_async16(tile[k] + i, from + i);
      } else {
        for (int i = t; i < n; i += threads) tile[k][i] = from[i];
      }
    }
    if (VEC) cp_async_wait();
    __syncthreads();
    // ---- one warp a row: its sums
    for (int k = warp; k < rows; k += warps) {
      const T *x = tx + (size_t)k * d, *dn = tdn + (size_t)k * d, *dr = tdr + (size_t)k * d;
      const T *y = ty + (size_t)k * d, *gt = tg + (size_t)k * d;
      const int c0 = VEC ? 4 * lane : lane;
      auto in = [&](int c, int q) { return VEC || c + 32 * q < d; };
      RowSums s = {0.f, 1.f, 0.f, 0.f, 0.f, 1.f, 0.f, 0.f};
      if (norm_layer || post_layer) {
        float sr = 0.f, sy = 0.f;
        for (int c = c0; c < d; c += 128) {
          float v[4];
          if (norm_layer) {
            load4<VEC>(x, c, 32, d, v);
            sr += (v[0] + v[1]) + (v[2] + v[3]);
          }
          if (post_layer) {
            load4<VEC>(y, c, 32, d, v);
            sy += (v[0] + v[1]) + (v[2] + v[3]);
          }
        }
        if (norm_layer) s.mean_r = warp_sum(sr) * inv_d;
        if (post_layer) s.mean_y = warp_sum(sy) * inv_d;
      }
      if (a.norm || a.post) {
        float m2r = 0.f, m2y = 0.f, sw = 0.f, swx = 0.f;
        for (int c = c0; c < d; c += 128) {
          float v[4], g[4], w[4];
          if (a.norm) {
            load4<VEC>(x, c, 32, d, v);
            load4<VEC>(dn, c, 32, d, g);
            load4<VEC>(ng, c, 32, d, w);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float e = in(c, q) ? v[q] - s.mean_r : 0.f;
              m2r = fmaf(e, e, m2r);
              w[q] *= g[q];
              sw += w[q];
              swx = fmaf(w[q], e, swx);
            }
          }
          if (a.post) {
            load4<VEC>(y, c, 32, d, v);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float e = in(c, q) ? v[q] - s.mean_y : 0.f;
              m2y = fmaf(e, e, m2y);
            }
          }
        }
        if (a.norm) {
          m2r = warp_sum(m2r);
          s.inv_r = inv_spread(m2r, a.norm, d, a.eps);
          swx = warp_sum(swx) * s.inv_r;
          if (norm_layer) {
            s.a_r = warp_sum(sw) * inv_d;
            s.b_r = swx * inv_d;
          } else {
            s.b_r = sqrtf(m2r) > a.eps ? swx : 0.f;
          }
        }
        if (a.post) {
          m2y = warp_sum(m2y);
          s.inv_y = inv_spread(m2y, a.post, d, a.eps);
          float sg = 0.f, sgy = 0.f;
          for (int c = c0; c < d; c += 128) {
            float dh[4] = {0.f, 0.f, 0.f, 0.f}, v[4], g[4], w[4];
            if (a.dr) load4<VEC>(dr, c, 32, d, dh);
            if (a.norm) {
              load4<VEC>(x, c, 32, d, v);
              load4<VEC>(dn, c, 32, d, g);
              load4<VEC>(ng, c, 32, d, w);
#pragma unroll
              for (int q = 0; q < 4; ++q)
                dh[q] += s.inv_r * (w[q] * g[q] - s.a_r - (v[q] - s.mean_r) * s.inv_r * s.b_r);
            }
            load4<VEC>(kp, c, 32, d, w);  // zero behind the row
            load4<VEC>(y, c, 32, d, v);
            if (a.gate) {
              load4<VEC>(gt, c, 32, d, g);
#pragma unroll
              for (int q = 0; q < 4; ++q) w[q] *= g[q];
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float e = dh[q] * w[q];
              sg += e;
              sgy = fmaf(e, v[q] - s.mean_y, sgy);
            }
          }
          sgy = warp_sum(sgy) * s.inv_y;
          if (post_layer) {
            s.a_y = warp_sum(sg) * inv_d;
            s.b_y = sgy * inv_d;
          } else {
            s.b_y = sqrtf(m2y) > a.eps ? sgy : 0.f;
          }
        }
      }
      if (lane == 0) sums[k] = s;
    }
    __syncthreads();
    // ---- four columns a thread and group: outputs and column sums
    if (active) {
      for (int k = sub; k < rows; k += a.subsets) {
        const RowSums s = sums[k];
        const long long out = (row0 + k) * d;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const int c = column(g);
          if (c >= d) continue;
          float dh[4] = {0.f, 0.f, 0.f, 0.f}, v[4], e[4];
          if (a.dr) load4<VEC>(tdr + (size_t)k * d, c, stride, d, dh);
          if (a.norm) {
            load4<VEC>(tx + (size_t)k * d, c, stride, d, v);
            load4<VEC>(tdn + (size_t)k * d, c, stride, d, e);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float u = (v[q] - s.mean_r) * s.inv_r;
              dh[q] += s.inv_r * (e[q] * gn[g][q] - s.a_r - u * s.b_r);
              acc[kNormG][g][q] = fmaf(e[q], u, acc[kNormG][g][q]);
              acc[kNormB][g][q] += e[q];
            }
          }
          store4<VEC>(static_cast<T *>(a.dh) + out, c, stride, d, dh);
          if (!a.dy) continue;
          float gv[4] = {1.f, 1.f, 1.f, 1.f};
          if (a.y) load4<VEC>(ty + (size_t)k * d, c, stride, d, v);
          else v[0] = v[1] = v[2] = v[3] = 0.f;
          if (a.gate) load4<VEC>(tg + (size_t)k * d, c, stride, d, gv);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float u = (v[q] - s.mean_y) * s.inv_y;
            const float p = dh[q] * fmaf(u, pg[g][q], pb[g][q]);
            acc[kScale][g][q] = fmaf(p, gv[q], acc[kScale][g][q]);
            const float dp = dh[q] * gv[q] * sc[g][q];
            acc[kPostG][g][q] = fmaf(dp, u, acc[kPostG][g][q]);
            acc[kPostB][g][q] += dp;
            v[q] = s.inv_y * (dp * pg[g][q] - s.a_y - u * s.b_y);
            e[q] = p * sc[g][q];
          }
          if (a.dgate) store4<VEC>(static_cast<T *>(a.dgate) + out, c, stride, d, e);
          store4<VEC>(static_cast<T *>(a.dy) + out, c, stride, d, v);
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
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c = VEC ? column(g) + q : column(g) + q * stride;
          if (c < d) part[s * (long long)d + c] = acc[s][g][q];
        }
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    float v = 0.f;
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int q = 0; q < 4; ++q) v += acc[s ? kPostG : kNormG][g][q];
    v = warp_sum(v);
    if (lane == 0) a.scalar_part[((long long)s * gridDim.x + blockIdx.x) * kMaxWarps + warp] = v;
  }
}

struct SumArgs {
  const float *part, *scalar_part;
  float *out[kSums];    // null: not wanted
  int scalar[kSums];    // a ScaleNorm's g: one value
  int parts, blocks, warps, d;
};

// Sums the parts in a fixed order: a thread block takes 32 columns of one
// kind (blockIdx.y), 32 threads a column.
__global__ void __launch_bounds__(1024) sum_parts_kernel(const SumArgs a) {
  ptx::griddep_wait();
  const int s = blockIdx.y;
  if (!a.out[s] || (a.scalar[s] && blockIdx.x)) return;
  __shared__ float buf[32][33];
  const int lane = threadIdx.x & 31, sub = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (a.scalar[s]) {
    const float *p = a.scalar_part + (s == kPostG ? (long long)a.blocks * kMaxWarps : 0);
    if (lane < a.warps)
      for (int b = sub; b < a.blocks; b += 32) v += p[(long long)b * kMaxWarps + lane];
  } else if (c < a.d) {
    const float *p = a.part + (long long)s * a.d + c;
    const long long step = (long long)kSums * a.d;
#pragma unroll 4
    for (int b = sub; b < a.parts; b += 32) v += p[b * step];
  }
  buf[lane][sub] = v;
  __syncthreads();
  // warp w joins column w
  v = warp_sum(buf[sub][lane]);
  if (a.scalar[s]) {
    __syncthreads();
    if (lane == 0) buf[0][sub] = v;
    __syncthreads();
    if (sub == 0) {
      v = warp_sum(buf[0][lane]);
      if (lane == 0) a.out[s][0] = v;
    }
  } else if (lane == 0 && blockIdx.x * 32 + sub < a.d) {
    a.out[s][blockIdx.x * 32 + sub] = v;
  }
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
  if (!vectors(a, sizeof(T)) || chunks > 8)
    return launch_pdl(residual_norm_any_kernel<T>, grid, block, 0, stream, a);
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

template <typename T, bool VEC, int NG, int MAXT>
cudaError_t launch_grad(const Args &a, const Shape &s, int blocks, size_t smem, cudaStream_t stream) {
  auto kernel = residual_norm_grad_kernel<T, VEC, NG, MAXT>;
  static size_t allowed[64];  // per device: the largest set so far
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (smem > 48 * 1024 && allowed[dev] == 0) {
    // the most that any call asks for
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kGradSmemMax);
    if (err != cudaSuccess) return err;
    allowed[dev] = kGradSmemMax;
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
  // few rows in all: spread them over the SMs
  const long long even = (a.M + num_sms - 1) / num_sms;
  if (rows > even) rows = even;
  a.rows = (int)rows;
  a.subsets = s.subsets;
  const size_t pitch = ((size_t)rows * a.d * sizeof(T) + 15) / 16 * 16;
  const size_t smem = pitch * arrays + (size_t)((a.d + 3) / 4 * 4) * 8 + rows * sizeof(RowSums);
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
  if (s.groups == 1) return launch_grad<T, VEC, 1, 256>(a, s, (int)blocks, smem, stream);
  if (s.groups == 2) return launch_grad<T, VEC, 2, 256>(a, s, (int)blocks, smem, stream);
  if (s.threads <= 256) return launch_grad<T, VEC, 4, 256>(a, s, (int)blocks, smem, stream);
  return launch_grad<T, VEC, 4, 512>(a, s, (int)blocks, smem, stream);
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
    err = vectors(a, 2) ? backward<__nv_bfloat16, true>(a, q.num_sms, &blocks, q.stream)
                        : backward<__nv_bfloat16, false>(a, q.num_sms, &blocks, q.stream);
  else
    err = vectors(a, 4) ? backward<float, true>(a, q.num_sms, &blocks, q.stream)
                        : backward<float, false>(a, q.num_sms, &blocks, q.stream);
  if (err != cudaSuccess) return err;
  SumArgs s = {};
  s.part = a.part;
  s.scalar_part = a.scalar_part;
  s.parts = blocks * a.subsets;
  s.blocks = blocks;
  s.warps = shape_of(q.d).threads / 32;
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
