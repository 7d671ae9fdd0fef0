// Activation checkpoints in 8 bits: the residual stream of a block's boundary
// kept between the forward and the backward pass as int8 codes, each 128
// neighbours of a row (a group) with an fp32 scale,
//   scale = max |x| * (1 / 127)  code = x / scale to the nearest, ties to even
// pack     r = h + y, n = norm(r), and the codes of r as it is stored
// restore  x = code * scale, and n = norm(x): what the layer's backward reads
// backward dh = dr + the norm's gradient at x, and its parameters' gradients
// with the norms of the residual stream's operator (LayerNorm, ScaleNorm).
//
// All three move rows once: in bf16 9, 5 and 7 bytes an element with the
// scales' 4 / 128, so memory bounds them.  A row belongs to one warp (up to
// 1024 columns) or to the four warps of a block, 8 consecutive columns a
// thread and step: 16 or 32 bytes of a row, 8 codes, and a group is 16
// neighbouring threads, whose maximum is four shuffles.
//
// A code is exact by its definition, not by the luck of a reciprocal: the
// rounded product x * (1 / scale) is at most one off, the remainder x - code *
// scale has no rounding error (it is below scale and a multiple of the smaller
// one's last place), and moves the code where it is above half a scale.
#include <cuda_bf16.h>

#include "flash_gau_internal.h"
#include "sm103_ptx.cuh"

namespace flashgau {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kGroup = kCheckpointGroup;
constexpr float kLeast = 0x1p-100f;  // a group below this is zero

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

// Eight columns of a row from column c on; `vec`: rows are whole vectors on
// their boundaries.  Columns behind d are zero and not stored.
__device__ __forceinline__ void load8(const __nv_bfloat16 *row, int c, int d, bool vec,
                                      float (&x)[8]) {
  if (vec) {
    const uint4 w = c < d ? *reinterpret_cast<const uint4 *>(row + c) : make_uint4(0, 0, 0, 0);
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 f = unpack_bf16(v[q]);
      x[2 * q] = f.x;
      x[2 * q + 1] = f.y;
    }
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = c + q < d ? __bfloat162float(row[c + q]) : 0.f;
  }
}
__device__ __forceinline__ void load8(const float *row, int c, int d, bool vec, float (&x)[8]) {
  if (vec) {
#pragma unroll
    for (int q = 0; q < 8; q += 4) {
      const float4 w = c < d ? *reinterpret_cast<const float4 *>(row + c + q)
                             : make_float4(0.f, 0.f, 0.f, 0.f);
      x[q] = w.x;
      x[q + 1] = w.y;
      x[q + 2] = w.z;
      x[q + 3] = w.w;
    }
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = c + q < d ? row[c + q] : 0.f;
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16 *row, int c, int d, bool vec,
                                       const float (&x)[8]) {
  if (vec) {
    if (c < d)
      *reinterpret_cast<uint4 *>(row + c) =
          make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                     pack_bf16(x[6], x[7]));
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (c + q < d) row[c + q] = __float2bfloat16_rn(x[q]);
  }
}
__device__ __forceinline__ void store8(float *row, int c, int d, bool vec, const float (&x)[8]) {
  if (vec) {
    if (c < d) {
      *reinterpret_cast<float4 *>(row + c) = make_float4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<float4 *>(row + c + 4) = make_float4(x[4], x[5], x[6], x[7]);
    }
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (c + q < d) row[c + q] = x[q];
  }
}
// Four codes as fp32: a code and 128 in the last digits of 2^23, less both.
__device__ __forceinline__ void four_codes(uint32_t w, float *c) {
  w ^= 0x80808080u;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    c[q] = __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 + q)) - 8388736.f;
}
// codes times their group's scale, the values that the checkpoint stands for
__device__ __forceinline__ void load_codes(const signed char *codes, const float *scales, int c,
                                           int d, bool vec, float (&x)[8]) {
  if (vec) {
    const uint2 w = c < d ? *reinterpret_cast<const uint2 *>(codes + c) : make_uint2(0, 0);
    const float s = c < d ? scales[c / kGroup] : 0.f;
    four_codes(w.x, x);
    four_codes(w.y, x + 4);
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] *= s;
  } else {
    const float s = c < d ? scales[c / kGroup] : 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = c + q < d ? (float)codes[c + q] * s : 0.f;
  }
}

__device__ __forceinline__ float rounded(float x, const float *) { return x; }
__device__ __forceinline__ float rounded(float x, const __nv_bfloat16 *) {
  return __bfloat162float(__float2bfloat16_rn(x));
}

// What the threads of a row share: WARPS warps, the block's `group`th so many.
template <int WARPS>
struct RowSum {
  float *part;  // [2][WARPS] shared, WARPS > 1
  int group;
  int turn = 0;
  __device__ float operator()(float v) {
    v = warp_sum(v);
    if (WARPS == 1) return v;
    float *p = part + turn * WARPS;  // two turns: the last sum may still be read
    turn ^= 1;
    if (threadIdx.x % 32 == 0) p[threadIdx.x / 32 % WARPS] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * WARPS) : "memory");
    v = 0.f;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) v += p[k];
    return v;
  }
};

// The normalised row without its parameters, in place of the row, and 1 /
// spread; the hardware's reciprocal square root as in the residual stream's
// operator.  `length2`: ScaleNorm's sum of squares.
template <int NC, int WARPS>
__device__ __forceinline__ float normalise(float (&x)[NC][8], int kind, int t, int d, float eps,
                                           RowSum<WARPS> &sum, float *length2) {
  const float inv_d = 1.0f / (float)d;
  float s = 0.f;
  if (kind == FLASH_GAU_NORM_LAYER) {
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int q = 0; q < 8; ++q) s += x[k][q];
    const float mean = sum(s) * inv_d;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = (k * 32 * WARPS + t) * 8;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        x[k][q] = c + q < d ? x[k][q] - mean : 0.f;
        s = fmaf(x[k][q], x[k][q], s);
      }
    }
    s = sum(s);
    s = rsqrtf(fmaf(s, inv_d, eps));
  } else {
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int q = 0; q < 8; ++q) s = fmaf(x[k][q], x[k][q], s);
    s = sum(s);
    *length2 = s;
    const float r = rsqrtf(s), most = 1.0f / eps;
    s = r > most ? most : r;  // not a number where the row is not
  }
#pragma unroll
  for (int k = 0; k < NC; ++k)
#pragma unroll
    for (int q = 0; q < 8; ++q) x[k][q] *= s;
  return s;
}

// n = u * g + b in the io type
template <int NC, int WARPS, typename T>
__device__ __forceinline__ void store_norm(const float (&u)[NC][8], const CheckpointArgs &a, int t,
                                           T *n, bool vec) {
  const bool layer = a.norm == FLASH_GAU_NORM_LAYER;
  const float g1 = layer ? 0.f : a.norm_g[0];
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const int c = (k * 32 * WARPS + t) * 8;
    if (c >= a.d) continue;
    float v[8], g[8], b[8];
    if (layer) {
      load8(a.norm_g, c, a.d, a.vec_param, g);
      if (a.norm_b) load8(a.norm_b, c, a.d, a.vec_param, b);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q)
      v[q] = layer ? fmaf(u[k][q], g[q], a.norm_b ? b[q] : 0.f) : u[k][q] * g1;
    store8(n, c, a.d, vec, v);
  }
}

// ------------------------------------------------------------------- pack --
template <typename T, int NC, int WARPS>
__global__ void __launch_bounds__(32 * (WARPS > 4 ? WARPS : 4)) pack_kernel(const CheckpointArgs a) {
  __shared__ float part[2 * WARPS];
  RowSum<WARPS> sum{part, 0};
  const int t = threadIdx.x % (32 * WARPS);
  const long long m = (long long)blockIdx.x * (WARPS == 1 ? 4 : 1) + threadIdx.x / (32 * WARPS);
  ptx::griddep_wait();
  if (m >= a.M) return;  // whole warps, and with four warps whole blocks
  const long long at = m * a.d;
  const T *h = static_cast<const T *>(a.h) + at;
  const T *y = a.y ? static_cast<const T *>(a.y) + at : nullptr;
  const bool vec = a.vec;
  float x[NC][8];
#pragma unroll
  for (int k = 0; k < NC; ++k) load8(h, (k * 32 * WARPS + t) * 8, a.d, vec, x[k]);
  if (y) {
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      float v[8];
      load8(y, (k * 32 * WARPS + t) * 8, a.d, vec, v);
#pragma unroll
      for (int q = 0; q < 8; ++q) x[k][q] += v[q];
    }
  }
  if (a.r) {
    T *r = static_cast<T *>(a.r) + at;
#pragma unroll
    for (int k = 0; k < NC; ++k) store8(r, (k * 32 * WARPS + t) * 8, a.d, vec, x[k]);
  }
  signed char *codes = a.codes + at;
  float *scales = a.scales + m * a.groups;
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const int c = (k * 32 * WARPS + t) * 8;
    float v[8], top = 0.f;
    bool odd = false;  // not a number: a maximum would pass over it
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      v[q] = rounded(x[k][q], h);
      top = fmaxf(top, fabsf(v[q]));
      odd |= v[q] != v[q];
    }
    if (odd) top = __int_as_float(0x7fffffff);
    // as integers, magnitudes keep their order and NaN lies above infinity
    int big = __float_as_int(top);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) big = max(big, __shfl_xor_sync(kAll, big, o));
    top = __int_as_float(big);
    if (c >= a.d) continue;
    const float s = top < kLeast ? 0.f : top * (1.f / 127.f);
    const float inv = s > 0.f && s < __int_as_float(0x7f800000) ? __fdiv_rn(1.f, s) : 0.f;
    if (t % 16 == 0) scales[c / kGroup] = s;
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      // in a group with an infinity or NaN every code is zero: it restores to NaN
      float e = inv > 0.f ? rintf(v[q] * inv) : 0.f;
      const float rest = inv > 0.f ? fmaf(-e, s, v[q]) : 0.f;
      const float twice = 2.f * fabsf(rest);
      const int i = (int)e;
      const int move = twice > s || (twice == s && (i & 1)) ? (rest > 0.f ? 1 : -1) : 0;
      w[q / 4] |= ((uint32_t)(i + move) & 0xffu) << (8 * (q & 3));
    }
    if (vec) {
      *reinterpret_cast<uint2 *>(codes + c) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (c + q < a.d) codes[c + q] = (signed char)(w[q / 4] >> (8 * (q & 3)));
    }
  }
  if (a.n) {
    float length2;
    normalise<NC, WARPS>(x, a.norm, t, a.d, a.eps, sum, &length2);
    store_norm<NC, WARPS>(x, a, t, static_cast<T *>(a.n) + at, vec);
  }
}

// ---------------------------------------------------------------- restore --
template <typename T, int NC, int WARPS>
__global__ void __launch_bounds__(32 * (WARPS > 4 ? WARPS : 4)) restore_kernel(const CheckpointArgs a) {
  __shared__ float part[2 * WARPS];
  RowSum<WARPS> sum{part, 0};
  const int t = threadIdx.x % (32 * WARPS);
  const long long m = (long long)blockIdx.x * (WARPS == 1 ? 4 : 1) + threadIdx.x / (32 * WARPS);
  ptx::griddep_wait();
  if (m >= a.M) return;
  const long long at = m * a.d;
  const bool vec = a.vec;
  float x[NC][8];
#pragma unroll
  for (int k = 0; k < NC; ++k)
    load_codes(a.codes + at, a.scales + m * a.groups, (k * 32 * WARPS + t) * 8, a.d, vec, x[k]);
  if (a.r) {
    T *r = static_cast<T *>(a.r) + at;
#pragma unroll
    for (int k = 0; k < NC; ++k) store8(r, (k * 32 * WARPS + t) * 8, a.d, vec, x[k]);
  }
  if (a.n) {
    float length2;
    normalise<NC, WARPS>(x, a.norm, t, a.d, a.eps, sum, &length2);
    store_norm<NC, WARPS>(x, a, t, static_cast<T *>(a.n) + at, vec);
  }
}

// --------------------------------------------------------------- backward --
// With u the normalised row without its parameters, i = 1 / spread and w = g
// dn: LayerNorm dx = i (w - mean(w) - u mean(w u)), ScaleNorm dx = i (w - u
// sum(w u)), the second term only where |x| > eps.  The row's warps walk rows
// and keep the column sums of dn u and dn in registers; each block leaves its
// sums in the workspace and a second kernel adds the blocks up in their order.
//
// A thread's column sums alone are 16 registers for each 8 columns, so few warps
// fit, and few loads with them (registers alone: 59 us at 16384 x 768 bf16, 1.0
// TB/s).  In rows on 16-byte boundaries each thread therefore brings its part of
// the next row into shared memory by asynchronous copies while it works on this
// one: no registers, no barrier, since it reads what it copied itself.

// dx in place of w = dn's row, from the row's values x, with the column sums.
template <int NC, int WARPS>
__device__ __forceinline__ void row_gradient(const CheckpointArgs &a, float (&x)[NC][8],
                                             float (&w)[NC][8], float (&sg)[NC][8],
                                             float (&sb)[NC][8], float &s1, int t,
                                             RowSum<WARPS> &sum) {
  const bool layer = a.norm == FLASH_GAU_NORM_LAYER;
  const float inv_d = 1.0f / (float)a.d;
  float length2 = 0.f;
  const float inv = normalise<NC, WARPS>(x, a.norm, t, a.d, a.eps, sum, &length2);
  float sw = 0.f, swu = 0.f;
  if (layer) {
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = (k * 32 * WARPS + t) * 8;
      float g[8];
      load8(a.norm_g, c, a.d, a.vec_param, g);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        sg[k][q] = fmaf(w[k][q], x[k][q], sg[k][q]);
        sb[k][q] += w[k][q];
        w[k][q] *= g[q];
        sw += w[k][q];
        swu = fmaf(w[k][q], x[k][q], swu);
      }
    }
    swu = sum(swu) * inv_d;
    sw = sum(sw) * inv_d;
  } else {
    const float g = a.norm_g[0];
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int q = 0; q < 8; ++q) swu = fmaf(w[k][q], x[k][q], swu);
    s1 += swu;
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int q = 0; q < 8; ++q) w[k][q] *= g;
    swu = length2 > a.eps * a.eps ? sum(swu) * g : 0.f;
  }
#pragma unroll
  for (int k = 0; k < NC; ++k)
#pragma unroll
    for (int q = 0; q < 8; ++q) w[k][q] = inv * (w[k][q] - sw - x[k][q] * swu);
}

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

__device__ __forceinline__ void widen(const uint4 *p, int step, float (&x)[8], const float *) {
  const uint4 v[2] = {p[0], p[step]};
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    x[4 * q] = __uint_as_float(v[q].x);
    x[4 * q + 1] = __uint_as_float(v[q].y);
    x[4 * q + 2] = __uint_as_float(v[q].z);
    x[4 * q + 3] = __uint_as_float(v[q].w);
  }
}
__device__ __forceinline__ void widen(const uint4 *p, int, float (&x)[8], const __nv_bfloat16 *) {
  const uint32_t v[4] = {p->x, p->y, p->z, p->w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float2 f = unpack_bf16(v[q]);
    x[2 * q] = f.x;
    x[2 * q + 1] = f.y;
  }
}

// Shared memory of a step: for each of a thread's NC runs of 8 columns dn, dr,
// codes and the scale, the threads' side by side.
template <typename T, int NC, int THREADS>
struct Ring {
  static constexpr int kPieces = sizeof(T) * 8 / 16;  // 16-byte pieces of a run
  static constexpr int kRun = THREADS * (2 * 16 * kPieces + 8 + 4);
  static constexpr int kStep = NC * kRun;
  static constexpr int kBytes = 2 * kStep;
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
  RowSum<WARPS> sum{part + group * 2 * WARPS, group};
  float sg[NC][8], sb[NC][8], s1 = 0.f;
#pragma unroll
  for (int k = 0; k < NC; ++k)
#pragma unroll
    for (int q = 0; q < 8; ++q) sg[k][q] = sb[k][q] = 0.f;
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
  fetch(m, 0);
  for (int turn = 0; m < a.M; m += step, turn ^= 1) {
    fetch(m + step, turn ^ 1);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    const R r{shared + turn * R::kStep};
    float x[NC][8], w[NC][8];
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const bool in = (k * 32 * WARPS + t) * 8 < a.d;
      const uint2 v = in ? *r.codes(k) : make_uint2(0, 0);
      const float s = in ? *r.scale(k) : 0.f;
      four_codes(v.x, x[k]);
      four_codes(v.y, x[k] + 4);
      if (in) widen(r.dn(k), THREADS, w[k], static_cast<const T *>(nullptr));
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        x[k][q] *= s;
        if (!in) w[k][q] = 0.f;
      }
    }
    row_gradient<NC, WARPS>(a, x, w, sg, sb, s1, t, sum);
    T *dh = static_cast<T *>(a.dh) + m * a.d;
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = (k * 32 * WARPS + t) * 8;
      if (c >= a.d) continue;
      if (a.dr) {
        float v[8];
        widen(r.dr(k), THREADS, v, static_cast<const T *>(nullptr));
#pragma unroll
        for (int q = 0; q < 8; ++q) w[k][q] += v[q];
      }
      store8(dh, c, a.d, true, w[k]);
    }
  }
  if (!a.part) return;
  if (a.norm != FLASH_GAU_NORM_LAYER) {
    s1 = warp_sum(s1);
    if (threadIdx.x % 32 == 0)
      a.part[(long long)blockIdx.x * (THREADS / 32) + threadIdx.x / 32] = s1;
    return;
  }
  // the block's sums: every group's in shared memory, then column by column
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  float *cols = reinterpret_cast<float *>(shared);
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const int c = (k * 32 * WARPS + t) * 8;
    if (c >= a.d) continue;
    store8(cols + (long long)group * 2 * a.d, c, a.d, true, sg[k]);
    store8(cols + (long long)group * 2 * a.d + a.d, c, a.d, true, sb[k]);
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

// Any rows, element by element where they are not on boundaries.
template <typename T, int NC, int WARPS>
__global__ void __launch_bounds__(32 * (WARPS > 4 ? WARPS : 4)) backward_kernel(const CheckpointArgs a) {
  constexpr int kThreads = 32 * (WARPS > 4 ? WARPS : 4), rows = kThreads / 32 / WARPS;
  __shared__ float part[2 * WARPS];
  extern __shared__ float cols[];  // [2][d], one row of warps after another
  RowSum<WARPS> sum{part, 0};
  const int t = threadIdx.x % (32 * WARPS);
  const bool layer = a.norm == FLASH_GAU_NORM_LAYER, vec = a.vec;
  float sg[NC][8], sb[NC][8], s1 = 0.f;
#pragma unroll
  for (int k = 0; k < NC; ++k)
#pragma unroll
    for (int q = 0; q < 8; ++q) sg[k][q] = sb[k][q] = 0.f;
  ptx::griddep_wait();
  for (long long m = (long long)blockIdx.x * rows + threadIdx.x / (32 * WARPS); m < a.M;
       m += (long long)gridDim.x * rows) {
    const long long at = m * a.d;
    float x[NC][8], w[NC][8];
#pragma unroll
    for (int k = 0; k < NC; ++k)
      load_codes(a.codes + at, a.scales + m * a.groups, (k * 32 * WARPS + t) * 8, a.d, vec, x[k]);
#pragma unroll
    for (int k = 0; k < NC; ++k)
      load8(static_cast<const T *>(a.dn) + at, (k * 32 * WARPS + t) * 8, a.d, vec, w[k]);
    row_gradient<NC, WARPS>(a, x, w, sg, sb, s1, t, sum);
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = (k * 32 * WARPS + t) * 8;
      if (a.dr) {
        float v[8];
        load8(static_cast<const T *>(a.dr) + at, c, a.d, vec, v);
#pragma unroll
        for (int q = 0; q < 8; ++q) w[k][q] += v[q];
      }
      store8(static_cast<T *>(a.dh) + at, c, a.d, vec, w[k]);
    }
  }
  if (!a.part) return;
  if (!layer) {
    s1 = warp_sum(s1);
    if (threadIdx.x % 32 == 0)
      a.part[(long long)blockIdx.x * (kThreads / 32) + threadIdx.x / 32] = s1;
    return;
  }
  for (int turn = 0; turn < rows; ++turn) {
    if (threadIdx.x / (32 * WARPS) == turn) {
#pragma unroll
      for (int k = 0; k < NC; ++k)
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int c = (k * 32 * WARPS + t) * 8 + q;
          if (c < a.d) {
            cols[c] = turn ? cols[c] + sg[k][q] : sg[k][q];
            cols[a.d + c] = turn ? cols[a.d + c] + sb[k][q] : sb[k][q];
          }
        }
    }
    __syncthreads();
  }
  float *to = a.part + (long long)blockIdx.x * 2 * a.d;
  for (int c = threadIdx.x; c < 2 * a.d; c += kThreads) to[c] = cols[c];
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

enum { kPack, kRestore, kBackward };

template <int WHAT, typename T, int NC, int WARPS>
cudaError_t launch(const CheckpointArgs &a, unsigned grid, cudaStream_t stream) {
  constexpr int kThreads = 32 * (WARPS > 4 ? WARPS : 4);
  if constexpr (WHAT == kPack) {
    return launch_pdl(pack_kernel<T, NC, WARPS>, dim3(grid), dim3(kThreads), 0, stream, a);
  } else if constexpr (WHAT == kRestore) {
    return launch_pdl(restore_kernel<T, NC, WARPS>, dim3(grid), dim3(kThreads), 0, stream, a);
  } else {
    const size_t smem = a.part && a.norm == FLASH_GAU_NORM_LAYER ? 2 * a.d * sizeof(float) : 0;
    if (smem > 48 * 1024) {
      const cudaError_t err = cudaFuncSetAttribute(
          backward_kernel<T, NC, WARPS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (err != cudaSuccess) return err;
    }
    return launch_pdl(backward_kernel<T, NC, WARPS>, dim3(grid), dim3(kThreads), smem, stream, a);
  }
}

// Warps of a row: one up to 1024 columns, four up to 4096, eight beyond.
int row_warps(int d) { return d <= 1024 ? 1 : d <= 4096 ? 4 : 8; }

template <int WHAT, typename T>
cudaError_t dispatch(const CheckpointArgs &a, unsigned most_blocks, cudaStream_t stream) {
  const int rows = row_warps(a.d) == 1 ? 4 : 1;
  const long long blocks = (a.M + rows - 1) / rows;
  const unsigned grid = (unsigned)(most_blocks && blocks > most_blocks ? most_blocks : blocks);
  if (a.d <= 256) return launch<WHAT, T, 1, 1>(a, grid, stream);
  if (a.d <= 512) return launch<WHAT, T, 2, 1>(a, grid, stream);
  if (a.d <= 768) return launch<WHAT, T, 3, 1>(a, grid, stream);
  if (a.d <= 1024) return launch<WHAT, T, 4, 1>(a, grid, stream);
  if (a.d <= 2048) return launch<WHAT, T, 2, 4>(a, grid, stream);
  if (a.d <= 4096) return launch<WHAT, T, 4, 4>(a, grid, stream);
  return launch<WHAT, T, 4, 8>(a, grid, stream);
}

template <int WHAT>
cudaError_t dispatch(const CheckpointArgs &a, int dtype, unsigned most_blocks,
                     cudaStream_t stream) {
  return dtype == FLASH_GAU_BF16 ? dispatch<WHAT, __nv_bfloat16>(a, most_blocks, stream)
                                 : dispatch<WHAT, float>(a, most_blocks, stream);
}

// The form with copies ahead, one block an SM.  Returns the blocks' number and
// their warps.
struct Grid {
  int blocks, warps;
};
template <typename T, int NC, int WARPS>
cudaError_t launch_ring(const CheckpointArgs &a, int num_sms, cudaStream_t stream, Grid *g) {
  // as many as the column sums' registers leave, in whole rows, and two steps' memory
  constexpr int kMost = NC < 4 ? 512 : WARPS <= 4 ? 384 : 256;
  constexpr int kThreads = Ring<T, NC, kMost>::kBytes <= 200 * 1024 ? kMost : 256;
  constexpr int kRows = kThreads / 32 / WARPS;
  auto kernel = ring_backward_kernel<T, NC, WARPS, kThreads>;
  // two steps, or the groups' column sums
  const size_t sums = (size_t)kRows * 2 * a.d * sizeof(float);
  const size_t smem = sums > Ring<T, NC, kThreads>::kBytes ? sums : Ring<T, NC, kThreads>::kBytes;
  const cudaError_t err =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
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
                        (const void *)a.dh})
    a.vec = a.vec && on(p, 16);
  a.vec_param = a.d % 8 == 0 && on(a.norm_g, 16) && on(a.norm_b, 16);
  return a;
}

}  // namespace

cudaError_t checkpoint_pack(const CheckpointArgs &a, int dtype, cudaStream_t stream) {
  return dispatch<kPack>(finish(a), dtype, 0, stream);
}

cudaError_t checkpoint_restore(const CheckpointArgs &a, int dtype, cudaStream_t stream) {
  return dispatch<kRestore>(finish(a), dtype, 0, stream);
}

size_t checkpoint_part_bytes(int d) {
  return (size_t)kCheckpointBlocks * 2 * (d < 8 ? 8 : d) * sizeof(float);
}

cudaError_t checkpoint_backward(const CheckpointArgs &args, float *dg, float *db, int dtype,
                                int num_sms, cudaStream_t stream) {
  CheckpointArgs a = finish(args);
  if (!dg && !db) a.part = nullptr;
  Grid g;
  cudaError_t err;
  if (a.vec) {
    err = dtype == FLASH_GAU_BF16 ? dispatch_ring<__nv_bfloat16>(a, num_sms, stream, &g)
                                  : dispatch_ring<float>(a, num_sms, stream, &g);
  } else {
    err = dispatch<kBackward>(a, dtype, kCheckpointBlocks, stream);
    const int warps = row_warps(a.d), rows = warps == 1 ? 4 : 1;
    const long long all = (a.M + rows - 1) / rows;
    g = {(int)(all < kCheckpointBlocks ? all : kCheckpointBlocks), warps > 4 ? warps : 4};
  }
  if (err != cudaSuccess || !a.part) return err;
  if (a.norm == FLASH_GAU_NORM_LAYER)
    return launch_pdl(join_columns_kernel, dim3((2 * a.d + 31) / 32), dim3(1024), 0, stream,
                      a.part, g.blocks, a.d, dg, db);
  return launch_pdl(join_scalar_kernel, dim3(1), dim3(1024), 0, stream, a.part,
                    g.blocks * g.warps, dg);
}

}  // namespace flashgau
