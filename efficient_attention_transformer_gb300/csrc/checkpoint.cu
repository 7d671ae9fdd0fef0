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
#include "packed_f32.cuh"
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

__device__ __forceinline__ uint32_t pack_bf16(f2 v) {
  const float2 f = split(v);
  const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ f2 unpack_bf16(uint32_t w) {
  return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// Eight columns of a row from column c on, in pairs; `vec`: rows are whole
// vectors on their boundaries.  Columns behind d are zero and not stored.
struct Eight {
  f2 v[4];
  __device__ float get(int q) const {
    const float2 f = split(v[q / 2]);
    return q % 2 ? f.y : f.x;
  }
  __device__ void of(const float (&x)[8]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = pair(x[2 * q], x[2 * q + 1]);
  }
  __device__ void zero_from(int n) {  // columns n .. 7
    float x[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = q < n ? get(q) : 0.f;
    of(x);
  }
};

__device__ __forceinline__ Eight load8(const __nv_bfloat16 *row, int c, int d, bool vec) {
  Eight e;
  if (vec) {
    const uint4 w = c < d ? *reinterpret_cast<const uint4 *>(row + c) : make_uint4(0, 0, 0, 0);
    e.v[0] = unpack_bf16(w.x);
    e.v[1] = unpack_bf16(w.y);
    e.v[2] = unpack_bf16(w.z);
    e.v[3] = unpack_bf16(w.w);
  } else {
    float x[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = c + q < d ? __bfloat162float(row[c + q]) : 0.f;
    e.of(x);
  }
  return e;
}
__device__ __forceinline__ Eight load8(const float *row, int c, int d, bool vec) {
  Eight e;
  if (vec) {
    ulonglong2 w[2] = {make_ulonglong2(0, 0), make_ulonglong2(0, 0)};
    if (c < d) {
      w[0] = *reinterpret_cast<const ulonglong2 *>(row + c);
      w[1] = *reinterpret_cast<const ulonglong2 *>(row + c + 4);
    }
    e.v[0] = w[0].x;
    e.v[1] = w[0].y;
    e.v[2] = w[1].x;
    e.v[3] = w[1].y;
  } else {
    float x[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = c + q < d ? row[c + q] : 0.f;
    e.of(x);
  }
  return e;
}
__device__ __forceinline__ void store8(__nv_bfloat16 *row, int c, int d, bool vec, const Eight &e) {
  if (vec) {
    if (c < d)
      *reinterpret_cast<uint4 *>(row + c) = make_uint4(pack_bf16(e.v[0]), pack_bf16(e.v[1]),
                                                       pack_bf16(e.v[2]), pack_bf16(e.v[3]));
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (c + q < d) row[c + q] = __float2bfloat16_rn(e.get(q));
  }
}
__device__ __forceinline__ void store8(float *row, int c, int d, bool vec, const Eight &e) {
  if (vec) {
    if (c < d) {
      *reinterpret_cast<ulonglong2 *>(row + c) = make_ulonglong2(e.v[0], e.v[1]);
      *reinterpret_cast<ulonglong2 *>(row + c + 4) = make_ulonglong2(e.v[2], e.v[3]);
    }
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (c + q < d) row[c + q] = e.get(q);
  }
}

// Eight codes times their group's scale, the values that the checkpoint stands
// for.  A code as fp32: it and 128 in the last digits of 2^23, less both.
__device__ __forceinline__ Eight times_scale(uint2 codes, float s) {
  const uint32_t w[2] = {codes.x ^ 0x80808080u, codes.y ^ 0x80808080u};
  Eight e;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const f2 c = pair(__uint_as_float(__byte_perm(w[q / 2], 0x4b000000u, 0x7440 + 2 * (q % 2))),
                      __uint_as_float(__byte_perm(w[q / 2], 0x4b000000u, 0x7441 + 2 * (q % 2))));
    e.v[q] = mul2(add2(c, both(-8388736.f)), both(s));
  }
  return e;
}
struct Packed {
  uint2 codes;
  float scale;
  __device__ void load(const signed char *row, const float *scales, int c, int d, bool vec) {
    codes = make_uint2(0, 0);
    scale = c < d ? scales[c / kGroup] : 0.f;
    if (vec) {
      if (c < d) codes = *reinterpret_cast<const uint2 *>(row + c);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const uint32_t b = c + q < d ? (uint32_t)(uint8_t)row[c + q] : 0u;
        (q < 4 ? codes.x : codes.y) |= b << (8 * (q & 3));
      }
    }
  }
  __device__ Eight values(int c, int d, bool vec) const {
    Eight e = times_scale(codes, scale);
    if (!vec && c + 8 > d) e.zero_from(d - c);  // 0 times a scale that is not finite
    return e;
  }
};

// The values as they are stored, and the bits of the largest magnitude: as whole
// numbers magnitudes keep their order, NaN above infinity.
__device__ __forceinline__ Eight stored(const Eight &e, const float *, uint32_t *top) {
  uint32_t m = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) m = max(m, __float_as_uint(e.get(q)) & 0x7fffffffu);
  *top = m;
  return e;
}
__device__ __forceinline__ Eight stored(const Eight &e, const __nv_bfloat16 *, uint32_t *top) {
  Eight r;
  uint32_t m = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t w = pack_bf16(e.v[q]);
    m = __vmaxu2(m, w & 0x7fff7fffu);
    r.v[q] = unpack_bf16(w);
  }
  *top = max(m << 16, m & 0xffff0000u);
  return r;
}

// Codes of eight values.  t = v / s to the nearest whole number in the digits of
// 1.5 * 2^23 is at most one off; the remainder v - t s is exact, and where one of
// eight is half a scale or more, each is looked at: it moves above a half, and
// from an odd number at a half.
__device__ __forceinline__ uint2 codes_of(const Eight &e, float s) {
  const float magic = 12582912.f;
  if (!(s > 0.f && s < __int_as_float(0x7f800000))) return make_uint2(0, 0);  // restores 0 or NaN
  const float inv = __fdiv_rn(1.f, s), half = 0.5f * s;
  f2 t[4], rest[4];
  float most = 0.f;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    t[q] = fma2(e.v[q], both(inv), both(magic));
    rest[q] = fma2(add2(both(magic), mul2(t[q], both(-1.f))), both(s), e.v[q]);
    const float2 f = split(rest[q]);
    most = fmaxf(most, fmaxf(fabsf(f.x), fabsf(f.y)));
  }
  uint32_t c[8];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float2 f = split(t[q]);
    c[2 * q] = __float_as_uint(f.x);
    c[2 * q + 1] = __float_as_uint(f.y);
  }
  if (most >= half) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float2 f = split(rest[q / 2]);
      const float x = q % 2 ? f.y : f.x;
      if (fabsf(x) > half || (fabsf(x) == half && (c[q] & 1))) c[q] += x > 0.f ? 1 : -1;
    }
  }
  // the last byte of each
  return make_uint2(__byte_perm(__byte_perm(c[0], c[1], 0x40), __byte_perm(c[2], c[3], 0x40), 0x5410),
                    __byte_perm(__byte_perm(c[4], c[5], 0x40), __byte_perm(c[6], c[7], 0x40), 0x5410));
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
__device__ __forceinline__ float normalise(Eight (&x)[NC], int kind, int t, int d, float eps,
                                           RowSum<WARPS> &row_sum, float *length2) {
  f2 s = 0;
  float scale;
  if (kind == FLASH_GAU_NORM_LAYER) {
    const float inv_d = 1.0f / (float)d;
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int q = 0; q < 4; ++q) s = add2(s, x[k].v[q]);
    const float mean = row_sum(sum(s)) * inv_d;
    s = 0;
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = (k * 32 * WARPS + t) * 8;
      const f2 less = both(c < d ? -mean : 0.f);
#pragma unroll
      for (int q = 0; q < 4; ++q) x[k].v[q] = add2(x[k].v[q], less);
      if (c < d && c + 8 > d) x[k].zero_from(d - c);
#pragma unroll
      for (int q = 0; q < 4; ++q) s = fma2(x[k].v[q], x[k].v[q], s);
    }
    scale = rsqrtf(fmaf(row_sum(sum(s)), inv_d, eps));
  } else {
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int q = 0; q < 4; ++q) s = fma2(x[k].v[q], x[k].v[q], s);
    *length2 = row_sum(sum(s));
    const float r = rsqrtf(*length2), most = 1.0f / eps;
    scale = r > most ? most : r;  // not a number where the row is not
  }
#pragma unroll
  for (int k = 0; k < NC; ++k)
#pragma unroll
    for (int q = 0; q < 4; ++q) x[k].v[q] = mul2(x[k].v[q], both(scale));
  return scale;
}

// n = u * g + b in the io type
template <int NC, int WARPS, typename T>
__device__ __forceinline__ void store_norm(const Eight (&u)[NC], const CheckpointArgs &a, int t,
                                           T *n) {
  const bool layer = a.norm == FLASH_GAU_NORM_LAYER;
  const f2 g1 = both(layer ? 0.f : a.norm_g[0]);
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const int c = (k * 32 * WARPS + t) * 8;
    if (c >= a.d) continue;
    Eight v;
    if (layer) {
      const Eight g = load8(a.norm_g, c, a.d, a.vec_param);
      Eight b = {{0, 0, 0, 0}};
      if (a.norm_b) b = load8(a.norm_b, c, a.d, a.vec_param);
#pragma unroll
      for (int q = 0; q < 4; ++q) v.v[q] = fma2(u[k].v[q], g.v[q], b.v[q]);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) v.v[q] = mul2(u[k].v[q], g1);
    }
    store8(n, c, a.d, a.vec, v);
  }
}

// ------------------------------------------------------------------- pack --
template <typename T, int NC, int WARPS>
__global__ void __launch_bounds__(32 * (WARPS > 4 ? WARPS : 4)) pack_kernel(const CheckpointArgs a) {
  __shared__ float part[2 * WARPS];
  RowSum<WARPS> row_sum{part, 0};
  const int t = threadIdx.x % (32 * WARPS);
  const long long m = (long long)blockIdx.x * (WARPS == 1 ? 4 : 1) + threadIdx.x / (32 * WARPS);
  ptx::griddep_wait();
  if (m >= a.M) return;  // whole warps, and with more than one whole blocks
  const long long at = m * a.d;
  const T *h = static_cast<const T *>(a.h) + at;
  const T *y = a.y ? static_cast<const T *>(a.y) + at : nullptr;
  const bool vec = a.vec;
  Eight x[NC];
#pragma unroll
  for (int k = 0; k < NC; ++k) x[k] = load8(h, (k * 32 * WARPS + t) * 8, a.d, vec);
  if (y) {
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const Eight v = load8(y, (k * 32 * WARPS + t) * 8, a.d, vec);
#pragma unroll
      for (int q = 0; q < 4; ++q) x[k].v[q] = add2(x[k].v[q], v.v[q]);
    }
  }
  T *r = a.r ? static_cast<T *>(a.r) + at : nullptr;
  signed char *codes = a.codes + at;
  float *scales = a.scales + m * a.groups;
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const int c = (k * 32 * WARPS + t) * 8;
    if (r) store8(r, c, a.d, vec, x[k]);
    uint32_t top;
    const Eight v = stored(x[k], h, &top);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(kAll, top, o));
    if (c >= a.d) continue;
    const float big = __uint_as_float(top), s = big < kLeast ? 0.f : big * (1.f / 127.f);
    if (t % 16 == 0) scales[c / kGroup] = s;
    const uint2 w = codes_of(v, s);
    if (vec) {
      *reinterpret_cast<uint2 *>(codes + c) = w;
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (c + q < a.d) codes[c + q] = (signed char)((q < 4 ? w.x : w.y) >> (8 * (q & 3)));
    }
  }
  if (a.n) {
    float length2;
    normalise<NC, WARPS>(x, a.norm, t, a.d, a.eps, row_sum, &length2);
    store_norm<NC, WARPS>(x, a, t, static_cast<T *>(a.n) + at);
  }
}

// ---------------------------------------------------------------- restore --
// (two or four rows a warp with all their codes asked for at first: 13.0 and 17.3
// us for 12.3 at 16384 x 768 bf16)
template <typename T, int NC, int WARPS>
__global__ void __launch_bounds__(32 * (WARPS > 4 ? WARPS : 4)) restore_kernel(const CheckpointArgs a) {
  __shared__ float part[2 * WARPS];
  RowSum<WARPS> row_sum{part, 0};
  const int t = threadIdx.x % (32 * WARPS);
  const long long m = (long long)blockIdx.x * (WARPS == 1 ? 4 : 1) + threadIdx.x / (32 * WARPS);
  ptx::griddep_wait();
  if (m >= a.M) return;  // whole warps, and with more than one whole blocks
  const long long at = m * a.d;
  Packed p[NC];
#pragma unroll
  for (int k = 0; k < NC; ++k)
    p[k].load(a.codes + at, a.scales + m * a.groups, (k * 32 * WARPS + t) * 8, a.d, a.vec);
  Eight x[NC];
#pragma unroll
  for (int k = 0; k < NC; ++k) x[k] = p[k].values((k * 32 * WARPS + t) * 8, a.d, a.vec);
  if (a.r) {
    T *r = static_cast<T *>(a.r) + at;
#pragma unroll
    for (int k = 0; k < NC; ++k) store8(r, (k * 32 * WARPS + t) * 8, a.d, a.vec, x[k]);
  }
  if (a.n) {
    float length2;
    normalise<NC, WARPS>(x, a.norm, t, a.d, a.eps, row_sum, &length2);
    store_norm<NC, WARPS>(x, a, t, static_cast<T *>(a.n) + at);
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
// TB/s).  For a LayerNorm of rows on 16-byte boundaries each thread therefore
// brings its part of the next rows into shared memory by asynchronous copies while
// it works on this one: no registers, no barrier, since it reads what it copied
// itself.  A ScaleNorm has no column sums; its rows go through registers alone,
// with as many warps as those leave.

// dx in place of w = dn's row, from the row's values x, with the column sums (a
// ScaleNorm has none, its one g's sum is s1).
// gain(k): a LayerNorm's g of the thread's k-th run.
template <bool LAYER, int NC, int WARPS, typename G>
__device__ __forceinline__ void row_gradient(const CheckpointArgs &a, Eight (&x)[NC],
                                             Eight (&w)[NC], Eight *sg, Eight *sb,
                                             float &s1, int t, RowSum<WARPS> &row_sum,
                                             const G &gain) {
  float length2 = 0.f;
  const float inv = normalise<NC, WARPS>(
      x, LAYER ? FLASH_GAU_NORM_LAYER : FLASH_GAU_NORM_SCALE, t, a.d, a.eps, row_sum, &length2);
  f2 sw2 = 0, swu2 = 0;
  float sw = 0.f, swu;
  if constexpr (LAYER) {
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const Eight g = gain(k);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        sg[k].v[q] = fma2(w[k].v[q], x[k].v[q], sg[k].v[q]);
        sb[k].v[q] = add2(sb[k].v[q], w[k].v[q]);
        w[k].v[q] = mul2(w[k].v[q], g.v[q]);
        sw2 = add2(sw2, w[k].v[q]);
        swu2 = fma2(w[k].v[q], x[k].v[q], swu2);
      }
    }
    const float inv_d = 1.0f / (float)a.d;
    swu = row_sum(sum(swu2)) * inv_d;
    sw = row_sum(sum(sw2)) * inv_d;
  } else {
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int q = 0; q < 4; ++q) swu2 = fma2(w[k].v[q], x[k].v[q], swu2);
    swu = sum(swu2);
    s1 += swu;
    const float g = a.norm_g[0];
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int q = 0; q < 4; ++q) w[k].v[q] = mul2(w[k].v[q], both(g));
    swu = length2 > a.eps * a.eps ? row_sum(swu) * g : 0.f;
  }
#pragma unroll
  for (int k = 0; k < NC; ++k)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      w[k].v[q] = mul2(fma2(x[k].v[q], both(-swu), add2(w[k].v[q], both(-sw))), both(inv));
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
      const int c = (k * 32 * WARPS + t) * 8;
      return c < a.d ? load8(gains, c, a.d, true) : none;
    });
    T *dh = static_cast<T *>(a.dh) + m * a.d;
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = (k * 32 * WARPS + t) * 8;
      if (c >= a.d) continue;
      if (a.dr) {
        const Eight v = widen(r.dr(k), THREADS, static_cast<const T *>(nullptr));
#pragma unroll
        for (int q = 0; q < 4; ++q) w[k].v[q] = add2(w[k].v[q], v.v[q]);
      }
      store8(dh, c, a.d, true, w[k]);
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
template <typename T, int NC, int WARPS, bool LAYER>
__global__ void __launch_bounds__(32 * (WARPS > 4 ? WARPS : 4), LAYER ? 1 : WARPS > 4 ? 3 : 6)
backward_kernel(const CheckpointArgs a) {
  constexpr int kThreads = 32 * (WARPS > 4 ? WARPS : 4), rows = kThreads / 32 / WARPS;
  __shared__ float part[2 * WARPS];
  extern __shared__ float cols[];  // [2][d], one row of warps after another
  RowSum<WARPS> row_sum{part, 0};
  const int t = threadIdx.x % (32 * WARPS);
  const bool vec = a.vec;
  float s1 = 0.f;
  Eight sg[LAYER ? NC : 1] = {}, sb[LAYER ? NC : 1] = {};
  ptx::griddep_wait();
  for (long long m = (long long)blockIdx.x * rows + threadIdx.x / (32 * WARPS); m < a.M;
       m += (long long)gridDim.x * rows) {
    const long long at = m * a.d;
    Eight x[NC], w[NC];
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = (k * 32 * WARPS + t) * 8;
      Packed p;
      p.load(a.codes + at, a.scales + m * a.groups, c, a.d, vec);
      x[k] = p.values(c, a.d, vec);
    }
#pragma unroll
    for (int k = 0; k < NC; ++k)
      w[k] = load8(static_cast<const T *>(a.dn) + at, (k * 32 * WARPS + t) * 8, a.d, vec);
    row_gradient<LAYER, NC, WARPS>(a, x, w, sg, sb, s1, t, row_sum, [&](int k) {
      return load8(a.norm_g, (k * 32 * WARPS + t) * 8, a.d, a.vec_param);
    });
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = (k * 32 * WARPS + t) * 8;
      if (a.dr) {
        const Eight v = load8(static_cast<const T *>(a.dr) + at, c, a.d, vec);
#pragma unroll
        for (int q = 0; q < 4; ++q) w[k].v[q] = add2(w[k].v[q], v.v[q]);
      }
      store8(static_cast<T *>(a.dh) + at, c, a.d, vec, w[k]);
    }
  }
  if (!a.part) return;
  if constexpr (!LAYER) {
    s1 = warp_sum(s1);
    if (threadIdx.x % 32 == 0)
      a.part[(long long)blockIdx.x * (kThreads / 32) + threadIdx.x / 32] = s1;
  } else {
    for (int turn = 0; turn < rows; ++turn) {
      if (threadIdx.x / (32 * WARPS) == turn) {
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const int c = (k * 32 * WARPS + t) * 8 + q;
            if (c < a.d) {
              cols[c] = turn ? cols[c] + sg[k].get(q) : sg[k].get(q);
              cols[a.d + c] = turn ? cols[a.d + c] + sb[k].get(q) : sb[k].get(q);
            }
          }
      }
      __syncthreads();
    }
    float *to = a.part + (long long)blockIdx.x * 2 * a.d;
    for (int c = threadIdx.x; c < 2 * a.d; c += kThreads) to[c] = cols[c];
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

enum { kPack, kRestore, kBackward };

template <int WHAT, typename T, int NC, int WARPS>
cudaError_t launch(const CheckpointArgs &a, unsigned grid, cudaStream_t stream) {
  constexpr int kThreads = 32 * (WARPS > 4 ? WARPS : 4);
  if constexpr (WHAT == kPack) {
    return launch_pdl(pack_kernel<T, NC, WARPS>, dim3(grid), dim3(kThreads), 0, stream, a);
  } else if constexpr (WHAT == kRestore) {
    return launch_pdl(restore_kernel<T, NC, WARPS>, dim3(grid), dim3(kThreads), 0, stream, a);
  } else {
    if (a.norm != FLASH_GAU_NORM_LAYER)
      return launch_pdl(backward_kernel<T, NC, WARPS, false>, dim3(grid), dim3(kThreads), 0, stream,
                        a);
    const size_t smem = a.part ? 2 * a.d * sizeof(float) : 0;
    if (smem > 48 * 1024) {
      const cudaError_t err =
          allow_shared<backward_kernel<T, NC, WARPS, true>>(2 * kCheckpointMaxD * sizeof(float));
      if (err != cudaSuccess) return err;
    }
    return launch_pdl(backward_kernel<T, NC, WARPS, true>, dim3(grid), dim3(kThreads), smem, stream,
                      a);
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
    err = dispatch<kBackward>(a, dtype, most, stream);
    const int warps = row_warps(a.d), rows = warps == 1 ? 4 : 1;
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
