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
#pragma once

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

// Eight columns of a row from column c on, in pairs; VEC: rows are whole
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

// A row of an array of M rows: where it begins, and where the array ends.
struct RowAt {
  long long at, end;
  __device__ RowAt(long long m, long long M, int d) : at(m * d), end(M * d) {}
};

// Rows that are not on vectors' boundaries are read in the aligned vectors that
// hold them, shifted by what they are off (the same for a row's whole warp), and
// written in aligned vectors that a thread puts together from its own and its
// neighbour's columns; what is left at the ends of a warp's columns goes element
// by element.  (16384 x 767 bf16 against element by element throughout: pack 56 us
// for 73, restore 32 for 59, the norm's gradient 100 for 106; whole vectors take
// 20, 12 and 23 at 16384 x 768, and one kernel that asks which form it has 31.)

// The words of `w` from byte s < 16 on.
template <int N>
__device__ __forceinline__ void shifted(uint32_t (&w)[N], uint32_t s) {
  if (s & 8)
#pragma unroll
    for (int i = 0; i + 2 < N; ++i) w[i] = w[i + 2];
  if (s & 4)
#pragma unroll
    for (int i = 0; i + 1 < N; ++i) w[i] = w[i + 1];
#pragma unroll
  for (int i = 0; i + 1 < N; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 8 * (s & 3));
}
__device__ __forceinline__ uint32_t off(const void *p, uint32_t bytes) {
  return (uint32_t)reinterpret_cast<uintptr_t>(p) & (bytes - 1);
}
// whether the vectors that hold eight columns may reach out of the array
__device__ __forceinline__ bool at_edge(const RowAt &row, int c) {
  return row.at + c < 8 || row.at + c + 16 > row.end;
}

template <bool VEC>
__device__ __forceinline__ Eight load8(const __nv_bfloat16 *array, const RowAt &row, int c, int d) {
  Eight e = {{0, 0, 0, 0}};
  if (c >= d) return e;
  const __nv_bfloat16 *p = array + row.at + c;
  if (!VEC && at_edge(row, c)) {
    float x[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = c + q < d ? __bfloat162float(p[q]) : 0.f;
    e.of(x);
    return e;
  }
  const uint32_t s = VEC ? 0 : off(p, 16);
  const uint4 *v = reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(p) - s);
  uint4 a = v[0];
  if (s) {
    const uint4 b = v[1];
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    shifted(w, s);
    a = make_uint4(w[0], w[1], w[2], w[3]);
  }
  e = {{unpack_bf16(a.x), unpack_bf16(a.y), unpack_bf16(a.z), unpack_bf16(a.w)}};
  if (!VEC && c + 8 > d) e.zero_from(d - c);
  return e;
}
template <bool VEC>
__device__ __forceinline__ Eight load8(const float *array, const RowAt &row, int c, int d) {
  Eight e = {{0, 0, 0, 0}};
  if (c >= d) return e;
  const float *p = array + row.at + c;
  if constexpr (VEC) {
    const ulonglong2 a = reinterpret_cast<const ulonglong2 *>(p)[0];
    const ulonglong2 b = reinterpret_cast<const ulonglong2 *>(p)[1];
    return {{a.x, a.y, b.x, b.y}};
  }
  float x[8];
  if (at_edge(row, c)) {
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = c + q < d ? p[q] : 0.f;
  } else {
    const uint32_t s = off(p, 16);
    const float4 *v = reinterpret_cast<const float4 *>(reinterpret_cast<const char *>(p) - s);
    const float4 f[3] = {v[0], v[1], s ? v[2] : make_float4(0.f, 0.f, 0.f, 0.f)};
    uint32_t w[12];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      w[4 * i] = __float_as_uint(f[i].x);
      w[4 * i + 1] = __float_as_uint(f[i].y);
      w[4 * i + 2] = __float_as_uint(f[i].z);
      w[4 * i + 3] = __float_as_uint(f[i].w);
    }
    shifted(w, s);
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = __uint_as_float(w[q]);
  }
  e.of(x);
  if (c + 8 > d) e.zero_from(d - c);
  return e;
}

// For whole warps: a thread's columns may be its neighbour's to store.
template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16 *array, const RowAt &row, int c, int d,
                                       const Eight &e) {
  const uint4 o = make_uint4(pack_bf16(e.v[0]), pack_bf16(e.v[1]), pack_bf16(e.v[2]),
                             pack_bf16(e.v[3]));
  __nv_bfloat16 *p = array + row.at + c;
  const uint32_t s = VEC ? 0 : off(p, 16);
  const bool full = c + 8 <= d;
  if (s == 0 && (VEC ? c < d : full)) *reinterpret_cast<uint4 *>(p) = o;
  if constexpr (VEC) return;
  const int lane = threadIdx.x % 32;
  uint32_t w[8] = {o.x, o.y, o.z, o.w, o.x, o.y, o.z, o.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __shfl_up_sync(kAll, w[i], 1);
  const bool next = __shfl_down_sync(kAll, (int)full, 1) && lane < 31, mine = full && lane > 0;
  if (s && mine) {
    shifted(w, 16 - s);
    *reinterpret_cast<uint4 *>(reinterpret_cast<char *>(p) - s) =
        make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (s == 0 ? full : mine && next) return;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const bool done = s == 0 ? false : q >= 8 - (int)s / 2 ? next : mine;
    if (c + q < d && !done) p[q] = __float2bfloat16_rn(e.get(q));
  }
}
template <bool VEC>
__device__ __forceinline__ void store8(float *array, const RowAt &row, int c, int d,
                                       const Eight &e) {
  float *p = array + row.at + c;
  const uint32_t s = VEC ? 0 : off(p, 16);
  const bool full = c + 8 <= d;
  if (s == 0 && (VEC ? c < d : full)) {
    reinterpret_cast<ulonglong2 *>(p)[0] = make_ulonglong2(e.v[0], e.v[1]);
    reinterpret_cast<ulonglong2 *>(p)[1] = make_ulonglong2(e.v[2], e.v[3]);
  }
  if constexpr (VEC) return;
  const int lane = threadIdx.x % 32;
  uint32_t w[12];  // the neighbour's last four columns, then these
#pragma unroll
  for (int i = 0; i < 8; ++i) w[4 + i] = __float_as_uint(e.get(i));
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __shfl_up_sync(kAll, w[8 + i], 1);
  const bool next = __shfl_down_sync(kAll, (int)full, 1) && lane < 31, mine = full && lane > 0;
  if (s && full) {
    shifted(w, 16 - s);
    uint4 *v = reinterpret_cast<uint4 *>(reinterpret_cast<char *>(p) - s);
    if (mine) v[0] = make_uint4(w[0], w[1], w[2], w[3]);
    v[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
  if (s == 0 ? full : mine && next) return;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int tail = 8 - (int)s / 4;
    const bool done = s == 0 ? false : q >= tail ? next : q < tail - 4 ? mine : full;
    if (c + q < d && !done) p[q] = e.get(q);
  }
}
template <bool VEC>
__device__ __forceinline__ void store_codes(signed char *array, const RowAt &row, int c, int d,
                                            uint2 o) {
  signed char *p = array + row.at + c;
  const uint32_t s = VEC ? 0 : off(p, 8);
  const bool full = c + 8 <= d;
  if (s == 0 && (VEC ? c < d : full)) *reinterpret_cast<uint2 *>(p) = o;
  if constexpr (VEC) return;
  const int lane = threadIdx.x % 32;
  uint32_t w[4] = {o.x, o.y, o.x, o.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) w[i] = __shfl_up_sync(kAll, w[i], 1);
  const bool next = __shfl_down_sync(kAll, (int)full, 1) && lane < 31, mine = full && lane > 0;
  if (s && mine) {
    shifted(w, 8 - s);
    *reinterpret_cast<uint2 *>(p - s) = make_uint2(w[0], w[1]);
  }
  if (s == 0 ? full : mine && next) return;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const bool done = s == 0 ? false : q >= 8 - (int)s ? next : mine;
    if (c + q < d && !done) p[q] = (signed char)((q < 4 ? o.x : o.y) >> (8 * (q & 3)));
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
template <bool VEC>
struct Packed {
  uint2 codes;
  float scale;
  __device__ void load(const signed char *array, const float *scales, const RowAt &row, int c,
                       int d) {
    codes = make_uint2(0, 0);
    scale = 0.f;
    if (c >= d) return;
    scale = scales[c / kGroup];
    const signed char *p = array + row.at + c;
    if (!VEC && at_edge(row, c)) {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const uint32_t b = c + q < d ? (uint32_t)(uint8_t)p[q] : 0u;
        (q < 4 ? codes.x : codes.y) |= b << (8 * (q & 3));
      }
      return;
    }
    const uint32_t s = VEC ? 0 : off(p, 8);
    const uint2 *v = reinterpret_cast<const uint2 *>(p - s);
    codes = v[0];
    if (s) {
      const uint2 b = v[1];
      uint32_t w[4] = {codes.x, codes.y, b.x, b.y};
      shifted(w, s);
      codes = make_uint2(w[0], w[1]);
    }
  }
  __device__ Eight values(int c, int d) const {
    Eight e = times_scale(codes, scale);
    if (!VEC && c + 8 > d) e.zero_from(d - c);  // 0 times a scale that is not finite
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
  auto four = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x40), __byte_perm(c, d, 0x40), 0x5410);
  };
  return make_uint2(four(c[0], c[1], c[2], c[3]), four(c[4], c[5], c[6], c[7]));
}

// A barrier of a row's warps, the block's `group`th so many.
template <int WARPS>
__device__ __forceinline__ void row_barrier(int group) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * WARPS) : "memory");
}
// What the threads of a row share.
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
    row_barrier<WARPS>(group);
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
template <bool VEC, int NC, int WARPS, typename T>
__device__ __forceinline__ void store_norm(const Eight (&u)[NC], const CheckpointArgs &a, int t,
                                           const RowAt &row) {
  const bool layer = a.norm == FLASH_GAU_NORM_LAYER;
  const f2 g1 = both(layer ? 0.f : a.norm_g[0]);
  const RowAt one(0, 1, a.d);
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const int c = (k * 32 * WARPS + t) * 8;
    Eight v;
    if (layer) {
      const Eight g = load8<VEC>(a.norm_g, one, c, a.d);
      Eight b = {{0, 0, 0, 0}};
      if (a.norm_b) b = load8<VEC>(a.norm_b, one, c, a.d);
#pragma unroll
      for (int q = 0; q < 4; ++q) v.v[q] = fma2(u[k].v[q], g.v[q], b.v[q]);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) v.v[q] = mul2(u[k].v[q], g1);
    }
    store8<VEC>(static_cast<T *>(a.n), row, c, a.d, v);
  }
}

// ------------------------------------------------------------------- pack --
template <typename T, int NC, int WARPS, bool VEC>
__global__ void __launch_bounds__(32 * (WARPS > 4 ? WARPS : 4))
pack_kernel(const CheckpointArgs a) {
  __shared__ float part[2 * WARPS];
  RowSum<WARPS> row_sum{part, 0};
  const int t = threadIdx.x % (32 * WARPS);
  const long long m = (long long)blockIdx.x * (WARPS == 1 ? 4 : 1) + threadIdx.x / (32 * WARPS);
  ptx::griddep_wait();
  if (m >= a.M) return;  // whole warps, and with more than one whole blocks
  const RowAt row(m, a.M, a.d);
  const T *h = static_cast<const T *>(a.h), *y = static_cast<const T *>(a.y);
  Eight x[NC];
#pragma unroll
  for (int k = 0; k < NC; ++k) x[k] = load8<VEC>(h, row, (k * 32 * WARPS + t) * 8, a.d);
  if (y) {
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const Eight v = load8<VEC>(y, row, (k * 32 * WARPS + t) * 8, a.d);
#pragma unroll
      for (int q = 0; q < 4; ++q) x[k].v[q] = add2(x[k].v[q], v.v[q]);
    }
  }
  // r may be h's or y's array: a row's stores follow its loads, in every warp of it
  if (WARPS > 1 && !VEC) row_barrier<WARPS>(0);
  float *scales = a.scales + m * a.groups;
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const int c = (k * 32 * WARPS + t) * 8;
    if (a.r) store8<VEC>(static_cast<T *>(a.r), row, c, a.d, x[k]);
    uint32_t top;
    const Eight v = stored(x[k], h, &top);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(kAll, top, o));
    const float big = __uint_as_float(top), s = big < kLeast ? 0.f : big * (1.f / 127.f);
    if (t % 16 == 0 && c < a.d) scales[c / kGroup] = s;
    store_codes<VEC>(a.codes, row, c, a.d, codes_of(v, s));
  }
  if (a.n) {
    float length2;
    normalise<NC, WARPS>(x, a.norm, t, a.d, a.eps, row_sum, &length2);
    store_norm<VEC, NC, WARPS, T>(x, a, t, row);
  }
}

// ---------------------------------------------------------------- restore --
// (two or four rows a warp with all their codes asked for at first: 13.0 and 17.3
// us for 12.3 at 16384 x 768 bf16)
template <typename T, int NC, int WARPS, bool VEC>
__global__ void __launch_bounds__(32 * (WARPS > 4 ? WARPS : 4))
restore_kernel(const CheckpointArgs a) {
  __shared__ float part[2 * WARPS];
  RowSum<WARPS> row_sum{part, 0};
  const int t = threadIdx.x % (32 * WARPS);
  const long long m = (long long)blockIdx.x * (WARPS == 1 ? 4 : 1) + threadIdx.x / (32 * WARPS);
  ptx::griddep_wait();
  if (m >= a.M) return;  // whole warps, and with more than one whole blocks
  const RowAt row(m, a.M, a.d);
  Packed<VEC> p[NC];
#pragma unroll
  for (int k = 0; k < NC; ++k)
    p[k].load(a.codes, a.scales + m * a.groups, row, (k * 32 * WARPS + t) * 8, a.d);
  Eight x[NC];
#pragma unroll
  for (int k = 0; k < NC; ++k) x[k] = p[k].values((k * 32 * WARPS + t) * 8, a.d);
  if (a.r) {
#pragma unroll
    for (int k = 0; k < NC; ++k)
      store8<VEC>(static_cast<T *>(a.r), row, (k * 32 * WARPS + t) * 8, a.d, x[k]);
  }
  if (a.n) {
    float length2;
    normalise<NC, WARPS>(x, a.norm, t, a.d, a.eps, row_sum, &length2);
    store_norm<VEC, NC, WARPS, T>(x, a, t, row);
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

// Any rows.
template <typename T, int NC, int WARPS, bool VEC, bool LAYER>
__global__ void __launch_bounds__(32 * (WARPS > 4 ? WARPS : 4), LAYER ? 1 : WARPS > 4 ? 3 : 6)
backward_kernel(const CheckpointArgs a) {
  constexpr int kThreads = 32 * (WARPS > 4 ? WARPS : 4), rows = kThreads / 32 / WARPS;
  __shared__ float part[2 * WARPS];
  extern __shared__ float cols[];  // [2][d], one row of warps after another
  RowSum<WARPS> row_sum{part, 0};
  const int t = threadIdx.x % (32 * WARPS);
  float s1 = 0.f;
  Eight sg[LAYER ? NC : 1] = {}, sb[LAYER ? NC : 1] = {};
  ptx::griddep_wait();
  for (long long m = (long long)blockIdx.x * rows + threadIdx.x / (32 * WARPS); m < a.M;
       m += (long long)gridDim.x * rows) {
    const RowAt row(m, a.M, a.d);
    Eight x[NC], w[NC];
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = (k * 32 * WARPS + t) * 8;
      Packed<VEC> p;
      p.load(a.codes, a.scales + m * a.groups, row, c, a.d);
      x[k] = p.values(c, a.d);
    }
#pragma unroll
    for (int k = 0; k < NC; ++k)
      w[k] = load8<VEC>(static_cast<const T *>(a.dn), row, (k * 32 * WARPS + t) * 8, a.d);
    row_gradient<LAYER, NC, WARPS>(a, x, w, sg, sb, s1, t, row_sum, [&](int k) {
      return load8<VEC>(a.norm_g, RowAt(0, 1, a.d), (k * 32 * WARPS + t) * 8, a.d);
    });
    // dh may be dr's array: all of the row's loads before its first store
    if (a.dr) {
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        const int c = (k * 32 * WARPS + t) * 8;
        const Eight v = load8<VEC>(static_cast<const T *>(a.dr), row, c, a.d);
#pragma unroll
        for (int q = 0; q < 4; ++q) w[k].v[q] = add2(w[k].v[q], v.v[q]);
      }
      if (!VEC && WARPS > 1) row_barrier<WARPS>(0);
      if (!VEC && WARPS == 1) __syncwarp();
    }
#pragma unroll
    for (int k = 0; k < NC; ++k)
      store8<VEC>(static_cast<T *>(a.dh), row, (k * 32 * WARPS + t) * 8, a.d, w[k]);
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

template <int WHAT, typename T, int NC, int WARPS, bool VEC>
cudaError_t launch(const CheckpointArgs &a, unsigned grid, cudaStream_t stream) {
  constexpr int kThreads = 32 * (WARPS > 4 ? WARPS : 4);
  if constexpr (WHAT == kCheckpointPack) {
    return launch_pdl(pack_kernel<T, NC, WARPS, VEC>, dim3(grid), dim3(kThreads), 0, stream, a);
  } else if constexpr (WHAT == kCheckpointRestore) {
    return launch_pdl(restore_kernel<T, NC, WARPS, VEC>, dim3(grid), dim3(kThreads), 0, stream, a);
  } else {
    if (a.norm != FLASH_GAU_NORM_LAYER)
      return launch_pdl(backward_kernel<T, NC, WARPS, VEC, false>, dim3(grid), dim3(kThreads), 0,
                        stream, a);
    if constexpr (!VEC) {  // with vectors the form with copies ahead is taken
      const size_t smem = a.part ? 2 * a.d * sizeof(float) : 0;
      if (smem > 48 * 1024) {
        constexpr size_t kMost = 2 * kCheckpointMaxD * sizeof(float);
        const cudaError_t err = allow_shared<backward_kernel<T, NC, WARPS, VEC, true>>(kMost);
        if (err != cudaSuccess) return err;
      }
      return launch_pdl(backward_kernel<T, NC, WARPS, VEC, true>, dim3(grid), dim3(kThreads), smem,
                        stream, a);
    }
    return cudaErrorInvalidValue;
  }
}

template <int WHAT, typename T, bool VEC>
cudaError_t dispatch(const CheckpointArgs &a, unsigned most_blocks, cudaStream_t stream) {
  const int rows = checkpoint_row_warps(a.d) == 1 ? 4 : 1;
  const long long blocks = (a.M + rows - 1) / rows;
  const unsigned grid = (unsigned)(most_blocks && blocks > most_blocks ? most_blocks : blocks);
  if (a.d <= 256) return launch<WHAT, T, 1, 1, VEC>(a, grid, stream);
  if (a.d <= 512) return launch<WHAT, T, 2, 1, VEC>(a, grid, stream);
  if (a.d <= 768) return launch<WHAT, T, 3, 1, VEC>(a, grid, stream);
  if (a.d <= 1024) return launch<WHAT, T, 4, 1, VEC>(a, grid, stream);
  if (a.d <= 2048) return launch<WHAT, T, 2, 4, VEC>(a, grid, stream);
  if (a.d <= 4096) return launch<WHAT, T, 4, 4, VEC>(a, grid, stream);
  return launch<WHAT, T, 4, 8, VEC>(a, grid, stream);
}

// A kernel over all rows, in `most_blocks` blocks at most (0: as many as it takes).
template <bool VEC>
cudaError_t rows(int what, const CheckpointArgs &a, int dtype, unsigned most_blocks,
                 cudaStream_t stream) {
  const bool bf16 = dtype == FLASH_GAU_BF16;
  if (what == kCheckpointPack)
    return bf16 ? dispatch<kCheckpointPack, __nv_bfloat16, VEC>(a, most_blocks, stream)
                : dispatch<kCheckpointPack, float, VEC>(a, most_blocks, stream);
  if (what == kCheckpointRestore)
    return bf16 ? dispatch<kCheckpointRestore, __nv_bfloat16, VEC>(a, most_blocks, stream)
                : dispatch<kCheckpointRestore, float, VEC>(a, most_blocks, stream);
  return bf16 ? dispatch<kCheckpointBackward, __nv_bfloat16, VEC>(a, most_blocks, stream)
              : dispatch<kCheckpointBackward, float, VEC>(a, most_blocks, stream);
}

}  // namespace
}  // namespace flashgau
