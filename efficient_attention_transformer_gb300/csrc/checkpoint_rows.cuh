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
// 1024 columns), to four or to the eight of a block, 8 consecutive columns a
// thread and step: 16 or 32 bytes of a row, 8 codes, and a group is 16
// neighbouring threads, whose maximum is four shuffles.  32768 x 1024 fp32 with
// ScaleNorm: pack 84 us, 6.8 TB/s, restore 55, 5.5, gradients 71, 6.1; 16384 x
// 768 bf16 with LayerNorm, half of it in L2: 20, 12 and 22 us.
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

// How rows lie in memory, all arrays of a call alike:
// kVectors   every row is whole vectors of eight elements on their boundaries
// kBlocks    the arrays begin on a boundary and rows where they may: a thread's
//            eight elements are a vector on its boundary that may begin before
//            the row (in front of the first column) and end behind it, and is
//            loaded whole and masked, and stored element by element where it is
//            not the row's alone
// kElements  anything else, element by element
// (16384 x 767 bf16 as blocks 66 us pack, 27 restore, 38 the norm's gradient;
// element by element 73, 59 and 106; whole vectors of 768 columns 20, 12 and 22.
// 2000 x 513 fp32 5.3, 3.5 and, of a ScaleNorm, 6.7 for 8.9, 8.7 and 8.5.)
enum { kElements, kVectors, kBlocks };

// Eight columns of a row from column c on, in pairs.  Columns before the row and
// behind it are zero and not stored.
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
  __device__ void keep(int c, int d) {  // what lies within the row
    float x[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = c + q >= 0 && c + q < d ? get(q) : 0.f;
    of(x);
  }
};

// A row of an array of M rows: where it begins, and where the array ends.
struct RowAt {
  long long at, end;
  __device__ RowAt(long long m, long long M, int d) : at(m * d), end(M * d) {}
};
// what the row's first vector holds in front of it
template <int FORM>
__device__ __forceinline__ int in_front(const RowAt &row) {
  return FORM == kBlocks ? (int)row.at & 7 : 0;
}
// The first of a thread's columns in its run k; only the first run's can lie in
// front of the row.
template <int WARPS>
__device__ __forceinline__ int column(int k, int t, int front) {
  const int c = (k * 32 * WARPS + t) * 8 - front;
  if (k > 0) __builtin_assume(c >= 0);
  return c;
}
template <int FORM>
__device__ __forceinline__ bool whole(int c, int d) {
  return FORM == kVectors || (c >= 0 && c + 8 <= d);
}

__device__ __forceinline__ Eight vector8(const __nv_bfloat16 *p) {
  const uint4 a = *reinterpret_cast<const uint4 *>(p);
  return {{unpack_bf16(a.x), unpack_bf16(a.y), unpack_bf16(a.z), unpack_bf16(a.w)}};
}
__device__ __forceinline__ Eight vector8(const float *p) {
  const ulonglong2 a = reinterpret_cast<const ulonglong2 *>(p)[0];
  const ulonglong2 b = reinterpret_cast<const ulonglong2 *>(p)[1];
  return {{a.x, a.y, b.x, b.y}};
}
__device__ __forceinline__ void vector8(__nv_bfloat16 *p, const Eight &e) {
  *reinterpret_cast<uint4 *>(p) =
      make_uint4(pack_bf16(e.v[0]), pack_bf16(e.v[1]), pack_bf16(e.v[2]), pack_bf16(e.v[3]));
}
__device__ __forceinline__ void vector8(float *p, const Eight &e) {
  reinterpret_cast<ulonglong2 *>(p)[0] = make_ulonglong2(e.v[0], e.v[1]);
  reinterpret_cast<ulonglong2 *>(p)[1] = make_ulonglong2(e.v[2], e.v[3]);
}
__device__ __forceinline__ float widened(float v) { return v; }
__device__ __forceinline__ float widened(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void narrow(float *p, float v) { *p = v; }
__device__ __forceinline__ void narrow(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

template <int FORM, typename T>
__device__ __forceinline__ Eight load8(const T *array, const RowAt &row, int c, int d) {
  Eight e = {{0, 0, 0, 0}};
  if (c >= d) return e;
  const T *p = array + (row.at + c);
  if (FORM == kVectors || (FORM == kBlocks && row.at + c + 8 <= row.end)) {
    e = vector8(p);
    if (!whole<FORM>(c, d)) e.keep(c, d);
  } else {
    float x[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)
      x[q] = (FORM == kElements || c + q >= 0) && c + q < d ? widened(p[q]) : 0.f;
    e.of(x);
  }
  return e;
}
template <int FORM, typename T>
__device__ __forceinline__ void store8(T *array, const RowAt &row, int c, int d, const Eight &e) {
  if (c >= d) return;
  T *p = array + (row.at + c);
  if constexpr (FORM == kVectors) {
    vector8(p, e);
  } else {
    if (FORM == kBlocks && whole<FORM>(c, d)) return vector8(p, e);
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (c + q >= 0 && c + q < d) narrow(p + q, e.get(q));
  }
}
template <int FORM>
__device__ __forceinline__ void store_codes(signed char *array, const RowAt &row, int c, int d,
                                            uint2 o) {
  if (c >= d) return;
  signed char *p = array + (row.at + c);
  if constexpr (FORM == kVectors) {
    *reinterpret_cast<uint2 *>(p) = o;
  } else {
    if (FORM == kBlocks && whole<FORM>(c, d)) {
      *reinterpret_cast<uint2 *>(p) = o;
      return;
    }
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (c + q >= 0 && c + q < d) p[q] = (signed char)((q < 4 ? o.x : o.y) >> (8 * (q & 3)));
  }
}
// A parameter of the columns; `p` on a vector's boundary but for kElements.
template <int FORM>
__device__ __forceinline__ Eight parameter8(const float *p, int c, int d) {
  if constexpr (FORM != kBlocks) {
    return load8<FORM>(p, RowAt(0, 1, d), c, d);
  } else {
    // three vectors, moved by what c is off; what lies outside is anything
    const int s = c & 3;
    float x[12];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int at = min(max(c - s + 4 * i, 0), (d - 1) & ~3);
      if (at + 4 <= d) {
        const float4 f = *reinterpret_cast<const float4 *>(p + at);
        x[4 * i] = f.x, x[4 * i + 1] = f.y, x[4 * i + 2] = f.z, x[4 * i + 3] = f.w;
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) x[4 * i + q] = p[min(at + q, d - 1)];
      }
    }
#pragma unroll
    for (int i = 0; i < 10; ++i) x[i] = s & 2 ? x[i + 2] : x[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = s & 1 ? x[i + 1] : x[i];
    return {{pair(x[0], x[1]), pair(x[2], x[3]), pair(x[4], x[5]), pair(x[6], x[7])}};
  }
}

// Groups of the eight columns from c on: as blocks the first `split` columns can
// belong to the group before the others'.
template <int FORM>
struct Groups {
  int before, group, split;
  __device__ Groups(int c, int d) {
    if constexpr (FORM == kBlocks) {
      before = max(c, 0) / kGroup;
      group = min(c + 7, d - 1) / kGroup;
      split = group != before ? group * kGroup - c : 0;
    } else {
      before = group = c / kGroup;
      split = 0;
    }
  }
};
// Eight codes times their groups' scales, the values that the checkpoint stands
// for.  A code as fp32: it and 128 in the last digits of 2^23, less both.
template <int FORM>
__device__ __forceinline__ Eight times_scale(uint2 codes, float before, float s, int split) {
  const uint32_t w[2] = {codes.x ^ 0x80808080u, codes.y ^ 0x80808080u};
  Eight e;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const f2 c = pair(__uint_as_float(__byte_perm(w[q / 2], 0x4b000000u, 0x7440 + 2 * (q % 2))),
                      __uint_as_float(__byte_perm(w[q / 2], 0x4b000000u, 0x7441 + 2 * (q % 2))));
    const f2 by = FORM == kBlocks ? pair(2 * q < split ? before : s, 2 * q + 1 < split ? before : s)
                                  : both(s);
    e.v[q] = mul2(add2(c, both(-8388736.f)), by);
  }
  return e;
}
template <int FORM>
struct Packed {
  uint2 codes;
  float before, scale;
  __device__ void load(const signed char *array, const float *scales, const RowAt &row, int c,
                       int d) {
    codes = make_uint2(0, 0);
    before = scale = 0.f;
    if (c >= d) return;
    const Groups<FORM> g(c, d);
    scale = scales[g.group];
    if (FORM == kBlocks && g.split) before = scales[g.before];
    const signed char *p = array + (row.at + c);
    if (FORM == kVectors || (FORM == kBlocks && row.at + c + 8 <= row.end)) {
      codes = *reinterpret_cast<const uint2 *>(p);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const uint32_t b = c + q >= 0 && c + q < d ? (uint32_t)(uint8_t)p[q] : 0u;
        (q < 4 ? codes.x : codes.y) |= b << (8 * (q & 3));
      }
    }
  }
  __device__ Eight values(int c, int d) const {
    Eight e = times_scale<FORM>(codes, before, scale, Groups<FORM>(c, d).split);
    if (!whole<FORM>(c, d)) e.keep(c, d);  // 0 times a scale that is not finite
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
// the same of stored values' first `split` columns, and of the others
__device__ __forceinline__ void largest(const Eight &e, int split, uint32_t *first,
                                        uint32_t *others) {
  *first = *others = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const uint32_t m = __float_as_uint(e.get(q)) & 0x7fffffffu;
    (q < split ? *first : *others) = max(q < split ? *first : *others, m);
  }
}

// Codes of eight values.  t = v / s to the nearest whole number in the digits of
// 1.5 * 2^23 is at most one off; the remainder v - t s is exact, and where one of
// eight is half a scale or more, each is looked at: it moves above a half, and
// from an odd number at a half.
// A scale and its reciprocal; of a scale that restores zero or NaN neither.
__device__ __forceinline__ float2 with_inverse(float s) {
  const bool some = s > 0.f && s < __int_as_float(0x7f800000);
  return some ? make_float2(s, __fdiv_rn(1.f, s)) : make_float2(0.f, 0.f);
}
template <int FORM>
__device__ __forceinline__ uint2 codes_of(const Eight &e, float2 before, float2 s, int front) {
  const float magic = 12582912.f;
  if (FORM != kBlocks && s.x == 0.f) return make_uint2(0, 0);
  auto of = [&](int q) { return FORM == kBlocks && q < front ? before : s; };
  f2 t[4], rest[4];
  bool any = false;
  float most = 0.f;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float2 a = of(2 * q), b = of(2 * q + 1);
    t[q] = fma2(e.v[q], pair(a.y, b.y), both(magic));
    rest[q] = fma2(add2(both(magic), mul2(t[q], both(-1.f))), pair(a.x, b.x), e.v[q]);
    const float2 f = split(rest[q]);
    if (FORM == kBlocks) any |= fabsf(f.x) >= 0.5f * a.x || fabsf(f.y) >= 0.5f * b.x;
    else most = fmaxf(most, fmaxf(fabsf(f.x), fabsf(f.y)));
  }
  uint32_t c[8];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float2 f = split(t[q]);
    c[2 * q] = __float_as_uint(f.x);
    c[2 * q + 1] = __float_as_uint(f.y);
  }
  if (FORM == kBlocks ? any : most >= 0.5f * s.x) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float2 f = split(rest[q / 2]);
      const float x = q % 2 ? f.y : f.x, half = 0.5f * of(q).x;
      if (fabsf(x) > half || (fabsf(x) == half && (c[q] & 1))) c[q] += x > 0.f ? 1 : -1;
    }
  }
  // the last byte of each
  auto four = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x40), __byte_perm(c, d, 0x40), 0x5410);
  };
  uint2 codes = make_uint2(four(c[0], c[1], c[2], c[3]), four(c[4], c[5], c[6], c[7]));
  if constexpr (FORM == kBlocks) {  // no scale, no code
    const uint64_t low = (uint64_t(1) << (8 * front)) - 1;  // the first columns' bytes
    const uint64_t keep = (before.x > 0.f ? low : 0) | (s.x > 0.f ? ~low : 0);
    codes.x &= (uint32_t)keep;
    codes.y &= (uint32_t)(keep >> 32);
  }
  return codes;
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
// `front`: what the row's first vector holds in front of it.
template <int FORM, int NC, int WARPS>
__device__ __forceinline__ float normalise(Eight (&x)[NC], int kind, int t, int d, int front,
                                           float eps, RowSum<WARPS> &row_sum,
                                           float *length2) {
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
      const int c = column<WARPS>(k, t, front);
      const f2 less = both(c < d ? -mean : 0.f);
#pragma unroll
      for (int q = 0; q < 4; ++q) x[k].v[q] = add2(x[k].v[q], less);
      if (c < d && !whole<FORM>(c, d)) x[k].keep(c, d);
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
template <int FORM, int NC, int WARPS, typename T>
__device__ __forceinline__ void store_norm(const Eight (&u)[NC], const CheckpointArgs &a, int t,
                                           const RowAt &row) {
  const bool layer = a.norm == FLASH_GAU_NORM_LAYER;
  const f2 g1 = both(layer ? 0.f : a.norm_g[0]);
  const int front = in_front<FORM>(row);
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const int c = column<WARPS>(k, t, front);
    Eight v;
    if (layer) {
      const Eight g = parameter8<FORM>(a.norm_g, c, a.d);
      Eight b = {{0, 0, 0, 0}};
      if (a.norm_b) b = parameter8<FORM>(a.norm_b, c, a.d);
#pragma unroll
      for (int q = 0; q < 4; ++q) v.v[q] = fma2(u[k].v[q], g.v[q], b.v[q]);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) v.v[q] = mul2(u[k].v[q], g1);
    }
    store8<FORM>(static_cast<T *>(a.n), row, c, a.d, v);
  }
}

// ------------------------------------------------------------------- pack --
__device__ __forceinline__ float scale_of(uint32_t top) {
  const float big = __uint_as_float(top);
  return big < kLeast ? 0.f : big * (1.f / 127.f);
}

template <typename T, int NC, int WARPS, int FORM>
__global__ void
__launch_bounds__(32 * (WARPS > 4 ? WARPS : 4), FORM == kBlocks && WARPS < 8 ? 5 : 0)
pack_kernel(const CheckpointArgs a) {
  __shared__ float part[2 * WARPS];
  RowSum<WARPS> row_sum{part, 0};
  const int t = threadIdx.x % (32 * WARPS);
  const long long m = (long long)blockIdx.x * (WARPS == 1 ? 4 : 1) + threadIdx.x / (32 * WARPS);
  ptx::griddep_wait();
  if (m >= a.M) return;  // whole warps, and with more than one whole blocks
  const RowAt row(m, a.M, a.d);
  const int front = in_front<FORM>(row);
  const T *h = static_cast<const T *>(a.h), *y = static_cast<const T *>(a.y);
  Eight x[NC];
#pragma unroll
  for (int k = 0; k < NC; ++k) x[k] = load8<FORM>(h, row, column<WARPS>(k, t, front), a.d);
  if (y) {
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const Eight v = load8<FORM>(y, row, column<WARPS>(k, t, front), a.d);
#pragma unroll
      for (int q = 0; q < 4; ++q) x[k].v[q] = add2(x[k].v[q], v.v[q]);
    }
  }
  float *scales = a.scales + m * a.groups;
  if constexpr (FORM != kBlocks) {
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = (k * 32 * WARPS + t) * 8;
      if (a.r) store8<FORM>(static_cast<T *>(a.r), row, c, a.d, x[k]);
      uint32_t top;
      const Eight v = stored(x[k], h, &top);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(kAll, top, o));
      const float s = scale_of(top);
      if (t % 16 == 0 && c < a.d) scales[c / kGroup] = s;
      const float2 by = with_inverse(s);
      store_codes<FORM>(a.codes, row, c, a.d, codes_of<FORM>(v, by, by, 0));
    }
  } else {
    // Sixteen threads' vectors hold a group but for its last columns, which are the
    // first of the next sixteen's: their largest and the scale go through memory.
    constexpr int kGroups = NC * 2 * WARPS;
    __shared__ uint32_t tail[WARPS == 1 ? 4 : 1][kGroups + 1];
    __shared__ float2 group_scale[WARPS == 1 ? 4 : 1][kGroups];
    const int line = threadIdx.x / (32 * WARPS);
    auto meet = [&] {
      if (WARPS == 1) __syncwarp();
      else row_barrier<WARPS>(0);
    };
    uint32_t top[NC];
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = column<WARPS>(k, t, front), g = (k * 32 * WARPS + t) / 16;
      if (a.r) store8<FORM>(static_cast<T *>(a.r), row, c, a.d, x[k]);
      uint32_t first = 0;
      const Eight v = stored(x[k], h, &top[k]);
      if (t % 16 == 0) {
        if (c > 0 && front) largest(v, front, &first, &top[k]);
        tail[line][g] = first;
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top[k] = max(top[k], __shfl_xor_sync(kAll, top[k], o));
    }
    if (t == 0) tail[line][kGroups] = 0;
    meet();
    float2 s[NC];
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int g = (k * 32 * WARPS + t) / 16;
      const float scale = scale_of(max(top[k], tail[line][g + 1]));
      s[k] = with_inverse(scale);
      if (t % 16 == 0) {
        group_scale[line][g] = s[k];
        if (g < a.groups) scales[g] = scale;
      }
    }
    meet();
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = column<WARPS>(k, t, front), g = (k * 32 * WARPS + t) / 16;
      const bool two = t % 16 == 0 && c > 0;
      uint32_t unused;
      const Eight v = stored(x[k], h, &unused);
      const float2 before = two ? group_scale[line][g - 1] : s[k];
      store_codes<FORM>(a.codes, row, c, a.d, codes_of<FORM>(v, before, s[k], two ? front : 0));
    }
  }
  if (a.n) {
    float length2;
    normalise<FORM, NC, WARPS>(x, a.norm, t, a.d, front, a.eps, row_sum, &length2);
    store_norm<FORM, NC, WARPS, T>(x, a, t, row);
  }
}

// ---------------------------------------------------------------- restore --
// (two or four rows a warp with all their codes asked for at first: 13.0 and 17.3
// us for 12.3 at 16384 x 768 bf16)
template <typename T, int NC, int WARPS, int FORM>
__global__ void __launch_bounds__(32 * (WARPS > 4 ? WARPS : 4))
restore_kernel(const CheckpointArgs a) {
  __shared__ float part[2 * WARPS];
  RowSum<WARPS> row_sum{part, 0};
  const int t = threadIdx.x % (32 * WARPS);
  const long long m = (long long)blockIdx.x * (WARPS == 1 ? 4 : 1) + threadIdx.x / (32 * WARPS);
  ptx::griddep_wait();
  if (m >= a.M) return;  // whole warps, and with more than one whole blocks
  const RowAt row(m, a.M, a.d);
  const int front = in_front<FORM>(row);
  Packed<FORM> p[NC];
#pragma unroll
  for (int k = 0; k < NC; ++k)
    p[k].load(a.codes, a.scales + m * a.groups, row, column<WARPS>(k, t, front), a.d);
  Eight x[NC];
#pragma unroll
  for (int k = 0; k < NC; ++k) x[k] = p[k].values(column<WARPS>(k, t, front), a.d);
  if (a.r) {
#pragma unroll
    for (int k = 0; k < NC; ++k)
      store8<FORM>(static_cast<T *>(a.r), row, column<WARPS>(k, t, front), a.d, x[k]);
  }
  if (a.n) {
    float length2;
    normalise<FORM, NC, WARPS>(x, a.norm, t, a.d, front, a.eps, row_sum, &length2);
    store_norm<FORM, NC, WARPS, T>(x, a, t, row);
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
// fit, and few loads with them (registers alone: 59 us at 16384 x 768 bf16, 1.5
// TB/s; with the copies 22; 32768 x 1024 fp32 104).  For a LayerNorm of rows on
// 16-byte boundaries each thread therefore brings its part of the next rows into
// shared memory by asynchronous copies while it works on this one: no registers,
// no barrier, since it reads what it copied itself.  A ScaleNorm has no column
// sums; its rows go through registers alone, with as many warps as those leave.

// dx in place of w = dn's row, from the row's values x, with the column sums (a
// ScaleNorm has none, its one g's sum is s1).
// gain(k): a LayerNorm's g of the thread's k-th run.
template <int FORM, bool LAYER, int NC, int WARPS, typename G>
__device__ __forceinline__ void row_gradient(const CheckpointArgs &a, Eight (&x)[NC],
                                             Eight (&w)[NC], Eight *sg, Eight *sb,
                                             float &s1, int t, int front,
                                             RowSum<WARPS> &row_sum, const G &gain) {
  float length2 = 0.f;
  const float inv =
      normalise<FORM, NC, WARPS>(x, LAYER ? FLASH_GAU_NORM_LAYER : FLASH_GAU_NORM_SCALE, t, a.d,
                                 front, a.eps, row_sum, &length2);
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

// From registers alone: a ScaleNorm's rows, and a LayerNorm's element by element.
template <typename T, int NC, int WARPS, int FORM, bool LAYER>
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
    const int front = in_front<FORM>(row);
    Eight x[NC], w[NC];
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = column<WARPS>(k, t, front);
      Packed<FORM> p;
      p.load(a.codes, a.scales + m * a.groups, row, c, a.d);
      x[k] = p.values(c, a.d);
    }
#pragma unroll
    for (int k = 0; k < NC; ++k)
      w[k] = load8<FORM>(static_cast<const T *>(a.dn), row, column<WARPS>(k, t, front), a.d);
    row_gradient<FORM, LAYER, NC, WARPS>(a, x, w, sg, sb, s1, t, front, row_sum, [&](int k) {
      return parameter8<FORM>(a.norm_g, (k * 32 * WARPS + t) * 8, a.d);
    });
    // dh may be dr's array: a thread stores what it has loaded
    if (a.dr) {
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        const int c = column<WARPS>(k, t, front);
        const Eight v = load8<FORM>(static_cast<const T *>(a.dr), row, c, a.d);
#pragma unroll
        for (int q = 0; q < 4; ++q) w[k].v[q] = add2(w[k].v[q], v.v[q]);
      }
    }
#pragma unroll
    for (int k = 0; k < NC; ++k)
      store8<FORM>(static_cast<T *>(a.dh), row, column<WARPS>(k, t, front), a.d, w[k]);
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

// A LayerNorm's gradients with copies ahead.
// BYTES asynchronously, of which the first `valid` are read and the rest is zero
template <int BYTES>
__device__ __forceinline__ void copy_ahead(void *dst, const void *src, int valid = BYTES) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(dst)),
                 "l"(src), "r"(valid)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(ptx::smem_u32(dst)),
                 "l"(src), "n"(BYTES), "r"(valid)
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
// codes and the scale (as blocks two scales), the threads' side by side.
constexpr int ring_run(int form, int io, int threads) {
  return threads * (2 * 8 * io + 8 + (form == kBlocks ? 8 : 4));
}
// steps under way: as many as fit, up to four
constexpr int ring_steps(int form, int io, int runs, int threads) {
  const int n = (form == kBlocks ? 184 : 200) * 1024 / (runs * ring_run(form, io, threads));
  return n < 4 ? n : 4;
}
template <int FORM, typename T, int NC, int THREADS>
struct Ring {
  static constexpr int kPieces = sizeof(T) * 8 / 16;  // 16-byte pieces of a run
  static constexpr int kRun = ring_run(FORM, sizeof(T), THREADS);
  static constexpr int kStep = NC * kRun;
  static constexpr int kSteps = ring_steps(FORM, sizeof(T), NC, THREADS);
  static constexpr int kBytes = kSteps * kStep;
  char *at;
  __device__ uint4 *dn(int k) const {
    return reinterpret_cast<uint4 *>(at + k * kRun) + threadIdx.x;
  }
  __device__ uint4 *dr(int k) const { return dn(k) + kPieces * THREADS; }
  __device__ uint2 *codes(int k) const {
    return reinterpret_cast<uint2 *>(at + k * kRun + 32 * kPieces * THREADS) + threadIdx.x;
  }
  __device__ float *scale(int k) const {
    return reinterpret_cast<float *>(at + k * kRun + (32 * kPieces + 8) * THREADS) + threadIdx.x;
  }
};

// As blocks: a row's first vector holds the same number of elements in front of
// the row in every row of a warp, since the rows between them make whole vectors
// (the grid is a multiple of eight where a warp has several), so that a thread's
// columns stay its own for the sums and for g.
template <int FORM, typename T, int NC, int WARPS, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) ring_backward_kernel(const CheckpointArgs a) {
  using R = Ring<FORM, T, NC, THREADS>;
  constexpr int kRows = THREADS / 32 / WARPS;
  extern __shared__ __align__(16) char shared[];
  __shared__ float part[kRows * 2 * WARPS];
  const int t = threadIdx.x % (32 * WARPS), group = threadIdx.x / (32 * WARPS);
  RowSum<WARPS> row_sum{part + group * 2 * WARPS, group};
  float s1;
  Eight sg[NC] = {}, sb[NC] = {};
  ptx::griddep_wait();
  const long long end = a.M * a.d, step = (long long)gridDim.x * kRows;
  long long m = (long long)blockIdx.x * kRows + group;
  const int front = in_front<FORM>(RowAt(m, a.M, a.d));
  auto fetch = [&](long long m, int turn) {
    const R r{shared + turn * R::kStep};
    if (m < a.M) {
      const long long at = m * a.d;
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        const int c = column<WARPS>(k, t, front);
        if (c >= a.d) continue;
        // the last row's last vector may reach out of the arrays
        const int left = FORM == kBlocks ? (int)min(end - (at + c), 8ll) : 8;
#pragma unroll
        for (int v = 0; v < R::kPieces; ++v) {
          constexpr int kElements = 16 / sizeof(T);
          const int some = min(max(left - v * kElements, 0), kElements) * (int)sizeof(T);
          // (nothing is read where nothing is left; the address stays in the array)
          const long long from = at + c + (FORM == kBlocks && some == 0 ? 0 : v * kElements);
          const T *dn = static_cast<const T *>(a.dn), *dr = static_cast<const T *>(a.dr);
          copy_ahead<16>(r.dn(k) + v * THREADS, dn + from, some);
          if (dr) copy_ahead<16>(r.dr(k) + v * THREADS, dr + from, some);
        }
        copy_ahead<8>(r.codes(k), a.codes + (at + c), left);
        const Groups<FORM> g(c, a.d);
        const float *scales = a.scales + m * a.groups;
        copy_ahead<4>(r.scale(k), scales + g.group);
        if (FORM == kBlocks && g.split) copy_ahead<4>(r.scale(k) + THREADS, scales + g.before);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < R::kSteps - 1; ++i) fetch(m + i * step, i);
  // a LayerNorm's g, behind the steps, as blocks each group's own
  constexpr int kWide = NC * WARPS * 256;  // columns and what is in front of them
  float *gains = reinterpret_cast<float *>(shared + R::kBytes);
  if constexpr (FORM == kBlocks) {
    gains += group * kWide;
    for (int i = t; i < kWide; i += 32 * WARPS)
      gains[i] = i >= front && i - front < a.d ? a.norm_g[i - front] : 0.f;
  } else {
    for (int c = threadIdx.x; c < a.d; c += THREADS) gains[c] = a.norm_g[c];
  }
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
      const int c = column<WARPS>(k, t, front);
      if (c < a.d) {
        const int split = Groups<FORM>(c, a.d).split;
        const float before = split ? r.scale(k)[THREADS] : 0.f;
        x[k] = times_scale<FORM>(*r.codes(k), before, *r.scale(k), split);
        w[k] = widen(r.dn(k), THREADS, static_cast<const T *>(nullptr));
        if (!whole<FORM>(c, a.d)) {
          x[k].keep(c, a.d);
          w[k].keep(c, a.d);
        }
      }
    }
    row_gradient<FORM, true, NC, WARPS>(a, x, w, sg, sb, s1, t, front, row_sum, [&](int k) {
      const int i = (k * 32 * WARPS + t) * 8;
      return FORM == kBlocks || i < a.d ? vector8(gains + i) : none;
    });
    const RowAt row(m, a.M, a.d);
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = column<WARPS>(k, t, front);
      if (c >= a.d) continue;
      if (a.dr) {
        const Eight v = widen(r.dr(k), THREADS, static_cast<const T *>(nullptr));
#pragma unroll
        for (int q = 0; q < 4; ++q) w[k].v[q] = add2(w[k].v[q], v.v[q]);
      }
      store8<FORM>(static_cast<T *>(a.dh), row, c, a.d, w[k]);
    }
  }
  if (!a.part) return;
  // the block's sums: every group's in shared memory, then column by column
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  float *cols = reinterpret_cast<float *>(shared);
  const int wide = FORM == kBlocks ? kWide : a.d;
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const int i = (k * 32 * WARPS + t) * 8;
    if (FORM != kBlocks && i >= a.d) continue;
    vector8(cols + 2 * group * wide + i, sg[k]);
    vector8(cols + (2 * group + 1) * wide + i, sb[k]);
  }
  __syncthreads();
  float *to = a.part + (long long)blockIdx.x * 2 * a.d;
  for (int c = threadIdx.x; c < 2 * a.d; c += THREADS) {
    float v = 0.f;
#pragma unroll
    for (int g = 0; g < kRows; ++g) {
      // where the group's row begins in its vectors; behind the last row it has none
      const int at = in_front<FORM>(RowAt((long long)blockIdx.x * kRows + g, a.M, a.d));
      v += cols[2 * g * wide + at + (c < a.d ? c : wide - a.d + c)];
    }
    to[c] = v;
  }
}

// The form with copies ahead, one block an SM.  Gives the blocks' number and their
// warps.
template <int FORM, typename T, int NC, int WARPS>
cudaError_t launch_ring(const CheckpointArgs &a, int num_sms, cudaStream_t stream,
                        CheckpointGrid *g) {
  // as many as the column sums' registers leave, and three steps' memory where a
  // row's warps allow
  constexpr int kMost = NC < 3 ? 512 : NC == 3 ? 384 : 256, kIo = sizeof(T);
  constexpr int kThreads = ring_steps(FORM, kIo, NC, kMost) >= 3               ? kMost
                           : kMost > 384 && ring_steps(FORM, kIo, NC, 384) >= 3 ? 384
                           : ring_steps(FORM, kIo, NC, 256) >= 3 || WARPS == 8 ? 256
                           : WARPS == 4                                  ? 128
                                                                         : 192;
  constexpr int kRows = kThreads / 32 / WARPS;
  constexpr auto kernel = ring_backward_kernel<FORM, T, NC, WARPS, kThreads>;
  // the steps and a LayerNorm's g, then the groups' column sums; d is at most kD,
  // and as blocks all kD columns are there
  constexpr size_t kD = NC * WARPS * 256, kSteps = Ring<FORM, T, NC, kThreads>::kBytes;
  constexpr size_t kSums = kRows * 2 * kD * sizeof(float);
  constexpr size_t kAll = kSteps + (FORM == kBlocks ? kRows : 1) * kD * sizeof(float);
  constexpr size_t kMostShared = kSums > kAll ? kSums : kAll;
  const cudaError_t err = allow_shared<kernel>(kMostShared);
  if (err != cudaSuccess) return err;
  const size_t sums = (size_t)kRows * 2 * a.d * sizeof(float);
  const size_t steps = kSteps + a.d * sizeof(float);
  const size_t smem = FORM == kBlocks ? kMostShared : sums > steps ? sums : steps;
  const long long all = (a.M + kRows - 1) / kRows;
  const int most = FORM != kBlocks ? num_sms : num_sms < 16 ? 8 : num_sms / 8 * 8;
  g->blocks = (int)(all < most ? all : most);
  if (g->blocks > kCheckpointBlocks) g->blocks = kCheckpointBlocks;  // (a multiple of 8)
  g->warps = kThreads / 32;
  return launch_pdl(kernel, dim3(g->blocks), dim3(kThreads), smem, stream, a);
}
template <int FORM, typename T>
cudaError_t dispatch_ring(const CheckpointArgs &a, int num_sms, cudaStream_t stream,
                          CheckpointGrid *g) {
  if (a.width <= 256) return launch_ring<FORM, T, 1, 1>(a, num_sms, stream, g);
  if (a.width <= 512) return launch_ring<FORM, T, 2, 1>(a, num_sms, stream, g);
  if (a.width <= 768) return launch_ring<FORM, T, 3, 1>(a, num_sms, stream, g);
  if (a.width <= 1024) return launch_ring<FORM, T, 4, 1>(a, num_sms, stream, g);
  if (a.width <= 2048) return launch_ring<FORM, T, 2, 4>(a, num_sms, stream, g);
  if (a.width <= 4096) return launch_ring<FORM, T, 4, 4>(a, num_sms, stream, g);
  return launch_ring<FORM, T, 4, 8>(a, num_sms, stream, g);
}

template <int WHAT, int FORM, typename T, int NC, int WARPS>
cudaError_t launch(const CheckpointArgs &a, cudaStream_t stream, CheckpointGrid *g) {
  constexpr int kThreads = 32 * (WARPS > 4 ? WARPS : 4), kRows = kThreads / 32 / WARPS;
  const long long blocks = (a.M + kRows - 1) / kRows;
  if constexpr (WHAT == kCheckpointPack) {
    return launch_pdl(pack_kernel<T, NC, WARPS, FORM>, dim3((unsigned)blocks), dim3(kThreads), 0,
                      stream, a);
  } else if constexpr (WHAT == kCheckpointRestore) {
    return launch_pdl(restore_kernel<T, NC, WARPS, FORM>, dim3((unsigned)blocks), dim3(kThreads),
                      0, stream, a);
  } else {
    const bool layer = a.norm == FLASH_GAU_NORM_LAYER;
    const int most = layer ? kCheckpointBlocks : kCheckpointScaleBlocks;
    *g = {(int)(blocks < most ? blocks : most), kThreads / 32};
    if (!layer)
      return launch_pdl(backward_kernel<T, NC, WARPS, FORM, false>, dim3(g->blocks),
                        dim3(kThreads), 0, stream, a);
    if constexpr (FORM == kElements) {  // the others take the form with copies ahead
      const size_t smem = a.part ? 2 * a.d * sizeof(float) : 0;
      if (smem > 48 * 1024) {
        constexpr size_t kMost = 2 * kCheckpointMaxD * sizeof(float);
        const cudaError_t err = allow_shared<backward_kernel<T, NC, WARPS, FORM, true>>(kMost);
        if (err != cudaSuccess) return err;
      }
      return launch_pdl(backward_kernel<T, NC, WARPS, FORM, true>, dim3(g->blocks),
                        dim3(kThreads), smem, stream, a);
    }
    return cudaErrorInvalidValue;
  }
}

template <int WHAT, int FORM, typename T>
cudaError_t dispatch(const CheckpointArgs &a, cudaStream_t stream, CheckpointGrid *g) {
  if constexpr (FORM != kElements) {  // element by element fewer variants will do
    if (a.width <= 256) return launch<WHAT, FORM, T, 1, 1>(a, stream, g);
    if (a.width <= 512) return launch<WHAT, FORM, T, 2, 1>(a, stream, g);
    if (a.width <= 768) return launch<WHAT, FORM, T, 3, 1>(a, stream, g);
    if (a.width > 1024 && a.width <= 2048) return launch<WHAT, FORM, T, 2, 4>(a, stream, g);
  }
  if (a.width <= 1024) return launch<WHAT, FORM, T, 4, 1>(a, stream, g);
  if (a.width <= 4096) return launch<WHAT, FORM, T, 4, 4>(a, stream, g);
  return launch<WHAT, FORM, T, 4, 8>(a, stream, g);
}

template <int FORM, typename T>
cudaError_t rows_of(int what, const CheckpointArgs &a, int num_sms, cudaStream_t stream,
                    CheckpointGrid *g) {
  if (what == kCheckpointPack) return dispatch<kCheckpointPack, FORM, T>(a, stream, g);
  if (what == kCheckpointRestore) return dispatch<kCheckpointRestore, FORM, T>(a, stream, g);
  if constexpr (FORM != kElements)
    if (a.norm == FLASH_GAU_NORM_LAYER) return dispatch_ring<FORM, T>(a, num_sms, stream, g);
  return dispatch<kCheckpointBackward, FORM, T>(a, stream, g);
}

// A kernel over all rows.
template <int FORM>
cudaError_t rows(int what, const CheckpointArgs &a, int dtype, int num_sms, cudaStream_t stream,
                 CheckpointGrid *g) {
  return dtype == FLASH_GAU_BF16 ? rows_of<FORM, __nv_bfloat16>(what, a, num_sms, stream, g)
                                 : rows_of<FORM, float>(what, a, num_sms, stream, g);
}

}  // namespace
}  // namespace flashgau
