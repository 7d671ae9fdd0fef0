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
// tensors), needs no workspace and can be captured; a warp takes 256 elements
// of one tensor at a time as two runs of 128, four consecutive elements a lane
// (16-byte accesses).  fp32 moments run at the copy rate (43.8 M parameters:
// 189 us, 6.7 TB/s), and 8-bit ones nearly do in long lists, whose values pass
// through shared memory (82.6 M with fp32 gradients and copies: 221 us); their
// values are written at 5.8 TB/s (133 us).
#include <cuda_bf16.h>
#include <math.h>

#include <atomic>

#include "flash_gau_internal.h"
#include "packed_f32.cuh"
#include "sm103_ptx.cuh"

namespace flashgau {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBlock = 256;  // elements that share a scale; a warp's at a time
constexpr int kRuns = 3;     // of them a warp takes from a long list of 8-bit moments

struct Entry {
  float *p;
  __nv_bfloat16 *copy;
  const void *g;
  void *m, *v;
  float *m_scale, *v_scale;
  long long n;
  float decay;    // 1 - lr * weight_decay
  int first;      // first thread block of the tensor in this launch
  int g_bf16;
  int vec;  // every pointer aligned for 1: four elements at a time, 2: 16 bytes
};

// The scalars of a step.
struct Step {
  float step_size, beta1, omb1, beta2, omb2, inv_c2, eps, one;
  const float *grad_scale;
};

template <int CAP>
struct List {
  Entry e[CAP];
  int count;
  int runs;  // blocks of 256 elements that a warp takes
  Step step;
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

// Four elements at i of an array, of which `n` are inside (FULL: all, on a
// boundary of four).
template <bool FULL>
__device__ __forceinline__ void load4(const float *a, long long i, int n, float (&x)[4]) {
  if (FULL) {
    const float4 t = *reinterpret_cast<const float4 *>(a + i);
    x[0] = t.x; x[1] = t.y; x[2] = t.z; x[3] = t.w;
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] = q < n ? a[i + q] : 0.f;
  }
}
template <bool FULL>
__device__ __forceinline__ void load4(const __nv_bfloat16 *a, long long i, int n,
                                      float (&x)[4]) {
  if (FULL) {
    const uint2 t = *reinterpret_cast<const uint2 *>(a + i);
    const float2 u = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&t.x));
    const float2 w = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&t.y));
    x[0] = u.x; x[1] = u.y; x[2] = w.x; x[3] = w.y;
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] = q < n ? __bfloat162float(a[i + q]) : 0.f;
  }
}
template <bool FULL>
__device__ __forceinline__ void store4(float *a, long long i, int n, const float (&x)[4]) {
  if (FULL) {
    *reinterpret_cast<float4 *>(a + i) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q < n) a[i + q] = x[q];
  }
}
template <bool FULL>
__device__ __forceinline__ void store4(__nv_bfloat16 *a, long long i, int n,
                                       const float (&x)[4]) {
  if (FULL) {
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
template <bool FULL>
__device__ __forceinline__ uint32_t load_codes(const void *a, long long i, int n) {
  const uint8_t *c = static_cast<const uint8_t *>(a) + i;
  if (FULL) return *reinterpret_cast<const uint32_t *>(c);
  uint32_t w = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (q < n) w |= (uint32_t)c[q] << (8 * q);
  return w;
}
template <bool FULL>
__device__ __forceinline__ void store_codes(void *a, long long i, int n, uint32_t w) {
  uint8_t *c = static_cast<uint8_t *>(a) + i;
  if (FULL) {
    *reinterpret_cast<uint32_t *>(c) = w;
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q < n) c[q] = (uint8_t)(w >> (8 * q));
  }
}

// Codes to and from fp32 without the conversion unit, which a step over 8-bit
// moments would keep busier than memory: a byte becomes the low digits of
// 2^23 (read) or is what adding 1.5 * 2^23 leaves in them (written, rounded to
// nearest even, negative values as two's complement).
// bytes 2 h and 2 h + 1 of a word, less what `bias` says
__device__ __forceinline__ f2 byte_floats(uint32_t w, int h, float bias) {
  const f2 x = pair(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7650 | (2 * h))),
                    __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7651 | (2 * h))));
  return add2(x, both(-bias));
}
// four codes of first moments are read as w ^ 0x80808080
__device__ __forceinline__ f2 decode_m(uint32_t w, int h, f2 scale) {
  const f2 c = byte_floats(w, h, 8388608.0f + 128.0f);
  const float2 x = split(c);
  return mul2(mul2(c, pair(fabsf(x.x), fabsf(x.y))), scale);
}
__device__ __forceinline__ f2 decode_root(uint32_t w, int h, f2 scale) {
  const f2 c = byte_floats(w, h, 8388608.0f);
  return mul2(mul2(c, c), scale);
}
__device__ __forceinline__ uint32_t pack_codes(const uint32_t (&c)[4]) {
  return __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
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

// The codes of eight elements, from correctly rounded roots or (EXACT not set)
// from the hardware's approximate ones; then the return value says how far
// from an integer the roots came at most.  abs_m: without the signs.
template <bool EXACT>
__device__ __forceinline__ float encode(const f2 (&m)[4], const f2 (&abs_m)[4], const f2 (&root)[4],
                                        float mi, float vi, float keep, uint32_t (&mw)[2],
                                        uint32_t (&vw)[2]) {
  float off = 0.f;
  const f2 magic = both(12582912.0f), back = both(-12582912.0f), minus = both(-1.f);
  auto rooted = [&](f2 x) {
    const float2 a = split(x);
    if (EXACT) return pair(__fsqrt_rn(a.x), __fsqrt_rn(a.y));
    float2 y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(a.x));
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(a.y));
    const f2 r = pair(y.x, y.y);
    const float2 d = split(fma2(add2(add2(r, magic), back), minus, r));
    off = fmaxf(off, fmaxf(fabsf(d.x), fabsf(d.y)));
    return r;
  };
  const f2 mi2 = both(mi), vi2 = both(vi);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t mq[4], vq[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = 2 * j + h;
      // the block's largest value comes out a rounding above 127 or 255 at
      // most, and rounds to it
      const float2 sm = split(m[k]), a = split(rooted(mul2(abs_m[k], mi2)));
      const float2 c = split(add2(pair(copysignf(a.x, sm.x), copysignf(a.y, sm.y)), magic));
      mq[2 * h] = __float_as_uint(c.x);
      mq[2 * h + 1] = __float_as_uint(c.y);
      // a nonzero root keeps a code of at least 1
      const float2 r = split(root[k]), b = split(rooted(mul2(root[k], vi2)));
      const float2 e = split(add2(pair(fmaxf(b.x, __saturatef(r.x * keep)),
                                       fmaxf(b.y, __saturatef(r.y * keep))), magic));
      vq[2 * h] = __float_as_uint(e.x);
      vq[2 * h + 1] = __float_as_uint(e.y);
    }
    mw[j] = pack_codes(mq);
    vw[j] = pack_codes(vq);
  }
  return off;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void to_pairs(const float (&x)[4], f2 *y) {
  y[0] = pair(x[0], x[1]);
  y[1] = pair(x[2], x[3]);
}
__device__ __forceinline__ void from_pairs(const f2 *y, float (&x)[4]) {
  const float2 a = split(y[0]), b = split(y[1]);
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
}

// Where a block's 256 elements are read: the tensor's arrays from there on, or
// their copies in shared memory.
struct Source {
  const float *p;
  const void *g, *m, *v;
  float ms, vs;  // 8-bit moments' scales
};

// One warp's 256 elements of a tensor, block `blk` of it; pairs 2 j and 2 j + 1
// are the lane's four elements of run j.
template <int BITS, bool FULL>
__device__ __forceinline__ void update(const Entry &e, const Source &src, const Step &l,
                                       long long blk, int lane, float gs) {
  const long long i0 = blk * kBlock + 4 * lane;
  int n[2];
  f2 p[4], g[4], m[4], v[4];
  float x[4];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const long long left = e.n - (i0 + 128 * j);
    const int i = 4 * lane + 128 * j;
    n[j] = FULL || left >= 4 ? 4 : (left > 0 ? (int)left : 0);
    load4<FULL>(src.p, i, n[j], x);
    to_pairs(x, p + 2 * j);
    if (e.g_bf16) load4<FULL>(static_cast<const __nv_bfloat16 *>(src.g), i, n[j], x);
    else load4<FULL>(static_cast<const float *>(src.g), i, n[j], x);
    to_pairs(x, g + 2 * j);
    if constexpr (BITS == 32) {
      load4<FULL>(static_cast<const float *>(src.m), i, n[j], x);
      to_pairs(x, m + 2 * j);
      load4<FULL>(static_cast<const float *>(src.v), i, n[j], x);
      to_pairs(x, v + 2 * j);
    }
  }
  if constexpr (BITS == 8) {
    const f2 ms = both(src.ms), vs = both(src.vs);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      // codes behind the end are read as zeros
      const uint32_t mc = load_codes<FULL>(src.m, 4 * lane + 128 * j, n[j]) ^ 0x80808080u;
      const uint32_t vc = load_codes<FULL>(src.v, 4 * lane + 128 * j, n[j]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        m[2 * j + h] = decode_m(mc, h, ms);
        const f2 r = decode_root(vc, h, vs);
        v[2 * j + h] = mul2(r, r);
      }
    }
  }
  f2 root[4], abs_m[4];
  uint32_t mmax = 0, rmax = 0;
  const f2 gs2 = both(gs), beta1 = both(l.beta1), omb1 = both(l.omb1), beta2 = both(l.beta2),
           omb2 = both(l.omb2), inv_c2 = both(l.inv_c2), eps = both(l.eps), decay = both(e.decay),
           minus_step = both(-l.step_size);
  // a sum of two rounded products: as x * 1 + y, which nothing contracts
  // (pairs' products and sums are, whatever rounding they name)
  const f2 one = both(l.one);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const f2 gg = mul2(g[k], gs2);  // exact where gs is one
    m[k] = fma2(mul2(m[k], beta1), one, mul2(gg, omb1));
    v[k] = fma2(mul2(v[k], beta2), one, mul2(mul2(gg, omb2), gg));
    const float2 w = split(v[k]);
    root[k] = pair(__fsqrt_rn(w.x), __fsqrt_rn(w.y));
    // a reciprocal of 1 unit in the last place is far finer than p's own digits
    const float2 den = split(fma2(root[k], inv_c2, eps));
    p[k] = fma2(mul2(m[k], minus_step), pair(rcp_approx(den.x), rcp_approx(den.y)),
                mul2(p[k], decay));
    if constexpr (BITS == 8) {
      const float2 a = split(m[k]), r = split(root[k]);
      abs_m[k] = pair(fabsf(a.x), fabsf(a.y));
      mmax = max(mmax, max(__float_as_uint(fabsf(a.x)), __float_as_uint(fabsf(a.y))));
      // (a root has no sign, unless it is not a number)
      rmax = max(rmax, max(__float_as_uint(fabsf(r.x)), __float_as_uint(fabsf(r.y))));
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const long long i = i0 + 128 * j;
    from_pairs(p + 2 * j, x);
    store4<FULL>(e.p, i, n[j], x);
    if (e.copy) store4<FULL>(e.copy, i, n[j], x);
    if constexpr (BITS == 32) {
      from_pairs(m + 2 * j, x);
      store4<FULL>(static_cast<float *>(e.m), i, n[j], x);
      from_pairs(v + 2 * j, x);
      store4<FULL>(static_cast<float *>(e.v), i, n[j], x);
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
    // a nonzero sqrt(v) is at least 2^-75
    const float keep = vs != 0.f ? 0x1p100f : 0.f;
    uint32_t mw[2], vw[2];
    const float off = encode<false>(m, abs_m, root, mi, vi, keep, mw, vw);
    // A root off by 2^-23 of itself, 2^-15 at 255, rounds as the exact one
    // does unless it comes this near to the middle between two codes.
    if (off > 0.5f - 0x1p-14f) encode<true>(m, abs_m, root, mi, vi, keep, mw, vw);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      store_codes<FULL>(e.m, i0 + 128 * j, n[j], mw[j]);
      store_codes<FULL>(e.v, i0 + 128 * j, n[j], vw[j]);
    }
  }
}

// The tensor's arrays from block `blk` on.
template <int BITS>
__device__ __forceinline__ Source source(const Entry &e, long long blk) {
  const long long i = blk * kBlock;
  Source s;
  s.p = e.p + i;
  s.g = static_cast<const uint8_t *>(e.g) + i * (e.g_bf16 ? 2 : 4);
  s.m = static_cast<const uint8_t *>(e.m) + i * (BITS / 8);
  s.v = static_cast<const uint8_t *>(e.v) + i * (BITS / 8);
  s.ms = s.vs = 0.f;  // the caller's to read
  return s;
}

// A warp's blocks of a tensor: first, and the one behind the last.
template <int CAP>
__device__ __forceinline__ const Entry &my_blocks(const List<CAP> &l, long long &blk, long long &end) {
  const Entry &e = l.e[find(l, blockIdx.x)];
  blk = ((long long)(blockIdx.x - e.first) * kWarps + (threadIdx.x >> 5)) * l.runs;
  end = min(blk + l.runs, (e.n + kBlock - 1) / kBlock);
  return e;
}

// 16 bytes from global into shared memory without passing through registers
__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(dst)), "l"(src)
               : "memory");
}

// A block's p, g, codes and scales of 8-bit moments in shared memory.
struct __align__(16) Staged {
  float p[kBlock];
  float g[kBlock];  // bf16 ones in its first half
  uint8_t m[kBlock], v[kBlock];
  float scales[4];
  __device__ void fetch(const Entry &e, long long blk, int lane) {
    const Source s = source<8>(e, blk);
    for (int i = lane; i < kBlock / 4; i += 32) cp_async16(p + 4 * i, s.p + 4 * i);
    const uint8_t *from = static_cast<const uint8_t *>(s.g);
    for (int i = lane; i < (e.g_bf16 ? kBlock / 8 : kBlock / 4); i += 32)
      cp_async16(g + 4 * i, from + 16 * i);
    const int i = 16 * (lane & 15);
    if (lane < 16) cp_async16(m + i, static_cast<const uint8_t *>(s.m) + i);
    else cp_async16(v + i, static_cast<const uint8_t *>(s.v) + i);
    if (lane < 2)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(ptx::smem_u32(scales + lane)),
                   "l"(lane ? e.v_scale + blk : e.m_scale + blk)
                   : "memory");
  }
};
constexpr size_t kStagedBytes = sizeof(Staged) * kRuns * kWarps;

// The blocks from blk on, values read where they are.
template <int BITS>
__device__ __forceinline__ void direct(const Entry &e, const Step &step, long long blk, long long end,
                                       float gs) {
  const int lane = threadIdx.x & 31;
  for (; blk < end; ++blk) {
    Source s = source<BITS>(e, blk);
    if (BITS == 8) {
      s.ms = e.m_scale[blk];
      s.vs = e.v_scale[blk];
    }
    if (e.vec && blk * kBlock + kBlock <= e.n) update<BITS, true>(e, s, step, blk, lane, gs);
    else update<BITS, false>(e, s, step, blk, lane, gs);
  }
}

// Blocks on an SM: 44 M parameters with fp32 moments take 0.188 ms with five,
// 0.199 with four (of 64 registers).
template <int BITS, int CAP>
__global__ void __launch_bounds__(kThreads, BITS == 8 ? 4 : 5) adamw_kernel(const __grid_constant__ List<CAP> l) {
  ptx::griddep_wait();
  long long blk, end;
  const Entry &e = my_blocks(l, blk, end);
  direct<BITS>(e, l.step, blk, end, l.step.grad_scale ? *l.step.grad_scale : 1.f);
}

// Long lists with 8-bit moments: a warp asks for the values of all its blocks
// at once (60 KB of shared memory, three thread blocks an SM) and codes one
// after the other.
template <int CAP>
__global__ void __launch_bounds__(kThreads, 3) adamw_staged_kernel(const __grid_constant__ List<CAP> l) {
  extern __shared__ __align__(16) uint8_t smem[];
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31;
  long long blk, end;
  const Entry &e = my_blocks(l, blk, end);
  const float gs = l.step.grad_scale ? *l.step.grad_scale : 1.f;
  if (e.vec == 2) {
    Staged *const mine = reinterpret_cast<Staged *>(smem) + (threadIdx.x >> 5) * kRuns;
    const long long whole = min(end, e.n / kBlock);
#pragma unroll
    for (int k = 0; k < kRuns; ++k) {
      if (blk + k < whole) mine[k].fetch(e, blk + k, lane);
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    for (int k = 0; blk < whole; ++k, ++blk) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kRuns - 1) : "memory");
      __syncwarp();
      const Staged &in = mine[k];
      const Source s = {in.p, in.g, in.m, in.v, in.scales[0], in.scales[1]};
      update<8, true>(e, s, l.step, blk, lane, gs);
      asm volatile("cp.async.commit_group;" ::: "memory");  // so that the wait counts on
    }
  }
  direct<8>(e, l.step, blk, end, gs);
}

// m and v of 8-bit moments as fp32: `p` holds m's values, `copy` v's.
template <bool FULL>
__device__ __forceinline__ void values(const Entry &e, long long blk, int lane) {
  const f2 ms = both(e.m_scale[blk]), vs = both(e.v_scale[blk]);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const long long i = blk * kBlock + 4 * lane + 128 * j, left = e.n - i;
    const int n = FULL || left >= 4 ? 4 : (left > 0 ? (int)left : 0);
    const uint32_t mc = load_codes<FULL>(e.m, i, n) ^ 0x80808080u;
    const uint32_t vc = load_codes<FULL>(e.v, i, n);
    f2 mp[2], vp[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mp[h] = decode_m(mc, h, ms);
      const f2 r = decode_root(vc, h, vs);
      vp[h] = mul2(r, r);
    }
    float m[4], v[4];
    from_pairs(mp, m);
    from_pairs(vp, v);
    store4<FULL>(e.p, i, n, m);
    store4<FULL>(reinterpret_cast<float *>(e.copy), i, n, v);
  }
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, 8) moments_kernel(const __grid_constant__ List<CAP> l) {
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31;
  long long blk, end;
  const Entry &e = my_blocks(l, blk, end);
  for (; blk < end; ++blk) {
    if (e.vec && blk * kBlock + kBlock <= e.n) values<true>(e, blk, lane);
    else values<false>(e, blk, lane);
  }
}

bool aligned(const void *p, unsigned bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

template <int CAP, typename Kernel, typename Fill>
cudaError_t run(Kernel kernel, const AdamwProblem &q, int runs, size_t smem, Fill fill) {
  List<CAP> l;
  l.step.step_size = (float)(q.lr / (1.0 - pow(q.beta1, (double)q.step)));
  l.step.beta1 = (float)q.beta1;
  l.step.omb1 = (float)(1.0 - q.beta1);
  l.step.beta2 = (float)q.beta2;
  l.step.omb2 = (float)(1.0 - q.beta2);
  l.step.inv_c2 = (float)(1.0 / sqrt(1.0 - pow(q.beta2, (double)q.step)));
  l.step.eps = (float)q.eps;
  l.step.one = 1.f;
  l.step.grad_scale = q.grad_scale;
  l.runs = runs;
  const long long chunk = (long long)kWarps * kBlock * l.runs;
  for (int k = 0; k < q.n_tensors;) {
    l.count = 0;
    long long blocks = 0;
    // as many tensors as fit the list and the grid
    for (; k < q.n_tensors && l.count < CAP; ++k) {
      const flash_gau_adamw_tensor &t = q.tensors[k];
      if (t.n == 0) continue;
      const long long b = (t.n + chunk - 1) / chunk;
      if (l.count && blocks + b > 0x7fffffffLL) break;
      Entry &e = l.e[l.count++];
      fill(k, e);
      e.n = t.n;
      e.first = (int)blocks;
      blocks += b;
    }
    if (!l.count) break;
    const cudaError_t err =
        launch_pdl(kernel, dim3((unsigned)blocks), dim3(kThreads), smem, q.stream, l);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

// short lists keep the launch's parameters small
constexpr int kSmall = 16, kLarge = 384;

// With 8-bit moments coding leaves too few loads under way, so long lists take
// the staged kernel (parameters, gradients and copies of 82 M elements: 0.30 ms
// direct, 0.22 staged; 9.4 M 35 and 27 us; 4.7 M 14.1 and 14.9 us).  With fp32
// moments the direct one runs at the copy rate.
template <int CAP, typename Fill>
cudaError_t step_by_size(const AdamwProblem &q, Fill fill) {
  if (q.state_bits != 8) return run<CAP>(adamw_kernel<32, CAP>, q, 1, 0, fill);
  long long n = 0;
  for (int k = 0; k < q.n_tensors; ++k) n += q.tensors[k].n;
  if (n < (1LL << 23)) return run<CAP>(adamw_kernel<8, CAP>, q, 1, 0, fill);
  auto kernel = adamw_staged_kernel<CAP>;
  static std::atomic<int> allowed[64];  // per device
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!allowed[dev].load(std::memory_order_acquire)) {
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kStagedBytes);
    if (err != cudaSuccess) return err;
    allowed[dev].store(1, std::memory_order_release);
  }
  return run<CAP>(kernel, q, kRuns, kStagedBytes, fill);
}

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
    if (e.vec && aligned(t.g, 16) && aligned(t.m, 16) && aligned(t.v, 16)) e.vec = 2;
  };
  if (q.n_tensors <= kSmall) return step_by_size<kSmall>(q, fill);
  return step_by_size<kLarge>(q, fill);
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
  return q.n_tensors <= kSmall ? run<kSmall>(moments_kernel<kSmall>, q, 1, 0, fill)
                               : run<kLarge>(moments_kernel<kLarge>, q, 1, 0, fill);
}

}  // namespace flashgau
