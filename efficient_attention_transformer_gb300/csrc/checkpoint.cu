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
// codes times their group's scale, the values that the checkpoint stands for
__device__ __forceinline__ void load_codes(const signed char *codes, const float *scales, int c,
                                           int d, bool vec, float (&x)[8]) {
  if (vec) {
    const uint2 w = c < d ? *reinterpret_cast<const uint2 *>(codes + c) : make_uint2(0, 0);
    const float s = c < d ? scales[c / kGroup] : 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const uint32_t v = q < 4 ? w.x : w.y;
      x[q] = (float)(signed char)(v >> (8 * (q & 3))) * s;
    }
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

// What the threads of a row share: WARPS warps, one row each time.
template <int WARPS>
struct RowSum {
  float *part;  // [2][WARPS] shared, WARPS > 1
  int turn = 0;
  __device__ float operator()(float v) {
    v = warp_sum(v);
    if (WARPS == 1) return v;
    float *p = part + turn * WARPS;  // two turns: the last sum may still be read
    turn ^= 1;
    if (threadIdx.x % 32 == 0) p[threadIdx.x / 32] = v;
    __syncthreads();
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
__global__ void __launch_bounds__(128) pack_kernel(const CheckpointArgs a) {
  __shared__ float part[2 * WARPS];
  RowSum<WARPS> sum{part};
  const int t = threadIdx.x % (32 * WARPS);
  const long long m = (long long)blockIdx.x * (4 / WARPS) + threadIdx.x / (32 * WARPS);
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
__global__ void __launch_bounds__(128) restore_kernel(const CheckpointArgs a) {
  __shared__ float part[2 * WARPS];
  RowSum<WARPS> sum{part};
  const int t = threadIdx.x % (32 * WARPS);
  const long long m = (long long)blockIdx.x * (4 / WARPS) + threadIdx.x / (32 * WARPS);
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
template <typename T, int NC, int WARPS>
__global__ void __launch_bounds__(128) backward_kernel(const CheckpointArgs a) {
  __shared__ float part[2 * WARPS];
  extern __shared__ float cols[];  // [2][d], one row of warps after another
  RowSum<WARPS> sum{part};
  const int t = threadIdx.x % (32 * WARPS), rows = 4 / WARPS;
  const bool layer = a.norm == FLASH_GAU_NORM_LAYER, vec = a.vec;
  const float inv_d = 1.0f / (float)a.d, g1 = layer ? 0.f : a.norm_g[0];
  float sg[NC][8], sb[NC][8], s1 = 0.f;
#pragma unroll
  for (int k = 0; k < NC; ++k)
#pragma unroll
    for (int q = 0; q < 8; ++q) sg[k][q] = sb[k][q] = 0.f;
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
    float length2 = 0.f;
    const float inv = normalise<NC, WARPS>(x, a.norm, t, a.d, a.eps, sum, &length2);
    float sw = 0.f, swu = 0.f;
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = (k * 32 * WARPS + t) * 8;
      float g[8];
      if (layer) load8(a.norm_g, c, a.d, a.vec_param, g);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (layer) {
          sg[k][q] = fmaf(w[k][q], x[k][q], sg[k][q]);
          sb[k][q] += w[k][q];
        } else {
          s1 = fmaf(w[k][q], x[k][q], s1);
        }
        w[k][q] *= layer ? g[q] : g1;
        sw += w[k][q];
        swu = fmaf(w[k][q], x[k][q], swu);
      }
    }
    swu = sum(swu);
    float mw = 0.f, mwu;
    if (layer) {
      mw = sum(sw) * inv_d;
      mwu = swu * inv_d;
    } else {
      mwu = length2 > a.eps * a.eps ? swu : 0.f;
    }
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = (k * 32 * WARPS + t) * 8;
      float v[8];
      if (a.dr) load8(static_cast<const T *>(a.dr) + at, c, a.d, vec, v);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float dx = inv * (w[k][q] - mw - x[k][q] * mwu);
        v[q] = a.dr ? v[q] + dx : dx;
      }
      store8(static_cast<T *>(a.dh) + at, c, a.d, vec, v);
    }
  }
  if (!a.part) return;
  if (!layer) {
    s1 = warp_sum(s1);
    if (threadIdx.x % 32 == 0) a.part[(long long)blockIdx.x * 4 + threadIdx.x / 32] = s1;
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
  for (int c = threadIdx.x; c < 2 * a.d; c += 128) to[c] = cols[c];
}

// Adds the blocks' sums up: 32 columns a block, 8 warps taking every eighth
// block's row, then the eight in order.
__global__ void __launch_bounds__(256)
join_columns_kernel(const float *__restrict__ part, int blocks, int d, float *__restrict__ dg,
                    float *__restrict__ db) {
  __shared__ float s[8][32];
  const int c = blockIdx.x * 32 + threadIdx.x % 32, w = threadIdx.x / 32;
  float v = 0.f;
  if (c < 2 * d)
    for (int b = w; b < blocks; b += 8) v += part[(long long)b * 2 * d + c];
  s[w][threadIdx.x % 32] = v;
  __syncthreads();
  if (w == 0 && c < 2 * d) {
#pragma unroll
    for (int k = 1; k < 8; ++k) v += s[k][threadIdx.x];
    float *to = c < d ? dg : db;
    if (to) to[c < d ? c : c - d] = v;
  }
}
// ScaleNorm's one g: n sums.  In 64 bits, because terms of both signs nearly cancel.
__global__ void __launch_bounds__(256)
join_scalar_kernel(const float *__restrict__ part, int n, float *__restrict__ dg) {
  __shared__ double s[256];
  double v = 0.0;
  for (int k = threadIdx.x; k < n; k += 256) v += (double)part[k];
  s[threadIdx.x] = v;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if (threadIdx.x < o) s[threadIdx.x] += s[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) *dg = (float)s[0];
}

enum { kPack, kRestore, kBackward };

template <int WHAT, typename T, int NC, int WARPS>
cudaError_t launch(const CheckpointArgs &a, unsigned grid, cudaStream_t stream) {
  if constexpr (WHAT == kPack) {
    pack_kernel<T, NC, WARPS><<<grid, 128, 0, stream>>>(a);
  } else if constexpr (WHAT == kRestore) {
    restore_kernel<T, NC, WARPS><<<grid, 128, 0, stream>>>(a);
  } else {
    const size_t smem = a.part && a.norm == FLASH_GAU_NORM_LAYER ? 2 * a.d * sizeof(float) : 0;
    if (smem > 48 * 1024) {
      const cudaError_t err = cudaFuncSetAttribute(
          backward_kernel<T, NC, WARPS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (err != cudaSuccess) return err;
    }
    backward_kernel<T, NC, WARPS><<<grid, 128, smem, stream>>>(a);
  }
  return cudaGetLastError();
}

// One warp a row up to 1024 columns, four beyond.
template <int WHAT, typename T>
cudaError_t dispatch(const CheckpointArgs &a, unsigned most_blocks, cudaStream_t stream) {
  const int rows = a.d <= 1024 ? 4 : 1;
  const long long blocks = (a.M + rows - 1) / rows;
  const unsigned grid = (unsigned)(most_blocks && blocks > most_blocks ? most_blocks : blocks);
  if (a.d <= 256) return launch<WHAT, T, 1, 1>(a, grid, stream);
  if (a.d <= 512) return launch<WHAT, T, 2, 1>(a, grid, stream);
  if (a.d <= 768) return launch<WHAT, T, 3, 1>(a, grid, stream);
  if (a.d <= 1024) return launch<WHAT, T, 4, 1>(a, grid, stream);
  if (a.d <= 2048) return launch<WHAT, T, 2, 4>(a, grid, stream);
  if (a.d <= 4096) return launch<WHAT, T, 4, 4>(a, grid, stream);
  return launch<WHAT, T, 8, 4>(a, grid, stream);
}

template <int WHAT>
cudaError_t dispatch(const CheckpointArgs &a, int dtype, unsigned most_blocks,
                     cudaStream_t stream) {
  return dtype == FLASH_GAU_BF16 ? dispatch<WHAT, __nv_bfloat16>(a, most_blocks, stream)
                                 : dispatch<WHAT, float>(a, most_blocks, stream);
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
  return (size_t)kCheckpointBlocks * 2 * (d < 4 ? 4 : d) * sizeof(float);
}

cudaError_t checkpoint_backward(const CheckpointArgs &args, float *dg, float *db, int dtype,
                                cudaStream_t stream) {
  CheckpointArgs a = finish(args);
  if (!dg && !db) a.part = nullptr;
  cudaError_t err = dispatch<kBackward>(a, dtype, kCheckpointBlocks, stream);
  if (err != cudaSuccess || !a.part) return err;
  const int rows = a.d <= 1024 ? 4 : 1;
  const long long all = (a.M + rows - 1) / rows;
  const int blocks = (int)(all < kCheckpointBlocks ? all : kCheckpointBlocks);
  if (a.norm == FLASH_GAU_NORM_LAYER)
    join_columns_kernel<<<(2 * a.d + 31) / 32, 256, 0, stream>>>(a.part, blocks, a.d, dg, db);
  else
    join_scalar_kernel<<<1, 256, 0, stream>>>(a.part, blocks * 4, dg);
  return cudaGetLastError();
}

}  // namespace flashgau
