// The residual stream around a block: the block's output, normalised, gated
// and scaled, is added to the stream, and the next block's pre-norm is taken
// in the same pass,
//   r = h + scale * gate * post(y)        n = norm(r)
// and its gradients.  post and norm are the flash_block norms:
//   LayerNorm  (x - mean) / sqrt(var + eps) * g + b     (biased variance)
//   ScaleNorm  g x / max(|x|, eps)                      (g a single scalar)
//
// Backward, with u the normalised row without its parameters and
// w = g * (gradient of the norm's output):
//   LayerNorm  dx = (w - mean(w) - u mean(w u)) / sqrt(var + eps)
//   ScaleNorm  dx = (w - u sum(w u)) / max(|x|, eps), the second term only
//              where |x| > eps
//   dh = dr + dx_norm(dn; r)      dgate = dh * post(y) * scale
//   dy = dx_post(dh * scale * gate; y)
// and the column sums over the rows for the parameters.
//
// Both directions only move rows (at d = 768, bf16: 4 rows in and out
// forward, 6 to 8 backward), so each value is read once and stays in
// registers.  A thread block is one row wide (8 columns a thread) and takes
// R rows at a time, so that the barriers of the row sums are shared by R rows
// and R rows' loads are in flight; a thread keeps its columns for the whole
// launch, so the parameters, and backward the column sums of their
// gradients, stay in registers too.  Statistics are fp32: within a warp the
// mean first and the squares around it second, warps joined by their counts
// (no difference of large squares).
#include <cuda_bf16.h>

#include "flash_gau_internal.h"
#include "sm103_ptx.cuh"

namespace flashgau {
namespace {

constexpr int kCols = 8;        // columns of a thread
constexpr int kMaxWarps = 16;   // of a block: d <= 4096
constexpr unsigned kAll = 0xffffffffu;

struct Args {
  const void *h, *y, *gate;  // backward: h is the stored r; y may be null there
                             // where nothing needs its values
  const void *dr, *dn;
  void *r, *n;               // forward outputs
  void *dh, *dy, *dgate;     // backward outputs
  const float *norm_g, *norm_b, *post_g, *post_b, *scale;
  float *part;               // backward: [blocks][kSums][d] column sums
  long long M;
  int d, norm, post;
  float eps;
};

// the column sums, in the workspace's order
enum { kNormG = 0, kNormB = 1, kPostG = 2, kPostB = 3, kScale = 4, kSums = 5 };

// Column q of thread t.  VEC elements are consecutive: 8 (bf16) or 4 (fp32)
// for 16-byte accesses, or 1, any d and alignment.
template <int VEC>
__device__ __forceinline__ int column(int t, int threads, int q) {
  if (VEC == 8) return t * 8 + q;
  if (VEC == 4) return (q / 4) * threads * 4 + t * 4 + q % 4;
  return q * threads + t;
}

// Eight values of one row as loaded (bf16 packed).
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  float x[8];
  __device__ float get(int q) const { return x[q]; }
  __device__ void set(int q, float v) { x[q] = v; }
};
template <>
struct Raw<__nv_bfloat16> {
  uint32_t w[4];
  __device__ float get(int q) const {
    return __uint_as_float((q & 1) ? (w[q / 2] & 0xffff0000u) : (w[q / 2] << 16));
  }
  __device__ void set2(int q2, float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    w[q2] = *reinterpret_cast<const uint32_t *>(&v);
  }
};

template <typename T, int VEC>
__device__ __forceinline__ void load_row(const void *base, long long row, int d, int t, int threads,
                                         Raw<T> &out) {
  const T *p = static_cast<const T *>(base) + row * d;
  if constexpr (VEC == 8) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (t * 8 < d) v = *reinterpret_cast<const uint4 *>(p + t * 8);
    out.w[0] = v.x; out.w[1] = v.y; out.w[2] = v.z; out.w[3] = v.w;
  } else if constexpr (VEC == 4) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = column<4>(t, threads, 4 * k);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c < d) v = *reinterpret_cast<const float4 *>(p + c);
      out.x[4 * k] = v.x; out.x[4 * k + 1] = v.y; out.x[4 * k + 2] = v.z; out.x[4 * k + 3] = v.w;
    }
  } else {
    float x[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int c = column<1>(t, threads, q);
      x[q] = c < d ? (float)p[c] : 0.f;
    }
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int q = 0; q < 8; ++q) out.set(q, x[q]);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) out.set2(q, x[2 * q], x[2 * q + 1]);
    }
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void store_row(void *base, long long row, int d, int t, int threads,
                                          const float (&x)[8]) {
  T *p = static_cast<T *>(base) + row * d;
  if constexpr (VEC == 8) {
    Raw<__nv_bfloat16> o;
#pragma unroll
    for (int q = 0; q < 4; ++q) o.set2(q, x[2 * q], x[2 * q + 1]);
    if (t * 8 < d) *reinterpret_cast<uint4 *>(p + t * 8) = make_uint4(o.w[0], o.w[1], o.w[2], o.w[3]);
  } else if constexpr (VEC == 4) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = column<4>(t, threads, 4 * k);
      if (c < d)
        *reinterpret_cast<float4 *>(p + c) =
            make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
    }
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int c = column<1>(t, threads, q);
      if (c < d) p[c] = (T)x[q];
    }
  }
}

// a parameter's values in this thread's columns (`fill` where there is none)
template <int VEC>
__device__ __forceinline__ void load_param(const float *p, int d, int t, int threads, float fill,
                                           float (&x)[8]) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int c = column<VEC>(t, threads, q);
    x[q] = p ? (c < d ? __ldg(p + c) : 0.f) : fill;
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// Sums and statistics over a row, R rows at a time, for a block of one or
// more warps.  Buffers alternate, so one barrier a reduction is enough: a
// warp writes a buffer again only after the barrier that follows every
// warp's reading of it.
template <int R>
struct Rows {
  float2 (*buf)[kMaxWarps][2 * R];  // [2]
  const float *count;               // columns of each warp
  int warps, warp, lane, d;
  int flip;

  // every warp's 2 R pairs; `use` reads them in order
  template <typename Use>
  __device__ void exchange(const float2 (&x)[2 * R], Use use) {
    if (warps == 1) {
#pragma unroll
      for (int k = 0; k < 2 * R; ++k) use(0, k, x[k]);
      return;
    }
    if (lane == 0) {
#pragma unroll
      for (int k = 0; k < 2 * R; ++k) buf[flip][warp][k] = x[k];
    }
    __syncthreads();
    for (int w = 0; w < warps; ++w)
#pragma unroll
      for (int k = 0; k < 2 * R; ++k) use(w, k, buf[flip][w][k]);
    flip ^= 1;
  }
};

// (mean, 1 / spread) of a row from its warps' (mean, squares around it): the
// LayerNorm's 1 / sqrt(var + eps), or the ScaleNorm's 1 / max(|x|, eps)
struct Stat {
  float mean, inv;
  bool long_;  // ScaleNorm: |x| > eps
};

// this warp's (mean, sum of squares around it) of one row
template <int VEC>
__device__ __forceinline__ float2 warp_stat(const float (&x)[8], int kind, float count, int d,
                                            int t, int threads) {
  float mean = 0.f;
  if (kind == FLASH_GAU_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) s += x[q];  // zeros behind the row
    mean = warp_sum(s) / count;
  }
  float s2 = 0.f;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const float c = column<VEC>(t, threads, q) < d ? x[q] - mean : 0.f;
    s2 = fmaf(c, c, s2);
  }
  return make_float2(mean, warp_sum(s2));
}

// Joins the warps' statistics: pairs 0 .. R - 1 are of norm ka, the others of
// norm kb.
template <int R>
__device__ __forceinline__ void join(Rows<R> &rows, const float2 (&x)[2 * R], int ka, int kb,
                                     float eps, Stat (&out)[2 * R]) {
  float m2[2 * R], means[2 * R];
#pragma unroll
  for (int k = 0; k < 2 * R; ++k) m2[k] = means[k] = 0.f;
  // joined one warp at a time: the running mean and the squares around it
  float seen = 0.f, ratio = 1.f, weight = 0.f;
  rows.exchange(x, [&](int w, int k, float2 v) {
    if (k == 0) {
      const float c = rows.count[w];
      ratio = c / (seen + c);
      weight = seen * ratio;
      seen += c;
    }
    const float delta = v.x - means[k];
    means[k] = fmaf(delta, ratio, means[k]);
    m2[k] += fmaf(delta * delta, weight, v.y);
  });
#pragma unroll
  for (int k = 0; k < 2 * R; ++k) {
    const int kind = k < R ? ka : kb;
    out[k].mean = means[k];
    if (kind == FLASH_GAU_NORM_LAYER) {
      out[k].inv = 1.0f / sqrtf(m2[k] / (float)rows.d + eps);
      out[k].long_ = true;
    } else {
      const float len = sqrtf(m2[k]);
      out[k].inv = 1.0f / fmaxf(len, eps);
      out[k].long_ = len > eps;
    }
  }
}

template <int R>
__device__ __forceinline__ Rows<R> make_rows(float2 (*buf)[kMaxWarps][2 * R], float *count, int d,
                                             int own) {
  Rows<R> rows;
  rows.buf = buf;
  rows.count = count;
  rows.warps = blockDim.x >> 5;
  rows.warp = threadIdx.x >> 5;
  rows.lane = threadIdx.x & 31;
  rows.d = d;
  rows.flip = 0;
  const float c = warp_sum((float)own);
  if (rows.lane == 0) count[rows.warp] = c;
  __syncthreads();
  return rows;
}

template <int VEC>
__device__ __forceinline__ int own_columns(int d, int t, int threads) {
  int n = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) n += column<VEC>(t, threads, q) < d;
  return n;
}

template <typename T, int VEC, int R, int MAXT>
__global__ void __launch_bounds__(MAXT) residual_norm_kernel(const Args a) {
  __shared__ float2 buf[2][kMaxWarps][2 * R];
  __shared__ float count[kMaxWarps];
  const int t = threadIdx.x, threads = blockDim.x, d = a.d;
  Rows<R> rows = make_rows<R>(buf, count, d, own_columns<VEC>(d, t, threads));
  ptx::griddep_wait();
  const bool post_layer = a.post == FLASH_GAU_NORM_LAYER, layer = a.norm == FLASH_GAU_NORM_LAYER;
  float pg[8], pb[8], sc[8], ng[8], nb[8];
  load_param<VEC>(post_layer ? a.post_g : nullptr, d, t, threads, a.post ? (post_layer ? 1.f : a.post_g[0]) : 1.f, pg);
  load_param<VEC>(post_layer ? a.post_b : nullptr, d, t, threads, 0.f, pb);
  load_param<VEC>(a.scale, d, t, threads, 1.f, sc);
  load_param<VEC>(layer ? a.norm_g : nullptr, d, t, threads, a.norm ? (layer ? 1.f : a.norm_g[0]) : 1.f, ng);
  load_param<VEC>(layer ? a.norm_b : nullptr, d, t, threads, 0.f, nb);
  const float wc = count[rows.warp];
  for (long long row0 = (long long)blockIdx.x * R; row0 < a.M; row0 += (long long)gridDim.x * R) {
    Raw<T> h[R], y[R], gt[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const long long row = min(row0 + k, a.M - 1);
      load_row<T, VEC>(a.h, row, d, t, threads, h[k]);
      if (a.y) load_row<T, VEC>(a.y, row, d, t, threads, y[k]);
      if (a.gate) load_row<T, VEC>(a.gate, row, d, t, threads, gt[k]);
    }
    float r[R][8];
    if (a.y) {
      Stat st[2 * R];
      if (a.post) {
        float2 w[2 * R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
          float x[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) x[q] = y[k].get(q);
          w[k] = warp_stat<VEC>(x, a.post, wc, d, t, threads);
          w[R + k] = make_float2(0.f, 0.f);
        }
        join<R>(rows, w, a.post, a.post, a.eps, st);
      }
#pragma unroll
      for (int k = 0; k < R; ++k)
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          float v = y[k].get(q);
          if (a.post) v = fmaf((v - st[k].mean) * st[k].inv, pg[q], pb[q]);
          if (a.gate) v *= gt[k].get(q);
          r[k][q] = fmaf(v, sc[q], h[k].get(q));
        }
      if (a.r) {
#pragma unroll
        for (int k = 0; k < R; ++k)
          if (row0 + k < a.M) store_row<T, VEC>(a.r, row0 + k, d, t, threads, r[k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < R; ++k)
#pragma unroll
        for (int q = 0; q < 8; ++q) r[k][q] = h[k].get(q);
    }
    if (a.norm) {
      float2 w[2 * R];
      Stat st[2 * R];
#pragma unroll
      for (int k = 0; k < R; ++k) {
        w[k] = warp_stat<VEC>(r[k], a.norm, wc, d, t, threads);
        w[R + k] = make_float2(0.f, 0.f);
      }
      join<R>(rows, w, a.norm, a.norm, a.eps, st);
#pragma unroll
      for (int k = 0; k < R; ++k) {
        float o[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) o[q] = fmaf((r[k][q] - st[k].mean) * st[k].inv, ng[q], nb[q]);
        if (row0 + k < a.M) store_row<T, VEC>(a.n, row0 + k, d, t, threads, o);
      }
    }
  }
}

// The input gradient of a norm from its row sums: x the row, w = g * (its
// output's gradient), s = (sum of w, sum of w u).
__device__ __forceinline__ float norm_grad(float u, float w, float2 s, const Stat &st, int kind,
                                           float inv_d) {
  if (kind == FLASH_GAU_NORM_LAYER) return st.inv * (w - s.x * inv_d - u * (s.y * inv_d));
  return st.inv * (w - (st.long_ ? u * s.y : 0.f));
}

template <typename T, int VEC, int R, int MAXT>
__global__ void __launch_bounds__(MAXT) residual_norm_grad_kernel(const Args a) {
  __shared__ float2 buf[2][kMaxWarps][2 * R];
  __shared__ float count[kMaxWarps];
  const int t = threadIdx.x, threads = blockDim.x, d = a.d;
  Rows<R> rows = make_rows<R>(buf, count, d, own_columns<VEC>(d, t, threads));
  ptx::griddep_wait();
  const bool post_layer = a.post == FLASH_GAU_NORM_LAYER, layer = a.norm == FLASH_GAU_NORM_LAYER;
  float pg[8], pb[8], sc[8], ng[8];
  load_param<VEC>(post_layer ? a.post_g : nullptr, d, t, threads, a.post ? (post_layer ? 1.f : a.post_g[0]) : 1.f, pg);
  load_param<VEC>(post_layer ? a.post_b : nullptr, d, t, threads, 0.f, pb);
  load_param<VEC>(a.scale, d, t, threads, 1.f, sc);
  load_param<VEC>(layer ? a.norm_g : nullptr, d, t, threads, a.norm ? (layer ? 1.f : a.norm_g[0]) : 1.f, ng);
  float acc[kSums][8] = {};
  const float wc = count[rows.warp], inv_d = 1.0f / (float)d;
  const bool need_y = a.y && (a.post || a.gate || a.scale);
  for (long long row0 = (long long)blockIdx.x * R; row0 < a.M; row0 += (long long)gridDim.x * R) {
    Raw<T> x[R], y[R], gt[R], dn[R], dr[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const long long row = min(row0 + k, a.M - 1);
      if (a.norm) {
        load_row<T, VEC>(a.h, row, d, t, threads, x[k]);
        load_row<T, VEC>(a.dn, row, d, t, threads, dn[k]);
      }
      if (need_y) load_row<T, VEC>(a.y, row, d, t, threads, y[k]);
      if (a.gate) load_row<T, VEC>(a.gate, row, d, t, threads, gt[k]);
      if (a.dr) load_row<T, VEC>(a.dr, row, d, t, threads, dr[k]);
    }
    Stat st[2 * R];  // of r, then of y
    if (a.norm || a.post) {
      float2 w[2 * R];
#pragma unroll
      for (int k = 0; k < R; ++k) {
        float v[8];
        w[k] = w[R + k] = make_float2(0.f, 0.f);
        if (a.norm) {
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] = x[k].get(q);
          w[k] = warp_stat<VEC>(v, a.norm, wc, d, t, threads);
        }
        if (a.post) {
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] = y[k].get(q);
          w[R + k] = warp_stat<VEC>(v, a.post, wc, d, t, threads);
        }
      }
      join<R>(rows, w, a.norm, a.post, a.eps, st);
    }
    float dh[R][8];
    if (a.norm) {
      float2 w[2 * R], s[2 * R];
#pragma unroll
      for (int k = 0; k < R; ++k) {
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float u = (x[k].get(q) - st[k].mean) * st[k].inv, g = dn[k].get(q) * ng[q];
          s1 += g;
          s2 = fmaf(g, u, s2);
        }
        w[k] = make_float2(layer ? warp_sum(s1) : 0.f, warp_sum(s2));
        w[R + k] = make_float2(0.f, 0.f);
        s[k] = make_float2(0.f, 0.f);
      }
      rows.exchange(w, [&](int, int k, float2 v) {
        if (k < R) {
          s[k].x += v.x;
          s[k].y += v.y;
        }
      });
#pragma unroll
      for (int k = 0; k < R; ++k) {
        const bool live = row0 + k < a.M;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float u = (x[k].get(q) - st[k].mean) * st[k].inv, g = dn[k].get(q);
          dh[k][q] = norm_grad(u, g * ng[q], s[k], st[k], a.norm, inv_d);
          if (a.dr) dh[k][q] += dr[k].get(q);
          if (live && column<VEC>(t, threads, q) < d) {
            acc[kNormG][q] = fmaf(g, u, acc[kNormG][q]);
            acc[kNormB][q] += g;
          }
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < R; ++k)
#pragma unroll
        for (int q = 0; q < 8; ++q) dh[k][q] = a.dr ? dr[k].get(q) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < R; ++k)
      if (row0 + k < a.M) store_row<T, VEC>(a.dh, row0 + k, d, t, threads, dh[k]);
    if (!a.dy) continue;
    // dh becomes the gradient of post(y)
    float2 w[2 * R], s[2 * R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const bool live = row0 + k < a.M;
      float s1 = 0.f, s2 = 0.f, dg[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const bool in = live && column<VEC>(t, threads, q) < d;
        float u = need_y ? y[k].get(q) : 0.f, p = u;
        if (a.post) {
          u = (u - st[R + k].mean) * st[R + k].inv;
          p = fmaf(u, pg[q], pb[q]);
        }
        const float gv = a.gate ? gt[k].get(q) : 1.f;
        dg[q] = dh[k][q] * p * sc[q];
        if (in) acc[kScale][q] = fmaf(dh[k][q] * p, gv, acc[kScale][q]);
        const float dp = dh[k][q] * gv * sc[q];
        if (in) {
          acc[kPostG][q] = fmaf(dp, u, acc[kPostG][q]);
          acc[kPostB][q] += dp;
        }
        const float g = dp * pg[q];
        dh[k][q] = g;
        if (column<VEC>(t, threads, q) < d) {
          s1 += g;
          s2 = fmaf(g, u, s2);
        }
      }
      if (a.gate && live && a.dgate) store_row<T, VEC>(a.dgate, row0 + k, d, t, threads, dg);
      w[R + k] = make_float2(0.f, 0.f);
      s[k] = make_float2(0.f, 0.f);
      if (a.post) w[k] = make_float2(post_layer ? warp_sum(s1) : 0.f, warp_sum(s2));
    }
    if (a.post) {
      rows.exchange(w, [&](int, int k, float2 v) {
        if (k < R) {
          s[k].x += v.x;
          s[k].y += v.y;
        }
      });
#pragma unroll
      for (int k = 0; k < R; ++k)
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float u = (y[k].get(q) - st[R + k].mean) * st[R + k].inv;
          dh[k][q] = norm_grad(u, dh[k][q], s[k], st[R + k], a.post, inv_d);
        }
    }
#pragma unroll
    for (int k = 0; k < R; ++k)
      if (row0 + k < a.M) store_row<T, VEC>(a.dy, row0 + k, d, t, threads, dh[k]);
  }
  // this block's column sums
  float *part = a.part + (long long)blockIdx.x * kSums * d;
#pragma unroll
  for (int s = 0; s < kSums; ++s)
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int c = column<VEC>(t, threads, q);
      if (c < d) part[s * (long long)d + c] = acc[s][q];
    }
}

struct SumArgs {
  const float *part;
  float *out[kSums];    // null: not wanted
  int scalar[kSums];    // the gradient of a single scalar: also summed over the columns
  int blocks, d;
};

// Sums the blocks' parts in a fixed order: a thread block takes 32 columns of
// one kind (blockIdx.y), 8 threads a column; a scalar's gradient one thread
// block for all its columns.
__global__ void __launch_bounds__(256) sum_parts_kernel(const SumArgs a) {
  ptx::griddep_wait();
  const int s = blockIdx.y;
  if (!a.out[s] || (a.scalar[s] && blockIdx.x)) return;
  __shared__ float buf[8][32];
  const int lane = threadIdx.x & 31, sub = threadIdx.x >> 5;
  float total = 0.f;
  for (int c0 = blockIdx.x * 32; c0 < a.d; c0 += a.scalar[s] ? 32 : a.d) {
    const int c = c0 + lane;
    float v = 0.f;
    if (c < a.d)
      for (int b = sub; b < a.blocks; b += 8) v += a.part[((long long)b * kSums + s) * a.d + c];
    total += v;
  }
  buf[sub][lane] = total;
  __syncthreads();
  if (sub) return;
  float v = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) v += buf[k][lane];
  if (a.scalar[s]) {
    v = warp_sum(v);
    if (lane == 0) a.out[s][0] = v;
  } else if (blockIdx.x * 32 + lane < a.d) {
    a.out[s][blockIdx.x * 32 + lane] = v;
  }
}

bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

constexpr int kRows = 2;  // rows a block takes at a time

int threads_of(int d) { return (d + 32 * kCols - 1) / (32 * kCols) * 32; }

template <typename T, int VEC, int R, int MAXT>
cudaError_t launch(const Args &a, bool grad, int blocks, cudaStream_t stream) {
  const dim3 grid(blocks), block(threads_of(a.d));
  return grad ? launch_pdl(residual_norm_grad_kernel<T, VEC, R, MAXT>, grid, block, 0, stream, a)
              : launch_pdl(residual_norm_kernel<T, VEC, R, MAXT>, grid, block, 0, stream, a);
}

template <typename T, int VEC>
cudaError_t dispatch(const Args &a, bool grad, int blocks, cudaStream_t stream) {
  if (threads_of(a.d) <= 128) return launch<T, VEC, kRows, 128>(a, grad, blocks, stream);
  return launch<T, VEC, 1, 32 * kMaxWarps>(a, grad, blocks, stream);
}

cudaError_t run(const Args &a, bool grad, int dtype, int blocks, cudaStream_t stream) {
  const bool bf16 = dtype == FLASH_GAU_BF16;
  bool vec = a.d % (bf16 ? 8 : 4) == 0;
  for (const void *p : {a.h, a.y, a.gate, a.dr, a.dn, (const void *)a.r, (const void *)a.n,
                        (const void *)a.dh, (const void *)a.dy, (const void *)a.dgate})
    vec = vec && aligned16(p);
  if (bf16)
    return vec ? dispatch<__nv_bfloat16, 8>(a, grad, blocks, stream)
               : dispatch<__nv_bfloat16, 1>(a, grad, blocks, stream);
  return vec ? dispatch<float, 4>(a, grad, blocks, stream)
             : dispatch<float, 1>(a, grad, blocks, stream);
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

int residual_norm_blocks(long long M, int d) {
  const int rows = threads_of(d) <= 128 ? kRows : 1;
  const long long n = (M + rows - 1) / rows;
  return (int)(n < kResidualMaxBlocks ? n : kResidualMaxBlocks);
}

cudaError_t residual_norm(const ResidualProblem &q, const void *h, void *r, void *n) {
  Args a = args_of(q);
  a.h = h;
  a.r = r;
  a.n = n;
  const int rows = threads_of(q.d) <= 128 ? kRows : 1;
  const long long blocks = (q.M + rows - 1) / rows;
  const int most = q.num_sms * (2048 / threads_of(q.d) < 8 ? 2048 / threads_of(q.d) : 8);
  return run(a, false, q.dtype, (int)(blocks < most ? blocks : most), q.stream);
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
  const int blocks = residual_norm_blocks(q.M, q.d);
  cudaError_t err = run(a, true, q.dtype, blocks, q.stream);
  if (err != cudaSuccess) return err;
  SumArgs s = {};
  s.part = a.part;
  s.blocks = blocks;
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
  return launch_pdl(sum_parts_kernel, dim3((q.d + 31) / 32, kSums), dim3(256), 0, q.stream, s);
}

}  // namespace flashgau
