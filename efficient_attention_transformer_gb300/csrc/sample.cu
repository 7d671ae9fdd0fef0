// The next token of each row of logits:
//   w_i = exp((l_i - max l) / T)
// words in falling order of l, equal ones by index; each filter keeps a
// beginning of that order,
//   top_k  the first k
//   top_p  those with less than p of top_k's mass before them
//   min_p  those with w_i >= min_p
// (the first word always), and the token is the first kept word with more
// than u of the kept mass up to its end.
//
// Everything asked of a row is therefore a place in one order: the k-th word,
// the word that reaches a mass.  No row is sorted.  One pass finds the
// largest logit, one adds words and masses into bins of l (2048 over the
// range in which w is not zero), a scan over the bins finds the bin of the
// place, and the few words of that bin are looked at one by one, or, where
// they are many, by bins of their keys, as often as it takes to come down to
// one value.
//
// Masses are whole numbers, w in units of 2^-44 (a power that leaves room for
// V of them): sums do not depend on their order, so a token does not depend on
// the launch, and a word's place is decided to 2^-41 of the mass where fp32
// sums would err once in some hundred tokens of a large vocabulary.  w comes
// from l in pairs of fp32 and 32-bit products: y = (l - max) log2(e) / T =
// k / 1024 + f, w = 2^(k / 1024) (from a table) * 2^f, |f| <= 2^-11, by the
// exponential series to its third power.
#include <cuda_bf16.h>

#include "flash_gau_internal.h"

namespace flashgau {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kBins = 2048, kPer = kBins / kThreads;
constexpr int kFew = 256;    // words of a bin that are compared with one another
constexpr int kList = 4096;  // words of a bin that are held in shared memory
constexpr int kUnit = 44;    // w = 1 is 2^kUnit, less for more than 2^18 words
constexpr float kNoTemperature = 1e-30f;  // below: the largest logit's word

using u64 = unsigned long long;

// 2^(j / 1024) in units of 2^-44, j = 0 .. 1023.
struct Powers {
  u64 v[1024];
  constexpr Powers() : v() {
    for (int j = 0; j < 1024; ++j) {
      // exp(j ln 2 / 1024) by its series, below 1 in argument
      const double x = j * (0.693147180559945309417232121458 / 1024.0);
      double term = 1.0, sum = 1.0;
      for (int i = 1; i < 24; ++i) {
        term *= x / i;
        sum += term;
      }
      v[j] = (u64)(sum * 17592186044416.0 + 0.5);
    }
  }
};
__device__ const Powers kPowers;

// What a row's words are weighed with.
struct Weigh {
  float top;     // largest logit
  float ch, cl;  // log2(e) / T as a pair
  int drop;      // bits of the unit given up for many words
  const u64 *pow;

  __device__ u64 operator()(float l) const {
    // l - top and its rounding error, times the pair
    const float dh = l - top, bv = l - dh, av = dh + bv;
    const float dl = (l - av) + (bv - top);
    const float yh = dh * ch;
    if (!(yh > -50.f)) return 0;  // minus infinity too
    const float yl = fmaf(dh, cl, fmaf(dl, ch, fmaf(dh, ch, -yh)));
    const float magic = 12582912.f;  // 1.5 * 2^23
    const float tm = fmaf(yh, 1024.f, magic), t = tm - magic;
    const int k = __float_as_int(tm) - 0x4b400000;
    const float fh = fmaf(t, -1.f / 1024.f, yh);
    // x = 2^f - 1 in units of 2^-41: f ln 2 + (f ln 2)^2 / 2 + (f ln 2)^3 / 6
    const float xf = fh * 0.693147181f, xl = yl * 0.693147181f;
    const float rest = fmaf(xl, 1.f + xf, xf * xf * fmaf(xf, 1.f / 6.f, 0.5f));
    const int fi = __float2int_rn(fh * 0x1p41f);
    const long long x1 = ((long long)fi * 2977044472LL) >> 32;  // ln 2 * 2^32
    const int x = (int)x1 + __float2int_rn(rest * 0x1p41f);
    const u64 p = pow[k & 1023];
    const u64 w = p + (u64)(((long long)(int)(p >> 14) * x) >> 27);
    const int down = drop - (k >> 10);
    return (w + ((1ull << down) >> 1)) >> down;
  }
};

__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t b = __float_as_uint(l + 0.f);  // minus zero is zero
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key ^ (key & 0x80000000u ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// f(l, i) for every word of a row: 16 bytes a load between its boundaries.
template <typename T, typename F>
__device__ __forceinline__ void each(const T *row, int V, const F &f) {
  constexpr int kVec = 16 / sizeof(T);
  const int head = min(V, (int)((16 - reinterpret_cast<uintptr_t>(row) % 16) % 16 / sizeof(T)));
  const int body = (V - head) / kVec, tail = head + body * kVec;
  if ((int)threadIdx.x < head) f(as_float(row[threadIdx.x]), (int)threadIdx.x);
  const uint4 *v = reinterpret_cast<const uint4 *>(row + head);
#pragma unroll 2
  for (int k = threadIdx.x; k < body; k += kThreads) {
    const uint4 w = v[k];
    const int i = head + k * kVec;
    const uint32_t part[4] = {w.x, w.y, w.z, w.w};
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int q = 0; q < 4; ++q) f(__uint_as_float(part[q]), i + q);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f(__uint_as_float(part[q] << 16), i + 2 * q);
        f(__uint_as_float(part[q] & 0xffff0000u), i + 2 * q + 1);
      }
    }
  }
  if (tail + (int)threadIdx.x < V) f(as_float(row[tail + threadIdx.x]), tail + (int)threadIdx.x);
}

struct Bins {
  uint32_t count[kBins], low[kBins], high[kBins];
  __device__ void clear() {
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int b = threadIdx.x + q * kThreads;
      count[b] = low[b] = high[b] = 0;
    }
  }
  __device__ void add(int b, u64 w) {
    atomicAdd(&count[b], 1u);
    const uint32_t l = (uint32_t)w;
    uint32_t h = (uint32_t)(w >> 32);
    if (l) h += atomicAdd(&low[b], l) + l < l;
    if (h) atomicAdd(&high[b], h);
  }
  __device__ u64 mass(int b) const { return (u64)high[b] << 32 | low[b]; }
};

struct Shared {
  Bins first, fine;
  u64 pow[1024];
  uint32_t key[kList];
  int index[kList];
  u64 weight[kFew];
  // scans
  u64 warp_mass[kWarps];
  uint32_t warp_count[kWarps];
  // results
  u64 mass;
  uint32_t count;
  int bin, listed;
  uint32_t lo, hi;
  float top;
  int bad, finite, at;
  u64 sum_mass, q_mass;
  uint32_t q_count;
};

// A place in the order of words: all words above `key`, and `ties` of those
// with that key.
struct Place {
  uint32_t key;
  uint32_t ties, equal;   // wanted, and how many there are
  u64 count, mass;        // through the place
  u64 weight;             // of a word with this key
  int index;              // of the word at the place where it is known, or -1
};

// The first bin in falling order of l (rising index) whose words or masses,
// with those of the bins before it and `count0`, `mass0`, reach `target`.
// Leaves it in s.bin, and what lies before it in s.count and s.mass.
__device__ void find_bin(Shared &s, const Bins &b, bool by_mass, u64 target, u64 count0,
                         u64 mass0) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  uint32_t c[kPer], ct = 0;
  u64 m[kPer], mt = 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int at = threadIdx.x * kPer + q;
    c[q] = b.count[at];
    m[q] = b.mass(at);
    ct += c[q];
    mt += m[q];
  }
  uint32_t ci = ct;
  u64 mi = mt;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t cu = __shfl_up_sync(kAll, ci, o);
    const u64 mu = __shfl_up_sync(kAll, mi, o);
    if (lane >= o) {
      ci += cu;
      mi += mu;
    }
  }
  if (lane == 31) {
    s.warp_count[warp] = ci;
    s.warp_mass[warp] = mi;
  }
  __syncthreads();
  if (warp == 0) {
    uint32_t cw = s.warp_count[lane];
    u64 mw = s.warp_mass[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t cu = __shfl_up_sync(kAll, cw, o);
      const u64 mu = __shfl_up_sync(kAll, mw, o);
      if (lane >= o) {
        cw += cu;
        mw += mu;
      }
    }
    s.warp_count[lane] = cw;
    s.warp_mass[lane] = mw;
  }
  __syncthreads();
  u64 cb = count0 + ci - ct + (warp ? s.warp_count[warp - 1] : 0);
  u64 mb = mass0 + mi - mt + (warp ? s.warp_mass[warp - 1] : 0);
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const u64 before = by_mass ? mb : cb, after = before + (by_mass ? m[q] : c[q]);
    if (before < target && target <= after) {
      s.bin = threadIdx.x * kPer + q;
      s.count = (uint32_t)cb;
      s.mass = mb;
    }
    cb += c[q];
    mb += m[q];
  }
  __syncthreads();
}

template <typename T>
struct Row {
  const T *row;
  int V;
  Weigh w;
  float per;  // bins of l a unit of l

  __device__ int bin(float l) const {
    return min(kBins - 1, __float2int_rz((w.top - l) * per));
  }

  // The place at which words (or masses) reach `target`, which lies in bin
  // s.bin of the first bins, s.count words and s.mass before it.
  __device__ Place place(Shared &s, bool by_mass, u64 target) const {
    const int b = s.bin;
    u64 count0 = s.count, mass0 = s.mass;
    const uint32_t n = s.first.count[b];
    __syncthreads();
    if (threadIdx.x == 0) {
      s.listed = 0;
      s.lo = 0xffffffffu;
      s.hi = 0;
    }
    __syncthreads();
    const bool list = n <= kList;
    {
      uint32_t lo = 0xffffffffu, hi = 0;
      each(row, V, [&](float l, int i) {
        if (l > __int_as_float(0xff800000) && bin(l) == b) {
          const uint32_t key = key_of(l);
          lo = min(lo, key);
          hi = max(hi, key);
          if (list) {
            const int at = atomicAdd(&s.listed, 1);
            if (at < kList) {
              s.key[at] = key;
              s.index[at] = i;
            }
          }
        }
      });
      if (lo <= hi) {
        atomicMin(&s.lo, lo);
        atomicMax(&s.hi, hi);
      }
    }
    __syncthreads();
    if (n <= kFew) return place_few(s, by_mass, target, count0, mass0, (int)n);
    uint32_t lo = s.lo, hi = s.hi;
    // down to one key: bins of (hi - key) >> shift, 11 bits of 32 each time
    for (int turn = 0; turn < 3 && lo < hi; ++turn) {
      const int shift = max(0, 32 - __clz(hi - lo) - 11);
      s.fine.clear();
      __syncthreads();
      if (list) {
        for (int k = threadIdx.x; k < (int)n; k += kThreads) {
          const uint32_t key = s.key[k];
          if (key >= lo && key <= hi) s.fine.add((hi - key) >> shift, w(value_of(key)));
        }
      } else {
        each(row, V, [&](float l, int) {
          const uint32_t key = key_of(l);
          if (key >= lo && key <= hi && bin(l) == b) s.fine.add((hi - key) >> shift, w(l));
        });
      }
      __syncthreads();
      find_bin(s, s.fine, by_mass, target, count0, mass0);
      count0 = s.count;
      mass0 = s.mass;
      const uint32_t first = (uint32_t)s.bin << shift;
      const uint32_t nlo = hi - min(hi - lo, first + ((1u << shift) - 1));
      hi -= first;
      lo = nlo;
      if (lo == hi) {
        Place p = at_key(lo, s.fine.count[s.bin], by_mass, target, count0, mass0);
        __syncthreads();
        return p;
      }
      __syncthreads();
    }
    return at_key(lo, n, by_mass, target, count0, mass0);
  }

  __device__ Place at_key(uint32_t key, uint32_t equal, bool by_mass, u64 target, u64 count0,
                          u64 mass0) const {
    Place p;
    p.key = key;
    p.equal = equal;
    p.weight = w(value_of(key));
    p.ties = by_mass ? (uint32_t)((target - mass0 + p.weight - 1) / p.weight)
                     : (uint32_t)(target - count0);
    p.count = count0 + p.ties;
    p.mass = mass0 + p.ties * p.weight;
    p.index = -1;
    return p;
  }

  // Each word of a short list against all of them.
  __device__ Place place_few(Shared &s, bool by_mass, u64 target, u64 count0, u64 mass0,
                             int n) const {
    const int t = threadIdx.x;
    if (t < n) s.weight[t] = w(value_of(s.key[t]));
    __syncthreads();
    if (t < n) {
      const uint32_t key = s.key[t];
      const int index = s.index[t];
      u64 c = count0, m = mass0;
      for (int k = 0; k < n; ++k)
        if (s.key[k] > key || (s.key[k] == key && s.index[k] < index)) {
          c += 1;
          m += s.weight[k];
        }
      const u64 before = by_mass ? m : c, after = before + (by_mass ? s.weight[t] : 1);
      if (before < target && target <= after) {
        s.at = t;
        s.count = (uint32_t)c;
        s.mass = m;
      }
    }
    __syncthreads();
    Place p;
    const int at = s.at;
    p.key = s.key[at];
    p.weight = s.weight[at];
    p.count = s.count + 1;
    p.mass = s.mass + p.weight;
    p.ties = p.equal = 0;
    p.index = s.index[at];
    __syncthreads();
    return p;
  }

  // The ties-th word with this key, by index.
  __device__ int find_index(Shared &s, uint32_t key, uint32_t ties) const {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int span = (V + kWarps - 1) / kWarps, i0 = min(V, warp * span), i1 = min(V, i0 + span);
    uint32_t n = 0;
    for (int i = i0 + lane; i < i1; i += 32) n += key_of(as_float(row[i])) == key;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(kAll, n, o);
    if (lane == 0) s.warp_count[warp] = n;
    __syncthreads();
    uint32_t before = 0;
    for (int k = 0; k < warp; ++k) before += s.warp_count[k];
    if (before < ties && ties <= before + n) {
      for (int i = i0; i < i1; i += 32) {
        const bool is = i + lane < i1 && key_of(as_float(row[i + lane])) == key;
        const unsigned all = __ballot_sync(kAll, is);
        if (is && before + __popc(all & ((2u << lane) - 1)) == ties) s.at = i + lane;
        before += __popc(all);
      }
    }
    __syncthreads();
    return s.at;
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads)
sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(16) unsigned char raw[];
  Shared &s = *reinterpret_cast<Shared *>(raw);
  const int tid = threadIdx.x, lane = tid % 32;
  const long long n = blockIdx.x;
  Row<T> r;
  r.row = static_cast<const T *>(a.logits) + n * a.ld;
  r.V = a.V;

  // the largest logit
  if (tid == 0) {
    s.bad = s.finite = s.bin = s.at = 0;
    s.lo = 0;
    s.sum_mass = s.q_mass = 0;
    s.q_count = 0;
  }
  s.first.clear();
  for (int j = tid; j < 1024; j += kThreads) s.pow[j] = kPowers.v[j];
  __syncthreads();
  {
    uint32_t top = 0;
    int bad = 0, finite = 0;
    each(r.row, a.V, [&](float l, int) {
      bad |= !(l < __int_as_float(0x7f800000));
      finite += l > __int_as_float(0xff800000);
      top = max(top, key_of(l));
    });
    bad = __any_sync(kAll, bad);
    top = __reduce_max_sync(kAll, top);
    finite = __reduce_add_sync(kAll, finite);
    if (lane == 0) {
      if (bad) s.bad = 1;
      atomicMax(&s.lo, top);
      atomicAdd(&s.finite, finite);
    }
  }
  __syncthreads();
  const uint32_t top_key = s.lo;
  const int finite = s.finite;
  const float temperature = a.temperature ? a.temperature[n] : 1.f;
  const int top_k = a.top_k ? a.top_k[n] : 0;
  const float top_p = a.top_p ? a.top_p[n] : 1.f, min_p = a.min_p ? a.min_p[n] : 0.f;
  float u = a.u[n];
  // settings that are no numbers, or a row without a distribution
  if (s.bad || !finite || !(temperature >= 0.f) || top_p != top_p || min_p != min_p ||
      !(u >= 0.f)) {
    if (tid == 0) {
      a.token[n] = -1;
      if (a.logp) a.logp[n] = __int_as_float(0x7fc00000);
      if (a.kept) a.kept[n] = 0;
    }
    return;
  }
  u = fminf(u, 0x1.fffffep-1f);
  r.w.top = value_of(top_key);
  if (temperature < kNoTemperature) {
    const int at = r.find_index(s, top_key, 1);
    if (tid == 0) {
      a.token[n] = at;
      if (a.logp) a.logp[n] = 0.f;
      if (a.kept) a.kept[n] = 1;
    }
    return;
  }
  const double c = 1.4426950408889634074 / (double)temperature;
  r.w.ch = (float)c;
  r.w.cl = (float)(c - (double)r.w.ch);
  r.w.drop = a.drop;
  r.w.pow = s.pow;
  // the bins' range: weights down to 2^-46
  r.per = (float)(kBins - 1) / 46.f * r.w.ch;

  // top_k's bin, so that no weight is taken behind it
  int last_bin = kBins - 1;
  u64 k_count = 0;
  if (top_k > 0 && top_k < finite) {
    k_count = (u64)top_k;
    each(r.row, a.V, [&](float l, int) {
      if (l > __int_as_float(0xff800000)) atomicAdd(&s.first.count[r.bin(l)], 1u);
    });
    __syncthreads();
    find_bin(s, s.first, false, k_count, 0, 0);
    last_bin = s.bin;
    __syncthreads();
    s.first.clear();
    __syncthreads();
  }
  // words and masses by bins; those that min_p keeps apart
  const bool by_min = min_p > 0.f;
  float least = 0.f;  // the smallest logit that min_p lets through
  if (by_min) {
    const double x = (double)r.w.top + (double)temperature * log((double)fminf(min_p, 1.f));
    least = __double2float_ru(x);
  }
  {
    u64 mass = 0, q_mass = 0;
    uint32_t q_count = 0;
    each(r.row, a.V, [&](float l, int) {
      if (!(l > __int_as_float(0xff800000))) return;
      const int b = r.bin(l);
      if (b > last_bin) return;
      const u64 w = r.w(l);
      s.first.add(b, w);
      mass += w;
      if (by_min && l >= least) {
        q_mass += w;
        ++q_count;
      }
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      mass += __shfl_xor_sync(kAll, mass, o);
      q_mass += __shfl_xor_sync(kAll, q_mass, o);
      q_count += __shfl_xor_sync(kAll, q_count, o);
    }
    if (lane == 0) {
      atomicAdd(&s.sum_mass, mass);
      atomicAdd(&s.q_mass, q_mass);
      atomicAdd(&s.q_count, q_count);
    }
  }
  __syncthreads();
  u64 kept = (u64)finite, mass = s.sum_mass;
  const u64 q_mass = s.q_mass;
  const uint32_t q_count = s.q_count;
  if (k_count) {
    find_bin(s, s.first, false, k_count, 0, 0);
    const Place p = r.place(s, false, k_count);
    kept = p.count;
    mass = p.mass;
  }
  if (top_p < 1.f) {
    const double share = top_p > 0.f ? (double)top_p * (double)mass : 0.0;
    u64 target = (u64)ceil(share);
    target = target < 1 ? 1 : target > mass ? mass : target;
    find_bin(s, s.first, true, target, 0, 0);
    const Place p = r.place(s, true, target);
    if (p.count < kept) {
      kept = p.count;
      mass = p.mass;
    }
  }
  if (by_min && q_count < kept) {
    kept = q_count;
    mass = q_mass;
  }
  u64 target = (u64)((double)u * (double)mass) + 1;
  if (target > mass) target = mass;
  find_bin(s, s.first, true, target, 0, 0);
  const Place p = r.place(s, true, target);
  const int at = p.index >= 0 ? p.index : r.find_index(s, p.key, p.ties);
  if (tid == 0) {
    a.token[n] = at;
    if (a.logp) {
      // (l - top) / T less the logarithm of the mass
      const double z = ((double)value_of(p.key) - (double)r.w.top) / (double)temperature;
      a.logp[n] = (float)(z - log(ldexp((double)mass, a.drop - kUnit)));
    }
    if (a.kept) a.kept[n] = (int)kept;
  }
}

template <typename T>
cudaError_t launch(const SampleArgs &a, int N, cudaStream_t stream) {
  const cudaError_t err = cudaFuncSetAttribute(
      sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared));
  if (err != cudaSuccess) return err;
  sample_kernel<T><<<N, kThreads, sizeof(Shared), stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t sample(SampleArgs a, int N, int dtype, cudaStream_t stream) {
  a.drop = 0;
  while (kUnit - a.drop > 0 && ((long long)a.V << (kUnit - a.drop)) > (1LL << 62)) ++a.drop;
  return dtype == FLASH_GAU_BF16 ? launch<__nv_bfloat16>(a, N, stream) : launch<float>(a, N, stream);
}

}  // namespace flashgau
