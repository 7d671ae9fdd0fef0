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
// the word that reaches a mass.  No row is sorted: words and masses are added
// into bins that keep the order, and a scan over the bins finds the one that
// holds a place.
//
// Masses are whole numbers, w in units of 2^-44 (a power that leaves room for
// V of them): sums do not depend on their order, so a token does not depend on
// the launch, and a word's place is decided to 2^-40 of the mass where fp32
// sums would err once in some hundred tokens of a large vocabulary.  Nothing
// here is in fp64, whose units are so few that one thread's logarithm took
// longer than a whole row's search: pairs of fp32 numbers and products of whole
// numbers give the digits.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "flash_gau_internal.h"

namespace flashgau {
namespace {

namespace cg = cooperative_groups;

constexpr unsigned kAll = 0xffffffffu;
constexpr int kBins = 2048;
constexpr int kFew = 256;    // words of a bin that are compared with one another
constexpr int kList = 1024;  // words of a bin that are held in shared memory
constexpr int kUnit = 44;    // w = 1 is 2^kUnit, less for more than 2^18 words
constexpr float kNoTemperature = 1e-30f;  // below: the largest logit's word
constexpr float kInf = __builtin_huge_valf();

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

// 2^(yh + yl) in units of 2^-(44 - drop), for -50 < yh <= 0 and yl below its last
// places: y = k / 1024 + f with |f| <= 2^-11, 2^(k / 1024) from the table and
// 2^f by the exponential series to its third power, in units of 2^-41.
__device__ __forceinline__ u64 power(float yh, float yl, int drop, const u64 *pow) {
  const float magic = 12582912.f;  // 1.5 * 2^23
  const float tm = fmaf(yh, 1024.f, magic), t = tm - magic;
  const int k = __float_as_int(tm) - 0x4b400000;
  const float fh = fmaf(t, -1.f / 1024.f, yh);
  const float xf = fh * 0.693147181f, xl = yl * 0.693147181f;
  const float rest = fmaf(xf, fmaf(xf, fmaf(xf, 1.f / 6.f, 0.5f), xl), xl);
  const int fi = __float2int_rn(fh * 0x1p41f);
  const long long x1 = ((long long)fi * 2977044472LL) >> 32;  // ln 2 * 2^32
  const int x = (int)x1 + __float2int_rn(rest * 0x1p41f);
  const u64 p = pow[k & 1023];
  const u64 w = p + (u64)(((long long)(int)(p >> 14) * x) >> 27);
  const int down = drop - (k >> 10);
  return (w + ((1ull << down) >> 1)) >> down;
}

// Sums (Knuth) and products (Dekker, by a fused addition) of fp32 numbers with
// what their rounding cuts off.
struct Pair {
  float h, l;
};
__device__ __forceinline__ Pair add(float a, float b) {
  const float s = a + b, bv = s - a, av = s - bv;
  return {s, (a - av) + (b - bv)};
}
__device__ __forceinline__ Pair times(float a, float bh, float bl) {
  const float p = a * bh;
  return {p, fmaf(a, bl, fmaf(a, bh, -p))};
}
// log2(e), and ln 2 in two parts, the first with 15 bits
constexpr float kLog2eH = 1.44269502f, kLog2eL = 1.92596303e-8f;
constexpr float kLn2H = 0.693145751953125f, kLn2L = 1.42860677e-6f;

// What a row's words are weighed with.  From a T of 2^64 on logits and T are
// taken 2^64 times smaller, so that finite logits have a finite difference and
// log2(e) / T its digits; below, a difference that overflows has no weight.
struct Weigh {
  float unit;    // 1, or 2^-64
  float top;     // the largest logit times unit
  float ch, cl;  // log2(e) / (T unit) as a pair
  int drop;      // bits of the unit given up for many words
  const u64 *pow;

  __device__ void temperature(float T) {
    unit = T >= 0x1p64f ? 0x1p-64f : 1.f;
    T *= unit;
    ch = kLog2eH / T;
    cl = T < 1e38f ? (fmaf(-ch, T, kLog2eH) + kLog2eL) / T : 0.f;
  }
  // (l - top) log2(e) / T
  __device__ Pair exponent(float l) const {
    // the sum of l unit and -top with its error, the product being exact
    const float s = fmaf(l, unit, -top), bv = fmaf(-l, unit, s), av = s - bv;
    const Pair d = {s, fmaf(l, unit, -av) - (top + bv)};
    const float yh = d.h * ch;
    return {yh, fmaf(d.h, cl, fmaf(d.l, ch, fmaf(d.h, ch, -yh)))};
  }
  __device__ u64 operator()(float l) const {
    const Pair y = exponent(l);
    // without a branch, so that several are under way at once; minus infinity: 0
    const bool some = y.h > -50.f;
    const u64 x = power(some ? y.h : 0.f, some ? y.l : 0.f, drop, pow);
    return some ? x : 0;
  }
};

// k ln 2 + ln(x / 2^63) for 2^63 <= x: an fp32 logarithm, and by how much its
// exponential misses x.
__device__ __noinline__ Pair logarithm(int k, u64 x, const u64 *pow) {
  const float l = __logf((float)(uint32_t)(x >> 32) * 0x1p-31f);
  const Pair y = times(-l, kLog2eH, kLog2eL);
  const u64 e = power(y.h, y.l, 0, pow);                   // exp(-l), 2^44 is 1
  const u64 near = __umul64hi(x, e << 19);                 // x exp(-l), 2^62 is 1
  const float miss = (float)(long long)(near - (1ull << 62)) * 0x1p-62f;
  const Pair s = add((float)k * kLn2H, l);
  return {s.h, s.l + fmaf((float)k, kLn2L, miss)};
}

// The whole part of x * m, 0 <= x < 1 (a zero of either sign), and whether
// anything is cut off.
__device__ __forceinline__ u64 part_of(float x, u64 m, bool *cut) {
  const uint32_t b = __float_as_uint(x) & 0x7fffffffu, e = b >> 23;
  const u64 digits = e ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
  const int shift = 150 - (int)(e ? e : 1);  // 24 or more
  const u64 hi = __umul64hi(digits, m), lo = digits * m;
  if (shift >= 128) {
    *cut = hi | lo;
    return 0;
  }
  if (shift >= 64) {
    *cut = (hi & ((1ull << (shift - 64)) - 1)) | lo;
    return hi >> (shift - 64);
  }
  *cut = lo & ((1ull << shift) - 1);
  return hi << (64 - shift) | lo >> shift;
}

// The fewest words of weight `one` that reach `mass`: an fp32 quotient is within
// a few units in the last place, two words where there are 2^22.
__device__ __forceinline__ uint32_t words_to(u64 mass, u64 one) {
  uint32_t n = (uint32_t)__fdividef((float)mass, (float)one);
  n = n > 3 ? n - 3 : 1;
  long long left = (long long)(mass - n * one);
#pragma unroll 1
  for (int i = 0; i < 8 && left > 0; ++i, ++n) left -= (long long)one;
  return n;
}

// A row's settings.  No word reaches a min_p above 1: the first one alone is left,
// as of top_k 1.
struct Settings {
  float temperature, top_p, min_p, u;
  int top_k;
  __device__ Settings(const SampleArgs &a, long long n)
      : temperature(a.temperature ? a.temperature[n] : 1.f),
        top_p(a.top_p ? a.top_p[n] : 1.f),
        min_p(a.min_p ? a.min_p[n] : 0.f),
        u(a.u[n]),
        top_k(a.top_k ? a.top_k[n] : 0) {
    if (min_p > 1.f) {
      min_p = 0.f;
      top_k = 1;
    }
  }
  __device__ bool usable() const {
    return temperature >= 0.f && top_p == top_p && min_p == min_p && u >= 0.f;
  }
  // the mass up to which words are kept: the one that reaches it is the last
  __device__ u64 share(u64 mass) const {
    if (!(top_p > 0.f)) return 1;
    bool cut;
    const u64 t = part_of(top_p, mass, &cut) + cut;
    return t ? t : 1;
  }
  // the word that reaches this mass is the token
  __device__ u64 draw(u64 mass) const {
    bool cut;
    return part_of(fminf(u, 0x1.fffffep-1f), mass, &cut) + 1;
  }
  // the smallest logit that min_p lets through: top + T ln(min_p), rounded up
  __device__ float least(float top, const u64 *pow) const {
    if (min_p == 1.f) return top;
    const uint32_t b = __float_as_uint(min_p), e = b >> 23;
    const uint32_t digits = e ? (b & 0x7fffffu) | 0x800000u : b;
    const int lead = __clz(digits);  // min_p = digits 2^(max(e, 1) - 150)
    const Pair ln = logarithm((int)(e ? e : 1) - 150 + 31 - lead, (u64)(digits << lead) << 32, pow);
    const Pair d = times(temperature, ln.h, ln.l);
    if (!(d.h > -kInf)) return -kInf;
    const Pair s = add(top, d.h);
    if (!(s.h > -kInf)) return -kInf;  // below every finite logit
    return __fadd_ru(s.h, s.l + d.l);
  }
};

// The logarithm of a mass, the largest logit's word being one.
__device__ __forceinline__ Pair log_mass(const Weigh &w, u64 mass) {
  const int lead = __clzll(mass);
  return logarithm(63 - lead - kUnit + w.drop, mass << lead, w.pow);
}
// The logarithm of the probability of a word with logit l.
__device__ __forceinline__ float log_share(const Weigh &w, float l, Pair log_mass) {
  const Pair y = w.exponent(l);
  // ln 2 = 0.693147182 - 1.9046543e-9
  const Pair z = times(y.h, 0.693147182f, -1.90465421e-9f);
  const Pair s = add(z.h, -log_mass.h);
  return s.h + (s.l + (fmaf(y.l, 0.693147182f, z.l) - log_mass.l));
}

__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t b = __float_as_uint(l + 0.f);  // minus zero is zero
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key ^ (key & 0x80000000u ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }

constexpr int kMostBlocks = 8;

// The blocks of a row: one, or a cluster's (two, four or eight), each of which
// reads a part of the row and then holds what all have found.  They decide on the
// same numbers, so that all come to the same barriers.
template <bool MANY>
struct Blocks {
  int rank = 0, size = 1;
  __device__ Blocks() {
    if constexpr (MANY) {
      rank = (int)cg::this_cluster().block_rank();
      size = (int)cg::this_cluster().num_blocks();
    }
  }
  __device__ void meet() const {
    if constexpr (MANY) cg::this_cluster().sync();
    else __syncthreads();
  }
  template <typename P>
  __device__ P *of(P *p, int other) const {
    if constexpr (MANY) return cg::this_cluster().map_shared_rank(p, other);
    else return p;
  }
};

// f(l, i) for every word of a row, or the block's part of it: 16 bytes a load
// between the row's boundaries.
template <int THREADS, typename T, typename B, typename F>
__device__ __forceinline__ void each(const T *row, int V, const B &blocks, const F &f) {
  constexpr int kVec = 16 / sizeof(T);
  const int head = min(V, (int)((16 - reinterpret_cast<uintptr_t>(row) % 16) % 16 / sizeof(T)));
  const int body = (V - head) / kVec, tail = head + body * kVec;
  const int first = blocks.rank * THREADS + (int)threadIdx.x, step = blocks.size * THREADS;
  if (first < head) f(as_float(row[first]), first);
  const uint4 *v = reinterpret_cast<const uint4 *>(row + head);
  uint4 next = make_uint4(0, 0, 0, 0);  // on its way while another is worked on
  if (first < body) next = v[first];
#pragma unroll 1
  for (int k = first; k < body; k += step) {
    const uint4 w = next;
    if (k + step < body) next = v[k + step];
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
  if (tail + first < V) f(as_float(row[tail + first]), tail + first);
}

struct Bins {
  uint32_t count[kBins], low[kBins], high[kBins];
  template <int THREADS>
  __device__ void clear() {
    for (int b = threadIdx.x; b < kBins; b += THREADS) count[b] = low[b] = high[b] = 0;
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

// The inclusive sums of a warp's (count, mass).
__device__ __forceinline__ void warp_scan(uint32_t &c, u64 &m) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t cu = __shfl_up_sync(kAll, c, o);
    const u64 mu = __shfl_up_sync(kAll, m, o);
    if ((int)(threadIdx.x % 32) >= o) {
      c += cu;
      m += mu;
    }
  }
}

// A barrier of the block's first `threads` threads.
__device__ __forceinline__ void first_threads(int threads) {
  asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
}

// What the scans and searches of a block share.
struct Tally {
  u64 warp_mass[32];
  uint32_t warp_count[32], turn_count[2][32];
  u64 mass, sum_mass, q_mass;
  uint32_t count, q_count;
  int bin, at, bad, finite;
  float least;
};

// A row as vectors of 16 bytes between its boundaries, what lies before the
// first boundary and behind the last being a vector too.
template <typename T>
struct Vectors {
  static constexpr int kVec = 16 / sizeof(T);
  const T *row;
  int V, head, body;
  __device__ Vectors(const T *row_, int V_) : row(row_), V(V_) {
    head = min(V, (int)((16 - reinterpret_cast<uintptr_t>(row) % 16) % 16 / sizeof(T)));
    body = (V - head) / kVec;
  }
  __device__ int count() const { return body + 2; }
  __device__ int start(int k) const { return k ? head + (k - 1) * kVec : 0; }
  __device__ uint4 load(int k) const {
    return k > 0 && k <= body ? reinterpret_cast<const uint4 *>(row + head)[k - 1]
                              : make_uint4(0, 0, 0, 0);
  }
  // the words of a vector that have value v, a bit each; w: load(k)
  __device__ unsigned matches(int k, uint4 w, float v) const {
    unsigned m = 0;
    if (k == 0 || k > body) {
      const int i0 = start(k), n = k ? V - i0 : head;
      if (k <= body + 1)
        for (int i = 0; i < n; ++i) m |= (unsigned)(as_float(row[i0 + i]) == v) << i;
      return m;
    }
    const uint32_t part[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if constexpr (sizeof(T) == 4) {
        m |= (unsigned)(__uint_as_float(part[q]) == v) << q;
      } else {
        m |= (unsigned)(__uint_as_float(part[q] << 16) == v) << (2 * q);
        m |= (unsigned)(__uint_as_float(part[q] & 0xffff0000u) == v) << (2 * q + 1);
      }
    }
    return m;
  }
};

// The index of the ties-th word of value v (zeros of both signs alike) among
// `equal` of them (0: not known), from the nearer end of the row, by the block's
// first THREADS threads.
template <int THREADS, typename T>
__device__ __noinline__ int find_index(Tally &s, const T *row, int V, float v, uint32_t ties,
                                       uint32_t equal) {
  constexpr int kWarps = THREADS / 32, kEach = 4, kStep = kEach * THREADS;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const Vectors<T> r(row, V);
  const int steps = (r.count() + kStep - 1) / kStep;
  const bool back = equal && ties > equal - ties + 1;
  uint32_t want = back ? equal - ties + 1 : ties;
  // a warp's vectors are neighbours, 32 of them a load; the next step's are under
  // way while this one's matches are counted
  auto first = [&](int step) {
    return (back ? steps - 1 - step : step) * kStep + 32 * kEach * warp + lane;
  };
  uint4 next[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) next[i] = r.load(first(0) + 32 * i);
#pragma unroll 1
  for (int step = 0; step < steps; ++step) {
    const int k = first(step);
    unsigned m[kEach];
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      m[i] = r.matches(k + 32 * i, next[i], v);
      n += __popc(m[i]);
    }
    if (step + 1 < steps) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) next[i] = r.load(first(step + 1) + 32 * i);
    }
    n = __reduce_add_sync(kAll, n);
    uint32_t *count = s.turn_count[step & 1];  // the last turn's may still be read
    if (lane == 0) count[warp] = n;
    first_threads(THREADS);
    const uint32_t c = lane < kWarps ? count[lane] : 0;
    const uint32_t total = __reduce_add_sync(kAll, c);
    if (want > total) {
      want -= total;
      continue;
    }
    const uint32_t rank = back ? total - want + 1 : want;
    uint32_t before = __reduce_add_sync(kAll, lane < warp ? c : 0);
    if (before < rank && rank <= before + n) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const uint32_t here = __popc(m[i]);
        uint32_t upto = here;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t x = __shfl_up_sync(kAll, upto, o);
          if (lane >= o) upto += x;
        }
        if (before + upto - here < rank && rank <= before + upto) {
          for (uint32_t left = rank - (before + upto - here); left > 1; --left) m[i] &= m[i] - 1;
          s.at = r.start(k + 32 * i) + __ffs(m[i]) - 1;
        }
        before += __shfl_sync(kAll, upto, 31);
      }
    }
    break;
  }
  first_threads(THREADS);
  return s.at;
}

struct Shared : Tally {
  Bins first, fine;
  u64 pow[1024];
  uint32_t key[kList];
  int index[kList];
  u64 weight[kFew];
  int listed;
  uint32_t lo, hi;
  // of all the row's blocks
  uint32_t all_top, all_q_count;
  int all_bad, all_finite;
  u64 all_mass, all_q_mass;
};

// What each block has added to its bins becomes what all have, and `also` is done
// by the first warp while the blocks' other sums stand.
template <bool MANY, typename F>
__device__ void share(const Blocks<MANY> &blocks, Bins &bins, const F &also) {
  blocks.meet();
  if constexpr (MANY) {  // a block adds up some of the bins for all
    const int some = kBins / blocks.size;
    for (int t = threadIdx.x; t < some; t += blockDim.x) {
      const int b = blocks.rank * some + t;
      uint32_t count = 0;
      u64 mass = 0;
#pragma unroll
      for (int k = 0; k < kMostBlocks; ++k) {  // their loads under way at once
        if (k >= blocks.size) continue;
        const Bins *other = blocks.of(&bins, (blocks.rank + k) & (blocks.size - 1));
        count += other->count[b];
        mass += other->mass(b);
      }
#pragma unroll
      for (int k = 0; k < kMostBlocks; ++k) {
        if (k >= blocks.size) continue;
        Bins *other = blocks.of(&bins, (blocks.rank + k) & (blocks.size - 1));
        other->count[b] = count;
        other->low[b] = (uint32_t)mass;
        other->high[b] = (uint32_t)(mass >> 32);
      }
    }
    if (threadIdx.x < 32) also();
    blocks.meet();
  }
}

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
template <int THREADS>
__device__ void find_bin(Shared &s, const Bins &b, bool by_mass, u64 target, u64 count0,
                         u64 mass0) {
  constexpr int kPer = kBins / THREADS, kWarps = THREADS / 32;
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
  first_threads(THREADS);
  if (warp == 0) {
    uint32_t cw = lane < kWarps ? s.warp_count[lane] : 0;
    u64 mw = lane < kWarps ? s.warp_mass[lane] : 0;
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
  first_threads(THREADS);
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
  first_threads(THREADS);
}

template <typename T, int THREADS, bool MANY>
struct Row {
  static constexpr int kThreads = THREADS, kWarps = THREADS / 32;
  const T *row;
  int V;
  Weigh w;
  float per;  // bins of l a (scaled) unit of l
  Blocks<MANY> blocks;

  __device__ int bin(float l) const {
    return min(kBins - 1, __float2int_rz(fmaf(-l, w.unit, w.top) * per));
  }

  // The place at which words (or masses) reach `target`, which lies in bin
  // s.bin of the first bins, s.count words and s.mass before it.
  __device__ Place place(Shared &s, bool by_mass, u64 target) const {
    const int b = s.bin;
    u64 count0 = s.count, mass0 = s.mass;
    const uint32_t n = s.first.count[b];
    first_threads(THREADS);
    if (threadIdx.x == 0) {
      s.listed = 0;
      s.lo = 0xffffffffu;
      s.hi = 0;
    }
    first_threads(THREADS);
    if (MANY) blocks.meet();  // before the others write to these
    const bool list = n <= kList;
    {
      uint32_t lo = 0xffffffffu, hi = 0;
      each<THREADS>(row, V, blocks, [&](float l, int i) {
        if (l > -kInf && bin(l) == b) {
          const uint32_t key = key_of(l);
          lo = min(lo, key);
          hi = max(hi, key);
          if (list) {
            const int at = atomicAdd(blocks.of(&s.listed, 0), 1);
            if (at < kList) {
              for (int k = 0; k < blocks.size; ++k) {
                blocks.of(s.key, k)[at] = key;
                blocks.of(s.index, k)[at] = i;
              }
            }
          }
        }
      });
      if (MANY) {
        lo = __reduce_min_sync(kAll, lo);
        hi = __reduce_max_sync(kAll, hi);
        if ((int)(threadIdx.x % 32) < blocks.size && lo <= hi) {
          atomicMin(blocks.of(&s.lo, threadIdx.x % 32), lo);
          atomicMax(blocks.of(&s.hi, threadIdx.x % 32), hi);
        }
      } else if (lo <= hi) {
        atomicMin(&s.lo, lo);
        atomicMax(&s.hi, hi);
      }
    }
    if (MANY) blocks.meet();
    else first_threads(THREADS);
    uint32_t lo = s.lo, hi = s.hi;
    if (lo < hi && n <= kFew) return place_few(s, by_mass, target, count0, mass0, (int)n);
    // down to one key: bins of (hi - key) >> shift, 11 bits of 32 each time
    for (int turn = 0; turn < 3 && lo < hi; ++turn) {
      const int shift = max(0, 32 - __clz(hi - lo) - 11);
      s.fine.template clear<THREADS>();
      first_threads(THREADS);
      if (list) {
        for (int k = threadIdx.x; k < (int)n; k += kThreads) {
          const uint32_t key = s.key[k];
          if (key >= lo && key <= hi) s.fine.add((hi - key) >> shift, w(value_of(key)));
        }
      } else {
        each<THREADS>(row, V, blocks, [&](float l, int) {
          const uint32_t key = key_of(l);
          if (key >= lo && key <= hi && bin(l) == b) s.fine.add((hi - key) >> shift, w(l));
        });
        if (MANY) share(blocks, s.fine, [] {});
      }
      first_threads(THREADS);
      find_bin<THREADS>(s, s.fine, by_mass, target, count0, mass0);
      count0 = s.count;
      mass0 = s.mass;
      const uint32_t first = (uint32_t)s.bin << shift;
      const uint32_t nlo = hi - min(hi - lo, first + ((1u << shift) - 1));
      hi -= first;
      lo = nlo;
      if (lo == hi) {
        Place p = at_key(lo, s.fine.count[s.bin], by_mass, target, count0, mass0);
        first_threads(THREADS);
        return p;
      }
      first_threads(THREADS);
    }
    return at_key(lo, n, by_mass, target, count0, mass0);
  }

  __device__ Place at_key(uint32_t key, uint32_t equal, bool by_mass, u64 target, u64 count0,
                          u64 mass0) const {
    Place p;
    p.key = key;
    p.equal = equal;
    p.weight = w(value_of(key));
    p.ties = by_mass ? words_to(target - mass0, p.weight)
                     : (uint32_t)(target - count0);
    p.count = count0 + p.ties;
    p.mass = mass0 + p.ties * p.weight;
    p.index = -1;
    return p;
  }

  // Each word of a short list against all of them, a warp a word.
  __device__ Place place_few(Shared &s, bool by_mass, u64 target, u64 count0, u64 mass0,
                             int n) const {
    const int lane = threadIdx.x % 32;
    for (int t = threadIdx.x; t < n; t += THREADS) s.weight[t] = w(value_of(s.key[t]));
    first_threads(THREADS);
    for (int t = threadIdx.x / 32; t < n; t += kWarps) {
      const uint32_t key = s.key[t];
      const int index = s.index[t];
      uint32_t c = 0;
      u64 m = 0;
      for (int k = lane; k < n; k += 32)
        if (s.key[k] > key || (s.key[k] == key && s.index[k] < index)) {
          c += 1;
          m += s.weight[k];
        }
      c = (uint32_t)count0 + __reduce_add_sync(kAll, c);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(kAll, m, o);
      m += mass0;
      const u64 before = by_mass ? m : c, after = before + (by_mass ? s.weight[t] : 1);
      if (lane == 0 && before < target && target <= after) {
        s.at = t;
        s.count = c;
        s.mass = m;
      }
    }
    first_threads(THREADS);
    Place p;
    const int at = s.at;
    p.key = s.key[at];
    p.weight = s.weight[at];
    p.count = s.count + 1;
    p.mass = s.mass + p.weight;
    p.ties = p.equal = 0;
    p.index = s.index[at];
    first_threads(THREADS);
    return p;
  }
};

__device__ void no_token(const SampleArgs &a, long long n) {
  a.token[n] = -1;
  if (a.logp) a.logp[n] = __int_as_float(0x7fc00000);
  if (a.kept) a.kept[n] = 0;
}

// The largest logit's word, where the temperature is zero.
template <int THREADS, typename T>
__device__ void greedy(Tally &s, const SampleArgs &a, long long n, const T *row, float top) {
  const int at = find_index<THREADS>(s, row, a.V, top, 1, 0);
  if (threadIdx.x == 0) {
    a.token[n] = at;
    if (a.logp) a.logp[n] = 0.f;
    if (a.kept) a.kept[n] = 1;
  }
}

// The token, once its value and which of its words is known: the last warp takes
// the logarithm while the others look for the word.
template <int THREADS, typename T>
__device__ void finish(Tally &s, const SampleArgs &a, long long n, const T *row, const Weigh &w,
                       float l, uint32_t ties, uint32_t equal, int index, u64 kept, u64 mass) {
  if (threadIdx.x >= THREADS - 32) {
    if (a.logp && threadIdx.x == THREADS - 1) a.logp[n] = log_share(w, l, log_mass(w, mass));
    return;
  }
  if (index < 0) index = find_index<THREADS - 32>(s, row, a.V, l, ties, equal);
  if (threadIdx.x == 0) {
    a.token[n] = index;
    if (a.kept) a.kept[n] = (int)kept;
  }
}

// ---- bf16 -------------------------------------------------------------------
// A bf16 row has few different words: 12289 between 2^-40 and 2^8 in magnitude,
// zero with them.  One pass counts them by value in shared memory, and a weight
// is taken once for each value that occurs rather than for each word.  128
// neighbouring values are a bin, as far down as a weight reaches; warps weigh the
// bins by turns, four values a lane.  One warp then holds what lies before each
// bin and finds one place after the other without a barrier of the block.  Rows
// with other words (but minus infinity) take the general form, such as those masked
// with a finite number: of 256 x 131072 with top_p, a tenth of the words at -1e4,
// 446 us for 38.  Vectors that hold minus infinity go word by word (240).
//
// The counting bounds it: 32 lanes add to random banks, and the fullest of the
// 32 sets the pace at 9 words a cycle and SM, whatever is done there (plain
// loads and stores too).
constexpr int kBinades = 48;                   // 2^-40 .. 2^8
constexpr uint32_t kLeast16 = 87 << 7;         // bits of 2^-40
constexpr uint32_t kValues = kBinades * 128;   // of one sign
constexpr int kBins16 = 2 * kBinades + 1;
// Words of shared memory: those of a sign by rising magnitude, zero behind the
// positive ones, the negative ones 2^15 bytes behind where those begin, so that
// a word's address is 4 times its magnitude's bits plus the sign's.
constexpr uint32_t kNegative = 8192;

struct Counted : Tally {
  alignas(16) uint32_t count[kNegative + kValues];  // read 16 bytes a load
  u64 pow[1024];
  // masses and words of a bin's places up to each four, falling; of all of them
  u64 lane_mass[32 * kBins16];
  uint32_t lane_count[32 * kBins16];
  u64 bin_mass[kBins16];
  uint32_t bin_count[kBins16];
  uint32_t most, least_bits, masked;
  int other;
  uint32_t token, ties, equal, kept;
  u64 kept_mass;
};

// Places in falling order, 0 for the largest positive value; the zero has a bin
// of its own between the signs.
__device__ __forceinline__ float value16(int place) {
  if (place < (int)kValues) return __uint_as_float((kLeast16 + kValues - 1 - place) << 16);
  const int k = place - (int)kValues - 128;
  return k < 0 ? 0.f : __uint_as_float((0x8000u | (kLeast16 + (uint32_t)k)) << 16);
}

// Counts of four neighbouring places from 4 k on, or of one.
__device__ __forceinline__ uint4 count4(const Counted &s, int k) {
  const uint4 *all = reinterpret_cast<const uint4 *>(s.count);
  constexpr int kQuarter = (int)kValues / 4;
  if (k >= kQuarter) return all[k < kQuarter + 32 ? k : k - 32 + (int)(kNegative - kValues) / 4];
  const uint4 v = all[kQuarter - 1 - k];
  return make_uint4(v.w, v.z, v.y, v.x);
}
__device__ __forceinline__ uint32_t count1(const Counted &s, int place) {
  if (place < (int)kValues) return s.count[(int)kValues - 1 - place];
  return s.count[place < (int)kValues + 128 ? place : place - 128 + (int)(kNegative - kValues)];
}

enum How { kByCount, kByMass, kByLeast };

// A place: `ties` of the `equal` words of a value, words and masses through them.
struct Found {
  int place;
  uint32_t ties, equal, count;
  u64 mass;
};

// The place at which words or masses reach `target`, or (kByLeast) that of the
// last word that is not below `least`; for one warp whose lanes hold four bins
// each and what lies before them.
__device__ __forceinline__ Found find_place(const Counted &s, const Weigh &w, uint32_t count,
                                         u64 mass, int top_bin, int bins, How how, u64 target,
                                         float least) {
  const int lane = threadIdx.x % 32;
  int hit = -1;
  uint32_t c0 = 0, c1 = count;
  u64 m0 = 0, m1 = mass;
#pragma unroll 1
  for (int b = 4 * lane; b < min(bins, 4 * lane + 4); ++b) {
    const uint32_t c = s.bin_count[b];
    const u64 m = s.bin_mass[b];
    bool is;
    if (how == kByLeast) {
      const int first = 128 * (top_bin + b);
      is = value16(first) >= least && (b == bins - 1 || !(value16(first + 128) >= least));
    } else {
      const u64 before = how == kByMass ? m1 : c1;
      is = before < target && target <= before + (how == kByMass ? m : c);
    }
    if (is) {
      hit = b;
      c0 = c1;
      m0 = m1;
    }
    c1 += c;
    m1 += m;
  }
  const int from = max(0, __ffs(__ballot_sync(kAll, hit >= 0)) - 1);
  hit = max(0, __shfl_sync(kAll, hit, from));
  c0 = __shfl_sync(kAll, c0, from);
  m0 = __shfl_sync(kAll, m0, from);
  // the four places, a lane each four
  const int k = 32 * (top_bin + hit);
  uint32_t c = c0 + s.lane_count[32 * hit + lane];
  u64 m = m0 + s.lane_mass[32 * hit + lane];
  bool mine = how == kByLeast ? value16(4 * (k + lane)) >= least : target <= (how == kByMass ? m : c);
  unsigned all = __ballot_sync(kAll, mine);
  // places and masses rise with the lane: the first that reaches, the last not below
  const int four = how == kByLeast ? 31 - __clz(all | 1) : max(0, __ffs(all) - 1);
  c0 = four ? __shfl_sync(kAll, c, four - 1) : c0;
  m0 = four ? __shfl_sync(kAll, m, four - 1) : m0;
  // the place, in every fourth lane alike
  Found p;
  p.place = 4 * (k + four) + lane % 4;
  p.equal = p.ties = count1(s, p.place);
  const float v = value16(p.place);
  const u64 one = w(v), here = p.equal * one;
  c = p.equal;
  m = here;
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    const uint32_t cu = __shfl_up_sync(kAll, c, o, 4);
    const u64 mu = __shfl_up_sync(kAll, m, o, 4);
    if (lane % 4 >= o) {
      c += cu;
      m += mu;
    }
  }
  p.count = c0 + c;
  p.mass = m0 + m;
  mine = how == kByLeast ? v >= least : target <= (how == kByMass ? p.mass : p.count);
  all = __ballot_sync(kAll, mine) & 15;
  const int at = how == kByLeast ? 31 - __clz(all | 1) : max(0, __ffs(all) - 1);
  if (how != kByLeast) {  // not all of its words
    p.ties = how == kByMass ? words_to(target - (p.mass - here), one)
                            : (uint32_t)target - (p.count - p.equal);
    p.count -= p.equal - p.ties;
    p.mass -= (p.equal - p.ties) * one;
  }
  p.place = __shfl_sync(kAll, p.place, at);
  p.ties = __shfl_sync(kAll, p.ties, at);
  p.equal = __shfl_sync(kAll, p.equal, at);
  p.count = __shfl_sync(kAll, p.count, at);
  p.mass = __shfl_sync(kAll, p.mass, at);
  return p;
}

// Whether the row is done.  A min_p below every weight is left to the general
// form, which counts words without weight too.
template <int THREADS>
__device__ bool counted_row(Counted &s, const SampleArgs &a, const Settings &set, long long n) {
  const int tid = threadIdx.x, lane = tid % 32, warp = __shfl_sync(kAll, tid / 32, 0);
  const __nv_bfloat16 *row = static_cast<const __nv_bfloat16 *>(a.logits) + n * a.ld;
  if (set.min_p > 0.f && set.min_p < 0x1p-45f) return false;
  for (int i = tid; i < (int)(kNegative + kValues) / 4; i += THREADS)
    reinterpret_cast<uint4 *>(s.count)[i] = make_uint4(0, 0, 0, 0);
  if (tid == 0) {
    s.most = s.masked = 0;
    s.least_bits = 0xffff;
    s.other = 0;
    s.at = 0;
  }
  for (int i = tid; i < 1024; i += THREADS) s.pow[i] = kPowers.v[i];
  Weigh w;
  w.temperature(set.temperature);
  w.drop = a.drop;
  w.pow = s.pow;
  __syncthreads();
  {
    // the largest positive word's bits and the smallest magnitude's, of two each
    uint32_t most = 0, least = 0xffffffffu, masked = 0;
    bool other = false;
    auto add = [&](uint32_t magnitude4, uint32_t sign) {
      atomicAdd(reinterpret_cast<uint32_t *>(reinterpret_cast<char *>(s.count) + magnitude4 + sign -
                                             4 * kLeast16), 1u);
    };
    auto one = [&](uint32_t b) {  // the low 16 bits, anything
      const uint32_t m = b & 0x7fffu;
      if (m - kLeast16 < kValues) {
        add(4 * m, b & 0x8000u);
        if (!(b & 0x8000u)) most = __vmaxs2(most, m);
        least = __vminu2(least, m | 0xffff0000u);
      } else if ((b & 0xffffu) == 0xff80u) {
        ++masked;
      } else if (!m) {
        atomicAdd(&s.count[kValues], 1u);
      } else {
        other = true;
      }
    };
    const Vectors<__nv_bfloat16> r(row, a.V);
    if (tid < r.head) one(__bfloat16_as_ushort(row[tid]));
    const uint4 *v = reinterpret_cast<const uint4 *>(row + r.head);
    auto eight = [&](uint4 w) {
      const uint32_t part[4] = {w.x, w.y, w.z, w.w};
      uint32_t m[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) m[q] = part[q] & 0x7fff7fffu;
      const uint32_t low = __vminu2(__vminu2(m[0], m[1]), __vminu2(m[2], m[3]));
      const uint32_t high = __vmaxu2(__vmaxu2(m[0], m[1]), __vmaxu2(m[2], m[3]));
      // all eight between 2^-40 and 2^8
      if (__vmaxu2(high, (kLeast16 + kValues - 1) * 0x10001u) == (kLeast16 + kValues - 1) * 0x10001u &&
          __vminu2(low, kLeast16 * 0x10001u) == kLeast16 * 0x10001u) {
        least = __vminu2(least, low);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          most = __vmaxs2(most, part[q]);
          add(part[q] << 2 & 0x1fffcu, part[q] & 0x8000u);
          add(part[q] >> 14 & 0x1fffcu, part[q] >> 16 & 0x8000u);
        }
      } else {
#pragma unroll 1
        for (int q = 0; q < 8; ++q) {
          one(w.x);
          w.x = __funnelshift_r(w.x, w.y, 16);
          w.y = __funnelshift_r(w.y, w.z, 16);
          w.z = __funnelshift_r(w.z, w.w, 16);
          w.w >>= 16;
        }
      }
    };
    int k = tid;
    for (; k + 3 * THREADS < r.body; k += 4 * THREADS) {  // four loads under way
      const uint4 w0 = v[k], w1 = v[k + THREADS], w2 = v[k + 2 * THREADS], w3 = v[k + 3 * THREADS];
      eight(w0);
      eight(w1);
      eight(w2);
      eight(w3);
    }
    for (; k < r.body; k += THREADS) eight(v[k]);
    const int tail = r.start(r.body + 1) + tid;
    if (tail < a.V) one(__bfloat16_as_ushort(row[tail]));
    most = __reduce_max_sync(kAll, max(most & 0xffffu, most >> 16));
    least = __reduce_min_sync(kAll, min(least & 0xffffu, least >> 16));
    masked = __reduce_add_sync(kAll, masked);
    other = __any_sync(kAll, other);
    if (lane == 0) {
      atomicMax(&s.most, most);
      atomicMin(&s.least_bits, least);
      if (masked) atomicAdd(&s.masked, masked);
      if (other) s.other = 1;
    }
  }
  __syncthreads();
  if (s.other) return false;
  const uint32_t finite = (uint32_t)a.V - s.masked;
  if (!finite || !set.usable()) {
    if (tid == 0) no_token(a, n);
    return true;
  }
  // the largest word: positive, or zero, or the smallest negative one
  const int top = s.most                 ? (int)(kLeast16 + kValues - 1 - s.most)
                  : s.count[kValues] ? (int)kValues
                                     : (int)(kValues + 128 + s.least_bits - kLeast16);
  const float largest = value16(top);
  if (set.temperature < kNoTemperature) {
    greedy<THREADS>(s, a, n, row, largest);
    return true;
  }
  w.top = largest * w.unit;
  // Values with a weight: 2^-45 lies 31.2 T below the largest.
  const uint32_t low = __float_as_uint(fmaf(-32.f, set.temperature, largest)) >> 16;
  const int size = (int)(low & 0x7fffu) - (int)kLeast16;
  const int last = size < 0           ? (int)kValues
                   : low & 0x8000u ? (int)kValues + 128 + min(size, (int)kValues - 1)
                                   : (int)kValues - 1 - min(size, (int)kValues - 1);
  const int top_bin = top >> 7, bins = (last >> 7) - top_bin + 1;
#pragma unroll 1
  for (int b = warp; b < bins; b += THREADS / 32) {
    const int k = 32 * (top_bin + b) + lane;
    const uint4 v = count4(s, k);
    uint32_t c = 0;
    u64 m = 0;
    if (__any_sync(kAll, v.x | v.y | v.z | v.w)) {
      c = v.x + v.y + v.z + v.w;
      m = v.x * w(value16(4 * k)) + v.y * w(value16(4 * k + 1)) + v.z * w(value16(4 * k + 2)) +
          v.w * w(value16(4 * k + 3));
      warp_scan(c, m);
    }
    s.lane_count[32 * b + lane] = c;
    s.lane_mass[32 * b + lane] = m;
    if (lane == 31) {
      s.bin_count[b] = c;
      s.bin_mass[b] = m;
    }
  }
  __syncthreads();
  if (warp == 0) {
    uint32_t count = 0;
    u64 mass = 0;
    for (int b = 4 * lane; b < min(bins, 4 * lane + 4); ++b) {
      count += s.bin_count[b];
      mass += s.bin_mass[b];
    }
    uint32_t own_count = count;
    u64 own_mass = mass;
    warp_scan(own_count, own_mass);
    const uint32_t all_count = __shfl_sync(kAll, own_count, 31);  // words with a weight
    u64 kept_mass = __shfl_sync(kAll, own_mass, 31);
    own_count -= count;
    own_mass -= mass;
    // top_k's place, top_p's, min_p's and the token's, one after the other: a loop,
    // so that there is one copy of the search
    const bool by_k = set.top_k > 0 && (uint32_t)set.top_k < finite;
    uint32_t kept = by_k ? (uint32_t)set.top_k : finite;
    u64 k_mass = kept_mass;
    Found p;
#pragma unroll 1
    for (int step = by_k && kept <= all_count ? 0 : 1; step < 4; ++step) {
      How how = kByMass;
      u64 target = 0;
      float least = 0.f;
      if (step == 0) {
        how = kByCount;
        target = kept;
      } else if (step == 1) {
        if (!(set.top_p < 1.f)) continue;
        target = set.share(k_mass);
      } else if (step == 2) {
        if (!(set.min_p > 0.f)) continue;
        how = kByLeast;
        least = set.least(largest, s.pow);
      } else {
        target = set.draw(kept_mass);
      }
      p = find_place(s, w, own_count, own_mass, top_bin, bins, how, target, least);
      if (step < 3 && p.count <= kept) {  // a beginning within the one so far
        kept = p.count;
        kept_mass = p.mass;
      }
      if (step == 0) k_mass = p.mass;
    }
    if (lane == 0) {
      s.token = p.place;
      s.ties = p.ties;
      s.equal = p.equal;
      s.kept = kept;
      s.kept_mass = kept_mass;
    }
  }
  __syncthreads();
  finish<THREADS>(s, a, n, row, w, value16((int)s.token), s.ties, s.equal, -1, s.kept, s.kept_mass);
  return true;
}

// ---- the general form ---------------------------------------------------------
// (Of few long rows each block of a cluster reads a part: what a pass finds is
// joined at its end, and the steps between the passes are taken by all alike.)
// One pass finds the largest logit, one adds words and masses into 2048 bins of l
// over the range in which w is not zero, a scan over the bins finds the bin of a
// place, and the few words of that bin are looked at one by one, or, where they
// are many, by bins of their keys, as often as it takes to come down to one value.
template <typename T, int THREADS, bool MANY>
__device__ void any_row(Shared &s, const SampleArgs &a, const Settings &set, long long n) {
  const int tid = threadIdx.x, lane = tid % 32;
  Row<T, THREADS, MANY> r;
  r.row = static_cast<const T *>(a.logits) + n * a.ld;
  r.V = a.V;

  // the largest logit
  if (tid == 0) {
    s.bad = s.finite = s.bin = s.at = 0;
    s.lo = 0;
    s.sum_mass = s.q_mass = 0;
    s.q_count = 0;
  }
  s.first.template clear<THREADS>();
  for (int j = tid; j < 1024; j += THREADS) s.pow[j] = kPowers.v[j];
  __syncthreads();
  {
    uint32_t top = 0;
    int bad = 0, finite = 0;
    each<THREADS>(r.row, a.V, r.blocks, [&](float l, int) {
      bad |= !(l < kInf);
      finite += l > -kInf;
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
  r.blocks.meet();
  if (MANY) {
    if (tid < 32) {
      const Shared *other = r.blocks.of(&s, tid < r.blocks.size ? tid : r.blocks.rank);
      const uint32_t most = __reduce_max_sync(kAll, other->lo);
      const int any_bad = __any_sync(kAll, other->bad);
      const int some = __reduce_add_sync(kAll, tid < r.blocks.size ? other->finite : 0);
      if (tid == 0) {
        s.all_top = most;
        s.all_bad = any_bad;
        s.all_finite = some;
      }
    }
    __syncthreads();
  }
  const uint32_t top_key = MANY ? s.all_top : s.lo;
  const int finite = MANY ? s.all_finite : s.finite;
  const float largest = value_of(top_key);
  // settings that are no numbers, or a row without a distribution
  const bool none = (MANY ? s.all_bad : s.bad) || !finite || !set.usable();
  if (none || set.temperature < kNoTemperature) {
    if (MANY) r.blocks.meet();  // the others may still read
    if (r.blocks.rank) return;
    if (!none) greedy<THREADS>(s, a, n, r.row, largest);
    else if (tid == 0) no_token(a, n);
    return;
  }
  r.w.temperature(set.temperature);
  r.w.top = largest * r.w.unit;
  r.w.drop = a.drop;
  r.w.pow = s.pow;
  const bool by_min = set.min_p > 0.f;
  if (by_min) {
    if (tid == 0) s.least = set.least(largest, s.pow);
    __syncthreads();
  }
  const float least = s.least;
  // the bins' range: weights down to 2^-46
  r.per = (float)(kBins - 1) / 46.f * r.w.ch;

  // top_k's bin, so that no weight is taken behind it
  int last_bin = kBins - 1;
  u64 k_count = 0;
  if (set.top_k > 0 && set.top_k < finite) {
    k_count = (u64)set.top_k;
    each<THREADS>(r.row, a.V, r.blocks, [&](float l, int) {
      if (l > -kInf) atomicAdd(&s.first.count[r.bin(l)], 1u);
    });
    share(r.blocks, s.first, [] {});
    find_bin<THREADS>(s, s.first, false, k_count, 0, 0);
    last_bin = s.bin;
    __syncthreads();
    s.first.template clear<THREADS>();
    __syncthreads();
  }
  // words and masses by bins; those that min_p keeps apart
  {
    u64 mass = 0, q_mass = 0;
    uint32_t q_count = 0;
    each<THREADS>(r.row, a.V, r.blocks, [&](float l, int) {
      const int b = r.bin(l);
      if (b > last_bin || !(l > -kInf)) return;
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
  share(r.blocks, s.first, [&] {
    const bool is = tid < r.blocks.size;
    const Shared *other = r.blocks.of(&s, is ? tid : r.blocks.rank);
    u64 all = is ? other->sum_mass : 0, q = is ? other->q_mass : 0;
    const uint32_t count = __reduce_add_sync(kAll, is ? other->q_count : 0);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      all += __shfl_xor_sync(kAll, all, o);
      q += __shfl_xor_sync(kAll, q, o);
    }
    if (tid == 0) {
      s.all_mass = all;
      s.all_q_mass = q;
      s.all_q_count = count;
    }
  });
  u64 kept = (u64)finite, mass = MANY ? s.all_mass : s.sum_mass;
  const u64 q_mass = MANY ? s.all_q_mass : s.q_mass;
  const uint32_t q_count = MANY ? s.all_q_count : s.q_count;
  if (k_count) {
    find_bin<THREADS>(s, s.first, false, k_count, 0, 0);
    const Place p = r.place(s, false, k_count);
    kept = p.count;
    mass = p.mass;
  }
  if (set.top_p < 1.f) {
    const u64 target = set.share(mass);
    find_bin<THREADS>(s, s.first, true, target, 0, 0);
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
  const u64 target = set.draw(mass);
  find_bin<THREADS>(s, s.first, true, target, 0, 0);
  const Place p = r.place(s, true, target);
  if (r.blocks.rank) return;
  finish<THREADS>(s, a, n, r.row, r.w, value_of(p.key), p.ties, p.equal, p.index, kept, mass);
}

template <int THREADS, bool MANY>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) sample_f32_kernel(const SampleArgs a) {
  extern __shared__ __align__(16) unsigned char raw[];
  const long long n = MANY ? blockIdx.y : blockIdx.x;
  const Settings set(a, n);
  any_row<float, THREADS, MANY>(*reinterpret_cast<Shared *>(raw), a, set, n);
}

template <int THREADS>
__device__ __noinline__ void any_bf16_row(Shared &s, const SampleArgs &a, const Settings &set,
                                          long long n) {
  any_row<__nv_bfloat16, THREADS, false>(s, a, set, n);
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) sample_bf16_kernel(const SampleArgs a) {
  extern __shared__ __align__(16) unsigned char raw[];
  const Settings set(a, blockIdx.x);
  if (counted_row<THREADS>(*reinterpret_cast<Counted *>(raw), a, set, blockIdx.x)) return;
  __syncthreads();
  any_bf16_row<THREADS>(*reinterpret_cast<Shared *>(raw), a, set, blockIdx.x);
}

template <auto KERNEL>
cudaError_t launch(size_t smem, bool most, int threads, const SampleArgs &a, int N,
                   cudaStream_t stream) {
  const cudaError_t err = allow_shared<KERNEL>(smem, most);
  if (err != cudaSuccess) return err;
  KERNEL<<<N, threads, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t sample(SampleArgs a, int N, int dtype, int num_sms, cudaStream_t stream) {
  a.drop = 0;
  while (kUnit - a.drop > 0 && ((long long)a.V << (kUnit - a.drop)) > (1LL << 62)) ++a.drop;
  // bf16: two blocks an SM, the memory that can be shared being theirs, so that one
  // counts while the other searches (256 x 131072: 42 us; one of 1024 threads 46;
  // a single row takes the same either way).  fp32: the same for more rows than
  // SMs (333 x 8003: 25 us for 32), else blocks of 1024 (64 x 32000 in one a row: 29
  // us for 39), which keep the row in the rest of that memory.
  constexpr size_t kSmem = sizeof(Counted) > sizeof(Shared) ? sizeof(Counted) : sizeof(Shared);
  if (dtype == FLASH_GAU_BF16)
    return launch<sample_bf16_kernel<512>>(kSmem, true, 512, a, N, stream);
  if (N > num_sms)
    return launch<sample_f32_kernel<512, false>>(sizeof(Shared), false, 512, a, N, stream);
  // Few long rows: a cluster of blocks a row, where its clusters find room at once
  // (fewer as they grow: a cluster is one GPC's) and a row's passes are long
  // enough for the two barriers and the exchange at each pass's end.  Of fp32, no
  // filter, one block, two, four and eight: 1 x 131072 79, 49, 31, 23 us; 14 x 131072
  // 87, 59, 41, 32; 33 x 50257 39, 31, 24, 50; 76 x 50257 47, 39, 61, 97; 4 x 24000
  // 21, 19, 17, 15.  The mean over all filters breaks even near 28000 words for
  // two, 20000 for four, 16000 for eight.
  int blocks = 1;
  if (a.V >= 16384 && N * kMostBlocks <= num_sms * 3 / 4) blocks = 8;
  else if (a.V >= 20480 && N * 4 <= num_sms * 7 / 8) blocks = 4;
  else if (a.V >= 28672 && N * 2 <= num_sms) blocks = 2;
  if (blocks == 1)
    return launch<sample_f32_kernel<1024, false>>(sizeof(Shared), false, 1024, a, N, stream);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, N);
  cfg.blockDim = dim3(1024);
  cfg.dynamicSmemBytes = sizeof(Shared);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = blocks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t err = allow_shared<sample_f32_kernel<1024, true>>(sizeof(Shared), false);
  if (err != cudaSuccess) return err;
  return cudaLaunchKernelEx(&cfg, sample_f32_kernel<1024, true>, a);
}

}  // namespace flashgau
