// sample.cu -- draws a token from each row of a logit matrix: temperature, top-k, top-p and
// min-p, and one uniform number a row.
//
// With M the row's largest logit and t the temperature, token i weighs w_i = e^((x_i - M) / t).
// In the order of the logits (larger first, equal ones by the index) top-k leaves the first k, of
// these top-p the shortest beginning whose weights reach p times their sum, and of these min-p
// the ones with w >= min_p; the first token always stays.  The draw is the first token, in the
// order of the vocabulary, at which the running sum of what stays passes u times its total.
//
// A draw near a border of that sum is decided by the last digits, and there are as many borders
// as tokens.  So the weights that decide are whole numbers, 2^42 w: x - M exactly (as two
// binary32 terms), its product with log2(e) / t in two terms, 2^y
// from a table of sixteenths of an octave and the series of the exponential function: 4e-11 of w, and
// half a unit (as fine as sums of 2^20 of them in 64 bits, and of a CTA's in bins of 32, allow).
// Weights below 2^-12 are computed in binary32 (3e-7 of w, 5e-7 of their sums).  Whole numbers add up the same in any order, so
// atomics do not change a result.
//
// A cluster of 1 to 16 CTAs takes a row, as many as fill the GPU.
//   1. One pass over the logits: the largest value of every block of 32 elements of a thread, and
//      for top-p without top-k the block's sum of weights relative to it (binary32).
//   2. A bound below which nothing can stay: for top-k, a CTA's j-th largest thread (or block)
//      maximum is reached by j elements, so the least of these over the row's CTAs, j = ceil(k /
//      CTAs), by k; for top-p the largest tried below which the blocks' sums hold no more than 1 - p
//      of all; for min-p its own.
//   3. Blocks that reach the bound are read again (from L2), their elements from the bound on
//      listed; for top-p the rest's weights are summed, blocks that do not reach it as they are.
//   4. The first CTA resolves the list (some hundreds).  Up to 256 elements (a longer list of a top-k is
//      cut down first) are ranked by comparing each with each; up to 2048 are sorted into 256 bins
//      by value, and by column for the draw: a border falls in one bin, whose elements compare themselves.
// A list that overflows (flat rows), or no filter at all, goes over the row (or the CTAs' lists)
// instead: 256 bins with counts and weights, the border's bin refined until it fits a list, and the
// draw by sums of ever smaller ranges.
//
// Measured (a graph of calls): one row of 248320 fp16 with top-k 200, top-p and min-p 12.9 us, 768 rows of
// 50257 bf16 with top-p 42.7 us (77 MB, 27 % of the copy rate of HBM: after the pass, 8 us of a CTA's 20,
// three short phases of block-wide steps follow, and 768 rows are 1.3 waves), 200 rows of 32000 with no
// filter 20.3 us.  Flat rows cost more: 64 x 128257 fp32 with a top-p of 0.95 22.6 us at a temperature of 0.8
// and 97 at 1, where it leaves thousands.
#include <math.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>
#include <atomic>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "launch.h"
#include "ptx.cuh"
#include "qgemm.h"

namespace qw {

constexpr int kSmThreads = 256;
constexpr int kSmWarps = kSmThreads / 32;
constexpr int kSmBlocks = 8;                      // blocks a thread keeps the maxima of
constexpr int kSmList = 2048;                     // elements a CTA lists
constexpr int kSmPairs = 256;                     // a list whose elements are compared each with each
constexpr int kSmShort = 2048;                    // of all CTAs of a row: the first one's alone
constexpr int kSmBins = 256;
constexpr int kSmMaxCluster = 16;
constexpr int kSmFix = 42;                        // weights in units of 2^-42

typedef unsigned long long u64;

struct SampleArgs {
  const void *logits;
  const float *u;
  const float *temps, *top_ps, *min_ps;           // [M], or nullptr: the number below for every row
  const int *top_ks;
  float temp, top_p, min_p;
  int top_k;
  long long row_stride;                           // elements
  int M, N;
  int *token;
  float *logprob;
};

struct SampleSmem {
  union {
    struct {
      float bmax[kSmBlocks][kSmThreads], bsum[kSmBlocks][kSmThreads];
    };
    u64 w[kSmList];                               // (the blocks are done with when elements are weighed)
  };
  u64 key[kSmList];                               // order key << 32 | ~index
  union {
    unsigned short work[kSmBlocks * kSmThreads];
    unsigned short order[kSmShort];
  };
  unsigned short start[kSmBins + 1];
  unsigned cnt[kSmBins];                          // bins: elements,
  unsigned limb[3][kSmBins];                      // and weights in three terms of 14 bits (the last up to 2^14; a row's slice has below 2^18
  u64 mass[kSmBins];                              // elements); or their sum
  float red[kSmWarps];
  int nkey[2][kSmWarps];
  u64 rsum[kSmWarps];
  float rsum3[3][kSmWarps];
  // read by the cluster's other CTAs
  float xmax, xsum, xsum3[2][3];
  unsigned xkey;
  u64 xtotal;
  // written by them (first CTA)
  unsigned n, gidx;
  u64 tail[kSmMaxCluster];
  // results of one thread or CTA for all
  int bin;
  u64 mbefore, total, top, thr;
  float rowmax, rowsum;
  unsigned rowkey;
  int nwork;
};

// ------------------------------------------------------------------ clusters --
__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ unsigned cluster_size() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ uint32_t peer(const void *p, unsigned rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t peer_ld32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ u64 peer_ld64(uint32_t a) {
  u64 v;
  asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void peer_st64(uint32_t a, u64 v) {
  asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ void peer_min(uint32_t a, unsigned v) {
  asm volatile("red.relaxed.cluster.shared::cluster.min.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// ------------------------------------------------------------------- numbers --
__device__ __forceinline__ float sm_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float sm_lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Pairs of binary32, two to an instruction.
struct F2 {
  u64 v;
  __device__ __forceinline__ F2() {}
  __device__ __forceinline__ F2(float x, float y) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y)); }
  __device__ __forceinline__ void get(float &x, float &y) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
};
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
// binary32 values as unsigned integers in the values' order, -0 as +0, NaN below all (as -inf
// it is never drawn)
__device__ __forceinline__ unsigned sm_key(float x) {
  const unsigned u = __float_as_uint(x + 0.0f);
  return x == x ? u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u) : 0u;
}
__device__ __forceinline__ float sm_value(unsigned k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

// A row's scale: M and log2(e) / t = chi + clo.
struct SampleScale {
  float M, chi, clo;
};
// 2^42 2^(k / 16), k = -8 .. 8
static __device__ const u64 kSmPowers[17] = {
    3109888511975ull, 3247575039328ull, 3391357470036ull, 3541505692798ull, 3698301545306ull, 3862039343274ull,
    4033026432885ull, 4211583767698ull, 4398046511104ull, 4592764665442ull, 4796103728980ull, 5008445381977ull,
    5230188203118ull, 5461748417677ull, 5703560678795ull, 5956078883349ull, 6219777023951ull};
constexpr float kSmLight = -12.0f;                // log2 of the weight from which on it is computed by sm_heavy
constexpr float kSmLn2 = 0.693147181f;

// 2^42 2^y for y = (x - M) chi, -12 < y <= 0, to 4e-11 and half a unit: y in two terms, the nearest sixteenth of an
// octave from a table, and the rest's exponential by its series, whose first term is exact; the low
// term's enters with the rest's exponential as its factor (without, it is 1e-8 off).
// x - M is rounded for 16-bit types too: fp16 values span 40 bits, and a logit of 2.4e-4 under a largest
// of 7.9 loses 2.4e-7 of its weight.
static __device__ __noinline__ u64 sm_heavy(float x, float M, float chi, float clo) {
  const float d = x - M, y = d * chi, b = d - x;  // (x - (d - b)) + (-M - b): what the difference rounded off
  const float yl = fmaf((x - (d - b)) + (-M - b), chi, fmaf(d, chi, -y) + d * clo);
  const float n = rintf(y), f = y - n;
  const float k = rintf(f * 16.0f), s = fmaf(k, -0.0625f, f);
  constexpr float L = 0.693147180559945f, Llo = (float)(0.69314718055994530942 - (double)L);
  const float p = s * L, pl = fmaf(s, L, -p) + s * Llo, low = yl * L;
  // (2^s - 1 - s ln 2) / s^2: ln(2)^k / k! s^(k - 2), k = 2 .. 5
  float q = fmaf(1.33335581e-3f, s, 9.61812911e-3f);
  q = fmaf(q, s, 5.55041087e-2f);
  q = fmaf(q, s, 0.240226507f);
  const float z = q * (s * s), rest = fmaf(low, p + z, low) + (z + pl);
  const long long t = (long long)__float2int_rn(p * 68719476736.0f) + __float2int_rn(rest * 68719476736.0f);
  const u64 w = kSmPowers[(int)k + 8];
  const u64 v = w + (u64)__mul64hi((long long)(w << 20), t << 8);
  const int r = -(int)n;
  return (v + ((1ull << r) >> 1)) >> r;
}
// e^((x - M) / t) in binary32, 0 below 2^-125 (and for NaN): 2^y, and times what y and x - M round off.
// (From y alone the weights of a row would all be off the same way, by up to 1.6e-6.)
__device__ __forceinline__ float sm_light(float x, const SampleScale &c) {
  const float d = x - c.M, y = d * c.chi, b = d - x;
  if (!(y > -125.0f)) return 0.0f;
  const float e = sm_ex2(y);
  return fmaf(e, kSmLn2 * fmaf((x - (d - b)) + (-c.M - b), c.chi, fmaf(d, c.chi, -y) + d * c.clo), e);
}
// 2^42 e^((x - M) / t), rounded; 0 for -inf and NaN.  Below 2^-12 in binary32: ex2's 2^-22 of the weight
// and 2^-24.
__device__ __forceinline__ u64 sm_weight(float x, const SampleScale &c) {
  if (x == c.M) return 1ull << kSmFix;            // (+inf too)
  if ((x - c.M) * c.chi > kSmLight) return sm_heavy(x, c.M, c.chi, c.clo);
  return __float2uint_rn(sm_light(x, c) * (float)(1ull << kSmFix));
}

// A row as 16-byte vectors: vector v holds columns v VE - pad .. + VE - 1, pad being how many
// elements the row starts past a 16-byte boundary.  Places outside the row read as -inf.
template <typename T>
struct SampleRow {
  static constexpr int VE = 16 / sizeof(T);
  static constexpr bool kF32 = sizeof(T) == 4;
  static constexpr bool kBf = sizeof(T) == 2 && !__is_same(T, __half);
  const T *row;
  int pad, N, nvec, in0, in1;                     // whole vectors: [in0, in1)
  __device__ __forceinline__ SampleRow(const T *r, int n) : row(r), N(n) {
    pad = (int)((reinterpret_cast<uintptr_t>(r) / sizeof(T)) % VE);
    nvec = (n + pad + VE - 1) / VE;
    in0 = pad > 0 ? 1 : 0;
    in1 = max((n + pad) / VE, in0);
  }
  __device__ __forceinline__ int col(int v) const { return v * VE - pad; }
  static constexpr uint32_t kLowest = kF32 ? 0xff800000u : kBf ? 0xff80u : 0xfc00u;      // -inf
  static __device__ __noinline__ uint4 edge(const T *row, int c, int N) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kF32) {
        const int j = c + i;
        w[i] = (unsigned)j < (unsigned)N ? __ldg(reinterpret_cast<const uint32_t *>(row) + j) : kLowest;
      } else {
        w[i] = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int j = c + 2 * i + h;
          const uint32_t x = (unsigned)j < (unsigned)N ? __ldg(reinterpret_cast<const uint16_t *>(row) + j) : kLowest;
          w[i] |= x << (16 * h);
        }
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ uint4 load(int v) const {
    return v >= in0 && v < in1 ? __ldg(reinterpret_cast<const uint4 *>(row + col(v))) : edge(row, col(v), N);
  }
  __device__ __forceinline__ static uint4 nothing() {
    constexpr uint32_t w = kF32 ? kLowest : kLowest * 0x10001u;
    return make_uint4(w, w, w, w);
  }
  __device__ __forceinline__ static void floats(const uint4 &r, float (&x)[VE]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kF32) {
        x[i] = __uint_as_float(w[i]);
      } else if constexpr (kBf) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        const float2 f = __half22float2(u32_as_h2(w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    }
  }
  // the largest of a vector's elements so far (packed for 16-bit types; NaN left out)
  __device__ __forceinline__ static uint32_t max2(uint32_t a, uint32_t b) {
    if constexpr (kF32) return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    else if constexpr (kBf) {
      const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
      return *reinterpret_cast<const uint32_t *>(&r);
    } else return h2_as_u32(__hmax2(u32_as_h2(a), u32_as_h2(b)));
  }
  // elements below `low` (or NaN) raised to it
  __device__ __forceinline__ static uint4 raised(const uint4 &r, uint32_t low) {
    return make_uint4(max2(r.x, low), max2(r.y, low), max2(r.z, low), max2(r.w, low));
  }
  // the value next below x, or x, twice for 16-bit types
  __device__ __forceinline__ static uint32_t packed(float x) {
    if constexpr (kF32) return __float_as_uint(x);
    else if constexpr (kBf) return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rd(x)) * 0x10001u;
    else return (uint32_t)__half_as_ushort(__float2half_rd(x)) * 0x10001u;
  }
  __device__ __forceinline__ static float max_of(uint32_t m) {
    float r;
    if constexpr (kF32) r = __uint_as_float(m);
    else if constexpr (kBf) r = fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    else {
      const float2 f = __half22float2(u32_as_h2(m));
      r = fmaxf(f.x, f.y);
    }
    return r == r ? r : -INFINITY;                // all NaN
  }
};

__device__ __forceinline__ int sm_bin_shift(u64 range) { return max(0, 56 - __clzll((long long)range)); }      // range >> it <= 255

// One CTA's place in the row's cluster.
template <typename T>
struct SampleCta {
  static constexpr int VE = SampleRow<T>::VE;
  SampleSmem &s;
  SampleRow<T> row;
  int tid, warp, lane;
  unsigned rank, size;
  int v0, v1;                                     // its vectors
  SampleScale sc;
  uint32_t lowest;                                // as vector_weight's, twice for 16-bit types

  __device__ __forceinline__ void sync() {        // the cluster's CTAs
    if (size > 1) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
  }
  __device__ __forceinline__ u64 weight(float x) const { return sm_weight(x, sc); }
  // The CTAs' lists at `list`, one behind the other in the first CTA's, if they are `most` together or
  // fewer; their number.  After a sync(), and ends with one.
  __device__ __forceinline__ unsigned join_lists(u64 *list, unsigned most, bool &full) {
    unsigned n = 0, before = 0;
    full = false;
    for (unsigned r = 0; r < size; ++r) {
      if (r == rank) before = n;
      const unsigned m = size > 1 ? peer_ld32(peer(&s.n, r)) : s.n;
      full |= m > kSmList;
      n += m;
    }
    if (n <= most && rank > 0) {
      const uint32_t to = peer(list, 0) + 8 * before;
      for (unsigned e = tid; e < s.n; e += kSmThreads) peer_st64(to + 8 * e, list[e]);
    }
    sync();
    return n;
  }

  // bin tid's count or weight `v`: the first bin at which `need` is reached (-1: none; before it:
  // s.mbefore), and the sum of all bins
  __device__ __forceinline__ int pick(u64 v, u64 need, u64 &total) {
    u64 incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    __syncthreads();
    if (lane == 31) s.rsum[warp] = incl;
    if (tid == 0) s.bin = -1;
    __syncthreads();
    total = 0;
    u64 before = 0;
    for (int w = 0; w < kSmWarps; ++w) {
      if (w == warp) before = total;
      total += s.rsum[w];
    }
    incl += before;
    if (incl >= need && incl - v < need) {
      s.bin = tid;
      s.mbefore = incl - v;
    }
    __syncthreads();
    return s.bin;
  }
  // Calls f(x, column) for the elements of vectors a, a + step, .. < b; four loads at a time.  Places
  // outside the row are -inf.
  template <typename F>
  __device__ __forceinline__ void walk(int a, int b, int step, F f) {
    for (int v = a; v < b; v += 4 * step) {
      uint4 raw[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) raw[i] = v + i * step < b ? row.load(v + i * step) : SampleRow<T>::nothing();
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        float x[VE];
        SampleRow<T>::floats(raw[0], x);
        raw[0] = raw[1];
        raw[1] = raw[2];
        raw[2] = raw[3];
        const int c = row.col(v + i * step);
#pragma unroll
        for (int e = 0; e < VE; ++e) f(x[e], c + e);
      }
    }
  }
  // The weights of one vector's elements, in sum: the light ones in binary32, as sm_light's, two at a
  // time.  (Of 16-bit types without what x - M rounds off, half a step of it: logits below 2^-9 in size
  // alone have bits there.)  Elements below `lowest` (also -inf and NaN) count as that, 2^-100.
  __device__ __forceinline__ u64 vector_weight(uint4 raw) const {
    raw = row.raised(raw, lowest);
    float x[VE];
    SampleRow<T>::floats(raw, x);
    const float top = row.max_of(row.max2(row.max2(raw.x, raw.y), row.max2(raw.z, raw.w)));
    u64 total = 0;
    if ((top - sc.M) * sc.chi > kSmLight) {
      const float low = row.max_of(lowest);
      unsigned heavy = 0;
#pragma unroll
      for (int e = 0; e < VE; ++e) heavy |= (x[e] - sc.M) * sc.chi > kSmLight ? 1u << e : 0u;
      for (; heavy; heavy &= heavy - 1) {
        const int k = __ffs(heavy) - 1;
        float v = x[0];
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          v = e == k ? x[e] : v;
          x[e] = e == k ? low : x[e];
        }
        total += weight(v);
      }
    }
    const F2 to(-sc.M, -sc.M), chi(sc.chi, sc.chi), less(-sc.chi, -sc.chi), clo(sc.clo, sc.clo);
    F2 w[VE / 2], off(0.0f, 0.0f);
#pragma unroll
    for (int e = 0; e < VE; e += 2) {
      const F2 v(x[e], x[e + 1]), d = add2(v, to), y = mul2(d, less);        // (-y)
      F2 r = fma2(d, clo, fma2(d, chi, y));
      if constexpr (SampleRow<T>::kF32) {         // what the difference rounded off
        const F2 minus(-1.0f, -1.0f), b = fma2(v, minus, d);
        r = fma2(add2(fma2(fma2(b, minus, d), minus, v), fma2(b, minus, to)), chi, r);
      }
      float y0, y1;
      y.get(y0, y1);
      w[e / 2] = F2(sm_ex2(-y0), sm_ex2(-y1));
      off = fma2(w[e / 2], r, off);
    }
    if constexpr (VE == 8) {
      w[0] = add2(w[0], w[1]);
      w[1] = add2(w[2], w[3]);
    }
    float s0, s1, o0, o1;
    add2(w[0], w[1]).get(s0, s1);
    off.get(o0, o1);
    const float sum = fmaf(kSmLn2, o0 + o1, s0 + s1);
    return total + ((u64)__float2uint_rn(sum * (float)(1ull << (kSmFix - 2))) << 2);       // (half of four units is at most half of one an element)
  }
  template <typename F>
  __device__ __forceinline__ void each(F f) {
    walk(v0 + tid, v1, kSmThreads, f);
  }
  template <bool ALL, typename F>
  __device__ __forceinline__ u64 warp_sum(F &f, int a, int b) {
    u64 sum = 0;
    if constexpr (ALL) {
      for (int v = a + lane; v < b; v += 128) {
        uint4 raw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) raw[i] = v + i * 32 < b ? row.load(v + i * 32) : SampleRow<T>::nothing();
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          sum += vector_weight(raw[0]);
          raw[0] = raw[1];
          raw[1] = raw[2];
          raw[2] = raw[3];
        }
      }
    } else {
      walk(a + lane, b, 32, [&](float x, int col) { sum += f(x, col); });
    }
    return reduce(sum);
  }
  __device__ __forceinline__ static u64 reduce(u64 x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
  }

  // The first column, in order, at which the running sum of f over the whole row passes
  // target(total): by the sums of the CTAs, of the warps' ranges and of pieces of one range.
  // done(column, logit, total) is called by one thread of the CTA that holds it.
  // ALL: f is every element's weight.
  template <bool ALL, typename F, typename G, typename H>
  __device__ __forceinline__ void find(F f, G target, H done) {
    const int per = (v1 - v0 + kSmWarps - 1) / kSmWarps;
    auto begin = [&](int w) { return min(v0 + w * per, v1); };
    __syncthreads();
    const u64 mine = warp_sum<ALL>(f, begin(warp), begin(warp + 1));
    if (lane == 0) s.rsum[warp] = mine;
    __syncthreads();
    if (tid == 0) {
      u64 t = 0;
      for (int w = 0; w < kSmWarps; ++w) t += s.rsum[w];
      s.xtotal = t;
    }
    sync();
    u64 total = 0, before = 0, own = 0;
    for (unsigned r = 0; r < size; ++r) {
      const u64 t = size > 1 ? peer_ld64(peer(&s.xtotal, r)) : s.xtotal;
      if (r == rank) {
        before = total;
        own = t;
      }
      total += t;
    }
    u64 at = target(total);
    const bool here = at >= before && at < before + own;
    if (here) {                                   // (the whole CTA)
      at -= before;
      int w = 0;
      while (w < kSmWarps - 1 && at >= s.rsum[w]) at -= s.rsum[w++];
      const int a = begin(w), b = begin(w + 1), len = (b - a + kSmWarps - 1) / kSmWarps;
      const int p0 = min(a + warp * len, b), p1 = min(p0 + len, b);
      const u64 piece = warp_sum<ALL>(f, p0, p1);
      __syncthreads();
      if (lane == 0) s.rsum[warp] = piece;
      __syncthreads();
      int q = 0;
      while (q < kSmWarps - 1 && at >= s.rsum[q]) at -= s.rsum[q++];
      if (q == warp) {
        for (int v = p0; v < p1; v += 32) {       // 32 vectors at a time
          float x[VE];
          u64 sum = 0;
          const int c = row.col(v + lane);
          const uint4 raw = v + lane < p1 ? row.load(v + lane) : SampleRow<T>::nothing();
          SampleRow<T>::floats(raw, x);
          if constexpr (ALL) {
            sum = vector_weight(raw);
          } else {
#pragma unroll
            for (int e = 0; e < VE; ++e) sum += f(x[e], c + e);
          }
          u64 incl = sum;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const u64 y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
          }
          const unsigned past = __ballot_sync(0xffffffffu, incl > at);
          if (past) {
            if (lane == __ffs(past) - 1) {
              // (one by one the elements may round to a little less than together: then the last, or
              // where all round to 0 the largest)
              u64 run = incl - sum;
              int found = -1;
              float logit = -INFINITY;
#pragma unroll
              for (int e = 0; e < VE; ++e) {
                const u64 y = f(x[e], c + e);
                if (run <= at && y > 0) {
                  found = c + e;
                  logit = x[e];
                }
                run += y;
              }
              if (found < 0) {
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                  if (x[e] > logit) {
                    logit = x[e];
                    found = c + e;
                  }
                }
              }
              done(found, logit, total);
            }
            break;
          }
          at -= __shfl_sync(0xffffffffu, incl, 31);
        }
      }
    }
  }
};

// The token of logit x, and the logarithm of its share: (x - M) / t less that of the total, which is 1
// and more.  Neither is above 0, so nothing cancels (a far token's weight has few bits left of its
// units: from the quotient of weights the logarithm was off by 1e-3 at 2^-30).
__device__ __forceinline__ void sample_write(const SampleArgs &a, int r, int token, float x, const SampleScale &c, u64 total) {
  a.token[r] = token;
  if (!a.logprob) return;
  float q = 0.0f, rest = 0.0f;
  if (x != c.M) {                                 // (not both infinite)
    constexpr float L = 0.693147180559945f, Llo = (float)(0.69314718055994530942 - (double)L);
    const float d = x - c.M, y = d * c.chi, b = d - x;
    q = y * L;
    rest = fmaf(y, L, -q) + y * Llo + L * fmaf((x - (d - b)) + (-c.M - b), c.chi, fmaf(d, c.chi, -y) + d * c.clo);
  }
  constexpr u64 one = 1ull << kSmFix;
  a.logprob[r] = q - log1pf((float)(total - one) * (1.0f / (float)one)) + rest;
}
// floor(u total), below total
__device__ __forceinline__ u64 sample_target(float u, u64 total) {
  const double t = (double)u * (double)total;
  return t > 0.0 ? min((u64)fmin(t, 1e19), total - 1) : 0;         // (NaN: 0)
}
// the least whole number that is not below p total
__device__ __forceinline__ u64 sample_mass(float p, u64 total) {
  return p > 0.0f ? (u64)ceil((double)p * (double)total) : 0;
}

// ------------------------------------------------------------------ the list --
// Keeps of a list what is not surely below its k-th element (k > 0): the key reached by k elements at
// least is raised by halving, until few more than k reach it.  Returns how many are left.
template <typename T>
__device__ __forceinline__ int sample_shrink(SampleCta<T> &t, int n, int k, unsigned low) {
  SampleSmem &s = t.s;
  constexpr int PER = kSmShort / kSmThreads;
  u64 key[PER];
  unsigned high = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = t.tid + i * kSmThreads;
    key[i] = e < n ? s.key[e] : 0;
    high = max(high, (unsigned)(key[i] >> 32));
  }
  high = __reduce_max_sync(0xffffffffu, high);
  if (t.lane == 0) s.cnt[t.warp] = high;
  if (t.tid == 0) s.nwork = 0;
  __syncthreads();
#pragma unroll
  for (int v = 0; v < kSmWarps; ++v) high = max(high, s.cnt[v]);
  const int enough = k + max(k / 4, 16);
  int left = n;
#pragma unroll 1
  for (int round = 0; round < 16 && left > enough && low < high; ++round) {
    const unsigned mid = low + (high - low) / 2 + 1;
    int c = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) c += (unsigned)(key[i] >> 32) >= mid;
    c = __reduce_add_sync(0xffffffffu, c);
    if (t.lane == 0) s.nkey[round & 1][t.warp] = c;
    __syncthreads();
    c = 0;
#pragma unroll
    for (int v = 0; v < kSmWarps; ++v) c += s.nkey[round & 1][v];
    if (c >= k) {
      low = mid;
      left = c;
    } else {
      high = mid - 1;
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if ((unsigned)(key[i] >> 32) >= low && key[i]) s.key[atomicAdd(&s.nwork, 1)] = key[i];
  __syncthreads();
  return left;
}

// A list of kSmPairs elements at most: sorted by comparing each with each, by a thread or a few an
// element; every filter then leaves a first part of it.  (min-p almost: weights of logits next to each
// other may round the other way round, so what stays is looked for up to the last of it.)
template <typename T>
__device__ __forceinline__ void sample_pairs(const SampleArgs &a, SampleCta<T> &t, int r, int n, int k, float p, float mp,
                                             float u) {
  SampleSmem &s = t.s;
  const int tid = t.tid, lane = t.lane, warp = t.warp;
  auto threads = [](int n) { return n <= 32 ? 3 : n <= 64 ? 2 : n <= 128 ? 1 : 0; };       // an element, log2
  u64 *const sorted = s.key + kSmPairs + 2;
  {
    const int lg = threads(n), e = tid >> lg, first = tid & ((1 << lg) - 1);
    if (tid < 2) s.key[n + tid] = 0;              // (below all)
    u64 tails = 0;
    if (p < 1.0f && k == 0 && tid < (int)t.size) tails = s.tail[tid];
    if (warp == 0) {
      tails = SampleCta<T>::reduce(tails);
      if (lane == 0) s.thr = tails;
    }
    __syncthreads();
    const u64 key = e < n ? s.key[e] : ~0ull;
    int above = 0;
#pragma unroll 4
    for (int q = 2 * first; q < n; q += 2 << lg) above += (s.key[q] > key) + (s.key[q + 1] > key);
    for (int o = 1; o < 1 << lg; o <<= 1) above += __shfl_xor_sync(0xffffffffu, above, o);
    if (e < n && first == 0) sorted[above] = key;
    __syncthreads();
  }
  const u64 key = tid < n ? sorted[tid] : 0;
  bool keep = tid < n && (k == 0 || tid < k);
  const u64 w = keep ? t.weight(sm_value((unsigned)(key >> 32))) : 0;
  if (p < 1.0f) {
    u64 incl = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) s.mass[warp] = incl;
    __syncthreads();
    u64 all = s.thr, before = incl - w;
#pragma unroll
    for (int v = 0; v < kSmWarps; ++v) {
      all += s.mass[v];
      if (v < warp) before += s.mass[v];
    }
    keep = keep && (before < sample_mass(p, all) || tid == 0);
  }
  if (mp > 0.0f) {
    const u64 least = (u64)ceil((double)mp * (double)(1ull << kSmFix));
    keep = keep && (w >= least || tid == 0);
  }
  // the draw among what stays, in the order of the vocabulary
  s.cnt[tid] = keep ? ~(unsigned)key : 0xffffffffu;
  s.w[tid] = keep ? w : 0;
  const u64 part = SampleCta<T>::reduce(keep ? w : 0);
  const unsigned stay = __ballot_sync(0xffffffffu, keep);
  if (lane == 0) {
    s.rsum[warp] = part;
    s.nkey[0][warp] = stay ? 32 * warp + 32 - __clz(stay) : 0;
  }
  __syncthreads();
  u64 all = 0, before = 0;
  int m = 0;
#pragma unroll
  for (int v = 0; v < kSmWarps; ++v) {
    all += s.rsum[v];
    m = max(m, s.nkey[0][v]);
  }
  const int lg = threads(m), e = tid >> lg;
  const unsigned col = s.cnt[e];
#pragma unroll 4
  for (int q = tid & ((1 << lg) - 1); q < m; q += 1 << lg) {
    const u64 other = s.w[q];
    before += s.cnt[q] < col ? other : 0;
  }
  for (int o = 1; o < 1 << lg; o <<= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  const u64 target = sample_target(u, all), mine = s.w[e];
  if ((tid & ((1 << lg) - 1)) == 0 && e < m && before <= target && before + mine > target)
    sample_write(a, r, (int)col, sm_value((unsigned)(sorted[e] >> 32)), t.sc, all);
}

// Resolves the list of n elements from the key `low` on (one CTA): which stay, and the draw among them.
// The elements are sorted into 256 bins, by their values for the filters' borders, by their columns
// for the draw; a border falls in one bin, whose elements compare themselves with each other.
template <typename T>
__device__ __forceinline__ void sample_list(const SampleArgs &a, SampleCta<T> &t, int r, int n, int k, float p, float mp,
                                            float u, unsigned low) {
  SampleSmem &s = t.s;
  const int tid = t.tid, lane = t.lane;
  if (k > 0 && n > 64 && n > k) n = sample_shrink(t, n, k, low);
  if (n <= kSmPairs) {
    sample_pairs(a, t, r, n, k, p, mp, u);
    return;
  }
  unsigned keep = 0;                              // bit i: element tid + i kSmThreads stays
  u64 best = 0, least = ~0ull;
  for (int e = tid, i = 0; e < n; e += kSmThreads, ++i) {
    const u64 key = s.key[e];
    s.w[e] = t.weight(sm_value((unsigned)(key >> 32)));
    keep |= 1u << i;
    best = max(best, key);
    least = min(least, key);
  }
  const unsigned k0 = __reduce_min_sync(0xffffffffu, (unsigned)(least >> 32));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
  if (lane == 0) {
    s.rsum[t.warp] = best;
    s.nkey[0][t.warp] = (int)k0;
  }
  __syncthreads();
  unsigned last = ~0u;
#pragma unroll
  for (int v = 0; v < kSmWarps; ++v) {
    best = max(best, s.rsum[v]);
    last = min(last, (unsigned)s.nkey[0][v]);
  }
  // bins of equal width from the largest value to the smallest (a NaN, as of infinities, is bin 0)
  const float from = sm_value((unsigned)(best >> 32)), per = (float)kSmBins * 0.9999f / (from - sm_value(last));
  auto value_bin = [&](u64 key) { return min(max((int)((from - sm_value((unsigned)(key >> 32))) * per), 0), kSmBins - 1); };
  const int width = (t.row.N + kSmBins - 1) / kSmBins;
  auto column_bin = [&](u64 key) { return (int)(~(unsigned)key) / width; };
  // what stays, by its bins: bin b's are s.order[s.start[b]] .. [s.start[b + 1] - 1]
  auto sort = [&](auto bin) {
    s.cnt[tid] = 0;
    __syncthreads();
    for (int e = tid, i = 0; e < n; e += kSmThreads, ++i)
      if (keep >> i & 1) atomicAdd(&s.cnt[bin(s.key[e])], 1u);
    __syncthreads();
    const unsigned own = s.cnt[tid];
    unsigned incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) s.nkey[0][t.warp] = (int)incl;
    __syncthreads();
    for (int v = 0; v < t.warp; ++v) incl += (unsigned)s.nkey[0][v];
    s.start[tid + 1] = (unsigned short)incl;
    if (tid == 0) s.start[0] = 0;
    s.cnt[tid] = incl - own;
    __syncthreads();
    for (int e = tid, i = 0; e < n; e += kSmThreads, ++i)
      if (keep >> i & 1) s.order[atomicAdd(&s.cnt[bin(s.key[e])], 1u)] = (unsigned short)e;
    __syncthreads();
  };
  auto others = [&](int b, auto f) {
    const int end = s.start[b + 1];
#pragma unroll 4
    for (int q = s.start[b]; q < end; ++q) f(s.order[q]);
  };
  // the first bin at which the running weight (or number) of what stays reaches `need`: s.bin
  // (kSmBins: none), and what lies before it: s.mbefore.  need(total): from all of it.
  auto border = [&](bool by_mass, auto need) {
    u64 own = s.start[tid + 1] - s.start[tid];
    if (by_mass) {
      own = 0;
      others(tid, [&](int e) { own += s.w[e]; });
    }
    u64 incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) s.rsum[t.warp] = incl;
    if (tid == 0) s.bin = kSmBins;
    __syncthreads();
    u64 total = 0, before = 0;
#pragma unroll
    for (int v = 0; v < kSmWarps; ++v) {
      if (v == t.warp) before = total;
      total += s.rsum[v];
    }
    incl += before;
    const u64 at = need(total);
    if (incl >= at && (incl - own < at || (at == 0 && tid == 0))) {        // (one thread)
      s.bin = tid;
      s.mbefore = incl - own;
    }
    __syncthreads();
    return at;
  };
  if ((k > 0 && n > k) || p < 1.0f) sort(value_bin);
  if (k > 0 && n > k) {
    (void)border(false, [&](u64) { return (u64)k; });
    const int kb = s.bin;
    const unsigned before = (unsigned)s.mbefore;
    unsigned out = 0;
    for (int e = tid, i = 0; e < n; e += kSmThreads, ++i) {
      const u64 key = s.key[e];
      const int b = value_bin(key);
      if (b < kb) continue;
      unsigned rank = before;
      if (b == kb) others(kb, [&](int o) { rank += s.key[o] > key; });
      if (b > kb || rank >= (unsigned)k) out |= 1u << i;
    }
    __syncthreads();
    keep &= ~out;
    for (int e = tid, i = 0; e < n; e += kSmThreads, ++i)
      if (out >> i & 1) s.w[e] = 0;
    __syncthreads();
  }
  if (p < 1.0f) {
    u64 tails = 0;
    if (k == 0)
      for (unsigned q = 0; q < t.size; ++q) tails += s.tail[q];
    const u64 thr = border(true, [&](u64 total) { return sample_mass(p, total + tails); });
    const int pb = s.bin;
    for (int e = tid, i = 0; e < n; e += kSmThreads, ++i) {
      const u64 key = s.key[e];
      const int b = value_bin(key);
      if (!(keep >> i & 1) || b < pb || key == best) continue;
      u64 above = thr;
      if (b == pb) {
        above = s.mbefore;
        others(pb, [&](int o) { if (s.key[o] > key) above += s.w[o]; });
      }
      if (above >= thr) keep &= ~(1u << i);
    }
  }
  if (mp > 0.0f) {
    const u64 bar = (u64)ceil((double)mp * (double)(1ull << kSmFix));
    for (int e = tid, i = 0; e < n; e += kSmThreads, ++i)
      if (s.w[e] < bar && s.key[e] != best) keep &= ~(1u << i);
  }
  // the draw, in the order of the vocabulary
  __syncthreads();
  sort(column_bin);
  u64 all = 0;
  const u64 target = border(true, [&](u64 total) {
    all = total;
    return sample_target(u, total) + 1;
  }) - 1;
  const int vb = s.bin;
  for (int e = tid, i = 0; e < n; e += kSmThreads, ++i) {
    const u64 key = s.key[e];
    if (!(keep >> i & 1) || column_bin(key) != vb) continue;
    const unsigned col = ~(unsigned)key;
    u64 run = s.mbefore;
    others(vb, [&](int o) { if (~(unsigned)s.key[o] < col) run += s.w[o]; });
    if (run <= target && run + s.w[e] > target) sample_write(a, r, (int)col, sm_value((unsigned)(key >> 32)), t.sc, all);
  }
}

// --------------------------------------------------------------- whole rows --
// What stays: keys above K, and those equal to it up to column I.
struct SampleCut {
  unsigned K;
  int I;
  __device__ __forceinline__ bool stays(unsigned key, int col) const { return key > K || (key == K && col <= I); }
};

// The draw among what the cut and min-p leave.
template <typename T, bool ALL>
__device__ __forceinline__ void sample_draw(const SampleArgs &a, SampleCta<T> &t, int r, const SampleCut &cut, float mp, float u) {
  const u64 least = (u64)ceil((double)mp * (double)(1ull << kSmFix));
  t.sync();
  t.template find<ALL>(
      [&](float x, int col) {
        if (!ALL && !cut.stays(sm_key(x), col)) return 0ull;
        const u64 w = t.weight(x);
        return ALL || w >= least ? w : 0ull;
      },
      [&](u64 total) { return sample_target(u, total); },
      [&](int col, float x, u64 total) { sample_write(a, r, col, x, t.sc, total); });
}
// The same from the CTAs' lists (n of them in this one).
template <typename T>
__device__ __forceinline__ void sample_draw_listed(const SampleArgs &a, SampleCta<T> &t, int r, int n, const SampleCut &cut, float mp, float u) {
  SampleSmem &s = t.s;
  const u64 least = (u64)ceil((double)mp * (double)(1ull << kSmFix));
  u64 sum = 0;
  t.sync();                                       // (the border's list, at the same place, has been read)
  for (int e = t.tid; e < n; e += kSmThreads) {
    const unsigned key = (unsigned)(s.key[e] >> 32);
    u64 w = 0;
    if (cut.stays(key, (int)~(unsigned)s.key[e])) w = t.weight(sm_value(key));
    if (w < least) w = 0;
    s.w[e] = w;
    sum += w;
  }
  u64 own;
  (void)t.pick(sum, ~0ull, own);
  if (t.tid == 0) s.xtotal = own;
  t.sync();
  u64 total = 0, before = 0;
  for (unsigned q = 0; q < t.size; ++q) {
    if (q == t.rank) before = total;
    total += t.size > 1 ? peer_ld64(peer(&s.xtotal, q)) : s.xtotal;
  }
  const u64 target = sample_target(u, total);
  if (target < before || target >= before + own) return;
  u64 need = target - before + 1;
  unsigned lo = 0, hi = (unsigned)t.row.N - 1;    // its column, refined by 256 bins a round
  while (lo != hi) {
    const int shift = sm_bin_shift(hi - lo);
    s.mass[t.tid] = 0;
    __syncthreads();
    for (int e = t.tid; e < n; e += kSmThreads) {
      const unsigned c = ~(unsigned)s.key[e];
      if (c >= lo && c <= hi && s.w[e]) atomicAdd(&s.mass[(c - lo) >> shift], s.w[e]);
    }
    __syncthreads();
    u64 all;
    const int b = max(t.pick(s.mass[t.tid], need, all), 0);
    need -= s.mbefore;
    lo += (unsigned)b << shift;
    hi = min(hi, lo + ((1u << shift) - 1));
    __syncthreads();
  }
  for (int e = t.tid; e < n; e += kSmThreads)
    if (~(unsigned)s.key[e] == lo) sample_write(a, r, (int)lo, sm_value((unsigned)(s.key[e] >> 32)), t.sc, total);
}

// A number in the elements' order: 4095 less the distance from the largest in steps of the first
// 41 octaves' (or of the bound's) 4095th part, the order key, the column backwards (N <= 2^20).  The
// first 12 bits spread the elements over bins, where the key alone crowds them into a few exponents
// (64 rows of 128257 fp32, top-p 0.95, nine tenths masked, temperatures of 0.8, 1 and 1.2: 44, 53 and 61 us, by keys
// 50, 59 and 67; unmasked, so with tens of thousands of them, 23, 97 and 147, by keys 24, 93 and 135).
struct SampleOrder {
  float M, steps;
  __device__ __forceinline__ SampleOrder(const SampleScale &c, unsigned T0)
      : M(c.M), steps(4095.0f / fminf(c.M - sm_value(T0), 41.0f / c.chi)) {}
  __device__ __forceinline__ u64 operator()(unsigned key, int col) const {
    const int d = min(max((int)((M - sm_value(key)) * steps), 0), 4095);         // (a NaN, as of infinities: 0)
    return (u64)(4095 - d) << 52 | (u64)key << 20 | (unsigned)(0xfffff - col);
  }
  static __device__ __forceinline__ unsigned key(u64 c) { return (unsigned)(c >> 20); }
  static __device__ __forceinline__ int column(u64 c) { return 0xfffff - (int)(c & 0xfffff); }
};

// The list that overflowed: the order numbers refined by 256 bins a round, all from one number of
// leading bits on, until the border's bin fits a list, which the first CTA refines further.
// items(f): calls f(order, x) for the CTA's elements from the bound T0 on.
template <typename T, typename I>
__device__ __forceinline__ SampleCut sample_flat(SampleCta<T> &t, const SampleOrder &order, int k, float p, u64 tail, unsigned T0, I items) {
  SampleSmem &s = t.s;
  const int tid = t.tid;
  auto pick = [&](u64 v, u64 need, u64 &total) { return t.pick(v, need, total); };
  // The order of the element up to which `need` is reached, in descending order from `high` down
  // to `low`: a number of elements, or (by_mass) a weight; share >= 0: that share of all weights and `tail`.
  auto border = [&](u64 high, u64 low, u64 need, bool by_mass, float share, u64 &found) {
    const u64 all = low;
    for (;;) {
      const u64 range = high - low;
      const int shift = sm_bin_shift(range);
      t.sync();                                   // the last round's bins have been read
      s.cnt[tid] = 0;
#pragma unroll
      for (int i = 0; i < 3; ++i) s.limb[i][tid] = 0;
      if (tid == 0) s.n = 0;
      __syncthreads();
      items([&](u64 c, float x) {
        if (c < low || c > high) return;
        const int b = (int)((high - c) >> shift);
        atomicAdd(&s.cnt[b], 1u);
        if (by_mass) {
          const u64 w = t.weight(x);
          atomicAdd(&s.limb[0][b], (unsigned)w & 0x3fffu);
          atomicAdd(&s.limb[1][b], (unsigned)(w >> 14) & 0x3fffu);
          atomicAdd(&s.limb[2][b], (unsigned)(w >> 28));
        }
      });
      __syncthreads();
      s.mass[tid] = (u64)s.limb[0][tid] + ((u64)s.limb[1][tid] << 14) + ((u64)s.limb[2][tid] << 28);
      t.sync();
      u64 mass = 0, number = 0, total;
      for (unsigned r = 0; r < t.size; ++r) {
        number += t.size > 1 ? peer_ld32(peer(&s.cnt[tid], r)) : s.cnt[tid];
        if (by_mass) mass += t.size > 1 ? peer_ld64(peer(&s.mass[tid], r)) : s.mass[tid];
      }
      if (share >= 0.0f) {
        (void)pick(mass, 0, total);
        need = max(sample_mass(share, total + tail), 1ull);
        share = -1.0f;
      }
      const int b = pick(by_mass ? mass : number, need, total);
      if (b < 0) {                                // all of them stay
        found = all;
        return;
      }
      need -= s.mbefore;
      if (tid == b) s.total = number;
      high -= (u64)b << shift;
      low = max(low, high - min(high, (1ull << shift) - 1));
      __syncthreads();
      if (s.total <= kSmList) break;
    }
    // the list of the border's bin
    items([&](u64 c, float) {
      if (c < low || c > high) return;
      s.w[atomicAdd(&s.n, 1u)] = c;
    });
    t.sync();
    bool full;
    const int n = (int)t.join_lists(s.w, kSmList, full);
    if (t.rank == 0) {
      auto weigh = [&](u64 c) { return by_mass ? t.weight(sm_value(SampleOrder::key(c))) : 1ull; };
      int left = n;
      while (left > kSmPairs && high != low) {
        const int shift = sm_bin_shift(high - low);
        __syncthreads();
        s.mass[tid] = 0;
        __syncthreads();
        for (int e = tid; e < n; e += kSmThreads)
          if (s.w[e] >= low && s.w[e] <= high) atomicAdd(&s.mass[(int)((high - s.w[e]) >> shift)], weigh(s.w[e]));
        __syncthreads();
        u64 total;
        const int b = max(pick(s.mass[tid], need, total), 0);
        need -= s.mbefore;
        high -= (u64)b << shift;
        low = max(low, high - min(high, (1ull << shift) - 1));
        left = 0;
        for (int e = tid; e < n + tid; e += kSmThreads) left += __syncthreads_count(e < n && s.w[e] >= low && s.w[e] <= high);
      }
      if (high != low) {                          // few: each against each
        if (tid == 0) s.n = 0;
        __syncthreads();
        for (int e = tid; e < n; e += kSmThreads)
          if (s.w[e] >= low && s.w[e] <= high) s.mass[atomicAdd(&s.n, 1u)] = s.w[e];
        __syncthreads();
        const u64 c = tid < left ? s.mass[tid] : 0, w = tid < left ? weigh(c) : 0;
        s.w[tid] = w;
        __syncthreads();
        u64 above = 0;
#pragma unroll 4
        for (int q = 0; q < left; ++q)
          if (s.mass[q] > c) above += s.w[q];
        if (above < need && need <= above + w) s.total = c;
        __syncthreads();
        high = s.total;
      }
      if (tid == 0)
        for (unsigned r = 0; r < t.size; ++r) peer_st64(peer(&s.top, r), high);
    }
    t.sync();
    found = s.top;
  };
  const u64 highest = order(sm_key(t.sc.M), 0);
  u64 floor = order(T0, 0xfffff);
  if (k > 0) border(highest, floor, (u64)k, false, -1.0f, floor);
  if (p < 1.0f) {
    u64 found;
    border(highest, floor, 0, true, p, found);    // (of what top-k left, or with the tail of all)
    floor = found;
  }
  return SampleCut{SampleOrder::key(floor), SampleOrder::column(floor)};
}

// ---------------------------------------------------------------- the kernel --
template <typename T>
__global__ void __launch_bounds__(kSmThreads, 4) sample_kernel(const __grid_constant__ SampleArgs a) {
  __shared__ SampleSmem s;
  constexpr int VE = SampleRow<T>::VE;
  const unsigned rank = cluster_rank(), size = cluster_size();
  const int r = (int)(blockIdx.x / size);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_wait();
  griddep_launch_dependents();
  const float tau = a.temps ? __ldg(a.temps + r) : a.temp;
  int k = a.top_ks ? __ldg(a.top_ks + r) : a.top_k;
  float p = a.top_ps ? __ldg(a.top_ps + r) : a.top_p;
  float mp = a.min_ps ? __ldg(a.min_ps + r) : a.min_p;
  const float u = __ldg(a.u + r);
  const bool greedy = !(tau > 0.0f);
  if (k <= 0 || k >= a.N) k = 0;
  p = p < 1.0f ? fmaxf(p, 0.0f) : 1.0f;         // (NaN: none)
  if (!(mp > 0.0f)) mp = 0.0f;
  if (mp > 1.0f) {                                // the first alone
    k = a.N > 1 ? 1 : 0;
    mp = 0.0f;
  }
  if (greedy) {
    k = 0;
    p = 1.0f;
    mp = 0.0f;
  }
  const bool sums = p < 1.0f && k == 0;

  SampleCta<T> t{s, SampleRow<T>(static_cast<const T *>(a.logits) + (long long)r * a.row_stride, a.N), tid, warp, lane, rank, size};
  const int per = (t.row.nvec + (int)size - 1) / (int)size;
  t.v0 = min((int)rank * per, t.row.nvec);
  t.v1 = min(t.v0 + per, t.row.nvec);
  // log2(e) / t in two terms: the quotient, and its remainder divided
  constexpr float E = 1.44269504f, Elo = (float)(1.4426950408889634074 - (double)E);
  t.sc.chi = fminf(__fdiv_rn(E, tau), 3.0e38f);
  t.sc.clo = __fdiv_rn(fmaf(-t.sc.chi, tau, E) + Elo, tau);
  if (greedy || !(fabsf(t.sc.clo) <= 1e-6f * t.sc.chi)) t.sc.clo = 0.0f;
  const float c = t.sc.chi, clo = t.sc.clo;
  // e^(d / t) for the sums of what lies below top-p's bound; the low term takes away an error that all would
  // share (7e-7 of them at 2^-18 and t = 1.1).  The pass goes without: what counts in a block lies a few octaves
  // below its largest, where it is 2e-7 (with it 768 x 50257 take 46.8 us, so 42.4).
  // (The distance of finite logits can be infinite too.)
  auto power = [&](float d) { return sm_ex2(fmaf(d, c, fmaxf(d, -3.0e38f) * clo)); };

  // ---- 1. blocks: U vectors of a thread, kSmThreads apart
  constexpr int U0 = 32 / VE;
  const int vecs = (t.v1 - t.v0 + kSmThreads - 1) / kSmThreads;
  int U = U0, logU = U0 == 4 ? 2 : 3;
  while (U * kSmBlocks < vecs) {
    U *= 2;
    ++logU;
  }
  const int nblk = (vecs + U - 1) / U;
  if (tid == 0) {
    s.n = s.nwork = 0;
    s.gidx = 0xffffffffu;
  }
  float top = -INFINITY;
  for (int b = 0; b < nblk; ++b) {
    const int first = t.v0 + b * U * kSmThreads + tid;
    float bm = -INFINITY, bs = 0.0f;
    for (int g = 0; g < U && first + g * kSmThreads < t.v1; g += U0) {
      uint4 raw[U0];
#pragma unroll
      for (int i = 0; i < U0; ++i) {
        const int v = first + (g + i) * kSmThreads;
        raw[i] = v < t.v1 ? t.row.load(v) : t.row.nothing();
      }
      uint32_t m = raw[0].x;
#pragma unroll
      for (int i = 0; i < U0; ++i) m = t.row.max2(m, t.row.max2(t.row.max2(raw[i].x, raw[i].y), t.row.max2(raw[i].z, raw[i].w)));
      const float gm = t.row.max_of(m);
      if (sums) {
        const float nm = fmaxf(bm, gm), ref = nm == -INFINITY ? 0.0f : nm;
        float sum = 0.0f, sum1 = 0.0f;
#pragma unroll
        for (int i = 0; i < U0; ++i) {
          float x[VE];
          t.row.floats(raw[i], x);
#pragma unroll
          for (int e = 0; e < VE; e += 2) {
            const F2 d = add2(F2(x[e], x[e + 1]), F2(-ref, -ref));
            float y0, y1;
            mul2(d, F2(c, c)).get(y0, y1);
            sum += sm_ex2(y0);
            sum1 += sm_ex2(y1);
          }
        }
        sum += sum1;
        if (!(sum < INFINITY)) {                  // NaN logits, or infinite ones
          sum = 0.0f;
#pragma unroll
          for (int i = 0; i < U0; ++i) {
            float x[VE];
            t.row.floats(raw[i], x);
#pragma unroll
            for (int e = 0; e < VE; ++e) sum += x[e] == ref ? 1.0f : x[e] > -INFINITY ? power(x[e] - ref) : 0.0f;
          }
        }
        bs = (bs == 0.0f ? 0.0f : bm == nm ? bs : bs * power(bm - nm)) + sum;
        bm = nm;
      } else {
        bm = fmaxf(bm, gm);
      }
    }
    s.bmax[b][tid] = bm;
    if (sums) s.bsum[b][tid] = bs;
    top = fmaxf(top, bm);
  }
  // ---- 2. the row's largest logit, sum and bound
  const float mine = top;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) s.red[warp] = top;
  if (k > 0) {
    // the j-th largest of the CTA's thread maxima, or for many of its block maxima, to 16 bits: by
    // halving
    const int j = (k + (int)size - 1) / (int)size;
    unsigned bound = 0;
    if (j <= kSmThreads / 2) {
      const unsigned key = sm_key(mine);
#pragma unroll 1
      for (unsigned bit = 0x80000000u; bit >= 0x10000u; bit >>= 1)
        if (__syncthreads_count(key >= (bound | bit)) >= j) bound |= bit;
    } else if (j <= kSmThreads * nblk) {
      unsigned key[kSmBlocks];
#pragma unroll
      for (int b = 0; b < kSmBlocks; ++b) key[b] = b < nblk ? sm_key(s.bmax[b][tid]) : 0u;
      int round = 0;
#pragma unroll 1
      for (unsigned bit = 0x80000000u; bit >= 0x10000u; bit >>= 1, round ^= 1) {
        int n = 0;
#pragma unroll
        for (int b = 0; b < kSmBlocks; ++b) n += key[b] >= (bound | bit);
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) s.nkey[round][warp] = n;
        __syncthreads();
        n = 0;
#pragma unroll
        for (int w = 0; w < kSmWarps; ++w) n += s.nkey[round][w];
        if (n >= j) bound |= bit;
      }
    }
    if (tid == 0) s.xkey = bound;
  }
  __syncthreads();
  float cm = s.red[0];
#pragma unroll
  for (int w = 1; w < kSmWarps; ++w) cm = fmaxf(cm, s.red[w]);
  auto rel = [&](float bm, float bs, float M) { return bs == 0.0f ? 0.0f : bm == M ? bs : bs * power(bm - M); };
  if (sums) {
    float sum = 0.0f;
    for (int b = 0; b < nblk; ++b) sum += rel(s.bmax[b][tid], s.bsum[b][tid], cm);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncthreads();
    if (lane == 0) s.red[warp] = sum;
    __syncthreads();
  }
  if (tid == 0) {
    float sum = 0.0f;
    if (sums)
      for (int w = 0; w < kSmWarps; ++w) sum += s.red[w];
    s.xmax = cm;
    s.xsum = sum;
  }
  t.sync();
  if (warp == 0) {
    float m = -INFINITY, sum = 0.0f;
    unsigned key = 0xffffffffu;
    if (lane < (int)size) {
      m = __uint_as_float(peer_ld32(peer(&s.xmax, lane)));
      sum = __uint_as_float(peer_ld32(peer(&s.xsum, lane)));
      key = peer_ld32(peer(&s.xkey, lane));
    }
    float M = m;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    sum = rel(m, sum, M);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
      key = min(key, __shfl_xor_sync(0xffffffffu, key, o));
    }
    if (lane == 0) {
      s.rowmax = M;
      s.rowsum = sum;
      s.rowkey = key;
    }
  }
  __syncthreads();
  t.sc.M = s.rowmax;
  const float M = t.sc.M;
  if (M == -INFINITY) {                           // nothing to draw from
    if (rank == 0 && tid == 0) {
      a.token[r] = -1;
      if (a.logprob) a.logprob[r] = -INFINITY;
    }
    t.sync();
    return;
  }
  // (2^-100 of the largest, if the type and the temperature have such a value; else as with filters)
  t.lowest = t.row.packed(M - 100.0f / c);
  const float low = t.row.max_of(t.lowest), far = (M - low) * c;
  if (!greedy && k == 0 && p == 1.0f && mp == 0.0f && low > -INFINITY && far > 60.0f && far < 1e4f) {
    sample_draw<T, true>(a, t, r, SampleCut{0u, 0x7fffffff}, 0.0f, u);
    t.sync();                                     // (its sums have been read)
    return;
  }
  // the bound, as an order key; a little lower where it is computed
  unsigned T0 = k > 0 ? s.rowkey : 0u;
  auto below = [&](float z) {                     // the key of M + z t ln 2, z <= 0
    const float d = z / c;
    return sm_key(M + d - (fabsf(d) * 1e-4f + fabsf(M) * 1e-6f));
  };
  if (sums) {
    const float most = (1.0f - p) * s.rowsum * 0.99f;             // what may be left out
    float z = fminf(sm_lg2(most / (float)a.N), 0.0f);
    {
      // Higher, from the blocks: with a bound of 2^z those below it leave out their sums and each
      // other at most 31 elements of weight 2^z.  Tried: sixteenths of the way, four at a time.
      const float step = -z * (1.0f / 16.0f), each = (float)(U * VE - 1);
      int lo = 16;
      for (int round = 0; round < 2; ++round) {
        const int at = round == 0 ? 4 : 1, from = round == 0 ? 0 : lo - 4;     // tried: from + at, from + 2 at, ..
        float sum[3] = {}, zt[3], wt[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          zt[i] = -step * (float)(from + at * (i + 1));
          wt[i] = each * sm_ex2(zt[i]);
        }
        for (int b = 0; b < nblk; ++b) {
          const float bm = s.bmax[b][tid], y = bm == M ? 0.0f : (bm - M) * c, bs = rel(bm, s.bsum[b][tid], M);
#pragma unroll
          for (int i = 0; i < 3; ++i) sum[i] += y < zt[i] ? bs : fminf(bs, wt[i]);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 3; ++i) {
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
          if (lane == 0) s.rsum3[i][warp] = sum[i];
        }
        __syncthreads();
        if (size > 1) {
          if (tid < 3) {
            float total = 0.0f;
            for (int w = 0; w < kSmWarps; ++w) total += s.rsum3[tid][w];
            s.xsum3[round][tid] = total;
          }
          t.sync();
        }
        int best = from + 4 * at;
#pragma unroll
        for (int i = 2; i >= 0; --i) {
          float total = 0.0f;
          if (size > 1)
            for (unsigned q = 0; q < size; ++q) total += __uint_as_float(peer_ld32(peer(&s.xsum3[round][i], q)));
          else
            for (int w = 0; w < kSmWarps; ++w) total += s.rsum3[i][w];
          if (total <= most) best = from + at * (i + 1);
        }
        lo = best;
      }
      z = -step * (float)lo;
    }
    T0 = max(T0, below(z - 0.01f));
  }
  if (mp > 0.0f && !(k > 0 && p < 1.0f)) T0 = max(T0, below(mp < 1.0f ? sm_lg2(mp) - 0.01f : 0.0f));
  if (greedy) T0 = sm_key(M);
  T0 = max(T0, 0x00800000u);                      // (the key of the lowest finite value: not -inf, not NaN)
  if (M == INFINITY) T0 = sm_key(M);              // (weights of 0 beside it)

  // ---- 3. the list
  u64 tail = 0;
  const bool counts = sums && M < INFINITY;       // (beside infinite logits the others weigh nothing)
  auto fixed = [&](float x) { return __float2ull_rn(x * (float)(1ull << kSmFix)); };
  for (int b = 0; b < nblk; ++b) {
    const float bm = s.bmax[b][tid];
    const bool hit = sm_key(bm) >= T0;
    const unsigned v = __ballot_sync(0xffffffffu, hit);
    int at = 0;
    if (v && lane == 0) at = atomicAdd(&s.nwork, __popc(v));
    at = __shfl_sync(0xffffffffu, at, 0);
    if (hit) s.work[at + __popc(v & ((1u << lane) - 1u))] = (unsigned short)(b * kSmThreads + tid);
    else if (counts) tail += fixed(rel(bm, s.bsum[b][tid], M));
  }
  __syncthreads();
  const uint32_t lead_g = peer(&s.gidx, 0);
  const int items = s.nwork * U;
  auto item = [&](int i) {                        // vector of work item i (t.v1: none)
    if (i >= items) return t.v1;
    const int id = s.work[i >> logU];
    return min(t.v0 + ((id / kSmThreads) * U + (i & (U - 1))) * kSmThreads + id % kSmThreads, t.v1);
  };
  // (the next vector is loaded while one is looked through)
  int vn = item(tid);
  uint4 next = vn < t.v1 ? t.row.load(vn) : t.row.nothing();
  for (int i = tid; i < items; i += kSmThreads) {
    const int v = vn;
    const uint4 raw = next;
    vn = item(i + kSmThreads);
    next = vn < t.v1 ? t.row.load(vn) : t.row.nothing();
    if (v >= t.v1) continue;
    float x[VE];
    t.row.floats(raw, x);
    unsigned hits = 0;
    float rest = 0.0f;
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      if (sm_key(x[e]) >= T0) hits |= 1u << e;
      else if (counts && x[e] > -INFINITY) rest += power(x[e] - M);
    }
    if (sums) tail += fixed(rest);
    if (hits) {
      const int col = t.row.col(v);               // (places outside the row are -inf)
      if (greedy) {
        peer_min(lead_g, (unsigned)(col + __ffs(hits) - 1));
      } else {
        // (a list that is full already is left alone: thousands would queue for its number)
        unsigned at = *static_cast<volatile unsigned *>(&s.n) > kSmList ? kSmList : atomicAdd(&s.n, __popc(hits));
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          if ((hits >> e & 1) && at < kSmList) s.key[at] = (u64)sm_key(x[e]) << 32 | (unsigned)~(col + e);
          at += hits >> e & 1;
        }
      }
    }
  }
  if (sums) {
    tail = SampleCta<T>::reduce(tail);
    if (lane == 0) s.rsum[warp] = tail;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kSmWarps; ++w) tail += s.rsum[w];
      peer_st64(peer(&s.tail[rank], 0), tail);
    }
  }
  t.sync();
  if (greedy) {
    if (rank == 0 && tid == 0) {
      a.token[r] = (int)s.gidx;
      if (a.logprob) a.logprob[r] = 0.0f;
    }
    return;                                       // (nobody reads another CTA's memory any more)
  }
  bool full;
  const unsigned n = t.join_lists(s.key, kSmShort, full);
  if (n <= kSmShort) {
    if (rank == 0) sample_list<T>(a, t, r, (int)n, k, p, mp, u, T0);
    return;
  }
  // ---- flat rows
  u64 rest = 0;
  if (sums)
    for (unsigned q = 0; q < size; ++q) rest += peer_ld64(peer(&s.tail[q], 0));
  const SampleOrder order(t.sc, T0);
  if (!full) {                                    // every CTA's list holds its elements
    const int own = (int)s.n;
    const SampleCut cut = sample_flat<T>(t, order, k, p, rest, T0, [&](auto f) {
      for (int e = tid; e < own; e += kSmThreads) {
        const unsigned key = (unsigned)(s.key[e] >> 32);
        f(order(key, (int)~(unsigned)s.key[e]), sm_value(key));
      }
    });
    sample_draw_listed<T>(a, t, r, own, cut, mp, u);
    t.sync();
    return;
  }
  const SampleCut cut = sample_flat<T>(t, order, k, p, rest, T0, [&](auto f) {
    auto at = [&](int i) {
      const int id = s.work[i >> logU];
      return t.v0 + ((id / kSmThreads) * U + (i & (U - 1))) * kSmThreads + id % kSmThreads;
    };
    for (int i = tid; i < items; i += 4 * kSmThreads) {
      uint4 raw[4];
      int v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[q] = i + q * kSmThreads < items ? at(i + q * kSmThreads) : t.v1;
        raw[q] = v[q] < t.v1 ? t.row.load(v[q]) : t.row.nothing();
      }
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        float x[VE];
        t.row.floats(raw[0], x);
        const int col = t.row.col(v[0]);
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const unsigned key = sm_key(x[e]);
          if (key >= T0) f(order(key, col + e), x[e]);
        }
#pragma unroll
        for (int z = 0; z < 3; ++z) {
          raw[z] = raw[z + 1];
          v[z] = v[z + 1];
        }
      }
    }
  });
  sample_draw<T, false>(a, t, r, cut, mp, u);
  t.sync();
}

namespace {
int bad(int code, const char *fmt, ...) {
  char msg[400];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof msg, fmt, ap);
  va_end(ap);
  return set_last_error(code, msg);
}
bool at(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }
}  // namespace
}  // namespace qw

using namespace qw;

extern "C" int sample_tokens(const void *logits, int dtype, int M, int N, long long row_stride, const float *u,
                             const qw_sampling_t *set, int32_t *token, float *logprob, qw_stream_t stream) {
  if (M < 0 || row_stride < 0) return bad(QW_ERR_INVALID_ARG, "negative size");
  if (dtype != QW_F16 && dtype != QW_BF16 && dtype != QW_F32) return bad(QW_ERR_INVALID_ARG, "logit type %d", dtype);
  if (N < 1 || N > (1 << 20)) return bad(QW_ERR_UNSUPPORTED_SHAPE, "1 <= N <= 2^20 (N=%d)", N);
  if (!set) return bad(QW_ERR_INVALID_ARG, "null settings");
  if (M == 0) return QW_OK;
  if (!logits || !u || !token) return bad(QW_ERR_INVALID_ARG, "null tensor pointer");
  if (!at(logits, dtype == QW_F32 ? 4 : 2) || !at(u, 4) || !at(token, 4) || !at(logprob, 4) || !at(set->temperatures, 4) ||
      !at(set->top_ps, 4) || !at(set->min_ps, 4) || !at(set->top_ks, 4))
    return bad(QW_ERR_ALIGNMENT, "arrays must be aligned to their elements");
  int sms = 0, rc = device_info(&sms, nullptr);
  if (rc) return rc;
  SampleArgs a{logits,           u,          set->temperatures, set->top_ps, set->min_ps, set->top_ks, set->temperature,
               set->top_p,       set->min_p, set->top_k,        row_stride,  M,           N,           token,
               logprob};
  int cluster = 1;
  // CTAs a row: the waves of CTAs (four an SM) times a CTA's elements, a row's steps counted as
  // 32768.  16 have to fit one part of the GPU; a CTA's part has below 2^18 elements.  (us with 1, 2, 4, 8 and 16
  // CTAs: 1 x 248320 31.5, 21.1, 16.0, 13.4, 12.9*; 16 x 128257 fp32 33.3, 21.6, 16.7, 14.6*; 64 x 128257 40.7, 26.4,
  // 21.3, 22.7*; 128 x 50257 16.2, 16.4, 18.4*, 32.1; 300 x 50257 21.2, 23.2*, 42.1; 768 x 50257 42.3*, 58.9;
  // *: the rule's.  Rows of a few thousand would do with fewer: 1 x 4096 8.5 us with one, 14.4 with the rule's 16.)
  long long best = 0;
  for (int c = 1; c <= ((long long)M * kSmMaxCluster <= sms / 2 ? kSmMaxCluster : 8); c *= 2) {
    const long long cost = ((long long)M * c + 4 * sms - 1) / (4 * sms) * (N / c + 32768);
    if (N / c < (1 << 18) - 16 && (best == 0 || cost < best)) {
      best = cost;
      cluster = c;
    }
  }
  if ((long long)M * cluster > 0x7fffffffll) return bad(QW_ERR_UNSUPPORTED_SHAPE, "too many rows");
  const void *f = dtype == QW_F16    ? reinterpret_cast<const void *>(sample_kernel<__half>)
                  : dtype == QW_BF16 ? reinterpret_cast<const void *>(sample_kernel<__nv_bfloat16>)
                                     : reinterpret_cast<const void *>(sample_kernel<float>);
  if (cluster > 8) {                              // (once a kernel and device)
    static std::atomic<unsigned long long> allowed[3];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && !(allowed[dtype].load(std::memory_order_relaxed) >> (dev & 63) & 1)) {
      e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e == cudaSuccess && dev < 64) allowed[dtype].fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    if (e != cudaSuccess) return bad(QW_ERR_CUDA, "cluster size: %s", cudaGetErrorString(e));
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(M * cluster));
  cfg.blockDim = dim3(kSmThreads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  void *argv[] = {&a};
  cudaError_t e = cudaLaunchKernelExC(&cfg, f, argv);
  count_launch();
  if (e != cudaSuccess) return bad(QW_ERR_CUDA, "sampling kernel launch: %s", cudaGetErrorString(e));
  return QW_OK;
}
