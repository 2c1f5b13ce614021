// token_logprobs.cu -- log probabilities of given tokens, entropy and the k most likely
// tokens of each row of a logit matrix, in one pass over the logits.
//
// With y_j = (x_j - r) log2(e) for a reference r near the row's largest x:
//   s = sum 2^y_j,  t = sum y_j 2^y_j
//   logsumexp = r + log2 s ln 2        log p_j = (x_j - r) - log2 s ln 2
//   entropy   = (log2 s - t / s) ln 2  (both terms are >= 0 up to rounding: no cancellation)
// The difference is taken first: x log2(e) - r log2(e) in one step saves an operation a pair, but
// then the rounding of r log2(e) moves every y by up to |r| 2^-24, and far from zero (a whole
// row masked with -1e30 or the type's lowest value) that is more than the exponents hold.
// A thread keeps (r, s, t) while it streams its 16-byte vectors; all sums in binary32, joined
// in a fixed order.
//
// The k most likely come from the same pass.  Each warp's j-th largest thread maximum, j =
// ceil(k / warps), is passed by j threads of that warp, so the smallest of these, T, is a lower
// bound of the k-th largest element: the blocks of vectors whose maximum (kept in shared
// memory) reaches T are read again (from L2), and their elements from T on listed as
// (value, column) composites -- distinct, ties ordered by column.  A list that overflows
// (many equal logits) gives a higher bound, the k-th largest of what it holds, and is filled
// again.
//
// Five CTAs of 128 threads an SM.  The vectors of all rows, laid end to end with a few places
// more for what a row costs by itself, are cut into one equal range a CTA, so the SMs finish
// together whatever the numbers of rows and columns; the last CTA to finish a cut row joins
// its parts' sums and selects among their lists the same way.  Each block of four vectors a
// thread is loaded while the one before is summed, across row borders too.
//
// What bounds it: the read of the logits (HBM); close to it the instructions, about ten a 16-bit
// element with everything counted (pairs go through two-wide binary32 operations), and some 500
// a warp and row; for few rows the launch and two chains of block-wide steps (the part's sums
// and list, then the join's).
//
// Measured: 2048 rows of 50257 bf16 (206 MB), no alternatives: 41.9 us, 4.9 TB/s; 64 of 128257
// binary32 with 20 alternatives: 17.2 us, 1.9 TB/s; one of 248320 fp16 with 20: 12.2 us.
#include <float.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "launch.h"
#include "ptx.cuh"
#include "qgemm.h"

namespace qw {

constexpr int kLpThreads = 128;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpPerSm = 5;                       // CTAs an SM (up to 96 registers a thread)
constexpr int kLpMaxK = 64;
constexpr int kLpLogUnroll = 2, kLpUnroll = 1 << kLpLogUnroll;      // vectors of a block a thread
constexpr int kLpBlock = kLpUnroll * kLpThreads;  // vectors of a block
constexpr int kLpMaxima = 16;                     // block maxima a thread keeps (of 2^g blocks for long rows)
constexpr int kLpBlocks = 256;                    // listed blocks of threads
constexpr int kLpList = 512;                      // listed elements
constexpr int kLpMinBlocks = 2;                   // blocks of vectors a CTA takes at least
constexpr int kLpRowCost = 256;                   // places of a row beside its vectors

struct LpArgs {
  const void *logits;
  const void *tokens;                             // [M][C] int32 or int64
  long long row_stride;                           // elements
  int M, N, C, k, tok64;
  int nv;                                         // vectors of a row, whatever its alignment
  long long share;                                // places a CTA
  int S, step;                                    // or, S > 0: CTAs a row and vectors of each
  float *logprob, *entropy, *lse, *top_lp;
  int *top_idx;
  float *part;                                    // [CTAs][2][4]: r, s, t of a cut row's part
  unsigned long long *cand;                       // [CTAs][2][k]
  int *counters;                                  // [CTAs], zero between calls
  int *err;
};

struct LpSmem {
  float red[3][kLpWarps];
  unsigned wkey[kLpWarps];
  unsigned long long list[kLpList];
  unsigned long long sel[kLpMaxK];
  unsigned long long T;
  int block[kLpBlocks];
  int n, nblock, first, parts;
};

__device__ __forceinline__ float lp_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// max that gives NaN when an operand is NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
// binary32 values as unsigned integers in the values' order; -0 as +0; NaN below every number
// (a maximum leaves NaN out, so what it bounds must not lie above it); no value gives 0
__device__ __forceinline__ unsigned order_key32(float x) {
  const unsigned u = __float_as_uint(x + 0.0f);
  return x == x ? u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u) : 1u;
}
__device__ __forceinline__ float key_value32(unsigned k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

template <typename T>
struct LpTwo {
  using type = __half2;
};
template <>
struct LpTwo<__nv_bfloat16> {
  using type = __nv_bfloat162;
};
template <typename T>
struct LpVec {
  static constexpr int VE = 16 / sizeof(T);
};
template <typename T>
__device__ __forceinline__ float lp_float(T x);
template <>
__device__ __forceinline__ float lp_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ float lp_float<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float lp_float<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

// A row as 16-byte vectors: vector v holds columns v VE - pad .. v VE - pad + VE - 1, where
// pad is how many elements the row starts past a 16-byte boundary.  Only the first and last
// vectors can reach past the row; their elements are read one by one.
template <typename T>
struct LpRow {
  static constexpr int VE = LpVec<T>::VE;
  static constexpr bool kBf = sizeof(T) == 2 && !__is_same(T, __half);
  const T *row;
  int pad, N, nvec, in0, in1;                     // whole vectors: [in0, in1)
  __device__ __forceinline__ LpRow(const T *r, int n) : row(r), N(n) {
    pad = (int)((reinterpret_cast<uintptr_t>(r) / sizeof(T)) % VE);
    nvec = (int)(((long long)n + pad + VE - 1) / VE);
    in0 = pad > 0 ? 1 : 0;
    in1 = max((int)(((long long)n + pad) / VE), in0);
  }
  __device__ __forceinline__ int col(int v) const { return v * VE - pad; }
  __device__ __forceinline__ uint4 raw(int v) const { return __ldg(reinterpret_cast<const uint4 *>(row + col(v))); }
};
template <typename T>
__device__ __forceinline__ void lp_unpack(const uint4 &w, float (&x)[LpVec<T>::VE]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      x[i] = __uint_as_float(u[i]);
    } else if constexpr (LpRow<T>::kBf) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    } else {
      const float2 f = __half22float2(u32_as_h2(u[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}
// The largest element of a vector (16-bit types: two at a time; NaN only where all are).
template <typename T>
__device__ __forceinline__ float lp_max(const uint4 &w) {
  if constexpr (sizeof(T) == 4) {
    return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
  } else {
    using T2 = typename LpTwo<T>::type;
    const T2 *e = reinterpret_cast<const T2 *>(&w);
    const T2 hi = __hmax2(__hmax2(e[0], e[1]), __hmax2(e[2], e[3]));
    return fmaxf(lp_float(hi.x), lp_float(hi.y));
  }
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNoRef = -3.402823466e38f;        // the reference of a sum of nothing: the lowest finite logit

struct LpSum {
  float r, s, t;
};
// two binary32 values in a register pair
__device__ __forceinline__ unsigned long long pair2(float a, float b) {
  unsigned long long d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float2 both2(unsigned long long a) {
  float2 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(a));
  return v;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// y moved from reference a to b: far below the exponents' range nothing is left, and no
// infinity may meet a zero (a reference +inf leaves NaN: its own sum is one)
__device__ __forceinline__ float lp_shift(float a, float b) { return fmaxf((a - b) * kLog2e, -1000.0f); }
__device__ __forceinline__ void lp_move(LpSum &a, float r) {       // to the reference r
  const float d = lp_shift(a.r, r), f = lp_ex2(d);
  a.t = a.s == 0.0f ? 0.0f : (a.t + d * a.s) * f;
  a.s *= f;
  a.r = r;
}
__device__ __forceinline__ LpSum lp_join(LpSum a, LpSum b) {
  const float r = fmaxf(a.r, b.r);
  lp_move(a, r);
  lp_move(b, r);
  return LpSum{r, a.s + b.s, a.t + b.t};
}
// to the largest reference among 2^n lanes, then plain sums (xor shuffles: a fixed order)
template <int LANES>
__device__ __forceinline__ LpSum lp_lanes(LpSum a) {
  float r = a.r;
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, o));
  lp_move(a, r);
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) {
    a.s += __shfl_xor_sync(0xffffffffu, a.s, o);
    a.t += __shfl_xor_sync(0xffffffffu, a.t, o);
  }
  return a;
}
// over the CTA; valid in every thread
__device__ __forceinline__ LpSum lp_block(LpSum a, LpSmem &sm) {
  a = lp_lanes<32>(a);
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
    sm.red[0][w] = a.r;
    sm.red[1][w] = a.s;
    sm.red[2][w] = a.t;
  }
  __syncthreads();
  return lp_lanes<kLpWarps>(LpSum{sm.red[0][lane % kLpWarps], sm.red[1][lane % kLpWarps], sm.red[2][lane % kLpWarps]});
}

// A lower bound of the k-th largest of the elements whose largest each thread holds in
// `key` (0: none), from the first `warps` warps, all of whose lanes hold one.
__device__ __forceinline__ unsigned lp_bound(unsigned key, int warps, int k, LpSmem &sm) {
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int j = warps > 0 ? (k + warps - 1) / warps : 33;
  unsigned best = 0u;
  if (w < warps && j <= 32)
    for (int i = 0; i < j; ++i) {                 // the warp's largest, one lane at a time
      best = __reduce_max_sync(0xffffffffu, key);
      if (lane == __ffs(__ballot_sync(0xffffffffu, key == best)) - 1) key = 0u;
    }
  if (lane == 0) sm.wkey[w] = best;
  __syncthreads();
  unsigned T = 0u;
  if (j <= 32) {
    T = 0xffffffffu;
#pragma unroll
    for (int i = 0; i < kLpWarps; ++i)
      if (i < warps) T = min(T, sm.wkey[i]);
  }
  return T;
}
// sm.T = the k-th largest of the (distinct) elements of a full list.
__device__ __forceinline__ void lp_raise(int k, LpSmem &sm) {
#pragma unroll 1
  for (int i = threadIdx.x; i < kLpList; i += kLpThreads) {
    const unsigned long long mine = sm.list[i];
    int above = 0;
#pragma unroll 8
    for (int j = 0; j < kLpList; ++j) above += sm.list[j] > mine;
    if (above == k - 1) sm.T = mine;
  }
  __syncthreads();
}
// Lists the elements from T on that `visit(T, put)` puts -- every thread its own --, raising T
// while they do not fit, and writes the k largest, largest first, to sm.sel (0 past the last).
template <typename F>
__device__ __forceinline__ void lp_select(unsigned long long T, int k, LpSmem &sm, const F &visit) {
  if ((int)threadIdx.x < k) sm.sel[threadIdx.x] = 0ull;
  if (threadIdx.x == 0) sm.n = 0;
  __syncthreads();
#pragma unroll 1
  for (;;) {
    visit(T, [&](unsigned long long p) {
      const int at = atomicAdd(&sm.n, 1);
      if (at < kLpList) sm.list[at] = p;
    });
    __syncthreads();
    if (sm.n <= kLpList) break;
    lp_raise(k, sm);
    T = sm.T;
    if (threadIdx.x == 0) sm.n = 0;
    __syncthreads();
  }
  const int n = sm.n;
  // rank: eight threads an element
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += kLpThreads / 8) {
    const int i = i0 + (int)threadIdx.x / 8;
    const unsigned long long mine = i < n ? sm.list[i] : 0ull;
    int above = 0;
    if (i < n)
#pragma unroll 4
      for (int j = threadIdx.x % 8; j < n; j += 8) above += sm.list[j] > mine;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) above += __shfl_xor_sync(0xffffffffu, above, o);
    if (i < n && threadIdx.x % 8 == 0 && above < k) sm.sel[above] = mine;
  }
  __syncthreads();
}
__device__ __forceinline__ unsigned long long lp_pair(unsigned key, int col) {
  return ((unsigned long long)key << 32) | (0xffffffffu - (unsigned)col);
}

__device__ __forceinline__ long long lp_token_id(const LpArgs &a, int m, int c) {
  const long long i = (long long)m * a.C + c;
  return a.tok64 ? __ldg(reinterpret_cast<const long long *>(a.tokens) + i) : __ldg(reinterpret_cast<const int *>(a.tokens) + i);
}
// The logit of the row's given token c; NaN when there is no such token.
template <typename T>
__device__ __forceinline__ float lp_token(const LpArgs &a, int m, const T *row, int c) {
  const long long tok = lp_token_id(a, m, c);
  if (tok >= 0 && tok < a.N) return lp_float(row[tok]);
  atomicCAS(a.err, 0, -9);
  return __uint_as_float(0x7fc00000u);
}
// The row's results from its sums and (k > 0) its k best pairs in sm.sel; xtok: token
// threadIdx.x's logit, where `given`.
template <typename T>
__device__ __forceinline__ void lp_write(const LpArgs &a, int m, const T *row, const LpSum &z, const LpSmem &sm, bool given,
                                         float xtok) {
  const float ls = log2f(z.s);
  const bool none = z.s == 0.0f;                  // every logit -inf
  if (threadIdx.x == 0) {
    a.lse[m] = none ? -INFINITY : fmaf(ls, kLn2, z.r);
    a.entropy[m] = none ? 0.0f : fmaxf(ls - z.t / z.s, z.s != z.s ? z.s : 0.0f) * kLn2;
  }
  // (a token that does not exist stays NaN)
  auto lp = [&](float x) { return none ? (x != x ? x : -INFINITY) : fmaf(-ls, kLn2, x - z.r); };
#pragma unroll 1
  for (int c = threadIdx.x; c < a.C; c += kLpThreads)
    a.logprob[(long long)m * a.C + c] = lp(given && c == (int)threadIdx.x ? xtok : lp_token<T>(a, m, row, c));
#pragma unroll 1
  for (int i = threadIdx.x; i < a.k; i += kLpThreads) {
    const unsigned long long p = sm.sel[i];
    a.top_lp[(long long)m * a.k + i] = lp(key_value32((unsigned)(p >> 32)));
    a.top_idx[(long long)m * a.k + i] = (int)(0xffffffffu - (unsigned)p);
  }
}

// TOP: the k most likely are wanted too
template <typename T, bool TOP>
__global__ void __launch_bounds__(kLpThreads, kLpPerSm) token_logprobs_kernel(const __grid_constant__ LpArgs a) {
  constexpr int VE = LpVec<T>::VE;
  __shared__ LpSmem sm;
  __shared__ float maxima[TOP ? kLpMaxima * kLpThreads : 1];
  const int tid = threadIdx.x, me = blockIdx.x, nv = a.nv;
  const long long span = nv + kLpRowCost;
  long long begin = a.share * me, end = min(begin + a.share, span * a.M);
  if (a.S > 0) {
    const int r = me / a.S, u = (me - r * a.S) * a.step;
    begin = r * span + kLpRowCost + u;
    end = begin + min(a.step, nv - u);
  }
  griddep_wait();
  griddep_launch_dependents();

  // ---- the copies, a block of vectors ahead of the sums: row lm (its places from lat)
  int lm = a.S > 0 ? me / a.S : (int)(begin / span);
  long long lat = lm * span;
  const int m0 = lm;
  const uint8_t *lsrc = nullptr;                  // the row's 16-byte boundary
  int lv = 0, lend = 0;
  auto open = [&]() {                             // the whole vectors of the row that lie in the range
    const LpRow<T> R(static_cast<const T *>(a.logits) + (long long)lm * a.row_stride, a.N);
    lsrc = reinterpret_cast<const uint8_t *>(R.row) - R.pad * (int)sizeof(T);
    lv = max((int)max(begin - lat - kLpRowCost, 0ll), R.in0);
    lend = min((int)min(end - lat - kLpRowCost, (long long)nv), R.in1);
  };
  open();
  auto fetch = [&](uint4 (&w)[kLpUnroll]) {
    while (lv >= lend) {
      lat += span;
      if (lat + kLpRowCost >= end) return;
      ++lm;
      open();
    }
    const uint4 *src = reinterpret_cast<const uint4 *>(lsrc) + lv + tid;
#pragma unroll
    for (int i = 0; i < kLpUnroll; ++i)
      if (lv + tid + i * kLpThreads < lend) w[i] = __ldg(src + i * kLpThreads);
    lv += kLpBlock;
    if (lv > lend) lv = lend;
  };
  uint4 w[kLpUnroll];
  fetch(w);

  long long at = m0 * span;
  int m = m0;
  long long tok = -1;
  if (tid < a.C) tok = lp_token_id(a, m, tid);
#pragma unroll 1
  for (; at + kLpRowCost < end; ++m, at += span) {
    const int u0 = (int)max(begin - at - kLpRowCost, 0ll), u1 = (int)min(end - at - kLpRowCost, (long long)nv);
    const T *row = static_cast<const T *>(a.logits) + (long long)m * a.row_stride;
    const LpRow<T> R(row, a.N);
    const int w0 = max(u0, R.in0), w1 = min(u1, R.in1);
    // an element of the row's cut vectors, by a thread of its own (loaded ahead of its use):
    // threads 0 .. those before the first whole vector, 32 .. those past the last
    int ec = -1;
    if (tid < VE) {
      if (u0 == 0 && R.in0 > 0 && tid < min(VE - R.pad, R.N)) ec = tid;
    } else if (tid >= 32 && tid < 32 + VE) {
      if (u0 <= R.in1 && R.in1 < min(u1, R.nvec) && R.col(R.in1) + tid - 32 < R.N) ec = R.col(R.in1) + tid - 32;
    }
    const T ex0 = row[max(ec, 0)];
    // the given tokens' logits likewise, thread c's token c of the row (the token itself was
    // loaded a row ahead)
    const bool known = tid < a.C && tok >= 0 && tok < a.N;
    const T xt0 = row[known ? tok : 0];
    if (tid < a.C && m + 1 < a.M) tok = lp_token_id(a, m + 1, tid);

    // ---- the sums, over even and odd elements.  The reference starts at the largest of the
    // warp's first blocks and moves when a block passes it by 4 (y stays below 6: nothing
    // overflows, and little cancels in log2 s - t / s).
    const float nothing = __uint_as_float(0x7fc00000u);        // (a maximum with NaN is the other)
    float top = nothing, r = kNoRef;              // this thread's largest element
    unsigned long long nr2 = pair2(-kNoRef, -kNoRef), s2 = pair2(0.0f, 0.0f), t2 = s2;
    const unsigned long long e2 = pair2(kLog2e, kLog2e);
    auto raise = [&](float x) {
      if (x > r + 4.0f) {
        const float d = lp_shift(r, x), f = lp_ex2(d);
        t2 = mul2(fma2(pair2(d, d), s2, t2), pair2(f, f));
        s2 = mul2(s2, pair2(f, f));
        r = x;
        nr2 = pair2(-x, -x);
      }
    };
    auto add = [&](float x0, float x1) {
      const float2 y = both2(mul2(add2(pair2(x0, x1), nr2), e2));
      const float y0 = max_nan(y.x, -150.0f), y1 = max_nan(y.y, -150.0f);       // 2^-150 is 0; -inf stays out of y 2^y
      const unsigned long long p2 = pair2(lp_ex2(y0), lp_ex2(y1));
      s2 = add2(s2, p2);
      t2 = fma2(pair2(y0, y1), p2, t2);
    };
    int g = 0;                                    // log2 of the blocks behind a kept maximum
    if (TOP)
      while ((w1 - w0 - 1) / kLpBlock >> g >= kLpMaxima) ++g;
    float run = nothing;
#pragma unroll 1
    for (int v = w0, blk = 0; v < w1; v += kLpBlock, ++blk) {
      uint4 x4[kLpUnroll];
      fetch(x4);
      float bm = nothing;
#pragma unroll
      for (int i = 0; i < kLpUnroll; ++i)
        if (v + tid + i * kLpThreads < w1) bm = fmaxf(bm, lp_max<T>(w[i]));
      top = fmaxf(top, bm);
      if (TOP) {
        run = (blk & ((1 << g) - 1)) == 0 ? bm : fmaxf(run, bm);
        maxima[(blk >> g) * kLpThreads + tid] = run;
      }
      if (blk == 0) {                             // (whole warp)
        r = fmaxf(key_value32(__reduce_max_sync(0xffffffffu, order_key32(bm))), kNoRef);
        nr2 = pair2(-r, -r);
      } else {
        raise(bm);
      }
#pragma unroll
      for (int i = 0; i < kLpUnroll; ++i)
        if (v + tid + i * kLpThreads < w1) {
          float x[VE];
          lp_unpack<T>(w[i], x);
#pragma unroll
          for (int e = 0; e < VE; e += 2) add(x[e], x[e + 1]);
        }
#pragma unroll
      for (int i = 0; i < kLpUnroll; ++i) w[i] = x4[i];
    }
    const float ex1 = lp_float(ex0);
    if (ec >= 0) {
      raise(ex1);
      add(ex1, -INFINITY);
    }
    const float2 ss = both2(s2), tt = both2(t2);
    LpSum z = lp_block(LpSum{r, ss.x + ss.y, tt.x + tt.y}, sm);
    if (TOP) {
      const unsigned bound = lp_bound(w0 + tid < w1 ? order_key32(top) : 0u, min(max(w1 - w0, 0) / 32, kLpWarps), a.k, sm);
      lp_select((unsigned long long)bound << 32, a.k, sm, [&](unsigned long long B, auto put) {
        const unsigned key0 = (unsigned)(B >> 32);
        auto offer = [&](float x, int c) {
          const unsigned long long p = lp_pair(order_key32(x), c);
          if (p >= B) put(p);
        };
        // element e of kept maximum b: vector j of its 4 2^g, b = (first block >> g) threads + thread
        auto element = [&](int b, int j, int e) {
          const int v = w0 + (((b / kLpThreads) << g) * kLpUnroll + j) * kLpThreads + b % kLpThreads;
          if (v < w1) offer(lp_float(row[R.col(v) + e]), R.col(v) + e);
        };
        const int kept = w0 < w1 ? ((w1 - w0 - 1) / kLpBlock >> g) + 1 : 0, eg = kLpLogUnroll + g;
        if (tid == 0) sm.nblock = 0;
        __syncthreads();
#pragma unroll 1
        for (int b = tid; b < kept * kLpThreads; b += kLpThreads)
          if (w0 + (b / kLpThreads << g) * kLpBlock + tid < w1 && order_key32(maxima[b]) >= key0) {
            const int i = atomicAdd(&sm.nblock, 1);
            if (i < kLpBlocks) sm.block[i] = b;
          }
        __syncthreads();
        if (sm.nblock <= kLpBlocks) {             // a thread an element of a listed block
#pragma unroll 4
          for (int i = tid; i < (sm.nblock << eg) * VE; i += kLpThreads) {
            const int q = i / VE;
            element(sm.block[q >> eg], q & ((1 << eg) - 1), i % VE);
          }
        } else {                                  // many (equal logits): every thread its own
#pragma unroll 1
          for (int b = tid; b < kept * kLpThreads; b += kLpThreads)
            if (order_key32(maxima[b]) >= key0) {
#pragma unroll 1
              for (int q = 0; q < VE << eg; ++q) element(b, q / VE, q % VE);
            }
        }
        if (ec >= 0) offer(ex1, ec);
      });
    }
    float xt = lp_float(xt0);
    if (u0 > 0 || u1 < nv) {
      // ---- a cut row: the last CTA to finish it joins its parts, in order
      if (tid == 0) {
        int c0 = me, c1 = me;
        if (a.S > 0) {
          c0 = m * a.S;
          c1 = c0 + a.S - 1;
        } else {
          if (u0 > 0) c0 = (int)((at + kLpRowCost) / a.share);
          if (u1 < nv) c1 = (int)((at + kLpRowCost + nv - 1) / a.share);
        }
        sm.first = c0;
        sm.parts = c1 - c0 + 1;
        *reinterpret_cast<float4 *>(a.part + (size_t)(2 * me + (c0 == me)) * 4) = make_float4(z.r, z.s, z.t, 0.0f);
      }
      __syncthreads();
      const int c0 = sm.first, parts = sm.parts;
      auto slot = [&](int i) { return (size_t)(2 * (c0 + i) + (i == 0)); };   // the first part: its CTA's slot 1
      if (TOP && tid < a.k) a.cand[slot(me - c0) * a.k + tid] = sm.sel[tid];
      __syncthreads();                            // (thread 0's release and acquire order every thread's accesses)
      if (tid == 0) {
        const int old = atom_add_acq_rel_gpu(a.counters + c0, 1);
        sm.n = old == parts - 1;
        if (sm.n) a.counters[c0] = 0;             // zero again for the next call
      }
      __syncthreads();
      const bool last = sm.n != 0;
      __syncthreads();
      if (!last) continue;
      z = LpSum{kNoRef, 0.0f, 0.0f};
      for (int i = tid; i < parts; i += kLpThreads) {
        const float4 q = __ldcg(reinterpret_cast<const float4 *>(a.part + slot(i) * 4));
        z = lp_join(z, LpSum{q.x, q.y, q.z});
      }
      z = lp_block(z, sm);
      if (TOP) {
        const int total = parts * a.k;
        auto pair = [&](int i) {
          const int q = i / a.k;
          return __ldcg(a.cand + slot(q) * a.k + i - q * a.k);
        };
        unsigned best = 0u;
#pragma unroll 4
        for (int i = tid; i < total; i += kLpThreads) best = max(best, (unsigned)(pair(i) >> 32));
        const unsigned bound = lp_bound(best, min(total / 32, kLpWarps), a.k, sm);
        lp_select((unsigned long long)bound << 32, a.k, sm, [&](unsigned long long B, auto put) {
          if (best < (unsigned)(B >> 32)) return;
#pragma unroll 4
          for (int i = tid; i < total; i += kLpThreads) {
            const unsigned long long p = pair(i);
            if (p >= B && p != 0ull) put(p);
          }
        });
      }
    }
    lp_write<T>(a, m, row, z, sm, tid < a.C && known, xt);
    __syncthreads();                              // sm is free for the next row
  }
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

// One range a CTA over the places of all rows; at least two blocks of vectors (fewer, and the
// join costs a short call more than the CTAs save).
constexpr size_t kLpCounterBytes = 8192;          // a counter a CTA, at a fixed place: calls of any shape share a workspace
struct LpPlan {
  int grid, nv, S, step;
  long long share;
  size_t part, cand;
};
size_t up(size_t n) { return (n + 255) & ~(size_t)255; }
LpPlan lp_plan(int M, int N, int es, int k, int sms) {
  LpPlan p{};
  const int ve = 16 / es;
  p.nv = (int)(((long long)N + 2 * ve - 2) / ve); // whatever the row's alignment
  const long long total = ((long long)p.nv + kLpRowCost) * M, most = (long long)kLpPerSm * sms;
  p.share = (total + most - 1) / most;
  if (p.share < kLpMinBlocks * kLpBlock) p.share = kLpMinBlocks * kLpBlock;
  p.grid = (int)((total + p.share - 1) / p.share);
  // Equal parts of each row instead, one a CTA, where a CTA of the ranges would finish two rows
  // one after the other and that costs more than the CTAs left over (a row's end takes a CTA
  // about as long as 700 vectors, 4000 with the top k).
  const int end = k > 0 ? 4000 : 700;
  long long S = most / M, fit = (p.nv + kLpMinBlocks * kLpBlock - 1) / (kLpMinBlocks * kLpBlock);
  if (S > fit) S = fit;
  if (S >= 1 && (p.nv + S - 1) / S + end <= p.share + 2 * end) {
    p.step = (int)((p.nv + S - 1) / S);
    p.S = (p.nv + p.step - 1) / p.step;
    p.grid = p.S * M;
  }
  p.part = up((size_t)p.grid * 2 * 16);
  p.cand = up((size_t)p.grid * 2 * k * 8);
  return p;
}
int lp_shape(int M, int N, int C, int k, int dtype) {
  if (M < 0 || N < 0 || C < 0 || k < 0) return bad(QW_ERR_INVALID_ARG, "negative size");
  if (dtype != QW_F16 && dtype != QW_BF16 && dtype != QW_F32) return bad(QW_ERR_INVALID_ARG, "logit type %d", dtype);
  if (N == 0 || k > kLpMaxK || k > N || N > (1 << 30))
    return bad(QW_ERR_UNSUPPORTED_SHAPE, "need 1 <= N <= 2^30 and k <= min(%d, N)", kLpMaxK);
  return QW_OK;
}

}  // namespace
}  // namespace qw

using namespace qw;

extern "C" {

size_t token_logprobs_workspace_bytes(int M, int N, int k, int dtype) {
  int sms = 0;
  if (lp_shape(M, N, 0, k, dtype) || M == 0 || device_info(&sms, nullptr)) return 0;
  const LpPlan p = lp_plan(M, N, dtype == QW_F32 ? 4 : 2, k, sms);
  return kLpCounterBytes + p.part + p.cand;
}
size_t token_logprobs_workspace_zero_bytes(int M, int N, int k, int dtype) {
  int sms = 0;
  if (lp_shape(M, N, 0, k, dtype) || M == 0 || device_info(&sms, nullptr)) return 0;
  return kLpCounterBytes;
}

int token_logprobs(const void *logits, int dtype, int M, int N, long long row_stride, const void *tokens,
                   int token_bytes, int C, int k, float *logprob, float *entropy, float *lse, float *top_logprob,
                   int32_t *top_idx, void *ws, size_t ws_bytes, qw_stream_t stream) {
  int rc = lp_shape(M, N, C, k, dtype);
  if (rc) return rc;
  if (token_bytes != 4 && token_bytes != 8) return bad(QW_ERR_INVALID_ARG, "tokens are int32 or int64");
  if (M == 0) return QW_OK;
  if (!logits || (C > 0 && (!tokens || !logprob)) || !entropy || !lse || (k > 0 && (!top_logprob || !top_idx)))
    return bad(QW_ERR_INVALID_ARG, "null tensor pointer");
  if (!at(logits, dtype == QW_F32 ? 4 : 2) || !at(tokens, token_bytes) || !at(logprob, 4) || !at(entropy, 4) ||
      !at(lse, 4) || !at(top_logprob, 4) || !at(top_idx, 4) || (ws && !at(ws, 256)))
    return bad(QW_ERR_ALIGNMENT, "arrays must be aligned to their elements, the workspace to 256 bytes");
  LpArgs a{};
  int sms = 0;
  if ((rc = device_info(&sms, &a.err))) return rc;
  const LpPlan p = lp_plan(M, N, dtype == QW_F32 ? 4 : 2, k, sms);
  const size_t need = kLpCounterBytes + p.part + p.cand;
  if ((size_t)kLpPerSm * sms * 4 > kLpCounterBytes) return bad(QW_ERR_ARCH, "more SMs than counters (%d)", sms);
  if ((!ws || ws_bytes < need))
    return bad(QW_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws ? ws_bytes : (size_t)0);
  uint8_t *w = static_cast<uint8_t *>(ws);
  a.logits = logits;
  a.tokens = tokens;
  a.row_stride = row_stride;
  a.M = M;
  a.N = N;
  a.C = C;
  a.k = k;
  a.tok64 = token_bytes == 8;
  a.nv = p.nv;
  a.share = p.share;
  a.S = p.S;
  a.step = p.step;
  a.logprob = logprob;
  a.entropy = entropy;
  a.lse = lse;
  a.top_lp = top_logprob;
  a.top_idx = top_idx;
  a.counters = reinterpret_cast<int *>(w);
  a.part = reinterpret_cast<float *>(w + kLpCounterBytes);
  a.cand = reinterpret_cast<unsigned long long *>(w + kLpCounterBytes + p.part);
#define QW_LP(T) (k > 0 ? reinterpret_cast<const void *>(token_logprobs_kernel<T, true>) \
                       : reinterpret_cast<const void *>(token_logprobs_kernel<T, false>))
  const void *f = dtype == QW_F16 ? QW_LP(__half) : dtype == QW_BF16 ? QW_LP(__nv_bfloat16) : QW_LP(float);
#undef QW_LP
  cudaError_t e = launch_pdl(f, dim3(p.grid), dim3(kLpThreads), 0, reinterpret_cast<cudaStream_t>(stream), a);
  count_launch();
  if (e != cudaSuccess) return bad(QW_ERR_CUDA, "log probability kernel launch: %s", cudaGetErrorString(e));
  return QW_OK;
}

}  // extern "C"
