// token_logprobs.cu -- log probabilities of given tokens, entropy and the k most likely
// tokens of each row of a logit matrix, in one pass over the logits.
//
// In base 2, with y_j = x_j log2(e) - r for a reference r near the row's largest x log2(e):
//   s = sum 2^y_j,  t = sum y_j 2^y_j
//   logsumexp = (r + log2 s) ln 2      log p_j = (y_j - log2 s) ln 2
//   entropy   = (log2 s - t / s) ln 2  (both terms are >= 0 up to rounding: no cancellation)
// A thread keeps (r, s, t) while it streams its 16-byte vectors; r moves only when a vector
// brings a new maximum.  All sums in binary32, joined in a fixed order.
//
// The k most likely come from the same pass.  Each warp's j-th largest thread maximum, j =
// ceil(k / warps), is passed by j threads of that warp, so the smallest of these, T, is a lower
// bound of the k-th largest element: the elements from T on lie in a few threads, which read
// the quarters of their elements that reach T again (from L2) and list them as
// (value, column) composites -- distinct, ties ordered by column.  A list that overflows
// (many equal logits) gives a higher bound, the k-th largest of what it holds, and is filled
// again.  A row is cut into slices (one CTA each); the last slice of a row to finish joins the
// sums and selects among the slices' lists the same way.
//
// What bounds it: the read of the logits (HBM), at about six operations and one ex2 an
// element; for few rows the launch and two chains of block-wide steps.
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

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpMaxK = 64;
constexpr int kLpMaxSlices = 128;                 // kLpMaxSlices k candidates: at most 32 a thread
constexpr int kLpList = 512;                      // listed elements
constexpr int kLpPerSm = 4;                       // CTAs an SM holds (64 registers a thread)
constexpr int kLpUnroll = 4;                      // vectors in flight a thread; maxima kept apart

struct LpArgs {
  const void *logits;
  const void *tokens;                             // [M][C] int32 or int64
  long long row_stride;                           // elements
  int M, N, C, k, tok64;
  int vps;                                        // vectors of a slice
  float *logprob, *entropy, *lse, *top_lp;
  int *top_idx;
  float *part;                                    // [M][S][4]: r, s, t
  unsigned long long *cand;                       // [M][S][k]
  int *counters;                                  // [M], zero between calls
  int *err;
};

struct LpSmem {
  float red[3][kLpWarps];
  unsigned wkey[kLpWarps];
  unsigned long long list[kLpList];
  unsigned long long sel[kLpMaxK];
  unsigned long long T;
  int n, last;
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
// binary32 values as unsigned integers in the values' order; -0 as +0; no value gives 0
__device__ __forceinline__ unsigned order_key32(float x) {
  const unsigned u = __float_as_uint(x + 0.0f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value32(unsigned k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

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

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNoRef = -1e30f;                  // the reference of a sum of nothing

struct LpSum {
  float r, s, t;
};
__device__ __forceinline__ void lp_move(LpSum &a, float r) {       // to the reference r
  const float d = a.r - r, f = lp_ex2(d);
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
// over the CTA, in a fixed order; valid in every thread
__device__ __forceinline__ LpSum lp_block(LpSum a, LpSmem &sm) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    a = lp_join(a, LpSum{__shfl_xor_sync(0xffffffffu, a.r, o), __shfl_xor_sync(0xffffffffu, a.s, o),
                         __shfl_xor_sync(0xffffffffu, a.t, o)});
  const int w = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) {
    sm.red[0][w] = a.r;
    sm.red[1][w] = a.s;
    sm.red[2][w] = a.t;
  }
  __syncthreads();
  a = LpSum{sm.red[0][0], sm.red[1][0], sm.red[2][0]};
#pragma unroll
  for (int i = 1; i < kLpWarps; ++i) a = lp_join(a, LpSum{sm.red[0][i], sm.red[1][i], sm.red[2][i]});
  return a;
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
  // rank: 4 threads an element while that many are free
  const int sub = n <= kLpThreads / 4 ? 4 : 1;
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += kLpThreads / sub) {
    const int i = i0 + (int)threadIdx.x / sub, e = (int)threadIdx.x % sub;
    const unsigned long long mine = i < n ? sm.list[i] : 0ull;
    int above = 0;
    if (i < n)
#pragma unroll 4
      for (int j = e; j < n; j += sub) above += sm.list[j] > mine;
    if (sub == 4) {
      above += __shfl_xor_sync(0xffffffffu, above, 1);
      above += __shfl_xor_sync(0xffffffffu, above, 2);
    }
    if (i < n && e == 0 && above < k) sm.sel[above] = mine;
  }
  __syncthreads();
}
__device__ __forceinline__ unsigned long long lp_pair(unsigned key, int col) {
  return ((unsigned long long)key << 32) | (0xffffffffu - (unsigned)col);
}

// The row's results from its sums and (k > 0) its k best pairs in sm.sel.
template <typename T>
__device__ __forceinline__ void lp_write(const LpArgs &a, int m, const T *row, const LpSum &z, const LpSmem &sm) {
  const float ls = log2f(z.s);
  const bool none = z.s == 0.0f;                  // every logit -inf
  if (threadIdx.x == 0) {
    a.lse[m] = none ? -INFINITY : (z.r + ls) * kLn2;
    a.entropy[m] = none ? 0.0f : fmaxf(ls - z.t / z.s, z.s != z.s ? z.s : 0.0f) * kLn2;
  }
  auto lp = [&](float x) { return none ? -INFINITY : (fmaf(x, kLog2e, -z.r) - ls) * kLn2; };
  for (int c = threadIdx.x; c < a.C; c += kLpThreads) {
    const long long i = (long long)m * a.C + c;
    const long long tok = a.tok64 ? reinterpret_cast<const long long *>(a.tokens)[i] : reinterpret_cast<const int *>(a.tokens)[i];
    float y = __uint_as_float(0x7fc00000u);       // no such token: NaN
    if (tok >= 0 && tok < a.N) y = lp(lp_float(row[tok]));
    else atomicCAS(a.err, 0, -9);
    a.logprob[i] = y;
  }
  for (int i = threadIdx.x; i < a.k; i += kLpThreads) {
    const unsigned long long p = sm.sel[i];
    a.top_lp[(long long)m * a.k + i] = lp(key_value32((unsigned)(p >> 32)));
    a.top_idx[(long long)m * a.k + i] = (int)(0xffffffffu - (unsigned)p);
  }
}

template <typename T>
__global__ void __launch_bounds__(kLpThreads, kLpPerSm) token_logprobs_kernel(const __grid_constant__ LpArgs a) {
  constexpr int VE = LpVec<T>::VE;
  __shared__ LpSmem sm;
  const int S = gridDim.x, sl = blockIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  for (int m = blockIdx.y; m < a.M; m += gridDim.y) {
    const T *row = static_cast<const T *>(a.logits) + (long long)m * a.row_stride;
    const LpRow<T> R(row, a.N);
    const int v0 = min(sl * a.vps, R.nvec), v1 = min(v0 + a.vps, R.nvec);
    LpSum z{kNoRef, 0.0f, 0.0f};
    float top = -INFINITY, quarter[kLpUnroll];
#pragma unroll
    for (int i = 0; i < kLpUnroll; ++i) quarter[i] = -INFINITY;
    const int w0 = max(v0, R.in0), w1 = min(v1, R.in1);
    auto raise = [&](float x) {                   // a new largest element: the reference follows
      if (x > top) {
        top = x;
        lp_move(z, x * kLog2e);
      }
    };
    auto add = [&](float x) {
      const float y = max_nan(fmaf(x, kLog2e, -z.r), -150.0f);     // 2^-150 is 0; -inf stays out of y 2^y
      const float p = lp_ex2(y);
      z.s += p;
      z.t = fmaf(y, p, z.t);
    };
    // the elements of the row's cut vectors: thread 0 takes those of its slice, once
    auto edges = [&](auto f) {
      if (threadIdx.x != 0) return;
#pragma unroll 1
      for (int end = 0; end < 2; ++end) {
        const int v = end ? R.in1 : 0;
        if (v < v0 || v >= v1 || (end ? v >= R.nvec : R.in0 == 0) ) continue;
#pragma unroll 1
        for (int c = max(R.col(v), 0); c < min(R.col(v) + VE, R.N); ++c) f(lp_float(row[c]), c);
      }
    };
#pragma unroll 1
    for (int v = w0 + (int)threadIdx.x; v < w1; v += kLpUnroll * kLpThreads) {
      uint4 w[kLpUnroll];
#pragma unroll
      for (int i = 0; i < kLpUnroll; ++i)
        if (v + i * kLpThreads < w1) w[i] = R.raw(v + i * kLpThreads);
#pragma unroll
      for (int i = 0; i < kLpUnroll; ++i) {
        if (v + i * kLpThreads >= w1) break;
        float x[VE];
        lp_unpack<T>(w[i], x);
        float vm = x[0];
#pragma unroll
        for (int e = 1; e < VE; ++e) vm = fmaxf(vm, x[e]);
        quarter[i] = fmaxf(quarter[i], vm);
        raise(vm);
#pragma unroll
        for (int e = 0; e < VE; ++e) add(x[e]);
      }
    }
    edges([&](float x, int) {
      raise(x);
      add(x);
    });
    z = lp_block(z, sm);
    if (a.k > 0) {
      unsigned reach = 0u;                        // order keys of the quarters
      const unsigned bound = lp_bound(w0 + (int)threadIdx.x < w1 ? order_key32(top) : 0u, min((w1 - w0) / 32, kLpWarps), a.k, sm);
      lp_select((unsigned long long)bound << 32, a.k, sm, [&](unsigned long long B, auto put) {
        const unsigned key0 = (unsigned)(B >> 32);
        reach = 0u;
#pragma unroll
        for (int i = 0; i < kLpUnroll; ++i) reach |= order_key32(quarter[i]) >= key0 ? 1u << i : 0u;
        auto offer = [&](float x, int c) {
          const unsigned long long p = lp_pair(order_key32(x), c);
          if (p >= B) put(p);
        };
#pragma unroll 1
        for (int v = w0 + (int)threadIdx.x; v < w1 && reach; v += kLpUnroll * kLpThreads) {
          uint4 w[kLpUnroll];
#pragma unroll
          for (int i = 0; i < kLpUnroll; ++i)
            if (v + i * kLpThreads < w1 && (reach >> i & 1u)) w[i] = R.raw(v + i * kLpThreads);
#pragma unroll 1
          for (int i = 0; i < kLpUnroll; ++i) {
            if (v + i * kLpThreads < w1 && (reach >> i & 1u)) {
              float x[VE];
              lp_unpack<T>(w[0], x);
#pragma unroll
              for (int e = 0; e < VE; ++e) offer(x[e], R.col(v + i * kLpThreads) + e);
            }
#pragma unroll
            for (int j = 0; j + 1 < kLpUnroll; ++j) w[j] = w[j + 1];
          }
        }
        edges(offer);
      });
    }
    if (S > 1) {
      // ---- publish; the last slice of the row joins
      unsigned long long *cand = a.cand + (size_t)m * S * a.k;
      if (threadIdx.x == 0) *reinterpret_cast<float4 *>(a.part + ((size_t)m * S + sl) * 4) = make_float4(z.r, z.s, z.t, 0.0f);
      if ((int)threadIdx.x < a.k) cand[(size_t)sl * a.k + threadIdx.x] = sm.sel[threadIdx.x];
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) {
        const int old = atom_add_acq_rel_gpu(a.counters + m, 1);
        sm.last = old == S - 1;
        if (sm.last) a.counters[m] = 0;           // zero again for the next call
      }
      __syncthreads();
      if (!sm.last) continue;
      __threadfence();
      z = LpSum{kNoRef, 0.0f, 0.0f};
      if ((int)threadIdx.x < S) {
        const float4 q = __ldcg(reinterpret_cast<const float4 *>(a.part + ((size_t)m * S + threadIdx.x) * 4));
        z = LpSum{q.x, q.y, q.z};
      }
      z = lp_block(z, sm);
      if (a.k > 0) {
        const int total = S * a.k;
        unsigned best = 0u;
        for (int i = threadIdx.x; i < total; i += kLpThreads) best = max(best, (unsigned)(__ldcg(cand + i) >> 32));
        const unsigned bound = lp_bound(best, min(total / 32, kLpWarps), a.k, sm);
        lp_select((unsigned long long)bound << 32, a.k, sm, [&](unsigned long long B, auto put) {
          if (best < (unsigned)(B >> 32)) return;
          for (int i = threadIdx.x; i < total; i += kLpThreads) {
            const unsigned long long p = __ldcg(cand + i);
            if (p >= B && p != 0ull) put(p);
          }
        });
      }
    }
    lp_write<T>(a, m, row, z, sm);
    __syncthreads();                              // sm free for the next row
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

// Slices a row is cut into: enough CTAs to fill the SMs twice, but at least two
// vectors a thread (a shorter slice costs more in the join than it saves).
// (several slices only where M < 8 SMs: one counter a row)
constexpr size_t kLpCounterBytes = 8192;
constexpr int kLpFill = 8;                        // CTAs an SM to aim for
struct LpPlan {
  int S, vps;
  size_t counters, part, cand;
};
size_t up(size_t n) { return (n + 255) & ~(size_t)255; }
LpPlan lp_plan(int M, int N, int es, int k, int sms) {
  LpPlan p{};
  const int ve = 16 / es;
  const long long nvec = ((long long)N + ve - 1 + ve - 1) / ve;     // whatever the row's alignment
  long long S = ((long long)kLpFill * sms + M - 1) / (M > 0 ? M : 1);
  const long long most = (nvec + 2 * kLpThreads - 1) / (2 * kLpThreads);
  if (S > most) S = most;
  if (S > kLpMaxSlices) S = kLpMaxSlices;
  if (S < 1) S = 1;
  p.vps = (int)((nvec + S - 1) / S);
  p.S = (int)((nvec + p.vps - 1) / p.vps);
  if (p.S > 1) {
    p.counters = kLpCounterBytes;      // a fixed place: calls of any M share a workspace
    p.part = up((size_t)M * p.S * 16);
    p.cand = up((size_t)M * p.S * k * 8);
  }
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
  return p.counters + p.part + p.cand;
}
size_t token_logprobs_workspace_zero_bytes(int M, int N, int k, int dtype) {
  int sms = 0;
  if (lp_shape(M, N, 0, k, dtype) || M == 0 || device_info(&sms, nullptr)) return 0;
  return lp_plan(M, N, dtype == QW_F32 ? 4 : 2, k, sms).counters;
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
  if ((size_t)kLpFill * sms * 4 > kLpCounterBytes) return bad(QW_ERR_ARCH, "more SMs than counters (%d)", sms);
  const LpPlan p = lp_plan(M, N, dtype == QW_F32 ? 4 : 2, k, sms);
  const size_t need = p.counters + p.part + p.cand;
  if (need > 0 && (!ws || ws_bytes < need))
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
  a.vps = p.vps;
  a.logprob = logprob;
  a.entropy = entropy;
  a.lse = lse;
  a.top_lp = top_logprob;
  a.top_idx = top_idx;
  a.counters = reinterpret_cast<int *>(w);
  a.part = reinterpret_cast<float *>(w + p.counters);
  a.cand = reinterpret_cast<unsigned long long *>(w + p.counters + p.part);
  const void *f = dtype == QW_F16    ? reinterpret_cast<const void *>(token_logprobs_kernel<__half>)
                  : dtype == QW_BF16 ? reinterpret_cast<const void *>(token_logprobs_kernel<__nv_bfloat16>)
                                     : reinterpret_cast<const void *>(token_logprobs_kernel<float>);
  cudaError_t e = launch_pdl(f, dim3(p.S, M < 65535 ? M : 65535), dim3(kLpThreads), 0, reinterpret_cast<cudaStream_t>(stream), a);
  count_launch();
  if (e != cudaSuccess) return bad(QW_ERR_CUDA, "log probability kernel launch: %s", cudaGetErrorString(e));
  return QW_OK;
}

}  // extern "C"
