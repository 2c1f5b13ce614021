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
// The k most likely come from the same pass: the k-th largest of the threads' maxima is a
// lower bound T of the k-th largest element, so the elements above T lie in fewer than k
// threads, which read their own elements again (from L1 and L2) and list them; elements
// equal to T fill up, lowest index first.  A row is cut into slices (one CTA each); the last
// slice of a row to finish joins the sums and selects among the slices' lists the same way.
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
constexpr int kLpListA = 2048;                    // elements above T
constexpr int kLpListB = 256;                     // elements equal to T
static_assert(kLpMaxSlices * kLpMaxK <= kLpListA / kLpMaxK * kLpThreads, "a joining thread's share, k times, fits list A");

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
  unsigned long long lista[kLpListA];
  unsigned listb[kLpListB];
  alignas(16) unsigned long long key[kLpThreads];
  unsigned long long sel[kLpMaxK];
  unsigned long long T;
  int na, nb, last, scan[kLpWarps];
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
// vectors can reach past the row; they are read element by element.
template <typename T>
struct LpRow {
  static constexpr int VE = LpVec<T>::VE;
  const T *row;
  int pad, N, nvec;
  __device__ __forceinline__ LpRow(const T *r, int n) : row(r), N(n) {
    pad = (int)((reinterpret_cast<uintptr_t>(r) / sizeof(T)) % VE);
    nvec = (int)(((long long)n + pad + VE - 1) / VE);
  }
  __device__ __forceinline__ int col(int v) const { return v * VE - pad; }
  __device__ __forceinline__ bool inner(int v) const { return col(v) >= 0 && col(v) + VE <= N; }
  __device__ __forceinline__ uint4 raw(int v) const {
    if (inner(v)) return __ldg(reinterpret_cast<const uint4 *>(row + col(v)));
    alignas(16) T e[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      const int c = col(v) + i;
      if (c >= 0 && c < N) e[i] = row[c];
      else if constexpr (sizeof(T) == 4) e[i] = -INFINITY;
      else *reinterpret_cast<uint16_t *>(&e[i]) = sizeof(T) == 2 && LpRow::kBf ? 0xff80u : 0xfc00u;   // -inf
    }
    return *reinterpret_cast<const uint4 *>(e);
  }
  static constexpr bool kBf = sizeof(T) == 2 && !__is_same(T, __half);
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

// sm.T = the k-th largest of n keys (k <= n), each thread counting for its own keys.
__device__ __forceinline__ void kth_largest(const unsigned long long *key, int n, int k, LpSmem &sm) {
  for (int i = threadIdx.x; i < n; i += kLpThreads) {
    const unsigned long long mine = key[i];
    int above = 0, equal = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) {
      above += key[j] > mine;
      equal += key[j] == mine;
    }
    if (above < k && k <= above + equal) sm.T = mine;
  }
  __syncthreads();
}
// The k largest of list[0 .. n) (distinct, n >= k or all of them), largest first, into sel.
__device__ __forceinline__ void rank_list(const unsigned long long *list, int n, int k, unsigned long long *sel) {
  for (int i = threadIdx.x; i < n; i += kLpThreads) {
    const unsigned long long mine = list[i];
    int above = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) above += list[j] > mine;
    if (above < k) sel[above] = mine;
  }
}
__device__ __forceinline__ unsigned long long lp_pair(unsigned key, int col) {
  return ((unsigned long long)key << 32) | (0xffffffffu - (unsigned)col);
}

// The slice's k best (key, column) pairs, best first, in sm.sel; 0 where the slice has
// fewer elements.  mymax: the key of this thread's largest element (0: it has none).
template <typename T>
__device__ void lp_slice_topk(const LpRow<T> &R, int v0, int v1, int k, unsigned mymax, LpSmem &sm) {
  constexpr int VE = LpVec<T>::VE;
  sm.key[threadIdx.x] = mymax;
  if (threadIdx.x < k) sm.sel[threadIdx.x] = 0ull;
  if (threadIdx.x == 0) sm.na = sm.nb = 0;
  __syncthreads();
  kth_largest(sm.key, kLpThreads, k, sm);
  unsigned T32 = (unsigned)sm.T;
  for (;;) {
    if (mymax >= T32 && mymax != 0u) {
      for (int v = v0 + (int)threadIdx.x; v < v1; v += kLpThreads) {
        float x[VE];
        lp_unpack<T>(R.raw(v), x);
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const int c = R.col(v) + e;
          const unsigned key = order_key32(x[e]);
          if (key < T32 || c < 0 || c >= R.N) continue;
          if (key > T32) {
            const int at = atomicAdd(&sm.na, 1);
            if (at < kLpListA) sm.lista[at] = lp_pair(key, c);
          } else {
            const int at = atomicAdd(&sm.nb, 1);
            if (at < kLpListB) sm.listb[at] = (unsigned)c;
          }
        }
      }
    }
    __syncthreads();
    if (sm.na <= kLpListA) break;
    // more above T than the list holds (they crowd into few threads): the k-th largest of
    // those listed is a higher lower bound; take its key and list again
    kth_largest(sm.lista, kLpListA, k, sm);
    T32 = (unsigned)(sm.T >> 32);
    __syncthreads();
    if (threadIdx.x == 0) sm.na = sm.nb = 0;
    __syncthreads();
  }
  const int na = sm.na, nb = sm.nb;
  rank_list(sm.lista, na, k, sm.sel);
  const int want = k - na;
  if (want > 0 && T32 != 0u) {
    if (nb <= kLpListB) {                         // few equal to T: rank them by column
      if ((int)threadIdx.x < nb) {
        const unsigned c = sm.listb[threadIdx.x];
        int before = 0;
        for (int j = 0; j < nb; ++j) before += sm.listb[j] < c;
        if (before < want) sm.sel[na + before] = lp_pair(T32, (int)c);
      }
    } else {                                      // many: the first `want`, in column order
      int got = 0;
      for (int base = v0; base < v1 && got < want; base += kLpThreads) {
        const int v = base + (int)threadIdx.x;
        unsigned hit = 0;
        if (v < v1) {
          float x[VE];
          lp_unpack<T>(R.raw(v), x);
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            const int c = R.col(v) + e;
            if (c >= 0 && c < R.N && order_key32(x[e]) == T32) hit |= 1u << e;
          }
        }
        int inc = __popc(hit);
        const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        if (lane == 31) sm.scan[w] = inc;
        __syncthreads();
        int at = got + inc - __popc(hit), all = 0;
        for (int i = 0; i < kLpWarps; ++i) {
          if (i < w) at += sm.scan[i];
          all += sm.scan[i];
        }
        while (hit && at < want) {
          const int e = __ffs(hit) - 1;
          hit &= hit - 1;
          sm.sel[na + at++] = lp_pair(T32, R.col(v) + e);
        }
        got += all;
        __syncthreads();
      }
    }
  }
  __syncthreads();
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
__global__ void __launch_bounds__(kLpThreads, 5) token_logprobs_kernel(const __grid_constant__ LpArgs a) {
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
    float top = -INFINITY;
    constexpr int UN = 4;                         // vectors in flight a thread
    auto take = [&](const uint4 &w) {
      float x[VE];
      lp_unpack<T>(w, x);
      float vm = x[0];
#pragma unroll
      for (int e = 1; e < VE; ++e) vm = fmaxf(vm, x[e]);
      if (vm > top) {
        top = vm;
        lp_move(z, vm * kLog2e);
      }
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float y = max_nan(fmaf(x[e], kLog2e, -z.r), -150.0f);      // 2^-150 is 0; -inf stays out of y 2^y
        const float p = lp_ex2(y);
        z.s += p;
        z.t = fmaf(y, p, z.t);
      }
    };
    int v = v0 + (int)threadIdx.x;
    const bool some = v < v1;
    for (; v + (UN - 1) * kLpThreads < v1; v += UN * kLpThreads) {
      uint4 w[UN];
#pragma unroll
      for (int i = 0; i < UN; ++i) w[i] = R.raw(v + i * kLpThreads);
#pragma unroll
      for (int i = 0; i < UN; ++i) take(w[i]);
    }
    for (; v < v1; v += kLpThreads) take(R.raw(v));
    z = lp_block(z, sm);
    if (a.k > 0) lp_slice_topk<T>(R, v0, v1, a.k, some ? order_key32(top) : 0u, sm);
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
        unsigned long long best = 0ull;
        for (int i = threadIdx.x; i < total; i += kLpThreads) best = max(best, __ldcg(cand + i));
        sm.key[threadIdx.x] = best;
        if ((int)threadIdx.x < a.k) sm.sel[threadIdx.x] = 0ull;
        if (threadIdx.x == 0) sm.na = 0;
        __syncthreads();
        kth_largest(sm.key, kLpThreads, a.k, sm);
        const unsigned long long T64 = sm.T;
        if (best >= T64 && best != 0ull)
          for (int i = threadIdx.x; i < total; i += kLpThreads) {
            const unsigned long long p = __ldcg(cand + i);
            if (p >= T64 && p != 0ull) sm.lista[atomicAdd(&sm.na, 1)] = p;
          }
        __syncthreads();
        rank_list(sm.lista, sm.na, a.k, sm.sel);
        __syncthreads();
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

// Slices a row is cut into: enough CTAs to fill the SMs at 5 CTAs each, but at least two
// vectors a thread (a shorter slice costs more in the join than it saves).
// (several slices only where M < 5 SMs: one counter a row)
constexpr size_t kLpCounterBytes = 4096;
constexpr int kLpPerSm = 5;
struct LpPlan {
  int S, vps;
  size_t counters, part, cand;
};
size_t up(size_t n) { return (n + 255) & ~(size_t)255; }
LpPlan lp_plan(int M, int N, int es, int k, int sms) {
  LpPlan p{};
  const int ve = 16 / es;
  const long long nvec = ((long long)N + ve - 1 + ve - 1) / ve;     // whatever the row's alignment
  long long S = ((long long)kLpPerSm * sms + M - 1) / (M > 0 ? M : 1);
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
  if ((size_t)kLpPerSm * sms * 4 > kLpCounterBytes) return bad(QW_ERR_ARCH, "more SMs than counters (%d)", sms);
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
