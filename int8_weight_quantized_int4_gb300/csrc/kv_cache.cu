// kv_cache.cu -- the paged key-value cache: writing new tokens into pages, copying pages,
// and the C entry points of the cache and of the attention over it (attn_paged.cuh).
//
// Both kernels only move bytes (2 d e a row, read and written), so what bounds them is HBM
// for large calls and the launch with its chain of dependent reads for small ones.
#include <math.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "launch.h"
#include "ptx.cuh"
#include "qgemm.h"

namespace qw {

// ------------------------------------------------------------------- append --
struct AppendArgs {
  const uint16_t *k, *v;
  uint8_t *kp, *vp;
  float *ks, *vs;
  const int *table, *lens, *cu;
  long long k_tok, k_head, v_tok, v_head, page_stride, head_stride, tok_stride;
  int B, T, Hkv, page, npages, max_pages;
  int *err;
};
constexpr int kAppendWarps = 4;

// One warp a new token.  Its K and V rows are loaded (16 bytes a lane) before the token's
// page is known; the chain cu -> sequence -> length, page table -> store is what a small
// call waits for, so a token that is alone in its sequence finds it in one step (cu[t] <= t
// < cu[t + 1]) and the others by a 32-way search of cu.  All loads of a token are under way
// before any is used (eight vectors a lane: 4 KB, a token of most caches), which is what
// fills HBM from four warps a CTA: 97 MB (12 prompts of up to 1400 tokens, 8 heads of 128, bf16)
// in 17.3 us, 5.6 TB/s; 64 tokens (4 heads of 256) in 2.6 us, all of it latency.
// int8: each row (one token of one KV head) becomes codes and a scale with the activation
// quantizer's arithmetic (s = amax / 127, IEEE; code = rne(x / s); a zero row: s = 0).
template <int D, bool I8>
__global__ void __launch_bounds__(32 * kAppendWarps) kv_append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int CH = D / 8;                      // 16-byte vectors of a source row
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  griddep_wait();
  griddep_launch_dependents();
  if (t >= a.T) return;                          // whole warp
  const int nvec = a.Hkv * CH, total = 2 * nvec;           // K vectors, then V vectors
  constexpr int kBatch = 8;
  uint4 x[kBatch];
  auto load = [&](int base) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int u = base + 32 * i + lane;
      if (u < total) {
        const bool isv = u >= nvec;
        const int w = isv ? u - nvec : u, h = w / CH, c = w % CH;
        const uint16_t *src = isv ? a.v + (long long)t * a.v_tok + (long long)h * a.v_head
                                  : a.k + (long long)t * a.k_tok + (long long)h * a.k_head;
        x[i] = __ldg(reinterpret_cast<const uint4 *>(src) + c);
      } else {
        x[i] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
  };
  load(0);
  // the token's sequence: the last b with cu[b] <= t
  int b = t;
  bool found = false;
  if (t < a.B) {
    const int c0 = __ldg(a.cu + t), c1 = __ldg(a.cu + t + 1);
    found = c0 <= t && t < c1;
    if (c0 < 0 || c1 < c0 || c1 > a.T) atomicCAS(a.err, 0, -9);      // offsets out of order
  }
  for (long long i = t + (lane + 1ll) * a.T; i < a.B; i += 32ll * a.T) {      // (sequences with no token)
    const int c0 = __ldg(a.cu + i), c1 = __ldg(a.cu + i + 1);
    if (c0 < 0 || c1 < c0 || c1 > a.T) atomicCAS(a.err, 0, -9);
  }
  if (!found) {
    int lo = 0, hi = a.B;                        // the answer is in [lo, hi)
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32;
      const int at = lo + step * lane;
      const bool le = at < hi && __ldg(a.cu + at) <= t;
      const int n = __popc(__ballot_sync(0xffffffffu, le));       // lanes 0 .. n - 1 (cu ascends)
      const int base = lo + step * (n > 0 ? n - 1 : 0);
      hi = min(hi, base + step);
      lo = base;
    }
    b = lo;
    found = __ldg(a.cu + b) <= t && t < __ldg(a.cu + b + 1);
  }
  if (!found) return;                            // a token of no sequence
  const int pos = __ldg(a.lens + b) - (__ldg(a.cu + b + 1) - t);
  const int pi = pos / a.page, po = pos - pi * a.page;
  int pid = -1;
  if (pos >= 0 && pi < a.max_pages) pid = __ldg(a.table + (size_t)b * a.max_pages + pi);
  if ((unsigned)pid >= (unsigned)a.npages) {     // no page to write to
    if (lane == 0) atomicCAS(a.err, 0, -9);
    return;
  }
  const long long row = pid * a.page_stride + po * a.tok_stride;
  for (int base = 0; base < total; base += 32 * kBatch) {
    if (base > 0) load(base);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int u = base + 32 * i + lane;
      const bool isv = u >= nvec;
      const int w = isv ? u - nvec : u, h = w / CH, c = w % CH;
      const long long off = row + h * a.head_stride;
      if constexpr (!I8) {
        if (u < total) reinterpret_cast<uint4 *>((isv ? a.vp : a.kp) + 2 * off)[c] = x[i];
      } else {
        // CH consecutive lanes hold a row (CH divides 32: all of a row or none is in range)
        if (base + 32 * i >= total) break;       // whole warp
        float f[8], amax = 0.0f;
        const uint32_t wd[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 p = __half22float2(u32_as_h2(wd[e]));
          f[2 * e] = p.x;
          f[2 * e + 1] = p.y;
          amax = fmaxf(amax, fmaxf(fabsf(p.x), fabsf(p.y)));
        }
#pragma unroll
        for (int o = CH / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const float s = __fdiv_rn(amax, 127.0f);
        uint32_t cw[2] = {0u, 0u};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int q = s == 0.0f ? 0 : __float2int_rn(__fdiv_rn(f[e], s));
          cw[e >> 2] |= (uint32_t)(max(-127, min(127, q)) & 0xff) << (8 * (e & 3));
        }
        if (u < total) {
          reinterpret_cast<uint2 *>((isv ? a.vp : a.kp) + off)[c] = make_uint2(cw[0], cw[1]);
          if (c == 0) (isv ? a.vs : a.ks)[((size_t)pid * a.Hkv + h) * a.page + po] = s;
        }
      }
    }
  }
}

// --------------------------------------------------------------- copy pages --
constexpr int kMaxPools = 4;
struct CopyPool {
  uint8_t *base;
  long long layer_stride, page_stride;           // bytes
  long long first;                               // index of its first piece
  int layers, npages;
  unsigned vecs;                                 // vectors of a page
  int wide;                                      // vectors of 16 bytes, else 4
  unsigned pieces;                               // pieces of a page
};
struct CopyArgs {
  CopyPool pool[kMaxPools];
  int npools, n;
  const int *pairs;
  long long total;
  int *err;
};
constexpr int kCopyWarps = 8;
constexpr int kCopyVecs = 8;                     // vectors a lane moves: a piece is 4 KB

template <typename V>
__device__ __forceinline__ void copy_piece(const uint8_t *src, uint8_t *dst, unsigned v0, unsigned vecs, int lane) {
  V r[kCopyVecs];
#pragma unroll
  for (int i = 0; i < kCopyVecs; ++i) {
    const unsigned u = v0 + 32u * i + lane;
    if (u < vecs) r[i] = __ldcs(reinterpret_cast<const V *>(src) + u);
  }
#pragma unroll
  for (int i = 0; i < kCopyVecs; ++i) {
    const unsigned u = v0 + 32u * i + lane;
    if (u < vecs) __stcs(reinterpret_cast<V *>(dst) + u, r[i]);
  }
}

// One warp a piece of 256 vectors of one page of one layer of one pool (eight loads in
// flight a lane); the pieces of all pools and layers in one launch.  1000 pages of 16 layers
// (int8 K and V and their scales, 2.13 GB read and written) in 312 us: 6.83 TB/s, the rate of a
// plain copy; one page of 16 layers in 2.3 us, its launch.
__global__ void __launch_bounds__(32 * kCopyWarps) kv_copy_kernel(const __grid_constant__ CopyArgs a) {
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * kCopyWarps + (threadIdx.x >> 5);
  griddep_wait();
  griddep_launch_dependents();
  if (w >= a.total) return;
  int p = 0;
  while (p + 1 < a.npools && w >= a.pool[p + 1].first) ++p;
  const CopyPool &q = a.pool[p];
  const unsigned long long x = (unsigned long long)(w - q.first);
  const unsigned piece = (unsigned)(x % q.pieces);
  const unsigned long long y = x / q.pieces;
  const int pair = (int)(y % (unsigned)a.n), layer = (int)(y / (unsigned)a.n);
  const int2 sd = __ldg(reinterpret_cast<const int2 *>(a.pairs) + pair);
  if ((unsigned)sd.x >= (unsigned)q.npages || (unsigned)sd.y >= (unsigned)q.npages) {
    if (lane == 0) atomicCAS(a.err, 0, -9);
    return;
  }
  if (sd.x == sd.y) return;
  const uint8_t *src = q.base + layer * q.layer_stride + sd.x * q.page_stride;
  uint8_t *dst = q.base + layer * q.layer_stride + sd.y * q.page_stride;
  const unsigned v0 = piece * (32u * kCopyVecs);
  if (q.wide) copy_piece<uint4>(src, dst, v0, q.vecs, lane);
  else copy_piece<uint32_t>(src, dst, v0, q.vecs, lane);
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

int check_cache(const qw_kv_cache_t *c) {
  if (!c) return bad(QW_ERR_INVALID_ARG, "null cache");
  if (c->dtype != QW_KV_F16 && c->dtype != QW_KV_BF16 && c->dtype != QW_KV_INT8)
    return bad(QW_ERR_INVALID_ARG, "cache type %d", c->dtype);
  if (c->num_pages < 0 || c->page < 1 || c->Hkv < 1) return bad(QW_ERR_INVALID_ARG, "bad cache size");
  if (c->d != 64 && c->d != 128 && c->d != 256)
    return bad(QW_ERR_UNSUPPORTED_SHAPE, "head dimension %d: 64, 128 or 256", c->d);
  if (c->Hkv > 1024 || c->page > (1 << 20)) return bad(QW_ERR_UNSUPPORTED_SHAPE, "Hkv <= 1024, page <= 2^20");
  if (c->num_pages > 0 && (!c->k || !c->v || (c->dtype == QW_KV_INT8 && (!c->k_scale || !c->v_scale))))
    return bad(QW_ERR_INVALID_ARG, "null cache pointer");
  const int es = c->dtype == QW_KV_INT8 ? 1 : 2;
  if (!at(c->k, 16) || !at(c->v, 16) || (c->dtype == QW_KV_INT8 && (!at(c->k_scale, 4) || !at(c->v_scale, 4))) ||
      c->page_stride * es % 16 || c->head_stride * es % 16 || c->token_stride * es % 16)
    return bad(QW_ERR_ALIGNMENT, "cache rows must start on 16-byte boundaries");
  if (c->page_stride < 0 || c->head_stride < 0 || c->token_stride < 0)
    return bad(QW_ERR_INVALID_ARG, "negative cache stride");
  return QW_OK;
}
int check_batch(const qw_kv_batch_t *b, int page, int T) {
  if (!b) return bad(QW_ERR_INVALID_ARG, "null batch");
  if (b->B < 0 || b->max_pages < 0 || T < 0) return bad(QW_ERR_INVALID_ARG, "negative size");
  if ((long long)b->max_pages * page > (1ll << 30))
    return bad(QW_ERR_UNSUPPORTED_SHAPE, "a page table names at most 2^30 keys");
  if (T == 0 || b->B == 0) return QW_OK;
  if (!b->page_table || !b->seq_lens || !b->cu_tokens) return bad(QW_ERR_INVALID_ARG, "null batch pointer");
  if (!at(b->page_table, 4) || !at(b->seq_lens, 4) || !at(b->cu_tokens, 4))
    return bad(QW_ERR_ALIGNMENT, "int32 arrays must be 4-byte aligned");
  return QW_OK;
}
template <bool I8>
const void *append_kernel(int d) {
  return d == 64    ? reinterpret_cast<const void *>(kv_append_kernel<64, I8>)
         : d == 128 ? reinterpret_cast<const void *>(kv_append_kernel<128, I8>)
                    : reinterpret_cast<const void *>(kv_append_kernel<256, I8>);
}

// ---- attention: the query columns of an item, and the workspace for them.  Eight where a
// step's columns (new tokens x heads a KV head) fit (half the MMAs of 16), else up to four blocks
// of 16.
int paged_columns(int max_new, int G) { return (long long)max_new * G <= 8 ? 8 : 64; }
constexpr size_t kPagedCounterBytes = 3 * kPagedMaxCtas * 4;   // three counters a CTA
size_t paged_ws(int d, int cols, int sms) {
  return kPagedCounterBytes + (size_t)2 * paged_ctas(d, cols) * sms * cols * (d + 2) * 4;
}
int check_heads(int d, int Hq, int Hkv, int max_new) {
  if (Hq < 1 || Hkv < 1 || max_new < 1) return bad(QW_ERR_INVALID_ARG, "Hq, Hkv and max_new must be positive");
  if (d != 64 && d != 128 && d != 256)
    return bad(QW_ERR_UNSUPPORTED_SHAPE, "head dimension %d: 64, 128 or 256", d);
  if (Hq % Hkv || Hq > 1024) return bad(QW_ERR_UNSUPPORTED_SHAPE, "Hkv must divide Hq <= 1024 (Hq=%d Hkv=%d)", Hq, Hkv);
  return QW_OK;
}

}  // namespace
}  // namespace qw

using namespace qw;

extern "C" {

int kv_append(const qw_kv_cache_t *c, const qw_kv_batch_t *b, const uint16_t *k, const uint16_t *v, int T,
              long long k_token_stride, long long k_head_stride, long long v_token_stride, long long v_head_stride,
              qw_stream_t stream) {
  int rc = check_cache(c);
  if (rc) return rc;
  if ((rc = check_batch(b, c->page, T))) return rc;
  if (T == 0 || b->B == 0) return QW_OK;
  if (!k || !v) return bad(QW_ERR_INVALID_ARG, "null tensor pointer");
  if (!at(k, 16) || !at(v, 16) || k_token_stride % 8 || k_head_stride % 8 || v_token_stride % 8 || v_head_stride % 8)
    return bad(QW_ERR_ALIGNMENT, "k and v rows must start on 16-byte boundaries");
  AppendArgs a{};
  if ((rc = device_info(nullptr, &a.err))) return rc;
  a.k = k;
  a.v = v;
  a.kp = static_cast<uint8_t *>(c->k);
  a.vp = static_cast<uint8_t *>(c->v);
  a.ks = c->k_scale;
  a.vs = c->v_scale;
  a.table = b->page_table;
  a.lens = b->seq_lens;
  a.cu = b->cu_tokens;
  a.k_tok = k_token_stride;
  a.k_head = k_head_stride;
  a.v_tok = v_token_stride;
  a.v_head = v_head_stride;
  a.page_stride = c->page_stride;
  a.head_stride = c->head_stride;
  a.tok_stride = c->token_stride;
  a.B = b->B;
  a.T = T;
  a.Hkv = c->Hkv;
  a.page = c->page;
  a.npages = c->num_pages;
  a.max_pages = b->max_pages;
  const void *f = c->dtype == QW_KV_INT8 ? append_kernel<true>(c->d) : append_kernel<false>(c->d);
  cudaError_t e = launch_pdl(f, dim3((T + kAppendWarps - 1) / kAppendWarps), dim3(32 * kAppendWarps), 0,
                             reinterpret_cast<cudaStream_t>(stream), a);
  count_launch();
  if (e != cudaSuccess) return bad(QW_ERR_CUDA, "append kernel launch: %s", cudaGetErrorString(e));
  return QW_OK;
}

int kv_copy_pages(const qw_page_pool_t *pools, int n_pools, const int32_t *pairs, int n, qw_stream_t stream) {
  if (n < 0 || n_pools < 0 || n_pools > kMaxPools) return bad(QW_ERR_INVALID_ARG, "bad count");
  if (n_pools > 0 && !pools) return bad(QW_ERR_INVALID_ARG, "null pools");
  CopyArgs a{};
  for (int i = 0; i < n_pools; ++i) {
    const qw_page_pool_t &p = pools[i];
    if (p.layers < 0 || p.num_pages < 0 || p.page_bytes < 0 || p.layer_stride < 0 || p.page_stride < 0)
      return bad(QW_ERR_INVALID_ARG, "negative pool size");
    if (p.page_bytes % 4 || p.page_bytes > (1ll << 30))
      return bad(QW_ERR_UNSUPPORTED_SHAPE, "a page is a multiple of 4 bytes, at most 2^30");
    if (p.layers == 0 || p.page_bytes == 0 || n == 0) continue;
    if (!p.base) return bad(QW_ERR_INVALID_ARG, "null pool pointer");
    if (p.page_stride < p.page_bytes) return bad(QW_ERR_INVALID_ARG, "pages overlap");
    if (!at(p.base, 4) || p.layer_stride % 4 || p.page_stride % 4)
      return bad(QW_ERR_ALIGNMENT, "pools are 4-byte aligned");
    CopyPool &q = a.pool[a.npools++];
    q.base = static_cast<uint8_t *>(p.base);
    q.layer_stride = p.layer_stride;
    q.page_stride = p.page_stride;
    q.layers = p.layers;
    q.npages = p.num_pages;
    q.wide = at(p.base, 16) && p.layer_stride % 16 == 0 && p.page_stride % 16 == 0 && p.page_bytes % 16 == 0;
    q.vecs = (unsigned)(p.page_bytes / (q.wide ? 16 : 4));
    q.pieces = (q.vecs + 32 * kCopyVecs - 1) / (32 * kCopyVecs);
    q.first = a.total;
    a.total += (long long)q.pieces * n * p.layers;
  }
  if (a.total == 0) return QW_OK;
  if (!pairs) return bad(QW_ERR_INVALID_ARG, "null pairs");
  if (!at(pairs, 8)) return bad(QW_ERR_ALIGNMENT, "pairs must be 8-byte aligned");
  const long long grid = (a.total + kCopyWarps - 1) / kCopyWarps;
  if (grid > 0x7fffffffll) return bad(QW_ERR_UNSUPPORTED_SHAPE, "too many pages for one call");
  int rc = device_info(nullptr, &a.err);
  if (rc) return rc;
  a.n = n;
  a.pairs = pairs;
  cudaError_t e = launch_pdl(reinterpret_cast<const void *>(kv_copy_kernel), dim3((unsigned)grid), dim3(32 * kCopyWarps),
                             0, reinterpret_cast<cudaStream_t>(stream), a);
  count_launch();
  if (e != cudaSuccess) return bad(QW_ERR_CUDA, "copy kernel launch: %s", cudaGetErrorString(e));
  return QW_OK;
}

size_t attn_paged_workspace_bytes(int d, int Hq, int Hkv, int max_new) {
  int sms = 0;
  if (check_heads(d, Hq, Hkv, max_new) || device_info(&sms, nullptr)) return 0;
  return paged_ws(d, paged_columns(max_new, Hq / Hkv), sms);
}
size_t attn_paged_workspace_zero_bytes(int d, int Hq, int Hkv, int max_new) {
  return check_heads(d, Hq, Hkv, max_new) ? 0 : kPagedCounterBytes;
}

int attn_paged(const qw_kv_cache_t *c, const qw_kv_batch_t *b, const uint16_t *q, int T, int Hq,
               long long q_token_stride, long long q_head_stride, int max_new, int window, int sinks, float scale,
               uint16_t *out, float *lse, void *ws, size_t ws_bytes, qw_stream_t stream) {
  int rc = check_cache(c);
  if (rc) return rc;
  if ((rc = check_batch(b, c->page, T))) return rc;
  if ((rc = check_heads(c->d, Hq, c->Hkv, max_new))) return rc;
  if (window < 0 || sinks < 0) return bad(QW_ERR_INVALID_ARG, "negative window or sinks");
  if (!isfinite(scale)) return bad(QW_ERR_INVALID_ARG, "scale is not finite");
  if ((long long)T * Hq > 0x7fffffffll) return bad(QW_ERR_UNSUPPORTED_SHAPE, "T * Hq above 2^31 - 1");
  if (T == 0 || b->B == 0) return QW_OK;
  if (!q || !out) return bad(QW_ERR_INVALID_ARG, "null tensor pointer");
  if (!at(q, 16) || !at(out, 16) || q_token_stride % 8 || q_head_stride % 8 || (lse && !at(lse, 4)) ||
      (ws && !at(ws, 256)))
    return bad(QW_ERR_ALIGNMENT, "q rows and out must start on 16-byte boundaries, the workspace on a 256-byte one");
  PagedArgs a{};
  int sms = 0;
  if ((rc = device_info(&sms, &a.err))) return rc;
  a.G = Hq / c->Hkv;
  const int cols = paged_columns(max_new, a.G);
  const size_t need = paged_ws(c->d, cols, sms);
  const int most_sms = kPagedMaxCtas / paged_ctas(c->d, cols);
  if (sms > most_sms) return bad(QW_ERR_ARCH, "more than %d SMs", most_sms);
  if (!ws || ws_bytes < need)
    return bad(QW_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws ? ws_bytes : (size_t)0);
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.k = static_cast<const uint8_t *>(c->k);
  a.v = static_cast<const uint8_t *>(c->v);
  a.ks = c->k_scale;
  a.vs = c->v_scale;
  a.table = b->page_table;
  a.lens = b->seq_lens;
  a.cu = b->cu_tokens;
  a.q_tok = q_token_stride;
  a.q_head = q_head_stride;
  a.page_stride = c->page_stride;
  a.head_stride = c->head_stride;
  a.tok_stride = c->token_stride;
  a.B = b->B;
  a.T = T;
  a.Hq = Hq;
  a.Hkv = c->Hkv;
  a.page = c->page;
  a.npages = c->num_pages;
  a.max_pages = b->max_pages;
  a.cap = b->max_pages * c->page;
  a.window = window < a.cap ? window : 0;        // (a window of all keys is none; and no sum with it overflows)
  a.sinks = a.window > 0 ? sinks : 0;
  a.page_shift = (c->page & (c->page - 1)) == 0 ? 0 : -1;
  while (a.page_shift >= 0 && c->page >> a.page_shift > 1) ++a.page_shift;
  a.strip_pages = c->page % 16 == 0;
  // every item's places, were all contexts as long as the page table: four for each strip of 16
  // keys, and up to 96 more
  long long most = ((long long)T * a.G / cols + b->B) * c->Hkv;
  if (most > (1ll << 28)) return bad(QW_ERR_UNSUPPORTED_SHAPE, "too many query columns");
  const long long blocks = most;
  for (most = blocks * (a.cap / 4 + 128); most > (long long)kPagedMaxPlaces; most = blocks * ((a.cap / 4 >> a.shift) + 128)) {
    if (++a.shift > 24) return bad(QW_ERR_UNSUPPORTED_SHAPE, "too many query columns");
  }
  // A CTA takes 12 places at least: with 6, one context of 1000 keys (8 heads of 128) takes 10.7 us
  // instead of 11.3 but one of 4000 14.8 instead of 13.6 (more parts to join); with 24, 1000 keys of
  // 4 heads of 256 with 12 columns 18.6 instead of 15.4, with 36 columns 22.6 instead of 24.7.
  a.min_places = 12;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.counters = static_cast<int *>(ws);
  a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + kPagedCounterBytes);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = c->dtype == QW_KV_F16    ? launch_attn_paged_f16(a, c->d, cols, sms, st)
                  : c->dtype == QW_KV_BF16 ? launch_attn_paged_bf16(a, c->d, cols, sms, st)
                                           : launch_attn_paged_i8(a, c->d, cols, sms, st);
  if (e != cudaSuccess) return bad(QW_ERR_CUDA, "attention kernel launch: %s", cudaGetErrorString(e));
  return QW_OK;
}

}  // extern "C"
