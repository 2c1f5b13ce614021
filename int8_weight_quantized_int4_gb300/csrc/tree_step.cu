// tree_step.cu -- what follows the attention and the draws of a verify step over trees of
// drafted tokens: the path that the draws accept, and its rows moved together in the cache.
//
// tree_accept, for the nodes of a sequence (parents p, tokens w, the tokens d drawn at the
// nodes): the path starts at node 0; from node c it goes on to the first child i (p_i = c) whose
// token is the one drawn, w_i = d_c, and ends where there is none.
//
// kv_keep_path, for the path a_0 < a_1 < ..: the row of slot s + a_i becomes the row of slot
// s + i (s the slot of node 0), in every layer and pool.  Since a_i >= i and the a_i ascend, a
// slot is written only after every row that comes from it was read, if each thread takes its
// 16 bytes of all rows in order.
//
// Both are chains of a few dependent reads: latency bounds them, and HBM the largest moves.
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>
#include "launch.h"
#include "ptx.cuh"
#include "qgemm.h"

namespace qw {

// ------------------------------------------------------------------- accept --
struct AcceptArgs {
  const int *tokens, *drawn, *parents, *cu;
  int *path, *count, *next;
  int B, T, width;
  int *err;
};
constexpr int kAcceptWarps = 4;
constexpr int kAcceptHeld = 4;                   // nodes a lane holds in registers

// One warp a sequence; a lane holds nodes lane, lane + 32, .. (128 in registers, later ones
// are read again at every step), so a step down the tree is a vote and a shuffle.
__global__ void __launch_bounds__(32 * kAcceptWarps) tree_accept_kernel(const __grid_constant__ AcceptArgs a) {
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.x * kAcceptWarps + (threadIdx.x >> 5);
  griddep_wait();
  griddep_launch_dependents();
  if (b >= a.B) return;                          // whole warp
  const int c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1);
  const int t0 = min(max(c0, 0), a.T), n = max(min(max(c1, 0), a.T) - t0, 0);
  if ((c0 != t0 || c1 != t0 + n) && lane == 0) atomicCAS(a.err, 0, -9);
  int par[kAcceptHeld], tok[kAcceptHeld], drw[kAcceptHeld];
#pragma unroll
  for (int k = 0; k < kAcceptHeld; ++k) {
    const int i = 32 * k + lane;
    par[k] = -1;
    tok[k] = drw[k] = 0;
    if (i < n) {
      par[k] = __ldg(a.parents + t0 + i);
      tok[k] = __ldg(a.tokens + t0 + i);
      drw[k] = __ldg(a.drawn + t0 + i);
    }
  }
  bool odd = false;
#pragma unroll
  for (int k = 0; k < kAcceptHeld; ++k) odd |= par[k] < -1 || par[k] >= max(32 * k + lane, 0);
  for (int i = 32 * kAcceptHeld + lane; i < n; i += 32) {
    const int p = __ldg(a.parents + t0 + i);
    odd |= p < -1 || p >= i;
  }
  if (__any_sync(0xffffffffu, odd) && lane == 0) atomicCAS(a.err, 0, -9);

  int *path = a.path + (long long)b * a.width;
  int len = 0, cur = n > 0 ? 0 : -1, last = -1;
  int mine = -1;                                 // the path's entry 32 j + lane of the block being filled
  while (cur >= 0 && len < a.width) {
    if (lane == (len & 31)) mine = cur;
    ++len;
    if ((len & 31) == 0) {
      path[len - 32 + lane] = mine;
      mine = -1;
    }
    int want = 0;
    if (cur < 32 * kAcceptHeld) {
#pragma unroll
      for (int k = 0; k < kAcceptHeld; ++k) {
        const int x = __shfl_sync(0xffffffffu, drw[k], cur & 31);
        if (cur >> 5 == k) want = x;
      }
    } else {
      want = __ldg(a.drawn + t0 + cur);
    }
    last = want;
    int found = -1;                              // a child comes after its parent
#pragma unroll
    for (int k = 0; k < kAcceptHeld; ++k) {
      const unsigned v = __ballot_sync(0xffffffffu, 32 * k + lane > cur && par[k] == cur && tok[k] == want);
      if (v && found < 0) found = 32 * k + __ffs(v) - 1;
    }
    for (int i = max(32 * kAcceptHeld, cur & ~31); found < 0 && i < n; i += 32) {
      const int j = i + lane;
      const bool hit = j < n && j > cur && __ldg(a.parents + t0 + j) == cur && __ldg(a.tokens + t0 + j) == want;
      const unsigned v = __ballot_sync(0xffffffffu, hit);
      if (v) found = i + __ffs(v) - 1;
    }
    cur = found;
  }
  for (int i = (len & ~31) + lane; i < a.width; i += 32) {
    path[i] = mine;
    mine = -1;
  }
  if (lane == 0) {
    a.count[b] = len;
    a.next[b] = last;
  }
}

// ---------------------------------------------------------------- keep path --
constexpr int kMaxRowPools = 4;
struct KeepPool {
  uint8_t *base;
  long long layer_stride, page_stride, head_stride, token_stride;      // bytes
  int npages, heads, vecs;                       // vectors of a row
  int wide;                                      // vectors of 16 bytes, else 4
  int first;                                     // its first warp of a sequence
  int columns;                                   // layers x heads x vecs
};
struct KeepArgs {
  KeepPool pool[kMaxRowPools];
  const int *path, *count, *table, *lens, *cu;
  int *new_lens;
  int npools, warps;                             // warps of a sequence
  int B, T, width, page, max_pages;
  int *err;
};
constexpr int kKeepWarps = 8;
// Rows in flight a lane.  Warps, not rows, hide the latency: with 8 rows and 100 registers 23 % of
// an SM's warps were active and 64 sequences of 48 int8 layers (62 MB in all) took 33 us, now 18.1.
// (2 rows: 17, and twice the round trips of a long path.)
constexpr int kKeepRows = 4;

// Moves a lane's column of the rows that lanes hold offsets of (from: -1 none), in the lanes' order.
template <typename V>
__device__ __forceinline__ void move_rows(uint8_t *at, bool on, long long from, long long to) {
  unsigned left = __ballot_sync(0xffffffffu, from >= 0);
  while (left) {
    V r[kKeepRows];
    unsigned rows = left;
#pragma unroll
    for (int k = 0; k < kKeepRows; ++k) {
      const long long x = __shfl_sync(0xffffffffu, from, (__ffs(rows) - 1) & 31);
      if (on && rows) r[k] = *reinterpret_cast<const V *>(at + x);
      rows &= rows - 1;
    }
#pragma unroll
    for (int k = 0; k < kKeepRows; ++k) {
      const long long x = __shfl_sync(0xffffffffu, to, (__ffs(left) - 1) & 31);
      if (on && left) *reinterpret_cast<V *>(at + x) = r[k];
      left &= left - 1;
    }
  }
}

// One warp 32 columns of a sequence: a column is 16 bytes (4 for scales) of a row's bytes in one
// layer and head.  Lane i looks up the i-th row's slots; kKeepRows rows are read before they are written.
__global__ void __launch_bounds__(32 * kKeepWarps, 4) kv_keep_kernel(const __grid_constant__ KeepArgs a) {
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * kKeepWarps + (threadIdx.x >> 5);
  griddep_wait();
  griddep_launch_dependents();
  const int b = (int)(w / a.warps);
  if (b >= a.B) return;                          // whole warp
  const int unit = (int)(w - (long long)b * a.warps);
  const int c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1), len = __ldg(a.lens + b), cnt = __ldg(a.count + b);
  const int *path = a.path + (long long)b * a.width;
  int src = lane < a.width ? __ldg(path + lane) : 0;      // (wanted for most calls, whatever the count)
  const int t0 = min(max(c0, 0), a.T), n = max(min(max(c1, 0), a.T) - t0, 0);
  const int m = min(max(cnt, 0), min(a.width, n));
  const int pos0 = len - n;                      // the slot of node 0
  if (unit == 0 && lane == 0) {
    if (a.new_lens) a.new_lens[b] = pos0 + m;
    if (c0 != t0 || c1 != t0 + n || m != cnt || pos0 < 0) atomicCAS(a.err, 0, -9);
  }
  if (a.npools == 0) return;
  int p = 0;
  while (p + 1 < a.npools && unit >= a.pool[p + 1].first) ++p;
  const KeepPool &q = a.pool[p];
  const int col = (unit - q.first) * 32 + lane;
  const bool on = col < q.columns;
  const int row = on ? col / q.vecs : 0, layer = on ? row / q.heads : 0;
  uint8_t *at = q.base + layer * q.layer_stride + (row - layer * q.heads) * q.head_stride + (col - row * q.vecs) * (q.wide ? 16 : 4);
  int before = -1;                               // the previous block's last entry
  for (int i0 = 0; i0 < m; i0 += 32) {
    const int i = i0 + lane;
    if (i0 > 0) src = i < a.width ? __ldg(path + i) : 0;
    int prev = __shfl_up_sync(0xffffffffu, src, 1);
    if (lane == 0) prev = before;
    before = __shfl_sync(0xffffffffu, src, 31);
    int sp = -1, so = 0, dp = -1, dof = 0;      // pages and rows of them
    long long from = -1, to = 0;
    if (i < m) {
      const long long s = (long long)pos0 + src, d = (long long)pos0 + i;
      const bool fine = src > prev && src >= i && src < n && pos0 >= 0;
      const bool moves = fine && src != i;        // (a row in its place stays)
      const int ps = (int)(s / a.page), pd = (int)(d / a.page);
      if (moves && ps < a.max_pages) {
        sp = __ldg(a.table + (long long)b * a.max_pages + ps);
        dp = __ldg(a.table + (long long)b * a.max_pages + pd);
        so = (int)(s - (long long)ps * a.page);
        dof = (int)(d - (long long)pd * a.page);
      }
      if (!fine || (moves && ((unsigned)sp >= (unsigned)q.npages || (unsigned)dp >= (unsigned)q.npages))) {
        atomicCAS(a.err, 0, -9);
      } else if (moves) {
        from = sp * q.page_stride + so * q.token_stride;
        to = dp * q.page_stride + dof * q.token_stride;
      }
    }
    if (q.wide) move_rows<uint4>(at, on, from, to);
    else move_rows<uint32_t>(at, on, from, to);
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

// A pool's rows start at base + sum i_k stride_k, i_k < n_k: its dimensions of several entries, the
// largest stride first.
struct RowDims {
  int count;
  long long n[4], stride[4];
};
RowDims row_dims(const qw_row_pool_t &p, int page) {
  const long long n[4] = {p.layers, p.num_pages, p.heads, page}, s[4] = {p.layer_stride, p.page_stride, p.head_stride, p.token_stride};
  RowDims d{};
  for (int i = 0; i < 4; ++i) {
    if (n[i] < 2) continue;
    int k = d.count++;
    for (; k > 0 && d.stride[k - 1] < s[i]; --k) {
      d.n[k] = d.n[k - 1];
      d.stride[k] = d.stride[k - 1];
    }
    d.n[k] = n[i];
    d.stride[k] = s[i];
  }
  return d;
}
typedef __int128 wide;                            // (products of sizes and strides pass 64 bits)
wide row_span(const RowDims &d, int from, long long row) {
  wide span = row;
  for (int i = from; i < d.count; ++i) span += (wide)(d.n[i] - 1) * d.stride[i];
  return span;
}
// Rows that overlap: strides that do not nest, each at least what the smaller ones span.
bool rows_overlap(const RowDims &d, long long row) {
  for (int i = 0; i < d.count; ++i)
    if (d.stride[i] < row_span(d, i + 1, row)) return true;
  return false;
}
// Whether x + sum k_i stride_i lies between -below and above (both excluded) for some lo_i <= k_i <= hi_i:
// the largest stride's k_i are those from which the others' reach it, one to three where strides nest.
struct RowGap {
  int count;
  long long lo[8], hi[8], stride[8];
  long long below, above;
  int left;                                       // more steps than these count as found
};
bool row_meets(RowGap &g, wide x, int i) {
  if (--g.left < 0) return true;
  wide least = 0, most = 0;                       // of what the later ones add
  for (int k = i + 1; k < g.count; ++k) {
    least += (wide)g.lo[k] * g.stride[k];
    most += (wide)g.hi[k] * g.stride[k];
  }
  if (i >= g.count) return x > -(wide)g.below && x < (wide)g.above;
  const wide s = g.stride[i];
  auto down = [&](wide a) { return a / s - (a % s != 0 && a < 0); };      // floor(a / s)
  const wide from = -down(x + g.below - 1 + most), to = down(g.above - 1 - x - least);
  for (wide k = from < g.lo[i] ? (wide)g.lo[i] : from; k <= g.hi[i] && k <= to; ++k)
    if (row_meets(g, x + k * s, i + 1)) return true;
  return false;
}
// Pools that share bytes of a row, or are laced in a way that 65536 steps do not tell apart.
bool pools_meet(const qw_row_pool_t &p, const RowDims &a, const qw_row_pool_t &q, const RowDims &b) {
  const wide x = (wide)reinterpret_cast<uintptr_t>(p.base) - (wide)reinterpret_cast<uintptr_t>(q.base);
  if (x + row_span(a, 0, p.row_bytes) <= 0 || x >= row_span(b, 0, q.row_bytes)) return false;
  RowGap g{0, {}, {}, {}, p.row_bytes, q.row_bytes, 65536};
  for (int i = 0, j = 0; i < a.count || j < b.count;) {       // equal strides together, largest first
    const bool first = j >= b.count || (i < a.count && a.stride[i] >= b.stride[j]);
    const bool both = first && j < b.count && a.stride[i] == b.stride[j];
    g.stride[g.count] = first ? a.stride[i] : b.stride[j];
    g.hi[g.count] = first ? a.n[i] - 1 : 0;
    g.lo[g.count] = !first || both ? 1 - b.n[j] : 0;
    ++g.count;
    i += first;
    j += !first || both;
  }
  return row_meets(g, x, 0);
}
}  // namespace
}  // namespace qw

using namespace qw;

extern "C" {

int tree_accept(const int32_t *tokens, const int32_t *drawn, const int32_t *parents, const int32_t *cu_tokens, int B,
                int T, int max_path, int32_t *path, int32_t *count, int32_t *next_token, qw_stream_t stream) {
  if (B < 0 || T < 0) return bad(QW_ERR_INVALID_ARG, "negative size");
  if (max_path < 1) return bad(QW_ERR_INVALID_ARG, "max_path must be positive");
  if (B == 0) return QW_OK;
  if (!cu_tokens || !path || !count || !next_token || (T > 0 && (!tokens || !drawn || !parents)))
    return bad(QW_ERR_INVALID_ARG, "null tensor pointer");
  if (!at(tokens, 4) || !at(drawn, 4) || !at(parents, 4) || !at(cu_tokens, 4) || !at(path, 4) || !at(count, 4) ||
      !at(next_token, 4))
    return bad(QW_ERR_ALIGNMENT, "int32 arrays must be 4-byte aligned");
  AcceptArgs a{tokens, drawn, parents, cu_tokens, path, count, next_token, B, T, max_path, nullptr};
  int rc = device_info(nullptr, &a.err);
  if (rc) return rc;
  cudaError_t e = launch_pdl(reinterpret_cast<const void *>(tree_accept_kernel),
                             dim3((unsigned)(((long long)B + kAcceptWarps - 1) / kAcceptWarps)), dim3(32 * kAcceptWarps), 0,
                             reinterpret_cast<cudaStream_t>(stream), a);
  count_launch();
  if (e != cudaSuccess) return bad(QW_ERR_CUDA, "accept kernel launch: %s", cudaGetErrorString(e));
  return QW_OK;
}

int kv_keep_path(const qw_row_pool_t *pools, int n_pools, const qw_kv_batch_t *batch, int T, int page,
                 const int32_t *path, const int32_t *count, int max_path, int32_t *new_lens, qw_stream_t stream) {
  if (n_pools < 0 || n_pools > kMaxRowPools) return bad(QW_ERR_INVALID_ARG, "zero to %d pools", kMaxRowPools);
  if (n_pools > 0 && !pools) return bad(QW_ERR_INVALID_ARG, "null pools");
  if (!batch) return bad(QW_ERR_INVALID_ARG, "null batch");
  if (batch->B < 0 || batch->max_pages < 0 || T < 0 || max_path < 0) return bad(QW_ERR_INVALID_ARG, "negative size");
  if (page < 1) return bad(QW_ERR_INVALID_ARG, "page must be positive");
  if (page > (1 << 20)) return bad(QW_ERR_UNSUPPORTED_SHAPE, "page <= 2^20");
  if ((long long)batch->max_pages * page > (1ll << 30))
    return bad(QW_ERR_UNSUPPORTED_SHAPE, "a page table names at most 2^30 keys");
  KeepArgs a{};
  long long warps = 0;
  RowDims dims[kMaxRowPools];
  const qw_row_pool_t *given[kMaxRowPools];
  for (int i = 0; i < n_pools; ++i) {
    const qw_row_pool_t &p = pools[i];
    if (p.layers < 0 || p.num_pages < 0 || p.heads < 0 || p.row_bytes < 0 || p.layer_stride < 0 || p.page_stride < 0 ||
        p.head_stride < 0 || p.token_stride < 0)
      return bad(QW_ERR_INVALID_ARG, "negative pool size");
    if (p.row_bytes % 4 || p.row_bytes > (1 << 20))
      return bad(QW_ERR_UNSUPPORTED_SHAPE, "a row is a multiple of 4 bytes, at most 2^20");
    if (p.layers == 0 || p.heads == 0 || p.row_bytes == 0 || p.num_pages == 0) continue;
    if (!p.base) return bad(QW_ERR_INVALID_ARG, "null pool pointer");
    if (!at(p.base, 4) || p.layer_stride % 4 || p.page_stride % 4 || p.head_stride % 4 || p.token_stride % 4)
      return bad(QW_ERR_ALIGNMENT, "rows start on 4-byte boundaries");
    KeepPool &q = a.pool[a.npools];
    q.base = static_cast<uint8_t *>(p.base);
    q.layer_stride = p.layer_stride;
    q.page_stride = p.page_stride;
    q.head_stride = p.head_stride;
    q.token_stride = p.token_stride;
    q.npages = p.num_pages;
    q.heads = p.heads;
    q.wide = at(p.base, 16) && p.layer_stride % 16 == 0 && p.page_stride % 16 == 0 && p.head_stride % 16 == 0 &&
             p.token_stride % 16 == 0 && p.row_bytes % 16 == 0;
    q.vecs = p.row_bytes / (q.wide ? 16 : 4);
    const long long columns = (long long)p.layers * p.heads * q.vecs;
    if (columns > (1ll << 30)) return bad(QW_ERR_UNSUPPORTED_SHAPE, "too many rows a token");
    dims[a.npools] = row_dims(p, page);
    if (rows_overlap(dims[a.npools], p.row_bytes)) return bad(QW_ERR_INVALID_ARG, "rows overlap: a stride below what the smaller ones span");
    for (int j = 0; j < a.npools; ++j)
      if (pools_meet(p, dims[a.npools], *given[j], dims[j])) return bad(QW_ERR_INVALID_ARG, "pools %d and %d share rows", (int)(given[j] - pools), i);
    given[a.npools++] = &p;
    q.columns = (int)columns;
    q.first = (int)warps;
    warps += (columns + 31) / 32;
  }
  if (batch->B == 0) return QW_OK;
  if (!path || !count || !batch->page_table || !batch->seq_lens || !batch->cu_tokens)
    if (a.npools > 0 || new_lens) return bad(QW_ERR_INVALID_ARG, "null batch pointer");
  if (!at(path, 4) || !at(count, 4) || !at(batch->page_table, 4) || !at(batch->seq_lens, 4) || !at(batch->cu_tokens, 4) ||
      !at(new_lens, 4))
    return bad(QW_ERR_ALIGNMENT, "int32 arrays must be 4-byte aligned");
  if (new_lens && new_lens == batch->seq_lens) return bad(QW_ERR_INVALID_ARG, "new_lens is the batch's seq_lens");
  if (a.npools == 0 && !new_lens) return QW_OK;
  a.warps = (int)(warps > 0 ? warps : 1);
  const long long grid = ((long long)a.warps * batch->B + kKeepWarps - 1) / kKeepWarps;
  if (grid > 0x7fffffffll) return bad(QW_ERR_UNSUPPORTED_SHAPE, "too many rows for one call");
  int rc = device_info(nullptr, &a.err);
  if (rc) return rc;
  a.path = path;
  a.count = count;
  a.table = batch->page_table;
  a.lens = batch->seq_lens;
  a.cu = batch->cu_tokens;
  a.new_lens = new_lens;
  a.B = batch->B;
  a.T = T;
  a.width = max_path;
  a.page = page;
  a.max_pages = batch->max_pages;
  cudaError_t e = launch_pdl(reinterpret_cast<const void *>(kv_keep_kernel), dim3((unsigned)grid), dim3(32 * kKeepWarps), 0,
                             reinterpret_cast<cudaStream_t>(stream), a);
  count_launch();
  if (e != cudaSuccess) return bad(QW_ERR_CUDA, "keep kernel launch: %s", cudaGetErrorString(e));
  return QW_OK;
}

}  // extern "C"
