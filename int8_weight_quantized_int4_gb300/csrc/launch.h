// launch.h -- internal interface between the C ABI (api.cu) and the kernel
// translation units.  Not part of the public ABI.
#pragma once
#include <stdint.h>
#include <stddef.h>
#include <cuda.h>            // CUtensorMap (type only; the driver is reached through the runtime)
#include <cuda_runtime.h>
#include "schedule.h"

namespace qw {

struct GemmArgs {
  CUtensorMap tmap;         // activations: fp16 [M,K] (64 x bn boxes, 128-byte swizzle) or
                            // int8 [M,K] (128 x bn boxes) for W4A8 at decode sizes
  CUtensorMap wmap, smap;   // row-block decode kernel: the packed int4 weights seen as
                            // [row tiles][groups][1056 x 8 B]: boxes of one row block's codes
                            // (1 KB) and scales (32 B) over 8 consecutive groups
  Plan P;
  const float *xs;          // token scales [M] (W4A8) or nullptr
  const uint16_t *xf16;     // W4A8 quantized in the kernel: the fp16 activations [M,K]
  const uint8_t *wpack;     // packed weights
  uint16_t *y;              // fp16 [M,N]
  int *counters;            // [tiles] arrival counters (stream-K)
  float *partials;          // [2*grid][bn][128] binary32 partial sums (stream-K)
  int *err;                 // device error word
  int early_weights;        // weights may be streamed before the preceding kernel ends
  unsigned long long wait_ns;   // time limit of a pipeline wait (QW_OPT_WAIT_LIMIT_US)
  uint32_t *tile_max;       // lm_head with top-k: [M][N/128] the largest order key of each
                            // token's outputs in each 128-row tile (raised with atomicMax),
                            // or nullptr
};

void count_launch();
// QW_OPT_WAIT_LIMIT_US in nanoseconds
unsigned long long wait_limit_ns();
// Record a host-side error for qw_last_error_string(); returns `code`.
int set_last_error(int code, const char *msg);
// Check the current device (sm_103) and return its SM count and the address of its
// device error word; QW_OK or a QW_ERR_* code (recorded for qw_last_error_string()).
int device_info(int *sms, int **err);

// Launch `func` with programmatic stream serialization: it may start while the
// preceding kernel on the stream finishes; every kernel of this library executes
// griddepcontrol.wait before its first global-memory access (the GEMM only
// prefetches weights into L2 before it).
template <typename... Args>
cudaError_t launch_pdl(const void *func, dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                       const Args &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void *argv[] = {const_cast<void *>(static_cast<const void *>(&args))...};
  return cudaLaunchKernelExC(&cfg, func, argv);
}
// Raise the dynamic shared-memory limit of `func` on the current device (once).
cudaError_t ensure_smem_attr(const void *func, int bytes);

// per-token quantizer: codes to q (int8 [M,K], or fp16 [M,K] when codes16), scales to s [M]
cudaError_t launch_quant_act(const uint16_t *x, int M, int K, void *q, bool codes16, float *s,
                             cudaStream_t st);
cudaError_t launch_widen_i8(const int8_t *src, uint16_t *dst, size_t n, int sms, cudaStream_t st);
cudaError_t launch_pack_w4(const int8_t *codes, const uint16_t *scales, int N, int K, void *packed,
                           int *err, int sms, cudaStream_t st);
cudaError_t launch_pack_w8(const int8_t *codes, const uint16_t *scales, int N, int K, void *packed,
                           int sms, cudaStream_t st);

// embedding gather and top-k (gather_topk.cu)
struct TopkPlan {
  int slices, slice_len;
  size_t ws_counters, ws_bytes;
};
constexpr int kTopkMaxN = 64 * 4096;
TopkPlan topk_plan(int M, int N, int k);
cudaError_t launch_embed_gather(const int32_t *ids, int T, const void *packed, int V, int D,
                                uint16_t *out, int *err, cudaStream_t st);
cudaError_t launch_topk(const uint16_t *logits, int M, int N, int k, uint16_t *vals, int32_t *idx,
                        void *ws, cudaStream_t st);
// lm_head with top-k: the k best of each row of y [M, N] from the GEMM's tile maxima
// (tile_max [M][N/128] and counters [M], zero, left zero), kTopkSlices CTAs a row whose
// (key, index) pairs go through `pairs` (topk_tiles_pair_bytes(M) bytes)
constexpr int kTopkSlices = 4;
size_t topk_tiles_pair_bytes(int M);
cudaError_t launch_topk_tiles(const uint16_t *y, int M, int N, int k, uint32_t *tile_max, int *counters,
                              unsigned long long *pairs, uint16_t *vals, int32_t *idx, cudaStream_t st);

// int8-QK causal prefill attention (attention.cu): head dimension and block sizes
constexpr int kAttnD = 256;       // head_dim
constexpr int kAttnBlk = 128;     // queries per block and keys per block
struct AttnLaunch {
  const uint16_t *q, *k, *v;      // [T][Hq][d], [S][Hkv][d], [S][Hkv][d] fp16
  uint16_t *out;                  // [T][Hq][d] fp16
  int T, S, Hq, Hkv;
  long long *part;                // [S/128][Hkv][d] channel partial sums (workspace)
  uint16_t *qc, *kc, *vt;         // [Hq][T][d], [Hkv][S][d] fp16 codes; [Hkv][d][S] fp16 V^T
  float *qs, *ks;                 // [Hq][T], [Hkv][S] row scales
  CUtensorMap tq, tk, tv;         // tensor maps of qc, kc, vt
  int *err;
  unsigned long long wait_ns;
};
size_t attn_fwd_smem_bytes();
cudaError_t launch_attn(const AttnLaunch &L, cudaStream_t st);

// Paged key-value cache (kv_cache.cu, attn_paged*.cu).  Cache types:
enum { kPagedF16 = 0, kPagedBf16 = 1, kPagedI8 = 2 };
constexpr int kPagedMaxCtas = 1024;
constexpr unsigned kPagedMaxPlaces = 1u << 30;   // of all items of a call
// CTAs an SM where there are many items; cols: the columns of an item, 8 or up to 64
constexpr int paged_ctas(int d, int cols) { return cols == 8 ? (d == 256 ? 2 : 4) : d == 64 ? 4 : d == 128 ? 2 : 1; }
struct PagedArgs {
  const uint16_t *q;            // [T][Hq][d], token and head strides q_tok, q_head (elements)
  uint16_t *out;                // [T][Hq][d] dense
  float *lse;                   // [T][Hq] or nullptr
  const uint8_t *k, *v;         // pages: element offset page * page_stride + g * head_stride
  const float *ks, *vs;         //   + row * tok_stride; int8: row scales [pages][Hkv][page]
  const int *table, *lens, *cu; // [B][max_pages], [B], [B + 1]
  long long q_tok, q_head, page_stride, head_stride, tok_stride;
  int B, T, Hq, Hkv, G, page, npages, max_pages;
  int cap;                      // keys the page table can name: max_pages * page
  int window, sinks;            // window 0: every key up to the position; sinks 0 without one
  int page_shift;               // log2(page), -1 where page is no power of two
  int strip_pages;              // page % 16 == 0: a strip of 16 keys lies in one page
  int shift;                    // the schedule counts places (a strip of 16 keys for a block of columns) in 2^shift
  int min_places;               // fewest of those units a CTA takes
  float scale_log2;             // softmax scale * log2(e)
  float *part;                  // [CTAs][2][rows (d + 2)] partial sums (workspace)
  int *counters;                // [kPagedMaxCtas] arrivals of an item's groups of parts, then [kPagedMaxCtas][2]
                                //   of a group's parts; zero between calls (workspace)
  int *err;
};
cudaError_t launch_attn_paged_f16(const PagedArgs &a, int d, int cols, int sms, cudaStream_t st);
cudaError_t launch_attn_paged_bf16(const PagedArgs &a, int d, int cols, int sms, cudaStream_t st);
cudaError_t launch_attn_paged_i8(const PagedArgs &a, int d, int cols, int sms, cudaStream_t st);

// Attention of trees over the paged cache (attn_tree*.cu)
constexpr unsigned kTreeMaxPlaces = 4000000000u;   // of all items of a call (sums of 32 bits)
struct TreeDesc {               // an item that several CTAs share, left by the first of them
  int tok0, col0, cols, g;      // its first row in q, first column, columns (0: none), KV head
  int parts, step;              // parts; CTAs from one to the next
};
struct TreeArgs {
  CUtensorMap qmap, kmap, vmap; // rows of d elements, boxes of 64 elements (int8: d) and one row
  CUtensorMap kbox, vbox;       // [pages][Hkv][page][d], boxes of 64 elements (int8: d) and `box` rows
  int box;                      // 0: gathers (pages of no multiple of 8 rows, a broadcast cache, no pages)
  CUtensorMap qbox;             // [T][Hkv][G][d], boxes of 64 elements and block_rows rows (G <= 128)
  int scale_boxes;              // int8: a box's scales are a multiple of 16 bytes, so aligned
  int block_rows;               // rows of an item: whole nodes (q_box), or 128
  int q_box;
  const uint16_t *q;            // as PagedArgs
  uint16_t *out;
  float *lse;
  const float *ks, *vs;
  const int *table, *lens, *cu, *parents;
  long long q_tok, q_head;
  int q_tok_rows, q_head_rows;  // strides in rows of the maps
  int page_rows, head_rows, tok_rows;
  int B, T, Hq, Hkv, G, page, npages, max_pages, cap, window, sinks, page_shift;
  int max_nodes, blocks;        // row blocks of a sequence of max_nodes
  float scale_log2;
  float *part;                  // [CTAs][2][128 (d + 2)] partial sums (workspace)
  TreeDesc *desc;               // [CTAs] (workspace)
  int *err;
  unsigned long long wait_ns;
};
// A tensor map of `rows` rows of d elements `pitch` bytes apart, in boxes of one row (int8: whole
// rows, unswizzled; 16 bits: 64 elements, 128-byte swizzle), for gathers.
int encode_row_map(CUtensorMap *map, const void *base, long long rows, int d, long long pitch, bool int8, bool bf16);
// [dim[2]][dim[1]][dim[0]][d] (strides in bytes), in boxes of `box` by 1 by `box2` rows: the cache as
// pages, heads and tokens, q as nodes, KV heads and the heads of each.
int encode_page_map(CUtensorMap *map, const void *base, const long long (&dim)[3], const long long (&stride)[3], int d, int box,
                    int box2, bool int8, bool bf16);
// CTAs an SM: TMEM holds O and two buffers of scores of two CTAs up to d = 128
constexpr int tree_ctas(int d) { return d == 256 ? 1 : 2; }
__host__ __device__ constexpr size_t tree_part_floats(int d) { return (size_t)128 * (d + 2); }
cudaError_t launch_attn_tree_f16(const TreeArgs &a, int d, int grid, cudaStream_t st);
cudaError_t launch_attn_tree_bf16(const TreeArgs &a, int d, int grid, cudaStream_t st);
cudaError_t launch_attn_tree_i8(const TreeArgs &a, int d, int grid, cudaStream_t st);

cudaError_t launch_gemm_w4a16(const GemmArgs &a, cudaStream_t st);
// W4A8 (token scales in the epilogue): act8, int8 codes widened in the kernel (token
// tiles up to kAct8InKernelMaxBn); otherwise fp16 codes read as fp16 tiles
cudaError_t launch_gemm_w4a8(const GemmArgs &a, bool act8, cudaStream_t st);
cudaError_t launch_gemm_w8a16(const GemmArgs &a, cudaStream_t st);
// decode batches (plan.ms_teams > 0); act: 0 fp16 activations (W4A16), 1 int8 codes and
// token scales (W4A8), 2 fp16 codes and token scales (W4A8 after the quantizer)
cudaError_t launch_gemm_ms(const GemmArgs &a, int act, cudaStream_t st);
// decode batches on layers of few rows (plan.rb_max > 0): the row-block kernel, act as above
// or 3: fp16 activations quantized per token in the kernel (plan.fused)
cudaError_t launch_gemm_rb(const GemmArgs &a, int act, cudaStream_t st);

}  // namespace qw
