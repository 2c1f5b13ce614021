// attn_tree.cuh -- attention of the nodes of trees of drafted tokens over a paged key-value cache.
//
// A sequence of length n whose last m positions hold the nodes of a tree: with s = n - m, node r at
// depth e (its ancestors) stands at position s + e and sees the keys j < s and those of its
// ancestors and itself (with a window W only positions above s + e - W or below `sinks`).  For head h
// of a node and KV head g = h / G,
//   x_j = q . k_j * scale,  p_j = e^(x_j - m),  out = sum_j p_j v_j / sum_j p_j.
//
// The G heads and m nodes that share a KV head are the rows of a 128-row tile, tiles of 64 keys
// stream past it: S = Q K^T and O += P V on tcgen05, S and O in TMEM, a row a thread in the
// softmax.  Reading K and V takes 4 D bytes a key (int8: 2 D) for 128 x 2 x 3 D flops (P enters P V as
// two 16-bit terms, below) whatever rows a small tree fills: 192 flops a byte a row block, int8 384, where
// the ridge lies at 281.  So HBM can bound one 16-bit row block alone; it does at d = 128 (74 % of its copy
// rate), while at d = 256, with several blocks and with int8 the softmax of a tile comes first.
//
// Roles of a CTA's warps: 8 of softmax (two groups that take tiles in turn), 1 issuing MMAs, 1 loading
// (d = 256: 2) and for an int8 cache 2 or 4 that widen codes to fp16 (exact).  Rings of K and of V
// tiles, each 64 rows: the scores of the next tile are computed while the softmax works on the last.
//   - Rows come by TMA straight to the 128-byte swizzle: pages of a multiple of 8 rows in boxes of up
//     to 64, other pages four rows a gather, from a map of rows one common divisor of the cache's
//     strides apart (rows outside it are zeros).  (Gathers move 6 to 9 bytes a clock an SM; cp.async
//     by two warps a CTA moved 10.)  Boxes without a row that a node sees are not read.  K is the K-major
//     operand and V, as it lies, the MN-major one, so nothing is transposed.
//   - P goes back into TMEM over the scores it came from.
//   - O is rescaled only when a score passes the reference by 2^8 (fp16: 2^15).
//   - A tile that some rows see partly gets a 64-bit mask a row: the window's and the length's
//     borders, and the bits of the row's ancestors (found by walking the parents once an item).
//
// Work: the tiles of every (sequence, KV head, block of 128 rows) item are laid end to end and cut into
// one equal range a CTA; an item that a border cuts leaves (m, l, O) parts in the workspace, which a
// second kernel joins.  Where sequences have several row blocks, teams of CTAs run one range, a
// row block each (tree_schedule).
//
// Measured (a graph of calls, inputs larger than L2): 40 contexts of up to 8190, 24 nodes of 32/8 heads
// of 128, bf16: 117 us, 585 MB, 74 % of the copy rate of HBM.  12 of up to 16384, 64 nodes of 24/4
// heads of 256, fp16: 197 us; a full row block's tile takes 2730 cycles, of which the MMAs are 1930
// (two terms of P), and the softmax of a tile bounds it.  5 of up to 65535 int8, 13 nodes: 155 us, 376
// MB: the same softmax, with scales, and shared memory (codes in, halves out, halves read) bound it.
//
// Roundings: each weight enters P V as two terms of the values' 16-bit type, p rounded and what
// that leaves, so the products keep 22 bits of it (bf16: 16), all sums are binary32 and the output's
// rounding is what remains.  In fp16 the reference starts 2^7 below the largest score, so that
// only weights below 2^-32 of it are lost.  With the int8 cache the value's scale joins its weight.
#pragma once
#include <stdint.h>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "launch.h"
#include "ptx.cuh"

namespace qw {

constexpr int kTreeKeys = 64;                     // keys of a tile
constexpr int kTreeRows = 128;                    // rows (columns of a KV head: node x head) of an item
constexpr int kTreeSegs = 16;                     // segments listed at a time
constexpr int kTreeMaxTeam = 4;
constexpr float kTreeNoScore = -3.402823466e38f;

struct TreeSeg {
  int b, g, rb;                                   // sequence, KV head, row block
  int u0, u1;                                     // tiles [u0, u1) of the item's
  int nsu, first;                                 // tiles of the sinks, tile of the first windowed key
  int lo, len, pos0;                              // keys [lo, len) and below `sinks`; the slot of node 0
  int tok0, nodes;
  int slot;                                       // -1: the whole item; 0: begins inside it; 1: begins it
  int parts;
};

struct TreeCtl {
  int nseg, more, member, size;                   // size: CTAs of a team
  int b, cost, all;                               // cost: what an item takes beside its tiles; all: one class alone
  unsigned off, pos, begin, end, share;
  unsigned part[16][kTreeMaxTeam], bare[16];
  unsigned long long bad[2];                      // keys of a group's tile whose values are not finite
  int zeroed;                                     // the segment (counted from 1) whose O was cleared before its first P V
};

template <int D, int KV>
struct TreeShape {
  static constexpr bool kI8 = KV == kPagedI8;
  static constexpr int kWideners = !kI8 ? 0 : D == 256 ? 4 : 2;
  static constexpr int kLoaders = D == 256 ? 2 : 1;       // two: one for K and Q, one for V
  static constexpr int kMmaWarp = 8, kLoadWarp = 9, kWiden0 = kLoadWarp + kLoaders;
  static constexpr int kWarps = kWiden0 + kWideners;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kCtas = tree_ctas(D);
  static constexpr int kStage = kTreeKeys * D * 2;
  // tiles of K, and of V, in shared memory: rings of their own, each filled in the tiles' order by one
  // warp and emptied by another, so that a wait's parity names one phase
  static constexpr int kTiles = kI8 ? (D == 128 ? 1 : 2) : D == 64 ? 4 : D == 256 ? 3 : 2;
  static constexpr int kRaw = kI8 ? kTreeKeys * D : 0;                // a stage of codes
  static constexpr int kRawK = !kI8 ? 0 : D == 64 ? 4 : 2, kRawV = kRawK;
  static constexpr int kScaleSlots = D == 64 ? 16 : D == 128 ? 6 : 8;     // tiles whose scales are kept (more than can be under way)
  // d = 256 (one CTA an SM): Q in TMEM.  From shared memory it would be read again for every 64 keys,
  // 64 KB beside the tile's 64, and shared memory's bandwidth bound the tile (Q there: 194 us for 12 x
  // 16k of 64 nodes); and it leaves 64 KB for tiles.
  static constexpr bool kQTmem = D == 256;
  static constexpr int kQ = kQTmem ? 0 : kTreeRows * D * 2;
  static constexpr int kAhead = 1, kBufs = kAhead + 1;    // tiles whose scores are computed before P V of one
  static constexpr uint32_t kTmem = D == 256 ? 512 : 256;
  static constexpr uint32_t kQCol = D, kSCol = kQTmem ? D + D / 2 : D;    // O [0, D), Q, then kBufs buffers of 64 columns of S and P
  static constexpr int kScaleBytes = kI8 ? kScaleSlots * kTreeKeys * 16 : 0;
  static constexpr int kMaskWords = 9;            // a row's ancestors (256 bits) and the first key of its window
  // barriers, parents, masks, an exchange between the groups, the segments
  static constexpr int kFixed = 512 + 512 + kTreeRows * kMaskWords * 4 + 4 * kTreeRows * 4 + kTreeSegs * (int)sizeof(TreeSeg) +
                                (int)sizeof(TreeCtl) + 64;
  static constexpr int kSmem = 1024 + kQ + 2 * kTiles * kStage + (kRawK + kRawV) * kRaw + kScaleBytes + kFixed;
  static_assert(kSmem * kCtas + 1024 * kCtas <= 228 * 1024 && kSmem <= 227 * 1024, "shared memory");
  static_assert(kAhead + kTiles + kRawK + 2 <= kScaleSlots, "scales outlive their use");
  // What an item costs beside its tiles, in tiles: about the time of 192 KB.  (us with none, 96, 192 and 384
  // KB: 40 x 8k bf16, 24 nodes 145, 115, 117, 121; with d = 64 117, 87, 92, 104; 12 x 16k fp16, 64 nodes 165, 201,
  // 196, 188; with d = 128 115, 114, 113, 116; 1 x 10k 32, 35, 27, 31; 40 windows of 1k 82, 56, 56, 55.)
  static constexpr int kItemCost = 196608 / (2 * kStage / (kI8 ? 2 : 1));
};

// Pairs of binary32, two to an instruction.
struct F2 {
  unsigned long long v;
  __device__ __forceinline__ F2() {}
  __device__ __forceinline__ F2(float x, float y) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y)); }
  __device__ __forceinline__ void get(float &x, float &y) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
};
struct alignas(16) F4 {
  F2 a, b;
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
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// mbar_wait without a call: one would keep a role's values in memory around it.
__device__ __forceinline__ bool tree_wait(uint32_t bar, uint32_t parity, volatile WaitBlock *w, bool no_limit) {
  if (no_limit ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    if (w->abort) return false;
    if (globaltimer_ns() - t0 >= w->limit_ns) {
      w->abort = 1;
      atomicCAS(w->err, 0, -7);
      return false;
    }
    if (mbar_try_wait_sleep(bar, parity)) return true;
  }
}

__device__ __forceinline__ float tree_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float tree_lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// arrive on `bar` when the thread's cp.async copies so far have landed (counted as one arrival)
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// Four rows of a 2-D tensor map (box one row high), row after row, from column x; rows outside the
// tensor are zero-filled.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const void *tmap, int x, const int (&r)[4], uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(bar)
      : "memory");
}
// The box at (x, y, z, w) of a 4-D tensor map.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void *tmap, int x, int y, int z, int w, uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void cp_async4_zfill(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// 32 bytes: a whole sector from one thread
__device__ __forceinline__ void st_global_v8(void *p, const uint32_t (&r)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
               "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// MN-major operand in the 128-byte swizzle: 128-byte rows of 64 channels, a row a key; groups of
// eight keys 1024 bytes apart, the next 64 channels a tile of keys further.
__device__ __forceinline__ uint64_t smem_desc_sw128_mn(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFF);
  d |= (uint64_t)(kTreeKeys * 128 >> 4) << 16;     // leading byte offset: along the channels
  d |= (uint64_t)(1024 >> 4) << 32;                // stride byte offset: along the keys
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
// Instruction descriptor, kind::f16: D fp32, A and B both fp16 or both bf16, B MN-major or not.
// (bit 13 negates A.)
__host__ __device__ constexpr uint32_t tree_idesc(bool bf, bool b_mn, int M, int N) {
  return (1u << 4) | (bf ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}
template <bool BF>
__device__ __forceinline__ uint32_t tree_pack(float x, float y) {
  if constexpr (BF) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&v);
  } else {
    return h2_as_u32(__floats2half2_rn(x, y));
  }
}
template <bool BF>
__device__ __forceinline__ float2 tree_unpack(uint32_t w) {
  if constexpr (BF) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  else return __half22float2(u32_as_h2(w));
}
// Two int8 codes of a word (xor 0x80 applied: code + 128) as fp16: 0x6400 | u is 1024 + u.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t tree_widen(uint32_t u) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(u), "r"(0x64646464u), "n"(SEL));
  return h2_as_u32(__hsub2(u32_as_h2(r), u32_as_h2(0x64806480u)));
}

// --------------------------------------------------------------- the schedule --
struct TreeSeq {
  int tok0, nodes, len;
  bool descends;                                  // its offsets do: its rows may be other sequences' too
};
// Sequence b's nodes and keys, clamped to what the buffers hold.
__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs &a, int b) {
  TreeSeq s;
  const int c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1), n = __ldg(a.lens + b);
  s.tok0 = min(max(c0, 0), a.T);
  s.nodes = max(min(max(c1, 0), a.T) - s.tok0, 0);
  s.descends = c1 < c0;
  s.len = min(max(n, 0), a.cap);
  if (c0 != s.tok0 || c1 != s.tok0 + s.nodes || n != s.len || s.nodes > a.max_nodes) atomicCAS(a.err, 0, -9);
  if (s.nodes > a.max_nodes) s.len = 0;           // rows of zeros
  return s;
}
struct TreeSpan {
  int lo, nsu, first, n, blocks;
};
__device__ __forceinline__ TreeSpan tree_span(const TreeArgs &a, const TreeSeq &s) {
  TreeSpan p;
  p.lo = a.window > 0 ? max(s.len - s.nodes - a.window + 1, 0) : 0;
  p.first = p.lo / kTreeKeys;
  p.nsu = min((min(a.sinks, s.len) + kTreeKeys - 1) / kTreeKeys, p.first);
  p.n = max(p.nsu + (s.len + kTreeKeys - 1) / kTreeKeys - p.first, 1);       // an item without keys still writes its rows
  p.blocks = (int)(((long long)s.nodes * a.G + a.block_rows - 1) / a.block_rows);
  return p;
}
// Places of a sequence for teams of R: a tile takes one, an item `cost` more by itself.  A
// sequence's stay below kTreeMaxPlaces, and so do all of a call's whose offsets ascend (the host's bound).
__device__ __forceinline__ unsigned tree_places(const TreeArgs &a, const TreeSpan &p, int R, int cost) {
  return (unsigned)((p.blocks + R - 1) / R) * (unsigned)a.Hkv * (unsigned)(p.n + cost);
}

// CTAs that share the row blocks of a sequence: one for each block, up to four; one where max_nodes
// says that every sequence has one block (whatever a sequence that breaks its word has)
__device__ __forceinline__ int tree_team(const TreeArgs &a, const TreeSpan &p) {
  return a.blocks > 1 ? min(max(p.blocks, 1), kTreeMaxTeam) : 1;
}

// Lists the range's next segments (one thread).
static __device__ __noinline__ void tree_walk(const TreeArgs &a, TreeSeg *segs, TreeCtl *ctl) {
  int n = 0, b = ctl->b;
  unsigned off = ctl->off, pos = ctl->pos;
  const unsigned begin = ctl->begin, end = ctl->end;
  const int R = ctl->size, cost = ctl->cost;
#pragma unroll 1
  while (pos < end && n < kTreeSegs && b < a.B) {
    const TreeSeq s = tree_seq(a, b);
    const TreeSpan p = tree_span(a, s);
    if ((!ctl->all && tree_team(a, p) != R) || off >= tree_places(a, p, R, cost)) {
      ++b;
      off = 0;
      continue;
    }
    const unsigned each = (unsigned)(p.n + cost);
    const int groups = (p.blocks + R - 1) / R;
    const unsigned item = off / each, in = off - item * each;
    const int g = groups == 1 ? (int)item : (int)item / groups, rb = ((int)item - g * groups) * R + ctl->member;
    // the item's first place is pos - in, its first tile's `cost` further
    const long long x0 = (long long)begin - pos + in - cost, x1 = (long long)end - pos + in - cost;
    const int u0 = x0 > 0 ? (int)x0 : 0, u1 = x1 < p.n ? (int)x1 : p.n;
    if (u0 < u1 && rb < p.blocks) {
      TreeSeg &q = segs[n++];
      q.b = b;
      q.g = g;
      q.rb = rb;
      q.u0 = u0;
      q.u1 = u1;
      q.nsu = p.nsu;
      q.first = p.first;
      q.lo = p.lo;
      q.len = s.len;
      q.pos0 = s.len - s.nodes;
      q.tok0 = s.tok0;
      q.nodes = s.nodes;
      q.slot = u0 == 0 && u1 == p.n ? -1 : u0 > 0 ? 0 : 1;
      // (begun here: the tiles that are left, in shares)
      q.parts = q.slot != 1 ? 0 : 1 + (int)((unsigned)(p.n - u1 + ctl->share - 1) / ctl->share);
    }
    pos += each - in;
    off += each - in;
  }
  ctl->nseg = n;
  ctl->more = pos < end && b < a.B;
  ctl->b = b;
  ctl->off = off;
  ctl->pos = pos;
}

// This CTA's team and range, and its first segments.  All threads.  Sequences of as many row
// blocks form a class, the CTAs are shared among the classes by their work, and a class's CTAs form
// teams of one CTA a block that run one range of tiles together: K and V then come from HBM once
// for all blocks, and no CTA idles beside a sequence of fewer.  (Teams of three for all, 12
// sequences of two and three blocks: 216 us, a quarter of the CTAs' time idle.)
template <int IC, int NW>
__device__ __noinline__ void tree_schedule(const TreeArgs &a, TreeSeg *segs, TreeCtl *ctl) {
  constexpr int NT = 32 * NW;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (a.B + NT - 1) / NT;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  const int classes = a.blocks > 1 ? kTreeMaxTeam : 1;
  unsigned sum[kTreeMaxTeam] = {}, bare = 0;
  bool descends = false;
  auto add = [](unsigned x, unsigned y) { return y > kTreeMaxPlaces - min(x, kTreeMaxPlaces) ? kTreeMaxPlaces + 1u : x + y; };
  for (int b = b0; b < b1; ++b) {
    const TreeSeq s = tree_seq(a, b);
    const TreeSpan p = tree_span(a, s);
    const int R = tree_team(a, p);
#pragma unroll
    for (int k = 0; k < kTreeMaxTeam; ++k)
      if (k == R - 1) sum[k] = add(sum[k], tree_places(a, p, R, IC));
    bare = add(bare, tree_places(a, p, 1, 0));
    descends |= s.descends;
  }
  if (tid == 0) {
    ctl->nseg = ctl->more = ctl->zeroed = 0;
    ctl->bad[0] = ctl->bad[1] = 0;
  }
  // totals; up to 32 sequences are the first warp's
  auto over_warp = [&](unsigned v) { return __reduce_add_sync(0xffffffffu, v); };
  if (a.B > 32 || warp == 0) {
#pragma unroll
    for (int k = 0; k < kTreeMaxTeam; ++k) {
      const unsigned v = k < classes ? over_warp(sum[k]) : 0u;
      if (lane == 0) ctl->part[warp][k] = v;
    }
    const unsigned v = over_warp(bare);
    if (lane == 0) ctl->bare[warp] = v;
  }
  // Offsets that descend (recorded by tree_seq) can name every node many times.  The sums above are
  // those of the call only if those in 64 bits stay below the limit; else nothing is computed.
  if (__syncthreads_or(descends)) {
    atomicAdd(&ctl->bad[0], (unsigned long long)sum[0] + sum[1] + sum[2] + sum[3]);
    atomicAdd(&ctl->bad[1], (unsigned long long)bare);
    __syncthreads();
    const unsigned long long most = max(ctl->bad[0], ctl->bad[1]);
    __syncthreads();
    if (tid == 0) ctl->bad[0] = ctl->bad[1] = 0;
    if (most > kTreeMaxPlaces) return;            // (the whole CTA; its list is empty)
  }
  unsigned total[kTreeMaxTeam] = {}, tiles = 0;
  for (int w = 0; w < (a.B <= 32 ? 1 : NW); ++w) {
    tiles += ctl->bare[w];
#pragma unroll
    for (int k = 0; k < kTreeMaxTeam; ++k) total[k] += ctl->part[w][k];
  }
  const unsigned grid = gridDim.x;
  int R = 1, cost = IC;
  unsigned W = total[0], teams = grid, from = 0;          // the class's work, teams and first CTA
  bool all = true;                                        // every sequence is of the class
  // Few tiles: one or two a CTA, whatever an item costs.  (One context of 100 keys 14.5 us, with items' costs
  // counted 15.2; 1003 keys 18.5 either way, and a limit of 1 or 4 tiles a CTA changes no form timed.)
  if (tiles <= 2 * grid) {
    cost = 0;
    W = tiles;
  } else if (classes > 1) {
    // CTAs of each class: its share of the work (a class of R: R a place), whole teams; what is left
    // over goes to the class with most
    float work[kTreeMaxTeam], sums = 0.0f;
    int most = 0;
#pragma unroll
    for (int k = 0; k < kTreeMaxTeam; ++k) {
      work[k] = (float)total[k] * (float)(k + 1);
      sums += work[k];
      if (k > 0 && work[k] > work[most]) most = k;
    }
    unsigned n[kTreeMaxTeam], used = 0, big = 1;
#pragma unroll
    for (int k = 0; k < kTreeMaxTeam; ++k) {
      n[k] = total[k] == 0 ? 0u : max(1u, (unsigned)(work[k] / sums * (float)grid / (float)(k + 1)));       // teams
      used += n[k] * (unsigned)(k + 1);
      if (k == most) big = n[k];
    }
    const unsigned spare = grid - min(used, grid), over = used - min(used, grid);
    unsigned at = 0;
#pragma unroll
    for (int k = 0; k < kTreeMaxTeam; ++k) {
      if (k == most) n[k] = max(big + spare / (unsigned)(k + 1), (over + k) / (unsigned)(k + 1) + 1) - (over + k) / (unsigned)(k + 1);
      const unsigned end = at + n[k] * (unsigned)(k + 1);
      if (blockIdx.x >= at && blockIdx.x < end) {
        R = k + 1;
        W = total[k];
        teams = n[k];
        from = at;
      }
      at = end;
    }
    if (blockIdx.x >= at) W = 0;                          // (fewer CTAs than a team are left over)
    all = false;
  }
  const unsigned team = R == 1 ? blockIdx.x - from : (blockIdx.x - from) / (unsigned)R;
  const unsigned share = W == 0 ? 1 : (W - 1) / teams + 1;
  const unsigned begin = team < teams && (unsigned long long)team * share < W ? team * share : W;
  const unsigned end = W - begin < share ? W : begin + share;
  // the sequence that the range begins in: running sums of the class
  unsigned mine = cost == 0 ? bare : 0u, incl;
  if (cost != 0) {
#pragma unroll
    for (int k = 0; k < kTreeMaxTeam; ++k) mine = k == R - 1 ? sum[k] : mine;
  }
  incl = mine;
  if (a.B > 32 || warp == 0) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
  }
  if (a.B > 32) {
    for (int w = 0; w < warp; ++w) incl += cost == 0 ? ctl->bare[w] : ctl->part[w][R - 1];
  }
  const unsigned start = incl - mine;
  if (begin < end && start <= begin && begin - start < mine) {     // one thread
    ctl->size = R;
    ctl->all = all;
    ctl->cost = cost;
    ctl->member = R == 1 ? 0 : (int)((blockIdx.x - from) % (unsigned)R);
    ctl->share = share;
    ctl->begin = begin;
    ctl->end = end;
    int b = b0;
    unsigned off = begin - start;
    for (; b + 1 < b1; ++b) {
      const TreeSpan p = tree_span(a, tree_seq(a, b));
      if (!all && tree_team(a, p) != R) continue;
      const unsigned c = tree_places(a, p, R, cost);
      if (off < c) break;
      off -= c;
    }
    ctl->b = b;
    ctl->off = off;
    ctl->pos = begin;
    tree_walk(a, segs, ctl);
  }
  __syncthreads();
}

// key base of tile u of a segment's item
__device__ __forceinline__ int tree_base(const TreeSeg &s, int u) { return (u < s.nsu ? u : u - s.nsu + s.first) * kTreeKeys; }

// bits a .. b - 1 of a word (clamped to 0 .. 64)
__device__ __forceinline__ unsigned long long tree_bits(int a, int b) {
  a = max(a, 0);
  b = min(b, 64);
  if (a >= b) return 0;
  return (~0ull >> (64 - (b - a))) << a;
}

// 16-byte chunk c of row r of a stage
__device__ __forceinline__ uint32_t tree_chunk(uint32_t stage, int r, int c) {
  return stage + (c >> 3) * (kTreeKeys * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}
__device__ __forceinline__ uint32_t tmem_ld1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr) : "memory");
  tmem_wait_ld();
  return r;
}
// O += p v for the keys of `found`, in the rows that see them; then their values are cleared.
// The warps of group grp; fresh: O holds nothing yet.
template <int D, bool BF>
__device__ __noinline__ void tree_add_bad(uint32_t o, uint32_t weights, uint32_t vst, unsigned long long found,
                                          unsigned long long vis, bool fresh, int grp) {
#pragma unroll 1
  for (int cc = 0; cc < D; cc += 32) {
    uint32_t v[32];
    if (fresh) {
#pragma unroll
      for (int c = 0; c < 32; ++c) v[c] = 0u;
    } else {
      tmem_ld32(o + cc, v);
      tmem_wait_ld();
    }
#pragma unroll 1
    for (unsigned long long k = found; k; k &= k - 1) {
      const int j = __ffsll((long long)k) - 1;
      if (!__any_sync(0xffffffffu, (vis >> j & 1) != 0)) continue;
      const uint32_t at = weights + (j & ~15) + (j & 15) / 2;     // its two terms
      const float2 hi = tree_unpack<BF>(tmem_ld1(at)), lw = tree_unpack<BF>(tmem_ld1(at + 8));
      const float p = j & 1 ? hi.y + lw.y : hi.x + lw.x;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t w[4];
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(tree_chunk(vst, j, cc / 8 + q)) : "memory");
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const float2 f = tree_unpack<BF>(w[h]);
          float x = __uint_as_float(v[8 * q + 2 * h]), y = __uint_as_float(v[8 * q + 2 * h + 1]);
          if (vis >> j & 1) {
            x = fmaf(p, f.x, x);
            y = fmaf(p, f.y, y);
          }
          v[8 * q + 2 * h] = __float_as_uint(x);
          v[8 * q + 2 * h + 1] = __float_as_uint(y);
        }
      }
    }
    tmem_st32(o + cc, v);
  }
  tmem_wait_st();
  named_bar_sync(10 + grp, 128);                  // everyone has read the values
  for (unsigned long long k = found; k; k &= k - 1) {
    const int j = __ffsll((long long)k) - 1;
    if ((int)(threadIdx.x & 127) < D / 8)
      asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(tree_chunk(vst, j, (int)(threadIdx.x & 127))), "r"(0) : "memory");
  }
  fence_proxy_async_smem();
}

// ---------------------------------------------------------------- the kernel --
template <int D, int KV>
__global__ void __launch_bounds__(TreeShape<D, KV>::kThreads, TreeShape<D, KV>::kCtas) attn_tree_kernel(const __grid_constant__ TreeArgs a) {
  using Sh = TreeShape<D, KV>;
  constexpr bool kI8 = Sh::kI8, kBf = KV == kPagedBf16;
  constexpr int F = Sh::kTiles;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw0 = smem_u32(smem_raw);
  const uint32_t sbase = (raw0 + 1023u) & ~1023u;
  uint8_t *gbase = smem_raw + (sbase - raw0);
  const uint32_t q_s = sbase, k_s = q_s + Sh::kQ, v_s = k_s + F * Sh::kStage, kc_s = v_s + F * Sh::kStage, vc_s = kc_s + Sh::kRawK * Sh::kRaw;      // (kc, vc: codes)
  constexpr int kAt = Sh::kQ + 2 * F * Sh::kStage + (Sh::kRawK + Sh::kRawV) * Sh::kRaw;
  // int8, by tile: [slots][64] of K's scales times the softmax's, V's scales vs, log2 |vs| and 1 / |vs|
  float *ksc = reinterpret_cast<float *>(gbase + kAt);
  float *vsc = ksc + Sh::kScaleSlots * kTreeKeys, *vlog = vsc + Sh::kScaleSlots * kTreeKeys, *vinv = vlog + Sh::kScaleSlots * kTreeKeys;
  const uint32_t bars = sbase + kAt + Sh::kScaleBytes;
  uint8_t *fixed = gbase + kAt + Sh::kScaleBytes;
  short *par = reinterpret_cast<short *>(fixed + 512);                       // parents of the segment's nodes (256)
  uint32_t *masks = reinterpret_cast<uint32_t *>(fixed + 1024);              // [128][kMaskWords]
  float *xch = reinterpret_cast<float *>(masks + kTreeRows * Sh::kMaskWords);   // [2][128], then [2][128] references
  TreeSeg *segs = reinterpret_cast<TreeSeg *>(xch + 4 * kTreeRows);
  TreeCtl *ctl = reinterpret_cast<TreeCtl *>(reinterpret_cast<uint8_t *>(segs) + kTreeSegs * sizeof(TreeSeg));
  volatile WaitBlock *wctl = reinterpret_cast<volatile WaitBlock *>(ctl + 1);
  volatile uint32_t *tslot = reinterpret_cast<volatile uint32_t *>(const_cast<WaitBlock *>(wctl) + 1);
  // barriers: of K's and V's rings ([4] each; int8 also of the codes'), then
  auto full = [&](int isv, int slot) { return bars + 8u * (8 * isv + slot); };
  auto empty = [&](int isv, int slot) { return bars + 8u * (8 * isv + 4 + slot); };
  auto raw_full = [&](int isv, int slot) { return bars + 8u * (16 + 8 * isv + slot); };
  auto raw_empty = [&](int isv, int slot) { return bars + 8u * (20 + 8 * isv + slot); };
  auto s_full = [&](int b) { return bars + 8u * (32 + b); };
  auto p_full = [&](int b) { return bars + 8u * (36 + b); };
  const uint32_t q_full = bars + 8 * 40, q_empty = bars + 8 * 41, o_done = bars + 8 * 43, o_free = bars + 8 * 44,
                 drain = bars + 8 * 45;
  // P V of tile gt is done.  One barrier a buffer: scores of tile gt follow P V of tile gt - kBufs, so
  // a wait for the tile before names one phase.
  auto o_step = [&](int gt) { return bars + 8u * (46 + gt % Sh::kBufs); };
  auto o_phase = [&](int gt) { return (uint32_t)((gt / Sh::kBufs) & 1); };
  auto pwait = [&](uint32_t bar, uint32_t parity) { return tree_wait(bar, parity, wctl, a.wait_ns == 0); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int v = 0; v < 2; ++v) {
      for (int i = 0; i < F; ++i) {
        mbar_init(full(v, i), kI8 ? 16 * Sh::kWideners : 1);
        mbar_init(empty(v, i), 1);
      }
      for (int i = 0; i < (v ? Sh::kRawV : Sh::kRawK); ++i) {
        mbar_init(raw_full(v, i), a.scale_boxes ? 1 : 33);
        mbar_init(raw_empty(v, i), Sh::kWideners / 2);
      }
    }
    for (int b = 0; b < Sh::kBufs; ++b) {
      mbar_init(s_full(b), 1);
      mbar_init(p_full(b), 4);
      mbar_init(o_step(b), 1);
    }
    mbar_init(q_full, Sh::kQTmem ? 8 : 1);
    mbar_init(q_empty, 1);
    mbar_init(o_done, 1);
    mbar_init(o_free, 8);
    mbar_init(drain, 1);
    wait_block_init(wctl, a.wait_ns, a.err);
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(const_cast<uint32_t *>(tslot)), Sh::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  griddep_wait();
  griddep_launch_dependents();
  tree_schedule<Sh::kItemCost, Sh::kWarps>(a, segs, ctl);

  // the roles' counters run over all segments of all lists
  int tiles = 0;                                  // tiles
  int nsegs = 0;                                  // segments
  bool ok = true;
  int last = -1, queries = 0;                     // loading: the last tile copied to slot `lane` (V: lane - 8); Qs copied
  TreeDesc desc{};                                // the item whose first part this CTA leaves

  for (;;) {
    const int nseg = ctl->nseg;
    if (warp >= Sh::kLoadWarp && warp < Sh::kWiden0) {
      // ------------------------------------------------------------ loading --
      // Pages of whole boxes (8 to 64 rows, a.box): box b of a tile is rows box * (b % boxes) .. of 128
      // bytes b / boxes (int8: of whole rows), and lane b's.  Other pages: a tile's 64 rows are
      // sixteen gathers of four rows, and as many for each 128 bytes; lane l finds the rows of quad
      // l % 16.  A box holds its warp about 70 cycles, so where a tile has most of them one warp
      // loads K and Q and the other V.  The loop over boxes is kept short: a warp that comes round
      // once a stage finds its instructions gone from the caches near it (250 of them took 1500
      // cycles).
      constexpr int CW = kI8 ? 1 : D / 64;                        // boxes or gathers side by side
      constexpr int NK = kI8 ? Sh::kRawK : F, NV = kI8 ? Sh::kRawV : F;
      constexpr int kRowBytes = kI8 ? D : 128;
      constexpr uint32_t kSlotBytes = kI8 ? Sh::kRaw : Sh::kStage;
      const int role = Sh::kLoaders == 2 ? warp - Sh::kLoadWarp : 2;      // 0: K and Q, 1: V, 2: all
      const int boxes = a.box ? kTreeKeys / a.box : 16;           // down a tile; a power of two
      const int chunk = lane / boxes;                             // this lane's 128 bytes (box: the only ones)
      const int first = a.box ? (lane & (boxes - 1)) * a.box : 4 * (lane & 15);        // its first row
      const uint32_t mine = (uint32_t)(first * kRowBytes + (a.box && !kI8 ? chunk * (kTreeKeys * 128) : 0));
      for (int si = 0; si < nseg && ok; ++si) {
        const TreeSeg &s = segs[si];
        const int n = s.u1 - s.u0, seg = nsegs + si;
        const int *table = a.table + (long long)s.b * a.max_pages;
        // waits for the slot of tile gt of K or V; its barrier, and where it lies (false: give up)
        auto room = [&](bool isv, int gt, uint32_t &bar, uint32_t &dst) {
          const int ring = isv ? NV : NK, slot = gt % ring;
          if (gt >= ring) ok = __all_sync(0xffffffffu, pwait(kI8 ? raw_empty(isv, slot) : empty(isv, slot), (uint32_t)((gt / ring - 1) & 1)));
          if (ok && lane == slot + (isv ? 8 : 0)) last = gt;
          bar = kI8 ? raw_full(isv, slot) : full(isv, slot);
          dst = (kI8 ? isv ? vc_s : kc_s : isv ? v_s : k_s) + slot * kSlotBytes + mine;
          return ok;
        };
        auto queries_in = [&] {
          // Q: row r is column rb * block_rows + r of the KV head: node column / G, head column % G
          if (seg > 0) ok = __all_sync(0xffffffffu, pwait(q_empty, (uint32_t)((seg - 1) & 1)));
          if (!ok) return;
          if (a.q_box) {                          // whole nodes: one box (rows beyond the sequence's are never written)
            if (lane == 0) mbar_arrive_expect_tx(q_full, a.block_rows * 2 * D);
            __syncwarp();
            if (lane < D / 64)
              tma_load_4d(q_s + lane * (kTreeRows * 128), &a.qbox, 64 * lane, 0, s.g, s.tok0 + s.rb * (a.block_rows / a.G), q_full);
          } else {
            if (lane == 0) mbar_arrive_expect_tx(q_full, Sh::kQ);
            __syncwarp();
            int row[4];
            const int cols = s.nodes * a.G;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int col = s.rb * kTreeRows + 4 * lane + e, node = col / a.G;
              row[e] = col < cols ? (s.tok0 + node) * a.q_tok_rows + (s.g * a.G + col - node * a.G) * a.q_head_rows : -1;
            }
#pragma unroll 1
            for (int c = 0; c < D / 64; ++c) tma_gather4(q_s + c * (kTreeRows * 128) + lane * 512, &a.qmap, 64 * c, row, q_full);
          }
          queries = seg + 1;
        };
        if (a.box) {
          // Tile t's box of this lane: page table entry pi, row r of it; advanced a tile at a time.
          // The table comes through a window of 64 entries, 32 ahead of their use.
          const int dpi = kTreeKeys / a.page, dr = kTreeKeys % a.page;
          int t = s.u0 - 1, j = 0, pi = 0, r = 0, wbase = -64, win = 0, ahead = 0;
          auto entry = [&](int e) { return e + lane < a.max_pages ? __ldg(table + e + lane) : 0; };
          int pid = -2, row = 0, vpid = -2, vrow = 0;             // of the tile whose K, V is next
          auto next = [&] {
            ++t;
            j += kTreeKeys;
            pi += dpi;
            r += dr;
            if (r >= a.page) {
              r -= a.page;
              ++pi;
            }
            if (t == s.u0 || t == s.nsu) {        // (the windowed tiles follow the sinks')
              j = tree_base(s, t) + first;
              pi = j / a.page;
              r = j - pi * a.page;
            }
            const int e0 = __shfl_sync(0xffffffffu, pi, 0);       // the tile's first entry; it has at most 8
            if (e0 - wbase >= 64 || e0 < wbase) {
              wbase = e0;
              win = entry(wbase);
              ahead = entry(wbase + 32);
            } else if (e0 - wbase >= 32) {
              wbase += 32;
              win = ahead;
              ahead = entry(wbase + 32);
            }
            const int at = pi - wbase;
            pid = __shfl_sync(0xffffffffu, win, at & 31);
            if (__any_sync(0xffffffffu, at >= 32)) {
              const int p = __shfl_sync(0xffffffffu, ahead, at & 31);
              pid = at >= 32 ? p : pid;
            }
            row = r;
            // boxes that no node sees a row of stay what they are: their keys are masked
            if (chunk >= CW || j >= s.len || (j + a.box <= s.lo && j >= a.sinks)) pid = -2;
          };
          const int stages = role == 2 ? 2 * n : n;
#pragma unroll 1
          for (int x = 0; x < stages; ++x) {      // K0 K1 V0 K2 V1 .., or a role's share of it
            const bool isv = role == 2 ? x == stages - 1 || (x >= 2 && !(x & 1)) : role == 1;
            const int i = role != 2 ? x : isv ? (x == stages - 1 ? n - 1 : x / 2 - 1) : (x + 1) / 2;
            if (role != 2 || !isv) {
              vpid = pid;
              vrow = row;
              next();
            } else if (x == stages - 1) {
              vpid = pid;
              vrow = row;
            }
            const int p = role == 2 && isv ? vpid : pid, r0 = role == 2 && isv ? vrow : row;
            uint32_t bar, dst;
            if (!room(isv, tiles + i, bar, dst)) break;
            const bool page = (unsigned)p < (unsigned)a.npages, on = p != -2;
            const int parts = __popc(__ballot_sync(0xffffffffu, on)), pages = kI8 ? __popc(__ballot_sync(0xffffffffu, page)) : 0;
            if constexpr (kI8) {
              // (scales of a page that is none are 0, not the tile's before: written ahead of lane 0's arrival)
              if (pages < parts && !isv && a.scale_boxes) {
                for (int q = 0; q < a.box && on && !page; ++q) {
                  const int to = ((tiles + i) % Sh::kScaleSlots) * kTreeKeys + first + q;
                  ksc[to] = vsc[to] = 0.0f;
                }
                __syncwarp();
              }
            }
            if (lane == 0)                        // (int8: the tile's scales come with its K)
              mbar_arrive_expect_tx(bar, parts * a.box * kRowBytes + (kI8 && !isv && a.scale_boxes ? pages * a.box * 8 : 0));
            __syncwarp();
            if (page) tma_load_4d(dst, isv ? &a.vbox : &a.kbox, kI8 ? 0 : 64 * chunk, r0, s.g, p, bar);
            if (on && !page) {                    // a page that is none: zeros
              atomicCAS(a.err, 0, -9);
              const int none[4] = {-1, -1, -1, -1};
              for (int q = 0; q < a.box; q += 4) tma_gather4(dst + q * kRowBytes, isv ? &a.vmap : &a.kmap, 0, none, bar);
            }
            if constexpr (kI8) {
              if (a.scale_boxes) {
                if (!isv && page) {
                  const int to = ((tiles + i) % Sh::kScaleSlots) * kTreeKeys + first;
                  const long long from = ((long long)p * a.Hkv + s.g) * a.page + r0;
                  bulk_g2s_nohint(smem_u32(ksc + to), a.ks + from, a.box * 4, bar);
                  bulk_g2s_nohint(smem_u32(vsc + to), a.vs + from, a.box * 4, bar);
                }
              } else {                            // (scales that are not aligned: one by one)
                for (int q = 0; q < a.box && !isv && on; ++q) {
                  const int to = ((tiles + i) % Sh::kScaleSlots) * kTreeKeys + first + q;
                  const long long from = page ? ((long long)p * a.Hkv + s.g) * a.page + r0 + q : 0;
                  cp_async4_zfill(smem_u32(ksc + to), a.ks + from, page ? 4u : 0u);
                  cp_async4_zfill(smem_u32(vsc + to), a.vs + from, page ? 4u : 0u);
                }
                cp_async_arrive(bar);
              }
            }
            if (!Sh::kQTmem && x == 0 && role != 1) queries_in();
          }
        } else {
          const int quad = lane & 15;
          auto seen = [&](int j) { return j < s.len && (j >= s.lo || j < a.sinks); };
#pragma unroll 1
          for (int x = 0; x < 2 * n; ++x) {
            const bool isv = x == 2 * n - 1 || (x >= 2 && !(x & 1));
            if (role != 2 && isv != (role == 1)) continue;
            const int i = isv ? (x == 2 * n - 1 ? n - 1 : x / 2 - 1) : (x + 1) / 2;
            const int j = tree_base(s, s.u0 + i) + 4 * quad;
            int pi = a.page_shift >= 0 ? j >> a.page_shift : j / a.page, r = j - pi * a.page;
            int row[4], pid[4], at[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              pid[e] = seen(j + e) ? __ldg(table + pi) : -2;
              at[e] = r;
              if (++r == a.page) {
                r = 0;
                ++pi;
              }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool page = (unsigned)pid[e] < (unsigned)a.npages;
              if (!page && pid[e] != -2) atomicCAS(a.err, 0, -9);
              row[e] = page ? pid[e] * a.page_rows + s.g * a.head_rows + at[e] * a.tok_rows : -1;
            }
            uint32_t bar, dst;
            if (!room(isv, tiles + i, bar, dst)) break;
            if (lane == 0) mbar_arrive_expect_tx(bar, kSlotBytes);
            __syncwarp();
            for (int c = chunk; c < CW; c += 2)
              tma_gather4(dst + c * (kTreeKeys * 128), isv ? &a.vmap : &a.kmap, kI8 ? 0 : 64 * c, row, bar);
            if constexpr (kI8) {                  // lanes 0 .. 15 K's scales, the others V's
              if (!isv) {
                const int to = ((tiles + i) % Sh::kScaleSlots) * kTreeKeys + 4 * quad;
                const float *from = lane < 16 ? a.ks : a.vs;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  cp_async4_zfill(smem_u32((lane < 16 ? ksc : vsc) + to + e), from + (row[e] < 0 ? 0 : ((long long)pid[e] * a.Hkv + s.g) * a.page + at[e]), row[e] < 0 ? 0u : 4u);
              }
              cp_async_arrive(bar);
            }
            if (!Sh::kQTmem && x == 0) queries_in();
          }
        }
        tiles += n;
      }
    } else if (kI8 && warp >= Sh::kWiden0) {
      // ----------------------------------------------------------- widening --
      // Half of the warps widen K, the others V.
      constexpr int WT = 16 * (kI8 ? Sh::kWideners : 2);          // threads a half
      const int isv = warp >= Sh::kWiden0 + Sh::kWideners / 2;
      const int t = threadIdx.x - 32 * Sh::kWiden0 - isv * WT;
      const int ring = isv ? max(Sh::kRawV, 1) : max(Sh::kRawK, 1);
      const uint32_t from_s = isv ? vc_s : kc_s, to_s = isv ? v_s : k_s;
      for (int si = 0; si < nseg && ok; ++si) {
        const int n = segs[si].u1 - segs[si].u0;
        for (int i = 0; i < n && ok; ++i) {
          const int gt = tiles + i, rs = gt % ring, fs = gt % F;
          ok = pwait(raw_full(isv, rs), (uint32_t)((gt / ring) & 1));
          if (ok && gt >= F) ok = pwait(empty(isv, fs), (uint32_t)((gt / F - 1) & 1));
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          // a tile's scales, with its K: logarithm and inverse of V's (of 0: of 2^-100, which times
          // vs is 0 again; at most 2^126, whose inverse is normal)
          if (!isv) {
            for (int e = t; e < kTreeKeys; e += WT) {
              const int at = (gt % Sh::kScaleSlots) * kTreeKeys + e;
              const float v = fabsf(vsc[at]);
              const float lv = v < INFINITY ? fminf(fmaxf(tree_lg2(v), -100.0f), 126.0f) : 0.0f;
              vlog[at] = lv;
              vinv[at] = tree_ex2(-lv);
              ksc[at] *= a.scale_log2;
            }
          }
          constexpr int CH = D / 16, PER = kTreeKeys * CH / WT, STEP = PER < 4 ? PER : 4;
#pragma unroll 1
          for (int k0 = 0; k0 < PER; k0 += STEP) {
            uint4 x[STEP];
#pragma unroll
            for (int k = 0; k < STEP; ++k) {
              const uint32_t at = from_s + rs * Sh::kRaw + 16 * ((k0 + k) * WT + t);
              asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x[k].x), "=r"(x[k].y), "=r"(x[k].z), "=r"(x[k].w) : "r"(at) : "memory");
            }
#pragma unroll
            for (int k = 0; k < STEP; ++k) {
              const int id = (k0 + k) * WT + t, row = id / CH, cc = id % CH;
              const uint32_t w[4] = {x[k].x ^ 0x80808080u, x[k].y ^ 0x80808080u, x[k].z ^ 0x80808080u, x[k].w ^ 0x80808080u};
#pragma unroll
              for (int h = 0; h < 2; ++h)
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(tree_chunk(to_s + fs * Sh::kStage, row, 2 * cc + h)),
                             "r"(tree_widen<0x4140>(w[2 * h])), "r"(tree_widen<0x4342>(w[2 * h])), "r"(tree_widen<0x4140>(w[2 * h + 1])),
                             "r"(tree_widen<0x4342>(w[2 * h + 1]))
                             : "memory");
            }
          }
          // (the codes' slot is given back only here, where every load's value has been used; right behind the
          // loads, whose values need not have arrived, the next copy was seen in them)
          __syncwarp();
          if (lane == 0) mbar_arrive(raw_empty(isv, rs));
          fence_proxy_async_smem();
          mbar_arrive(full(isv, fs));
        }
        tiles += n;
      }
    } else if (warp == Sh::kMmaWarp) {
      // ---------------------------------------------------------------- MMA --
      // The whole warp runs the loop and the leader lane issues: see mma_f16_ts_w.
      const uint32_t leader = elect_leader();
      auto wwait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, pwait(bar, parity)); };
      constexpr uint32_t kIdO = tree_idesc(kBf, true, kTreeRows, D);
      const uint32_t kIdS = tree_idesc(kBf, false, kTreeRows, kTreeKeys) | (a.scale_log2 < 0.0f && !kI8 ? 1u << 13 : 0u);
      for (int si = 0; si < nseg && ok; ++si) {
        const int n = segs[si].u1 - segs[si].u0;
        const int seg = nsegs + si;
        if (!wwait(q_full, (uint32_t)(seg & 1))) { ok = false; break; }
        for (int i = -Sh::kAhead; i < n; ++i) {   // scores of tile i + kAhead, then P V of tile i
          const int k = i + Sh::kAhead;
          if (k < n) {
            const int gt = tiles + k, slot = gt % F, b = gt % Sh::kBufs;
            if (!wwait(full(0, slot), (uint32_t)((gt / F) & 1))) { ok = false; break; }
            tc_fence_after();
            // (descriptors count 16 bytes; the loops are kept rolled: see the loading loop)
            uint64_t qd = smem_desc_sw128(q_s), kd = smem_desc_sw128(k_s + slot * Sh::kStage);
#pragma unroll 1
            for (int c = 0; c < D / 64; ++c, qd += kTreeRows * 8, kd += kTreeKeys * 8) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                const uint32_t to = tmem + Sh::kSCol + (uint32_t)(b * kTreeKeys);
                if constexpr (Sh::kQTmem) mma_f16_ts_w(leader, to, tmem + Sh::kQCol + (uint32_t)(32 * c + 8 * kk), kd + 2 * kk, kIdS, (uint32_t)(c + kk));
                else mma_f16_ss_w(leader, to, qd + 2 * kk, kd + 2 * kk, kIdS, (uint32_t)(c + kk));
              }
            }
            mma_commit_w(leader, s_full(b));
            mma_commit_w(leader, empty(0, slot));
            if (!Sh::kQTmem && k == n - 1) mma_commit_w(leader, q_empty);
          }
          if (i >= 0) {
            const int gt = tiles + i, slot = gt % F, b = gt % Sh::kBufs;
            if (!wwait(p_full(b), (uint32_t)((gt / Sh::kBufs) & 1))) { ok = false; break; }
            if (!wwait(full(1, slot), (uint32_t)((gt / F) & 1))) { ok = false; break; }
            tc_fence_after();
            // (O of the segment before has been read; a tile with values that are not finite starts it at 0)
            if (i == 0 && seg > 0 && !wwait(o_free, (uint32_t)((seg - 1) & 1))) { ok = false; break; }
            const uint32_t more = i > 0 || *static_cast<volatile int *>(&ctl->zeroed) == seg + 1;
            uint64_t vd = smem_desc_sw128_mn(v_s + slot * Sh::kStage);
            uint32_t pt = tmem + Sh::kSCol + (uint32_t)(b * kTreeKeys);
#pragma unroll 1
            for (int kk = 0; kk < kTreeKeys / 16; ++kk, vd += 128, pt += 16) {
              mma_f16_ts_w(leader, tmem, pt, vd, kIdO, more | (uint32_t)kk);
              mma_f16_ts_w(leader, tmem, pt + 8, vd, kIdO, 1u);
            }
            mma_commit_w(leader, empty(1, slot));
            mma_commit_w(leader, o_step(gt));
            if (i == n - 1) mma_commit_w(leader, o_done);
          }
        }
        if (!ok) break;
        tiles += n;
      }
    } else if (warp < 8) {
      // ------------------------------------------------------------ softmax --
      // Two groups of four warps take tiles in turn, a thread a row: while one group's weights are
      // under way the other finds the next tile's largest scores (loads and stores of TMEM take
      // hundreds of cycles beside the MMAs; with both groups on one tile, half the keys each, a tile
      // took 2700 cycles, 3600 with int8).  The reference passes from tile to tile through shared memory.
      // Warps whose rows are all beyond the item's only keep the barriers going.
      constexpr int ST = 256;
      const int grp = warp >> 2, row = threadIdx.x & 127;              // (TMEM lane)
      const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
      constexpr float kHead = kBf ? 0.0f : 7.0f, kPass = kBf ? 8.0f : 15.0f;
      constexpr int DH = D / 2;
      const float scale = fabsf(a.scale_log2);    // (a negative one negates Q)
      bool aborted = !ok;
      for (int si = 0; si < nseg && !aborted; ++si) {
        const TreeSeg &s = segs[si];
        const int n = s.u1 - s.u0, seg = nsegs + si;
        const int col = s.rb * a.block_rows + row, node = col / a.G, head = s.g * a.G + col - node * a.G;
        const bool real = node < s.nodes && row < a.block_rows;
        const bool busy = __any_sync(0xffffffffu, real);
        if constexpr (Sh::kQTmem) {
          // the row of Q, a group half of it: two elements a column (the segment before has its scores)
          uint4 v[D / 16];
          const uint16_t *from = a.q + (long long)(s.tok0 + (real ? node : 0)) * a.q_tok + (long long)head * a.q_head + grp * (D / 2);
#pragma unroll
          for (int c = 0; c < D / 16; ++c) v[c] = real ? __ldg(reinterpret_cast<const uint4 *>(from) + c) : make_uint4(0u, 0u, 0u, 0u);
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < D / 16; c += 2) {
            const uint32_t w[8] = {v[c].x, v[c].y, v[c].z, v[c].w, v[c + 1].x, v[c + 1].y, v[c + 1].z, v[c + 1].w};
            tmem_st8(tmem + lane_base + Sh::kQCol + (uint32_t)(grp * (D / 4) + 4 * c), w);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(q_full);
        }
        // the row's ancestors, as bits over the nodes, and the first key its window holds
        uint32_t *mine = masks + row * Sh::kMaskWords;
        if ((tree_base(s, s.u1 - 1) + kTreeKeys > s.pos0 || a.window > 0) && s.nodes <= 256) {   // (else none is needed)
          named_bar_sync(1, ST);                  // the last segment's have been read
          for (int i = threadIdx.x; i < s.nodes; i += ST) {
            int p = __ldg(a.parents + s.tok0 + i);
            if (p < -1 || p >= i) {
              atomicCAS(a.err, 0, -9);
              p = -1;
            }
            par[i] = (short)p;
          }
          named_bar_sync(1, ST);
          if (grp == 0) {
            int depth = 0;
            if (real && a.window > 0)
              for (int i = par[node]; i >= 0; i = par[i]) ++depth;
#pragma unroll
            for (int w = 0; w < 8; ++w) mine[w] = 0u;
            mine[8] = (uint32_t)(a.window > 0 ? max(s.pos0 + depth - a.window + 1, 0) : 0);
            if (real && s.len > 0) {
              int e = 0;
              for (int i = node; i >= 0; i = par[i], ++e)
                if (a.window == 0 || e < a.window || s.pos0 + depth - e < a.sinks) mine[i >> 5] |= 1u << (i & 31);
            }
          }
          named_bar_sync(1, ST);
        }
        // keys from this one on (before the tree) are in every row's window
        const int whole = a.window > 0 ? s.pos0 + s.nodes - a.window : 0;
        float m_ref = kTreeNoScore, l = 0.0f;     // the group's sum, to the reference of its latest tile
        float *refs = xch + 2 * kTreeRows + row;  // [2][128]: of the latest tiles
        const int pass_on = 2 + 4 * grp + (warp & 3), take_over = 2 + 4 * (grp ^ 1) + (warp & 3);      // barriers of a row's two warps
        for (int i = (tiles & 1) == grp ? 0 : 1; i < n; i += 2) {
          const int gt = tiles + i, b = gt % Sh::kBufs;
          const int base = tree_base(s, s.u0 + i);
          const bool masked = base + kTreeKeys > s.pos0 || (base < whole && base + kTreeKeys > a.sinks);
          unsigned long long vis = ~0ull;
          if (masked) {
            const int lo = a.window > 0 ? (int)mine[8] : 0;
            vis = tree_bits(lo - base, s.pos0 - base) | tree_bits(0, min(a.sinks, s.pos0) - base);
            const int at = base - s.pos0;         // the tile's first key among the nodes
            if (at > -kTreeKeys && at < 256) {
              unsigned long long t = 0;
              for (int w = max(at, 0) >> 5; w < 8 && 32 * w - at < 64; ++w) {
                const int sh = 32 * w - at;       // where word w starts in the tile
                t |= sh >= 0 ? (unsigned long long)mine[w] << sh : (unsigned long long)mine[w] >> -sh;
              }
              vis |= t & tree_bits(0, s.len - base);
            }
            if (!real) vis = 0;
          }
          bool stop = !pwait(s_full(b), (uint32_t)((gt / Sh::kBufs) & 1));
          tc_fence_after();
          const uint32_t sadr = tmem + lane_base + Sh::kSCol + (uint32_t)(b * kTreeKeys);
          const int sc = (gt % Sh::kScaleSlots) * kTreeKeys;
          // NX scores from c0 on; int8: log2 of the weight times its value's scale.  Where the registers
          // do not hold all 64 they are read twice.
          constexpr int NX = D < 256 ? 16 : kI8 ? 32 : 64;
          F2 x[NX / 2];
          auto scores = [&](int c0) {
            uint32_t v[NX];
            if constexpr (NX == 16) tmem_ld16(sadr + (uint32_t)c0, v);
            else if constexpr (NX == 32) tmem_ld32(sadr + (uint32_t)c0, v);
            else {
              tmem_ld32(sadr, *reinterpret_cast<uint32_t(*)[32]>(v));
              tmem_ld32(sadr + 32u, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
            }
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < NX; c += 4) {
              x[c / 2] = F2(__uint_as_float(v[c]), __uint_as_float(v[c + 1]));
              x[c / 2 + 1] = F2(__uint_as_float(v[c + 2]), __uint_as_float(v[c + 3]));
              if constexpr (kI8) {                // (16 bytes a load: the loads of scales alone are 1500 cycles a tile by 8)
                const F4 k = *reinterpret_cast<const F4 *>(ksc + sc + c0 + c), e = *reinterpret_cast<const F4 *>(vlog + sc + c0 + c);
                x[c / 2] = fma2(x[c / 2], k.a, e.a);
                x[c / 2 + 1] = fma2(x[c / 2 + 1], k.b, e.b);
              }
            }
          };
          float top = -INFINITY;
          if (busy) {
#pragma unroll 1
            for (int c0 = 0; c0 < kTreeKeys; c0 += NX) {
              scores(c0);
              float t0 = -INFINITY, t1 = -INFINITY;
              if (masked) {
                const unsigned long long vm = vis >> c0;
#pragma unroll
                for (int c = 0; c < NX / 2; ++c) {
                  float p, r;
                  x[c].get(p, r);
                  t0 = max3(t0, vm >> (2 * c) & 1 ? p : -INFINITY, vm >> (2 * c + 1) & 1 ? r : -INFINITY);
                }
              } else {
#pragma unroll
                for (int c = 0; c < NX / 2; c += 2) {
                  float p, r;
                  x[c].get(p, r);
                  t0 = max3(t0, p, r);
                  x[c + 1].get(p, r);
                  t1 = max3(t1, p, r);
                }
              }
              top = max3(top, t0, t1);
            }
            if (!kI8) top = top == -INFINITY ? top : top * scale;
          }
          // The reference of the tile before, which moves only when a score passes it by 2^kPass; then O
          // is rescaled, once the previous P V is done.
          stop = stop || wctl->abort;
          float before = kTreeNoScore;
          if (i > 0) {
            named_bar_sync(take_over, 64);
            before = refs[(grp ^ 1) * kTreeRows];
          }
          const bool moves = top > before + kPass;
          const float now = moves ? top - kHead : before;
          if (i + 1 < n) {
            refs[grp * kTreeRows] = now;
            asm volatile("bar.arrive %0, %1;" ::"r"(pass_on), "r"(64) : "memory");
          }
          l *= tree_ex2(m_ref - now);
          m_ref = now;
          if (__any_sync(0xffffffffu, moves) && i > 0) {
            const float f = tree_ex2(before - now);
            if (!__all_sync(0xffffffffu, pwait(o_step(gt - 1), o_phase(gt - 1)))) stop = true;
            tc_fence_after();
#pragma unroll 1
            for (int cc = 0; cc < (stop ? 0 : D); cc += 32) {
              uint32_t v[32];
              tmem_ld32(tmem + lane_base + cc, v);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 32; ++c) v[c] = __float_as_uint(__uint_as_float(v[c]) * f);
              tmem_st32(tmem + lane_base + cc, v);
            }
            tmem_wait_st();
          }
          // the weights of 16 keys over their scores: 8 columns of rounded pairs, 8 of what they leave
          auto weights = [&](auto partly) {
            const F2 sc2(scale, scale), neg(-m_ref, -m_ref), minus(-1.0f, -1.0f);
            F2 sum(0.0f, 0.0f);
#pragma unroll 1
            for (int c0 = 0; c0 < kTreeKeys; c0 += NX) {
              if constexpr (NX < kTreeKeys) scores(c0);
              const unsigned long long vm = vis >> c0;
#pragma unroll
              for (int h = 0; h < NX; h += 16) {
                uint32_t hi[8], lw[8];
                F4 iv, vs;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                  if constexpr (kI8) {
                    if (!(c & 1)) {
                      iv = *reinterpret_cast<const F4 *>(vinv + sc + c0 + h + 2 * c);
                      vs = *reinterpret_cast<const F4 *>(vsc + sc + c0 + h + 2 * c);
                    }
                  }
                  F2 w = kI8 ? add2(x[h / 2 + c], neg) : fma2(x[h / 2 + c], sc2, neg);
                  float p, r;
                  w.get(p, r);
                  w = F2(tree_ex2(p), tree_ex2(r));
                  if constexpr (kI8) {
                    w = mul2(w, c & 1 ? iv.b : iv.a);
                    if constexpr (decltype(partly)::value) {
                      w.get(p, r);
                      w = F2(vm >> (h + 2 * c) & 1 ? p : 0.0f, vm >> (h + 2 * c + 1) & 1 ? r : 0.0f);
                    }
                    sum = add2(sum, w);
                    w = mul2(w, c & 1 ? vs.b : vs.a);
                  }
                  w.get(p, r);
                  if constexpr (decltype(partly)::value) {    // (hidden: also with scores or scales that are not finite)
                    p = vm >> (h + 2 * c) & 1 ? p : 0.0f;
                    r = vm >> (h + 2 * c + 1) & 1 ? r : 0.0f;
                    w = F2(p, r);
                  }
                  if constexpr (!kI8) sum = add2(sum, w);
                  hi[c] = tree_pack<kBf>(p, r);
                  const float2 q = tree_unpack<kBf>(hi[c]);
                  fma2(F2(q.x, q.y), minus, w).get(p, r);
                  lw[c] = tree_pack<kBf>(p, r);
                }
                tmem_st8(sadr + (uint32_t)(c0 + h), hi);
                tmem_st8(sadr + (uint32_t)(c0 + h) + 8u, lw);
              }
            }
            float p, r;
            sum.get(p, r);
            l += p + r;
            tmem_wait_st();
          };
          if (busy) {
            if (masked) weights(std::true_type{});
            else weights(std::false_type{});
          }
          if constexpr (!kI8) {
            // A value that is not finite would reach the rows that do not see its key (0 times it is NaN),
            // so tiles seen partly are searched for such keys.  They are added here, to the rows
            // that see them, and cleared for the MMA.  (Not where no row sees anything: a sequence of more nodes
            // than are allowed has no masks, so no barrier between this and the other group's rows of the last segment.)
            if (masked && s.len > 0) {
              const uint32_t vst = v_s + (gt % F) * Sh::kStage;
              stop = stop || !pwait(full(1, gt % F), (uint32_t)((gt / F) & 1));
              if (row == 0) ctl->bad[grp] = 0;
              named_bar_sync(10 + grp, 128);
              constexpr uint32_t e = kBf ? 0x7f80u : 0x7c00u;
              bool bad = false;
#pragma unroll
              for (int c = 0; c < D / 16; ++c) {
                const uint32_t at = tree_chunk(vst, row >> 1, (row & 1) * (D / 16) + c);
                uint32_t w[4];
                asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
#pragma unroll
                for (int k = 0; k < 4; ++k) bad |= (w[k] & e) == e || (w[k] >> 16 & e) == e;
              }
              if (bad) atomicOr(&ctl->bad[grp], 1ull << (row >> 1));
              named_bar_sync(10 + grp, 128);
              const unsigned long long found = *static_cast<volatile unsigned long long *>(&ctl->bad[grp]);
              if (found) {
                stop = stop || !__all_sync(0xffffffffu, i == 0 || pwait(o_step(gt - 1), o_phase(gt - 1)));
                tc_fence_after();
                // (after a wait that gave up everyone goes on to the segment's end without waiting)
                if (!named_bar_or(10 + grp, 128, stop)) tree_add_bad<D, kBf>(tmem + lane_base, tmem + lane_base + Sh::kSCol + (uint32_t)(b * kTreeKeys), vst, found, vis, i == 0, grp);
                if (row == 0 && i == 0) *static_cast<volatile int *>(&ctl->zeroed) = seg + 1;
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (stop) wctl->abort = 1;
            mbar_arrive(p_full(b));
          }
        }
        // ---- the rows, or their parts
        const bool got = !aborted && pwait(o_done, (uint32_t)(seg & 1));
        xch[grp * kTreeRows + row] = l;
        refs[grp * kTreeRows] = m_ref;
        if (named_bar_or(1, ST, !got || wctl->abort)) { aborted = true; break; }
        tc_fence_after();
        {
          const float other = refs[(grp ^ 1) * kTreeRows], m = fmaxf(m_ref, other);      // (the latest tile's)
          l = l * tree_ex2(m_ref - m) + xch[(grp ^ 1) * kTreeRows + row] * tree_ex2(other - m);
          m_ref = m;
        }
        named_bar_sync(1, ST);                    // (both have read them)
        if (s.slot < 0) {
          const float inv = 1.0f / l;
          const long long at = (long long)(s.tok0 + node) * a.Hq + head;
#pragma unroll 1
          for (int cc = grp * DH; cc < grp * DH + DH; cc += 32) {
            uint32_t v[32];
            tmem_ld32(tmem + lane_base + cc, v);
            tmem_wait_ld();
            if (real) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t o[8];
#pragma unroll
                for (int c = 0; c < 8; ++c)
                  o[c] = l == 0.0f ? 0u : tree_pack<kBf>(__uint_as_float(v[16 * h + 2 * c]) * inv, __uint_as_float(v[16 * h + 2 * c + 1]) * inv);
                uint4 *to = reinterpret_cast<uint4 *>(a.out + at * D + cc + 16 * h);
                to[0] = make_uint4(o[0], o[1], o[2], o[3]);
                to[1] = make_uint4(o[4], o[5], o[6], o[7]);
              }
            }
          }
          if (real && grp == 0 && a.lse) a.lse[at] = l == 0.0f ? -INFINITY : (m_ref + log2f(l)) * 0.693147180559945309f;
        } else {
          const int ps = 2 * (int)blockIdx.x + s.slot;
          float *part = a.part + (size_t)ps * tree_part_floats(D) + (size_t)row * D;
#pragma unroll 1
          for (int cc = grp * DH; cc < grp * DH + DH; cc += 32) {
            uint32_t v[32];
            tmem_ld32(tmem + lane_base + cc, v);
            tmem_wait_ld();
            if (real) {
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                uint32_t o[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) o[c] = l == 0.0f ? 0u : v[8 * h + c];
                st_global_v8(part + cc + 8 * h, o);
              }
            }
          }
          float2 *ml = reinterpret_cast<float2 *>(a.part + (size_t)ps * tree_part_floats(D) + (size_t)kTreeRows * D) + row;
          if (real && grp == 0) *ml = make_float2(m_ref, l);
          if (s.slot == 1) {
            desc.tok0 = s.tok0;
            desc.col0 = s.rb * a.block_rows;
            desc.cols = min(s.nodes * a.G - s.rb * a.block_rows, a.block_rows);
            desc.g = s.g;
            desc.parts = s.parts;
            desc.step = ctl->size;
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_free);
        tiles += n;
      }
      ok = !aborted;
    }
    nsegs += nseg;
    if (!ctl->more) break;
    __syncthreads();                              // everyone has done the list
    if (threadIdx.x == 0) tree_walk(a, segs, ctl);
    __syncthreads();
    if (ctl->nseg == 0 && !ctl->more) break;
  }

  // what was started ends before the CTA does
  // (the MMAs have waited for all copies, unless a wait gave up)
  if (warp >= Sh::kLoadWarp && warp < Sh::kWiden0 && wctl->abort) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    const int isv = lane >= 8, ring = max(kI8 ? isv ? Sh::kRawV : Sh::kRawK : F, 1);
    if (last >= 0) mbar_drain(kI8 ? raw_full(isv, lane & 7) : full(isv, lane & 7), (uint32_t)((last / ring) & 1), wctl);
    if (lane == 0 && queries > 0) mbar_drain(q_full, (uint32_t)((queries - 1) & 1), wctl);
  }
  if (warp == Sh::kMmaWarp) {
    const uint32_t leader = elect_leader();
    mma_commit_w(leader, drain);
    mbar_drain(drain, 0u, wctl);
  }
  if (threadIdx.x == 0) a.desc[blockIdx.x] = desc;
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, Sh::kTmem);
  }
}

// ------------------------------------------------------------------ the join --
// A warp a row of the item whose first part CTA blockIdx.x of attn_tree_kernel left: its parts are
// that CTA's second slot and the first slots of the same member of the next teams.
constexpr int kJoinWarps = 8;
template <int D, bool BF>
__global__ void __launch_bounds__(32 * kJoinWarps) attn_tree_join_kernel(const __grid_constant__ TreeArgs a) {
  constexpr int PER = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_wait();
  griddep_launch_dependents();
  const TreeDesc d = a.desc[blockIdx.x];
  const size_t size = tree_part_floats(D);
  auto part = [&](int k) { return a.part + (size_t)(k == 0 ? 2 * (int)blockIdx.x + 1 : 2 * ((int)blockIdx.x + k * d.step)) * size; };
  const int r = blockIdx.y * kJoinWarps + warp;
  if (r < d.cols) {
    // the parts' references and sums, 32 at a time
    auto head_of = [&](int k) { return k < d.parts ? reinterpret_cast<const float2 *>(part(k) + (size_t)kTreeRows * D)[r] : make_float2(kTreeNoScore, 0.0f); };
    const float2 first = head_of(lane);
    float m = first.x;
    for (int k = lane + 32; k < d.parts; k += 32) m = fmaxf(m, head_of(k).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = 0.0f, acc[PER] = {};
    for (int k0 = 0; k0 < d.parts; k0 += 32) {
      const float2 ml = k0 == 0 ? first : head_of(k0 + lane);
      const float w = k0 + lane < d.parts ? tree_ex2(ml.x - m) : 0.0f, lk = ml.y * w;
      const int n = min(d.parts - k0, 32);
#pragma unroll 8
      for (int k = 0; k < n; ++k) {
        const float *p = part(k0 + k) + (size_t)r * D + lane * PER;
        const float f = __shfl_sync(0xffffffffu, w, k);
        l += __shfl_sync(0xffffffffu, lk, k);
        float x[PER];
        if constexpr (PER == 2) {
          const float2 v = *reinterpret_cast<const float2 *>(p);
          x[0] = v.x;
          x[1] = v.y;
        } else {
#pragma unroll
          for (int q = 0; q < PER / 4; ++q) {
            const float4 v = reinterpret_cast<const float4 *>(p)[q];
            x[4 * q] = v.x;
            x[4 * q + 1] = v.y;
            x[4 * q + 2] = v.z;
            x[4 * q + 3] = v.w;
          }
        }
#pragma unroll
        for (int c = 0; c < PER; ++c) acc[c] = fmaf(f, x[c], acc[c]);
      }
    }
    const int col = d.col0 + r, node = col / a.G, head = d.g * a.G + col - node * a.G;
    const long long at = (long long)(d.tok0 + node) * a.Hq + head;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint32_t o[PER / 2];
#pragma unroll
    for (int c = 0; c < PER / 2; ++c) o[c] = tree_pack<BF>(acc[2 * c] * inv, acc[2 * c + 1] * inv);
    uint32_t *to = reinterpret_cast<uint32_t *>(a.out + at * D) + lane * (PER / 2);
    if constexpr (PER == 8) *reinterpret_cast<uint4 *>(to) = make_uint4(o[0], o[1], o[2], o[3]);
    else if constexpr (PER == 4) *reinterpret_cast<uint2 *>(to) = make_uint2(o[0], o[1]);
    else *to = o[0];
    if (a.lse && lane == 0) a.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
  }
}

template <int D, int KV>
cudaError_t launch_tree(const TreeArgs &a, int grid, cudaStream_t st) {
  using Sh = TreeShape<D, KV>;
  const void *f = reinterpret_cast<const void *>(attn_tree_kernel<D, KV>);
  cudaError_t e = ensure_smem_attr(f, Sh::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(f, dim3(grid), dim3(Sh::kThreads), Sh::kSmem, st, a);
  count_launch();
  if (e != cudaSuccess) return e;
  e = launch_pdl(reinterpret_cast<const void *>(attn_tree_join_kernel<D, KV == kPagedBf16>), dim3(grid, kTreeRows / kJoinWarps), dim3(32 * kJoinWarps),
                 0, st, a);
  count_launch();
  return e;
}
template <int KV>
cudaError_t launch_tree_kv(const TreeArgs &a, int d, int grid, cudaStream_t st) {
  return d == 64 ? launch_tree<64, KV>(a, grid, st) : d == 128 ? launch_tree<128, KV>(a, grid, st) : launch_tree<256, KV>(a, grid, st);
}

}  // namespace qw
