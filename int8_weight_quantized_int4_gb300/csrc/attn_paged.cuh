// attn_paged.cuh -- attention of each sequence's new tokens over a paged key-value cache.
//
// For query head h of a new token at position pos of its sequence, KV head g = h / G
// (G = Hq / Hkv), over the keys j it can see (j <= pos and, with a window W, j > pos - W or
// j < sinks):
//   x_j = q . k_j * scale,  p_j = e^(x_j - m),  out = sum_j p_j v_j / sum_j p_j.
// One pass over K and V: a running reference m of the exponents (moved only when a score
// passes it by 2^8, in fp16 2^15, which rescales the sums), the sums in binary32.
//
// What bounds it: reading K and V, 2 S d e bytes a (sequence, KV head) for 4 S d flops a
// query row -- a few rows a KV head (G x new tokens), so 1..64 flops a byte, far below the
// ridge of any matrix unit here (warp-level MMA: 606 TFLOP/s measured against 6.7 TB/s, 90
// flops a byte).  So the design is about keeping loads in flight and instructions few:
//   - The G heads and the new tokens of a sequence that share a KV head are the columns of an
//     MMA whose rows are keys (S^T = K Q^T) and then channels (O^T = V^T P^T), so K and V are
//     read once for all of them and eight columns (the common case, G <= 8) cost half of what
//     a 16-row query tile would, in instructions and in accumulator registers.
//   - One CTA, or up to four (paged_launch), share an SM.  Each of its KW groups streams its own strips of 16 keys through its
//     own ring of half stages (the K rows, then the V rows of a strip; cp.async, 16 bytes a
//     thread; rows beyond the visible keys are zero-filled, not read) and waits only for
//     itself: no CTA-wide barrier between the strips of a sequence.  A group is one warp, but
//     where 16 columns of d = 256 would fill a thread's registers, two warps halve the channels
//     (of both products: the halves' scores meet in shared memory), which lets twelve warps
//     hide each other's waits where six could not.
//   - More than 16 columns are dealt to the groups in blocks of 16: the groups of different
//     blocks stream the same strips at the same time, the first from HBM and the others from
//     L2.  (16 sequences of up to 16384, 6 to 36 columns, d = 256, with one product a weight: 149
//     us.  As items of their own the blocks came too far apart, 5 % L2 hits and 21 us more; groups
//     of two to four warps with 16 columns each, reading a strip once for all of them, took 188
//     to 421 us, rings shared through counting barriers 151 at best.)
//   - Work is split evenly over the SMs whatever the lengths: the visible strips of every
//     (sequence, column block, KV head) item are laid end to end and cut into one equal range
//     a CTA (every CTA finds its own range from the lengths on the device, so a captured graph
//     follows growing contexts).  An item that a range border cuts leaves partial sums (m, l,
//     O) in the workspace, and the last CTA to finish it joins them in CTA order: results do
//     not depend on arrival order.
//   - The ring runs ahead across item borders, so the next item's keys arrive while one item
//     is being finished.
//
// Measured (K and V rows read / time): 64 ragged contexts of up to 8190, 32/8 heads of 128, bf16:
// 177 to 183 us, 6.3 to 6.5 TB/s; 4 of up to 131071, 24/4 heads of 256, int8: 116 us, 5.75 TB/s (the
// codes' conversion to fp16 takes half of the issue slots); 16 of up to 16384 with up to 6 new
// tokens, fp16: 157 us, 4.5 TB/s (up to 36 columns: a strip is read once from HBM and up to
// twice more from L2, at 31 bytes a clock an SM with one product a weight); a window of
// 1024, 48 contexts, 64/8 heads of 64, fp16: 26.9 us, 3.7 TB/s (items of 66 strips: their
// starts and joins); one context of 1003, 24/4 heads of 256, fp16: 12.2 us, nearly all of it the
// chain launch -> lengths -> page table -> keys -> exchange -> partial sums -> join.
//
// Roundings: each weight enters P.V as two terms of the values' 16-bit type, p rounded and what
// that leaves, so it keeps 22 bits (bf16 16) where one term has 11 (8): all products are exact and
// all sums binary32, and the output's own rounding is what remains (one term gave 1.32 times the
// error of a binary32 softmax in fp16 and 1.26 in bf16, against binary64; two give 1.00).  The
// second product costs nothing where 8 columns read at HBM's rate, 3.5 % for int8 and 6 % for up to
// 36 columns of d = 256.  fp16 has no relative bound below 2^-14, and rounds what lies below 2^-25
// to 0, always the same way: the reference starts 2^7 below the largest score, so that only
// weights below 2^-32 of it are lost (131k of them hold 2^-15 of the mass; with the reference at
// the largest it was 2^-8), and weights stay below 2^15.  bf16 has binary32's exponents.  With the
// int8 cache the value's scale joins its weight (w_j = p_j vs_j) and the reference follows w_j,
// not p_j, so that w keeps its bits whatever the scales' size.
#pragma once
#include <stdint.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "launch.h"
#include "ptx.cuh"

namespace qw {

constexpr int kPagedMaxSegs = 32;       // work segments listed at a time
constexpr int kStrip = 16;              // keys of a strip: the MMA's rows of S^T, its depth of O^T
constexpr int kPagedSmem = 227 * 1024;
constexpr float kNoScore = -3.402823466e38f;   // the reference of a sum of nothing: the lowest finite score

struct PagedSeg {
  int b, g, rb;                 // sequence, KV head, block of kRows columns
  int nblk;                     // blocks of kCols columns in it
  int u0, u1;                   // strips of the item [u0, u1)
  int nsu, first;               // strips of the sinks, strip of the first windowed key
  int lo, hi;                   // visible keys of the column block: [lo, hi) and below `sinks`
  int pos0, rows;               // position of the sequence's first new token; its query columns
  int tok0;                     // its first row in q and out
  int c0, c1;                   // CTAs holding the item's first and last strip
};

// A CTA's list of work and the state to list the rest, in shared memory.
struct PagedCtl {
  int nseg, more;               // segments listed; whether others follow
  int njoin, last;              // groups of parts this CTA was the last to finish
  PagedSeg join[2];             // their items
  int group[2];                 // and the first part of each
  int b;                        // walk: sequence
  int off, pos;                 // walk: place in the sequence, in all
  int begin, end, share;        // the range
  int part[16];
};

// Shapes.  NB: MMA column tiles (of 8) a warp; GW: warps of a group, which share the channels.
// The warps an SM has are what the registers allow: accumulators take D NB / 4 / GW registers a
// thread and the Q fragments half of that.  CTAS: CTAs that share it.
template <int D, int KV, int NB, int CTAS>
struct PagedShape {
  static constexpr int kES = KV == kPagedI8 ? 1 : 2;
  static constexpr int kGW = D * NB == 512 ? 2 : 1;
  static constexpr int kMaxWarps = (D * NB >= 256 ? 12 : 16) / CTAS;
  static constexpr int kKW = kMaxWarps / kGW;
  static constexpr int kWarps = kGW * kKW;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kCols = 8 * NB;                 // columns a group
  // columns of an item, at most (kernels of 8 are called for up to 8: then the blocks' logic is
  // left out, 1 to 3 us a call)
  static constexpr int kRows = NB == 1 ? kCols : 4 * kCols;
  static_assert(NB == 1 || kKW >= 4, "a group a block");
  static constexpr int kRowBytes = D * kES;
  static constexpr int kHalf = kStrip * kRowBytes + (KV == kPagedI8 ? 2 * kStrip * 4 : 0);      // (whole 128 bytes)
  // the exchange at an item's end: SW channels of each warp at a time, rows of SW + 4 floats
  // (column pairs 2 c and channels r8 of a warp's lanes fall on distinct banks); in between it
  // holds the halves' scores
  static constexpr int kSW = D == 64 || kWarps * kCols * 68 * 4 <= 28 * 1024 ? 64 : 32;
  static constexpr int kRedBytes = kWarps * kCols * (kSW + 4) * 4;
  static_assert(kGW == 1 || kWarps * NB * 512 <= kRedBytes, "room for the scores");
  static constexpr int kFixed = kRedBytes + 2 * kWarps * kCols * 4 + kRows * 8 + kPagedMaxSegs * (int)sizeof(PagedSeg) + (int)sizeof(PagedCtl);
  static constexpr int kFit = (kPagedSmem / CTAS - (CTAS - 1) * 1024 / CTAS - kFixed) / (kKW * kHalf);
  static constexpr int kRing = kFit > 12 ? 12 : kFit;  // half stages a group
  static constexpr int kSmem = kFixed + kRing * kKW * kHalf;
  static_assert(kRing >= (kGW > 1 ? 3 : 2), "K and V of a strip in flight");
  // What an item costs beside its strips, in strips: the groups that wait for the last one, its
  // join and the next Q take an SM about the time of 192 KB (64 x 8k bf16, one CTA an SM: 202 us
  // with 64 KB, 196 with 128, 193 with 192, 188 with 256; 4 x 128k int8: 119, 117, 117, 124; four CTAs,
  // 200 x 700: 63 with 128, 58 with 192, 57 with 288, and 48 x 1024 of d = 64: 19.8, 19.4, 22.3).
  static constexpr int kItemCost = 196608 / CTAS / (2 * kStrip * kRowBytes);
  static constexpr size_t kPartFloats = (size_t)kRows * (D + 2);
};

__device__ __forceinline__ float paged_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float paged_lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
template <bool BF>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  if constexpr (BF) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&v);
  } else {
    const __half2 v = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&v);
  }
}
template <bool BF>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (BF) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  else return __half22float2(u32_as_h2(w));
}
// Two int8 codes of a word (xor 0x80 applied: u = code + 128) as an fp16 pair: 0x6400 | u
// is 1024 + u exactly, minus 1152.  SEL picks the two bytes.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t codes_f16(uint32_t u) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(u), "r"(0x64646464u), "n"(SEL));
  return h2_as_u32(__hsub2(u32_as_h2(r), u32_as_h2(0x64806480u)));
}
__device__ __forceinline__ void cp_async16_full(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 4-byte asynchronous copy (zero-filled when src_bytes is 0)
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, uint32_t src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}

// Byte offset of 16-byte chunk c of row r in a strip: chunks of eight consecutive rows at
// one chunk index fall on distinct bank groups, for ldmatrix.
template <int RB>
__device__ __forceinline__ uint32_t strip_off(int r, int c) {
  if constexpr (RB >= 128) return (uint32_t)(r * RB + ((c ^ (r & 7)) << 4));
  else return (uint32_t)(r * RB + ((c ^ ((r >> 1) & 3)) << 4));      // 64-byte rows: two a bank line
}

// 8 x 8 matrix of 16-bit elements, a row pair a lane, transposed across the warp.
__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Whether a strip of 16 value rows (16-bit) holds an infinity or a NaN; whole warp.
template <int D, bool BF>
__device__ __noinline__ bool strip_nonfinite(uint32_t vst, int lane) {
  const uint32_t e = BF ? 0x7f80u : 0x7c00u;
  bool bad = false;
  for (int i = lane; i < 16 * D / 2; i += 32) {
    uint32_t w;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(vst + 4 * i) : "memory");
    bad |= (w & e) == e || ((w >> 16) & e) == e;
  }
  return __any_sync(0xffffffffu, bad);
}
// acc += V^T P^T of one strip over the visible keys alone (score above -inf), term by term.
// s[nb]: the scores of keys r8 + 8 h and columns 2 c4, 2 c4 + 1; m: those columns' references.
// n0: the warp's first chunk of 8 channels.
template <int D, int DT, int NB, bool BF>
__device__ __forceinline__ void add_visible(float (&acc)[DT][NB][4], const float (&s)[NB][4], const float (&m)[NB][2],
                                            uint32_t vst, int n0, int lane) {
  const int c4 = lane & 3, r8 = lane >> 2;
#pragma unroll 1
  for (int j = 0; j < kStrip; ++j) {
    const int src = (j & 7) * 4 + c4, h = j >> 3;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const float s0 = __shfl_sync(0xffffffffu, h ? s[nb][2] : s[nb][0], src);
      const float s1 = __shfl_sync(0xffffffffu, h ? s[nb][3] : s[nb][1], src);
      const float w0 = paged_ex2(s0 - m[nb][0]), w1 = paged_ex2(s1 - m[nb][1]);
#pragma unroll
      for (int n = 0; n < 2 * DT; ++n) {             // channel 8 n + r8: rows r8 (+ 8) of tile n / 2
        unsigned short v;
        asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(vst + strip_off<D * 2>(j, n0 + n) + 2 * r8) : "memory");
        const float f = BF ? __uint_as_float((uint32_t)v << 16) : __half2float(__ushort_as_half(v));
        float(&a)[4] = acc[n / 2][nb];
        if (s0 != -INFINITY) a[2 * (n & 1)] = fmaf(w0, f, a[2 * (n & 1)]);
        if (s1 != -INFINITY) a[2 * (n & 1) + 1] = fmaf(w1, f, a[2 * (n & 1) + 1]);
      }
    }
  }
}

// Chunk s of a row, s = 2 k + h (k the MMA step, h this lane's half): the offsets of steps
// 0 .. 3; step k is 128 (k / 4) bytes past step k % 4 (the swizzle permutes 128 bytes).
template <int RB>
struct LaneOffs {
  uint32_t x[RB >= 128 ? 4 : 2];
  __device__ __forceinline__ LaneOffs(int row, int half) {
#pragma unroll
    for (int k = 0; k < (RB >= 128 ? 4 : 2); ++k) x[k] = strip_off<RB>(row, 2 * k + half);
  }
  __device__ __forceinline__ uint32_t operator()(int k) const { return x[k % (RB >= 128 ? 4 : 2)] + (uint32_t)(k / 4 * 128); }
};

// --------------------------------------------------------------- the schedule --
// a / b for 0 <= a, 0 < b.  Below 2^22 by a binary32 quotient, at most one off, and its
// remainder: a fraction of the general division's latency, which a short call waits for.
__device__ __forceinline__ int paged_div(int a, int b) {
  if ((unsigned)(a | b) >> 22) return (int)((unsigned)a / (unsigned)b);
  int q = (int)__fdividef((float)a, (float)b);
  const int r = a - q * b;
  q += r >= b;
  q -= r < 0;
  return q;
}

// Sequence b's new tokens and keys, clamped to what the buffers hold (a length beyond the
// page table or offsets out of order record QW_ERR_BAD_INDEX).
struct PagedSeq {
  int tok0, nq, len;
};
__device__ __forceinline__ PagedSeq paged_seq(const PagedArgs &a, int b) {
  PagedSeq s;
  const int c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1), n = __ldg(a.lens + b);
  s.tok0 = min(max(c0, 0), a.T);
  s.nq = max(min(max(c1, 0), a.T) - s.tok0, 0);
  s.len = min(max(n, 0), a.cap);
  if (c0 != s.tok0 || c1 != s.tok0 + s.nq || n != s.len) atomicCAS(a.err, 0, -9);
  return s;
}
struct PagedSpan {
  int lo, hi, nsu, first, n;
};
// The keys that column block rb can see and their strips.
template <int ROWS>
__device__ __forceinline__ PagedSpan paged_span(const PagedArgs &a, const PagedSeq &s, int rb) {
  PagedSpan p;
  const int rows = s.nq * a.G, pos0 = s.len - s.nq;
  int t0 = 0, t1 = s.nq - 1;                            // its first and last token
  if (rows > ROWS) {
    t0 = paged_div(rb * ROWS, a.G);
    t1 = paged_div(min(rows, rb * ROWS + ROWS) - 1, a.G);
  }
  p.hi = max(pos0 + t1 + 1, 0);
  p.lo = a.window > 0 ? max(pos0 + t0 - a.window + 1, 0) : 0;
  p.first = p.lo / kStrip;
  p.nsu = min((min(a.sinks, p.hi) + kStrip - 1) / kStrip, p.first);
  p.n = max(p.nsu + (p.hi + kStrip - 1) / kStrip - p.first, 1);      // an item with no key still writes its rows
  return p;
}

// Blocks of a group's columns in block rb of a sequence's `rows` columns.
template <int ROWS>
__device__ __forceinline__ int paged_blocks(int rows, int rb) {
  return ROWS == 8 ? 1 : (min(rows - rb * ROWS, ROWS) + 15) / 16;
}
template <int ROWS>
__device__ __forceinline__ void paged_fill(PagedSeg &g, const PagedSeq &s, const PagedSpan &p, int b, int rb, int head,
                                          int G) {
  g.b = b;
  g.rb = rb;
  g.g = head;
  g.nsu = p.nsu;
  g.first = p.first;
  g.lo = p.lo;
  g.hi = p.hi;
  g.pos0 = s.len - s.nq;
  g.rows = s.nq * G;
  g.nblk = paged_blocks<ROWS>(g.rows, rb);
  g.tok0 = s.tok0;
}


// Places: a strip takes as many as its item has column blocks w (its groups' work), an item IC
// more by itself.  They are counted in units of 2^shift (shift is 0 unless all keys of a call
// could pass 2^30 places).
__device__ __forceinline__ int paged_places(const PagedArgs &a, int n, int w) { return (n * w + (1 << a.shift) - 1) >> a.shift; }
// the strips that end within the first x places of an item's strips
__device__ __forceinline__ int paged_strips(const PagedArgs &a, int x, int w) { return w == 1 ? x << a.shift : paged_div(x << a.shift, w); }

// One segment: the strips of the item that starts at place `at` which lie in the range; false
// if there are none.
template <int ROWS, int IC>
__device__ __forceinline__ bool paged_emit(const PagedArgs &a, PagedSeg &g, const PagedSeq &s, const PagedSpan &p, int b,
                                           int rb, int head, int at, int begin, int end, int share) {
  const int w = paged_blocks<ROWS>(s.nq * a.G, rb), n = paged_places(a, p.n, w), x1 = min(end - at - IC, n);
  const int u0 = paged_strips(a, max(begin - at - IC, 0), w), u1 = x1 == n ? p.n : paged_strips(a, x1, w);
  if (u0 >= u1) return false;
  g.u0 = u0;
  g.u1 = u1;
  g.c0 = u0 == 0 ? (int)blockIdx.x : paged_div(at + IC + paged_places(a, 1, w) - 1, share);
  g.c1 = u1 == p.n ? (int)blockIdx.x : paged_div(at + IC + n - 1, share);
  paged_fill<ROWS>(g, s, p, b, rb, head, a.G);
  return true;
}
// Parts of an item of n strips when CTAs of their own take `size` places, and their strips.
__device__ __forceinline__ int paged_parts(const PagedArgs &a, int n, int w, int size, int &len) {
  const int np = paged_div(paged_places(a, n, w) + size - 1, size);
  len = paged_div(n + np - 1, np);
  return paged_div(n + len - 1, len);
}

// Lists the range's next segments (one thread).
template <int ROWS, int IC>
__device__ __forceinline__ void paged_walk(const PagedArgs &a, PagedSeg *segs, PagedCtl *ctl) {
  int n = 0, b = ctl->b, off = ctl->off, pos = ctl->pos;
  const int end = ctl->end;
#pragma unroll 1
  while (pos < end && n < kPagedMaxSegs) {
    const PagedSeq s = paged_seq(a, b);
    const int nrb = (s.nq * a.G + ROWS - 1) / ROWS;
    int o = off, rb = 0, each = 1;
    PagedSpan p{};
#pragma unroll 1
    for (; rb < nrb; ++rb) {
      p = paged_span<ROWS>(a, s, rb);
      each = paged_places(a, p.n, paged_blocks<ROWS>(s.nq * a.G, rb)) + IC;
      if (o < each * a.Hkv) break;
      o -= each * a.Hkv;
    }
    if (rb == nrb) {
      ++b;
      off = 0;
      continue;
    }
    const int head = paged_div(o, each), in = o - head * each;
    // (a range may end among an item's first places)
    if (pos - in + IC < end && paged_emit<ROWS, IC>(a, segs[n], s, p, b, rb, head, pos - in, ctl->begin, end, ctl->share)) ++n;
    pos += each - in;
    off += each - in;
  }
  ctl->nseg = n;
  ctl->more = pos < end;
  ctl->b = b;
  ctl->off = off;
  ctl->pos = pos;
}

// This CTA's work: its first segments and the state to list the others; false: none.  The
// places of all items, in order, are cut into equal ranges -- or, where that costs little more
// than the equal share, each item gets CTAs of its own: no CTA then finishes two items one
// after the other, which is what a short call would wait for.  Up to 32 sequences one warp
// does it, a sequence a lane; otherwise the CTA, one or more sequences a thread.
template <int ROWS, int IC, int NW>
__device__ __forceinline__ bool paged_schedule(const PagedArgs &a, PagedSeg *segs, PagedCtl *ctl) {
  constexpr int NT = 32 * NW;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    ctl->nseg = ctl->more = ctl->njoin = 0;
  }
  __syncwarp();                  // before the first warp's other lanes count up (shuffles order no memory)
  if (a.B > 32 || warp == 0) {
    const int per = a.B > 32 ? (a.B + NT - 1) / NT : 1;
    const int b_lo = min(tid * per, a.B), b_hi = min(b_lo + per, a.B);
    auto blocks = [&](const PagedSeq &s) { return (s.nq * a.G + ROWS - 1) / ROWS; };
    auto cost = [&](const PagedSeq &s) {
      int c = 0;
#pragma unroll 1
      for (int rb = 0, n = blocks(s); rb < n; ++rb) c += paged_places(a, paged_span<ROWS>(a, s, rb).n, paged_blocks<ROWS>(s.nq * a.G, rb)) + IC;
      return c * a.Hkv;
    };
    // Sums stop past kPagedMaxPlaces.  Offsets in order stay below it (the host's shift); sequences
    // whose offsets overlap could name more tokens than there are, and pass 2^31.
    auto add = [](int x, int y) { return (int)min((unsigned)x + (unsigned)y, kPagedMaxPlaces + 1u); };
    // sums before this thread and over all (of the warp, or through shared memory)
    auto scan = [&](int v, int &before, int &all) {
      int inc = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc = add(inc, t);
      }
      before = inc - v;
      all = __shfl_sync(0xffffffffu, inc, 31);
      if (a.B > 32) {
        __syncthreads();
        if (lane == 0) ctl->part[warp] = all;
        __syncthreads();
        all = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const int x = ctl->part[w];
          before = add(before, w < warp ? x : 0);
          all = add(all, x);
        }
      }
    };
    PagedSeq own{};                                     // per == 1: this thread's sequence
    PagedSpan first{};                                  // and its first block's keys
    int mine = 0, items = 0;
#pragma unroll 1
    for (int b = b_lo; b < b_hi; ++b) {
      own = paged_seq(a, b);
      const int n = blocks(own);
      if (n == 1) {
        first = paged_span<ROWS>(a, own, 0);
        mine = add(mine, (paged_places(a, first.n, paged_blocks<ROWS>(own.nq * a.G, 0)) + IC) * a.Hkv);
      } else {
        mine = add(mine, cost(own));
      }
      items += n * a.Hkv;
    }
    auto span = [&](int rb) { return blocks(own) == 1 ? first : paged_span<ROWS>(a, own, rb); };
    int pre, total, dummy, all_items;
    scan(mine, pre, total);
    if (a.B > 32) scan(min(items, 1 << 16), dummy, all_items);
    else all_items = __reduce_add_sync(0xffffffffu, min(items, 1 << 16));
    const int grid = gridDim.x, me = blockIdx.x;
    const int share = max(paged_div(total + grid - 1, grid), a.min_places);
    // places a CTA takes when items have CTAs of their own (the items' parts then fit the grid)
    const int left = grid - all_items;
    const int size = per == 1 && left > 0 && a.shift == 0 ? max(paged_div(total - IC * all_items + left - 1, left), a.min_places) : 0;
    if (total > (int)kPagedMaxPlaces) {
      // offsets that overlap (recorded by paged_seq): no places to cut, so nothing is computed
    } else if (size > 0 && size <= share + 2 * IC) {
      int parts = 0, pp;
#pragma unroll 1
      for (int rb = 0, n = blocks(own), len; rb < n; ++rb)
        parts += paged_parts(a, span(rb).n, paged_blocks<ROWS>(own.nq * a.G, rb), size, len) * a.Hkv;
      scan(parts, pp, dummy);
      if (me >= pp && me < pp + parts) {                // one thread, if any
        int at = pp;
#pragma unroll 1
        for (int rb = 0, n = blocks(own); rb < n; ++rb) {
          const PagedSpan p = span(rb);
          int len;
          const int np = paged_parts(a, p.n, paged_blocks<ROWS>(own.nq * a.G, rb), size, len);
          if (me < at + np * a.Hkv) {
            PagedSeg &g = segs[0];
            const int head = paged_div(me - at, np), j = me - at - head * np;
            g.u0 = j * len;
            g.u1 = min(p.n, g.u0 + len);
            g.c0 = me - j;
            g.c1 = g.c0 + np - 1;
            paged_fill<ROWS>(g, own, p, b_lo, rb, head, a.G);
            ctl->nseg = 1;
            break;
          }
          at += np * a.Hkv;
        }
      }
    } else {
      const int begin = (int)min((long long)share * me, (long long)total), end = min(total - begin, share) + begin;
      // Up to a sequence a thread and kPagedMaxSegs segments: every thread lists its own
      // sequence's (in any order); otherwise thread 0 walks, a list at a time.
      if (begin < end && pre < end && begin < pre + mine) {
        int at = pre;
        if (per == 1) {
#pragma unroll 1
          for (int rb = 0, n = blocks(own); rb < n && at < end; ++rb) {
            const PagedSpan p = span(rb);
            const int each = paged_places(a, p.n, paged_blocks<ROWS>(own.nq * a.G, rb)) + IC;
            int head = begin > at ? min(paged_div(begin - at, each), a.Hkv) : 0;
            int x = at + head * each;
#pragma unroll 1
            for (; head < a.Hkv && x + IC < end; ++head, x += each)
              if (x + each > begin) {
                PagedSeg g;
                if (paged_emit<ROWS, IC>(a, g, own, p, b_lo, rb, head, x, begin, end, share)) {
                  const int i = atomicAdd(&ctl->nseg, 1);
                  if (i < kPagedMaxSegs) segs[i] = g;
                }
              }
            at += a.Hkv * each;
          }
        }
        if (begin >= pre) {                             // the owner of the range's first place
          int off = begin - pre, b = b_lo;
          if (per > 1) {
#pragma unroll 1
            for (; b + 1 < b_hi; ++b) {
              const int c = cost(paged_seq(a, b));
              if (off < c) break;
              off -= c;
            }
            ctl->more = 1;
          }
          ctl->b = b;
          ctl->off = off;
          ctl->pos = ctl->begin = begin;
          ctl->end = end;
          ctl->share = share;
        }
      }
    }
  }
  __syncthreads();
  if (ctl->nseg > kPagedMaxSegs) {                      // too many: walk instead
    __syncthreads();
    if (tid == 0) {
      ctl->nseg = 0;
      ctl->more = 1;
    }
    __syncthreads();
  }
  return ctl->nseg != 0 || ctl->more != 0;
}

// More than 16 parts of a cut item are joined in groups of 2^this, then the groups: one CTA
// reading 152 parts took longer than all the rest (131k keys of one KV head of 128: 51 us, in
// groups of 16 31; of 256 with 64 columns, 60k keys: 207 and 89).
__device__ __forceinline__ int paged_group(int parts) { return parts <= 16 ? 4 : parts <= 64 ? 3 : parts <= 256 ? 4 : 5; }

// Joins n parts of a cut item, first, first + step, .., in order (all threads of the last CTA to
// finish them): the item's rows, or (not FINAL) one part in place of the first.
template <int D, int KV, int NB, int CTAS>
__device__ __forceinline__ void paged_join(const PagedArgs &a, const PagedSeg &g, int first, int step, int n, bool final,
                                           float *red) {
  using P = PagedShape<D, KV, NB, CTAS>;
  constexpr int NT = P::kThreads, ROWS = P::kRows;
  constexpr bool BF = KV == kPagedBf16;
  const int tid = threadIdx.x, lane = tid & 31;
  const int row0 = g.rb * ROWS, nrows = min(ROWS, g.rows - row0);
  // the item's first part is in its CTA's slot 1, the others in their slots 0
  auto slot = [&](int i) {
    const int k = first + i * step;
    return a.part + (size_t)(2 * (g.c0 + k) + (k == 0 ? 1 : 0)) * P::kPartFloats;
  };
  // `chunk` columns at a time: their parts' m and l in shared memory, then each part's weight
  const int chunk = min(nrows, P::kRedBytes / 8 / n);
  float *mm = red, *ll = red + chunk * n;
#pragma unroll 1
  for (int r0 = 0; r0 < nrows; r0 += chunk) {
    const int nr = min(chunk, nrows - r0);
#pragma unroll 1
    for (int i = tid; i < n * nr; i += NT) {
      const int k = i / nr, r = i - k * nr;
      const float *s = slot(k) + r0 + r;
      mm[k * nr + r] = __ldcg(s);
      ll[k * nr + r] = __ldcg(s + ROWS);
    }
    __syncthreads();
    // eight lanes a column
#pragma unroll 1
    for (int r = tid >> 3; r < (nr + 3) / 4 * 4; r += NT / 8) {       // whole warps
      const int e = lane & 7;
      float Mx = kNoScore, Ls = 0.0f;
      if (r < nr)
#pragma unroll 1
        for (int k = e; k < n; k += 8) Mx = fmaxf(Mx, mm[k * nr + r]);
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) Mx = fmaxf(Mx, __shfl_xor_sync(0xffffffffu, Mx, o));
      if (r < nr)
#pragma unroll 1
        for (int k = e; k < n; k += 8) {
          const float w = paged_ex2(mm[k * nr + r] - Mx);
          Ls += ll[k * nr + r] * w;
          mm[k * nr + r] = w;
        }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) Ls += __shfl_xor_sync(0xffffffffu, Ls, o);
      if (!final) {
        if (r < nr && e == 0) {
          slot(0)[r0 + r] = Mx;
          slot(0)[ROWS + r0 + r] = Ls;
        }
        continue;
      }
      const float inv = Ls == 0.0f ? 0.0f : 1.0f / Ls;
      if (r < nr)
#pragma unroll 1
        for (int k = e; k < n; k += 8) mm[k * nr + r] *= inv;
      if (a.lse && r < nr && e == 0) {
        const int gr = row0 + r0 + r;
        a.lse[(long long)(g.tok0 + gr / a.G) * a.Hq + g.g * a.G + gr % a.G] =
            Ls > 0.0f || Ls != Ls ? (Mx + log2f(Ls)) * 0.6931471805599453f : -INFINITY;
      }
    }
    __syncthreads();
#pragma unroll 1
    for (int i = tid; i < nr * (D / 4); i += NT) {
      const int r = i / (D / 4);
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
      for (int k0 = 0; k0 < n; k0 += 8) {            // eight parts in flight
        float4 v[8];
#pragma unroll
        for (int x = 0; x < 8; ++x)
          if (k0 + x < n)
            v[x] = __ldcg(reinterpret_cast<const float4 *>(slot(k0 + x) + 2 * ROWS + (size_t)r0 * D) + i);
#pragma unroll
        for (int x = 0; x < 8; ++x)
          if (k0 + x < n) {
            const float w = mm[(k0 + x) * nr + r];
            o.x += v[x].x * w;
            o.y += v[x].y * w;
            o.z += v[x].z * w;
            o.w += v[x].w * w;
          }
      }
      if (!final) {
        reinterpret_cast<float4 *>(slot(0) + 2 * ROWS + (size_t)r0 * D)[i] = o;
        continue;
      }
      const int gr = row0 + r0 + r;
      uint16_t *dst = a.out + ((long long)(g.tok0 + gr / a.G) * a.Hq + g.g * a.G + gr % a.G) * D + 4 * (i % (D / 4));
      *reinterpret_cast<uint2 *>(dst) = make_uint2(pack2<BF>(o.x, o.y), pack2<BF>(o.z, o.w));
    }
    __syncthreads();
  }
}

template <int D, int KV, int NB, int CTAS>
__global__ void __launch_bounds__(PagedShape<D, KV, NB, CTAS>::kThreads, CTAS)
    attn_paged_kernel(const __grid_constant__ PagedArgs a) {
  using P = PagedShape<D, KV, NB, CTAS>;
  constexpr bool BF = KV == kPagedBf16;
  constexpr bool I8 = KV == kPagedI8;
  constexpr int KW = P::kKW, NT = P::kThreads, ROWS = P::kRows, COLS = P::kCols, RB = P::kRowBytes;
  constexpr int R = P::kRing, SW = P::kSW, GW = P::kGW;
  constexpr int DT = D / 16 / GW;                       // 16-channel tiles a warp
  // the reference lies kHead below a strip's largest score when it moves, and moves when one
  // passes it by kRise (exponents of 2; fp16 weights reach 2^kRise)
  constexpr float kHead = BF ? 0.0f : 7.0f, kRise = BF ? 8.0f : 15.0f;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t *fixed = smem + R * KW * P::kHalf;
  float *red = reinterpret_cast<float *>(fixed);                      // [KW][GW][COLS][SW + 4]
  float *sm_m = red + P::kRedBytes / 4;                               // [KW][COLS]
  float *sm_l = sm_m + P::kWarps * COLS;
  long long *sm_row = reinterpret_cast<long long *>(sm_l + P::kWarps * COLS);   // [ROWS]
  PagedSeg *segs = reinterpret_cast<PagedSeg *>(sm_row + ROWS);
  PagedCtl *ctl = reinterpret_cast<PagedCtl *>(segs + kPagedMaxSegs);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gi = warp % GW, kw = warp / GW;             // place in its group, group
  const int c4 = lane & 3, r8 = lane >> 2;
  uint8_t *ring = smem + kw * R * P::kHalf;                           // this group's half stages
  const uint32_t ring_s = smem_u32(ring);

  // this lane's row and half of the four matrices it addresses: K as keys x channels, V
  // transposed (channels x keys)
  const LaneOffs<RB> koff((lane & 7) + ((lane >> 3) & 1) * 8, lane >> 4), voff((lane & 7) + (lane >> 4) * 8, (lane >> 3) & 1);
  const uint32_t half = (uint32_t)(gi * (RB / 2));      // this warp's channels in a row (GW = 2: a multiple of 128 bytes)

  griddep_wait();
  griddep_launch_dependents();

  if (!paged_schedule<ROWS, P::kItemCost, P::kWarps>(a, segs, ctl)) return;       // whole CTA

  float acc[DT][NB][4];
  for (;;) {
    if (ctl->nseg == 0) {                                // the whole CTA
      __syncthreads();
      if (tid == 0) paged_walk<ROWS, P::kItemCost>(a, segs, ctl);
      __syncthreads();
      if (ctl->nseg == 0) break;                         // (only places of no strip were left)
    }
    const int nseg = ctl->nseg;
    const bool more = ctl->more != 0;

    // Group kw of an item of nblk column blocks takes block kw % nblk and its strips
    // u0 + kw / nblk, + KW / nblk, .. (the groups left over take none).
    auto deal = [&](const PagedSeg &g, int &first, int &step) {
      const int n = ROWS == COLS ? 1 : g.nblk;
      step = n == 1 ? KW : n == 2 ? KW / 2 : n == 3 ? KW / 3 : KW / 4;
      first = n == 1 ? kw : n == 2 ? kw >> 1 : n == 3 ? (kw * 11) >> 5 : kw >> 2;     // kw / n, kw < 16
      const int block = kw - first * n;
      if (first >= step) first = 1 << 28;
      first += g.u0;
      return block;
    };
    // ---- the ring: this group's strips, ahead of the arithmetic, each as two half stages: its
    // K rows, then its V rows
    int ls = -1, lu = 0, lend = 0, lstep = KW, lbuf = 0;
    bool lv = false;
    auto advance = [&]() {                                 // to the next segment with a strip
#pragma unroll 1
      while (ls < nseg && lu >= lend)
        if (++ls < nseg) {
          deal(segs[ls], lu, lstep);
          lend = segs[ls].u1;
        }
    };
    advance();
    // Of the strip being loaded: byte offset of row lane & 15 (-1: not read) and, int8, of its
    // scale; the rows that are read; whether the strip lies in one page and is read whole.
    long long off = -1, soff = -1;
    bool plain = false;
    auto load_next = [&]() {
      if (ls < nseg) {
        const PagedSeg &g = segs[ls];
        const uint32_t st = ring_s + (uint32_t)(lbuf * P::kHalf);
        if (!lv) {
          const int unit = lu < g.nsu ? lu : g.first + lu - g.nsu;
          const int key = unit * kStrip + (lane & 15);
          off = soff = -1;
          if (key < g.hi && (key >= g.lo || key < a.sinks)) {
            const int pi = a.page_shift >= 0 ? key >> a.page_shift : paged_div(key, a.page), po = key - pi * a.page;
            const int pid = __ldg(a.table + (size_t)g.b * a.max_pages + pi);
            if ((unsigned)pid < (unsigned)a.npages) {
              off = (pid * a.page_stride + g.g * a.head_stride + po * a.tok_stride) * P::kES;
              if constexpr (I8) soff = ((long long)pid * a.Hkv + g.g) * a.page + po;
            } else {
              atomicCAS(a.err, 0, -9);
            }
          }
          plain = a.strip_pages && __all_sync(0xffffffffu, off >= 0);
        }
        const uint8_t *base = lv ? a.v : a.k;
        if constexpr (I8)
          if (gi == 0 && lane < 16)
            cp_async4(st + kStrip * RB + lane * 4, (lv ? a.vs : a.ks) + (soff >= 0 ? soff : 0), soff >= 0 ? 4u : 0u);
        constexpr int CH = RB / 16;                        // 16-byte chunks a row
        constexpr int RPI = 32 / CH;                       // rows a warp instruction covers
        constexpr int NI = kStrip / RPI;
        // (computed here again for each half: kept, these would take eight registers)
        int ln = lane;
        asm volatile("" : "+r"(ln));
        const int lr = ln / CH, lc = ln % CH;
        if (plain) {                                       // rows at equal distances
          const long long o0 = __shfl_sync(0xffffffffu, off, 0);
          const uint8_t *src = base + o0 + (gi * RPI + lr) * a.tok_stride * P::kES + lc * 16;
          // row i of this lane: the swizzle changes by bits of i alone (stages start on 128 bytes)
          constexpr int NR = GW * RPI;
          static_assert(NI % GW == 0 && (RB >= 128 || NR % 8 == 0) && P::kHalf % (RB < 128 ? RB : 128) == 0, "");
          const uint32_t dst = st + strip_off<RB>(gi * RPI + lr, lc);
          if (a.tok_stride == D) {                         // one after the other: no address to compute
#pragma unroll
            for (int i = 0; i < NI / GW; ++i)
              cp_async16_full((dst ^ (((i * NR) & 7) << 4)) + i * NR * RB, src + i * NR * RB);
          } else {
            const long long step = NR * a.tok_stride * P::kES;
#pragma unroll
            for (int i = 0; i < NI / GW; ++i) {
              cp_async16_full((dst ^ (((i * NR) & 7) << 4)) + i * NR * RB, src);
              src += step;
            }
          }
        } else {
#pragma unroll 1
          for (int i = gi; i < NI; i += GW) {
            const int r = i * RPI + lr;
            const long long o = __shfl_sync(0xffffffffu, off, r);
            cp_async16(st + strip_off<RB>(r, lc), base + (o >= 0 ? o + lc * 16 : 0), o >= 0 ? 16u : 0u);
          }
        }
        if (lv) {
          lu += lstep;
          advance();
        }
        lv = !lv;
      }
      cp_async_commit();
      lbuf = lbuf + 1 == R ? 0 : lbuf + 1;
    };
    // One warp a group refills a buffer as soon as it has read it (R loads ahead); several
    // warps refill it after the next half's barrier (R - 1 ahead).
    constexpr int kAhead = GW == 1 ? R : R - 1;
    int buf = 0;
    auto acquire = [&]() {                                 // the next half: its shared address
      cp_async_wait<kAhead - 1>();
      if constexpr (GW == 1) {
        __syncwarp();
      } else {
        named_bar_sync(1 + kw, 32 * GW);
        load_next();
      }
      const int b = buf;
      buf = buf + 1 == R ? 0 : buf + 1;
      return b * P::kHalf;
    };
    auto release = [&]() {
      if constexpr (GW == 1) {
        __syncwarp();
        load_next();
      }
    };

    // ---- Q as B fragments: column r8 of tile nb, channels 2 c4, + 1, + 8, + 9 of each 16
    // (int8: 4 c4 .. 4 c4 + 3, the order in which the codes of a word are widened).  Loaded
    // while the item before is joined.
    uint32_t qr[DT][NB][2];
    auto load_q = [&](const PagedSeg &g) {
      int first, step;
      const int row0 = g.rb * ROWS + deal(g, first, step) * COLS;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        // (a column past the last repeats the first: its sums are its own and unused)
        const int gr = row0 + nb * 8 + r8;
        const int tok = gr < g.rows ? gr / a.G : 0, hd = gr < g.rows ? gr - tok * a.G : 0;
        const uint16_t *src = a.q + (long long)(g.tok0 + tok) * a.q_tok + (long long)(g.g * a.G + hd) * a.q_head + gi * (D / 2) + (I8 ? 4 : 2) * c4;
#pragma unroll
        for (int ks = 0; ks < DT; ++ks) {
          if constexpr (I8) {
            const uint2 v = __ldg(reinterpret_cast<const uint2 *>(src + ks * 16));
            qr[ks][nb][0] = v.x;
            qr[ks][nb][1] = v.y;
          } else {
            qr[ks][nb][0] = __ldg(reinterpret_cast<const uint32_t *>(src + ks * 16));
            qr[ks][nb][1] = __ldg(reinterpret_cast<const uint32_t *>(src + ks * 16 + 8));
          }
        }
      }
    };

    load_q(segs[0]);
#pragma unroll 1
    for (int i = 0; i < kAhead; ++i) load_next();

    for (int sg = 0; sg < nseg; ++sg) {
      const PagedSeg &g = segs[sg];
      int u, step;
      const int block = deal(g, u, step);
      const int row0 = g.rb * ROWS + block * COLS;         // the group's first column
      // positions of this lane's columns (-1: no such column)
      int pos[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int gr = row0 + nb * 8 + 2 * c4 + e;
          pos[nb][e] = gr < g.rows ? g.pos0 + gr / a.G : -1;
        }
      const int pmin = g.pos0 + row0 / a.G, pmax = g.pos0 + (min(g.rows, row0 + COLS) - 1) / a.G;
      // whether the item's columns, whose keys are loaded together, lie at several positions
      const bool mixed = g.rb * ROWS / a.G != (min(g.rows, g.rb * ROWS + ROWS) - 1) / a.G;
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[t][nb][e] = 0.0f;
      float m[NB][2], l[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        m[nb][0] = m[nb][1] = kNoScore;
        l[nb][0] = l[nb][1] = 0.0f;
      }

#pragma unroll 1
      for (; u < g.u1; u += step) {
        const int key0 = (u < g.nsu ? u : g.first + u - g.nsu) * kStrip;
        // ---- S^T = K Q^T: element e of tile nb: key r8 + 8 (e / 2), column 2 c4 + (e & 1)
        constexpr int CN = NB == 1 ? 2 : 1;                // independent sums (MMA latency)
        float sp[CN][NB][4] = {};
        float ksc[2] = {a.scale_log2, a.scale_log2};
        {
          const int hb = acquire();
          const uint32_t kst = ring_s + (uint32_t)hb + half;
          if constexpr (!I8) {
            // A tile: matrices (keys 0-7, 8-15) x (channels 0-7, 8-15) of each 16
#pragma unroll
            for (int ks = 0; ks < DT; ++ks) {
              uint32_t kf[4];
              ldsm4(kf, kst + koff(ks));
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) mma16816<BF>(sp[ks % CN][nb], kf, qr[ks][nb][0], qr[ks][nb][1]);
            }
          } else {
            const float *sc = reinterpret_cast<const float *>(ring + hb + kStrip * RB);
            ksc[0] *= sc[r8];
            ksc[1] *= sc[r8 + 8];
            // matrices: (keys 0-7, 8-15) x (channels 0-15, 16-31); a word holds four channels
#pragma unroll
            for (int kk = 0; kk < DT / 2; ++kk) {
              uint32_t kf[4];
              ldsm4(kf, kst + koff(kk));
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t u0 = kf[2 * h] ^ 0x80808080u, u1 = kf[2 * h + 1] ^ 0x80808080u;
                const uint32_t af[4] = {codes_f16<0x4140>(u0), codes_f16<0x4140>(u1), codes_f16<0x4342>(u0), codes_f16<0x4342>(u1)};
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                  mma16816<false>(sp[(kk * 2 + h) % CN][nb], af, qr[kk * 2 + h][nb][0], qr[kk * 2 + h][nb][1]);
              }
            }
          }
          release();
        }
        float s[NB][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[nb][e] = sp[0][nb][e];
#pragma unroll
            for (int i = 1; i < CN; ++i) s[nb][e] += sp[i][nb][e];
          }
        if constexpr (GW == 2) {
          // the other half's scores (read before the values' barrier, written again after it)
          float4 *xs = reinterpret_cast<float4 *>(red) + kw * 2 * NB * 32 + lane;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) xs[(gi * NB + nb) * 32] = make_float4(s[nb][0], s[nb][1], s[nb][2], s[nb][3]);
          named_bar_sync(1 + kw, 32 * GW);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const float4 o = xs[((gi ^ 1) * NB + nb) * 32];
            s[nb][0] += o.x;
            s[nb][1] += o.y;
            s[nb][2] += o.z;
            s[nb][3] += o.w;
          }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nb][e] *= ksc[e >> 1];
        const bool masked = key0 + kStrip - 1 > pmin ||
                            (a.window > 0 && key0 <= pmax - a.window && key0 + kStrip > a.sinks);
        if (masked) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = key0 + r8 + 8 * (e >> 1), ps = pos[nb][e & 1];
              if (j > ps || (a.window > 0 && j <= ps - a.window && j >= a.sinks)) s[nb][e] = -INFINITY;
            }
        }
        const int hb = acquire();
        const uint32_t vst = ring_s + (uint32_t)hb;
        float vsc[2] = {1.0f, 1.0f}, lvs[2] = {0.0f, 0.0f};
        if constexpr (I8) {
          const float *sc = reinterpret_cast<const float *>(ring + hb + kStrip * RB);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            vsc[h] = sc[r8 + 8 * h];
            lvs[h] = fmaxf(paged_lg2(fabsf(vsc[h])), -64.0f);
          }
        }
        // ---- weights.  The reference moves only when a weight passes it by 2^kRise, so the
        // largest score of a strip is seldom needed exactly.
        bool up = false;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) up |= (I8 ? s[nb][e] + lvs[e >> 1] : s[nb][e]) > m[nb][e & 1] + kRise;
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float top = fmaxf(s[nb][e] + lvs[0], s[nb][2 + e] + lvs[1]);
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
              float f = 1.0f;
              if (top > m[nb][e] + kRise) {
                top -= kHead;
                f = paged_ex2(m[nb][e] - top);
                m[nb][e] = top;
              }
              l[nb][e] *= f;
#pragma unroll
              for (int t = 0; t < DT; ++t) {
                acc[t][nb][e] *= f;
                acc[t][nb][2 + e] *= f;
              }
            }
        }
        uint32_t pf[2][NB][2];                             // the rounded weights, and what that leaves
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float p0 = paged_ex2(s[nb][2 * h] - m[nb][0]), p1 = paged_ex2(s[nb][2 * h + 1] - m[nb][1]);
            l[nb][0] += p0;
            l[nb][1] += p1;
            if constexpr (I8) {          // (a hidden key's weight is 0 whatever its value's scale holds)
              p0 = s[nb][2 * h] == -INFINITY ? 0.0f : p0 * vsc[h];
              p1 = s[nb][2 * h + 1] == -INFINITY ? 0.0f : p1 * vsc[h];
            }
            const uint32_t pk = pack2<BF>(p0, p1);
            const float2 r = unpack2<BF>(pk);
            pf[0][nb][h] = movm_t(pk);
            pf[1][nb][h] = movm_t(pack2<BF>(p0 - r.x, p1 - r.y));
          }
        }
        // ---- O^T += V^T P^T
        bool odd = false;
        if constexpr (!I8) {
          // an item's columns at several positions: a key hidden from some (this group's may
          // all be at one) has weight 0 there, and 0 times an infinite or NaN value would reach
          // them through the MMA.  Strips that hold such a value are summed without the hidden
          // products.
          odd = masked && mixed && strip_nonfinite<D, BF>(vst, lane);
        }
        if (!I8 && odd) {
          if constexpr (!I8) add_visible<D, DT, NB, BF>(acc, s, m, vst, gi * 2 * DT, lane);
        } else if constexpr (!I8) {
          // A tile (transposed): (channels 0-7, 8-15) x (keys 0-7, 8-15)
#pragma unroll
          for (int dt = 0; dt < DT; ++dt) {
            uint32_t vf[4];
            ldsm4_t(vf, vst + half + voff(dt));
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) mma16816<BF>(acc[dt][nb], vf, pf[i][nb][0], pf[i][nb][1]);
          }
        } else {
          // a transposed 16-bit element holds two channels: rows 0-7 of tile dt are the even
          // channels of its 16, rows 8-15 the odd ones
#pragma unroll
          for (int kk = 0; kk < DT / 2; ++kk) {
            uint32_t vf[4];
            ldsm4_t(vf, vst + half + voff(kk));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t u0 = vf[h] ^ 0x80808080u, u1 = vf[2 + h] ^ 0x80808080u;
              const uint32_t af[4] = {codes_f16<0x4240>(u0), codes_f16<0x4341>(u0), codes_f16<0x4240>(u1), codes_f16<0x4341>(u1)};
#pragma unroll
              for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) mma16816<false>(acc[2 * kk + h][nb], af, pf[i][nb][0], pf[i][nb][1]);
            }
          }
        }
        release();
      }

      // ---- join the CTA's groups: out rows, or partial sums of a cut item
      if (sg + 1 < nseg) load_q(segs[sg + 1]);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) l[nb][e] += __shfl_xor_sync(0xffffffffu, l[nb][e], o);
          if (r8 == 0 && gi == 0) {
            sm_m[kw * COLS + nb * 8 + 2 * c4 + e] = m[nb][e];
            sm_l[kw * COLS + nb * 8 + 2 * c4 + e] = l[nb][e];
          }
        }
      __syncthreads();                                   // also: Q is no longer read
      // bit w: group w takes the item's first block; shifted by b, its block b
      const unsigned groups = ROWS == COLS || g.nblk == 1 ? 0xffffu : g.nblk == 2 ? 0x5555u : g.nblk == 3 ? 0x9249u : 0x1111u;
      float f[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float M = kNoScore;
#pragma unroll
          for (int w = 0; w < KW; ++w)
            if (ROWS == COLS || ((groups << block >> w) & 1u)) M = fmaxf(M, sm_m[w * COLS + nb * 8 + 2 * c4 + e]);
          f[nb][e] = paged_ex2(m[nb][e] - M);
        }
      const bool cut = g.c0 != g.c1;
      float *part = a.part + (size_t)(2 * blockIdx.x + (g.c0 == (int)blockIdx.x ? 1 : 0)) * P::kPartFloats;
      const int first = g.rb * ROWS, nrows = min(ROWS, g.rows - first);
      // column sums: M and L of each column (thread r), and its row of out
      float M = kNoScore, L = 0.0f;
      if (tid < nrows) {
        const int tok = (first + tid) / a.G;
        const long long orow = (long long)(g.tok0 + tok) * a.Hq + g.g * a.G + first + tid - tok * a.G;
        sm_row[tid] = orow;
        const unsigned mine = groups << (tid / COLS);
        const int cl = tid % COLS;
#pragma unroll
        for (int w = 0; w < KW; ++w)
          if (ROWS == COLS || (mine >> w & 1u)) M = fmaxf(M, sm_m[w * COLS + cl]);
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          if (ROWS == COLS || (mine >> w & 1u)) L += sm_l[w * COLS + cl] * paged_ex2(sm_m[w * COLS + cl] - M);
        }
        if (cut) {
          part[tid] = M;
          part[ROWS + tid] = L;
        } else if (a.lse) {
          a.lse[orow] = L > 0.0f || L != L ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
        }
      }
      __syncthreads();
      if (tid < nrows) sm_l[tid] = L == 0.0f ? 0.0f : 1.0f / L;      // no key: a row of zeros
#pragma unroll
      for (int sl = 0; sl < 16 * DT / SW; ++sl) {
        float *w = red + warp * COLS * (SW + 4);
#pragma unroll
        for (int t = 0; t < SW / 16; ++t)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const float(&x)[4] = acc[sl * (SW / 16) + t][nb];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float *dst = w + (nb * 8 + 2 * c4 + e) * (SW + 4) + 16 * t;
              if constexpr (!I8) {
                dst[r8] = x[e] * f[nb][e];
                dst[r8 + 8] = x[2 + e] * f[nb][e];
              } else {
                *reinterpret_cast<float2 *>(dst + 2 * r8) = make_float2(x[e] * f[nb][e], x[2 + e] * f[nb][e]);
              }
            }
          }
        __syncthreads();
#pragma unroll 1
        for (int i = tid; i < nrows * (GW * SW / 2); i += NT) {
          const int r = i / (GW * SW / 2), hc = i % (GW * SW / 2) / (SW / 2), cp = i % (SW / 2);
          float2 o = make_float2(0.0f, 0.0f);
          const unsigned mine = groups << (r / COLS);
#pragma unroll
          for (int w2 = 0; w2 < KW; ++w2) {
            if (ROWS != COLS && !(mine >> w2 & 1u)) continue;
            const float2 v = *reinterpret_cast<const float2 *>(red + ((w2 * GW + hc) * COLS + r % COLS) * (SW + 4) + 2 * cp);
            o.x += v.x;
            o.y += v.y;
          }
          const int col = hc * (D / 2) + SW * sl + 2 * cp;
          if (cut) {
            *reinterpret_cast<float2 *>(part + 2 * ROWS + (size_t)r * D + col) = o;
          } else {
            const float inv = sm_l[r];
            *reinterpret_cast<uint32_t *>(a.out + sm_row[r] * D + col) = pack2<BF>(o.x * inv, o.y * inv);
          }
        }
        __syncthreads();
      }
      if (!cut) continue;

      // ---- a cut item: the last CTA to finish a group of its parts joins them, in CTA order
      // (the barrier and thread 0's release and acquire order every thread's accesses)
      __syncthreads();
      if (tid == 0) {
        const int n = g.c1 - g.c0 + 1, lg = paged_group(n), head = ((int)blockIdx.x - g.c0) >> lg << lg;
        // (a CTA's first and last part may each begin a group: two counters)
        int *counter = a.counters + kPagedMaxCtas + 2 * (g.c0 + head) + (head == 0 ? 1 : 0);
        if (atom_add_acq_rel_gpu(counter, 1) == min(1 << lg, n - head) - 1) {
          *counter = 0;                                  // zero again for the next call
          ctl->group[ctl->njoin] = head;
          ctl->join[ctl->njoin++] = g;                   // (a range cuts two items at most)
        }
      }
    }
    if (!more) break;
    __syncthreads();
    if (tid == 0) ctl->nseg = 0;
    __syncthreads();
  }
  // ---- the groups that this CTA was the last to finish; the last of an item's groups: the item
  __syncthreads();
#pragma unroll 1
  for (int i = 0; i < ctl->njoin; ++i) {
    const PagedSeg &g = ctl->join[i];
    const int n = g.c1 - g.c0 + 1, lg = paged_group(n), groups = (n + (1 << lg) - 1) >> lg;
    if (groups == 1) {                                   // (apart, with its constants: 0.3 us a short call)
      paged_join<D, KV, NB, CTAS>(a, g, 0, 1, n, true, red);
      continue;
    }
    int first = ctl->group[i], step = 1, count = min(1 << lg, n - first);
    bool final = false;
#pragma unroll 1
    for (;;) {
      paged_join<D, KV, NB, CTAS>(a, g, first, step, count, final, red);
      if (final) break;
      if (tid == 0) {                                    // (the join ends with a barrier)
        ctl->last = atom_add_acq_rel_gpu(a.counters + g.c0, 1) == groups - 1;
        if (ctl->last) a.counters[g.c0] = 0;
      }
      __syncthreads();
      final = ctl->last != 0;
      __syncthreads();
      if (!final) break;
      first = 0;
      step = 1 << lg;
      count = groups;
    }
  }
}

template <int D, int KV, int NB, int CTAS>
cudaError_t paged_launch_one(const PagedArgs &a, int sms, cudaStream_t st) {
  using P = PagedShape<D, KV, NB, CTAS>;
  const void *f = reinterpret_cast<const void *>(attn_paged_kernel<D, KV, NB, CTAS>);
  cudaError_t e = ensure_smem_attr(f, P::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(f, dim3(sms * CTAS), dim3(P::kThreads), P::kSmem, st, a);
  count_launch();
  return e;
}
// cols: the columns of an item, 8 or 64 (paged_columns).
//
// Several CTAs share an SM where there are many items (one CTA's exchange and join then overlap
// the others' strips), one has it alone where there are few (a short call waits for one item,
// which more warps finish sooner).  Measured, one against several: 64 of 1000 to 8190 tokens, 32/8
// heads of 128, bf16: 187.5 and 184.5 us; 200 x 700: 98.2 and 95.5; 48 windows of 1024, 64/8 heads of
// 64: 32.7 and 27.9; 64 x 3000, 24/4 heads of 256: 126.3 and 127.6 (int8 81.6 and 76.4), 16 x 3000: 41.0 and
// 40.3, 4 x 3000: 16.3 and 17.4; 2 x 3000 of 8 heads of 128: 12.5 and 13.0; 4 x 131071 of 4 heads of 256, int8:
// 176 and 186; 32 x 16000, 24 columns of 8 heads of 128: 437 and 439.  Sixteen columns of d = 256 leave
// no registers for it (48 x 16k, 24 columns, with one product a weight: 299 and 382 us).
template <int KV>
cudaError_t paged_launch(const PagedArgs &a, int d, int cols, int sms, cudaStream_t st) {
  const bool many = 3ll * a.B * a.Hkv > sms;
#define QW_PAGED(DD)                                                                       \
  case DD:                                                                                  \
    return cols == 8 ? many ? paged_launch_one<DD, KV, 1, paged_ctas(DD, 8)>(a, sms, st)    \
                            : paged_launch_one<DD, KV, 1, 1>(a, sms, st)                    \
                     : many ? paged_launch_one<DD, KV, 2, paged_ctas(DD, 64)>(a, sms, st)   \
                            : paged_launch_one<DD, KV, 2, 1>(a, sms, st);
  switch (d) {
    QW_PAGED(64)
    QW_PAGED(128)
    QW_PAGED(256)
  }
#undef QW_PAGED
  return cudaErrorInvalidValue;
}

}  // namespace qw
