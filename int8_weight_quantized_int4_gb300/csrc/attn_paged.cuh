// attn_paged.cuh -- attention of each sequence's new tokens over a paged key-value cache.
//
// For query head h of new token t at position pos of its sequence, KV head g = h / G
// (G = Hq / Hkv), over the keys j it can see (j <= pos and, with a window W, j > pos - W or
// j < sinks):
//   x_j = q . k_j * scale,  p_j = e^(x_j - m),  out = sum_j p_j v_j / sum_j p_j.
// One pass over K and V: a running reference m of the exponents (moved only when a score
// passes it by 2^8, which rescales the sums), the sums in binary32.
//
// What bounds it: reading K and V, 2 S d e bytes a (sequence, KV head) for 4 S d flops a
// query row -- a few rows a KV head (G x new tokens), so 1..64 flops a byte, far below the
// ridge of any matrix unit here (warp-level MMA: 606 TFLOP/s measured against 6.7 TB/s, 90
// flops a byte).  So the design is about keeping loads in flight:
//   - The G heads and the new tokens of a sequence that share a KV head are the rows of one
//     16-row MMA tile (RW tiles for more rows), so K and V are read once for all of them.
//   - A CTA of RW x KW warps owns an SM.  Each of its KW groups streams its own strips of 16
//     keys through its own ring of shared-memory stages (cp.async, 16 bytes a thread; rows
//     beyond the visible keys are zero-filled, not read) and waits only for itself: no
//     CTA-wide barrier between the strips of a sequence.  The RW warps of a group share its
//     strips, one row tile each.
//   - Work is split evenly over the SMs whatever the lengths: the visible keys of every
//     (sequence, row block, KV head) item are cut into units of 16 KW keys, the units of all
//     items laid end to end and cut into one equal range a CTA (every CTA finds its own range
//     from the lengths on the device, so a captured graph follows growing contexts).  An item
//     that a range border cuts leaves partial sums (m, l, O) in the workspace, and the last
//     CTA to finish it joins them in CTA order: results do not depend on arrival order.
//   - The ring runs ahead across item borders, so the next item's keys arrive while one item
//     is being finished.
//
// Roundings: p is rounded to the values' 16-bit type for the P.V product (fp16 2^-11, bf16
// 2^-8 relative, half a step; both sums are exact products accumulated in binary32) -- the
// error of each p is independent, so it stays of the order of the output's own rounding; the
// denominator sums the unrounded p.  With the int8 cache the value's scale joins its weight
// (w_j = p_j vs_j) and the reference follows w_j, not p_j, so that w keeps its bits whatever
// the scales' size.
#pragma once
#include <stdint.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "launch.h"
#include "ptx.cuh"

namespace qw {

constexpr int kPagedMaxSegs = 32;       // work segments listed at a time
constexpr int kStrip = 16;              // keys a group handles per step: the MMA's K of P.V
constexpr int kRedStride = 40;          // floats a row of the 32-column exchange buffer
                                        // (8 rows x 4 column pairs on distinct banks)
constexpr int kPagedSmem = 227 * 1024;

struct PagedSeg {
  int b, g, rb;                 // sequence, KV head, row block
  int u0, u1;                   // units of the item [u0, u1)
  int nsu, first;               // units of the sinks, unit of the first windowed key
  int lo, hi;                   // visible keys of the row block: [lo, hi) and below `sinks`
  int pos0, rows;               // position of the sequence's first new token; its query rows
  int tok0;                     // its first row in q and out
  int c0, c1;                   // CTAs holding the item's first and last unit
};

template <int D, int KV, int RW>
struct PagedShape {
  static constexpr int kES = KV == kPagedI8 ? 1 : 2;
  static constexpr int kKW = KV != kPagedI8 && D == 256 && RW == 1 ? 4 : 8 / RW;
  static constexpr int kWarps = RW * kKW;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kRows = 16 * RW;
  static constexpr int kUnit = kStrip * kKW;
  static constexpr int kRowBytes = D * kES;
  static constexpr int kStageBytes = 2 * kStrip * kRowBytes + (KV == kPagedI8 ? 2 * kStrip * 4 : 0);
  static constexpr int kQBytes = RW * D * 32;
  static constexpr int kRedBytes = kWarps * 16 * kRedStride * 4;
  static constexpr int kQRed = kQBytes > kRedBytes ? kQBytes : kRedBytes;   // Q and the exchange share it
  static constexpr int kFixed = kQRed + 2 * kWarps * 16 * 4 + kPagedMaxSegs * (int)sizeof(PagedSeg) + 256;
  static constexpr int kFit = (kPagedSmem - kFixed) / (kKW * kStageBytes);
  static constexpr int kStages = kFit > 8 ? 8 : kFit;
  static constexpr int kSmem = kFixed + kStages * kKW * kStageBytes;
  static_assert(kStages >= 3, "a ring of at least three stages");
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
// Two int8 codes of a word (xor 0x80 applied: u = code + 128) as an fp16 pair: 0x6400 | u
// is 1024 + u exactly, minus 1152.  SEL picks the two bytes.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t codes_f16(uint32_t u) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(u), "r"(0x64646464u), "n"(SEL));
  return h2_as_u32(__hsub2(u32_as_h2(r), u32_as_h2(0x64806480u)));
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
// acc += P . V of one strip over the visible keys alone (score above -inf), term by term.
// p: the A fragments, s: the scores (tile t, element e: row r8 + 8 (e / 2), key 8 t + 2 c4 + (e & 1)).
template <int D, bool BF>
__device__ __forceinline__ void add_visible(float (&acc)[D / 8][4], const uint32_t (&p)[4], const float (&s)[2][4],
                                            uint32_t vst, int lane) {
#pragma unroll 1
  for (int j = 0; j < kStrip; ++j) {
    const int src = (lane & ~3) | ((j & 7) >> 1), t = j >> 3, e = j & 1;
    float w[2];
    bool see[2];
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const uint32_t pw = __shfl_sync(0xffffffffu, t ? p[2 + hh] : p[hh], src) >> (16 * e);
      const float sv = __shfl_sync(0xffffffffu, t ? (e ? s[1][2 * hh + 1] : s[1][2 * hh])
                                                  : (e ? s[0][2 * hh + 1] : s[0][2 * hh]), src);
      w[hh] = BF ? __uint_as_float(pw << 16) : __half2float(__ushort_as_half((unsigned short)pw));
      see[hh] = sv != -INFINITY;
    }
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
      uint32_t v;
      asm volatile("ld.shared.b32 %0, [%1];"
                   : "=r"(v) : "r"(vst + strip_off<D * 2>(j, n) + 4 * (lane & 3)) : "memory");
      const float v0 = BF ? __uint_as_float(v << 16) : __half2float(__ushort_as_half((unsigned short)v));
      const float v1 = BF ? __uint_as_float(v & 0xffff0000u) : __half2float(__ushort_as_half((unsigned short)(v >> 16)));
#pragma unroll
      for (int hh = 0; hh < 2; ++hh)
        if (see[hh]) {
          acc[n][2 * hh] = fmaf(w[hh], v0, acc[n][2 * hh]);
          acc[n][2 * hh + 1] = fmaf(w[hh], v1, acc[n][2 * hh + 1]);
        }
    }
  }
}

// --------------------------------------------------------------- the schedule --
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
// The keys that row block rb can see and their units.
template <int ROWS, int UNIT>
__device__ __forceinline__ PagedSpan paged_span(const PagedArgs &a, const PagedSeq &s, int rb) {
  PagedSpan p;
  const int rows = s.nq * a.G, pos0 = s.len - s.nq;
  const int t0 = rb * ROWS / a.G, t1 = (min(rows, rb * ROWS + ROWS) - 1) / a.G;
  p.hi = max(pos0 + t1 + 1, 0);
  p.lo = a.window > 0 ? max(pos0 + t0 - a.window + 1, 0) : 0;
  p.first = p.lo / UNIT;
  p.nsu = min((min(a.sinks, p.hi) + UNIT - 1) / UNIT, p.first);
  p.n = max(p.nsu + (p.hi + UNIT - 1) / UNIT - p.first, 1);      // an item with no key still writes its rows
  return p;
}

template <int D, int KV, int RW>
__global__ void __launch_bounds__(PagedShape<D, KV, RW>::kThreads, 1)
    attn_paged_kernel(const __grid_constant__ PagedArgs a) {
  using P = PagedShape<D, KV, RW>;
  constexpr bool BF = KV == kPagedBf16;
  constexpr bool I8 = KV == kPagedI8;
  constexpr int KW = P::kKW, NT = P::kThreads, ROWS = P::kRows, U = P::kUnit, RB = P::kRowBytes;
  constexpr int ST = P::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t ring_s = smem_u32(smem);
  uint8_t *fixed = smem + ST * KW * P::kStageBytes;
  uint4 *qf = reinterpret_cast<uint4 *>(fixed);                       // [RW][D/16][32] A fragments
  float *red = reinterpret_cast<float *>(fixed);                      // [KW][RW][16][kRedStride]
  float *sm_m = reinterpret_cast<float *>(fixed + P::kQRed);          // [KW][ROWS]
  float *sm_l = sm_m + P::kWarps * 16;
  PagedSeg *segs = reinterpret_cast<PagedSeg *>(sm_l + P::kWarps * 16);
  int *ctl = reinterpret_cast<int *>(segs + kPagedMaxSegs);           // [0..63]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rw = warp % RW, kw = warp / RW;
  const int c4 = lane & 3, r8 = lane >> 2;

  griddep_wait();
  griddep_launch_dependents();

  // ---- this CTA's range of units
  long long total = 0, pre = 0, mine = 0;
  const int per = (a.B + NT - 1) / NT;
  const int b_lo = min(tid * per, a.B), b_hi = min(b_lo + per, a.B);
  auto cost = [&](const PagedSeq &s) {
    long long c = 0;
    for (int rb = 0, n = (s.nq * a.G + ROWS - 1) / ROWS; rb < n; ++rb) c += paged_span<ROWS, U>(a, s, rb).n;
    return c * a.Hkv;
  };
  for (int b = b_lo; b < b_hi; ++b) mine += cost(paged_seq(a, b));
  {
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += t;
    }
    long long *ws = reinterpret_cast<long long *>(red);
    if (lane == 31) ws[warp] = inc;
    __syncthreads();
    for (int w = 0; w < P::kWarps; ++w) {
      if (w < warp) pre += ws[w];
      total += ws[w];
    }
    pre += inc - mine;
  }
  const long long share = max((total + gridDim.x - 1) / gridDim.x, (long long)a.min_units);
  const long long begin = share * blockIdx.x, end = min(total, begin + share);
  if (begin >= end) return;                                           // whole CTA
  // the sequence holding `begin`: ctl[0] its index, ctl[2..3] the offset in it
  if (begin >= pre && begin < pre + mine) {
    long long off = begin - pre;
    int b = b_lo;
    for (; b < b_hi; ++b) {
      const long long c = cost(paged_seq(a, b));
      if (off < c) break;
      off -= c;
    }
    ctl[0] = b;
    *reinterpret_cast<long long *>(ctl + 2) = off;
  }
  __syncthreads();
  // the walk's state, kept by thread 0: sequence, offset in it, units done
  int wb = ctl[0];
  long long woff = *reinterpret_cast<long long *>(ctl + 2), wpos = begin;

  float acc[D / 8][4];
  for (;;) {
    // ---- list the next segments
    __syncthreads();
    if (tid == 0) {
      int n = 0;
      while (wpos < end && n < kPagedMaxSegs) {
        const PagedSeq s = paged_seq(a, wb);
        const int rows = s.nq * a.G, nrb = (rows + ROWS - 1) / ROWS;
        long long off = woff;
        int rb = 0;
        PagedSpan p{};
        for (; rb < nrb; ++rb) {
          p = paged_span<ROWS, U>(a, s, rb);
          if (off < (long long)p.n * a.Hkv) break;
          off -= (long long)p.n * a.Hkv;
        }
        if (rb == nrb) {
          ++wb;
          woff = 0;
          continue;
        }
        PagedSeg &g = segs[n++];
        g.b = wb;
        g.rb = rb;
        g.g = (int)(off / p.n);
        g.u0 = (int)(off % p.n);
        g.u1 = (int)min((long long)p.n, g.u0 + (end - wpos));
        g.nsu = p.nsu;
        g.first = p.first;
        g.lo = p.lo;
        g.hi = p.hi;
        g.pos0 = s.len - s.nq;
        g.rows = rows;
        g.tok0 = s.tok0;
        g.c0 = (int)((wpos - g.u0) / share);
        g.c1 = (int)((wpos - g.u0 + p.n - 1) / share);
        wpos += g.u1 - g.u0;
        woff += g.u1 - g.u0;
      }
      ctl[4] = n;
      ctl[5] = wpos < end;
    }
    __syncthreads();
    const int nseg = ctl[4];
    const bool more = ctl[5] != 0;

    // ---- the ring: this group's strips, ahead of the arithmetic
    int ls = 0, lu = segs[0].u0, lstage = 0;
    auto load_next = [&]() {
      if (ls < nseg) {
        const PagedSeg &g = segs[ls];
        const int unit = lu < g.nsu ? lu : g.first + lu - g.nsu;
        const int key0 = unit * U + kw * kStrip;
        const uint32_t st = ring_s + (uint32_t)((lstage * KW + kw) * P::kStageBytes);
        // lane r (and r + 16): row r of the strip -- its element offset, -1 when not read
        long long off = -1;
        int srow = -1;
        {
          const int key = key0 + (lane & 15);
          if (key < g.hi && (key >= g.lo || key < a.sinks)) {
            const int pi = key / a.page, po = key - pi * a.page;
            const int pid = __ldg(a.table + (size_t)g.b * a.max_pages + pi);
            if ((unsigned)pid < (unsigned)a.npages) {
              off = pid * a.page_stride + g.g * a.head_stride + po * a.tok_stride;
              srow = 1;
              if constexpr (I8) {
                if (rw == 0) {
                  const float *sc = (lane < 16 ? a.ks : a.vs) + ((size_t)pid * a.Hkv + g.g) * a.page + po;
                  cp_async4(st + 2 * kStrip * RB + lane * 4, sc, 4);
                }
              }
            } else {
              atomicCAS(a.err, 0, -9);
            }
          }
          if constexpr (I8)
            if (rw == 0 && srow < 0) cp_async4(st + 2 * kStrip * RB + lane * 4, a.ks, 0);
        }
        constexpr int CH = RB / 16;                        // 16-byte chunks a row
        constexpr int RPI = 32 / CH > 0 ? 32 / CH : 1;     // rows a warp instruction covers
        constexpr int NI = kStrip / RPI;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          if (NI >= RW ? (i % RW != rw) : (rw >= NI || i != rw)) continue;
          const int r = i * RPI + (CH < 32 ? lane / CH : 0), c = lane % CH;
          const long long o = __shfl_sync(0xffffffffu, off, r);
          const uint32_t d = st + strip_off<RB>(r, c), nb = o >= 0 ? 16u : 0u;
          const size_t so = o >= 0 ? (size_t)o * P::kES + c * 16 : 0;
          cp_async16(d, a.k + so, nb);
          cp_async16(d + kStrip * RB, a.v + so, nb);
        }
        if (++lu == g.u1 && ++ls < nseg) lu = segs[ls].u0;
      }
      cp_async_commit();
      lstage = lstage + 1 == ST ? 0 : lstage + 1;
    };
#pragma unroll 1
    for (int i = 0; i < ST - 1; ++i) load_next();

    int stage = 0;
    for (int sg = 0; sg < nseg; ++sg) {
      const PagedSeg &g = segs[sg];
      const int row0 = g.rb * ROWS;
      // ---- Q rows as A fragments
      for (int i = tid; i < RW * (D / 16) * 32; i += NT) {
        const int ln = i & 31, ks = (i >> 5) % (D / 16), w = i / (32 * (D / 16));
        uint32_t f[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int gr = row0 + w * 16 + (ln >> 2) + 8 * hh;
          if (gr < g.rows) {
            const uint16_t *src = a.q + (long long)(g.tok0 + gr / a.G) * a.q_tok + (long long)(g.g * a.G + gr % a.G) * a.q_head + ks * 16;
            if constexpr (I8) {       // k = 2c, 2c+1 and 2c+8, 2c+9 are channels 4c .. 4c+3
              const uint2 v = __ldg(reinterpret_cast<const uint2 *>(src + 4 * (ln & 3)));
              f[hh] = v.x;
              f[2 + hh] = v.y;
            } else {
              f[hh] = __ldg(reinterpret_cast<const uint32_t *>(src + 2 * (ln & 3)));
              f[2 + hh] = __ldg(reinterpret_cast<const uint32_t *>(src + 2 * (ln & 3) + 8));
            }
          }
        }
        qf[i] = make_uint4(f[0], f[1], f[2], f[3]);
      }
      __syncthreads();
      // positions of this lane's two rows (-1: no such row)
      int pos[2];
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int gr = row0 + rw * 16 + r8 + 8 * hh;
        pos[hh] = gr < g.rows ? g.pos0 + gr / a.G : -1;
      }
      const int pmin = g.pos0 + row0 / a.G, pmax = g.pos0 + (min(g.rows, row0 + ROWS) - 1) / a.G;
#pragma unroll
      for (int t = 0; t < D / 8; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[t][e] = 0.0f;
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

#pragma unroll 1
      for (int u = g.u0; u < g.u1; ++u) {
        cp_async_wait<ST - 2>();
        if constexpr (RW == 1) __syncwarp();
        else named_bar_sync(1 + kw, 32 * RW);
        load_next();
        const uint32_t kst = ring_s + (uint32_t)((stage * KW + kw) * P::kStageBytes), vst = kst + kStrip * RB;
        const float *sc = reinterpret_cast<const float *>(smem + (stage * KW + kw) * P::kStageBytes + 2 * kStrip * RB);
        const int unit = u < g.nsu ? u : g.first + u - g.nsu;
        const int key0 = unit * U + kw * kStrip;
        stage = stage + 1 == ST ? 0 : stage + 1;
        if (key0 >= g.hi) continue;                      // nothing of this strip is visible
        // ---- scores of 16 rows x 16 keys
        float s[2][4] = {};
        const int mi = lane >> 3;
        const int krow = (lane & 7) + (mi >> 1) * 8;
        if constexpr (!I8) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t kf[4];
            ldsm4(kf, kst + strip_off<RB>(krow, ks * 2 + (mi & 1)));
            const uint4 q4 = qf[(rw * (D / 16) + ks) * 32 + lane];
            const uint32_t af[4] = {q4.x, q4.y, q4.z, q4.w};
            mma16816<BF>(s[0], af, kf[0], kf[1]);
            mma16816<BF>(s[1], af, kf[2], kf[3]);
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk) {
            uint32_t kf[4];
            ldsm4(kf, kst + strip_off<RB>(krow, kk * 2 + (mi & 1)));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint4 q4 = qf[(rw * (D / 16) + kk * 2 + h) * 32 + lane];
              const uint32_t af[4] = {q4.x, q4.y, q4.z, q4.w};
              const uint32_t u0 = kf[h] ^ 0x80808080u, u1 = kf[2 + h] ^ 0x80808080u;
              mma16816<false>(s[0], af, codes_f16<0x4140>(u0), codes_f16<0x4342>(u0));
              mma16816<false>(s[1], af, codes_f16<0x4140>(u1), codes_f16<0x4342>(u1));
            }
          }
        }
        // ---- weights: element (tile t, e): row r8 + 8 (e / 2), key key0 + 8 t + 2 c4 + (e & 1)
        const bool masked = key0 + kStrip - 1 > pmin ||
                            (a.window > 0 && key0 <= pmax - a.window && key0 + kStrip > a.sinks);
        float vs[2][2], lvs[2][2];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if constexpr (I8) {
              const int j = 8 * t + 2 * c4 + e;
              const float ksc = sc[j] * a.scale_log2;
              s[t][e] *= ksc;
              s[t][2 + e] *= ksc;
              vs[t][e] = sc[kStrip + j];
              lvs[t][e] = fmaxf(paged_lg2(fabsf(vs[t][e])), -64.0f);
            } else {
              s[t][e] *= a.scale_log2;
              s[t][2 + e] *= a.scale_log2;
              vs[t][e] = 1.0f;
              lvs[t][e] = 0.0f;
            }
          }
        if (masked) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = key0 + 8 * t + 2 * c4 + (e & 1), ps = pos[e >> 1];
              if (j > ps || (a.window > 0 && j <= ps - a.window && j >= a.sinks)) s[t][e] = -INFINITY;
            }
        }
        float top[2];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          float x = fmaxf(fmaxf(s[0][2 * hh] + lvs[0][0], s[0][2 * hh + 1] + lvs[0][1]),
                          fmaxf(s[1][2 * hh] + lvs[1][0], s[1][2 * hh + 1] + lvs[1][1]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
          top[hh] = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
        }
        // the reference moves only when a weight passes it by 2^8 (a weight then fits fp16)
        const bool up = top[0] > m[0] + 8.0f || top[1] > m[1] + 8.0f;
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            float f = 1.0f;
            if (top[hh] > m[hh] + 8.0f) {
              f = paged_ex2(m[hh] - top[hh]);
              m[hh] = top[hh];
            }
            l[hh] *= f;
#pragma unroll
            for (int t = 0; t < D / 8; ++t) {
              acc[t][2 * hh] *= f;
              acc[t][2 * hh + 1] *= f;
            }
          }
        }
        uint32_t pf[4];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const float ref = m[hh] == -INFINITY ? 0.0f : m[hh];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const float p0 = paged_ex2(s[t][2 * hh] - ref), p1 = paged_ex2(s[t][2 * hh + 1] - ref);
            l[hh] += p0 + p1;
            // (a hidden key's weight is 0 whatever its value's scale holds)
            if constexpr (I8)
              pf[2 * t + hh] = pack2<false>(s[t][2 * hh] == -INFINITY ? 0.0f : p0 * vs[t][0],
                                            s[t][2 * hh + 1] == -INFINITY ? 0.0f : p1 * vs[t][1]);
            else
              pf[2 * t + hh] = pack2<BF>(p0, p1);
          }
        }
        // ---- P . V
        const int vrow = (lane & 7) + (mi & 1) * 8;
        if constexpr (!I8) {
          // rows at several positions: a key hidden from some rows has weight 0 there, and 0
          // times an infinite or NaN value would reach them through the MMA.  Strips that
          // hold such a value are summed without the hidden products.
          if (masked && pmin != pmax && strip_nonfinite<D, BF>(vst, lane)) {
            add_visible<D, BF>(acc, pf, s, vst, lane);
            continue;
          }
#pragma unroll
          for (int dt = 0; dt < D / 16; ++dt) {
            uint32_t vf[4];
            ldsm4_t(vf, vst + strip_off<RB>(vrow, dt * 2 + (mi >> 1)));
            mma16816<BF>(acc[2 * dt], pf, vf[0], vf[1]);
            mma16816<BF>(acc[2 * dt + 1], pf, vf[2], vf[3]);
          }
        } else {
          // a transposed 16-bit element holds two channels: the even and the odd ones go to
          // two tiles (tile 2c: channels 16 c + 0, 2, .. 14; tile 2c + 1: 1, 3, .. 15)
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk) {
            uint32_t vf[4];
            ldsm4_t(vf, vst + strip_off<RB>(vrow, kk * 2 + (mi >> 1)));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t u0 = vf[2 * h] ^ 0x80808080u, u1 = vf[2 * h + 1] ^ 0x80808080u;
              mma16816<false>(acc[4 * kk + 2 * h], pf, codes_f16<0x4240>(u0), codes_f16<0x4240>(u1));
              mma16816<false>(acc[4 * kk + 2 * h + 1], pf, codes_f16<0x4341>(u0), codes_f16<0x4341>(u1));
            }
          }
        }
      }

      // ---- join the CTA's groups: out rows, or partial sums of a cut item
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 1);
        l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 2);
        if (c4 == 0) {
          sm_m[kw * ROWS + rw * 16 + r8 + 8 * hh] = m[hh];
          sm_l[kw * ROWS + rw * 16 + r8 + 8 * hh] = l[hh];
        }
      }
      __syncthreads();                                   // also: Q is no longer read
      float f[2];
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < KW; ++w) M = fmaxf(M, sm_m[w * ROWS + rw * 16 + r8 + 8 * hh]);
        f[hh] = m[hh] == -INFINITY ? 0.0f : paged_ex2(m[hh] - M);
      }
      const bool cut = g.c0 != g.c1;
      float *part = a.part + (size_t)(2 * blockIdx.x + (g.c0 == (int)blockIdx.x ? 1 : 0)) * P::kPartFloats;
      const int nrows = min(ROWS, g.rows - row0);
      // row sums: M and L of each row (thread r)
      float M = -INFINITY, L = 0.0f;
      if (tid < nrows) {
        for (int w = 0; w < KW; ++w) M = fmaxf(M, sm_m[w * ROWS + tid]);
        for (int w = 0; w < KW; ++w) {
          const float mw = sm_m[w * ROWS + tid];
          if (mw != -INFINITY) L += sm_l[w * ROWS + tid] * paged_ex2(mw - M);
        }
        if (cut) {
          part[tid] = M;
          part[ROWS + tid] = L;
        } else if (a.lse) {
          const int gr = row0 + tid;
          a.lse[(long long)(g.tok0 + gr / a.G) * a.Hq + g.g * a.G + gr % a.G] = L > 0.0f || L != L ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
        }
      }
      __syncthreads();
      if (tid < nrows) sm_l[tid] = L == 0.0f ? 0.0f : 1.0f / L;      // no key: a row of zeros
#pragma unroll
      for (int sl = 0; sl < D / 32; ++sl) {
        float *w = red + (warp * 16) * kRedStride;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const float(&x)[4] = acc[4 * sl + t];
          if constexpr (!I8) {
            *reinterpret_cast<float2 *>(w + r8 * kRedStride + 8 * t + 2 * c4) = make_float2(x[0] * f[0], x[1] * f[0]);
            *reinterpret_cast<float2 *>(w + (r8 + 8) * kRedStride + 8 * t + 2 * c4) = make_float2(x[2] * f[1], x[3] * f[1]);
          } else if (t % 2 == 0) {
            const float(&y)[4] = acc[4 * sl + t + 1];
            *reinterpret_cast<float4 *>(w + r8 * kRedStride + 8 * t + 4 * c4) =
                make_float4(x[0] * f[0], y[0] * f[0], x[1] * f[0], y[1] * f[0]);
            *reinterpret_cast<float4 *>(w + (r8 + 8) * kRedStride + 8 * t + 4 * c4) =
                make_float4(x[2] * f[1], y[2] * f[1], x[3] * f[1], y[3] * f[1]);
          }
        }
        __syncthreads();
        for (int i = tid; i < nrows * 16; i += NT) {
          const int r = i >> 4, cp = i & 15;
          float2 o = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int w2 = 0; w2 < KW; ++w2) {
            const float2 v = *reinterpret_cast<const float2 *>(red + ((w2 * RW + (r >> 4)) * 16 + (r & 15)) * kRedStride + 2 * cp);
            o.x += v.x;
            o.y += v.y;
          }
          const int col = 32 * sl + 2 * cp;
          if (cut) {
            *reinterpret_cast<float2 *>(part + 2 * ROWS + (size_t)r * D + col) = o;
          } else {
            const float inv = sm_l[r];
            const int gr = row0 + r;
            uint16_t *dst = a.out + ((long long)(g.tok0 + gr / a.G) * a.Hq + g.g * a.G + gr % a.G) * D + col;
            *reinterpret_cast<uint32_t *>(dst) = pack2<BF>(o.x * inv, o.y * inv);
          }
        }
        __syncthreads();
      }
      if (!cut) continue;

      // ---- a cut item: the last CTA to finish it joins the parts, in CTA order
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const int n = g.c1 - g.c0 + 1;
        const int old = atom_add_acq_rel_gpu(a.counters + g.c0, 1);
        ctl[6] = old == n - 1;
        if (old == n - 1) a.counters[g.c0] = 0;          // zero again for the next call
      }
      __syncthreads();
      if (ctl[6] == 0) continue;
      __threadfence();
      const float *p0 = a.part + (size_t)(2 * g.c0 + 1) * P::kPartFloats;         // the first part: slot 1
      auto slot = [&](int i) { return i == 0 ? p0 : a.part + (size_t)(2 * (g.c0 + i)) * P::kPartFloats; };
      const int n = g.c1 - g.c0 + 1;
      for (int i = tid; i < nrows * (D / 4); i += NT) {
        const int r = i / (D / 4), col = 4 * (i % (D / 4));
        float Mx = -INFINITY;
        for (int k = 0; k < n; ++k) Mx = fmaxf(Mx, __ldcg(slot(k) + r));
        float Ls = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
          const float *s = slot(k);
          const float mk = __ldcg(s + r), lk = __ldcg(s + ROWS + r);
          const float4 v = __ldcg(reinterpret_cast<const float4 *>(s + 2 * ROWS + (size_t)r * D + col));
          const float wgt = mk == -INFINITY ? 0.0f : paged_ex2(mk - Mx);
          Ls += lk * wgt;
          o.x += v.x * wgt;
          o.y += v.y * wgt;
          o.z += v.z * wgt;
          o.w += v.w * wgt;
        }
        const float inv = Ls == 0.0f ? 0.0f : 1.0f / Ls;
        const int gr = row0 + r;
        const long long orow = (long long)(g.tok0 + gr / a.G) * a.Hq + g.g * a.G + gr % a.G;
        *reinterpret_cast<uint2 *>(a.out + orow * D + col) =
            make_uint2(pack2<BF>(o.x * inv, o.y * inv), pack2<BF>(o.z * inv, o.w * inv));
        if (a.lse && col == 0)
          a.lse[orow] = Ls > 0.0f || Ls != Ls ? (Mx + log2f(Ls)) * 0.6931471805599453f : -INFINITY;
      }
      __syncthreads();
    }
    if (!more) break;
  }
}

template <int D, int KV, int RW>
cudaError_t paged_launch_one(const PagedArgs &a, int sms, cudaStream_t st) {
  using P = PagedShape<D, KV, RW>;
  const void *f = reinterpret_cast<const void *>(attn_paged_kernel<D, KV, RW>);
  cudaError_t e = ensure_smem_attr(f, P::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(f, dim3(sms), dim3(P::kThreads), P::kSmem, st, a);
  count_launch();
  return e;
}
template <int KV>
cudaError_t paged_launch(const PagedArgs &a, int d, int rw, int sms, cudaStream_t st) {
#define QW_PAGED(DD)                                                     \
  case DD:                                                               \
    return rw == 1   ? paged_launch_one<DD, KV, 1>(a, sms, st)           \
           : rw == 2 ? paged_launch_one<DD, KV, 2>(a, sms, st)           \
                     : paged_launch_one<DD, KV, 4>(a, sms, st);
  switch (d) {
    QW_PAGED(64)
    QW_PAGED(128)
    QW_PAGED(256)
  }
#undef QW_PAGED
  return cudaErrorInvalidValue;
}

}  // namespace qw
