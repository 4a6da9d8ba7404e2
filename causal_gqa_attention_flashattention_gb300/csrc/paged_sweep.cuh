// The sweep of the newest tokens' attention over a paged key/value cache (sm_103a). paged.cu
// launches it for sequences of their own, paged_prefix.cu for a batch with a shared prefix.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "paged.cuh"
#include "paged_prefix.cuh"
#include "ptx.cuh"
#include "rope.cuh"

namespace ne {
namespace {

// ====================================================================== attention
// Work: the key tiles (kTK positions) of every (sequence, key/value head), laid end
// to end in that order, cut into one equal stretch for each block.  Every block
// works the stretches out for itself from the lengths, so nothing is planned on the
// host and a captured graph follows the lengths it finds.  A segment, the part of
// one (sequence, head) in one block's stretch, that is not the whole of it leaves
// its unnormalised O, running maximum and sum; the block that finishes a (sequence,
// head) last adds the segments in order: the result does not depend on which one.
//
// Rows: the R = Tq * G queries of a key/value head (row t * G + g).  With at most 8 a
// matrix tile of 16 rows holds them twice: rows 0-7 the high fp16 part of the rotated query,
// rows 8-15 its remainder, so that one m16n8k16 product gives both parts of a score
// in one thread; the same goes for the weights' two bf16 parts in P V.  That
// precision is free: the tile has 16 rows anyway.  With more rows the parts are two products of
// a tile of 16 rows each.  mma.sync and not tcgen05: with so few rows the sweep is bound by the bytes
// of the cache, and a warp that owns its 16 keys end to end (copies, scores, weights,
// P V in registers) needs no hand-off between warps per tile.  It works two tiles off in
// 0.7 us, HBM delivers them in 1.4 us (7.1 TB/s over a long context); the contiguous cache's
// tcgen05 sweep takes 0.9 us for one.  16 contexts around 8192 positions (127 MB) 28.0 us,
// one of 131001 29.0 us; a short context 7.2 us, the chain of lengths, table, page and join.  The
// 16 contexts with 16 rows take 30.5 us, with 32 (bound by the products) 45.9, with 64 81.
template <int D>
struct Sweep {
  static constexpr uint32_t kSpan = D * 2;
  static constexpr int kSlot = 2 * 16 * (int)kSpan;  // 16 keys and their values
};
constexpr int kTK = 128;  // positions of a tile: a slice of 16 for each consumer warp
// Slices that a consumer warp has room for (more than 16 rows are bound by the products: 32 rows of
// 64 columns 45.9 us with two, 47.4 with three; of 32 columns 34.9 with four, 34.3 with six).
template <int D, int MT>
constexpr int kDepth = D == 64 ? (MT < 4 ? 4 : 2) : (MT < 4 ? 8 : 6);
// Eight consumer warps, then a warpgroup for the queries and the finished segments.
// (Sixteen consumers in two groups on alternate tiles measured slower: a short context 8.4 us
// against 7.4, 16 contexts around 8192 positions 31.9 against 31.4.)
constexpr int kWarps = 8;
constexpr int kSweepThreads = (kWarps + 4) * 32;
// What a segment costs beside its tiles (queries, its parts' way out), in tiles of the sweep: blocks get
// equal shares of both (128 sequences up to 1000 long 20.9 us, without it 22.4; 8 around 1700 11.5, 12.9).
constexpr int seg_cost(int D) { return D == 64 ? 1 : 2; }
// Joining a cut (sequence, head) costs about 3 us at the end, as much as five tiles.  One of at
// most so many tiles is never cut (32 sequences up to 1500 long 14.3 us, with 4 for 8 15.0) ...
constexpr int whole_tiles(int D) { return D == 64 ? 8 : 16; }
// ... and a boundary moves by so many to an end of a longer one (those 32 sequences 13.4 us, with 2
// 14.3, with 0 15.1; 64 up to 4000 long 29.8, 29.2, 31.2).
constexpr int max_slack(int D) { return D == 64 ? 3 : 6; }

// Buffers for the warps' parts of a finished segment, each with a finishing warp of its own.
constexpr int sweep_bufs(int D, int mt) { return D * mt <= 64 ? 2 : 1; }
// Warps that pack queries: with more than 8 rows those that do not finish segments (one of them alone
// takes about 1 us for 8 rows, in front of the block's first tile).
constexpr int query_warps(int D, int mt) { return mt == 1 ? 1 : 4 - sweep_bufs(D, mt); }

// Shared memory: barriers, the block's plan and the sequences' lengths first, then (from a
// 1024-byte boundary) the ring and what else a role keeps.  tiles: packed row tiles, mt: of one warp.
constexpr int kOffVars = 256, kOffCum = 384;
__host__ __device__ constexpr int paged_head(int B) { return (kOffCum + (2 * B + 1) * 4 + 1023) / 1024 * 1024; }
struct SweepSmem {
  int ring, q, scratch, ml, total;
};
// Query tiles of two segments, where there are not too many.
__host__ __device__ constexpr int sweep_qbufs(int tiles) { return tiles <= 8 ? 2 : 1; }
__host__ __device__ constexpr SweepSmem sweep_smem(int D, int depth, int tiles, int mt, int B) {
  SweepSmem m = {};
  const int rows = sweep_bufs(D, mt) * kWarps * mt * 8;
  m.ring = paged_head(B);
  m.q = m.ring + kWarps * depth * 2 * 16 * D * 2;
  m.scratch = m.q + sweep_qbufs(tiles) * tiles * 16 * D * 2;
  m.ml = m.scratch + rows * D * 4;
  m.total = m.ml + rows * 8 + 1024;
  return m;
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// L2 policy of the cache's keys and values: read once a step, they are the first to leave, and page
// tables, queries and the rotary table stay (16 contexts around 8192 positions 30.2 -> 28.8 us).
__device__ __forceinline__ uint64_t evict_first() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
// 16 bytes global -> shared past L1; n = 0 reads nothing and writes zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t n, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint.L2::128B [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(n),
               "l"(policy)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until all but the newest N groups of this thread have landed.
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_b16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The work: a (sequence, head) of n tiles takes `over` + n places of a line, (sequence, head) by
// (sequence, head), tile i of one at s0 the place s0 + over + i; G blocks have equal stretches of it.
struct SweepPlan {
  int W, G, base, rem;  // the first rem blocks have base + 1, the others base
  int slack;            // tiles by which a boundary moves to spare a cut
  int w, end;           // the block's stretch, boundaries moved as below
  int b, g, n0;         // its first tile: sequence, head, key tile
};
struct Tiles {
  const int* cum;  // shared memory: the cost of one head before sequence b
  int B, Hkv, over, whole;
  // the last b with Hkv * cum[b] <= x, by a whole warp: 32 probes at a time
  __device__ int find_warp(int x, int lane) const {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) >> 5, i = lo + lane * step;
      const unsigned le = __ballot_sync(0xffffffffu, i < hi && cum[i] * Hkv <= x);
      lo += (31 - __clz((int)le)) * step;
      hi = min(hi, lo + step);
    }
    return lo;
  }
  // The boundary x, in sequence i: at an end of its (sequence, head) if that is at most `slack` tiles away
  // or the whole has at most `whole`, else as it is.
  __device__ int moved(int x, int i, int slack) const {
    const int n = cum[i + 1] - cum[i], y = x - cum[i] * Hkv;
    int off = y - (int)__fdividef((float)y, (float)n) * n;  // y mod n, the quotient within one
    off += off < 0 ? n : 0;
    off -= off >= n ? n : 0;
    const int up = n - off, down = off - over;
    if (n - over <= whole) slack = n;
    if (down <= slack && down <= up) return x - off;
    return up <= slack ? x + up : x;
  }
  __device__ int nt(int b) const { return cum[b + 1] - cum[b] - over; }
  // The block whose unmoved stretch has x.
  __device__ int at(const SweepPlan& p, int x) const {
    const int big = p.rem * (p.base + 1);
    return x < big ? x / (p.base + 1) : p.rem + (x - big) / p.base;
  }
  // The first and last block of a (sequence, head) of n tiles that is cut, so has more than 2 slack
  // + 1 of them: the boundaries within `slack` of its ends have moved there.
  __device__ int first(const SweepPlan& p, int s0) const { return at(p, s0 + over + p.slack); }
  __device__ int last(const SweepPlan& p, int s0, int n) const { return at(p, s0 + over + n - 1 - p.slack); }
};
// cum[0 .. B]: the running sum of cost(b), by the block's THREADS threads (wsum: a word for each warp).
template <int THREADS, class F>
__device__ __forceinline__ void running_costs(int B, int* cum, int* wsum, int tid, F cost) {
  const int warp = tid >> 5, lane = tid & 31;
  if (tid == 0) cum[0] = 0;
  int before = 0;
  for (int b0 = 0; b0 < B; b0 += THREADS) {
    const int b = b0 + tid;
    int x = b < B ? cost(b) : 0;
    if (b0 + warp * 32 < B) {
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, m);
        if (lane >= m) x += y;
      }
    }
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    if (b0 + warp * 32 < B) {
      int low = lane < warp ? wsum[lane] : 0;  // at most 12 warps
#pragma unroll
      for (int m = 16; m; m >>= 1) low += __shfl_xor_sync(0xffffffffu, low, m);
      if (b < B) cum[b + 1] = before + low + x;
    }
    if (b0 + THREADS < B) {
      for (int i = 0; i < THREADS / 32; i++) before += wsum[i];
      __syncthreads();
    }
  }
  __syncthreads();
}
// Block blk of nblk: its stretch and its first tile, into splan (slack: see SweepPlan; div(W, G) = W / G).
// Two warps divide the work (a division costs every warp its issue slots): the block's first tile and
// the next block's.
template <class F>
__device__ __forceinline__ void divide_work(const Tiles& tl, volatile SweepPlan* splan, int blk, int nblk, int slack,
                                            int warp, int lane, F div) {
  if (warp < 2) {
    SweepPlan p;
    p.W = tl.cum[tl.B] * tl.Hkv;
    p.G = min(p.W, nblk);
    p.base = p.W == p.G ? 1 : div(p.W, p.G);
    p.rem = p.W - p.base * p.G;
    const int c = blk + warp, x = c * p.base + min(c, p.rem);
    const bool any = blk < p.G && x < p.W;
    p.b = tl.find_warp(min(x, p.W - 1), lane);
    p.slack = min(slack, p.base / 2);
    p.w = any ? tl.moved(x, p.b, p.slack) : p.W;
    if (lane == 0 && warp == 1) splan->end = p.w;
    if (lane == 0 && warp == 0) {
      if (p.w == tl.cum[p.b + 1] * tl.Hkv) p.b++;  // moved to the next sequence's first tile
      if (p.b == tl.B) p.b--;                      // nothing left
      const int n = tl.cum[p.b + 1] - tl.cum[p.b], off = p.w - tl.cum[p.b] * tl.Hkv;
      p.g = (int)__fdividef((float)off, (float)n);  // within one of off / n
      p.n0 = off - p.g * n;
      while (p.n0 < 0) p.g--, p.n0 += n;
      while (p.n0 >= n) p.g++, p.n0 -= n;
      p.n0 = max(p.n0 - tl.over, 0);
      splan->slack = p.slack;
      splan->W = p.W;
      splan->G = p.G;
      splan->base = p.base;
      splan->rem = p.rem;
      splan->w = p.w;
      splan->b = p.b;
      splan->g = p.g;
      splan->n0 = p.n0;
    }
  }
}
// Walks a block's stretch segment by segment.
template <int OVER>
struct SegWalk {
  const int* cum;
  int Hkv, w, end;
  int b, g, n0, n1, nt;  // the segment: key tiles [n0, n1) of nt
  __device__ void init(const Tiles& t, const volatile SweepPlan* p) {
    cum = t.cum;
    Hkv = t.Hkv;
    w = p->w;
    end = p->end;
    b = p->b;
    g = p->g;
    n0 = p->n0;
    nt = -1;
  }
  __device__ bool next() {
    if (nt >= 0) {  // the segment before ended with its (sequence, head), or the stretch with it
      n0 = 0;
      if (++g == Hkv) {
        g = 0;
        b++;
      }
    }
    if (n0 == 0) w += OVER;
    if (w >= end) return false;
    nt = cum[b + 1] - cum[b] - OVER;
    n1 = min(nt, n0 + (end - w));
    w += n1 - n0;
    return true;
  }
};

// A row's parts (maximum z in log2 units, sum, O), some lanes each with a few: the maximum of
// all, then sums of the rescaled parts (0 where a part's sum is 0: the row saw none of its keys).
struct RowSum {
  float M = -INFINITY, S = 0.f;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  // to the maximum `top`, which is at least M
  __device__ void raise(float top) {
    const float f = S == 0.f ? 0.f : ex2(M - top);
    M = top;
    S *= f;
    v = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
  }
  __device__ void add(float top, float2 z, const float4& u) {
    const float f = z.y == 0.f ? 0.f : ex2(z.x - top);
    S = fmaf(f, z.y, S);
    v = make_float4(fmaf(f, u.x, v.x), fmaf(f, u.y, v.y), fmaf(f, u.z, v.z), fmaf(f, u.w, v.w));
  }
};

struct SweepBars {
  uint64_t *q_full, *q_empty, *parts_full, *parts_empty, *fin, *stored;
};

// What a consumer warp holds of a segment: its rows' queries (in registers for at most 16 rows, else
// read from shared memory as they are used), O, running maximum and sum.  Up to 8 rows they are
// twice in one matrix tile, high and low parts; with more a tile has 16 rows, and the parts are
// two products into the same sums, which halves O's registers (16 contexts around 8192, 32 rows: 56 us
// for 69).
template <int D, int MT>
struct SweepState {
  static constexpr int KS = D / 16;
  static constexpr bool kTwice = MT == 1;
  static constexpr int MF = kTwice ? 1 : MT / 2;      // matrix tiles
  static constexpr int kParts = kTwice ? 1 : 2, kH = kTwice ? 1 : 2;  // products of a score; rows of a lane in a tile
  static constexpr bool kQRegs = MT <= 2;
  uint32_t q[kQRegs ? MF : 1][kParts][KS][4], qbase;
  float o[MF][2 * KS][4], mx[MF][kH], ls[MF][kH];
  int lim[MF][kH];  // last visible position of this lane's rows, from the own part's start
  int own, pos0;    // positions of the own part; row 0's position

  // Part p of the queries of tile m, columns 16 k ..: rows 8 .. 15 of the fragment come from the low
  // parts behind the eight rows, or from the next eight rows.
  __device__ __forceinline__ uint32_t q_at(int m, int p, int k, int lane) const {
    constexpr uint32_t kSpan = Sweep<D>::kSpan;
    const uint32_t lrow = lane & 15, lchk = lane >> 4;
    if (kTwice) return qbase + swz(lrow, 2 * k + lchk, kSpan);
    return qbase + (2 * m + (lrow >> 3)) * 16 * kSpan + swz((lrow & 7) + 8 * p, 2 * k + lchk, kSpan);
  }
  __device__ __forceinline__ void begin(const PagedDecodeArgs& a, int mg, int lane) {
#pragma unroll
    for (int m = 0; m < MF; m++) {
#pragma unroll
      for (int h = 0; h < kH; h++) {
        mx[m][h] = -INFINITY;
        ls[m][h] = 0.f;
        const int r = (mg * MT + kH * m + h) * 8 + (lane >> 2);
        lim[m][h] = r < a.R ? pos0 + (int)fdiv((uint32_t)r, a.div_g) : own - 1;
      }
#pragma unroll
      for (int i = 0; i < 2 * KS; i++)
#pragma unroll
        for (int e = 0; e < 4; e++) o[m][i][e] = 0.f;
    }
  }
  // The segment's parts: row (lane / 4) of each eight, maximum in log2 units.
  __device__ __forceinline__ void store(float* scratch, float2* ml, int warp, float sl2, int lane) {
#pragma unroll
    for (int m = 0; m < MF; m++)
#pragma unroll
      for (int h = 0; h < kH; h++) {
        float l = ls[m][h];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        const int row = (warp * MT + kH * m + h) * 8 + (lane >> 2);
        if ((lane & 3) == 0) ml[row] = make_float2(mx[m][h] == -INFINITY ? -INFINITY : __fmul_rn(mx[m][h], sl2), l);
#pragma unroll
        for (int i = 0; i < 2 * KS; i++)
          *reinterpret_cast<float2*>(scratch + row * D + i * 8 + (lane & 3) * 2) =
              kTwice ? make_float2(o[m][i][0] + o[m][i][2], o[m][i][1] + o[m][i][3])
                     : make_float2(o[m][i][2 * h], o[m][i][2 * h + 1]);
      }
  }
};
// Slices of 16 keys that a warp takes together: two where the registers allow it, which gives
// its chain of dependent steps (scores, maximum, weights, P V) something to overlap with.
template <int D, int MT>
constexpr int kSlicesAtOnce = MT * D <= 128 ? 2 : 1;

// N slices (keys at kb, values at vb, first position j0) into the state.
template <int D, int MT, int N>
__device__ __forceinline__ void sweep_slices(SweepState<D, MT>& w, const uint32_t (&kb)[N], const uint32_t (&vb)[N],
                                             const int (&j0)[N], float sl2, int lane) {
  constexpr int KS = D / 16;
  constexpr uint32_t kSpan = Sweep<D>::kSpan;
  // this lane's ldmatrix row and chunk parity (keys, values and queries alike)
  const uint32_t lrow = lane & 15, lchk = lane >> 4;
  uint32_t kf[N][KS][4], vf[N][KS][4];
#pragma unroll
  for (int i = 0; i < N; i++)
#pragma unroll
    for (int k = 0; k < KS; k++) ldsm4(kf[i][k], kb[i] + swz(lrow, 2 * k + lchk, kSpan));
#pragma unroll
  for (int i = 0; i < N; i++) {
#pragma unroll
    for (int k = 0; k < KS; k++) ldsm4t(vf[i][k], vb[i] + swz(lrow, 2 * k + lchk, kSpan));
    if (j0[i] + 16 > w.own) {
      // what lies behind the last position may be anything: its weight is 0, but 0 times a
      // NaN is not
      const int v0 = w.own - j0[i] - (lane & 3) * 2;
      const uint32_t m0 = (v0 > 0 ? 0xffffu : 0u) | (v0 > 1 ? 0xffff0000u : 0u);
      const uint32_t m1 = (v0 > 8 ? 0xffffu : 0u) | (v0 > 9 ? 0xffff0000u : 0u);
#pragma unroll
      for (int k = 0; k < KS; k++) {
        vf[i][k][0] &= m0;
        vf[i][k][1] &= m1;
        vf[i][k][2] &= m0;
        vf[i][k][3] &= m1;
      }
    }
  }
  using W = SweepState<D, MT>;
  constexpr int kH = W::kH, kV = 4 * kH;  // rows and values of a slice per lane
#pragma unroll
  for (int m = 0; m < W::MF; m++) {
    float sa[N][4], sb[N][4];
#pragma unroll
    for (int i = 0; i < N; i++)
#pragma unroll
      for (int e = 0; e < 4; e++) sa[i][e] = sb[i][e] = 0.f;
#pragma unroll
    for (int k = 0; k < KS; k++)
#pragma unroll
      for (int p = 0; p < W::kParts; p++) {
        uint32_t qt[4];
        if (W::kQRegs) {
#pragma unroll
          for (int e = 0; e < 4; e++) qt[e] = w.q[W::kQRegs ? m : 0][p][k][e];
        } else {
          ldsm4(qt, w.q_at(m, p, k, lane));
        }
#pragma unroll
        for (int i = 0; i < N; i++) {
          mma_f16(sa[i], qt, kf[i][k][0], kf[i][k][2]);
          mma_f16(sb[i], qt, kf[i][k][1], kf[i][k][3]);
        }
      }
    // row h, keys (lane & 3) * 2 + {0, 1} and those + 8 at 4 h .. 4 h + 3
    float x[N][kV], t[kH];
#pragma unroll
    for (int h = 0; h < kH; h++) t[h] = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; i++) {
      if (W::kTwice) {  // high + low part
        x[i][0] = sa[i][0] + sa[i][2];
        x[i][1] = sa[i][1] + sa[i][3];
        x[i][2] = sb[i][0] + sb[i][2];
        x[i][3] = sb[i][1] + sb[i][3];
      } else {
#pragma unroll
        for (int e = 0; e < kV; e++) x[i][e] = (e & 2 ? sb : sa)[i][(e >> 2) * 2 + (e & 1)];
      }
      if (j0[i] + 16 > w.pos0 + 1) {  // some row does not see every key of the slice
        const int k0 = j0[i] + (lane & 3) * 2;
#pragma unroll
        for (int e = 0; e < kV; e++)
          if (k0 + (e & 1) + ((e >> 1) & 1) * 8 > w.lim[m][e >> 2]) x[i][e] = -INFINITY;
      }
#pragma unroll
      for (int h = 0; h < kH; h++)
        t[h] = fmaxf(t[h], fmaxf(fmaxf(x[i][4 * h], x[i][4 * h + 1]), fmaxf(x[i][4 * h + 2], x[i][4 * h + 3])));
    }
    // O and the sum follow the maximum only when it grew by more than 2^8
    bool grow[kH], any = false;
#pragma unroll
    for (int h = 0; h < kH; h++) {
      t[h] = fmaxf(t[h], __shfl_xor_sync(0xffffffffu, t[h], 1));
      t[h] = fmaxf(t[h], __shfl_xor_sync(0xffffffffu, t[h], 2));
      const float mx = w.mx[m][h];
      grow[h] = mx == -INFINITY ? t[h] > -INFINITY : __fmul_rn(t[h], sl2) > __fmul_rn(mx, sl2) + 8.f;
      any = any || grow[h];
    }
    if (__any_sync(0xffffffffu, any)) {
#pragma unroll
      for (int h = 0; h < kH; h++) {
        const float mx = w.mx[m][h];
        const float al = grow[h] && mx != -INFINITY ? ex2(__fmul_rn(mx, sl2) - __fmul_rn(t[h], sl2)) : 1.f;
        w.mx[m][h] = grow[h] ? t[h] : mx;
        w.ls[m][h] *= al;
#pragma unroll
        for (int i = 0; i < 2 * KS; i++)
#pragma unroll
          for (int e = 0; e < 4; e++)
            if (W::kTwice || (e >> 1) == h) w.o[m][i][e] *= al;
      }
    }
    float mu[kH];
#pragma unroll
    for (int h = 0; h < kH; h++) mu[h] = w.mx[m][h] == -INFINITY ? 0.f : __fmul_rn(w.mx[m][h], sl2);
#pragma unroll
    for (int i = 0; i < N; i++) {
      float p[kV];
#pragma unroll
      for (int e = 0; e < kV; e++) p[e] = ex2(fmaf(x[i][e], sl2, -mu[e >> 2]));
#pragma unroll
      for (int h = 0; h < kH; h++) w.ls[m][h] += (p[4 * h] + p[4 * h + 1]) + (p[4 * h + 2] + p[4 * h + 3]);
      // the weights' bf16 high parts and remainders, by row and eight keys
      uint32_t hi[2 * kH], lo[2 * kH];
#pragma unroll
      for (int e = 0; e < 2 * kH; e++) {
        hi[e] = pack_bf16(p[2 * e], p[2 * e + 1]);
        lo[e] = pack_bf16(p[2 * e] - bf_lo(hi[e]), p[2 * e + 1] - bf_hi(hi[e]));
      }
      if constexpr (W::kTwice) {
        const uint32_t pa[4] = {hi[0], lo[0], hi[1], lo[1]};
#pragma unroll
        for (int k = 0; k < KS; k++) {
          mma_b16(w.o[m][2 * k], pa, vf[i][k][0], vf[i][k][1]);
          mma_b16(w.o[m][2 * k + 1], pa, vf[i][k][2], vf[i][k][3]);
        }
      } else {
        const uint32_t ph[4] = {hi[0], hi[kH], hi[1], hi[kH + 1]}, pl[4] = {lo[0], lo[kH], lo[1], lo[kH + 1]};
#pragma unroll
        for (int k = 0; k < KS; k++) {
          mma_b16(w.o[m][2 * k], ph, vf[i][k][0], vf[i][k][1]);
          mma_b16(w.o[m][2 * k + 1], ph, vf[i][k][2], vf[i][k][3]);
        }
#pragma unroll
        for (int k = 0; k < KS; k++) {
          mma_b16(w.o[m][2 * k], pl, vf[i][k][0], vf[i][k][1]);
          mma_b16(w.o[m][2 * k + 1], pl, vf[i][k][2], vf[i][k][3]);
        }
      }
    }
  }
}

// A finished row: written out, or (prefix) kept as the sequence's own part for k_prefix_join.
template <int D, bool PREFIX>
__device__ __forceinline__ void put_row(const PagedDecodeArgs& a, bool prefix, int b, int g, int r, int q, float4 v,
                                        float M, float S) {
  if (PREFIX && prefix) {
    const size_t row = (size_t)g * a.pre.tiles * kTile + (size_t)b * a.R + r;
    reinterpret_cast<float4*>(a.pre.o + row * D)[q] = v;
    if (q == 0) a.pre.ml[row] = make_float2(M, S);
  } else {
    write_row<D>(a, b, g, r, q, v, M, S);
  }
}

// Joins the consumers' parts of a segment, thread t of n: a whole (sequence, head) is written out, a
// part of one left in the workspace.
template <int D, int MT, bool PREFIX>
__device__ __forceinline__ void join_warps(const PagedDecodeArgs& a, const SegWalk<seg_cost(D)>& sw, const int* len,
                                           const float* scratch, const float2* ml, int blk, int t, int n) {
  const int parts = MT < 4 ? kWarps : kWarps / a.MG;  // warps that hold a part of a row
  const bool whole = sw.n0 == 0 && sw.n1 == sw.nt;
  const int slot = sw.n0 > 0 ? 0 : 1;  // a block's first segment is the only one that begins inside
  const bool pre = PREFIX && sweep_base(a, len[sw.b]) > 0;
  // a thread takes columns 4 q .. and 4 (q + D / 8) .. of a row
  constexpr int kQ = D / 8;
  const int items = a.R * kQ;
  for (int i = t; i < items; i += n) {
    const int r = i / kQ, q = i % kQ, tile = r >> 3;
    const int at0 = ((tile / MT) * parts * MT + tile % MT) * 8 + (r & 7);
    RowSum x, y;
#pragma unroll
    for (int k = 0; k < kWarps; k++)
      if (MT < 4 || k < parts) x.M = fmaxf(x.M, ml[at0 + k * MT * 8].x);
#pragma unroll 4
    for (int k = 0; k < parts; k++) {
      const int from = at0 + k * MT * 8;
      const float2 z = ml[from];
      x.add(x.M, z, *reinterpret_cast<const float4*>(scratch + from * D + 4 * q));
      y.add(x.M, z, *reinterpret_cast<const float4*>(scratch + from * D + 4 * (q + kQ)));
    }
    if (whole) {
      put_row<D, PREFIX>(a, pre, sw.b, sw.g, r, q, x.v, x.M, x.S);
      put_row<D, PREFIX>(a, pre, sw.b, sw.g, r, q + kQ, y.v, x.M, x.S);
    } else {
      const size_t at1 = (size_t)(2 * blk + slot) * a.R + r;
      float4* to = reinterpret_cast<float4*>(a.part_o + at1 * D) + q;
      to[0] = x.v;
      to[kQ] = y.v;
      if (q == 0) a.part_ml[at1] = make_float2(x.M, x.S);
    }
  }
}

template <int D, int MT, bool PREFIX>
__device__ bool sweep_consume(const PagedDecodeArgs& a, SegWalk<seg_cost(D)> sw, const int* len, uint8_t* smem, const SweepSmem& L,
                              const SweepBars& bar, const volatile int* abort, int blk, int warp, int lane) {
  using C = Sweep<D>;
  constexpr int KS = D / 16;
  constexpr int kBufs = sweep_bufs(D, MT);
  const int KG = MT < 4 ? kWarps : kWarps / a.MG;  // warps over a tile's keys; the rest share the row tiles out
  const int mg = warp / KG, kg = warp - mg * KG;
  const uint64_t policy = evict_first();
  const float sl2 = a.scale_log2;
  constexpr int S = kDepth<D, MT>, kN = kSlicesAtOnce<D, MT>;
  constexpr int kCPR = D / 8, kCopies = 16 * kCPR / 32;  // 16-byte chunks of a row; of a slice, per lane
  const int lm = MT < 4 ? 0 : (a.MG == 1 ? 0 : (a.MG == 2 ? 1 : 2));  // log2 of a tile's slices per warp
  const uint32_t ring = smem_u32(smem + L.ring) + (uint32_t)warp * S * C::kSlot;
  // Slice k of a segment is 16 positions from place(segment, k).  The warp copies its own slices,
  // S ahead of the one it works on: no other warp reads them, so a copy needs no barrier, and a
  // slice lies in one page, so small pages cost nothing (with tiled copies by a producer warp,
  // pages of 16 took 0.87 us a tile and larger ones 0.70).
  const auto slices = [&](const auto& s) { return (s.n1 - s.n0) << lm; };
  const auto place = [&](const auto& s, int k) {
    return (s.n0 + (k >> lm)) * kTK + (kg + (k & ((1 << lm) - 1)) * KG) * 16;
  };
  // Page numbers come 32 slices at a time, one to a lane and a window ahead: -1 where nothing is
  // to be read, -2 for a bad page.
  const auto window = [&](const auto& s, int k0) {
    const int base = sweep_base(a, len[s.b]), own = len[s.b] - base, k = k0 + lane;
    int id = -1;
    if (k < slices(s)) {
      const int j0 = place(s, k);
      if (j0 < own) {
        const int i = (base + j0) >> a.page_shift;
        id = i < (a.prefix_len >> a.page_shift) ? a.prefix_table[i] : a.table[(size_t)s.b * a.max_pages + i];
        if (id < 0 || id >= a.num_pages) {
          record_page(a.status);
          id = -2;
        }
      }
    }
    return id;
  };
  SegWalk<seg_cost(D)> is = sw, ls = sw;  // the segment being copied, and that of the window after this one
  bool ion = is.next(), lon = ls.next();
  int ik = 0, iw = 0, lk = 0, islot = 0, id = -1, nid = -1;
  const auto look = [&]() {
    if (!lon) return;
    if (lk + 32 < slices(ls)) {
      lk += 32;
    } else {
      lon = ls.next();
      lk = 0;
    }
    nid = lon ? window(ls, lk) : -1;
  };
  if (ion) id = window(is, 0);
  look();
  const auto issue = [&]() {
    if (ion && (ik - iw == 32 || ik == slices(is))) {
      is = ls;
      ion = lon;
      ik = iw = lk;
      id = nid;
      look();
    }
    if (ion) {
      const int page = __shfl_sync(0xffffffffu, id, ik - iw);
      if (page != -1) {
        const int j0 = place(is, ik);
        const size_t at = (size_t)max(page, 0) * a.page_stride +
                          (((size_t)is.g << a.page_shift) + (j0 & ((1 << a.page_shift) - 1))) * D + lane * 8;
        const uint32_t n = page < 0 ? 0u : 16u, to = ring + islot * C::kSlot;
#pragma unroll
        for (int i = 0; i < kCopies; i++) {
          const uint32_t row = i * (32 / kCPR) + lane / kCPR, off = swz(row, lane % kCPR, C::kSpan);
          copy16(to + off, a.kp + at + i * 256, n, policy);
          copy16(to + C::kSlot / 2 + off, a.vp + at + i * 256, n, policy);
        }
      }
      ik++;
    }
    copy_commit();
    islot = islot + 1 == S ? 0 : islot + 1;
  };
#pragma unroll 1
  for (int i = 0; i < S; i++) issue();
  int cslot = 0, seg = 0;
  const int qbufs = sweep_qbufs(a.tiles);
  for (; sw.next(); seg++) {
    SweepState<D, MT> w;
    const int total = len[sw.b];
    w.own = total - sweep_base(a, total);
    w.pos0 = w.own - a.Tq;
    const int qs = qbufs == 2 ? seg & 1 : 0;
    if (!__all_sync(0xffffffffu, mbar_wait(bar.q_full + qs, (qbufs == 2 ? seg >> 1 : seg) & 1, abort))) {
      copy_wait<0>();
      return false;
    }
    w.qbase = smem_u32(smem + L.q) + (uint32_t)((qs * a.tiles + mg * MT) * 16) * C::kSpan;
    if (w.kQRegs) {
#pragma unroll
      for (int m = 0; m < w.MF; m++)
#pragma unroll
        for (int p = 0; p < w.kParts; p++)
#pragma unroll
          for (int k = 0; k < KS; k++) ldsm4(w.q[w.kQRegs ? m : 0][p][k], w.q_at(m, p, k, lane));
      warp_arrive(bar.q_empty + qs);
    }
    w.begin(a, mg, lane);
    const int cnt = slices(sw);
    for (int k = 0; k < cnt;) {
      const int j0 = place(sw, k);
      const uint32_t k0 = ring + cslot * C::kSlot;
      cslot = cslot + 1 == S ? 0 : cslot + 1;
      if (kN == 2 && k + 1 < cnt) {
        const uint32_t k1 = ring + cslot * C::kSlot;
        cslot = cslot + 1 == S ? 0 : cslot + 1;
        copy_wait<S - 2>();
        __syncwarp();
        if (j0 < w.own) {
          const uint32_t kb[2] = {k0, k1}, vb[2] = {k0 + C::kSlot / 2, k1 + C::kSlot / 2};
          const int jn[2] = {j0, place(sw, k + 1)};
          sweep_slices<D, MT, 2>(w, kb, vb, jn, sl2, lane);
        }
        __syncwarp();
        issue();
        issue();
        k += 2;
      } else {
        copy_wait<S - 1>();
        __syncwarp();
        if (j0 < w.own) {
          const uint32_t kb[1] = {k0}, vb[1] = {k0 + C::kSlot / 2};
          const int jn[1] = {j0};
          sweep_slices<D, MT, 1>(w, kb, vb, jn, sl2, lane);
        }
        __syncwarp();
        issue();
        k++;
      }
    }
    if (!w.kQRegs) warp_arrive(bar.q_empty + qs);
    // the warps' parts go to shared memory, where they are joined
    const int buf = seg % kBufs, use = seg / kBufs;
    if (use > 0 && !__all_sync(0xffffffffu, mbar_wait(bar.parts_empty + buf, (use - 1) & 1, abort))) {
      copy_wait<0>();
      return false;
    }
    float* scratch = reinterpret_cast<float*>(smem + L.scratch) + buf * kWarps * MT * 8 * D;
    float2* ml = reinterpret_cast<float2*>(smem + L.ml) + buf * kWarps * MT * 8;
    w.store(scratch, ml, warp, sl2, lane);
    if (kBufs == 1) {
      warp_arrive(bar.stored);
      if (!__all_sync(0xffffffffu, mbar_wait(bar.stored, seg & 1, abort))) {
        copy_wait<0>();
        return false;
      }
      join_warps<D, MT, PREFIX>(a, sw, len, scratch, ml, blk, warp * 32 + lane, kWarps * 32);
    }
    warp_arrive(bar.parts_full + buf);
  }
  copy_wait<0>();
  return true;
}

// Counts a segment, the last one (number `last`) back to 0: its part is visible before the
// count, and the parts of those counted before are visible after it.
__device__ __forceinline__ bool count_segment(unsigned* done, unsigned last) {
  unsigned old;
  asm volatile("atom.inc.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(old) : "l"(done), "r"(last) : "memory");
  return old == last;
}

// Finishing warp f: joins the consumers' parts of every kBufs-th segment (with one buffer, more rows,
// the consumers do that themselves: one warp took 2.6 us for 32 rows).  A part of a (sequence, head) is
// counted, and the block that counts the last one notes it in todo[first or second cut segment of the
// block] for its consumers.
template <int D, int MT, bool PREFIX>
__device__ bool sweep_finish(const PagedDecodeArgs& a, SegWalk<seg_cost(D)> sw, const Tiles& tl, const SweepPlan& plan,
                             const int* len, uint8_t* smem, const SweepSmem& L, const SweepBars& bar, volatile int* todo,
                             const volatile int* abort, int blk, int f, int lane) {
  constexpr int kBufs = sweep_bufs(D, MT);
  const float* scratch = reinterpret_cast<const float*>(smem + L.scratch) + f * kWarps * MT * 8 * D;
  const float2* ml = reinterpret_cast<const float2*>(smem + L.ml) + f * kWarps * MT * 8;
  bool waited = false;
  for (int seg = 0; sw.next(); seg++) {
    if (seg % kBufs != f) continue;
    if (!waited) {
      pdl_wait();  // the kernel before clears the workspace's counters
      waited = true;
    }
    if (!__all_sync(0xffffffffu, mbar_wait(bar.parts_full + f, (seg / kBufs) & 1, abort))) return false;
    if (kBufs == 2) join_warps<D, MT, PREFIX>(a, sw, len, scratch, ml, blk, lane, 32);
    warp_arrive(bar.parts_empty + f);
    if (sw.n0 == 0 && sw.n1 == sw.nt) continue;
    __syncwarp();  // the other lanes' parts before lane 0's release
    if (lane == 0) {
      const int s0 = tl.cum[sw.b] * tl.Hkv + sw.g * (sw.nt + tl.over);
      const int c0 = tl.first(plan, s0), c1 = tl.last(plan, s0, sw.nt);
      if (count_segment(a.done + c0, (unsigned)(c1 - c0))) todo[sw.n0 > 0 ? 0 : 1] = sw.b * tl.Hkv + sw.g;
    }
    __syncwarp();
  }
  warp_arrive(bar.fin);
  return true;
}

// The (sequence, head)s whose last segment this block counted: their segments in order, up to four
// neighbouring lanes to four columns of a row, as the threads suffice for all rows at once (each its
// own share, then lane by lane: the same sum whichever block does it).
template <int D, int MT, bool PREFIX>
__device__ bool sweep_join(const PagedDecodeArgs& a, const Tiles& tl, const SweepPlan& plan, const int* len,
                           const SweepBars& bar, const volatile int* todo, const volatile int* abort, int tid) {
  constexpr int kThreads = kWarps * 32, kAhead = 4;
  if (!__all_sync(0xffffffffu, mbar_wait(bar.fin, 0, abort))) return false;
  for (int k = 0; k < 2; k++) {
    const int sh = todo[k];
    if (sh < 0) continue;
    __threadfence();
    const int b = sh / tl.Hkv, g = sh - b * tl.Hkv, nt = tl.nt(b);
    const int s0 = tl.cum[b] * tl.Hkv + g * (nt + tl.over);
    const int c0 = tl.first(plan, s0), c1 = tl.last(plan, s0, nt);
    const int items = a.R * (D / 4), lg = items <= kThreads / 4 ? 2 : (items <= kThreads / 2 ? 1 : 0);
    const int split = 1 << lg, sub = tid & (split - 1);
    for (int i0 = 0; i0 < items; i0 += kThreads >> lg) {
      const int i = min(i0 + (tid >> lg), items - 1);
      const int r = i / (D / 4), q = i % (D / 4);
      const auto at = [&](int c) { return (size_t)(2 * c + (c == c0 ? 1 : 0)) * a.R + r; };
      RowSum x;
      for (int c = c0 + sub; c <= c1; c += kAhead << lg) {
        float2 z[kAhead];
        float4 u[kAhead];
#pragma unroll
        for (int e = 0; e < kAhead; e++) {
          z[e] = make_float2(-INFINITY, 0.f);
          u[e] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (c + (e << lg) <= c1) {
            z[e] = __ldcg(a.part_ml + at(c + (e << lg)));
            u[e] = __ldcg(reinterpret_cast<const float4*>(a.part_o + at(c + (e << lg)) * D) + q);
          }
        }
        float top = x.M;
#pragma unroll
        for (int e = 0; e < kAhead; e++) top = fmaxf(top, z[e].x);
        x.raise(top);
#pragma unroll
        for (int e = 0; e < kAhead; e++) x.add(top, z[e], u[e]);
      }
      float top = x.M;
      for (int m = 1; m < split; m <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
      x.raise(top);
      for (int m = 1; m < split; m <<= 1) {
        x.S += __shfl_xor_sync(0xffffffffu, x.S, m);
        x.v.x += __shfl_xor_sync(0xffffffffu, x.v.x, m);
        x.v.y += __shfl_xor_sync(0xffffffffu, x.v.y, m);
        x.v.z += __shfl_xor_sync(0xffffffffu, x.v.z, m);
        x.v.w += __shfl_xor_sync(0xffffffffu, x.v.w, m);
      }
      if (sub == 0 && i0 + (tid >> lg) < items) put_row<D, PREFIX>(a, PREFIX && sweep_base(a, len[b]) > 0, b, g, r, q, x.v, top, x.S);
    }
  }
  return true;
}

// With PREFIX the first blocks take the shared prefix's tiles, the others the sweep: the one is bound
// by the tensor cores and exponentials, the other by HBM, and they run side by side.
template <int D, int MT, bool PREFIX>
__global__ void __launch_bounds__(kSweepThreads, 1) k_paged_sweep(const __grid_constant__ PagedDecodeArgs a) {
  constexpr int kThreads = kSweepThreads, kBufs = sweep_bufs(D, MT);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const SweepSmem L = sweep_smem(D, kDepth<D, MT>, a.tiles, MT, a.B);
  SweepBars bar;
  bar.q_full = reinterpret_cast<uint64_t*>(smem);  // [2]
  bar.q_empty = bar.q_full + 2;             // [2]
  bar.parts_full = bar.q_empty + 2;         // [2] a segment's parts are in shared memory
  bar.parts_empty = bar.parts_full + 2;     // [2] and have been read
  bar.fin = bar.parts_empty + 2;            // the finishing warps are done
  bar.stored = bar.fin + 1;                 // one buffer: all consumers' parts are in it
  volatile int* abort = reinterpret_cast<volatile int*>(smem + kOffVars);
  volatile int* todo = abort + 1;                              // [2]
  volatile SweepPlan* splan = reinterpret_cast<volatile SweepPlan*>(const_cast<int*>(abort) + 3);
  int* wsum = const_cast<int*>(abort) + 16;                    // [12] the scan's warp totals
  int* cum = reinterpret_cast<int*>(smem + kOffCum);
  int* len = cum + a.B + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // lengths, and the running count of the tiles of the parts read here
  const int cap = a.max_pages << a.page_shift;
  running_costs<kThreads>(a.B, cum, wsum, tid, [&](int b) {
    int n = a.len[b];
    if (n > cap) {
      if (blockIdx.x == 0) record_page(a.status);
      n = cap;
    }
    n = max(n, 0);
    len[b] = n;
    return seg_cost(D) + max(1, (n - sweep_base(a, n) + kTK - 1) / kTK);  // one even where nothing is read: its rows are written
  });
  int blk = (int)blockIdx.x, nblk = (int)gridDim.x;
  if constexpr (PREFIX) {
    const int P = prefix_blocks(a, cum[a.B] * a.Hkv, nblk);
    if (blk < P) {
      prefix_role<D>(a, len, smem + paged_head(a.B), P, tid);
      return;
    }
    blk -= P;
    nblk -= P;
  }
  if (tid == 32) {
    *abort = 0;
    todo[0] = todo[1] = -1;
    for (int i = 0; i < 2; i++) {
      mbar_init(bar.q_full + i, query_warps(D, MT));
      mbar_init(bar.q_empty + i, kWarps);
      mbar_init(bar.parts_full + i, kWarps);
      mbar_init(bar.parts_empty + i, 1);
    }
    mbar_init(bar.fin, kBufs);
    mbar_init(bar.stored, kWarps);
    fence_mbar_init();
  }
  Tiles tl;
  tl.cum = cum;
  tl.B = a.B;
  tl.Hkv = a.Hkv;
  tl.over = seg_cost(D);
  tl.whole = whole_tiles(D);
  divide_work(tl, splan, blk, nblk, max_slack(D), warp, lane,
              [&](int W, int G) { return PREFIX ? W / G : (int)fdiv((uint32_t)W, a.div_grid); });
  __syncthreads();
  SegWalk<seg_cost(D)> sw;
  sw.init(tl, splan);
  // registers: 384 x 168 at launch; 256 x 216 for the consumers, 128 x 72 for the others
  if (warp < kWarps) {
    regs_inc<216>();
    bool ok = sweep_consume<D, MT, PREFIX>(a, sw, len, smem, L, bar, abort, blk, warp, lane);
    if (ok) {
      SweepPlan p;
      p.W = splan->W;
      p.base = splan->base;
      p.rem = splan->rem;
      p.slack = splan->slack;
      ok = sweep_join<D, MT, PREFIX>(a, tl, p, len, bar, todo, abort, tid);
    }
    if (!ok && lane == 0) {
      *abort = 1;
      atomicExch(a.status, kStatusTimeout);
    }
    return;
  }
  regs_dec<72>();
  bool ok = true;
  const int qw = warp == kWarps ? 0 : warp - kWarps - kBufs;
  if (warp == kWarps || (qw > 0 && qw < query_warps(D, MT))) {
    // ------------------------------------------------------------ queries, two passes of rows at a time
    constexpr int kCPR = D / 8, kRows = 32 / kCPR;
    const int c = lane % kCPR;
    const bool norm = a.qw != nullptr;
    const int qbufs = sweep_qbufs(a.tiles);
    constexpr uint32_t kSpan = Sweep<D>::kSpan;
    uint4 wv = make_uint4(0, 0, 0, 0);
    if (norm) wv = load_rope_chunk<D>(a.qw, c, a.rope_half != 0);
    for (int seg = 0; ok && sw.next(); seg++) {
      const int qs = qbufs == 2 ? seg & 1 : 0, use = qbufs == 2 ? seg >> 1 : seg;
      if (use > 0) ok = __all_sync(0xffffffffu, mbar_wait(bar.q_empty + qs, (use - 1) & 1, abort));
      if (!ok) break;
      const int pos0 = len[sw.b] - a.Tq;
      uint8_t* q = smem + L.q + qs * a.tiles * 16 * kSpan;
      for (int r0 = qw * 2 * kRows; r0 < a.tiles * 8; r0 += query_warps(D, MT) * 2 * kRows) {
        const int r = r0 + lane / kCPR, r2 = r + kRows;
        const QueryChunk x = query_load<D>(a, sw.b, sw.g, r, c, pos0), y = query_load<D>(a, sw.b, sw.g, r2, c, pos0);
        uint4 hi, lo;
        query_finish<D>(a, x, norm, wv, hi, lo);
        *reinterpret_cast<uint4*>(q + (r >> 3) * 16 * kSpan + swz(r & 7, c, kSpan)) = hi;
        *reinterpret_cast<uint4*>(q + (r >> 3) * 16 * kSpan + swz((r & 7) + 8, c, kSpan)) = lo;
        query_finish<D>(a, y, norm, wv, hi, lo);
        if (r2 < a.tiles * 8) {
          *reinterpret_cast<uint4*>(q + (r2 >> 3) * 16 * kSpan + swz(r2 & 7, c, kSpan)) = hi;
          *reinterpret_cast<uint4*>(q + (r2 >> 3) * 16 * kSpan + swz((r2 & 7) + 8, c, kSpan)) = lo;
        }
      }
      warp_arrive(bar.q_full + qs);
    }
  } else if (warp - kWarps - 1 < kBufs) {
    // ------------------------------------------------------------ finished segments
    SweepPlan p;
    p.W = splan->W;
    p.base = splan->base;
    p.rem = splan->rem;
    p.slack = splan->slack;
    ok = sweep_finish<D, MT, PREFIX>(a, sw, tl, p, len, smem, L, bar, todo, abort, blk, warp - kWarps - 1, lane);
  }
  if (!ok && lane == 0) {
    *abort = 1;
    atomicExch(a.status, kStatusTimeout);
  }
}

// The counters of the (sequence, head)s that several blocks share.
__global__ void k_paged_clear(unsigned* done, int n) {
  pdl_launch();
  for (int i = threadIdx.x; i < n; i += blockDim.x) done[i] = 0u;
}

template <int D, int MT, bool PREFIX>
cudaError_t launch_sweep_t(const PagedDecodeArgs& a, int nsm, cudaStream_t s) {
  static bool attr_set[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(k_paged_sweep<D, MT, PREFIX>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  PagedDecodeArgs b = a;
  int bytes = sweep_smem(D, kDepth<D, MT>, b.tiles, MT, b.B).total;
  if constexpr (PREFIX) bytes = bytes > prefix_smem(D, b.B) ? bytes : prefix_smem(D, b.B);
  if (bytes > kSmemMax) return cudaErrorInvalidValue;
  const int grid = nsm < kPagedMaxBlocks ? nsm : kPagedMaxBlocks;
  b.div_grid = make_fastdiv((uint32_t)grid);
  if (b.own_counters) {  // they are 0 before and after every call
    k_paged_sweep<D, MT, PREFIX><<<grid, kSweepThreads, (size_t)bytes, s>>>(b);
    return cudaGetLastError();
  }
  k_paged_clear<<<1, 256, 0, s>>>(b.done, kPagedMaxBlocks);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_pdl(k_paged_sweep<D, MT, PREFIX>, grid, kSweepThreads, (size_t)bytes, s, b);
}

template <bool PREFIX>
cudaError_t launch_sweep(const PagedDecodeArgs& a, int mt, int nsm, cudaStream_t s) {
  if (a.D == 64)
    return mt == 1 ? launch_sweep_t<64, 1, PREFIX>(a, nsm, s)
                   : (mt == 2 ? launch_sweep_t<64, 2, PREFIX>(a, nsm, s) : launch_sweep_t<64, 4, PREFIX>(a, nsm, s));
  return mt == 1 ? launch_sweep_t<32, 1, PREFIX>(a, nsm, s)
                 : (mt == 2 ? launch_sweep_t<32, 2, PREFIX>(a, nsm, s) : launch_sweep_t<32, 4, PREFIX>(a, nsm, s));
}

}  // namespace
}  // namespace ne
