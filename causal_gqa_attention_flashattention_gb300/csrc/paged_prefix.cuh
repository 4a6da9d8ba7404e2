// Shared prefix of a batch over a paged key/value cache (sm_103a).
//
// Every sequence of the batch starts with the same pages.  Their attention is
// computed once for all: the queries of one key/value head, of every sequence and
// new token, fill 128-row tiles (row b * R + r), and each key/value tile of the
// prefix is read once for two of them.  S = Q K^T and O += P V run on the tensor
// cores over the key tiles of the prefix, laid end to end over (head, pair of row
// tiles) and cut into one equal stretch per block; the softmax warps pack the queries
// (normalised, rotated, fp16) themselves while the first keys are on their way, and each
// segment leaves its unnormalised O and its rows' maximum and sum.  k_prefix_join
// (paged_prefix.cu) adds these parts and the sequences' own:
//   O = sum_s 2^(m_s - m) O_s / sum_s 2^(m_s - m) l_s.
//
// A sequence takes part if its first query sees the whole prefix, so no score is
// masked here but for the columns behind the prefix in its last tile; the sweep
// reads the prefix pages itself for one that does not.
// Precision: as the sweep's, so that a call gives the same o with and without a shared prefix: q as
// two fp16 parts (two products; with one the LSE is off by 1e-5), the weights as two bf16
// parts (2^-17; one part is 2^-9 off, and the call with a prefix then differs from the one without by
// more than a bf16 o's rounding). Both parts of all 128 keys would not fit the tensor memory, so P
// goes out in quarters of 32 keys through two buffers. 128 sequences on 16384 positions 39.7 us, with
// one part in halves 34.8: a third each for the second part's arithmetic, its products and the
// hand-offs (halves through one buffer 46.5 where quarters take 45.6).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"
#include "rope.cuh"

namespace ne {
namespace {

constexpr int kPagedHead0 = 384;  // a block's barriers and variables, before the lengths

template <int D>
struct PreCfg {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr uint32_t kSpan = D * 2;
  static constexpr uint32_t kSwz = D == 64 ? kSw128 : kSw64;
  static constexpr uint32_t kSBO = 8 * kSpan;
  static constexpr int kQSlots = 4;  // high and low part of each unit's row tile
  static constexpr int kStages = 4;
  static constexpr uint32_t kColO = 0, kColS = 128, kColP = 384;  // unit u: O at 64u, S at 128 + 128u, P at 384 + 64u:
  // two buffers of 32 columns, a quarter's high parts and then its low parts in each
  static constexpr uint32_t kTmemCols = 512;
  static constexpr int kThreads = 384;
  static constexpr int kOffK = kQSlots * kTileBytes;  // Q first: unit u at 2 u and 2 u + 1
  static constexpr int kOffV = kOffK + kStages * kTileBytes;
  static constexpr int kOffBar = kOffV + kStages * kTileBytes;
  static constexpr int kNumBars = 4 + 2 * kStages + 14 + 3;
  static constexpr int kBytes = kOffBar + kNumBars * 8 + 16;
};

inline int prefix_smem(int D, int B) {
  return (kPagedHead0 + (2 * B + 1) * 4 + 1023) / 1024 * 1024 + (D == 64 ? PreCfg<64>::kBytes : PreCfg<32>::kBytes) + 1024;
}

// The blocks that take the prefix, of all: their share of the work, a tile of a pair of row tiles
// counted as 3.25 of the sweep's (measured: 128 sequences on 16384 positions 40.1 us, with 3 42.3, with 3.5
// 40.2; 100 on 2048 21.0, 24.5, 21.0), and a (sequence, head) as one tile more than in the sweep's own
// plan, whose blocks share that cost alike (100 sequences of one own position on 131072 68.8 us, without
// 100; 64 of up to 16 on 65536 46.7, 49.5; 128 of up to 20 on 1024 20.4, 18.7). Above 16 rows the sweep is
// bound by its products, for every 32 rows a tile counts three times (40 sequences of 20 rows on 8192
// positions 34.0 us, with 1 52.9, 2 36.1, 4 37.7, 5 37.7; 20 of 64 rows on 4096 21.3, 22.0, 22.2, 21.6, 23.3).
__device__ __forceinline__ int prefix_blocks(const PagedDecodeArgs& a, int sweep_tiles, int blocks) {
  const float mine = 3.25f * (float)a.pre.W;
  const float theirs = ((float)sweep_tiles + (float)(a.B * a.Hkv)) * (a.D == 64 ? 1.f : 0.5f) * (a.R > 16 ? 3.f * (float)a.MG : 1.f);
  const int P = max(1, min(min(__float2int_rn((float)blocks * __fdiv_rn(mine, mine + theirs)), blocks - 1), a.pre.W));
  // the same number for every (head, pair), so that no block has parts of two (which costs it
  // a second packing and a second epilogue, about 4 us)
  const int segs = a.Hkv * a.pre.pairs;
  if (P < segs) return P;
  const int most = min(blocks - 1, a.pre.W) / segs;
  const int k = max(1, min((P + segs / 2) / segs, most)), n = (a.pre.ntk + k - 1) / k;
  return segs * ((a.pre.ntk + n - 1) / n);  // fewer, where the busiest of them then has no more tiles
}

struct PreSeg {
  int w, end;       // tiles of the block's stretch that are left
  int s, n0, n1;    // the segment: (head, pair) s, key tiles [n0, n1)
  __device__ void init(const PrefixArgs& p, int block, int blocks) {
    const PrefixCut cut(p.ntk, p.W / p.ntk, blocks);
    w = cut.start(block);
    end = cut.start(block + 1);
  }
  __device__ bool next(const PrefixArgs& p) {
    if (w >= end) return false;
    s = w / p.ntk;
    n0 = w - s * p.ntk;
    n1 = min(p.ntk, n0 + (end - w));
    w += n1 - n0;
    return true;
  }
  __device__ int units(const PrefixArgs& p) const { return 2 * (s % p.pairs) + 1 < p.tiles ? 2 : 1; }
};

// Rows r0 .. r0 + 31 of a packed tile whose first row is rho0, normalised and rotated, as fp16 high and low
// parts into the swizzled tiles at dst and behind it.  D / 8 neighbouring lanes to a row, so that a
// load takes whole lines (100 sequences on 2048 positions 23.9 us, with a lane to a row 25.4; 64 on 8192
// 20.5, 20.2, each with one part of the weights), all of the warp's rows under way at once.
template <int D>
__device__ __forceinline__ void pack_query_rows(const PagedDecodeArgs& a, const int* len, int g, int rho0, uint8_t* dst,
                                                int r0, int lane) {
  constexpr int kCPR = D / 8, kRows = 32 / kCPR, kPasses = 32 / kRows;
  const int c = lane % kCPR;
  uint4 wv = make_uint4(0, 0, 0, 0);
  if (a.qw) wv = load_rope_chunk<D>(a.qw, c, a.rope_half != 0);
  QueryChunk x[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; i++) {
    const int rho = rho0 + r0 + i * kRows + lane / kCPR, b = (int)fdiv((uint32_t)rho, a.div_r);
    const bool on = b < a.B;
    x[i] = query_load<D>(a, on ? b : 0, g, on ? rho - b * a.R : a.R, c, on ? len[b] - a.Tq : 0);
  }
#pragma unroll
  for (int i = 0; i < kPasses; i++) {
    const int r = r0 + i * kRows + lane / kCPR;
    uint4 hi, lo;
    query_finish<D>(a, x[i], a.qw != nullptr, wv, hi, lo);
    *reinterpret_cast<uint4*>(dst + swz(r, c, D * 2)) = hi;
    *reinterpret_cast<uint4*>(dst + PreCfg<D>::kTileBytes + swz(r, c, D * 2)) = lo;
  }
}

// Block pb of P of the prefix's part; len: the sequences' lengths in shared memory, smem: behind the
// block's head, 1024-byte aligned.
template <int D>
__device__ void prefix_role(const PagedDecodeArgs& a, const int* len, uint8_t* smem, int P, int tid) {
  using C = PreCfg<D>;
  constexpr int S = C::kStages;
  constexpr int TB = C::kTileBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* q_full = bars;                  // [2] per unit: its 128 rows are packed
  uint64_t* q_empty = q_full + 2;           // [2] the segment's last S has completed
  uint64_t* kv_full = q_empty + 2;          // [S]
  uint64_t* kv_empty = kv_full + S;         // [S] both O += P V issuers are done with the stage
  uint64_t* s_full = kv_empty + S;          // [2] per unit
  uint64_t* s_read = s_full + 2;            // [2] the unit's warpgroup holds its scores in registers
  uint64_t* p_ready = s_read + 2;           // [2][2] per unit and P buffer: twice a tile
  uint64_t* pv_done = p_ready + 4;          // [2][2] per unit and P buffer
  uint64_t* o_free = pv_done + 4;           // [2] the unit's O has been read out
  uint64_t* drain = o_free + 2;             // [3] one per issuing thread
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kNumBars);
  volatile int* abort = reinterpret_cast<volatile int*>(bars + C::kNumBars) + 1;
  const int warp = tid >> 5, lane = tid & 31, pb = (int)blockIdx.x;
  const PrefixArgs& p = a.pre;

  if (tid == 0) {
    *abort = 0;
    for (int k = 0; k < 2; k++) {
      mbar_init(q_full + k, 4);
      mbar_init(q_empty + k, 1);
    }
    for (int k = 0; k < S; k++) {
      mbar_init(kv_full + k, 1);
      mbar_init(kv_empty + k, 2);
    }
    for (int u = 0; u < 2; u++) {
      mbar_init(s_full + u, 1);
      mbar_init(s_read + u, 4);
      mbar_init(p_ready + 2 * u, 4);
      mbar_init(p_ready + 2 * u + 1, 4);
      mbar_init(pv_done + 2 * u, 1);
      mbar_init(pv_done + 2 * u + 1, 1);
      mbar_init(o_free + u, 4);
    }
    for (int k = 0; k < 3; k++) mbar_init(drain + k, 1);
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const volatile int never = 0;
  PreSeg sg;
  sg.init(p, pb, P);
  // registers: 128 x 72 + 256 x 216 of the 384 x 168 at launch
  if (warp < 4) regs_dec<72>();
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      prefetch_tmap(&a.map_pk);
      prefetch_tmap(&a.map_pv);
    }
    const int prows = min(1 << a.page_shift, kTile), per = kTile / prows;
    const uint32_t pbytes = (uint32_t)prows * C::kSpan;
    const int np = a.prefix_len >> a.page_shift;
    bool ok = true;
    int g = 0;  // K/V stages handed out so far
    while (ok && sg.next(p)) {
      const int kvh = sg.s / p.pairs;
      int win = -1, id = 0;
      for (int n = sg.n0; ok && n < sg.n1; n++, g++) {
        const int first = (n * kTile) >> a.page_shift;
        if ((first >> 5) != win) {
          win = first >> 5;
          id = a.num_pages;  // pages behind the prefix in its last tile: outside the pool, read as zeros
          if (win * 32 + lane < np) {
            id = a.prefix_table[win * 32 + lane];
            if (id < 0 || id >= a.num_pages) {
              record_page(a.status);
              id = a.num_pages;
            }
          }
        }
        const int mine = __shfl_sync(0xffffffffu, id, (first & 31) + (lane < per ? lane : 0));
        const int st = g % S, use = g / S;
        if (use > 0) ok = __all_sync(0xffffffffu, mbar_wait(kv_empty + st, (use - 1) & 1, abort));
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(kv_full + st, 2 * TB);
        __syncwarp();
        if (lane < per) {
          const int off = (n * kTile) & ((1 << a.page_shift) - 1);
          tma_load_4d(smem + C::kOffK + st * TB + lane * pbytes, &a.map_pk, kv_full + st, 0, off, kvh, mine);
          tma_load_4d(smem + C::kOffV + st * TB + lane * pbytes, &a.map_pv, kv_full + st, 0, off, kvh, mine);
        }
      }
    }
    if (!ok && lane == 0) {
      *abort = 1;
      atomicExch(a.status, kStatusTimeout);
    }
    // let every copy issued above land before the block can exit
    if (lane == 0) {
      for (int x = g - S < 0 ? 0 : g - S; x < g; x++) mbar_wait(kv_full + x % S, (x / S) & 1, &never);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ S = Q K^T issuer (both units)
    if (lane == 0) {
      constexpr uint32_t idS = idesc_fp16(128, 128, false, false);
      constexpr uint32_t kStepK = 32 >> 4;
      constexpr uint32_t tstep = (uint32_t)TB >> 4;
      const uint64_t dQ0 = smem_desc(smem_u32(smem), 16, C::kSBO, C::kSwz);
      const uint64_t dK0 = smem_desc(smem_u32(smem + C::kOffK), 16, C::kSBO, C::kSwz);
      bool ok = true;
      int g = 0, e[2] = {0, 0}, m[2] = {0, 0};  // K/V stages; segments and S issued per unit
      while (ok && sg.next(p)) {
        const int nu = sg.units(p);
        for (int n = sg.n0; ok && n < sg.n1; n++, g++) {
          const int st = g % S;
          if (!(ok = mbar_wait(kv_full + st, (g / S) & 1, abort))) break;
          for (int u = 0; u < nu; u++) {
            if (n == sg.n0 && !(ok = mbar_wait(q_full + u, e[u] & 1, abort))) break;
            // the unit's previous scores are in its warpgroup's registers
            if (m[u] > 0 && !(ok = mbar_wait(s_read + u, (m[u] - 1) & 1, abort))) break;
            tc_fence_after();
            const uint64_t dq = dQ0 + (uint64_t)(2 * u * tstep), dk = dK0 + (uint64_t)(st * tstep);
            mma_ss_chain<D / 16>(tmem + C::kColS + 128u * u, dq, kStepK, dk, kStepK, idS, 0u);
            mma_ss_chain<D / 16>(tmem + C::kColS + 128u * u, dq + (uint64_t)tstep, kStepK, dk, kStepK, idS, 1u);
            mma_commit(s_full + u);
            if (n + 1 == sg.n1) mma_commit(q_empty + u);
            m[u]++;
          }
        }
        for (int u = 0; u < nu; u++) e[u]++;
      }
      if (!ok) {
        *abort = 1;
        atomicExch(a.status, kStatusTimeout);
      }
      mma_commit(drain);
      mbar_wait(drain, 0, &never);
    }
  } else if (warp == 2 || warp == 3) {
    // ------------------------------------------------------------ O_u += P_u V issuers
    if (lane == 0) {
      const int u = warp - 2;
      constexpr uint32_t idPV = idesc_bf16(128, D, false, true);
      constexpr uint32_t kStepMN = (16 * C::kSpan) >> 4;
      constexpr uint32_t tstep = (uint32_t)TB >> 4;
      const uint64_t dV0 = smem_desc(smem_u32(smem + C::kOffV), 16, C::kSBO, C::kSwz);
      bool ok = true;
      int g = 0, e = 0;  // K/V stages, this unit's segments
      while (ok && sg.next(p)) {
        const bool act = u < sg.units(p);
        for (int n = sg.n0; ok && n < sg.n1; n++, g++) {
          const int st = g % S;
          if (act) {
            // the first quarters of P go out while the warpgroup still computes the others: quarter j in
            // buffer j & 1, the buffer's use 2 m + (j >> 1)
            const uint64_t dv = dV0 + (uint64_t)(st * tstep);
            for (int j = 0; ok && j < 4; j++) {
              if (!(ok = mbar_wait(p_ready + 2 * u + (j & 1), j >> 1, abort))) break;
              if (j == 0 && n == sg.n0 && e > 0 && !(ok = mbar_wait(o_free + u, (e - 1) & 1, abort))) break;
              tc_fence_after();
              const uint32_t pb = tmem + C::kColP + 64u * u + 32u * (j & 1);
              const uint64_t dvj = dv + (uint64_t)(2 * j * kStepMN);
              mma_ts_chain<2, false>(tmem + C::kColO + 64u * u, pb, dvj, kStepMN, idPV, n > sg.n0 || j > 0 ? 1u : 0u);
              mma_ts_chain<2, false>(tmem + C::kColO + 64u * u, pb + 16u, dvj, kStepMN, idPV, 1u);
              mma_commit(pv_done + 2 * u + (j & 1));
            }
            if (!ok) break;
            mma_commit(kv_empty + st);  // V by this PV; K by this unit's S, complete before its P existed
          } else {
            // the segment has one unit: once for each use of the stage, so not before the stage is full
            if (!(ok = mbar_wait(kv_full + st, (g / S) & 1, abort))) break;
            mbar_arrive(kv_empty + st);
          }
        }
        if (act) e++;
      }
      if (!ok) {
        *abort = 1;
        atomicExch(a.status, kStatusTimeout);
      }
      mma_commit(drain + 1 + u);
      mbar_wait(drain + 1 + u, 0, &never);
    }
  } else {
    // ------------------------------------------------------------ softmax warpgroup of unit u
    regs_inc<216>();
    const int u = (warp - 4) >> 2;  // 0: warps 4-7, 1: warps 8-11
    const int q4 = warp & 3;        // TMEM lane quarter
    const int r = q4 * 32 + lane;   // row within the tile
    const uint32_t trow = tmem + ((uint32_t)(q4 * 32) << 16);
    const uint32_t sbuf = trow + C::kColS + 128u * u;
    const uint32_t pbuf = trow + C::kColP + 64u * u;
    const uint32_t obuf = trow + C::kColO + 64u * u;
    const float sl2 = a.scale_log2;
    bool ok = true, waited = false;
    int m = 0, e = 0;  // this unit's steps and segments so far
    while (ok && sg.next(p)) {
      if (u >= sg.units(p)) continue;
      {
        if (e >= 1) ok = __all_sync(0xffffffffu, mbar_wait(q_empty + u, (e - 1) & 1, abort));
        if (!ok) break;
        pack_query_rows<D>(a, len, sg.s / p.pairs, (2 * (sg.s % p.pairs) + u) * kTile, smem + 2 * u * TB, q4 * 32, lane);
        fence_proxy_async_smem();
        warp_arrive(q_full + u);
        e++;
      }
      float r_run = 0.f, l_run = 0.f;  // running maximum (raw logit units) and sum of the row
      float m_use = 0.f;
      for (int n = sg.n0; n < sg.n1; n++, m++) {
        ok = __all_sync(0xffffffffu, mbar_wait(s_full + u, m & 1, abort));
        if (!ok) break;
        tc_fence_after();
        uint32_t sc[128];
#pragma unroll
        for (int c = 0; c < 4; c++) tmem_ld32(sbuf + c * 32, *reinterpret_cast<uint32_t(*)[32]>(sc + 32 * c));
        tmem_wait_ld();
        tc_fence_before();
        warp_arrive(s_read + u);
        const int rem = a.prefix_len - n * kTile;  // columns of the tile that are in the prefix
        if (rem < kTile) {
#pragma unroll
          for (int e = 0; e < 128; e++)
            if (e >= rem) sc[e] = 0xff800000u;
        }
        float mx8[8];
#pragma unroll
        for (int e = 0; e < 8; e++) mx8[e] = -INFINITY;
#pragma unroll
        for (int e = 0; e < 128; e += 2)
          mx8[(e >> 1) & 7] = fmax3(mx8[(e >> 1) & 7], __uint_as_float(sc[e]), __uint_as_float(sc[e + 1]));
        const float mxr = fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                                fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
        float r_use = mxr, alpha = 1.f;
        if (n > sg.n0) {
          r_use = r_run;
          const float m_old = __fmul_rn(r_run, sl2);
          const float r_new = fmaxf(r_run, mxr);
          const float m_new = __fmul_rn(r_new, sl2);
          // lazy rescale: only when some row's maximum grew by more than 2^8
          if (__any_sync(0xffffffffu, m_new > m_old + 8.0f)) {
            // the last quarter of the step before: use 2 m - 1 of the second buffer
            ok = __all_sync(0xffffffffu, mbar_wait(pv_done + 2 * u + 1, 1, abort));
            if (!ok) break;
            tc_fence_after();
            r_use = r_new;
            alpha = ex2(m_old - m_new);
            uint32_t w[32];
#pragma unroll
            for (int c = 0; c < D / 32; c++) {
              tmem_ld32(obuf + c * 32, w);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; e++) w[e] = __float_as_uint(__uint_as_float(w[e]) * alpha);
              tmem_st32(obuf + c * 32, w);
            }
            tmem_wait_st();
            tc_fence_before();
          }
        }
        r_run = r_use;
        m_use = __fmul_rn(r_use, sl2);
        uint64_t sum4[4] = {0ull, 0ull, 0ull, 0ull};
        const uint64_t sl2x2 = f2(sl2, sl2), negm = f2(-m_use, -m_use);
        const uint64_t minus = f2(-1.f, -1.f);
#pragma unroll
        for (int c = 0; c < 8; c++) {
          const int j = c >> 1, h = j & 1;  // quarter and its buffer
          uint32_t ph[8], pl[8];
#pragma unroll
          for (int e = 0; e < 8; e++) {
            const int k = 16 * c + 2 * e;
            float x0, x1, l0, l1;
            f2_split(f2_fma(f2(__uint_as_float(sc[k]), __uint_as_float(sc[k + 1])), sl2x2, negm), x0, x1);
            const uint64_t pp = f2(ex2(x0), ex2(x1));
            f2_split(pp, x0, x1);
            ph[e] = pack_bf16(x0, x1);
            f2_split(f2_fma(f2(bf_lo(ph[e]), bf_hi(ph[e])), minus, pp), l0, l1);
            pl[e] = pack_bf16(l0, l1);
            sum4[e & 3] = f2_add(sum4[e & 3], pp);
          }
          if ((c & 1) == 0) {
            if (c > 0) {  // the quarter before: its stores have had 16 keys' time
              tmem_wait_st();
              tc_fence_before();
              warp_arrive(p_ready + 2 * u + (h ^ 1));
            }
            // the buffer's use before, 2 m + (j >> 1) - 1, has been read
            if ((j > 1 || m > 0) && !__all_sync(0xffffffffu, mbar_wait(pv_done + 2 * u + h, j > 1 ? 0 : 1, abort))) {
              ok = false;
              break;
            }
            tc_fence_after();
          }
          tmem_st8(pbuf + 32 * h + 8 * (c & 1), ph);
          tmem_st8(pbuf + 32 * h + 16 + 8 * (c & 1), pl);
        }
        if (!ok) break;
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(p_ready + 2 * u + 1);
        float s0, s1, s2, s3, s4, s5, s6, s7;
        f2_split(sum4[0], s0, s1);
        f2_split(sum4[1], s2, s3);
        f2_split(sum4[2], s4, s5);
        f2_split(sum4[3], s6, s7);
        const float l = ((s0 + s1) + (s2 + s3)) + ((s4 + s5) + (s6 + s7));
        l_run = n > sg.n0 ? fmaf(l_run, alpha, l) : l;
      }
      if (!ok) break;
      // the segment's unnormalised O, maximum (log2 units) and sum
      ok = __all_sync(0xffffffffu, mbar_wait(pv_done + 2 * u + 1, 1, abort));
      if (!ok) break;
      tc_fence_after();
      if (!waited) {
        pdl_wait();  // everything before in the stream is done with the workspace
        waited = true;
        if (pb == 0 && tid == 128) *p.cut = P;
      }
      const size_t part = prefix_part(pb + sg.s, u);
      float4* dst = reinterpret_cast<float4*>(p.part_o) + prefix_quad<D>(part, r, 0);
#pragma unroll
      for (int c = 0; c < D / 32; c++) {
        uint32_t w[32];
        tmem_ld32(obuf + c * 32, w);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 8; e++)
          dst[(c * 8 + e) * 32] = make_float4(__uint_as_float(w[4 * e]), __uint_as_float(w[4 * e + 1]),
                                              __uint_as_float(w[4 * e + 2]), __uint_as_float(w[4 * e + 3]));
      }
      tc_fence_before();
      warp_arrive(o_free + u);
      p.part_ml[part * kTile + r] = make_float2(m_use, l_run);
    }
    if (!ok) {
      *abort = 1;
      atomicExch(a.status, kStatusTimeout);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    tmem_relinquish();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

}  // namespace
}  // namespace ne
