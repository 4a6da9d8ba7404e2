// Shared prefix of a batch over a paged key/value cache (sm_103a).
//
// Every sequence of the batch starts with the same pages.  Their attention is
// computed once for all: the queries of one key/value head, of every sequence and
// new token, fill 128-row tiles, and each key/value tile of the prefix is read once
// for two of them.
//
//   k_prefix_q  queries normalised, rotated and packed: [Hkv, tiles * 128, D] fp16,
//               row b * R + r (zeros behind the last)
//   k_prefix    S = Q K^T and O += P V on the tensor cores over the key tiles of the
//               prefix, laid end to end over (head, pair of row tiles) and cut into one
//               equal stretch per block; each segment leaves its unnormalised O and its
//               rows' maximum and sum
//   k_prefix_join  the segments of every row: O = sum_s 2^(m_s - m) O_s, l likewise
// The sweep over the sequences' own pages (paged.cu) takes the joined part in with its own.
//
// A sequence takes part if its first query sees the whole prefix, so no score is
// masked here but for the columns behind the prefix in its last tile; the sweep
// reads the prefix pages itself for one that does not (and leaves the parts out).
// Precision: q as one fp16, the weights as one bf16, as the forward (2^-12 and 2^-9
// relative roundings, at random over the keys).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"
#include "rope.cuh"

namespace ne {
namespace {

// ====================================================================== packed queries
template <int D>
__global__ void __launch_bounds__(128) k_prefix_q(const PagedDecodeArgs a) {
  constexpr int kCPR = D / 8;
  pdl_launch();
  const int rows = a.pre.tiles * kTile;
  const long long n = (long long)a.Hkv * rows * kCPR;
  const long long it = blockIdx.x * 128LL + threadIdx.x;
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < kPagedMaxBlocks; i += 128) a.done[i] = 0u;
  if ((it & ~31LL) >= n) return;
  const int c = (int)(it % kCPR);
  const long long row = (it < n ? it : 0) / kCPR;
  const int g = (int)(row / rows), rho = (int)(row - (long long)g * rows);
  const int b = rho / a.R, r = rho - b * a.R;
  int pos0 = 0;
  const bool in = b < a.B && it < n;
  if (in) pos0 = min(a.len[b], a.max_pages << a.page_shift) - a.Tq;
  const bool norm = a.qw != nullptr;
  uint4 wv = make_uint4(0, 0, 0, 0), hi, lo;
  if (norm) wv = load_rope_chunk<D>(a.qw, c, a.rope_half != 0);
  const QueryChunk x = query_load<D>(a, in ? b : 0, g, in ? r : a.R, c, pos0);  // row R: zeros
  query_finish<D>(a, x, norm, wv, hi, lo);
  if (it < n) reinterpret_cast<uint4*>(a.pre.q)[it] = hi;
}

// ====================================================================== the prefix's tiles
template <int D>
struct PreCfg {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr uint32_t kSpan = D * 2;
  static constexpr uint32_t kSwz = D == 64 ? kSw128 : kSw64;
  static constexpr uint32_t kSBO = 8 * kSpan;
  static constexpr int kQSlots = 4;  // two segments' worth of row tiles
  static constexpr int kStages = 4;
  static constexpr uint32_t kColO = 0, kColS = 128, kColP = 384;  // unit u: O at 64u, S at 128 + 128u, P at 384 + 64u
  static constexpr uint32_t kTmemCols = 512;
  static constexpr int kThreads = 384;
  static constexpr int kOffK = kQSlots * kTileBytes;
  static constexpr int kOffV = kOffK + kStages * kTileBytes;
  static constexpr int kOffBar = kOffV + kStages * kTileBytes;
  static constexpr int kNumBars = 2 * kQSlots + 2 * kStages + 14 + 3;
  static constexpr int kSmemBytes = kOffBar + kNumBars * 8 + 16 + 1024;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

struct PreSeg {
  int w, end;       // tiles of the block's stretch that are left
  int s, n0, n1;    // the segment: (head, pair) s, key tiles [n0, n1)
  __device__ void init(const PrefixArgs& p) {
    w = (int)((long long)blockIdx.x * p.W / p.blocks);
    end = (int)((long long)(blockIdx.x + 1) * p.W / p.blocks);
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

template <int D>
__global__ void __launch_bounds__(384, 1) k_prefix(const __grid_constant__ PagedDecodeArgs a) {
  using C = PreCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  constexpr int S = C::kStages;
  constexpr int TB = C::kTileBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* q_full = bars;                  // [4] Q slots
  uint64_t* q_empty = q_full + 4;           // [4] the slot's last S has completed
  uint64_t* kv_full = q_empty + 4;          // [S]
  uint64_t* kv_empty = kv_full + S;         // [S] both O += P V issuers are done with the stage
  uint64_t* s_full = kv_empty + S;          // [2] per unit
  uint64_t* s_read = s_full + 2;            // [2] the unit's warpgroup holds its scores in registers
  uint64_t* p_ready = s_read + 2;           // [2][2] per unit and key half
  uint64_t* pv_done = p_ready + 4;          // [2][2] per unit and key half
  uint64_t* o_free = pv_done + 4;           // [2] the unit's O has been read out
  uint64_t* drain = o_free + 2;             // [3] one per issuing thread
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kNumBars);
  volatile int* abort = reinterpret_cast<volatile int*>(bars + C::kNumBars) + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PrefixArgs& p = a.pre;

  if (tid == 0) {
    *abort = 0;
    for (int k = 0; k < C::kQSlots; k++) {
      mbar_init(q_full + k, 1);
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
  pdl_launch();
  PreSeg sg;
  sg.init(p);
  // registers: 128 x 72 + 256 x 216 of the 384 x 168 at launch
  if (warp < 4) regs_dec<72>();
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      prefetch_tmap(&a.map_q);
      prefetch_tmap(&a.map_pk);
      prefetch_tmap(&a.map_pv);
    }
    const int prows = min(1 << a.page_shift, kTile), per = kTile / prows;
    const uint32_t pbytes = (uint32_t)prows * C::kSpan;
    const int np = a.prefix_len >> a.page_shift;
    bool ok = true, waited = false;
    int g = 0, c = 0;  // K/V stages and Q slots handed out so far
    while (ok && sg.next(p)) {
      const int kvh = sg.s / p.pairs, tile0 = 2 * (sg.s % p.pairs), nu = sg.units(p);
      int win = -1, id = 0;
      bool q_sent = false;
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
        if (!q_sent) {  // the segment's row tiles, behind its first keys
          q_sent = true;
          if (!waited) {
            pdl_wait();  // the packed queries of the kernel before
            waited = true;
          }
          for (int u = 0; ok && u < nu; u++, c++) {
            const int sl = c & 3, quse = c >> 2;
            if (quse > 0) ok = __all_sync(0xffffffffu, mbar_wait(q_empty + sl, (quse - 1) & 1, abort));
            if (ok && lane == 0) {
              mbar_arrive_expect_tx(q_full + sl, TB);
              tma_load_4d(smem + sl * TB, &a.map_q, q_full + sl, 0, 0, (kvh * p.tiles + tile0 + u) * kTile, 0);
            }
            if (!ok) break;
          }
          if (!ok) g++;  // this step's keys and values are on their way
        }
        if (!ok) break;
      }
    }
    if (!ok && lane == 0) {
      *abort = 1;
      atomicCAS(a.status, 0, kStatusTimeout);
    }
    // let every copy issued above land before the block can exit
    if (lane == 0) {
      for (int x = c - 4 < 0 ? 0 : c - 4; x < c; x++) mbar_wait(q_full + (x & 3), (x >> 2) & 1, &never);
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
      int g = 0, c = 0, m[2] = {0, 0};  // K/V stages, Q slots, S issued per unit
      while (ok && sg.next(p)) {
        const int nu = sg.units(p);
        for (int n = sg.n0; ok && n < sg.n1; n++, g++) {
          const int st = g % S;
          if (!(ok = mbar_wait(kv_full + st, (g / S) & 1, abort))) break;
          for (int u = 0; u < nu; u++) {
            const int q = c + u, sl = q & 3;
            if (n == sg.n0 && !(ok = mbar_wait(q_full + sl, (q >> 2) & 1, abort))) break;
            // the unit's previous scores are in its warpgroup's registers
            if (m[u] > 0 && !(ok = mbar_wait(s_read + u, (m[u] - 1) & 1, abort))) break;
            tc_fence_after();
            mma_ss_chain<D / 16>(tmem + C::kColS + 128u * u, dQ0 + (uint64_t)(sl * tstep), kStepK,
                                 dK0 + (uint64_t)(st * tstep), kStepK, idS, 0u);
            mma_commit(s_full + u);
            if (n + 1 == sg.n1) mma_commit(q_empty + sl);
            m[u]++;
          }
        }
        c += nu;
      }
      if (!ok) {
        *abort = 1;
        atomicCAS(a.status, 0, kStatusTimeout);
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
      int g = 0, m = 0, e = 0;  // K/V stages, this unit's steps, this unit's segments
      while (ok && sg.next(p)) {
        const bool act = u < sg.units(p);
        for (int n = sg.n0; ok && n < sg.n1; n++, g++) {
          const int st = g % S;
          if (act) {
            // keys 0..63 of P go out while the warpgroup still computes keys 64..127
            if (!(ok = mbar_wait(p_ready + 2 * u, m & 1, abort))) break;
            if (n == sg.n0 && e > 0 && !(ok = mbar_wait(o_free + u, (e - 1) & 1, abort))) break;
            tc_fence_after();
            const uint64_t dv = dV0 + (uint64_t)(st * tstep);
            mma_ts_chain<4, false>(tmem + C::kColO + 64u * u, tmem + C::kColP + 64u * u, dv, kStepMN, idPV,
                                   n > sg.n0 ? 1u : 0u);
            mma_commit(pv_done + 2 * u);
            if (!(ok = mbar_wait(p_ready + 2 * u + 1, m & 1, abort))) break;
            tc_fence_after();
            mma_ts_chain<4, false>(tmem + C::kColO + 64u * u, tmem + C::kColP + 64u * u + 32u,
                                   dv + (uint64_t)(4 * kStepMN), kStepMN, idPV, 1u);
            mma_commit(pv_done + 2 * u + 1);
            mma_commit(kv_empty + st);  // V by this PV; K by this unit's S, complete before its P existed
            m++;
          } else {
            mbar_arrive(kv_empty + st);  // the segment has one unit
          }
        }
        if (act) e++;
      }
      if (!ok) {
        *abort = 1;
        atomicCAS(a.status, 0, kStatusTimeout);
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
    int m = 0;  // this unit's steps so far
    while (ok && sg.next(p)) {
      if (u >= sg.units(p)) continue;
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
            ok = __all_sync(0xffffffffu, mbar_wait(pv_done + 2 * u + 1, (m - 1) & 1, abort));
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
        if (m > 0) {  // keys 0..63 of the P buffer: read by the first half of the previous step's P V
          ok = __all_sync(0xffffffffu, mbar_wait(pv_done + 2 * u, (m - 1) & 1, abort));
          if (!ok) break;
        }
        tc_fence_after();
        uint64_t sum4[4] = {0ull, 0ull, 0ull, 0ull};
        const uint64_t sl2x2 = f2(sl2, sl2), negm = f2(-m_use, -m_use);
#pragma unroll
        for (int c = 0; c < 8; c++) {
          if (c == 4) {
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(p_ready + 2 * u);
            if (m > 0 && !__all_sync(0xffffffffu, mbar_wait(pv_done + 2 * u + 1, (m - 1) & 1, abort))) {
              ok = false;
              break;
            }
            tc_fence_after();
          }
          uint32_t pk[8];
#pragma unroll
          for (int e = 0; e < 8; e++) {
            const int k = 16 * c + 2 * e;
            float x0, x1;
            f2_split(f2_fma(f2(__uint_as_float(sc[k]), __uint_as_float(sc[k + 1])), sl2x2, negm), x0, x1);
            const float p0 = ex2(x0), p1 = ex2(x1);
            pk[e] = pack_bf16(p0, p1);
            sum4[e & 3] = f2_add(sum4[e & 3], f2(p0, p1));
          }
          tmem_st8(pbuf + c * 8, pk);
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
      ok = __all_sync(0xffffffffu, mbar_wait(pv_done + 2 * u + 1, (m - 1) & 1, abort));
      if (!ok) break;
      tc_fence_after();
      if (!waited) {
        pdl_wait();  // everything before in the stream is done with the workspace
        waited = true;
      }
      const size_t part = prefix_part(blockIdx.x + sg.s, u);
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
      atomicCAS(a.status, 0, kStatusTimeout);
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

// ====================================================================== the segments of a tile joined
// A thread takes four columns of a row and its segments in order, rescaling as the maximum grows.  32 neighbouring rows of one column quad lie side by side in a
// segment (prefix_quad); the result is row by row.
template <int D>
__global__ void __launch_bounds__(128) k_prefix_join(const __grid_constant__ PagedDecodeArgs a) {
  const PrefixArgs& p = a.pre;
  pdl_wait();
  pdl_launch();
  const int lane = threadIdx.x & 31;
  const long long w = blockIdx.x * 4LL + threadIdx.x / 32;  // (head, tile, 32 rows, quad)
  const int q = (int)(w % (D / 4)), r32 = (int)(w / (D / 4) % (kTile / 32));
  const long long gt = w / (D / 4) / (kTile / 32);
  const int g = (int)(gt / p.tiles), tile = (int)(gt - (long long)g * p.tiles);
  if (g >= a.Hkv) return;
  const int row = r32 * 32 + lane, s = g * p.pairs + (tile >> 1), u = tile & 1;
  const int lo = prefix_owner(p, s * p.ntk), hi = prefix_owner(p, s * p.ntk + p.ntk - 1);
  // eight segments' loads under way at a time
  constexpr int kAhead = 8;
  float top = -INFINITY, S = 0.f;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c0 = lo; c0 <= hi; c0 += kAhead) {
    float2 z[kAhead];
    float4 x[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; k++) {
      const size_t part = prefix_part(min(c0 + k, hi) + s, u);
      z[k] = __ldcg(p.part_ml + part * kTile + row);
      x[k] = __ldcg(reinterpret_cast<const float4*>(p.part_o) + prefix_quad<D>(part, row, q));
    }
    float t = top;
#pragma unroll
    for (int k = 0; k < kAhead; k++) t = fmaxf(t, z[k].x);
    const float r = top == -INFINITY ? 0.f : ex2(top - t);
    S *= r;
    v = make_float4(v.x * r, v.y * r, v.z * r, v.w * r);
    top = t;
#pragma unroll
    for (int k = 0; k < kAhead; k++) {
      const float f = c0 + k <= hi ? ex2(z[k].x - top) : 0.f;
      S = fmaf(f, z[k].y, S);
      v = make_float4(fmaf(f, x[k].x, v.x), fmaf(f, x[k].y, v.y), fmaf(f, x[k].z, v.z), fmaf(f, x[k].w, v.w));
    }
  }
  const size_t out = (size_t)gt * kTile + row;
  reinterpret_cast<float4*>(p.o)[out * (D / 4) + q] = v;
  if (q == 0) p.ml[out] = make_float2(top, S);
}

template <int D>
cudaError_t launch_t(const PagedDecodeArgs& a, cudaStream_t s) {
  using C = PreCfg<D>;
  static bool attr_set[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(k_prefix<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  const long long n = (long long)a.Hkv * a.pre.tiles * kTile * (D / 8);
  k_prefix_q<D><<<(unsigned)((n + 127) / 128), 128, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = launch_pdl(k_prefix<D>, a.pre.blocks, C::kThreads, (size_t)C::kSmemBytes, s, a);
  if (e != cudaSuccess) return e;
  const long long warps = (long long)a.Hkv * a.pre.tiles * (kTile / 32) * (D / 4);
  return launch_pdl(k_prefix_join<D>, (int)((warps + 3) / 4), 128, 0, s, a);
}

}  // namespace

cudaError_t launch_prefix(const PagedDecodeArgs& a, cudaStream_t s) {
  return a.D == 64 ? launch_t<64>(a, s) : launch_t<32>(a, s);
}

}  // namespace ne
