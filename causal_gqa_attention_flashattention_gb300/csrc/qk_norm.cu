// RMS norm of each query and key head with the rotary embedding in the same
// pass, and its backward (sm_103a).
//
// Row x (one head of one position, D values), weight w [D] shared by the heads:
//   r = 1 / sqrt(mean_d x_d^2 + eps),  xh = x r,  n = w o xh,  y = R_t n
// The forward writes y as fp16 at the start of the attention's workspace, so
// ne_attn_fwd_ex and ne_attn_bwd (NE_ATTN_QK_ROTATED) take it without another
// pass over q and k.  ne_attn_bwd turns its gradients back by R_t^T and returns
// them with respect to n; with g = dL/dn the norm's own backward is
//   dx = r (w o g - xh mean_d(w o g o xh)),   dw = sum over rows of g o xh
//
// Both passes are a handful of operations per value: bound by the bytes they
// stream (HBM, or L2 when a step's tensors fit there).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace ne {
namespace {

// The eight values of chunk c of a bf16 row as fp32, pairs of the rotation side
// by side (as load_rope_chunk orders them).
__device__ __forceinline__ void unpack8(const uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int p = 0; p < 4; p++) {
    x[2 * p] = bf_lo(w[p]);
    x[2 * p + 1] = bf_hi(w[p]);
  }
}

// Sum over the kLanes neighbouring lanes that hold one row.
template <int kLanes>
__device__ __forceinline__ float row_sum(float s) {
#pragma unroll
  for (int m = 1; m < kLanes; m <<= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
  return s;
}

constexpr int kThreads = 256;
constexpr int kHeads = 4;  // heads of one position per thread: one read of its table row serves them

// A thread takes chunk c of up to kHeads heads of one position; the D / 8
// threads of a row are neighbouring lanes and add up their squares by shuffles.
// The chunk index is the same for every item of a thread (the grid's stride is a
// multiple of D / 8), so its weights stay in registers.
template <int D>
__global__ void __launch_bounds__(kThreads) k_qk_norm(const QkNormArgs a) {
  constexpr int kCPR = D / 8;
  const uint32_t H = a.Hq + a.Hkv;
  const uint32_t n = (uint32_t)a.B * a.T * a.div_hg.d * kCPR;
  const int c = (int)(threadIdx.x % kCPR);
  const bool half = a.rope_half != 0;
  float wq[8], wk[8];
  unpack8(load_rope_chunk<D>(a.qw, c, half), wq);
  unpack8(load_rope_chunk<D>(a.kw, c, half), wk);
  // whole warps run together: lanes past the end take part in the shuffles only
  for (uint32_t it = blockIdx.x * kThreads + threadIdx.x; (it & ~31u) < n; it += gridDim.x * kThreads) {
    const bool on = it < n;
    const uint32_t row = (on ? it : 0u) / kCPR;
    const uint32_t bt = fdiv(row, a.div_hg);
    const uint32_t h0 = (row - bt * a.div_hg.d) * kHeads;
    const uint32_t t = bt - fdiv(bt, a.div_t) * a.T;
    float x[kHeads][8], ss[kHeads];
#pragma unroll
    for (int e = 0; e < kHeads; e++) {
      const uint32_t h = h0 + e;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (on && h < H)
        v = load_rope_chunk<D>(h < (uint32_t)a.Hq ? a.q + (size_t)bt * a.q_stride + h * D
                                                  : a.k + (size_t)bt * a.k_stride + (h - a.Hq) * D,
                               c, half);
      unpack8(v, x[e]);
    }
    float4 c0, c1;
    rope_coeffs<D>(a.rope, (int)t, c, c0, c1);
#pragma unroll
    for (int e = 0; e < kHeads; e++) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; i++) s = fmaf(x[e][i], x[e][i], s);
      ss[e] = row_sum<kCPR>(s);
    }
    const float cs[4] = {c0.x, c0.z, c1.x, c1.z}, sn[4] = {c0.y, c0.w, c1.y, c1.w};
#pragma unroll
    for (int e = 0; e < kHeads; e++) {
      const uint32_t h = h0 + e;
      if (!on || h >= H) continue;
      const bool isq = h < (uint32_t)a.Hq;
      const float r = rsqrtf(fmaf(ss[e], 1.f / D, a.eps));
      uint32_t o[4];
#pragma unroll
      for (int p = 0; p < 4; p++) {
        const float x0 = x[e][2 * p] * r * (isq ? wq[2 * p] : wk[2 * p]);
        const float x1 = x[e][2 * p + 1] * r * (isq ? wq[2 * p + 1] : wk[2 * p + 1]);
        o[p] = pack_f16(fmaf(x0, cs[p], -x1 * sn[p]), fmaf(x0, sn[p], x1 * cs[p]));
      }
      uint4* dst = isq ? reinterpret_cast<uint4*>(a.qr) + ((size_t)bt * a.Hq + h) * kCPR
                       : reinterpret_cast<uint4*>(a.kr) + ((size_t)bt * a.Hkv + (h - a.Hq)) * kCPR;
      dst[c] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// Whether this block is the last of n to count itself (the counter goes back to 0); what the
// block wrote before is visible to the last one after.
__device__ __forceinline__ bool last_to_count(unsigned* done, unsigned n) {
  __shared__ bool last;
  __syncthreads();
  if (threadIdx.x == 0) {
    unsigned old;
    asm volatile("atom.inc.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(old) : "l"(done), "r"(n - 1) : "memory");
    last = old == n - 1;
  }
  __syncthreads();
  return last;
}

// Sum of n partial rows of 2 D values, n at most 4 kOver, in a fixed order; true for the first
// 2 D / 4 threads, which then have a quad each in t.
template <int D>
__device__ __forceinline__ bool add_partials(const float* part, unsigned n, float4& t) {
  constexpr unsigned kQuads = 2 * D / 4, kOver = kThreads / kQuads;
  __shared__ float4 red4[kOver][kQuads];
  const unsigned q = threadIdx.x % kQuads, o = threadIdx.x / kQuads;
  float4 u[4];
#pragma unroll
  for (unsigned k = 0; k < 4; k++)
    u[k] = o + k * kOver < n ? __ldcg(reinterpret_cast<const float4*>(part) + (size_t)(o + k * kOver) * kQuads + q)
                             : make_float4(0.f, 0.f, 0.f, 0.f);
  red4[o][q] = make_float4((u[0].x + u[1].x) + (u[2].x + u[3].x), (u[0].y + u[1].y) + (u[2].y + u[3].y),
                           (u[0].z + u[1].z) + (u[2].z + u[3].z), (u[0].w + u[1].w) + (u[2].w + u[3].w));
  __syncthreads();
  if (threadIdx.x >= kQuads) return false;
  t = red4[0][q];
#pragma unroll
  for (unsigned k = 1; k < kOver; k++) {
    const float4 x = red4[k][q];
    t = make_float4(t.x + x.x, t.y + x.y, t.z + x.z, t.w + x.w);
  }
  return true;
}
static_assert(kQkNormGroup <= 32 && kQkNormMaxSms * kQkNormBlocksPerSm <= 32 * kQkNormGroup, "partials of a sum");

// Backward.  dw is summed in fp32: over the rows of a thread, over the threads of
// a block that share a chunk (in a fixed order), one partial per block and weight
// in the workspace, added in two steps by the blocks that end last, always in the
// same order: the result does not depend on which ones, and is bitwise reproducible.
template <int D, bool F32>
__global__ void __launch_bounds__(kThreads) k_qk_norm_bwd(const QkNormBwdArgs a) {
  constexpr int kCPR = D / 8;
  constexpr int kPer = 2;  // heads per thread
  const uint32_t H = a.Hq + a.Hkv;
  const uint32_t n = (uint32_t)a.B * a.T * a.div_hg.d * kCPR;
  const int c = (int)(threadIdx.x % kCPR);
  float wq[8], wk[8], dwq[8], dwk[8];
  unpack8(__ldg(reinterpret_cast<const uint4*>(a.qw) + c), wq);
  unpack8(__ldg(reinterpret_cast<const uint4*>(a.kw) + c), wk);
#pragma unroll
  for (int i = 0; i < 8; i++) dwq[i] = dwk[i] = 0.f;
  for (uint32_t it = blockIdx.x * kThreads + threadIdx.x; (it & ~31u) < n; it += gridDim.x * kThreads) {
    const bool on = it < n;
    const uint32_t row = (on ? it : 0u) / kCPR;
    const uint32_t bt = fdiv(row, a.div_hg);
    const uint32_t h0 = (row - bt * a.div_hg.d) * kPer;
    float x[kPer][8], g[kPer][8];
#pragma unroll
    for (int e = 0; e < kPer; e++) {
      const uint32_t h = h0 + e;
      const bool isq = h < (uint32_t)a.Hq;
      uint4 v = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 8; i++) g[e][i] = 0.f;
      if (on && h < H) {
        v = __ldg(reinterpret_cast<const uint4*>(isq ? a.q + (size_t)bt * a.q_stride + h * D
                                                     : a.k + (size_t)bt * a.k_stride + (h - a.Hq) * D) + c);
        const size_t gi = isq ? ((size_t)bt * a.Hq + h) * D + 8 * c : ((size_t)bt * a.Hkv + (h - a.Hq)) * D + 8 * c;
        const void* gp = isq ? a.gq : a.gk;
        if (F32) {  // plain loads: dq may be the same buffer as gq
          const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(gp) + gi);
          const float4 u = p[0], w = p[1];
          g[e][0] = u.x, g[e][1] = u.y, g[e][2] = u.z, g[e][3] = u.w;
          g[e][4] = w.x, g[e][5] = w.y, g[e][6] = w.z, g[e][7] = w.w;
        } else {
          unpack8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(gp) + gi), g[e]);
        }
      }
      unpack8(v, x[e]);
    }
#pragma unroll
    for (int e = 0; e < kPer; e++) {
      const uint32_t h = h0 + e;
      const bool isq = h < (uint32_t)a.Hq;
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int i = 0; i < 8; i++) {
        s1 = fmaf(x[e][i], x[e][i], s1);
        s2 = fmaf(g[e][i] * (isq ? wq[i] : wk[i]), x[e][i], s2);
      }
      s1 = row_sum<kCPR>(s1);
      s2 = row_sum<kCPR>(s2);
      if (!on || h >= H) continue;
      const float r = rsqrtf(fmaf(s1, 1.f / D, a.eps));
      const float m = s2 * r * (1.f / D);  // mean(w g xh)
      float d[8];
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const float xh = x[e][i] * r;
        d[i] = r * fmaf(-xh, m, g[e][i] * (isq ? wq[i] : wk[i]));
        if (isq)
          dwq[i] = fmaf(g[e][i], xh, dwq[i]);
        else
          dwk[i] = fmaf(g[e][i], xh, dwk[i]);
      }
      const size_t di = isq ? (size_t)bt * a.dq_stride + h * D + 8 * c : (size_t)bt * a.dk_stride + (h - a.Hq) * D + 8 * c;
      void* dp = isq ? a.dq : a.dk;
      if (F32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(dp) + di);
        p[0] = make_float4(d[0], d[1], d[2], d[3]);
        p[1] = make_float4(d[4], d[5], d[6], d[7]);
      } else {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(dp) + di) =
            make_uint4(pack_bf16(d[0], d[1]), pack_bf16(d[2], d[3]), pack_bf16(d[4], d[5]), pack_bf16(d[6], d[7]));
      }
    }
  }
  // the block's dw: lanes of a warp with the same chunk, then the warps
  __shared__ float red[kThreads / 32][2 * D];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
  for (int i = 0; i < 8; i++)
#pragma unroll
    for (int m = kCPR; m < 32; m <<= 1) {
      dwq[i] += __shfl_xor_sync(0xffffffffu, dwq[i], m);
      dwk[i] += __shfl_xor_sync(0xffffffffu, dwk[i], m);
    }
  if (lane < kCPR) {
#pragma unroll
    for (int i = 0; i < 8; i++) {
      red[warp][8 * c + i] = dwq[i];
      red[warp][D + 8 * c + i] = dwk[i];
    }
  }
  __syncthreads();
  if (threadIdx.x < 2 * D) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; w++) s += red[w][threadIdx.x];
    a.part[(size_t)blockIdx.x * 2 * D + threadIdx.x] = s;
  }
  // the last of kQkNormGroup neighbouring blocks adds their partials in order, the last of those
  // blocks the groups' sums
  const unsigned grp = blockIdx.x / kQkNormGroup, groups = (gridDim.x + kQkNormGroup - 1) / kQkNormGroup;
  const unsigned b0 = grp * kQkNormGroup, nb = min((unsigned)kQkNormGroup, gridDim.x - b0);
  float4 t;
  if (!last_to_count(a.done + 1 + grp, nb)) return;
  const bool mine = add_partials<D>(a.part + (size_t)b0 * 2 * D, nb, t);
  float4* sums = reinterpret_cast<float4*>(a.part + (size_t)gridDim.x * 2 * D);
  if (mine) sums[(size_t)grp * (2 * D / 4) + threadIdx.x] = t;
  if (!last_to_count(a.done, groups)) return;
  if (add_partials<D>(reinterpret_cast<const float*>(sums), groups, t))
    *reinterpret_cast<float4*>((threadIdx.x < D / 4 ? a.dqw : a.dkw - D) + 4 * threadIdx.x) = t;
}

int blocks_for(long long threads, int most) {
  const long long b = (threads + kThreads - 1) / kThreads;
  return (int)(b < most ? b : most);
}

}  // namespace

int qk_norm_heads_per_item(bool bwd) { return bwd ? 2 : kHeads; }

cudaError_t launch_qk_norm(const QkNormArgs& a, int D, int nsm, cudaStream_t s) {
  const int grid = blocks_for((long long)a.B * a.T * a.div_hg.d * (D / 8), nsm * 8);
  if (D == 64)
    k_qk_norm<64><<<grid, kThreads, 0, s>>>(a);
  else
    k_qk_norm<32><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

int qk_norm_bwd_blocks(int B, int T, int hg, int D, int nsm) {
  return blocks_for((long long)B * T * hg * (D / 8), (nsm < kQkNormMaxSms ? nsm : kQkNormMaxSms) * kQkNormBlocksPerSm);
}

cudaError_t launch_qk_norm_bwd(const QkNormBwdArgs& a, int D, bool f32, int blocks, cudaStream_t s) {
  if (D == 64) {
    if (f32)
      k_qk_norm_bwd<64, true><<<blocks, kThreads, 0, s>>>(a);
    else
      k_qk_norm_bwd<64, false><<<blocks, kThreads, 0, s>>>(a);
  } else {
    if (f32)
      k_qk_norm_bwd<32, true><<<blocks, kThreads, 0, s>>>(a);
    else
      k_qk_norm_bwd<32, false><<<blocks, kThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace ne
