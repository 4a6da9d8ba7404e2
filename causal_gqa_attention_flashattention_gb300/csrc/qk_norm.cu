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
constexpr int kAtOnce = 2;  // rows a thread has under way

// A block works on q or on k (the first nbq blocks on q): one weight, a thread takes the same
// chunk of every row it gets, so its part of the weight stays in registers.  Few registers, and
// as many blocks as the SMs hold at once, carry these kernels: with four heads of a position per
// thread (one read of its table row for them, both weights in registers) the forward took 15.0 us
// at 16 x 512 positions, 12/4 heads, D = 64, with two heads 11.6 us, in this form 8.1 us (33.6 MB,
// 4.1 TB/s); the backward 28.3 us, in this form 14.3 us (50 MB, with the sums of dw).
template <int D>
struct Side {
  bool isq;
  const __nv_bfloat16 *x, *w;
  long long stride;
  uint32_t H, n, first, step;  // heads; row chunks; this thread's first chunk and the distance to its next
};
template <int D, typename Args>
__device__ __forceinline__ Side<D> side_of(const Args& a) {
  Side<D> s;
  s.isq = blockIdx.x < (uint32_t)a.nbq;
  s.x = s.isq ? a.q : a.k;
  s.w = s.isq ? a.qw : a.kw;
  s.stride = s.isq ? a.q_stride : a.k_stride;
  s.H = s.isq ? a.Hq : a.Hkv;
  s.n = (uint32_t)a.B * a.T * s.H * (D / 8);
  const uint32_t blk = s.isq ? blockIdx.x : blockIdx.x - a.nbq;
  s.first = blk * kThreads + threadIdx.x;
  s.step = (s.isq ? a.nbq : gridDim.x - a.nbq) * kThreads;
  return s;
}

// The D / 8 threads of a row are neighbouring lanes and add up their squares by shuffles: whole
// warps run together, lanes past the end take part in the shuffles only.
template <int D>
__global__ void __launch_bounds__(kThreads) k_qk_norm(const QkNormArgs a) {
  constexpr int kCPR = D / 8;
  const Side<D> s = side_of<D>(a);
  const FastDiv div_h = s.isq ? a.div_hq : a.div_hkv;
  uint4* out = reinterpret_cast<uint4*>(s.isq ? a.qr : a.kr);
  const int c = (int)(threadIdx.x % kCPR);
  const bool half = a.rope_half != 0;
  float w[8];
  unpack8(load_rope_chunk<D>(s.w, c, half), w);
  for (uint32_t it = s.first; (it & ~31u) < s.n; it += kAtOnce * s.step) {
    uint4 v[kAtOnce];
    float4 c0[kAtOnce], c1[kAtOnce];
#pragma unroll
    for (int e = 0; e < kAtOnce; e++) {
      const uint32_t i = it + e * s.step, row = (i < s.n ? i : 0u) / kCPR;
      const uint32_t bt = fdiv(row, div_h), h = row - bt * s.H, t = bt - fdiv(bt, a.div_t) * a.T;
      v[e] = load_rope_chunk<D>(s.x + (size_t)bt * s.stride + h * D, c, half);
      rope_coeffs<D>(a.rope, (int)t, c, c0[e], c1[e]);
    }
#pragma unroll
    for (int e = 0; e < kAtOnce; e++) {
      const uint32_t i = it + e * s.step;
      float x[8], ss = 0.f;
      unpack8(v[e], x);
#pragma unroll
      for (int j = 0; j < 8; j++) ss = fmaf(x[j], x[j], ss);
      const float r = rsqrtf(fmaf(row_sum<kCPR>(ss), 1.f / D, a.eps));
      const float cs[4] = {c0[e].x, c0[e].z, c1[e].x, c1[e].z}, sn[4] = {c0[e].y, c0[e].w, c1[e].y, c1[e].w};
      uint32_t o[4];
#pragma unroll
      for (int p = 0; p < 4; p++) {
        const float x0 = x[2 * p] * r * w[2 * p], x1 = x[2 * p + 1] * r * w[2 * p + 1];
        o[p] = pack_f16(fmaf(x0, cs[p], -x1 * sn[p]), fmaf(x0, sn[p], x1 * cs[p]));
      }
      if (i < s.n) out[i] = make_uint4(o[0], o[1], o[2], o[3]);
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

// Sum of n <= 32 partial rows of D values, in a fixed order; true for the first D / 4 threads,
// which then have a quad each in t.
template <int D>
__device__ __forceinline__ bool add_partials(const float* part, unsigned n, float4& t) {
  constexpr unsigned kQuads = D / 4, kOver = kThreads / kQuads, kEach = (32 + kOver - 1) / kOver;
  __shared__ float4 red4[kOver][kQuads];
  const unsigned q = threadIdx.x % kQuads, o = threadIdx.x / kQuads;
  float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (unsigned k = 0; k < kEach; k++)
    if (o + k * kOver < n) {
      const float4 x = __ldcg(reinterpret_cast<const float4*>(part) + (size_t)(o + k * kOver) * kQuads + q);
      u = make_float4(u.x + x.x, u.y + x.y, u.z + x.z, u.w + x.w);
    }
  red4[o][q] = u;
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
static_assert(kQkNormGroup <= 32 && kQkNormMaxBlocks <= 32 * kQkNormGroup, "partials of a sum");

// Backward.  dw is summed in fp32: over the rows of a thread, over the threads of
// a block that share a chunk (in a fixed order), one partial per block in the
// workspace, added in two steps by the blocks that end last, always in the
// same order: the result does not depend on which ones, and is bitwise reproducible.
template <int D, bool F32>
__global__ void __launch_bounds__(kThreads) k_qk_norm_bwd(const QkNormBwdArgs a) {
  constexpr int kCPR = D / 8;
  const Side<D> s = side_of<D>(a);
  const FastDiv div_h = s.isq ? a.div_hq : a.div_hkv;
  const void* gp = s.isq ? a.gq : a.gk;
  void* dp = s.isq ? a.dq : a.dk;
  const long long d_stride = s.isq ? a.dq_stride : a.dk_stride;
  const int c = (int)(threadIdx.x % kCPR);
  float w[8], dw[8];
  unpack8(__ldg(reinterpret_cast<const uint4*>(s.w) + c), w);
#pragma unroll
  for (int j = 0; j < 8; j++) dw[j] = 0.f;
  for (uint32_t it = s.first; (it & ~31u) < s.n; it += kAtOnce * s.step) {
    uint4 v[kAtOnce], g0[kAtOnce], g1[kAtOnce];
    size_t to[kAtOnce];
#pragma unroll
    for (int e = 0; e < kAtOnce; e++) {
      const uint32_t i = it + e * s.step, row = (i < s.n ? i : 0u) / kCPR;
      const uint32_t bt = fdiv(row, div_h), h = row - bt * s.H;
      v[e] = __ldg(reinterpret_cast<const uint4*>(s.x + (size_t)bt * s.stride + h * D) + c);
      // plain loads: dq may be the same buffer as gq
      g0[e] = g1[e] = make_uint4(0, 0, 0, 0);
      if (i < s.n) {
        const uint4* p = static_cast<const uint4*>(gp) + (size_t)i * (F32 ? 2 : 1);
        g0[e] = p[0];
        if (F32) g1[e] = p[1];
      }
      to[e] = (size_t)bt * d_stride + h * D + 8 * c;
    }
#pragma unroll
    for (int e = 0; e < kAtOnce; e++) {
      float x[8], g[8];
      unpack8(v[e], x);
      if (F32) {
        const uint32_t u[8] = {g0[e].x, g0[e].y, g0[e].z, g0[e].w, g1[e].x, g1[e].y, g1[e].z, g1[e].w};
#pragma unroll
        for (int j = 0; j < 8; j++) g[j] = __uint_as_float(u[j]);
      } else {
        unpack8(g0[e], g);
      }
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int j = 0; j < 8; j++) {
        s1 = fmaf(x[j], x[j], s1);
        s2 = fmaf(g[j] * w[j], x[j], s2);
      }
      s1 = row_sum<kCPR>(s1);
      s2 = row_sum<kCPR>(s2);
      if (it + e * s.step >= s.n) continue;
      const float r = rsqrtf(fmaf(s1, 1.f / D, a.eps));
      const float m = s2 * r * (1.f / D);  // mean(w g xh)
      float d[8];
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const float xh = x[j] * r;
        d[j] = r * fmaf(-xh, m, g[j] * w[j]);
        dw[j] = fmaf(g[j], xh, dw[j]);
      }
      if (F32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(dp) + to[e]);
        p[0] = make_float4(d[0], d[1], d[2], d[3]);
        p[1] = make_float4(d[4], d[5], d[6], d[7]);
      } else {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(dp) + to[e]) =
            make_uint4(pack_bf16(d[0], d[1]), pack_bf16(d[2], d[3]), pack_bf16(d[4], d[5]), pack_bf16(d[6], d[7]));
      }
    }
  }
  // the block's dw: lanes of a warp with the same chunk, then the warps
  __shared__ float red[kThreads / 32][D];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
  for (int j = 0; j < 8; j++)
#pragma unroll
    for (int m = kCPR; m < 32; m <<= 1) dw[j] += __shfl_xor_sync(0xffffffffu, dw[j], m);
  if (lane < kCPR) {
#pragma unroll
    for (int j = 0; j < 8; j++) red[warp][8 * c + j] = dw[j];
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < kThreads / 32; k++) t += red[k][threadIdx.x];
    pdl_wait();  // where the kernel before clears the workspace's counters
    a.part[(size_t)blockIdx.x * D + threadIdx.x] = t;
  }
  // the last of kQkNormGroup neighbouring blocks of a side adds their partials in order, the last of
  // those blocks the groups' sums
  const unsigned first = s.isq ? 0 : a.nbq, count = s.isq ? a.nbq : gridDim.x - a.nbq;
  const unsigned grp = (blockIdx.x - first) / kQkNormGroup, groups = (count + kQkNormGroup - 1) / kQkNormGroup;
  const unsigned b0 = grp * kQkNormGroup, nb = min((unsigned)kQkNormGroup, count - b0);
  const unsigned g0 = s.isq ? 0 : (a.nbq + kQkNormGroup - 1) / kQkNormGroup;  // the side's first group
  float4 t;
  if (!last_to_count(a.done + 2 + g0 + grp, nb)) return;
  float* sums = a.part + (size_t)(gridDim.x + g0) * D;
  if (add_partials<D>(a.part + (size_t)(first + b0) * D, nb, t))
    reinterpret_cast<float4*>(sums + (size_t)grp * D)[threadIdx.x] = t;
  if (!last_to_count(a.done + (s.isq ? 0 : 1), groups)) return;
  if (add_partials<D>(sums, groups, t)) reinterpret_cast<float4*>(s.isq ? a.dqw : a.dkw)[threadIdx.x] = t;
}

// The counters of a caller's workspace.
__global__ void k_qk_norm_clear(unsigned* done) {
  pdl_launch();
  if (threadIdx.x < 2 + kQkNormMaxGroups) done[threadIdx.x] = 0u;
}
static_assert(2 + kQkNormMaxGroups <= 64, "threads of the clear");

}  // namespace

// Blocks of q and of both: as many as the rows need or the SMs hold, in proportion to the heads.
int qk_norm_blocks(int B, int T, int Hq, int Hkv, int D, int nsm, bool bwd, int* nbq) {
  const auto need = [&](int H) {
    const long long chunks = (long long)B * T * H * (D / 8);
    return (int)((chunks + kThreads * kAtOnce - 1) / (kThreads * kAtOnce));
  };
  const int nq = need(Hq), nk = need(Hkv);
  int most = (nsm < kQkNormMaxSms ? nsm : kQkNormMaxSms) * (bwd ? kQkNormBlocksPerSm : kQkNormFwdBlocksPerSm);
  if (nq + nk <= most) {
    *nbq = nq;
    return nq + nk;
  }
  *nbq = (int)((long long)most * Hq / (Hq + Hkv));
  return most;
}

cudaError_t launch_qk_norm(const QkNormArgs& a, int D, int blocks, cudaStream_t s) {
  if (D == 64)
    k_qk_norm<64><<<blocks, kThreads, 0, s>>>(a);
  else
    k_qk_norm<32><<<blocks, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_qk_norm_bwd(const QkNormBwdArgs& a, int D, bool f32, int blocks, bool clear, cudaStream_t s) {
  const auto k = D == 64 ? (f32 ? k_qk_norm_bwd<64, true> : k_qk_norm_bwd<64, false>)
                         : (f32 ? k_qk_norm_bwd<32, true> : k_qk_norm_bwd<32, false>);
  if (!clear) {
    k<<<blocks, kThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  k_qk_norm_clear<<<1, 64, 0, s>>>(a.done);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_pdl(k, blocks, kThreads, 0, s, a);
}

}  // namespace ne
