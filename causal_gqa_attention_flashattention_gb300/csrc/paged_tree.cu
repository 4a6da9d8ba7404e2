// Attention of a tree of drafted tokens over a paged key/value cache (sm_103a).
//
// Sequence b has len[b] positions in the cache, the last nodes[b] of them a tree: token t hangs on token
// parents[t] < t, or on the context (-1).  With ctx = len - nodes and depth the number of ancestors,
//   q^_t = R_(ctx + depth(t)) q_t,   s_tj = q^_t . k^_j / sqrt(D)
// for j < ctx and for the positions ctx + u of t's ancestors u and of t itself; o and lse as ever.
#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"
#include "rope.cuh"

namespace ne {
namespace {

// Sequence b: its positions and tokens, both 0 for an idle slot of the batch (or one that cannot be).
struct TreeShape {
  int len, nodes;
};
__device__ __forceinline__ TreeShape tree_shape(const PagedTreeArgs& a, int b, bool record) {
  TreeShape x = {a.len[b], a.nodes ? a.nodes[b] : a.Tq};
  if (x.len <= 0) return {0, 0};
  if (x.nodes < 0 || x.nodes > a.Tq) {
    if (record) record_tree(a.status);
    return {0, 0};
  }
  if (x.len > a.max_pages << a.page_shift) {
    if (record) record_page(a.status);
    return {0, 0};
  }
  if (x.len < x.nodes) return {0, 0};
  return x;
}

// A warp to a query row (sequence, token, head), its lanes on the positions in turn.
template <int D>
__global__ void __launch_bounds__(128) k_tree_rows(const PagedTreeArgs a) {
  __shared__ float sq[4][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = blockIdx.x * 4LL + warp;
  if (row >= (long long)a.B * a.Tq * a.Hq) return;
  const int h = (int)(row % a.Hq), t = (int)(row / a.Hq % a.Tq), b = (int)(row / a.Hq / a.Tq), g = h / a.G;
  const TreeShape x = tree_shape(a, b, lane == 0);
  const int len = x.len, ctx = x.len - x.nodes;
  const bool live = t < x.nodes;
  unsigned long long mask = 0;
  int depth = -1;
  if (live) {
    for (int x = t; x >= 0;) {
      mask |= 1ull << x;
      depth++;
      int p = a.parents[b * a.parent_stride + x];
      if (p < -1 || p >= x) {
        record_tree(a.status);
        p = -1;
      }
      x = p;
    }
    // the rotated query
    const __nv_bfloat16* q = a.q + (size_t)(b * a.Tq + t) * a.q_stride + (size_t)h * D;
    for (int i = lane; i < D / 2; i += 32) {
      const int i0 = a.rope_half ? i : 2 * i, i1 = a.rope_half ? i + D / 2 : 2 * i + 1;
      float x0 = __bfloat162float(q[i0]), x1 = __bfloat162float(q[i1]);
      if (a.qw) {
        float ss = 0.f;
        for (int d = 0; d < D; d++) ss = fmaf(__bfloat162float(q[d]), __bfloat162float(q[d]), ss);
        const float r = rsqrtf(fmaf(ss, 1.f / D, a.eps));
        x0 *= r * __bfloat162float(a.qw[i0]);
        x1 *= r * __bfloat162float(a.qw[i1]);
      }
      const float2 cs = a.rope[(size_t)(ctx + depth) * (D / 2) + i];
      sq[warp][2 * i] = x0 * cs.x - x1 * cs.y;
      sq[warp][2 * i + 1] = x0 * cs.y + x1 * cs.x;
    }
  }
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[D];
#pragma unroll
  for (int d = 0; d < D; d++) o[d] = 0.f;
  for (int j = lane; j < (live ? len : 0); j += 32) {
    if (j >= ctx && !((mask >> (j - ctx)) & 1)) continue;
    const int page = a.table[(size_t)b * a.max_pages + (j >> a.page_shift)];
    const bool there = page >= 0 && page < a.num_pages;
    if (!there) record_page(a.status);
    const size_t at = (size_t)(there ? page : 0) * a.page_stride + (((size_t)g << a.page_shift) + (j & ((1 << a.page_shift) - 1))) * D;
    float s = 0.f;
    if (there) {
#pragma unroll
      for (int d = 0; d < D; d++) s = fmaf(sq[warp][d], __half2float(a.kp[at + d]), s);
    }
    s *= a.scale_log2;
    const float top = fmaxf(m, s), f = m == -INFINITY ? 0.f : ex2(m - top), p = ex2(s - top);
    m = top;
    l = fmaf(l, f, p);
#pragma unroll
    for (int d = 0; d < D; d++) o[d] = fmaf(o[d], f, there ? p * __bfloat162float(a.vp[at + d]) : 0.f);
  }
  float top = m;
  for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
  const float f = m == -INFINITY && l == 0.f ? 0.f : ex2(m - top);
  l *= f;
  for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const size_t to = (size_t)row * D;
#pragma unroll
  for (int d = 0; d < D; d++) {
    float v = o[d] * f;
    for (int x = 16; x; x >>= 1) v += __shfl_xor_sync(0xffffffffu, v, x);
    if (lane == (d & 31)) {
      if (a.o_fp32) static_cast<float*>(a.o)[to + d] = v * inv;
      else static_cast<__nv_bfloat16*>(a.o)[to + d] = __float2bfloat16(v * inv);
    }
  }
  if (lane == 0 && a.lse) a.lse[((size_t)b * a.Hq + h) * a.Tq + t] = l == 0.f ? -INFINITY : (top + log2f(l)) * kPagedLn2;
}

}  // namespace

cudaError_t launch_decode_tree(const PagedTreeArgs& a, cudaStream_t s) {
  const long long rows = (long long)a.B * a.Tq * a.Hq;
  const unsigned grid = (unsigned)((rows + 3) / 4);
  if (a.D == 64)
    k_tree_rows<64><<<grid, 128, 0, s>>>(a);
  else
    k_tree_rows<32><<<grid, 128, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace ne
