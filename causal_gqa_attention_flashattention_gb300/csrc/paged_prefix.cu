// Attention of the newest tokens over a paged key/value cache for a batch with a shared prefix
// (sm_103a): the sweep with some of its blocks on the prefix (paged_prefix.cuh), then
// the join of the prefix's parts with the sequences' own.
#include "paged_sweep.cuh"

namespace ne {
namespace {

// A thread takes four columns of a row and its segments in order, rescaling as the maximum grows,
// then the sequence's own part.  32 neighbouring rows of one column quad lie side by side in a
// segment (prefix_quad), so that a warp's loads are whole sectors.
template <int D>
__global__ void __launch_bounds__(128) k_prefix_join(const __grid_constant__ PagedDecodeArgs a) {
  const PrefixArgs& p = a.pre;
  const int lane = threadIdx.x & 31, tile = blockIdx.y, g = blockIdx.z;
  const int w = blockIdx.x * 4 + threadIdx.x / 32, q = w % (D / 4), r32 = w / (D / 4);
  const int row = r32 * 32 + lane, s = g * p.pairs + (tile >> 1), u = tile & 1;
  const int rho = tile * kTile + row, b = (int)fdiv((uint32_t)rho, a.div_r), r = rho - b * a.R;
  if (b >= a.B) return;
  const int len = max(0, min(a.len[b], a.max_pages << a.page_shift));
  pdl_wait();
  const int blocks = __ldcg(p.cut);
  const size_t own = ((size_t)g * p.tiles + tile) * kTile + row;
  const float2 zo = __ldcg(p.ml + own);
  const float4 xo = __ldcg(reinterpret_cast<const float4*>(p.o + own * D) + q);
  if (sweep_base(a, len) == 0) return;  // the sweep has written it
  const PrefixCut cut(p.ntk, a.Hkv * p.pairs, max(1, min(blocks, min(kPagedMaxBlocks, p.W))));
  const int lo = cut.first(s), hi = cut.last(s);
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
  const float t = fmaxf(top, zo.x), f = ex2(top - t), fo = zo.y == 0.f ? 0.f : ex2(zo.x - t);
  write_row<D>(a, b, g, r, q,
               make_float4(fmaf(fo, xo.x, f * v.x), fmaf(fo, xo.y, f * v.y), fmaf(fo, xo.z, f * v.z), fmaf(fo, xo.w, f * v.w)),
               t, fmaf(fo, zo.y, f * S));
}

template <int D>
cudaError_t launch_join(const PagedDecodeArgs& a, cudaStream_t s) {
  return launch_pdl(k_prefix_join<D>, dim3(kTile / 32 * (D / 4) / 4, a.pre.tiles, a.Hkv), 128, 0, s, a);
}

}  // namespace

cudaError_t launch_decode_prefix(const PagedDecodeArgs& a, int mt, int nsm, cudaStream_t s) {
  const cudaError_t e = launch_sweep<true>(a, mt, nsm, s);
  if (e != cudaSuccess) return e;
  return a.D == 64 ? launch_join<64>(a, s) : launch_join<32>(a, s);
}

}  // namespace ne
