// Shared by the paged cache's kernels: the status of a bad page, and queries on the
// way to the tensor cores.
#pragma once
#include "internal.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace ne {

__device__ __forceinline__ void record_page(int* status) { atomicCAS(status, 0, kStatusPage); }

// Rotated (and normalised) query row chunk as fp16 high and low parts.
template <int D>
__device__ __forceinline__ void query_chunk(const PagedDecodeArgs& a, int b, int g, int r, int c, int pos0, uint4& hi,
                                            uint4& lo) {
  constexpr int kCPR = D / 8;
  const bool on = r < a.R;
  const int t = on ? r / a.G : 0, gg = r - t * a.G;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (on) v = load_rope_chunk<D>(a.q + (size_t)(b * a.Tq + t) * a.q_stride + (g * a.G + gg) * D, c, a.rope_half != 0);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float x[8];
#pragma unroll
  for (int p = 0; p < 4; p++) {
    x[2 * p] = bf_lo(w[p]);
    x[2 * p + 1] = bf_hi(w[p]);
  }
  if (a.qw) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; i++) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int m = 1; m < kCPR; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
    const float rs = rsqrtf(fmaf(ss, 1.f / D, a.eps));
    const uint4 wv = load_rope_chunk<D>(a.qw, c, a.rope_half != 0);
    const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
    for (int p = 0; p < 4; p++) {
      x[2 * p] *= rs * bf_lo(ww[p]);
      x[2 * p + 1] *= rs * bf_hi(ww[p]);
    }
  }
  float4 c0, c1;
  rope_coeffs<D>(a.rope, max(pos0 + t, 0), c, c0, c1);
  const float cs[4] = {c0.x, c0.z, c1.x, c1.z}, sn[4] = {c0.y, c0.w, c1.y, c1.w};
  uint32_t h[4], l[4];
#pragma unroll
  for (int p = 0; p < 4; p++) {
    const float y0 = fmaf(x[2 * p], cs[p], -x[2 * p + 1] * sn[p]), y1 = fmaf(x[2 * p], sn[p], x[2 * p + 1] * cs[p]);
    h[p] = pack_f16(y0, y1);
    l[p] = pack_f16(y0 - f16_lo(h[p]), y1 - f16_hi(h[p]));
  }
  if (!on) {
#pragma unroll
    for (int p = 0; p < 4; p++) h[p] = l[p] = 0;
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

}  // namespace ne
