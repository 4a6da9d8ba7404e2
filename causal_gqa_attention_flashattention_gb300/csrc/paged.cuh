// Shared by the paged cache's kernels: the status of a bad page, and queries on the
// way to the tensor cores.
#pragma once
#include "internal.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace ne {

constexpr float kPagedLn2 = 0.69314718055994531f;
constexpr int kSmemMax = 232448;

__device__ __forceinline__ void record_page(int* status) { atomicCAS(status, 0, kStatusPage); }

// Chunk c (8 values) of query row r of (sequence b, key/value head g) on its way to the
// tensor cores, in two steps so that a warp can have the loads of several rows under way.
struct QueryChunk {
  uint4 v;
  float4 c0, c1;
  bool on;
};
template <int D>
__device__ __forceinline__ QueryChunk query_load(const PagedDecodeArgs& a, int b, int g, int r, int c, int pos0) {
  QueryChunk x;
  x.on = r < a.R;
  const int t = x.on ? (int)fdiv((uint32_t)r, a.div_g) : 0, gg = r - t * a.G;
  x.v = make_uint4(0, 0, 0, 0);
  if (x.on) x.v = load_rope_chunk<D>(a.q + (size_t)(b * a.Tq + t) * a.q_stride + (g * a.G + gg) * D, c, a.rope_half != 0);
  rope_coeffs<D>(a.rope, max(pos0 + t, 0), c, x.c0, x.c1);
  return x;
}
// Normalises with the weight chunk w (where norm is set) and rotates in fp32; hi is the fp16
// rounding, lo that of the remainder.  The D / 8 lanes of a row are neighbours (every lane of
// the warp takes part); rows past the last come out as zeros.
template <int D>
__device__ __forceinline__ void query_finish(const PagedDecodeArgs& a, const QueryChunk& q, bool norm, const uint4& wv,
                                             uint4& hi, uint4& lo) {
  const uint32_t w[4] = {q.v.x, q.v.y, q.v.z, q.v.w};
  float x[8];
#pragma unroll
  for (int p = 0; p < 4; p++) {
    x[2 * p] = bf_lo(w[p]);
    x[2 * p + 1] = bf_hi(w[p]);
  }
  if (norm) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; i++) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int m = 1; m < D / 8; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
    const float rs = rsqrtf(fmaf(ss, 1.f / D, a.eps));
    const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
    for (int p = 0; p < 4; p++) {
      x[2 * p] *= rs * bf_lo(ww[p]);
      x[2 * p + 1] *= rs * bf_hi(ww[p]);
    }
  }
  const float cs[4] = {q.c0.x, q.c0.z, q.c1.x, q.c1.z}, sn[4] = {q.c0.y, q.c0.w, q.c1.y, q.c1.w};
  uint32_t h[4], l[4];
#pragma unroll
  for (int p = 0; p < 4; p++) {
    const float y0 = fmaf(x[2 * p], cs[p], -x[2 * p + 1] * sn[p]), y1 = fmaf(x[2 * p], sn[p], x[2 * p + 1] * cs[p]);
    h[p] = q.on ? pack_f16(y0, y1) : 0u;
    l[p] = q.on ? pack_f16(y0 - f16_lo(h[p]), y1 - f16_hi(h[p])) : 0u;
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// Row r of (sequence b, head g), columns 4 q .. 4 q + 3: normalise and write. L is 0 for a row that saw no
// key, and only then; a NaN stays one in o and lse.
template <int D>
__device__ __forceinline__ void write_row(const PagedDecodeArgs& a, int b, int g, int r, int q, float4 v, float M, float L) {
  const int t = (int)fdiv((uint32_t)r, a.div_g), h = g * a.G + (r - t * a.G);
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const size_t at = (((size_t)b * a.Tq + t) * a.Hq + h) * D + 4 * q;
  v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
  if (a.o_fp32)
    *reinterpret_cast<float4*>(static_cast<float*>(a.o) + at) = v;
  else
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + at) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
  if (q == 0 && a.lse) a.lse[((size_t)b * a.Hq + h) * a.Tq + t] = L == 0.f ? -INFINITY : (M + log2f(L)) * kPagedLn2;
}

// Positions of a sequence that the sweep leaves to the prefix kernel: the whole shared
// prefix if the first query sees all of it, else none.
__device__ __forceinline__ int sweep_base(const PagedDecodeArgs& a, int len) {
  return a.base > 0 && len - a.Tq + 1 >= a.base ? a.base : 0;
}

}  // namespace ne
