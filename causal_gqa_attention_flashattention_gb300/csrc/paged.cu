// Paged key/value cache (sm_103a): appending new tokens, and the attention of
// the newest tokens of every sequence over it.
//
// The pools hold num_pages pages of `page` positions, head-major inside a page
// ([num_pages, Hkv, page, D]: rotated keys fp16, values bf16), so that a page of
// one key/value head is one stretch of memory.  Position j of sequence b lies in
// row j % page of page table[b, j / page].  Lengths, tables and the places of new
// tokens are read on the device: a captured graph replays with new ones.  Every
// table entry is checked against num_pages before it is used; a bad one is
// recorded in the status word (kStatusPage) and never followed.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "paged_sweep.cuh"

namespace ne {
namespace {

// ====================================================================== append
// New row n belongs to the sequence s with cu[s] <= n < cu[s + 1] (rows at or
// past cu[B] belong to none and are skipped) and to position pos0[s] + n - cu[s].
// A thread takes one 16-byte chunk of a key row and of the value row; the D / 8
// threads of a row are neighbouring lanes (the norm adds up squares by shuffles).  Bound by the
// bytes: 23 prompts with 17,000 rows of four heads (34.9 MB) take 9.3 us, a step of 64 tokens 3.1 us.
// With SLOTS every row is given its place in the pool and its rotary position (negative slot: no place): 256 rows of
// four heads 1.7 us, 16381 (33.3 MB) 8.0 us: two and a quarter waves of blocks (12 an SM).
template <int D, bool SLOTS>
__global__ void __launch_bounds__(128) k_kv_append_paged(const PagedAppendArgs a) {
  if (SLOTS) pdl_wait();
  constexpr int kCPR = D / 8;
  const int lane = threadIdx.x & 31;
  const long long total = (long long)a.N * a.Hkv * kCPR;
  const long long it = blockIdx.x * 128LL + threadIdx.x;
  if ((it & ~31LL) >= total) return;  // whole warps leave: the rest shuffle together
  const bool in = it < total;
  const uint32_t row = (uint32_t)((in ? it : 0) / kCPR);
  const int c = (int)(it % kCPR);
  const uint32_t n = fdiv(row, a.div_hkv);
  const uint32_t g = row - n * a.Hkv;
  // the row itself first: its loads are under way while its place is looked up
  bool on = in;
  int slot = -1, pos = 0, page = -1;
  if (SLOTS) {
    slot = in ? a.slots[n] : -1;
    pos = in ? a.positions[n] : 0;  // at once: the rotation's coefficients are one trip nearer
    on = slot >= 0;
  } else {
    on = in && (!a.cu || (int)n < a.cu[a.B]);
  }
  uint4 kv = make_uint4(0, 0, 0, 0), vv = kv, wv = kv;
  if (SLOTS ? in : on) {
    kv = load_rope_chunk<D>(a.k + (size_t)n * a.k_stride + g * D, c, a.rope_half != 0);
    vv = __ldg(reinterpret_cast<const uint4*>(a.v + (size_t)n * a.v_stride + g * D) + c);
  }
  if (a.kw) wv = load_rope_chunk<D>(a.kw, c, a.rope_half != 0);
  if constexpr (SLOTS) {
    page = slot >> a.page_shift;
    if (on && (page >= a.num_pages || pos < 0 || pos >= a.capacity)) {
      record_page(a.status);
      on = false;
    }
    slot &= (1 << a.page_shift) - 1;
  } else {
    // the row's sequence and position
    int s = 0, first = 0;
    if (a.cu) {
      // last s with cu[s] <= n: 32 probes at a time for the warp's lowest row, then
      // each lane steps on to its own
      const int n0 = (int)__shfl_sync(0xffffffffu, n, 0);
      int lo = 0, hi = a.B;  // the answer is in [lo, hi)
      while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int i = lo + lane * step;
        const unsigned le = __ballot_sync(0xffffffffu, i < hi && (lane == 0 || a.cu[i] <= n0));
        const int top = 31 - __clz((int)le);
        lo += top * step;
        hi = min(hi, lo + step);
      }
      s = lo;
      while (s + 1 < a.B && a.cu[s + 1] <= (int)n) s++;
      first = a.cu[s];
      on = on && (int)n >= first;
    } else {
      s = (int)fdiv(n, a.div_per);
      first = s * (int)a.div_per.d;
    }
    pos = on ? a.pos0[s] + ((int)n - first) : 0;
    if (on) {
      const int i = pos >> a.page_shift;
      if (pos >= 0 && i < a.max_pages) page = a.table[(size_t)s * a.max_pages + i];
      if (page < 0 || page >= a.num_pages) {
        record_page(a.status);
        on = false;
      }
    }
    slot = pos & ((1 << a.page_shift) - 1);
  }
  float4 c0 = make_float4(0.f, 0.f, 0.f, 0.f), c1 = c0;
  if (on) rope_coeffs<D>(a.rope, pos, c, c0, c1);
  const uint32_t w[4] = {kv.x, kv.y, kv.z, kv.w};
  float x[8];
#pragma unroll
  for (int p = 0; p < 4; p++) {
    x[2 * p] = bf_lo(w[p]);
    x[2 * p + 1] = bf_hi(w[p]);
  }
  if (a.kw) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; i++) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int m = 1; m < kCPR; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
    const float r = rsqrtf(fmaf(ss, 1.f / D, a.eps));
    const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
    for (int p = 0; p < 4; p++) {
      x[2 * p] *= r * bf_lo(ww[p]);
      x[2 * p + 1] *= r * bf_hi(ww[p]);
    }
  }
  if (!on) return;
  const float cs[4] = {c0.x, c0.z, c1.x, c1.z}, sn[4] = {c0.y, c0.w, c1.y, c1.w};
  uint32_t o[4];
#pragma unroll
  for (int p = 0; p < 4; p++)
    o[p] = pack_f16(fmaf(x[2 * p], cs[p], -x[2 * p + 1] * sn[p]), fmaf(x[2 * p], sn[p], x[2 * p + 1] * cs[p]));
  const size_t dst = (size_t)page * a.page_stride +
                     (((size_t)g << a.page_shift) + slot) * D;
  reinterpret_cast<uint4*>(a.kp + dst)[c] = make_uint4(o[0], o[1], o[2], o[3]);
  reinterpret_cast<uint4*>(a.vp + dst)[c] = vv;
}

}  // namespace

template <bool SLOTS>
static cudaError_t launch_append(const PagedAppendArgs& a, int D, cudaStream_t s) {
  const long long n = (long long)a.N * a.Hkv * (D / 8);
  const unsigned grid = (unsigned)((n + 127) / 128);
  if (SLOTS) {
    return D == 64 ? launch_pdl(k_kv_append_paged<64, SLOTS>, dim3(grid), 128, 0, s, a)
                   : launch_pdl(k_kv_append_paged<32, SLOTS>, dim3(grid), 128, 0, s, a);
  }
  if (D == 64)
    k_kv_append_paged<64, SLOTS><<<grid, 128, 0, s>>>(a);
  else
    k_kv_append_paged<32, SLOTS><<<grid, 128, 0, s>>>(a);
  return cudaGetLastError();
}
cudaError_t launch_kv_append_paged(const PagedAppendArgs& a, int D, cudaStream_t s) { return launch_append<false>(a, D, s); }
cudaError_t launch_kv_append_slots(const PagedAppendArgs& a, int D, cudaStream_t s) { return launch_append<true>(a, D, s); }

void paged_rows(int R, int* mt, int* tiles, int* mg) {
  *mt = R <= 8 ? 1 : (R <= 16 ? 2 : 4);
  *mg = R <= 32 ? 1 : (R <= 64 ? 2 : 4);
  *tiles = *mt * *mg;
}

cudaError_t launch_decode_paged(const PagedDecodeArgs& a, int mt, int nsm, cudaStream_t s) {
  return launch_sweep<false>(a, mt, nsm, s);
}

}  // namespace ne
