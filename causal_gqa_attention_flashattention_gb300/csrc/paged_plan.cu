// The paged cache's bookkeeping on the device (sm_103a): block tables and slot maps from the
// lengths of the requests, and the accepted path of a drafted tree moved into place.
#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace ne {
namespace {

// ====================================================================== tables and slots
// Sequence b has len[b] positions and is to have add[b] more.  With want = ceil((len + add) / page):
//   need = max(0, want - held), give = max(0, held - want), run = inclusive sum of need over b;
//   granted where need = 0 or run <= count;  the i-th page handed out is ring[(first + i) % P], in the
//   order of the sequences and their tables, the j-th returned goes to ring[(first + count + j) % P].
// A returned page serves the next call, so what is read of the ring and what is written are different
// places.  One block does the sums and moves the pages: the state is a few KB, and what bounds the
// kernel is its chain of round trips, not the bytes: launch and lengths, ring, table, parents.  64 sequences
// of one new token 4.4 us on the device (4.7 if the launch waits for the kernel in front), 48 trees of 5 to 24 tokens 6.1 us.
constexpr int kPlanThreads = 1024;
constexpr int kPlanMaxB = 2048;
// Rows up to which that block writes the slots too (64 sequences with 2048 rows in all 6.1 us, with a second launch
// 7.5; 4096 rows 7.8 and 7.3, 16384 rows 17.2 and 6.9).
constexpr int kPlanRows = 4096;

// Exclusive sum of v over the block's threads, and the total of all.
__device__ __forceinline__ unsigned long long block_scan(unsigned long long v, unsigned long long* wsum, unsigned long long* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  unsigned long long x = v;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, x, m);
    if (lane >= m) x += y;
  }
  if (lane == 31) wsum[warp] = x;
  __syncthreads();
  unsigned long long t = wsum[lane], low = lane < warp ? t : 0;
#pragma unroll
  for (int m = 16; m; m >>= 1) {
    t += __shfl_xor_sync(0xffffffffu, t, m);
    low += __shfl_xor_sync(0xffffffffu, low, m);
  }
  *total = t;
  __syncthreads();
  return low + x - v;
}
// The last b in [0, B) with start[b] <= x.
__device__ __forceinline__ int find(const int* start, int B, int x) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (start[m] <= x) lo = m;
    else hi = m;
  }
  return lo;
}
// Depth of token t of a tree; a parent that does not come before its child counts as the context.
__device__ __forceinline__ int tree_depth(const int* parents, int t, int* status) {
  int d = 0;
  for (;;) {
    const int p = parents[t];
    if (p < -1 || p >= t) {
      record_tree(status);
      return d;
    }
    if (p < 0) return d;
    t = p;
    d++;
  }
}

// Row n: token t = n - first of sequence b, which had len positions.
__device__ __forceinline__ void plan_row(const PagedPlanArgs& a, int n, int b, int t, int len, bool granted) {
  const int at = (int)((unsigned)len + (unsigned)t);  // a refused length may be anything
  int slot = -1;
  if (granted) {
    const int page = a.table[(size_t)b * a.max_pages + (at >> a.page_shift)];
    if (page >= 0 && page < a.num_pages)
      slot = (page << a.page_shift) + (at & ((1 << a.page_shift) - 1));
    else
      record_page(a.status);
  }
  a.slots[n] = slot;
  a.positions[n] = a.parents && t < a.Tq ? (int)((unsigned)len + tree_depth(a.parents + b * a.parent_stride, t, a.status)) : at;
}

__global__ void __launch_bounds__(kPlanThreads, 1) k_paged_plan(const PagedPlanArgs a) {
  __shared__ int s_got[kPlanMaxB], s_give[kPlanMaxB], s_cu[kPlanMaxB], s_from[kPlanMaxB], s_len[kPlanMaxB];
  __shared__ bool s_ok[kPlanMaxB];
  __shared__ unsigned long long wsum[32];
  __shared__ int s_first_short;
  pdl_wait();
  pdl_launch();
  const int tid = threadIdx.x, P = a.num_pages, cap = a.max_pages << a.page_shift;
  int first = a.span[0], count = a.span[1];
  const bool ring_ok = first >= 0 && first < P && count >= 0 && count <= P;
  if (!ring_ok) {
    if (tid == 0) record_page(a.status);
    first = count = 0;
  }
  if (tid == 0) s_first_short = 0x7fffffff;
  // two neighbouring sequences a thread
  int len[2], add[2], held[2], want[2];
  bool ok[2];
  unsigned long long pages = 0, rows = 0;
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const int b = 2 * tid + i;
    len[i] = add[i] = held[i] = want[i] = 0;
    ok[i] = true;
    if (b >= a.B) continue;
    len[i] = a.len[b];
    add[i] = a.add[b];
    held[i] = want[i] = a.held[b];
    ok[i] = ring_ok && len[i] >= 0 && len[i] <= cap && add[i] >= 0 && add[i] <= cap - len[i] && held[i] >= 0 &&
            held[i] <= a.max_pages && (!a.parents || add[i] <= a.Tq);
    if (ok[i])
      want[i] = (len[i] + add[i] + (1 << a.page_shift) - 1) >> a.page_shift;
    else if (ring_ok)
      record_page(a.status);
    rows += (unsigned)max(add[i], 0);
  }
  unsigned long long all_rows, all_pages;
  unsigned long long row0 = block_scan(rows, wsum, &all_rows);
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const int b = 2 * tid + i;
    if (b >= a.B) continue;
    const unsigned long long end = row0 + (unsigned)max(add[i], 0);
    if (end > (unsigned long long)a.N && ok[i] && add[i] > 0) {  // its rows are not all there
      ok[i] = false;
      want[i] = held[i];
      record_page(a.status);
    }
    s_cu[b] = (int)min(row0, (unsigned long long)a.N);
    a.cu[b] = s_cu[b];
    if (b == a.B - 1) a.cu[a.B] = (int)min(end, (unsigned long long)a.N);
    row0 = end;
    pages += ((unsigned long long)max(0, want[i] - held[i]) << 32) + (unsigned)max(0, held[i] - want[i]);
  }
  unsigned long long at = block_scan(pages, wsum, &all_pages);
  // pages are handed out in order as long as they last
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const int b = 2 * tid + i, need = max(0, want[i] - held[i]), give = max(0, held[i] - want[i]);
    if (b >= a.B) continue;
    const int n0 = (int)(at >> 32);
    s_got[b] = n0;
    s_give[b] = (int)(unsigned)at;
    s_from[b] = min(held[i], want[i]);
    if (need > 0 && n0 + need > count) {
      ok[i] = false;
      atomicMin(&s_first_short, n0);
    }
    if (need > 0 && !ok[i]) want[i] = held[i];
    at += ((unsigned long long)need << 32) + (unsigned)give;
    // a refused sequence keeps what it has
    a.held_out[b] = want[i];
    a.len_out[b] = len[i] + (ok[i] ? add[i] : 0);
    if (a.new_out) a.new_out[b] = ok[i] ? add[i] : 0;
    s_len[b] = len[i];
    s_ok[b] = ok[i];
  }
  __syncthreads();
  const int taken = min((int)(all_pages >> 32), s_first_short), given = (int)(unsigned)all_pages;
  for (int i = tid; i < taken; i += kPlanThreads) {
    const int b = find(s_got, a.B, i);
    int x = first + i;
    if (x >= P) x -= P;
    const int page = a.ring[x];
    if (page < 0 || page >= P) record_page(a.status);
    a.table[(size_t)b * a.max_pages + s_from[b] + (i - s_got[b])] = page;
  }
  for (int j = tid; j < given; j += kPlanThreads) {
    const int b = find(s_give, a.B, j);
    a.ring[((unsigned)first + (unsigned)count + (unsigned)j) % (unsigned)P] =
        a.table[(size_t)b * a.max_pages + s_from[b] + (j - s_give[b])];
  }
  if (tid == 0 && ring_ok) {
    int left = count - taken + given;
    if (left > P) {
      record_page(a.status);
      left = P;
    }
    a.span_out[0] = first + taken >= P ? first + taken - P : first + taken;
    a.span_out[1] = left;
  } else if (tid == 0) {
    a.span_out[0] = a.span[0];
    a.span_out[1] = a.span[1];
  }
  if (a.N > kPlanRows) return;  // k_paged_slots writes them
  __syncthreads();
  const int total = (int)min(all_rows, (unsigned long long)a.N);
  for (int n = tid; n < a.N; n += kPlanThreads) {
    if (n >= total) {
      a.slots[n] = -1;
      a.positions[n] = 0;
      continue;
    }
    const int b = find(s_cu, a.B, n);
    plan_row(a, n, b, n - s_cu[b], s_len[b], s_ok[b]);
  }
}

// The slots of many rows: 128 neighbouring ones a warp, whose threads look a sequence up again only where it changes.  With
// the plan in front 11.3 us for 200 prompts of 33 to 4096 tokens: the plan's block, a launch, and the
// trips cu -> table -> slot (the rows' 3.3 MB take 0.5 us).
constexpr int kSlotRows = 4;
__global__ void __launch_bounds__(256) k_paged_slots(const PagedPlanArgs a) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int w0 = (blockIdx.x * 8 + threadIdx.x / 32) * 32 * kSlotRows;
  if (w0 >= a.N) return;
  const int total = a.cu[a.B];
  int lo = 0, hi = a.B;  // the warp's first row: 32 probes at a time
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, i = lo + lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, i < hi && (lane == 0 || a.cu[i] <= w0));
    lo += (31 - __clz((int)le)) * step;
    hi = min(hi, lo + step);
  }
  int b = lo, first = a.cu[b], end = a.cu[b + 1], len = a.len[b];
  bool granted = a.len_out[b] == len + (end - first);
#pragma unroll
  for (int i = 0; i < kSlotRows; i++) {
    const int n = w0 + 32 * i + lane;
    if (n >= a.N) return;
    if (n >= total) {
      a.slots[n] = -1;
      a.positions[n] = 0;
      continue;
    }
    if (n >= end) {
      do {
        b++;
        end = a.cu[b + 1];
      } while (n >= end);
      first = a.cu[b];
      len = a.len[b];
      granted = a.len_out[b] == len + (end - first);
    }
    plan_row(a, n, b, n - first, len, granted);
  }
}

// ====================================================================== the accepted path
// Sequence b has len[b] positions, the last nodes[b] of them a tree; path[b, 0 .. count[b]) are the tokens
// that stay, in rising order: token path[i] moves to position len - nodes + i.  path[i] >= i, so a row may be
// both a source and a place, but a place only of a token before it: a warp takes a (sequence, head) and moves some rows
// at a time, in order, all of them read before one is written.  Bound by the trips lengths -> path -> table ->
// row: one tree of 8 tokens 2.0 us, 64 trees with 64 heads (16 layers of 4), 13.8 MB, 3.8 us; 6.5 us with a block for
// each, whose threads wait for one another.
constexpr int kKeepThreads = 128, kKeepChunks = 8;
template <int D>
__global__ void __launch_bounds__(kKeepThreads) k_kv_keep(const PagedKeepArgs a) {
  constexpr int kCPR = D / 8;
  __shared__ long long s_src[kTreeMax], s_dst[kTreeMax];
  pdl_wait();
  const int g0 = blockIdx.x * (kKeepThreads / 32), b = blockIdx.y, tid = threadIdx.x;
  const int cap = a.max_pages << a.page_shift, mask = (1 << a.page_shift) - 1;
  const int len = a.len[b], nodes = a.nodes ? a.nodes[b] : a.tokens;
  int m = a.count[b];
  int x = 0, before = -1;  // at once with the lengths
  if (tid < a.width) {
    x = a.path[(size_t)b * a.width + tid];
    if (tid > 0) before = a.path[(size_t)b * a.width + tid - 1];
  }
  if (nodes == 0) m = 0;  // no tree (the plan gave it no place): whatever its path holds
  if (len < nodes || len <= 0) {  // an idle slot of the batch
    if (g0 == 0 && tid == 0) a.len_out[b] = max(len, 0);
    return;
  }
  const int base = len - nodes;
  bool bad = nodes < 0 || m < 0 || m > min(nodes, a.width) || len > cap;
  if (!bad && tid < m) {
    bad = x <= before || x >= nodes;
    if (!bad) {
      const int from = base + x, to = base + tid;
      const int ps = a.table[(size_t)b * a.max_pages + (from >> a.page_shift)];
      const int pd = a.table[(size_t)b * a.max_pages + (to >> a.page_shift)];
      const bool there = ps >= 0 && ps < a.num_pages && pd >= 0 && pd < a.num_pages;
      if (!there) record_page(a.status);
      s_src[tid] = (long long)ps * a.page_stride + (long long)(from & mask) * D;
      s_dst[tid] = there && x != tid ? (long long)pd * a.page_stride + (long long)(to & mask) * D : -1;
    }
  }
  if (__syncthreads_or(bad)) {
    if (g0 == 0 && tid == 0) {
      record_tree(a.status);
      a.len_out[b] = max(min(base, len), 0);
    }
    return;
  }
  if (g0 == 0 && tid == 0) a.len_out[b] = base + m;
  const int g = g0 + tid / 32, lane = tid & 31, c = lane % kCPR;
  if (g >= a.Hkv) return;
  // chunk c of keys or values in turn, of row after row: 32 / kCPR of them a step
  constexpr int kRows = kKeepChunks * 32 / kCPR / 2;
  const long long head = ((long long)g << a.page_shift) * D + c * 8;
  for (int r0 = 0; r0 < m; r0 += kRows) {
    uint4 v[kKeepChunks];
#pragma unroll
    for (int k = 0; k < kKeepChunks; k++) {
      const int i = k * (32 / kCPR) + lane / kCPR, r = r0 + i / 2;
      if (r >= m || s_dst[r] < 0) continue;
      v[k] = *(i & 1 ? reinterpret_cast<const uint4*>(a.vp + s_src[r] + head) : reinterpret_cast<const uint4*>(a.kp + s_src[r] + head));
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kKeepChunks; k++) {
      const int i = k * (32 / kCPR) + lane / kCPR, r = r0 + i / 2;
      if (r >= m || s_dst[r] < 0) continue;
      *(i & 1 ? reinterpret_cast<uint4*>(a.vp + s_dst[r] + head) : reinterpret_cast<uint4*>(a.kp + s_dst[r] + head)) = v[k];
    }
    __syncwarp();
  }
}

}  // namespace

cudaError_t launch_paged_plan(const PagedPlanArgs& a, cudaStream_t s) {
  const cudaError_t e = launch_pdl(k_paged_plan, dim3(1), kPlanThreads, 0, s, a);
  if (e != cudaSuccess || a.N <= kPlanRows) return e;
  return launch_pdl(k_paged_slots, dim3((unsigned)((a.N + 256 * kSlotRows - 1) / (256 * kSlotRows))), 256, 0, s, a);
}

cudaError_t launch_kv_keep(const PagedKeepArgs& a, int D, cudaStream_t s) {
  const dim3 grid((unsigned)((a.Hkv + kKeepThreads / 32 - 1) / (kKeepThreads / 32)), (unsigned)a.B);
  return D == 64 ? launch_pdl(k_kv_keep<64>, grid, kKeepThreads, 0, s, a) : launch_pdl(k_kv_keep<32>, grid, kKeepThreads, 0, s, a);
}

}  // namespace ne
