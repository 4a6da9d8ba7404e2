// Internal interfaces between the C-ABI layer (api.cu) and the kernel files.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace ne {

constexpr int kTile = 128;  // query rows / key rows per tile

// Device-side status codes (mirror ne_status in include/ne_attn.h). The word keeps the first bad page,
// but a timeout takes its place: counters that the library keeps may then be half way.
constexpr int kStatusTimeout = -6;
constexpr int kStatusPage = -8;
constexpr int kStatusTree = -9;

// Flag bits shared with include/ne_attn.h.
constexpr int kFlagOFp32 = 1;      // o is float32
constexpr int kFlagGradFp32 = 2;   // dq, dk, dv are float32
constexpr int kFlagPreciseQK = 4;  // logits from hi + lo fp16 parts of rotated q and k
constexpr int kFlagQKRotated = 8;  // backward: the workspace already holds the forward's rotated q and k
constexpr int kFlagRopeHalf = 16;  // RoPE pairs (x[i], x[i + D/2]) instead of (x[2i], x[2i+1])
constexpr int kFlagFp8 = 32;       // forward: rotated q, k as e4m3 with per-head scales

// Largest number of query heads one forward CTA handles (TMEM/smem budget).
inline int fwd_max_heads(int D, bool precise) { return D == 64 ? (precise ? 3 : 4) : 8; }

struct FwdArgs {
  // 4-D tiled maps over [B, T, H, D], box D x 1 x 128 x 1.  Default precision:
  // map_q / map_k cover the rotated fp16 copies in the workspace (e4m3 with
  // FP8); precise logits: the bf16 inputs (the kernel rotates them itself).
  CUtensorMap map_q, map_k, map_v;
  CUtensorMap map_o;                // store map over o (default precision): 128-byte (or 64-byte) column boxes x 32 rows
  void* o;                          // [B, T, Hq, D] bf16 or fp32
  float* lse;                       // [B, Hq, T]
  float* lse_lo;                    // [B, Hq, T] fp32 remainder of lse (precise logits only)
  const float2* rope;               // [Tcap][D/2] (cos, sin)
  int* status;                      // device status word
  int B, T, Hq, Hkv, D, G, HC;      // HC: query heads per CTA (divides G; precise-logits kernel)
  int nt;                           // number of 128-row tiles
  int o_fp32;
  float scale_log2;                 // log2(e) / sqrt(D), rounded to fp32
  float scale_log2_lo;              // remainder log2(e)/sqrt(D) - scale_log2
  const float* qk_amax;             // FP8 forward: per-head max |rotated value|, [Hq] for q then [Hkv] for k
  const int* sched;                 // [grid, sched_k] int4 work items of each CTA (b = -1: none), see fwd_pair_schedule
  int sched_k;
  int grid;                         // CTAs of the persistent forward
};

// Division of a non-negative 32-bit n < 2^31 by a runtime divisor d >= 1 with
// a multiply-high and a shift (round-up magic number):
//   l = ceil(log2 d), m = floor(2^32 (2^l - d) / d) + 1, n / d = (umulhi(n, m) + n) >> l.
struct FastDiv {
  uint32_t d, m, l;
};
inline FastDiv make_fastdiv(uint32_t d) {
  uint32_t l = 0;
  while ((1ull << l) < d) l++;
  const uint64_t m = ((1ull << 32) * ((1ull << l) - d)) / d + 1;
  return FastDiv{d, (uint32_t)m, l};
}

#ifdef __CUDACC__
__device__ __forceinline__ uint32_t fdiv(uint32_t n, const FastDiv& f) { return (__umulhi(n, f.m) + n) >> f.l; }
#endif

// RoPE pre-pass of the forward: q, k (bf16) -> rotated fp16 copies qr, kr.
struct RopeArgs {
  const __nv_bfloat16 *q, *k;
  __half *qr, *kr;
  const float2* rope;
  int B, T, Hq, Hkv;
  int rope_half;  // half-split pair layout of q and k
  FastDiv div_hq, div_hkv, div_t;
  FastDiv div_hg;    // by the groups of four heads (Hq + Hkv, four per thread) of k_rope_qk
  uint8_t *q8, *k8;  // FP8 forward: rotated q, k as e4m3 scaled by 448 / max |value| of their head
  float* amax;       // FP8 forward: [Hq + Hkv] per-head max |rotated value| (zeroed before the max pass)
};

struct BwdArgs {
  CUtensorMap map_qr, map_kr, map_v, map_do;  // 4-D maps as above (qr/kr: rotated fp16 copies)
  CUtensorMap map_qlo, map_klo;               // fp16 remainders (precise logits only)
  CUtensorMap map_dqacc;                      // 2-D map over [B*Hq*Tp, D] fp32, box 32 x 128
  CUtensorMap map_dk, map_dv;                 // 4-D store maps over [B, T, Hkv, D] (fp32 or bf16), box
                                              // 128 bytes of columns x 1 x 128 rows x 1, same swizzle span
  const float* lse2;                          // [B, Hq, Tp]  lse * log2(e); +inf on pad rows
  const float* lse2_lo;                       // [B, Hq, Tp]  its fp32 remainder (precise logits only)
  const float* delta;                         // [B, Hq, Tp]
  void* dk;                                   // [B, T, Hkv, D] bf16 or fp32
  void* dv;
  const float2* rope;
  int* status;
  int B, T, Hq, Hkv, D, G, nt, Tp;
  int grad_fp32;
  int rope_half;  // dk leaves in the half-split pair layout
  float scale_log2, scale_log2_lo, scale;
};

struct PrepArgs {
  const __nv_bfloat16 *q, *k, *dout;
  const void* o;  // bf16 or fp32
  const float* lse;
  const float* lse_lo;          // null unless precise logits
  __half *qr, *kr, *qlo, *klo;  // qlo/klo null unless precise logits
  float *lse2, *lse2_lo, *delta, *dqacc;
  const float2* rope;
  int B, T, Hq, Hkv, D, Tp, o_fp32;
  int rotate_qk;                            // 0: qr / kr already hold the rotated q and k
  int rope_half;                            // half-split pair layout of q and k
  int negate;                               // 1: store -lse * log2(e) and -Delta (default-precision sweep)
  FastDiv div_hq, div_hkv, div_t, div_pad;  // by Hq, Hkv, T and Tp - T (pad rows; d = 1 if none)
};

struct DqArgs {
  const float* dqacc;  // [B, Hq, Tp, D]
  void* dq;            // [B, T, Hq, D]
  const float2* rope;
  int B, T, Hq, D, Tp, grad_fp32;
  int rope_half;  // dq leaves in the half-split pair layout
  float scale;
  FastDiv div_hq, div_t;
  FastDiv div_hg;  // by the groups of four query heads (four per thread)
};

// Key/value cache append: rotated keys (fp16) and values (bf16) of Tn new positions.
struct KvAppendArgs {
  const __nv_bfloat16 *k, *v;  // [B, Tn, Hkv, D]
  __half* kc;                  // [B, Hkv, Tcap, D] rotated keys
  __nv_bfloat16* vc;           // [B, Hkv, Tcap, D]
  const float2* rope;
  int B, Tn, Hkv, Tcap, pos0;
  int rope_half;  // half-split pair layout of the new keys
  FastDiv div_hkv, div_tn;
};

// Decode over a key/value cache (see attn_decode.cu).
struct DecodeArgs {
  CUtensorMap map_q;         // packed rotated queries [B*Hkv*128, D] fp16 (4-D map, box D x 1 x 128 x 1)
  CUtensorMap map_k, map_v;  // caches [B, Hkv, Tkv valid of Tcap, D] (fp16 keys, bf16 values)
  const __nv_bfloat16* q;    // [B, Tq, Hq, D]
  __half* qpk;               // [B, Hkv, 128, D] packed rotated queries (workspace)
  float* part_o;             // [B, Hkv, nsplit, F, R, D] unnormalised O per split and copy (workspace)
  float* part_ml;            // [B, Hkv, nsplit, F, R] (max in log2 units, sum) pairs (workspace)
  unsigned* done;            // [B * Hkv] finished splits per group (workspace; zeroed by the query pass)
  void* o;                   // [B, Tq, Hq, D] bf16 or fp32
  float* lse;                // [B, Hq, Tq]
  const float2* rope;
  int* status;
  int B, Tq, Tkv, Hq, Hkv, D, G, R, ntk, nsplit, o_fp32;
  int F;                     // copies of the R query rows in the 128-row tile: 4 if R <= 32, 2 if R <= 64, else 1
  int rope_half;             // half-split pair layout of q (and of the cached keys)
  float scale_log2;
};

// RMSNorm + fused Q/K/V projection (see qkv_proj.cu).  Rows r = b * T + t of
// x [M, C]; projection features n of w_qkv [N, C], N = (Hq + 2 Hkv) D.
struct QkvArgs {
  CUtensorMap map_x;              // x [M, C] bf16, box 64 x 128, 128-byte swizzle
  CUtensorMap map_w;              // folded weight [N, C] bf16, box 64 x BN, 128-byte swizzle
  CUtensorMap map_qr, map_kr;     // store maps over the rotated fp16 q [M, Hq, D], k [M, Hkv, D]
  CUtensorMap map_vst;            // store map over v [M, Hkv, D] bf16 (boxes 32 x 1 x 128, 64-byte swizzle)
  const __nv_bfloat16* x;         // [M, C]
  const __nv_bfloat16* norm_w;    // [C]
  const __nv_bfloat16* w;         // [N, C]
  __nv_bfloat16* wf;              // [N, C] w_qkv[n', c] * norm_w[c], rows permuted for half-split q, k
  float* rstd;                    // [M]
  __nv_bfloat16 *q, *k, *v;       // [M, Hq, D], [M, Hkv, D], [M, Hkv, D] (q and k may be null)
  __half *qr, *kr;                // rotated fp16 q and k (null: not written)
  const float2* rope;
  int* status;
  int M, C, N, T, Hq, Hkv, D;
  int nkb, ntn, tiles;            // 64-wide K blocks, BN-wide column tiles, 128 x BN tiles
  int rope_half;
  float eps;
};

// Norms of the query and key heads with the rotation, and their backward (see qk_norm.cu).
struct QkNormArgs {
  const __nv_bfloat16 *q, *k;    // [B, T, H, D], rows of one position q_stride / k_stride values apart
  const __nv_bfloat16 *qw, *kw;  // [D]
  __half *qr, *kr;               // [B, T, Hq, D], [B, T, Hkv, D] rotated
  const float2* rope;
  long long q_stride, k_stride;
  int B, T, Hq, Hkv, rope_half;
  float eps;
  int nbq;                       // blocks that work on q; the others on k
  FastDiv div_t, div_hq, div_hkv;
};
struct QkNormBwdArgs {
  const __nv_bfloat16 *q, *k, *qw, *kw;
  const void *gq, *gk;  // gradients of the normalised q, k [B, T, H, D], bf16 or fp32
  void *dq, *dk;        // gradients of q, k (same type), rows dq_stride / dk_stride values apart
  float* part;          // [blocks + groups, D] partial weight gradients (workspace)
  unsigned* done;       // [2 + groups] groups of a side, and blocks of a group, that have left theirs; 0
                        // before and after (workspace or the library's)
  float *dqw, *dkw;     // [D]
  long long q_stride, k_stride, dq_stride, dk_stride;
  int B, T, Hq, Hkv;
  float eps;
  int nbq;              // blocks that work on q; the others on k
  FastDiv div_hq, div_hkv;
};
constexpr int kQkNormMaxSms = 160, kQkNormBlocksPerSm = 3, kQkNormFwdBlocksPerSm = 5;
constexpr int kQkNormMaxBlocks = kQkNormMaxSms * kQkNormBlocksPerSm;  // bounds the backward's partials
constexpr int kQkNormGroup = 32;  // blocks whose partials are added first
constexpr int kQkNormMaxGroups = kQkNormMaxBlocks / kQkNormGroup + 2;

// Append of new keys and values to a paged cache (see paged.cu).
struct PagedAppendArgs {
  const __nv_bfloat16 *k, *v, *kw;  // new rows [N, Hkv, D], k_stride / v_stride values apart; kw [D] or null
  __half* kp;                       // [num_pages, Hkv, page, D] rotated keys, pages page_stride values apart
  __nv_bfloat16* vp;
  const int *table, *pos0, *cu;     // [B, max_pages], [B], [B + 1] or null (N / B rows for every sequence)
  const float2* rope;
  int* status;
  long long k_stride, v_stride, page_stride;
  int N, B, Hkv, page_shift, num_pages, max_pages, rope_half;
  float eps;
  FastDiv div_hkv, div_per;         // by Hkv and by N / B (cu null)
  const int *slots, *positions;     // append to slots: [N] each; table, pos0 and cu are then not used
  int capacity;                     // positions of the rotary table
};

// Block tables and slot maps from lengths (see paged_plan.cu).
constexpr int kTreeMax = 64;  // tokens of a drafted tree: one bit each in a mask of ancestors
struct PagedPlanArgs {
  int *table, *ring;                           // [B, max_pages], [num_pages]
  const int *held, *span, *len, *add;          // [B], [2] (first, count), [B], [B]
  const int* parents;                          // [B, Tq] parent_stride apart, or null
  int *held_out, *span_out, *len_out;          // the first two may be held and span
  int* new_out;                                // [B] or null; may be add
  int *cu, *slots, *positions;                 // [B + 1], [N], [N] (N may be 0)
  int* status;
  long long parent_stride;
  int N, B, Tq, page_shift, num_pages, max_pages;
};

// The accepted path of a drafted tree moved behind the cached positions (see paged_plan.cu).
struct PagedKeepArgs {
  __half* kp;
  __nv_bfloat16* vp;
  const int *table, *len, *nodes, *path, *count;  // [B, max_pages], [B], [B] or null (all `tokens`), [B, width], [B]
  int* len_out;                                   // [B]
  int* status;
  long long page_stride;
  int B, Hkv, width, tokens, page_shift, num_pages, max_pages;
};


// Attention of a drafted tree over a paged cache (see paged_tree.cu).
struct TreeInfo {               // a sequence's tree
  unsigned long long mask[kTreeMax];  // a token and its ancestors
  int ctx, nodes;
};
struct PagedTreeArgs {
  CUtensorMap map_pk, map_pv;   // pools {D, page, Hkv, num_pages}, box D x min(page, 128) rows
  const __nv_bfloat16 *q, *qw;  // [B, Tq, Hq, D], positions q_stride values apart; qw [D] or null
  const int *table, *len;       // [B, max_pages], [B]
  const int *parents, *nodes;   // [B, Tq] rows parent_stride apart; [B] or null (all Tq)
  const float2* rope;
  int* status;
  void* o;
  float* lse;                   // or null
  float* part_o;                // [2 blocks, rows, D] unnormalised O of a block's first and last segment (workspace)
  float2* part_ml;              // [2 blocks, rows] their maximum (log2 units) and sum
  int4* cut;                    // [blocks] the cut (sequence, head) that begins in the block or goes through it: sequence
                                // (-1: none), head, first and last block (workspace)
  long long q_stride, parent_stride;
  int B, Tq, Hq, Hkv, D, G, R, page_shift, num_pages, max_pages, rope_half, o_fp32;
  int pairs, rows;              // pairs of 128-row tiles of a head's queries, rows of the largest
  FastDiv div_g, div_grid;      // by G and the sweep's blocks
  float eps, scale_log2;
};
inline int tree_pairs(int R) { return (R + 2 * kTile - 1) / (2 * kTile); }

// Attention of the newest tokens over a paged cache (see paged.cu).
constexpr int kPagedMaxBlocks = 160;  // blocks of the sweep: bounds its partial results
// The shared prefix's part of it (see paged_prefix.cu): key tiles of 128 positions over every
// (key/value head, pair of 128-row tiles), in one line, block c's stretch [c W / blocks, ..).
struct PrefixArgs {
  float* part_o;    // unnormalised O of segment (block c, (head, pair) s), unit u: part prefix_part(c + s, u),
                    // float4 prefix_quad of it (workspace)
  float2* part_ml;  // [part, 128] maximum (log2 units) and sum of the rows
  float* o;         // [Hkv, tiles * 128, D] the sequences' own parts, unnormalised (workspace)
  float2* ml;       // [Hkv, tiles * 128]
  int* cut;         // blocks that took the prefix (workspace)
  int tiles, pairs, ntk, W;
};
#ifdef __CUDACC__
__device__ __forceinline__ size_t prefix_part(int segment, int unit) { return (size_t)segment * 2 + unit; }
// Columns 4 q .. of a row: the 32 rows of a warp lie side by side, so that the warp's stores
// (and the loads of a sequence's neighbouring rows) are whole sectors.
template <int D>
__device__ __forceinline__ size_t prefix_quad(size_t part, int row, int q) {
  return ((part * (kTile / 32) + row / 32) * (D / 4) + q) * 32 + row % 32;
}
// The prefix's tiles, `ntk` of each of its segs (head, pair)s, cut among its blocks: with at least a
// block for each (head, pair) (blocks is then a multiple of segs) every one is cut for itself, else
// all of them in one line.
struct PrefixCut {
  int ntk, per, base, rem;  // per: blocks of a (head, pair), 0: in one line; the first rem blocks have base + 1
  __device__ PrefixCut(int ntk_, int segs, int blocks) : ntk(ntk_), per(blocks >= segs ? blocks / segs : 0) {
    const int n = per ? per : blocks, tiles = per ? ntk : ntk * segs;
    base = tiles / n;
    rem = tiles - base * n;
  }
  __device__ int start(int c) const {
    const int s = per ? c / per : 0, i = c - s * per;
    return s * ntk + i * base + min(i, rem);
  }
  // the first and last block of the (head, pair) s
  __device__ int first(int s) const { return per ? s * per : at(s * ntk); }
  __device__ int last(int s) const { return per ? s * per + min(per, ntk) - 1 : at(s * ntk + ntk - 1); }
  __device__ int at(int x) const {  // the block with tile x of the one line
    const int big = rem * (base + 1);
    return x < big ? x / (base + 1) : rem + (x - big) / base;
  }
};
#endif

struct PagedDecodeArgs {
  CUtensorMap map_pk, map_pv;   // prefix: pools {D, page, Hkv, num_pages}, box D x min(page, 128) rows
  const __half* kp;             // pools, pages page_stride values apart
  const __nv_bfloat16* vp;
  long long page_stride;
  PrefixArgs pre;
  const __nv_bfloat16 *q, *qw;  // [B, Tq, Hq, D], positions q_stride values apart; qw [D] or null
  const int *table, *len, *prefix_table;
  const float2* rope;
  int* status;
  void* o;
  float* lse;       // or null
  float* part_o;    // [2 blocks, R, D] unnormalised O of a block's first and last segment (workspace)
  float2* part_ml;  // [2 blocks, R] their maximum (log2 units) and sum
  unsigned* done;   // [blocks] segments finished of the (sequence, head) whose first one is the block's
  long long q_stride;
  int B, Tq, Hq, Hkv, D, G, R, page_shift, num_pages, max_pages, prefix_len, rope_half, o_fp32;
  int base;         // shared positions that the prefix kernel reads (0: none, the sweep reads all)
  int tiles, MG;    // packed row tiles (8 rows each) and the groups of warps that share them
  FastDiv div_grid; // by the sweep's blocks
  FastDiv div_r, div_g;  // by R, G
  int own_counters; // done is the library's: 0 before and after every call
  float eps, scale_log2;
};

// Launch that may start before the kernel ahead of it in the stream ends; the
// kernel calls pdl_wait before it touches what that one writes.
#ifdef __CUDACC__
template <typename... P, typename... A>
cudaError_t launch_pdl(void (*k)(P...), dim3 grid, int block, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, static_cast<P>(args)...);
}
#endif

int qk_norm_blocks(int B, int T, int Hq, int Hkv, int D, int nsm, bool bwd, int* nbq);
cudaError_t launch_qk_norm(const QkNormArgs& a, int D, int blocks, cudaStream_t s);
cudaError_t launch_qk_norm_bwd(const QkNormBwdArgs& a, int D, bool f32, int blocks, bool clear, cudaStream_t s);
cudaError_t launch_kv_append_paged(const PagedAppendArgs& a, int D, cudaStream_t s);
cudaError_t launch_kv_append_slots(const PagedAppendArgs& a, int D, cudaStream_t s);
cudaError_t launch_paged_plan(const PagedPlanArgs& a, cudaStream_t s);
cudaError_t launch_kv_keep(const PagedKeepArgs& a, int D, cudaStream_t s);
cudaError_t launch_decode_tree(const PagedTreeArgs& a, int nsm, cudaStream_t s);
void paged_rows(int R, int* mt, int* tiles, int* mg);
cudaError_t launch_decode_paged(const PagedDecodeArgs& a, int mt, int nsm, cudaStream_t s);
cudaError_t launch_decode_prefix(const PagedDecodeArgs& a, int mt, int nsm, cudaStream_t s);

cudaError_t launch_qkv_prep(const QkvArgs& a, cudaStream_t s);
cudaError_t launch_qkv_gemm(const QkvArgs& a, int BN, int grid, cudaStream_t s);
int qkv_pick_bn(int M, int N, int nsm, int* grid);

cudaError_t launch_fwd(const FwdArgs& a, bool precise, cudaStream_t s);
cudaError_t launch_kv_append(const KvAppendArgs& a, int D, cudaStream_t s);
cudaError_t launch_decode_q(const DecodeArgs& a, cudaStream_t s);
cudaError_t launch_decode(const DecodeArgs& a, int nsm, cudaStream_t s);
cudaError_t launch_rope_qk(const RopeArgs& a, int D, cudaStream_t s);
cudaError_t launch_rope_amax(const RopeArgs& a, cudaStream_t s);  // D = 64
cudaError_t launch_rope_q8(const RopeArgs& a, cudaStream_t s);    // D = 64
cudaError_t launch_fwd_fp8(const FwdArgs& a, cudaStream_t s);      // D = 64
cudaError_t launch_bwd_prep(const PrepArgs& a, cudaStream_t s);
cudaError_t launch_bwd_dkdv(const BwdArgs& a, bool precise, cudaStream_t s);
cudaError_t launch_bwd_dq(const DqArgs& a, cudaStream_t s);
cudaError_t launch_rope_table(float2* tab, int Tcap, int D, double base, cudaStream_t s);
cudaError_t launch_timeout_probe(int* status, long long limit_ns, cudaStream_t s);

}  // namespace ne
