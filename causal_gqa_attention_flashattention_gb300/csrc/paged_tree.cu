// Attention of a tree of drafted tokens over a paged key/value cache (sm_103a).
//
// Sequence b has len[b] positions in the cache, the last nodes[b] of them a tree: token t hangs on token
// parents[t] < t, or on the context (-1).  With ctx = len - nodes and depth the number of ancestors,
//   q^_t = R_(ctx + depth(t)) q_t,   s_tj = q^_t . k^_j / sqrt(D)
// for j < ctx and for the positions ctx + u of t's ancestors u and of t itself; o and lse as ever.  A token's
// ancestors and itself are a mask of 64 bits.
//
// The R = Tq * G queries of a key/value head fill tiles of 128 rows (row t * G + g). The key tiles of every
// (sequence, head, pair of row tiles) lie in one line that is cut into one equal stretch for each block, as in the
// sweep of the paged decode, and each tile is worked off on the tensor cores: S = Q K^T and O += P V with TMEM
// accumulators, q as two fp16 parts and the weights as two bf16 parts (the paged decode's precision: a tree's rows are
// the decode's of the accepted path). A step is one key tile for one row tile; two groups of four softmax warps take the
// steps in turn, each with an O of its own. With up to 128 rows the groups share the row tile and take alternate key
// tiles (their two O are added at the end), with more each has one of the pair's.
//
// A product of 128 rows and 64 columns takes the tensor cores as long as one of 128 columns (64 clocks for 16 keys), so
// the two parts of the weights cost as much again as the two of the scores. Up to 64 rows therefore have two lanes each:
// of a warp's 32 lanes the first 16 hold the scores of its 16 rows and the high parts of their weights, the others the
// low parts, and one product takes both. The warp reads the 16 lanes as a matrix fragment (two rows of four neighbouring
// threads each), so that every thread works on half as many scores. (16 trees of 4 and of 16 tokens, 12 and 48 rows, on
// contexts around 8192: 30.6 and 32.2 us; with a lane for each row 36.4 and 38.2.)
//
// The softmax warps pack the queries (normalised, rotated, two parts) and work the trees out themselves: those of a
// block's first segments while its first keys are on their way, those of a later one when its slot is free, by the group
// that does not write the rows of the segment before out; that one reads the other's O where it is, in TMEM. (16 trees of
// 16: 32.5 us, with a kernel in front of the sweep 34.5, with four more warps for it 36 to 38. 64 trees of 32 with 128
// rows: 54.4; with one group doing both 61.5, with the kernel 58.0.)
//
// The warps wait for instructions as often as for scores, so code that is not part of a step is kept small (its loops
// rolled, its waits short), and registers are kept for the steps: four spilled words or a part of a segment's end unrolled
// took 2 to 4 us of a call.
//
// A segment that is not the whole of its (sequence, head) leaves its parts to k_tree_join; a join inside the sweep, by
// the block that is last to finish, kept the others waiting for memory fences (34.6 -> 39.8 us) and was taken out.
//
// What bounds it (device times; 4 key/value heads of 64): up to 64 rows and a long context the bytes of K and V, 0.74 us
// for a tile of every block (a steady 6.8 TB/s); the call adds the start (lengths, tables, first tiles: 4 us), the last
// tiles' steps (3 us) and the join (2 to 6 us). 16 trees of 16 on contexts around 8192, pages of 64: 32.5 us, 19.1 of them
// the bytes; with pages of 16 39 us (eight copies a tile, each of 2 KB). With 128 rows a step takes the tensor cores
// 1536 clocks for two parts of both factors and the softmax as long: 64 trees of 32 on 700 to 4096 positions, 53.3 us.
// With 256 rows and an fp32 o (three parts), 64 tokens on 131001 positions, 110 us.
#include "paged_sweep.cuh"

namespace ne {
namespace {

// Sequence b: its positions and tokens, both 0 for an idle slot of the batch (or one that cannot be, or one without a
// tree in this call: nothing of its context is read).
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
  if (x.len < x.nodes || x.nodes == 0) return {0, 0};
  return x;
}

// mbar_wait in fewer instructions: the sweep's warps wait for instructions as it is (16 trees of 16 on contexts around
// 8192 33.6 -> 32.6 us). At most 2^17 tries of at most 20 us.
__device__ __forceinline__ bool tree_wait(uint64_t* bar, uint32_t parity, const volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
#pragma unroll 1
  for (int i = 0; i < 1 << 17; i++) {
    if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
    if (*abort) return false;
  }
  return false;
}

constexpr int kTreeThreads = 384;
// A segment's cost beside its tiles, in tiles; a (sequence, head) of at most so many tiles is never cut; a
// boundary moves by so many to an end of a longer one.
// Over 17 batches: a segment's cost of 1 takes up to 6 % more, one of 3 up to 4 % more or less, one of 4 up to 4 % more;
// whole up to 8 and a boundary moved by 3 up to 3 % more; no moves 4 % more for 128 short sequences, and others 0 to 4 % less.
constexpr int kTreeOver = 2, kTreeWhole = 4, kTreeSlack = 2;

template <int D>
struct TreeCfg {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr uint32_t kSpan = D * 2;
  static constexpr uint32_t kSwz = D == 64 ? kSw128 : kSw64;
  static constexpr uint32_t kSBO = 8 * kSpan;
  // A key tile is free once its scores are done, a value tile two to three steps later: 3 and 6 stages (together 4: the
  // loads' 1.25 us under load then bounded a step, 1750 clocks with 48 rows where 1450 are possible).
  static constexpr int kKStages = D == 64 ? 3 : 4, kVStages = D == 64 ? 6 : 8;
  static constexpr int kOffK = 4 * kTileBytes;  // Q first: two slots of (high, low), or a pair's two row tiles
  static constexpr int kOffV = kOffK + kKStages * kTileBytes;
  static constexpr int kBytes = kOffV + kVStages * kTileBytes;
  // Tensor memory: group g's O at 64 g. With both parts of the weights in one lane step n has its S at 128 +
  // 128 (n % 3), and P in its place; with SPLIT a group has S at 128 + 128 g and P, 64 columns, at 384 + 64 g, so that
  // its next scores are worked out while it is on its weights. With FULL a group has one buffer of S, at 128 + 128 g, and
  // the third parts go to 384 + 64 g, with SPLIT in the place of S.
  static constexpr uint32_t kColO = 0, kColS = 128, kColP = 384;
};
constexpr int kTreeVars = 480, kTreePlan = 488, kTreeSums = 544, kTreeInfo = 608, kTrees = 5, kTreeMl = 3248;
constexpr int kTreeWalk = kTreeMl + 4 * kTile * 8, kTreeCum = kTreeWalk + 8 * 2 * 6 * 4;
static_assert(kTreeInfo + kTrees * sizeof(TreeInfo) <= kTreeMl && kTreePlan + sizeof(SweepPlan) <= kTreeSums, "head");
static_assert((2 + 2 * TreeCfg<32>::kKStages + 2 * TreeCfg<32>::kVStages + 4 + 8 + 3 + 4 + 8 + 2 + 3) * 8 <= kTreeVars,
              "barriers");
__host__ __device__ constexpr int tree_head(int B) { return (kTreeCum + (B + 1) * 4 + B + 1023) / 1024 * 1024; }

// The tile's bits of a mask over positions that begins `r` positions before position 0 of the tree (r < 0: in the
// context, all ones): 32 columns from there.
__device__ __forceinline__ uint32_t tree_word(unsigned long long mask, int r) {
  if (r <= -32) return 0xffffffffu;
  if (r < 0) return (uint32_t)(mask << -r) | ((1u << -r) - 1u);
  return r < 64 ? (uint32_t)(mask >> r) : 0u;
}
__device__ __forceinline__ unsigned long long shfl64(unsigned long long x, int lane) {
  return ((unsigned long long)__shfl_sync(0xffffffffu, (uint32_t)(x >> 32), lane) << 32) |
         __shfl_sync(0xffffffffu, (uint32_t)x, lane);
}

// Tokens lane and lane + 32 of a tree: masks of ancestors by doubling (after k rounds a token's mask holds itself and
// 2^k - 1 ancestors, `up`, their parents at first, the next one).
__device__ __forceinline__ void tree_masks(int (&up)[2], int nodes, int lane, int* status, unsigned long long (&mask)[2]) {
#pragma unroll
  for (int h = 0; h < 2; h++) {
    const int t = lane + 32 * h;
    mask[h] = t < nodes ? 1ull << t : 0ull;
    if (t >= nodes) up[h] = -1;
    if (up[h] < -1 || up[h] >= t) {
      if (status) record_tree(status);
      up[h] = -1;
    }
  }
#pragma unroll 1
  while (__any_sync(0xffffffffu, up[0] >= 0 || up[1] >= 0)) {
    unsigned long long m[2];
    int u[2];
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const int s = up[h] & 31;
      const bool high = up[h] >= 32;
      const unsigned long long m0 = shfl64(mask[0], s), m1 = shfl64(mask[1], s);
      const int u0 = __shfl_sync(0xffffffffu, up[0], s), u1 = __shfl_sync(0xffffffffu, up[1], s);
      m[h] = up[h] < 0 ? 0 : (high ? m1 : m0);
      u[h] = up[h] < 0 ? -1 : (high ? u1 : u0);
    }
#pragma unroll
    for (int h = 0; h < 2; h++) {
      mask[h] |= m[h];
      up[h] = u[h];
    }
  }
}

// N values to place `to` of o (bf16 or fp32), scaled.
template <int N>
__device__ __forceinline__ void put_columns(const PagedTreeArgs& a, size_t to, const float (&v)[N], float inv, bool live) {
  if (a.o_fp32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(a.o) + to);
#pragma unroll
    for (int e = 0; e < N / 4; e++)
      p[e] = live ? make_float4(v[4 * e] * inv, v[4 * e + 1] * inv, v[4 * e + 2] * inv, v[4 * e + 3] * inv)
                  : make_float4(0.f, 0.f, 0.f, 0.f);
  } else {
    uint4* p = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + to);
#pragma unroll
    for (int e = 0; e < N / 8; e++)
      p[e] = live ? make_uint4(pack_bf16(v[8 * e] * inv, v[8 * e + 1] * inv), pack_bf16(v[8 * e + 2] * inv, v[8 * e + 3] * inv),
                               pack_bf16(v[8 * e + 4] * inv, v[8 * e + 5] * inv), pack_bf16(v[8 * e + 6] * inv, v[8 * e + 7] * inv))
                  : make_uint4(0u, 0u, 0u, 0u);
  }
}

// RT: row tiles of a pair (2: more than 128 rows). SPLIT: at most 64 rows, two lanes each (see above). FULL: o is
// float32, and the weights have a third part (2^-25; two are 2^-17 off, an eighth of a bf16 o's rounding but ten
// times what fp32 sums are off).
template <int D, int RT, bool SPLIT, bool FULL>
__global__ void __launch_bounds__(kTreeThreads, 1) k_tree_sweep(const __grid_constant__ PagedTreeArgs a) {
  using C = TreeCfg<D>;
  constexpr int SK = C::kKStages, SV = C::kVStages, TB = C::kTileBytes;
  constexpr int NR = SPLIT ? kTile / 2 : kTile;  // rows of a tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* head = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* q_full = reinterpret_cast<uint64_t*>(head);  // [2] the slot's queries are packed
  uint64_t* k_full = q_full + 2;           // [SK]
  uint64_t* k_empty = k_full + SK;         // [SK] the last S = Q K^T of the stage has completed
  uint64_t* v_full = k_empty + SK;         // [SV]
  uint64_t* v_empty = v_full + SV;         // [SV] the O += P V of the stage have completed
  uint64_t* s_full = v_empty + SV;         // [group][2] the group's steps in turn
  uint64_t* p_ready = s_full + 4;          // [group][2][2] weights of the tile's last 64 keys, and of the first (SPLIT: all)
  // [3] per buffer of S and P its weights are read (FULL: [group]); SPLIT, not FULL: [group] the scores are in registers
  uint64_t* pv_done = p_ready + 8;
  uint64_t* o_done = pv_done + 3;          // [group][2] the group's steps in turn: O has the step
  uint64_t* part_full = o_done + 4;        // [group][4] the other group is done with a segment that this one finishes
  uint64_t* o_read = part_full + 8;        // [group] the group's O of such a segment has been read by the other
  uint64_t* drain = o_read + 2;             // [3] per issuing thread
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(head + kTreeVars);
  volatile int* abort = reinterpret_cast<volatile int*>(head + kTreeVars) + 1;
  volatile SweepPlan* splan = reinterpret_cast<volatile SweepPlan*>(head + kTreePlan);
  int* wsum = reinterpret_cast<int*>(head + kTreeSums);
  // [kTrees] segments in turn. Scores wait for the weights three steps before, so while a group packs segment e + 2 (the
  // last scores of e are there) the other may still read the tree of e - 2, e - 1 or e.
  TreeInfo* info = reinterpret_cast<TreeInfo*>(head + kTreeInfo);
  float2* ml_other = reinterpret_cast<float2*>(head + kTreeMl);    // [4][128] segments in turn
  int* cum = reinterpret_cast<int*>(head + kTreeCum);
  uint8_t* pad = reinterpret_cast<uint8_t*>(cum + a.B + 1);  // positions that a sequence's last tile lacks
  uint8_t* smem = head + tree_head(a.B);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, blk = (int)blockIdx.x;
  if (tid == 0) {
    *abort = 0;
    for (int k = 0; k < 2; k++) {
      mbar_init(q_full + k, RT * 4);  // the warps that pack a row tile
      mbar_init(o_read + k, 4);
    }
    for (int k = 0; k < SK; k++) {
      mbar_init(k_full + k, 1);
      mbar_init(k_empty + k, 1);
    }
    for (int k = 0; k < SV; k++) {
      mbar_init(v_full + k, 1);
      mbar_init(v_empty + k, RT);  // one for each row tile of the pair
    }
    for (int k = 0; k < 4; k++) {
      mbar_init(s_full + k, 2);
      mbar_init(p_ready + 2 * k, 4);
      mbar_init(p_ready + 2 * k + 1, 4);
      mbar_init(o_done + k, 1);
      mbar_init(part_full + k, 4);
      mbar_init(part_full + 4 + k, 4);
    }
    for (int k = 0; k < 3; k++) {
      mbar_init(pv_done + k, SPLIT && !FULL ? 4 : 1);
      mbar_init(drain + k, 1);
    }
    fence_mbar_init();
  }
  pdl_wait();  // before the tensor memory is taken: the kernel in front may still need some
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  running_costs<kTreeThreads>(a.B, cum, wsum, tid, [&](int b) {
    const TreeShape x = tree_shape(a, b, blk == 0);
    const int nt = max(1, (x.len + kTile - 1) / kTile);  // one even where nothing is read: its rows are written
    pad[b] = (uint8_t)(nt * kTile - x.len);
    return kTreeOver + nt;
  });
  Tiles tl;
  tl.cum = cum;
  tl.B = a.B;
  tl.Hkv = a.Hkv * a.pairs;
  tl.over = kTreeOver;
  tl.whole = kTreeWhole;
  divide_work(tl, splan, blk, (int)gridDim.x, kTreeSlack, warp, lane,
              [&](int W, int) { return (int)fdiv((uint32_t)W, a.div_grid); });
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const volatile int never = 0;
  SegWalk<kTreeOver> sw;
  sw.init(tl, splan);
  const auto head_of = [&](int g) { return RT == 1 ? g : g / a.pairs; };  // (up to 128 rows are one pair)
  const auto pair_of = [&](int g) { return RT == 1 ? 0 : g % a.pairs; };
  const auto units = [&](const SegWalk<kTreeOver>& x) {  // row tiles of the segment's pair
    return RT == 1 ? 1 : (2 * (pair_of(x.g)) * kTile + kTile < a.R ? 2 : 1);
  };
  const auto slot_of = [](int e) { return RT == 1 ? e & 1 : 0; };
  const auto use_of = [](int e) { return RT == 1 ? e >> 1 : e; };
  // registers: 384 x 168 at launch; 128 x 120 + 256 x 192, with O in registers 128 x 72 + 256 x 216
  if (warp < 4) regs_dec<FULL ? 72 : 120>();
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      prefetch_tmap(&a.map_pk);
      prefetch_tmap(&a.map_pv);
    }
    const uint64_t policy = evict_first();
    const int prows = min(1 << a.page_shift, kTile), per = kTile / prows;
    const uint32_t pbytes = (uint32_t)prows * C::kSpan;
    // Page numbers 32 at a time, one to a lane, a window ahead; behind the last position num_pages, outside the
    // pool, which is read as zeros.
    const auto window = [&](const SegWalk<kTreeOver>& x, int w) {
      const int i = w * 32 + lane;
      return (i << a.page_shift) < x.nt * kTile - pad[x.b] ? a.table[(size_t)x.b * a.max_pages + i] : a.num_pages;
    };
    const auto page_of = [&](int n) { return (n * kTile) >> a.page_shift; };
    SegWalk<kTreeOver> ls = sw;  // the segment of the next window
    bool lon = ls.next();
    int lw = 0, id = 0, nid = 0;
    if (lon) {
      lw = page_of(ls.n0) >> 5;
      nid = window(ls, lw);
    }
    const auto look = [&]() {
      id = nid;  // looked at only now: the next window's are still on their way
      if (id < 0 || id > a.num_pages || (id == a.num_pages && (lw * 32 + lane) << a.page_shift < ls.nt * kTile - pad[ls.b])) {
        record_page(a.status);
        id = a.num_pages;
      }
      if (!lon) return;
      if (lw < page_of(ls.n1 - 1) >> 5) {
        lw++;
      } else {
        lon = ls.next();
        if (lon) lw = page_of(ls.n0) >> 5;
      }
      if (lon) nid = window(ls, lw);
    };
    SweepPlan plan;
    plan.base = splan->base;
    plan.rem = splan->rem;
    plan.slack = splan->slack;
    int4 cut = make_int4(-1, 0, 0, 0);
    bool ok = true;
    int k = 0;  // tiles so far
    while (ok && sw.next()) {
      const int kvh = head_of(sw.g);
      if (sw.n1 < sw.nt) {  // a cut one that begins here, or goes through the whole stretch
        const int s0 = cum[sw.b] * tl.Hkv + sw.g * (sw.nt + tl.over);
        cut = make_int4(sw.b, sw.g, sw.n0 == 0 ? blk : tl.first(plan, s0), tl.last(plan, s0, sw.nt));
      }
      int win = -1;
#pragma unroll 1
      for (int n = sw.n0; ok && n < sw.n1; n++, k++) {
        const int first = page_of(n);
        if ((first >> 5) != win) {
          win = first >> 5;
          look();
        }
        const int mine = __shfl_sync(0xffffffffu, id, (first & 31) + (lane < per ? lane : 0));
        const int off = (n * kTile) & ((1 << a.page_shift) - 1);
        const bool again = RT == 2 && a.pairs > 1;  // the other pairs read it too
        const auto load = [&](const CUtensorMap* map, uint8_t* to, uint64_t* full, uint64_t* empty, int use) {
          if (use > 0) ok = __all_sync(0xffffffffu, tree_wait(empty, (use - 1) & 1, abort));
          if (!ok) return;
          if (lane == 0) mbar_arrive_expect_tx(full, TB);
          __syncwarp();
          if (lane < per) {
            if (again)
              tma_load_4d(to + lane * pbytes, map, full, 0, off, kvh, mine);
            else
              tma_load_4d(to + lane * pbytes, map, full, 0, off, kvh, mine, policy);
          }
        };
        load(&a.map_pk, smem + C::kOffK + k % SK * TB, k_full + k % SK, k_empty + k % SK, k / SK);
        if (!ok) {
          // V of this tile is not on its way: below, only what is
          for (int x = k - SK < 0 ? 0 : k - SK; lane == 0 && x < k; x++) tree_wait(k_full + x % SK, (x / SK) & 1, &never);
          for (int x = k - SV < 0 ? 0 : k - SV; lane == 0 && x < k; x++) tree_wait(v_full + x % SV, (x / SV) & 1, &never);
          break;
        }
        load(&a.map_pv, smem + C::kOffV + k % SV * TB, v_full + k % SV, v_empty + k % SV, k / SV);
        if (!ok) {
          const int k0 = k - SK + 1 < 0 ? 0 : k - SK + 1;
          for (int x = k0; lane == 0 && x <= k; x++) tree_wait(k_full + x % SK, (x / SK) & 1, &never);
          for (int x = k - SV < 0 ? 0 : k - SV; lane == 0 && x < k; x++) tree_wait(v_full + x % SV, (x / SV) & 1, &never);
          break;
        }
      }
    }
    if (lane == 0) {
      a.cut[blk] = cut;
      if (!ok) {
        *abort = 1;
        atomicExch(a.status, kStatusTimeout);
      } else {
        // let every copy issued above land before the block can exit
        for (int x = k - SK < 0 ? 0 : k - SK; x < k; x++) tree_wait(k_full + x % SK, (x / SK) & 1, &never);
        for (int x = k - SV < 0 ? 0 : k - SV; x < k; x++) tree_wait(v_full + x % SV, (x / SV) & 1, &never);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ S = Q K^T issuer
    if (lane == 0) {
      constexpr uint32_t idS = idesc_fp16(128, 128, false, false);
      constexpr uint32_t kStepK = 32 >> 4, tstep = (uint32_t)TB >> 4;
      const uint64_t dQ0 = smem_desc(smem_u32(smem), 16, C::kSBO, C::kSwz);
      const uint64_t dK0 = smem_desc(smem_u32(smem + C::kOffK), 16, C::kSBO, C::kSwz);
      bool ok = true;
      int n = 0, k = 0, e = 0;  // steps, tiles, segments
      while (ok && sw.next()) {
        const int nu = units(sw), slot = slot_of(e);
        if (!(ok = tree_wait(q_full + slot, use_of(e) & 1, abort))) break;
#pragma unroll 1
        for (int i = sw.n0; ok && i < sw.n1; i++, k++) {
          const int st = k % SK;
          if (!(ok = tree_wait(k_full + st, (k / SK) & 1, abort))) break;
#pragma unroll 1
          for (int u = 0; u < nu; u++, n++) {
            // the buffer's weights have been read (SPLIT, not FULL: the group's scores)
            const int buf = SPLIT || FULL ? n & 1 : n % 3, use = SPLIT || FULL ? n >> 1 : n / 3;
            if (use > 0 && !(ok = tree_wait(pv_done + buf, (use - 1) & 1, abort))) break;
            tc_fence_after();
            const uint64_t dq = dQ0 + (uint64_t)((RT == 1 ? 2 * slot : 2 * u) * tstep), dk = dK0 + (uint64_t)(st * tstep);
            const uint32_t to = tmem + C::kColS + 128u * buf;
            mma_ss_chain<D / 16>(to, dq, kStepK, dk, kStepK, idS, 0u);
            mma_ss_chain<D / 16>(to, dq + (uint64_t)tstep, kStepK, dk, kStepK, idS, 1u);
            uint64_t* full = s_full + 2 * (n & 1) + ((n >> 1) & 1);
            mma_commit(full);
            mbar_arrive(full);  // what this thread has seen (the tree of the segment) comes with it
          }
          if (ok) mma_commit(k_empty + st);
        }
        e++;
      }
      if (!ok) {
        *abort = 1;
        atomicExch(a.status, kStatusTimeout);
      }
      mma_commit(drain);
      tree_wait(drain, 0, &never);
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------ O += P V issuer of a group
    if (lane == 0) {
      const int grp = warp - 2;
      constexpr uint32_t idPV = idesc_bf16(128, D, false, true);
      constexpr uint32_t kStepMN = (16 * C::kSpan) >> 4, tstep = (uint32_t)TB >> 4;
      const uint64_t dV0 = smem_desc(smem_u32(smem + C::kOffV), 16, C::kSBO, C::kSwz);
      const uint32_t o = tmem + C::kColO + 64u * grp;
      bool ok = true, lent = false;  // the other group reads O of the last segment
      int n = 0, k = 0, reads = 0;
      while (ok && sw.next()) {
        const int nu = units(sw), first = n, tiles = sw.n1 - sw.n0, end = first + tiles * nu;
#pragma unroll 1
        for (n = first + ((first ^ grp) & 1); n < end; n += 2) {
          const int kt = k + (RT == 2 && nu == 2 ? (n - first) >> 1 : n - first), st = kt % SV, i = n >> 1;
          // the group has also read the O of its last segment before it arrives for this one
          uint64_t* ready = p_ready + 4 * grp + 2 * (i & 1);
          if (!(ok = tree_wait(ready, (i >> 1) & 1, abort))) break;
          if (!(ok = tree_wait(v_full + st, (kt / SV) & 1, abort))) break;
          if (lent) {
            if (!(ok = tree_wait(o_read + grp, reads++ & 1, abort))) break;
            lent = false;
          }
          const uint64_t dv = dV0 + (uint64_t)(st * tstep), dv2 = dv + (uint64_t)(4 * kStepMN);
          const uint32_t sb = tmem + C::kColS + 128u * (FULL ? grp : n % 3), pb = tmem + C::kColP + 64u * grp;
          const uint32_t p = SPLIT ? pb : sb, third = SPLIT ? sb : pb;
          constexpr uint32_t kHalf = SPLIT ? 32u : 64u;  // columns of P for 64 keys
          tc_fence_after();
          mma_ts_chain<4, false>(o, p + kHalf, dv2, kStepMN, idPV, !FULL && n - first >= 2 ? 1u : 0u);
          if (!SPLIT) {
            mma_ts_chain<4, false>(o, p + kHalf + 32u, dv2, kStepMN, idPV, 1u);
            if (!(ok = tree_wait(ready + 1, (i >> 1) & 1, abort))) break;
            tc_fence_after();
          }
          mma_ts_chain<4, false>(o, p, dv, kStepMN, idPV, 1u);
          if (!SPLIT) mma_ts_chain<4, false>(o, p + 32u, dv, kStepMN, idPV, 1u);
          if (FULL) {
            mma_ts_chain<4, false>(o, third + 32u, dv2, kStepMN, idPV, 1u);
            mma_ts_chain<4, false>(o, third, dv, kStepMN, idPV, 1u);
          }
          if (!SPLIT || FULL) mma_commit(pv_done + (FULL ? grp : n % 3));
          mma_commit(o_done + 2 * grp + (i & 1));
          mma_commit(v_empty + st);
          if (RT == 2 && nu == 1) mbar_arrive(v_empty + st);
        }
        lent = lent || (nu == 1 && tiles >= 2 && ((end - 1) & 1) != grp);
        n = end;
        k += tiles;
      }
      if (!ok) {
        *abort = 1;
        atomicExch(a.status, kStatusTimeout);
      }
      mma_commit(drain + 1 + grp);
      tree_wait(drain + 1 + grp, 0, &never);
    }
  } else {
    // ------------------------------------------------------------ softmax group
    regs_inc<FULL ? 216 : 192>();
    const int grp = (warp - 4) >> 2, q4 = warp & 3;
    const int r = q4 * 32 + lane, rr = SPLIT ? q4 * 16 + (lane & 15) : r;  // lane of the tile and its row
    const uint32_t trow = tmem + ((uint32_t)(q4 * 32) << 16);
    const uint32_t obuf = trow + C::kColO + 64u * grp;
    const float sl2 = a.scale_log2;
    uint4 wv = make_uint4(0, 0, 0, 0);
    // This group packs row tile u of a segment, number e of the block, and signals it `times` times.
    const auto pack = [&](const SegWalk<kTreeOver>& x, int e, int u, int times) {
      constexpr int kCPR = D / 8, kItems = NR * kCPR / 128, kBatch = kItems < 4 ? kItems : 4;  // 16-byte chunks of a thread
      const int pr = pair_of(x.g), g = head_of(x.g), c = lane % kCPR, r0 = pr * 2 * kTile + u * kTile;
      uint8_t* to = smem + (RT == 1 ? 2 * slot_of(e) : 2 * u) * TB;
      const int total = x.nt * kTile - pad[x.b];
      int up[2];
#pragma unroll
      for (int h = 0; h < 2; h++) up[h] = lane + 32 * h < a.Tq ? a.parents[x.b * a.parent_stride + lane + 32 * h] : -1;
      const int nodes = total > 0 ? (a.nodes ? a.nodes[x.b] : a.Tq) : 0;
      TreeInfo& tree = info[(unsigned)e % kTrees];
      if (a.qw) wv = load_rope_chunk<D>(a.qw, c, a.rope_half != 0);
      unsigned long long mask[2];
      tree_masks(up, nodes, lane, q4 == 0 ? a.status : nullptr, mask);
      const int depth[2] = {__popcll(mask[0]) - 1, __popcll(mask[1]) - 1};
      if (q4 == 0) {
        tree.mask[lane] = mask[0];
        tree.mask[lane + 32] = mask[1];
        if (lane == 0) {
          tree.ctx = total - nodes;
          tree.nodes = nodes;
        }
      }
#pragma unroll 1
      for (int i0 = 0; i0 < kItems; i0 += kBatch) {
        QueryChunk q[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; i++) {
          const int rt = ((i0 + i) * 128 + r) / kCPR, row = r0 + rt, t = row < a.R ? (int)fdiv((uint32_t)row, a.div_g) : 0;
          const int d0 = __shfl_sync(0xffffffffu, depth[0], t & 31), d1 = __shfl_sync(0xffffffffu, depth[1], t & 31);
          q[i] = query_load_at<D>(a, row < a.R && t < nodes, x.b, g, row, t, c, total - nodes + (t < 32 ? d0 : d1));
        }
#pragma unroll
        for (int i = 0; i < kBatch; i++) {
          const int rt = ((i0 + i) * 128 + r) / kCPR;
          uint4 hi, lo;
          query_finish<D>(a, q[i], a.qw != nullptr, wv, hi, lo);
          const uint32_t at = swz(SPLIT ? 32 * (rt / 16) + rt % 16 : rt, c, C::kSpan);
          *reinterpret_cast<uint4*>(to + at) = hi;
          *reinterpret_cast<uint4*>(to + TB + at) = lo;
        }
      }
      fence_proxy_async_smem();
      for (int i = 0; i < times; i++) warp_arrive(q_full + slot_of(e));
    };
    // Segments are packed two ahead where two have slots of their own (RT == 1), else one.
    constexpr int kAhead = RT == 1 ? 2 : 1;
    // The walks to the segment that is worked off and to the one that is packed lie in shared memory (the warp's own): the
    // steps between need the registers.
    volatile int* walk = reinterpret_cast<volatile int*>(head + kTreeWalk) + (warp - 4) * 12;
    const auto put = [&](const SegWalk<kTreeOver>& x, int i) {
      __syncwarp();
      if (lane == 0) {
        walk[6 * i] = x.w;
        walk[6 * i + 1] = x.b;
        walk[6 * i + 2] = x.g;
        walk[6 * i + 3] = x.n0;
        walk[6 * i + 4] = x.n1;
        walk[6 * i + 5] = x.nt;
      }
      __syncwarp();
    };
    const auto get = [&](int i) {
      SegWalk<kTreeOver> x;
      x.cum = cum;
      x.Hkv = tl.Hkv;
      x.end = splan->end;
      x.w = walk[6 * i];
      x.b = walk[6 * i + 1];
      x.g = walk[6 * i + 2];
      x.n0 = walk[6 * i + 3];
      x.n1 = walk[6 * i + 4];
      x.nt = walk[6 * i + 5];
      return x;
    };
    put(sw, 0);
    put(sw, 1);
    bool qon = true;
    bool ok = true;
    int n = 0, kt = 0;                 // steps, stages
    int joined0 = 0, joined1 = 0;      // segments that each group finished with the other
    for (int e = -kAhead; ok; e++) {
      int pack0 = 0, pack1 = 0, times = 1;  // this group packs row tiles pack0 .. pack1 - 1 of segment e + kAhead
      if (qon) {
        SegWalk<kTreeOver> qs = get(1);
        qon = qs.next();
        put(qs, 1);
      }
      if (e < 0) {
        if (!qon) continue;
        if (RT == 1) {
          pack1 = grp == e + kAhead ? 1 : 0;
        } else {
          const int next = units(get(1));
          pack0 = grp;
          pack1 = min(grp + 1, next);
          times = next == 2 ? 1 : 2;
        }
      } else {
        SegWalk<kTreeOver> sw = get(0);
        if (!sw.next()) break;
        put(sw, 0);
        const int n0 = sw.n0, nu = units(sw), first = n, end = first + (sw.n1 - sw.n0) * nu;
        const int mine = first + ((first ^ grp) & 1);           // this group's first step
        const bool joint = nu == 1 && end - first >= 2;         // both groups have a part of the same rows
        const int last = (end - 1) & 1;                         // the group of the last step
        const int k0 = kt;
        n = end;
        kt += sw.n1 - sw.n0;
        const int turn = last ? joined1 : joined0;
        if (joint) last ? joined1++ : joined0++;
        const int u = nu == 2 ? (mine - first) & 1 : 0;
        if (mine < end) {
          const auto token = [&](int x) { return x < a.R ? (int)fdiv((uint32_t)x, a.div_g) : kTreeMax; };
          const TreeInfo& tree = info[(unsigned)e % kTrees];
          const auto row_of = [&](int x) { return pair_of(get(0).g) * 2 * kTile + u * kTile + x; };  // row of the (sequence, head)
          int ctx = 0;
          bool live = false;
          // a thread's row, or (SPLIT) its two rows lane / 4 and lane / 4 + 8 of the warp's 16: maximum, sum
          constexpr int NQ = SPLIT ? 2 : 1;
          float r_run[NQ], l_run[NQ];
          float acc[FULL ? D : 1];  // FULL: O of the lane's row so far
#pragma unroll
          for (int x = 0; FULL && x < D; x++) acc[x] = 0.f;
          // FULL: adds the O of step n to it, then scales both
          const auto flush = [&](int n, float f) {
            if (!__all_sync(0xffffffffu, tree_wait(o_done + 2 * grp + ((n >> 1) & 1), (n >> 2) & 1, abort))) return false;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < (FULL ? D / 16 : 0); c++) {
              uint32_t w[16];
              tmem_ld16(obuf + c * 16, w);
              tmem_wait_ld();
#pragma unroll
              for (int x = 0; x < 16; x++) {
                float& y = acc[FULL ? 16 * c + x : 0];
                y = (y + __uint_as_float(w[x])) * f;
              }
            }
            return true;
          };
          int s = mine;
          for (; s < end; s += 2) {
            const int buf = SPLIT || FULL ? grp : s % 3, tile = n0 + (nu == 2 ? (s - first) >> 1 : s - first);
            const uint32_t sbuf = trow + C::kColS + 128u * buf, pown = trow + C::kColP + 64u * grp;
            const uint32_t pbuf = SPLIT ? pown : sbuf, third = SPLIT ? sbuf : pown;
            ok = __all_sync(0xffffffffu, tree_wait(s_full + 2 * grp + ((s >> 1) & 1), (s >> 2) & 1, abort));
            if (!ok) break;
            tc_fence_after();
            if (s == mine) {
              ctx = tree.ctx;
              live = token(row_of(rr)) < tree.nodes;
            }
            const bool edge = (tile + 1) * kTile > ctx;  // the tile ends in the tree or behind it
            // What a row does not see becomes -infinity: a lane's scores where they lie, SPLIT a thread's once it has them (less
            // code in a step against a trip to TMEM in the last ones: 64 trees of 32 54.4 -> 53.4 us; 16 of 16 32.6 -> 33.1).
            unsigned long long mask[NQ];
            if (edge) {
              const int nodes = tree.nodes, row0 = row_of(0), past = ctx + nodes - tile * kTile;
#pragma unroll
              for (int i = 0; i < NQ; i++) {
                const int t = token(row0 + (SPLIT ? q4 * 16 + lane / 4 + 8 * i : r));
                mask[i] = t < nodes ? tree.mask[t] : 0ull;
              }
#pragma unroll 1
              for (int c = SPLIT ? kTile / 16 : max(0, ctx - tile * kTile) / 16; c < kTile / 16; c++) {
                const uint32_t see = tree_word(mask[0], tile * kTile + c * 16 - ctx);
                uint32_t w[16];
                tmem_ld16(sbuf + c * 16, w);
                tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < 16; x++)
                  if (!(see & (1u << x))) w[x] = 0xff800000u;
                tmem_st16(sbuf + c * 16, w);
              }
              if (!SPLIT) tmem_wait_st();
              if (past < kTile) {
                // what lies behind the last position may be anything: its weight is 0, but 0 times a NaN is not
                const int kt = k0 + tile - n0;
                ok = __all_sync(0xffffffffu, tree_wait(v_full + kt % SV, (kt / SV) & 1, abort));
                if (!ok) break;
                if (r >= past) {
                  uint4* v = reinterpret_cast<uint4*>(smem + C::kOffV + kt % SV * TB + r * C::kSpan);
#pragma unroll
                  for (int c = 0; c < D / 8; c++) v[c] = make_uint4(0u, 0u, 0u, 0u);
                  fence_proxy_async_smem();
                }
              }
            }
            // 64 scores of a thread at a time. With one row and 128 they are read once for the maximum and (but for the last 64)
            // once more for the weights: with all in registers the loop does not fit the schedulers' instruction caches
            // (warps then wait for instructions longer than they issue them).
            uint32_t sc[64];
            const auto load = [&](int h) {
              uint32_t(&lo)[32] = *reinterpret_cast<uint32_t(*)[32]>(sc);
              uint32_t(&hi)[32] = *reinterpret_cast<uint32_t(*)[32]>(sc + 32);
              if (SPLIT) {
                tmem_ld16x64(sbuf, lo);
                tmem_ld16x64(sbuf + 64, hi);
              } else {
                tmem_ld32(sbuf + h * 64, lo);
                tmem_ld32(sbuf + h * 64 + 32, hi);
              }
              tmem_wait_ld();
              if (SPLIT && edge) {
#pragma unroll
                for (int c = 0; c < 4; c++) {
                  const int at = tile * kTile + c * 32 - ctx;
                  const int by = 2 * (lane & 3);
                  const uint32_t see[2] = {tree_word(mask[0], at) >> by, tree_word(mask[NQ - 1], at) >> by};
#pragma unroll
                  for (int x = 0; x < 16; x++)  // columns 8 (x / 4) + 2 (lane % 4) + x % 2 of the 32, row x / 2 % 2
                    if (!(see[x / 2 % 2] & (1u << (8 * (x / 4) + x % 2)))) sc[16 * c + x] = 0xff800000u;
                }
              }
            };
            float mxr[NQ];
            if (SPLIT) {
              load(0);
              if (!FULL) {
                tc_fence_before();
                warp_arrive(pv_done + grp);
              }
              float m2[2][2] = {{-INFINITY, -INFINITY}, {-INFINITY, -INFINITY}};
#pragma unroll
              for (int x = 0; x < 64; x += 2) {
                float& y = m2[(x >> 1) & 1][(x >> 2) & 1];
                y = fmax3(y, __uint_as_float(sc[x]), __uint_as_float(sc[x + 1]));
              }
#pragma unroll
              for (int i = 0; i < NQ; i++) {
                float m = fmaxf(m2[i][0], m2[i][1]);
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                mxr[i] = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
              }
            } else {
              float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
              for (int h = 0; h < 2; h++) {
                load(h);
#pragma unroll
                for (int x = 0; x < 64; x += 2)
                  mx4[(x >> 1) & 3] = fmax3(mx4[(x >> 1) & 3], __uint_as_float(sc[x]), __uint_as_float(sc[x + 1]));
              }
              mxr[0] = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
            }
            float alpha[NQ];
            if (s == mine) {
#pragma unroll
              for (int i = 0; i < NQ; i++) {
                r_run[i] = mxr[i];
                alpha[i] = 0.f;
                l_run[i] = 0.f;
              }
            } else {
              // O and the sum follow the maximum only when some row's grew by more than 2^8 (or came out of nothing)
              bool grow = false;
#pragma unroll
              for (int i = 0; i < NQ; i++) {
                alpha[i] = 1.f;
                grow = grow || __fmul_rn(fmaxf(r_run[i], mxr[i]), sl2) > __fmul_rn(r_run[i], sl2) + 8.0f;
              }
              float lane_a = 1.f;  // of the lane's row
              if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int i = 0; i < NQ; i++) {
                  const float r_new = fmaxf(r_run[i], mxr[i]);
                  alpha[i] = r_run[i] == -INFINITY ? 0.f : ex2(__fmul_rn(r_run[i], sl2) - __fmul_rn(r_new, sl2));
                  r_run[i] = r_new;
                }
                lane_a = alpha[0];
                if (SPLIT) {
                  const float x = __shfl_sync(0xffffffffu, alpha[0], 4 * (lane & 7));
                  const float y = __shfl_sync(0xffffffffu, alpha[NQ - 1], 4 * (lane & 7));
                  lane_a = lane & 8 ? y : x;
                }
                if (!FULL) {
                  ok = __all_sync(0xffffffffu, tree_wait(o_done + 2 * grp + (((s - 2) >> 1) & 1), ((s - 2) >> 2) & 1, abort));
                  if (!ok) break;
                  tc_fence_after();
#pragma unroll 1
                  for (int c = 0; c < D / 16; c++) {
                    uint32_t w[16];
                    tmem_ld16(obuf + c * 16, w);
                    tmem_wait_ld();
#pragma unroll
                    for (int x = 0; x < 16; x++) w[x] = __float_as_uint(__uint_as_float(w[x]) * lane_a);
                    tmem_st16(obuf + c * 16, w);
                  }
                }
              }
              if (FULL && !(ok = flush(s - 2, lane_a))) break;
            }
            if (SPLIT ? s >= 2 : FULL && s >= 2 && s == mine) {  // the weights of the step before have been read
              ok = __all_sync(0xffffffffu, tree_wait(o_done + 2 * grp + (((s - 2) >> 1) & 1), ((s - 2) >> 2) & 1, abort));
              if (!ok) break;
              tc_fence_after();
            }
            uint64_t sum[NQ][4 / NQ], negm[NQ];
#pragma unroll
            for (int i = 0; i < NQ; i++) {
              const float m = r_run[i] == -INFINITY ? 0.f : __fmul_rn(r_run[i], sl2);
              negm[i] = f2(-m, -m);
#pragma unroll
              for (int j = 0; j < 4 / NQ; j++) sum[i][j] = 0ull;
            }
            const uint64_t sl2x2 = f2(sl2, sl2), minus = f2(-1.f, -1.f);
#pragma unroll 1
            for (int h = 1; h >= (SPLIT ? 1 : 0); h--) {
              if (h == 0) load(0);
              uint32_t ph[32], pl[32], pt[32];
#pragma unroll
              for (int x = 0; x < 32; x++) {
                constexpr int kSums = 4 / NQ;
                const int i = SPLIT ? x & 1 : 0, j = (SPLIT ? x >> 1 : x) % kSums;
                float x0, x1, l0, l1;
                f2_split(f2_fma(f2(__uint_as_float(sc[2 * x]), __uint_as_float(sc[2 * x + 1])), sl2x2, negm[i]), x0, x1);
                const uint64_t pp = f2(ex2(x0), ex2(x1));
                f2_split(pp, x0, x1);
                ph[x] = pack_bf16(x0, x1);
                const uint64_t ll = f2_fma(f2(bf_lo(ph[x]), bf_hi(ph[x])), minus, pp);
                f2_split(ll, l0, l1);
                pl[x] = pack_bf16(l0, l1);
                if (FULL) {
                  f2_split(f2_fma(f2(bf_lo(pl[x]), bf_hi(pl[x])), minus, ll), l0, l1);
                  pt[x] = pack_bf16(l0, l1);
                }
                sum[i][j] = f2_add(sum[i][j], pp);
                if (!SPLIT && x % 8 == 7) {
                  tmem_st8(pbuf + 64 * h + x - 7, *reinterpret_cast<uint32_t(*)[8]>(ph + x - 7));
                  tmem_st8(pbuf + 64 * h + 32 + x - 7, *reinterpret_cast<uint32_t(*)[8]>(pl + x - 7));
                  if (FULL) tmem_st8(third + 32 * h + x - 7, *reinterpret_cast<uint32_t(*)[8]>(pt + x - 7));
                }
                if (SPLIT && x % 16 == 15) {
                  tmem_st16x32(pbuf + 2 * (x - 15), *reinterpret_cast<uint32_t(*)[16]>(ph + x - 15));
                  tmem_st16x32(pbuf + (16u << 16) + 2 * (x - 15), *reinterpret_cast<uint32_t(*)[16]>(pl + x - 15));
                  if (FULL) {  // beside the low parts
                    const uint32_t none[16] = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
                    tmem_st16x32(third + 2 * (x - 15), none);
                    tmem_st16x32(third + (16u << 16) + 2 * (x - 15), *reinterpret_cast<uint32_t(*)[16]>(pt + x - 15));
                  }
                }
              }
              tmem_wait_st();
              tc_fence_before();
              warp_arrive(p_ready + 4 * grp + 2 * ((s >> 1) & 1) + (h == 0 ? 1 : 0));
            }
#pragma unroll
            for (int i = 0; i < NQ; i++) {
              uint64_t t = f2_add(sum[i][0], sum[i][1]);
              if (NQ == 1) t = f2_add(t, f2_add(sum[i][4 / NQ - 2], sum[i][4 / NQ - 1]));
              float x, y;
              f2_split(t, x, y);
              l_run[i] = fmaf(l_run[i], alpha[i], x + y);
            }
          }
          if (!ok) break;
          float lane_m = r_run[0], lane_l = l_run[0];  // of the lane's row
          if (SPLIT) {
            float m2[2], l2[2];
#pragma unroll
            for (int i = 0; i < NQ; i++) {
              float l = l_run[i];
              l += __shfl_xor_sync(0xffffffffu, l, 1);
              l += __shfl_xor_sync(0xffffffffu, l, 2);
              l2[i] = __shfl_sync(0xffffffffu, l, 4 * (lane & 7));
              m2[i] = __shfl_sync(0xffffffffu, r_run[i], 4 * (lane & 7));
            }
            lane_m = lane & 8 ? m2[1] : m2[0];
            lane_l = lane & 8 ? l2[1] : l2[0];
          }
          lane_m = lane_m == -INFINITY ? 0.f : __fmul_rn(lane_m, sl2);
          sw = get(0);
          const int row = row_of(rr);
          // the segment's unnormalised O, maximum (log2 units) and sum
          if (FULL) {
            if (!(ok = flush(s - 2, 1.f))) break;
#pragma unroll
            for (int c = 0; c < (FULL ? D / 16 : 0); c++) {
              uint32_t w[16];
#pragma unroll
              for (int x = 0; x < 16; x++) w[x] = __float_as_uint(acc[FULL ? 16 * c + x : 0]);
              tmem_st16(obuf + c * 16, w);
            }
            tmem_wait_st();
          }
          if (joint && grp != last) {
            // the other group reads this one's O where it is
            ml_other[(e & 3) * kTile + r] = make_float2(lane_m, lane_l);
            tc_fence_before();
            warp_arrive(part_full + 4 * last + (turn & 3));
          } else {
            const auto done = [&](int g, int n) {
              return __all_sync(0xffffffffu, tree_wait(o_done + 2 * g + ((n >> 1) & 1), (n >> 2) & 1, abort));
            };
            if (!(ok = done(grp, s - 2))) break;
            const bool whole = sw.n0 == 0 && sw.n1 == sw.nt;
            const size_t part = (size_t)(2 * blk + (sw.n0 > 0 ? 0 : 1)) * a.rows + u * kTile + rr;
            const int g = head_of(sw.g), t = row < a.R ? (int)fdiv((uint32_t)row, a.div_g) : 0, h = g * a.G + (row - t * a.G);
            float M = lane_m, L = lane_l, mine_f = 1.f, other_f = 0.f;
            if (joint) {
              ok = __all_sync(0xffffffffu, tree_wait(part_full + 4 * grp + (turn & 3), (turn >> 2) & 1, abort));
              if (!ok || !(ok = done(grp ^ 1, end - 2))) break;
              const float2 z = ml_other[(e & 3) * kTile + r];
              M = L == 0.f ? z.x : (z.y == 0.f ? M : fmaxf(M, z.x));
              mine_f = L == 0.f ? 0.f : ex2(lane_m - M);
              other_f = z.y == 0.f ? 0.f : ex2(z.x - M);
              L = fmaf(L, mine_f, z.y * other_f);
            }
            tc_fence_after();
            const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll 1
            for (int c = 0; c < D / 16; c++) {
              uint32_t w[16], x[16];
              float v[16];
              tmem_ld16(obuf + c * 16, w);
              if (joint) tmem_ld16(trow + C::kColO + 64u * (grp ^ 1) + c * 16, x);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; i++) {
                v[i] = __uint_as_float(w[i]) * mine_f;
                if (joint) v[i] = fmaf(__uint_as_float(x[i]), other_f, v[i]);
                if (SPLIT) v[i] += __shfl_xor_sync(0xffffffffu, v[i], 16);  // a row's two lanes, each of which writes half
              }
              if (row < a.R && !(SPLIT && (c < D / 32) != (lane < 16))) {
                if (whole) {
                  put_columns(a, (((size_t)sw.b * a.Tq + t) * a.Hq + h) * D + c * 16, v, inv, live);
                } else {
                  float4* to = reinterpret_cast<float4*>(a.part_o + part * D) + c * 4;
#pragma unroll
                  for (int q = 0; q < 4; q++)
                    to[q] = live ? make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
                }
              }
              __syncwarp();
            }
            tc_fence_before();
            if (joint) warp_arrive(o_read + (grp ^ 1));
            if (row < a.R && !(SPLIT && lane >= 16)) {
              if (!whole)
                a.part_ml[part] = make_float2(M, live ? L : 0.f);
              else if (a.lse)
                a.lse[((size_t)sw.b * a.Hq + h) * a.Tq + t] = live ? (M + log2f(L)) * kPagedLn2 : -INFINITY;
            }
          }
        }
        // The slot of a segment is free once its last scores are there. With one row tile the group without the last step
        // packs, while the other finishes the segment; with two each its own.
        if (qon && nu == 2) {
          const int next = units(get(1));
          times = next == 2 ? 1 : 2;
          pack0 = u;
          pack1 = min(u + 1, next);
        } else if (qon && grp != last) {
          pack1 = RT == 1 ? 1 : units(get(1));
          times = RT == 1 || pack1 == 2 ? 1 : 2;
          ok = __all_sync(0xffffffffu, tree_wait(s_full + 2 * last + (((end - 1) >> 1) & 1), ((end - 1) >> 2) & 1, abort));
          if (!ok) break;
        }
      }
      for (int u = pack0; u < pack1; u++) pack(get(1), e + kAhead, u, times);
    }
    if (!ok) {
      *abort = 1;
      atomicExch(a.status, kStatusTimeout);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    tmem_relinquish();
    tmem_dealloc(tmem, 512);
  }
}

// The cut (sequence, head)s: one that lies in the sweep's blocks c .. c + n is joined by n columns of this grid, each
// of which finds it with one load. A thread, or four neighbouring ones where there are many parts, takes four columns of a
// row, its parts in order (each its own share, then thread by thread: the same sum whichever block does it).
constexpr int kJoinThreads = 128, kJoinSlices = 8;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) k_tree_join(const __grid_constant__ PagedTreeArgs a) {
  const int tid = threadIdx.x;
  pdl_wait();
  const int4 cut = __ldcg(a.cut + blockIdx.x);
  if (cut.x < 0) return;
  const int first = cut.z, last = cut.w, slice = ((int)blockIdx.x - first) * kJoinSlices + (int)blockIdx.y;
  const int share = (last - first) * kJoinSlices, parts = last - first + 1;
  const int g = cut.y / a.pairs, r0 = cut.y % a.pairs * 2 * kTile, rows = min(a.rows, a.R - r0);
  constexpr int kAhead = 8;
  const int split = parts > kAhead ? 4 : 1, sub = tid & (split - 1), items = rows * (D / 4);
  for (int i0 = (slice * kJoinThreads + tid) / split; i0 - tid / split < items; i0 += share * kJoinThreads / split) {
    const int i = min(i0, items - 1), row = i / (D / 4), q = i % (D / 4);
    RowSum x;
    for (int c = first + sub; c <= last; c += kAhead * split) {
      float2 z[kAhead];
      float4 v[kAhead];
#pragma unroll
      for (int e = 0; e < kAhead; e++) {
        z[e] = make_float2(-INFINITY, 0.f);
        v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        const int at = c + e * split;
        if (at <= last) {
          const size_t p = (size_t)(2 * at + (at == first ? 1 : 0)) * a.rows + row;
          z[e] = __ldcg(a.part_ml + p);
          v[e] = __ldcg(reinterpret_cast<const float4*>(a.part_o + p * D) + q);
        }
      }
      float top = x.M;
#pragma unroll
      for (int e = 0; e < kAhead; e++)
        if (z[e].y != 0.f) top = fmaxf(top, z[e].x);
      x.raise(top);
#pragma unroll
      for (int e = 0; e < kAhead; e++) x.add(top, z[e], v[e]);
    }
    float top = x.M;
    for (int m = 1; m < split; m <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
    x.raise(top);
    for (int m = 1; m < split; m <<= 1) {
      x.S += __shfl_xor_sync(0xffffffffu, x.S, m);
      x.v.x += __shfl_xor_sync(0xffffffffu, x.v.x, m);
      x.v.y += __shfl_xor_sync(0xffffffffu, x.v.y, m);
      x.v.z += __shfl_xor_sync(0xffffffffu, x.v.z, m);
      x.v.w += __shfl_xor_sync(0xffffffffu, x.v.w, m);
    }
    if (sub == 0 && i0 < items) write_row<D>(a, cut.x, g, r0 + row, q, x.v, x.M, x.S);
  }
}

template <int D, int RT, bool SPLIT, bool FULL>
cudaError_t launch_tree_t(const PagedTreeArgs& a, int grid, cudaStream_t s) {
  static bool attr_set[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(k_tree_sweep<D, RT, SPLIT, FULL>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  static_assert(tree_head(2048) + TreeCfg<D>::kBytes + 1024 <= kSmemMax, "the largest batch");
  const int bytes = tree_head(a.B) + TreeCfg<D>::kBytes + 1024;
  if (bytes > kSmemMax) return cudaErrorInvalidValue;
  const cudaError_t e = launch_pdl(k_tree_sweep<D, RT, SPLIT, FULL>, dim3((unsigned)grid), kTreeThreads, (size_t)bytes, s, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_tree_join<D>, dim3((unsigned)grid, kJoinSlices), kJoinThreads, 0, s, a);
}
template <int D, bool FULL>
cudaError_t launch_tree(const PagedTreeArgs& a, int grid, cudaStream_t s) {
  if (a.R > kTile) return launch_tree_t<D, 2, false, FULL>(a, grid, s);
  return a.R > kTile / 2 ? launch_tree_t<D, 1, false, FULL>(a, grid, s) : launch_tree_t<D, 1, true, FULL>(a, grid, s);
}

}  // namespace

cudaError_t launch_decode_tree(const PagedTreeArgs& a, int nsm, cudaStream_t s) {
  PagedTreeArgs b = a;
  const int grid = nsm < kPagedMaxBlocks ? nsm : kPagedMaxBlocks;
  b.div_grid = make_fastdiv((uint32_t)grid);
  if (b.D == 64) return b.o_fp32 ? launch_tree<64, true>(b, grid, s) : launch_tree<64, false>(b, grid, s);
  return b.o_fp32 ? launch_tree<32, true>(b, grid, s) : launch_tree<32, false>(b, grid, s);
}

}  // namespace ne
