// Attention of a tree of drafted tokens over the paged cache (the verification step of tree
// speculation). Node i of sequence b is a token at cache position seq_len + i; it sees the context
// (all of it, a sliding window ending at its own logical position, or an index set) and, of the
// nodes, itself and its ancestors:
//
//   out[b, i, hq] = sum_t p_t v_t,  p = softmax_t(scale q[b, i, hq] . k_t)
//
// over t in the node's context and { seq_len + a : a = i or an ancestor of i }.
//
// The n G query rows of one (sequence, KV head) share every K / V row, so a row of 2 d bf16 feeds
// 4 d n G operations: HBM-bound up to about 250 rows, tensor-bound beyond. On the 5th-generation
// tensor cores:
//   * Work: the 64-token tiles of all (sequence, KV head) pairs in one line, split evenly over one
//     CTA per SM (ragged lengths balance by themselves; a CTA has at most two partial pairs). With
//     more than 256 rows (128 at d = 256) the CTAs form row groups that walk the line side by side
//     and share the rows through L2.
//   * 4 copy warps bring K / V rows straight from their pages (16-byte cp.async) into a ring of
//     stages, as 64-dimension column blocks with the 128-byte swizzle: the K-major operand of
//     S = Q K^T and the MN-major operand of O += P V. They run ahead over pair boundaries. The
//     nodes' rows come from k_new when given; another warp writes them to the cache.
//   * Groups of 4 warps, one thread per query row (tensor-memory lane): S from tensor memory, online
//     softmax in registers (fp32, lazy rescale of O), P as two bf16 parts back to tensor memory as the A
//     operands of P V. A further warp per group issues its MMAs; S of the next tile is computed while
//     the softmax of this one runs. At d = 128 two groups: both halves of 256 rows, or, with at most
//     128 rows, the even and the odd tiles of the same rows, whose O are merged at the end through
//     tensor memory (the two groups' warps share lanes). Their S, P and O fill tensor memory, so Q is
//     an operand in shared memory. At d = 256 O takes 256 columns, one group remains, and Q fits.
//   * The tensor cores take bf16 beside the bf16 V, so P = h + l (split_weights): a weight is off by at
//     most 2^-14 of itself, as close as the decode kernels' split. The sum of the weights is kept
//     from the fp32 ones.
//   * Pairs cut between CTAs leave fp32 (m, l, O) partials; a second kernel merges them.
// Masked positions must not reach the output even when V holds inf or NaN there (0 * inf): tiles
// in which a row masks a position that others see are scanned; non-finite elements are added to
// the rows that see them by hand and cleared in shared memory before the MMA.
// Measured on one B200 (32/8 heads, d 128; replayed in a graph): 104 rows over 8 contexts of 32K down to
// 16K 183 us, 4.2 TB/s of cache rows (the dense decode kernel: 156 us for one query each); 256 rows over
// 16 such contexts 588 us, 2.7 TB/s and 0.67 PFLOP/s: there the softmax warps are the bound (2900 cycles
// per tile, of which the exponentials and the split of P take 1400; the tensor pipe needs 1800, the bytes
// 1400). With P as one bf16 the two took 490 and 154 us: the split adds instructions to the softmax, the
// second product to the tensor pipe, and a stage is held longer. A chain of 5 nodes over one
// context of 700: 16 us.
// Every wait is bounded: after a timeout a thread goes on without waiting (all barriers still
// match), the flag is raised, and what was issued is drained before the tensor memory is freed.
#include <limits.h>

#include "common.cuh"
#include "tcgen05.cuh"

namespace jssa {

namespace tree_detail {

constexpr int kM = 128;   // rows of an MMA = threads of a group
constexpr int kTT = 64;   // tokens per tile (a tree of at most 64 nodes spans at most two)
constexpr uint32_t kCols = 512;
constexpr int kCopiers = 128;  // threads that copy rows: 16 of a tile per warp
// Row offsets are looked up for kBatch tiles of a pair at once, two batches ahead of the copies: the
// dependent loads (index set, page table) take microseconds under load.
constexpr int kBatch = 4;
constexpr float kRescaleSlack = 8.f;  // log2 units
constexpr unsigned kAll = 0xffffffffu;
// A branch that the tile loop hardly ever takes: its code is laid out away from the loop's.
__device__ __forceinline__ bool rare(bool x) { return __builtin_expect(x, 0); }

constexpr int kMinTiles = 4;  // tiles per CTA, before more CTAs take part

template <int D, bool TWO>
struct Cfg {
  static constexpr int kGroups = D == 128 ? 2 : 1;
  static constexpr bool kHalves = kGroups == 2 && !TWO;  // the groups share rows and split the tiles
  // + a warpgroup of which a warp per group issues its MMAs and one stores the new rows
  static constexpr int kThreads = kGroups * kM + kCopiers + 128;
  // registers per thread of the softmax, copy and MMA warpgroups; they add up to the launch's
  // (65536 / kThreads, a multiple of 8, per thread)
  static constexpr int kRegsSoftmax = D == 128 ? 168 : 232, kRegsCopy = D == 128 ? 96 : 136,
                       kRegsIssue = D == 128 ? 80 : 136;
  static_assert(kGroups * kM * kRegsSoftmax + 128 * (kRegsCopy + kRegsIssue) ==
                    kThreads * (65536 / kThreads / 8 * 8), "register split");
  static constexpr int kBlockBytes = kTT * 128;              // 64 tokens x 64 dimensions
  static constexpr int kTileBytes = D / 64 * kBlockBytes;    // K (or V) of one tile
  static constexpr int kStageBytes = 2 * kTileBytes;         // K then V
  // Q: in shared memory at d = 128 (of both groups, or of the rows they share), in tensor memory at
  // d = 256
  static constexpr bool kQTmem = D != 128;
  static constexpr int kQGroup = kM * D * 2;
  static constexpr int kQBytes = kQTmem ? 0 : (TWO ? 2 : 1) * kQGroup;
  static constexpr int kStages = D == 128 ? (TWO ? 4 : 5) : 3;
  static constexpr int kSmem = 1024 + kQBytes + kStages * kStageBytes;
  // tensor memory columns: Q (d = 256) and P (high parts, then low parts) as bf16 A operands, S and O
  // (fp32); P, S and O of each group
  static constexpr int kPiece = D == 128 ? 8 : 32;  // pairs of weights written to P at a time
  static constexpr uint32_t kQ = 0, kP = D == 128 ? 0 : 192, kS = 128, kO = 256;
};

// What the tiles of one (sequence, KV head) walk over: list index j < n_ctx is context position
// lo + j (or idx[j]), j - n_ctx < n a node.
struct Pair {
  int b, h, L, lo, n_ctx, tiles;
};
__device__ __forceinline__ Pair pair_of(const TreeArgs& a, int pair) {
  Pair p;
  p.b = pair / a.h_kv;
  p.h = pair - p.b * a.h_kv;
  const int max_len = a.max_pages * a.page_size;
  p.L = min(max(a.seq_lens[p.b], 0), max_len);
  p.lo = a.window > 0 ? max(0, p.L - a.window + 1) : 0;
  p.n_ctx = a.idx ? min(max(a.count[pair], 0), a.budget) : p.L - p.lo;
  p.tiles = (p.n_ctx + a.n + kTT - 1) / kTT;
  return p;
}

// Ancestor sets of the tree by pointer doubling over a warp: this lane's nodes are lane and
// lane + 32. Unused nodes have an empty set.
struct Tree {
  uint64_t see[2];
  __device__ __forceinline__ uint64_t of(int node) const {  // (warp-collective)
    const uint64_t lo = __shfl_sync(kAll, see[0], node & 31), hi = __shfl_sync(kAll, see[1], node & 31);
    return node < 32 ? lo : hi;
  }
};
// (parents: the n parents of one sequence)
__device__ __forceinline__ Tree tree_of(const int32_t* parents, int n, int lane, bool report) {
  Tree t;
  int ptr[2];
  bool bad[2], named[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = lane + 32 * u;
    const int p = i < n ? parents[i] : -2;
    t.see[u] = 1ull << i;
    named[u] = p >= -1;
    bad[u] = p < -1 || p >= i;
    ptr[u] = bad[u] ? -1 : p;
  }
  // (a tree of depth d takes log2 d rounds)
#pragma unroll 1
  while (__any_sync(kAll, ptr[0] >= 0 || ptr[1] >= 0)) {
    uint64_t s[2];
    int np[2];
    bool nb[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int src = ptr[u] & 31;
      const uint64_t s0 = __shfl_sync(kAll, t.see[0], src), s1 = __shfl_sync(kAll, t.see[1], src);
      const int p0 = __shfl_sync(kAll, ptr[0], src), p1 = __shfl_sync(kAll, ptr[1], src);
      const int b0 = __shfl_sync(kAll, (int)bad[0], src), b1 = __shfl_sync(kAll, (int)bad[1], src);
      const bool far = ptr[u] >= 32, on = ptr[u] >= 0;
      s[u] = on ? (far ? s1 : s0) : 0ull;
      np[u] = on ? (far ? p1 : p0) : -1;
      nb[u] = on && (far ? b1 : b0);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      t.see[u] |= s[u];
      ptr[u] = np[u];
      bad[u] |= nb[u];
    }
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    if (bad[u] && named[u] && report) raise_flag(2u);
    if (bad[u]) t.see[u] = 0ull;
  }
  return t;
}

// Two weights p = h + l as pairs of bf16 (the first one in the low half): h is p cut off, l the rest,
// with 2^-20 p added so that l > 0 wherever p > 0: an infinite value keeps its sign under both products
// and never meets a zero weight that the formula does not have. l < 2^-7 p; its rounding (half a step)
// and the addition are off by less than 2^-14 p.
__device__ __forceinline__ void split_weights(float2 p, uint32_t& h, uint32_t& l) {
  const uint32_t x = __float_as_uint(p.x), y = __float_as_uint(p.y);
  h = __byte_perm(x, y, 0x7632);
  const float2 minus_h = make_float2(__uint_as_float((x & 0xFFFF0000u) | 0x80000000u),
                                     __uint_as_float((y & 0xFFFF0000u) | 0x80000000u));
  const float2 rest = fma2(p, make_float2(1.f + 0x1p-20f, 1.f + 0x1p-20f), minus_h);
  l = pack_bf16x2(rest.x, rest.y);
}

// Weight of a partial (m, l) under the merged maximum M; a row whose every score was NaN keeps it.
__device__ __forceinline__ float merge_weight(float m, float l, float M) {
  return m == -INFINITY ? (l == l ? 0.f : l) : fast_exp2(m - M);
}
__device__ __forceinline__ float inverse_sum(float l) { return l > 0.f ? 1.f / l : (l == l ? 0.f : l); }

// Workspace: [where each CTA's tiles begin: pair (-1: none), tile][(m, l) of each partial row]
// [O of each partial row].
struct Work {
  int2* at;    // [CTAs]
  float2* ml;  // [2 * CTAs][rows]
  float* o;    // [2 * CTAs][rows][D]
};
__host__ __device__ inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }
__host__ __device__ inline Work work_of(void* ws, int64_t ctas, int64_t rows) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  Work w;
  w.at = reinterpret_cast<int2*>(p);
  p += up256(ctas * sizeof(int2));
  w.ml = reinterpret_cast<float2*>(p);
  p += up256(2 * ctas * rows * sizeof(float2));
  w.o = reinterpret_cast<float*>(p);
  return w;
}

struct Plan {
  bool two;        // both groups hold rows of their own (d = 128, more than 128 rows)
  int group_rows;  // rows of a row group
  int row_groups, ctas;
  int slot_rows;   // partial rows kept per slot
};
inline Plan plan_tree(int n, int G, int d) {
  Plan p;
  const int rows = n * G;
  p.two = d == 128 && rows > kM;
  p.group_rows = p.two ? 2 * kM : kM;
  p.row_groups = (rows + p.group_rows - 1) / p.group_rows;
  p.ctas = num_sms() / p.row_groups * p.row_groups;
  if (p.ctas < p.row_groups) p.ctas = p.row_groups;
  p.slot_rows = rows < p.group_rows ? rows : p.group_rows;
  return p;
}

template <int D, bool TWO>
__global__ void __launch_bounds__(Cfg<D, TWO>::kThreads, 1)
    tree_kernel(TreeArgs a, int row_groups, int slot_rows, long long limit) {
  using C = Cfg<D, TWO>;
  constexpr int kGroups = C::kGroups;
  constexpr bool kHalves = C::kHalves;
  extern __shared__ __align__(1024) uint8_t tree_smem[];
  __shared__ __align__(8) uint64_t s_full[C::kStages], s_empty[C::kStages];
  // per group: S ready, P V done (commits), S read, P ready, Q ready (an arrival of each warp)
  enum { kBarS, kBarO, kBarFree, kBarP, kBarQ, kBars };
  __shared__ __align__(8) uint64_t s_bar[kBars * kGroups + 1];  // the last one: drain
  __shared__ __align__(8) uint64_t s_valid[C::kStages];         // usable positions of a stage
  // offset (elements, a multiple of 8) of each row in the caches, or in k_new / v_new with bit 0
  // set; -1: not usable
  __shared__ int64_t s_off[kCopiers / 32][kBatch * 16];
  __shared__ float2 s_ml[2][kM];
  __shared__ uint32_t s_bad[kGroups][4], s_keep[kGroups];
  __shared__ int64_t s_sum[C::kThreads / 32];
  __shared__ int64_t s_todo;
  __shared__ int s_pair, s_tile;
  __shared__ uint32_t s_tmem;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t q_smem = (smem_u32(tree_smem) + 1023u) & ~1023u, ring = q_smem + C::kQBytes;
  const int pairs = a.batch * a.h_kv, G = a.h_q / a.h_kv, rows = a.n * G;
  const int rg = blockIdx.x % row_groups, cta = blockIdx.x / row_groups;

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      tc::mbar_init(smem_u32(&s_full[i]), kCopiers + kCopiers / 32);
      tc::mbar_init(smem_u32(&s_empty[i]), TWO ? 2 : 1);
    }
    for (int i = 0; i < kBars * kGroups + 1; ++i)
      tc::mbar_init(smem_u32(&s_bar[i]), i == kBars * kGroups ? kGroups : i % kBars < kBarFree ? 1 : 4);
    tc::fence_mbar_init();
  }
  if (warp == 0) {
    tc::tmem_alloc(smem_u32(&s_tmem), kCols);
    tc::tmem_relinquish();
  }
  pdl_wait();
  // ---- this CTA's tiles: prefix sums over the pairs' tile counts --------------------------------
  {
    const int per = (pairs + C::kThreads - 1) / C::kThreads;
    const int q0 = min(tid * per, pairs), q1 = min(q0 + per, pairs);
    int64_t mine = 0;
    for (int q = q0; q < q1; ++q) mine += pair_of(a, q).tiles;
    int64_t incl = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(kAll, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    int64_t before = incl - mine, total = 0;
    for (int w = 0; w < C::kThreads / 32; ++w) {
      if (w < warp) before += s_sum[w];
      total += s_sum[w];
    }
    const int64_t n_cta = gridDim.x / row_groups;
    const int64_t n_work = min(n_cta, (total + kMinTiles - 1) / kMinTiles);
    const int64_t begin = cta < n_work ? cta * total / n_work : total;
    const int64_t end = cta < n_work ? (cta + 1) * total / n_work : total;
    if (tid == 0) s_todo = end - begin;
    int2* at = work_of(a.ws, gridDim.x, slot_rows).at + cta;
    if (tid == 0 && rg == 0 && begin == end) *at = make_int2(-1, 0);
    for (int q = q0; q < q1 && begin < end; ++q) {
      const int t = pair_of(a, q).tiles;
      if (begin >= before && begin < before + t) {
        s_pair = q;
        s_tile = (int)(begin - before);
        if (rg == 0) *at = make_int2(q, (int)(begin - before));
      }
      before += t;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  pdl_trigger();
  const uint32_t tmem = s_tmem;
  const int64_t todo = s_todo;
  int pair = s_pair, t0 = s_tile;
  bool fail = false;

  if (warp >= kGroups * 4 + 4) {
    tc::regs_dec<C::kRegsIssue>();
    if (warp < kGroups * 4 + 4 + kGroups) {
      // ---- MMA issue, a warp per group: all lanes run the loop, one issues --------------------------
      // The S of the group's next tile goes before the P V of this one, under whose softmax it is
      // computed. The warp sleeps in its waits: one that polls takes issue slots from the softmax.
      const int g = warp - (kGroups * 4 + 4);
      constexpr uint32_t kIdescS = tc::idesc_bf16(kM, kTT, false);
      constexpr uint32_t kIdescO = tc::idesc_bf16(kM, D, true);
      constexpr int kStride = kHalves ? 2 : 1;  // tiles from one tile of the group to its next
      const uint32_t on = tc::elect_one();
      auto bar = [&](int which) { return smem_u32(&s_bar[kBars * g + which]); };
      auto wait = [&](uint32_t b, uint32_t parity) {  // (the whole warp agrees)
        if (!fail) fail = __any_sync(kAll, !tc::mbar_wait(b, parity & 1u, limit));
      };
      const uint32_t ts = tmem + C::kS + g * kTT, tp = tmem + C::kP + g * kTT, to = tmem + C::kO + g * D;
      uint32_t n_s = 0, n_p = 0, n_q = 0;  // S and P V issued, segments with a tile
      int64_t k0 = 0;
      while (k0 < todo && !fail) {
        const int tiles = pair_of(a, pair).tiles;
        const int n = (int)min((int64_t)tiles - t0, todo - k0);  // tiles of the segment
        int i_s = kHalves ? g : 0;  // the next S, with its stage
        int st_s = (int)((k0 + i_s) % C::kStages), st_p = st_s;
        uint32_t lap = (uint32_t)((k0 + i_s) / C::kStages);
        auto issue_s = [&]() {
          if (n_s > 0) wait(bar(kBarFree), n_s - 1);
          wait(smem_u32(&s_full[st_s]), lap);
          if (fail) return;
          // the rows came by cp.async (generic proxy); the tensor cores read by the async proxy
          tc::fence_proxy_async_smem();
          tc::fence_after_sync();
          const uint64_t b0 = tc::sw128_desc(ring + st_s * C::kStageBytes, 16, 1024);
          const uint64_t a0 = tc::sw128_desc(q_smem + (TWO ? g * C::kQGroup : 0), 16, 1024);
          if (!C::kQTmem) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              tc::mma_ss_warp(on, ts, a0 + (uint64_t)(((kk >> 2) * kM * 128 + (kk & 3) * 32) >> 4),
                              b0 + (uint64_t)(((kk >> 2) * C::kBlockBytes + (kk & 3) * 32) >> 4),
                              kIdescS, kk > 0);
          } else {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              tc::mma_ts_warp(on, ts, tmem + C::kQ + kk * 8,
                              b0 + (uint64_t)(((kk >> 2) * C::kBlockBytes + (kk & 3) * 32) >> 4),
                              kIdescS, kk > 0);
          }
          tc::mma_commit_warp(on, bar(kBarS));
          ++n_s;
          i_s += kStride;
          st_s += kStride;
          if (st_s >= C::kStages) {
            st_s -= C::kStages;
            ++lap;
          }
        };
        // Q is announced to a group's warp only in segments with a tile for it: those it cannot fall
        // behind in (a warp two phases late could not tell them apart)
        if (i_s < n) wait(bar(kBarQ), n_q++);
        if (i_s < n) issue_s();
        for (int i = kHalves ? g : 0; i < n && !fail; i += kStride) {
          if (i_s < n) issue_s();
          wait(bar(kBarP), n_p);
          if (fail) break;
          tc::fence_after_sync();
          const uint64_t b0 = tc::sw128_desc(ring + st_p * C::kStageBytes + C::kTileBytes,
                                             C::kBlockBytes, 1024);
          const bool add = *(volatile uint32_t*)&s_keep[g] != 0u;
#pragma unroll
          for (int kk = 0; kk < kTT / 8; ++kk)  // the high parts of P, then the low ones
            tc::mma_ts_warp(on, to, tp + kk * 8, b0 + (uint64_t)((kk % (kTT / 16) * 16 * 128) >> 4),
                            kIdescO, add || kk > 0);
          tc::mma_commit_warp(on, bar(kBarO));
          tc::mma_commit_warp(on, smem_u32(&s_empty[st_p]));
          ++n_p;
          st_p += kStride;
          if (st_p >= C::kStages) st_p -= C::kStages;
        }
        k0 += n;
        t0 = 0;
        ++pair;
      }
      // everything issued has completed before the tensor memory is freed
      tc::mma_commit_warp(on, smem_u32(&s_bar[kBars * kGroups]));
      if (!tc::mbar_wait(smem_u32(&s_bar[kBars * kGroups]), 0)) fail = true;
    } else if (warp == kGroups * 4 + 4 + kGroups && rg == 0) {
      // ---- bad lengths and parents are reported, the new nodes' rows written to the cache -----------
      const int max_len = a.max_pages * a.page_size;
      for (int64_t k0 = 0; k0 < todo;) {
        const Pair p = pair_of(a, pair);
        const int t1 = (int)min((int64_t)p.tiles, t0 + todo - k0);
        if (lane == 0 && a.seq_lens[p.b] != p.L) raise_flag(4u);
        const Tree tree = tree_of(a.parents + (int64_t)p.b * a.n, a.n, lane, true);
        if (a.k_new) {
          int64_t to[2];  // of nodes lane and lane + 32
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int node = lane + 32 * u, j = p.n_ctx + node, pos = p.L + node;
            to[u] = -1;
            if (tree.see[u] && j >= t0 * kTT && j < t1 * kTT && pos < max_len) {
              const int pg = a.block_table[(int64_t)p.b * a.max_pages + pos / a.page_size];
              if (pg >= 0 && (int64_t)pg < a.num_pages)
                to[u] = (int64_t)pg * a.page_stride + (int64_t)(pos % a.page_size) * a.slot_stride +
                        (int64_t)p.h * a.head_stride;
            }
          }
          // 4 rows at a time; lanes 0-15 K and 16-31 V at d = 128, chunk `lane` of both at d = 256
          const int c = D == 128 ? lane & 15 : lane;
          const bool is_v = D == 128 && lane >= 16;
#pragma unroll 1
          for (int i0 = 0; i0 < a.n; i0 += 4) {
            int64_t dst[4];
            uint4 x[4], y[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int i = i0 + u;
              const int64_t d0 = __shfl_sync(kAll, to[0], i & 31), d1 = __shfl_sync(kAll, to[1], i & 31);
              dst[u] = i < 32 ? d0 : d1;
              const int64_t src = (((int64_t)p.b * a.n + i) * a.h_kv + p.h) * D + c * 8;
              if (dst[u] >= 0) {
                x[u] = *reinterpret_cast<const uint4*>((is_v ? a.v_new : a.k_new) + src);
                if (D == 256) y[u] = *reinterpret_cast<const uint4*>(a.v_new + src);
              }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              if (dst[u] < 0) continue;
              *reinterpret_cast<uint4*>((is_v ? a.v_cache : a.k_cache) + dst[u] + c * 8) = x[u];
              if (D == 256) *reinterpret_cast<uint4*>(a.v_cache + dst[u] + c * 8) = y[u];
            }
          }
        }
        k0 += t1 - t0;
        t0 = 0;
        ++pair;
      }
    }
  } else if (warp >= kGroups * 4) {
    // ---- row copies: 16 rows of a tile per warp -----------------------------------------------------
    tc::regs_dec<C::kRegsCopy>();
    const int pw = warp - kGroups * 4;
    constexpr int kChunks = D / 8;                             // 16-byte chunks per row
    constexpr int kRowsPer = 32 / kChunks ? 32 / kChunks : 1;  // rows per copy instruction
    constexpr int kIters = 16 / kRowsPer, kUnroll = 8;
    const int c = lane % kChunks, half = kRowsPer == 2 ? lane >> 4 : 0;
    const int shift = 31 - __clz(a.page_size), max_len = a.max_pages * a.page_size;
    // Offsets of a batch (tiles t .. t + n - 1 of one pair): this lane's rows are row
    // 16 pw + lane % 16 of tiles t + lane / 16 and t + 2 + lane / 16. The positions (index set) of
    // the batch after next and the pages of the next one are in flight while a batch is copied.
    constexpr int kNone = INT_MIN;
    struct Batch {
      int b, h, n_ctx, t, n;
    };
    Batch next = {};
    int64_t left = todo;
    int tiles = 0, L = 0, lo = 0;
    auto advance = [&]() {  // the next batch of the line; n = 0 behind its end
      if (left <= 0) {
        next.n = 0;
        return;
      }
      next.t += next.n;
      if (next.t == tiles) {  // (also at the start, with tiles = t = 0)
        const Pair p = pair_of(a, pair);
        next.b = p.b; next.h = p.h; next.n_ctx = p.n_ctx;
        next.t = t0;
        tiles = p.tiles; L = p.L; lo = p.lo;
        t0 = 0;
        ++pair;
      }
      next.n = (int)min(min((int64_t)kBatch, left), (int64_t)(tiles - next.t));
      left -= next.n;
    };
    auto position = [&](int x) {  // of row x of `next`; kNone: no token there
      const int i = 2 * x + (lane >> 4);
      const int j = (next.t + i) * kTT + 16 * pw + (lane & 15), node = j - next.n_ctx;
      if (i >= next.n || node >= a.n) return kNone;
      if (node < 0)
        return a.idx ? max(a.idx[((int64_t)next.b * a.h_kv + next.h) * a.budget + j], -1) : lo + j;
      const int par = a.parents[(int64_t)next.b * a.n + node];
      return par >= -1 && par < node ? L + node : kNone;
    };
    auto page = [&](int b, int pos) {
      return pos >= 0 && pos < max_len ? a.block_table[(int64_t)b * a.max_pages + (pos >> shift)] : -1;
    };
    advance();
    Batch now = next;
    int pos0 = position(0), pos1 = position(1);
    int pg0 = page(now.b, pos0), pg1 = page(now.b, pos1);
    advance();
    int npos0 = position(0), npos1 = position(1);
    int st = 0;
    uint32_t lap = 0;
    while (now.n > 0) {
      const int n = now.n;
      uint32_t bad = 0u;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int ps = x ? pos1 : pos0, pg = x ? pg1 : pg0;
        int64_t off = -1;
        if (ps != kNone) {
          if (ps < 0 || ps >= max_len) {
            bad |= 2u;
          } else if (pg < 0 || (int64_t)pg >= a.num_pages) {
            bad |= 1u;
          } else {
            const int node = (now.t + 2 * x + (lane >> 4)) * kTT + 16 * pw + (lane & 15) - now.n_ctx;
            if (node >= 0 && a.k_new)
              off = ((((int64_t)now.b * a.n + node) * a.h_kv + now.h) * D) | 1;
            else
              off = (int64_t)pg * a.page_stride + (int64_t)(ps & (a.page_size - 1)) * a.slot_stride +
                    (int64_t)now.h * a.head_stride;
          }
        }
        s_off[pw][32 * x + lane] = off;
      }
      if (bad) raise_flag(bad);
      __syncwarp();
      now = next;
      pos0 = npos0;
      pos1 = npos1;
      pg0 = page(now.b, pos0);
      pg1 = page(now.b, pos1);
      advance();
      npos0 = position(0);
      npos1 = position(1);
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        const int64_t* offs = &s_off[pw][16 * i];
        if (!fail) fail = !tc::mbar_wait(smem_u32(&s_empty[st]), (lap & 1) ^ 1u, limit);
        const uint32_t stage = ring + st * C::kStageBytes + (c >> 3) * C::kBlockBytes;
#pragma unroll 1
        for (int i0 = 0; i0 < kIters; i0 += kUnroll) {
          int64_t off[kUnroll];  // (all of them first: the copies are not reordered with loads)
#pragma unroll
          for (int u = 0; u < kUnroll; ++u) off[u] = offs[(i0 + u) * kRowsPer + half];
#pragma unroll
          for (int u = 0; u < kUnroll; ++u) {
            const int64_t at = (off[u] >= 0 ? off[u] & ~1ll : 0) + c * 8;
            const bool fresh = off[u] >= 0 && (off[u] & 1);
            const int tr = pw * 16 + (i0 + u) * kRowsPer + half, n_bytes = off[u] >= 0 ? 16 : 0;
            const uint32_t dst = stage + tr * 128 + (((c & 7) ^ (tr & 7)) << 4);
            cp_async16(dst, (fresh ? a.k_new : a.k_cache) + at, n_bytes);
            cp_async16(dst + C::kTileBytes, (fresh ? a.v_new : a.v_cache) + at, n_bytes);
          }
        }
        const unsigned ok = __ballot_sync(kAll, offs[lane & 15] >= 0);
        if (lane == 0) reinterpret_cast<uint16_t*>(&s_valid[st])[pw] = (uint16_t)ok;
        tc::mbar_arrive_cp_async(smem_u32(&s_full[st]));
        if (lane == 0) tc::mbar_arrive(smem_u32(&s_full[st]));  // (s_valid is written)
        if (++st == C::kStages) {
          st = 0;
          ++lap;
        }
      }
      __syncwarp();  // the offsets have been read
    }
    cp_async_wait_all();
  } else {
    // ---- softmax groups ----------------------------------------------------------------------------
    tc::regs_inc<C::kRegsSoftmax>();
    const int g = warp >> 2, gt = tid & (kM - 1);  // group, thread of the group = tensor-memory lane
    const int gbar = 1 + g;                        // the group's named barrier; 3: both groups
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);  // this warp's lanes
    const uint32_t ts = tl + C::kS + g * kTT, tp = tl + C::kP + g * kTT, to = tl + C::kO + g * D;
    const uint32_t q_group = q_smem + (TWO ? g * C::kQGroup : 0);
    auto bar = [&](int which) { return smem_u32(&s_bar[kBars * g + which]); };
    // this warp has done its part: its tensor-memory accesses are complete before the arrival
    auto arrive = [&](int which) {
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar(which));
    };
    // (a negative scale is a negated Q; a zero scale must not turn the mask's -inf into NaN)
    const float scale_log2 = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1e-37f);
    const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
    const int r = rg * (TWO ? 2 * kM : kM) + (TWO ? g * kM : 0) + gt;  // query row of this thread
    const int node = min(r / G, kTreeMaxNodes - 1);
    uint32_t n_t = 0;  // tiles of this group so far (phases of its barriers)
    int64_t k0 = 0;    // line index (within the CTA) of the segment's first tile
    while (k0 < todo) {
      // Q: this thread's row (on its way to L1 while the pair and the tree are resolved)
      const bool q_mine = !kHalves || g == 0;
      const int pb = pair / a.h_kv;
      const int64_t q_off = r < rows ? (((int64_t)pb * a.n + node) * a.h_q + (int64_t)(pair - pb * a.h_kv) * G + r % G) * D : 0;
      const uint4* qrow = reinterpret_cast<const uint4*>(a.q + q_off);
      if (q_mine)
#pragma unroll
        for (int u = 0; u < D / 64; ++u) prefetch_l1(qrow + 8 * u);
      const Pair p = pair_of(a, pair);
      const int t1 = (int)min((int64_t)p.tiles, t0 + todo - k0);
      const Tree tree = tree_of(a.parents + (int64_t)p.b * a.n, a.n, lane, false);
      uint64_t see = tree.of(node);
      if (r >= rows) see = 0ull;
      const bool used = see != 0ull;
      const int depth = __popcll(see) - 1;
      int lo = 0;  // first list index this row sees
      if (a.window > 0) {
        lo = min(max(0, p.L + depth - a.window + 1) - p.lo, p.n_ctx);
        for (int x = depth + 1 - a.window; x > 0; --x) see &= see - 1;  // (ancestors: ascending depth)
      }
      if (q_mine) {
#pragma unroll(D == 128 ? 2 : 1)
        for (int c = 0; c < D / 64; ++c) {
          uint32_t v[32];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const uint4 x = qrow[8 * c + u];
            v[4 * u] = used ? x.x ^ flip : 0u;
            v[4 * u + 1] = used ? x.y ^ flip : 0u;
            v[4 * u + 2] = used ? x.z ^ flip : 0u;
            v[4 * u + 3] = used ? x.w ^ flip : 0u;
          }
          if (C::kQTmem) {
            tc::tmem_st32(tl + C::kQ + 32 * c, v);
          } else {
#pragma unroll
            for (int u = 0; u < 8; ++u)
              st_shared_v4(q_group + c * kM * 128 + gt * 128 + ((u ^ (gt & 7)) << 4), v[4 * u],
                           v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
          }
        }
        if (C::kQTmem) tc::tmem_wait_st();
        else tc::fence_proxy_async_smem();
        arrive(kBarQ);
        if (kHalves && t1 - t0 > 1 && lane == 0) tc::mbar_arrive(smem_u32(&s_bar[kBars + kBarQ]));
      }
      float m_ref = -INFINITY, l = 0.f;
      bool have_o = false;
      const bool active = __any_sync(kAll, used);  // a warp of padding rows only keeps the barriers
      int st = (int)((k0 + (kHalves ? g : 0)) % C::kStages);
      uint32_t lap = (uint32_t)((k0 + (kHalves ? g : 0)) / C::kStages);
#pragma unroll 1
      for (int t = t0 + (kHalves ? g : 0); t < t1; t += kHalves ? 2 : 1) {
        const uint32_t stage = ring + st * C::kStageBytes;
        // S of this tile; its rows' validity (they are in long since, when S is: the tests overlap)
        {
          const bool s_in = tc::mbar_test(bar(kBarS), n_t & 1);
          const bool rows_in = tc::mbar_test(smem_u32(&s_full[st]), lap & 1);
          if (rare(!s_in) && !fail) fail = !tc::mbar_wait(bar(kBarS), n_t & 1, limit);
          if (rare(!rows_in) && !fail) fail = !tc::mbar_wait(smem_u32(&s_full[st]), lap & 1, limit);
        }
        tc::fence_after_sync();
        uint32_t s0[32], s1[32];
        if (active) {
          tc::tmem_ld32(ts, s0);
          tc::tmem_ld32(ts + 32, s1);
        }
        uint64_t see_t = s_valid[st];  // the list indexes of this tile that the row sees
        const int j0 = t * kTT, c_left = p.n_ctx - j0;  // context positions from here on
        // uniform over the CTA: some row may mask a position that is in the tile
        const bool special = c_left < kTT || (a.window > 0 && t == 0);
        if (rare(special)) {
          if (c_left < kTT) {
            const uint64_t ctx = c_left > 0 ? (1ull << c_left) - 1ull : 0ull;
            const uint64_t tr = c_left >= 0 ? see << c_left : (-c_left < 64 ? see >> -c_left : 0ull);
            see_t &= ctx | tr;
          }
          if (lo > j0) see_t &= lo - j0 < 64 ? ~0ull << (lo - j0) : 0ull;
          if (!used) see_t = ~0ull;  // (its row is discarded)
        }
        if (active) tc::tmem_wait_ld();
        arrive(kBarFree);
        if (active) {
          if (rare(!__all_sync(kAll, see_t == ~0ull))) {
            const uint32_t lo32 = (uint32_t)see_t, hi32 = (uint32_t)(see_t >> 32);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              if (!((lo32 >> j) & 1u)) s0[j] = 0xFF800000u;  // -inf
              if (!((hi32 >> j) & 1u)) s1[j] = 0xFF800000u;
            }
          }
          float mx[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) mx[u] = fmaxf(__uint_as_float(s0[u]), __uint_as_float(s1[u]));
#pragma unroll
          for (int j = 4; j < 32; j += 4)
#pragma unroll
            for (int u = 0; u < 4; ++u)
              mx[u] = fmaxf(mx[u], fmaxf(__uint_as_float(s0[j + u]), __uint_as_float(s1[j + u])));
          const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale_log2;
          // lazy rescale: weights are relative to m_ref, which moves only when the row's maximum
          // exceeds it by more than the slack (weights stay <= 2^8)
          const bool grow = mt > m_ref + kRescaleSlack;
          const float m_new = grow ? mt : m_ref;
          const float corr = grow && m_ref != -INFINITY ? fast_exp2(m_ref - m_new) : 1.f;
          // P V of the group's previous tile: done with P and O (tested here, its latency under the
          // exponentials)
          bool o_done = n_t == 0 || tc::mbar_test(bar(kBarO), (n_t - 1) & 1);
          auto previous_done = [&]() {
            if (rare(!o_done) && !fail) fail = !tc::mbar_wait(bar(kBarO), (n_t - 1) & 1, limit);
            o_done = true;
            tc::fence_after_sync();
          };
          if (rare(have_o && __any_sync(kAll, corr != 1.f))) {
            previous_done();
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tc::tmem_ld32(to + 32 * c, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
              tc::tmem_st32(to + 32 * c, o);
            }
          }
          m_ref = m_new;
          const float m_sub = m_ref == -INFINITY ? 0.f : m_ref;
          const float2 sc2 = make_float2(scale_log2, scale_log2), ms2 = make_float2(-m_sub, -m_sub);
          float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
          // kPiece pairs at a time, so that P takes the registers that S gives up (d = 256 has registers for the
          // whole tile, and the previous P V is later)
#pragma unroll
          for (int j0 = 0; j0 < 32; j0 += C::kPiece) {
            uint32_t ph[C::kPiece], pl[C::kPiece];
#pragma unroll
            for (int u = 0; u < C::kPiece; ++u) {
              const int j = j0 + u;
              float2 p = j < 16 ? make_float2(__uint_as_float(s0[2 * j]), __uint_as_float(s0[2 * j + 1]))
                                : make_float2(__uint_as_float(s1[2 * j - 32]), __uint_as_float(s1[2 * j - 31]));
              p = fma2(p, sc2, ms2);
              p.x = fast_exp2(p.x);
              p.y = fast_exp2(p.y);
              if (j & 1) sum1 = add2(sum1, p);
              else sum0 = add2(sum0, p);
              split_weights(p, ph[u], pl[u]);
            }
            if (j0 == 0) previous_done();
#pragma unroll
            for (int u = 0; u < C::kPiece; u += 8) {
              tc::tmem_st8(tp + j0 + u, ph + u);
              tc::tmem_st8(tp + kTT / 2 + j0 + u, pl + u);
            }
          }
          sum0 = add2(sum0, sum1);
          l = l * corr + (sum0.x + sum0.y);
          tc::tmem_wait_st();
        } else {
          // (keeps this warp's arrivals in step: P of the previous tile has been taken)
          if (n_t > 0 && !fail) fail = !tc::mbar_wait(bar(kBarO), (n_t - 1) & 1, limit);
          tc::fence_after_sync();
        }
        bool keep_o = have_o;
        if (rare(special)) {
          // this thread's half row of V: any exponent of all ones
          const uint32_t vrow = stage + C::kTileBytes + (gt >> 1) * 128;
          constexpr int kPer = D / 16;  // 16-byte chunks of half a row
          auto chunk = [&](int q) {
            const int c = (gt & 1) * kPer + q;
            return vrow + (c >> 3) * C::kBlockBytes + (((c & 7) ^ ((gt >> 1) & 7)) << 4);
          };
          auto odd = [](uint32_t w) { return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u; };
          bool mine = false;
#pragma unroll
          for (int q = 0; q < kPer; ++q) {
            const uint4 y = ld_shared_v4(chunk(q));
            mine |= odd(y.x) | odd(y.y) | odd(y.z) | odd(y.w);
          }
          const int vbar = TWO ? 3 : gbar, vthreads = TWO ? 2 * kM : kM;
          if (tc::bar_or(vbar, vthreads, mine)) {
            const unsigned two = __ballot_sync(kAll, mine);
            if (lane == 0) s_bad[g][warp & 3] = two;  // bit 2 i (+ 1): token 16 w + i
            tc::bar_sync(gbar, kM);
            // add p v of the non-finite elements to the rows that see them (O = 0 first; the high part
            // of p has its sign, and is 0 or NaN where p is)
            uint32_t pw[32];
            tc::tmem_ld32(tp, pw);
            tc::tmem_wait_ld();
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              if (have_o) {
                tc::tmem_ld32(to + 32 * c, o);
                tc::tmem_wait_ld();
              } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = 0u;
              }
#pragma unroll 1
              for (int j = 0; j < kTT; ++j) {
                if (!((s_bad[g][j >> 4] >> (2 * (j & 15))) & 3u)) continue;
                const uint32_t w = pw[j >> 1];
                const float pj = (j & 1) ? bf16_hi(w) : bf16_lo(w);
                const bool sees = (see_t >> j) & 1ull;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const int cc = 4 * c + q;
                  const uint4 y = ld_shared_v4(stage + C::kTileBytes + (cc >> 3) * C::kBlockBytes + j * 128 +
                                     (((cc & 7) ^ (j & 7)) << 4));
                  const uint32_t yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const float v0 = bf16_lo(yw[e]), v1 = bf16_hi(yw[e]);
                    uint32_t& o0 = o[8 * q + 2 * e];
                    uint32_t& o1 = o[8 * q + 2 * e + 1];
                    if (sees && (yw[e] & 0x7F80u) == 0x7F80u)
                      o0 = __float_as_uint(__uint_as_float(o0) + pj * v0);
                    if (sees && (yw[e] & 0x7F800000u) == 0x7F800000u)
                      o1 = __float_as_uint(__uint_as_float(o1) + pj * v1);
                  }
                }
              }
              tc::tmem_st32(to + 32 * c, o);
            }
            tc::tmem_wait_st();
            keep_o = true;
            tc::bar_sync(vbar, vthreads);  // everyone has read V
            if (!TWO || g == 0) {          // clear the elements for the MMA
#pragma unroll 1
              for (int q = 0; q < kPer; ++q) {
                const uint4 y = ld_shared_v4(chunk(q));
                uint32_t yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  if ((yw[e] & 0x7F80u) == 0x7F80u) yw[e] &= 0xFFFF0000u;
                  if ((yw[e] & 0x7F800000u) == 0x7F800000u) yw[e] &= 0x0000FFFFu;
                }
                st_shared_v4(chunk(q), yw[0], yw[1], yw[2], yw[3]);
              }
              tc::fence_proxy_async_smem();
            }
            if (TWO) tc::bar_sync(vbar, vthreads);
          }
        }
        // (thread 0 of the group also says whether P V adds to O: the same for all its tiles but the
        // first, and but for the slow path above)
        if (rare(t < t0 + 2 * (kHalves ? 2 : 1) || special) && gt == 0) *(volatile uint32_t*)&s_keep[g] = keep_o;
        arrive(kBarP);
        have_o = true;
        ++n_t;
        st += kHalves ? 2 : 1;
        if (st >= C::kStages) {
          st -= C::kStages;
          ++lap;
        }
      }
      if (have_o && !fail) fail = !tc::mbar_wait(bar(kBarO), (n_t - 1) & 1, limit);
      tc::fence_after_sync();

      // ---- the segment's rows: into the output when the pair is whole, else into a partial slot
      const Work ws = work_of(a.ws, gridDim.x, slot_rows);
      const bool whole = t0 == 0 && t1 == p.tiles;
      if (!used) {
        m_ref = -INFINITY;
        l = 0.f;
      }
      float w0 = merge_weight(m_ref, l, m_ref), w1 = 0.f;  // of this group's and the other group's O
      bool other = false;
      if (kHalves) {
        s_ml[g][gt] = make_float2(m_ref, l);
        tc::fence_before_sync();
        tc::bar_sync(3, 2 * kM);
        tc::fence_after_sync();
        const float2 o = s_ml[g ^ 1][gt];
        const float M = fmaxf(m_ref, o.x);
        w0 = merge_weight(m_ref, l, M);
        w1 = merge_weight(o.x, o.y, M);
        // (a group without tiles has no O)
        l = (have_o ? w0 * l : 0.f) + (w1 != 0.f ? w1 * o.y : 0.f);
        m_ref = M;
        other = w1 != 0.f;
      }
      const bool mine = have_o && w0 != 0.f;
      const float inv = whole ? inverse_sum(l) : 1.f;
      const int slot = 2 * blockIdx.x + (k0 > 0 ? 1 : 0), lr = (TWO ? g * kM : 0) + gt;
      const int64_t prow = (int64_t)slot * slot_rows + lr;
      if (!whole && r < rows && (!kHalves || g == 0)) ws.ml[prow] = make_float2(m_ref, l);
      uint16_t* orow = a.out + q_off;
      constexpr int kPart = kHalves ? D / 64 : D / 32;  // 32-column pieces written by this group
#pragma unroll 1
      for (int c = (kHalves ? g * kPart : 0); c < (kHalves ? g * kPart : 0) + kPart; ++c) {
        uint32_t o[32];
        if (have_o) {
          tc::tmem_ld32(to + 32 * c, o);
          tc::tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = mine ? __float_as_uint(__uint_as_float(o[e]) * w0) : 0u;
        if (kHalves) {
          if (__any_sync(kAll, other)) {
            uint32_t y[32];
            tc::tmem_ld32(tl + C::kO + (g ^ 1) * D + 32 * c, y);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (other) o[e] = __float_as_uint(__uint_as_float(o[e]) + w1 * __uint_as_float(y[e]));
          }
        }
        if (r >= rows) continue;
        if (whole) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
              w[u] = pack_bf16x2(__uint_as_float(o[8 * e + 2 * u]) * inv, __uint_as_float(o[8 * e + 2 * u + 1]) * inv);
            reinterpret_cast<uint4*>(orow + 32 * c)[e] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
          float4* dst = reinterpret_cast<float4*>(ws.o + prow * D + 32 * c);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            dst[e] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                 __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
        }
      }
      tc::fence_before_sync();
      if (kHalves) tc::bar_sync(3, 2 * kM);  // both groups are done with both O and s_ml
      tc::fence_after_sync();
      k0 += t1 - t0;
      t0 = 0;
      ++pair;
    }
  }
  if (fail) raise_flag(JSSA_DEVERR_TIMEOUT);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kCols);
  }
}

// Merge of the pairs that several CTAs share,
//   M = max m_i,  w_i = 2^(m_i - M),  out = sum w_i O_i / sum w_i l_i.
// Block (x, y): the pair in whose middle CTA x begins, if it is the first such CTA, and 8 of its rows,
// one per warp. Latency-bound: the (m, l) and O of kMergeParts partials are read at once, and the weights
// applied as they come (a running maximum). One row per warp keeps all blocks resident at once: with 4
// (126 registers) the merge of 148 x 256 rows took 12 us longer.
constexpr int kMergeWarps = 8, kMergeParts = 4;
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32)
    merge_kernel(TreeArgs a, int row_groups, int group_rows, int slot_rows, int ctas) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int x = blockIdx.x / row_groups + 1, rg = blockIdx.x % row_groups, n_cta = ctas / row_groups;
  const Work ws = work_of(a.ws, ctas, slot_rows);
  pdl_wait();
  // lane i: where CTA x - 1 + i begins
  const int2 at = x - 1 + lane < n_cta ? ws.at[x - 1 + lane] : make_int2(-1, 0);
  const int pair = __shfl_sync(kAll, at.x, 1);
  const bool inside = at.x == pair && at.y > 0;  // it begins in the middle of the pair
  unsigned in = __ballot_sync(kAll, inside);
  if (pair < 0 || !(in & 2u) || (in & 1u)) return;  // CTA x is not the first that does
  const int first = __shfl_sync(kAll, at.x, 0) == pair ? 0 : 1;
  // partial 0: CTA x - 1's last segment; partial i > 0: the first segment of CTA x - 1 + i
  int parts = __ffs(~(in | 1u)) - 1;
  if (parts < 0) {
    parts = 32;
    for (int y = x + 31; y < n_cta; y += 32) {
      const int2 more = y + lane < n_cta ? ws.at[y + lane] : make_int2(-1, 0);
      in = __ballot_sync(kAll, more.x == pair && more.y > 0);
      parts += in == kAll ? 32 : __ffs(~in) - 1;
      if (in != kAll) break;
    }
  }
  auto slot_of = [&](int i) {
    return (int64_t)(2 * ((x - 1 + i) * row_groups + rg) + (i == 0 ? first : 0)) * slot_rows;
  };
  const int G = a.h_q / a.h_kv, rows = a.n * G;
  const int lr = blockIdx.y * kMergeWarps + warp, r = rg * group_rows + lr;
  if (lr >= slot_rows || r >= rows) return;
  float M = -INFINITY, l = 0.f, acc[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) acc[e] = 0.f;
#pragma unroll 1
  for (int i0 = 0; i0 < parts; i0 += kMergeParts) {
    float2 ml[kMergeParts];
    float4 o[kMergeParts][D / 128];
#pragma unroll
    for (int i = 0; i < kMergeParts; ++i) {
      ml[i] = make_float2(-INFINITY, 0.f);
      if (i0 + i >= parts) continue;
      const int64_t row = slot_of(i0 + i) + lr;
      ml[i] = __ldcg(ws.ml + row);
#pragma unroll
      for (int q = 0; q < D / 128; ++q)
        o[i][q] = __ldcg(reinterpret_cast<const float4*>(ws.o + row * D) + q * 32 + lane);
    }
    float top = M;
#pragma unroll
    for (int i = 0; i < kMergeParts; ++i) top = fmaxf(top, ml[i].x);
    const float keep = M == -INFINITY ? 1.f : fast_exp2(M - top);  // (of zeros, or of NaN sums)
    M = top;
    l *= keep;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc[e] *= keep;
#pragma unroll
    for (int i = 0; i < kMergeParts; ++i) {
      const float w = merge_weight(ml[i].x, ml[i].y, top);
      if (w == 0.f) continue;
      l += w * ml[i].y;
#pragma unroll
      for (int q = 0; q < D / 128; ++q) {
        acc[4 * q] += w * o[i][q].x;
        acc[4 * q + 1] += w * o[i][q].y;
        acc[4 * q + 2] += w * o[i][q].z;
        acc[4 * q + 3] += w * o[i][q].w;
      }
    }
  }
  const int b = pair / a.h_kv, h = pair % a.h_kv;
  const float inv = inverse_sum(l);
  uint16_t* out = a.out + (((int64_t)b * a.n + r / G) * a.h_q + (int64_t)h * G + r % G) * D;
#pragma unroll
  for (int q = 0; q < D / 128; ++q)
    reinterpret_cast<uint2*>(out)[q * 32 + lane] =
        make_uint2(pack_bf16x2(acc[4 * q] * inv, acc[4 * q + 1] * inv),
                   pack_bf16x2(acc[4 * q + 2] * inv, acc[4 * q + 3] * inv));
}

// What a draft needs before its attention: the cache slots of the used nodes, and the mean of their
// queries (fp32 sums, rounded once). Block (b, x): kPrepareThreads x 8 elements of the mean of sequence
// b, x = 0 also its slots. Unused nodes' rows are not read. Latency-bound: one chain of parents, tree and
// rows.
constexpr int kPrepareThreads = 128;
__global__ void __launch_bounds__(kPrepareThreads) prepare_kernel(TreeArgs a, int64_t* slots, uint16_t* mean) {
  __shared__ uint64_t s_used;
  const int tid = threadIdx.x, lane = tid & 31, b = blockIdx.x;
  if (tid < 32) {
    const Tree tree = tree_of(a.parents + (int64_t)b * a.n, a.n, lane, false);
    const unsigned lo = __ballot_sync(kAll, tree.see[0] != 0ull), hi = __ballot_sync(kAll, tree.see[1] != 0ull);
    if (lane == 0) s_used = (uint64_t)hi << 32 | lo;
  }
  __syncthreads();
  const uint64_t used = s_used;
  if (blockIdx.y == 0 && tid < a.n) {
    const int max_len = a.max_pages * a.page_size;
    const int pos = min(max(a.seq_lens[b], 0), max_len) + tid;
    int64_t slot = -1;
    if ((used >> tid & 1ull) && pos < max_len) {
      const int pg = a.block_table[(int64_t)b * a.max_pages + pos / a.page_size];
      if (pg >= 0 && (int64_t)pg < a.num_pages) slot = (int64_t)pg * a.page_size + pos % a.page_size;
    }
    slots[(int64_t)b * a.n + tid] = slot;
  }
  const int width = a.h_q * a.d, e = (blockIdx.y * kPrepareThreads + tid) * 8;
  if (!mean || e >= width) return;
  const uint16_t* q = a.q + (int64_t)b * a.n * width + e;
  float2 sum[4] = {};
#pragma unroll 4
  for (uint64_t left = used; left; left &= left - 1) {
    const uint4 x = *reinterpret_cast<const uint4*>(q + (int64_t)(__ffsll((long long)left) - 1) * width);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int u = 0; u < 4; ++u) sum[u] = add2(sum[u], make_float2(bf16_lo(w[u]), bf16_hi(w[u])));
  }
  const float n = (float)max(__popcll(used), 1);
  uint32_t w[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) w[u] = pack_bf16x2(sum[u].x / n, sum[u].y / n);
  *reinterpret_cast<uint4*>(mean + (int64_t)b * width + e) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <int D, bool TWO>
cudaError_t launch_t(const TreeArgs& a, const Plan& plan, cudaStream_t s) {
  using C = Cfg<D, TWO>;
  auto kern = tree_kernel<D, TWO>;
  cudaError_t e = configure_kernel((const void*)kern, C::kSmem, false);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(plan.ctas, 1, 1);
  cfg.blockDim = dim3(C::kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, a, plan.row_groups, plan.slot_rows, tc_wait_limit());
  if (e != cudaSuccess) return e;
  if (plan.ctas == plan.row_groups) return cudaGetLastError();  // one CTA has every pair whole
  cfg.gridDim = dim3(plan.ctas - plan.row_groups, (plan.slot_rows + kMergeWarps - 1) / kMergeWarps, 1);
  cfg.blockDim = dim3(kMergeWarps * 32, 1, 1);
  cfg.dynamicSmemBytes = 0;
  e = cudaLaunchKernelEx(&cfg, merge_kernel<D>, a, plan.row_groups, plan.group_rows, plan.slot_rows,
                         plan.ctas);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace tree_detail

size_t tree_ws_bytes(int batch, int n, int h_q, int h_kv, int d) {
  using namespace tree_detail;
  if (batch * h_kv == 0 || n == 0) return 0;
  const Plan p = plan_tree(n, h_q / h_kv, d);
  const size_t rows = 2 * (size_t)p.ctas * p.slot_rows;
  return up256(p.ctas * sizeof(int2)) + up256(rows * sizeof(float2)) + rows * d * sizeof(float);
}

cudaError_t launch_tree_prepare(const TreeArgs& a, int64_t* slots, uint16_t* mean, cudaStream_t s) {
  using namespace tree_detail;
  if (a.batch == 0 || (a.n == 0 && !mean)) return cudaSuccess;
  const int per = kPrepareThreads * 8;
  prepare_kernel<<<dim3(a.batch, mean ? (a.h_q * a.d + per - 1) / per : 1), kPrepareThreads, 0, s>>>(a, slots, mean);
  return cudaGetLastError();
}

cudaError_t launch_tree(const TreeArgs& a, cudaStream_t s) {
  using namespace tree_detail;
  if (a.batch == 0 || a.n == 0) return cudaSuccess;
  const Plan p = plan_tree(a.n, a.h_q / a.h_kv, a.d);
  if (a.d == 128) return p.two ? launch_t<128, true>(a, p, s) : launch_t<128, false>(a, p, s);
  if (a.d == 256) return launch_t<256, false>(a, p, s);
  return cudaErrorInvalidValue;
}

}  // namespace jssa
