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
//   * 4 producer warps copy K / V rows straight from their pages (16-byte cp.async) into a ring of
//     stages, as 64-dimension column blocks with the 128-byte swizzle: the K-major operand of
//     S = Q K^T and the MN-major operand of O += P V. They run ahead over pair boundaries. The
//     nodes' rows come from k_new when given, and are written to the cache on the way.
//   * Groups of 4 warps, one thread per query row (tensor-memory lane): S from tensor memory,
//     online softmax in registers (fp32, lazy rescale of O), P as bf16 back over S. Q and P are the
//     A operands from tensor memory. At d = 128 two groups: both halves of 256 rows, or, with at
//     most 128 rows, the even and the odd tiles of the same rows, whose O are merged at the end
//     through tensor memory (the two groups' warps share lanes). At d = 256 O takes 256 columns
//     and one group remains.
//   * P is rounded to bf16 (half a step, 2^-9 of a weight): the tensor cores take bf16 beside the
//     bf16 V; the sum l is kept from the fp32 weights.
//   * Pairs cut between CTAs leave fp32 (m, l, O) partials; a second kernel merges them.
// Masked positions must not reach the output even when V holds inf or NaN there (0 * inf): tiles
// in which a row masks a position that others see are scanned; non-finite elements are added to
// the rows that see them by hand and cleared in shared memory before the MMA.
// Every wait is bounded: after a timeout a thread goes on without waiting (all barriers still
// match), the flag is raised, and what was issued is drained before the tensor memory is freed.
#include "common.cuh"
#include "tcgen05.cuh"

namespace jssa {

namespace tree_detail {

constexpr int kM = 128;   // rows of an MMA = threads of a group
constexpr int kTT = 64;   // tokens per tile (a tree of at most 64 nodes spans at most two)
constexpr uint32_t kCols = 512;
constexpr int kProducers = 128;
constexpr float kRescaleSlack = 8.f;  // log2 units
constexpr unsigned kAll = 0xffffffffu;
constexpr int kMinTiles = 2;  // tiles per CTA, before more CTAs take part

template <int D>
struct Cfg {
  static constexpr int kGroups = D == 128 ? 2 : 1;
  static constexpr int kThreads = kGroups * kM + kProducers;
  static constexpr int kBlockBytes = kTT * 128;              // 64 tokens x 64 dimensions
  static constexpr int kTileBytes = D / 64 * kBlockBytes;    // K (or V) of one tile
  static constexpr int kStageBytes = 2 * kTileBytes;         // K then V
  static constexpr int kStages = D == 128 ? 6 : 3;
  static constexpr int kAhead = D == 128 ? 3 : 1;            // newer tiles in flight behind a landed one
  static constexpr int kSmem = 1024 + kStages * kStageBytes;
  // tensor memory columns: Q (bf16 A operand), S / P, O of each group
  static constexpr uint32_t kQ = 0, kQCols = D / 2;
  static constexpr uint32_t kS = 128, kO = 256;
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
__device__ __forceinline__ Tree tree_of(const TreeArgs& a, int b, int lane, bool report) {
  Tree t;
  int ptr[2];
  bool bad[2], named[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = lane + 32 * u;
    const int p = i < a.n ? a.parents[(int64_t)b * a.n + i] : -2;
    t.see[u] = 1ull << i;
    named[u] = p >= -1;
    bad[u] = p < -1 || p >= i;
    ptr[u] = bad[u] ? -1 : p;
  }
#pragma unroll 1
  for (int step = 1; step < a.n; step <<= 1) {
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

// Weight of a partial (m, l) under the merged maximum M; a row whose every score was NaN keeps it.
__device__ __forceinline__ float merge_weight(float m, float l, float M) {
  return m == -INFINITY ? (l == l ? 0.f : l) : fast_exp2(m - M);
}
__device__ __forceinline__ float inverse_sum(float l) { return l > 0.f ? 1.f / l : (l == l ? 0.f : l); }

// Workspace: [tiles in the line, CTAs per row group that share them][first tile of each pair]
// [(m, l) of each partial row][O of each partial row].
struct Work {
  int64_t* head;
  int64_t* first;  // [pairs + 1]
  float2* ml;      // [2 * CTAs][rows]
  float* o;        // [2 * CTAs][rows][D]
};
__host__ __device__ inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }
__host__ __device__ inline Work work_of(void* ws, int64_t pairs, int64_t ctas, int64_t rows) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  Work w;
  w.head = reinterpret_cast<int64_t*>(p);
  w.first = w.head + 2;
  p += up256((pairs + 3) * 8);
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
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
    tree_kernel(TreeArgs a, int row_groups, int slot_rows, long long limit) {
  using C = Cfg<D>;
  constexpr int kGroups = C::kGroups;
  constexpr bool kHalves = kGroups == 2 && !TWO;  // the groups share rows and split the tiles
  extern __shared__ __align__(1024) uint8_t tree_smem[];
  __shared__ __align__(8) uint64_t s_full[C::kStages], s_empty[C::kStages];
  __shared__ __align__(8) uint64_t s_bar[3 * kGroups];  // per group: S ready, P V done, drain
  __shared__ uint16_t s_valid[C::kStages][kTT / 16];    // usable positions of a stage
  __shared__ float2 s_ml[2][kM];
  __shared__ uint32_t s_bad[kGroups][4];
  __shared__ int64_t s_sum[C::kThreads / 32];
  __shared__ int64_t s_begin, s_end;
  __shared__ int s_pair, s_tile;
  __shared__ uint32_t s_tmem;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t ring = (smem_u32(tree_smem) + 1023u) & ~1023u;
  const int pairs = a.batch * a.h_kv, G = a.h_q / a.h_kv, rows = a.n * G;
  const int rg = blockIdx.x % row_groups, cta = blockIdx.x / row_groups;
  const int n_cta = gridDim.x / row_groups;
  const Work ws = work_of(a.ws, pairs, gridDim.x, slot_rows);

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      tc::mbar_init(smem_u32(&s_full[i]), kProducers / 32);
      tc::mbar_init(smem_u32(&s_empty[i]), TWO ? 2 : 1);
    }
    for (int i = 0; i < 3 * kGroups; ++i) tc::mbar_init(smem_u32(&s_bar[i]), 1);
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
    const int64_t n_work = min((int64_t)n_cta, (total + kMinTiles - 1) / kMinTiles);
    const int64_t begin = cta < n_work ? cta * total / n_work : total;
    const int64_t end = cta < n_work ? (cta + 1) * total / n_work : total;
    if (tid == 0) {
      s_begin = begin;
      s_end = end;
      if (blockIdx.x == 0) {
        ws.head[0] = total;
        ws.head[1] = n_work;
        ws.first[pairs] = total;
      }
    }
    for (int q = q0; q < q1; ++q) {
      const int t = pair_of(a, q).tiles;
      if (begin >= before && begin < before + t) {
        s_pair = q;
        s_tile = (int)(begin - before);
      }
      if (blockIdx.x == 0) ws.first[q] = before;
      before += t;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  pdl_trigger();
  const uint32_t tmem = s_tmem;
  const int64_t todo = s_end - s_begin;
  int pair = s_pair, t0 = s_tile;
  bool fail = false;

  if (warp >= kGroups * 4) {
    // ---- producers: 16 rows of a tile per warp ---------------------------------------------------
    const int pw = warp - kGroups * 4;
    constexpr int kChunks = D / 8;                 // 16-byte chunks per row
    constexpr int kRowsPer = 32 / kChunks ? 32 / kChunks : 1;  // rows per warp copy
    const int shift = 31 - __clz(a.page_size), max_len = a.max_pages * a.page_size;
    // cursor over (pair, tile), one tile ahead of the copies
    Pair p = {};
    Tree tree = {};
    int cur = t0, at_pair = pair;
    int64_t left = todo;
    if (left > 0) {
      p = pair_of(a, at_pair);
      tree = tree_of(a, p.b, lane, pw == 0 && rg == 0);
      if (pw == 0 && lane == 0 && a.seq_lens[p.b] != p.L) raise_flag(4u);
    }
    struct Row {
      const uint16_t* k;  // null: not usable
      const uint16_t* v;
      int64_t store;      // cache offset a new row goes to, or -1
    };
    // the source of row (16 pw + lane) of the cursor's tile (lanes 0-15); the cursor moves on
    auto next_row = [&]() {
      Row r = {nullptr, nullptr, -1};
      const uint64_t used0 = __ballot_sync(kAll, tree.see[0] != 0ull);
      const uint64_t used1 = __ballot_sync(kAll, tree.see[1] != 0ull);
      const uint64_t used = used0 | (used1 << 32);
      const int j = cur * kTT + pw * 16 + lane;
      int node = -1, pos = -1;
      bool want = false;
      if (lane < 16) {
        if (j < p.n_ctx) {
          pos = a.idx ? a.idx[(int64_t)at_pair * a.budget + j] : p.lo + j;
          want = true;
        } else if (j - p.n_ctx < a.n && ((used >> (j - p.n_ctx)) & 1ull)) {
          node = j - p.n_ctx;
          pos = p.L + node;
          want = true;
        }
      }
      if (want) {
        if (pos < 0 || pos >= max_len) {
          raise_flag(2u);
        } else {
          const int pg = a.block_table[(int64_t)p.b * a.max_pages + (pos >> shift)];
          if (pg < 0 || (int64_t)pg >= a.num_pages) {
            raise_flag(1u);
          } else {
            const int64_t off = (int64_t)pg * a.page_stride +
                                (int64_t)(pos & (a.page_size - 1)) * a.slot_stride +
                                (int64_t)p.h * a.head_stride;
            if (node >= 0 && a.k_new) {
              const int64_t src = (((int64_t)p.b * a.n + node) * a.h_kv + p.h) * D;
              r.k = a.k_new + src;
              r.v = a.v_new + src;
              r.store = off;
            } else {
              r.k = a.k_cache + off;
              r.v = a.v_cache + off;
            }
          }
        }
      }
      if (--left > 0 && ++cur == p.tiles) {
        p = pair_of(a, ++at_pair);
        cur = 0;
        tree = tree_of(a, p.b, lane, pw == 0 && rg == 0);
        if (pw == 0 && lane == 0 && a.seq_lens[p.b] != p.L) raise_flag(4u);
      }
      return r;
    };
    Row row = {nullptr, nullptr, -1};
    if (todo > 0) row = next_row();
    const int c = lane % kChunks;
    for (int64_t k = 0; k < todo; ++k) {
      const int st = (int)(k % C::kStages);
      const Row now = row;
      if (k + 1 < todo) row = next_row();
      if (!fail) fail = !tc::mbar_wait(smem_u32(&s_empty[st]), (uint32_t)((k / C::kStages) & 1) ^ 1u, limit);
      const unsigned ok = __ballot_sync(kAll, now.k != nullptr);
      if (lane == 0) s_valid[st][pw] = (uint16_t)ok;
      const uint32_t stage = ring + st * C::kStageBytes;
      bool any_new = false;
#pragma unroll
      for (int it = 0; it < 16 / kRowsPer; ++it) {
        const int u = it * kRowsPer + (kRowsPer == 2 ? lane >> 4 : 0);
        const uint16_t* ks = reinterpret_cast<const uint16_t*>(__shfl_sync(kAll, (unsigned long long)now.k, u));
        const uint16_t* vs = reinterpret_cast<const uint16_t*>(__shfl_sync(kAll, (unsigned long long)now.v, u));
        const int tr = pw * 16 + u;
        const uint32_t dst = stage + (c >> 3) * C::kBlockBytes + tr * 128 + (((c & 7) ^ (tr & 7)) << 4);
        cp_async16(dst, (ks ? ks : a.k_cache) + c * 8, ks ? 16 : 0);
        cp_async16(dst + C::kTileBytes, (vs ? vs : a.v_cache) + c * 8, vs ? 16 : 0);
      }
      cp_async_commit();
      any_new = __any_sync(kAll, now.store >= 0);
      if (any_new && rg == 0) {  // the new nodes' rows into the cache
#pragma unroll 1
        for (int u = 0; u < 16; ++u) {
          const int64_t to = __shfl_sync(kAll, now.store, u);
          const uint4* ks = reinterpret_cast<const uint4*>(__shfl_sync(kAll, (unsigned long long)now.k, u));
          const uint4* vs = reinterpret_cast<const uint4*>(__shfl_sync(kAll, (unsigned long long)now.v, u));
          if (to >= 0 && lane < kChunks) {
            *(reinterpret_cast<uint4*>(a.k_cache + to) + lane) = ks[lane];
            *(reinterpret_cast<uint4*>(a.v_cache + to) + lane) = vs[lane];
          }
        }
      }
      if (k >= C::kAhead) {
        cp_async_wait<C::kAhead>();
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(smem_u32(&s_full[(k - C::kAhead) % C::kStages]));
      }
    }
    cp_async_wait<0>();
    tc::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0)
      for (int64_t k = max((int64_t)0, todo - C::kAhead); k < todo; ++k)
        tc::mbar_arrive(smem_u32(&s_full[k % C::kStages]));
  } else {
    // ---- softmax groups ----------------------------------------------------------------------------
    const int g = warp >> 2, gt = tid & (kM - 1);  // group, thread of the group = tensor-memory lane
    const int gbar = 1 + g;                        // the group's named barrier; 3: both groups
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tq = tmem + C::kQ + g * C::kQCols, ts = tmem + C::kS + g * kTT,
                   to = tmem + C::kO + g * D;
    const uint32_t bar_s = smem_u32(&s_bar[3 * g]), bar_o = smem_u32(&s_bar[3 * g + 1]),
                   bar_d = smem_u32(&s_bar[3 * g + 2]);
    constexpr uint32_t kIdescS = tc::idesc_bf16(kM, kTT, false);
    constexpr uint32_t kIdescO = tc::idesc_bf16(kM, D, true);
    // (a negative scale is a negated Q; a zero scale must not turn the mask's -inf into NaN)
    const float scale_log2 = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1e-37f);
    const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
    const int r = rg * (TWO ? 2 * kM : kM) + (TWO ? g * kM : 0) + gt;  // query row of this thread
    const int node = min(r / G, kTreeMaxNodes - 1);
    uint32_t n_s = 0, n_o = 0;  // phases of bar_s and bar_o so far
    int64_t k0 = 0;             // line index (within the CTA) of the segment's first tile
    while (k0 < todo) {
      const Pair p = pair_of(a, pair);
      const int t1 = (int)min((int64_t)p.tiles, t0 + todo - k0);
      const Tree tree = tree_of(a, p.b, lane, false);
      uint64_t see = tree.of(node);
      if (r >= rows) see = 0ull;
      const bool used = see != 0ull;
      const int depth = __popcll(see) - 1;
      int lo = 0;  // first list index this row sees
      if (a.window > 0) {
        lo = min(max(0, p.L + depth - a.window + 1) - p.lo, p.n_ctx);
        for (int x = depth + 1 - a.window; x > 0; --x) see &= see - 1;  // (ancestors: ascending depth)
      }
      // Q: this thread's row into its lane
      {
        const int64_t qo = (((int64_t)p.b * a.n + node) * a.h_q + (int64_t)p.h * G + r % G) * D;
        const uint4* src = reinterpret_cast<const uint4*>(a.q + (used ? qo : 0));
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint32_t v[32];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const uint4 x = used ? __ldg(src + c * 8 + u) : make_uint4(0u, 0u, 0u, 0u);
            v[4 * u] = x.x ^ flip;
            v[4 * u + 1] = x.y ^ flip;
            v[4 * u + 2] = x.z ^ flip;
            v[4 * u + 3] = x.w ^ flip;
          }
          tc::tmem_st32(tq + lane_base + 32 * c, v);
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        tc::bar_sync(gbar, kM);
      }
      float m_ref = -INFINITY, l = 0.f;
      bool have_o = false;
      const bool active = __any_sync(kAll, used);  // a warp of padding rows only keeps the barriers
      for (int t = t0 + (kHalves ? g : 0); t < t1; t += kHalves ? 2 : 1) {
        const int64_t k = k0 + (t - t0);
        const int st = (int)(k % C::kStages);
        const uint32_t stage = ring + st * C::kStageBytes;
        if (!fail) fail = !tc::mbar_wait(smem_u32(&s_full[st]), (uint32_t)((k / C::kStages) & 1), limit);
        if (gt == 0 && !fail) {
          // (P of the previous tile lies over S: its P V has to be done)
          if (n_o > 0) fail = !tc::mbar_wait(bar_o, (n_o - 1) & 1, limit);
          if (!fail) {
            tc::fence_after_sync();
            const uint64_t b0 = tc::sw128_desc(stage, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              tc::mma_ts(ts, tq + kk * 8,
                         b0 + (uint64_t)(((kk >> 2) * C::kBlockBytes + (kk & 3) * 32) >> 4), kIdescS,
                         kk > 0);
            tc::mma_commit(bar_s);
          }
        }
        // the list indexes of this tile that the row sees
        const uint16_t* vp = s_valid[st];
        uint64_t see_t = (uint64_t)vp[0] | ((uint64_t)vp[1] << 16) | ((uint64_t)vp[2] << 32) | ((uint64_t)vp[3] << 48);
        const int j0 = t * kTT, c_left = p.n_ctx - j0;  // context positions from here on
        if (c_left < kTT) {
          const uint64_t ctx = c_left > 0 ? (1ull << c_left) - 1ull : 0ull;
          const uint64_t tr = c_left >= 0 ? see << c_left : (-c_left < 64 ? see >> -c_left : 0ull);
          see_t &= ctx | tr;
        }
        if (lo > j0) see_t &= lo - j0 < 64 ? ~0ull << (lo - j0) : 0ull;
        if (!used) see_t = ~0ull;  // (its row is discarded)
        // uniform over the CTA: some row may mask a position that is in the tile
        const bool special = c_left < kTT || (a.window > 0 && t == 0);

        if (!fail) fail = !tc::mbar_wait(bar_s, n_s & 1, limit);
        ++n_s;
        tc::fence_after_sync();
        uint32_t ph[32];
        if (active) {
          uint32_t s0[32], s1[32];
          tc::tmem_ld32(ts + lane_base, s0);
          tc::tmem_ld32(ts + lane_base + 32, s1);
          tc::tmem_wait_ld();
          float x[kTT];
          if (__all_sync(kAll, see_t == ~0ull)) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              x[j] = __uint_as_float(s0[j]);
              x[j + 32] = __uint_as_float(s1[j]);
            }
          } else {
            const uint32_t lo32 = (uint32_t)see_t, hi32 = (uint32_t)(see_t >> 32);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              x[j] = ((lo32 >> j) & 1u) ? __uint_as_float(s0[j]) : -INFINITY;
              x[j + 32] = ((hi32 >> j) & 1u) ? __uint_as_float(s1[j]) : -INFINITY;
            }
          }
          float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int j = 4; j < kTT; j += 4)
#pragma unroll
            for (int u = 0; u < 4; ++u) mx[u] = fmaxf(mx[u], x[j + u]);
          const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale_log2;
          // lazy rescale: weights are relative to m_ref, which moves only when the row's maximum
          // exceeds it by more than the slack (weights stay <= 2^8)
          const bool grow = mt > m_ref + kRescaleSlack;
          const float m_new = grow ? mt : m_ref;
          const float corr = grow && m_ref != -INFINITY ? fast_exp2(m_ref - m_new) : 1.f;
          if (have_o && __any_sync(kAll, corr != 1.f)) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tc::tmem_ld32(to + lane_base + 32 * c, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
              tc::tmem_st32(to + lane_base + 32 * c, o);
            }
          }
          m_ref = m_new;
          const float m_sub = m_ref == -INFINITY ? 0.f : m_ref;
          float sum[2] = {0.f, 0.f};
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float p0 = fast_exp2(fmaf(x[2 * j], scale_log2, -m_sub));
            const float p1 = fast_exp2(fmaf(x[2 * j + 1], scale_log2, -m_sub));
            sum[0] += p0;
            sum[1] += p1;
            ph[j] = pack_bf16x2(p0, p1);
          }
          l = l * corr + (sum[0] + sum[1]);
          tc::tmem_st32(ts + lane_base, ph);
        }
        bool keep_o = have_o;
        if (special) {
          // this thread's half row of V: any exponent of all ones
          const uint32_t vrow = stage + C::kTileBytes + (gt >> 1) * 128;
          constexpr int kPer = D / 16;  // 16-byte chunks of half a row
          auto chunk = [&](int q) {
            const int c = (gt & 1) * kPer + q;
            return vrow + (c >> 3) * C::kBlockBytes + (((c & 7) ^ ((gt >> 1) & 7)) << 4);
          };
          auto odd = [](uint32_t w) { return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u; };
          auto ld = [](uint32_t at) {
            uint4 y;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w) : "r"(at) : "memory");
            return y;
          };
          bool mine = false;
#pragma unroll
          for (int q = 0; q < kPer; ++q) {
            const uint4 y = ld(chunk(q));
            mine |= odd(y.x) | odd(y.y) | odd(y.z) | odd(y.w);
          }
          const int vbar = TWO ? 3 : gbar, vthreads = TWO ? 2 * kM : kM;
          if (tc::bar_or(vbar, vthreads, mine)) {
            const unsigned two = __ballot_sync(kAll, mine);
            if (lane == 0) s_bad[g][warp & 3] = two;  // bit 2 i (+ 1): token 16 w + i
            tc::bar_sync(gbar, kM);
            // add p v of the non-finite elements to the rows that see them (O = 0 first)
            tc::tmem_wait_st();
            uint32_t pl[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) pl[j] = ph[j];
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              if (have_o) {
                tc::tmem_ld32(to + lane_base + 32 * c, o);
                tc::tmem_wait_ld();
              } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = 0u;
              }
#pragma unroll 1
              for (int j = 0; j < kTT; ++j) {
                if (!((s_bad[g][j >> 4] >> (2 * (j & 15))) & 3u)) continue;
                const uint32_t w = pl[j >> 1];
                const float pj = (j & 1) ? bf16_hi(w) : bf16_lo(w);
                const bool sees = (see_t >> j) & 1ull;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const int cc = 4 * c + q;
                  const uint4 y = ld(stage + C::kTileBytes + (cc >> 3) * C::kBlockBytes + j * 128 +
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
              tc::tmem_st32(to + lane_base + 32 * c, o);
            }
            keep_o = true;
            tc::bar_sync(vbar, vthreads);  // everyone has read V
            if (!TWO || g == 0) {          // clear the elements for the MMA
#pragma unroll 1
              for (int q = 0; q < kPer; ++q) {
                const uint4 y = ld(chunk(q));
                uint32_t yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  if ((yw[e] & 0x7F80u) == 0x7F80u) yw[e] &= 0xFFFF0000u;
                  if ((yw[e] & 0x7F800000u) == 0x7F800000u) yw[e] &= 0x0000FFFFu;
                }
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(chunk(q)), "r"(yw[0]),
                             "r"(yw[1]), "r"(yw[2]), "r"(yw[3]) : "memory");
              }
              tc::fence_proxy_async_smem();
            }
            if (TWO) tc::bar_sync(vbar, vthreads);
          }
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        tc::bar_sync(gbar, kM);
        if (gt == 0 && !fail) {
          tc::fence_after_sync();
#pragma unroll
          for (int kk = 0; kk < kTT / 16; ++kk)
            tc::mma_ts(to, ts + kk * 8,
                       tc::sw128_desc(stage + C::kTileBytes + kk * 16 * 128, C::kBlockBytes, 1024),
                       kIdescO, keep_o || kk > 0);
          tc::mma_commit(bar_o);
          tc::mma_commit(smem_u32(&s_empty[st]));
        }
        ++n_o;
        have_o = true;
      }
      if (have_o && !fail) fail = !tc::mbar_wait(bar_o, (n_o - 1) & 1, limit);
      tc::fence_after_sync();

      // ---- the segment's rows: into the output when the pair is whole, else into a partial slot
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
      uint16_t* orow = a.out + (((int64_t)p.b * a.n + node) * a.h_q + (int64_t)p.h * G + r % G) * D;
      constexpr int kPart = kHalves ? D / 64 : D / 32;  // 32-column pieces written by this group
#pragma unroll 1
      for (int c = (kHalves ? g * kPart : 0); c < (kHalves ? g * kPart : 0) + kPart; ++c) {
        uint32_t o[32];
        if (have_o) {
          tc::tmem_ld32(to + lane_base + 32 * c, o);
          tc::tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = mine ? __float_as_uint(__uint_as_float(o[e]) * w0) : 0u;
        if (kHalves) {
          if (__any_sync(kAll, other)) {
            uint32_t y[32];
            tc::tmem_ld32(tmem + C::kO + (g ^ 1) * D + lane_base + 32 * c, y);
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
    // everything this group issued has completed before the tensor memory is freed
    if (gt == 0) {
      tc::mma_commit(bar_d);
      if (!tc::mbar_wait(bar_d, 0)) fail = true;
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

// Merge of the pairs that several CTAs share: one warp per query row,
//   M = max m_i,  w_i = 2^(m_i - M),  out = sum w_i O_i / sum w_i l_i.
constexpr int kMergeWarps = 8;
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32)
    merge_kernel(TreeArgs a, int row_groups, int group_rows, int slot_rows, int ctas) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int pair = blockIdx.x / row_groups, rg = blockIdx.x % row_groups;
  const int pairs = a.batch * a.h_kv, G = a.h_q / a.h_kv;
  const Work ws = work_of(a.ws, pairs, ctas, slot_rows);
  pdl_wait();
  const int64_t total = ws.head[0], n = ws.head[1], s0 = ws.first[pair], s1 = ws.first[pair + 1];
  // CTA c covers tiles [c total / n, (c + 1) total / n): the one that holds tile t
  auto holder = [&](int64_t t) {
    int64_t c = t * n / total;
    while ((c + 1) * total / n <= t) ++c;
    while (c * total / n > t) --c;
    return (int)c;
  };
  const int c0 = holder(s0), c1 = holder(s1 - 1);
  if (c0 == c1) return;  // written by the CTA itself
  const int lr = blockIdx.y * kMergeWarps + warp, r = rg * group_rows + lr;
  if (lr >= slot_rows || r >= a.n * G) return;
  // partial i: CTA c0 + i; the first one is its CTA's last segment, the others' their first
  const int parts = c1 - c0 + 1;
  auto row_of = [&](int i) {
    const int64_t c = c0 + i;
    const int second = i == 0 && c * total / n < s0 ? 1 : 0;
    return (2 * (c * row_groups + rg) + second) * (int64_t)slot_rows + lr;
  };
  float M = -INFINITY;
  for (int i = lane; i < parts; i += 32) M = fmaxf(M, ws.ml[row_of(i)].x);
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kAll, M, o));
  float acc[D / 32], l = 0.f;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) acc[e] = 0.f;
  for (int i0 = 0; i0 < parts; i0 += 32) {
    float w = 0.f;
    if (i0 + lane < parts) {
      const float2 ml = ws.ml[row_of(i0 + lane)];
      w = merge_weight(ml.x, ml.y, M);
      if (w != 0.f) l += w * ml.y;
    }
    const int m = min(32, parts - i0);
#pragma unroll 4
    for (int i = 0; i < m; ++i) {
      const float wi = __shfl_sync(kAll, w, i);
      const float4* o = reinterpret_cast<const float4*>(ws.o + row_of(i0 + i) * D);
#pragma unroll
      for (int q = 0; q < D / 128; ++q) {
        const float4 x = o[q * 32 + lane];
        if (wi != 0.f) {
          acc[4 * q] += wi * x.x;
          acc[4 * q + 1] += wi * x.y;
          acc[4 * q + 2] += wi * x.z;
          acc[4 * q + 3] += wi * x.w;
        }
      }
    }
  }
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(kAll, l, o);
  const float inv = inverse_sum(l);
  const int b = pair / a.h_kv, h = pair % a.h_kv;
  uint16_t* out = a.out + (((int64_t)b * a.n + r / G) * a.h_q + (int64_t)h * G + r % G) * D;
#pragma unroll
  for (int q = 0; q < D / 128; ++q)
    reinterpret_cast<uint2*>(out)[q * 32 + lane] =
        make_uint2(pack_bf16x2(acc[4 * q] * inv, acc[4 * q + 1] * inv),
                   pack_bf16x2(acc[4 * q + 2] * inv, acc[4 * q + 3] * inv));
}

template <int D, bool TWO>
cudaError_t launch_t(const TreeArgs& a, const Plan& plan, cudaStream_t s) {
  auto kern = tree_kernel<D, TWO>;
  cudaError_t e = configure_kernel((const void*)kern, Cfg<D>::kSmem, false);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(plan.ctas, 1, 1);
  cfg.blockDim = dim3(Cfg<D>::kThreads, 1, 1);
  cfg.dynamicSmemBytes = Cfg<D>::kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, a, plan.row_groups, plan.slot_rows, tc_wait_limit());
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(a.batch * a.h_kv * plan.row_groups, (plan.slot_rows + kMergeWarps - 1) / kMergeWarps, 1);
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
  return up256(((size_t)batch * h_kv + 3) * 8) + up256(rows * sizeof(float2)) + rows * d * sizeof(float);
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
