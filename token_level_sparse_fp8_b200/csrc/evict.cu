// Moves of cached rows inside the paged cache: commit (the accepted nodes of a drafted tree become
// consecutive positions) and eviction (the positions that keep their place are those with the
// largest accumulated attention mass, plus the most recent ones; heavy-hitter eviction). A row is
// everything the cache holds of one position and KV head: K, V, the scoring code and, for
// eviction, the running mass.
//
// Order of reads and writes. Eviction's sources ascend, src[i] >= i = dst[i], so a row read for a
// later i is never one that an earlier i writes; only a write must wait for the reads of the rows
// before it. Rows are therefore moved in tiles: a tile's rows are read into registers, all of them
// (barrier), then written. That order makes the move safe in place.
#include <limits.h>

#include "common.cuh"

namespace jssa {

namespace evict_detail {

constexpr unsigned kAll = 0xffffffffu;

// The part of one position's row that a lane moves: 16-byte chunks of K and V (lanes 0-15 K and
// 16-31 V at d = 128; chunk `lane` of both at d = 256).
template <int D>
struct LaneRow {
  static constexpr int kParts = D / 128;
  uint4 x[kParts];
  __device__ __forceinline__ static int64_t chunk(int lane) {
    return D == 128 ? (lane & 15) * 8 : lane * 8;
  }
  __device__ __forceinline__ void load(const uint16_t* k, const uint16_t* v, int64_t off, int lane) {
    if (D == 128) {
      x[0] = *reinterpret_cast<const uint4*>((lane < 16 ? k : v) + off + chunk(lane));
    } else {
      x[0] = *reinterpret_cast<const uint4*>(k + off + chunk(lane));
      x[kParts - 1] = *reinterpret_cast<const uint4*>(v + off + chunk(lane));
    }
  }
  __device__ __forceinline__ void store(uint16_t* k, uint16_t* v, int64_t off, int lane) const {
    if (D == 128) {
      *reinterpret_cast<uint4*>((lane < 16 ? k : v) + off + chunk(lane)) = x[0];
    } else {
      *reinterpret_cast<uint4*>(k + off + chunk(lane)) = x[0];
      *reinterpret_cast<uint4*>(v + off + chunk(lane)) = x[kParts - 1];
    }
  }
};

// Page of logical position `pos` in a table row of `max_pages` pages; -1 (flagged) when unusable.
__device__ __forceinline__ int page_of(const RowMove& m, const int32_t* table, int max_pages, int pos) {
  if (pos < 0 || pos >= max_pages * m.page_size) {
    raise_flag(2u);
    return -1;
  }
  const int pg = table[pos / m.page_size];
  if (pg < 0 || (int64_t)pg >= m.num_pages) {
    raise_flag(1u);
    return -1;
  }
  return pg;
}
__device__ __forceinline__ int64_t kv_offset(const RowMove& m, int pg, int pos, int h) {
  return (int64_t)pg * m.page_stride + (int64_t)(pos % m.page_size) * m.slot_stride +
         (int64_t)h * m.head_stride;
}
__device__ __forceinline__ int64_t code_offset(const RowMove& m, int pg, int pos, int h) {
  return (((int64_t)pg * m.h_kv + h) * m.page_size + pos % m.page_size) * m.code_bytes;
}

// Where a warp's rows come from and go to: lane u holds row u's positions and pages (-1: the row is
// not moved).
struct Ends {
  int src_pos, dst_pos, src_pg, dst_pg;
};

// A warp's tile of at most kRows (4 or 8) rows: the K / V chunks of every row, one scoring chunk and one mass value
// per lane.
template <int D, int kRows>
struct WarpTile {
  LaneRow<D> kv[kRows];
  uint4 code;
  float mass;

  __device__ __forceinline__ void load(const RowMove& m, int h, const float* mass_row, const Ends& e,
                                       int lane) {
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int pg = __shfl_sync(kAll, e.src_pg, u), pos = __shfl_sync(kAll, e.src_pos, u);
      if (pg >= 0) kv[u].load(m.k_cache, m.v_cache, kv_offset(m, pg, pos, h), lane);
    }
    if (m.code_bytes) {
      const int per = m.code_bytes >> 4, u = lane / per;  // chunks per row; this lane's row
      const int pg = __shfl_sync(kAll, e.src_pg, u & 7), pos = __shfl_sync(kAll, e.src_pos, u & 7);
      if (u < kRows && pg >= 0)
        code = *reinterpret_cast<const uint4*>(m.score_cache + code_offset(m, pg, pos, h) + (lane % per) * 16);
    }
    if (mass_row && lane < kRows && e.src_pg >= 0) mass = mass_row[e.src_pos];
  }
  __device__ __forceinline__ void store(const RowMove& m, int h, float* mass_row, const Ends& e,
                                        int lane) const {
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int pg = __shfl_sync(kAll, e.dst_pg, u), pos = __shfl_sync(kAll, e.dst_pos, u);
      if (pg >= 0) kv[u].store(m.k_cache, m.v_cache, kv_offset(m, pg, pos, h), lane);
    }
    if (m.code_bytes) {
      const int per = m.code_bytes >> 4, u = lane / per;
      const int pg = __shfl_sync(kAll, e.dst_pg, u & 7), pos = __shfl_sync(kAll, e.dst_pos, u & 7);
      if (u < kRows && pg >= 0)
        *reinterpret_cast<uint4*>(m.score_cache + code_offset(m, pg, pos, h) + (lane % per) * 16) = code;
    }
    if (mass_row && lane < kRows && e.dst_pg >= 0) mass_row[e.dst_pos] = mass;
  }
};

__device__ __forceinline__ int clamped_len(const RowMove& m, int b, bool report) {
  const int max_len = m.max_pages * m.page_size;
  int L = m.seq_lens[b];
  if (L < 0 || L > max_len) {
    if (report) raise_flag(4u);
    L = L < 0 ? 0 : max_len;
  }
  return L;
}

// ---- commit --------------------------------------------------------------------------------
// Grid batch * h_kv; 8 warps hold the at most 64 rows of one (sequence, KV head) at once, so the
// order of the path does not matter. Latency-bound: one dependent chain of path, page and row (3.6 us
// for one sequence, 5.2 us for 64 of 9 rows each).
constexpr int kCommitThreads = 256;
constexpr int kCommitRows = 8;
static_assert(kCommitThreads / 32 * kCommitRows == kTreeMaxNodes, "all rows of a tree in registers");

template <int D>
__global__ void __launch_bounds__(kCommitThreads)
    commit_kernel(RowMove m, const int32_t* path, const int32_t* n_path, int max_path) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.x / m.h_kv, h = blockIdx.x % m.h_kv;
  const bool report = h == 0 && threadIdx.x == 0;
  const int L = clamped_len(m, b, report);
  int n = n_path[b];
  if (n < 0 || n > max_path) {
    if (report) raise_flag(2u);
    n = n < 0 ? 0 : max_path;
  }
  const int room = m.max_pages * m.page_size - L;
  if (n > room) {
    if (report) raise_flag(2u);
    n = room;
  }
  if (report) m.lens_out[b] = L + n;
  const int32_t* table = m.block_table + (int64_t)b * m.max_pages;
  Ends ends = {-1, -1, -1, -1};
  const int i = warp * kCommitRows + lane;
  if (lane < kCommitRows && i < n) {
    const int node = path[(int64_t)b * max_path + i];
    if (node < 0 || node >= kTreeMaxNodes) {
      raise_flag(2u);
    } else {  // (a node that keeps its position only has its page checked)
      const int sp = page_of(m, table, m.max_pages, L + node);
      const int dp = node != i ? page_of(m, table, m.max_pages, L + i) : -1;
      if (sp >= 0 && dp >= 0) ends = {L + node, L + i, sp, dp};
    }
  }
  WarpTile<D, kCommitRows> t;
  t.load(m, h, nullptr, ends, lane);
  __syncthreads();
  t.store(m, h, nullptr, ends, lane);
}

// ---- evict ---------------------------------------------------------------------------------
// Selection: a cluster of C CTAs per (sequence, KV head), C as large as fits one wave.
//   (1) The key of rank keep - recent among positions [0, L - recent): exact radix selection, 11 +
//       11 + 10 bits, each CTA counting its slice of the positions; the C histograms are summed
//       through distributed shared memory.
//   (2) The kept positions in ascending order: each warp owns a contiguous range, counts its keys
//       above and at the threshold, and writes its part after a scan over warps and CTAs.
// Measured on one B200: 16 sequences of 64K down to 32K cut to 16K (8 heads, d 128, 32-byte codes) 62 us
// of selection and 386 us of moves (5.9 TB/s read and written); one of 4K cut to 2K 10 + 5 us.
// The selection passes five times over the 4 bytes of each position, the last four out of L2: bound by the
// instructions of a pass. The rows then move (HBM-bound: each is read once and written once)
//   * into other pages by a kernel of its own with a short-lived warp per few rows: nothing orders
//     them, and many small blocks keep more rows in flight than a persistent loop (6.2 against 4.5
//     TB/s of a copy of random 256-byte rows);
//   * in place by the cluster that selected them, in tiles of C x 128 rows (64 at d = 256): the rows
//     of the next tile, the pages of the one after and the positions of the one after that are in
//     flight while a tile is written, with a cluster barrier between a tile's reads and its writes.
constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kEvictMaxCluster = 8;  // the portable size
constexpr int kBins = 2048;          // four per thread
constexpr int kFlight = 8;           // loads of mass in flight per lane
constexpr int kClusterSpan = 8192;   // positions per CTA before more CTAs take part

// Order-preserving key of a running mass; every NaN counts as the largest value.
constexpr uint32_t kNanKey = 0xffffffffu;
__device__ __forceinline__ uint32_t mass_key(float x) {
  return x != x ? kNanKey : score_key(x);
}
// The value of a key other than NaN's (-0 has become +0, which compares the same).
__device__ __forceinline__ float key_mass(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// f(position, value, whether the position is in [lo, hi)) for a warp's positions, kFlight x 32 at a
// time; every lane makes every call.
template <class F>
__device__ __forceinline__ void each_mass(const float* mass, int lo, int hi, int lane, F f) {
  int p = lo;
  for (; p + 32 * kFlight <= hi; p += 32 * kFlight) {
    float x[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) x[u] = mass[p + 32 * u + lane];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) f(p + 32 * u + lane, x[u], true);
  }
#pragma unroll 1
  for (; p < hi; p += 32) {
    const int q = p + lane;
    f(q, q < hi ? mass[q] : 0.f, q < hi);
  }
}

struct SelectShared {
  __align__(16) uint32_t hist[2][kBins];  // alternating, so one barrier a round is enough
  __align__(16) uint4 counts;             // of this CTA: above, equal, first position out
  int above[kEvictWarps], equal[kEvictWarps], first, want;
  uint32_t bin, scan[kEvictWarps];
};
struct Kept {
  int L, n_keep, first_out;  // length, positions kept, the first one that is not (or above)
};

// Writes idx, count and lens_out of the cluster's pair; on return they are visible to the cluster.
__device__ __forceinline__ Kept select_kept(const RowMove& m, const EvictArgs& e, SelectShared& sh,
                                            int cluster) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % cluster, pair = blockIdx.x / cluster;
  const int b = pair / m.h_kv, h = pair % m.h_kv;
  const int L = clamped_len(m, b, h == 0 && rank == 0 && tid == 0);
  const int n_keep = min(L, e.keep);
  const float* mass = e.mass + (int64_t)pair * e.mass_stride;
  int32_t* idx = e.idx + (int64_t)pair * e.keep;
  if (tid == 0) {
    sh.first = INT_MAX;
    if (rank == 0) {
      e.count[pair] = n_keep;
      if (h == 0) m.lens_out[b] = n_keep;
    }
  }
  __syncthreads();
  // this warp's positions: the CTA's slice of [0, L), a 16th of it
  const int per_warp = ((L + cluster * kEvictWarps - 1) / (cluster * kEvictWarps) + 31) / 32 * 32;
  const int p_lo = min((int64_t)L, (int64_t)(rank * kEvictWarps + warp) * per_warp);
  const int p_hi = max(p_lo, min(L, p_lo + per_warp));
  const int n_cand = L > e.keep ? L - e.recent : 0;  // positions that compete
  int want = L > e.keep ? e.keep - e.recent : 0;     // for so many places
  const bool pick = want > 0;
  uint32_t edge = 0u;
  if (pick) {
#pragma unroll 1
    for (int round = 0; round < 3; ++round) {
      uint32_t* hist = sh.hist[round & 1];
      const int shift = round == 0 ? 21 : round == 1 ? 10 : 0;
      reinterpret_cast<uint4*>(hist)[tid] = make_uint4(0u, 0u, 0u, 0u);
      __syncthreads();
      const int hi = min(p_hi, n_cand);
      if (round == 0) {
        each_mass(mass, p_lo, hi, lane, [&](int, float x, bool in) {
          const uint32_t bin = mass_key(x) >> 21, bin0 = __shfl_sync(kAll, bin, 0);
          // (equal keys in a whole warp, as of untouched positions, would serialise)
          if (__all_sync(kAll, in && bin == bin0)) {
            if (lane == 0) atomicAdd(&hist[bin], 32u);
          } else if (in) {
            atomicAdd(&hist[bin], 1u);
          }
        });
      } else {
        const int low = round == 1 ? 21 : 10;  // bits below the prefix found so far
        each_mass(mass, p_lo, hi, lane, [&](int, float x, bool in) {
          const uint32_t key = mass_key(x);
          if (in && (key ^ edge) >> low == 0u) atomicAdd(&hist[(key >> shift) & ((1u << (low - shift)) - 1u)], 1u);
        });
      }
      if (cluster > 1) cluster_sync();
      else __syncthreads();
      // thread t: bins of descending order 4 t .. 4 t + 3, over the whole cluster
      const uint32_t at = smem_u32(hist) + (kBins - 4 - 4 * tid) * 4;
      uint4 c = make_uint4(0u, 0u, 0u, 0u);
      for (int r = 0; r < cluster; ++r) {
        const uint4 x = cluster > 1 ? ld_cluster_v4(cluster_addr(at, r)) : ld_shared_v4(at);
        c.x += x.x; c.y += x.y; c.z += x.z; c.w += x.w;
      }
      const uint32_t mine = c.x + c.y + c.z + c.w;
      uint32_t incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(kAll, incl, o);
        if (lane >= o) incl += x;
      }
      if (lane == 31) sh.scan[warp] = incl;
      __syncthreads();
      uint32_t before = incl - mine;
      for (int w = 0; w < warp; ++w) before += sh.scan[w];
      if (before < (uint32_t)want && before + mine >= (uint32_t)want) {
        const uint32_t n[4] = {c.w, c.z, c.y, c.x};  // descending
        uint32_t left = want - before, bin = kBins - 1 - 4 * tid;
        for (int u = 0; u < 4 && n[u] < left; ++u) {
          left -= n[u];
          --bin;
        }
        sh.want = left;
        sh.bin = bin;
      }
      __syncthreads();
      want = sh.want;  // keys to take of those with this prefix
      edge |= sh.bin << shift;
    }
  }
  const int n_equal = pick ? want : 0;  // keys equal to the edge that stay, lowest positions first
  // positions before n_cand stay if they are above the edge, or equal to it and early enough; those
  // from n_cand on (the recent ones, or all when nothing is evicted) stay
  const bool nan_edge = pick && edge == kNanKey;
  const float edge_x = pick ? key_mass(edge) : 0.f;
  auto is_above = [&](float x) { return pick && !nan_edge && !(x <= edge_x); };
  auto is_equal = [&](float x) { return pick && (nan_edge ? x != x : x == edge_x); };
  const int split = max(p_lo, min(p_hi, n_cand));  // this warp's first position that stays anyway
  int above = 0, equal = 0, first = INT_MAX;
  each_mass(mass, p_lo, split, lane, [&](int q, float x, bool in) {
    const bool a = in && is_above(x);
    above += a;
    equal += in && is_equal(x);
    if (in && !a) first = min(first, q);
  });
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    above += __shfl_xor_sync(kAll, above, o);
    equal += __shfl_xor_sync(kAll, equal, o);
    first = min(first, __shfl_xor_sync(kAll, first, o));
  }
  above += p_hi - split;
  if (lane == 0) {
    sh.above[warp] = above;
    sh.equal[warp] = equal;
    if (first != INT_MAX) atomicMin(&sh.first, first);
  }
  __syncthreads();
  if (warp == 0) {
    int a = lane < kEvictWarps ? sh.above[lane] : 0, q = lane < kEvictWarps ? sh.equal[lane] : 0;
    for (int o = 16; o; o >>= 1) {
      a += __shfl_xor_sync(kAll, a, o);
      q += __shfl_xor_sync(kAll, q, o);
    }
    if (lane == 0) sh.counts = make_uint4(a, q, sh.first, 0u);
  }
  if (cluster > 1) cluster_sync();
  else __syncthreads();
  int base = 0, eq_before = 0, first_out = INT_MAX;
  for (int r = 0; r < cluster; ++r) {
    const uint32_t at = smem_u32(&sh.counts);
    const uint4 c = cluster > 1 ? ld_cluster_v4(cluster_addr(at, r)) : ld_shared_v4(at);
    first_out = min(first_out, (int)c.z);
    if (r < rank) {
      base += c.x + max(0, min((int)c.y, n_equal - eq_before));
      eq_before += c.y;
    }
  }
  for (int w = 0; w < warp; ++w) {
    base += sh.above[w] + max(0, min(sh.equal[w], n_equal - eq_before));
    eq_before += sh.equal[w];
  }
  const unsigned below = (1u << lane) - 1u;
  each_mass(mass, p_lo, split, lane, [&](int q, float x, bool in) {
    const unsigned eq = __ballot_sync(kAll, in && is_equal(x));
    bool stay = in && is_above(x);
    if (eq) {
      stay = stay || (in && is_equal(x) && eq_before + __popc(eq & below) < n_equal);
      eq_before += __popc(eq);
    }
    const unsigned st = __ballot_sync(kAll, stay);
    if (stay) __stcg(&idx[base + __popc(st & below)], q);
    base += __popc(st);
  });
  for (int q = split + lane; q < p_hi; q += 32) __stcg(&idx[base + q - split], q);
  for (int i = n_keep + rank * kEvictThreads + tid; i < e.keep; i += cluster * kEvictThreads) idx[i] = -1;
  if (cluster > 1) cluster_sync();
  else __syncthreads();
  return {L, n_keep, first_out};
}

// Selection alone, and zeros in the mass of the positions left over (mass_out is not mass).
__global__ void __launch_bounds__(kEvictThreads, 2) select_kernel(RowMove m, EvictArgs e, int cluster) {
  __shared__ SelectShared sh;
  const Kept k = select_kept(m, e, sh, cluster);
  const int rank = blockIdx.x % cluster, pair = blockIdx.x / cluster;
  float* mass_out = e.mass_out + (int64_t)pair * e.mass_stride;
  for (int p = k.n_keep + rank * kEvictThreads + threadIdx.x; p < k.L; p += cluster * kEvictThreads)
    mass_out[p] = 0.f;
}

// Looks up a row's pages; they may still be in flight on return (see usable).
__device__ __forceinline__ Ends look_up(const RowMove& m, const EvictArgs& e, const int32_t* table,
                                        const int32_t* dst_table, int src, int dst) {
  Ends r = {-1, -1, -1, -1};
  if (src >= 0) {
    r.src_pos = src;
    r.dst_pos = dst;
    r.src_pg = src < m.max_pages * m.page_size ? table[src / m.page_size] : -2;
    r.dst_pg = dst < e.dst_max_pages * m.page_size ? dst_table[dst / m.page_size] : -2;
  }
  return r;
}
// Both pages have to be usable (-2: beyond the table).
__device__ __forceinline__ void usable(const RowMove& m, Ends& r) {
  if (r.src_pos < 0) return;
  const bool beyond = r.src_pg == -2 || r.dst_pg == -2;
  const bool bad = (r.src_pg != -2 && (r.src_pg < 0 || r.src_pg >= m.num_pages)) ||
                   (r.dst_pg != -2 && (r.dst_pg < 0 || r.dst_pg >= m.num_pages));
  if (beyond || bad) {
    raise_flag((beyond ? 2u : 0u) | (bad ? 1u : 0u));
    r.src_pg = r.dst_pg = -1;
  }
}

// The rows of one eviction into other pages: grid (row blocks, pairs), 32 rows per warp. Lane u looks
// up row u; the K / V chunks then go through registers in groups, one being read while one is written.
constexpr int kMoveThreads = 128;
template <int D>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(RowMove m, EvictArgs e) {
  constexpr int kGroup = D == 128 ? 4 : 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int pair = blockIdx.y, b = pair / m.h_kv, h = pair % m.h_kv;
  pdl_wait();
  const int i = (blockIdx.x * (kMoveThreads / 32) + warp) * 32 + lane;
  const int src = i < e.keep ? e.idx[(int64_t)pair * e.keep + i] : -1;  // (-1: padding)
  if (__all_sync(kAll, src < 0)) return;
  Ends ends = look_up(m, e, m.block_table + (int64_t)b * m.max_pages,
                      e.dst_table + (int64_t)b * e.dst_max_pages, src, i);
  usable(m, ends);
  const int64_t from = ends.src_pg >= 0 ? kv_offset(m, ends.src_pg, ends.src_pos, h) : -1;
  const int64_t to = ends.dst_pg >= 0 ? kv_offset(m, ends.dst_pg, ends.dst_pos, h) : -1;
  LaneRow<D> x[2][kGroup];
  auto read = [&](LaneRow<D>(&r)[kGroup], int g) {
#pragma unroll
    for (int u = 0; u < kGroup; ++u) {
      const int64_t off = __shfl_sync(kAll, from, g * kGroup + u);
      if (off >= 0) r[u].load(m.k_cache, m.v_cache, off, lane);
    }
  };
  auto write = [&](const LaneRow<D>(&r)[kGroup], int g) {
#pragma unroll
    for (int u = 0; u < kGroup; ++u) {
      const int64_t off = __shfl_sync(kAll, to, g * kGroup + u);
      if (off >= 0) r[u].store(m.k_cache, m.v_cache, off, lane);
    }
  };
  read(x[0], 0);
  // mass: lane u's row; scoring codes: 16-byte chunks, `per` of a row side by side
  const float mass = src >= 0 ? e.mass[(int64_t)pair * e.mass_stride + src] : 0.f;
  if (to >= 0) e.mass_out[(int64_t)pair * e.mass_stride + i] = mass;
#pragma unroll 1
  for (int g = 0; g < 32 / kGroup; g += 2) {
    read(x[1], g + 1);
    write(x[0], g);
    if (g + 2 < 32 / kGroup) read(x[0], g + 2);
    write(x[1], g + 1);
  }
  const int per = m.code_bytes >> 4;
#pragma unroll 1
  for (int c = 0; c < per; ++c) {
    const int u = (c * 32 + lane) / per, at = (c * 32 + lane) % per * 16;
    const int sp = __shfl_sync(kAll, ends.src_pg, u), ss = __shfl_sync(kAll, ends.src_pos, u);
    const int dp = __shfl_sync(kAll, ends.dst_pg, u), ds = __shfl_sync(kAll, ends.dst_pos, u);
    if (sp >= 0)
      *reinterpret_cast<uint4*>(m.score_cache + code_offset(m, dp, ds, h) + at) =
          *reinterpret_cast<const uint4*>(m.score_cache + code_offset(m, sp, ss, h) + at);
  }
}

template <int D>
__global__ void __launch_bounds__(kEvictThreads, 1)
    evict_in_place_kernel(RowMove m, EvictArgs e, int cluster) {
  constexpr int kRows = D == 128 ? 8 : 4;  // per warp and tile: two tiles in registers
  __shared__ SelectShared sh;
  const Kept k = select_kept(m, e, sh, cluster);
  const int L = k.L, n_keep = k.n_keep;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % cluster, pair = blockIdx.x / cluster;
  const int b = pair / m.h_kv, h = pair % m.h_kv;
  const float* mass = e.mass + (int64_t)pair * e.mass_stride;
  float* mass_out = e.mass_out + (int64_t)pair * e.mass_stride;
  const int32_t* idx = e.idx + (int64_t)pair * e.keep;
  // the rows before the first one out stay where they are (unless the mass or the pages are others)
  const int32_t* table = m.block_table + (int64_t)b * m.max_pages;
  const int32_t* dst_table = e.dst_table + (int64_t)b * e.dst_max_pages;
  const int span = cluster * kEvictWarps * kRows;
  const bool stays = e.dst_table == m.block_table && e.mass_out == e.mass;
  const int i_begin = stays ? min(k.first_out, n_keep) : 0;
  const int n_tiles = (n_keep - i_begin + span - 1) / span;
  const int row0 = i_begin + (rank * kEvictWarps + warp) * kRows + lane;  // (the first lanes)
  auto position = [&](int t) {  // of this lane's row of tile t; -1: none
    const int i = row0 + t * span;
    return lane < kRows && t < n_tiles && i < n_keep ? __ldcg(&idx[i]) : -1;
  };
  auto ends_of = [&](int t, int pos) { return look_up(m, e, table, dst_table, pos, row0 + t * span); };
  // a step writes tile t (`cur`) after the reads of tile t + 1 (`nxt`) have been issued
  WarpTile<D, kRows> ta, tb;
  Ends ea, eb, ahead;
  ea = ends_of(0, position(0));
  ahead = ends_of(1, position(1));
  int pos = position(2);
  usable(m, ea);
  ta.load(m, h, mass, ea, lane);
  auto step = [&](int t, const WarpTile<D, kRows>& cur, const Ends& ce, WarpTile<D, kRows>& nxt, Ends& ne) {
    ne = ahead;
    usable(m, ne);
    nxt.load(m, h, mass, ne, lane);
    ahead = ends_of(t + 2, pos);
    pos = position(t + 3);
    if (cluster > 1) cluster_sync();
    else __syncthreads();
    cur.store(m, h, mass_out, ce, lane);
  };
#pragma unroll 1
  for (int t = 0; t < n_tiles; t += 2) {
    step(t, ta, ea, tb, eb);
    if (t + 1 < n_tiles) step(t + 1, tb, eb, ta, ea);
  }
  // (the last tile's barrier came after the last read of the mass)
  for (int p = n_keep + rank * kEvictThreads + tid; p < L; p += cluster * kEvictThreads) mass_out[p] = 0.f;
}

}  // namespace evict_detail

cudaError_t launch_commit(const RowMove& m, const int32_t* path, const int32_t* n_path, int max_path,
                          cudaStream_t s) {
  using namespace evict_detail;
  const int pairs = m.batch * m.h_kv;
  if (pairs == 0) return cudaSuccess;
  if (m.d == 128) commit_kernel<128><<<pairs, kCommitThreads, 0, s>>>(m, path, n_path, max_path);
  else if (m.d == 256) commit_kernel<256><<<pairs, kCommitThreads, 0, s>>>(m, path, n_path, max_path);
  else return cudaErrorInvalidValue;
  return cudaGetLastError();
}

cudaError_t launch_evict(const RowMove& m, const EvictArgs& e, cudaStream_t s) {
  using namespace evict_detail;
  const int pairs = m.batch * m.h_kv;
  if (pairs == 0) return cudaSuccess;
  const bool in_place = e.dst_table == m.block_table || e.mass_out == e.mass;
  const int slots = (in_place ? 1 : 2) * num_sms();  // CTAs of one wave
  // a round over a cluster costs some 3 us more than one inside a CTA (barriers, remote reads), about
  // what a CTA takes for kClusterSpan more positions; in place the cluster also shares the moves
  const int64_t len = (int64_t)m.max_pages * m.page_size, span = in_place ? kClusterSpan / 4 : kClusterSpan;
  int cluster = 1;
  while (cluster < kEvictMaxCluster && 2 * cluster * pairs <= slots && cluster * span < len) cluster *= 2;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(pairs * cluster, 1, 1);
  cfg.blockDim = dim3(kEvictThreads, 1, 1);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (in_place) {
    const cudaError_t err = m.d == 128 ? cudaLaunchKernelEx(&cfg, evict_in_place_kernel<128>, m, e, cluster)
                                       : cudaLaunchKernelEx(&cfg, evict_in_place_kernel<256>, m, e, cluster);
    return err != cudaSuccess ? err : cudaGetLastError();
  }
  cudaError_t err = cudaLaunchKernelEx(&cfg, select_kernel, m, e, cluster);
  if (err != cudaSuccess) return err;
  const int rows = kMoveThreads;
  cfg.gridDim = dim3((e.keep + rows - 1) / rows, pairs, 1);
  cfg.blockDim = dim3(kMoveThreads, 1, 1);
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  err = m.d == 128 ? cudaLaunchKernelEx(&cfg, move_kernel<128>, m, e)
                   : cudaLaunchKernelEx(&cfg, move_kernel<256>, m, e);
  if (err != cudaSuccess) return err;
  return cudaGetLastError();
}

}  // namespace jssa
