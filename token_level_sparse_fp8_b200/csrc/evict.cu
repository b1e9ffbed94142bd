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
    if (mass_row && lane < kRows && e.src_pos >= 0) mass = mass_row[e.src_pos];
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
    if (mass_row && lane < kRows && e.src_pos >= 0) mass_row[e.dst_pos] = mass;
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
// order of the path does not matter. Latency-bound: one dependent chain of path, page and row.
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
    } else if (node != i) {
      const int sp = page_of(m, table, m.max_pages, L + node);
      const int dp = page_of(m, table, m.max_pages, L + i);
      if (sp >= 0 && dp >= 0) ends = {L + node, L + i, sp, dp};
    }
  }
  WarpTile<D, kCommitRows> t;
  t.load(m, h, nullptr, ends, lane);
  __syncthreads();
  t.store(m, h, nullptr, ends, lane);
}

// ---- evict ---------------------------------------------------------------------------------
// A cluster of C CTAs per (sequence, KV head), C as large as fits one wave of one CTA per SM.
//   (1) The key of rank keep - recent among positions [0, L - recent): exact radix selection, 11 +
//       11 + 10 bits, each CTA counting its slice of the positions; the C histograms are summed
//       through distributed shared memory.
//   (2) The kept positions in ascending order: each warp owns a contiguous range, counts its keys
//       above and at the threshold, and writes its part after a scan over warps and CTAs.
//   (3) The rows, in tiles of C x 128 (64 at d = 256). The rows of the next tile, the pages of the one after and the
//       positions of the one after that are in flight while a tile is written.
//   (4) Zeros in the mass of the positions left over.
// Bound by HBM in (3) (a kept row is read once and written once) and by L2 latency in (1) and (2),
// which pass five times over the 4 bytes of each position.
constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kEvictMaxCluster = 8;  // the portable size
constexpr int kBins = 2048;          // four per thread
constexpr int kFlight = 8;           // loads of mass in flight per lane

// Order-preserving key of a running mass; every NaN counts as the largest value.
__device__ __forceinline__ uint32_t mass_key(float x) {
  return x != x ? 0xffffffffu : score_key(x);
}

template <int D>
__global__ void __launch_bounds__(kEvictThreads, 1)
    evict_kernel(RowMove m, EvictArgs e, int cluster, bool in_place) {
  constexpr int kRows = D == 128 ? 8 : 4;  // per warp and tile: two tiles in registers
  __shared__ __align__(16) uint32_t s_hist[2][kBins];  // alternating, so one barrier a round is enough
  __shared__ __align__(16) uint4 s_counts;             // of this CTA: above, equal, first position out
  __shared__ int s_above[kEvictWarps], s_equal[kEvictWarps], s_first, s_want;
  __shared__ uint32_t s_bin, s_scan[kEvictWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % cluster, pair = blockIdx.x / cluster;
  const int b = pair / m.h_kv, h = pair % m.h_kv;
  const int L = clamped_len(m, b, h == 0 && rank == 0 && tid == 0);
  const int n_keep = min(L, e.keep);
  const float* mass = e.mass + (int64_t)pair * e.mass_stride;
  float* mass_out = e.mass_out + (int64_t)pair * e.mass_stride;
  int32_t* idx = e.idx + (int64_t)pair * e.keep;
  if (tid == 0) {
    s_first = INT_MAX;
    if (rank == 0) {
      e.count[pair] = n_keep;
      if (h == 0) m.lens_out[b] = n_keep;
    }
  }
  __syncthreads();
  // this warp's positions: the CTA's slice of [0, L), a 16th of it
  const int per_warp = ((L + cluster * kEvictWarps - 1) / (cluster * kEvictWarps) + 31) / 32 * 32;
  const int p_lo = min((int64_t)L, (int64_t)(rank * kEvictWarps + warp) * per_warp);
  const int p_hi = min(L, p_lo + per_warp);
  const int n_cand = L > e.keep ? L - e.recent : 0;  // positions that compete
  int want = L > e.keep ? e.keep - e.recent : 0;     // for so many places
  const bool pick = want > 0;
  // (1)
  uint32_t edge = 0u;
  if (pick) {
#pragma unroll 1
    for (int round = 0; round < 3; ++round) {
      uint32_t* hist = s_hist[round & 1];
      const int shift = round == 0 ? 21 : round == 1 ? 10 : 0;
      reinterpret_cast<uint4*>(hist)[tid] = make_uint4(0u, 0u, 0u, 0u);
      __syncthreads();
      const int hi = min(p_hi, n_cand);
      for (int p = p_lo; p < hi; p += 32 * kFlight) {
        float x[kFlight];
#pragma unroll
        for (int u = 0; u < kFlight; ++u)
          if (p + 32 * u + lane < hi) x[u] = mass[p + 32 * u + lane];
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
          const bool in = p + 32 * u + lane < hi;
          const uint32_t key = in ? mass_key(x[u]) : 0u;
          const uint32_t bin = (key >> shift) & (kBins - 1);
          if (round == 0) {
            // (equal keys in a whole warp, as of untouched positions, would serialise)
            const uint32_t bin0 = __shfl_sync(kAll, bin, 0);
            if (__all_sync(kAll, in && bin == bin0)) {
              if (lane == 0) atomicAdd(&hist[bin], 32u);
            } else if (in) {
              atomicAdd(&hist[bin], 1u);
            }
          } else if (in && (round == 1 ? key >> 21 == edge >> 21 : key >> 10 == edge >> 10)) {
            atomicAdd(&hist[round == 1 ? bin : key & 1023u], 1u);
          }
        }
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
      if (lane == 31) s_scan[warp] = incl;
      __syncthreads();
      uint32_t before = incl - mine;
      for (int w = 0; w < warp; ++w) before += s_scan[w];
      if (before < (uint32_t)want && before + mine >= (uint32_t)want) {
        const uint32_t n[4] = {c.w, c.z, c.y, c.x};  // descending
        uint32_t left = want - before, bin = kBins - 1 - 4 * tid;
        for (int u = 0; u < 4 && n[u] < left; ++u) {
          left -= n[u];
          --bin;
        }
        s_want = left;
        s_bin = bin;
      }
      __syncthreads();
      want = s_want;  // keys to take of those with this prefix
      edge |= s_bin << shift;
    }
  }
  const int n_equal = pick ? want : 0;  // keys equal to the edge that stay, lowest positions first
  // (2) 2: stays, 1: equal to the edge, 0: out; nothing is evicted when everything fits
  auto state = [&](int p, float x) {
    if (p >= L) return 0;
    if (L <= e.keep || p >= n_cand) return 2;
    if (!pick) return 0;
    const uint32_t key = mass_key(x);
    return key > edge ? 2 : key == edge ? 1 : 0;
  };
  int above = 0, equal = 0, first = INT_MAX;
  for (int p = p_lo; p < p_hi; p += 32 * kFlight) {
    float x[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int q = p + 32 * u + lane;
      x[u] = q < min(p_hi, n_cand) ? mass[q] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int q = p + 32 * u + lane, s = q < p_hi ? state(q, x[u]) : -1;
      above += __popc(__ballot_sync(kAll, s == 2));
      equal += __popc(__ballot_sync(kAll, s == 1));
      const unsigned out = __ballot_sync(kAll, s == 0 || s == 1);
      if (out && first == INT_MAX) first = p + 32 * u + __ffs(out) - 1;
    }
  }
  if (lane == 0) {
    s_above[warp] = above;
    s_equal[warp] = equal;
    if (first != INT_MAX) atomicMin(&s_first, first);
  }
  __syncthreads();
  if (warp == 0) {
    int a = lane < kEvictWarps ? s_above[lane] : 0, q = lane < kEvictWarps ? s_equal[lane] : 0;
    for (int o = 16; o; o >>= 1) {
      a += __shfl_xor_sync(kAll, a, o);
      q += __shfl_xor_sync(kAll, q, o);
    }
    if (lane == 0) s_counts = make_uint4(a, q, s_first, 0u);
  }
  if (cluster > 1) cluster_sync();
  else __syncthreads();
  int base = 0, eq_before = 0, first_out = INT_MAX;
  for (int r = 0; r < cluster; ++r) {
    const uint32_t at = smem_u32(&s_counts);
    const uint4 c = cluster > 1 ? ld_cluster_v4(cluster_addr(at, r)) : ld_shared_v4(at);
    first_out = min(first_out, (int)c.z);
    if (r < rank) {
      base += c.x + max(0, min((int)c.y, n_equal - eq_before));
      eq_before += c.y;
    }
  }
  for (int w = 0; w < warp; ++w) {
    base += s_above[w] + max(0, min(s_equal[w], n_equal - eq_before));
    eq_before += s_equal[w];
  }
  const unsigned below = (1u << lane) - 1u;
  for (int p = p_lo; p < p_hi; p += 32 * kFlight) {
    float x[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int q = p + 32 * u + lane;
      x[u] = q < min(p_hi, n_cand) ? mass[q] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int q = p + 32 * u + lane, s = q < p_hi ? state(q, x[u]) : -1;
      const unsigned eq = __ballot_sync(kAll, s == 1);
      const bool stay = s == 2 || (s == 1 && eq_before + __popc(eq & below) < n_equal);
      const unsigned st = __ballot_sync(kAll, stay);
      if (stay) __stcg(&idx[base + __popc(st & below)], q);
      base += __popc(st);
      eq_before += __popc(eq);
    }
  }
  for (int i = n_keep + rank * kEvictThreads + tid; i < e.keep; i += cluster * kEvictThreads) idx[i] = -1;
  if (cluster > 1) cluster_sync();
  else __syncthreads();
  // (3) in place, the rows before the first one out stay where they are
  const int32_t* table = m.block_table + (int64_t)b * m.max_pages;
  const int32_t* dst_table = e.dst_table + (int64_t)b * e.dst_max_pages;
  const int span = cluster * kEvictWarps * kRows;
  const bool stays = e.dst_table == m.block_table && e.mass_out == e.mass;
  const int i_begin = stays ? min(first_out, n_keep) : 0;
  const int n_tiles = (n_keep - i_begin + span - 1) / span;
  const int row0 = i_begin + (rank * kEvictWarps + warp) * kRows + lane;  // (the first lanes)
  auto position = [&](int t) {  // of this lane's row of tile t; -1: none
    const int i = row0 + t * span;
    return lane < kRows && t < n_tiles && i < n_keep ? __ldcg(&idx[i]) : -1;
  };
  const int src_len = m.max_pages * m.page_size, dst_len = e.dst_max_pages * m.page_size;
  auto look_up = [&](int t, int pos) {
    Ends r = {-1, -1, -1, -1};
    if (pos >= 0) {
      const int i = row0 + t * span;
      r.src_pos = pos;
      r.dst_pos = i;
      r.src_pg = pos < src_len ? table[pos / m.page_size] : -2;
      r.dst_pg = i < dst_len ? dst_table[i / m.page_size] : -2;
    }
    return r;
  };
  auto check = [&](Ends& r) {  // both pages have to be usable (-2: beyond the table)
    if (r.src_pos < 0) return;
    const uint32_t bad = (r.src_pg == -2 || r.dst_pg == -2 ? 2u : 0u) |
                         ((r.src_pg != -2 && (r.src_pg < 0 || r.src_pg >= m.num_pages)) ||
                                  (r.dst_pg != -2 && (r.dst_pg < 0 || r.dst_pg >= m.num_pages))
                              ? 1u : 0u);
    if (bad) {
      raise_flag(bad);
      r.src_pg = r.dst_pg = -1;
    }
  };
  // a step writes tile t (`cur`) after the reads of tile t + 1 (`nxt`) have been issued
  WarpTile<D, kRows> ta, tb;
  Ends ea, eb, ahead;
  ea = look_up(0, position(0));
  ahead = look_up(1, position(1));
  int pos = position(2);
  check(ea);
  ta.load(m, h, mass, ea, lane);
  auto step = [&](int t, const WarpTile<D, kRows>& cur, const Ends& ce, WarpTile<D, kRows>& nxt, Ends& ne) {
    ne = ahead;
    check(ne);
    nxt.load(m, h, mass, ne, lane);
    ahead = look_up(t + 2, pos);
    pos = position(t + 3);
    if (in_place) {
      if (cluster > 1) cluster_sync();
      else __syncthreads();
    }
    cur.store(m, h, mass_out, ce, lane);
  };
#pragma unroll 1
  for (int t = 0; t < n_tiles; t += 2) {
    step(t, ta, ea, tb, eb);
    if (t + 1 < n_tiles) step(t + 1, tb, eb, ta, ea);
  }
  // (4) (in place, the last tile's barrier came after the last read of the mass)
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
  int cluster = 1;
  while (cluster < kEvictMaxCluster && 2 * cluster * pairs <= num_sms()) cluster *= 2;
  const bool in_place = e.dst_table == m.block_table || e.mass_out == e.mass;
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
  cudaError_t err = cudaErrorInvalidValue;
  if (m.d == 128) err = cudaLaunchKernelEx(&cfg, evict_kernel<128>, m, e, cluster, in_place);
  else if (m.d == 256) err = cudaLaunchKernelEx(&cfg, evict_kernel<256>, m, e, cluster, in_place);
  if (err != cudaSuccess) return err;
  return cudaGetLastError();
}

}  // namespace jssa
