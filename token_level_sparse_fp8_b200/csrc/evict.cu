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
#include "common.cuh"

namespace jssa {

namespace evict_detail {

constexpr int kWarpRows = 8;  // rows a warp holds in registers
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

// A warp's tile of at most 8 rows: sources and destinations by lane (lane u < 8 holds row u's
// pages, or -1), the K / V chunks of every row, one scoring chunk and one mass value per lane.
template <int D>
struct WarpTile {
  int src_pos, dst_pos, src_pg, dst_pg;  // lanes 0-7
  LaneRow<D> kv[kWarpRows];
  uint4 code;
  float mass;

  __device__ __forceinline__ void load(const RowMove& m, int h, const float* mass_row, int lane) {
#pragma unroll
    for (int u = 0; u < kWarpRows; ++u) {
      const int pg = __shfl_sync(kAll, src_pg, u), pos = __shfl_sync(kAll, src_pos, u);
      if (pg >= 0) kv[u].load(m.k_cache, m.v_cache, kv_offset(m, pg, pos, h), lane);
    }
    if (m.code_bytes) {
      const int per = m.code_bytes >> 4, u = lane / per;  // chunks per row; this lane's row
      const int pg = __shfl_sync(kAll, src_pg, u & 7), pos = __shfl_sync(kAll, src_pos, u & 7);
      if (u < kWarpRows && pg >= 0)
        code = *reinterpret_cast<const uint4*>(m.score_cache + code_offset(m, pg, pos, h) + (lane % per) * 16);
    }
    if (mass_row && lane < kWarpRows && src_pos >= 0) mass = mass_row[src_pos];
  }
  __device__ __forceinline__ void store(const RowMove& m, int h, float* mass_row, int lane) {
#pragma unroll
    for (int u = 0; u < kWarpRows; ++u) {
      const int pg = __shfl_sync(kAll, dst_pg, u), pos = __shfl_sync(kAll, dst_pos, u);
      if (pg >= 0) kv[u].store(m.k_cache, m.v_cache, kv_offset(m, pg, pos, h), lane);
    }
    if (m.code_bytes) {
      const int per = m.code_bytes >> 4, u = lane / per;
      const int pg = __shfl_sync(kAll, dst_pg, u & 7), pos = __shfl_sync(kAll, dst_pos, u & 7);
      if (u < kWarpRows && pg >= 0)
        *reinterpret_cast<uint4*>(m.score_cache + code_offset(m, pg, pos, h) + (lane % per) * 16) = code;
    }
    if (mass_row && lane < kWarpRows && src_pos >= 0) mass_row[dst_pos] = mass;
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
static_assert(kCommitThreads / 32 * kWarpRows == kTreeMaxNodes, "all rows of a tree in registers");

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
  WarpTile<D> t;
  t.src_pos = t.dst_pos = t.src_pg = t.dst_pg = -1;
  const int i = warp * kWarpRows + lane;
  if (lane < kWarpRows && i < n) {
    const int node = path[(int64_t)b * max_path + i];
    if (node < 0 || node >= kTreeMaxNodes) {
      raise_flag(2u);
    } else if (node != i) {
      const int sp = page_of(m, table, m.max_pages, L + node);
      const int dp = page_of(m, table, m.max_pages, L + i);
      if (sp >= 0 && dp >= 0) {
        t.src_pos = L + node; t.src_pg = sp;
        t.dst_pos = L + i; t.dst_pg = dp;
      }
    }
  }
  t.load(m, h, nullptr, lane);
  __syncthreads();
  t.store(m, h, nullptr, lane);
}

// ---- evict ---------------------------------------------------------------------------------
constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;

// Order-preserving key of a running mass; every NaN counts as the largest value.
__device__ __forceinline__ uint32_t mass_key(float x) {
  return x != x ? 0xffffffffu : score_key(x);
}

// Grid batch * h_kv. (1) The key of rank keep - recent among positions [0, L - recent) by an exact
// radix selection, 8 bits a round; (2) the kept positions in ascending order: each warp owns a
// contiguous range, counts its keys above and at the threshold, and writes its part after a scan
// over the warps; (3) the rows, tile by tile; (4) zeros in the mass of the positions left over.
template <int D>
__global__ void __launch_bounds__(kEvictThreads) evict_kernel(RowMove m, EvictArgs e) {
  __shared__ int s_hist[256];
  __shared__ int s_above[kEvictWarps], s_equal[kEvictWarps];
  __shared__ uint32_t s_prefix;
  __shared__ int s_want;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pair = blockIdx.x, b = pair / m.h_kv, h = pair % m.h_kv;
  const int L = clamped_len(m, b, h == 0 && tid == 0);
  const int n_keep = min(L, e.keep);
  const float* mass = e.mass + (int64_t)pair * e.mass_stride;
  float* mass_out = e.mass_out + (int64_t)pair * e.mass_stride;
  int32_t* idx = e.idx + (int64_t)pair * e.keep;
  if (tid == 0) {
    e.count[pair] = n_keep;
    if (h == 0) m.lens_out[b] = n_keep;
  }
  // (1)
  const int n_cand = L > e.keep ? L - e.recent : 0;  // positions that compete
  if (tid == 0) {
    s_prefix = 0u;
    s_want = L > e.keep ? e.keep - e.recent : 0;
  }
  __syncthreads();
  const bool pick = s_want > 0;
  if (pick) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kEvictThreads) s_hist[i] = 0;
      __syncthreads();
      const uint32_t prefix = s_prefix;
      for (int p = tid; p < n_cand; p += kEvictThreads) {
        const uint32_t key = mass_key(mass[p]);
        if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8)))
          atomicAdd(&s_hist[(key >> shift) & 255u], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int want = s_want, bin = 255;
        while (bin > 0 && s_hist[bin] < want) want -= s_hist[bin--];
        s_want = want;  // keys to take from the chosen bin
        s_prefix = prefix | ((uint32_t)bin << shift);
      }
      __syncthreads();
    }
  }
  const uint32_t edge = s_prefix;
  const int n_equal = pick ? s_want : 0;  // keys equal to the edge that stay, lowest positions first
  // (2) every position below n_keep stays when nothing is evicted
  auto state = [&](int p) {  // 2 above, 1 equal, 0 out
    if (p >= L) return 0;
    if (L <= e.keep || p >= n_cand) return 2;
    if (!pick) return 0;
    const uint32_t key = mass_key(mass[p]);
    return key > edge ? 2 : key == edge ? 1 : 0;
  };
  const int per_warp = ((L + kEvictWarps - 1) / kEvictWarps + 31) / 32 * 32;
  const int p0 = warp * per_warp, p1 = min(L, p0 + per_warp);
  int above = 0, equal = 0;
  for (int p = p0; p < p1; p += 32) {
    const int s = state(p + lane);
    above += __popc(__ballot_sync(kAll, s == 2));
    equal += __popc(__ballot_sync(kAll, s == 1));
  }
  if (lane == 0) {
    s_above[warp] = above;
    s_equal[warp] = equal;
  }
  __syncthreads();
  int eq_before = 0, base = 0;
  for (int w = 0; w < warp; ++w) {
    base += s_above[w] + max(0, min(s_equal[w], n_equal - eq_before));
    eq_before += s_equal[w];
  }
  for (int p = p0; p < p1; p += 32) {
    const int s = state(p + lane);
    const unsigned eq = __ballot_sync(kAll, s == 1), below = (1u << lane) - 1u;
    const bool stay = s == 2 || (s == 1 && eq_before + __popc(eq & below) < n_equal);
    const unsigned st = __ballot_sync(kAll, stay);
    if (stay) idx[base + __popc(st & below)] = p + lane;
    base += __popc(st);
    eq_before += __popc(eq);
  }
  for (int i = n_keep + tid; i < e.keep; i += kEvictThreads) idx[i] = -1;
  __syncthreads();
  // (3)
  const int32_t* table = m.block_table + (int64_t)b * m.max_pages;
  const int32_t* dst_table = e.dst_table + (int64_t)b * e.dst_max_pages;
  for (int i0 = 0; i0 < n_keep; i0 += kEvictWarps * kWarpRows) {
    WarpTile<D> t;
    t.src_pos = t.dst_pos = t.src_pg = t.dst_pg = -1;
    const int i = i0 + warp * kWarpRows + lane;
    if (lane < kWarpRows && i < n_keep) {
      t.src_pos = idx[i];
      t.dst_pos = i;
      t.src_pg = page_of(m, table, m.max_pages, t.src_pos);
      t.dst_pg = page_of(m, dst_table, e.dst_max_pages, i);
      if (t.src_pg < 0 || t.dst_pg < 0) t.src_pg = t.dst_pg = -1;
    }
    t.load(m, h, mass, lane);
    __syncthreads();
    t.store(m, h, mass_out, lane);
  }
  __syncthreads();
  // (4)
  for (int p = n_keep + tid; p < L; p += kEvictThreads) mass_out[p] = 0.f;
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
  if (m.d == 128) evict_kernel<128><<<pairs, kEvictThreads, 0, s>>>(m, e);
  else if (m.d == 256) evict_kernel<256><<<pairs, kEvictThreads, 0, s>>>(m, e);
  else return cudaErrorInvalidValue;
  return cudaGetLastError();
}

}  // namespace jssa
