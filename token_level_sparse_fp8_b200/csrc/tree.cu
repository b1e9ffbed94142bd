// Attention of a tree of drafted tokens over the paged cache (the verification step of tree
// speculation). Node i of sequence b is a token at cache position seq_len + i; it sees the context
// (all of it, a sliding window ending at its own logical position, or an index set) and, of the
// nodes, itself and its ancestors:
//
//   out[b, i, hq] = sum_t p_t v_t,  p = softmax_t(scale q[b, i, hq] . k_t)
//
// over t in the node's context and { seq_len + a : a = i or an ancestor of i }.
#include "common.cuh"

namespace jssa {

namespace tree_detail {

// The new nodes' rows into the cache (unused nodes are not written). Grid (n, batch).
__global__ void store_kernel(TreeArgs a) {
  const int i = blockIdx.x, b = blockIdx.y;
  const int max_len = a.max_pages * a.page_size;
  const int L = min(max(a.seq_lens[b], 0), max_len);
  if (a.parents[b * a.n + i] < -1) return;
  const int pos = L + i;
  if (pos >= max_len) {
    raise_flag(2u);
    return;
  }
  const int pg = a.block_table[(int64_t)b * a.max_pages + pos / a.page_size];
  if (pg < 0 || (int64_t)pg >= a.num_pages) {
    raise_flag(1u);
    return;
  }
  const int64_t row = (int64_t)pg * a.page_stride + (int64_t)(pos % a.page_size) * a.slot_stride;
  for (int e = threadIdx.x; e < a.h_kv * a.d; e += blockDim.x) {
    const int64_t dst = row + (int64_t)(e / a.d) * a.head_stride + e % a.d;
    const int64_t src = ((int64_t)b * a.n + i) * a.h_kv * a.d + e;
    a.k_cache[dst] = a.k_new[src];
    a.v_cache[dst] = a.v_new[src];
  }
}

// One warp per (node, query head, sequence): 32 positions at a time, one per lane.
template <int D>
__global__ void __launch_bounds__(32) tree_kernel(TreeArgs a) {
  __shared__ float s_q[D];
  const int lane = threadIdx.x, i = blockIdx.x, hq = blockIdx.y, b = blockIdx.z;
  const int G = a.h_q / a.h_kv, h = hq / G;
  const int max_len = a.max_pages * a.page_size;
  int L = a.seq_lens[b];
  if (L < 0 || L > max_len) {
    if (lane == 0) raise_flag(4u);
    L = L < 0 ? 0 : max_len;
  }
  const int32_t* par = a.parents + (int64_t)b * a.n;
  uint16_t* out = a.out + (((int64_t)b * a.n + i) * a.h_q + hq) * D;
  // ancestors; depth
  uint64_t see = 0;
  int depth = -1;
  bool used = true;
  for (int x = i; x >= 0;) {
    const int p = par[x];
    if (p < -1) {
      if (x != i && lane == 0) raise_flag(2u);
      used = false;
      break;
    }
    if (p >= x) {
      if (lane == 0) raise_flag(2u);
      used = false;
      break;
    }
    if (a.window <= 0 || depth + 1 < a.window) see |= 1ull << x;
    ++depth;
    x = p;
  }
  for (int e = lane; e < D; e += 32)
    s_q[e] = bf16_to_f(a.q[(((int64_t)b * a.n + i) * a.h_q + hq) * D + e]);
  __syncwarp();
  float o[D / 32];
  for (int e = 0; e < D / 32; ++e) o[e] = 0.f;
  float m = -INFINITY, l = 0.f;
  int n_ctx = L, lo = 0;
  if (a.idx) n_ctx = min(max(a.count[b * a.h_kv + h], 0), a.budget);
  else if (a.window > 0) lo = max(0, L + depth - a.window + 1);
  const float scale_log2 = a.scale * 1.4426950408889634f;
  for (int t0 = lo & ~31; used && t0 < n_ctx + a.n; t0 += 32) {
    const int t = t0 + lane;
    int pos = -1;
    if (t >= lo && t < n_ctx) {
      pos = a.idx ? a.idx[((int64_t)b * a.h_kv + h) * a.budget + t] : t;
      if (pos < 0 || pos >= max_len) {
        raise_flag(2u);
        pos = -1;
      }
    } else if (t >= n_ctx && t < n_ctx + a.n && ((see >> (t - n_ctx)) & 1)) {
      pos = L + t - n_ctx;
      if (pos >= max_len) {
        raise_flag(2u);
        pos = -1;
      }
    }
    int64_t off = -1;
    float x = -INFINITY;
    if (pos >= 0) {
      const int pg = a.block_table[(int64_t)b * a.max_pages + pos / a.page_size];
      if (pg < 0 || (int64_t)pg >= a.num_pages) {
        raise_flag(1u);
      } else {
        off = (int64_t)pg * a.page_stride + (int64_t)(pos % a.page_size) * a.slot_stride +
              (int64_t)h * a.head_stride;
        float s = 0.f;
        for (int e = 0; e < D; ++e) s += s_q[e] * bf16_to_f(a.k_cache[off + e]);
        x = s * scale_log2;
      }
    }
    float mt = x;
    for (int w = 16; w; w >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, w));
    const float mn = fmaxf(m, mt), mu = mn == -INFINITY ? 0.f : mn;
    const float corr = fast_exp2(m - mu), p = fast_exp2(x - mu);
    float ps = p;
    for (int w = 16; w; w >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, w);
    l = l * corr + ps;
    m = mn;
    for (int e = 0; e < D / 32; ++e) o[e] *= corr;
    for (int j = 0; j < 32; ++j) {
      const int64_t oj = __shfl_sync(0xffffffffu, off, j);
      const float pj = __shfl_sync(0xffffffffu, p, j);
      if (oj < 0) continue;
      for (int e = 0; e < D / 32; ++e) o[e] += pj * bf16_to_f(a.v_cache[oj + lane + 32 * e]);
    }
  }
  const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
  for (int e = 0; e < D / 32; ++e) out[lane + 32 * e] = f_to_bf16(o[e] * inv);
}

}  // namespace tree_detail

size_t tree_ws_bytes(int batch, int n, int h_q, int h_kv, int d) { return 0; }

cudaError_t launch_tree(const TreeArgs& a, cudaStream_t s) {
  using namespace tree_detail;
  if (a.batch == 0 || a.n == 0) return cudaSuccess;
  if (a.k_new) store_kernel<<<dim3(a.n, a.batch), 256, 0, s>>>(a);
  const dim3 grid(a.n, a.h_q, a.batch);
  if (a.d == 128) tree_kernel<128><<<grid, 32, 0, s>>>(a);
  else if (a.d == 256) tree_kernel<256><<<grid, 32, 0, s>>>(a);
  else return cudaErrorInvalidValue;
  return cudaGetLastError();
}

}  // namespace jssa
