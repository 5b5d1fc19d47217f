// s4kv_tree_attention device side: attention of a tree of drafted tokens over
// the paged cache, its ancestors and itself ("KV-Cache-Optimierung --
// PagedAttention, quantisierter KV, Speculative Cache", "Kernpunkte").
//
// For node i of sequence b and query head j (kv head j / G):
//   out = softmax(sm_scale * q K^T) V
// over the cached tokens (full pages dequantized, code * scale + zero; the
// partial page from the fp16 residual), the node's ancestors and the node.
//
// One CTA takes eight query rows of a (sequence, kv head) over all its keys, 16
// at a time, in fp32 with an online softmax.
#include "code_map.cuh"
#include "kernels.cuh"

namespace s4kv {

namespace {
constexpr int kRowsT = 8;
}

__global__ void __launch_bounds__(128) tree_kernel(const TreeParams p) {
  __shared__ float ks[kPage][kHeadDim + 1], vs[kPage][kHeadDim], qs[kRowsT][kHeadDim];
  __shared__ float ss[kRowsT][kPage];
  __shared__ unsigned long long anc[kRowsT];
  const int b = blockIdx.y, h = blockIdx.z, tid = threadIdx.x, H = p.num_kv_heads, G = p.group;
  const int c0 = __ldg(p.cu_nodes + b), c1 = __ldg(p.cu_nodes + b + 1), n = c1 - c0;
  const bool first = blockIdx.x == 0 && h == 0 && tid == 0;
  if (c0 < 0 || n < 0 || c1 > p.n_nodes || n > p.max_nodes) {
    if (first) flag_error(p.err, S4KV_EFLAG_TREE);
    return;
  }
  const int L = __ldg(p.seq_lens + b);
  if (n == 0) return;
  if (L < 0 || L > p.max_pages * kPage) {
    if (first) flag_error(p.err, S4KV_EFLAG_SEQ_LEN);
    return;
  }
  const int r0 = blockIdx.x * kRowsT, rows = min(kRowsT, n * G - r0);
  if (rows <= 0) return;
  if (tid < rows) {
    unsigned long long m = 0;
    for (int a = (r0 + tid) / G; a >= 0;) {
      m |= 1ull << a;
      const int up = __ldg(p.parents + c0 + a);
      if (up < -1 || up >= a) {
        flag_error(p.err, S4KV_EFLAG_TREE);
        break;
      }
      a = up;
    }
    anc[tid] = m;
  }
  for (int r = 0; r < kRowsT; ++r)
    qs[r][tid] = r < rows ? __half2float(p.q[(static_cast<long>(c0 + (r0 + r) / G) * p.num_q_heads + h * G + (r0 + r) % G) * kHeadDim + tid]) : 0.f;
  float O[kRowsT], mref[kRowsT], l[kRowsT];
  for (int r = 0; r < kRowsT; ++r) {
    O[r] = l[r] = 0.f;
    mref[r] = -INFINITY;
  }
  const int nfull = L / kPage, res = L % kPage;
  const int tiles = nfull + (res ? 1 : 0) + (n + kPage - 1) / kPage;
  const int code_bytes = kPage * kHeadDim * p.bits / 8;
  for (int tile = 0; tile < tiles; ++tile) {
    __syncthreads();
    int count = kPage, node0 = -1;
    if (tile < nfull) {
      int phys = __ldg(p.block_tables + static_cast<long>(b) * p.max_pages + tile);
      if (static_cast<unsigned>(phys) >= static_cast<unsigned>(p.num_pages)) {
        if (tid == 0) flag_error(p.err, S4KV_EFLAG_PAGE_RANGE);
        phys = 0;
      }
      const uint8_t *blk = p.pool + (static_cast<long>(phys) * H + h) * block_bytes_for(p.bits);
      const __half *meta = reinterpret_cast<const __half *>(blk + 2 * code_bytes);
      const int c = tid, g = c / kVGroup;
      const float sk = __half2float(meta[c]), zk = __half2float(meta[kHeadDim + key_zero_slot(c)]);
      for (int t = 0; t < kPage; ++t) {
        int w, j;
        key_position(t, c, w, j);
        ks[t][c] = static_cast<float>(code_at(blk, w, j, p.bits)) * sk + zk;
        value_position(t, c, w, j);
        vs[t][c] = static_cast<float>(code_at(blk + code_bytes, w, j, p.bits)) *
                       __half2float(meta[2 * kHeadDim + value_scale_slot(t, g)]) +
                   __half2float(meta[2 * kHeadDim + 64 + g * kPage + t]);
      }
    } else if (tile == nfull && res) {
      count = res;
      const long base = (static_cast<long>(b) * H + h) * kPage * kHeadDim + tid;
      for (int t = 0; t < count; ++t) {
        ks[t][tid] = __half2float(p.res_k[base + t * kHeadDim]);
        vs[t][tid] = __half2float(p.res_v[base + t * kHeadDim]);
      }
    } else {
      node0 = (tile - nfull - (res ? 1 : 0)) * kPage;
      count = min(kPage, n - node0);
      for (int t = 0; t < count; ++t) {
        const long at = (static_cast<long>(c0 + node0 + t) * H + h) * kHeadDim + tid;
        ks[t][tid] = __half2float(p.k[at]);
        vs[t][tid] = __half2float(p.v[at]);
      }
    }
    __syncthreads();
    {
      const int r = tid >> 4, t = tid & 15;
      float s = 0.f;
      bool seen = r < rows && t < count;
      if (seen && node0 >= 0) seen = (anc[r] >> (node0 + t)) & 1;
      if (seen)
        for (int c = 0; c < kHeadDim; ++c) s += qs[r][c] * ks[t][c];
      ss[r][t] = seen ? s * p.scale_log2 : -INFINITY;
    }
    __syncthreads();
    for (int r = 0; r < rows; ++r) {
      float m = mref[r];
      for (int t = 0; t < count; ++t) m = fmaxf(m, ss[r][t]);
      if (m == -INFINITY) continue;
      const float a = exp2f(mref[r] - m);
      O[r] *= a;
      l[r] *= a;
      mref[r] = m;
      for (int t = 0; t < count; ++t) {
        const float w = exp2f(ss[r][t] - m);
        l[r] += w;
        O[r] += w * vs[t][tid];
      }
    }
  }
  for (int r = 0; r < rows; ++r)
    p.out[(static_cast<long>(c0 + (r0 + r) / G) * p.num_q_heads + h * G + (r0 + r) % G) * kHeadDim + tid] =
        __float2half_rn(O[r] / l[r]);
}

cudaError_t launch_tree(const TreeParams &p, cudaStream_t stream) {
  const dim3 grid((p.max_nodes * p.group + kRowsT - 1) / kRowsT, p.batch, p.num_kv_heads);
  tree_kernel<<<grid, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace s4kv
