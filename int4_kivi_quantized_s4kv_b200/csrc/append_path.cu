// s4kv_append_path device side: the accepted path of a drafted tree enters the
// cache.  Sequence b's token j (node path[b][j], j < path_len[b]) takes position
// seq_lens[b] + j; pages that fill up are quantized from the old residual rows
// and the path's rows, the rest goes to the residual -- s4kv_append with the
// rows reached through the path and every length read on the device ("KV-Cache-
// Optimierung -- PagedAttention, quantisierter KV, Speculative Cache").
//
// Grid: (page slot, sequence, kv head), 128 threads, as in s4kv_append: slot s
// takes the s-th page that the path touches, and slot 0 writes the partial tail
// after it has read the residual rows that its own page needed.
//
// Bound by latency: a chain of launch, lengths and path, rows, quantization, and a
// few KB a CTA.  The lengths, the path, the page's id and the residual rows are
// therefore fetched at once.  Measured, captured and warm, 8 kv heads: one sequence's
// path of up to 4 nodes 1.9 us, 128 sequences' paths of up to 1, 8 and 64 nodes 8.8, 10.4 and
// 23.3 us; followed by s4kv_dequant_pages, 128 paths of up to 8, 18 us.
#include "kernels.cuh"
#include "quant.cuh"

namespace s4kv {

template <int kBits>
__global__ void __launch_bounds__(128) append_path_kernel(const PathParams p) {
  const int slot = blockIdx.x, b = blockIdx.y, h = blockIdx.z, tid = threadIdx.x;
  const int H = p.num_kv_heads;
  __shared__ __align__(16) __half ks[kPage][kHeadDim];
  __shared__ __align__(16) __half vs[kPage][kHeadDim];
  __shared__ uint8_t kc[kPage][kHeadDim];
  __shared__ uint8_t vc[kPage][kHeadDim];

  __shared__ int nodes[S4KV_MAX_TREE_NODES];

  // everything that depends on nothing is fetched at once: the call's time is the chain of its loads
  const int c0 = __ldg(p.cu_nodes + b), c1 = __ldg(p.cu_nodes + b + 1);
  const int m = __ldg(p.path_len + b), L = __ldg(p.seq_lens + b);
  const int node = tid < p.max_nodes ? __ldg(p.path + static_cast<long>(b) * p.max_nodes + tid) : 0;
  // every CTA of the sequence comes to the same verdict on its whole path
  bool tree_ok = c0 >= 0 && c1 >= c0 && c1 <= p.n_nodes && m >= 0 && m <= p.max_nodes;
  const bool len_ok = L >= 0 && L <= p.max_pages * kPage - (tree_ok ? m : 0);
  if (tid < p.max_nodes) nodes[tid] = node;
  if (tid < m) tree_ok = tree_ok && node >= 0 && node < c1 - c0;  // (m <= max_nodes where the rest is right)
  // the page that this CTA may complete
  const int pg = len_ok ? L / kPage + slot : 0;
  int phys = -1;
  if (len_ok && pg < p.max_pages) phys = __ldg(p.block_tables + static_cast<long>(b) * p.max_pages + pg);
  tree_ok = __syncthreads_and(tree_ok);
  const bool first = slot == 0 && h == 0 && tid == 0;
  if (first) p.new_lens[b] = (tree_ok && len_ok) ? L + m : L;
  if (!tree_ok || !len_ok) {
    if (first) flag_error(p.err, (tree_ok ? 0u : S4KV_EFLAG_TREE) | (len_ok ? 0u : S4KV_EFLAG_SEQ_LEN));
    return;
  }
  if (m == 0) return;
  const int end = L + m;
  const int pl = (end - 1) / kPage;
  if (pg > pl) return;
  const bool full = (pg + 1) * kPage <= end;
  if (!full && slot != 0) return;  // the partial tail belongs to slot 0
  const long res_base = (static_cast<long>(b) * H + h) * kPage * kHeadDim;

  if (full) {
    const bool phys_ok = static_cast<unsigned>(phys) < static_cast<unsigned>(p.num_pages);
    for (int ch = tid; ch < kPage * (kHeadDim / 8); ch += 128) {
      const int t = ch / (kHeadDim / 8), c8 = (ch % (kHeadDim / 8)) * 8;
      const int pos = pg * kPage + t;
      const __half *sk = p.res_k + res_base + t * kHeadDim + c8, *sv = p.res_v + res_base + t * kHeadDim + c8;
      if (pos >= L) {
        const long row = (static_cast<long>(c0 + nodes[pos - L]) * H + h) * kHeadDim + c8;
        sk = p.k + row;
        sv = p.v + row;
      }
      *reinterpret_cast<uint4 *>(&ks[t][c8]) = *reinterpret_cast<const uint4 *>(sk);
      *reinterpret_cast<uint4 *>(&vs[t][c8]) = *reinterpret_cast<const uint4 *>(sv);
    }
    if (!phys_ok && tid == 0) flag_error(p.err, S4KV_EFLAG_PAGE_RANGE);
    __syncthreads();
    if (phys_ok)
      quantize_page_cta<kBits>(ks, vs, kc, vc, p.pool + (static_cast<long>(phys) * H + h) * Fmt<kBits>::kBlock, tid);
    if (slot != 0) return;
    __syncthreads();  // the residual rows are read before the tail overwrites them
  }
  if (end % kPage != 0) {
    const int tail0 = max(L, pl * kPage);
    for (int ch = tid; ch < (end - tail0) * (kHeadDim / 8); ch += 128) {
      const int pos = tail0 + ch / (kHeadDim / 8), c8 = (ch % (kHeadDim / 8)) * 8;
      const long row = (static_cast<long>(c0 + nodes[pos - L]) * H + h) * kHeadDim + c8;
      const long dst = res_base + (pos % kPage) * kHeadDim + c8;
      *reinterpret_cast<uint4 *>(p.res_k + dst) = *reinterpret_cast<const uint4 *>(p.k + row);
      *reinterpret_cast<uint4 *>(p.res_v + dst) = *reinterpret_cast<const uint4 *>(p.v + row);
    }
  }
}

cudaError_t launch_append_path(const PathParams &p, int batch, cudaStream_t stream) {
  // pages that max_nodes tokens can touch
  const dim3 grid((kPage - 1 + p.max_nodes + kPage - 1) / kPage, batch, p.num_kv_heads);
  if (p.bits == 8) append_path_kernel<8><<<grid, 128, 0, stream>>>(p);
  else if (p.bits == 2) append_path_kernel<2><<<grid, 128, 0, stream>>>(p);
  else append_path_kernel<4><<<grid, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace s4kv
