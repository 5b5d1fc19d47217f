// s4kv_verify_tree device side: acceptance of drafted tokens against the
// target's probabilities from given random numbers ("KV-Cache-Optimierung --
// PagedAttention, quantisierter KV, Speculative Cache", "Kernpunkte").
//
// The walk: cur = node 0; child c (token x) of cur is accepted when
// u_c M Q(x) < R(x), where R starts as cur's target row P with mass M = 1.
// After rejections with masses M_0, M_1, ... the rest is
//   R = max(.. max(P - M_0 Q, 0) - M_1 Q .., 0) = max(P - A Q, 0),  A = sum M_i
// (every M_i Q >= 0), so one number A describes it and R is never stored.  The
// next token is drawn from R by inverting its cumulative sum at u_0.  Sums are
// held in 64 bits: a border of the cumulative sum then moves by about 1e-16 of
// the mass whatever the order of the additions, and with it the answer.
//
// A cluster of CTAs takes a sequence, each a part of the vocabulary, and meets in
// distributed shared memory only to add up a row.  The entries that the walk tests
// (one a node) are fetched all at once before it, so that it runs without waiting for
// memory.  A row is summed in chunks of 256 consecutive entries, one a warp; their sums
// stay in shared memory, and the draw reads again only the chunk that holds its answer.
// 64 registers a thread let 4 CTAs share an SM, so that a batch of 64 sequences in
// clusters of 8 is on the card at once (128 registers: two waves).
// Bound by HBM for many sequences (one target row each, and one draft row after a
// rejection), by the chain of a row's sum and its exchange for few.  Measured, captured
// and warm: 64 chains of 8 over 128256 fp32 entries with draft rows 19.5 us (21.4 a call
// with an empty L2: 3.1 TB/s), 48 trees over bf16 rows without 14.0, 16 trees of 12 over 32000
// fp16 entries with draft rows 10.6, one chain of 5 over 32000 6.5.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "kernels.cuh"

namespace s4kv {

namespace cg = cooperative_groups;

namespace {

constexpr int kThreadsV = 256, kWarpsV = kThreadsV / 32;
constexpr int kPerLane = 8, kBlockV = 32 * kPerLane;  // entries a warp reads at once
constexpr int kMaxChunks = 1024;                       // chunk sums a CTA keeps
constexpr int kMaxCluster = 8, kCtasAnSm = 4, kWaveEntries = 9000;
constexpr unsigned kAllV = 0xFFFFFFFFu;

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
// negative entries and NaN count as 0
__device__ __forceinline__ double positive(double x) { return x > 0.0 ? x : 0.0; }
template <typename T>
__device__ __forceinline__ double prob(T x) {
  return static_cast<double>(fmaxf(as_float(x), 0.0f));  // fmaxf passes a NaN over
}

// This lane's entries v0 + 32 e of a row (0 behind its end), all loads in flight before the first is used.
template <typename T>
__device__ __forceinline__ void load_block(const T *row, int v0, int V, int lane, T (&x)[kPerLane]) {
  row += v0 + lane;
  if (v0 + kBlockV <= V) {
#pragma unroll
    for (int e = 0; e < kPerLane; ++e) x[e] = __ldg(row + 32 * e);
  } else {
#pragma unroll
    for (int e = 0; e < kPerLane; ++e) x[e] = v0 + lane + 32 * e < V ? __ldg(row + 32 * e) : T(0.0f);
  }
}

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(kAllV, x, off);
  return x;
}

}  // namespace

// blocks: groups of kBlockV entries in a chunk (1 but for vocabularies in the millions).
template <typename T>
__global__ void __launch_bounds__(kThreadsV, kCtasAnSm) verify_kernel(const VerifyParams p, int blocks) {
  __shared__ int tok[S4KV_MAX_TREE_NODES], out_path[S4KV_MAX_TREE_NODES];
  __shared__ double at_p[S4KV_MAX_TREE_NODES], at_q[S4KV_MAX_TREE_NODES], at_u[S4KV_MAX_TREE_NODES];
  __shared__ double chunk_sum[kMaxChunks];
  __shared__ double part[2];  // this CTA's share of a row's sum, for two rows in turn
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int b = blockIdx.x / C, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c0 = __ldg(p.cu_nodes + b), c1 = __ldg(p.cu_nodes + b + 1), n = c1 - c0;
  int32_t *path = p.path + static_cast<long>(b) * p.max_nodes;
  const bool ok = c0 >= 0 && c1 >= c0 && c1 <= p.n_nodes && n <= p.max_nodes;
  if (!ok || n == 0) {  // the whole cluster
    if (rank == 0) {
      if (tid < p.max_nodes) path[tid] = -1;
      if (tid == 0) {
        p.path_len[b] = 0;
        p.next_token[b] = -1;
        if (!ok) flag_error(p.err, S4KV_EFLAG_TREE);
      }
    }
    return;
  }
  const T *target = static_cast<const T *>(p.target) + static_cast<long long>(c0) * p.target_stride;
  const T *draft = p.draft ? static_cast<const T *>(p.draft) + static_cast<long long>(c0) * p.draft_stride : nullptr;
  const int V = p.vocab;

  // ---- the entries that the walk may test
  if (tid < n) {
    const int x = __ldg(p.tokens + c0 + tid), up = __ldg(p.parents + c0 + tid);
    const bool known = static_cast<unsigned>(x) < static_cast<unsigned>(V);
    if (tid > 0 && !known && rank == 0) flag_error(p.err, S4KV_EFLAG_TREE);
    tok[tid] = known ? x : -1;
    const bool child = known && up >= 0 && up < tid;
    at_p[tid] = child ? prob(__ldg(target + up * p.target_stride + x)) : 0.0;
    at_q[tid] = child && draft ? prob(__ldg(draft + up * p.draft_stride + x)) : 1.0;
    at_u[tid] = static_cast<double>(__ldg(p.uniforms + c0 + tid));
    out_path[tid] = -1;
  }
  // parents of nodes lane, lane + 32 (every warp walks by itself, all alike)
  const int up0 = lane < n ? __ldg(p.parents + c0 + lane) : -1, up1 = lane + 32 < n ? __ldg(p.parents + c0 + lane + 32) : -1;
  __syncthreads();

  int cur = 0, len = 1, sums = 0;
  double M = 1.0, A = 0.0;
  unsigned long long gone = 0;  // rejected children of cur (no draft rows)
  const T *P = target, *Q = draft;

  // this CTA's chunks of a row
  const int chunk = kBlockV * blocks;
  const int chunks = (V - 1) / chunk + 1;
  const int k0 = static_cast<int>(static_cast<long long>(chunks) * rank / C);
  const int k1 = static_cast<int>(static_cast<long long>(chunks) * (rank + 1) / C);
  // what is left of this lane's entries v0 + 32 e of a block
  auto rest = [&](int v0, double (&x)[kPerLane]) {
    T raw[kPerLane];
    load_block(P, v0, V, lane, raw);
    if (Q && A > 0.0) {
      T q[kPerLane];
      load_block(Q, v0, V, lane, q);
#pragma unroll
      for (int e = 0; e < kPerLane; ++e) x[e] = positive(prob(raw[e]) - A * prob(q[e]));
    } else {
#pragma unroll
      for (int e = 0; e < kPerLane; ++e) x[e] = prob(raw[e]);
      for (unsigned long long m = gone; m; m &= m - 1) {
        const int x0 = tok[__ffsll(m) - 1] - v0;
        if (x0 >= 0 && x0 < kBlockV) {
#pragma unroll
          for (int e = 0; e < kPerLane; ++e)
            if (x0 == 32 * e + lane) x[e] = 0.0;
        }
      }
    }
  };
  // Sum of the rest over the row; `before`: the share of the CTAs of lower rank.  Every thread of the cluster calls it.
  auto mass = [&](double &before) {
    for (int k = k0 + warp; k < k1; k += kWarpsV) {
      double s = 0.0;
      for (int e = 0; e < blocks; ++e) {
        double x[kPerLane];
        rest(k * chunk + e * kBlockV, x);
#pragma unroll
        for (int j = 0; j < kPerLane; ++j) s += x[j];
      }
      s = warp_sum(s);
      if (lane == 0) chunk_sum[k - k0] = s;
    }
    __syncthreads();
    if (warp == 0) {
      double s = 0.0;
      for (int k = lane; k < k1 - k0; k += 32) s += chunk_sum[k];
      s = warp_sum(s);
      if (lane == 0) part[sums & 1] = s;
    }
    cluster.sync();
    double total = 0.0;
    for (int r = 0; r < C; ++r) {
      if (r == rank) before = total;
      total += *cluster.map_shared_rank(&part[sums & 1], r);
    }
    ++sums;  // the slot is written again only after the next sum's meeting
    return total;
  };

  // ---- the walk
  while (true) {
    unsigned long long children = __ballot_sync(kAllV, up0 == cur && lane > cur) |
                                  static_cast<unsigned long long>(__ballot_sync(kAllV, up1 == cur && lane + 32 > cur)) << 32;
    bool moved = false;
    while (children && !moved) {  // in the order in which they are tried
      const int c = __ffsll(children) - 1;
      children &= children - 1;
      if (tok[c] < 0) continue;
      double r = at_p[c];
      if (Q) r = positive(r - A * at_q[c]);
      else
        for (unsigned long long m = gone; m; m &= m - 1)
          if (tok[__ffsll(m) - 1] == tok[c]) r = 0.0;
      if (at_u[c] * M * at_q[c] < r) {
        moved = true;
        cur = c;
        if (tid == 0) out_path[len] = c;
        ++len;
        M = 1.0;
        A = 0.0;
        gone = 0;
        P = target + static_cast<long long>(c) * p.target_stride;
        if (Q) Q = draft + static_cast<long long>(c) * p.draft_stride;
      } else if (Q) {
        A += M;
        double before;
        if (children) M = mass(before);  // needed only by another child
      } else {
        M -= r;
        gone |= 1ull << c;
      }
    }
    if (!moved) break;
  }

  // ---- the draw, from the rest; where nothing is left, from cur's own row
  double before = 0.0, total = mass(before);
  if (!(total > 0.0) && (A > 0.0 || gone)) {
    A = 0.0;
    gone = 0;
    total = mass(before);
  }
  if (!(total > 0.0) || isinf(total)) {
    if (rank == 0 && tid == 0) {
      p.next_token[b] = -1;
      flag_error(p.err, S4KV_EFLAG_PROBS);
    }
  } else {
    double t = positive(at_u[0] * total);
    // the CTA whose share holds t; where t is the end of the sum, the last one with any mass
    bool holds = before <= t && before + part[(sums - 1) & 1] > t;
    if (t >= total) {
      int last = 0;
      for (int r = 0; r < C; ++r)
        if (*cluster.map_shared_rank(&part[(sums - 1) & 1], r) > 0.0) last = r;
      holds = rank == last;
    }
    if (holds && warp == 0) {
      // the chunk, then the entry: the first whose cumulative sum passes t, or the last with any mass where
      // rounding lets none pass
      int pick = -1, last = -1;
      double run = before, at = before;
      for (int k = 0; k < k1 - k0 && pick < 0; k += 32) {
        const double x = k + lane < k1 - k0 ? chunk_sum[k + lane] : 0.0;
        double incl = x;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const double o = __shfl_up_sync(kAllV, incl, off);
          if (lane >= off) incl += o;
        }
        const unsigned hit = __ballot_sync(kAllV, x > 0.0 && run + incl > t), some = __ballot_sync(kAllV, x > 0.0);
        if (hit) {
          pick = k + __ffs(hit) - 1;
          at = __shfl_sync(kAllV, run + incl - x, __ffs(hit) - 1);
        } else if (some) {
          last = k + 31 - __clz(some);
        }
        run += __shfl_sync(kAllV, incl, 31);
      }
      if (pick < 0) {
        pick = last;
        t = INFINITY;  // its last entry with any mass
      }
      int answer = -1;
      last = -1;
      for (int e = 0; e < blocks && answer < 0; ++e) {
        const int v0 = (k0 + pick) * chunk + e * kBlockV;
        double x[kPerLane];
        rest(v0, x);
#pragma unroll
        for (int j = 0; j < kPerLane; ++j) {
          double incl = x[j];
#pragma unroll
          for (int off = 1; off < 32; off <<= 1) {
            const double o = __shfl_up_sync(kAllV, incl, off);
            if (lane >= off) incl += o;
          }
          const unsigned hit = __ballot_sync(kAllV, x[j] > 0.0 && at + incl > t), some = __ballot_sync(kAllV, x[j] > 0.0);
          if (hit && answer < 0) answer = v0 + 32 * j + __ffs(hit) - 1;
          if (some) last = v0 + 32 * j + 31 - __clz(some);
          at += __shfl_sync(kAllV, incl, 31);
        }
      }
      if (lane == 0) p.next_token[b] = answer >= 0 ? answer : last;
    }
  }
  if (rank == 0) {
    __syncthreads();
    if (tid < p.max_nodes) path[tid] = tid == 0 ? 0 : tid < n ? out_path[tid] : -1;
    if (tid == 0) p.path_len[b] = len;
  }
  cluster.sync();  // no CTA leaves while another reads its share
}

template <typename T>
static cudaError_t launch_verify_for(const VerifyParams &p, cudaStream_t stream) {
  // CTAs a sequence: the number that takes the shortest time, as waves of what is on the card at once, each of a fixed
  // part (walk, exchange, draw) as long as kWaveEntries entries and a CTA's share of the row.  Of 4 CTAs an SM clusters
  // of 4 and 8 leave one in 25 idle (148 SMs: 71 clusters of 8, 142 of 4, 296 of 2, by the occupancy query); no more
  // CTAs than leave each warp a chunk of its own.  Measured, fp32 with draft rows, us for 8 / 4 / 2 / 1:
  //   128256 entries: 70 sequences 16 / 21 / 34 / -, 74 22.5 / 22.3 / 35 / 61, 136 31 / 26 / 40 / -, 200 44 / 45 / 43 / 71,
  //   296 66 / 61 / 47 / 72, 400 83 / 70 / 77 / 77, 592 119 / 105 / 89 / 85, 800 158 / 131 / 120 / 140, 1600 - / - / 224 / 217
  //   32000: 70 8.4 / 8.5 / 10.7 / -, 74 12.6 / 8.7 / 10.7 / 15.3, 136 15 / 10.3 / 11.3 / -, 144 18 / 13.9 / 11.5 / -,
  //   296 36 / 26 / 16 / 21, 400 46 / 31 / 29 / 25, 800 89 / 58 / 44 / 46, 1600 - / - / 81 / 69
  //   4000: 70 7.5 / 6.5 / 6.5 / 6.6
  int cluster = 1;
  long long best = 0;
  for (int c = 1; c <= kMaxCluster && (c == 1 || p.vocab > kBlockV * kWarpsV * (c / 2)); c *= 2) {
    const int slots = kCtasAnSm * p.num_sms, at_once = (c > 2 ? slots - slots / 25 : slots) / c;
    const long long t = static_cast<long long>((p.batch - 1) / at_once + 1) * (p.vocab / c + kWaveEntries);
    if (c == 1 || t < best) {
      best = t;
      cluster = c;
    }
  }
  const int blocks = static_cast<int>((static_cast<long long>(p.vocab) / cluster + 1) / (static_cast<long long>(kBlockV) * (kMaxChunks - 2)) + 1);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.batch) * cluster);
  cfg.blockDim = dim3(kThreadsV);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_kernel<T>, p, blocks);
}

cudaError_t launch_verify(const VerifyParams &p, cudaStream_t stream) {
  return p.prob_type == S4KV_PROB_F16 ? launch_verify_for<__half>(p, stream)
         : p.prob_type == S4KV_PROB_BF16 ? launch_verify_for<__nv_bfloat16>(p, stream) : launch_verify_for<float>(p, stream);
}

}  // namespace s4kv
