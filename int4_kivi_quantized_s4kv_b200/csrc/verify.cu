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
// One CTA a sequence; the row is taken in chunks of consecutive entries whose
// sums stay in shared memory, so that the second pass reads only the chunk that
// holds the answer.
#include <cuda_bf16.h>

#include "kernels.cuh"

namespace s4kv {

namespace {

constexpr int kThreadsV = 512;
constexpr int kPerThread = 8;
constexpr int kChunk = kThreadsV * kPerThread;

__device__ __forceinline__ double prob(const float *p) { return static_cast<double>(*p); }
__device__ __forceinline__ double prob(const __half *p) { return static_cast<double>(__half2float(*p)); }
__device__ __forceinline__ double prob(const __nv_bfloat16 *p) { return static_cast<double>(__bfloat162float(*p)); }
// negative entries and NaN count as 0
__device__ __forceinline__ double positive(double x) { return x > 0.0 ? x : 0.0; }

// Sum over the CTA, given to every thread; `scratch`: one double a warp.
__device__ __forceinline__ double cta_sum(double x, double *scratch) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, off);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = x;
  __syncthreads();
  double s = 0.0;
  for (int w = 0; w < kThreadsV / 32; ++w) s += scratch[w];
  return s;
}

}  // namespace

template <typename T>
__global__ void __launch_bounds__(kThreadsV) verify_kernel(const VerifyParams p) {
  __shared__ int tok[S4KV_MAX_TREE_NODES], par[S4KV_MAX_TREE_NODES], out_path[S4KV_MAX_TREE_NODES];
  __shared__ double scratch[kThreadsV / 32];
  __shared__ int answer;
  const int b = blockIdx.x, tid = threadIdx.x;
  const int c0 = __ldg(p.cu_nodes + b), c1 = __ldg(p.cu_nodes + b + 1), n = c1 - c0;
  int32_t *path = p.path + static_cast<long>(b) * p.max_nodes;
  const bool ok = c0 >= 0 && n >= 0 && c1 <= p.n_nodes && n <= p.max_nodes;
  if (!ok || n == 0) {
    if (tid < p.max_nodes) path[tid] = -1;
    if (tid == 0) {
      p.path_len[b] = 0;
      p.next_token[b] = -1;
      if (!ok) flag_error(p.err, S4KV_EFLAG_TREE);
    }
    return;
  }
  if (tid < n) {
    tok[tid] = __ldg(p.tokens + c0 + tid);
    par[tid] = __ldg(p.parents + c0 + tid);
    if (tid > 0 && static_cast<unsigned>(tok[tid]) >= static_cast<unsigned>(p.vocab)) flag_error(p.err, S4KV_EFLAG_TREE);
  }
  if (tid < p.max_nodes) out_path[tid] = tid == 0 ? 0 : -1;
  __syncthreads();

  const T *target = static_cast<const T *>(p.target), *draft = static_cast<const T *>(p.draft);
  const int V = p.vocab;
  int cur = 0, len = 1;
  double M = 1.0, A = 0.0;
  unsigned long long gone = 0;  // rejected children of cur
  const T *P = target + static_cast<long long>(c0) * p.target_stride;
  const T *Q = draft ? draft + static_cast<long long>(c0) * p.draft_stride : nullptr;
  // what is left of entry v
  auto rest = [&](int v) {
    if (Q) return positive(positive(prob(P + v)) - A * positive(prob(Q + v)));
    for (unsigned long long g = gone; g; g &= g - 1)
      if (tok[__ffsll(g) - 1] == v) return 0.0;
    return positive(prob(P + v));
  };
  for (int c = 1; c < n; ++c) {  // children come after their parent, in the order they are tried
    if (par[c] != cur || static_cast<unsigned>(tok[c]) >= static_cast<unsigned>(V)) continue;
    const double r = rest(tok[c]), u = static_cast<double>(__ldg(p.uniforms + c0 + c));
    const double q = Q ? positive(prob(Q + tok[c])) : 1.0;
    if (u * M * q < r) {
      if (tid == 0) out_path[len] = c;
      ++len;
      cur = c;
      M = 1.0;
      A = 0.0;
      gone = 0;
      P = target + static_cast<long long>(c0 + c) * p.target_stride;
      if (Q) Q = draft + static_cast<long long>(c0 + c) * p.draft_stride;
    } else if (Q) {
      A += M;
      bool more = false;  // the new mass is needed only by another child
      for (int d = c + 1; d < n; ++d) more |= par[d] == cur;
      if (more) {
        double s = 0.0;
        for (int v = tid; v < V; v += kThreadsV) s += rest(v);
        M = cta_sum(s, scratch);
      }
    } else {
      M -= r;
      gone |= 1ull << c;
    }
  }

  // draw from the rest; where nothing is left, from cur's own row
  auto draw = [&]() -> int {
    double total = 0.0;
    for (int v = tid; v < V; v += kThreadsV) total += rest(v);
    total = cta_sum(total, scratch);
    if (!(total > 0.0) || isinf(total)) return -1;
    const double t = static_cast<double>(__ldg(p.uniforms + c0)) * total;
    if (tid == 0) answer = -1;
    double before = 0.0;
    for (int v0 = 0; v0 < V; v0 += kChunk) {
      const int lo = v0 + tid * kPerThread;
      double mine = 0.0;
      int last = -1;
      for (int k = 0; k < kPerThread; ++k)
        if (lo + k < V) {
          const double r = rest(lo + k);
          mine += r;
          if (r > 0.0) last = lo + k;
        }
      const double chunk = cta_sum(mine, scratch);
      if (before + chunk > t) {
        // inclusive scan over the threads
        double incl = mine;
        for (int off = 1; off < 32; off <<= 1) {
          const double o = __shfl_up_sync(0xFFFFFFFFu, incl, off);
          if ((tid & 31) >= off) incl += o;
        }
        __syncthreads();
        if ((tid & 31) == 31) scratch[tid >> 5] = incl;
        __syncthreads();
        double base = before;
        for (int w = 0; w < (tid >> 5); ++w) base += scratch[w];
        const double excl = base + incl - mine;
        if (excl <= t && base + incl > t) {
          double run = excl;
          int hit = last;
          for (int k = 0; k < kPerThread; ++k)
            if (lo + k < V) {
              run += rest(lo + k);
              if (run > t) {
                hit = lo + k;
                break;
              }
            }
          atomicMax(&answer, hit);
        }
        __syncthreads();
        if (answer >= 0) return answer;
      }
      before += chunk;
    }
    // t reaches the end of the sum: the last entry with any mass
    __syncthreads();
    for (int v = tid; v < V; v += kThreadsV)
      if (rest(v) > 0.0) atomicMax(&answer, v);
    __syncthreads();
    return answer;
  };
  int next = draw();
  if (next < 0 && (A > 0.0 || gone)) {
    A = 0.0;
    gone = 0;
    __syncthreads();
    next = draw();
  }
  if (tid < p.max_nodes) path[tid] = out_path[tid];
  if (tid == 0) {
    p.path_len[b] = len;
    p.next_token[b] = next;
    if (next < 0) flag_error(p.err, S4KV_EFLAG_PROBS);
  }
}

cudaError_t launch_verify(const VerifyParams &p, cudaStream_t stream) {
  if (p.prob_type == S4KV_PROB_F16) verify_kernel<__half><<<p.batch, kThreadsV, 0, stream>>>(p);
  else if (p.prob_type == S4KV_PROB_BF16) verify_kernel<__nv_bfloat16><<<p.batch, kThreadsV, 0, stream>>>(p);
  else verify_kernel<float><<<p.batch, kThreadsV, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace s4kv
