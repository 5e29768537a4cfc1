// accept.cu -- acceptance of drafted tokens and the draw of the token that
// follows them (glinattn_accept_drafts).
//
// Mathematics: draft i with token x is accepted iff u_i q_i(x) < p_i(x); the
// next token comes from the normalised residual max(p_a - q_a, 0) at the first
// rejected position a (or from p_n).  The cumulative draw runs over whole
// numbers W(v) = trunc(w(v) 2^40), whose sums (at most 2^62) are exact in any
// order, so splitting a row over CTAs cannot move the drawn token.
//
// Bound: HBM bytes, one pass over one row of p (and one of q after a
// rejection); a single request is bound by latency.  One cluster of 8 CTAs
// owns a request: 64 warps sum one contiguous 64th of the row each, every
// CTA gets all 64 sums through distributed shared memory, and the CTA whose
// piece holds the threshold reads that piece (V / 64 elements, from L2) again
// to find the token.
#include "common.cuh"

namespace glinattn {
namespace {

constexpr int kCluster = 8, kThreads = 256, kWarps = kThreads / 32;
constexpr int kPieces = kCluster * kWarps;
constexpr int kAhead = 8;  // elements of a row that a lane has in flight
constexpr float kWeight = 1099511627776.f;  // 2^40

typedef unsigned long long u64;

__device__ __forceinline__ u64 weight(float w) {
  return (u64)(fminf(fmaxf(w, 0.f), 1.f) * kWeight);  // fmaxf(NaN, 0) is 0
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void st_remote(u64 *p, uint32_t rank, u64 v) {
  const uint32_t a = (uint32_t)__cvta_generic_to_shared(p);
  asm volatile("{\n\t.reg .b32 ra;\n\tmapa.shared::cluster.u32 ra, %0, %1;\n\tst.shared::cluster.u64 [ra], %2;\n\t}" ::"r"(a), "r"(rank),
               "l"(v)
               : "memory");
}

// The weights of one request's draw.
struct Row {
  const float *p, *q;  // q NULL: none is taken off
  int zero;            // the element without weight (the rejected point mass), or -1
  __device__ __forceinline__ float at(int v) const { return q ? p[v] - q[v] : v == zero ? 0.f : p[v]; }
};

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads) accept_kernel(const glinattn_accept_args a) {
  __shared__ u64 s_piece[2][kPieces];
  __shared__ u64 s_warp[kWarps];
  __shared__ int s_accept;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int r = blockIdx.x / kCluster;
  const int D = a.draft_len, V = a.vocab;
  const int n = a.num_drafts ? a.num_drafts[r] : D;
  const float *target = a.target_probs + (size_t)r * (D + 1) * V;
  const float *draft = a.draft_probs ? a.draft_probs + (size_t)r * D * V : nullptr;
  const int32_t *tokens = a.draft_tokens + (size_t)r * D;
  const float *u = a.uniforms + (size_t)r * (D + 1);

  // ---- accepted drafts: every CTA's warp 0, a lane per draft -------------------
  if (n < 0 || n > D) {  // the same in all CTAs of the cluster, as every exit before the barriers
    if (rank == 0 && tid == 0 && a.dev_status) atomicOr(a.dev_status, GLINATTN_DEV_BAD_COUNT);
    return;
  }
  if (warp == 0) {
    int acc = n, bad = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int i = i0 + lane;
      bool reject = false, wrong = false;
      if (i < n) {
        const int x = tokens[i];
        wrong = x < 0 || x >= V;
        if (!wrong) {
          const float qx = draft ? draft[(size_t)i * V + x] : 1.f;
          reject = !(__fmul_rn(u[i], qx) < target[(size_t)i * V + x]);
        }
      }
      const unsigned rej = __ballot_sync(0xffffffffu, reject);
      bad |= __any_sync(0xffffffffu, wrong);
      if (rej && acc == n) acc = i0 + __ffs(rej) - 1;
    }
    if (lane == 0) s_accept = bad ? -1 : acc;
  }
  __syncthreads();
  const int acc = s_accept;
  if (acc < 0) {
    if (rank == 0 && tid == 0 && a.dev_status) atomicOr(a.dev_status, GLINATTN_DEV_BAD_TOKEN);
    return;
  }

  // ---- the row of weights, its 64 pieces' sums -----------------------------------
  const bool rejected = acc < n;
  Row w;
  w.p = target + (size_t)acc * V;
  w.q = rejected && draft ? draft + (size_t)acc * V : nullptr;
  w.zero = rejected && !draft ? tokens[acc] : -1;
  const int len = (V + kPieces - 1) / kPieces;  // elements of a piece
  const int piece = (int)rank * kWarps + warp;
  const int v0 = min(piece * len, V), v1 = min(v0 + len, V);
  cluster_sync();  // every CTA of the cluster runs: its shared memory may be written
  u64 total = 0;
  for (int pass = 0; pass < 2; ++pass) {
    u64 sum = 0;
    for (int b = v0 + lane; b < v1; b += 32 * kAhead) {
      float x[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) x[k] = b + 32 * k < v1 ? w.at(b + 32 * k) : 0.f;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) sum += weight(x[k]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane < kCluster) st_remote(&s_piece[pass][piece], (uint32_t)lane, sum);
    __syncwarp();
    cluster_sync();
    total = 0;
    for (int k = 0; k < kPieces; ++k) total += s_piece[pass][k];
    if (total > 0) {
      // ---- the piece that holds the threshold, and in it the token -----------------
      const double prod = (double)u[D] * (double)total;
      u64 t = prod > 0. ? (u64)prod : 0;
      if (!(t < total)) t = total - 1;
      u64 before = 0;
      int hit = 0;
      for (; hit < kPieces - 1 && before + s_piece[pass][hit] <= t; ++hit) before += s_piece[pass][hit];
      if (hit / kWarps != (int)rank) return;
      const int h0 = hit * len, h1 = min(h0 + len, V);
      const int per = (len + kThreads - 1) / kThreads;  // contiguous elements of a thread
      const int e0 = min(h0 + tid * per, h1), e1 = min(e0 + per, h1);
      u64 mine = 0;
      for (int v = e0; v < e1; ++v) mine += weight(w.at(v));
      u64 upto = mine;  // inclusive scan over the CTA
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      if (lane == 31) s_warp[warp] = upto;
      __syncthreads();
      for (int k = 0; k < warp; ++k) upto += s_warp[k];
      const u64 start = before + upto - mine;
      if (start <= t && t < start + mine) {  // exactly one thread
        u64 run = start;
        int v = e0;
        for (; v < e1 - 1; ++v) {
          run += weight(w.at(v));
          if (run > t) break;
        }
        a.tokens[(size_t)r * (D + 1) + acc] = v;
        a.accept[r] = acc;
      }
      for (int i = tid; i <= D; i += kThreads)
        if (i != acc) a.tokens[(size_t)r * (D + 1) + i] = i < acc ? tokens[i] : -1;
      return;
    }
    if (!rejected) break;
    w.q = nullptr;  // the residual has no mass: the target's own row
    w.zero = -1;
  }
  if (rank == 0 && tid == 0 && a.dev_status) atomicOr(a.dev_status, GLINATTN_DEV_BAD_PROB);
}

}  // namespace
}  // namespace glinattn

extern "C" glinattn_status glinattn_accept_drafts(const glinattn_accept_args *a, glinattn_stream_t stream) {
  using namespace glinattn;
  if (!a) return GLINATTN_ERR_INVALID_ARG;
  if (a->num_req < 0 || a->num_req > (1 << 24) || a->draft_len < 0 || a->draft_len > 1024 || a->vocab < 1 ||
      a->vocab > (1 << 22))
    return GLINATTN_ERR_INVALID_ARG;
  if (a->num_req == 0) return GLINATTN_OK;
  if (!a->target_probs || !a->uniforms || !a->accept || !a->tokens || (a->draft_len > 0 && !a->draft_tokens))
    return GLINATTN_ERR_INVALID_ARG;
  const void *list[] = {a->target_probs, a->draft_probs, a->draft_tokens, a->num_drafts, a->uniforms, a->accept, a->tokens};
  for (const void *p : list)
    if ((uintptr_t)p & 3u) return GLINATTN_ERR_INVALID_ARG;
  accept_kernel<<<(unsigned)a->num_req * kCluster, kThreads, 0, (cudaStream_t)stream>>>(*a);
  return cudaGetLastError() == cudaSuccess ? GLINATTN_OK : GLINATTN_ERR_CUDA;
}
