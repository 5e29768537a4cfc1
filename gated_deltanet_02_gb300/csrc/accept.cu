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
// owns a request: every warp sums one contiguous piece of the row, all CTAs
// get all pieces' sums through distributed shared memory, and the CTA whose
// piece holds the threshold reads that piece again (from L2; its warps sum an
// eighth each, then one warp walks to the token).  256 threads with 12 elements
// each in flight and 5 CTAs per SM: 256 requests of V = 160,000 take 52 us (58 us
// with 8 elements and 6 CTAs, 53 with 16 and 4, 70 with CTAs of 512 threads; clusters
// of 4, 2 and 1 CTAs were slower too); one request of V = 100,003 takes 7 us, most of
// it launch, barriers and the chain of loads.
#include "common.cuh"

namespace glinattn {
namespace {

constexpr int kCluster = 8;
constexpr int kThreads = 256;
constexpr int kAhead = 12;  // elements of a row that a lane has in flight

typedef unsigned long long u64;

// trunc(w 2^40) of two weights in [0, 1] as hi 2^20 + lo, hi and lo each below
// the exponent field of 2^23 (kBias): w 2^20 + 2^23 rounded towards zero holds
// floor(w 2^20) in its low bits, what that leaves is exact, and so once more.  Two-lane
// fp32 arithmetic, 3.5 instructions a weight with its share of the sums; shifting
// the significand in 64 bits, 256 requests of V = 160,000 took 61 us.
constexpr uint32_t kBias = 0x4b000000u;
__device__ __forceinline__ void parts(float2 w, uint2 &hi, uint2 &lo) {
  const float2 one = make_float2(8388608.f, 8388608.f), scale = make_float2(1048576.f, 1048576.f);
  const float2 x = __fmul2_rn(w, scale);
  const float2 t = __fadd2_rz(x, one);
  const float2 f = __fadd2_rn(x, __fadd2_rn(one, make_float2(-t.x, -t.y)));
  const float2 y = __ffma2_rz(f, scale, one);
  hi = make_uint2(__float_as_uint(t.x), __float_as_uint(t.y));
  lo = make_uint2(__float_as_uint(y.x), __float_as_uint(y.y));
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
  // weights of the elements b + 32 k < end, k < kAhead, in [0, 1] (NaN: 0), all loaded before the first is used
  template <bool kFull>
  __device__ __forceinline__ void load(int b, int end, float (&x)[kAhead]) const {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) x[k] = kFull || b + 32 * k < end ? __ldg(p + b + 32 * k) : 0.f;
    if (q) {
      float y[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) y[k] = kFull || b + 32 * k < end ? __ldg(q + b + 32 * k) : 0.f;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) x[k] = __saturatef(x[k] - y[k]);
    } else {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) x[k] = __saturatef(x[k]);
    }
    if (zero >= 0) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) x[k] = b + 32 * k == zero ? 0.f : x[k];
    }
  }
  // the warp's sum over [v0, v1), in every lane: at most 2^11 elements a lane, so
  // that 32 bits hold the sums of their parts (2^20 at most each) once the biases,
  // which wrap, are taken off
  __device__ __forceinline__ u64 sum(int v0, int v1, int lane) const {
    uint32_t hi = 0, lo = 0, bias = 0;
    auto add = [&](const float (&x)[kAhead]) {
#pragma unroll
      for (int k = 0; k < kAhead; k += 2) {
        uint2 h, l;
        parts(make_float2(x[k], x[k + 1]), h, l);
        hi += h.x + h.y;
        lo += l.x + l.y;
      }
      bias += kBias * kAhead;
    };
    int b = v0;
    float x[kAhead];
    for (; b + 32 * kAhead <= v1; b += 32 * kAhead) {
      load<true>(b + lane, v1, x);
      add(x);
    }
    if (b < v1) {
      load<false>(b + lane, v1, x);
      add(x);
    }
    u64 s = ((u64)(hi - bias) << 20) + (lo - bias);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
  }
};

__device__ __forceinline__ u64 warp_scan(u64 x, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 5) accept_kernel(const glinattn_accept_args a) {
  constexpr int kWarps = kThreads / 32, kPieces = kCluster * kWarps, kPer = kPieces / 32;
  __shared__ u64 s_piece[2][kPieces];
  __shared__ u64 s_sub[kWarps];
  __shared__ u64 s_t, s_before, s_total;
  __shared__ int s_accept, s_hit;
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
  for (int pass = 0; pass < 2; ++pass) {
    const u64 sum = w.sum(v0, v1, lane);
    if (lane < kCluster) st_remote(&s_piece[pass][piece], (uint32_t)lane, sum);
    __syncwarp();
    cluster_sync();
    if (warp == 0) {  // lane l has pieces kPer l ..; the threshold and its piece
      u64 mine[kPer], group = 0;
#pragma unroll
      for (int k = 0; k < kPer; ++k) group += mine[k] = s_piece[pass][kPer * lane + k];
      const u64 upto = warp_scan(group, lane);
      const u64 all = __shfl_sync(0xffffffffu, upto, 31);
      if (lane == 0) s_total = all;
      if (all > 0) {
        const double prod = (double)u[D] * (double)all;
        u64 t = prod > 0. ? (u64)prod : 0;
        if (!(t < all)) t = all - 1;
        if (upto - group <= t && t < upto) {  // one lane
          u64 before = upto - group;
          int hit = kPer * lane;
#pragma unroll
          for (int k = 0; k < kPer - 1; ++k)
            if (hit == kPer * lane + k && before + mine[k] <= t) {
              before += mine[k];
              ++hit;
            }
          s_hit = hit;
          s_before = before;
          s_t = t;
        }
      }
    }
    __syncthreads();
    const u64 total = s_total;
    if (total > 0) {
      const u64 t = s_t, before = s_before;
      const int hit = s_hit;
      if (hit / kWarps != (int)rank) return;
      for (int i = tid; i <= D; i += kThreads)
        if (i != acc) a.tokens[(size_t)r * (D + 1) + i] = i < acc ? tokens[i] : -1;
      const int h0 = min(hit * len, V), h1 = min(h0 + len, V);
      const int sl = (len + kWarps - 1) / kWarps;
      const int e0 = min(h0 + warp * sl, h1), e1 = min(e0 + sl, h1);
      const u64 s = w.sum(e0, e1, lane);
      if (lane == 0) s_sub[warp] = s;
      __syncthreads();
      u64 run = before;
      for (int k = 0; k < warp; ++k) run += s_sub[k];
      if (!(run <= t && t < run + s)) return;  // exactly one warp goes on
      for (int b = e0; b < e1; b += 32 * kAhead) {
        float x[kAhead];
        w.load<false>(b + lane, e1, x);
#pragma unroll 1
        for (int k = 0; k < kAhead; ++k) {
          float y = 0.f;
#pragma unroll
          for (int j = 0; j < kAhead; ++j) y = j == k ? x[j] : y;
          uint2 h, l;
          parts(make_float2(y, 0.f), h, l);
          const u64 c = run + warp_scan(((u64)(h.x - kBias) << 20) + (l.x - kBias), lane);
          const unsigned over = __ballot_sync(0xffffffffu, c > t);
          if (over) {
            if (lane == 0) {
              a.tokens[(size_t)r * (D + 1) + acc] = b + 32 * k + __ffs(over) - 1;
              a.accept[r] = acc;
            }
            return;
          }
          run = __shfl_sync(0xffffffffu, c, 31);
        }
      }
      return;
    }
    if (!rejected) break;
    __syncthreads();  // s_total is read
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
