// scan_packed.cu -- the selective scan over packed rows with its step bias, skip
// and gate, the states in a slot-indexed pool (glinattn_selective_scan_packed).
//
// Mathematics, per channel d and state index n, dt = softplus(delta + bias):
//   h_t = exp(dt A) h_{t-1} + dt B_t x_t,   y_t = (sum_n h_t C_t + skip x_t) silu(z_t).
// A thread owns a channel and its N states in registers and runs its request's
// rows in order; the rows' B and C are in shared memory.
#include "packed.cuh"

namespace glinattn {
namespace scan {
namespace {

using namespace packed;

struct Params {
  Rows rows;
  const void *x, *delta, *z, *Bm, *Cm;
  long long x_stride, delta_stride, z_stride, b_stride, c_stride;
  const float *A, *skip, *delta_bias;
  float *pool;
  void *y;
  int D, update, out_bf16;
};

constexpr int kThreads = 128, kRows = 32;

__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x))); }

template <bool kBf16, int N>
__global__ void __launch_bounds__(kThreads) scan_kernel(const Params p) {
  __shared__ float sB[kRows][N], sC[kRows][N];
  if (blockIdx.x == 0 && blockIdx.y == 0) check_requests(p.rows, threadIdx.x, kThreads);
  const Request q = request(p.rows, blockIdx.y);
  if (!q.ok || q.run == 0) return;
  const int d = blockIdx.x * kThreads + threadIdx.x;
  const bool in = d < p.D;
  float A[N], h[N];
  float *state = p.pool + ((size_t)q.slot * p.D + d) * N;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    A[n] = in ? p.A[(size_t)d * N + n] * 1.4426950408889634f : 0.0f;
    h[n] = in && q.resumed ? state[n] : 0.0f;
  }
  const float bias = in && p.delta_bias ? p.delta_bias[d] : 0.0f, skip = in && p.skip ? p.skip[d] : 0.0f;
  for (int base = 0; base < q.run; base += kRows) {
    const int rows = min(kRows, q.run - base);
    __syncthreads();
    for (int e = threadIdx.x; e < rows * N; e += kThreads) {
      const size_t t = (size_t)q.s0 + base + e / N;
      sB[e / N][e % N] = load_one<kBf16>(p.Bm, t * p.b_stride + e % N);
      if (p.y) sC[e / N][e % N] = load_one<kBf16>(p.Cm, t * p.c_stride + e % N);
    }
    __syncthreads();
    if (!in) continue;
    for (int i = 0; i < rows; ++i) {
      const size_t t = (size_t)q.s0 + base + i;
      const float x = load_one<kBf16>(p.x, t * p.x_stride + d);
      const float dt = softplus(load_one<kBf16>(p.delta, t * p.delta_stride + d) + bias), dtx = dt * x;
      float y = skip * x;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        h[n] = fmaf(exp2f(dt * A[n]), h[n], dtx * sB[i][n]);
        if (p.y) y = fmaf(h[n], sC[i][n], y);
      }
      if (!p.y) continue;
      if (p.z) {
        const float z = load_one<kBf16>(p.z, t * p.z_stride + d);
        y *= z / (1.0f + expf(-z));
      }
      if (p.out_bf16) store_one<true>(p.y, t * p.D + d, y);
      else store_one<false>(p.y, t * p.D + d, y);
    }
  }
  if (p.update && in)
#pragma unroll
    for (int n = 0; n < N; ++n) state[n] = h[n];
}

template <bool kBf16>
void launch(const Params &p, int N, cudaStream_t s) {
  const dim3 grid((unsigned)((p.D + kThreads - 1) / kThreads), (unsigned)p.rows.R);
  if (N == 8) scan_kernel<kBf16, 8><<<grid, kThreads, 0, s>>>(p);
  else if (N == 16) scan_kernel<kBf16, 16><<<grid, kThreads, 0, s>>>(p);
  else scan_kernel<kBf16, 32><<<grid, kThreads, 0, s>>>(p);
}

bool activation(int dtype) { return dtype == GLINATTN_F32 || dtype == GLINATTN_BF16; }

glinattn_status run(const glinattn_scan_packed_args *a, cudaStream_t stream) {
  if (!a || !activation(a->in_dtype) || !activation(a->out_dtype) || a->num_req < 0 || a->num_tok < 0 || a->channels <= 0 ||
      a->state <= 0 || a->max_q_len < 0 || a->x_stride < 0 || a->delta_stride < 0 || a->z_stride < 0 || a->b_stride < 0 ||
      a->c_stride < 0)
    return GLINATTN_ERR_INVALID_ARG;
  if ((a->state != 8 && a->state != 16 && a->state != 32) || a->num_req > 65535 || a->channels > (1 << 20)) return GLINATTN_ERR_UNSUPPORTED;
  if ((a->state_pool == nullptr) != (a->slot_ids == nullptr) || (a->state_pool && a->pool_slots <= 0)) return GLINATTN_ERR_INVALID_ARG;
  if (!a->q_start && a->num_tok != a->num_req) return GLINATTN_ERR_INVALID_ARG;
  if (a->num_req == 0 || a->num_tok == 0) return GLINATTN_OK;
  const bool update = a->update_state && a->state_pool;
  if (!a->x || !a->delta || !a->Bm || !a->A || (a->y && !a->Cm) || (!a->y && !update)) return GLINATTN_ERR_INVALID_ARG;
  const size_t es = a->in_dtype == GLINATTN_BF16 ? 2 : 4, os = a->out_dtype == GLINATTN_BF16 ? 2 : 4;
  const int D = a->channels, N = a->state;
  const long long strides[] = {a->x_stride ? a->x_stride : D, a->delta_stride ? a->delta_stride : D, a->z_stride ? a->z_stride : D,
                               a->b_stride ? a->b_stride : N, a->c_stride ? a->c_stride : N};
  const void *rows[] = {a->x, a->delta, a->z, a->Bm, a->Cm};
  const size_t ny = (size_t)a->num_tok * D * os, np = a->state_pool ? (size_t)a->pool_slots * D * N * 4 : 0;
  for (int i = 0; i < 5; ++i) {
    if (!rows[i]) continue;
    const int width = i < 3 ? D : N;
    if ((strides[i] < width && a->num_tok > 1) || !aligned(rows[i], es)) return GLINATTN_ERR_INVALID_ARG;
    const size_t n = row_bytes(a->num_tok, width, strides[i], es);
    if (overlap(a->y, ny, rows[i], n) || (update && overlap(a->state_pool, np, rows[i], n))) return GLINATTN_ERR_INVALID_ARG;
  }
  if (overlap(a->y, ny, a->state_pool, np)) return GLINATTN_ERR_INVALID_ARG;
  const void *list[] = {a->A, a->skip, a->delta_bias, a->state_pool, a->y};
  for (const void *q : list)
    if (!aligned(q, 16)) return GLINATTN_ERR_INVALID_ARG;
  const void *ints[] = {a->slot_ids, a->q_start, a->resume, a->count};
  for (const void *q : ints)
    if (!aligned(q, 4)) return GLINATTN_ERR_INVALID_ARG;
  Params p;
  p.rows = {a->num_req, a->num_tok, a->pool_slots, a->max_q_len, a->state_pool != nullptr, a->q_start, a->slot_ids, a->resume, a->count,
            a->dev_status};
  p.x = a->x, p.delta = a->delta, p.z = a->z, p.Bm = a->Bm, p.Cm = a->Cm;
  p.x_stride = strides[0], p.delta_stride = strides[1], p.z_stride = strides[2], p.b_stride = strides[3], p.c_stride = strides[4];
  p.A = a->A, p.skip = a->skip, p.delta_bias = a->delta_bias, p.pool = a->state_pool, p.y = a->y;
  p.D = D, p.update = update, p.out_bf16 = a->out_dtype == GLINATTN_BF16;
  if (a->in_dtype == GLINATTN_BF16) launch<true>(p, N, stream);
  else launch<false>(p, N, stream);
  return cudaGetLastError() == cudaSuccess ? GLINATTN_OK : GLINATTN_ERR_CUDA;
}

}  // namespace
}  // namespace scan
}  // namespace glinattn

extern "C" glinattn_status glinattn_selective_scan_packed(const glinattn_scan_packed_args *args, glinattn_stream_t stream) {
  return glinattn::scan::run(args, (cudaStream_t)stream);
}
