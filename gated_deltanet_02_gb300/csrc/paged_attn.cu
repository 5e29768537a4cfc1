// paged_attn.cu -- causal softmax attention of new tokens over the paged cache
// (glinattn_paged_attention).
//
// Mathematics: for each (token, head) row one pass over the keys it sees, with
// the running maximum m and sum l of the softmax and an output accumulator that
// is rescaled by 2^(m_old - m_new) whenever m grows; scores in log2 units.
#include <math.h>

#include "paged_sched.cuh"

namespace glinattn {
namespace paged {
namespace {

constexpr int kWarps = 4;

// One warp per (token row, head), lane = D / 32 channels.
template <int D, bool kE4m3>
__global__ void __launch_bounds__(32 * kWarps) attn_row_kernel(const glinattn_paged_attn_args a) {
  constexpr int kE = D / 32;
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int i = (int)(unit / a.heads), h = (int)(unit % a.heads);
  if (i >= a.num_tok) return;
  const int r = find_request(a.q_start, a.num_req, i, lane);
  const int s0 = a.q_start[r], s1 = a.q_start[r + 1], len = a.kv_len[r];
  if (i < s0 || i >= s1) return;
  if (!request_ok(s0, s1, len, a.num_tok, (long long)a.max_pages * a.page_size) || s1 - s0 > a.max_q_len) {
    if (lane == 0 && a.dev_status) atomicOr(a.dev_status, GLINATTN_DEV_BAD_COUNT);
    return;
  }
  const int seen = len - (s1 - i) + 1;
  const int hk = h / (a.heads / a.kv_heads);
  const float c = a.scale * 1.44269504088896341f;
  float q[kE], o[kE], m = -INFINITY, l = 0.f;
  const __nv_bfloat16 *qp = reinterpret_cast<const __nv_bfloat16 *>(a.q) + ((size_t)i * a.heads + h) * D + lane * kE;
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    q[e] = __bfloat162float(qp[e]);
    o[e] = 0.f;
  }
  for (int j = 0; j < seen; ++j) {
    const int page = a.page_table[(size_t)r * a.max_pages + j / a.page_size];
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0 && a.dev_status) atomicOr(a.dev_status, GLINATTN_DEV_BAD_SLOT);
      return;
    }
    const size_t cr = ((size_t)page * a.kv_heads + hk) * a.page_size + j % a.page_size;
    float k[kE], v[kE], ks = 1.f, vs = 1.f;
    if (kE4m3) {
      const uint16_t *kp = reinterpret_cast<const uint16_t *>(reinterpret_cast<const uint8_t *>(a.k_cache) + cr * D + lane * kE);
      const uint16_t *vp = reinterpret_cast<const uint16_t *>(reinterpret_cast<const uint8_t *>(a.v_cache) + cr * D + lane * kE);
#pragma unroll
      for (int e = 0; e < kE; e += 2) {
        const float2 fk = e4m3x2(kp[e / 2]), fv = e4m3x2(vp[e / 2]);
        k[e] = fk.x, k[e + 1] = fk.y, v[e] = fv.x, v[e + 1] = fv.y;
      }
      ks = scale_value(a.k_scale[cr]);
      vs = scale_value(a.v_scale[cr]);
    } else {
      const __nv_bfloat16 *kp = reinterpret_cast<const __nv_bfloat16 *>(a.k_cache) + cr * D + lane * kE;
      const __nv_bfloat16 *vp = reinterpret_cast<const __nv_bfloat16 *>(a.v_cache) + cr * D + lane * kE;
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        k[e] = __bfloat162float(kp[e]);
        v[e] = __bfloat162float(vp[e]);
      }
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < kE; ++e) s = fmaf(q[e], k[e], s);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= ks * c;
    const float mn = fmaxf(m, s), ms = mn == -INFINITY ? 0.f : mn;
    const float f = exp2f(m - ms), p = exp2f(s - ms);
    m = mn;
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < kE; ++e) o[e] = fmaf(p * vs, v[e], o[e] * f);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  __nv_bfloat16 *op = reinterpret_cast<__nv_bfloat16 *>(a.o) + ((size_t)i * a.heads + h) * D + lane * kE;
#pragma unroll
  for (int e = 0; e < kE; ++e) op[e] = __float2bfloat16_rn(l == 0.f ? 0.f : o[e] * inv);
}

glinattn_status check(const glinattn_paged_attn_args *a) {
  if (!a) return GLINATTN_ERR_INVALID_ARG;
  const glinattn_status st =
      check_cache(a->cache_dtype, a->num_req, a->num_tok, a->kv_heads, a->head_dim, a->page_size, a->num_pages,
                  a->max_pages, a->k_cache, a->v_cache, a->k_scale, a->v_scale, a->page_table, a->kv_len, a->q_start);
  if (st != GLINATTN_OK) return st;
  if (a->heads <= 0 || a->heads % a->kv_heads != 0 || a->max_q_len < 0) return GLINATTN_ERR_INVALID_ARG;
  if ((long long)a->num_tok * a->heads > (1ll << 30)) return GLINATTN_ERR_INVALID_ARG;
  if (!(a->scale > 0.f) || isinf(a->scale)) return GLINATTN_ERR_INVALID_ARG;
  if (a->num_req == 0 || a->num_tok == 0) return GLINATTN_OK;
  if (!a->q || !a->o || (((uintptr_t)a->q | (uintptr_t)a->o) & 15u)) return GLINATTN_ERR_INVALID_ARG;
  return GLINATTN_OK;
}

// Rows of an item that the decode kernel's accumulators are built for.
int item_rows(const glinattn_paged_attn_args *a) {
  const long long rows = (long long)a->max_q_len * (a->heads / a->kv_heads);
  return rows <= 16 ? 16 : rows <= kDecodeRows ? 32 : 0;
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    return 152;
  return n;
}

// The workspace's parts, each 16-byte aligned: desc, skip, ml, part.
size_t carve(int ctas, int rows, int d, AttnParams *p, uint8_t *base) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t *x = base + at;
    at += (bytes + 15) & ~(size_t)15;
    return x;
  };
  uint8_t *desc = take((size_t)ctas * sizeof(int4));
  uint8_t *skip = take((size_t)ctas * 2 * sizeof(int));
  uint8_t *ml = take((size_t)ctas * 2 * rows * sizeof(float2));
  uint8_t *part = take((size_t)ctas * 2 * rows * d * sizeof(float));
  if (p) {
    p->desc = reinterpret_cast<int4 *>(desc);
    p->skip = reinterpret_cast<int *>(skip);
    p->ml = reinterpret_cast<float2 *>(ml);
    p->part = reinterpret_cast<float *>(part);
  }
  return at;
}

}  // namespace
}  // namespace paged
}  // namespace glinattn

extern "C" {

size_t glinattn_paged_attention_workspace_size(const glinattn_paged_attn_args *a) {
  using namespace glinattn::paged;
  if (check(a) != GLINATTN_OK || a->num_req == 0 || a->num_tok == 0) return 0;
  const int rows = item_rows(a);
  return rows ? carve(2 * sm_count(), rows, a->head_dim, nullptr, nullptr) : 0;
}

glinattn_status glinattn_paged_attention(const glinattn_paged_attn_args *a, glinattn_stream_t stream) {
  using namespace glinattn::paged;
  const glinattn_status st = check(a);
  if (st != GLINATTN_OK) return st;
  if (a->num_req == 0 || a->num_tok == 0) return GLINATTN_OK;
  const bool f8 = a->cache_dtype == GLINATTN_E4M3;
  if (const int rows = item_rows(a)) {
    const int ctas = 2 * sm_count();
    if (!a->workspace || ((uintptr_t)a->workspace & 15u) ||
        a->workspace_bytes < carve(ctas, rows, a->head_dim, nullptr, nullptr))
      return GLINATTN_ERR_INVALID_ARG;
    AttnParams p = {};
    p.R = a->num_req;
    p.N = a->num_tok;
    p.H = a->heads;
    p.Hkv = a->kv_heads;
    p.G = a->heads / a->kv_heads;
    p.page = a->page_size;
    p.page_shift = a->page_size == 16 ? 4 : a->page_size == 32 ? 5 : a->page_size == 64 ? 6 : 7;
    p.P = a->num_pages;
    p.max_pages = a->max_pages;
    p.max_q = a->max_q_len;
    p.tp = 1 << 30;
    p.c = a->scale * 1.44269504088896341f;
    p.q = reinterpret_cast<const __nv_bfloat16 *>(a->q);
    p.k_scale = a->k_scale;
    p.v_scale = a->v_scale;
    p.table = a->page_table;
    p.kv_len = a->kv_len;
    p.q_start = a->q_start;
    p.o = reinterpret_cast<__nv_bfloat16 *>(a->o);
    p.dev_status = a->dev_status;
    carve(ctas, rows, a->head_dim, &p, reinterpret_cast<uint8_t *>(a->workspace));
    return launch_decode(p, f8, a->head_dim, rows, a->k_cache, a->v_cache, ctas, (cudaStream_t)stream) == cudaSuccess
               ? GLINATTN_OK
               : GLINATTN_ERR_CUDA;
  }
  auto kernel = a->head_dim == 128 ? (f8 ? attn_row_kernel<128, true> : attn_row_kernel<128, false>)
                                   : (f8 ? attn_row_kernel<64, true> : attn_row_kernel<64, false>);
  const long long units = (long long)a->num_tok * a->heads;
  kernel<<<(unsigned)((units + kWarps - 1) / kWarps), 32 * kWarps, 0, (cudaStream_t)stream>>>(*a);
  return cudaGetLastError() == cudaSuccess ? GLINATTN_OK : GLINATTN_ERR_CUDA;
}

}  // extern "C"
