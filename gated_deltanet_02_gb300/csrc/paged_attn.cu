// paged_attn.cu -- the host side of glinattn_paged_attention: argument checks,
// the workspace, and the choice between the kernels.
//
// A call whose items (query tokens x heads of a group) have few rows runs the
// transposed kernel of paged_decode.cu, any other call, mixtures of prompts and
// single tokens among them, the one of paged_prefill.cu with 256 rows an item.
#include <math.h>

#include "paged_sched.cuh"
#include "paged_tc.cuh"

namespace glinattn {
namespace paged {

bool encode_map(CUtensorMap *m, const void *base, CUtensorMapDataType type, int elem_bytes, const long long dims[3],
                const int box[3], CUtensorMapSwizzle swizzle) {
  static const auto encode = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found);
    return (decltype(&cuTensorMapEncodeTiled))(e == cudaSuccess && found == cudaDriverEntryPointSuccess ? f : nullptr);
  }();
  if (!encode) return false;
  const cuuint64_t size[3] = {(cuuint64_t)dims[0], (cuuint64_t)dims[1], (cuuint64_t)dims[2]};
  const cuuint64_t stride[2] = {size[0] * elem_bytes, size[0] * size[1] * elem_bytes};
  const cuuint32_t extent[3] = {(cuuint32_t)box[0], (cuuint32_t)box[1], (cuuint32_t)box[2]}, step[3] = {1, 1, 1};
  return encode(m, type, 3, const_cast<void *>(base), size, stride, extent, step, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

constexpr float kLog2e = 1.44269504088896341f;

glinattn_status check(const glinattn_paged_attn_args *a) {
  if (!a) return GLINATTN_ERR_INVALID_ARG;
  const glinattn_status st =
      check_cache(a->cache_dtype, a->num_req, a->num_tok, a->kv_heads, a->head_dim, a->page_size, a->num_pages,
                  a->max_pages, a->k_cache, a->v_cache, a->k_scale, a->v_scale, a->page_table, a->kv_len, a->q_start);
  if (st != GLINATTN_OK) return st;
  if (a->heads <= 0 || a->heads % a->kv_heads != 0 || a->max_q_len < 0) return GLINATTN_ERR_INVALID_ARG;
  if ((long long)a->num_tok * a->heads > (1ll << 30)) return GLINATTN_ERR_INVALID_ARG;
  if (a->heads / a->kv_heads > kPrefillRows) return GLINATTN_ERR_UNSUPPORTED;
  if (!(a->scale > 0.f) || isinf(a->scale * kLog2e)) return GLINATTN_ERR_INVALID_ARG;
  if (a->num_req == 0 || a->num_tok == 0) return GLINATTN_OK;
  if (!a->q || !a->o || (((uintptr_t)a->q | (uintptr_t)a->o) & 15u)) return GLINATTN_ERR_INVALID_ARG;
  return GLINATTN_OK;
}

// Rows of an item: what the kernel's accumulators are built for.  Single tokens
// and drafts run the kernel for few rows, in which query rows are the narrow side
// of the tensor-core tile.  64 requests after 8,192 tokens, 4 kv heads of 128:
//   rows          8    16    24    32    40    48
//   bf16 few    165   170   (no accumulators for more: a build that had them took 182 .. 206)
//        many   169   170   173   174   176   177 us
//   e4m3 few     97   104   115   122   156   163
//        many   209   210   211   213   214   214
// One request after 30,000: e4m3 21 .. 37 us against 39, bf16 24 and 26 against 35; four
// after 900: e4m3 12 .. 17 against 17 up to 32 rows, 19 and 21 against 18 with 40 and 48, bf16
// 12.7 and 14.2 against 14.2.  The lengths are not known here, so short caches lose the 2 us.
int item_rows(const glinattn_paged_attn_args *a) {
  const long long rows = (long long)a->max_q_len * (a->heads / a->kv_heads);
  if (rows <= 16) return 16;
  if (a->cache_dtype != GLINATTN_E4M3 || rows > 48) return kPrefillRows;
  return rows <= 32 ? 32 : 48;
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    return 152;
  return n;
}

// CTAs of a call: as many as the SMs hold at a time.
int item_ctas(int rows) { return rows == kPrefillRows ? sm_count() : 2 * sm_count(); }

// The workspace's parts, each 16-byte aligned: desc, skip, ml, part.
size_t carve(int ctas, int rows, int d, AttnParams *p, uint8_t *base) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t *x = base + at;
    at += (bytes + 15) & ~(size_t)15;
    return x;
  };
  uint8_t *desc = take((size_t)ctas * sizeof(int4));
  uint8_t *skip = take((size_t)ctas * 4 * sizeof(int));
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
  return carve(item_ctas(rows), rows, a->head_dim, nullptr, nullptr);
}

glinattn_status glinattn_paged_attention(const glinattn_paged_attn_args *a, glinattn_stream_t stream) {
  using namespace glinattn::paged;
  const glinattn_status st = check(a);
  if (st != GLINATTN_OK) return st;
  if (a->num_req == 0 || a->num_tok == 0) return GLINATTN_OK;
  const bool f8 = a->cache_dtype == GLINATTN_E4M3;
  const int rows = item_rows(a), ctas = item_ctas(rows);
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
  p.tp = rows == kPrefillRows ? kPrefillRows / p.G : 1 << 30;
  p.c = a->scale * kLog2e;
  p.q = reinterpret_cast<const __nv_bfloat16 *>(a->q);
  p.k_scale = a->k_scale;
  p.v_scale = a->v_scale;
  p.table = a->page_table;
  p.kv_len = a->kv_len;
  p.q_start = a->q_start;
  p.o = reinterpret_cast<__nv_bfloat16 *>(a->o);
  p.dev_status = a->dev_status;
  carve(ctas, rows, a->head_dim, &p, reinterpret_cast<uint8_t *>(a->workspace));
  const cudaError_t e =
      rows == kPrefillRows
          ? launch_prefill(p, f8, a->head_dim, a->k_cache, a->v_cache, ctas, (cudaStream_t)stream)
          : launch_decode(p, f8, a->head_dim, rows, a->k_cache, a->v_cache, ctas, (cudaStream_t)stream);
  return e == cudaSuccess ? GLINATTN_OK : GLINATTN_ERR_CUDA;
}

}  // extern "C"
