// kv_cache.cu -- writing new tokens' keys and values to the paged cache and
// reading cached rows back (glinattn_kv_append, glinattn_kv_gather).
//
// Mathematics: a row x of d elements becomes e4m3 values times a power of two
// 2^e, e the smallest exponent for which max |x| <= 448 * 2^e.  A power of two
// makes x * 2^-e exact, so the one rounding is that to e4m3 (half a step,
// 2^-4 relative), and the way back is exact in bf16.
//
// Bound: HBM bytes, 2 d bytes of bf16 and d (+ 1) of e4m3 per row and head.
// A warp finds its packed row's request (32-way search, all lanes), then moves
// every (head, k / v) row of it, 8 elements a lane, with all loads of a round in
// flight before the first store.  Appending 8 prompts of
// 1,500 .. 8,000 tokens (8 heads of 128, e4m3) takes 35.5 us, 6,100 GB/s; gathering 4
// prefixes of 20,000 .. 32,768 tokens (4 heads) 56 us, 6,000 GB/s; one token of 256
// requests 2.7 us (other numbers of loads in flight and of warps a CTA measured no better).
#include "paged.cuh"

namespace glinattn {
namespace paged {

glinattn_status check_cache(int cache_dtype, int num_req, int num_tok, int kv_heads, int head_dim, int page_size,
                            int num_pages, int max_pages, const void *k_cache, const void *v_cache, const void *k_scale,
                            const void *v_scale, const void *page_table, const void *kv_len, const void *q_start) {
  if (cache_dtype != GLINATTN_BF16 && cache_dtype != GLINATTN_E4M3) return GLINATTN_ERR_INVALID_ARG;
  if (num_req < 0 || num_req > 65536 || num_tok < 0 || kv_heads <= 0 || head_dim <= 0 || page_size <= 0 ||
      num_pages < 0 || max_pages < 0)
    return GLINATTN_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return GLINATTN_ERR_UNSUPPORTED;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) return GLINATTN_ERR_UNSUPPORTED;
  // the (page, head) planes of the cache and the positions of a request are 32-bit numbers
  if ((long long)num_pages * kv_heads > (1ll << 30) || (long long)max_pages * page_size > (1ll << 30))
    return GLINATTN_ERR_INVALID_ARG;
  if (num_req == 0 || num_tok == 0) return GLINATTN_OK;
  if (!kv_len || !q_start || (max_pages > 0 && !page_table) || (num_pages > 0 && (!k_cache || !v_cache)))
    return GLINATTN_ERR_INVALID_ARG;
  if (cache_dtype == GLINATTN_E4M3 && num_pages > 0 && (!k_scale || !v_scale)) return GLINATTN_ERR_INVALID_ARG;
  const void *list[] = {k_cache, v_cache, k_scale, v_scale};
  for (const void *p : list)
    if ((uintptr_t)p & 15u) return GLINATTN_ERR_INVALID_ARG;
  const void *ints[] = {page_table, kv_len, q_start};
  for (const void *p : ints)
    if ((uintptr_t)p & 3u) return GLINATTN_ERR_INVALID_ARG;
  return GLINATTN_OK;
}

namespace {

constexpr int kWarps = 4;   // of a CTA
constexpr int kRound = 4;   // steps of a lane in flight: half of them k rows, half v rows

// Code (exponent plus 127) of a row's scale from the largest finite |x| as bf16
// bits, x = 1.m * 2^(E - 127) <= 1.75 * 2^8 * 2^e: e = E - 135, one more where m
// is above 0x60 (then the addition carries into E); subnormals end at -100.
__device__ __forceinline__ uint32_t scale_code(uint32_t amax) {
  return (uint32_t)min(max((int)((amax + 0x1fu) >> 7) - 8, 27), 246);
}

__device__ __forceinline__ uint32_t finite_mag(uint32_t bits16) {
  const uint32_t a = bits16 & 0x7fffu;
  return a < 0x7f80u ? a : 0u;
}

// The magnitudes' maximum, with some sign; a NaN gives way to a number.
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Largest finite |x| of two rows, as bf16 bits in the halves of the result; a row
// is in kLanes lanes, 8 elements each.  Rows with infinities (or NaN alone) again
// with those left out.
template <int kLanes>
__device__ __forceinline__ uint32_t rows_amax(const uint4 &x, const uint4 &y) {
  const uint32_t a = max_abs_bf16x2(max_abs_bf16x2(x.x, x.y), max_abs_bf16x2(x.z, x.w));
  const uint32_t b = max_abs_bf16x2(max_abs_bf16x2(y.x, y.y), max_abs_bf16x2(y.z, y.w));
  uint32_t m = max_abs_bf16x2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) m = max_abs_bf16x2(m, __shfl_xor_sync(0xffffffffu, m, o));
  m &= 0x7fff7fffu;
  if (__any_sync(0xffffffffu, ((m + 0x00800080u) & 0x80008000u) != 0)) {
    const uint32_t w[2][4] = {{x.x, x.y, x.z, x.w}, {y.x, y.y, y.z, y.w}};
    uint32_t v[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[i] = max(v[i], max(finite_mag(w[i][k]), finite_mag(w[i][k] >> 16)));
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) v[i] = max(v[i], __shfl_xor_sync(0xffffffffu, v[i], o));
    }
    m = v[0] | v[1] << 16;
  }
  return m;
}

// Eight bf16 times 2^-e as e4m3; eight e4m3 times their scale as bf16.
__device__ __forceinline__ uint2 quantise(const uint4 &x, uint32_t code) {
  const float f = __uint_as_float((254u - code) << 23);
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t q[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 y = __fmul2_rn(make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u)), make_float2(f, f));
    q[k] = to_e4m3x2(y.x, y.y);
  }
  return make_uint2(__byte_perm(q[0], q[1], 0x5410), __byte_perm(q[2], q[3], 0x5410));
}
__device__ __forceinline__ uint4 dequantise(const uint2 &y, uint32_t code) {
  const float f = scale_value(code);
  const uint32_t w[4] = {y.x & 0xffffu, y.x >> 16, y.y & 0xffffu, y.y >> 16};
  uint32_t q[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 v = __fmul2_rn(e4m3x2(w[k]), make_float2(f, f));
    q[k] = pack_bf16(v.x, v.y);
  }
  return make_uint4(q[0], q[1], q[2], q[3]);
}

// Where the packed rows of a warp, one after the other, are in the cache.
struct Place {
  int r = 0, s1 = 0, pos = 0, page = -1;
  bool good = false;  // the last row was in a request that is in bounds
  // Whether row i is to be moved; then `page` and pos % page_size say where.
  __device__ __forceinline__ bool find(const glinattn_kv_args &a, int i, int lane) {
    if (good && i < s1) {  // the next position of the same request
      ++pos;
    } else {
      r = find_request(a.q_start, a.num_req, i, lane);
      const int s0 = a.q_start[r], len = a.kv_len[r];
      s1 = a.q_start[r + 1];
      // a row in no request's range: the search lands in the range before it, or in a decreasing one
      good = i >= s0 && i < s1 && request_ok(s0, s1, len, a.num_tok, (long long)a.max_pages * a.page_size);
      if (!good) return false;
      pos = len - (s1 - i);
      page = -1;
    }
    if (pos < 0) return false;
    const int row = pos & (a.page_size - 1);
    if (page == -1 || row == 0) {
      page = a.page_table[(size_t)r * a.max_pages + pos / a.page_size];
      if (page < 0 || page >= a.num_pages) {
        if (lane == 0 && a.dev_status) atomicOr(a.dev_status, GLINATTN_DEV_BAD_SLOT);
        page = -2;
      }
    }
    return page >= 0;
  }
};

// The ranges themselves are checked once, request by request, by the first CTAs.
__device__ __forceinline__ void check_requests(const glinattn_kv_args &a) {
  if (!a.dev_status) return;
  const long long max_len = (long long)a.max_pages * a.page_size;
  for (int r = blockIdx.x * blockDim.x + threadIdx.x; r < a.num_req; r += gridDim.x * blockDim.x)
    if (!request_ok(a.q_start[r], a.q_start[r + 1], a.kv_len[r], a.num_tok, max_len))
      atomicOr(a.dev_status, GLINATTN_DEV_BAD_COUNT);
}

// kRows: packed rows of a warp.
template <int D, bool kE4m3, bool kAppend, int kRows>
__global__ void __launch_bounds__(32 * kWarps) kv_move_kernel(const glinattn_kv_args a) {
  constexpr int kLanes = D / 8;             // lanes of one (head, k / v) row
  constexpr int kPer = 32 / kLanes;         // such rows a warp moves at a time
  constexpr int kHeads = kRound / 2 * kPer; // heads of a round
  constexpr int kEsz = kE4m3 ? 1 : 2;
  check_requests(a);
  const int lane = threadIdx.x & 31;
  const int i0 = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * kRows, i1 = min(i0 + kRows, a.num_tok);
  const int H = a.kv_heads, sub = lane / kLanes, c = lane % kLanes;
  Place place;
  for (int i = i0; i < i1; ++i) {           // whole warps
    // eight elements of head h in the token's row, its step 0 .. kRound - 1 of a round: k rows, then v rows
    const size_t token = ((size_t)i * H + sub) * D + c * 8;
    auto token_at = [&](int u, int h0) {
      return reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(u < kRound / 2 ? a.k : a.v) + token + (h0 + u % (kRound / 2) * kPer) * D);
    };
    auto there = [&](int u, int h0) { return h0 + u % (kRound / 2) * kPer + sub < H; };
    uint4 x[kRound];
    auto read_tokens = [&](int h0) {
#pragma unroll
      for (int u = 0; u < kRound; ++u) x[u] = there(u, h0) ? __ldcs(token_at(u, h0)) : make_uint4(0, 0, 0, 0);
    };
    if (kAppend) read_tokens(0);              // in flight while the row is located
    if (!place.find(a, i, lane)) continue;
    size_t cr = ((size_t)place.page * H + sub) * a.page_size + (place.pos & (a.page_size - 1));  // the lane's first row of the cache
    for (int h0 = 0; h0 < H; h0 += kHeads, cr += (size_t)kHeads * a.page_size) {
      auto cached_at = [&](int u) {
        const size_t at = cr + (uint32_t)(u % (kRound / 2) * kPer * a.page_size);
        return reinterpret_cast<uint8_t *>(u < kRound / 2 ? a.k_cache : a.v_cache) + (at * D + c * 8) * kEsz;
      };
      auto scale_at = [&](int u) {
        return (u < kRound / 2 ? a.k_scale : a.v_scale) + (cr + (uint32_t)(u % (kRound / 2) * kPer * a.page_size));
      };
      if (kAppend) {
        if (h0 > 0) read_tokens(h0);
        if constexpr (kE4m3) {
#pragma unroll
          for (int u = 0; u < kRound; u += 2) {
            const uint32_t m = rows_amax<kLanes>(x[u], x[u + 1]);
            const uint32_t code[2] = {scale_code(m & 0xffffu), scale_code(m >> 16)};
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              const uint2 q = quantise(x[u + v], code[v]);
              if (there(u + v, h0)) {
                *reinterpret_cast<uint2 *>(cached_at(u + v)) = q;
                if (c == 0) *scale_at(u + v) = (uint8_t)code[v];
              }
            }
          }
        } else {
#pragma unroll
          for (int u = 0; u < kRound; ++u)
            if (there(u, h0)) *reinterpret_cast<uint4 *>(cached_at(u)) = x[u];
        }
      } else {
        uint32_t code[kRound];
#pragma unroll
        for (int u = 0; u < kRound; ++u) {
          x[u] = make_uint4(0, 0, 0, 0);
          code[u] = 0;
          if (!there(u, h0)) continue;
          if (kE4m3) {
            const uint2 y = *reinterpret_cast<const uint2 *>(cached_at(u));
            x[u].x = y.x;
            x[u].y = y.y;
            code[u] = *scale_at(u);
          } else {
            x[u] = *reinterpret_cast<const uint4 *>(cached_at(u));
          }
        }
#pragma unroll
        for (int u = 0; u < kRound; ++u) {
          const uint4 y = kE4m3 ? dequantise(make_uint2(x[u].x, x[u].y), code[u]) : x[u];
          if (there(u, h0)) __stcs(token_at(u, h0), y);
        }
      }
    }
  }
}

template <bool kAppend>
glinattn_status move(const glinattn_kv_args *a, cudaStream_t stream) {
  if (!a) return GLINATTN_ERR_INVALID_ARG;
  const glinattn_status st =
      check_cache(a->cache_dtype, a->num_req, a->num_tok, a->kv_heads, a->head_dim, a->page_size, a->num_pages,
                  a->max_pages, a->k_cache, a->v_cache, a->k_scale, a->v_scale, a->page_table, a->kv_len, a->q_start);
  if (st != GLINATTN_OK) return st;
  if (a->num_req == 0 || a->num_tok == 0) return GLINATTN_OK;
  if (!a->k || !a->v || (((uintptr_t)a->k | (uintptr_t)a->v) & 15u)) return GLINATTN_ERR_INVALID_ARG;
  // Four rows a warp where e4m3 rows are read and there are enough of them to fill
  // the SMs: the look-ups for the next rows cost little, and a row has few bytes in
  // flight.  4 heads of 128, one row and four: 4,096 rows 4.2 and 5.1 us, 16,384 rows
  // 8.6 and 7.7 us, 109,688 rows 60 and 56 us; of bf16 rows 43 and 43.5 us (65,536);
  // appending 35.5 and 41 us (8 prompts of 1,500 .. 8,000 tokens, 8 heads).
  auto run = [&](auto kernel, int rows) {
    kernel<<<(unsigned)((a->num_tok - 1) / (rows * kWarps) + 1), 32 * kWarps, 0, stream>>>(*a);
  };
  if (a->cache_dtype == GLINATTN_BF16) {
    if (a->head_dim == 128) run(kv_move_kernel<128, false, kAppend, 1>, 1);
    else run(kv_move_kernel<64, false, kAppend, 1>, 1);
  } else if (kAppend || a->num_tok < 8192) {
    if (a->head_dim == 128) run(kv_move_kernel<128, true, kAppend, 1>, 1);
    else run(kv_move_kernel<64, true, kAppend, 1>, 1);
  } else {
    if (a->head_dim == 128) run(kv_move_kernel<128, true, false, 4>, 4);
    else run(kv_move_kernel<64, true, false, 4>, 4);
  }
  return cudaGetLastError() == cudaSuccess ? GLINATTN_OK : GLINATTN_ERR_CUDA;
}

}  // namespace
}  // namespace paged
}  // namespace glinattn

extern "C" {

glinattn_status glinattn_kv_append(const glinattn_kv_args *args, glinattn_stream_t stream) {
  return glinattn::paged::move<true>(args, (cudaStream_t)stream);
}

glinattn_status glinattn_kv_gather(const glinattn_kv_args *args, glinattn_stream_t stream) {
  return glinattn::paged::move<false>(args, (cudaStream_t)stream);
}

}  // extern "C"
