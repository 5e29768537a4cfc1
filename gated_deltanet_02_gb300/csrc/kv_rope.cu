// kv_rope.cu -- writing new tokens' keys and values to the paged cache with the
// position rotation applied to keys and queries on the way (glinattn_kv_append_rope).
//
// Mathematics: pair i at position p turns by p f_i radians.  f / (2 pi) is held as a
// 64-bit fraction of a turn, so that p times it, modulo 2^64, is the exact fraction
// of a turn but for p 2^-64: no position is too far.  The fraction is split into a
// quarter turn and a rest within an eighth, whose sine and cosine need no reduction.
//
// Bound: HBM bytes.  A warp moves one packed row: its lanes make the sines and
// cosines of all pairs once (two or fewer each, shared through shared memory),
// then each lane moves units of 16 channels, 8 pairs, of the row's heads.  8 prompts of 1,500 .. 8,000 tokens,
// 32 heads over 8 of 128, into an e4m3 cache take 153 us (5,990 GB/s); one token of 256 requests, 16 heads
// over 4, 4.8 us (the look-ups in q_start and the page table, one behind the other).
#include "packed.cuh"

namespace glinattn {
namespace paged {
namespace {

using packed::finite_bits;
using packed::load_raw8;
using packed::overlap;
using packed::Raw8;
using packed::row_bytes;
using packed::unpack8;

constexpr int kWarps = 4;  // of a CTA

// f / (2 pi) modulo 1 as a fraction of 2^64, for |f| < 2^24: the 24 bits of f's
// significand times 1 / (2 pi), of which 128 bits are kept, shifted into place.
__device__ __forceinline__ unsigned long long turn_of(float f) {
  const uint32_t bits = __float_as_uint(f), e = (bits >> 23) & 0xffu;
  const unsigned long long m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);
  // m 2^(max(e, 1) - 150) / (2 pi) 2^64 = m c 2^(max(e, 1) - 86 - 128), c = 2^128 / (2 pi)
  const unsigned long long hi = 0x28be60db9391054aull, lo = 0x7f09d5f47d4d3770ull;
  const int right = 214 - (int)max(e, 1u) - 64;  // 64 of the shift: m lo's low half
  const unsigned long long p0 = m * hi, p1 = __umul64hi(m, hi), c0 = __umul64hi(m, lo);
  const unsigned long long low = p0 + c0, high = p1 + (low < p0 ? 1 : 0);
  const unsigned long long u = right >= 128 ? 0 : right >= 64 ? high >> (right - 64) : right == 0 ? low : low >> right | high << (64 - right);
  return (bits >> 31) ? 0ull - u : u;
}

// Cosine and sine of a fraction of a turn.
__device__ __forceinline__ float2 cos_sin(unsigned long long turn) {
  const uint32_t quarter = (uint32_t)((turn + (1ull << 61)) >> 62);
  const long long rest = (long long)(turn - ((unsigned long long)quarter << 62));  // within an eighth
  float s, c;
  sincospif((float)rest * 0x1p-63f, &s, &c);  // its argument is in half turns
  const float cs = quarter & 1 ? s : c, sn = quarter & 1 ? c : s;
  return make_float2(quarter == 1 || quarter == 2 ? -cs : cs, quarter & 2 ? -sn : sn);
}

template <int D, bool kE4m3>
__global__ void __launch_bounds__(32 * kWarps) rope_kernel(const glinattn_kv_rope_args a) {
  constexpr int kUnits = D / 16;         // 16 channels each, of one head
  constexpr int kHeads = 32 / kUnits;    // heads a warp moves at a time
  __shared__ float2 turns[kWarps][D / 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long max_len = (long long)a.max_pages * a.page_size;
  if (a.dev_status)
    for (int r = blockIdx.x * blockDim.x + threadIdx.x; r < a.num_req; r += gridDim.x * blockDim.x)
      if (!request_ok(a.q_start[r], a.q_start[r + 1], a.kv_len[r], a.num_tok, max_len))
        atomicOr(a.dev_status, GLINATTN_DEV_BAD_COUNT);
  const long long row = (long long)blockIdx.x * kWarps + warp;
  if (row >= a.num_tok) return;
  const int i = (int)row;
  const int r = find_request(a.q_start, a.num_req, i, lane);
  const int s0 = a.q_start[r], s1 = a.q_start[r + 1], len = a.kv_len[r];
  if (i < s0 || i >= s1 || !request_ok(s0, s1, len, a.num_tok, max_len)) return;
  const int pos = len - (s1 - i);
  if (pos < 0) return;
  int page = a.page_table[(size_t)r * a.max_pages + pos / a.page_size];
  if (page < 0 || page >= a.num_pages) {
    if (lane == 0 && a.dev_status) atomicOr(a.dev_status, GLINATTN_DEV_BAD_SLOT);
    page = -1;
  }
  const int pairs = a.rotary_dim / 2;
  for (int k = lane; k < pairs; k += 32) {
    const float f = a.inv_freq[k];
    float2 t = cos_sin(turn_of(f) * (unsigned long long)(uint32_t)pos);
    if (!(fabsf(f) < 16777216.0f)) t.x = t.y = __uint_as_float(0x7fffffffu);
    turns[warp][k] = make_float2(t.x * a.rope_scale, t.y * a.rope_scale);
  }
  __syncwarp();
  const int unit = lane % kUnits, sub = lane / kUnits;
  const bool turned = unit < a.rotary_dim / 16;
  // the unit's two groups of 8 channels
  const int c0 = turned && !a.interleaved ? 8 * unit : 16 * unit, c1 = turned && !a.interleaved ? pairs + 8 * unit : 16 * unit + 8;
  float cs[8], sn[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 t = turned ? turns[warp][8 * unit + k] : make_float2(1.0f, 0.0f);
    cs[k] = t.x, sn[k] = t.y;
  }
  auto rotate = [&](float *u, float *v) {  // the 16 channels in place
    if (!a.interleaved) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float x = u[k], y = v[k];
        u[k] = fmaf(x, cs[k], -(y * sn[k]));
        v[k] = fmaf(y, cs[k], x * sn[k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float *w = k < 4 ? u + 2 * k : v + 2 * (k - 4);
        const float x = w[0], y = w[1];
        w[0] = fmaf(x, cs[k], -(y * sn[k]));
        w[1] = fmaf(y, cs[k], x * sn[k]);
      }
    }
  };
  // a unit to bf16 memory: rotated, or bit for bit
  auto store_turned = [&](void *to, size_t at, const Raw8<true> &x, const Raw8<true> &y, bool turn) {
    if (turn) {
      float u[8], v[8];
      unpack8(x, u);
      unpack8(y, v);
      rotate(u, v);
      packed::store8<true>(to, at + c0, u);
      packed::store8<true>(to, at + c1, v);
    } else {
      packed::store_raw8(to, at + c0, x);
      packed::store_raw8(to, at + c1, y);
    }
  };
  // queries
  for (int h = sub; h < a.heads; h += kHeads) {
    const size_t at = (size_t)i * a.q_stride + h * D, to = (size_t)i * a.q_out_stride + h * D;
    const Raw8<true> x = load_raw8<true>(a.q, at + c0), y = load_raw8<true>(a.q, at + c1);
    store_turned(a.q_out, to, x, y, turned);
  }
  if (page < 0) return;
  // keys, then values
  for (int s = 0; s < 2; ++s) {
    const void *src = s ? a.v : a.k;
    void *dst = s ? a.v_cache : a.k_cache;
    const long long stride = s ? a.v_stride : a.k_stride;
    for (int h0 = 0; h0 < a.kv_heads; h0 += kHeads) {  // whole warps: the maximum is over lanes
      const int h = h0 + sub;
      const bool in = h < a.kv_heads;
      Raw8<true> x = {}, y = {};
      if (in) {
        x = load_raw8<true>(src, (size_t)i * stride + h * D + c0);
        y = load_raw8<true>(src, (size_t)i * stride + h * D + c1);
      }
      const size_t line = ((size_t)page * a.kv_heads + h) * a.page_size + (pos & (a.page_size - 1));
      if constexpr (kE4m3) {
        float u[8], v[8];
        unpack8(x, u);
        unpack8(y, v);
        if (s == 0 && turned) rotate(u, v);
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) top = max(top, max(finite_bits(u[k]), finite_bits(v[k])));
#pragma unroll
        for (int o = kUnits / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const uint32_t code = packed::scale_code(top);
        const float f = __uint_as_float((254u - code) << 23);
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] *= f, v[k] *= f;
        if (in) {
          uint8_t *to = reinterpret_cast<uint8_t *>(dst) + line * D;
          *reinterpret_cast<uint2 *>(to + c0) = packed::to_e4m3x8(u);
          *reinterpret_cast<uint2 *>(to + c1) = packed::to_e4m3x8(v);
          if (unit == 0) (s ? a.v_scale : a.k_scale)[line] = (uint8_t)code;
        }
      } else if (in) {
        store_turned(dst, line * D, x, y, s == 0 && turned);
      }
    }
  }
}

glinattn_status run(const glinattn_kv_rope_args *args, cudaStream_t stream) {
  if (!args) return GLINATTN_ERR_INVALID_ARG;
  glinattn_kv_rope_args a = *args;
  const glinattn_status st = check_cache(a.cache_dtype, a.num_req, a.num_tok, a.kv_heads, a.head_dim, a.page_size, a.num_pages, a.max_pages,
                                         a.k_cache, a.v_cache, a.k_scale, a.v_scale, a.page_table, a.kv_len, a.q_start);
  if (st != GLINATTN_OK) return st;
  if (a.heads < 0 || a.rotary_dim <= 0 || a.rotary_dim > a.head_dim || !(a.rope_scale > 0.0f && a.rope_scale <= 1e30f))
    return GLINATTN_ERR_INVALID_ARG;
  if (a.rotary_dim % 16) return GLINATTN_ERR_UNSUPPORTED;
  if (a.heads > 65536 || a.kv_heads > 65536) return GLINATTN_ERR_UNSUPPORTED;
  if (a.num_req == 0 || a.num_tok == 0) return GLINATTN_OK;
  const long long d = a.head_dim, nq = a.heads * d, nk = a.kv_heads * d;
  int64_t *strides[] = {&a.q_stride, &a.q_out_stride, &a.k_stride, &a.v_stride};
  const void *rows[] = {a.q, a.q_out, a.k, a.v};
  size_t bytes[4];
  for (int i = 0; i < 4; ++i) {
    const long long width = i < 2 ? nq : nk;
    if (*strides[i] == 0) *strides[i] = width;
    if (*strides[i] < 0 || *strides[i] % 8 || (*strides[i] < width && a.num_tok > 1)) return GLINATTN_ERR_INVALID_ARG;
    if ((width && !rows[i]) || !packed::aligned(rows[i], 16)) return GLINATTN_ERR_INVALID_ARG;
    bytes[i] = width ? row_bytes(a.num_tok, width, *strides[i], 2) : 0;
  }
  if (!a.inv_freq || !packed::aligned(a.inv_freq, 4)) return GLINATTN_ERR_INVALID_ARG;
  // q_out may be q itself; it may lie between k's and v's rows (slices of the same rows), not share bytes with them
  if (overlap(a.q_out, bytes[1], a.q, bytes[0]) && !(a.q_out == a.q && a.q_out_stride == a.q_stride)) return GLINATTN_ERR_INVALID_ARG;
  for (int i = 2; i < 4; ++i) {
    if (!overlap(a.q_out, bytes[1], rows[i], bytes[i])) continue;
    if (*strides[i] != a.q_out_stride) return GLINATTN_ERR_INVALID_ARG;
    const long long pitch = 2 * a.q_out_stride, off = (((intptr_t)rows[i] - (intptr_t)a.q_out) % pitch + pitch) % pitch;
    if (off < 2 * nq || off + 2 * nk > pitch) return GLINATTN_ERR_INVALID_ARG;
  }
  const unsigned grid = (unsigned)(((long long)a.num_tok + kWarps - 1) / kWarps);
  if (a.head_dim == 128) {
    if (a.cache_dtype == GLINATTN_E4M3) rope_kernel<128, true><<<grid, 32 * kWarps, 0, stream>>>(a);
    else rope_kernel<128, false><<<grid, 32 * kWarps, 0, stream>>>(a);
  } else {
    if (a.cache_dtype == GLINATTN_E4M3) rope_kernel<64, true><<<grid, 32 * kWarps, 0, stream>>>(a);
    else rope_kernel<64, false><<<grid, 32 * kWarps, 0, stream>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? GLINATTN_OK : GLINATTN_ERR_CUDA;
}

}  // namespace
}  // namespace paged
}  // namespace glinattn

extern "C" glinattn_status glinattn_kv_append_rope(const glinattn_kv_rope_args *args, glinattn_stream_t stream) {
  return glinattn::paged::run(args, (cudaStream_t)stream);
}
