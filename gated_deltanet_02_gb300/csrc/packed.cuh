// packed.cuh -- packed token rows, states by slot and element access: what the
// calls around the sequence mixers share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "glinattn.h"
#include "paged.cuh"

namespace glinattn {
namespace packed {

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Element i of an activation array.
template <bool kBf16>
__device__ __forceinline__ float load_one(const void *p, size_t i) {
  if (kBf16) return __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(p)[i] << 16);
  return reinterpret_cast<const float *>(p)[i];
}
template <bool kBf16>
__device__ __forceinline__ void store_one(void *p, size_t i, float v) {
  if (kBf16)
    reinterpret_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
  else
    reinterpret_cast<float *>(p)[i] = v;
}

// Eight elements from element i on, whose address is 16-byte aligned.
template <bool kBf16>
struct Raw8 {
  uint4 w[kBf16 ? 1 : 2];
};
template <bool kBf16>
__device__ __forceinline__ Raw8<kBf16> load_raw8(const void *p, size_t i) {
  Raw8<kBf16> r;
  const uint4 *q = reinterpret_cast<const uint4 *>(reinterpret_cast<const uint8_t *>(p) + i * (kBf16 ? 2 : 4));
#pragma unroll
  for (int k = 0; k < (kBf16 ? 1 : 2); ++k) r.w[k] = q[k];
  return r;
}
__device__ __forceinline__ void store_raw8(void *p, size_t i, const Raw8<true> &r) {
  *reinterpret_cast<uint4 *>(reinterpret_cast<uint8_t *>(p) + i * 2) = r.w[0];
}
template <bool kBf16>
__device__ __forceinline__ void unpack8(const Raw8<kBf16> &r, float *f) {
  if constexpr (kBf16) {
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) f[2 * k] = bf16_lo(w[k]), f[2 * k + 1] = bf16_hi(w[k]);
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      f[4 * k] = __uint_as_float(r.w[k].x), f[4 * k + 1] = __uint_as_float(r.w[k].y);
      f[4 * k + 2] = __uint_as_float(r.w[k].z), f[4 * k + 3] = __uint_as_float(r.w[k].w);
    }
  }
}
template <bool kBf16>
__device__ __forceinline__ void store8(void *p, size_t i, const float *f) {
  uint4 *q = reinterpret_cast<uint4 *>(reinterpret_cast<uint8_t *>(p) + i * (kBf16 ? 2 : 4));
  if constexpr (kBf16) {
    q[0] = make_uint4(paged::pack_bf16(f[0], f[1]), paged::pack_bf16(f[2], f[3]), paged::pack_bf16(f[4], f[5]),
                      paged::pack_bf16(f[6], f[7]));
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      q[k] = make_uint4(__float_as_uint(f[4 * k]), __float_as_uint(f[4 * k + 1]), __float_as_uint(f[4 * k + 2]),
                        __float_as_uint(f[4 * k + 3]));
  }
}

// Code (exponent plus 127) of the smallest 2^e with e in [-100, 119] and
// amax <= 448 * 2^e, from the bits of amax = 1.m * 2^(E - 127): 448 = 1.75 * 2^8,
// so e + 127 = E - 8, one more where m is above 0x600000 (the addition carries into E).
__device__ __forceinline__ uint32_t scale_code(uint32_t amax) {
  return (uint32_t)min(max((int)((amax + 0x1fffffu) >> 23) - 8, 27), 246);
}
// The bits of |x|, 0 where x is not finite: such bits compare like the numbers.
__device__ __forceinline__ uint32_t finite_bits(float x) {
  const uint32_t a = __float_as_uint(x) & 0x7fffffffu;
  return a < 0x7f800000u ? a : 0u;
}
__device__ __forceinline__ uint2 to_e4m3x8(const float *f) {
  uint32_t q[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) q[k] = paged::to_e4m3x2(f[2 * k], f[2 * k + 1]);
  return make_uint2(__byte_perm(q[0], q[1], 0x5410), __byte_perm(q[2], q[3], 0x5410));
}

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// z / (1 + e^-z), the exponential and the reciprocal within 2^-22 (and |z| 2^-23) of themselves; 0 below z = -87.3, where
// the reciprocal is subnormal (the result is above -10^-36 there).
__device__ __forceinline__ float silu(float z) { return z * rcp_fast(1.0f + exp2_fast(-z * kLog2e)); }
__device__ __forceinline__ float2 silu2(float2 z) {
  const float2 e = __fmul2_rn(z, make_float2(-kLog2e, -kLog2e));
  const float2 w = __fadd2_rn(make_float2(exp2_fast(e.x), exp2_fast(e.y)), make_float2(1.0f, 1.0f));
  return __fmul2_rn(z, make_float2(rcp_fast(w.x), rcp_fast(w.y)));
}

// The packed rows and slots of a call (the members that the argument structs share).
struct Rows {
  int R, num_tok, pool_slots, max_len;  // max_len: no request is longer, else it is skipped
  bool has_pool;
  const int32_t *q_start, *slot_ids, *resume, *count;
  uint32_t *dev_status;
};

// One request: its range, the rows of it that are run, its slot and whether it resumes.
struct Request {
  int s0, s1, run, slot;
  bool ok, resumed;
};

// All lanes of a warp may call it with the same r in [0, R).
__device__ __forceinline__ Request request(const Rows &p, int r) {
  Request q;
  q.s0 = p.q_start ? p.q_start[r] : r;
  q.s1 = p.q_start ? p.q_start[r + 1] : r + 1;
  q.run = p.count ? p.count[r] : q.s1 - q.s0;
  q.slot = p.has_pool ? p.slot_ids[r] : 0;
  q.resumed = p.has_pool && (!p.resume || p.resume[r] != 0);
  q.ok = q.s0 >= 0 && q.s0 <= q.s1 && q.s1 <= p.num_tok && q.s1 - q.s0 <= p.max_len && q.run >= 0 &&
         q.run <= q.s1 - q.s0 && (!p.has_pool || (q.slot >= 0 && q.slot < p.pool_slots));
  return q;
}

// The error bits of all requests, request by request; called by every thread of a grid.
__device__ __forceinline__ void check_requests(const Rows &p, long long thread, long long threads) {
  if (!p.dev_status) return;
  for (long long r = thread; r < p.R; r += threads) {
    const Request q = request(p, (int)r);
    if (q.ok) continue;
    const bool range = q.s0 >= 0 && q.s0 <= q.s1 && q.s1 <= p.num_tok && q.s1 - q.s0 <= p.max_len && q.run >= 0 &&
                       q.run <= q.s1 - q.s0;
    const bool slot = !p.has_pool || (q.slot >= 0 && q.slot < p.pool_slots);
    atomicOr(p.dev_status, (range ? 0u : GLINATTN_DEV_BAD_COUNT) | (slot ? 0u : GLINATTN_DEV_BAD_SLOT));
  }
}

// Host: bytes from the first to behind the last element of rows `stride` apart.
inline size_t row_bytes(long long rows, long long width, long long stride, size_t size) {
  return rows > 0 ? ((size_t)(rows - 1) * (size_t)stride + (size_t)width) * size : 0;
}
inline bool overlap(const void *a, size_t na, const void *b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a && b && na && nb && x < y + nb && y < x + na;
}
inline bool aligned(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

}  // namespace packed
}  // namespace glinattn
