// paged.cuh -- the paged key / value cache: what its kernels share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "glinattn.h"

namespace glinattn {
namespace paged {

// Request of packed row i: the last r with q_start[r] <= i, found by a whole
// warp 32 ways at a time (two rounds of loads for up to 1024 requests).  The
// caller checks that i really is in [q_start[r], q_start[r + 1]).
__device__ __forceinline__ int find_request(const int32_t *q_start, int R, int i, int lane) {
  int lo = 0, n = R;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int r = lo + lane * step;
    const bool le = lane == 0 || (lane * step < n && q_start[r] <= i);
    const unsigned b = __ballot_sync(0xffffffffu, le);
    const int k = 31 - __clz(b);
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// Whether request r's range and length are in bounds.
__device__ __forceinline__ bool request_ok(int s0, int s1, int len, int num_tok, long long max_len) {
  return s0 >= 0 && s0 <= s1 && s1 <= num_tok && len >= 0 && (long long)len <= max_len;
}

// 2^(code - 127) for a stored scale (code 0 is 2^-127, 255 NaN).
__device__ __forceinline__ float scale_value(uint32_t code) {
  return __uint_as_float(code == 0 ? 0x00400000u : code == 255 ? 0x7fffffffu : code << 23);
}

// Two e4m3 (low byte first) as floats.
__device__ __forceinline__ float2 e4m3x2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)two));
  float2 f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}" : "=f"(f.x), "=f"(f.y) : "r"(h));
  return f;
}

// Two floats as e4m3 (x in the low byte), rounded to nearest even; beyond 448
// (infinities) +-448, NaN stays NaN.
__device__ __forceinline__ uint32_t to_e4m3x2(float x, float y) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  return r;
}

// Host: the argument checks that the calls on the cache share.
glinattn_status check_cache(int cache_dtype, int num_req, int num_tok, int kv_heads, int head_dim, int page_size,
                            int num_pages, int max_pages, const void *k_cache, const void *v_cache, const void *k_scale,
                            const void *v_scale, const void *page_table, const void *kv_len, const void *q_start);

}  // namespace paged
}  // namespace glinattn
