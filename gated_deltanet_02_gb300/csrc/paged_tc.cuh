// paged_tc.cuh -- device helpers of the two paged-attention kernels: the
// e4m3 tensor-core instruction, its operands' descriptors, and the split of a
// query row into e4m3 parts.
#pragma once

#include "paged.cuh"
#include "sm100.cuh"

namespace glinattn {
namespace paged {

using sm100::smem_u32;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// ---- tensor-core instructions, their operands' descriptors as two words --------
// One MMA lasts 32 .. 64 cycles, and one thread issues them all, so their
// descriptors must cost next to nothing: the high word (group stride, format
// version 1, swizzle) is a constant, and a step along K adds a constant to the
// low one (address, block stride; 16-byte units, no carry out of the address).
enum : uint32_t { kSwNone = 0, kSw128 = 2, kSw64 = 4 };
__host__ __device__ constexpr uint32_t desc_hi(uint32_t sbo, uint32_t swizzle) {
  return (sbo >> 4) | (1u << 14) | (swizzle << 29);
}
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return ((saddr >> 4) & 0x3FFFu) | (lbo >> 4) << 16; }

// D[tmem] (+)= A[smem] B[smem]: bf16 x bf16, or e4m3 x e4m3 (or e5m2, as the
// descriptor says), -> fp32.
template <bool kF8>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t alo, uint32_t ahi, uint32_t blo, uint32_t bhi, uint32_t idesc,
                                       uint32_t acc) {
  if constexpr (kF8)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %6, 0;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, p;\n\t}\n" ::"r"(d),
        "r"(alo), "r"(ahi), "r"(blo), "r"(bhi), "r"(idesc), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %6, 0;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}\n" ::"r"(d),
        "r"(alo), "r"(ahi), "r"(blo), "r"(bhi), "r"(idesc), "r"(acc)
        : "memory");
}
// D[tmem] (+)= A[tmem] B[smem], bf16.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t blo, uint32_t bhi, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}\n" ::"r"(d),
      "r"(a), "r"(blo), "r"(bhi), "r"(idesc), "r"(acc)
      : "memory");
}
// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}\n" : "=r"(e));
  return e != 0;
}
// Instruction descriptor for e4m3 operands (formats 0; B e5m2: 1), fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, bool a_mn, bool b_mn, bool b_e5m2 = false) {
  return (1u << 4) | ((b_e5m2 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

// 8 bf16 of a query row (kLanes lanes hold the row) as two e4m3 parts of 2^-e
// times the value, e bringing the row's largest element into [128, 256); returns
// 2^e.  bf16's 8 bits are 4 + 4, so the parts are exact but for elements below
// 2^-9 of the row's largest (1/4 here, whose last bit is the smallest e4m3), where a
// step is 2^-16 of it.  An infinite or NaN
// element becomes NaN.
template <int kLanes>
__device__ __forceinline__ float split_q(const uint4 &x, uint2 &hi, uint2 &lo) {
  const uint32_t u[4] = {x.x, x.y, x.z, x.w};
  float f[8], am = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = __uint_as_float(u[k] << 16);
    f[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (fabsf(f[k]) <= 3.4e38f) am = fmaxf(am, fabsf(f[k]));
    else f[k] = __int_as_float(0x7fffffff);
  }
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
  const int e = min(max((int)(__float_as_uint(am) >> 23) - 127 - 7, -100), 120);
  const float down = __uint_as_float((uint32_t)(127 - e) << 23);
  uint32_t h[4], l[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float a = f[2 * k] * down, b = f[2 * k + 1] * down;
    h[k] = to_e4m3x2(a, b);
    const float2 y = e4m3x2(h[k]);
    l[k] = to_e4m3x2(a - y.x, b - y.y);
  }
  hi = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
  lo = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
  return __uint_as_float((uint32_t)(127 + e) << 23);
}

// 128 columns of this thread's lane, one wait.
__device__ __forceinline__ void tmem_ld128(uint32_t a, float (&v)[128]) {
  uint32_t r[128];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%128];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%129];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, "
      "%80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95}, [%130];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%96, %97, %98, %99, %100, %101, %102, %103, %104, %105, %106, %107, %108, %109, %110, %111, "
      "%112, %113, %114, %115, %116, %117, %118, %119, %120, %121, %122, %123, %124, %125, %126, %127}, [%131];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63]),
        "=r"(r[64]), "=r"(r[65]), "=r"(r[66]), "=r"(r[67]), "=r"(r[68]), "=r"(r[69]), "=r"(r[70]), "=r"(r[71]),
        "=r"(r[72]), "=r"(r[73]), "=r"(r[74]), "=r"(r[75]), "=r"(r[76]), "=r"(r[77]), "=r"(r[78]), "=r"(r[79]),
        "=r"(r[80]), "=r"(r[81]), "=r"(r[82]), "=r"(r[83]), "=r"(r[84]), "=r"(r[85]), "=r"(r[86]), "=r"(r[87]),
        "=r"(r[88]), "=r"(r[89]), "=r"(r[90]), "=r"(r[91]), "=r"(r[92]), "=r"(r[93]), "=r"(r[94]), "=r"(r[95]),
        "=r"(r[96]), "=r"(r[97]), "=r"(r[98]), "=r"(r[99]), "=r"(r[100]), "=r"(r[101]), "=r"(r[102]), "=r"(r[103]),
        "=r"(r[104]), "=r"(r[105]), "=r"(r[106]), "=r"(r[107]), "=r"(r[108]), "=r"(r[109]), "=r"(r[110]), "=r"(r[111]),
        "=r"(r[112]), "=r"(r[113]), "=r"(r[114]), "=r"(r[115]), "=r"(r[116]), "=r"(r[117]), "=r"(r[118]), "=r"(r[119]),
        "=r"(r[120]), "=r"(r[121]), "=r"(r[122]), "=r"(r[123]), "=r"(r[124]), "=r"(r[125]), "=r"(r[126]), "=r"(r[127])
      : "r"(a), "r"(a + 32), "r"(a + 64), "r"(a + 96)
      : "memory");
#pragma unroll
  for (int k = 0; k < 128; ++k) v[k] = __uint_as_float(r[k]);
}

// After a wait that gave up, before a CTA leaves its shared memory and TMEM: time
// (1 ms) for the copies and products that it still has in flight.
__device__ __forceinline__ void let_copies_land() {
  const uint64_t t0 = sm100::global_timer_ns();
  while (sm100::global_timer_ns() - t0 < 1000000ull) __nanosleep(1000);
}

// Host: a tiled map of a contiguous array [dims[2], dims[1], dims[0]] of elements
// of elem_bytes, false when it is refused.
bool encode_map(CUtensorMap *m, const void *base, CUtensorMapDataType type, int elem_bytes, const long long dims[3],
                const int box[3], CUtensorMapSwizzle swizzle);

}  // namespace paged
}  // namespace glinattn
