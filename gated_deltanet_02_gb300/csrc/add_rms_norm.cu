// add_rms_norm.cu -- the residual's addition, the root-mean-square norm and its
// 8-bit output (glinattn_add_rms_norm).
//
// Mathematics: h = x + residual, y = h / sqrt(mean(h^2) + eps) * w.  A row is read
// once and kept in registers: a row's threads hold kChunks chunks of 8
// elements each, sum their squares, join the sums, and scale.  A scale's block of 32, 64 or 128
// elements is in 4, 8 or 16 neighbouring lanes.
//
// Bound: HBM bytes (x, residual in; residual, y out).  A CTA goes through many rows and has the next one
// on its way while it joins the sums of this one: 15,001 rows of 4,096 in bf16 to e4m3 with a scale a row
// take 71 us (6,050 GB/s), 2,049 rows of 8,192 with an fp32 residual in blocks of 32 34 us (5,500 GB/s; 16,392
// rows 225 us, 6,570 GB/s).  One CTA a row took 80 and 41 us; weights in registers for rows above 2,048
// elements 43 us (spilled).  Four rows of 2,048: 2.1 us.
#include "packed.cuh"

namespace glinattn {
namespace norm {
namespace {

using namespace packed;

struct Params {
  const void *x, *residual;
  const float *weight;
  void *residual_out, *y, *scale;
  long long rows, x_stride;
  int width, group;
  float eps;
};

constexpr float kMinScale = 7.888609052210118e-31f;  // 2^-100
// Squares of values up to 2^128 times this factor add up without an overflow.
constexpr float kShrink = 1.262177448353619e-29f;    // 2^-96
constexpr float kLargest = 3.4028234663852886e38f;   // finite fp32

template <bool kMax>
__device__ __forceinline__ float join(float a, float b) {
  return kMax ? __uint_as_float(max(__float_as_uint(a), __float_as_uint(b))) : a + b;
}

// The sum (or the maximum of non-negative bits) over a row's `threads` threads, for all of them.  Calls
// take turns with the halves of `shared`, so that one barrier each is enough: a half is written again
// behind the next call's barrier.
struct Shared {
  float half[2][32];
};
template <bool kMax>
__device__ __forceinline__ float over_row(float v, Shared &shared, int &turn, int threads) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = join<kMax>(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (threads == 32) return v;
  const int warps = threads >> 5;
  float *mine = shared.half[turn];
  turn ^= 1;
  if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = mine[0];
  for (int k = 1; k < warps; ++k) s = join<kMax>(s, mine[k]);
  return s;
}

// 1 / sqrt(mean + eps) as a product of two factors: `shrink`, which the values are
// multiplied with first, and the result.
__device__ __forceinline__ float inverse_root(float sum, int width, float eps) { return 1.0f / sqrtf(sum / (float)width + eps); }

// The scale of a maximum (its bits), what is stored and what values are multiplied with.
// `root`: what the values, and their maximum, still have to be multiplied with (fp32 scales), 1 or in
// [1, 2): so no factor here leaves fp32, 448 / top neither where top * root / 448 is above 2^-100.
template <bool kPow2>
__device__ __forceinline__ float scale_of(uint32_t amax, float root, void *scale, size_t at, bool store) {
  if (kPow2) {
    const uint32_t code = scale_code(amax);
    if (store) reinterpret_cast<uint8_t *>(scale)[at] = (uint8_t)code;
    return __uint_as_float((254u - code) << 23);
  }
  const float top = __uint_as_float(amax), s = fmaxf(top * root / 448.0f, kMinScale);
  if (store) reinterpret_cast<float *>(scale)[at] = s;
  return s > kMinScale ? 448.0f / top : root / kMinScale;
}

__device__ __forceinline__ float2 pair(const float *f, int i) { return make_float2(f[2 * i], f[2 * i + 1]); }
__device__ __forceinline__ void flat(const float2 *h, float *f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[2 * i] = h[i].x, f[2 * i + 1] = h[i].y;
}

// kOut: 0 fp32, 1 bf16, 2 e4m3 with fp32 scales, 3 e4m3 with powers of two.
// kRes: 0 none, 1 bf16, 2 fp32.  A CTA goes through every gridDim.x-th (group of) rows: its threads
// keep their weights, and the next row is on its way while this one's sums are formed.
template <bool kXBf16, int kRes, int kOut, int kChunks>
__global__ void __launch_bounds__(kChunks == 1 ? 128 : kChunks == 2 ? 256 : 512, kChunks == 1 ? 8 : kChunks == 2 ? 3 : 1) norm_rows_kernel(const Params p) {
  __shared__ Shared shared;
  const int threads = blockDim.x, chunks = p.width >> 3;
  int turn = 0;
  // A thread's weights: in registers, or where these would not be enough in shared memory
  constexpr bool kKept = kChunks < 4;
  extern __shared__ float4 weights[];
  float w[kKept ? kChunks : 1][8];
#pragma unroll
  for (int k = 0; k < kChunks; ++k) {
    const int c = k * threads + threadIdx.x;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 1.0f;
    if (p.weight && c < chunks) unpack8(load_raw8<false>(p.weight, 8 * c), v);
    if constexpr (kKept) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[k][i] = v[i];
    } else {  // its own, 16 bytes next to its neighbours'
      weights[2 * k * threads + threadIdx.x] = make_float4(v[0], v[1], v[2], v[3]);
      weights[(2 * k + 1) * threads + threadIdx.x] = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
  Raw8<kXBf16> rx[kChunks];
  Raw8<kRes == 1> rr[kChunks];
  auto read = [&](long long row) {
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      const int c = k * threads + threadIdx.x;
      rx[k] = {};
      rr[k] = {};
      if (row < p.rows && c < chunks) {
        rx[k] = load_raw8<kXBf16>(p.x, (size_t)row * p.x_stride + 8 * c);
        if (kRes) rr[k] = load_raw8<kRes == 1>(p.residual, (size_t)row * p.width + 8 * c);
      }
    }
  };
  const long long step = (long long)gridDim.x * blockDim.y;
  long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  read(row);
  // all threads of a CTA go on while its first row is there (of more than one row a CTA, 32 threads each)
  for (long long first = (long long)blockIdx.x * blockDim.y; first < p.rows; first += step, row += step) {
    const bool there = row < p.rows;
    float2 h[kChunks][4], squares = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      float x[8], r[8];
      unpack8(rx[k], x);
      if (kRes) unpack8(rr[k], r);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[k][i] = pair(x, i);
        if (kRes) h[k][i] = __fadd2_rn(h[k][i], pair(r, i));
        squares = __ffma2_rn(h[k][i], h[k][i], squares);
      }
    }
    read(row + step);
    float sum = over_row<false>(squares.x + squares.y, shared, turn, threads);
    if (kRes && there) {
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        const int c = k * threads + threadIdx.x;
        float o[8];
        flat(h[k], o);
        if (c < chunks) store8<kRes == 1>(p.residual_out, (size_t)row * p.width + 8 * c, o);
      }
    }
    float eps = p.eps;
    if (!(sum <= 3.0e38f)) {  // uniform over the row: an overflow, an infinity or a NaN
      squares = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < kChunks; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          h[k][i] = __fmul2_rn(h[k][i], make_float2(kShrink, kShrink));
          squares = __ffma2_rn(h[k][i], h[k][i], squares);
        }
      eps = 0.0f;                    // 2^-192 eps
      sum = over_row<false>(squares.x + squares.y, shared, turn, threads);
    }
    float inv = inverse_root(sum, p.width, eps);
    // With scales in fp32 y / scale is h w * 448 / max |h w|: the root enters the scale alone, and the
    // quotient has two roundings less.  Its power of two, an exact factor, stays with the values, so these are
    // within a factor of 2 of y: none leaves fp32 that y does not, whatever eps and the weights.  Rows with an
    // infinity or NaN get theirs from the root.
    float root = 1.0f;
    if (kOut == 2 && inv > 0.0f) {  // a normal number: in 2^-64 .. 2^34, of shrunken values in 2^-32 .. 2^48
      root = __uint_as_float((__float_as_uint(inv) & 0x007fffffu) | 0x3f800000u);
      inv = __uint_as_float(__float_as_uint(inv) & 0x7f800000u);
    }
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      float v[8];
      if constexpr (kKept) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = w[k][i];
      } else {
        const float4 lo = weights[2 * k * threads + threadIdx.x], hi = weights[(2 * k + 1) * threads + threadIdx.x];
        v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w, v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) h[k][i] = __fmul2_rn(__fmul2_rn(h[k][i], make_float2(inv, inv)), pair(v, i));
    }
    if constexpr (kOut < 2) {
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        const int c = k * threads + threadIdx.x;
        float o[8];
        flat(h[k], o);
        if (there && c < chunks) store8<kOut == 1>(p.y, (size_t)row * p.width + 8 * c, o);
      }
    } else {
      uint32_t top[kChunks];
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        float m = 0.0f;  // fmaxf leaves NaN out
#pragma unroll
        for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(h[k][i].x), fabsf(h[k][i].y)));
        top[k] = __float_as_uint(m);
        if (!(m * root <= kLargest)) {  // outputs that are infinite, or that the root would make so
          top[k] = 0;
          if (root != 1.0f)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 y = __fmul2_rn(h[k][i], make_float2(root, root));
              h[k][i] = make_float2(fabsf(y.x) <= kLargest ? h[k][i].x : y.x, fabsf(y.y) <= kLargest ? h[k][i].y : y.y);
            }
#pragma unroll
          for (int i = 0; i < 4; ++i) top[k] = max(top[k], max(finite_bits(h[k][i].x), finite_bits(h[k][i].y)));
        }
      }
      const int lanes = p.group >> 3, shift = 31 - __clz(lanes | 1);  // a power of two
      if (p.group) {
        for (int o = 1; o < lanes; o <<= 1)
#pragma unroll
          for (int k = 0; k < kChunks; ++k) top[k] = max(top[k], __shfl_xor_sync(0xffffffffu, top[k], o));
      } else {
#pragma unroll
        for (int k = 1; k < kChunks; ++k) top[0] = max(top[0], top[k]);
        top[0] = __float_as_uint(over_row<true>(__uint_as_float(top[0]), shared, turn, threads));
      }
      float f = 0.0f;
      if (!p.group) f = scale_of<kOut == 3>(top[0], root, p.scale, (size_t)row, there && threadIdx.x == 0);
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        const int c = k * threads + threadIdx.x;
        const bool in = there && c < chunks;
        if (p.group)
          f = scale_of<kOut == 3>(top[k], root, p.scale, (size_t)row * (chunks >> shift) + (c >> shift), in && (c & (lanes - 1)) == 0);
        float q[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = __fmul2_rn(h[k][i], make_float2(f, f));
          q[2 * i] = v.x, q[2 * i + 1] = v.y;
        }
        if (in) *reinterpret_cast<uint2 *>(reinterpret_cast<uint8_t *>(p.y) + (size_t)row * p.width + 8 * c) = to_e4m3x8(q);
      }
    }
  }
}

// Any width and alignment: one CTA a row, the row read again (from L2) for each of its
// passes; every element is read and written by one thread in the last of them.  Scalar loads bound it, two readings or, to
// e4m3, three: 15,001 rows of 4,095 in bf16 with a residual 194 us (2,540 GB/s, 79 with 4,096 in the kernel above), rows of 4,096 off
// by an element to e4m3 395, 2,048 rows of 32,768 301 us (1,780 GB/s), four rows of 2,047 4.4.
template <bool kXBf16, int kRes, int kOut>
__global__ void __launch_bounds__(512) norm_any_kernel(const Params p) {
  __shared__ Shared shared;
  int turn = 0;
  const long long row = blockIdx.x;
  const size_t x0 = (size_t)row * p.x_stride, y0 = (size_t)row * p.width;
  auto at = [&](int i) {
    float h = load_one<kXBf16>(p.x, x0 + i);
    if (kRes) h += load_one<kRes == 1>(p.residual, y0 + i);
    return h;
  };
  float sum = 0.0f, shrink = 1.0f, eps = p.eps;
  for (int i = threadIdx.x; i < p.width; i += blockDim.x) {
    const float h = at(i);
    sum = fmaf(h, h, sum);
  }
  sum = over_row<false>(sum, shared, turn, blockDim.x);
  if (!(sum <= 3.0e38f)) {
    shrink = kShrink, sum = 0.0f, eps = 0.0f;
    for (int i = threadIdx.x; i < p.width; i += blockDim.x) {
      const float h = at(i) * shrink;
      sum = fmaf(h, h, sum);
    }
    sum = over_row<false>(sum, shared, turn, blockDim.x);
  }
  const float inv = inverse_root(sum, p.width, eps);
  auto normed = [&](float h, int i) { return h * shrink * inv * (p.weight ? p.weight[i] : 1.0f); };
  if constexpr (kOut < 2) {
    for (int i = threadIdx.x; i < p.width; i += blockDim.x) {
      const float h = at(i);
      if (kRes) store_one<kRes == 1>(p.residual_out, y0 + i, h);
      store_one<kOut == 1>(p.y, y0 + i, normed(h, i));
    }
  } else {
    // a group's elements by one warp, a row's by all
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int group = p.group ? p.group : p.width, groups = p.width / group;
    const int first = p.group ? threadIdx.x >> 5 : 0, step = p.group ? warps : 1;
    const int begin = p.group ? lane : threadIdx.x, stride = p.group ? 32 : blockDim.x;
    for (int g = first; g < groups; g += step) {
      uint32_t top = 0;
      for (int i = begin; i < group; i += stride) top = max(top, finite_bits(normed(at(g * group + i), g * group + i)));
      if (p.group) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      } else {
        top = __float_as_uint(over_row<true>(__uint_as_float(top), shared, turn, blockDim.x));
      }
      const float f = scale_of<kOut == 3>(top, 1.0f, p.scale, (size_t)row * groups + g, begin == 0);
      for (int j = begin; j < group; j += stride) {
        const int i = g * group + j;
        const float h = at(i);
        if (kRes) store_one<kRes == 1>(p.residual_out, y0 + i, h);
        reinterpret_cast<uint8_t *>(p.y)[y0 + i] = (uint8_t)paged::to_e4m3x2(normed(h, i) * f, 0.0f);
      }
    }
  }
}

template <bool kXBf16, int kRes, int kOut>
void launch(const Params &p, bool vector, cudaStream_t s) {
  const int chunks = p.width >> 3;
  if (!vector || chunks > 2048) {
    norm_any_kernel<kXBf16, kRes, kOut><<<(unsigned)p.rows, 512, 0, s>>>(p);
    return;
  }
  // as many CTAs as the SMs hold, each of them with about the same number of rows
  auto grid = [&](int threads, int rows, int held) {  // threads that an SM holds
    const long long all = (p.rows + rows - 1) / rows, most = 152ll * (held / (threads * rows));
    const long long each = (all + most - 1) / most;
    return dim3((unsigned)((all + each - 1) / each));
  };
  auto up = [](int n) { int t = 32; while (t < n) t *= 2; return t; };
  if (chunks <= 32) {
    norm_rows_kernel<kXBf16, kRes, kOut, 1><<<grid(32, 4, 1024), dim3(32, 4), 0, s>>>(p);
  } else if (chunks <= 256) {
    const int t = up((chunks + 1) / 2);
    norm_rows_kernel<kXBf16, kRes, kOut, 2><<<grid(t, 1, 3 * 256), dim3(t, 1), 0, s>>>(p);
  } else {
    const int t = up((chunks + 3) / 4);
    cudaFuncSetAttribute(norm_rows_kernel<kXBf16, kRes, kOut, 4>, cudaFuncAttributeMaxDynamicSharedMemorySize, 512 * 128);
    norm_rows_kernel<kXBf16, kRes, kOut, 4><<<grid(t, 1, 512), dim3(t, 1), (size_t)t * 128, s>>>(p);
  }
}

template <bool kXBf16, int kRes>
void by_out(const Params &p, int out, bool vector, cudaStream_t s) {
  switch (out) {
    case 0: launch<kXBf16, kRes, 0>(p, vector, s); break;
    case 1: launch<kXBf16, kRes, 1>(p, vector, s); break;
    case 2: launch<kXBf16, kRes, 2>(p, vector, s); break;
    default: launch<kXBf16, kRes, 3>(p, vector, s); break;
  }
}

size_t size_of(int dtype) { return dtype == GLINATTN_F32 ? 4 : dtype == GLINATTN_BF16 ? 2 : 1; }

bool activation(int dtype) { return dtype == GLINATTN_F32 || dtype == GLINATTN_BF16; }

glinattn_status run(const glinattn_norm_args *a, cudaStream_t stream) {
  if (!a || !activation(a->in_dtype) || !(activation(a->out_dtype) || a->out_dtype == GLINATTN_E4M3) || a->rows < 0 ||
      a->width <= 0 || a->x_stride < 0 || !(a->eps >= 1e-20f && a->eps <= 1e20f))
    return GLINATTN_ERR_INVALID_ARG;
  const bool e4m3 = a->out_dtype == GLINATTN_E4M3;
  if (e4m3) {
    if ((a->scale_dtype != GLINATTN_F32 && a->scale_dtype != GLINATTN_E8M0) || a->group < 0) return GLINATTN_ERR_INVALID_ARG;
    if (a->group != 0 && a->group != 32 && a->group != 64 && a->group != 128) return GLINATTN_ERR_UNSUPPORTED;
    if (a->group && a->width % a->group) return GLINATTN_ERR_INVALID_ARG;
  } else if (a->group || a->scale) {
    return GLINATTN_ERR_INVALID_ARG;
  }
  if ((a->residual == nullptr) != (a->residual_out == nullptr)) return GLINATTN_ERR_INVALID_ARG;
  if (a->residual && !activation(a->residual_dtype)) return GLINATTN_ERR_INVALID_ARG;
  if (a->rows == 0) return GLINATTN_OK;
  const long long stride = a->x_stride ? a->x_stride : a->width;
  const size_t xs = size_of(a->in_dtype);
  if (stride < a->width && a->rows > 1) return GLINATTN_ERR_INVALID_ARG;
  if (!a->x || !a->y || (e4m3 && !a->scale) || !aligned(a->x, xs)) return GLINATTN_ERR_INVALID_ARG;
  const void *list[] = {a->residual, a->residual_out, a->weight, a->y, a->scale};
  for (const void *q : list)
    if (!aligned(q, 16)) return GLINATTN_ERR_INVALID_ARG;
  // outputs may be their inputs exactly, and otherwise overlap nothing
  const size_t nx = row_bytes(a->rows, a->width, stride, xs), elements = (size_t)a->rows * a->width;
  const size_t nr = a->residual ? elements * size_of(a->residual_dtype) : 0, ny = elements * size_of(a->out_dtype);
  const size_t ns = e4m3 ? (size_t)a->rows * (a->group ? a->width / a->group : 1) * (a->scale_dtype == GLINATTN_F32 ? 4 : 1) : 0;
  const size_t nw = a->weight ? (size_t)a->width * 4 : 0;
  const bool x_whole = stride == a->width || a->rows == 1;
  struct Out { const void *p; size_t n; int dtype; bool may_x, may_res; };
  const Out outs[] = {{a->residual_out, nr, a->residual_dtype, true, true}, {a->y, ny, a->out_dtype, true, false}, {a->scale, ns, -1, false, false}};
  for (int i = 0; i < 3; ++i) {
    const Out &o = outs[i];
    if (overlap(o.p, o.n, a->x, nx) && !(o.may_x && o.p == a->x && x_whole && o.dtype == a->in_dtype)) return GLINATTN_ERR_INVALID_ARG;
    if (overlap(o.p, o.n, a->residual, nr) && !(o.may_res && o.p == a->residual)) return GLINATTN_ERR_INVALID_ARG;
    if (overlap(o.p, o.n, a->weight, nw)) return GLINATTN_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(o.p, o.n, outs[j].p, outs[j].n)) return GLINATTN_ERR_INVALID_ARG;
  }
  const Params p = {a->x, a->residual, a->weight, a->residual_out, a->y, a->scale, a->rows, stride, a->width, a->group, a->eps};
  const bool vector = a->width % 8 == 0 && aligned(a->x, 16) && (a->rows == 1 || (stride * (long long)xs) % 16 == 0);
  const int out = e4m3 ? (a->scale_dtype == GLINATTN_F32 ? 2 : 3) : a->out_dtype == GLINATTN_F32 ? 0 : 1;
  const int res = !a->residual ? 0 : a->residual_dtype == GLINATTN_BF16 ? 1 : 2;
  if (a->in_dtype == GLINATTN_BF16) {
    if (res == 0) by_out<true, 0>(p, out, vector, stream);
    else if (res == 1) by_out<true, 1>(p, out, vector, stream);
    else by_out<true, 2>(p, out, vector, stream);
  } else {
    if (res == 0) by_out<false, 0>(p, out, vector, stream);
    else if (res == 1) by_out<false, 1>(p, out, vector, stream);
    else by_out<false, 2>(p, out, vector, stream);
  }
  return cudaGetLastError() == cudaSuccess ? GLINATTN_OK : GLINATTN_ERR_CUDA;
}

}  // namespace
}  // namespace norm
}  // namespace glinattn

extern "C" glinattn_status glinattn_add_rms_norm(const glinattn_norm_args *args, glinattn_stream_t stream) {
  return glinattn::norm::run(args, (cudaStream_t)stream);
}
