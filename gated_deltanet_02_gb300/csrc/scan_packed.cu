// scan_packed.cu -- the selective scan over packed rows with its step bias, skip
// and gate, the states in a slot-indexed pool (glinattn_selective_scan_packed).
//
// Mathematics, per channel d and state index n, dt = softplus(delta + bias):
//   h_t = exp(dt A) h_{t-1} + dt B_t x_t,   y_t = (sum_n h_t C_t + skip x_t) silu(z_t).
//
// Every (d, n) is a recurrence of its own whose only serial step is one fused
// multiply-add a row; the exponential, the products and the sum over n of any row
// do not wait for the row before.  So the rows of a request are run in order, once,
// with one exponential per element, and what fills the SMs is that a warp always has
// the work of several rows in flight.
//
// scan_kernel: a CTA owns 32 channels of a request and has two kinds of warps.  The scan
// warps keep kK states of a channel in each thread and go through tiles of 32 rows that lie
// ready in shared memory: the steps (dt, dt x), B and C.  A thread forms the decays and terms of
// the next four rows while it runs the recurrence of these four, so that a warp alone
// keeps its scheduler busy.  The helper warps turn the inputs of the tile after next into
// steps, and the last tile's partial sums into outputs (sum over the channel's threads,
// skip, gate).  One barrier a tile.
//
// few_kernel (single tokens, drafts): a thread owns four states of a channel for
// kReqs requests, all of whose loads are in flight together.
//
// Bound: scan_kernel by instruction issue (per element an exponential and packed fp32
// instructions of a half each for its argument, dt x B, h and y, beside loads of B and C and the
// helpers' share), few_kernel by HBM bytes, the states in and out.
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
  int D, update, out_bf16, bc_vector;
};

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

// log(1 + e^x) = max(x, 0) + log(1 + e), e = e^-|x| in (0, 1]; log(1 + e) = e P(e), P of degree 8
// fitted to log(1 + e) / e on [0, 1] with a relative error of 3e-8, so a small result keeps its
// relative error.  Two at a time.
__device__ __forceinline__ float2 softplus2(float2 x) {
  const float2 e = make_float2(exp2_fast(-fabsf(x.x) * kLog2e), exp2_fast(-fabsf(x.y) * kLog2e));
  constexpr float c[9] = {0.9999999403953552f, -0.4999949336051941f, 0.3331909775733948f, -0.2484298199415207f, 0.19106005132198334f,
                          -0.13663242757320404f, 0.07822591066360474f, -0.029505213722586632f, 0.0052326880395412445f};
  float2 r = make_float2(c[8], c[8]);
#pragma unroll
  for (int i = 7; i >= 0; --i) r = __ffma2_rn(r, e, make_float2(c[i], c[i]));
  return __ffma2_rn(r, e, make_float2(fmaxf(x.x, 0.0f), fmaxf(x.y, 0.0f)));
}
__device__ __forceinline__ float softplus(float x) { return softplus2(make_float2(x, x)).x; }
__device__ __forceinline__ float silu(float z) { return z * rcp_fast(1.0f + exp2_fast(-z * kLog2e)); }

// ---------------------------------------------------------------------------
// many rows
// ---------------------------------------------------------------------------

constexpr int kCh = 32, kL = 32;            // channels of a CTA, rows of a tile
constexpr int kHelpers = kL * (kCh / 8);    // helper threads: one for 8 channels of one row

template <int N, int kK, int kC>
struct Tile {
  static constexpr int kG = N / kK;              // threads of a channel
  static constexpr int kScan = kCh / kC * kG;    // scan threads
  static constexpr int kPlane = kL * kCh + 4;    // partial sums of one of a channel's threads (4: other banks)
  float step[3][kL][2 * kCh];                    // (dt, dt x) of the channels, permuted: step_at
  float b[3][kL][N], c[3][kL][N];
  float part[2][kG][kPlane];                     // the channels permuted: part_at
  float bias[kCh], skip[kCh];
};

// The permutations keep the banks of 8 neighbouring lanes apart on both sides.  Where the step of
// channel 8 u + c of row t is: helper threads (four u, two rows) write one 16-byte pair of channels each.
__device__ __forceinline__ int step_at(int t, int u, int c) { return 4 * (4 * u + ((c >> 1) ^ ((u >> 1) + 2 * (t & 1)))) + 2 * (c & 1); }
// Where the partial sum of channel 8 u + c of row t is: helper threads read 16 bytes each.
__device__ __forceinline__ int part_at(int t, int u, int c) { return t * kCh + 4 * ((u + (c & 4)) ^ (4 * (t & 1))) + (c & 3); }

// Eight elements of a row as they are in memory; those outside [0, left) are zeros.
template <bool kBf16>
__device__ __forceinline__ Raw8<kBf16> load_unit(const void *p, size_t at, int left, bool vector) {
  if (vector) return load_raw8<kBf16>(p, at);
  uint32_t w[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    w[k] = 0;
    if (k < left) w[k] = kBf16 ? reinterpret_cast<const uint16_t *>(p)[at + k] : reinterpret_cast<const uint32_t *>(p)[at + k];
  }
  Raw8<kBf16> r;
  if constexpr (kBf16) {
    r.w[0] = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
  } else {
    r.w[0] = make_uint4(w[0], w[1], w[2], w[3]);
    r.w[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
  return r;
}

// kK floats of B or C.
template <int kK>
__device__ __forceinline__ void load_states(const float *p, float *f) {
  if constexpr (kK == 2) {
    const float2 v = *reinterpret_cast<const float2 *>(p);
    f[0] = v.x, f[1] = v.y;
  } else {
#pragma unroll
    for (int k = 0; k < kK / 4; ++k) {
      const float4 v = reinterpret_cast<const float4 *>(p)[k];
      f[4 * k] = v.x, f[4 * k + 1] = v.y, f[4 * k + 2] = v.z, f[4 * k + 3] = v.w;
    }
  }
}

template <bool kBf16, int N, int kK, int kC, bool kVec>
__global__ void __launch_bounds__(kCh / kC *(N / kK) + kHelpers, kC == 1 ? 2 : 3) scan_kernel(const Params p) {
  using T = Tile<N, kK, kC>;
  extern __shared__ __align__(16) uint8_t smem[];
  T &s = *reinterpret_cast<T *>(smem);
  if (blockIdx.x == 0 && blockIdx.y == 0) check_requests(p.rows, threadIdx.x, blockDim.x);
  const Request q = request(p.rows, blockIdx.y);
  if (!q.ok || q.run == 0) return;
  const int d0 = blockIdx.x * kCh, tiles = (q.run + kL - 1) / kL;
  if (threadIdx.x < T::kScan) {
    // --- scan warps: thread g of channels ch .. ch + kC - 1 has their states g kK .. g kK + kK - 1.
    // Lanes 2 i and 2 i + 1 have the same g, lanes i and i ^ 2 the same channels: loads of shared
    // memory in which such lanes read the same 16 (or 8) bytes take half the cycles.
    constexpr int kLogG = T::kG == 2 ? 1 : T::kG == 4 ? 2 : 3;
    const int lane = threadIdx.x & 31, g = (lane >> 1) & (T::kG - 1);
    const int ch = kC * ((threadIdx.x >> 5) * (32 / T::kG) + (lane & 1) + 2 * (lane >> (1 + kLogG))), d = d0 + ch;
    float2 A[kC][kK / 2], h[kC][kK / 2];
    float *state = p.pool + ((size_t)q.slot * p.D + d) * N + g * kK;
#pragma unroll
    for (int i = 0; i < kC; ++i)
#pragma unroll
      for (int k = 0; k < kK / 2; ++k) {
        const bool in = d + i < p.D;
        const float2 a = in ? reinterpret_cast<const float2 *>(p.A + (size_t)(d + i) * N + g * kK)[k] : make_float2(0.0f, 0.0f);
        A[i][k] = make_float2(a.x * kLog2e, a.y * kLog2e);
        h[i][k] = in && q.resumed ? reinterpret_cast<const float2 *>(state + i * N)[k] : make_float2(0.0f, 0.0f);
      }
    const int steps[2] = {step_at(0, ch >> 3, ch & 7), step_at(1, ch >> 3, ch & 7)};
    const int parts[2] = {part_at(0, ch >> 3, ch & 7), part_at(1, ch >> 3, ch & 7) - kCh};
    // A block of kRows rows: what is read for it, and its decays and terms.  While one block's recurrence
    // runs, the next one's decays are formed and the one's after that is read: nothing waits
    // for a load, and the exponentials lie between the multiply-adds.
    constexpr int kRows = 2, kBlocks = kL / kRows;
    struct Lines {
      float st[kRows][2 * kC], b[kRows][kK];
    };
    struct Block {
      float2 a[kRows][kC][kK / 2], b[kRows][kC][kK / 2];
    };
    struct Outs {
      float c[kRows][kK];
    };
    auto fetch = [&](Lines &l, int slot, int t0) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        load_states<2 * kC>(&s.step[slot][t0 + r][steps[(t0 + r) & 1]], l.st[r]);
        load_states<kK>(&s.b[slot][t0 + r][g * kK], l.b[r]);
      }
    };
    auto fetch_c = [&](Outs &o, int slot, int t0) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) load_states<kK>(&s.c[slot][t0 + r][g * kK], o.c[r]);
    };
    auto form = [&](Block &w, const Lines &l, int r) {
#pragma unroll
      for (int i = 0; i < kC; ++i)
#pragma unroll
        for (int k = 0; k < kK / 2; ++k) {
          const float2 e = __fmul2_rn(A[i][k], make_float2(l.st[r][2 * i], l.st[r][2 * i]));
          w.a[r][i][k] = make_float2(exp2_fast(e.x), exp2_fast(e.y));
          w.b[r][i][k] = __fmul2_rn(make_float2(l.st[r][2 * i + 1], l.st[r][2 * i + 1]), make_float2(l.b[r][2 * k], l.b[r][2 * k + 1]));
        }
    };
    auto run = [&](const Block &w, const Outs &o, int r, float *y) {
#pragma unroll
      for (int i = 0; i < kC; ++i) {
        float2 sum;
#pragma unroll
        for (int k = 0; k < kK / 2; ++k) {
          h[i][k] = __ffma2_rn(w.a[r][i][k], h[i][k], w.b[r][i][k]);
          const float2 c2 = make_float2(o.c[r][2 * k], o.c[r][2 * k + 1]);
          sum = k ? __ffma2_rn(h[i][k], c2, sum) : __fmul2_rn(h[i][k], c2);
        }
        y[i] = sum.x + sum.y;
      }
    };
    __syncthreads();
    Block w[2];
    Lines l[2];
    Outs o[2];
    fetch(l[0], 0, 0);
    fetch(l[1], 0, kRows);
    fetch_c(o[0], 0, 0);
#pragma unroll
    for (int r = 0; r < kRows; ++r) form(w[0], l[0], r);
    int slot = 0;
    for (int i = 0; i < tiles; ++i) {
      const int next = slot == 2 ? 0 : slot + 1;
      float *part = &s.part[i & 1][g][0];
#pragma unroll
      for (int m = 0; m < kBlocks; ++m) {
        // behind the last tile lies an old one or nothing: read and formed, not used
        fetch(l[m & 1], m + 2 < kBlocks ? slot : next, kRows * ((m + 2) % kBlocks));
        fetch_c(o[(m + 1) & 1], m + 1 < kBlocks ? slot : next, kRows * ((m + 1) % kBlocks));
        float y[kRows][kC];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          run(w[m & 1], o[m & 1], r, y[r]);
          form(w[(m + 1) & 1], l[(m + 1) & 1], r);
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          float *to = part + (kRows * m + r) * kCh + parts[(kRows * m + r) & 1];
          if constexpr (kC == 1) to[0] = y[r][0];
          else *reinterpret_cast<float2 *>(to) = make_float2(y[r][0], y[r][1]);
        }
      }
      slot = next;
      __syncthreads();
    }
    if (p.update)
#pragma unroll
      for (int i = 0; i < kC; ++i)
#pragma unroll
        for (int k = 0; k < kK / 2; ++k)
          if (d + i < p.D) reinterpret_cast<float2 *>(state + i * N)[k] = h[i][k];
    return;
  }
  // --- helper warps: thread (t, u) has row t, channels 8 u .. 8 u + 7 of every tile
  const int j = threadIdx.x - T::kScan, u = j & 3, t = j >> 2, d = d0 + 8 * u, left = min(8, p.D - d);
  const bool in = left > 0;
  if (j < kCh) {
    s.bias[j] = d0 + j < p.D && p.delta_bias ? p.delta_bias[d0 + j] : 0.0f;
    s.skip[j] = d0 + j < p.D && p.skip ? p.skip[d0 + j] : 0.0f;
  }
  constexpr int kUnits = 2 * kL * N / 8, kBc = (kUnits + kHelpers - 1) / kHelpers;  // units of 8 elements of B and C: all, of a thread
  Raw8<kBf16> x, delta, z, bc[kBc];  // of the next tile
  const bool gate = p.z && p.y;
  auto load = [&](int i) {
    const int row = i * kL + t;
    const size_t r = (size_t)q.s0 + row;
    if (in && row < q.run) {
      x = load_unit<kBf16>(p.x, r * p.x_stride + d, left, kVec);
      delta = load_unit<kBf16>(p.delta, r * p.delta_stride + d, left, kVec);
      if (gate) z = load_unit<kBf16>(p.z, r * p.z_stride + d, left, kVec);
    } else {  // a step of softplus(-infinity) = 0, no term
      const uint32_t inf = kBf16 ? 0xff80ff80u : 0xff800000u;
      x = {};
#pragma unroll
      for (int k = 0; k < (kBf16 ? 1 : 2); ++k) delta.w[k] = make_uint4(inf, inf, inf, inf);
    }
#pragma unroll
    for (int m = 0; m < kBc; ++m) {
      const int e = j + m * kHelpers, line = e / (N / 8), rr = i * kL + (line >> 1), n = (e % (N / 8)) * 8;
      const bool c = line & 1;
      bc[m] = {};
      if ((kUnits % kHelpers && e >= kUnits) || rr >= q.run || (c && !p.y)) continue;
      bc[m] = load_unit<kBf16>(c ? p.Cm : p.Bm, ((size_t)q.s0 + rr) * (c ? p.c_stride : p.b_stride) + n, 8, p.bc_vector);
    }
  };
  auto produce = [&](int slot) {
    float *to = &s.step[slot][t][0];
    float xs[8], ds[8], bias[8];
    unpack8(x, xs);
    unpack8(delta, ds);
    load_states<8>(&s.bias[8 * u], bias);
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      const float2 dt = softplus2(make_float2(ds[k] + bias[k], ds[k + 1] + bias[k + 1]));
      const float2 dtx = __fmul2_rn(dt, make_float2(xs[k], xs[k + 1]));
      *reinterpret_cast<float4 *>(to + step_at(t, u, k)) = make_float4(dt.x, dtx.x, dt.y, dtx.y);
    }
#pragma unroll
    for (int m = 0; m < kBc; ++m) {
      const int e = j + m * kHelpers, line = e / (N / 8), n = (e % (N / 8)) * 8;
      if (kUnits % kHelpers && e >= kUnits) continue;
      float f[8];
      unpack8(bc[m], f);
      float4 *to_bc = reinterpret_cast<float4 *>(line & 1 ? &s.c[slot][line >> 1][n] : &s.b[slot][line >> 1][n]);
      to_bc[0] = make_float4(f[0], f[1], f[2], f[3]);
      to_bc[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
  };
  auto finish = [&](int i, const Raw8<kBf16> &rx, const Raw8<kBf16> &rz) {
    const int row = i * kL + t;
    if (!p.y || !in || row >= q.run) return;
    float f[8], skip[8];
    float2 y[4];
    unpack8(rx, f);
    load_states<8>(&s.skip[8 * u], skip);
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = __fmul2_rn(make_float2(skip[2 * k], skip[2 * k + 1]), make_float2(f[2 * k], f[2 * k + 1]));
#pragma unroll
    for (int g = 0; g < T::kG; ++g) {
      float part[8];
      load_states<4>(&s.part[i & 1][g][part_at(t, u, 0)], part);
      load_states<4>(&s.part[i & 1][g][part_at(t, u, 4)], part + 4);
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] = __fadd2_rn(y[k], make_float2(part[2 * k], part[2 * k + 1]));
    }
    if (gate) {
      unpack8(rz, f);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 z = make_float2(f[2 * k], f[2 * k + 1]), e = __fmul2_rn(z, make_float2(-kLog2e, -kLog2e));
        const float2 w = __fadd2_rn(make_float2(exp2_fast(e.x), exp2_fast(e.y)), make_float2(1.0f, 1.0f));
        y[k] = __fmul2_rn(y[k], __fmul2_rn(z, make_float2(rcp_fast(w.x), rcp_fast(w.y))));
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) f[2 * k] = y[k].x, f[2 * k + 1] = y[k].y;
    const size_t at = ((size_t)q.s0 + row) * p.D + d;
    if (kVec) {
      if (p.out_bf16) store8<true>(p.y, at, f);
      else store8<false>(p.y, at, f);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < left) {
          if (p.out_bf16) store_one<true>(p.y, at + k, f[k]);
          else store_one<false>(p.y, at + k, f[k]);
        }
    }
  };
  // x and z of the last tile, of the one that is being scanned and of the next
  Raw8<kBf16> x0, z0, x1, z1, x2, z2;
  load(0);
  asm volatile("bar.sync 1, %0;" ::"n"(kHelpers) : "memory");  // bias and skip are there, for the helpers
  produce(0);
  x1 = x, z1 = z;
  load(1);
  produce(1);
  x2 = x, z2 = z;
  load(2);
  __syncthreads();
  int slot = 2;
  for (int i = 0; i < tiles; ++i) {
    if (i > 0) finish(i - 1, x0, z0);
    x0 = x1, z0 = z1, x1 = x2, z1 = z2, x2 = x, z2 = z;
    if (i + 2 < tiles) {
      produce(slot);
      load(i + 3);
    }
    slot = slot == 2 ? 0 : slot + 1;
    __syncthreads();
  }
  finish(tiles - 1, x0, z0);
}

// ---------------------------------------------------------------------------
// few rows
// ---------------------------------------------------------------------------

constexpr int kFewThreads = 256, kFewRows = 16;  // requests of more rows take the other kernel

template <bool kBf16>
__device__ __forceinline__ float4 load4(const void *p, size_t at, bool vector) {
  if (!vector) return make_float4(load_one<kBf16>(p, at), load_one<kBf16>(p, at + 1), load_one<kBf16>(p, at + 2), load_one<kBf16>(p, at + 3));
  if constexpr (kBf16) {
    const uint2 w = *reinterpret_cast<const uint2 *>(reinterpret_cast<const uint16_t *>(p) + at);
    return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
  } else {
    return *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(p) + at);
  }
}

template <bool kBf16, int N, int kReqs>
__global__ void __launch_bounds__(kFewThreads) few_kernel(const Params p) {
  constexpr int kQ = N / 4;  // threads of a channel, four states each
  if (blockIdx.x == 0) check_requests(p.rows, (long long)blockIdx.y * kFewThreads + threadIdx.x, (long long)gridDim.y * kFewThreads);
  const int g = threadIdx.x % kQ, d = blockIdx.x * (kFewThreads / kQ) + threadIdx.x / kQ;
  const bool in = d < p.D;
  const int dd = in ? d : 0;
  const float4 a4 = reinterpret_cast<const float4 *>(p.A + (size_t)dd * N)[g];
  const float A[4] = {a4.x * kLog2e, a4.y * kLog2e, a4.z * kLog2e, a4.w * kLog2e};
  const float bias = p.delta_bias ? p.delta_bias[dd] : 0.0f, skip = p.skip ? p.skip[dd] : 0.0f;
  Request q[kReqs];
  float4 h4[kReqs];
  struct Row {
    float x, delta, z;
    float4 b, c;
  };
  auto row = [&](size_t r) {
    Row v;
    v.x = load_one<kBf16>(p.x, r * p.x_stride + dd);
    v.delta = load_one<kBf16>(p.delta, r * p.delta_stride + dd);
    v.z = p.z && p.y ? load_one<kBf16>(p.z, r * p.z_stride + dd) : 0.0f;
    v.b = load4<kBf16>(p.Bm, r * p.b_stride + 4 * g, p.bc_vector);
    v.c = p.y ? load4<kBf16>(p.Cm, r * p.c_stride + 4 * g, p.bc_vector) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    return v;
  };
  Row first[kReqs];
#pragma unroll
  for (int i = 0; i < kReqs; ++i) {
    const int r = blockIdx.y * kReqs + i;
    if (r < p.rows.R) q[i] = request(p.rows, r);
    else q[i].ok = false;
    if (!q[i].ok) q[i].run = 0, q[i].slot = 0, q[i].resumed = false;
  }
#pragma unroll
  for (int i = 0; i < kReqs; ++i) {
    h4[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (q[i].run == 0) continue;  // whole CTAs
    if (q[i].resumed && in) h4[i] = reinterpret_cast<const float4 *>(p.pool + ((size_t)q[i].slot * p.D + d) * N)[g];
    first[i] = row((size_t)q[i].s0);
  }
#pragma unroll
  for (int i = 0; i < kReqs; ++i) {
    if (q[i].run == 0) continue;
    float h[4] = {h4[i].x, h4[i].y, h4[i].z, h4[i].w};
    Row v = first[i];
    for (int t = 0; t < q[i].run; ++t) {
      const Row now = v;
      if (t + 1 < q[i].run) v = row((size_t)q[i].s0 + t + 1);
      const float dt = softplus(now.delta + bias), dtx = dt * now.x;
      const float b[4] = {now.b.x, now.b.y, now.b.z, now.b.w}, c[4] = {now.c.x, now.c.y, now.c.z, now.c.w};
      float y = 0.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        h[k] = fmaf(exp2_fast(dt * A[k]), h[k], dtx * b[k]);
        y = fmaf(h[k], c[k], y);
      }
      if (!p.y) continue;
#pragma unroll
      for (int o = kQ / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
      if (!in || g != 0) continue;
      y = fmaf(skip, now.x, y);
      if (p.z) y *= silu(now.z);
      const size_t at = ((size_t)q[i].s0 + t) * p.D + d;
      if (p.out_bf16) store_one<true>(p.y, at, y);
      else store_one<false>(p.y, at, y);
    }
    if (p.update && in)
      reinterpret_cast<float4 *>(p.pool + ((size_t)q[i].slot * p.D + d) * N)[g] = make_float4(h[0], h[1], h[2], h[3]);
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

template <bool kBf16, int N, int kK, int kC, bool kVec>
cudaError_t launch_scan(const Params &p, cudaStream_t s) {
  using T = Tile<N, kK, kC>;
  static_assert(sizeof(T) <= 227 * 1024, "a tile's buffers have to fit an SM");
  const cudaError_t e = cudaFuncSetAttribute(scan_kernel<kBf16, N, kK, kC, kVec>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(T));
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((p.D + kCh - 1) / kCh), (unsigned)p.rows.R);
  scan_kernel<kBf16, N, kK, kC, kVec><<<grid, T::kScan + kHelpers, sizeof(T), s>>>(p);
  return cudaGetLastError();
}

template <bool kBf16, int N>
cudaError_t launch(const Params &p, bool vector, cudaStream_t s) {
  if (p.rows.max_len <= kFewRows) {
    constexpr int kPer = kFewThreads / (N / 4);
    auto grid = [&](int reqs) { return dim3((unsigned)((p.D + kPer - 1) / kPer), (unsigned)((p.rows.R + reqs - 1) / reqs)); };
    few_kernel<kBf16, N, 1><<<grid(1), kFewThreads, 0, s>>>(p);
    return cudaGetLastError();
  }
  constexpr int kK = 4;
  // two channels a thread where that leaves a scan warp for each of the SMs' schedulers
  const bool two = (long long)p.rows.R * p.D * (N / kK) / 64 >= 608;
  if (two) return vector ? launch_scan<kBf16, N, kK, 2, true>(p, s) : launch_scan<kBf16, N, kK, 2, false>(p, s);
  return vector ? launch_scan<kBf16, N, kK, 1, true>(p, s) : launch_scan<kBf16, N, kK, 1, false>(p, s);
}

template <bool kBf16>
cudaError_t by_state(const Params &p, int N, bool vector, cudaStream_t s) {
  if (N == 8) return launch<kBf16, 8>(p, vector, s);
  if (N == 16) return launch<kBf16, 16>(p, vector, s);
  return launch<kBf16, 32>(p, vector, s);
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
  bool vec[5];  // rows that can be read 16 bytes at a time
  for (int i = 0; i < 5; ++i)
    vec[i] = !rows[i] || (aligned(rows[i], 16) && (a->num_tok == 1 || strides[i] * (long long)es % 16 == 0));
  p.bc_vector = vec[3] && vec[4];
  const bool vector = D % 8 == 0 && vec[0] && vec[1] && vec[2];
  const cudaError_t e = a->in_dtype == GLINATTN_BF16 ? by_state<true>(p, N, vector, stream) : by_state<false>(p, N, vector, stream);
  return e == cudaSuccess ? GLINATTN_OK : GLINATTN_ERR_CUDA;
}

}  // namespace
}  // namespace scan
}  // namespace glinattn

extern "C" glinattn_status glinattn_selective_scan_packed(const glinattn_scan_packed_args *args, glinattn_stream_t stream) {
  return glinattn::scan::run(args, (cudaStream_t)stream);
}
