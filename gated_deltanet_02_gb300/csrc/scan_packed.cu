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
// scan_kernel (prompts and pieces of prompts): a CTA owns 32 channels of a request and has two kinds
// of warps.  The scan warps keep four states of one or two channels in each thread and go
// through tiles of 32 rows that lie ready in shared memory: the steps (dt, dt x), B and C.  A thread
// forms the decays and terms of the next rows while it runs the recurrence of these, so that a
// warp alone keeps its scheduler busy.  The helper warps turn the inputs of the tile after next into
// steps, and the last tile's partial sums into outputs (sum over the channel's threads, skip,
// gate).  One barrier a tile.  Long requests that would leave SMs idle are run in pieces of 512 rows,
// twice: for the states behind them, and from these for the outputs.
//
// ring_kernel (single tokens, drafts): a thread owns a channel; states and rows come, and states go,
// by bulk copies through a ring of buffers.  few_kernel does the same from registers where rows are
// not made of whole 16 bytes.
//
// Bound.  scan_kernel: reads of shared memory.  A warp's 16-byte load takes 4 cycles of the SM's one port, 2
// where neighbouring lanes share it; per row and four states of a channel B, C, the step and the partial
// sum take 6 cycles, with two channels a thread 4; the helpers 13 a row.  At 16 states that is 39 cycles a row of
// 512 elements with one channel a thread, 2.4 for 32 elements, and 1.5 with two (counted: 38.8 M wavefronts beside 25.5 M
// instructions of the exponential unit), beside 1 for their exponentials (32 lanes a cycle) and 1 for their packed arithmetic.  One
// prompt of 8,191 rows, 4,096 channels, 16 states: 204 us (2.6 10^12 elements/s, 0.8 us a tile for each of 128
// CTAs on 152 SMs); 8 prompts of 200 .. 4,001 rows, 2,048 channels: 240 us (2.8 10^12), the port busy 62% of it. With 8 and 32
// states 179 and 312, 219 and 353 us; in fp32 with 16 states 276 and 326; rows that no 16 bytes fit 570 (4,095 channels) and 434.
// ring_kernel: HBM bytes, the states in and out: 256 tokens of 2,048 channels 13.6 us, 5,270 GB/s.
//
// Measured and not kept: groups of scan warps that hand the states on from 8 rows to the next 8 (305 us
// for the prompt above), barriers between the roles instead of one for all (231 us), tiles of 16
// rows (270 us), inputs read ahead into registers (536 us: waits for one load are waits for all).
#include "packed.cuh"
#include "sm100.cuh"

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
  // requests in pieces of `piece` rows: per piece that is not its request's last, the state behind
  // it and the sum of its steps; per request of more than one piece, the state before it
  int piece;
  float *ends, *sums, *starts;
};

// log(1 + e^x) = max(x, 0) + log(1 + e), e = e^-|x| in (0, 1]; log(1 + e) = e P(e), P of degree 8
// fitted to log(1 + e) / e on [0, 1]: the rounded coefficients are within 7.1e-8 of it, from below (6e-8
// for small e, c[0] being 1 - 2^-24), so a small result keeps its relative error but for the exponential's
// argument, whose rounding adds about |x| 2^-24 (5e-6 at x = -80).  Two at a time.
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

// ---------------------------------------------------------------------------
// many rows
// ---------------------------------------------------------------------------

constexpr int kCh = 32, kL = 32;            // channels of a CTA, rows of a tile
constexpr int kHelpers = kL * (kCh / 8);    // helper threads: one for 8 channels of one row

template <bool kBf16, int N, int kK, int kC>
struct Tile {
  static constexpr int kUnits = 2 * kL * N / 8, kBc = (kUnits + kHelpers - 1) / kHelpers;  // units of 8 of B and C: all, of a thread
  // One thread a channel: its CTAs are few, and their helper warps are two groups, one for the inputs
  // and one for the outputs.  Else one group does both in turn.
  static constexpr bool kTwo = kC == 1 && kBf16;  // in fp32 the buffers would not fit
  static constexpr int kThreads = kCh / kC * (N / kK) + (kTwo ? 2 : 1) * kHelpers;
  // Tiles' inputs: asked for kAhead tiles before they become steps, x and z kept until the outputs
  // are formed (three tiles later; in the next iteration where others do that).
  static constexpr int kAhead = 2, kStages = kAhead + 3 + kTwo;
  uint4 raw[kStages][3 + kBc][kBf16 ? 1 : 2][kHelpers];  // x, delta, z, B and C: every input thread's own
  static constexpr int kG = N / kK;              // threads of a channel
  static constexpr int kScan = kCh / kC * kG;    // scan threads
  static constexpr int kPlane = kL * kCh + 4;    // partial sums of one of a channel's threads (4: other banks)
  float step[3][kL][2 * kCh];                    // (dt, dt x) of the channels, permuted: step_at
  float b[3][kL][N], c[3][kL][N];
  float part[2][kG][kPlane];                     // the channels permuted: part_at
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

// 16 bytes to shared memory; zeros, and nothing read, where `there` is false.
__device__ __forceinline__ void copy_async16(void *to, const void *from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sm100::smem_u32(to)), "l"(from), "r"(there ? 16 : 0) : "memory");
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

// What a CTA runs: rows [first, first + rows) of request r, its piece k of `pieces`; `index` is
// the place of the request's first piece among all requests' pieces that are not their last.
struct Piece {
  int r, k, pieces, index, first, rows;
};

// Block y is request y's first piece for y < R, then come the others' in order.  A warp looks
// 32 requests at a time for the one that the block is in.
__device__ __forceinline__ int more_pieces(const Params &p, int r) {
  if (r >= p.rows.R) return 0;
  const Request q = request(p.rows, r);
  return q.ok && q.run > 0 ? (q.run - 1) / p.piece : 0;
}
__device__ __forceinline__ Piece find_piece(const Params &p, int y, int lane) {
  Piece f = {-1, 0, 1, 0, 0, 0};
  int before = 0;  // pieces that are not the last of the requests before these 32
  for (int r0 = 0; r0 < p.rows.R; r0 += 32) {
    const int n = more_pieces(p, r0 + lane);
    int upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    const int first = before + upto - n;
    const int e = y - p.rows.R;  // the block's place among the pieces that are not first
    const bool here = e < 0 ? y == r0 + lane : n > 0 && e >= first && e < first + n;
    const unsigned who = __ballot_sync(0xffffffffu, here);
    if (who) {
      const int l = __ffs(who) - 1;
      f.r = r0 + l;
      f.index = __shfl_sync(0xffffffffu, first, l);
      f.pieces = __shfl_sync(0xffffffffu, n, l) + 1;
      f.k = e < 0 ? 0 : e - f.index + 1;
      break;
    }
    before = min(before + __shfl_sync(0xffffffffu, upto, 31), 1 << 30);
  }
  // ranges that overlap (a decreasing q_start) may have more pieces than the workspace has room for
  if (f.pieces > 1 && f.index + f.pieces - 1 > p.rows.num_tok / p.piece) f.r = -1;
  return f;
}

// Up to 32 requests: the one with the y-th most rows, so that no long one begins when others end.
__device__ __forceinline__ int by_length(const Rows &rows, int y, int lane) {
  int n = -1;
  if (lane < rows.R) {
    const Request q = request(rows, lane);
    n = q.ok ? q.run : 0;
  }
  int rank = 0;
  for (int k = 0; k < rows.R; ++k) {
    const int other = __shfl_sync(0xffffffffu, n, k);
    rank += other > n || (other == n && k < lane);
  }
  return __ffs(__ballot_sync(0xffffffffu, lane < rows.R && rank == y)) - 1;
}

// kPass 0: whole requests.  1: pieces that are not their request's last, for their ends alone (the
// first one's from the request's state, the others' from zeros).  2: all pieces, from the
// state that the ends before them add up to.
template <bool kBf16, int N, int kK, int kC, bool kVec, int kPass>
__global__ void __launch_bounds__(Tile<kBf16, N, kK, kC>::kThreads, kC == 1 ? 1 : 2) scan_kernel(const Params p) {
  using T = Tile<kBf16, N, kK, kC>;
  constexpr bool kOut = kPass != 1;
  extern __shared__ __align__(16) uint8_t smem[];
  T &s = *reinterpret_cast<T *>(smem);
  if (blockIdx.x == 0 && blockIdx.y == 0 && kPass != 1) check_requests(p.rows, threadIdx.x, blockDim.x);
  Piece f = {(int)blockIdx.y, 0, 1, 0, 0, 0};
  if (kPass) f = find_piece(p, blockIdx.y, threadIdx.x & 31);
  else if (p.rows.R > 1 && p.rows.R <= 32) f.r = by_length(p.rows, blockIdx.y, threadIdx.x & 31);
  if (f.r < 0 || (kPass == 1 && f.k == f.pieces - 1)) return;
  Request q = request(p.rows, f.r);
  if (!q.ok || q.run == 0) return;
  if (kPass) {  // the piece's rows in the request's place
    q.s0 += f.k * p.piece;
    q.run = min(p.piece, q.run - f.k * p.piece);
  }
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
        h[i][k] = make_float2(0.0f, 0.0f);
        if (f.k == 0 && in && q.resumed) {
          const size_t at = ((size_t)f.index * p.D + d + i) * N + g * kK;
          // the last piece may have written the pool by now: the first pass has kept what was there
          h[i][k] = kPass == 2 && f.pieces > 1 ? reinterpret_cast<const float2 *>(p.starts + at)[k] : reinterpret_cast<const float2 *>(state + i * N)[k];
          if (kPass == 1) reinterpret_cast<float2 *>(p.starts + at)[k] = h[i][k];
        }
      }
    if (kPass == 2) {
      for (int e = 0; e < f.k; ++e)
#pragma unroll
        for (int i = 0; i < kC; ++i)
          if (d + i < p.D) {
            const size_t at = (size_t)(f.index + e) * p.D + d + i;
            const float sum = p.sums[at];
#pragma unroll
            for (int k = 0; k < kK / 2; ++k) {
              const float2 end = reinterpret_cast<const float2 *>(p.ends + at * N + g * kK)[k];
              const float2 x = __fmul2_rn(A[i][k], make_float2(sum, sum));
              h[i][k] = e ? __ffma2_rn(make_float2(exp2_fast(x.x), exp2_fast(x.y)), h[i][k], end) : end;
            }
          }
    }
    float sum[kC] = {};
    const int steps[2] = {step_at(0, ch >> 3, ch & 7), step_at(1, ch >> 3, ch & 7)};
    const int parts[2] = {part_at(0, ch >> 3, ch & 7), part_at(1, ch >> 3, ch & 7) - kCh};
    // A block of kRows rows: what is read for it, and its decays and terms.  While one block's recurrence
    // runs, the next one's decays are formed and the one's after that is read: nothing waits
    // for a load, and the exponentials lie between the multiply-adds.
    constexpr int kRows = kC == 1 ? 4 : 2, kBlocks = kL / kRows;
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
    auto form = [&](Block &w, const Lines &l, int r, bool counts) {
#pragma unroll
      for (int i = 0; i < kC; ++i)
#pragma unroll
        for (int k = 0; k < kK / 2; ++k) {
          const float2 e = __fmul2_rn(A[i][k], make_float2(l.st[r][2 * i], l.st[r][2 * i]));
          w.a[r][i][k] = make_float2(exp2_fast(e.x), exp2_fast(e.y));
          w.b[r][i][k] = __fmul2_rn(make_float2(l.st[r][2 * i + 1], l.st[r][2 * i + 1]), make_float2(l.b[r][2 * k], l.b[r][2 * k + 1]));
        }
      if (kPass == 1 && counts)
#pragma unroll
        for (int i = 0; i < kC; ++i) sum[i] += l.st[r][2 * i];
    };
    auto run = [&](const Block &w, const Outs &o, int r, float *y) {
#pragma unroll
      for (int i = 0; i < kC; ++i) {
        float2 out;
#pragma unroll
        for (int k = 0; k < kK / 2; ++k) {
          h[i][k] = __ffma2_rn(w.a[r][i][k], h[i][k], w.b[r][i][k]);
          const float2 c2 = make_float2(o.c[r][2 * k], o.c[r][2 * k + 1]);
          if (kOut) out = k ? __ffma2_rn(h[i][k], c2, out) : __fmul2_rn(h[i][k], c2);
        }
        if (kOut) y[i] = out.x + out.y;
      }
    };
    __syncthreads();
    Block w[2];
    Lines l[2];
    Outs o[2];
    fetch(l[0], 0, 0);
    fetch(l[1], 0, kRows);
    if (kOut) fetch_c(o[0], 0, 0);
#pragma unroll
    for (int r = 0; r < kRows; ++r) form(w[0], l[0], r, true);
    int slot = 0;
    for (int i = 0; i < tiles; ++i) {
      const int next = slot == 2 ? 0 : slot + 1;
      float *part = &s.part[i & 1][g][0];
#pragma unroll
      for (int m = 0; m < kBlocks; ++m) {
        // behind the last tile lies an old one or nothing: read and formed, not used
        fetch(l[m & 1], m + 2 < kBlocks ? slot : next, kRows * ((m + 2) % kBlocks));
        if (kOut) fetch_c(o[(m + 1) & 1], m + 1 < kBlocks ? slot : next, kRows * ((m + 1) % kBlocks));
        float y[kRows][kC];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          run(w[m & 1], o[m & 1], r, y[r]);
          form(w[(m + 1) & 1], l[(m + 1) & 1], r, m + 1 < kBlocks || i + 1 < tiles);
        }
#pragma unroll
        for (int r = 0; r < kRows && kOut; ++r) {
          float *to = part + (kRows * m + r) * kCh + parts[(kRows * m + r) & 1];
          if constexpr (kC == 1) to[0] = y[r][0];
          else *reinterpret_cast<float2 *>(to) = make_float2(y[r][0], y[r][1]);
        }
      }
      slot = next;
      __syncthreads();
    }
    if (kPass == 1) {
#pragma unroll
      for (int i = 0; i < kC; ++i)
        if (d + i < p.D) {
          const size_t at = (size_t)(f.index + f.k) * p.D + d + i;
          if (g == 0) p.sums[at] = sum[i];
#pragma unroll
          for (int k = 0; k < kK / 2; ++k) reinterpret_cast<float2 *>(p.ends + at * N + g * kK)[k] = h[i][k];
        }
    } else if (p.update && f.k == f.pieces - 1) {
#pragma unroll
      for (int i = 0; i < kC; ++i)
#pragma unroll
        for (int k = 0; k < kK / 2; ++k)
          if (d + i < p.D) reinterpret_cast<float2 *>(state + i * N)[k] = h[i][k];
    }
    return;
  }
  // --- helper warps: thread (t, u) has row t, channels 8 u .. 8 u + 7 of every tile
  const int helper = threadIdx.x - T::kScan, j = helper % kHelpers, u = j & 3, t = j >> 2, d = d0 + 8 * u, left = min(8, p.D - d);
  const bool in = left > 0;
  constexpr int kUnits = T::kUnits, kBc = T::kBc, kWords = kBf16 ? 1 : 2, kStages = T::kStages, kAhead = T::kAhead;
  const bool out = kOut && p.y, gate = p.z && out;
  float bias[8], skip[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    bias[k] = k < left && p.delta_bias ? p.delta_bias[d + k] : 0.0f;
    skip[k] = k < left && p.skip ? p.skip[d + k] : 0.0f;
  }
  // The inputs come through shared memory, a thread's own and several tiles ahead: registers that
  // wait for memory would hold up the other loads.  Zeros where there are none.
  auto bring = [&](int stage, int what, const void *src, size_t at, int n, bool there, bool vector) {
    uint4 *to = &s.raw[stage][what][0][j];
    if (vector) {
#pragma unroll
      for (int k = 0; k < kWords; ++k)
        copy_async16(to + k * kHelpers, reinterpret_cast<const uint8_t *>(src) + (there ? at * (kBf16 ? 2 : 4) + 16 * k : 0), there);
    } else {
      const Raw8<kBf16> v = load_unit<kBf16>(src, at, there ? n : 0, false);
#pragma unroll
      for (int k = 0; k < kWords; ++k) to[k * kHelpers] = v.w[k];
    }
  };
  auto load = [&](int i) {
    const int row = i * kL + t, stage = i % kStages;
    const size_t r = (size_t)q.s0 + row;
    const bool there = in && row < q.run;
    if (i < tiles) {
      bring(stage, 0, p.x, r * p.x_stride + d, left, there, kVec);
      bring(stage, 1, p.delta, r * p.delta_stride + d, left, there, kVec);
      if (gate) bring(stage, 2, p.z, r * p.z_stride + d, left, there, kVec);
#pragma unroll
      for (int m = 0; m < kBc; ++m) {
        const int e = j + m * kHelpers, line = e / (N / 8), rr = i * kL + (line >> 1), n = (e % (N / 8)) * 8;
        const bool c = line & 1;
        if ((kUnits % kHelpers && e >= kUnits) || (c && !out)) continue;
        bring(stage, 3 + m, c ? p.Cm : p.Bm, ((size_t)q.s0 + rr) * (c ? p.c_stride : p.b_stride) + n, 8, rr < q.run, p.bc_vector);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto take = [&](int stage, int what) {
    Raw8<kBf16> v;
#pragma unroll
    for (int k = 0; k < kWords; ++k) v.w[k] = s.raw[stage][what][k][j];
    return v;
  };
  auto produce = [&](int i, int slot) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    const int stage = i % kStages;
    const bool there = in && i * kL + t < q.run;
    float *to = &s.step[slot][t][0];
    float xs[8], ds[8];
    Raw8<kBf16> x = take(stage, 0), delta = take(stage, 1);
    if (!there) {  // a step of softplus(-infinity) = 0
      const uint32_t inf = kBf16 ? 0xff80ff80u : 0xff800000u;
#pragma unroll
      for (int k = 0; k < kWords; ++k) delta.w[k] = make_uint4(inf, inf, inf, inf);
      x = {};
    }
    unpack8(x, xs);
    unpack8(delta, ds);
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
      float v[8];
      unpack8(take(stage, 3 + m), v);
      float4 *to_bc = reinterpret_cast<float4 *>(line & 1 ? &s.c[slot][line >> 1][n] : &s.b[slot][line >> 1][n]);
      to_bc[0] = make_float4(v[0], v[1], v[2], v[3]);
      to_bc[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  };
  auto finish = [&](int i) {
    const int row = i * kL + t, stage = i % kStages;
    if (!out || !in || row >= q.run) return;
    float f[8];
    float2 y[4];
    unpack8(take(stage, 0), f);
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
      unpack8(take(stage, 2), f);
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] = __fmul2_rn(y[k], silu2(make_float2(f[2 * k], f[2 * k + 1])));
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
  const bool inputs = !T::kTwo || helper < kHelpers, outputs = !T::kTwo || helper >= kHelpers;
  if (inputs) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(i);
    // behind the last tile there are two more, of zero steps: their inputs are not read
    produce(0, 0);
    load(kAhead);
    produce(1, 1);
    load(kAhead + 1);
  }
  __syncthreads();
  int slot = 2;
  for (int i = 0; i < tiles; ++i) {
    if (outputs && i > 0) finish(i - 1);
    if (inputs && i + 2 < tiles) {
      produce(i + 2, slot);
      load(i + 2 + kAhead);
    }
    slot = slot == 2 ? 0 : slot + 1;
    __syncthreads();
  }
  if (outputs) finish(tiles - 1);
}

// ---------------------------------------------------------------------------
// few rows
// ---------------------------------------------------------------------------

constexpr int kFewThreads = 256, kFewRows = 24;  // requests of more rows take the other kernel

// Four elements as they are in memory, and as floats.
template <bool kBf16>
struct Raw4 {
  uint32_t w[kBf16 ? 2 : 4];
};
template <bool kBf16>
__device__ __forceinline__ Raw4<kBf16> load4(const void *p, size_t at, bool vector) {
  Raw4<kBf16> r;
  if constexpr (kBf16) {
    const uint16_t *q = reinterpret_cast<const uint16_t *>(p) + at;
    if (vector) {
      const uint2 v = *reinterpret_cast<const uint2 *>(q);
      r.w[0] = v.x, r.w[1] = v.y;
    } else {
      r.w[0] = q[0] | (uint32_t)q[1] << 16, r.w[1] = q[2] | (uint32_t)q[3] << 16;
    }
  } else {
    const uint32_t *q = reinterpret_cast<const uint32_t *>(p) + at;
    if (vector) {
      const uint4 v = *reinterpret_cast<const uint4 *>(q);
      r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) r.w[k] = q[k];
    }
  }
  return r;
}
template <bool kBf16>
__device__ __forceinline__ void open4(const Raw4<kBf16> &r, float2 *f) {
  if constexpr (kBf16) {
    f[0] = make_float2(bf16_lo(r.w[0]), bf16_hi(r.w[0])), f[1] = make_float2(bf16_lo(r.w[1]), bf16_hi(r.w[1]));
  } else {
    f[0] = make_float2(__uint_as_float(r.w[0]), __uint_as_float(r.w[1])), f[1] = make_float2(__uint_as_float(r.w[2]), __uint_as_float(r.w[3]));
  }
}

// A thread runs kReqs requests one after the other, kBatch rows at a time; the states and the first
// rows of all of them are asked for before any is run.
template <bool kBf16, int N, int kReqs, int kBatch>
__global__ void __launch_bounds__(kFewThreads, 3) few_kernel(const Params p) {
  constexpr int kQ = N / 4;  // threads of a channel, four states each
  if (blockIdx.x == 0) check_requests(p.rows, (long long)blockIdx.y * kFewThreads + threadIdx.x, (long long)gridDim.y * kFewThreads);
  const int g = threadIdx.x % kQ, d = blockIdx.x * (kFewThreads / kQ) + threadIdx.x / kQ;
  const bool in = d < p.D;
  const int dd = in ? d : 0;
  struct Row {
    uint32_t x, delta, z;
    Raw4<kBf16> b, c;
  };
  auto one = [&](const void *src, size_t at) -> uint32_t {
    return kBf16 ? (uint32_t) reinterpret_cast<const uint16_t *>(src)[at] << 16 : reinterpret_cast<const uint32_t *>(src)[at];
  };
  auto row = [&](Row &v, size_t r) {
    v.x = one(p.x, r * p.x_stride + dd);
    v.delta = one(p.delta, r * p.delta_stride + dd);
    v.b = load4<kBf16>(p.Bm, r * p.b_stride + 4 * g, p.bc_vector);
    if (!p.y) return;
    if (p.z) v.z = one(p.z, r * p.z_stride + dd);
    v.c = load4<kBf16>(p.Cm, r * p.c_stride + 4 * g, p.bc_vector);
  };
  Request q[kReqs];
  float4 h4[kReqs];
  Row v[kReqs][kBatch];
#pragma unroll
  for (int i = 0; i < kReqs; ++i) {
    const int r = blockIdx.y * kReqs + i;
    q[i].ok = false;
    if (r < p.rows.R) q[i] = request(p.rows, r);
    if (!q[i].ok) q[i].run = 0, q[i].slot = 0, q[i].resumed = false;
  }
#pragma unroll
  for (int i = 0; i < kReqs; ++i) {
    h4[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (q[i].resumed && in && q[i].run > 0) h4[i] = reinterpret_cast<const float4 *>(p.pool + ((size_t)q[i].slot * p.D + d) * N)[g];
#pragma unroll
    for (int t = 0; t < kBatch; ++t)
      if (t < q[i].run) row(v[i][t], (size_t)q[i].s0 + t);
  }
  const float4 a4 = reinterpret_cast<const float4 *>(p.A + (size_t)dd * N)[g];
  const float2 A[2] = {make_float2(a4.x * kLog2e, a4.y * kLog2e), make_float2(a4.z * kLog2e, a4.w * kLog2e)};
  const float bias = p.delta_bias ? p.delta_bias[dd] : 0.0f, skip = p.skip ? p.skip[dd] : 0.0f;
#pragma unroll
  for (int i = 0; i < kReqs; ++i) {
    if (q[i].run == 0) continue;  // whole CTAs
    float2 h[2] = {make_float2(h4[i].x, h4[i].y), make_float2(h4[i].z, h4[i].w)};
    for (int t0 = 0; t0 < q[i].run; t0 += kBatch) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int t = t0 + k;
        if (t >= q[i].run) break;
        const Row now = v[i][k];
        if (t + kBatch < q[i].run) row(v[i][k], (size_t)q[i].s0 + t + kBatch);
        const float dt = softplus(__uint_as_float(now.delta) + bias), x = __uint_as_float(now.x), dtx = dt * x;
        float2 b[2], c[2], y2 = make_float2(0.0f, 0.0f);
        open4(now.b, b);
        if (p.y) open4(now.c, c);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const float2 e = __fmul2_rn(A[m], make_float2(dt, dt));
          h[m] = __ffma2_rn(make_float2(exp2_fast(e.x), exp2_fast(e.y)), h[m], __fmul2_rn(make_float2(dtx, dtx), b[m]));
          if (p.y) y2 = m ? __ffma2_rn(h[m], c[m], y2) : __fmul2_rn(h[m], c[m]);
        }
        if (!p.y) continue;
        float y = y2.x + y2.y;
#pragma unroll
        for (int o = kQ / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        if (!in || g != 0) continue;
        y = fmaf(skip, x, y);
        if (p.z) y *= silu(__uint_as_float(now.z));
        const size_t at = ((size_t)q[i].s0 + t) * p.D + d;
        if (p.out_bf16) store_one<true>(p.y, at, y);
        else store_one<false>(p.y, at, y);
      }
    }
    if (p.update && in)
      reinterpret_cast<float4 *>(p.pool + ((size_t)q[i].slot * p.D + d) * N)[g] = make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
  }
}

// The same over a ring of buffers that bulk copies fill and empty: a stage is the states of 128 channels
// and the rows of one request, several are on their way to and from each CTA while one is
// run.  A thread has all N states of a channel.  A CTA keeps its channels and goes through every
// `gridDim.x / blocks`-th request.  Rows have to be made of whole 16 bytes.
constexpr int kRingStages = 8, kRingCh = 128;
constexpr size_t kRingBytes = 56 * 1024;  // of a CTA: four on an SM

template <bool kBf16, int N>
struct Ring {
  static constexpr int kSize = kBf16 ? 2 : 4;
  static constexpr int kRowBytes = (3 * kRingCh + 2 * N) * kSize, kStateBytes = kRingCh * N * 4;  // x, delta, z, B, C
};
struct RingHead {
  uint64_t full[kRingStages], empty[kRingStages];
  int4 meta[kRingStages];  // first row, rows, slot, whether it resumes
};

// Shared -> global, both 16-byte aligned, a multiple of 16 bytes.
__device__ __forceinline__ void bulk_store(void *to, const void *from, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"((uint64_t)to), "r"(sm100::smem_u32(from)), "r"(bytes) : "memory");
}

template <bool kBf16, int N>
__global__ void __launch_bounds__(kRingCh + 32, 4) ring_kernel(const Params p, int blocks, int stages, int stage_bytes) {
  using G = Ring<kBf16, N>;
  extern __shared__ __align__(16) uint8_t smem[];
  RingHead &head = *reinterpret_cast<RingHead *>(smem);
  uint8_t *ring = smem + ((sizeof(RingHead) + 127) & ~(size_t)127);
  const int block = blockIdx.x % blocks, r0 = blockIdx.x / blocks, rstep = gridDim.x / blocks;
  const int d0 = block * kRingCh, width = min(kRingCh, p.D - d0), rows_at = G::kStateBytes;
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      sm100::mbar_init(&head.full[i], 1);
      sm100::mbar_init(&head.empty[i], kRingCh / 32);
    }
    sm100::fence_mbar_init();
  }
  __syncthreads();
  auto wait = [&](uint64_t *bar, int parity) {
    const bool ok = sm100::mbar_wait(bar, (uint32_t)parity & 1u);
    if (!ok && p.rows.dev_status) atomicOr(p.rows.dev_status, GLINATTN_DEV_WAIT_TIMEOUT);
    return __all_sync(0xffffffffu, ok) != 0;  // whole warps go on or leave their loop
  };
  bool ok = true;  // no wait of the warp has given up
  if (threadIdx.x >= kRingCh) {
    // --- the warp that brings: 32 requests are looked up at a time, one lane each
    const int lane = threadIdx.x & 31;
    check_requests(p.rows, (long long)blockIdx.x * 32 + lane, (long long)gridDim.x * 32);
    int stage = 0, round = 0, issued = 0;  // stages filled so far
    for (int n0 = r0; ok && n0 < p.rows.R; n0 += 32 * rstep) {
      Request mine;
      mine.ok = false;
      const long long r = n0 + (long long)lane * rstep;
      if (r < p.rows.R) mine = request(p.rows, (int)r);
      if (!mine.ok) mine.s0 = 0, mine.run = 0, mine.slot = 0, mine.resumed = false;
      const int many = min(32, (int)((p.rows.R - n0 + (long long)rstep - 1) / rstep));
      for (int l = 0; l < many; ++l) {
        const int s0 = __shfl_sync(0xffffffffu, mine.s0, l), run = __shfl_sync(0xffffffffu, mine.run, l);
        const int slot = __shfl_sync(0xffffffffu, mine.slot, l), resumed = __shfl_sync(0xffffffffu, (int)mine.resumed, l);
        ok = wait(&head.empty[stage], round ^ 1);
        if (!ok) break;
        uint8_t *to = ring + (size_t)stage * stage_bytes;
        uint64_t *bar = &head.full[stage];
        const int parts = (p.y ? (p.z ? 5 : 4) : 3), row_bytes = (width * (p.y && p.z ? 3 : 2) + N * (p.y ? 2 : 1)) * G::kSize;
        if (lane == 0) {
          head.meta[stage] = make_int4(s0, run, slot, resumed);
          const uint32_t bytes = run ? (uint32_t)(run * row_bytes + (resumed ? width * N * 4 : 0)) : 0u;
          if (bytes) sm100::mbar_arrive_expect_tx(bar, bytes);
          else sm100::mbar_arrive(bar);
        }
        __syncwarp();
        if (lane == 0 && run && resumed) sm100::bulk_load(to, p.pool + ((size_t)slot * p.D + d0) * N, (uint32_t)(width * N * 4), bar);
        // x, delta, B, C, z of each row
        for (int e = lane; e < run * parts; e += 32) {
          const int t = e / parts, what = e - t * parts;
          const size_t row = (size_t)s0 + t;
          const uint8_t *src = reinterpret_cast<const uint8_t *>(what == 0 ? p.x : what == 1 ? p.delta : what == 2 ? p.Bm : what == 3 ? p.Cm : p.z);
          const long long stride = what == 0 ? p.x_stride : what == 1 ? p.delta_stride : what == 2 ? p.b_stride : what == 3 ? p.c_stride : p.z_stride;
          const bool states = what == 2 || what == 3;
          const int at = what == 0 ? 0 : what == 1 ? kRingCh : what == 4 ? 2 * kRingCh : 3 * kRingCh + (what - 2) * N;
          sm100::bulk_load(to + rows_at + t * G::kRowBytes + at * G::kSize, src + (row * stride + (states ? 0 : d0)) * G::kSize,
                           (uint32_t)((states ? N : width) * G::kSize), bar);
        }
        if (++stage == stages) stage = 0, round ^= 1;
        ++issued;
      }
    }
    // After a wait that gave up, here or below, the copies on their way land before the CTA leaves its
    // shared memory to another: a stage's barrier counts their bytes.
    if (!__syncthreads_and(ok))
      for (int i = max(0, issued - stages); i < issued; ++i)
        if (!sm100::mbar_wait(&head.full[i % stages], (uint32_t)(i / stages) & 1u)) break;
    return;
  }
  // --- the warps that run: a thread has a channel.  It goes through its states 16 bytes at a time in an
  // order of its own, in which 8 neighbouring threads are at different banks.
  constexpr int kQ = N / 4;
  const int ch = threadIdx.x, lane = ch & 31, d = d0 + ch, turn = (ch & 7) / (8 / kQ);
  const bool in = ch < width;
  const int dd = in ? d : d0;
  float2 A[kQ][2];
#pragma unroll
  for (int k = 0; k < kQ; ++k) {
    const float4 v = reinterpret_cast<const float4 *>(p.A + (size_t)dd * N)[(k + turn) & (kQ - 1)];
    A[k][0] = make_float2(v.x * kLog2e, v.y * kLog2e), A[k][1] = make_float2(v.z * kLog2e, v.w * kLog2e);
  }
  const float bias = p.delta_bias ? p.delta_bias[dd] : 0.0f, skip = p.skip ? p.skip[dd] : 0.0f;
  const int mine = min(32, width - (ch & ~31)) * N * 4;  // bytes of the warp's states
  int stage = 0, round = 0, leaving = -1;                // the stage whose states are on their way back
  for (long long r = r0; r < p.rows.R; r += rstep) {
    ok = wait(&head.full[stage], round);
    if (!ok) break;
    const int4 m = head.meta[stage];
    const int s0 = m.x, run = m.y;
    uint8_t *from = ring + (size_t)stage * stage_bytes;
    float4 *state = reinterpret_cast<float4 *>(from) + ch * kQ;
    float2 h[kQ][2];
#pragma unroll
    for (int k = 0; k < kQ; ++k) {
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (run && m.w) v = state[(k + turn) & (kQ - 1)];
      h[k][0] = make_float2(v.x, v.y), h[k][1] = make_float2(v.z, v.w);
    }
    for (int t = 0; t < run; ++t) {  // threads without a channel run what lies there, and store nothing
      const uint8_t *row = from + rows_at + t * G::kRowBytes;
      const float x = load_one<kBf16>(row, ch), dt = softplus(load_one<kBf16>(row, kRingCh + ch) + bias), dtx = dt * x;
      float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
      for (int k = 0; k < kQ; ++k) {
        const int at = 4 * ((k + turn) & (kQ - 1));
        float2 b[2], c[2];
        open4(load4<kBf16>(row, 3 * kRingCh + at, true), b);
        if (p.y) open4(load4<kBf16>(row, 3 * kRingCh + N + at, true), c);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 e = __fmul2_rn(A[k][i], make_float2(dt, dt));
          h[k][i] = __ffma2_rn(make_float2(exp2_fast(e.x), exp2_fast(e.y)), h[k][i], __fmul2_rn(make_float2(dtx, dtx), b[i]));
          if (p.y) sum[i] = __ffma2_rn(h[k][i], c[i], sum[i]);
        }
      }
      if (!p.y || !in) continue;
      sum[0] = __fadd2_rn(sum[0], sum[1]);
      float y = fmaf(skip, x, sum[0].x + sum[0].y);
      if (p.z) y *= silu(load_one<kBf16>(row, 2 * kRingCh + ch));
      const size_t at = ((size_t)s0 + t) * p.D + d;
      if (p.out_bf16) store_one<true>(p.y, at, y);
      else store_one<false>(p.y, at, y);
    }
    const bool store = p.update && run;
    if (store) {
#pragma unroll
      for (int k = 0; k < kQ; ++k) state[(k + turn) & (kQ - 1)] = make_float4(h[k][0].x, h[k][0].y, h[k][1].x, h[k][1].y);
      sm100::fence_proxy_async_smem();
    }
    __syncwarp();
    if (lane == 0) {
      if (store) {
        if (mine > 0) bulk_store(p.pool + ((size_t)m.z * p.D + d) * N, state, (uint32_t)mine);
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        if (leaving >= 0) {
          asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
          sm100::mbar_arrive(&head.empty[leaving]);
        }
      } else {
        if (leaving >= 0) {
          asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          sm100::mbar_arrive(&head.empty[leaving]);
        }
        sm100::mbar_arrive(&head.empty[stage]);
      }
    }
    leaving = store ? stage : -1;
    if (++stage == stages) stage = 0, round ^= 1;
  }
  if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  __syncthreads_and(ok);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

template <bool kBf16, int N>
cudaError_t launch_ring(const Params &p, cudaStream_t s) {
  using G = Ring<kBf16, N>;
  const int stage_bytes = (G::kStateBytes + p.rows.max_len * G::kRowBytes + 127) & ~127;
  const size_t head = (sizeof(RingHead) + 127) & ~(size_t)127;
  int stages = (int)((kRingBytes - head) / stage_bytes);  // two at least, with a larger share of the SM where rows are many
  stages = stages < 2 ? 2 : stages > kRingStages ? kRingStages : stages;
  const size_t bytes = head + (size_t)stages * stage_bytes;
  // The limit is the kernel's, for all host threads: what the largest call takes, whatever this one does.
  constexpr size_t two = ((sizeof(RingHead) + 127) & ~(size_t)127) + 2 * (G::kStateBytes + kFewRows * G::kRowBytes + 128);
  constexpr size_t most = two > kRingBytes ? two : kRingBytes;
  static_assert(most <= 200 * 1024, "two stages have to fit");
  const cudaError_t e = cudaFuncSetAttribute(ring_kernel<kBf16, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
  if (e != cudaSuccess) return e;
  const int blocks = (p.D + kRingCh - 1) / kRingCh, together = 4 * 152 / blocks;
  const int per = together < 1 ? 1 : together < p.rows.R ? together : p.rows.R;
  ring_kernel<kBf16, N><<<(unsigned)(blocks * per), kRingCh + 32, bytes, s>>>(p, blocks, stages, stage_bytes);
  return cudaGetLastError();
}

constexpr int kPiece = 512;        // rows of a piece
constexpr int kPiecedReqs = 1024;  // requests at most: every block looks through their lengths

// Whether requests are run in pieces, which costs a second pass over nearly all rows
// (without outputs) and balances the SMs.
bool pieced(int R, int num_tok, int max_len, int D, int N) {
  if (R > kPiecedReqs || max_len <= 2 * kPiece || num_tok / kPiece + R > 65535) return false;
  // In ns, at N = 16 in bf16: a tile of 32 rows and channels takes 850 where its CTA has an SM to itself, 1,430 where two
  // share one; both passes over pieces, on full SMs, take 9.2 a tile.  (One request of 8,192 rows and
  // 4,096 channels: 210 us whole, 305 in pieces; 2,048 channels: 210 and 169.)
  // A piece reads what all pieces before it in its request end with, at 3,000 bytes a ns, half of that where
  // they do not fit in L2.  (One request of 2^17 rows and 2,048 channels: 3.2 ms whole, 3.9 in pieces;
  // 2^20: 26 and 231; 2^18 and 2^20 rows of 256 channels: 6.3 and 25 whole, 1.4 and 15 in pieces.)
  const double ctas = (double)R * ((D + kCh - 1) / kCh), tiles = (max_len + kL - 1) / kL;
  const double whole = ctas <= 152 ? 850.0 * tiles : 1430.0 * tiles * (double)(((long long)ctas + 303) / 304);
  const double before = 0.5 * ((double)num_tok / kPiece) * ((double)max_len / kPiece) * (double)D * (N + 1) * 4.0;
  return 15000.0 + 9.2 * ((double)num_tok / kL) * ((D + kCh - 1) / kCh) + before / 3000.0 < 0.9 * whole;
}
size_t up16(size_t n) { return (n + 15) & ~(size_t)15; }

template <bool kBf16, int N, int kC, bool kVec, int kPass>
cudaError_t launch_scan(const Params &p, int pieces, cudaStream_t s) {
  constexpr int kK = 4;
  using T = Tile<kBf16, N, kK, kC>;
  static_assert(sizeof(T) <= 227 * 1024, "a tile's buffers have to fit an SM");
  const auto kernel = scan_kernel<kBf16, N, kK, kC, kVec, kPass>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(T));
  if (e != cudaSuccess) return e;
  kernel<<<dim3((unsigned)((p.D + kCh - 1) / kCh), (unsigned)(p.rows.R + pieces)), T::kThreads, sizeof(T), s>>>(p);
  return cudaGetLastError();
}

template <bool kBf16, int N, bool kVec>
cudaError_t launch_many(const Params &p, cudaStream_t s) {
  if (p.piece) {
    const int pieces = p.rows.num_tok / p.piece;
    const cudaError_t e = launch_scan<kBf16, N, 2, kVec, 1>(p, pieces, s);
    return e == cudaSuccess ? launch_scan<kBf16, N, 2, kVec, 2>(p, pieces, s) : e;
  }
  // one channel a thread, a CTA alone on its SM, while there are as many SMs (4 requests of 4,096 rows and 2,048
  // channels, 256 CTAs: 217 us, with two channels a thread 183)
  const bool two = (long long)p.rows.R * ((p.D + kCh - 1) / kCh) > 152;
  return two ? launch_scan<kBf16, N, 2, kVec, 0>(p, 0, s) : launch_scan<kBf16, N, 1, kVec, 0>(p, 0, s);
}

template <bool kBf16, int N>
cudaError_t launch(const Params &p, bool vector, cudaStream_t s) {
  // Rows one after the other with all states in flight, or 32 channels a CTA; measured at N = 16 in bf16: 8 requests of 2,048 channels take 3 + 0.43 us
  // a row and, up to 32 rows, 7.8 us; 64 requests of 17, 24 and 32 rows 23, 31, 48 us and 46, 48, 50 us.
  const bool many = (long long)p.rows.R * ((p.D + kCh - 1) / kCh) > 304;
  if (p.rows.max_len <= (many ? kFewRows : 11)) {
    constexpr int kPer = kFewThreads / (N / 4);
    auto grid = [&](int reqs) { return dim3((unsigned)((p.D + kPer - 1) / kPer), (unsigned)((p.rows.R + reqs - 1) / reqs)); };
    if (vector && p.bc_vector) return launch_ring<kBf16, N>(p, s);
    if (p.rows.max_len == 1) few_kernel<kBf16, N, 2, 1><<<grid(2), kFewThreads, 0, s>>>(p);
    else few_kernel<kBf16, N, 1, 2><<<grid(1), kFewThreads, 0, s>>>(p);
    return cudaGetLastError();
  }
  return vector ? launch_many<kBf16, N, true>(p, s) : launch_many<kBf16, N, false>(p, s);
}

template <bool kBf16>
cudaError_t by_state(const Params &p, int N, bool vector, cudaStream_t s) {
  if (N == 8) return launch<kBf16, 8>(p, vector, s);
  if (N == 16) return launch<kBf16, 16>(p, vector, s);
  return launch<kBf16, 32>(p, vector, s);
}

bool activation(int dtype) { return dtype == GLINATTN_F32 || dtype == GLINATTN_BF16; }

glinattn_status check_sizes(const glinattn_scan_packed_args *a) {
  if (!a || !activation(a->in_dtype) || !activation(a->out_dtype) || a->num_req < 0 || a->num_tok < 0 || a->channels <= 0 ||
      a->state <= 0 || a->max_q_len < 0 || a->x_stride < 0 || a->delta_stride < 0 || a->z_stride < 0 || a->b_stride < 0 ||
      a->c_stride < 0)
    return GLINATTN_ERR_INVALID_ARG;
  if ((a->state != 8 && a->state != 16 && a->state != 32) || a->num_req > 65535 || a->num_tok > (1 << 30) || a->channels > (1 << 20))
    return GLINATTN_ERR_UNSUPPORTED;
  return GLINATTN_OK;
}

// Bytes of the workspace, and where its parts begin; 0 where requests are run whole.
size_t workspace(const glinattn_scan_packed_args *a, size_t *sums, size_t *starts) {
  const int longest = a->max_q_len < a->num_tok ? a->max_q_len : a->num_tok;
  if (a->num_req == 0 || a->num_tok == 0 || !pieced(a->num_req, a->num_tok, longest, a->channels, a->state)) return 0;
  const size_t pieces = (size_t)(a->num_tok / kPiece), ends = pieces * a->channels * a->state * 4, each = up16(pieces * a->channels * 4);
  if (sums) *sums = ends, *starts = ends + each;
  return 2 * ends + each;
}

glinattn_status run(const glinattn_scan_packed_args *a, cudaStream_t stream) {
  const glinattn_status st = check_sizes(a);
  if (st != GLINATTN_OK) return st;
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
  size_t sums = 0, starts = 0;
  const size_t need = workspace(a, &sums, &starts);
  p.piece = need ? kPiece : 0;
  p.ends = p.sums = p.starts = nullptr;
  if (need) {
    if (!a->workspace || a->workspace_bytes < need || !aligned(a->workspace, 16)) return GLINATTN_ERR_INVALID_ARG;
    uint8_t *ws = static_cast<uint8_t *>(a->workspace);
    p.ends = reinterpret_cast<float *>(ws);
    p.sums = reinterpret_cast<float *>(ws + sums);
    p.starts = reinterpret_cast<float *>(ws + starts);
  }
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

extern "C" size_t glinattn_selective_scan_packed_workspace_size(const glinattn_scan_packed_args *args) {
  return glinattn::scan::check_sizes(args) == GLINATTN_OK ? glinattn::scan::workspace(args, nullptr, nullptr) : 0;
}

extern "C" glinattn_status glinattn_selective_scan_packed(const glinattn_scan_packed_args *args, glinattn_stream_t stream) {
  return glinattn::scan::run(args, (cudaStream_t)stream);
}
