// short_conv.cu -- the state-space block's causal depthwise convolution over
// packed rows, its history in a slot-indexed pool (glinattn_short_conv).
//
// Mathematics: y_t = act(bias + sum_j w_j x_{t - (W - 1) + j}) per channel.  A warp
// owns a tile of token rows and 32 * kVec channels; the last W - 1 inputs of the
// request move along in registers.
//
// A request's slot is read and written by one warp per channel block, the one whose
// tile has the request's first row: that warp also runs the request's first W - 1
// rows where they pass the tile's end (they are the ones that need the history), and
// the next tile leaves them out.  So nothing reads a slot after it was written.
//
// Bound: HBM bytes, x in and y out, at 27% of the warps an SM can hold (95 registers): 8 prompts of 200 ..
// 4,001 rows, 4,096 channels in bf16, take 63 us (4,740 GB/s); 256 single tokens of 2,048 channels 4.7 us.  Eight
// channels a lane took 72 us (182 registers), without reading ahead 80 us, scalar arithmetic with a
// division 251 us.
#include "packed.cuh"

namespace glinattn {
namespace conv {
namespace {

using namespace packed;

struct Params {
  Rows rows;
  const void *x;
  long long x_stride;
  const float *w, *bias;
  void *pool, *y;
  int C, silu, update;
};

constexpr int kWarps = 4;  // of a CTA

template <bool kBf16, int kVec>
struct Lane {  // kVec channels of one row as they are in memory
  uint32_t w[kVec == 1 ? 1 : kBf16 ? kVec / 2 : kVec];
};
template <bool kBf16, int kVec>
__device__ __forceinline__ Lane<kBf16, kVec> load_lane(const void *p, size_t i, bool in) {
  Lane<kBf16, kVec> l = {};
  if (!in) return l;
  const uint8_t *at = reinterpret_cast<const uint8_t *>(p) + i * (kBf16 ? 2 : 4);
  if constexpr (kVec == 1) {
    l.w[0] = kBf16 ? *reinterpret_cast<const uint16_t *>(at) : *reinterpret_cast<const uint32_t *>(at);
  } else if constexpr (kBf16) {
    const uint2 v = *reinterpret_cast<const uint2 *>(at);
    l.w[0] = v.x, l.w[1] = v.y;
  } else {
    const uint4 v = *reinterpret_cast<const uint4 *>(at);
    l.w[0] = v.x, l.w[1] = v.y, l.w[2] = v.z, l.w[3] = v.w;
  }
  return l;
}
template <bool kBf16, int kVec>
__device__ __forceinline__ void open_lane(const Lane<kBf16, kVec> &l, float *f) {
  if constexpr (kBf16) {
    f[0] = bf16_lo(l.w[0]);
    if constexpr (kVec == 4) f[1] = bf16_hi(l.w[0]), f[2] = bf16_lo(l.w[1]), f[3] = bf16_hi(l.w[1]);
  } else {
#pragma unroll
    for (int k = 0; k < kVec; ++k) f[k] = __uint_as_float(l.w[k]);
  }
}
template <bool kBf16, int kVec>
__device__ __forceinline__ void store_lane(void *p, size_t i, const float *f) {
  uint8_t *at = reinterpret_cast<uint8_t *>(p) + i * (kBf16 ? 2 : 4);
  if constexpr (kVec == 1) store_one<kBf16>(p, i, f[0]);
  else if constexpr (kBf16) *reinterpret_cast<uint2 *>(at) = make_uint2(paged::pack_bf16(f[0], f[1]), paged::pack_bf16(f[2], f[3]));
  else *reinterpret_cast<float4 *>(at) = make_float4(f[0], f[1], f[2], f[3]);
}

// A lane's weights and bias: kVec channels' are next to each other.
template <int W, int kVec>
__device__ __forceinline__ void load_weights(const Params &p, int c, bool in, float (*w)[kVec], float *b) {
  if constexpr (kVec == 1) {
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][0] = in ? p.w[(size_t)c * W + j] : 0.0f;
    b[0] = in && p.bias ? p.bias[c] : 0.0f;
  } else {
    float f[kVec * W];
#pragma unroll
    for (int k = 0; k < kVec * W / 4; ++k) {
      const float4 v = in ? reinterpret_cast<const float4 *>(p.w + (size_t)c * W)[k] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      f[4 * k] = v.x, f[4 * k + 1] = v.y, f[4 * k + 2] = v.z, f[4 * k + 3] = v.w;
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i)
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][i] = f[i * W + j];
#pragma unroll
    for (int k = 0; k < kVec / 4; ++k) {
      const float4 v = in && p.bias ? reinterpret_cast<const float4 *>(p.bias + c)[k] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      b[4 * k] = v.x, b[4 * k + 1] = v.y, b[4 * k + 2] = v.z, b[4 * k + 3] = v.w;
    }
  }
}

// kTile: rows of a warp, kLoad of them in flight at a time.
template <bool kBf16, int kVec, int W, int kTile>
__global__ void __launch_bounds__(32 * kWarps) conv_kernel(const Params p) {
  constexpr int kLoad = kTile < 8 ? kTile : 8;
  const int lane = threadIdx.x & 31;
  if (blockIdx.y == 0) check_requests(p.rows, (long long)blockIdx.x * blockDim.x + threadIdx.x, (long long)gridDim.x * blockDim.x);
  const long long first = ((long long)blockIdx.x * kWarps + (threadIdx.x >> 5)) * kTile;
  if (first >= p.rows.num_tok) return;  // whole warps
  const int t0 = (int)first, t1 = (int)min(first + kTile, (long long)p.rows.num_tok);
  const int c = (blockIdx.y * 32 + lane) * kVec;
  const bool in = c < p.C;
  float w[W][kVec], b[kVec];
  load_weights<W, kVec>(p, c, in, w, b);
  float past[W - 1][kVec];  // the last W - 1 inputs, oldest first
  Request q;
  q.ok = false;
  q.s0 = q.s1 = t0;
  auto x_at = [&](int t) { return (size_t)t * p.x_stride + c; };
  auto history = [&](float(*h)[kVec]) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      open_lane<kBf16, kVec>(load_lane<kBf16, kVec>(p.pool, ((size_t)q.slot * (W - 1) + j) * p.C + c, in && q.resumed), h[j]);
  };
  auto shift = [&](const Lane<kBf16, kVec> &raw) {
    float x[kVec];
    open_lane<kBf16, kVec>(raw, x);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
      for (int i = 0; i < kVec; ++i) past[j][i] = j < W - 2 ? past[j + 1][i] : x[i];
  };
  auto step = [&](int t, const Lane<kBf16, kVec> &raw) {
    float x[kVec], o[kVec];
    open_lane<kBf16, kVec>(raw, x);
    if constexpr (kVec == 1) {
      o[0] = b[0];
#pragma unroll
      for (int j = 0; j < W - 1; ++j) o[0] = fmaf(w[j][0], past[j][0], o[0]);
      o[0] = fmaf(w[W - 1][0], x[0], o[0]);
      if (p.silu) o[0] = silu(o[0]);
    } else {
      auto two = [](const float *f, int i) { return make_float2(f[i], f[i + 1]); };
#pragma unroll
      for (int i = 0; i < kVec; i += 2) {
        float2 s = two(b, i);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) s = __ffma2_rn(two(w[j], i), two(past[j], i), s);
        s = __ffma2_rn(two(w[W - 1], i), two(x, i), s);
        if (p.silu) s = silu2(s);
        o[i] = s.x, o[i + 1] = s.y;
      }
    }
    shift(raw);
    if (in) store_lane<kBf16, kVec>(p.y, (size_t)t * p.C + c, o);
  };
  // A request's first row: its history, and its state after the rows that it runs.
  auto begin = [&]() {
    if (!q.ok || q.run == 0) return;
    history(past);
    if (!p.update || !p.pool) return;
    float now[W - 1][kVec];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int at = q.run - (W - 1) + j;  // row of the request, or a place in its history
      if (at >= 0) {
        open_lane<kBf16, kVec>(load_lane<kBf16, kVec>(p.x, x_at(q.s0 + at), in), now[j]);
      } else {
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
          if (k == W - 1 + at)
#pragma unroll
            for (int i = 0; i < kVec; ++i) now[j][i] = past[k][i];
      }
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      if (in) store_lane<kBf16, kVec>(p.pool, ((size_t)q.slot * (W - 1) + j) * p.C + c, now[j]);
  };
  // The request of row t, when the warp comes upon it.
  auto enter = [&](int t) {
    const int r = p.rows.q_start ? paged::find_request(p.rows.q_start, p.rows.R, t, lane) : t;
    q = request(p.rows, r);
    if (t < q.s0 || t >= q.s1) {  // a row of no request: looked at again at the next row
      q.ok = false;
      q.s0 = q.s1 = t + 1;
      return;
    }
    if (t == q.s0) {
      begin();
    } else if (q.s0 >= t0) {  // a decreasing q_start hid the request's first row
      q.ok = false;
    } else if (q.ok) {
#pragma unroll
      for (int j = 0; j < W - 1; ++j) {
        const int row = t - (W - 1) + j;  // rows before the request's first are not used: see the head
        open_lane<kBf16, kVec>(load_lane<kBf16, kVec>(p.x, x_at(row), in && row >= q.s0), past[j]);
      }
    }
  };
  auto live = [&](int t) { return q.ok && p.y && t - q.s0 < q.run; };
  Lane<kBf16, kVec> next[kLoad];
  auto ahead = [&](int base) {
#pragma unroll
    for (int u = 0; u < kLoad; ++u) next[u] = load_lane<kBf16, kVec>(p.x, x_at(base + u), in && p.y && base + u < t1);
  };
  ahead(t0);
  enter(t0);
  for (int base = t0; base < t1; base += kLoad) {
    Lane<kBf16, kVec> raw[kLoad];
#pragma unroll
    for (int u = 0; u < kLoad; ++u) raw[u] = next[u];
    if (kTile > kLoad) ahead(base + kLoad);
    // all of these rows belong to the request and are this warp's to run
    if (base + kLoad <= t1 && base + kLoad <= q.s1 && live(base + kLoad - 1) && (q.s0 >= t0 || base - q.s0 >= W - 1)) {
#pragma unroll
      for (int u = 0; u < kLoad; ++u) step(base + u, raw[u]);
      continue;
    }
    const int end = min(base + kLoad, t1);
#pragma unroll 1
    for (int t = base; t < end; ++t) {
      if (t >= q.s1) enter(t);
      if (!live(t)) continue;
      const Lane<kBf16, kVec> raw = load_lane<kBf16, kVec>(p.x, x_at(t), in);
      if (q.s0 < t0 && t - q.s0 < W - 1) shift(raw);  // run by the warp of the request's first row
      else step(t, raw);
    }
  }
  if (q.s0 >= t0 && q.s1 > t1)  // the first rows of the last request, past the tile's end
    for (int t = t1; t < q.s1 && t - q.s0 < W - 1 && live(t); ++t) step(t, load_lane<kBf16, kVec>(p.x, x_at(t), in));
}

template <bool kBf16, int kVec, int W, int kTile>
void launch(const Params &p, cudaStream_t s) {
  const long long tiles = ((long long)p.rows.num_tok + kTile - 1) / kTile;
  const dim3 grid((unsigned)((tiles + kWarps - 1) / kWarps), (unsigned)((p.C + 32 * kVec - 1) / (32 * kVec)));
  conv_kernel<kBf16, kVec, W, kTile><<<grid, 32 * kWarps, 0, s>>>(p);
}

template <bool kBf16, int W>
void by_size(const Params &p, bool vector, cudaStream_t s) {
  // Rows of a warp: two where every request has one; else as many as leave 16 warps an SM, as a
  // tile's weights and history are read once.  (20,800 rows of 4,096 channels with 16, 32 and 64:
  // 75, 65 and 63 us; 256 single tokens of 2,048 channels with 1 and 2: 5.4 and 4.6 us.)
  constexpr int kVec = 4;
  const long long units = (long long)p.rows.num_tok * ((p.C + 31) / 32) / (vector ? kVec : 1), enough = 152 * 16;
  const int tile = !p.rows.q_start || units / 16 < enough ? 2 : units / 64 < enough ? 16 : 64;
  if (vector) {
    if (tile == 64) launch<kBf16, kVec, W, 64>(p, s);
    else if (tile == 16) launch<kBf16, kVec, W, 16>(p, s);
    else launch<kBf16, kVec, W, 2>(p, s);
  } else {
    if (tile == 64) launch<kBf16, 1, W, 64>(p, s);
    else if (tile == 16) launch<kBf16, 1, W, 16>(p, s);
    else launch<kBf16, 1, W, 2>(p, s);
  }
}

glinattn_status run(const glinattn_short_conv_args *a, cudaStream_t stream) {
  if (!a || (a->in_dtype != GLINATTN_F32 && a->in_dtype != GLINATTN_BF16) || a->num_req < 0 || a->num_tok < 0 ||
      a->channels <= 0 || a->x_stride < 0 || (a->activation != 0 && a->activation != 1))
    return GLINATTN_ERR_INVALID_ARG;
  if (a->width < 2 || a->width > 4 || a->num_req > 65535 || a->num_tok > (1 << 30) || a->channels > (1 << 20))
    return GLINATTN_ERR_UNSUPPORTED;
  if ((a->conv_pool == nullptr) != (a->slot_ids == nullptr) || (a->conv_pool && a->pool_slots <= 0)) return GLINATTN_ERR_INVALID_ARG;
  if (!a->q_start && a->num_tok != a->num_req) return GLINATTN_ERR_INVALID_ARG;
  if (a->num_req == 0 || a->num_tok == 0) return GLINATTN_OK;
  const bool update = a->update_state && a->conv_pool;
  if (!a->x || !a->w || (!a->y && !update)) return GLINATTN_ERR_INVALID_ARG;
  const size_t es = a->in_dtype == GLINATTN_BF16 ? 2 : 4;
  const long long stride = a->x_stride ? a->x_stride : a->channels;
  if (stride < a->channels && a->num_tok > 1) return GLINATTN_ERR_INVALID_ARG;
  const void *list[] = {a->w, a->bias, a->conv_pool, a->y};
  for (const void *q : list)
    if (!aligned(q, 16)) return GLINATTN_ERR_INVALID_ARG;
  const void *ints[] = {a->slot_ids, a->q_start, a->resume, a->count};
  for (const void *q : ints)
    if (!aligned(q, 4)) return GLINATTN_ERR_INVALID_ARG;
  if (!aligned(a->x, es)) return GLINATTN_ERR_INVALID_ARG;
  const size_t nx = row_bytes(a->num_tok, a->channels, stride, es), ny = (size_t)a->num_tok * a->channels * es;
  const size_t np = a->conv_pool ? (size_t)a->pool_slots * (a->width - 1) * a->channels * es : 0;
  if (overlap(a->y, ny, a->x, nx) || overlap(a->y, ny, a->conv_pool, np) || (update && overlap(a->conv_pool, np, a->x, nx)))
    return GLINATTN_ERR_INVALID_ARG;
  Params p;
  p.rows = {a->num_req, a->num_tok, a->pool_slots, INT32_MAX, a->conv_pool != nullptr, a->q_start, a->slot_ids, a->resume, a->count, a->dev_status};
  p.x = a->x, p.x_stride = stride, p.w = a->w, p.bias = a->bias, p.pool = a->conv_pool, p.y = a->y;
  p.C = a->channels, p.silu = a->activation, p.update = update;
  const bool vector = a->channels % 4 == 0 && aligned(a->x, 16) && (a->num_tok == 1 || (stride * (long long)es) % 16 == 0);
  const bool bf16 = a->in_dtype == GLINATTN_BF16;
  switch (a->width) {
    case 2: bf16 ? by_size<true, 2>(p, vector, stream) : by_size<false, 2>(p, vector, stream); break;
    case 3: bf16 ? by_size<true, 3>(p, vector, stream) : by_size<false, 3>(p, vector, stream); break;
    default: bf16 ? by_size<true, 4>(p, vector, stream) : by_size<false, 4>(p, vector, stream); break;
  }
  return cudaGetLastError() == cudaSuccess ? GLINATTN_OK : GLINATTN_ERR_CUDA;
}

}  // namespace
}  // namespace conv
}  // namespace glinattn

extern "C" glinattn_status glinattn_short_conv(const glinattn_short_conv_args *args, glinattn_stream_t stream) {
  return glinattn::conv::run(args, (cudaStream_t)stream);
}
