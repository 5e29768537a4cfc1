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
// Bound: HBM bytes, x in and y out.
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
  Raw8<kBf16> v;
  float s;
};
template <bool kBf16, int kVec>
__device__ __forceinline__ Lane<kBf16, kVec> load_lane(const void *p, size_t i, bool in) {
  Lane<kBf16, kVec> l = {};
  if (in) {
    if constexpr (kVec == 8) l.v = load_raw8<kBf16>(p, i);
    else l.s = load_one<kBf16>(p, i);
  }
  return l;
}
template <bool kBf16, int kVec>
__device__ __forceinline__ void open_lane(const Lane<kBf16, kVec> &l, float *f) {
  if constexpr (kVec == 8) unpack8(l.v, f);
  else f[0] = l.s;
}
template <bool kBf16, int kVec>
__device__ __forceinline__ void store_lane(void *p, size_t i, const float *f) {
  if constexpr (kVec == 8) store8<kBf16>(p, i, f);
  else store_one<kBf16>(p, i, f[0]);
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
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][i] = in ? p.w[(size_t)(c + i) * W + j] : 0.0f;
    b[i] = in && p.bias ? p.bias[c + i] : 0.0f;
  }
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
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      o[i] = b[i];
#pragma unroll
      for (int j = 0; j < W - 1; ++j) o[i] = fmaf(w[j][i], past[j][i], o[i]);
      o[i] = fmaf(w[W - 1][i], x[i], o[i]);
      if (p.silu) o[i] = o[i] / (1.0f + expf(-o[i]));
    }
    shift(raw);
    if (in && p.y) store_lane<kBf16, kVec>(p.y, (size_t)t * p.C + c, o);
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
  for (int base = t0; base < t1; base += kLoad) {
    Lane<kBf16, kVec> raw[kLoad];
    if (p.y) {
#pragma unroll
      for (int u = 0; u < kLoad; ++u) raw[u] = load_lane<kBf16, kVec>(p.x, x_at(base + u), in && base + u < t1);
    }
#pragma unroll
    for (int u = 0; u < kLoad; ++u) {
      const int t = base + u;
      if (t >= t1) break;
      if (t >= q.s1) enter(t);
      const bool others = q.s0 < t0 && t - q.s0 < W - 1;  // run by the warp of the request's first row
      if (!live(t)) continue;
      if (others) shift(raw[u]);
      else step(t, raw[u]);
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
  // rows of a warp: one where every request has one, more rows (whose halo is
  // read once) where there are enough of them
  const bool many = p.rows.q_start && (long long)p.rows.num_tok * p.C > (1 << 22);
  if (vector) {
    if (many) launch<kBf16, 8, W, 16>(p, s);
    else launch<kBf16, 8, W, 2>(p, s);
  } else {
    if (many) launch<kBf16, 1, W, 16>(p, s);
    else launch<kBf16, 1, W, 2>(p, s);
  }
}

glinattn_status run(const glinattn_short_conv_args *a, cudaStream_t stream) {
  if (!a || (a->in_dtype != GLINATTN_F32 && a->in_dtype != GLINATTN_BF16) || a->num_req < 0 || a->num_tok < 0 ||
      a->channels <= 0 || a->x_stride < 0 || (a->activation != 0 && a->activation != 1))
    return GLINATTN_ERR_INVALID_ARG;
  if (a->width < 2 || a->width > 4 || a->num_req > 65535 || a->channels > (1 << 20)) return GLINATTN_ERR_UNSUPPORTED;
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
  const bool vector = a->channels % 8 == 0 && aligned(a->x, 16) && (a->num_tok == 1 || (stride * (long long)es) % 16 == 0);
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
