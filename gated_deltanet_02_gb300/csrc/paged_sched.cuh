// paged_sched.cuh -- how the attention kernels share their work out, and the
// merge of partial results.
//
// The work of a call is a row of units, one unit being the 128 keys of one
// cache tile for one item; an item is (request, key / value head, tile of query
// tokens), and its units are kCost for its own beginning and end (reading q,
// writing outputs) and then the cache tiles that its last token sees (one at
// least).  Requests come in order, then heads, then token tiles.  CTA c takes
// units [c n, (c + 1) n), n = ceil(units / CTAs): every SM reads the same number
// of cache tiles whatever the lengths are, and a long request is shared by many.
// An item whose units fall to several CTAs leaves one partial result per CTA
// (running maximum, sum, unscaled outputs) that merge_kernel joins in CTA
// order, so results depend on the lengths only.
//
// The lengths are in device memory, so every CTA finds its own units: a sum
// over the requests, then a scan up to the request that holds its first one.
#pragma once

#include <math.h>

#include "paged.cuh"

namespace glinattn {
namespace paged {

constexpr int kTileKeys = 128;
// What an item costs beside its cache tiles, in cache tiles.  Without it the SMs
// that get many short items end last: packed prompts of 200 .. 4001 tokens, 16
// heads over 4, take 159, 144, 149, 155 us with 1, 2, 3, 4 from a bf16 cache (a prompt
// of 16,000 tokens 701, 670, 671, 676 us) and 238, 212, 194, 194 us from an e4m3 one,
// whose q is split for every item.  With few rows a tile is bound by HBM and hides
// the next item's beginning (0 and 1 measured the same).
constexpr int kItemCostMany = 2, kItemCostManyF8 = 3, kItemCostFew = 0;

// Everything that the attention kernels are told.
struct AttnParams {
  int R, N, H, Hkv, G;     // requests, packed rows, heads, kv heads, heads per kv head
  int page, page_shift, P, max_pages;
  int max_q;               // longest allowed range
  int tp;                  // query tokens of an item
  float c;                 // scale * log2(e)
  const __nv_bfloat16 *q;
  const uint8_t *k_scale, *v_scale;
  const int32_t *table, *kv_len, *q_start;
  __nv_bfloat16 *o;
  uint32_t *dev_status;
  // workspace: the item that begins in CTA c and goes on behind it, if any
  // (first row, kv head, tokens, last CTA); per CTA two partial results
  // (0: an item begun before the CTA, 1: one that goes on behind it)
  int4 *desc;              // [CTAs]
  int *skip;               // [CTAs, 2, row tile]: rows 128 w .. of the piece met a bad page (few rows: w = 0 alone)
  float2 *ml;              // [CTAs, 2, rows]: maximum (log2 units) and sum
  float *part;             // [CTAs, 2, rows x D], in the order that the merge reads
};

struct Req {
  int s0, q_len, pos0, len, ntile;
  bool ok;
};

__device__ __forceinline__ Req load_req(const AttnParams &p, int r) {
  Req x;
  const int s0 = p.q_start[r], s1 = p.q_start[r + 1];
  x.len = p.kv_len[r];
  x.ok = request_ok(s0, s1, x.len, p.N, (long long)p.max_pages * p.page) && s1 - s0 <= p.max_q;
  x.s0 = s0;
  x.q_len = x.ok ? s1 - s0 : 0;
  x.pos0 = x.len - x.q_len;
  x.ntile = x.q_len > 0 ? (x.q_len - 1) / p.tp + 1 : 0;
  return x;
}

// Units of token tile t: the cache tiles up to its last token's position.
__device__ __forceinline__ int tile_units(int tp, int pos0, int q_len, int t) {
  const long long end = (long long)(t + 1) * tp;
  const long long vis = pos0 + (end < q_len ? end : (long long)q_len);
  return vis <= kTileKeys ? 1 : (int)((vis + kTileKeys - 1) / kTileKeys);
}

// Sum of floor((a i + b) / 128) over i in [0, n), 128 being the keys of a cache tile: the
// sum of all a i + b less that of their remainders, over 128.  The remainders repeat
// every q = 128 / g steps, g the largest power of two in a (128 at most): a whole
// period meets each of b mod g, b mod g + g, .. once, and what is left of the last period
// (127 steps at most) is added up, four remainders at a time in the bytes of a word.
// n < 2^24, a and b below 2^31: sums stay below 2^63.
__host__ __device__ inline long long tiles_sum(unsigned n, unsigned a, unsigned b) {
  static_assert(kTileKeys == 128, "remainders of 7 bits");
  const unsigned low = a & 127u, g = low ? low & (0u - low) : 128u, q = 128u / g;
  const long long periods = n / q;
  long long rest = periods * (q * (b & (g - 1u)) + g * (q * (q - 1u) / 2u));
  const unsigned m = n % q;
  unsigned x = (b + 3u * low & 127u) << 24 | (b + 2u * low & 127u) << 16 | (b + low & 127u) << 8 | (b & 127u);
  const unsigned step = (4u * low & 127u) * 0x01010101u;
  unsigned even = 0, odd = 0;  // two sums each, 32 terms below 2^7
  unsigned i = 0;
  for (; i + 4u <= m; i += 4u) {
    even += x & 0x00ff00ffu;
    odd += x >> 8 & 0x00ff00ffu;
    x = x + step & 0x7f7f7f7fu;
  }
  for (; i < m; ++i, x >>= 8) rest += x & 0x7fu;
  rest += (even & 0xffffu) + (even >> 16) + (odd & 0xffffu) + (odd >> 16);
  const long long pairs = (long long)n * ((long long)n - 1) / 2;
  return (pairs * a + (long long)n * b - rest) / kTileKeys;
}

// a / b for non-negative numbers, in 32 bits where they fit (a 64-bit division
// costs a few hundred cycles of the planning step).
__device__ __forceinline__ long long div_pos(long long a, long long b) {
  return ((unsigned long long)(a | b) >> 32) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

// Units and the items' own cost of the tiles before tile t (t = ntile: of one
// kv head of the request).  Not inlined: the planning code runs once per CTA, and
// what it costs is mostly the fetching of its instructions.
static __device__ __noinline__ long long units_before(int tp, int cost, int pos0, int q_len, int ntile, int t) {
  long long s = (long long)t * cost;
  int n = t;
  if (t == ntile && t > 0) {  // the last tile may be a short one
    s += tile_units(tp, pos0, q_len, t - 1);
    n = t - 1;
  }
  if (n <= 0) return s;
  const long long room = (long long)kTileKeys - pos0;  // tiles that end within the first cache tile: one unit
  const int z = room < tp ? 0 : (int)min((long long)n, div_pos(room, tp));
  s += z;
  // the tiles are of more than 128 rows, and a call has at most 2^30 rows: n < 2^24
  if (n > z) s += tiles_sum((unsigned)(n - z), (unsigned)tp, (unsigned)(pos0 + (long long)(z + 1) * tp + kTileKeys - 1));
  return s;
}

struct Plan {
  long long u0, u1, per;  // this CTA's units; units of a CTA
  int r;                  // request of u0
  long long off;          // u0's offset in that request
  long long per_head;     // units of one kv head of that request
};

// Shared memory of the planning step.
struct PlanShared {
  long long scan[16];
  long long first_off, first_per_head;
  int first_r;
};

// Called by the whole CTA (blockDim a multiple of 32, at most 512); kOneTile:
// p.tp covers any range, so that a request has one tile.
template <bool kOneTile, int kCost>
__device__ inline Plan make_plan(const AttnParams &p, PlanShared *sh) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
  auto head_units = [&](int r) -> long long {  // of one kv head of request r
    if (r >= p.R) return 0;
    const Req x = load_req(p, r);
    if (!x.ok && blockIdx.x == 0 && p.dev_status) atomicOr(p.dev_status, GLINATTN_DEV_BAD_COUNT);
    if (x.ntile == 0) return 0;
    return kOneTile ? kCost + tile_units(p.tp, x.pos0, x.q_len, 0)
                    : units_before(p.tp, kCost, x.pos0, x.q_len, x.ntile, x.ntile);
  };
  Plan pl;
  pl.r = 0;
  pl.per = pl.u0 = pl.u1 = pl.off = pl.per_head = 0;
  // more requests than threads: their total first
  const bool one_chunk = p.R <= nt;
  long long total = 0;
  if (!one_chunk) {
    for (int r = tid; r < p.R; r += nt) total += head_units(r);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane == 0) sh->scan[warp] = total;
    __syncthreads();
    total = 0;
    for (int w = 0; w < nw; ++w) total += sh->scan[w];
    total *= p.Hkv;
    __syncthreads();
  }
  // a scan of nt requests at a time, up to the one that holds the CTA's first unit
  long long before = 0;
  for (int base = 0;; base += nt) {
    const long long head = head_units(base + tid), u = head * p.Hkv;
    long long upto = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) sh->scan[warp] = upto;
    __syncthreads();
    long long all = 0;
    for (int w = 0; w < nw; ++w) {
      if (w < warp) upto += sh->scan[w];
      all += sh->scan[w];
    }
    if (base == 0) {
      if (one_chunk) total = all;
      pl.per = max(1ll, div_pos(total + gridDim.x - 1, gridDim.x));
      pl.u0 = min((long long)blockIdx.x * pl.per, total);
      pl.u1 = min(pl.u0 + pl.per, total);
      if (pl.u0 >= pl.u1) return pl;  // the same in all threads
    }
    const long long a = before + upto - u;
    if (a <= pl.u0 && pl.u0 < a + u) {
      sh->first_r = base + tid;
      sh->first_off = pl.u0 - a;
      sh->first_per_head = head;
    }
    __syncthreads();
    before += all;
    if (before > pl.u0 || base + nt >= p.R) break;
  }
  pl.r = sh->first_r;
  pl.off = sh->first_off;
  pl.per_head = sh->first_per_head;
  return pl;
}

// One item's share of this CTA, as the producer hands it to the other roles.
struct Item {
  int r, hk;
  int row0;      // first packed row of its tokens
  int ntok;      // tokens
  int pos0;      // position of the first token
  int j0, j1;    // cache tiles of this CTA
  int kind;      // 0: the whole item, 1: its beginning, 2: a later piece; -1: no more items
};

// The items of a CTA, in order (run by one warp, all lanes alike).
template <bool kOneTile, int kCost>
struct Walk {
  const AttnParams &p;
  Plan pl;
  Req x;
  int r, hk, t, off;      // off: units of the item that are before this CTA
  long long left, at;

  __device__ Walk(const AttnParams &p_, const Plan &pl_, int lane) : p(p_), pl(pl_) {
    left = pl.u1 - pl.u0;
    at = pl.u0;
    r = pl.r;
    hk = t = off = 0;
    if (left <= 0) return;
    x = load_req(p, r);
    hk = (int)div_pos(pl.off, pl.per_head);
    const long long y = pl.off - hk * pl.per_head;
    if (!kOneTile) {  // the last tile with units_before <= y, 32 ways at a time
      long long before = 0;
      for (int n = x.ntile; n > 1;) {
        const int step = (n + 31) >> 5;
        const long long u = units_before(p.tp, kCost, x.pos0, x.q_len, x.ntile, min(t + lane * step, x.ntile));
        const int k = 31 - __clz(__ballot_sync(0xffffffffu, lane == 0 || (lane * step < n && u <= y)));
        before = __shfl_sync(0xffffffffu, u, k);
        t += k * step;
        n = min(step, n - k * step);
      }
      off = (int)(y - before);
    } else {
      off = (int)y;
    }
  }

  // The next item with cache tiles in this CTA; false when there is none.
  __device__ bool next(Item &it, int lane) {
    if (left <= 0) return false;
    const int units = kCost + tile_units(p.tp, x.pos0, x.q_len, t);
    const int take = (int)min((long long)(units - off), left);
    it.r = r;
    it.hk = hk;
    const int tok0 = kOneTile ? 0 : t * p.tp;
    it.row0 = x.s0 + tok0;
    it.ntok = kOneTile ? x.q_len : min(p.tp, x.q_len - tok0);
    it.pos0 = x.pos0 + tok0;
    it.j0 = max(0, off - kCost);
    it.j1 = max(0, off + take - kCost);
    if (it.j1 == 0) return false;  // only the item's own cost: it begins in the next CTA
    it.kind = it.j0 > 0 ? 2 : it.j1 == units - kCost ? 0 : 1;
    if (it.kind == 1 && lane == 0)
      p.desc[blockIdx.x] = make_int4(it.row0, hk, it.ntok, (int)div_pos(at - off + units - 1, pl.per));
    left -= take;
    at += take;
    off = 0;
    if (left > 0) {
      if (++t >= x.ntile) {
        t = 0;
        if (++hk >= p.Hkv) {
          hk = 0;
          do {
            if (++r >= p.R) {  // only when the lengths changed under the call
              left = 0;
              return true;
            }
            x = load_req(p, r);
          } while (x.ntile == 0);
        }
      }
    }
    return true;
  }
};

// A running (maximum, sum, outputs) triple of one row, kE channels a lane.
template <int kE>
struct Partial {
  float m = -INFINITY, l = 0.f, o[kE] = {};
  // Adds a piece; one without weight adds nothing, whatever its outputs hold.  The
  // maxima of an e4m3 cache hold its values' scales, which the sums do not: a sum may
  // be far above 1 and a factor below fp32's range, so it is applied in two halves.
  __device__ __forceinline__ void add(float pm, float pl, const float (&x)[kE]) {
    const float mn = fmaxf(m, pm), ms = mn == -INFINITY ? 0.f : mn;
    const float f2 = exp2f(0.5f * (m - ms)), g2 = exp2f(0.5f * (pm - ms)), f = f2 * f2, g = g2 * g2;
    l = l * f2 * f2 + (pm == -INFINITY ? 0.f : pl * g2 * g2);
#pragma unroll
    for (int e = 0; e < kE; ++e) o[e] = o[e] * f + (pm == -INFINITY ? 0.f : x[e] * g);
    m = mn;
  }
};

// Whether row tile w of a piece of the item that begins in CTA c0 met a bad page (whole CTA).
__device__ __forceinline__ bool any_bad(const AttnParams &p, int c0, int c1, int w) {
  int bad = 0;
  for (int c = c0 + (int)threadIdx.x; c <= c1; c += (int)blockDim.x) bad |= p.skip[2 * (2 * c + (c == c0 ? 1 : 0)) + w];
  return __syncthreads_or(bad) != 0;
}

// Joins the pieces of the item that begins in CTA blockIdx.x and goes on
// behind it, with few rows and possibly many pieces: blockIdx.y = its row, 8
// warps share the pieces, a lane holds D / 32 channels.  Bound by latency, a few
// L2 reads per piece.  Partial outputs are [row][channel].
template <int D, int kRows>
__global__ void __launch_bounds__(256) merge_few_rows_kernel(const AttnParams p) {
  constexpr int kE = D / 32;
  __shared__ float s_m[8], s_l[8], s_o[8][D];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c0 = blockIdx.x, row = blockIdx.y;
  const int4 d = p.desc[c0];
  if (d.w < 0 || row >= d.z * p.G) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto piece = [&](int c, float (&x)[kE]) -> float2 {
    const size_t at = (size_t)(2 * c + (c == c0 ? 1 : 0)) * kRows + row;
#pragma unroll
    for (int e = 0; e < kE; ++e) x[e] = p.part[at * D + lane * kE + e];
    return p.ml[at];
  };
  // the warp's first piece is read beside the flags
  float first[kE];
  float2 fml = make_float2(-INFINITY, 0.f);
  if (c0 + warp <= d.w) fml = piece(c0 + warp, first);
  if (any_bad(p, c0, d.w, 0)) return;
  Partial<kE> a;
  if (c0 + warp <= d.w) a.add(fml.x, fml.y, first);
#pragma unroll 4
  for (int c = c0 + warp + 8; c <= d.w; c += 8) {
    float x[kE];
    const float2 ml = piece(c, x);
    a.add(ml.x, ml.y, x);
  }
  if (lane == 0) {
    s_m[warp] = a.m;
    s_l[warp] = a.l;
  }
#pragma unroll
  for (int e = 0; e < kE; ++e) s_o[warp][lane * kE + e] = a.o[e];
  __syncthreads();
  if (threadIdx.x < D) {
    Partial<1> b;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const float x[1] = {s_o[w][threadIdx.x]};
      b.add(s_m[w], s_l[w], x);
    }
    const int tok = row / p.G, g = row - tok * p.G;
    p.o[((size_t)(d.x + tok) * p.H + d.y * p.G + g) * D + threadIdx.x] = __float2bfloat16_rn(b.l == 0.f ? 0.f : b.o[0] / b.l);
  }
}

// The same with many rows and mostly two pieces: 32 rows per CTA (blockIdx.y),
// lane = row, warp w the D / 8 channels from w D / 8.  Partial outputs are
// [channel / 4][row][4], so that the lanes' reads (and the attention kernel's
// writes, a row per lane there too) are contiguous.
template <int D, int kRows>
__global__ void __launch_bounds__(256) merge_many_rows_kernel(const AttnParams p) {
  constexpr int kE = D / 8;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c0 = blockIdx.x;
  const int4 d = p.desc[c0];
  const int nrow = d.z * p.G;
  if (d.w < 0 || (int)blockIdx.y * 32 >= nrow) return;
  const int row = blockIdx.y * 32 + (threadIdx.x & 31), warp = threadIdx.x >> 5;
  auto piece = [&](int c, float (&x)[kE]) -> float2 {
    const size_t slot = (size_t)(2 * c + (c == c0 ? 1 : 0));
    const float4 *src = reinterpret_cast<const float4 *>(p.part) + (slot * (D / 4) + warp * (kE / 4)) * kRows + row;
#pragma unroll
    for (int k = 0; k < kE / 4; ++k) {
      const float4 v = src[k * kRows];
      x[4 * k] = v.x, x[4 * k + 1] = v.y, x[4 * k + 2] = v.z, x[4 * k + 3] = v.w;
    }
    return p.ml[slot * kRows + row];
  };
  // the first two pieces (there are two at least) are read beside the flags
  float x0[kE], x1[kE];
  float2 ml0, ml1;
  if (row < nrow) {
    ml0 = piece(c0, x0);
    ml1 = piece(c0 + 1, x1);
  }
  if (any_bad(p, c0, d.w, blockIdx.y / 4) || row >= nrow) return;
  Partial<kE> a;
  a.add(ml0.x, ml0.y, x0);
  a.add(ml1.x, ml1.y, x1);
  for (int c = c0 + 2; c <= d.w; ++c) {
    const float2 ml = piece(c, x0);
    a.add(ml.x, ml.y, x0);
  }
  const int tok = row / p.G, g = row - tok * p.G;
  uint4 *o = reinterpret_cast<uint4 *>(p.o + ((size_t)(d.x + tok) * p.H + d.y * p.G + g) * D + warp * kE);
  const float inv = a.l == 0.f ? 0.f : 1.f / a.l;
#pragma unroll
  for (int e = 0; e < kE; e += 8) {
    uint32_t u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) u[k] = a.l == 0.f ? 0u : pack_bf16(a.o[e + 2 * k] * inv, a.o[e + 2 * k + 1] * inv);
    o[e / 8] = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

// The merge, launched so that it is in place when the attention kernel ends.
template <int D, int kRows, bool kFewRows>
cudaError_t launch_merge(const AttnParams &p, int ctas, cudaStream_t stream) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  // rows that an item can have, however many there is room for
  const int rows = (int)max(1ll, min((long long)kRows, (long long)min(p.max_q, p.tp) * p.G));
  cfg.gridDim = dim3((unsigned)ctas, (unsigned)(kFewRows ? rows : (rows + 31) / 32), 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if constexpr (kFewRows)
    return cudaLaunchKernelEx(&cfg, merge_few_rows_kernel<D, kRows>, p);
  else
    return cudaLaunchKernelEx(&cfg, merge_many_rows_kernel<D, kRows>, p);
}

// Few rows: items of at most 16 query rows (tokens x heads of a group), with an
// e4m3 cache also 32 or 48.
cudaError_t launch_decode(const AttnParams &p, bool f8, int d, int rows, const void *k_cache, const void *v_cache,
                          int ctas, cudaStream_t stream);

// more of them: items of kPrefillRows / G tokens
constexpr int kPrefillRows = 256;
cudaError_t launch_prefill(const AttnParams &p, bool f8, int d, const void *k_cache, const void *v_cache, int ctas,
                           cudaStream_t stream);

}  // namespace paged
}  // namespace glinattn
