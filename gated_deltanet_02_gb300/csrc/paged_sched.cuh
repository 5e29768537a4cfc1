// paged_sched.cuh -- how the attention kernels share their work out, and the
// merge of partial results.
//
// The work of a call is a row of units, one unit being the 128 keys of one
// cache tile for one item; an item is (request, key / value head, tile of query
// tokens), and its units are the cache tiles that its last token sees (one at
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
  int *skip;               // [CTAs, 2]: the piece met a bad page
  float2 *ml;              // [CTAs, 2, rows]: maximum (log2 units) and sum
  float *part;             // [CTAs, 2, rows, D]
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
__device__ __forceinline__ int tile_units(const AttnParams &p, const Req &x, int t) {
  const long long end = (long long)(t + 1) * p.tp;
  const long long vis = x.pos0 + (end < x.q_len ? end : (long long)x.q_len);
  return vis <= kTileKeys ? 1 : (int)((vis + kTileKeys - 1) / kTileKeys);
}

// sum of floor((a i + b) / m) over i in [0, n), by the Euclidean recursion.
__device__ inline long long floor_sum(long long n, unsigned m, unsigned a, unsigned b) {
  long long s = 0;
  while (true) {
    if (a >= m) {
      s += n * (n - 1) / 2 * (a / m);
      a %= m;
    }
    if (b >= m) {
      s += n * (b / m);
      b %= m;
    }
    const unsigned long long y = (unsigned long long)a * (unsigned long long)n + b;
    if (y < m) return s;
    n = (long long)(y / m);
    b = (unsigned)(y % m);
    const unsigned x = m;
    m = a;
    a = x;
  }
}

// Units of the tiles before tile t (t = ntile: of one kv head of the request).
__device__ inline long long units_before(const AttnParams &p, const Req &x, int t) {
  long long s = 0;
  int n = t;
  if (t == x.ntile && t > 0) {
    s = tile_units(p, x, t - 1);  // the last tile may be a short one
    n = t - 1;
  }
  if (n <= 0) return s;
  const long long room = (long long)kTileKeys - x.pos0;  // tiles that end within the first cache tile: one unit
  const int z = room < p.tp ? 0 : (int)min((long long)n, room / p.tp);
  s += z;
  if (n > z) s += floor_sum(n - z, kTileKeys, (unsigned)p.tp, (unsigned)(x.pos0 + (long long)(z + 1) * p.tp + kTileKeys - 1));
  return s;
}

struct Plan {
  long long u0, u1, per;  // this CTA's units; units of a CTA
  int r;                  // request of u0
  long long off;          // u0's offset in that request
};

// Shared memory of the planning step.
struct PlanShared {
  long long scan[32];
  long long first_off;
  int first_r;
};

// Called by the whole CTA (blockDim a multiple of 32); kOneTile: p.tp covers
// any range, so that a request has one tile.
template <bool kOneTile>
__device__ inline Plan make_plan(const AttnParams &p, PlanShared *sh) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
  auto units = [&](int r, bool flag) -> long long {
    if (r >= p.R) return 0;
    const Req x = load_req(p, r);
    if (!x.ok) {
      if (flag && p.dev_status) atomicOr(p.dev_status, GLINATTN_DEV_BAD_COUNT);
      return 0;
    }
    if (x.ntile == 0) return 0;
    return (long long)p.Hkv * (kOneTile ? (long long)tile_units(p, x, 0) : units_before(p, x, x.ntile));
  };
  long long mine = 0;
  for (int r = tid; r < p.R; r += nt) mine += units(r, blockIdx.x == 0);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) sh->scan[warp] = mine;
  __syncthreads();
  long long total = 0;
  for (int w = 0; w < nw; ++w) total += sh->scan[w];
  __syncthreads();
  Plan pl;
  pl.per = max(1ll, (total + gridDim.x - 1) / gridDim.x);
  pl.u0 = min((long long)blockIdx.x * pl.per, total);
  pl.u1 = min(pl.u0 + pl.per, total);
  pl.r = 0;
  pl.off = 0;
  if (pl.u0 >= pl.u1) return pl;
  long long before = 0;
  for (int base = 0; base < p.R; base += nt) {
    const long long u = units(base + tid, false);
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
    const long long a = before + upto - u;
    if (a <= pl.u0 && pl.u0 < a + u) {
      sh->first_r = base + tid;
      sh->first_off = pl.u0 - a;
    }
    before += all;
    __syncthreads();
    if (before > pl.u0) break;
  }
  pl.r = sh->first_r;
  pl.off = sh->first_off;
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
template <bool kOneTile>
struct Walk {
  const AttnParams &p;
  Plan pl;
  Req x;
  int r, hk, t, off;
  long long left, at;

  __device__ Walk(const AttnParams &p_, const Plan &pl_, int lane) : p(p_), pl(pl_) {
    left = pl.u1 - pl.u0;
    at = pl.u0;
    r = pl.r;
    hk = t = off = 0;
    if (left <= 0) return;
    x = load_req(p, r);
    const long long per_head = kOneTile ? tile_units(p, x, 0) : units_before(p, x, x.ntile);
    hk = (int)(pl.off / per_head);
    const long long y = pl.off - hk * per_head;
    if (!kOneTile) {  // the last tile with units_before <= y, 32 ways at a time
      int lo = 0, n = x.ntile;
      while (n > 1) {
        const int step = (n + 31) >> 5;
        const bool le = lane == 0 || (lane * step < n && units_before(p, x, lo + lane * step) <= y);
        const int k = 31 - __clz(__ballot_sync(0xffffffffu, le));
        lo += k * step;
        n = min(step, n - k * step);
      }
      t = lo;
      off = (int)(y - units_before(p, x, t));
    } else {
      off = (int)y;
    }
  }

  // The next item; false when the CTA's units are used up.
  __device__ bool next(Item &it, int lane) {
    if (left <= 0) return false;
    const int units = tile_units(p, x, t);
    const int take = (int)min((long long)(units - off), left);
    it.r = r;
    it.hk = hk;
    const int tok0 = kOneTile ? 0 : t * p.tp;
    it.row0 = x.s0 + tok0;
    it.ntok = kOneTile ? x.q_len : min(p.tp, x.q_len - tok0);
    it.pos0 = x.pos0 + tok0;
    it.j0 = off;
    it.j1 = off + take;
    it.kind = off > 0 ? 2 : take == units ? 0 : 1;
    if (it.kind == 1 && lane == 0)
      p.desc[blockIdx.x] = make_int4(it.row0, hk, it.ntok, (int)((at + units - 1) / pl.per));
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
  // Adds a piece; one without weight adds nothing, whatever its outputs hold.
  __device__ __forceinline__ void add(float pm, float pl, const float (&x)[kE]) {
    const float mn = fmaxf(m, pm), ms = mn == -INFINITY ? 0.f : mn;
    const float f = exp2f(m - ms), g = exp2f(pm - ms);
    l = l * f + (pm == -INFINITY ? 0.f : pl * g);
#pragma unroll
    for (int e = 0; e < kE; ++e) o[e] = o[e] * f + (pm == -INFINITY ? 0.f : x[e] * g);
    m = mn;
  }
};

// Joins the pieces of the item that begins in CTA blockIdx.x and goes on
// behind it, kRowsPerCta rows per CTA (blockIdx.y); a lane holds D / 32
// channels.  Bound by latency, a few L2 reads per piece: with few pieces a
// warp takes a row, with many the 8 warps share the pieces of one row at a time.
template <int D, int kRows, int kRowsPerCta>
__global__ void __launch_bounds__(256) merge_kernel(const AttnParams p) {
  constexpr int kE = D / 32;
  __shared__ float s_m[8], s_l[8], s_o[8][D];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c0 = blockIdx.x;
  const int4 d = p.desc[c0];
  const int nrow = d.z * p.G, row0 = blockIdx.y * kRowsPerCta;
  if (d.w < 0 || row0 >= nrow) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int bad = 0;
  for (int c = c0 + (int)threadIdx.x; c <= d.w; c += 256) bad |= p.skip[2 * c + (c == c0 ? 1 : 0)];
  if (__syncthreads_or(bad)) return;
  auto pieces = [&](int row, int first, int step, Partial<kE> &a) {
#pragma unroll 4
    for (int c = c0 + first; c <= d.w; c += step) {
      const size_t at = (size_t)(2 * c + (c == c0 ? 1 : 0)) * kRows + row;
      const float2 ml = p.ml[at];
      float x[kE];
      if constexpr (kE == 4) {
        const float4 v = *reinterpret_cast<const float4 *>(p.part + at * D + lane * 4);
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
      } else {
        const float2 v = *reinterpret_cast<const float2 *>(p.part + at * D + lane * 2);
        x[0] = v.x, x[1] = v.y;
      }
      a.add(ml.x, ml.y, x);
    }
  };
  auto out = [&](int row) {
    const int tok = row / p.G, g = row - tok * p.G;
    return p.o + ((size_t)(d.x + tok) * p.H + d.y * p.G + g) * D;
  };
  if (kRowsPerCta == 8 && d.w - c0 < 8) {
    const int row = row0 + warp;
    if (row >= nrow) return;
    Partial<kE> a;
    pieces(row, 0, 1, a);
    __nv_bfloat16 *o = out(row) + lane * kE;
#pragma unroll
    for (int e = 0; e < kE; e += 2)
      *reinterpret_cast<uint32_t *>(o + e) = a.l == 0.f ? 0u : pack_bf16(a.o[e] / a.l, a.o[e + 1] / a.l);
    return;
  }
  for (int row = row0; row < min(row0 + kRowsPerCta, nrow); ++row) {
    Partial<kE> a;
    pieces(row, warp, 8, a);
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
      out(row)[threadIdx.x] = __float2bfloat16_rn(b.l == 0.f ? 0.f : b.o[0] / b.l);
    }
    __syncthreads();
  }
}

// The merge, launched so that it is in place when the attention kernel ends.
template <int D, int kRows, int kRowsPerCta>
cudaError_t launch_merge(const AttnParams &p, int ctas, cudaStream_t stream) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas, kRows / kRowsPerCta, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, merge_kernel<D, kRows, kRowsPerCta>, p);
}

// rows <= kDecodeRows query rows (tokens x heads of a group) per item
constexpr int kDecodeRows = 32;
cudaError_t launch_decode(const AttnParams &p, bool f8, int d, int rows, const void *k_cache, const void *v_cache,
                          int ctas, cudaStream_t stream);

// more of them: items of kPrefillRows / G tokens
constexpr int kPrefillRows = 256;
cudaError_t launch_prefill(const AttnParams &p, bool f8, int d, const void *k_cache, const void *v_cache, int ctas,
                           cudaStream_t stream);

}  // namespace paged
}  // namespace glinattn
