// paged_decode.cu -- attention over the paged cache for few query rows per
// (request, key / value head): single tokens and drafts (glinattn_paged_attention).
//
// Mathematics: one pass over the keys with the running maximum m of the
// softmax (log2 units), in the transposed form
//   S^T = K Q^T   [128 keys x rows],   W = 2^(S^T - m),   O^T += V^T W   [d x rows]
// so that the 128-wide side of the tensor-core tile is filled by keys and
// channels and the few query rows (tokens x heads of the group) are the N side.  m only
// moves when a tile exceeds it by 2^kSlack (then O^T and the sums are
// rescaled), which leaves the result unchanged: m is a common factor.
//
// Precision: scores, m, sums and O^T are fp32.  The weights enter the second
// product as two bf16 parts (together 2^-16 relative), with an e4m3 cache as three
// e5m2 parts: 2^-9 of the weight, half of what rounding it to bf16 would do, and
// 2^-33 of the largest weight times value scale of the row (two e4m3 parts end at 2^-18,
// and 32,000 keys below that under one dominating key moved an output by 0.11).
// With an e4m3 cache both products run on the stored values
// (kind::f8f6f4): q is split into two e4m3 parts of 4 bits (bf16 has 8) with a
// power-of-two scale per row, exact but for elements below 2^-9 of the row's
// largest, where a step is 2^-16 of it; the key's scale multiplies its score, and
// the value's scale 2^e is folded into the weight's exponent: W = 2^(S + e - m)
// with m the maximum of S + e.  The sums hold 2^(S - m), between 2^-119 and 2^104 a
// key for the exponents that a cache can have.
//
// Bound: HBM, one read of the cache; 2 CTAs per SM, each with a ring of 16 KiB
// stages (TMA, one box per page), so that about 190 KiB per SM are in flight (128 KiB
// with 48 rows, where 160 measured the same).  Warps:
// 0 TMA and the walk over the items, 1 MMA issue, then groups of four softmax
// warps, a key per thread and 16 rows per group (24 rows per group, fewer warps
// that repeat a tile's fixed cost, were 17% slower for 40 rows of e4m3).  With many
// rows the softmax's instructions count beside the bytes: items are read from shared
// memory where they are needed, for with 48 rows a thread has 72 registers (kept in
// registers they cost 64 requests of 40 rows after 32,768 tokens 15%).
//
// 256 single tokens after 1,000 .. 6,000, 16 heads over 4 of 128, bf16: 283-287 us,
// 6,600 GB/s; the 40 rows above, e4m3: 445 us, 4,700 GB/s (382 us with weights in two
// parts and sums that could lose keys); 4 single tokens: 11 us, launches and latency.
#include "paged_sched.cuh"
#include "paged_tc.cuh"
#include "tc_common.cuh"

namespace glinattn {
namespace paged {
namespace {

using namespace sm100;
using tc::wait_bar;
using tc::wait_bar_warp;
using tc::warp_arrive;

constexpr int kItems = 4;              // depth of the item queue
constexpr int kScaleSlots = 12;        // tiles of scales in flight, see ScaleRing below
constexpr uint32_t kStageBytes = 16384;

template <int D, bool kF8, int N>
struct Cfg {
  static constexpr int kTQ = kF8 ? 2 : 1;            // parts of q
  static constexpr int kTP = kF8 ? 3 : 2;            // parts of a weight
  static constexpr int kNO = N * kTP;                // columns of O^T (S^T has N)
  static constexpr int kEsz = kF8 ? 1 : 2;
  static constexpr int kTileStages = D * kEsz * kTileKeys > (int)kStageBytes ? 2 : 1;
  static constexpr int kRows = 16;                   // rows of a softmax group of four warps
  static constexpr int kGroups = N / kRows;
  static constexpr int kThreads = 64 + 128 * kGroups;
  static constexpr uint32_t kBytesQ = N * kTQ * D * kEsz;
  static constexpr uint32_t kBytesP = N * kTP * kTileKeys * kEsz;
  static constexpr uint32_t kBytesScale = kF8 ? kScaleSlots * 2 * kTileKeys : 0;
  static constexpr uint32_t kBytesRows = 4 * N * 4 + 5 * N * 4;  // [row][warp] maxima or sums, then five numbers a row
  static constexpr uint32_t kBytesBars = 640;
  static constexpr uint32_t kFixed = kBytesQ + kBytesP + kBytesScale + kBytesRows + kBytesBars + 1024;
  // two CTAs of an SM share 228 KiB, 1 KiB of each reserved
  static constexpr int kFit = (int)((112 * 1024 - kFixed) / kStageBytes);
  static constexpr int kStages = kFit < 6 ? kFit : 6;
  static constexpr uint32_t kSmem = kFixed + kStages * kStageBytes;
  static constexpr uint32_t kOffQ = kStages * kStageBytes, kOffP = kOffQ + kBytesQ, kOffScale = kOffP + kBytesP,
                            kOffRows = kOffScale + kBytesScale, kOffBars = kOffRows + kBytesRows;
  static constexpr uint32_t kColO = 2 * N;
  static constexpr uint32_t kCols = kColO + kNO <= 64 ? 64 : kColO + kNO <= 128 ? 128 : 256;
  static_assert(kColO + kNO <= 256, "two CTAs share the SM's 512 columns");
  static_assert(kStages >= 2 * kTileStages, "K and V tiles of one step");
  // the first tile index whose scales the producer may be loading is that of
  // the oldest unread tile + 1 (its S issued early) + the ring's K tiles
  static_assert(!kF8 || kScaleSlots >= kStages + 3, "scale slots");
};

struct Bars {
  uint64_t full[6], empty[6];
  uint64_t s_ready[2], s_free[2], q_ready, p_ready, o_done;
  uint64_t item_full[kItems], item_empty[kItems];
  Item item[kItems];
  PlanShared plan;
  uint64_t sync[3];  // the four warps of a softmax group among themselves
  uint32_t tmem;
  int abort;
};

__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Two weights of at most 2^15 as three e5m2 parts each, the second times 4, the third
// times 32.  e5m2 is the upper byte of f16: the first two parts are cut off the weight's
// f16 (parts 0 and 1: bytes 1 and 3), the third is what is left, rounded (bytes 0 and 1).  Off by
// 2^-9 of the weight's leading power (3 bits a part; 2^-12 for the f16), or by 2^-22
// where that is more (half the smallest e5m2, over 32).
__device__ __forceinline__ void split_e5m2x2(float w0, float w1, uint32_t (&part)[3]) {
  constexpr uint32_t kUp[2] = {0x44004400u, 0x48004800u};  // 4, 8
  uint32_t x;
  unsigned short e;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(x) : "f"(w1), "f"(w0));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    part[i] = x;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(x) : "r"(x), "r"(x & 0xff00ff00u));
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(x) : "r"(x), "r"(kUp[i]));
  }
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(e) : "r"(x));
  part[2] = e;
}

// 16 columns from a of this thread's lane, times f[0 ..] (shared memory) twice.
__device__ __forceinline__ void tmem_scale16(uint32_t a, const float *f) {
  float t[16];
  tmem_ld16(a, t);
#pragma unroll
  for (int k = 0; k < 16; k += 8) {
    uint32_t u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = __float_as_uint(t[k + j] * f[k + j] * f[k + j]);
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(a + k), "r"(u[0]), "r"(u[1]),
                 "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                 : "memory");
  }
  tmem_wait_st();
}

template <int D, bool kF8, int N>
__global__ void __launch_bounds__(Cfg<D, kF8, N>::kThreads, 2)
    decode_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const AttnParams p) {
  using C = Cfg<D, kF8, N>;
  constexpr int ST = C::kStages, NS = C::kTileStages, W = C::kGroups, R = C::kRows;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Bars *bars = reinterpret_cast<Bars *>(smem + C::kOffBars);
  static_assert(sizeof(Bars) <= C::kBytesBars, "barrier block");
  __shared__ __align__(16) int s_flag[2][W][4];  // [tile parity][group][warp]: a row's maximum moves
  __shared__ int s_look[W];                      // 1: rows of the group have to be looked at in every tile, 2: huge scores in this one
  __shared__ int s_bad[kItems];
  volatile int *abort = &bars->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->s_ready[i], 1);
      mbar_init(&bars->s_free[i], 4 * W);
    }
    mbar_init(&bars->q_ready, 4 * W);
    mbar_init(&bars->p_ready, 4 * W);
    mbar_init(&bars->o_done, 1);
    for (int i = 0; i < W; ++i) mbar_init(&bars->sync[i], 4);
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&bars->item_full[i], 1);
      mbar_init(&bars->item_empty[i], 1 + 4 * W);
      s_bad[i] = 0;
    }
    bars->abort = 0;
    p.desc[blockIdx.x].w = -1;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem, C::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  const Plan plan = make_plan<true, kItemCostFew>(p, &bars->plan);  // has CTA barriers
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == 0) {
    // ============ the walk over the items, and TMA (a page per lane) ============
    Walk<true, kItemCostFew> walk(p, plan, lane);
    Item it;
    uint32_t sc = 0;                 // stages used so far
    uint32_t g = 0;                  // tiles so far
    const int pages = kTileKeys >> p.page_shift;  // pages of a tile
    bool ok = true;
    uint32_t slot = 0;
    if (lane == 0) {
      prefetch_tensormap(&tk);
      prefetch_tensormap(&tv);
    }
    while (ok) {
      const bool more = walk.next(it, lane);
      const int si = slot % kItems;
      if (!(ok = wait_bar_warp(&bars->item_empty[si], ((slot / kItems) & 1u) ^ 1u, abort))) break;
      if (!more) it.kind = -1;
      if (lane == 0) {
        bars->item[si] = it;
        s_bad[si] = 0;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->item_full[si]);
      ++slot;
      if (!more) break;
      const int npage = (int)(((long long)it.pos0 + it.ntok + p.page - 1) >> p.page_shift);  // pages of the request
      const int32_t *table = p.table + (size_t)it.r * p.max_pages;
      // ids of pages base + lane, and of the 32 behind them
      int base = it.j0 * pages;
      int ids = base + lane < npage ? table[base + lane] : 0;
      int ids_next = base + 32 + lane < npage ? table[base + 32 + lane] : 0;
      int vbase = base, vids = ids;  // the value tiles come one tile behind
      // One tile's loads.  K: [16-byte swizzled columns of 64][128 keys], a stage per
      // 64 bf16 columns; V: a stage per 64 keys when the tile has two stages.
      auto load = [&](int j, bool isv, int b0, int id_reg) -> bool {
        const int pg0 = j * pages, np = min(pages, npage - pg0);
        const int id = __shfl_sync(0xffffffffu, id_reg, (pg0 - b0) + (lane & (pages - 1)));
        const bool mine = (lane & (pages - 1)) < np;
        const bool good = id >= 0 && id < p.P;
        const unsigned bad = __ballot_sync(0xffffffffu, mine && !good);
        if (bad && lane == 0) s_bad[si] = 1;
        const int ngood = __popc(__ballot_sync(0xffffffffu, lane < np && good));
        const int pl = lane & (pages - 1);
        const int plane = id * p.Hkv + it.hk;
        const CUtensorMap *map = isv ? &tv : &tk;
        if constexpr (NS == 2) {
          // ops per page: 2 column blocks (x 2 key halves of a 128-key page for V)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t s = (sc + h) % ST;
            if (!wait_bar_warp(&bars->empty[s], (((sc + h) / ST) & 1u) ^ 1u, abort)) return false;
            uint8_t *dst = smem + s * kStageBytes;
            if (!isv) {
              if (lane == 0) mbar_arrive_expect_tx(&bars->full[s], (uint32_t)ngood << (p.page_shift + 7));
              __syncwarp();
              if (lane < np && good) tma_load_3d(dst + (pl << (p.page_shift + 7)), map, &bars->full[s], 64 * h, 0, plane);
            } else {
              // keys 64 h .. 64 h + 63: pages of this half (a page of 128 keys: its half)
              const int per = pages > 1 ? pages / 2 : 1;
              const bool in = pages > 1 ? (pl / per == h) : true;
              const int rows = min(p.page, 64);
              const int n = __popc(__ballot_sync(0xffffffffu, lane < np && good && in));
              if (lane == 0) mbar_arrive_expect_tx(&bars->full[s], (uint32_t)(n * rows) * 256u);
              __syncwarp();
              const int l2 = lane & 15, col = lane >> 4;  // lanes 16 .. 31: the second column block
              const int idv = __shfl_sync(0xffffffffu, id, l2 & (pages - 1));
              const bool goodv = idv >= 0 && idv < p.P;
              const int plv = l2 & (pages - 1);
              if (l2 < np && goodv && (pages > 1 ? plv / per == h : true))
                tma_load_3d(dst + col * 8192 + (pages > 1 ? (plv % per) << (p.page_shift + 7) : 0), map, &bars->full[s], 64 * col,
                            pages > 1 ? 0 : 64 * h, idv * p.Hkv + it.hk);
            }
          }
        } else {
          const uint32_t s = sc % ST;
          if (!wait_bar_warp(&bars->empty[s], ((sc / ST) & 1u) ^ 1u, abort)) return false;
          uint8_t *dst = smem + s * kStageBytes;
          constexpr int kRow = D * C::kEsz;  // bytes of a cached row
          const uint32_t bytes = (uint32_t)ngood * (uint32_t)p.page * (kRow + (kF8 && !isv ? 2 : 0));
          if (lane == 0) mbar_arrive_expect_tx(&bars->full[s], bytes);
          __syncwarp();
          if (lane < np && good) {
            tma_load_3d(dst + pl * p.page * kRow, map, &bars->full[s], 0, 0, plane);
            if (kF8 && !isv) {  // both scales travel with the keys
              uint8_t *ss = smem + C::kOffScale + (g % kScaleSlots) * 2 * kTileKeys + pl * p.page;
              bulk_load(ss, p.k_scale + (size_t)plane * p.page, (uint32_t)p.page, &bars->full[s]);
              bulk_load(ss + kTileKeys, p.v_scale + (size_t)plane * p.page, (uint32_t)p.page, &bars->full[s]);
            }
          }
        }
        sc += NS;
        return true;
      };
      for (int j = it.j0; j < it.j1 && ok; ++j) {
        if (j * pages >= base + 32) {
          base += 32;
          ids = ids_next;
          ids_next = base + 32 + lane < npage ? table[base + 32 + lane] : 0;
        }
        ok = load(j, false, base, ids);
        ++g;
        if (ok && j > it.j0) {
          ok = load(j - 1, true, vbase, vids);
        }
        vbase = base;
        vids = ids;
      }
      if (ok) ok = load(it.j1 - 1, true, vbase, vids);
    }
  } else if (warp == 1) {
    {
      // ============ MMA issue (one lane) ============
      constexpr uint32_t id_s = kF8 ? idesc_f8(128, N, false, false) : idesc_bf16(128, N, false, false);
      constexpr uint32_t id_o = kF8 ? idesc_f8(D, C::kNO, true, true, true) : idesc_bf16(D, C::kNO, true, true);
      constexpr uint32_t hi_r = kF8 && D == 64 ? desc_hi(512, kSw64) : desc_hi(1024, kSw128);  // K, V, q
      // weights: 16-byte units of consecutive rows (no swizzle, MN-major), a unit's 8 keys 16
      // bytes apart, 128 bytes between groups of 8 keys, 2048 between units
      constexpr uint32_t hi_w = desc_hi(2048, kSwNone);
      const bool leader = elect_one();
      const uint32_t sb = smem_u32(smem), q0 = desc_lo(sb + C::kOffQ, 16), p0 = desc_lo(sb + C::kOffP, 128);
      const uint32_t k0 = desc_lo(sb, 16), v0 = desc_lo(sb, 8192);
      uint32_t sc = 0, g = 0, slot = 0;
      auto issue_s = [&](uint32_t gi) -> bool {
        for (int h = 0; h < NS; ++h)
          if (!wait_bar_warp(&bars->full[(sc + h) % ST], ((sc + h) / ST) & 1u, abort)) return false;
        const uint32_t buf = gi & 1;
        if (!wait_bar_warp<false>(&bars->s_free[buf], ((gi >> 1) & 1u) ^ 1u, abort)) return false;
        tc_fence_after();
        const uint32_t d = tmem + buf * N;
        const uint32_t a0 = k0 + (sc % ST) * (kStageBytes >> 4), a1 = k0 + ((sc + 1) % ST) * (kStageBytes >> 4);
        if (leader) {
          if constexpr (!kF8) {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
              mma_ss<false>(d, (ks < 4 ? a0 : a1) + ((ks & 3) * 32 >> 4), hi_r, q0 + ((ks >> 2) * (N * 128) + (ks & 3) * 32 >> 4), hi_r, id_s,
                            ks > 0);
          } else {
            // both parts of q against the same keys
#pragma unroll
            for (int ks = 0; ks < 2 * (D / 32); ++ks) {
              const uint32_t k = ks % (D / 32) * 32;
              mma_ss<true>(d, a0 + (k >> 4), hi_r, q0 + (ks / (D / 32) * (N * D) + k >> 4), hi_r, id_s, ks > 0);
            }
          }
          umma_commit(&bars->s_ready[buf]);
          for (int h = 0; h < NS; ++h) umma_commit(&bars->empty[(sc + h) % ST]);
        }
        sc += NS;
        return true;
      };
      auto issue_o = [&](uint32_t gi, bool first) -> bool {
        if (!wait_bar_warp<false>(&bars->p_ready, gi & 1u, abort)) return false;
        for (int h = 0; h < NS; ++h)
          if (!wait_bar_warp(&bars->full[(sc + h) % ST], ((sc + h) / ST) & 1u, abort)) return false;
        tc_fence_after();
        const uint32_t d = tmem + C::kColO;
        const uint32_t a0 = v0 + (sc % ST) * (kStageBytes >> 4), a1 = v0 + ((sc + 1) % ST) * (kStageBytes >> 4);
        if (leader) {
          if constexpr (!kF8) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              mma_ss<false>(d, (NS == 1 || ks < 4 ? a0 : a1) + ((NS == 1 ? ks : ks & 3) * 2048 >> 4), hi_r, p0 + (ks * 256 >> 4), hi_w,
                            id_o, ks > 0 || !first);
          } else {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_ss<true>(d, a0 + (ks * (32 * D) >> 4), hi_r, p0 + (ks * 512 >> 4), hi_w, id_o, ks > 0 || !first);
          }
          umma_commit(&bars->o_done);
          for (int h = 0; h < NS; ++h) umma_commit(&bars->empty[(sc + h) % ST]);
        }
        sc += NS;
        return true;
      };
      for (bool ok = true; ok;) {
        const int si = slot % kItems;
        if (!wait_bar_warp(&bars->item_full[si], (slot / kItems) & 1u, abort)) break;
        const int kind = bars->item[si].kind, n = bars->item[si].j1 - bars->item[si].j0;
        warp_arrive(&bars->item_empty[si]);
        if (kind < 0) break;
        if (!wait_bar_warp(&bars->q_ready, slot & 1u, abort)) break;
        ++slot;
        for (int j = 0; j < n && ok; ++j) {
          ok = issue_s(g + j);
          if (ok && j > 0) ok = issue_o(g + j - 1, j == 1);
        }
        if (ok) ok = issue_o(g + n - 1, n == 1);
        g += n;
      }
    }
  } else {
    // ============ softmax: thread = key, group w = rows R w .. R w + R - 1 ============
    const int w = (warp - 2) >> 2, q4 = warp & 3, kk = 32 * q4 + lane;
    const int st = tid - 64 - 128 * w;               // 0 .. 127
    const int rb = R * w;                            // the group's first row
    const uint32_t lane_base = (uint32_t)(32 * q4) << 16;
    const uint32_t sb = smem_u32(smem);
    float *s_red = reinterpret_cast<float *>(smem + C::kOffRows) + 4 * rb;  // [row][warp]
    // per row: m (0 while there is no maximum), the root of the factor of its step in
    // this tile (applied twice: with an e4m3 cache a sum may be far from 1, and the
    // factor beyond fp32's range), the scale of q, the last key that it sees; with an
    // e4m3 cache m is m + lo for huge scores, beside which a value's exponent is lost in fp32
    float *s_m = reinterpret_cast<float *>(smem + C::kOffRows) + 4 * N + rb, *s_f = s_m + N, *s_qs = s_f + N, *s_lo = s_qs + N;
    int *s_lim = reinterpret_cast<int *>(s_lo + N);
    // How far a score may be above the maximum before m moves (log2), and how far above the
    // maximum m then is: bf16 weights are 1 at most, so that no value overflows.
    constexpr float kSlack = kF8 ? 4.f : 8.f, kAbove = kF8 ? 0.f : kSlack;
    constexpr float kTop = 11.f;                     // e4m3: log2 of what the weights' parts are times, 2^15 at most
    uint32_t g = 0, slot = 0, syncs = 0;
    // the group's barrier; like every wait here it gives up after a limit
    auto group_sync = [&]() -> bool {
      warp_arrive(&bars->sync[w]);
      return wait_bar_warp<false>(&bars->sync[w], syncs++ & 1u, abort);
    };
    for (bool ok = true; ok;) {
      if (!(ok = wait_bar_warp(&bars->item_full[slot % kItems], (slot / kItems) & 1u, abort))) break;
      const Item &it = bars->item[slot % kItems];                 // read where needed: registers are short
      if (it.kind < 0) break;
      ++slot;
      // ---- q: rows of tokens x heads, 8 channels a lane, swizzled; rows past nrow are zero
      {
        constexpr int kLanes = D / 8, kPer = 128 / kLanes;
        const int c = st % kLanes, nrow = it.ntok * p.G;
#pragma unroll
        for (int r0 = 0; r0 < R; r0 += kPer) {
          const int row = rb + r0 + st / kLanes;
          uint4 x = make_uint4(0, 0, 0, 0);
          if (row < nrow) {
            const int tok = row / p.G, gh = row - tok * p.G;
            x = *reinterpret_cast<const uint4 *>(p.q + ((size_t)(it.row0 + tok) * p.H + it.hk * p.G + gh) * D + c * 8);
          }
          if constexpr (!kF8) {
            sts128(sb + C::kOffQ + sw128_offset(row, c * 8, N), x);
          } else {
            uint2 vh, vl;
            const float scale = split_q<kLanes>(x, vh, vl);
            if (c == 0) s_qs[row - rb] = scale * p.c;
            const uint32_t ch = c >> 1, in = (c & 1) * 8;
            auto at = [&](int rr) {
              return D == 128 ? rr * 128u + ((ch ^ (rr & 7u)) << 4) + in : rr * 64u + ((ch ^ ((rr >> 1) & 3u)) << 4) + in;
            };
            *reinterpret_cast<uint2 *>(smem + C::kOffQ + at(row)) = vh;
            *reinterpret_cast<uint2 *>(smem + C::kOffQ + at(N + row)) = vl;
          }
        }
        fence_proxy_async_smem();
        warp_arrive(&bars->q_ready);
        if (st < R) {
          s_m[st] = s_lo[st] = 0.f;
          s_lim[st] = it.pos0 + min(rb + st, nrow - 1) / p.G;
        }
        if (!(ok = group_sync())) break;
      }
      bool has_max = false;  // of the row st (threads 0 .. R - 1 of the group)
      float2 l[R / 2];
#pragma unroll
      for (int r = 0; r < R / 2; ++r) l[r] = make_float2(0.f, 0.f);
      const int j1 = it.j1;
      bool first = true;                               // the item's first tile
      for (int j = it.j0; j < j1; ++j, ++g, first = false) {
        const uint32_t buf = g & 1, tS = tmem + buf * N + rb + lane_base;
        if (!(ok = wait_bar_warp<false>(&bars->s_ready[buf], (g >> 1) & 1u, abort))) break;
        tc_fence_after();
        const int key = j * kTileKeys + kk;
        // ---- scores in log2 units, less m where `less` is set
        float x[R], ev = 0.f;                             // e4m3: the value's exponent
        float ks = p.c;
        if constexpr (kF8) {
          const uint8_t *ss = smem + C::kOffScale + (g % kScaleSlots) * 2 * kTileKeys;
          const uint32_t vc = ss[kTileKeys + kk];
          const bool there = key < it.pos0 + it.ntok;     // a stale scale may be anything
          ks = scale_value(ss[kk]);
          ev = !there ? 0.f : vc == 255 ? __int_as_float(0x7fffffff) : (float)((int)vc - 127);
        }
        // The product is rounded before the difference, as m was: with a fused one equal keys of
        // huge scores would differ.  (Another rounding of the difference, exact near 0, so that
        // the two are not fused after all.)
        auto scores = [&](bool less) {
          tmem_ld16(tS, x);
#pragma unroll
          for (int r = 0; r < R; r += 4) {
            const float4 m = *reinterpret_cast<const float4 *>(s_m + r);
            float2 q0 = make_float2(ks, ks), q1 = q0;
            if constexpr (kF8) {
              const float4 qs = *reinterpret_cast<const float4 *>(s_qs + r);
              q1 = __fmul2_rn(q0, make_float2(qs.z, qs.w));
              q0 = __fmul2_rn(q0, make_float2(qs.x, qs.y));
            }
            float2 a = __fmul2_rn(make_float2(x[r], x[r + 1]), q0), b = __fmul2_rn(make_float2(x[r + 2], x[r + 3]), q1);
            if (less) {
              a = __fadd2_rz(a, make_float2(-m.x, -m.y));
              b = __fadd2_rz(b, make_float2(-m.z, -m.w));
            }
            x[r] = a.x, x[r + 1] = a.y, x[r + 2] = b.x, x[r + 3] = b.y;
          }
          if (j * kTileKeys + kTileKeys - 1 > it.pos0) {    // some row does not see the whole tile
#pragma unroll
            for (int r = 0; r < R; r += 4) {
              const int4 lim = *reinterpret_cast<const int4 *>(s_lim + r);
              x[r] = key > lim.x ? -INFINITY : x[r];
              x[r + 1] = key > lim.y ? -INFINITY : x[r + 1];
              x[r + 2] = key > lim.z ? -INFINITY : x[r + 2];
              x[r + 3] = key > lim.w ? -INFINITY : x[r + 3];
            }
          }
        };
        scores(true);
        // ---- does a row's maximum move?  (In its first tile always; later once in a while.)
        {
          float t = x[0];
#pragma unroll
          for (int r = 1; r < R - 1; r += 2) t = max3(t, x[r], x[r + 1]);
          const bool any = __any_sync(0xffffffffu, fmaxf(t, x[R - 1]) + ev > kSlack - kAbove);
          if (lane == 0) s_flag[g & 1][w][q4] = any || first;
        }
        if (!(ok = group_sync())) break;
        const int4 fl = *reinterpret_cast<const int4 *>(s_flag[g & 1][w]);
        const bool moves = fl.x | fl.y | fl.z | fl.w | (!first && s_look[w]);
        if (moves) {
          // from the scores themselves: a difference to an m far below has lost their last digits (masked
          // keys of -1e30 before ordinary ones)
          if (!first) scores(false);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float v = warp_max(x[r] + ev);
            if (lane == r) s_red[r * 4 + q4] = v;
          }
          if (!(ok = group_sync())) break;
          float old = 0.f;                                // the row's m before a huge score
          bool huge = false;
          if (st < 32) {
            bool look = false;
            if (st < R) {
              const float4 v = *reinterpret_cast<const float4 *>(s_red + st * 4);
              const float t = fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)), m = s_m[st];
              huge = kF8 && fabsf(t) > 0x1p20f && fabsf(t) < INFINITY;
              if (huge) {
                old = m;
                s_m[st] = has_max ? fmaxf(m, t) : t;
              } else {
                const bool up = has_max ? t - m > kSlack - kAbove : t > -INFINITY;
                s_f[st] = up && has_max ? ex2(-0.5f * (t + kAbove - m)) : 1.f;  // nothing to rescale before the first maximum
                if (up) {
                  s_m[st] = t + kAbove;
                  s_lo[st] = 0.f;
                }
                has_max |= up;
              }
              look = !has_max || huge || s_lo[st] != 0.f;
            }
            const int bits = (__any_sync(0xffffffffu, look) ? 1 : 0) | (__any_sync(0xffffffffu, huge) ? 2 : 0);
            if (st == 0) s_look[w] = bits;
          }
          if (!(ok = group_sync())) break;
          const int look = s_look[w];
          if (look & 2) {                                 // the scores less the new m are small again: lo from them
#pragma unroll
            for (int r = 0; r < R; ++r) {
              const float v = warp_max(__fadd_rn(x[r], -s_m[r]) + ev);
              if (lane == r) s_red[r * 4 + q4] = v;
            }
            if (!(ok = group_sync())) break;
            if (huge) {
              const float4 v = *reinterpret_cast<const float4 *>(s_red + st * 4);
              const float t = fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)), was = old - s_m[st] + s_lo[st];
              const float lo = has_max ? fmaxf(t, was) : t;
              s_f[st] = has_max ? ex2(-0.5f * (lo - was)) : 1.f;
              s_lo[st] = lo;
              has_max = true;
            }
            if (!(ok = group_sync())) break;
          }
#pragma unroll
          for (int r = 0; r < R; r += 4) {
            const float4 m = *reinterpret_cast<const float4 *>(s_m + r);
            const float2 a = __fadd2_rz(make_float2(x[r], x[r + 1]), make_float2(-m.x, -m.y));
            const float2 b = __fadd2_rz(make_float2(x[r + 2], x[r + 3]), make_float2(-m.z, -m.w));
            x[r] = a.x, x[r + 1] = a.y, x[r + 2] = b.x, x[r + 3] = b.y;
          }
          if (kF8 && look) {
#pragma unroll
            for (int r = 0; r < R; ++r) x[r] -= s_lo[r];
          }
#pragma unroll
          for (int r = 0; r < R; r += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(s_f + r);
            const float2 f0 = make_float2(f.x, f.y), f1 = make_float2(f.z, f.w);
            l[r / 2] = __fmul2_rn(__fmul2_rn(l[r / 2], f0), f0);
            l[r / 2 + 1] = __fmul2_rn(__fmul2_rn(l[r / 2 + 1], f1), f1);
          }
        }
        tc_fence_before();
        warp_arrive(&bars->s_free[buf]);                  // (the buffer's next product comes behind this tile's weights)
        if (g > 0 && !(ok = wait_bar_warp<false>(&bars->o_done, (g - 1) & 1u, abort))) break;  // W is read, O^T complete
        if (moves && !first) {
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < C::kTP; ++k) tmem_scale16(tmem + C::kColO + k * N + rb + lane_base, s_f);
        }
        // ---- weights, rounded into their parts, as the second product's B operand: a key's
        // rows are contiguous, 16 bytes a unit
        const uint32_t wp = sb + C::kOffP + kk * 16;
        if constexpr (!kF8) {
#pragma unroll
          for (int c = 0; c < R; c += 8) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int r = 0; r < 8; r += 2) {
              const float2 v = make_float2(ex2(x[c + r]), ex2(x[c + r + 1]));
              l[(c + r) / 2] = __fadd2_rn(l[(c + r) / 2], v);
              hi[r / 2] = pack_bf16(v.x, v.y);
              lo[r / 2] = pack_bf16(v.x - __uint_as_float(hi[r / 2] << 16), v.y - __uint_as_float(hi[r / 2] & 0xffff0000u));
            }
            sts128(wp + (rb + c) / 8 * 2048, make_uint4(hi[0], hi[1], hi[2], hi[3]));
            sts128(wp + (N + rb + c) / 8 * 2048, make_uint4(lo[0], lo[1], lo[2], lo[3]));
          }
        } else {
          // One exponential 2^(x + h) for both, the sum's 2^x and the weight, 2^kTop times 2^x and
          // the value's power of two.  m being the maximum of S + e, the x that count for the sum
          // are above -119 - 30 and those of the weight above -e - 36, and all are at most 4 - e:
          // with h = 23 (e - 90 above 113) the exponential stays between 2^-126 and 2^127 for e in
          // -100 .. 119, and neither loses a key to the other's scale.
          const float h = fmaxf(23.f, ev - 90.f), down = ex2(-h), up = ex2(ev + kTop - h);
          const float2 h2 = make_float2(h, h), down2 = make_float2(down, down), up2 = make_float2(up, up);
          uint32_t q[3][4];
#pragma unroll
          for (int r = 0; r < 16; r += 4) {
            uint32_t a[3], b[3];
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
              float2 u = __fadd2_rn(make_float2(x[r + k], x[r + k + 1]), h2);
              u.x = ex2(u.x);
              u.y = ex2(u.y);
              l[(r + k) / 2] = __ffma2_rn(u, down2, l[(r + k) / 2]);
              u = __fmul2_rn(u, up2);
              split_e5m2x2(u.x, u.y, k ? b : a);
            }
            q[0][r / 4] = __byte_perm(a[0], b[0], 0x7531);
            q[1][r / 4] = __byte_perm(a[1], b[1], 0x7531);
            q[2][r / 4] = __byte_perm(a[2], b[2], 0x5410);
          }
#pragma unroll
          for (int k = 0; k < 3; ++k) sts128(wp + (k * (N / 16) + w) * 2048, make_uint4(q[k][0], q[k][1], q[k][2], q[k][3]));
        }
        if (j == j1 - 1) {
          // the last tile: its values have landed, and rows behind the cache's end become zeros
          const uint32_t vs = NS * (2 * g + 1);  // K of every tile and V of the earlier ones come first
          for (int h = 0; h < NS && ok; ++h) ok = wait_bar_warp(&bars->full[(vs + h) % ST], ((vs + h) / ST) & 1u, abort);
          if (!ok) break;
          if (w == 0 && key >= it.pos0 + it.ntok) {
            if constexpr (NS == 2) {
              const uint32_t a = sb + ((vs + (kk >> 6)) % ST) * kStageBytes + (kk & 63) * 128;
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                sts128(a + 16 * k, make_uint4(0, 0, 0, 0));
                sts128(a + 8192 + 16 * k, make_uint4(0, 0, 0, 0));
              }
            } else {
              constexpr int kRow = D * C::kEsz;
              const uint32_t a = sb + (vs % ST) * kStageBytes + kk * kRow;
#pragma unroll
              for (int k = 0; k < kRow / 16; ++k) sts128(a + 16 * k, make_uint4(0, 0, 0, 0));
            }
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        warp_arrive(&bars->p_ready);
      }
      if (!ok) break;
      // ---- sums over the keys; the item's outputs or its partial result
      const int si = (slot - 1) % kItems, bad = s_bad[si], nrow = it.ntok * p.G;
#pragma unroll
      for (int r = 0; r < R; ++r) {  // the maxima of the last tile have been read
        float v = r & 1 ? l[r / 2].y : l[r / 2].x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == r) s_red[r * 4 + q4] = v;
      }
      if (!(ok = group_sync())) break;
      if (!(ok = wait_bar_warp<false>(&bars->o_done, (g - 1) & 1u, abort))) break;
      tc_fence_after();
      float o[R];
      {
        float o1[R];
        tmem_ld16x2(tmem + C::kColO + rb + lane_base, tmem + C::kColO + N + rb + lane_base, o, o1);
#pragma unroll
        for (int r = 0; r < R; ++r) o[r] = kF8 ? o[r] + 0.25f * o1[r] : o[r] + o1[r];
        if constexpr (kF8) {
          tmem_ld16(tmem + C::kColO + 2 * N + rb + lane_base, o1);
#pragma unroll
          for (int r = 0; r < R; ++r) o[r] = 0x1p-11f * (o[r] + 0.03125f * o1[r]);
        }
      }
      tc_fence_before();
      const int ch = D == 128 ? kk : 16 * q4 + lane;   // channel of this TMEM lane
      const bool has = D == 128 || lane < 16;
      const int pslot = 2 * blockIdx.x + (it.kind == 1 ? 1 : 0);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int row = rb + r;
        if (row < nrow && has) {
          const float4 v = *reinterpret_cast<const float4 *>(s_red + r * 4);
          float lt = (v.x + v.y) + (v.z + v.w);
          if (it.kind == 0) {
            if (!bad) {
              const int tok = row / p.G, gh = row - tok * p.G;
              p.o[((size_t)(it.row0 + tok) * p.H + it.hk * p.G + gh) * D + ch] = __float2bfloat16_rn(lt == 0.f ? 0.f : o[r] / lt);
            }
          } else {
            if (kF8 && s_lo[r] != 0.f) {                  // relative to m alone
              const float f = ex2(0.5f * s_lo[r]);
              o[r] = o[r] * f * f;
              lt = lt * f * f;
            }
            p.part[((size_t)pslot * N + row) * D + ch] = o[r];
            if (ch == 0) p.ml[(size_t)pslot * N + row] = make_float2(lt == 0.f ? -INFINITY : s_m[r], lt);
          }
        }
      }
      if (st == 0 && w == 0) {
        if (it.kind != 0) p.skip[2 * pslot] = bad;
        if (bad && p.dev_status) atomicOr(p.dev_status, GLINATTN_DEV_BAD_SLOT);
      }
      if (!(ok = group_sync())) break;  // s_red and s_m are rewritten by the next item
      warp_arrive(&bars->item_empty[si]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort) {
    if (tid == 0 && p.dev_status) atomicOr(p.dev_status, GLINATTN_DEV_WAIT_TIMEOUT);
    let_copies_land();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

template <int D, bool kF8, int N>
cudaError_t launch(const AttnParams &p, const CUtensorMap &tk, const CUtensorMap &tv, int ctas, cudaStream_t stream) {
  auto kernel = decode_kernel<D, kF8, N>;
  const int bytes = (int)Cfg<D, kF8, N>::kSmem;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  kernel<<<ctas, Cfg<D, kF8, N>::kThreads, bytes, stream>>>(tk, tv, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_merge<D, N, true>(p, ctas, stream);
}

}  // namespace

cudaError_t launch_decode(const AttnParams &p, bool f8, int d, int rows, const void *k_cache, const void *v_cache,
                          int ctas, cudaStream_t stream) {
  const int esz = f8 ? 1 : 2;
  const CUtensorMapDataType type = f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const CUtensorMapSwizzle sw = f8 && d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  const long long dims[3] = {d, p.page, p.P > 0 ? (long long)p.P * p.Hkv : 1};
  if (p.P == 0) k_cache = v_cache = p.q;  // an empty pool: nothing is ever loaded
  const int inner = f8 ? d : 64;
  const int kbox[3] = {inner, p.page, 1};
  const int vbox[3] = {inner, !f8 && d == 128 ? min(p.page, 64) : p.page, 1};
  CUtensorMap tk, tv;
  if (!encode_map(&tk, k_cache, type, esz, dims, kbox, sw) ||
      !encode_map(&tv, v_cache, type, esz, dims, vbox, sw))
    return cudaErrorInvalidValue;
  // more than 16 rows only with an e4m3 cache (item_rows)
  if (d == 128) {
    if (!f8) return launch<128, false, 16>(p, tk, tv, ctas, stream);
    return rows == 16   ? launch<128, true, 16>(p, tk, tv, ctas, stream)
           : rows == 32 ? launch<128, true, 32>(p, tk, tv, ctas, stream)
                        : launch<128, true, 48>(p, tk, tv, ctas, stream);
  }
  if (!f8) return launch<64, false, 16>(p, tk, tv, ctas, stream);
  return rows == 16   ? launch<64, true, 16>(p, tk, tv, ctas, stream)
         : rows == 32 ? launch<64, true, 32>(p, tk, tv, ctas, stream)
                      : launch<64, true, 48>(p, tk, tv, ctas, stream);
}

}  // namespace paged
}  // namespace glinattn
