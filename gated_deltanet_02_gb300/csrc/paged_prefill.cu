// paged_prefill.cu -- attention over the paged cache for many query rows per
// (request, key / value head): prompts, pieces of prompts, and batches that mix
// them with single tokens (glinattn_paged_attention).
//
// Mathematics: one pass over the keys with the running maximum m (log2 units)
// and sum l of the softmax per row,
//   S = Q K^T,   P = 2^(S - m),   O += P V,   l += sum P,
// m only moving (and O, l being rescaled) when a tile exceeds it by 2^8 (P is
// relative to 2^8 times m, 1 at most): a common factor of P, O and l.  S, m, l and O are fp32; P is rounded to bf16
// for the second product (half a step, 2^-8 relative to a weight), which adds
// to the output about what its own rounding to bf16 does.
//
// Kernel: one CTA per SM works on 256 query rows (tokens x heads of a group),
// two tiles of 128 whose S, P and O are in TMEM (S: 2 x 128 columns, O: 2 x D, P
// over S for D = 128 and beside it for D = 64).  For D = 128 one warp issues the
// MMAs, the row tiles in turn, so that one tile's products run while the other's
// softmax does:  P0 V, Q0 K' | P1 V, Q1 K' | ...  (with a warp for each tile their
// products interleave and both tiles' softmaxes run at once, which took packed
// prompts 6% and e4m3 keys 30% longer).  For D = 64 the softmaxes take longer than
// the products: the next S starts as soon as this one is read, and a warp for each
// tile saves their waiting for each other's hand-overs (together 18% for 8191
// tokens, 8 heads).  A softmax thread owns a row, so no reduction crosses threads.
// An item's q is one TMA box per 64 channels, [tokens][heads of the group], that a
// warp of its own loads as soon as the last product with the q before it is done
// (copied by the softmax warps it cost every item 2.3 us of their time).  K and V
// tiles of 128 keys come through a shared-memory ring: TMA, one box per page and
// 64 channels (bf16); of an e4m3 cache the keys go into the first product as they
// are (kind::f8f6f4, q split in place into two e4m3 parts as in paged_decode.cu;
// the keys' scales multiply the scores' columns), while four more warps turn the
// value tiles, times their powers of two, into the bf16 tiles (exact) that the
// second product reads.  Everything but the softmax is kept in short loops: its
// unrolled code streams through the instruction caches (the conversion unrolled
// over 8 keys instead of 2: 811 instead of 760 us for the chunk below).
//
// Bound: the tensor core for long prompts, next to it the softmax of the tile
// that waits for it.  A causal prompt of 16,000 tokens, 16 heads over 4 of 128,
// takes 646 us, 1620 TFLOP/s; packed prompts of 200 .. 4001 tokens 142 us (1110);
// 8191 tokens, 8 heads of 64, 78 us (882); 4096 tokens behind 12,288 of an e4m3
// cache, 32 heads over 8, 783 us (1229).
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

constexpr int kItems = 4;
// How far a score may be above the running maximum (log2); the weights are taken
// relative to 2^kSlack times it, so that none is above 1 and no value overflows.
constexpr float kSlack = 8.f;
constexpr int kNoTile = 0x7fffffff;
// e4m3: the keys' scales are taken times this, for products (2^24 at most) with a scale
// of 2^119, as rows with an infinity get it, stay finite; the scales of q take it out again.
constexpr float kKeyScale = 0x1p-24f;

template <int D, bool kF8>
struct Cfg {
  static constexpr int kThreads = kF8 ? 512 : 384, kCost = kF8 ? kItemCostManyF8 : kItemCostMany;
  // q: planes of 256 rows of 128 bytes (64 channels, bf16), or the two e4m3 parts;
  // they come as the same planes of half the channels each
  static constexpr uint32_t kQRow = kF8 ? D : 128, kQPlane = 2 * 128 * kQRow, kQPlanes = 512 * D / kQPlane;
  static constexpr uint32_t kStageBytes = kTileKeys * D * 2;  // a bf16 tile
  static constexpr uint32_t kRawBytes = kTileKeys * D;        // an e4m3 tile
  // bf16: K and V tiles in turn; e4m3: V tiles after their conversion, and K
  // and V tiles as they are in the cache
  static constexpr int kStages = kF8 ? 2 : D == 128 ? 4 : 6;
  static constexpr int kRawK = kF8 ? 3 : 0, kRawV = kF8 ? 2 : 0;
  static constexpr int kScaleSlots = kF8 ? 8 : 0;             // tiles of key scales as floats
  static constexpr uint32_t kOffRing = kQPlanes * kQPlane;
  static constexpr uint32_t kOffRawK = kOffRing + kStages * kStageBytes;
  static constexpr uint32_t kOffRawV = kOffRawK + kRawK * kRawBytes;
  static constexpr uint32_t kOffCode = kOffRawV + kRawV * kRawBytes;      // scale codes beside the raw tiles
  static constexpr uint32_t kOffScale = kOffCode + (kRawK + kRawV) * kTileKeys;
  // bf16, D = 128: 32 rows of 64 output channels for each softmax warp, which TMA
  // then writes (64 prompts of 100 .. 600 tokens, 16 heads over 4: 77 us, with
  // stores of the registers 83 us; longer prompts the same).  D = 64 has half the
  // outputs and gains nothing, e4m3 has no room.
  static constexpr bool kStaged = !kF8 && D == 128;
  static constexpr uint32_t kOffOut = kOffScale + kScaleSlots * kTileKeys * 4;
  static constexpr uint32_t kOffBars = kOffOut + (kStaged ? 8 * 4096 : 0);
  static constexpr uint32_t kBytesBars = 1024 + (kF8 ? 1024 : 0);         // e4m3: and a scale per q row
  static constexpr uint32_t kSmem = kOffBars + kBytesBars + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  // the keys' scales of tile j are read before S of tile j + 1 is issued, so
  // that a tile at most kRawK ahead can be written meanwhile
  static_assert(!kF8 || kScaleSlots > kRawK, "scale slots");
  // TMEM columns: S, O, and P over S (D = 128 takes all 512) or beside it
  static constexpr bool kSepP = D == 64;
  static constexpr int kIssuers = kSepP ? 2 : 1;
  static constexpr uint32_t kColS = 0, kColO = 256, kColP = kSepP ? kColO + 2 * D : kColS, kPStep = kSepP ? 64 : 128;
};

struct Bars {
  uint64_t full[6], empty[6];             // bf16 tiles
  uint64_t rawk_full[3], rawk_empty[3], rawv_full[2], rawv_empty[2], scale_ready[8];
  uint64_t s_ready[2], s_free[2], p_ready[2][2], q_empty, q_ready[2], o_done[2];
  uint64_t item_full[kItems], item_empty[kItems];
  // an item's q; one for each slot, since a row tile without work in an item does not wait for its q
  uint64_t q_full[kItems];
  Item item[kItems];
  PlanShared plan;
  int bad[kItems];  // the item's first cache tile with a bad page
  uint32_t tmem;
  int abort;
};

template <int kRegs>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// Tiles [j0, j1) that row tile w of the item looks at: up to its last row's key.
__device__ __forceinline__ int last_tile(const Item &it, int G, uint32_t inv_g, int w) {
  const int nrow = it.ntok * G;
  const int last = max(min(128 * (w + 1), nrow) - 1, 0);  // its last row
  const int end = it.pos0 + (int)((uint32_t)last * inv_g >> 16) + 1;
  const int n = end <= kTileKeys ? 1 : (end + kTileKeys - 1) / kTileKeys;
  return 128 * w >= nrow ? it.j0 : max(it.j0, min(it.j1, n));
}

// Two e4m3 (bytes 0 and 1 of `two`) as bf16 of 2^-120 times their value: the
// e4m3 fields moved under bf16's (a subnormal stays one).
__device__ __forceinline__ uint32_t e4m3x2_bf16_small(uint32_t two) {
  const uint32_t v = __byte_perm(two, 0, 0x1404);  // bytes 0, 1 to the top of each half
  return (v & 0x80008000u) | ((v >> 4) & 0x07f007f0u);
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A box from shared memory, by the calling lane; its stores are one group each.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, uint32_t src, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];\n\tcp.async.bulk.commit_group;" ::"l"(map),
      "r"(src), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// 64 bytes to global memory, as two 32-byte stores where the address allows it.
__device__ __forceinline__ void store64(void *dst, const uint32_t (&u)[16]) {
  if (((uintptr_t)dst & 31) == 0) {
#pragma unroll
    for (int k = 0; k < 16; k += 8)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(reinterpret_cast<uint32_t *>(dst) + k), "r"(u[k]),
                   "r"(u[k + 1]), "r"(u[k + 2]), "r"(u[k + 3]), "r"(u[k + 4]), "r"(u[k + 5]), "r"(u[k + 6]), "r"(u[k + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int k = 0; k < 16; k += 4) reinterpret_cast<uint4 *>(dst)[k / 4] = make_uint4(u[k], u[k + 1], u[k + 2], u[k + 3]);
  }
}

template <int D, bool kF8>
__global__ void __launch_bounds__(kF8 ? 512 : 384, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                   const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap to, const AttnParams p,
                   const uint8_t *v_cache) {
  using C = Cfg<D, kF8>;
  constexpr int ST = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Bars *bars = reinterpret_cast<Bars *>(smem + C::kOffBars);
  static_assert(sizeof(Bars) <= 1024, "barrier block");
  static_assert(ST <= 6 && C::kRawK <= 3 && C::kRawV <= 2 && C::kScaleSlots <= 8, "barriers of the rings");
  float *s_qs = reinterpret_cast<float *>(smem + C::kOffBars + 1024);  // e4m3: scale of a q row
  volatile int *abort = &bars->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sb = smem_u32(smem);

  if (tid == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(&bars->full[s], kF8 ? 4 : 1);
      mbar_init(&bars->empty[s], C::kIssuers);
    }
    for (int s = 0; s < C::kRawK; ++s) {
      mbar_init(&bars->rawk_full[s], 1);
      mbar_init(&bars->rawk_empty[s], C::kIssuers + 4);  // and the scales' readers
    }
    for (int s = 0; s < C::kRawV; ++s) {
      mbar_init(&bars->rawv_full[s], 1);
      mbar_init(&bars->rawv_empty[s], 4);
    }
    for (int s = 0; s < C::kScaleSlots; ++s) mbar_init(&bars->scale_ready[s], 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->s_ready[i], 1);
      mbar_init(&bars->s_free[i], 4);
      mbar_init(&bars->p_ready[i][0], 4);
      mbar_init(&bars->p_ready[i][1], 4);
      mbar_init(&bars->q_ready[i], 4);
      mbar_init(&bars->o_done[i], 1);
    }
    mbar_init(&bars->q_empty, C::kIssuers);
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&bars->item_full[i], 1);
      mbar_init(&bars->q_full[i], 1);
      mbar_init(&bars->item_empty[i], 1 + C::kIssuers + 8 + (kF8 ? 4 : 0));
      bars->bad[i] = kNoTile;
    }
    bars->abort = 0;
    p.desc[blockIdx.x].w = -1;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  const Plan plan = make_plan<false, C::kCost>(p, &bars->plan);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int pages = kTileKeys >> p.page_shift;  // pages of a tile
  const uint32_t inv_g = (65535u + p.G) / p.G;  // row / G is row * inv_g >> 16 for row, G <= 256

  if (warp < 4) {
    // registers a thread: 64 + 2 x 192 + 64 of 4 x 128 (e4m3), 80 + 2 x 208 of 3 x 168
    regs_dec<kF8 ? 64 : 80>();
    if (warp == 0) {
      // ============ the walk over the items, and TMA ============
      Walk<false, C::kCost> walk(p, plan, lane);
      Item it;
      uint32_t sc = 0, slot = 0;
      for (bool ok = true; ok;) {
        const bool more = walk.next(it, lane);
        const int si = slot % kItems;
        if (!(ok = wait_bar_warp(&bars->item_empty[si], ((slot / kItems) & 1u) ^ 1u, abort))) break;
        if (!more) it.kind = -1;
        if (lane == 0) {
          bars->item[si] = it;
          bars->bad[si] = kNoTile;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->item_full[si]);
        ++slot;
        if (!more) break;
        const int npage = (int)(((long long)it.pos0 + it.ntok + p.page - 1) >> p.page_shift);
        const int32_t *table = p.table + (size_t)it.r * p.max_pages;
        int base = it.j0 * pages;
        int ids = base + lane < npage ? table[base + lane] : 0;
        int ids_next = base + 32 + lane < npage ? table[base + 32 + lane] : 0;
        for (int j = it.j0; j < it.j1 && ok; ++j) {
          if (j * pages >= base + 32) {
            base += 32;
            ids = ids_next;
            ids_next = base + 32 + lane < npage ? table[base + 32 + lane] : 0;
          }
          // bf16: a page and 64 channels per lane; e4m3: a page per lane
          const int pl = lane & (pages - 1), col = lane / pages;
          const int np = min(pages, npage - j * pages);
          const int id = __shfl_sync(0xffffffffu, ids, j * pages - base + pl);
          const bool good = id >= 0 && id < p.P, op = pl < np && col < (kF8 ? 1 : D / 64);
          if (__any_sync(0xffffffffu, op && !good) && lane == 0) bars->bad[si] = min(bars->bad[si], j);
          const uint32_t ops = (uint32_t)__popc(__ballot_sync(0xffffffffu, op && good));
          const uint32_t bytes = kF8 ? ops * (uint32_t)p.page * (D + 1) : ops << (p.page_shift + 7);
          const size_t plane = (size_t)(good ? id : 0) * p.Hkv + it.hk;
#pragma unroll
          for (int v = 0; v < 2; ++v, ++sc) {
            if constexpr (kF8) {
              const uint32_t g = sc >> 1, s = v ? g % C::kRawV : g % C::kRawK;
              uint64_t *f = v ? &bars->rawv_full[s] : &bars->rawk_full[s];
              if (!(ok = v ? wait_bar_warp(&bars->rawv_empty[s], ((g / C::kRawV) & 1u) ^ 1u, abort)
                           : wait_bar_warp(&bars->rawk_empty[s], ((g / C::kRawK) & 1u) ^ 1u, abort)))
                break;
              if (lane == 0) mbar_arrive_expect_tx(f, bytes);
              __syncwarp();
              if (op && good) {
                if (v)
                  bulk_load(smem + C::kOffRawV + s * C::kRawBytes + pl * p.page * D, v_cache + plane * p.page * D,
                            (uint32_t)p.page * D, f);
                else
                  tma_load_3d(smem + C::kOffRawK + s * C::kRawBytes + pl * p.page * D, &tk, f, 0, 0, (int)plane);
                bulk_load(smem + C::kOffCode + (v ? C::kRawK + s : s) * kTileKeys + pl * p.page,
                          (v ? p.v_scale : p.k_scale) + plane * p.page, (uint32_t)p.page, f);
              }
            } else {
              const uint32_t s = sc % ST;
              if (!(ok = wait_bar_warp(&bars->empty[s], ((sc / ST) & 1u) ^ 1u, abort))) break;
              if (lane == 0) mbar_arrive_expect_tx(&bars->full[s], bytes);
              __syncwarp();
              if (op && good)
                tma_load_3d(smem + C::kOffRing + s * C::kStageBytes + col * 16384 + (pl << (p.page_shift + 7)), v ? &tv : &tk,
                            &bars->full[s], 64 * col, 0, (int)plane);
            }
          }
        }
      }
    } else if (warp <= C::kIssuers) {
      // ============ MMA issue (one lane): kMine row tiles from w0 on ============
      constexpr int kMine = 2 / C::kIssuers;
      const int w0 = C::kIssuers == 2 ? warp - 1 : 0;
      constexpr uint32_t id_s = kF8 ? idesc_f8(128, 128, false, false) : idesc_bf16(128, 128, false, false);
      constexpr uint32_t id_o = idesc_bf16(128, D, false, true);
      constexpr uint32_t hi_s = kF8 && D == 64 ? desc_hi(512, kSw64) : desc_hi(1024, kSw128);
      const bool leader = elect_one();
      uint32_t g = 0, slot = 0, np[kMine] = {}, nq[kMine] = {}, nf[kMine] = {};  // g: cache tiles so far
      // stages of tile t's keys and values
      auto k_stage = [](uint32_t t) { return kF8 ? t % C::kRawK : 2 * t % ST; };
      auto v_stage = [](uint32_t t) { return kF8 ? t % ST : (2 * t + 1) % ST; };
      auto k_landed = [&](uint32_t t) -> bool {
        return kF8 ? wait_bar_warp<false>(&bars->rawk_full[k_stage(t)], (t / C::kRawK) & 1u, abort)
                   : wait_bar_warp<false>(&bars->full[k_stage(t)], (2 * t / ST) & 1u, abort);
      };
      auto v_landed = [&](uint32_t t) -> bool {
        return wait_bar_warp<false>(&bars->full[v_stage(t)], (kF8 ? t / ST : (2 * t + 1) / ST) & 1u, abort);
      };
      // S_w = Q_w K^T; with P beside S the scores before it have to be read
      auto issue_s = [&](int i, uint32_t t) -> bool {
        const int w = w0 + i;
        if (C::kSepP && !wait_bar_warp<false>(&bars->s_free[w], (nf[i]++ & 1u) ^ 1u, abort)) return false;
        tc_fence_after();
        const uint32_t d = tmem + C::kColS + 128 * w, a = desc_lo(sb + w * (C::kQPlane / 2), 16);
        const uint32_t b = desc_lo(kF8 ? sb + C::kOffRawK + k_stage(t) * C::kRawBytes : sb + C::kOffRing + k_stage(t) * C::kStageBytes, 16);
        if (leader) {
          if constexpr (kF8) {  // both parts of q against the same keys
#pragma unroll
            for (int ks = 0; ks < 2 * (D / 32); ++ks) {
              const uint32_t k = ks % (D / 32) * 32;
              mma_ss<true>(d, a + (ks / (D / 32) * C::kQPlane + k >> 4), hi_s, b + (k >> 4), hi_s, id_s, ks > 0);
            }
          } else {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              const uint32_t k = (ks & 3) * 32;
              mma_ss<false>(d, a + ((ks >> 2) * C::kQPlane + k >> 4), hi_s, b + ((ks >> 2) * 16384 + k >> 4), hi_s, id_s, ks > 0);
            }
          }
          umma_commit(&bars->s_ready[w]);
        }
        return true;
      };
      // O_w (+)= P_w V, 64 keys' weights at a time
      auto issue_o = [&](int i, uint32_t t, bool first) -> bool {
        const int w = w0 + i;
        const uint32_t b = desc_lo(sb + C::kOffRing + v_stage(t) * C::kStageBytes, 16384), ph = np[i]++ & 1u;
        const uint32_t d = tmem + C::kColO + D * w, a = tmem + C::kColP + C::kPStep * w;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!wait_bar_warp<false>(&bars->p_ready[w][h], ph, abort)) return false;
          tc_fence_after();
          if (leader) {
#pragma unroll
            for (int ks = 4 * h; ks < 4 * h + 4; ++ks)
              mma_ts(d, a + 8 * ks, b + ks * (2048 >> 4), desc_hi(1024, kSw128), id_o, ks > 0 || !first);
          }
        }
        return true;
      };
      Item it;
      int nw[kMine], most;
      // a stage (and q) is free when every issuer says so: behind its products, or at
      // once (but not before it is filled) where its row tiles have none in it
      auto release = [&](uint64_t *bar, bool used) {
        if (!leader) return;
        if (used) umma_commit(bar);
        else mbar_arrive(bar);
      };
      // behind the products with the item's tile j: is it the last that reads q?
      auto q_release = [&](int j) {
        if (j == max(most, 1) - 1) release(&bars->q_empty, most > 0);
      };
      auto k_release = [&](uint32_t t, bool used) { release(kF8 ? &bars->rawk_empty[k_stage(t)] : &bars->empty[k_stage(t)], used); };
      auto next_item = [&]() -> bool {
        const int si = slot % kItems;
        if (!wait_bar_warp<false>(&bars->item_full[si], (slot / kItems) & 1u, abort)) return false;
        it = bars->item[si];
        warp_arrive(&bars->item_empty[si]);
        ++slot;
#pragma unroll
        for (int i = 0; i < kMine; ++i) nw[i] = it.kind < 0 ? 0 : last_tile(it, p.G, inv_g, w0 + i) - it.j0;
        most = max(nw[0], nw[kMine - 1]);
        return true;
      };
      auto q_there = [&](int i) -> bool {
        return kF8 ? wait_bar_warp<false>(&bars->q_ready[w0 + i], nq[i]++ & 1u, abort)
                   : wait_bar_warp<false>(&bars->q_full[(slot - 1) % kItems], ((slot - 1) / kItems) & 1u, abort);
      };
      bool ok = next_item();
      while (ok && it.kind >= 0) {
        const int n = it.j1 - it.j0;
        // first scores
        if (!(ok = k_landed(g))) break;
#pragma unroll
        for (int i = 0; i < kMine; ++i)
          if (ok && nw[i] > 0) ok = q_there(i) && issue_s(i, g);
        if (C::kIssuers == 2 && ok && most <= 0)
          ok = wait_bar_warp<false>(&bars->q_full[(slot - 1) % kItems], ((slot - 1) / kItems) & 1u, abort);
        if (!ok) break;
        k_release(g, most > 0);
        q_release(0);
        for (int j = 0; j < n && ok; ++j) {
          const bool last = j + 1 == n;
          if (C::kSepP && !last) {  // the next scores before this tile's second product
            if (!(ok = k_landed(g + j + 1))) break;
#pragma unroll
            for (int i = 0; i < kMine; ++i)
              if (ok && j + 1 < nw[i]) ok = issue_s(i, g + j + 1);
            if (!ok) break;
            k_release(g + j + 1, j + 1 < most);
            q_release(j + 1);
          }
          if (!(ok = v_landed(g + j))) break;
          if (!C::kSepP && !last && !(ok = k_landed(g + j + 1))) break;
#pragma unroll
          for (int i = 0; i < kMine; ++i) {
            if (ok && j < nw[i]) {
              ok = issue_o(i, g + j, j == 0);
              if (ok && leader && (C::kSepP || j + 1 == nw[i])) umma_commit(&bars->o_done[w0 + i]);
            }
            if (!C::kSepP && ok && j + 1 < nw[i]) ok = issue_s(i, g + j + 1);
          }
          if (!ok) break;
          release(&bars->empty[v_stage(g + j)], j < most);
          if (!C::kSepP && !last) {
            k_release(g + j + 1, j + 1 < most);
            q_release(j + 1);
          }
        }
        g += n;
        if (ok) ok = next_item();
      }
    } else if (warp == 3) {
      // ============ q: an item's rows (tokens x heads of the group) are a box ============
      // Rows behind the item's last hold other tokens' q, or zeros behind the last
      // token; nothing that comes of them is stored.
      for (uint32_t slot = 0;; ++slot) {
        const int si = slot % kItems;
        if (!wait_bar_warp(&bars->item_full[si], (slot / kItems) & 1u, abort)) break;
        const int kind = bars->item[si].kind, row0 = bars->item[si].row0, hk = bars->item[si].hk;
        warp_arrive(&bars->item_empty[si]);
        if (kind < 0 || !wait_bar_warp(&bars->q_empty, (slot & 1u) ^ 1u, abort)) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars->q_full[si], C::kQPlanes * (uint32_t)(p.tp * p.G) * C::kQRow);
#pragma unroll
          for (uint32_t h = 0; h < C::kQPlanes; ++h)
            tma_load_3d(smem + h * C::kQPlane, &tq, &bars->q_full[si], (int)(h * C::kQRow / 2), hk * p.G, row0);
        }
        __syncwarp();
      }
    }
  } else if (warp < 12) {
    // ============ softmax: row tile w, thread = row ============
    regs_inc<kF8 ? 192 : 208>();
    const int w = warp >= 8 ? 1 : 0, q4 = warp & 3;
    const int lrow = 32 * q4 + lane, row = 128 * w + lrow;
    const uint32_t lane_base = (uint32_t)(32 * q4) << 16;
    const uint32_t tS = tmem + C::kColS + 128 * w + lane_base, tO = tmem + C::kColO + D * w + lane_base;
    const uint32_t tP = tmem + C::kColP + C::kPStep * w + lane_base;
    uint32_t g = 0, slot = 0, ns = 0, nd = 0;  // g: cache tiles so far
    // a row's place among the item's rows of q and o, in elements
    auto row_at = [&](const Item &it, int r) -> size_t {
      const int tok = (int)((uint32_t)r * inv_g >> 16);
      return ((size_t)(it.row0 + tok) * p.H + it.hk * p.G + (r - tok * p.G)) * D;
    };
    // An e4m3 cache's q, D / 8 lanes a row: split in place, row by row, half a row
    // of bf16 where each part goes.  Only for a row tile that has work in the item:
    // its softmax warps then wait for the MMA warp's answer, so that q_ready is
    // never a phase ahead of its reader.
    auto split_rows = [&](uint32_t slot) -> bool {
      const Item &it = bars->item[slot % kItems];
      if (!kF8 || it.kind < 0 || last_tile(it, p.G, inv_g, w) <= it.j0) return true;
      if (!wait_bar_warp(&bars->q_full[slot % kItems], (slot / kItems) & 1u, abort)) return false;
      constexpr uint32_t kLanes = D / 8, kPer = 32 / kLanes, kQU = 2;
      const uint32_t c = lane % kLanes, half = c / (kLanes / 2);
      auto at = [&](uint32_t r, uint32_t unit) { return r * C::kQRow + ((unit ^ (D == 128 ? r & 7u : r >> 1 & 3u)) << 4); };
#pragma unroll 1
      for (uint32_t r0 = row - lane + lane / kLanes, n = 0; n < kLanes; n += kQU, r0 += kQU * kPer) {
        uint4 x[kQU];
#pragma unroll
        for (uint32_t k = 0; k < kQU; ++k) x[k] = lds128(sb + half * C::kQPlane + at(r0 + k * kPer, c % (kLanes / 2)));
        __syncwarp();
#pragma unroll
        for (uint32_t k = 0; k < kQU; ++k) {
          const uint32_t r = r0 + k * kPer;
          uint2 hi, lo;
          const float scale = split_q<kLanes>(x[k], hi, lo);
          // never 0 (nor infinite), which a masked score of -infinity (or one of 0) would turn into
          // NaN: scores, 2^119 at most before it, are next to 0 then
          if (c == 0) s_qs[r] = fminf(fmaxf(scale * (p.c / kKeyScale), 0x1p-126f), 3.4e38f);
          uint8_t *dst = smem + at(r, c >> 1) + (c & 1) * 8;
          *reinterpret_cast<uint2 *>(dst) = hi;
          *reinterpret_cast<uint2 *>(dst + C::kQPlane) = lo;
        }
      }
      fence_proxy_async_smem();
      warp_arrive(&bars->q_ready[w]);
      return true;
    };
    bool ok = wait_bar_warp(&bars->item_full[0], 0, abort);
    if (ok) ok = split_rows(0);
    while (ok) {
      const Item &it = bars->item[slot % kItems];
      if (it.kind < 0) break;
      const int j0 = it.j0, n = it.j1 - j0, nw = last_tile(it, p.G, inv_g, w) - j0;
      const int end = it.pos0 + it.ntok;                    // keys behind it are not there
      const int lim = it.pos0 + (int)((uint32_t)row * inv_g >> 16);  // the row's last key
      const int first_lim = it.pos0 + (int)((uint32_t)(128 * w) * inv_g >> 16);  // the first row's
      const float c = kF8 ? s_qs[row] : p.c;                // written by this warp
      const float slack = fminf(kSlack / c, 1e38f);
      float m = -INFINITY, l = 0.f;                         // the maximum in the scores' units, before c
      for (int jj = 0; jj < nw; ++jj) {
        const int j = j0 + jj;
        if (!(ok = wait_bar_warp<false>(&bars->s_ready[w], ns++ & 1u, abort))) break;
        tc_fence_after();
        float s[128];
        if constexpr (D == 64) {  // (78 us instead of 80 for 8191 tokens; D = 128 does not gain)
          tmem_ld128(tS, s);
        } else {
          tmem_ld32x2(tS, tS + 32, *reinterpret_cast<float(*)[32]>(s), *reinterpret_cast<float(*)[32]>(s + 32));
          tmem_ld32x2(tS + 64, tS + 96, *reinterpret_cast<float(*)[32]>(s + 64), *reinterpret_cast<float(*)[32]>(s + 96));
        }
        if (C::kSepP) {
          tc_fence_before();
          warp_arrive(&bars->s_free[w]);
        }
        if constexpr (kF8) {  // the keys' scales
          const uint32_t ss = (g + jj) % C::kScaleSlots;
          if (!(ok = wait_bar_warp(&bars->scale_ready[ss], ((g + jj) / C::kScaleSlots) & 1u, abort))) break;
          const float4 *ks = reinterpret_cast<const float4 *>(smem + C::kOffScale + ss * kTileKeys * 4);
#pragma unroll
          for (int k = 0; k < 128; k += 4) {
            const float4 v = ks[k / 4];
            const float2 a = __fmul2_rn(make_float2(s[k], s[k + 1]), make_float2(v.x, v.y));
            const float2 b = __fmul2_rn(make_float2(s[k + 2], s[k + 3]), make_float2(v.z, v.w));
            s[k] = a.x, s[k + 1] = a.y, s[k + 2] = b.x, s[k + 3] = b.y;
          }
        }
        if (j * kTileKeys + kTileKeys - 1 > first_lim) {
          const int left = lim - j * kTileKeys;             // columns 0 .. left are seen
#pragma unroll
          for (int k = 0; k < 128; ++k) s[k] = k <= left ? s[k] : -INFINITY;
        }
        float mt;
        {
          float a[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int k = 4; k < 124; k += 8) {
#pragma unroll
            for (int u = 0; u < 4; ++u) a[u] = max3(a[u], s[k + u], s[k + 4 + u]);
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) a[u] = fmaxf(a[u], s[124 + u]);
          mt = fmaxf(max3(a[0], a[1], a[2]), a[3]);
        }
        const bool need = mt > m + slack;
        // the previous P is read and O complete: with P over S this tile's S was issued behind P V
        if (C::kSepP && jj > 0) {
          if (!(ok = wait_bar_warp<false>(&bars->o_done[w], nd++ & 1u, abort))) break;
          tc_fence_after();
        }
        if (__any_sync(0xffffffffu, need)) {
          const float mn = need ? mt : m;
          const float f = need ? ex2((m - mn) * c) : 1.f;
          l *= f;
          m = mn;
          if (jj > 0) {
#pragma unroll 1
            for (int k = 0; k < D; k += 32) {
              float o[32];
              uint32_t u[32];
              tmem_ld32(tO + k, o);
#pragma unroll
              for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(o[e] * f);
              tmem_st32(tO + k, u);
            }
          }
        }
        // S c - m c, fused, is off by the rounding of m c, the same for all keys: next to nothing
        // for ordinary scores, a factor beyond fp32's range for huge ones.  There, with c cut to
        // a power of two, it is exact: keys that equal the maximum have weight 1, and
        // any other, a step of 2^5 (2^4 with that c) below at least, next to none.
        float cc = c, ms = m * c + kSlack;
        if (ms == -INFINITY) ms = 0.f;  // no score above -infinity, in these units
        if (fabsf(ms) > 0x1p29f) {
          cc = __uint_as_float(__float_as_uint(c) & 0x7f800000u);
          ms = m * cc;
        }
        const float2 c2 = make_float2(cc, cc), m2 = make_float2(-ms, -ms);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t u[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float2 x = __ffma2_rn(make_float2(s[64 * h + 2 * e], s[64 * h + 2 * e + 1]), c2, m2);
            x.x = ex2(x.x);
            x.y = ex2(x.y);
            sum[e & 1] = __fadd2_rn(sum[e & 1], x);
            u[e] = pack_bf16(x.x, x.y);
          }
          if (h == 0 && jj == nw - 1) {
            // the row tile's last cache tile: its values have landed; rows behind the cache's end become
            // zeros (where both row tiles see them, both write the zeros that their own product needs)
            const uint32_t vs = kF8 ? g + jj : 2 * (g + jj) + 1;
            if (!(ok = wait_bar_warp(&bars->full[vs % ST], (vs / ST) & 1u, abort))) break;
            if (!kF8 && j * kTileKeys + lrow >= end) {
              const uint32_t a = sb + C::kOffRing + (vs % ST) * C::kStageBytes + lrow * 128;
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                sts128(a + 16 * k, make_uint4(0, 0, 0, 0));
                if (D == 128) sts128(a + 16384 + 16 * k, make_uint4(0, 0, 0, 0));
              }
            }
            fence_proxy_async_smem();
          }
          tmem_st32(tP + 32 * h, u);
          tc_fence_before();
          warp_arrive(&bars->p_ready[w][h]);
        }
        if (!ok) break;
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      }
      if (!ok) break;
      g += n;
      // ---- the next item's q, before this item's outputs
      ++slot;
      if (!(ok = wait_bar_warp(&bars->item_full[slot % kItems], (slot / kItems) & 1u, abort))) break;
      if (!(ok = split_rows(slot))) break;
      // a bad page counts for the row tiles that read it; the producer may be past this one's last tile
      const int si = (slot - 1) % kItems, bad = bars->bad[si] < j0 + nw;
      const bool has = row < it.ntok * p.G;
      const size_t pslot = (size_t)(2 * blockIdx.x + (it.kind == 1 ? 1 : 0));
      if (nw > 0) {
        if (!(ok = wait_bar_warp(&bars->o_done[w], nd++ & 1u, abort))) break;
        tc_fence_after();
        const float inv = l == 0.f ? 0.f : 1.f / l;
        __nv_bfloat16 *dst = p.o + row_at(it, row);
        const bool put = it.kind == 0 && has && !bad;
        // a warp whose 32 rows are all there, and whole tokens: a box of them for 64 channels
        const bool boxes = C::kStaged && it.kind == 0 && !bad && 32 % p.G == 0 && row - lane + 32 <= it.ntok * p.G;
        if (boxes) {
          const uint32_t out = sb + C::kOffOut + (warp - 4) * 4096;
          const int x = it.hk * p.G, y = it.row0 + (row - lane) / p.G;
#pragma unroll 1
          for (int k = 0; k < D; k += 64) {
            float o[64];
            tmem_ld32x2(tO + k, tO + k + 32, *reinterpret_cast<float(*)[32]>(o), *reinterpret_cast<float(*)[32]>(o + 32));
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the last box has been read
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 64; e += 8) {
              uint32_t u[4];
#pragma unroll
              for (int v = 0; v < 4; ++v) u[v] = l == 0.f ? 0u : pack_bf16(o[e + 2 * v] * inv, o[e + 2 * v + 1] * inv);
              sts128(out + lane * 128 + ((e / 8 ^ (lane & 7)) << 4), make_uint4(u[0], u[1], u[2], u[3]));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tma_store_3d(&to, out, k, x, y);
          }
        }
#pragma unroll 1
        for (int k = 0; k < D && !boxes; k += 32) {
          float o[32];
          tmem_ld32(tO + k, o);
          if (it.kind == 0) {
            // 64 contiguous bytes of the lane's row, whole 32-byte sectors
            uint32_t u[16];
#pragma unroll
            for (int x = 0; x < 16; ++x) u[x] = l == 0.f ? 0u : pack_bf16(o[2 * x] * inv, o[2 * x + 1] * inv);
            if (put) store64(dst + k, u);
          } else if (has) {
            float4 *part = reinterpret_cast<float4 *>(p.part) + (pslot * (D / 4) + k / 4) * kPrefillRows + row;
#pragma unroll
            for (int e = 0; e < 32; e += 4) part[e / 4 * kPrefillRows] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
        }
        tc_fence_before();
      }
      // a sum beside no maximum is NaN (scores of NaN alone): the merge leaves out pieces whose maximum is
      // -infinity; so it is here where the row tile has no work, and c is not this item's
      const float ml = m > -INFINITY ? m * c + kSlack : l != 0.f ? 0.f : m;
      if (it.kind != 0 && has) p.ml[pslot * kPrefillRows + row] = make_float2(ml, l);
      if (lrow == 0) {
        if (it.kind != 0) p.skip[2 * pslot + w] = bad;
        if (bad && p.dev_status) atomicOr(p.dev_status, GLINATTN_DEV_BAD_SLOT);
      }
      warp_arrive(&bars->item_empty[si]);
    }
  } else if constexpr (kF8) {
    // ============ e4m3 cache: the keys' scales as floats; values times their scale, as the bf16 tile ============
    regs_dec<64>();
    const int ct = tid - 384;
    constexpr int kLanes = D / 16;                   // lanes of a key's row, 16 values each
    constexpr int kKeys = 128 / kLanes;              // keys a pass of the 128 threads takes: 16 or 32
    constexpr int kPass = kTileKeys / kKeys, kCU = 2;
    const int c16 = ct % kLanes, k0 = ct / kLanes;   // key of pass i: i kKeys + k0
    uint32_t g = 0, slot = 0;
    for (bool ok = true; ok;) {
      const int si = slot % kItems;
      if (!(ok = wait_bar_warp(&bars->item_full[si], (slot / kItems) & 1u, abort))) break;
      const int kind = bars->item[si].kind, j1 = bars->item[si].j1;
      const int end = bars->item[si].pos0 + bars->item[si].ntok;
      int j = bars->item[si].j0;
      warp_arrive(&bars->item_empty[si]);
      if (kind < 0) break;
      ++slot;
      for (; j < j1; ++j, ++g) {
        const uint32_t rk = g % C::kRawK, rv = g % C::kRawV, s = g % ST, ss = g % C::kScaleSlots;
        if (!(ok = wait_bar_warp(&bars->rawk_full[rk], (g / C::kRawK) & 1u, abort))) break;
        reinterpret_cast<float *>(smem + C::kOffScale)[ss * kTileKeys + ct] = kKeyScale * scale_value(smem[C::kOffCode + rk * kTileKeys + ct]);
        warp_arrive(&bars->rawk_empty[rk]);
        warp_arrive(&bars->scale_ready[ss]);
        if (!(ok = wait_bar_warp(&bars->rawv_full[rv], (g / C::kRawV) & 1u, abort))) break;
        if (!(ok = wait_bar_warp(&bars->empty[s], ((g / ST) & 1u) ^ 1u, abort))) break;
        const uint32_t raw = sb + C::kOffRawV + rv * C::kRawBytes;
        const uint8_t *code = smem + C::kOffCode + (C::kRawK + rv) * kTileKeys;
        const uint32_t base = sb + C::kOffRing + s * C::kStageBytes;
        const int there = end - j * kTileKeys;              // keys of the tile that are there
        // a short loop: the unrolled one takes the softmax's code out of the instruction caches
#pragma unroll 1
        for (int i0 = 0; i0 < kPass; i0 += kCU) {
          uint4 y[kCU];
          uint32_t cd[kCU];
#pragma unroll
          for (int i = 0; i < kCU; ++i) {
            const int key = (i0 + i) * kKeys + k0;
            y[i] = lds128(raw + key * D + c16 * 16);
            cd[i] = code[key];
          }
#pragma unroll
          for (int i = 0; i < kCU; ++i) {
            const int key = (i0 + i) * kKeys + k0;
            if (key >= there) {                             // whatever was in the stage
              y[i] = make_uint4(0, 0, 0, 0);
              cd[i] = 127;
            }
            // 2^(code - 127) 2^120 in two factors within bf16's range
            const int e = (int)cd[i] - 7;                   // exponent of the product, as 120 + code - 127
            const int e1 = min(e, 127), e2 = e - e1;
            const uint32_t f1 = cd[i] == 255 ? 0x7fff7fffu : (uint32_t)(e1 + 127) * 0x00800080u;
            const uint32_t src[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
            uint32_t o[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              o[2 * k] = mul_bf16x2(e4m3x2_bf16_small(src[k]), f1);
              o[2 * k + 1] = mul_bf16x2(e4m3x2_bf16_small(src[k] >> 16), f1);
            }
            // NaN (a magnitude of 0x7f), which the moved fields would turn into 480
            uint32_t nan[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) nan[k] = (src[k] & 0x7f7f7f7fu) + 0x01010101u;
            if ((nan[0] | nan[1] | nan[2] | nan[3]) & 0x80808080u) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                o[2 * k] |= (__byte_perm(nan[k], 0, 0x1404) >> 15 & 0x00010001u) * 0x7fffu;
                o[2 * k + 1] |= (__byte_perm(nan[k], 0, 0x3424) >> 15 & 0x00010001u) * 0x7fffu;
              }
            }
            if (e2 > 0) {
              const uint32_t f2 = (uint32_t)(e2 + 127) * 0x00800080u;
#pragma unroll
              for (int k = 0; k < 8; ++k) o[k] = mul_bf16x2(o[k], f2);
            }
            sts128(base + sw128_offset(key, c16 * 16, 128), make_uint4(o[0], o[1], o[2], o[3]));
            sts128(base + sw128_offset(key, c16 * 16 + 8, 128), make_uint4(o[4], o[5], o[6], o[7]));
          }
        }
        warp_arrive(&bars->rawv_empty[rv]);
        fence_proxy_async_smem();
        warp_arrive(&bars->full[s]);
      }
    }
  }

  if (C::kStaged && warp >= 4 && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  if (*abort) {
    if (tid == 0 && p.dev_status) atomicOr(p.dev_status, GLINATTN_DEV_WAIT_TIMEOUT);
    let_copies_land();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool kF8>
cudaError_t launch(const AttnParams &p, const void *k_cache, const void *v_cache, int ctas, cudaStream_t stream) {
  using C = Cfg<D, kF8>;
  CUtensorMap tq = {}, tk = {}, tv = {}, to = {};
  const long long dims[3] = {D, p.page, p.P > 0 ? (long long)p.P * p.Hkv : 1};
  if (p.P == 0) k_cache = v_cache = p.q;  // an empty pool: nothing is ever loaded
  const long long q_dims[3] = {D, p.H, p.N};
  const int q_box[3] = {(int)C::kQRow / 2, p.G, p.tp};
  if (!encode_map(&tq, p.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, q_dims, q_box,
                              C::kQRow == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  const int o_box[3] = {64, p.G, 32 / p.G};
  if (C::kStaged && 32 % p.G == 0 && !encode_map(&to, p.o, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, q_dims, o_box, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  if (kF8) {
    const int box[3] = {D, p.page, 1};
    if (!encode_map(&tk, k_cache, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, dims, box,
                                D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
      return cudaErrorInvalidValue;
  } else {
    const int box[3] = {64, p.page, 1};
    if (!encode_map(&tk, k_cache, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, dims, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_map(&tv, v_cache, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, dims, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  auto kernel = prefill_kernel<D, kF8>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
  if (e != cudaSuccess) return e;
  kernel<<<ctas, C::kThreads, C::kSmem, stream>>>(tq, tk, tv, to, p, (const uint8_t *)v_cache);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_merge<D, kPrefillRows, false>(p, ctas, stream);
}

}  // namespace

cudaError_t launch_prefill(const AttnParams &p, bool f8, int d, const void *k_cache, const void *v_cache, int ctas,
                           cudaStream_t stream) {
  if (d == 128) return f8 ? launch<128, true>(p, k_cache, v_cache, ctas, stream) : launch<128, false>(p, k_cache, v_cache, ctas, stream);
  return f8 ? launch<64, true>(p, k_cache, v_cache, ctas, stream) : launch<64, false>(p, k_cache, v_cache, ctas, stream);
}

}  // namespace paged
}  // namespace glinattn
