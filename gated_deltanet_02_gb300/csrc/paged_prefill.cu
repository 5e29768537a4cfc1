// paged_prefill.cu -- attention over the paged cache for many query rows per
// (request, key / value head): prompts, pieces of prompts, and batches that mix
// them with single tokens (glinattn_paged_attention).
//
// Mathematics: one pass over the keys with the running maximum m (log2 units)
// and sum l of the softmax per row,
//   S = Q K^T,   P = 2^(S - m),   O += P V,   l += sum P,
// m only moving (and O, l being rescaled) when a tile exceeds it by 2^8: a
// common factor of P, O and l.  S, m, l and O are fp32; P is rounded to bf16
// for the second product (half a step, 2^-8 relative to a weight), which adds
// to the output about what its own rounding to bf16 does.
//
// Kernel: one CTA per SM works on 256 query rows (tokens x heads of a group),
// two tiles of 128 whose S, P and O are in TMEM (P over S: 2 x 128 columns, O:
// 2 x D).  One thread issues the MMAs so that one tile's products run while the
// other's softmax does:  P0 V, Q0 K' | P1 V, Q1 K' | ...  A softmax thread
// owns a row, so no reduction crosses threads.  K and V tiles of 128 keys come
// through a shared-memory ring: TMA, one box per page and 64 channels (bf16);
// an e4m3 cache is read by four converting warps, which scale the values by
// their power of two and write the bf16 tile (exact) where TMA would have put it.
//
// Bound: the tensor core for long prompts (two 128 x 128 x D products per tile
// pair and 128 keys), next to it the exponentials.
#include "paged_sched.cuh"
#include "prefill_tc.cuh"
#include "tc_common.cuh"

namespace glinattn {
namespace paged {
namespace {

using namespace sm100;
using tc::wait_bar;
using tc::wait_bar_warp;
using tc::warp_arrive;

constexpr int kItems = 4;
constexpr float kSlack = 8.f;  // log2 of the largest weight

template <int D, bool kF8>
struct Cfg {
  static constexpr int kThreads = kF8 ? 512 : 384;
  static constexpr uint32_t kQTile = 128 * D * 2;
  static constexpr uint32_t kStageBytes = kTileKeys * D * 2;
  static constexpr int kStages = D == 128 ? (kF8 ? 3 : 4) : 6;
  // e4m3: tiles as they are in the cache (with their scales), before the conversion
  static constexpr int kRawStages = kF8 ? (D == 128 ? 3 : 6) : 0;
  static constexpr uint32_t kRawBytes = kTileKeys * D;
  static constexpr uint32_t kOffRing = 2 * kQTile;
  static constexpr uint32_t kOffRaw = kOffRing + kStages * kStageBytes;
  static constexpr uint32_t kOffScale = kOffRaw + kRawStages * kRawBytes;
  static constexpr uint32_t kOffOut = kOffScale + kRawStages * kTileKeys;  // 2 KiB per softmax warp
  static constexpr uint32_t kOffBars = kOffOut + 8 * 2048;
  static constexpr uint32_t kBytesBars = 1024;
  static constexpr uint32_t kSmem = kOffBars + kBytesBars + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static constexpr uint32_t kColS = 0, kColO = 256;
};

struct Bars {
  uint64_t full[6], empty[6], raw_full[6], raw_empty[6];
  uint64_t s_ready[2], p_ready[2][2], q_ready[2], o_done[2];
  uint64_t item_full[kItems], item_empty[kItems];
  Item item[kItems];
  PlanShared plan;
  int bad[kItems];
  uint32_t tmem;
  int abort;
};

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
template <int kRegs>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// Tiles [j0, j1) that row tile w of the item looks at: up to its last row's key.
__device__ __forceinline__ int last_tile(const Item &it, int G, int w) {
  const int nrow = it.ntok * G;
  const int last = min(128 * (w + 1), nrow) - 1;  // its last row
  const int end = it.pos0 + last / G + 1;
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

template <int D, bool kF8>
__global__ void __launch_bounds__(kF8 ? 512 : 384, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const AttnParams p,
                   const uint8_t *k_cache, const uint8_t *v_cache) {
  using C = Cfg<D, kF8>;
  constexpr int ST = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Bars *bars = reinterpret_cast<Bars *>(smem + C::kOffBars);
  static_assert(sizeof(Bars) <= C::kBytesBars, "barrier block");
  volatile int *abort = &bars->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sb = smem_u32(smem);

  if (tid == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(&bars->full[s], kF8 ? 4 : 1);
      mbar_init(&bars->empty[s], 1);
    }
    for (int s = 0; s < C::kRawStages; ++s) {
      mbar_init(&bars->raw_full[s], 1);
      mbar_init(&bars->raw_empty[s], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->s_ready[i], 1);
      mbar_init(&bars->p_ready[i][0], 4);
      mbar_init(&bars->p_ready[i][1], 4);
      mbar_init(&bars->q_ready[i], 4);
      mbar_init(&bars->o_done[i], 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&bars->item_full[i], 1);
      mbar_init(&bars->item_empty[i], 1 + 8 + (kF8 ? 4 : 0));
      bars->bad[i] = 0;
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
  const Plan plan = make_plan<false>(p, &bars->plan);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int pages = kTileKeys >> p.page_shift;  // pages of a tile

  if (warp < 4) {
    // registers a thread: 64 + 2 x 184 + 80 of 4 x 128 (e4m3), 80 + 2 x 208 of 3 x 168
    regs_dec<kF8 ? 64 : 80>();
    if (warp == 0) {
      // ============ the walk over the items, and TMA ============
      Walk<false> walk(p, plan, lane);
      Item it;
      uint32_t sc = 0, slot = 0;
      for (bool ok = true; ok;) {
        const bool more = walk.next(it, lane);
        const int si = slot % kItems;
        if (!(ok = wait_bar_warp(&bars->item_empty[si], ((slot / kItems) & 1u) ^ 1u, abort))) break;
        if (!more) it.kind = -1;
        if (lane == 0) {
          bars->item[si] = it;
          bars->bad[si] = 0;
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
          if (__any_sync(0xffffffffu, op && !good) && lane == 0) bars->bad[si] = 1;
          const uint32_t ops = (uint32_t)__popc(__ballot_sync(0xffffffffu, op && good));
          const uint32_t bytes = kF8 ? ops * (uint32_t)p.page * (D + 1) : ops << (p.page_shift + 7);
          const size_t plane = (size_t)(good ? id : 0) * p.Hkv + it.hk;
#pragma unroll
          for (int v = 0; v < 2; ++v, ++sc) {
            if constexpr (kF8) {
              const uint32_t s = sc % C::kRawStages;
              if (!(ok = wait_bar_warp(&bars->raw_empty[s], ((sc / C::kRawStages) & 1u) ^ 1u, abort))) break;
              if (lane == 0) mbar_arrive_expect_tx(&bars->raw_full[s], bytes);
              __syncwarp();
              if (op && good) {
                bulk_load(smem + C::kOffRaw + s * C::kRawBytes + pl * p.page * D, (v ? v_cache : k_cache) + plane * p.page * D,
                          (uint32_t)p.page * D, &bars->raw_full[s]);
                bulk_load(smem + C::kOffScale + s * kTileKeys + pl * p.page, (v ? p.v_scale : p.k_scale) + plane * p.page,
                          (uint32_t)p.page, &bars->raw_full[s]);
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
    } else if (warp == 1 && lane == 0) {
      // ============ MMA issue ============
      constexpr uint32_t id_s = idesc_bf16(128, 128, false, false), id_o = idesc_bf16(128, D, false, true);
      uint32_t sc = 0, slot = 0, np[2] = {0, 0}, nq[2] = {0, 0};
      // S_w = Q_w K^T from the stage of number k
      auto issue_s = [&](int w, uint32_t k) {
        const uint32_t a = sb + w * C::kQTile, b = sb + C::kOffRing + (k % ST) * C::kStageBytes;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = (ks >> 2) * 16384 + (ks & 3) * 32;
          umma_bf16(tmem + C::kColS + 128 * w, desc_sw128(a + off, 16, 1024), desc_sw128(b + off, 16, 1024), id_s, ks > 0);
        }
        umma_commit(&bars->s_ready[w]);
      };
      // O_w (+)= P_w V
      auto issue_o = [&](int w, uint32_t k, bool first) -> bool {
        const uint32_t b = sb + C::kOffRing + (k % ST) * C::kStageBytes, ph = np[w]++ & 1u;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          if (ks % 4 == 0) {  // 64 keys' weights at a time
            if (!wait_bar(&bars->p_ready[w][ks / 4], ph, abort)) return false;
            tc_fence_after();
          }
          umma_bf16_tmem_a(tmem + C::kColO + D * w, tmem + C::kColS + 128 * w + 8 * ks, desc_sw128(b + ks * 2048, 16384, 1024), id_o,
                           ks > 0 || !first);
        }
        return true;
      };
      auto landed = [&](uint32_t k) -> bool {
        if (!wait_bar(&bars->full[k % ST], (k / ST) & 1u, abort)) return false;
        tc_fence_after();
        return true;
      };
      for (bool ok = true; ok;) {
        const int si = slot % kItems;
        if (!wait_bar(&bars->item_full[si], (slot / kItems) & 1u, abort)) break;
        const Item it = bars->item[si];
        mbar_arrive(&bars->item_empty[si]);
        if (it.kind < 0) break;
        ++slot;
        const int n = it.j1 - it.j0, n0 = last_tile(it, p.G, 0) - it.j0, n1 = last_tile(it, p.G, 1) - it.j0;
        // tile j of the item: K at stage number sc + 2 j, V behind it
        if (!(ok = landed(sc))) break;
        for (int w = 0; w < 2 && ok; ++w) {
          if ((w ? n1 : n0) <= 0) continue;
          ok = wait_bar(&bars->q_ready[w], nq[w]++ & 1u, abort);
          if (ok) issue_s(w, sc);
        }
        if (!ok) break;
        umma_commit(&bars->empty[sc % ST]);
        for (int j = 0; j < n && ok; ++j) {
          const uint32_t kv = sc + 2 * j + 1, kk = kv + 1;
          ok = landed(kv) && (j + 1 >= n || landed(kk));
          if (!ok) break;
          for (int w = 0; w < 2 && ok; ++w) {
            const int nw = w ? n1 : n0;
            if (j < nw) {
              ok = issue_o(w, kv, j == 0);
              if (ok && j + 1 == nw) umma_commit(&bars->o_done[w]);
            }
            if (ok && j + 1 < nw) issue_s(w, kk);
          }
          if (!ok) break;
          umma_commit(&bars->empty[kv % ST]);
          if (j + 1 < n) umma_commit(&bars->empty[kk % ST]);
        }
        sc += 2 * n;
      }
    }
  } else if (warp < 12) {
    // ============ softmax: row tile w, thread = row ============
    regs_inc<kF8 ? 184 : 208>();
    const int w = warp >= 8 ? 1 : 0, q4 = warp & 3;
    const int lrow = 32 * q4 + lane, row = 128 * w + lrow;
    const uint32_t lane_base = (uint32_t)(32 * q4) << 16;
    const uint32_t tS = tmem + C::kColS + 128 * w + lane_base, tO = tmem + C::kColO + D * w + lane_base;
    uint32_t sc = 0, slot = 0, ns = 0, nd = 0;
    const uint32_t inv_g = (65535u + p.G) / p.G;  // row / G is row * inv_g >> 16 for row, G <= 256
    // a row's place among the item's rows of q and o, in elements
    auto row_at = [&](const Item &it, int r) -> size_t {
      const int tok = (int)((uint32_t)r * inv_g >> 16);
      return ((size_t)(it.row0 + tok) * p.H + it.hk * p.G + (r - tok * p.G)) * D;
    };
    // q of the warp's 32 rows into shared memory, D / 8 lanes a row; rows past
    // the last are zero.  Only for a row tile that has work in the item: its
    // softmax warps then wait for the MMA warp's answer, so that q_ready is
    // never a phase ahead of its reader.
    auto load_q = [&](const Item &it) {
      if (it.kind < 0 || last_tile(it, p.G, w) <= it.j0) return;
      constexpr int kLanes = D / 8, kPer = 32 / kLanes;
      const int c = lane % kLanes, nrow = it.ntok * p.G;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 x[16 / kPer];
#pragma unroll
        for (int k = 0; k < 16 / kPer; ++k) {
          const int r = 128 * w + 32 * q4 + 16 * h + k * kPer + lane / kLanes;
          x[k] = r < nrow ? __ldg(reinterpret_cast<const uint4 *>(p.q + row_at(it, r)) + c) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < 16 / kPer; ++k)
          sts128(sb + w * C::kQTile + sw128_offset(32 * q4 + 16 * h + k * kPer + lane / kLanes, c * 8, 128), x[k]);
      }
      fence_proxy_async_smem();
      warp_arrive(&bars->q_ready[w]);
    };
    bool ok = wait_bar_warp(&bars->item_full[0], 0, abort);
    Item it;
    if (ok) {
      it = bars->item[0];
      load_q(it);
    }
    while (ok && it.kind >= 0) {
      const int si = slot % kItems;
      const int n = it.j1 - it.j0, nw = last_tile(it, p.G, w) - it.j0;
      const int end = it.pos0 + it.ntok;                    // keys behind it are not there
      const int lim = it.pos0 + (int)((uint32_t)row * inv_g >> 16);  // the row's last key
      const int first_lim = it.pos0 + (128 * w) / p.G;      // the first row's
      const bool zero0 = last_tile(it, p.G, 0) == it.j1;    // tile 0 looks at the last cache tile
      float m = -INFINITY, l = 0.f;
      for (int jj = 0; jj < nw; ++jj) {
        const int j = it.j0 + jj;
        if (!(ok = wait_bar_warp(&bars->s_ready[w], ns++ & 1u, abort))) break;
        tc_fence_after();
        float s[128];
        tmem_ld32x2(tS, tS + 32, *reinterpret_cast<float(*)[32]>(s), *reinterpret_cast<float(*)[32]>(s + 32));
        tmem_ld32x2(tS + 64, tS + 96, *reinterpret_cast<float(*)[32]>(s + 64), *reinterpret_cast<float(*)[32]>(s + 96));
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
          mt = fmaxf(max3(a[0], a[1], a[2]), a[3]) * p.c;
        }
        const bool need = mt > m + kSlack;
        if (__any_sync(0xffffffffu, need)) {
          // S of this tile was issued behind the previous tile's P V, so O is complete
          const float mn = need ? mt : m;
          const float f = need ? ex2(m - mn) : 1.f;
          l *= f;
          m = mn;
          if (jj > 0) {
#pragma unroll
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
        const float ms = m == -INFINITY ? 0.f : m;
        const float2 c2 = make_float2(p.c, p.c), m2 = make_float2(-ms, -ms);
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
            // the row tile's last cache tile: its values have landed; rows behind the cache's end become zeros
            const uint32_t vs = sc + 2 * jj + 1;
            if (!(ok = wait_bar_warp(&bars->full[vs % ST], (vs / ST) & 1u, abort))) break;
            if (!kF8 && j == it.j1 - 1 && (w == 0 || !zero0) && j * kTileKeys + lrow >= end) {
              const uint32_t a = sb + C::kOffRing + (vs % ST) * C::kStageBytes + lrow * 128;
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                sts128(a + 16 * k, make_uint4(0, 0, 0, 0));
                if (D == 128) sts128(a + 16384 + 16 * k, make_uint4(0, 0, 0, 0));
              }
            }
            fence_proxy_async_smem();
          }
          tmem_st32(tS + 32 * h, u);
          tc_fence_before();
          warp_arrive(&bars->p_ready[w][h]);
        }
        if (!ok) break;
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      }
      if (!ok) break;
      sc += 2 * n;
      // ---- the next item's q, before this item's outputs
      ++slot;
      if (!(ok = wait_bar_warp(&bars->item_full[slot % kItems], (slot / kItems) & 1u, abort))) break;
      const Item nx = bars->item[slot % kItems];
      load_q(nx);
      const int bad = bars->bad[si];
      const bool has = row < it.ntok * p.G;
      const size_t pslot = (size_t)(2 * blockIdx.x + (it.kind == 1 ? 1 : 0));
      if (nw > 0) {
        if (!(ok = wait_bar_warp(&bars->o_done[w], nd++ & 1u, abort))) break;
        tc_fence_after();
        const float inv = l == 0.f ? 0.f : 1.f / l;
        // outputs through shared memory, 32 channels of the warp's 32 rows at a
        // time, so that 4 lanes write 64 contiguous bytes of a row
        const uint32_t stage = sb + C::kOffOut + (warp - 4) * 2048;
        __nv_bfloat16 *dst[4];
        bool put[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 128 * w + 32 * q4 + 8 * i + (lane >> 2);
          put[i] = it.kind == 0 && !bad && r < it.ntok * p.G;
          dst[i] = p.o + row_at(it, r) + (lane & 3) * 8;
        }
#pragma unroll
        for (int k = 0; k < D; k += 32) {
          float o[32];
          tmem_ld32(tO + k, o);
          if (it.kind == 0) {
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint32_t u[4];
#pragma unroll
              for (int x = 0; x < 4; ++x)
                u[x] = l == 0.f ? 0u : pack_bf16(o[e + 2 * x] * inv, o[e + 2 * x + 1] * inv);
              sts128(stage + lane * 64 + (((e / 8) ^ ((lane >> 1) & 3)) << 4), make_uint4(u[0], u[1], u[2], u[3]));
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = 8 * i + (lane >> 2);
              const uint4 v = lds128(stage + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) << 4));
              if (put[i]) *reinterpret_cast<uint4 *>(dst[i] + k) = v;
            }
          } else if (has) {
            float4 *part = reinterpret_cast<float4 *>(p.part) + (pslot * (D / 4) + k / 4) * kPrefillRows + row;
#pragma unroll
            for (int e = 0; e < 32; e += 4) part[e / 4 * kPrefillRows] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
        }
        tc_fence_before();
      }
      if (it.kind != 0 && has) p.ml[pslot * kPrefillRows + row] = make_float2(m, l);
      if (lrow == 0) {
        if (it.kind != 0 && w == 0) p.skip[pslot] = bad;
        if (bad && p.dev_status) atomicOr(p.dev_status, GLINATTN_DEV_BAD_SLOT);
      }
      warp_arrive(&bars->item_empty[si]);
      it = nx;
    }
  } else if constexpr (kF8) {
    // ============ e4m3 cache: raw tile -> values times their scale, as the bf16 tile ============
    regs_dec<80>();
    const int ct = tid - 384;
    constexpr int kLanes = D / 16;                   // lanes of a key's row, 16 values each
    constexpr int kKeys = 128 / kLanes;              // keys a pass of the 128 threads takes: 16 or 32
    constexpr int kPass = kTileKeys / kKeys;
    const int c16 = ct % kLanes, k0 = ct / kLanes;   // key of pass i: i kKeys + k0
    uint32_t sc = 0, slot = 0;
    for (bool ok = true; ok;) {
      const int si = slot % kItems;
      if (!(ok = wait_bar_warp(&bars->item_full[si], (slot / kItems) & 1u, abort))) break;
      const int kind = bars->item[si].kind, j1 = bars->item[si].j1;
      const int end = bars->item[si].pos0 + bars->item[si].ntok;
      int j = bars->item[si].j0;
      warp_arrive(&bars->item_empty[si]);
      if (kind < 0) break;
      ++slot;
      for (; j < j1 && ok; ++j) {
#pragma unroll 1
        for (int v = 0; v < 2; ++v, ++sc) {
          const uint32_t rs = sc % C::kRawStages, s = sc % ST;
          if (!(ok = wait_bar_warp(&bars->raw_full[rs], (sc / C::kRawStages) & 1u, abort))) break;
          const uint32_t raw = sb + C::kOffRaw + rs * C::kRawBytes;
          const uint8_t *scale = smem + C::kOffScale + rs * kTileKeys;
          uint4 y[kPass];
          uint32_t cd[kPass];
#pragma unroll
          for (int i = 0; i < kPass; ++i) {
            const int key = i * kKeys + k0;
            y[i] = lds128(raw + key * D + c16 * 16);
            cd[i] = scale[key];
            if (j * kTileKeys + key >= end) {  // not there: whatever was in the stage
              y[i] = make_uint4(0, 0, 0, 0);
              cd[i] = 127;
            }
          }
          warp_arrive(&bars->raw_empty[rs]);
          if (!(ok = wait_bar_warp(&bars->empty[s], ((sc / ST) & 1u) ^ 1u, abort))) break;
          const uint32_t base = sb + C::kOffRing + s * C::kStageBytes;
#pragma unroll
          for (int i = 0; i < kPass; ++i) {
            // 2^(code - 127) 2^120 in two factors within bf16's range
            const int e = (int)cd[i] - 7;                     // exponent of the product, as 120 + code - 127
            const int e1 = min(e, 127), e2 = e - e1;
            const uint32_t f1 = cd[i] == 255 ? 0x7fff7fffu : (uint32_t)(e1 + 127) * 0x00800080u;
            const uint32_t f2 = (uint32_t)(e2 + 127) * 0x00800080u;
            const uint32_t src[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
            uint32_t o[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              o[2 * k] = mul_bf16x2(e4m3x2_bf16_small(src[k] & 0xffffu), f1);
              o[2 * k + 1] = mul_bf16x2(e4m3x2_bf16_small(src[k] >> 16), f1);
            }
            if (e2 > 0) {
#pragma unroll
              for (int k = 0; k < 8; ++k) o[k] = mul_bf16x2(o[k], f2);
            }
            const int key = i * kKeys + k0;
            const uint32_t a = base + sw128_offset(key, c16 * 16, 128), b = base + sw128_offset(key, c16 * 16 + 8, 128);
            sts128(a, make_uint4(o[0], o[1], o[2], o[3]));
            sts128(b, make_uint4(o[4], o[5], o[6], o[7]));
          }
          fence_proxy_async_smem();
          warp_arrive(&bars->full[s]);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort && tid == 0 && p.dev_status) atomicOr(p.dev_status, GLINATTN_DEV_WAIT_TIMEOUT);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool kF8>
cudaError_t launch(const AttnParams &p, const void *k_cache, const void *v_cache, int ctas, cudaStream_t stream) {
  using C = Cfg<D, kF8>;
  CUtensorMap tk = {}, tv = {};
  if (!kF8) {
    const long long dims[3] = {D, p.page, p.P > 0 ? (long long)p.P * p.Hkv : 1};
    const int box[3] = {64, p.page, 1};
    if (p.P == 0) k_cache = v_cache = p.q;  // an empty pool: nothing is ever loaded
    if (!encode_3d_map(&tk, k_cache, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, dims, box, true) ||
        !encode_3d_map(&tv, v_cache, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, dims, box, true))
      return cudaErrorInvalidValue;
  }
  auto kernel = prefill_kernel<D, kF8>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
  if (e != cudaSuccess) return e;
  kernel<<<ctas, C::kThreads, C::kSmem, stream>>>(tk, tv, p, (const uint8_t *)k_cache, (const uint8_t *)v_cache);
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
