// bf16 scored-attention forward on tcgen05 tensor cores (d, dv <= 128).
//
// The pipeline is that of the plain forward (fwd_bf16.cu): one persistent CTA
// per SM, a unit of two 128-row query tiles that share every K/V tile, a
// producer warp (TMA, one K/V ring), an MMA warp, and two softmax warpgroups
// with a thread per query row, which keep a row's 128 scores in registers and
// write P (bf16) over them in tensor memory. What differs:
//   - rows are the packed rows of a key head (scored.h), so grouped query
//     heads share key tiles with no copy;
//   - each row tile of a unit runs over its own key tiles, those its ranges'
//     hull meets, and only tiles with a key that some row does not see are
//     masked, by each row's range;
//   - scores are capped and biased in the softmax threads (scored_math.cuh);
//   - units are claimed at run time (documents make their lengths unequal),
//     longest first under a causal mask;
//   - rows of V outside the unit's hull are zeroed in shared memory (P is 0
//     there, but 0 times what an unused cache row holds need not be).
// TMEM: row tile t keeps S_t (and P_t over it) at columns [256 t, 256 t +
// 128) and O_t at [256 t + 128, 256 t + 128 + dv).
#include <cuda.h>
#include <cuda_bf16.h>
#include <math_constants.h>
#include <stdint.h>

#include <type_traits>

#include "bwd_common.cuh"
#include "common.cuh"
#include "ptx.cuh"
#include "scored.h"
#include "scored_math.cuh"
#include "scored_queue.cuh"

namespace attn {
namespace scored_fwd {

using scored::Cap;
using scored::add2;
using scored::dup;
using scored::f2;
using scored::F2;
using scored::fma2;
using scored::mul2;

constexpr int BM = 128, BN = 128;
constexpr int BOX_BYTES = 128 * 64 * 2;
constexpr float TAU = 8.0f;        // the running reference moves when the maximum grows by more (log2 units)
constexpr int NUM_THREADS = 384;
constexpr int REG_CTRL = 96;
constexpr int REG_SOFTMAX = 200;

// A unit: the row tiles 2 qb and 2 qb + 1 of key head bh, the key tiles
// [s[t], e[t]) of each, [s0, e0) of both, and the hull [lo, hi) of their keys.
// With few units the key tiles are cut into ranges (splits), as units of their
// own: the tiles are then those of the unit's range.
struct Unit {
  int bh, b, qb, split, s[2], e[2], s0, e0, lo, hi;
  int all_lo[2], all_hi[2];   // keys that every row of the tile sees
};
using Ring = scored::UnitRing<Unit>;

// One tile width for Q, K, V and O rows: 64 where d and dv fit, else 128.
template <int HD>
struct Cfg {
  static constexpr int KB = HD / 64;
  static constexpr int TILE = BM * HD * 2;
  static constexpr int NSLOT_FIT = (227 * 1024 - 2 * TILE - 1024) / TILE;
  static constexpr int NSLOT = NSLOT_FIT < 10 ? NSLOT_FIT : 10;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_KV = OFF_Q + 2 * TILE;
  static constexpr int OFF_BAR = OFF_KV + NSLOT * TILE;
  // q_full, q_empty, full[NSLOT], empty[NSLOT], s_full[2], p_full[2], o_full[2], drain, unit queue
  static constexpr int NBAR = 2 + 2 * NSLOT + 7 + 2 * Ring::N;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM = OFF_MISC + 16 + Ring::BYTES;
  static constexpr int READERS = 1 + 256;
  static constexpr uint32_t IDESC_S = ptx::idesc_bf16(BM, BN, false, false);
  static constexpr uint32_t IDESC_PV = ptx::idesc_bf16(BM, HD, false, true);
};

struct Params {
  ScoredProblem p;
  ScoredPlan plan;
  __nv_bfloat16* O;
  float* LSE;
  uint32_t* status;
  int n_pairs, total, group;
  float sc2;   // scale * log2(e)
  Cap cap;
  int n_splits, split_tiles;
  float* Opart;     // [n_splits][B * Hkv * R][dv]
  float* LSEpart;   // [n_splits][B * Hkv * R]
};

__device__ __forceinline__ Unit load_unit(const Params& P, int x) {
  Unit u;
  bwd::grouped_unit(x, P.n_pairs * P.n_splits, P.p.B * P.p.Hkv, P.group, true, &u.bh, &u.qb);
  u.split = u.qb % P.n_splits;
  u.qb = scored::packed_block(u.qb / P.n_splits, P.n_pairs, P.p.G);
  u.b = u.bh / P.p.Hkv;
  u.lo = 0x7fffffff;
  u.hi = 0;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int rt = 2 * u.qb + t;
    const int4 tile = rt < P.p.n_rt ? __ldg(P.plan.tiles + static_cast<long long>(u.b) * P.p.n_rt + rt)
                                    : make_int4(0, 0, 0x7fffffff, 0);
    const bool live = tile.y > 0;
    u.s[t] = live ? max(tile.x / BN, u.split * P.split_tiles) : 0;
    u.e[t] = live ? max(min((tile.y + BN - 1) / BN, (u.split + 1) * P.split_tiles), u.s[t]) : 0;
    u.all_lo[t] = tile.z;
    u.all_hi[t] = tile.w;
    if (live) {
      u.lo = min(u.lo, tile.x);
      u.hi = max(u.hi, tile.y);
    }
  }
  u.s0 = u.hi > 0 ? max(u.lo / BN, u.split * P.split_tiles) : 0;
  u.e0 = max(min((u.hi + BN - 1) / BN, (u.split + 1) * P.split_tiles), u.s0);
  return u;
}

// SPLIT: key ranges as units of their own, with partial results.
template <int HD, bool CAP, bool BIAS, bool SPLIT>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    scored_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Params P) {
  using C = Cfg<HD>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if ((ptx::smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicOr(P.status, ATTN_DEV_BAD_SMEM);
    return;
  }
  uint8_t* sQ = smem + C::OFF_Q;
  uint8_t* sKV = smem + C::OFF_KV;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* q_full = bars + 0;
  uint64_t* q_empty = bars + 1;
  uint64_t* kv_full = bars + 2;
  uint64_t* kv_empty = kv_full + C::NSLOT;
  uint64_t* s_full = kv_empty + C::NSLOT;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 2;
  uint64_t* drain = o_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC + 4);
  const Ring ring{reinterpret_cast<Unit*>(smem + C::OFF_MISC + 16), drain + 1, drain + 1 + Ring::N};

  if (threadIdx.x == 0) {
    ptx::mbar_init(q_full, 1);
    ptx::mbar_init(q_empty, 1);
    for (int s = 0; s < C::NSLOT; ++s) {
      ptx::mbar_init(kv_full + s, 1);
      ptx::mbar_init(kv_empty + s, 1);
    }
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(s_full + t, 1);
      ptx::mbar_init(p_full + t, 128);
      ptx::mbar_init(o_full + t, 1);
    }
    ptx::mbar_init(drain, 1);
    ring.init(C::READERS);
    *abort_flag = 0u;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(tmem_slot, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // Item i of the K/V stream (K and V of the units' key tiles in order) sits
  // in ring slot i % NSLOT; the counters run across units.
  auto slot = [](uint32_t i) { return static_cast<int>(i % C::NSLOT); };
  auto par = [](uint32_t i) { return (i / C::NSLOT) & 1u; };

  const int wg = warp >> 2;
  if (wg == 0) {
    ptx::reg_release<REG_CTRL>();
    if (warp == 0 && lane == 0) {
      // ------------------------------------------------------------ producer
      ptx::WaitCtx w{abort_flag, P.status, 1u};
      ptx::tma_prefetch_desc(&tmQ);
      ptx::tma_prefetch_desc(&tmK);
      ptx::tma_prefetch_desc(&tmV);
      uint32_t item = 0, u_it = 0, pu = 0;
      bool ok = true;
      auto load = [&](int x) { return load_unit(P, x); };
      auto work = [](const Unit& u) { return u.e0 > u.s0; };
      scored::NextUnit<Unit> cur{}, next{};
      ok = cur.first(P.plan.counters, P.total, load, work, ring, &pu, w);
      for (; ok && cur.u.bh >= 0; cur = next) {
        const Unit& u = cur.u;
        if (!(ok = ptx::mbar_wait(q_empty, (u_it & 1u) ^ 1u, w))) break;
        ptx::mbar_arrive_expect_tx(q_full, 2 * C::TILE);
        for (int t = 0; t < 2; ++t)
          for (int c = 0; c < C::KB; ++c)
            ptx::tma_load_3d(sQ + t * C::TILE + c * BOX_BYTES, &tmQ, q_full, c * 64, (2 * u.qb + t) * BM, u.bh);
        ++u_it;
        for (int j = u.s0; ok && j < u.e0; ++j) {
          if (!(ok = next.step(j - u.s0, u.e0 - u.s0, P.plan.counters, P.total, load, work, ring, &pu, w))) break;
          for (int kv = 0; kv < 2; ++kv, ++item) {
            const int sl = slot(item);
            if (!(ok = ptx::mbar_wait(kv_empty + sl, par(item) ^ 1u, w))) break;
            ptx::mbar_arrive_expect_tx(kv_full + sl, C::TILE);
            for (int c = 0; c < C::KB; ++c)
              ptx::tma_load_3d(sKV + sl * C::TILE + c * BOX_BYTES, kv ? &tmV : &tmK, kv_full + sl, c * 64, j * BN,
                               u.bh);
          }
        }
      }
      if (!ok) {
        // let the copies in flight land before the CTA exits
        for (uint32_t n = (item > (uint32_t)C::NSLOT ? item - C::NSLOT : 0u); n < item; ++n)
          ptx::mbar_wait_drain(kv_full + slot(n), par(n));
        if (u_it > 0) ptx::mbar_wait_drain(q_full, (u_it - 1) & 1u);
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      // The whole warp follows the schedule; the lane elect.sync picks (lane
      // 0) issues the MMAs and commits (see fwd_bf16.cu).
      ptx::WaitCtx w{abort_flag, P.status, 3u};
      const uint32_t sQa = ptx::smem_u32(sQ), sKVa = ptx::smem_u32(sKV);
      const uint64_t q_desc[2] = {scored::formed(ptx::sdesc_sw128(sQa, 16, 1024)),
                                  scored::formed(ptx::sdesc_sw128(sQa + C::TILE, 16, 1024))};
      auto k_desc = [&](int sl) { return scored::formed(ptx::sdesc_sw128(sKVa + sl * C::TILE, 16, 1024)); };
      auto v_desc = [&](int sl) { return scored::formed(ptx::sdesc_sw128(sKVa + sl * C::TILE, BOX_BYTES, 1024)); };
      // (unrolled by 4: whole, the eight products of each call fill the
      // instruction cache, 141 in place of 138 us at B=2 H=16 T=4096 d=128
      // with a cap; one at a time, the loop holds them up, 149)
      auto mma_S = [&](int t, uint64_t k) {
        const uint32_t d = tmem + t * 256;
#pragma unroll 4
        for (int kk = 0; kk < HD / 16; ++kk) {
          const uint32_t off = (kk >> 2) * BOX_BYTES + (kk & 3) * 32;
          ptx::mma_ss(d, ptx::sdesc_advance(q_desc[t], off), ptx::sdesc_advance(k, off), C::IDESC_S, kk > 0 ? 1u : 0u);
        }
        ptx::mma_commit(s_full + t);
      };
      auto mma_PV = [&](int t, uint64_t v, bool acc) {
        const uint32_t d = tmem + t * 256 + 128, a = tmem + t * 256;
#pragma unroll 4
        for (int kk = 0; kk < BN / 16; ++kk)
          ptx::mma_ts(d, a + kk * 8, ptx::sdesc_advance(v, kk * 2048), C::IDESC_PV, (acc || kk > 0) ? 1u : 0u);
      };
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, w));
      };
      uint32_t item = 0, u_it = 0, ru = 0, pp[2] = {0u, 0u};
      bool moved = false;
      auto next_unit = [&](Unit* u) {
        if (!ring.read(ru, u, w)) return false;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ring.empty + ru % Ring::N);
        ++ru;
        return true;
      };
      Unit u, un;
      bool ok = next_unit(&u);
      while (ok && u.bh >= 0) {
        const int n = u.e0 - u.s0;
        const uint64_t k0 = k_desc(slot(item));
        if (!(ok = wait(q_full, u_it & 1u))) break;
        if (!(ok = wait(kv_full + slot(item), par(item)))) break;
        ptx::tc_fence_after();
        // (selects by constant index keep pp, s and e in registers)
        if (ptx::elect_one()) {
          moved |= lane != 0;
          if (u.s[0] == u.s0 && u.e[0] > u.s[0]) mma_S(0, k0);
          if (u.s[1] == u.s0 && u.e[1] > u.s[1]) mma_S(1, k0);
          ptx::mma_commit(kv_empty + slot(item));
          if (n == 1) ptx::mma_commit(q_empty);   // no later MMA reads Q: the next unit's may load
        }
        __syncwarp();
        // each step waits for the next step's tiles while its own MMAs run
        if (!(ok = wait(kv_full + slot(item + 1), par(item + 1)))) break;
        if (n > 1 && !(ok = wait(kv_full + slot(item + 2), par(item + 2)))) break;
        for (int j = u.s0; j < u.e0; ++j, item += 2) {
          if (j + 1 == u.e0 && !(ok = next_unit(&un))) break;
          const uint32_t iv = item + 1, ikn = item + 2;   // V_j, K_{j+1}: resident
          const uint64_t v = v_desc(slot(iv)), k = k_desc(slot(ikn));
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const bool act = j >= u.s[t] && j < u.e[t];
            const bool next = j + 1 >= u.s[t] && j + 1 < u.e[t];
            if (act) {
              if (!(ok = wait(p_full + t, pp[t] & 1u))) break;
              ++pp[t];
              ptx::tc_fence_after();
            }
            if (ptx::elect_one()) {
              moved |= lane != 0;
              if (act) mma_PV(t, v, j > u.s[t]);
              if (next) mma_S(t, k);
              if (act && !next) ptx::mma_commit(o_full + t);
              if (t == 1) {
                ptx::mma_commit(kv_empty + slot(iv));
                if (j + 1 < u.e0) ptx::mma_commit(kv_empty + slot(ikn));
                if (j + 2 == u.e0) ptx::mma_commit(q_empty);   // the unit's last S products are out
              }
            }
            __syncwarp();
          }
          if (!ok) break;
          if (j + 1 < u.e0 && !(ok = wait(kv_full + slot(iv + 2), par(iv + 2)))) break;
          if (j + 2 < u.e0 && !(ok = wait(kv_full + slot(ikn + 2), par(ikn + 2)))) break;
        }
        if (!ok) break;
        ++u_it;
        u = un;
      }
      if (!ok) {
        if (ptx::elect_one()) ptx::mma_commit(drain);
        __syncwarp();
        ptx::mbar_wait_drain(drain, 0u);
      }
      if (__any_sync(0xffffffffu, moved) && lane == 0) atomicOr(P.status, ATTN_DEV_ISSUER);
    }
  } else {
    ptx::reg_acquire<REG_SOFTMAX>();
    // ------------------------------------------------------------ softmax
    const int t = wg - 1;
    const int quad = warp & 3;
    const int r = quad * 32 + lane;
    const uint32_t tS = tmem + (static_cast<uint32_t>(quad * 32) << 16) + t * 256;
    const uint32_t tO = tS + 128;
    ptx::WaitCtx w{abort_flag, P.status, 4u + t};
    const float sc2 = P.sc2;
    const F2 sc2v = dup(sc2);
    const int R = P.p.R, dv = P.p.dv;
    uint32_t sp = 0, op = 0, ru = 0, item = 0;
    // A unit as this thread sees it: its row tile's key tiles, its row's range
    // and slope. The next one is read before this one's epilogue, which
    // covers the loads.
    struct Mine {
      int bh, split, row;          // bh < 0: the end; row: of this thread; n_rt * 128 where the tile does not exist
      int s0, items;               // the unit's first key tile, its K/V items
      int s, e;                    // this row tile's key tiles
      int lo, hi;                  // hull of the unit's keys
      int all_lo, all_hi;          // keys every row of the tile sees
      int from, to, pos;           // this row's range and position
      float slope2;
    };
    auto next_unit = [&](Mine* m) {
      Unit u;
      if (!ring.read(ru, &u, w)) return false;
      ptx::mbar_arrive(ring.empty + ru % Ring::N);
      ++ru;
      m->bh = u.bh;
      if (u.bh < 0) return true;
      if (SPLIT) m->split = u.split;
      m->s0 = u.s0;
      m->items = 2 * (u.e0 - u.s0);
      m->lo = u.lo;
      m->hi = u.hi;
      m->s = t ? u.s[1] : u.s[0];
      m->e = t ? u.e[1] : u.e[0];
      m->all_lo = t ? u.all_lo[1] : u.all_lo[0];
      m->all_hi = t ? u.all_hi[1] : u.all_hi[0];
      m->row = min(2 * u.qb + t, P.p.n_rt) * BM + r;
      if (2 * u.qb + t < P.p.n_rt) {
        const int4 ri = __ldg(P.plan.rows + static_cast<long long>(u.b) * P.p.rpad() + m->row);
        m->from = ri.x;
        m->to = ri.y;
        m->pos = ri.z;
        if (BIAS && m->row < R)
          m->slope2 =
              __ldg(P.p.slopes + (u.bh - u.b * P.p.Hkv) * P.p.G + m->row / P.p.Tq) * scored::kLog2e;
      }
      return true;
    };
    Mine me{}, nx{};
    bool ok = next_unit(&me);
    while (ok && me.bh >= 0) {
      const int s_t = me.s, e_t = me.e;
      const float slope2 = me.slope2;
      float m_used = -CUDART_INF_F, l = 0.f;
      for (int j = s_t; j < e_t; ++j) {
        const int kv0 = j * BN;
        // every lane must agree before the warp-wide tcgen05 loads
        if (!(ok = __all_sync(0xffffffffu, ptx::mbar_wait(s_full + t, sp & 1u, w)))) break;
        ++sp;
        ptx::tc_fence_after();
        uint32_t raw[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) ptx::tmem_ld32(tS + c * 32, raw[c]);
        // a key of the tile that some row does not see
        const bool partial = kv0 < me.all_lo || kv0 + BN > me.all_hi;
        if (partial && (kv0 < me.lo || kv0 + BN > me.hi)) {
          // the unit's first or last key tile: zero the rows of V that no row sees
          const uint32_t iv = item + 2 * (j - me.s0) + 1;
          if (!(ok = __all_sync(0xffffffffu, ptx::mbar_wait(kv_full + slot(iv), par(iv), w)))) break;
          if (kv0 + r < me.lo || kv0 + r >= me.hi) {
#pragma unroll
            for (int c = 0; c < C::KB; ++c) scored::zero_box_row(sKV + slot(iv) * C::TILE + c * BOX_BYTES, r);
          }
          ptx::fence_proxy_async_smem();
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) ptx::tmem_ld_wait(raw[c]);
        float* s = reinterpret_cast<float*>(&raw[0][0]);
        // Maxima of the raw scores, with a bias in groups of 8 keys.
        constexpr int NG = BIAS ? 16 : 4;
        float gm[NG];
        auto maxima = [&] {
          if constexpr (BIAS) {
#pragma unroll
            for (int g = 0; g < 16; ++g)
              gm[g] = ptx::fmax3(ptx::fmax3(s[8 * g], s[8 * g + 1], s[8 * g + 2]),
                                 ptx::fmax3(s[8 * g + 3], s[8 * g + 4], s[8 * g + 5]),
                                 fmaxf(s[8 * g + 6], s[8 * g + 7]));
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) gm[k] = fmaxf(s[k], s[k + 4]);
#pragma unroll
            for (int i = 8; i < 128; i += 8)
#pragma unroll
              for (int k = 0; k < 4; ++k) gm[k] = ptx::fmax3(gm[k], s[i + k], s[i + 4 + k]);
          }
        };
        auto all_max = [&] {
          float m = fmaxf(gm[NG - 2], gm[NG - 1]);
#pragma unroll
          for (int g = 0; g < NG - 2; g += 2) m = ptx::fmax3(m, gm[g], gm[g + 1]);
          return m;
        };
        int form = 0;   // of the cap
        if constexpr (CAP) {
          // (minima and maxima in one instruction each; absolute values would take one of their own)
          maxima();
          float n4[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) n4[k] = fminf(s[k], s[k + 4]);
#pragma unroll
          for (int i = 8; i < 128; i += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) n4[k] = ptx::fmin3(n4[k], s[i + k], s[i + 4 + k]);
          form = scored::cap_form(P.cap, ptx::fmin3(n4[0], n4[1], fminf(n4[2], n4[3])), all_max());
        }
        if (partial) {
          // bit i of a word: this row sees the chunk's key i
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t seen = scored::bit_range(me.from - kv0 - 32 * c, me.to - kv0 - 32 * c);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(seen & (1u << i))) s[32 * c + i] = -CUDART_INF_F;
          }
        }
        if (!CAP || partial) maxima();
        // The bias of key i of the tile is c1 * (delta + i) on one side of the
        // row's position; where it changes sides inside the tile for some row
        // of the warp (cross) it is -slope2 |delta + i|.
        const int dist = kv0 - me.pos;
        const float delta = static_cast<float>(dist);
        const float c1 = dist < 0 ? slope2 : -slope2;
        const bool cross = BIAS && __any_sync(0xffffffffu, dist < 0 && dist > -(BN - 1));
        float mx;
        if constexpr (BIAS) {
          // An upper bound of the row's changed scores: per group, its largest
          // score (the cap is monotone) plus its largest bias. It lies above
          // the maximum by at most 8 |slope2|, which moves the exponentials
          // down by so many powers of two and costs no digit; for slopes
          // above 2.7, where that could reach fp32's range, the maximum
          // itself is formed.
          mx = -CUDART_INF_F;
          auto value = [&](float x) {
            if constexpr (CAP)
              return x == -CUDART_INF_F ? x : scored::cap_rough(x, P.cap);
            else
              return x * sc2;
          };
          if (__all_sync(0xffffffffu, fabsf(slope2) <= 4.f)) {
#pragma unroll
            for (int g = 0; g < 16; ++g) {
              // distances of the group's ends; 0 lies between them where their signs differ
              const float a = delta + static_cast<float>(8 * g), z = a + 7.f;
              const float near = fmaxf(fmaxf(a, -z), 0.f), far = fmaxf(fabsf(a), fabsf(z));
              mx = fmaxf(mx, fmaf(-slope2, slope2 > 0.f ? near : far, value(gm[g])));
            }
          } else {
#pragma unroll
            for (int i = 0; i < 128; ++i) mx = fmaxf(mx, fmaf(-slope2, fabsf(delta + static_cast<float>(i)), value(s[i])));
          }
        } else {
          mx = all_max();
          if constexpr (CAP)
            mx = mx == -CUDART_INF_F ? mx : scored::cap_rough(mx, P.cap);   // the cap is monotone
          else
            mx *= sc2;
        }
        const float m_new = fmaxf(m_used, mx);
        bool need = false;
        float corr = 1.0f;
        if (j == s_t) {
          m_used = m_new;
        } else if (m_new > m_used + TAU) {
          need = true;
          corr = ptx::ex2(m_used - m_new);   // 0 when m_used = -inf
          l *= corr;
          m_used = m_new;
        }
        const float ref = (m_used == -CUDART_INF_F) ? 0.f : m_used;   // no key seen yet
        F2 ls[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) ls[k] = dup(0.f);
        const F2 nref = dup(-ref);
        // p = 2^(changed score - ref), in place of the scores. MASKED: under a
        // cap the -inf of a masked score does not pass through, so its p is
        // set; CROSS: the bias by absolute distance.
        auto exps = [&](auto capped, auto masked, auto crossing) {
          constexpr int kForm = decltype(capped)::value;
          constexpr bool kMasked = decltype(masked)::value, kCross = decltype(crossing)::value;
          const scored::CapPoly<kForm == scored::kCapPoly2 ? kForm : scored::kCapPoly4> poly(P.cap);
          F2 off[BIAS && !kCross ? 4 : 1];   // c1 * i of a group's pairs
          if constexpr (BIAS && !kCross) {
#pragma unroll
            for (int k = 0; k < 4; ++k) off[k] = f2(c1 * static_cast<float>(2 * k), c1 * static_cast<float>(2 * k + 1));
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t pk[16];
            uint32_t seen = 0xffffffffu;
            if constexpr (kMasked) seen = scored::bit_range(me.from - kv0 - 32 * c, me.to - kv0 - 32 * c);
            F2 base = nref;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int n = 32 * c + 2 * i;   // key of the tile
              if constexpr (BIAS && !kCross) {
                if (i % 4 == 0) base = dup(fmaf(c1, delta + static_cast<float>(n), -ref));
              }
              F2 b = base;
              if constexpr (BIAS && !kCross) b = add2(off[i % 4], base);
              if constexpr (BIAS && kCross)
                b = f2(fmaf(-slope2, fabsf(delta + static_cast<float>(n)), -ref),
                       fmaf(-slope2, fabsf(delta + static_cast<float>(n + 1)), -ref));
              const F2 v = f2(s[n], s[n + 1]);
              F2 x;
              if constexpr (kForm == 0)
                x = fma2(v, sc2v, b);
              else if constexpr (kForm == scored::kCapFormula)
                x = add2(scored::cap_any(v, P.cap), b);
              else
                x = fma2(v, poly(v), b);
              F2 p = scored::ex2(x);
              if constexpr (kMasked && CAP)
                p = f2(seen & (1u << (2 * i)) ? p.x : 0.f, seen & (2u << (2 * i)) ? p.y : 0.f);
              ls[i & 3] = add2(ls[i & 3], p);
              pk[i] = scored::pack_bf16(p);
            }
            ptx::tmem_st16(tS + 16 * c, pk);
          }
        };
        // (variants of their own where they are frequent: a condition per
        // element would become selects that every tile pays for)
        using bias = std::integral_constant<bool, BIAS>;
        auto either = [&](auto capped) {
          if (BIAS && cross)
            exps(capped, std::true_type{}, bias{});
          else if (CAP && partial)
            exps(capped, std::true_type{}, std::false_type{});
          else
            exps(capped, std::false_type{}, std::false_type{});
        };
        if constexpr (!CAP) {
          either(std::integral_constant<int, 0>{});
        } else {
          if (form == scored::kCapPoly2 && !partial && !(BIAS && cross))
            exps(std::integral_constant<int, scored::kCapPoly2>{}, std::false_type{}, std::false_type{});
          else if (form != scored::kCapFormula)
            either(std::integral_constant<int, scored::kCapPoly4>{});
          else
            exps(std::integral_constant<int, scored::kCapFormula>{}, std::true_type{}, bias{});
        }
        const F2 lsum = add2(add2(ls[0], ls[1]), add2(ls[2], ls[3]));
        l += lsum.x + lsum.y;
        if (__any_sync(0xffffffffu, need)) {
          // O_t *= corr before the next PV product adds to it; the previous
          // one is complete (issued before the S product just consumed)
#pragma unroll 1
          for (int c = 0; c < HD / 32; ++c) {
            uint32_t o[32];
            ptx::tmem_ld32(tO + c * 32, o);
            ptx::tmem_ld_wait(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * corr);
            ptx::tmem_st32(tO + c * 32, o);
          }
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        ptx::mbar_arrive(p_full + t);
      }
      if (!ok) break;
      item += me.items;
      if (!(ok = next_unit(&nx))) break;
      // ---------------------------------------------------------- epilogue
      if (me.row >= P.p.rpad()) {   // an odd number of row tiles
        me = nx;
        continue;
      }
      if (e_t > s_t) {
        if (!(ok = __all_sync(0xffffffffu, ptx::mbar_wait(o_full + t, op & 1u, w)))) break;
        ++op;
        ptx::tc_fence_after();
      }
      const bool none = l == 0.f;   // no key seen (a NaN among the row's scores goes through)
      const float inv_l = none ? 0.f : 1.0f / l;
      const float lse = none ? -CUDART_INF_F : (m_used + log2f(l)) * 0.69314718055994530942f;
      // the four rows of this lane's quad, of which it stores every fourth 16-byte piece
      const int row4 = me.row & ~3;
      const long long head = static_cast<long long>(me.bh) * R;
      const long long part = SPLIT ? static_cast<long long>(me.split) * P.p.B * P.p.Hkv * R + head : 0;
      // (not unrolled: it would displace the softmax code in the instruction
      // cache; 106 in place of 97 us at H=32 Hkv=8 T=8192 d=128 over documents of
      // about 1000 tokens)
#pragma unroll 1
      for (int c = 0; c < HD / 32; ++c) {
        uint32_t o[32];
        ptx::tmem_ld32(tO + c * 32, o);
        ptx::tmem_ld_wait(o);
        uint4 pk[4];
        if constexpr (SPLIT) {   // partial rows, fp32: 16 columns at a time
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t v[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                v[e] = none ? 0u : __float_as_uint(__uint_as_float(o[16 * h + 4 * i + e]) * inv_l);
              pk[i] = make_uint4(v[0], v[1], v[2], v[3]);
            }
            scored::quad_transpose(pk, lane);
            const int col = 32 * c + 16 * h + 4 * (lane & 3);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (row4 + i < R && col < dv)
                *reinterpret_cast<uint4*>(P.Opart + (part + row4 + i) * dv + col) = pk[i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v[e] = none ? 0u
                          : ptx::pack_bf16(__uint_as_float(o[8 * i + 2 * e]) * inv_l,
                                           __uint_as_float(o[8 * i + 2 * e + 1]) * inv_l);
            pk[i] = make_uint4(v[0], v[1], v[2], v[3]);
          }
          scored::quad_transpose(pk, lane);
          const int col = 32 * c + 8 * (lane & 3);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (row4 + i < R && col < dv) *reinterpret_cast<uint4*>(P.O + (head + row4 + i) * dv + col) = pk[i];
        }
      }
      if (me.row < R) (SPLIT ? P.LSEpart + part : P.LSE + head)[me.row] = lse;
      ptx::tc_fence_before();
      me = nx;
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

template <int HD, bool CAP, bool BIAS>
cudaError_t launch(const ScoredFwd& a) {
  using C = Cfg<HD>;
  static_assert(C::SMEM <= 227 * 1024, "shared memory");
  Params P;
  P.p = a.p;
  P.plan = a.plan;
  P.O = static_cast<__nv_bfloat16*>(a.O);
  P.LSE = a.LSE;
  P.status = a.status;
  P.sc2 = a.p.scale * scored::kLog2e;
  P.cap = scored::make_cap(a.p.scale, a.p.softcap);
  const int heads = a.p.B * a.p.Hkv;
  P.n_pairs = scored::packed_blocks((a.p.n_rt + 1) / 2, a.p.G);
  P.n_splits = a.n_splits;
  P.split_tiles = a.split_keys / BN;
  P.Opart = a.Opart;
  P.LSEpart = a.LSEpart;
  P.total = P.n_pairs * P.n_splits * heads;
  // heads in groups whose keys and values fill about half of L2
  const size_t per_head = static_cast<size_t>(a.p.Tk) * (a.p.d + a.p.dv) * 2;
  size_t g = per_head * heads <= 2 * a.l2_bytes ? heads : a.l2_bytes / 2 / per_head;
  P.group = static_cast<int>(g < 1 ? 1 : g > static_cast<size_t>(heads) ? heads : g);
  const int grid = P.total < a.num_sms ? P.total : a.num_sms;
  auto kern = a.n_splits > 1 ? scored_fwd_kernel<HD, CAP, BIAS, true> : scored_fwd_kernel<HD, CAP, BIAS, false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  // the register split must fit the launch allocation (see ptx::reg_acquire)
  cudaFuncAttributes fa;
  if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
  if (fa.numRegs < REG_CTRL || fa.numRegs > REG_SOFTMAX || 3 * fa.numRegs < REG_CTRL + 2 * REG_SOFTMAX)
    return cudaErrorInvalidConfiguration;
  kern<<<grid, NUM_THREADS, C::SMEM, a.stream>>>(*a.tmQ, *a.tmK, *a.tmV, P);
  return cudaGetLastError();
}

template <int HD>
cudaError_t modes(const ScoredFwd& a) {
  const bool cap = a.p.softcap > 0.f, bias = a.p.slopes != nullptr;
  if (cap) return bias ? launch<HD, true, true>(a) : launch<HD, true, false>(a);
  return bias ? launch<HD, false, true>(a) : launch<HD, false, false>(a);
}

}  // namespace scored_fwd

cudaError_t launch_scored_fwd_bf16(const ScoredFwd& a) {
  return a.p.d <= 64 && a.p.dv <= 64 ? scored_fwd::modes<64>(a) : scored_fwd::modes<128>(a);
}

}  // namespace attn
