// bf16 scored-attention backward on tcgen05 tensor cores (d, dv <= 128).
//
//   D  = rowsum(dO o O),  P = 2^(S2 - LSE2)  (scores in log2 units)
//   dV = P^T dO,  dS = P o T o (dO V^T - D),  dQ = scale dS K,  dK = scale dS^T Q
// with T = 1 - (capped score / cap)^2, or 1 without a cap. Two kernels, with
// the pipelines of the plain backward (bwd_bf16.cu):
//   - dq_kernel: a unit is one 128-row tile of packed rows; Q and dO stay in
//     shared memory, dQ accumulates in tensor memory over the key tiles the
//     rows see, and D and -LSE log2(e) go to the workspace;
//   - dkdv_kernel: a unit is one 128-key tile; K and V stay in shared memory,
//     and dK and dV accumulate in tensor memory over the row tiles that see
//     a key of it (a bit list from the plan), which with packed rows sums
//     them over the query heads that share the key head.
// Both sum in a fixed order. Differences from the plain kernels: the units'
// tile lists come from the plan and are claimed at run time; the factor P T,
// which dS needs, takes the place of P in the registers between the two
// passes over a tile (the dQ kernel keeps P too, in 11 bits, where there is a
// cap); ranges and bias are applied per row (dq) and per column (dkdv).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <limits.h>
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
namespace scored_bwd {

using bwd::BOX_BYTES;
using bwd::BT;
using bwd::packed_col;
using bwd::sw128_offset;
using scored::Cap;
using scored::add2;
using scored::dup;
using scored::f2;
using scored::F2;
using scored::fma2;
using scored::mul2;

// The dK/dV kernel works on 2^kLift P: what it keeps of P T between its passes
// is fp16, and from 4e-9 on that holds P T in 11 bits.
constexpr float kLift = 14.f, kLower = 0x1p-14f;

struct Params {
  ScoredProblem p;
  ScoredPlan plan;
  const float* LSE;
  float* NL;
  float* D;
  __nv_bfloat16* dQ;
  __nv_bfloat16* dK;
  __nv_bfloat16* dV;
  float* dKpart;
  float* dVpart;
  uint32_t* status;
  uint32_t* counter;   // this launch's unit counter
  int n_blocks, total, group;
  float sc2;           // scale * log2(e)
  Cap cap;
};

// Zeroes the bf16 values of w whose bits of `seen` (value e of word i: bit 2 i + e) are not set.
__device__ __forceinline__ void mask_pairs(uint32_t (&w)[16], uint32_t seen) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (!(seen & (1u << (2 * i)))) w[i] &= 0xffff0000u;
    if (!(seen & (2u << (2 * i)))) w[i] &= 0x0000ffffu;
  }
}

// ---------------------------------------------------------------- dQ

struct UnitQ {
  int bh, b, rt, j0, n;   // row tile rt of key head bh; key tiles [j0, j0 + n)
  int4 tile;
};
using RingQ = scored::UnitRing<UnitQ>;

template <int HD>
struct CfgQ {
  static constexpr int KB = HD / 64;
  static constexpr int TILE = BT * HD * 2;
  static constexpr int SUMS_BYTES = 2 * BT * 8;   // [row group][128]: sums of P (dP - D) and of P
  static constexpr int NSLOT_FIT = (227 * 1024 - 2 * TILE - SUMS_BYTES - 512) / TILE;
  static constexpr int NSLOT = NSLOT_FIT < 12 ? NSLOT_FIT : 12;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_DO = OFF_Q + TILE;
  static constexpr int OFF_RING = OFF_DO + TILE;
  static constexpr int OFF_SUMS = OFF_RING + NSLOT * TILE;
  static constexpr int OFF_BAR = OFF_SUMS + SUMS_BYTES;
  // full[NSLOT], empty[NSLOT], q_full, q_empty, o_read, s_full, s_free, dp_full, ds_full, dq_full, sums_full, drain,
  // unit queue
  static constexpr int NBAR = 2 * NSLOT + 10 + 2 * RingQ::N;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM = OFF_MISC + 16 + RingQ::BYTES;
  static constexpr int READERS = 1 + 256;
  static constexpr uint32_t IDESC_S = ptx::idesc_bf16(BT, BT, false, false);
  static constexpr uint32_t IDESC_DQ = ptx::idesc_bf16(BT, HD, false, true);
  // two tiles, of alternate key tiles: S, then dP, then dS and P T; the
  // accumulators of dS K and of P T K
  static constexpr uint32_t T_X = 0, T_DQ = 256, T_PK = 384;
};
constexpr int DQ_THREADS = 384;
constexpr int DQ_REG_CTRL = 96, DQ_REG_ROWS = 200;
constexpr float kWhole = 0x1p-10f;   // how near 1 a row's sum of P is where the call holds all its keys

__device__ __forceinline__ UnitQ load_unit_q(const Params& P, int x) {
  UnitQ u;
  bwd::grouped_unit(x, P.n_blocks, P.p.B * P.p.Hkv, P.group, true, &u.bh, &u.rt);
  u.rt = scored::packed_block(u.rt, P.n_blocks, P.p.G);
  u.b = u.bh / P.p.Hkv;
  u.tile = u.rt < P.p.n_rt ? __ldg(P.plan.tiles + static_cast<long long>(u.b) * P.p.n_rt + u.rt)
                           : make_int4(0, 0, 0, 0);
  u.j0 = u.tile.y > 0 ? u.tile.x / BT : 0;
  u.n = u.tile.y > 0 ? (u.tile.y + BT - 1) / BT - u.j0 : 0;
  return u;
}

// Warps: 0 producer, 1 MMA, 4-7 and 8-11 two row groups of a thread per query
// row; group g works on key columns [64 g, 64 g + 64) of every row.
//
// D enters dS linearly, and rowsum(dO o O) with the rounded O is off by enough
// to show: where a row's weight lies on few keys, dP - D is small beside D, and
// dQ and dK were off by 0.0026 of their norm over long rows, 0.0035 over
// documents of 16 tokens and up to 0.02 where rows see two to four keys. So that
// D is only a first estimate; the difference to the exact one,
//   rowsum P o (dP - D) = rowsum(P o dP) - D   (the rows of P sum to 1),
// is summed in fp32 along the way, a fourth product accumulates P T K, and at
// the end dQ = dS K - difference * P T K. The dK/dV kernel reads the exact D.
// dQ and dK are now off by 0.0024, what the roundings of dS and of the result
// make. Where a row's P does not sum to 1 (a call on a part of its keys, with O
// and LSE of them all) the difference is something else, and the estimate stays.
// It costs this kernel 176 -> 221 us at B=2 H=16 T=4096 d=128 causal with a cap,
// 83 -> 95 at B=4 H=16 T=2048 d=64 with a bias: a product more, at d = 128 Q and
// dO in shared memory for its accumulator's sake, and a quarter more arithmetic.
//
// dP_j goes where S_j was, dS_j and P_j T_j where dP_j was, and the next tile's
// S into the other place, so that the products run in the order dQ_j-1, dP_j,
// (P T K)_j-1, S_j+1 and both products of K fall behind what the threads wait
// for. (dP first: 617 in place of 611 us for a step over documents, H=32 Hkv=8
// T=8192 d=128; P T over S and the products of K together before the next S:
// 604 there, 622 in place of 610 with the cap.)
template <int HD, bool CAP, bool BIAS>
__global__ void __launch_bounds__(DQ_THREADS, 1)
    dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
              const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmdO,
              const __grid_constant__ CUtensorMap tmO, const __grid_constant__ Params P) {
  using C = CfgQ<HD>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if ((ptx::smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicOr(P.status, ATTN_DEV_BAD_SMEM);
    return;
  }
  uint8_t* sQ = smem + C::OFF_Q;
  uint8_t* sdO = smem + C::OFF_DO;
  uint8_t* ring = smem + C::OFF_RING;
  float2* sums = reinterpret_cast<float2*>(smem + C::OFF_SUMS);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* full = bars;
  uint64_t* empty = full + C::NSLOT;
  uint64_t* q_full = empty + C::NSLOT;   // Q and dO
  uint64_t* q_empty = q_full + 1;
  uint64_t* o_read = q_full + 2;         // the row threads have read a unit's dO and O
  uint64_t* s_full = q_full + 3;
  uint64_t* s_free = q_full + 4;
  uint64_t* dp_full = q_full + 5;
  uint64_t* ds_full = q_full + 6;
  uint64_t* dq_full = q_full + 7;
  uint64_t* sums_full = q_full + 8;
  uint64_t* drain = q_full + 9;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC + 4);
  const RingQ units{reinterpret_cast<UnitQ*>(smem + C::OFF_MISC + 16), q_full + 10, q_full + 10 + RingQ::N};
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NSLOT; ++s) {
      ptx::mbar_init(full + s, 1);
      ptx::mbar_init(empty + s, 1);
    }
    units.init(C::READERS);
    ptx::mbar_init(q_full, 1);
    ptx::mbar_init(q_empty, 1);
    ptx::mbar_init(o_read, 256);
    ptx::mbar_init(s_full, 1);
    ptx::mbar_init(s_free, 256);
    ptx::mbar_init(dp_full, 1);
    ptx::mbar_init(ds_full, 256);
    ptx::mbar_init(dq_full, 1);
    ptx::mbar_init(sums_full, 256);
    ptx::mbar_init(drain, 1);
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
  // Ring item i sits in slot i % NSLOT. A unit whose first item is i0 has O at
  // i0 and K_j, V_j at i0 + 1 + 2 j and i0 + 2 + 2 j; its Q and dO have tiles
  // of their own.
  auto slot = [](uint32_t i) { return static_cast<int>(i % C::NSLOT); };
  auto par = [](uint32_t i) { return (i / C::NSLOT) & 1u; };

  const int wg = warp >> 2;
  if (wg == 0) {
    ptx::reg_release<DQ_REG_CTRL>();
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- producer
      ptx::WaitCtx w{abort_flag, P.status, 5u};
      ptx::tma_prefetch_desc(&tmQ);
      ptx::tma_prefetch_desc(&tmK);
      ptx::tma_prefetch_desc(&tmV);
      ptx::tma_prefetch_desc(&tmdO);
      ptx::tma_prefetch_desc(&tmO);
      uint32_t item = 0, u_it = 0, pu = 0;
      auto load = [&](const CUtensorMap* map, int row, int bh) {
        const int s = slot(item);
        if (!ptx::mbar_wait(empty + s, par(item) ^ 1u, w)) return false;
        ptx::mbar_arrive_expect_tx(full + s, C::TILE);
        for (int c = 0; c < C::KB; ++c)
          ptx::tma_load_3d(ring + s * C::TILE + c * BOX_BYTES, map, full + s, c * 64, row, bh);
        ++item;
        return true;
      };
      // Q and dO, when the unit before needs its own no more
      auto load_rows = [&](int row, int bh) {
        if (!ptx::mbar_wait(q_empty, (u_it & 1u) ^ 1u, w)) return false;
        ptx::mbar_arrive_expect_tx(q_full, 2 * C::TILE);
        for (int c = 0; c < C::KB; ++c) {
          ptx::tma_load_3d(sQ + c * BOX_BYTES, &tmQ, q_full, c * 64, row, bh);
          ptx::tma_load_3d(sdO + c * BOX_BYTES, &tmdO, q_full, c * 64, row, bh);
        }
        ++u_it;
        return true;
      };
      auto look = [&](int x) { return load_unit_q(P, x); };
      auto work = [](const UnitQ& u) { return u.n > 0; };
      scored::NextUnit<UnitQ> cur{}, next{};
      bool ok = cur.first(P.counter, P.total, look, work, units, &pu, w);
      for (; ok && cur.u.bh >= 0; cur = next) {
        const UnitQ& u = cur.u;
        ok = load(&tmO, u.rt * BT, u.bh);
        for (int j = 0; ok && j < u.n; ++j) {
          if (!(ok = next.step(j, u.n, P.counter, P.total, look, work, units, &pu, w))) break;
          ok = load(&tmK, (u.j0 + j) * BT, u.bh) && load(&tmV, (u.j0 + j) * BT, u.bh) &&
               (j > 0 || load_rows(u.rt * BT, u.bh));
        }
      }
      if (!ok) {
        // let the copies in flight land before the CTA exits
        for (uint32_t n = (item > static_cast<uint32_t>(C::NSLOT) ? item - C::NSLOT : 0u); n < item; ++n)
          ptx::mbar_wait_drain(full + slot(n), par(n));
        if (u_it > 0) ptx::mbar_wait_drain(q_full, (u_it - 1) & 1u);
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer
      ptx::WaitCtx w{abort_flag, P.status, 6u};
      const uint32_t aR = ptx::smem_u32(ring);
      auto kmaj = [](uint64_t base, int kk) { return ptx::sdesc_advance(base, (kk >> 2) * BOX_BYTES + (kk & 3) * 32); };
      auto mnmaj = [](uint64_t base, int kk) { return ptx::sdesc_advance(base, kk * 2048); };
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, w));
      };
      const uint64_t q_desc = scored::formed(ptx::sdesc_sw128(ptx::smem_u32(sQ), 16, 1024));
      const uint64_t do_desc = scored::formed(ptx::sdesc_sw128(ptx::smem_u32(sdO), 16, 1024));
      // K-major and M/N-major descriptors of the tile of ring item i
      auto kdesc = [&](uint32_t i) { return scored::formed(ptx::sdesc_sw128(aR + slot(i) * C::TILE, 16, 1024)); };
      auto mdesc = [&](uint32_t i) { return scored::formed(ptx::sdesc_sw128(aR + slot(i) * C::TILE, BOX_BYTES, 1024)); };
      // (unrolled whole: the issue is on the way of every product)
      auto mma_s = [&](uint32_t x, uint64_t k) {
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
          ptx::mma_ss(x, kmaj(q_desc, kk), kmaj(k, kk), C::IDESC_S, kk > 0);
        ptx::mma_commit(s_full);
      };
      auto mma_dp = [&](uint32_t x, uint64_t v, uint32_t iv) {
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
          ptx::mma_ss(x, kmaj(do_desc, kk), kmaj(v, kk), C::IDESC_S, kk > 0);
        ptx::mma_commit(dp_full);
        ptx::mma_commit(empty + slot(iv));
      };
      // dS (at 0) or P T (at 16) times K: the row threads put 16 columns of
      // each, packed, in the place of 32 keys of dP
      auto mma_k = [&](uint32_t acc, uint32_t x, uint64_t k, bool add) {
#pragma unroll
        for (int kk = 0; kk < BT / 16; ++kk)
          ptx::mma_ts(tmem + acc, x + (kk >> 1) * 32 + (kk & 1) * 8, mnmaj(k, kk), C::IDESC_DQ,
                      (add || kk > 0) ? 1u : 0u);
      };
      auto place = [&](uint32_t t) { return tmem + C::T_X + 128 * (t & 1u); };
      uint32_t item = 0, u_it = 0, sp = 0, ru = 0;
      bool moved = false;
      // key tiles of the next unit, 0 at the end, -1 on a timeout
      auto next_unit = [&]() {
        UnitQ u;
        if (!units.read(ru, &u, w)) return -1;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(units.empty + ru % RingQ::N);
        ++ru;
        return u.bh < 0 ? 0 : u.n;
      };
      int nk = next_unit(), nk_next = 0;
      bool ok = nk >= 0;
      while (ok && nk > 0) {
        const uint32_t i0 = item;
        const uint64_t k0 = kdesc(i0 + 1);
        // (the products that read what this one overwrites have been issued: they run in order)
        if (!(ok = wait(q_full, u_it & 1u))) break;
        if (!(ok = wait(full + slot(i0 + 1), par(i0 + 1)))) break;
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
          moved |= lane != 0;
          mma_s(place(sp), k0);
        }
        __syncwarp();
        for (int j = 0; j < nk; ++j, ++sp) {
          if (j + 1 == nk) {
            nk_next = next_unit();
            ok = nk_next >= 0;
            if (!ok) break;
          }
          const uint32_t ik = i0 + 1 + 2 * j, x = place(sp), y = place(sp + 1);   // K_j; V_j = ik + 1, K_{j+1} = ik + 2
          const uint64_t v = kdesc(ik + 1), kn = kdesc(ik + 2), kl = mdesc(ik - 2), k = mdesc(ik);
          if (!(ok = wait(full + slot(ik + 1), par(ik + 1)))) break;
          if (!(ok = wait(s_free, sp & 1u))) break;
          if (j == 0) {   // O goes back to the ring
            if (!(ok = wait(o_read, u_it & 1u))) break;
            if (lane == 0) ptx::mbar_arrive(empty + slot(i0));
            __syncwarp();
          }
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
            moved |= lane != 0;
            mma_dp(x, v, ik + 1);
            if (j + 1 == nk) ptx::mma_commit(q_empty);   // the last product of Q and dO
            if (j > 0) {
              mma_k(C::T_PK, y + 16, kl, j > 1);
              ptx::mma_commit(empty + slot(ik - 2));
            }
          }
          __syncwarp();
          if (j + 1 < nk) {
            if (!(ok = wait(full + slot(ik + 2), par(ik + 2)))) break;
            ptx::tc_fence_after();
            if (ptx::elect_one()) {
              moved |= lane != 0;
              mma_s(y, kn);
            }
            __syncwarp();
          }
          if (!(ok = wait(ds_full, sp & 1u))) break;
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
            moved |= lane != 0;
            mma_k(C::T_DQ, x, k, j > 0);
            if (j + 1 == nk) {
              mma_k(C::T_PK, x + 16, k, j > 0);
              ptx::mma_commit(empty + slot(ik));
              ptx::mma_commit(dq_full);
            }
          }
          __syncwarp();
        }
        if (!ok) break;
        item = i0 + 1 + 2 * nk;
        ++u_it;
        nk = nk_next;
      }
      if (!ok) {
        if (ptx::elect_one()) ptx::mma_commit(drain);
        __syncwarp();
        ptx::mbar_wait_drain(drain, 0u);
      }
      if (__any_sync(0xffffffffu, moved) && lane == 0) atomicOr(P.status, ATTN_DEV_ISSUER);
    }
  } else {
    ptx::reg_acquire<DQ_REG_ROWS>();
    // ------------------------------------------------------------ row groups
    const int g = wg - 1;
    const int quad = warp & 3;
    const int r = quad * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tX = tmem + lane_off + C::T_X + 64 * g;
    const uint32_t tDQ = tmem + lane_off + C::T_DQ + (HD / 2) * g, tPK = tmem + lane_off + C::T_PK + (HD / 2) * g;
    ptx::WaitCtx w{abort_flag, P.status, 7u + g};
    const float sc2 = P.sc2, scale = P.p.scale;
    const F2 sc2v = dup(sc2), ninv2 = dup(P.cap.ninv2), one = dup(1.f);
    const int R = P.p.R, d = P.p.d, rpad = P.p.rpad();
    // rowsum(dO o O) of this thread's row. Rows past R load as zeros.
    auto estimate = [&](uint32_t i0, uint32_t u, float* sum) {
      if (!__all_sync(0xffffffffu, ptx::mbar_wait(q_full, u & 1u, w))) return false;
      if (!__all_sync(0xffffffffu, ptx::mbar_wait(full + slot(i0), par(i0), w))) return false;
      const uint8_t* so = ring + slot(i0) * C::TILE;
      F2 part = dup(0.f);
#pragma unroll 4
      for (int k = 0; k < HD / 8; ++k) {
        const uint32_t off = sw128_offset(r, 8 * k);
        const uint4 x = *reinterpret_cast<const uint4*>(sdO + off);
        const uint4 o = *reinterpret_cast<const uint4*>(so + off);
        const __nv_bfloat162* dov = reinterpret_cast<const __nv_bfloat162*>(&x);
        const __nv_bfloat162* ov = reinterpret_cast<const __nv_bfloat162*>(&o);
#pragma unroll
        for (int e = 0; e < 4; ++e) part = fma2(__bfloat1622float2(ov[e]), __bfloat1622float2(dov[e]), part);
      }
      *sum = part.x + part.y;
      ptx::mbar_arrive(o_read);
      return true;
    };
    // the next unit: 1, 0 at the end, -1 on a timeout (with what this
    // thread's row needs: read one unit ahead, so that the loads' latency
    // does not fall between units)
    uint32_t ru = 0;
    struct Mine {
      UnitQ u;
      int4 row;
      float lse, slope2;
    };
    auto next_unit = [&](Mine* m) {
      if (!units.read(ru, &m->u, w)) return -1;
      ptx::mbar_arrive(units.empty + ru % RingQ::N);
      ++ru;
      const UnitQ& u = m->u;
      if (u.bh < 0) return 0;
      const int row = u.rt * BT + r;
      m->row = __ldg(P.plan.rows + static_cast<long long>(u.b) * rpad + row);
      m->lse = row < R ? __ldg(P.LSE + static_cast<long long>(u.bh) * R + row) : -CUDART_INF_F;
      if (BIAS) m->slope2 = __ldg(P.plan.slope2 + static_cast<long long>(u.bh - u.b * P.p.Hkv) * rpad + row);
      return 1;
    };
    uint32_t item = 0, u_it = 0, sp = 0;
    Mine me{}, nx{};
    const int first = next_unit(&me);
    bool have = first == 1;
    bool ok = first >= 0;
    while (ok && have) {
      const UnitQ& u = me.u;
      const int row = u.rt * BT + r;
      const int4 ri = me.row;
      const float lse = me.lse, slope2 = me.slope2;
      bool have_next = false;
      const float nlse2 = (lse == -CUDART_INF_F) ? -CUDART_INF_F : fmaf(-lse, scored::kLog2e, kLift);
      const F2 nlv = dup(nlse2);
      float dd;
      if (!(ok = estimate(item, u_it, &dd))) break;
      if (ri.y == 0) dd = 0.f;   // (rows that see no key may hold anything)
      const F2 ndd = dup(-dd);
      F2 rest = dup(0.f), weight = dup(0.f);   // sums of P (dP - D) and of P
      for (int j = 0; j < u.n; ++j, ++sp) {
        if (!(ok = __all_sync(0xffffffffu, ptx::mbar_wait(s_full, sp & 1u, w)))) break;
        ptx::tc_fence_after();
        const uint32_t tx = tX + 128 * (sp & 1u);
        float f[64];                      // P T
        uint32_t whole[CAP ? 2 : 1][16];  // P where T is not 1, as fp16: for the sums
        const int kv0 = (u.j0 + j) * BT + 64 * g;   // key of this thread's first column
        // a key of the group's that some row does not see
        const bool partial = kv0 < u.tile.z || kv0 + 64 > u.tile.w;
        {
          uint32_t v[2][32];
#pragma unroll
          for (int c = 0; c < 2; ++c) ptx::tmem_ld32(tx + c * 32, v[c]);
#pragma unroll
          for (int c = 0; c < 2; ++c) ptx::tmem_ld_wait(v[c]);
          // S is in registers: the dP product may overwrite it
          ptx::tc_fence_before();
          ptx::mbar_arrive(s_free);
          const float* s = reinterpret_cast<const float*>(&v[0][0]);
          int form = 0;   // of the cap
          if constexpr (CAP) {
            float hi = s[0], lo = s[0];
#pragma unroll
            for (int i = 0; i < 64; i += 2) {
              hi = ptx::fmax3(hi, s[i], s[i + 1]);
              lo = ptx::fmin3(lo, s[i], s[i + 1]);
            }
            form = scored::cap_form(P.cap, lo, hi);
          }
          const int dist = kv0 - ri.z;
          const float delta = static_cast<float>(dist);
          const float c1 = dist < 0 ? slope2 : -slope2;
          const F2 c1v = dup(c1), base = dup(fmaf(c1, delta, nlse2));
          bool cross = false;
          if constexpr (BIAS) cross = __any_sync(0xffffffffu, dist < 0 && dist > -63);
          auto tile = [&](auto capped) {
            constexpr int kForm = decltype(capped)::value;
            const scored::CapPoly<kForm == scored::kCapPoly2 ? kForm : scored::kCapPoly4> cap_poly(P.cap);
#pragma unroll
            for (int i = 0; i < 64; i += 2) {
              const F2 t = f2(s[i], s[i + 1]);
              F2 add = nlv, p;
              if constexpr (BIAS) {
                add = fma2(f2(static_cast<float>(i), static_cast<float>(i + 1)), c1v, base);
                if (cross)
                  add = f2(fmaf(-slope2, fabsf(delta + static_cast<float>(i)), nlse2),
                           fmaf(-slope2, fabsf(delta + static_cast<float>(i + 1)), nlse2));
              }
              if constexpr (kForm == 0) {
                p = scored::ex2(fma2(t, sc2v, add));
              } else {
                F2 y;
                if constexpr (kForm != scored::kCapFormula)
                  y = mul2(t, cap_poly(t));
                else
                  y = scored::cap_any(t, P.cap);
                p = scored::ex2(add2(y, add));
                whole[i / 32][i / 2 % 16] = ptx::pack_f16_sat(p.x, p.y);
                p = mul2(p, fma2(mul2(y, y), ninv2, one));
              }
              f[i] = p.x;
              f[i + 1] = p.y;
            }
          };
          if constexpr (!CAP) {
            tile(std::integral_constant<int, 0>{});
          } else {
            switch (form) {
              case scored::kCapPoly2: tile(std::integral_constant<int, scored::kCapPoly2>{}); break;
              case scored::kCapPoly4: tile(std::integral_constant<int, scored::kCapPoly4>{}); break;
              default: tile(std::integral_constant<int, scored::kCapFormula>{});
            }
          }
        }
        uint32_t seen[2] = {0xffffffffu, 0xffffffffu};
        if (partial) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            seen[c] = scored::bit_range(ri.x - kv0 - 32 * c, ri.y - kv0 - 32 * c);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(seen[c] & (1u << i))) f[32 * c + i] = 0.f;
            if constexpr (CAP) mask_pairs(whole[c], seen[c]);
          }
        }
        // Keys that no row of the tile sees may hold anything, which a weight of
        // 0 would not hold back: their K is zeroed, now that the S product has
        // read it (each group a box of 64 columns).
        const int k0 = kv0 - 64 * g;
        if (k0 < u.tile.x || k0 + BT > u.tile.y) {
          if (k0 + r < u.tile.x || k0 + r >= u.tile.y)
            for (int c = g; c < C::KB; c += 2)
              scored::zero_box_row(ring + slot(item + 1 + 2 * j) * C::TILE + c * BOX_BYTES, r);
          ptx::fence_proxy_async_smem();
        }
        if (j + 1 == u.n) {
          const int more = next_unit(&nx);
          ok = more >= 0;
          if (!ok) break;
          have_next = more == 1;
        }
        if (!(ok = __all_sync(0xffffffffu, ptx::mbar_wait(dp_full, sp & 1u, w)))) break;
        ptx::tc_fence_after();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t v[32], pk[32];
          ptx::tmem_ld32(tx + c * 32, v);
          ptx::tmem_ld_wait(v);
          if (partial) {   // (what the row does not see may hold anything)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(seen[c] & (1u << i))) v[i] = __float_as_uint(dd);
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const F2 pt = f2(f[c * 32 + 2 * i], f[c * 32 + 2 * i + 1]);
            const F2 e = add2(f2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), ndd);
            const F2 ds = mul2(pt, e);
            pk[i] = scored::pack_bf16(ds);
            pk[16 + i] = scored::pack_bf16(pt);
            if constexpr (CAP) {
              const F2 p = __half22float2(*reinterpret_cast<const __half2*>(&whole[c][i]));
              rest = fma2(p, e, rest);
              weight = add2(weight, p);
            } else {
              rest = add2(rest, ds);
              weight = add2(weight, pt);
            }
          }
          ptx::tmem_st32(tx + c * 32, pk);   // over the columns just read
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        ptx::mbar_arrive(ds_full);
      }
      if (!ok) break;
      if (!(ok = __all_sync(0xffffffffu, ptx::mbar_wait(dq_full, u_it & 1u, w)))) break;
      ptx::tc_fence_after();
      // The two groups' sums. (Every thread has read the last unit's: dq_full
      // came after its first dS of this one.)
      sums[g * BT + r] = f2(rest.x + rest.y, weight.x + weight.y);
      ptx::mbar_arrive(sums_full);
      if (!(ok = __all_sync(0xffffffffu, ptx::mbar_wait(sums_full, u_it & 1u, w)))) break;
      const F2 sum = mul2(add2(sums[r], sums[BT + r]), dup(kLower));
      const float off = fabsf(sum.y - 1.f) <= kWhole ? sum.x : 0.f;
      if (g == 0) {   // for every row of the padded tile: the dK/dV kernel reads whole 128-row slices
        P.D[static_cast<long long>(u.bh) * rpad + row] = ri.y > 0 ? dd + off : 0.f;
        P.NL[static_cast<long long>(u.bh) * rpad + row] = nlse2;
      }
      const float mul = scale * kLower;
      const F2 mulv = dup(mul), offv = dup(-off * mul);
      const int row4 = row & ~3;   // (see scored::quad_transpose)
      __nv_bfloat16* out = P.dQ + (static_cast<long long>(u.bh) * R + row4) * d;
#pragma unroll 1
      for (int c = 0; c < HD / 64; ++c) {
        uint32_t v[32], k[32];
        ptx::tmem_ld32(tDQ + c * 32, v);
        ptx::tmem_ld32(tPK + c * 32, k);
        ptx::tmem_ld_wait(v);
        ptx::tmem_ld_wait(k);
        uint4 pk[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t x[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int i = 8 * e + 2 * q;
            const F2 y = fma2(f2(__uint_as_float(k[i]), __uint_as_float(k[i + 1])), offv,
                              mul2(f2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), mulv));
            x[q] = ri.y == 0 ? 0u : scored::pack_bf16(y);   // sees no key: 0 times what others see may be NaN
          }
          pk[e] = make_uint4(x[0], x[1], x[2], x[3]);
        }
        scored::quad_transpose(pk, lane);
        const int col = (HD / 2) * g + c * 32 + 8 * (lane & 3);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (row4 + i < R && col < d) *reinterpret_cast<uint4*>(out + static_cast<long long>(i) * d + col) = pk[i];
      }
      // (the next unit's first products into the accumulators wait for this
      // group's first dS of that unit, stored after this)
      ptx::tc_fence_before();
      item += 1 + 2 * u.n;
      ++u_it;
      have = have_next;
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

// ---------------------------------------------------------------- dK, dV

constexpr int KV_THREADS = 512;
constexpr int KV_REG_CTRL = 96, KV_REG_PDS = 168, KV_REG_EPI = 80, KV_REG_LAUNCH = 128;

struct UnitKV {
  int bh, b, kb, part, n;   // part of the row tiles of key tile kb of key head bh, n row tiles
  int lo, hi;               // keys outside are seen by no row
  int blank;                // some row tile has a row that sees no key
  const uint32_t* bits;      // those of the key tile as bits
};
using RingKV = scored::UnitRing<UnitKV>;

// What the P / dS threads need of a row tile, in its slot of the slices' ring:
// written by the producer (the first four) and copied from the plan.
struct alignas(16) TileRec {
  int kb, b, kvh, rt;   // kb < 0: the end
  int4 hull;            // the plan's
  int4 even;            // .x: position of the first row, or kScoredUneven
  float4 slope2;        // .x: the first row's
};

template <int HD>
struct CfgKV {
  static constexpr int KB = HD / 64;
  static constexpr int TILE = BT * HD * 2;
  static constexpr int NQ = 3, NO = 2, NL = 2;   // rings: Q tiles, dO tiles, slices of NL and D
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = OFF_K + TILE;
  static constexpr int OFF_Q = OFF_V + TILE;
  static constexpr int OFF_DO = OFF_Q + NQ * TILE;
  static constexpr int OFF_LSE = OFF_DO + NO * TILE;
  static constexpr int OFF_D = OFF_LSE + NL * BT * 4;
  static constexpr int OFF_REC = OFF_D + NL * BT * 4;
  static constexpr int OFF_BAR = OFF_REC + NL * static_cast<int>(sizeof(TileRec));
  // kv_full, kv_empty, q_full[NQ], q_empty[NQ], o_full[NO], o_empty[NO], l_full[NL], l_empty[NL], raw_q[NQ],
  // raw_o[NO], s_full, dp_full, p_full, ds_full, acc_full, dv_free, dk_free, drain, unit queue
  static constexpr int NBAR = 2 + 3 * NQ + 3 * NO + 2 * NL + 8 + 2 * RingKV::N;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM = OFF_MISC + 16 + RingKV::BYTES;
  static constexpr int READERS = 2 + 128;   // of the units: the MMA warp and the cleaner (once), the epilogue threads
  static constexpr uint32_t IDESC_S = ptx::idesc_bf16(BT, BT, false, false);
  static constexpr uint32_t IDESC_ACC = ptx::idesc_bf16(BT, HD, false, true);
};

__device__ __forceinline__ UnitKV load_unit_kv(const Params& P, int x) {
  UnitKV u;
  int blk;
  bwd::grouped_unit(x, P.n_blocks, P.p.B * P.p.Hkv, P.group, false, &u.bh, &blk);
  u.kb = blk / P.p.kv_splits;
  u.part = blk - u.kb * P.p.kv_splits;
  u.b = u.bh / P.p.Hkv;
  const long long at = static_cast<long long>(u.b) * P.p.n_kt + u.kb;
  u.n = __ldg(P.plan.kcount + at * P.p.kv_splits + u.part);
  u.bits = P.plan.kbits + at * P.p.n_words();
  const int4 hull = __ldg(P.plan.khull + at);
  u.lo = hull.x;
  u.hi = hull.y;
  u.blank = hull.z;
  return u;
}

// Walks the set bits of a list from bit `first` on; the caller takes a unit's n of them.
struct TileList {
  const uint32_t* words;
  int base;
  uint32_t bits;
  __device__ __forceinline__ TileList(const uint32_t* w, int first) : words(w + first / 32), base(first & ~31), bits(0u) {
    if (w) bits = __ldg(words++) & (0xffffffffu << (first % 32));
  }
  __device__ __forceinline__ int next() {
    while (bits == 0u) {
      base += 32;
      bits = __ldg(words++);
    }
    const int i = __ffs(bits) - 1;
    bits &= bits - 1u;
    return base + i;
  }
};

// 32 x 32 bits, row i in lane i; returns column `lane` (bit i from lane i).
__device__ __forceinline__ uint32_t transpose32(uint32_t x, int lane) {
  uint32_t m = 0x0000ffffu;
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) {
    const uint32_t y = __shfl_xor_sync(0xffffffffu, x, j);
    x = (lane & j) ? ((x & ~m) | ((y & ~m) >> j)) : ((x & m) | ((y & m) << j));
    m ^= m << (j >> 1);
  }
  return x;
}

// Warps: 0 producer, 1 MMA, 2 cleaner, 4-7 and 8-11 P / dS (a thread per key; group h
// works on query columns [64 h, 64 h + 64)), 12-15 epilogue.
// TMEM: dV [0, 128), dK [128, 256), S^T [256, 384), dP^T [384, 512).
// PARTS: units are parts of a key tile's row tiles, with partial results.
template <int HD, bool CAP, bool BIAS, bool PARTS>
__global__ void __launch_bounds__(KV_THREADS, 1)
    dkdv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmdO,
                const __grid_constant__ Params P) {
  using C = CfgKV<HD>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if ((ptx::smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicOr(P.status, ATTN_DEV_BAD_SMEM);
    return;
  }
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sV = smem + C::OFF_V;
  uint8_t* sQ = smem + C::OFF_Q;
  uint8_t* sdO = smem + C::OFF_DO;
  float* sLSE = reinterpret_cast<float*>(smem + C::OFF_LSE);
  float* sD = reinterpret_cast<float*>(smem + C::OFF_D);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* kv_full = bars + 0;
  uint64_t* kv_empty = bars + 1;
  uint64_t* q_full = bars + 2;
  uint64_t* q_empty = q_full + C::NQ;
  uint64_t* o_full = q_empty + C::NQ;
  uint64_t* o_empty = o_full + C::NO;
  uint64_t* l_full = o_empty + C::NO;
  uint64_t* l_empty = l_full + C::NL;
  uint64_t* raw_q = l_empty + C::NL;   // as q_full and o_full, in units that go by way of the cleaner
  uint64_t* raw_o = raw_q + C::NQ;
  uint64_t* s_full = raw_o + C::NO;
  uint64_t* dp_full = s_full + 1;
  uint64_t* p_full = s_full + 2;
  uint64_t* ds_full = s_full + 3;
  uint64_t* acc_full = s_full + 4;
  uint64_t* dv_free = s_full + 5;
  uint64_t* dk_free = s_full + 6;
  uint64_t* drain = s_full + 7;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC + 4);
  const RingKV units{reinterpret_cast<UnitKV*>(smem + C::OFF_MISC + 16), s_full + 8, s_full + 8 + RingKV::N};
  TileRec* recs = reinterpret_cast<TileRec*>(smem + C::OFF_REC);   // [NL]

  if (threadIdx.x == 0) {
    units.init(C::READERS);
    ptx::mbar_init(kv_full, 1);
    ptx::mbar_init(kv_empty, 1);
    for (int s = 0; s < C::NQ; ++s) {
      ptx::mbar_init(q_full + s, 1);
      ptx::mbar_init(q_empty + s, 1);
      ptx::mbar_init(raw_q + s, 1);
    }
    for (int s = 0; s < C::NO; ++s) {
      ptx::mbar_init(o_full + s, 1);
      ptx::mbar_init(o_empty + s, 1);
      ptx::mbar_init(raw_o + s, 1);
    }
    for (int s = 0; s < C::NL; ++s) {
      ptx::mbar_init(l_full + s, 1);
      ptx::mbar_init(l_empty + s, 256);
    }
    ptx::mbar_init(s_full, 1);
    ptx::mbar_init(dp_full, 1);
    ptx::mbar_init(p_full, 256);
    ptx::mbar_init(ds_full, 256);
    ptx::mbar_init(acc_full, 1);
    ptx::mbar_init(dv_free, 128);
    ptx::mbar_init(dk_free, 128);
    ptx::mbar_init(drain, 1);
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
  const uint32_t T_DV = 0, T_DK = 128, T_ST = 256, T_DP = 384;
  // Row tile number n (counted across units) uses slot n % NQ, n % NO, n % NL.
  auto qslot = [](uint32_t n) { return static_cast<int>(n % C::NQ); };
  auto qpar = [](uint32_t n) { return (n / C::NQ) & 1u; };
  auto oslot = [](uint32_t n) { return static_cast<int>(n % C::NO); };
  auto opar = [](uint32_t n) { return (n / C::NO) & 1u; };
  auto lslot = [](uint32_t n) { return static_cast<int>(n % C::NL); };
  auto lpar = [](uint32_t n) { return (n / C::NL) & 1u; };
  const int rpad = P.p.rpad();

  const int wg = warp >> 2;
  if (wg == 0) {
    ptx::reg_release<KV_REG_CTRL>();
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- producer
      ptx::WaitCtx w{abort_flag, P.status, 1u};
      ptx::tma_prefetch_desc(&tmQ);
      ptx::tma_prefetch_desc(&tmK);
      ptx::tma_prefetch_desc(&tmV);
      ptx::tma_prefetch_desc(&tmdO);
      uint32_t u_it = 0, q_it = 0, q_issued = 0, o_issued = 0, l_issued = 0, pu = 0;
      auto look = [&](int x) { return load_unit_kv(P, x); };
      auto work = [](const UnitKV& u) { return u.n > 0; };
      scored::NextUnit<UnitKV> cur{}, next{};
      bool ok = cur.first(P.counter, P.total, look, work, units, &pu, w);
      for (; ok && cur.u.bh >= 0; cur = next) {
        const UnitKV& u = cur.u;
        if (!(ok = ptx::mbar_wait(kv_empty, (u_it & 1u) ^ 1u, w))) break;
        ptx::mbar_arrive_expect_tx(kv_full, 2 * C::TILE);
        for (int c = 0; c < C::KB; ++c) {
          ptx::tma_load_3d(sK + c * BOX_BYTES, &tmK, kv_full, c * 64, u.kb * BT, u.bh);
          ptx::tma_load_3d(sV + c * BOX_BYTES, &tmV, kv_full, c * 64, u.kb * BT, u.bh);
        }
        ++u_it;
        TileList list(u.bits, u.part * P.p.kv_split_tiles);
        // Q and dO of a unit some of whose rows see no key go by way of the
        // cleaner. (Chosen per unit: a choice per tile in this thread cost 4 %.)
        uint64_t *q_to = u.blank ? raw_q : q_full, *o_to = u.blank ? raw_o : o_full;
        for (int ii = 0; ii < u.n; ++ii, ++q_it) {
          if (!(ok = next.step(ii, u.n, P.counter, P.total, look, work, units, &pu, w))) break;
          const int rt = list.next();
          const int qs = qslot(q_it), os = oslot(q_it), ls = lslot(q_it);
          const long long row0 = static_cast<long long>(u.bh) * rpad + static_cast<long long>(rt) * BT;
          if (!(ok = ptx::mbar_wait(q_empty + qs, qpar(q_it) ^ 1u, w))) break;
          ptx::mbar_arrive_expect_tx(q_to + qs, C::TILE);
          for (int c = 0; c < C::KB; ++c)
            ptx::tma_load_3d(sQ + qs * C::TILE + c * BOX_BYTES, &tmQ, q_to + qs, c * 64, rt * BT, u.bh);
          q_issued = q_it + 1;
          if (!(ok = ptx::mbar_wait(l_empty + ls, lpar(q_it) ^ 1u, w))) break;
          const int kvh = u.bh - u.b * P.p.Hkv;
          const long long at = static_cast<long long>(u.b) * P.p.n_rt + rt;
          TileRec* rec = recs + ls;
          rec->kb = u.kb;
          rec->b = u.b;
          rec->kvh = kvh;
          rec->rt = rt;
          ptx::mbar_arrive_expect_tx(l_full + ls, 2 * BT * 4 + 16 + (BIAS ? 32 : 0));
          ptx::bulk_load(&rec->hull, P.plan.tiles + at, 16, l_full + ls);
          if (BIAS) {
            ptx::bulk_load(&rec->even, P.plan.even + at, 16, l_full + ls);
            ptx::bulk_load(&rec->slope2, P.plan.slope2 + static_cast<long long>(kvh) * rpad + rt * BT, 16, l_full + ls);
          }
          ptx::bulk_load(sLSE + ls * BT, P.NL + row0, BT * 4, l_full + ls);
          ptx::bulk_load(sD + ls * BT, P.D + row0, BT * 4, l_full + ls);
          l_issued = q_it + 1;
          if (!(ok = ptx::mbar_wait(o_empty + os, opar(q_it) ^ 1u, w))) break;
          ptx::mbar_arrive_expect_tx(o_to + os, C::TILE);
          for (int c = 0; c < C::KB; ++c)
            ptx::tma_load_3d(sdO + os * C::TILE + c * BOX_BYTES, &tmdO, o_to + os, c * 64, rt * BT, u.bh);
          o_issued = q_it + 1;
        }
      }
      // the end for the P / dS threads: a record without slices
      if (ok && (ok = ptx::mbar_wait(l_empty + lslot(q_it), lpar(q_it) ^ 1u, w))) {
        recs[lslot(q_it)].kb = -1;
        ptx::mbar_arrive(l_full + lslot(q_it));
      }
      if (!ok) {
        // let the copies in flight land before the CTA exits (those that the
        // cleaner no longer hands on have, when a wait here gives up)
        if (u_it > 0) ptx::mbar_wait_drain(kv_full, (u_it - 1) & 1u);
        for (uint32_t n = (q_issued > (uint32_t)C::NQ ? q_issued - C::NQ : 0u); n < q_issued; ++n)
          ptx::mbar_wait_drain(q_full + qslot(n), qpar(n));
        for (uint32_t n = (o_issued > (uint32_t)C::NO ? o_issued - C::NO : 0u); n < o_issued; ++n)
          ptx::mbar_wait_drain(o_full + oslot(n), opar(n));
        for (uint32_t n = (l_issued > (uint32_t)C::NL ? l_issued - C::NL : 0u); n < l_issued; ++n)
          ptx::mbar_wait_drain(l_full + lslot(n), lpar(n));
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer
      ptx::WaitCtx w{abort_flag, P.status, 2u};
      const uint32_t aK = ptx::smem_u32(sK), aV = ptx::smem_u32(sV), aQ = ptx::smem_u32(sQ), adO = ptx::smem_u32(sdO);
      auto kmaj = [](uint64_t base, int kk) { return ptx::sdesc_advance(base, (kk >> 2) * BOX_BYTES + (kk & 3) * 32); };
      auto mnmaj = [](uint64_t base, int kk) { return ptx::sdesc_advance(base, kk * 2048); };
      const uint64_t k_desc = scored::formed(ptx::sdesc_sw128(aK, 16, 1024));
      const uint64_t v_desc = scored::formed(ptx::sdesc_sw128(aV, 16, 1024));
      // K-major and M/N-major descriptors of row tile n's Q and dO
      auto q_k = [&](uint32_t n) { return scored::formed(ptx::sdesc_sw128(aQ + qslot(n) * C::TILE, 16, 1024)); };
      auto q_m = [&](uint32_t n) { return scored::formed(ptx::sdesc_sw128(aQ + qslot(n) * C::TILE, BOX_BYTES, 1024)); };
      auto o_k = [&](uint32_t n) { return scored::formed(ptx::sdesc_sw128(adO + oslot(n) * C::TILE, 16, 1024)); };
      auto o_m = [&](uint32_t n) { return scored::formed(ptx::sdesc_sw128(adO + oslot(n) * C::TILE, BOX_BYTES, 1024)); };
      // (products unrolled by 4: see the forward)
      auto mma_st = [&](uint64_t q) {   // S^T = K Q^T
#pragma unroll 4
        for (int kk = 0; kk < HD / 16; ++kk)
          ptx::mma_ss(tmem + T_ST, kmaj(k_desc, kk), kmaj(q, kk), C::IDESC_S, kk > 0);
        ptx::mma_commit(s_full);
      };
      auto mma_dpt = [&](uint64_t o) {   // dP^T = V dO^T
#pragma unroll 4
        for (int kk = 0; kk < HD / 16; ++kk)
          ptx::mma_ss(tmem + T_DP, kmaj(v_desc, kk), kmaj(o, kk), C::IDESC_S, kk > 0);
        ptx::mma_commit(dp_full);
      };
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, w));
      };
      uint32_t u_it = 0, q_it = 0, pp = 0, ru = 0;
      bool moved = false;
      // row tiles of the next unit, 0 at the end, -1 on a timeout
      auto next_unit = [&]() {
        UnitKV u;
        if (!units.read(ru, &u, w)) return -1;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(units.empty + ru % RingKV::N);
        ++ru;
        return u.bh < 0 ? 0 : u.n;
      };
      int nq = next_unit(), nq_next = 0;
      bool ok = nq >= 0;
      while (ok && nq > 0) {
        const uint64_t q0 = q_k(q_it), o0 = o_k(q_it);
        if (!(ok = wait(kv_full, u_it & 1u))) break;
        if (!(ok = wait(q_full + qslot(q_it), qpar(q_it)))) break;
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
          moved |= lane != 0;
          mma_st(q0);
        }
        __syncwarp();
        if (!(ok = wait(o_full + oslot(q_it), opar(q_it)))) break;
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
          moved |= lane != 0;
          mma_dpt(o0);
          // K and V are read by no later MMA of a one-tile unit
          if (nq == 1) ptx::mma_commit(kv_empty);
        }
        __syncwarp();
        if (nq > 1 && !(ok = wait(q_full + qslot(q_it + 1), qpar(q_it + 1)))) break;
        for (int ii = 0; ii < nq; ++ii) {
          if (ii + 1 == nq) {
            nq_next = next_unit();
            ok = nq_next >= 0;
            if (!ok) break;
          }
          const uint32_t it = q_it + ii;
          const bool more = ii + 1 < nq;
          const uint64_t om = o_m(it), qm = q_m(it), qn = q_k(it + 1), on = o_k(it + 1);
          // dV += P^T dO, then the next S^T (which overwrites P^T). A unit's
          // first dV (dK) overwrites the accumulator: the epilogue must have
          // read the previous unit's.
          if (ii == 0 && !(ok = wait(dv_free, (u_it & 1u) ^ 1u))) break;
          if (!(ok = wait(p_full, pp & 1u))) break;
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
            moved |= lane != 0;
#pragma unroll 4
            for (int kk = 0; kk < BT / 16; ++kk)
              ptx::mma_ts(tmem + T_DV, tmem + T_ST + packed_col(kk), mnmaj(om, kk),
                          C::IDESC_ACC, (ii > 0 || kk > 0) ? 1u : 0u);
            ptx::mma_commit(o_empty + oslot(it));
            if (more) mma_st(qn);
          }
          __syncwarp();
          if (ii == 0 && !(ok = wait(dk_free, (u_it & 1u) ^ 1u))) break;
          if (!(ok = wait(ds_full, pp & 1u))) break;
          ++pp;
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
            moved |= lane != 0;
#pragma unroll 4
            for (int kk = 0; kk < BT / 16; ++kk)
              ptx::mma_ts(tmem + T_DK, tmem + T_DP + packed_col(kk), mnmaj(qm, kk),
                          C::IDESC_ACC, (ii > 0 || kk > 0) ? 1u : 0u);
            ptx::mma_commit(q_empty + qslot(it));
          }
          __syncwarp();
          if (more) {
            if (!(ok = wait(o_full + oslot(it + 1), opar(it + 1)))) break;
            ptx::tc_fence_after();
            if (ptx::elect_one()) {
              moved |= lane != 0;
              mma_dpt(on);
              if (ii + 2 == nq) ptx::mma_commit(kv_empty);   // the unit's last product of K or V
            }
            __syncwarp();
          }
          if (ii + 2 < nq && !(ok = wait(q_full + qslot(it + 2), qpar(it + 2)))) break;
        }
        if (!ok) break;
        if (ptx::elect_one()) {
          moved |= lane != 0;
          ptx::mma_commit(acc_full);
        }
        __syncwarp();
        q_it += nq;
        ++u_it;
        nq = nq_next;
      }
      if (!ok) {
        if (ptx::elect_one()) ptx::mma_commit(drain);
        __syncwarp();
        ptx::mbar_wait_drain(drain, 0u);
      }
      if (__any_sync(0xffffffffu, moved) && lane == 0) atomicOr(P.status, ATTN_DEV_ISSUER);
    } else if (warp == 2) {
      // ---------------------------------------------------------- cleaner
      // Rows that see no key (padding) may hold anything, which weights of 0
      // would not hold back: their Q and dO become zeros before the products
      // read them (D and P are 0 there). A warp of its own: branches for it
      // among the P / dS threads cost every tile 3 to 8 %.
      ptx::WaitCtx w{abort_flag, P.status, 2u};
      uint32_t raw = 0;   // bit s: parity of the next phase of raw_q[s], bit 16 + s: of raw_o[s]
      uint32_t n = 0, ru = 0;
      bool ok = true;
      while (ok) {
        UnitKV u;
        if (!__all_sync(0xffffffffu, units.read(ru, &u, w))) break;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(units.empty + ru % RingKV::N);
        ++ru;
        if (u.bh < 0) break;
        TileList list(u.bits, u.part * P.p.kv_split_tiles);
        for (int i = 0; u.blank && i < u.n; ++i) {
          const long long rt = list.next();
          const bool some = __ldg(&P.plan.tiles[static_cast<long long>(u.b) * P.p.n_rt + rt].z) == INT_MAX;
          const int4* rows = P.plan.rows + static_cast<long long>(u.b) * rpad + rt * BT;
          // passes a tile on when it has landed, without what such rows hold
          auto pass = [&](uint64_t* from, uint32_t bit, uint8_t* tile, uint64_t* to) {
            if (!__all_sync(0xffffffffu, ptx::mbar_wait(from, raw >> bit & 1u, w))) return false;
            raw ^= 1u << bit;
            if (some) {
              for (int r = lane; r < BT; r += 32)
                if (__ldg(&rows[r].y) == 0)
                  for (int c = 0; c < C::KB; ++c) scored::zero_box_row(tile + c * BOX_BYTES, r);
              ptx::fence_proxy_async_smem();
              __syncwarp();
            }
            if (lane == 0) ptx::mbar_arrive(to);
            return true;
          };
          const int qs = qslot(n + i), os = oslot(n + i);
          ok = pass(raw_q + qs, qs, sQ + qs * C::TILE, q_full + qs) &&
               pass(raw_o + os, 16 + os, sdO + os * C::TILE, o_full + os);
          if (!ok) break;
        }
        n += u.n;
      }
    }
  } else if (wg <= 2) {
    ptx::reg_acquire<KV_REG_PDS>();
    // ------------------------------------------------------------ P / dS (thread = key row)
    const int h = wg - 1;
    const int quad = warp & 3;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tST = tmem + lane_off + T_ST + 64 * h, tDP = tmem + lane_off + T_DP + 64 * h;
    ptx::WaitCtx w{abort_flag, P.status, 3u};
    const float sc2 = P.sc2;
    const F2 sc2v = dup(sc2), ninv2 = dup(P.cap.ninv2), one = dup(1.f), neg1 = dup(-1.f);
    // A row tile as these threads see it, from its record, and (for a partial
    // tile, or one whose rows' positions are uneven) what its rows need,
    // loaded as soon as the record is there: columns c and 32 + c of this
    // group for lane c.
    struct Tile {
      int kb, all_lo, all_hi, even;
      float slope2;
      int4 r[2];
      float cslope[2];
    };
    auto is_partial = [&](const Tile& t) { return t.kb * BT < t.all_lo || t.kb * BT + BT > t.all_hi; };
    auto fetch = [&](uint32_t n, Tile* t) {   // once l_full says so
      const TileRec* rec = recs + lslot(n);
      t->kb = rec->kb;
      if (t->kb < 0) return;
      t->all_lo = rec->hull.z;
      t->all_hi = rec->hull.w;
      if constexpr (BIAS) {
        t->even = rec->even.x;
        t->slope2 = rec->slope2.x;
      }
      const bool uneven = BIAS && t->even == kScoredUneven;
      if (!is_partial(*t) && !uneven) return;
      const int row = rec->rt * BT + 64 * h + lane;
      const int4* rows = P.plan.rows + static_cast<long long>(rec->b) * rpad + row;
      t->r[0] = __ldg(rows);
      t->r[1] = __ldg(rows + 32);
      if (uneven) {
        const float* sl = P.plan.slope2 + static_cast<long long>(rec->kvh) * rpad + row;
        t->cslope[0] = __ldg(sl);
        t->cslope[1] = __ldg(sl + 32);
      }
    };
    uint32_t q_it = 0;
    Tile cur{}, nxt{};
    bool ok = __all_sync(0xffffffffu, ptx::mbar_wait(l_full + lslot(0), lpar(0), w));
    if (ok) fetch(0, &cur);
    {
      while (ok && cur.kb >= 0) {
        const int ls = lslot(q_it);
        const float* nlse2 = sLSE + ls * BT + 64 * h;
        const float* dd = sD + ls * BT + 64 * h;
        const int key0 = cur.kb * BT + quad * 32;   // key of lane 0
        const int key = key0 + lane;
        // Which of this warp's keys each of the 64 columns' rows sees, unless
        // all rows see all keys of the tile: bit c of seen[c / 32] for this
        // thread's key.
        const bool partial = is_partial(cur);
        uint32_t seen[2] = {0xffffffffu, 0xffffffffu};
        if (partial) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
            seen[c] = transpose32(scored::bit_range(cur.r[c].x - key0, cur.r[c].y - key0), lane);
        }
        // bias: one slope and consecutive positions for the tile's rows (the
        // plan says), else each column's own, from lanes c and c + 32
        const bool even = !BIAS || cur.even != kScoredUneven;
        const float pos0 = BIAS && even ? static_cast<float>(key - cur.even - 64 * h) : 0.f;   // key - position of column 0
        const float slope2 = cur.slope2;
        if (!(ok = __all_sync(0xffffffffu, ptx::mbar_wait(s_full, q_it & 1u, w)))) break;
        ptx::tc_fence_after();
        // pass 1: P^T, packed bf16 (the product's type) over the first half of
        // this group's S^T columns; P^T T stays in registers for pass 2, as
        // fp16: as fp32 it would take 64 of 168 registers, and as bf16 it would
        // be a third rounding of dK, as large as dS's and the result's.
        uint32_t keep[2][16];
        {
          uint32_t rs[2][32];
          ptx::tmem_ld32(tST, rs[0]);
          ptx::tmem_ld32(tST + 32, rs[1]);
          ptx::tmem_ld_wait(rs[0]);
          ptx::tmem_ld_wait(rs[1]);
          int form = 0;   // of the cap
          if constexpr (CAP) {
            float hi = __uint_as_float(rs[0][0]), lo = hi;
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                hi = ptx::fmax3(hi, __uint_as_float(rs[c][i]), __uint_as_float(rs[c][i + 1]));
                lo = ptx::fmin3(lo, __uint_as_float(rs[c][i]), __uint_as_float(rs[c][i + 1]));
              }
            form = scored::cap_form(P.cap, lo, hi);
          }
          // the distance pos0 - column changes sign inside the tile for some key of the warp
          const bool cross = BIAS && __any_sync(0xffffffffu, pos0 > 0.f && pos0 < 63.f);
          const float c1 = pos0 > 0.f ? -slope2 : slope2;   // -slope2 |pos0 - column| = c1 (pos0 - column)
          const F2 nc1 = dup(-c1), base = dup(c1 * pos0);
          auto tile = [&](auto capped, auto distance, auto masked) {
            constexpr int kForm = decltype(capped)::value;
            const scored::CapPoly<kForm == scored::kCapPoly2 ? kForm : scored::kCapPoly4> cap_poly(P.cap);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t pk[16];
#pragma unroll
              for (int i = 0; i < 16; i += 2) {
                const float4 l4 = ptx::lds128(nlse2 + c * 32 + 2 * i);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                  const int a = 2 * (i + q);   // column within the 32
                  const F2 t = f2(__uint_as_float(rs[c][a]), __uint_as_float(rs[c][a + 1]));
                  F2 add = q ? f2(l4.z, l4.w) : f2(l4.x, l4.y);
                  if constexpr (BIAS) {
                    const float n0 = static_cast<float>(c * 32 + a), n1 = static_cast<float>(c * 32 + a + 1);
                    if constexpr (decltype(distance)::value == 0) {
                      add = add2(add, fma2(f2(n0, n1), nc1, base));
                    } else if constexpr (decltype(distance)::value == 1) {
                      add = f2(fmaf(-slope2, fabsf(pos0 - n0), add.x), fmaf(-slope2, fabsf(pos0 - n1), add.y));
                    } else {
                      const int q0 = __shfl_sync(0xffffffffu, cur.r[c].z, a),
                                q1 = __shfl_sync(0xffffffffu, cur.r[c].z, a + 1);
                      const float s0 = __shfl_sync(0xffffffffu, cur.cslope[c], a),
                                  s1 = __shfl_sync(0xffffffffu, cur.cslope[c], a + 1);
                      add = f2(fmaf(-s0, fabsf(static_cast<float>(key - q0)), add.x),
                               fmaf(-s1, fabsf(static_cast<float>(key - q1)), add.y));
                    }
                  }
                  F2 p, grad;
                  if constexpr (kForm == 0) {
                    p = scored::ex2(fma2(t, sc2v, add));
                  } else {
                    F2 y;
                    if constexpr (kForm != scored::kCapFormula)
                      y = mul2(t, cap_poly(t));
                    else
                      y = scored::cap_any(t, P.cap);
                    p = scored::ex2(add2(y, add));
                    grad = fma2(mul2(y, y), ninv2, one);
                  }
                  if constexpr (decltype(masked)::value)
                    p = f2(seen[c] & (1u << a) ? p.x : 0.f, seen[c] & (2u << a) ? p.y : 0.f);
                  pk[i + q] = scored::pack_bf16(p);
                  if constexpr (kForm != 0) p = mul2(p, grad);
                  keep[c][i + q] = ptx::pack_f16_sat(p.x, p.y);
                }
              }
              ptx::tmem_st16(tST + c * 16, pk);
            }
          };
          // (variants of their own where they are frequent; the others mask always)
          auto either = [&](auto capped) {
            using zero = std::integral_constant<int, 0>;
            if (BIAS && !even)
              tile(capped, std::integral_constant<int, BIAS ? 2 : 0>{}, std::true_type{});
            else if (cross)
              tile(capped, std::integral_constant<int, BIAS ? 1 : 0>{}, std::true_type{});
            else if (partial)
              tile(capped, zero{}, std::true_type{});
            else
              tile(capped, zero{}, std::false_type{});
          };
          if constexpr (!CAP) {
            either(std::integral_constant<int, 0>{});
          } else {
            constexpr int kF = scored::kCapFormula, kUneven = BIAS ? 2 : 0, kAbs = BIAS ? 1 : 0;
            if (form == scored::kCapPoly2 && !partial && !(BIAS && (cross || !even)))
              tile(std::integral_constant<int, scored::kCapPoly2>{}, std::integral_constant<int, 0>{}, std::false_type{});
            else if (form != kF)   // (degree 4 covers the range of degree 2: fewer variants, 224 in place of 241 us)
              either(std::integral_constant<int, scored::kCapPoly4>{});
            else if (BIAS && !even)
              tile(std::integral_constant<int, kF>{}, std::integral_constant<int, kUneven>{}, std::true_type{});
            else
              tile(std::integral_constant<int, kF>{}, std::integral_constant<int, kAbs>{}, std::true_type{});
          }
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        ptx::mbar_arrive(p_full);
        // the next tile's record, where it is there already (behind the last
        // tile of a unit it waits for that tile's products)
        const bool early = __all_sync(0xffffffffu, ptx::mbar_test(l_full + lslot(q_it + 1), lpar(q_it + 1)));
        if (early) fetch(q_it + 1, &nxt);
        // pass 2: dS^T = P^T T (dP^T - D), bf16 over dP^T
        if (!(ok = __all_sync(0xffffffffu, ptx::mbar_wait(dp_full, q_it & 1u, w)))) break;
        ptx::tc_fence_after();
        {
          uint32_t rd[2][32];
          ptx::tmem_ld32(tDP, rd[0]);
          ptx::tmem_ld32(tDP + 32, rd[1]);
          ptx::tmem_ld_wait(rd[0]);
          ptx::tmem_ld_wait(rd[1]);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float4 d4 = ptx::lds128(dd + c * 32 + 2 * i);
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const F2 pt = __half22float2(*reinterpret_cast<const __half2*>(&keep[c][i + q]));
                const F2 e = fma2(q ? f2(d4.z, d4.w) : f2(d4.x, d4.y), neg1,
                                  f2(__uint_as_float(rd[c][2 * (i + q)]), __uint_as_float(rd[c][2 * (i + q) + 1])));
                pk[i + q] = scored::pack_bf16(mul2(pt, e));
              }
            }
            ptx::tmem_st16(tDP + c * 16, pk);
          }
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        ptx::mbar_arrive(ds_full);
        ptx::mbar_arrive(l_empty + ls);
        ++q_it;
        if (!early) {
          if (!(ok = __all_sync(0xffffffffu, ptx::mbar_wait(l_full + lslot(q_it), lpar(q_it), w)))) break;
          fetch(q_it, &nxt);
        }
        cur = nxt;
      }
    }
  } else {
    ptx::reg_release<KV_REG_EPI>();
    // ------------------------------------------------------------ dK / dV epilogue
    const int quad = warp & 3;
    const int r = quad * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    ptx::WaitCtx w{abort_flag, P.status, 4u};
    const float scale = P.p.scale;
    const int Tk = P.p.Tk;
    uint32_t u_it = 0, ru = 0;
    bool ok = true;
    while (ok) {
      UnitKV u;
      if (!(ok = units.read(ru, &u, w))) break;
      ptx::mbar_arrive(units.empty + ru % RingKV::N);
      ++ru;
      if (u.bh < 0) break;
      const int key = u.kb * BT + r;
      const bool unseen = key < u.lo || key >= u.hi;
      const long long head = static_cast<long long>(u.bh) * Tk;
      const long long part_row = (static_cast<long long>(u.part) * P.p.B * P.p.Hkv + u.bh) * Tk;
      if (!(ok = __all_sync(0xffffffffu, ptx::mbar_wait(acc_full, u_it & 1u, w)))) break;
      ptx::tc_fence_after();
      // (Loops, not unrolled: the roles of this kernel together fill the
      // instruction cache, and unrolled this part, which runs once per unit,
      // displaced the others' code: 116 in place of 111 us at B=4 H=16 T=2048
      // d=64 with a bias.)
#pragma unroll 1
      for (int acc = 0; acc < 2; ++acc) {   // dV first, released as soon as it is read, then scale * dK
        const uint32_t tcol = tmem + lane_off + (acc ? T_DK : T_DV);
        const int width = acc ? P.p.d : P.p.dv;
        const int key4 = key & ~3;   // (see scored::quad_transpose)
        const float mul = acc ? scale * kLower : kLower;
#pragma unroll 1
        for (int c = 0; c < HD / 32; ++c) {
          uint32_t v[32];
          ptx::tmem_ld32(tcol + c * 32, v);
          ptx::tmem_ld_wait(v);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * mul);
          if (unseen) {   // (it may hold anything)
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0u;
          }
          uint4 pk[4];
          if constexpr (PARTS) {   // fp32: 16 columns at a time
            float* out = (acc ? P.dKpart : P.dVpart) + (part_row + key4) * width;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                pk[e] = make_uint4(v[16 * h + 4 * e], v[16 * h + 4 * e + 1], v[16 * h + 4 * e + 2], v[16 * h + 4 * e + 3]);
              scored::quad_transpose(pk, lane);
              const int col = 32 * c + 16 * h + 4 * (lane & 3);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (key4 + i < Tk && col < width)
                  *reinterpret_cast<uint4*>(out + static_cast<long long>(i) * width + col) = pk[i];
            }
          } else {
            __nv_bfloat16* out = (acc ? P.dK : P.dV) + (head + key4) * width;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t x[4];
#pragma unroll
              for (int q = 0; q < 4; ++q)
                x[q] = ptx::pack_bf16(__uint_as_float(v[8 * e + 2 * q]), __uint_as_float(v[8 * e + 2 * q + 1]));
              pk[e] = make_uint4(x[0], x[1], x[2], x[3]);
            }
            scored::quad_transpose(pk, lane);
            const int col = c * 32 + 8 * (lane & 3);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (key4 + i < Tk && col < width)
                *reinterpret_cast<uint4*>(out + static_cast<long long>(i) * width + col) = pk[i];
          }
        }
        ptx::tc_fence_before();
        ptx::mbar_arrive(acc ? dk_free : dv_free);
      }
      ++u_it;
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
cudaError_t launch(const ScoredBwd& a) {
  static_assert(CfgQ<HD>::SMEM <= 227 * 1024 && CfgKV<HD>::SMEM <= 227 * 1024, "shared memory");
  static_assert(KV_REG_CTRL + 2 * KV_REG_PDS + KV_REG_EPI <= 4 * KV_REG_LAUNCH, "register split");
  const ScoredProblem& p = a.p;
  Params P;
  P.p = p;
  P.plan = a.plan;
  P.LSE = a.LSE;
  P.NL = a.NL;
  P.D = a.D;
  P.dQ = static_cast<__nv_bfloat16*>(a.dQ);
  P.dK = static_cast<__nv_bfloat16*>(a.dK);
  P.dV = static_cast<__nv_bfloat16*>(a.dV);
  P.dKpart = a.dKpart;
  P.dVpart = a.dVpart;
  P.status = a.status;
  P.sc2 = p.scale * scored::kLog2e;
  P.cap = scored::make_cap(p.scale, p.softcap);
  const int heads = p.B * p.Hkv;
  // heads in groups whose streamed tiles fill about half of L2
  auto group = [&](size_t per_head) {
    size_t g = per_head * heads <= 2 * a.l2_bytes ? heads : a.l2_bytes / 2 / per_head;
    return static_cast<int>(g < 1 ? 1 : g > static_cast<size_t>(heads) ? heads : g);
  };
  auto kq = dq_kernel<HD, CAP, BIAS>;
  auto kk = p.kv_splits > 1 ? dkdv_kernel<HD, CAP, BIAS, true> : dkdv_kernel<HD, CAP, BIAS, false>;
  cudaError_t e = cudaFuncSetAttribute(kq, cudaFuncAttributeMaxDynamicSharedMemorySize, CfgQ<HD>::SMEM);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(kk, cudaFuncAttributeMaxDynamicSharedMemorySize, CfgKV<HD>::SMEM);
  if (e != cudaSuccess) return e;
  // the register splits must fit the launch allocations (see ptx::reg_acquire)
  cudaFuncAttributes fa;
  if ((e = cudaFuncGetAttributes(&fa, kq)) != cudaSuccess) return e;
  if (fa.numRegs < DQ_REG_CTRL || fa.numRegs > DQ_REG_ROWS || 3 * fa.numRegs < DQ_REG_CTRL + 2 * DQ_REG_ROWS)
    return cudaErrorInvalidConfiguration;
  if ((e = cudaFuncGetAttributes(&fa, kk)) != cudaSuccess) return e;
  if (fa.numRegs != KV_REG_LAUNCH) return cudaErrorInvalidConfiguration;
  P.n_blocks = scored::packed_blocks(p.n_rt, p.G);
  P.total = P.n_blocks * heads;
  P.group = group(static_cast<size_t>(p.Tk) * (p.d + p.dv) * 2);
  P.counter = a.plan.counters;
  kq<<<P.total < a.num_sms ? P.total : a.num_sms, DQ_THREADS, CfgQ<HD>::SMEM, a.stream>>>(*a.tmQ, *a.tmK, *a.tmV,
                                                                                          *a.tmdO, *a.tmO, P);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  P.n_blocks = p.n_kt * p.kv_splits;
  P.total = P.n_blocks * heads;
  P.group = group(static_cast<size_t>(p.R) * ((p.d + p.dv) * 2 + 8));
  P.counter = a.plan.counters + 1;
  kk<<<P.total < a.num_sms ? P.total : a.num_sms, KV_THREADS, CfgKV<HD>::SMEM, a.stream>>>(*a.tmQ, *a.tmK, *a.tmV,
                                                                                           *a.tmdO, P);
  return cudaGetLastError();
}

template <int HD>
cudaError_t modes(const ScoredBwd& a) {
  const bool cap = a.p.softcap > 0.f, bias = a.p.slopes != nullptr;
  if (cap) return bias ? launch<HD, true, true>(a) : launch<HD, true, false>(a);
  return bias ? launch<HD, false, true>(a) : launch<HD, false, false>(a);
}

}  // namespace scored_bwd

cudaError_t launch_scored_bwd_bf16(const ScoredBwd& a) {
  return a.p.d <= 64 && a.p.dv <= 64 ? scored_bwd::modes<64>(a) : scored_bwd::modes<128>(a);
}

}  // namespace attn
