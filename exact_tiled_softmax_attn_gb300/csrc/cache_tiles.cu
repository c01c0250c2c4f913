// bf16 scored attention of a tile of query rows over a paged cache of e4m3
// codes (d, dv <= 128, more than a few and at most 128 packed rows of a key
// head in a tile) on tcgen05 tensor cores.
//
// With some tens of rows a key's codes are used often enough that converting
// them for every 8 or 16 rows is what the few-row kernel spends its time on
// (64 rows: 0.6 of its instructions). Here a tile of 128 keys is converted
// once, by a warpgroup of its own, to fp16 (exact) in the swizzled layout that
// tcgen05.mma reads, for all rows of the tile:
//   producer warps  look pages up and copy their codes as they lie (bulk
//                   copies; a page of a head is contiguous) into rings, one of
//                   K, which also hands on the scales, and one of V
//   converters      codes -> fp16 tiles, a warpgroup each for K and for V (one
//                   for both had K wait for V's buffer); zeros for V's rows
//                   that no query sees and for pages that are none
//   MMA warp        S = Q K^T (two buffers), O += P V
//   softmax         a thread per row; scores in registers, weights (fp16) over
//                   the scores in tensor memory
// Q goes through fp16 at a power of two of its row, the key scale multiplies
// the scores, and the value scale's logarithm is added to them, as in
// cache_tokens.cu; stages, shares and the join are cache_walk.cuh's.
//
// Weights are p vs as fp16, relative to the largest of the row, so a page of
// zeros (or of tokens that no row sees) whose scale is 2^30 times the others'
// must not set what they are relative to. A warp looks over the scales of a run
// ahead of it. Where they lie more than 2^8 apart, or a page is none, it steps
// between the producer of V and the converter: it finds the largest code (but
// NaN) that is seen of every 16 keys, multiplies their codes by the power of two that brings
// it above 224 - exact, codes have no more bits - and divides the scale by it.
// Weights are then relative to the largest of what keys add to O, whatever the
// scales. That costs other runs 6 % (57 -> 60.5 us with 64 rows, 78 -> 84 with
// 128, by the code's size: the roles' loops together just fit the instruction
// cache); a factor on the converted values instead 16 %, a product per band of
// scales 30 %.
//
// Order of the tensor core's work, tile i: S(i + 1) is issued before O += P V
// of tile i, so that the softmax of the next tile need not wait for it. S(i)
// goes over P(i - 2), which the product before it in the queue has read by
// then. A thread waits for the product of tile i - 1 before it lets that of
// tile i go, which is also when it may rescale O.
// TMEM: S and P of even tiles at column 0, of odd ones at 128, O at 256.
//
// 16 sequences of up to 12000 keys, Hkv=4 d=128: 64 rows a key head 60 us (113
// by groups of 32 rows in cache_tokens.cu), 128 rows 84. A tile of 128 keys
// takes about 2300 cycles with 64 rows: the products 1260, shared memory 1750
// (the codes in and out, the converted tiles in and out, Q), a converter 1150, a
// softmax thread 1350; they wait for one another in turn.
#include <cuda_bf16.h>
#include <math_constants.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "cache.h"
#include "cache_walk.cuh"
#include "common.cuh"
#include "ptx.cuh"
#include "scored.h"
#include "scored_math.cuh"

namespace attn {
namespace cache_tiles {

using cache_walk::Params;
using scored::add2;
using scored::dup;
using scored::f2;
using scored::F2;
using scored::fma2;

constexpr int BM = 128, BN = 128;
constexpr int BOX = 128 * 64 * 2;      // 128 rows of 64 fp16
constexpr float TAU = 8.0f, SHIFT = 7.0f;   // weights up to 2^(TAU + SHIFT)
constexpr float kWide = 256.0f;      // value scales further apart than this: a wide run
constexpr int THREADS = 512;
constexpr int REG_CTRL = 88, REG_CONVERT = 88, REG_SOFTMAX = 240;
constexpr int NSC = 8;   // tiles whose scales are held (see the producer)

// CP copies of a tile's rows, RP of them each: where half of the tile's rows
// are free, they hold the same queries, and the threads of each copy take half
// of the keys.
template <int HD, int CP>
struct Cfg {
  static constexpr int RP = BM / CP, KEYS = BN / CP;
  static constexpr int TILE = BN * HD * 2;     // fp16
  static constexpr int RAW = BN * HD;          // codes of a tile of keys or of values
  // Even: a place of the ring is then always keys' or always values', and its converters see every phase of its barriers.
  static constexpr int NRAW = HD == 128 ? 4 : 8;
  static_assert(NRAW % 2 == 0 && NRAW <= 8, "ring");
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + TILE;
  static constexpr int OFF_V = OFF_K + 2 * TILE;   // two of K: the next is converted while S is formed from one
  static constexpr int OFF_RAW = OFF_V + TILE;
  // raw_full[NRAW], raw_empty[NRAW], k_full[2], k_empty[2], v_full, v_empty, s_full[2], p_full[2], pv_done, q_full, drain,
  // sc_full[NSC], unit_full[2], run_full[2], run_empty[2], wide_full[NRAW]
  static constexpr int NBAR = 3 * NRAW + 19 + NSC;
  static constexpr int OFF_SUMS = OFF_RAW + NRAW * RAW;   // [2][RP][32] fp32: columns that a copy hands to the other
  static constexpr int OFF_BAR = OFF_SUMS + (CP > 1 ? 2 * RP * 128 : 0);
  static constexpr int OFF_NONE = OFF_BAR + (NBAR * 8 + 15) / 16 * 16;   // [NRAW]: 16-key groups of a slot that hold nothing
  static constexpr int OFF_SCALE = OFF_NONE + (NRAW * 4 + 15) / 16 * 16;   // [NSC][8] float4
  static constexpr int OFF_MISC = OFF_SCALE + NSC * 8 * 16;
  static constexpr int OFF_ML = OFF_MISC + 128;              // [128] float2: maxima and sums of the rows' copies
  static constexpr int OFF_UNIT = OFF_ML + 1024;             // [2][128] float: the powers of two of Q's rows, of a run
  static constexpr int OFF_HULL = OFF_UNIT + 1024;
  static constexpr int SMEM = OFF_HULL + 8 * THREADS;
  // fp16 operands (format 0), fp32 accumulator
  static constexpr uint32_t idesc(int N, bool b_mn_major) {
    return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(BM >> 4) << 24);
  }
  static constexpr uint32_t IDESC_S = idesc(BN, false), IDESC_PV = idesc(HD, true);
};

using Walk = cache_walk::Walk<BM, BN>;

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Barrier of the softmax warps; whether `ok` holds in all of them.
__device__ __forceinline__ bool softmax_barrier_all(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"(ok ? 1u : 0u)
      : "memory");
  return r != 0;
}

template <int HD, int CP>
__global__ void __launch_bounds__(THREADS, 1) tiles_kernel(const __grid_constant__ Params P) {
  using C = Cfg<HD, CP>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if ((ptx::smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicOr(P.status, ATTN_DEV_BAD_SMEM);
    return;
  }
  uint8_t* sQ = smem + C::OFF_Q;
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sV = smem + C::OFF_V;
  uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* raw_empty = raw_full + C::NRAW;
  uint64_t* k_full = raw_empty + C::NRAW;
  uint64_t* k_empty = k_full + 2;
  uint64_t* v_full = k_empty + 2;
  uint64_t* v_empty = v_full + 1;
  uint64_t* s_full = v_empty + 1;
  uint64_t* p_full = s_full + 2;
  uint64_t* pv_done = p_full + 2;
  uint64_t* q_full = pv_done + 1;
  uint64_t* drain = q_full + 1;
  uint64_t* sc_full = drain + 1;
  uint64_t* unit_full = sc_full + NSC;
  uint64_t* run_full = unit_full + 2;    // whether a run is wide
  uint64_t* run_empty = run_full + 2;
  uint64_t* wide_full = run_empty + 2;   // values of wide runs, before they are raw_full
  float* units = reinterpret_cast<float*>(smem + C::OFF_UNIT);
  float4* scales = reinterpret_cast<float4*>(smem + C::OFF_SCALE);   // of 16-key groups: ks, log2 vs, 1 / vs
  volatile uint32_t* none_of = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_NONE);
  volatile uint32_t* run_wide = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC + 8);   // [2]
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC + 4);
  int* found = reinterpret_cast<int*>(smem + C::OFF_MISC + 16);
  int* scan = reinterpret_cast<int*>(smem + C::OFF_MISC + 32);   // one per warp
  int2* hulls = reinterpret_cast<int2*>(smem + C::OFF_HULL);
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NRAW; ++s) {
      ptx::mbar_init(raw_full + s, 1);
      ptx::mbar_init(raw_empty + s, 128);
    }
    ptx::mbar_init(v_full, 128);
    ptx::mbar_init(v_empty, 1);
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(k_full + t, 128);
      ptx::mbar_init(k_empty + t, 1);
      ptx::mbar_init(s_full + t, 1);
      ptx::mbar_init(p_full + t, 128);
    }
    ptx::mbar_init(pv_done, 1);
    ptx::mbar_init(q_full, 128);
    ptx::mbar_init(drain, 1);
    for (int k = 0; k < NSC; ++k) ptx::mbar_init(sc_full + k, 1);
    for (int k = 0; k < 2; ++k) {
      ptx::mbar_init(unit_full + k, 128);
      ptx::mbar_init(run_full + k, 1);
      ptx::mbar_init(run_empty + k, 2);
    }
    for (int k = 0; k < C::NRAW; ++k) ptx::mbar_init(wide_full + k, 1);
    *abort_flag = 0u;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(tmem_slot, 512);
    ptx::tmem_relinquish();
  }
  // columns from d (dv) on stay zero: the converters write only what there is, all of it in every tile
  if (P.p.d < HD || P.p.dv < HD) {
    for (int i = threadIdx.x; i < 3 * C::TILE / 16; i += THREADS)
      reinterpret_cast<uint4*>(sK)[i] = make_uint4(0u, 0u, 0u, 0u);
    ptx::fence_proxy_async_smem();
  }
  // (the launch overlaps the end of the kernel before; the join's, earlier than this one's end, costs 1 to 3 us)
  ptx::grid_wait();
  ptx::tc_fence_before();
  int first, last;
  const bool one = cache_walk::share<BM, BN, THREADS>(P, hulls, scan, found, &first, &last);
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Walk wk;
  if (last > first) wk.begin(P, one ? hulls : nullptr, found[0], found[1], last - first);
  // Items 2 i and 2 i + 1 of the ring are the keys and the values of the CTA's tile i.
  auto slot = [](uint32_t i) { return static_cast<int>(i % C::NRAW); };
  auto par = [](uint32_t i) { return (i / C::NRAW) & 1u; };

  const int wg = warp >> 2;
  if (wg == 0) {
    ptx::reg_release<REG_CTRL>();
    const int shift = P.c.shift, rows = 1 << shift, nb = BN >> shift;   // nb boxes of a tile, of `rows` keys each
    // box `box` of the run: its plane of the pool, or -1
    auto find = [&](int box, bool* seen) {
      const int key = wk.key0(wk.s0) + box * rows;
      *seen = box < wk.run * nb && key < wk.hull.y && key + rows > wk.hull.x;
      const int at = *seen ? cache::page_of(P.c, wk.e / P.groups, key >> shift) : -1;
      return at >= 0 ? at * P.p.Hkv + wk.h : -1;
    };
    if ((warp == 0 || warp == 2) && last > first) {
      // ------------------------------------------------------------ producers, of K (and the scales) and of V
      const int side = warp >> 1;
      ptx::WaitCtx w{abort_flag, P.status, 1u};
      const uint32_t bytes = static_cast<uint32_t>(rows * (side ? P.p.dv : P.p.d));   // of a box
      uint32_t item = side, runs = 0;
      bool ok = true, seen;
      do {
        const int n_box = wk.run * nb;
        bool wide = false;
        // lane i looks up box i of the next 32
        int plane = find(lane, &seen);
        for (int box0 = 0; ok && box0 < n_box; box0 += 32) {
          float ks = 1.f, vs = 1.f;
          if (side == 0 && plane >= 0) {
            ks = P.c.scale[0][plane];
            vs = P.c.scale[1][plane];
          }
          const int next = find(box0 + 32 + lane, &seen);
          const int boxes = min(32, n_box - box0);
          for (int j = 0; ok && j < boxes; j += nb) {
            const int at = __shfl_sync(0xffffffffu, plane, (j + lane) & 31);
            const bool there = lane < nb && at >= 0;
            const unsigned got = __ballot_sync(0xffffffffu, there);
            const int from = j + ((16 * (lane & 7)) >> shift);   // box of 16-key group lane % 8
            // 16-key groups of the boxes that are not there
            const uint32_t none = 0xffu & ~__ballot_sync(0xffffffffu, __shfl_sync(0xffffffffu, plane, from) >= 0);
            const int sl = slot(item);
            if (lane == 0) ok = ptx::mbar_wait(raw_empty + sl, par(item) ^ 1u, w);
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
            if (!ok) break;
            if (side && box0 + j == 0) {
              if (!(ok = __all_sync(0xffffffffu, ptx::mbar_wait(run_full + (runs & 1u), (runs >> 1) & 1u, w)))) break;
              wide = run_wide[runs & 1u] != 0u;
            }
            uint64_t* full = (side && wide ? wide_full : raw_full) + sl;
            if (lane == 0) {
              none_of[sl] = none;
              ptx::mbar_arrive_expect_tx(full, bytes * __popc(got));
            }
            __syncwarp();
            if (there)
              ptx::bulk_load(smem + C::OFF_RAW + sl * C::RAW + lane * bytes,
                             static_cast<const uint8_t*>(P.c.pool[side]) + static_cast<long long>(at) * bytes, bytes,
                             full);
            const uint32_t tile = item / 2;
            item += 2;
            if (side) continue;
            if (box0 + j == 0) {
              if (!(ok = __all_sync(0xffffffffu, ptx::mbar_wait(run_full + (runs & 1u), (runs >> 1) & 1u, w)))) break;
              wide = run_wide[runs & 1u] != 0u;
            }
            // The scales of the tile j (of the CTA), behind its copies. They replace those of j - NSC, which the softmax
            // has done with: the ring had room for j's keys, so those of j - NRAW / 2 (j - 4 at least) were converted,
            // so S of the tile two before them (j - 6) was out, which is issued after the softmax of the one two before
            // it (j - 8) was waited for. (Of a wide run: below.)
            if (wide) continue;
            const float k = cache::clamp_scale(__shfl_sync(0xffffffffu, ks, from));
            const float v = cache::clamp_scale(__shfl_sync(0xffffffffu, vs, from));
            if (lane < 8) scales[(tile % NSC) * 8 + lane] = make_float4(k, log2f(v), 1.f / v, 0.f);
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(sc_full + tile % NSC);
          }
          plane = next;
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(run_empty + (runs & 1u));
        ++runs;
      } while (ok && wk.next(P));
      if (!ok && lane == 0)   // let the copies in flight land before the CTA exits (a wide run's: while this wait runs out)
        for (uint32_t n = item > static_cast<uint32_t>(C::NRAW) ? item - C::NRAW : side; n < item; n += 2)
          ptx::mbar_wait_drain(raw_full + slot(n), par(n));
    } else if (warp == 3 && last > first) {
      // ------------------------------------------------------------ value scales that lie far apart
      ptx::WaitCtx w{abort_flag, P.status, 5u};
      uint32_t runs = 0, tile = 0, phase = 0;   // phase: of wide_full, a bit each
      bool ok = true, seen;
      do {
        float least = CUDART_INF_F, most = 0.f;
        bool wide = false;
        for (int box = lane; box < wk.run * nb; box += 4 * 32) {
          int at[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            at[u] = find(box + 32 * u, &seen);
            if (seen && at[u] < 0) wide = true;
          }
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (at[u] >= 0) {
              const float v = cache::clamp_scale(P.c.scale[1][at[u]]);
              least = fminf(least, v);
              most = fmaxf(most, v);
            }
        }
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        }
        wide = __any_sync(0xffffffffu, wide || most > kWide * least);
        if (lane == 0 && (ok = ptx::mbar_wait(run_empty + (runs & 1u), ((runs >> 1) & 1u) ^ 1u, w))) {
          run_wide[runs & 1u] = wide;
          ptx::mbar_arrive(run_full + (runs & 1u));
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        ++runs;
        if (wide) {
          for (int j = 0; ok && j < wk.run; ++j, ++tile) {
            // Four lanes a group of 16 keys: the rows that are seen, 16 codes at a time.
            const int g = lane >> 2, box = j * nb + (16 * g >> shift), per = P.p.dv / 16;
            const int plane = find(box, &seen);
            const float ks = plane >= 0 ? cache::clamp_scale(P.c.scale[0][plane]) : 1.f;
            const float vs = plane >= 0 ? cache::clamp_scale(P.c.scale[1][plane]) : 1.f;
            const int key0 = wk.key0(wk.s0 + j) + 16 * g;
            const int r0 = max(0, min(16, wk.hull.x - key0)), r1 = plane >= 0 ? max(0, min(16, wk.hull.y - key0)) : 0;
            const int sl = slot(2 * tile + 1);
            // (every lane reads what was copied)
            if (!(ok = __all_sync(0xffffffffu, ptx::mbar_wait(wide_full + sl, phase >> sl & 1u, w)))) {   // let the copies in flight land before the CTA exits
              if (lane == 0) ptx::mbar_wait_drain(wide_full + sl, phase >> sl & 1u);
              break;
            }
            phase ^= 1u << sl;
            uint4* codes = reinterpret_cast<uint4*>(smem + C::OFF_RAW + sl * C::RAW) + 16 * g * per;
            uint32_t m = 0;
            for (int i = r0 * per + (lane & 3); i < r1 * per; i += 4) {
              const uint4 u = codes[i];
              constexpr uint32_t SIZE = 0x7f7f7f7fu;   // without the signs; four NaN
              auto larger = [&](uint32_t x) { m = __vmaxu4(m, x & SIZE & ~__vcmpeq4(x & SIZE, SIZE)); };
              larger(u.x), larger(u.y), larger(u.z), larger(u.w);
            }
            uint32_t top = max(max(m & 255u, m >> 8 & 255u), max(m >> 16 & 255u, m >> 24));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float size = cache::half2_to_float2(cache::codes_to_half2(static_cast<uint16_t>(top))).x;
            int up = 0;   // to 17
            if (top > 0) {
              up = 8 - ilogbf(size);
              if (ldexpf(size, up) > kCodeMost) --up;
            }
            if (up > 0) {
              const float f = ldexpf(1.f, up);
              for (int i = r0 * per + (lane & 3); i < r1 * per; i += 4) {
                uint4 u = codes[i];
                uint32_t* q = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float2 a = cache::half2_to_float2(cache::codes_to_half2(static_cast<uint16_t>(q[e])));
                  const float2 c = cache::half2_to_float2(cache::codes_to_half2(static_cast<uint16_t>(q[e] >> 16)));
                  q[e] = static_cast<uint32_t>(cache::float2_to_codes(a.x * f, a.y * f)) |
                         static_cast<uint32_t>(cache::float2_to_codes(c.x * f, c.y * f)) << 16;
                }
                codes[i] = u;
              }
            }
            ptx::fence_proxy_async_smem();   // (the slot's next copies come after these writes)
            // Zeros: a scale below all others', 2^-40 2^-17. The place is free: the copies had room, so the values of the
            // tile four before at least were converted, after the product of the one before that.
            if ((lane & 3) == 0)
              scales[(tile % NSC) * 8 + g] = make_float4(ks, top == 0 ? -60.f : log2f(vs) - static_cast<float>(up),
                                                         top == 0 ? 0x1p60f : ldexpf(1.f / vs, up), 0.f);
            __syncwarp();
            if (lane == 0) {
              ptx::mbar_arrive(raw_full + sl);
              ptx::mbar_arrive(sc_full + tile % NSC);
            }
          }
        } else {
          tile += wk.run;
        }
      } while (ok && wk.next(P));
    } else if (warp == 1 && last > first) {
      // ------------------------------------------------------------ MMA issuer
      // The whole warp follows the schedule; the lane elect.sync picks issues.
      ptx::WaitCtx w{abort_flag, P.status, 3u};
      const uint64_t q_desc = scored::formed(ptx::sdesc_sw128(ptx::smem_u32(sQ), 16, 1024));
      const uint64_t k_desc[2] = {scored::formed(ptx::sdesc_sw128(ptx::smem_u32(sK), 16, 1024)),
                                  scored::formed(ptx::sdesc_sw128(ptx::smem_u32(sK) + C::TILE, 16, 1024))};
      const uint64_t v_desc = scored::formed(ptx::sdesc_sw128(ptx::smem_u32(sV), BOX, 1024));
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, w));
      };
      bool moved = false, ok = true;
      auto mma_S = [&](uint32_t i) {
        if (ptx::elect_one()) {
          moved |= lane != 0;
          const uint32_t dst = tmem + (i & 1u) * 128;
          const uint64_t k = i & 1u ? k_desc[1] : k_desc[0];
#pragma unroll 4
          for (int kk = 0; kk < HD / 16; ++kk) {
            const uint32_t off = (kk >> 2) * BOX + (kk & 3) * 32;
            ptx::mma_ss(dst, ptx::sdesc_advance(q_desc, off), ptx::sdesc_advance(k, off), C::IDESC_S, kk > 0 ? 1u : 0u);
          }
          ptx::mma_commit(s_full + (i & 1u));
          ptx::mma_commit(k_empty + (i & 1u));
        }
        __syncwarp();
      };
      uint32_t i = 0, runs = 0;
      do {
        if (!(ok = wait(q_full, runs & 1u))) break;
        ++runs;
        if (!(ok = wait(k_full + (i & 1u), (i >> 1) & 1u))) break;
        ptx::tc_fence_after();
        mma_S(i);
        for (int s = 0; s < wk.run; ++s, ++i) {
          if (s + 1 < wk.run) {
            if (!(ok = wait(k_full + ((i + 1) & 1u), ((i + 1) >> 1) & 1u))) break;
            ptx::tc_fence_after();
            mma_S(i + 1);
          }
          if (!(ok = wait(p_full + (i & 1u), (i >> 1) & 1u))) break;
          if (!(ok = wait(v_full, i & 1u))) break;
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
            moved |= lane != 0;
#pragma unroll 4
            for (int kk = 0; kk < BN / 16; ++kk)
              ptx::mma_ts(tmem + 256, tmem + (i & 1u) * 128 + kk * 8, ptx::sdesc_advance(v_desc, kk * 2048), C::IDESC_PV,
                          (s > 0 || kk > 0) ? 1u : 0u);
            ptx::mma_commit(v_empty);
            ptx::mma_commit(pv_done);
          }
          __syncwarp();
        }
      } while (ok && wk.next(P));
      if (!ok) {
        if (ptx::elect_one()) ptx::mma_commit(drain);
        __syncwarp();
        ptx::mbar_wait_drain(drain, 0u);
      }
      if (__any_sync(0xffffffffu, moved) && lane == 0) atomicOr(P.status, ATTN_DEV_ISSUER);
    }
  } else if (wg < 3) {
    ptx::reg_release<REG_CONVERT>();
    // -------------------------------------------------------------- converters
    // A thread takes one 16-code piece of every 128 / P-th row (P threads a row), so that its places are a constant
    // step apart in the codes and, eight rows being the swizzle's period, in the tile.
    if (last > first) {
      const int side = wg - 1;   // K, V
      ptx::WaitCtx w{abort_flag, P.status, 2u};
      const int tid = threadIdx.x & 127;
      const int per = (side ? P.p.dv : P.p.d) / 16;                 // pieces of a row
      const int lanes = per > 4 ? 8 : per > 2 ? 4 : per;            // threads of a row
      const int r1 = tid / lanes, c = tid - r1 * lanes, step = 128 / lanes;
      const bool mine = c < per;
      // the two 16-byte pieces of the tile; those of the second 64 columns in the other order, so that the eight threads
      // of a phase write to eight different 16-byte columns
      const int block = c >> 2, at = 2 * (c & 3);
      uint8_t* to = (side ? sV : sK) + block * BOX + r1 * 128;
      uint8_t* const to0 = to + (((at + block) ^ (r1 & 7)) << 4);
      uint8_t* const to1 = to + (((at + 1 - block) ^ (r1 & 7)) << 4);
      const uint32_t places = side ? 1u : 2u;   // of tiles
      uint64_t* full = side ? v_full : k_full;
      uint64_t* empty = side ? v_empty : k_empty;
      uint32_t i = 0, runs = 0;
      bool ok = true;
      do {
        if (side == 0) {
          // -------------------------------------------------------- the run's queries, as fp16 at powers of two
          // HD / 8 lanes a row. (By the softmax warps, each its own rows, 6 us before a run's first product.) The units
          // have two places: those of the run after next come when S of the next run's last tile is out, which waits for
          // this run's softmax.
          // (no product reads Q any more)
          if (i > 0 && !(ok = ptx::mbar_wait(empty + ((i - 1) & 1u), ((i - 1) >> 1) & 1u, w))) break;
          constexpr int LANES = HD / 8, ROWS = 128 / LANES;
          const int b = wk.e / P.groups, r0 = (wk.e - b * P.groups) * BM, R = P.p.R - r0, d = P.p.d;
          const long long head = static_cast<long long>(b * P.p.Hkv + wk.h) * P.p.R + r0;
          const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(P.Q) + head * d;
          const int q = tid % LANES;   // this lane's 8 columns
          // loads on their way together: 8 (58 in place of 60 us at 64 rows), with 128 rows 2 (for want of registers: 89 in
          // place of 85 us with 8)
          constexpr int N = CP > 1 ? (C::RP / ROWS < 8 ? C::RP / ROWS : 8) : 2;
          for (int k0 = 0; k0 < C::RP / ROWS; k0 += N) {
            uint4 raw[N];
#pragma unroll
            for (int k = 0; k < N; ++k) {
              const int r = (k0 + k) * ROWS + tid / LANES;
              raw[k] = make_uint4(0u, 0u, 0u, 0u);
              if (r < R && 8 * q < d)
                raw[k] = *reinterpret_cast<const uint4*>(src + static_cast<long long>(r) * d + 8 * q);
            }
#pragma unroll
            for (int k = 0; k < N; ++k) {
              const int r = (k0 + k) * ROWS + tid / LANES;
              const uint32_t u[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
              float top = 0.f;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                top = ptx::fmax3(top, fabsf(__uint_as_float(u[e] << 16)), fabsf(__uint_as_float(u[e] & 0xffff0000u)));
#pragma unroll
              for (int o = 1; o < LANES; o *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
              // the largest to [2^14, 2^15), by the exponent's bits (0 and infinities: as they are)
              const int bits = static_cast<int>(__float_as_uint(top) >> 23);
              const int ex = top > 0.f && bits < 255 ? max(bits - 141, -126) : 0;
              const float up = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
              if (q == 0) units[(runs & 1u) * 128 + r] = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
              uint32_t h[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                h[e] = pack_f16(__uint_as_float(u[e] << 16) * up, __uint_as_float(u[e] & 0xffff0000u) * up);
#pragma unroll
              for (int k2 = 0; k2 < CP; ++k2) {
                const int row = k2 * C::RP + r;
                *reinterpret_cast<uint4*>(sQ + (q >> 3) * BOX + row * 128 + (((q & 7) ^ (row & 7)) << 4)) =
                    make_uint4(h[0], h[1], h[2], h[3]);
              }
            }
          }
          ptx::fence_proxy_async_smem();
          ptx::mbar_arrive(q_full);
          ptx::mbar_arrive(unit_full + (runs & 1u));
          ++runs;
        }
        for (int s = wk.s0; ok && s < wk.s0 + wk.run; ++s, ++i) {
          const uint32_t item = 2 * i + side;
          const int sl = slot(item);
          if (!(ok = ptx::mbar_wait(raw_full + sl, par(item), w))) break;
          const uint32_t place = i % places;
          if (!(ok = ptx::mbar_wait(empty + place, (i / places & 1u) ^ 1u, w))) break;
          if (mine) {
            const uint32_t none = none_of[sl];
            const int key0 = wk.key0(s);
            const int lo = side ? wk.hull.x - key0 : 0, hi = side ? wk.hull.y - key0 : BN;   // rows outside: zeros
            const bool plain = none == 0u && lo <= 0 && hi >= BN;
            const uint8_t* from = smem + C::OFF_RAW + sl * C::RAW + (r1 * per + c) * 16;
#pragma unroll
            for (int k0 = 0; k0 < 8; k0 += 4) {   // the loads of four on their way together
              if (k0 >= lanes) break;
              uint4 u[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (k0 + k < lanes) u[k] = *reinterpret_cast<const uint4*>(from + (k0 + k) * step * per * 16);
              if (!plain) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const int r = r1 + (k0 + k) * step;
                  if (r < lo || r >= hi || (none >> ((r >> 4) & 31) & 1u)) u[k] = make_uint4(0u, 0u, 0u, 0u);
                }
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if (k0 + k >= lanes) break;
                const uint32_t v[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
                uint32_t h[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  h[2 * e] = cache::codes_to_half2(static_cast<uint16_t>(v[e]));
                  h[2 * e + 1] = cache::codes_to_half2(static_cast<uint16_t>(v[e] >> 16));
                }
                const uint4 p0 = make_uint4(h[0], h[1], h[2], h[3]), p1 = make_uint4(h[4], h[5], h[6], h[7]);
                const int off = (k0 + k) * step * 128 + static_cast<int>(place) * C::TILE;
                *reinterpret_cast<uint4*>(to0 + off) = block ? p1 : p0;
                *reinterpret_cast<uint4*>(to1 + off) = block ? p0 : p1;
              }
            }
          }
          ptx::fence_proxy_async_smem();
          ptx::mbar_arrive(full + place);
          ptx::mbar_arrive(raw_empty + sl);
        }
      } while (ok && wk.next(P));
    }
  } else {
    ptx::reg_acquire<REG_SOFTMAX>();
    // -------------------------------------------------------------- softmax
    if (last > first) {
      const int quad = warp & 3, row = quad * 32 + lane;
      const int copy = row / C::RP, r = row - copy * C::RP;   // (the copy is the warp's)
      const uint32_t tS0 = tmem + (static_cast<uint32_t>(quad * 32) << 16);
      const uint32_t tO = tS0 + 256;
      ptx::WaitCtx w{abort_flag, P.status, 4u};
      constexpr int GROUPS = C::KEYS / 16;
      const int Tq = P.p.Tq, dv = P.p.dv;
      const bool cap = P.p.softcap > 0.f, bias = P.p.slopes != nullptr;
      uint32_t i = 0, runs = 0;
      bool ok = true;
      do {
        const int b = wk.e / P.groups, r0 = (wk.e - b * P.groups) * BM;
        const int bh = b * P.p.Hkv + wk.h;
        const int R = P.p.R - r0;   // rows from the group on
        const bool live = r < R;
        const long long head = static_cast<long long>(bh) * P.p.R + r0;
        const bool idle = quad * 32 % C::RP >= R;   // a warp without live rows has nothing to compute
        int from = 0x7fffffff, to = 0, pos = 0;
        float slope2 = 0.f;
        if (live) {
          const int tok = (r0 + r) % Tq;
          cache::row_range(P.mask, static_cast<long long>(b) * Tq + tok, tok, cache::tokens_of(P.c, b),
                           cache::new_of(P.c, b, Tq), P.p.Tk, P.window, &from, &to, &pos);
          if (bias) slope2 = P.p.slopes[wk.h * P.p.G + (r0 + r) / Tq] * scored::kLog2e;
        }
        if (!(ok = __all_sync(0xffffffffu, ptx::mbar_wait(unit_full + (runs & 1u), (runs >> 1) & 1u, w)))) {
          if constexpr (CP == 1) break;
        }
        const float fac = units[(runs & 1u) * 128 + r] * (cap ? 1.f : P.sc2);
        ++runs;
        // keys that every live row of the warp sees
        const int all_lo = __reduce_max_sync(0xffffffffu, live ? from : 0);
        const int all_hi = __reduce_min_sync(0xffffffffu, live ? to : 0x7fffffff);
        float m_used = -CUDART_INF_F, l = 0.f;
        for (int s = wk.s0; ok && s < wk.s0 + wk.run; ++s, ++i) {
          const int key0 = wk.key0(s) + copy * C::KEYS;   // the thread's keys of the tile: KEYS from there on
          const float4* sc = scales + (i % NSC) * 8 + copy * GROUPS;
          const uint32_t tS = tS0 + (i & 1u) * 128;
          // every lane must agree before the warp-wide tcgen05 loads
          if (!(ok = __all_sync(0xffffffffu, ptx::mbar_wait(sc_full + i % NSC, (i / NSC) & 1u, w) &&
                                                 ptx::mbar_wait(s_full + (i & 1u), (i >> 1) & 1u, w))))
            break;
          ptx::tc_fence_after();
          bool need = false;
          float corr = 1.f;
          if (!idle) {
            constexpr int N = C::KEYS;
            uint32_t raw[N / 32][32];
#pragma unroll
            for (int c = 0; c < N / 32; ++c) ptx::tmem_ld32(tS + copy * N + c * 32, raw[c]);
#pragma unroll
            for (int c = 0; c < N / 32; ++c) ptx::tmem_ld_wait(raw[c]);
            float* x = reinterpret_cast<float*>(&raw[0][0]);
            // scores in log2 units with the value scale; the raw ones may hold anything where no row sees the key
            if (cap) {
#pragma unroll
              for (int g = 0; g < GROUPS; ++g) {
                const float f = fac * sc[g].x;
#pragma unroll
                for (int e = 0; e < 16; ++e) x[16 * g + e] *= f;
              }
              float top = 0.f;
#pragma unroll
              for (int e = 0; e < N; e += 2) top = ptx::fmax3(top, fabsf(x[e]), fabsf(x[e + 1]));
              if (__all_sync(0xffffffffu, !(top > P.cap.limit4))) {
                const scored::CapPoly<scored::kCapPoly4> poly(P.cap);
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) {
                  const F2 lv = dup(sc[g].y);
#pragma unroll
                  for (int e = 0; e < 16; e += 2) {
                    const F2 v = f2(x[16 * g + e], x[16 * g + e + 1]), y = fma2(v, poly(v), lv);
                    x[16 * g + e] = y.x, x[16 * g + e + 1] = y.y;
                  }
                }
              } else {
#pragma unroll
                for (int e = 0; e < N; ++e) x[e] = scored::cap_any(x[e], P.cap) + sc[e >> 4].y;
              }
            } else {
#pragma unroll
              for (int g = 0; g < GROUPS; ++g) {
                const F2 f = dup(fac * sc[g].x), lv = dup(sc[g].y);
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                  const F2 y = fma2(f2(x[16 * g + e], x[16 * g + e + 1]), f, lv);
                  x[16 * g + e] = y.x, x[16 * g + e + 1] = y.y;
                }
              }
            }
            if (bias) {
              const float delta = static_cast<float>(key0 - pos);
#pragma unroll
              for (int e = 0; e < N; ++e) x[e] = fmaf(-slope2, fabsf(delta + static_cast<float>(e)), x[e]);
            }
            if (key0 < all_lo || key0 + N > all_hi) {
#pragma unroll
              for (int c = 0; c < N / 32; ++c) {
                const uint32_t seen = scored::bit_range(from - key0 - 32 * c, to - key0 - 32 * c);
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (!(seen & (1u << e))) x[32 * c + e] = -CUDART_INF_F;
              }
            }
            float g4[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) g4[k] = fmaxf(x[k], x[k + 4]);
#pragma unroll
            for (int e = 8; e < N; e += 8)
#pragma unroll
              for (int k = 0; k < 4; ++k) g4[k] = ptx::fmax3(g4[k], x[e + k], x[e + 4 + k]);
            const float m_new = fmaxf(m_used, ptx::fmax3(g4[0], g4[1], fmaxf(g4[2], g4[3])));
            if (s == wk.s0) {
              m_used = m_new;
            } else if (m_new > m_used + TAU) {
              need = true;
              corr = ptx::ex2(m_used - m_new);   // 0 when m_used = -inf
              l *= corr;
              m_used = m_new;
            }
            const float ref = m_used == -CUDART_INF_F ? 0.f : m_used - SHIFT;   // no key seen yet
            const F2 nref = dup(-ref);
            F2 ls[2] = {dup(0.f), dup(0.f)};
#pragma unroll
            for (int c = 0; c < N / 32; ++c) {
              uint32_t pk[16];
#pragma unroll
              for (int g = 0; g < 2; ++g) {
                const F2 iv = dup(sc[2 * c + g].z);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const int n = 32 * c + 16 * g + 2 * e;
                  const F2 p = scored::ex2(add2(f2(x[n], x[n + 1]), nref));
                  ls[e & 1] = fma2(p, iv, ls[e & 1]);
                  pk[8 * g + e] = pack_f16(p.x, p.y);
                }
              }
              ptx::tmem_st16(tS + copy * (N / 2) + 16 * c, pk);
            }
            if constexpr (CP > 1) {   // the other copies' keys
              uint32_t zero[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) zero[e] = 0u;
#pragma unroll
              for (int c = 0; c < 4; ++c)
                if (c / (N / 32) != copy) ptx::tmem_st16(tS + 16 * c, zero);
            }
            const F2 sum = add2(ls[0], ls[1]);
            l += sum.x + sum.y;
          }
          if (i > 0 && !(ok = __all_sync(0xffffffffu, ptx::mbar_wait(pv_done, (i - 1) & 1u, w)))) break;
          if (__any_sync(0xffffffffu, need)) {   // O *= corr before the product of this tile adds to it
            ptx::tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < HD / 32; ++c) {
              uint32_t o[32];
              ptx::tmem_ld32(tO + c * 32, o);
              ptx::tmem_ld_wait(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
              ptx::tmem_st32(tO + c * 32, o);
            }
          }
          ptx::tmem_st_wait();
          ptx::tc_fence_before();
          ptx::mbar_arrive(p_full + (i & 1u));
        }
        // (the four warps leave together where one's wait gave up)
        if (CP > 1 && !softmax_barrier_all(ok)) break;
        if (!ok) break;
        // ---------------------------------------------------------- epilogue
        if (!(ok = __all_sync(0xffffffffu, ptx::mbar_wait(pv_done, (i - 1) & 1u, w)))) {
          if constexpr (CP == 1) break;
        }
        ptx::tc_fence_after();
        // the copies' maxima and sums: this copy's weight w_c of the row, and the row's sum
        float weight = 1.f, top = m_used, sum = l;
        if constexpr (CP > 1) {
          float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
          ml[row] = make_float2(m_used, l);
          if (!softmax_barrier_all(ok)) break;
#pragma unroll
          for (int c = 0; c < CP; ++c) top = fmaxf(top, ml[c * C::RP + r].x);
          const float ref = top == -CUDART_INF_F ? 0.f : top;
          sum = 0.f;
#pragma unroll
          for (int c = 0; c < CP; ++c) sum += ml[c * C::RP + r].y * ptx::ex2(ml[c * C::RP + r].x - ref);
          weight = ptx::ex2(m_used - ref);
        }
        const bool none = sum == 0.f;   // no key seen (a NaN among the row's scores goes through)
        const float inv_l = none ? 0.f : weight / sum;
        const float lse = none ? -CUDART_INF_F : (top - SHIFT + log2f(sum)) * 0.69314718055994530942f;
        const bool whole = wk.run == wk.n;
        const long long part = (static_cast<long long>(blockIdx.x) * 2 + (wk.s0 > 0 ? 0 : 1)) * BM;
        const long long base = whole ? head : part;
        // the four rows of this lane's quad, of which it stores every fourth 16-byte piece
        const int row4 = r & ~3;
        // 32 columns from c on of this thread's row, to the result or the part
        auto store = [&](float (&f)[32], int c) {
          uint4 pk[4];
          if (!whole) {   // fp32: 16 columns at a time
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int e = 16 * h + 4 * k;
                pk[k] = make_uint4(__float_as_uint(f[e]), __float_as_uint(f[e + 1]), __float_as_uint(f[e + 2]),
                                   __float_as_uint(f[e + 3]));
              }
              scored::quad_transpose(pk, lane);
              const int col = c + 16 * h + 4 * (lane & 3);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (row4 + k < R && col < dv) *reinterpret_cast<uint4*>(P.Opart + (base + row4 + k) * dv + col) = pk[k];
            }
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              pk[k] = make_uint4(ptx::pack_bf16(f[8 * k], f[8 * k + 1]), ptx::pack_bf16(f[8 * k + 2], f[8 * k + 3]),
                                 ptx::pack_bf16(f[8 * k + 4], f[8 * k + 5]), ptx::pack_bf16(f[8 * k + 6], f[8 * k + 7]));
            scored::quad_transpose(pk, lane);
            const int col = c + 8 * (lane & 3);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (row4 + k < R && col < dv)
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(P.O) + (base + row4 + k) * dv + col) = pk[k];
          }
        };
        auto load = [&](float (&f)[32], int c) {
          uint32_t o[32];
          ptx::tmem_ld32(tO + c, o);
          ptx::tmem_ld_wait(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) f[e] = none ? 0.f : __uint_as_float(o[e]) * inv_l;
        };
        if constexpr (CP == 1) {
          if (!idle) {
#pragma unroll 1
            for (int c = 0; c < HD; c += 32) {
              float f[32];
              load(f, c);
              store(f, c);
            }
          }
        } else {
          // each copy finishes half of the columns: 32 at a time, the other half's go to the other copy (RP >= R, so that
          // the copies have the same live warps)
#pragma unroll 1
          for (int c = 0; c < HD / 2; c += 32) {
            float f[32];
            float4* to = reinterpret_cast<float4*>(smem + C::OFF_SUMS) + ((1 - copy) * C::RP + r) * 8;
            const float4* from4 = reinterpret_cast<const float4*>(smem + C::OFF_SUMS) + (copy * C::RP + r) * 8;
            if (!idle) {
              load(f, (1 - copy) * (HD / 2) + c);
#pragma unroll
              for (int k = 0; k < 8; ++k) to[k ^ (r & 7)] = make_float4(f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]);
            }
            softmax_barrier_all(true);
            if (!idle) {
              load(f, copy * (HD / 2) + c);
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float4 v = from4[k ^ (r & 7)];
                f[4 * k] += v.x, f[4 * k + 1] += v.y, f[4 * k + 2] += v.z, f[4 * k + 3] += v.w;
              }
              store(f, copy * (HD / 2) + c);
            }
            softmax_barrier_all(true);
          }
        }
        if (live && copy == 0) (whole ? P.LSE : P.LSEpart)[base + r] = lse;
        ptx::tc_fence_before();
      } while (wk.next(P));
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

template <int HD, int CP>
cudaError_t launch(const CacheTokens& a) {
  using C = Cfg<HD, CP>;
  static_assert(C::SMEM <= 227 * 1024, "shared memory");
  const Params P = cache_walk::params(a);
  auto kern = tiles_kernel<HD, CP>;
  // the register split must fit the launch allocation (see ptx::reg_acquire)
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(kern, C::SMEM, done);
  if (e != cudaSuccess) return e;
  static std::atomic<int> regs{0};   // (of the code, the same on every device; a query that fails is made again)
  int n = regs.load(std::memory_order_relaxed);
  if (n == 0) {
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
    regs.store(n = fa.numRegs, std::memory_order_relaxed);
  }
  if (n < REG_CONVERT || n > REG_SOFTMAX || 4 * n < REG_CTRL + 2 * REG_CONVERT + REG_SOFTMAX)
    return cudaErrorInvalidConfiguration;
  if ((e = launch_over(kern, a.grid, THREADS, C::SMEM, a.stream, P)) != cudaSuccess) return e;
  return cache_walk::launch_join<false>(P, a.grid, BM, a.stream);
}

template <int HD>
cudaError_t rows(const CacheTokens& a) {
  return a.p.R <= 64 ? launch<HD, 2>(a) : launch<HD, 1>(a);
}

}  // namespace cache_tiles

cudaError_t launch_cache_tiles(const CacheTokens& a) {
  return a.p.d <= 64 && a.p.dv <= 64 ? cache_tiles::rows<64>(a) : cache_tiles::rows<128>(a);
}

}  // namespace attn
