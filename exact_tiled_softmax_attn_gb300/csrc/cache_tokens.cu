// Scored attention of few query rows over a paged cache (d, dv <= 128), whose
// pages hold e4m3 codes with a scale per page and head, or bf16.
//
// Reads every seen key and value once, where it lies: bound by memory. The
// keys that a group of at most 8, 16 or 32 packed rows of a key head sees - the
// hull of their ranges - are cut into stages of 64 at multiples of 64; all
// stages of the launch form one list, of which every CTA takes an equal
// contiguous share, so sequences of any lengths load the SMs evenly. A CTA
// that holds all stages of a group writes its rows' results; the others leave
// partial results, which a second kernel joins in order. Short sequences have
// no list and no second kernel: a cluster of up to eight CTAs for each group,
// which read each other's states through distributed shared memory.
//
// A producer warp looks the pages up, 32 at a time and ahead of their use, and
// fills a ring of stages by TMA, a box per page (or 64 tokens of one), with the
// scales beside the ring; 4 warps per row tile each take 16 of a stage's 64
// keys - which lie in one page - and keep a running maximum, sum and
// accumulator of their own, joined at the end of the run. The products run on
// mma.m16n8k16, keys (or columns of V) as its 16 and rows as its 8: S^T = K Q^T
// and O^T = V^T P^T, so that eight rows cost half of what they would as half of
// a 16-row operand, and what was read and converted of K and V serves all rows
// of a warp. With few rows the tcgen05 tile of 128 would be mostly empty, and
// at this intensity the memory is what counts.
//
// e4m3 codes go through fp16, which holds every one of them exactly (pairs by
// one conversion; for V after a byte permute that pairs two keys). Queries go
// through fp16 too, each row times a power of two that brings its largest
// element to [2^14, 2^15): bf16's 8 bits fit, and what falls below fp16's range
// is 2^-38 of the row's largest. fp32 queries are two fp16 terms each, and so
// are their weights. The scales cost nothing per element: the key scale is part
// of the factor that each score is multiplied by anyway, and the value scale
// enters as its logarithm, added in the same instruction: weights are held as
// p vs, relative to a reference, and the sum takes p = (p vs) / vs in the FMA
// that adds it.
//
// As fp16 the weights keep their 11 bits down to 2^-21 of that reference, so it
// may not stand for a page of zeros, or of tokens that no row sees, whose scale
// is 2^30 times the others'. Where the value scales since it was set are more
// than 2^8 apart, it is set anew: to min(W, S vs), W the largest p vs and S the
// largest p so far, vs the scale from here on, but no less than W 2^-72. A weight
// is then in full as long as p is at least 2^-13 of the largest p, whatever the
// scales (up to 2^72 apart; at 2^80, the most there is, 2^-5), and smaller ones
// are off by 2^-32 of the reference. Sums and accumulators take the ratio of two
// references in 32 bits: 2^15 of a weight, 448, 2^30 keys and 2^72 are below
// 2^126. The producer compares the scales, of all that a CTA takes on.
//
// Fragments are read as 16-byte vectors: the columns of Q and K are permuted
// alike, so that a thread's fragments of K are 16 adjacent codes of a row; the
// weights become an operand by an 8x8 transpose in registers. Within a 16-key
// group fragment row g stands for key g (g even) or g ^ 4 (g odd): the eight
// threads of one shared-memory phase then touch eight different 16-byte columns
// in both reads.
//
// 32 sequences of up to 32768 keys, H=32 Hkv=8 d=128, 1.27 GB of codes: 194 us,
// 6.5 TB/s (with the rows as the 16 of the products 203); fp32 queries 202 us
// (341); bf16 pages, 2.53 GB, 363 us, 7.0 TB/s. 16 rows a key head cost more
// than memory: 16 sequences of up to 12000 keys, Hkv=4, 33 us with 4 rows, 43
// with 16, 66 with 32. A step of 16 keys is a chain of about 950 cycles a warp;
// what hides it is the three CTAs (twelve such warps) of an SM.
#include <cuda.h>
#include <cuda_bf16.h>
#include <math_constants.h>
#include <stdint.h>

#include "cache.h"
#include "cache_walk.cuh"
#include "common.cuh"
#include "ptx.cuh"
#include "scored.h"
#include "scored_math.cuh"

namespace attn {
namespace cache_tokens {

using cache_walk::Params;
using cache_walk::share;
using cache_walk::Walk;

constexpr int BK = 64;              // keys per stage
constexpr float TAU = 8.0f;
// The value scales that a reference stands for lie within 2^8 of one
// another, and it is let down by at most 2^DEPTH (see the header).
constexpr float SPREAD = 8.01f, DEPTH = 72.0f;   // (8, and the logarithms' rounding)
// Where they do not, a stage's scales come with the largest of those before plus APART (log2), else with 0.
constexpr float APART = 256.0f;

// E: uint8_t (e4m3) or bf16; SPLIT: fp32 queries and results (e4m3 only); a
// warp has 8 NT rows, and RT row tiles of 4 warps share the stages.
template <typename E, bool SPLIT, int HD, int NT, int RT>
struct Cfg {
  static constexpr bool CODES = sizeof(E) == 1;
  static constexpr int RW = 8 * NT;               // rows of a warp
  static constexpr int RB = RW * RT;              // rows of a group
  static constexpr int KB = CODES ? 1 : HD / 64;  // boxes of a key's row
  static constexpr int BOX = BK * (CODES ? HD : 128);
  static constexpr int STAGE = 2 * KB * BOX;
  static constexpr int WARPS = 4 * RT;            // compute warps
  static constexpr int THREADS = 32 * (WARPS + 1);
  static constexpr int CTAS = cache_token_ctas(RB, CODES);   // per SM
  static constexpr float SHIFT = CODES ? 7.f : 0.f;   // weights up to 2^(TAU + SHIFT) keep more of fp16's range
  static constexpr int LDO = HD + 4;
  static constexpr int JOIN = RB * 2 * (LDO + 2) * 4;        // rows, maxima and sums of two key groups
  static constexpr int BUDGET = 227 * 1024 / CTAS - 1024 - JOIN - 2048;
  static constexpr int NST = BUDGET / STAGE < 8 ? BUDGET / STAGE : 8;
  static constexpr int OFF_JOIN = NST * STAGE;
  static constexpr int OFF_BAR = OFF_JOIN + JOIN;
  static constexpr int OFF_SCALE = OFF_BAR + 2 * NST * 8;    // [NST][4] float4: of a stage's 16-key groups
  static constexpr int OFF_MISC = OFF_SCALE + NST * 64;
  static constexpr int OFF_HULL = OFF_MISC + 64 + 128;   // after the scan: [THREADS] hulls
  static constexpr int OFF_TOP = OFF_HULL + 8 * THREADS;     // [WARPS][RW] float2: log2 of W and S of a row
  static constexpr int SMEM = OFF_TOP + (CODES ? 8 * WARPS * RW : 0);
};

template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t lo_codes(uint32_t w) { return cache::codes_to_half2(static_cast<uint16_t>(w)); }
__device__ __forceinline__ uint32_t hi_codes(uint32_t w) { return cache::codes_to_half2(static_cast<uint16_t>(w >> 16)); }

// Barriers of the compute warps alone; the second tells whether `ok` holds in all of them.
template <int N>
__device__ __forceinline__ void compute_barrier() {
  asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ bool compute_barrier_all(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"(ok ? 1u : 0u), "n"(N)
      : "memory");
  return r != 0;
}

// The transpose of an 8x8 matrix of 16-bit elements, a row per four lanes.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Byte offset of 16-byte piece c of row r in a box of rows of 64 or 128 bytes, as TMA's swizzles lay it out.
template <int WIDTH>
__device__ __forceinline__ int piece(int r, int c) {
  return r * WIDTH + ((WIDTH == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4);
}

// The CTA's share of the stages. In a cluster its rows' states are left in the
// slots 0 of `join`.
template <typename E, bool SPLIT, int HD, int NT, int RT, bool CLUSTER>
__device__ __forceinline__ void attend(const CUtensorMap& tmK, const CUtensorMap& tmV, const Params& P, uint8_t* smem) {
  using C = Cfg<E, SPLIT, HD, NT, RT>;
  constexpr bool CODES = C::CODES;
  constexpr int RB = C::RB;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if ((ptx::smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicOr(P.status, ATTN_DEV_BAD_SMEM);
    return;
  }
  float* join = reinterpret_cast<float*>(smem + C::OFF_JOIN);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + C::NST;
  float4* scales = reinterpret_cast<float4*>(smem + C::OFF_SCALE);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC);
  int* found = reinterpret_cast<int*>(smem + C::OFF_MISC + 16);   // {entry, offset}
  int* scan = reinterpret_cast<int*>(smem + C::OFF_MISC + 64);
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NST; ++s) {
      ptx::mbar_init(full + s, CODES ? 2 : 1);   // the boxes, and the scales
      ptx::mbar_init(empty + s, C::WARPS);
    }
    *abort_flag = 0u;
    ptx::fence_mbar_init();
    ptx::tma_prefetch_desc(&tmK);
    ptx::tma_prefetch_desc(&tmV);
  }
  // (the launch overlaps the end of the kernel before; the join's, earlier than this one's end, costs 1 to 3 us)
  ptx::grid_wait();
  // This CTA's share of the launch's stages.
  int2* hulls = reinterpret_cast<int2*>(smem + C::OFF_HULL);
  int first, last;
  const bool one = share<RB, BK, C::THREADS>(P, hulls, scan, found, &first, &last);
  if (last <= first) return;
  Walk<RB, BK> wk;
  wk.begin(P, one ? hulls : nullptr, found[0], found[1], last - first);

  if (warp == C::WARPS) {
    // ------------------------------------------------------------ producer
    ptx::WaitCtx w{abort_flag, P.status, 1u};
    bool ok = true;
    uint32_t it = 0;
    const int shift = P.c.shift;
    const int nb = shift < 6 ? 64 >> shift : 1;               // boxes of a stage, of `rows` keys each
    const int rows = shift < 6 ? 1 << shift : 64;
    const int planes = P.c.pages * P.p.Hkv;                   // (a plane past the last reads as zeros)
    do {
      float vs_lo = CUDART_INF_F, vs_hi = -CUDART_INF_F;   // log2 of the value scales since the references were set
      const int b = wk.e / P.groups;
      const int key_s0 = wk.key0(wk.s0), n_box = wk.run * nb;
      // lane i looks up box i of the next 32: its plane, and its scales
      auto find = [&](int box) {
        const int key = key_s0 + box * rows;
        const bool seen = box < n_box && key < wk.hull.y && key + rows > wk.hull.x;
        const int at = seen ? cache::page_of(P.c, b, key >> shift) : -1;
        return at >= 0 ? at * P.p.Hkv + wk.h : -1;
      };
      int plane = find(lane);
      for (int box0 = 0; ok && box0 < n_box; box0 += 32) {
        float ks = 1.f, vs = 1.f;
        if (CODES && plane >= 0) {
          ks = P.c.scale[0][plane];
          vs = P.c.scale[1][plane];
        }
        const int next = find(box0 + 32 + lane);
        ks = cache::clamp_scale(ks);
        vs = cache::clamp_scale(vs);
        const float lv = CODES ? log2f(vs) : 0.f, iv = 1.f / vs;
        const int boxes = min(32, n_box - box0);
        for (int j = 0; j < boxes; j += nb, ++it) {
          const int st = it % C::NST;
          if (lane == 0) ok = ptx::mbar_wait(empty + st, ((it / C::NST) & 1u) ^ 1u, w);
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          if (!ok) break;
          if (lane == 0) ptx::mbar_arrive_expect_tx(full + st, C::STAGE);
          __syncwarp();
          const int i = lane / (2 * C::KB), what = lane % (2 * C::KB);   // this lane's box: K's, then V's
          const int at = __shfl_sync(0xffffffffu, plane, (j + i) & 31);
          if (i < nb) {
            const int key = key_s0 + (box0 + j + i) * rows;
            const bool is_v = what >= C::KB;
            const int col = what - (is_v ? C::KB : 0);
            ptx::tma_load_3d(smem + st * C::STAGE + what * C::BOX + i * rows * (C::BOX / BK), is_v ? &tmV : &tmK,
                             full + st, col * 64, key & ((1 << shift) - 1), at >= 0 ? at : planes);
          }
          if constexpr (CODES) {
            const int from = j + (shift < 6 ? (16 * (lane & 3)) >> shift : 0);   // box of 16-key group lane % 4
            float4 s = make_float4(__shfl_sync(0xffffffffu, ks, from), __shfl_sync(0xffffffffu, lv, from),
                                   __shfl_sync(0xffffffffu, iv, from), 0.f);
            const bool is = __shfl_sync(0xffffffffu, plane, from) >= 0;
            float lo = is ? s.y : CUDART_INF_F, hi = is ? s.y : -CUDART_INF_F;
#pragma unroll
            for (int o = 1; o < 4; o *= 2) {
              lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
              hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
            }
            const bool apart = vs_hi >= vs_lo && hi >= lo && fmaxf(hi, vs_hi) - fminf(lo, vs_lo) > SPREAD;
            if (apart) s.w = vs_hi + APART;
            vs_lo = apart ? lo : fminf(lo, vs_lo), vs_hi = apart ? hi : fmaxf(hi, vs_hi);
            if (!is) {   // zeros: any scale, before the first page a small one
              s.y = vs_lo < CUDART_INF_F ? vs_lo : -60.f;
              s.z = exp2f(-s.y);
            }
            if (lane < 4) scales[st * 4 + lane] = s;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(full + st);
          }
        }
        plane = next;
      }
    } while (ok && wk.next(P));
    if (!ok && lane == 0)   // let the copies in flight land before the CTA exits
      for (uint32_t n = it > static_cast<uint32_t>(C::NST) ? it - C::NST : 0u; n < it; ++n)
        ptx::mbar_wait_drain(full + n % C::NST, (n / C::NST) & 1u);
    return;
  }

  // -------------------------------------------------------------- compute
  ptx::WaitCtx w{abort_flag, P.status, 2u};
  const int rt = warp >> 2, kg = warp & 3;
  const int g = lane >> 2, t = lane & 3;
  const int Tq = P.p.Tq, d = P.p.d, dv = P.p.dv;
  const int krow = (g & 1) ? g ^ 4 : g;                 // key of fragment row g within 8
  const int k_lo = 2 * t, k_hi = (2 * t + 1) ^ 4;       // keys of operand elements 2t, 2t + 1 within 8
  constexpr float SHIFT = C::SHIFT;
  float2* top = reinterpret_cast<float2*>(smem + C::OFF_TOP) + warp * C::RW + 2 * t;   // [8 n + e]
  uint32_t it = 0;
  bool ok = true;
  // The fragments of Q: row 8 n + g of the warp's. Codes: elements 64 c + 16 t + 4 j .. + 3 as words 2 (4 c + j) and the
  // next (SPLIT: the second terms too); bf16: elements 32 c + 8 t .. + 7 as words 4 c ..
  uint32_t q[SPLIT ? 2 : 1][NT][HD / 8];
  float o[NT][HD / 16][4];   // [n][i][2 h + e]: row 8 n + 2 t + e, column col_of(i, h)
  auto col_of = [&](int i, int h) { return CODES ? (HD / 8) * g + 2 * i + h : (i >> 2) * 64 + 8 * g + 2 * (i & 3) + h; };
  do {
    const int b = wk.e / P.groups, r0 = (wk.e - b * P.groups) * RB + rt * C::RW;   // the warp's first row
    const int bh = b * P.p.Hkv + wk.h;
    const int R = P.p.R - r0;                           // rows from there on
    const int len = cache::tokens_of(P.c, b), n_new = cache::new_of(P.c, b, Tq);
    int lo[NT][2], hi[NT][2], pos[NT][2];
    float slope2[NT][2], fac[NT][2];
    int lo_all = 0, hi_all = 0x7fffffff;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        lo[n][e] = 0x7fffffff, hi[n][e] = 0, pos[n][e] = 0;
        slope2[n][e] = 0.f;
        const int row = 8 * n + 2 * t + e;
        if (row < R) {
          const int r = r0 + row, tok = r % Tq;
          cache::row_range(P.mask, static_cast<long long>(b) * Tq + tok, tok, len, n_new, P.p.Tk, P.window, &lo[n][e],
                           &hi[n][e], &pos[n][e]);
          if (P.p.slopes) slope2[n][e] = P.p.slopes[wk.h * P.p.G + r / Tq] * scored::kLog2e;
          lo_all = max(lo_all, lo[n][e]);
          hi_all = min(hi_all, hi[n][e]);
        }
      }
      const bool live = 8 * n + g < R;
      const long long at = (static_cast<long long>(bh) * P.p.R + r0 + 8 * n + g) * d;
      float unit = 1.f;
      if constexpr (!CODES) {
#pragma unroll
        for (int c = 0; c < HD / 32; ++c) {
          const int col = 32 * c + 8 * t;
          const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(P.Q) + at + col;
          const uint4 v = live && col < d ? *reinterpret_cast<const uint4*>(src) : make_uint4(0u, 0u, 0u, 0u);
          q[0][n][4 * c] = v.x, q[0][n][4 * c + 1] = v.y, q[0][n][4 * c + 2] = v.z, q[0][n][4 * c + 3] = v.w;
        }
      } else {
        float f[HD / 4];
        float top = 0.f;
#pragma unroll
        for (int c = 0; c < HD / 64; ++c) {
          const int col = 64 * c + 16 * t;
          const bool there = live && col < d;
          if constexpr (SPLIT) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(P.Q) + at + col);
              const float4 v = there ? src[j] : make_float4(0.f, 0.f, 0.f, 0.f);
              float* to = f + 16 * c + 4 * j;
              to[0] = v.x, to[1] = v.y, to[2] = v.z, to[3] = v.w;
            }
          } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(P.Q) + at + col);
              const uint4 v = there ? src[j] : make_uint4(0u, 0u, 0u, 0u);
              const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                f[16 * c + 8 * j + 2 * e] = __uint_as_float(u[e] << 16);
                f[16 * c + 8 * j + 2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
              }
            }
          }
        }
#pragma unroll
        for (int e = 0; e < HD / 4; ++e) top = fmaxf(top, fabsf(f[e]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // times 2^(14 - exponent of the largest); an infinity stays one
        const int ex = top > 0.f && top < CUDART_INF_F ? max(ilogbf(top) - 14, -126) : 0;
        const float up = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
        unit = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
#pragma unroll
        for (int e = 0; e < HD / 8; ++e) {
          const float x0 = f[2 * e] * up, x1 = f[2 * e + 1] * up;
          q[0][n][e] = pack_f16(x0, x1);
          if constexpr (SPLIT) {
            const float2 h = cache::half2_to_float2(q[0][n][e]);
            q[SPLIT ? 1 : 0][n][e] = pack_f16(x0 - h.x, x1 - h.y);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)   // (row 2 t + e's, from its lanes)
        fac[n][e] = __shfl_sync(0xffffffffu, unit, 4 * (2 * t + e)) * (P.p.softcap > 0.f ? 1.f : P.sc2);
    }
    // keys that every row of the warp sees
    lo_all = __reduce_max_sync(0xffffffffu, lo_all);
    hi_all = __reduce_min_sync(0xffffffffu, hi_all);
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -CUDART_INF_F;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int i = 0; i < HD / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
    }
    if (CODES) {
      __syncwarp();   // (the last run's are read)
      if (g == 0) {
#pragma unroll
        for (int n = 0; n < NT; ++n) top[8 * n] = top[8 * n + 1] = make_float2(-CUDART_INF_F, -CUDART_INF_F);
      }
      __syncwarp();
    }

    for (int s = wk.s0; s < wk.s0 + wk.run; ++s, ++it) {
      const int st = it % C::NST;
      if (!(ok = __all_sync(0xffffffffu, ptx::mbar_wait(full + st, (it / C::NST) & 1u, w)))) break;
      const int key0 = wk.key0(s) + 16 * kg;   // of this warp's 16
      if (key0 < wk.hull.y && key0 + 16 > wk.hull.x && R > 0) {
        const uint8_t* sK = smem + st * C::STAGE + 16 * kg * (C::BOX / BK);
        const uint8_t* sV = sK + C::KB * C::BOX;
        float4 sc = make_float4(1.f, 0.f, 1.f, 0.f);   // key scale, log2 of the value scale, 1 / value scale, see APART
        if constexpr (CODES) sc = scales[st * 4 + kg];
        // x[n][2 h + e]: key krow + 8 h, row 8 n + 2 t + e; two chains of products where a warp has eight rows
        constexpr int CH = NT == 1 ? 2 : 1;
        float part[CH][NT][4];
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) part[c][n][e] = 0.f;
        if constexpr (CODES) {
#pragma unroll
          for (int c = 0; c < HD / 64; ++c) {
            const uint4 k0 = *reinterpret_cast<const uint4*>(sK + piece<HD>(krow, 4 * c + t));
            const uint4 k1 = *reinterpret_cast<const uint4*>(sK + piece<HD>(8 + krow, 4 * c + t));
            const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t a0 = lo_codes(w0[j]), a1 = lo_codes(w1[j]), a2 = hi_codes(w0[j]), a3 = hi_codes(w1[j]);
              const int e = 2 * (4 * c + j);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                mma16816<true>(part[j % CH][n], a0, a1, a2, a3, q[0][n][e], q[0][n][e + 1]);
                if constexpr (SPLIT)
                  mma16816<true>(part[j % CH][n], a0, a1, a2, a3, q[SPLIT ? 1 : 0][n][e], q[SPLIT ? 1 : 0][n][e + 1]);
              }
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < HD / 32; ++c) {
            const uint4 k0 = *reinterpret_cast<const uint4*>(sK + (c >> 1) * C::BOX + piece<128>(krow, 4 * (c & 1) + t));
            const uint4 k1 = *reinterpret_cast<const uint4*>(sK + (c >> 1) * C::BOX + piece<128>(8 + krow, 4 * (c & 1) + t));
            const int e = 4 * c;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma16816<false>(part[0][n], k0.x, k1.x, k0.y, k1.y, q[0][n][e], q[0][n][e + 1]);
              mma16816<false>(part[CH - 1][n], k0.z, k1.z, k0.w, k1.w, q[0][n][e + 2], q[0][n][e + 3]);
            }
          }
        }
        float x[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[n][e] = CH == 2 ? part[0][n][e] + part[CH - 1][n][e] : part[0][n][e];
        // changed and masked scores, in log2 units and with the value scale
        if (P.p.softcap > 0.f) {   // the cap's form by the warp's scores; degree 4 holds where degree 2 does
          float top = 0.f;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if constexpr (CODES) x[n][e] *= fac[n][e & 1] * sc.x;
              top = fmaxf(top, fabsf(x[n][e]));
            }
          if (__all_sync(0xffffffffu, !(top > P.cap.limit4))) {
            const scored::CapPoly<scored::kCapPoly4> poly(P.cap);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 4; e += 2) {
                const scored::F2 v = scored::f2(x[n][e], x[n][e + 1]), y = poly(v);
                x[n][e] = fmaf(v.x, y.x, sc.y), x[n][e + 1] = fmaf(v.y, y.y, sc.y);
              }
          } else {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) x[n][e] = scored::cap_any(x[n][e], P.cap) + sc.y;
          }
        } else {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[n][e] = fmaf(x[n][e], fac[n][e & 1] * sc.x, sc.y);
        }
        if (P.p.slopes) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = key0 + krow + 8 * (e >> 1);
              x[n][e] = fmaf(-slope2[n][e & 1], fabsf(static_cast<float>(key - pos[n][e & 1])), x[n][e]);
            }
        }
        if (key0 < lo_all || key0 + 16 > hi_all) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = key0 + krow + 8 * (e >> 1);
              x[n][e] = key >= lo[n][e & 1] && key < hi[n][e & 1] ? x[n][e] : -CUDART_INF_F;
            }
        }
        if constexpr (CODES) {
          if (sc.w != 0.f) {   // the references as these scales want them
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float2 ws = top[8 * n + e];
                ws.x = fmaxf(ws.x, m[n][e]);
                ws.y = fmaxf(ws.y, m[n][e] - (sc.w - APART));
                const float mn = fmaxf(fminf(ws.x, ws.y + sc.y), ws.x - DEPTH);
                const float corr = m[n][e] == mn ? 1.f : ptx::ex2(m[n][e] - mn);
                m[n][e] = mn;
                l[n][e] *= corr;
#pragma unroll
                for (int i = 0; i < HD / 16; ++i) o[n][i][e] *= corr, o[n][i][2 + e] *= corr;
                __syncwarp();
                if (g == 0) top[8 * n + e] = ws;
                __syncwarp();
              }
          }
        }
        bool need = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) need = need || fmaxf(x[n][e], x[n][2 + e]) > m[n][e] + TAU;   // (from -inf: any score)
        if (__any_sync(0xffffffffu, need)) {
          // the running references move to the maxima
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float mn = fmaxf(x[n][e], x[n][2 + e]);
#pragma unroll
              for (int k = 4; k <= 16; k *= 2) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, k));
              mn = fmaxf(m[n][e], mn);
              const float corr = m[n][e] == mn ? 1.f : ptx::ex2(m[n][e] - mn);
              m[n][e] = mn;
              l[n][e] *= corr;
#pragma unroll
              for (int i = 0; i < HD / 16; ++i) o[n][i][e] *= corr, o[n][i][2 + e] *= corr;
            }
        }
        // Weights, and as the operand: keys 2 t, 2 t + 1 (word 0) and 8 + .. (word 1) of row 8 n + g. Over bf16 pages that
        // is bf16, V's type: O is off by 0.0022 of its norm, with fp16 by 0.0017. A second term, as fp32 queries have it,
        // would give 0.0017 too, at 0 to 3 % of the time with 8 and 16 rows and 12 % with 32 (90 -> 101 us, 16 sequences to
        // 16384 keys).
        uint32_t pb[SPLIT ? 2 : 1][NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float ref[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) ref[e] = m[n][e] == -CUDART_INF_F ? 0.f : m[n][e] - SHIFT;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[n][e] = ptx::ex2(x[n][e] - ref[e & 1]);
            l[n][e & 1] = CODES ? fmaf(x[n][e], sc.z, l[n][e & 1]) : l[n][e & 1] + x[n][e];
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t u = CODES ? pack_f16(x[n][2 * h], x[n][2 * h + 1]) : ptx::pack_bf16(x[n][2 * h], x[n][2 * h + 1]);
            pb[0][n][h] = transposed(u);
            if constexpr (SPLIT) {
              const float2 f = cache::half2_to_float2(u);
              pb[SPLIT ? 1 : 0][n][h] = transposed(pack_f16(x[n][2 * h] - f.x, x[n][2 * h + 1] - f.y));
            }
          }
        }
        // rows of V outside the hull may hold anything: P is 0 there, 0 * NaN is not
        const bool edge = key0 + 16 > wk.hull.y || key0 < wk.hull.x;
        auto outside = [&](int kr) { return key0 + kr >= wk.hull.y || key0 + kr < wk.hull.x; };
        if constexpr (CODES) {
          constexpr int W = HD / 32;   // words of a thread's columns: HD / 8 columns from (HD / 8) g on
          uint32_t v[4][W];            // keys k_lo, k_hi, 8 + k_lo, 8 + k_hi
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int kr = (i >> 1) * 8 + ((i & 1) ? k_hi : k_lo);
            if constexpr (HD == 128) {
              const uint4 u = *reinterpret_cast<const uint4*>(sV + piece<HD>(kr, g));
              v[i][0] = u.x, v[i][1] = u.y, v[i][W - 2] = u.z, v[i][W - 1] = u.w;
            } else {
              const uint2 u = *reinterpret_cast<const uint2*>(sV + piece<HD>(kr, g >> 1) + 8 * (g & 1));
              v[i][0] = u.x, v[i][1] = u.y;
            }
            if (edge && outside(kr)) {
#pragma unroll
              for (int j = 0; j < W; ++j) v[i][j] = 0u;
            }
          }
#pragma unroll
          for (int j = 0; j < W; ++j) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {   // columns 4 j + 2 half and the next: keys of a pair side by side
              const uint32_t sel = half ? 0x7362u : 0x5140u;
              const uint32_t u0 = __byte_perm(v[0][j], v[1][j], sel), u1 = __byte_perm(v[2][j], v[3][j], sel);
              const uint32_t a0 = lo_codes(u0), a1 = hi_codes(u0), a2 = lo_codes(u1), a3 = hi_codes(u1);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                mma16816<true>(o[n][2 * j + half], a0, a1, a2, a3, pb[0][n][0], pb[0][n][1]);
                if constexpr (SPLIT)
                  mma16816<true>(o[n][2 * j + half], a0, a1, a2, a3, pb[SPLIT ? 1 : 0][n][0], pb[SPLIT ? 1 : 0][n][1]);
              }
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < C::KB; ++c) {
            uint32_t v[4][4];   // keys k_lo, k_hi, 8 + k_lo, 8 + k_hi; elements 64 c + 8 g .. + 7
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int kr = (i >> 1) * 8 + ((i & 1) ? k_hi : k_lo);
              uint4 u = *reinterpret_cast<const uint4*>(sV + c * C::BOX + piece<128>(kr, g));
              if (edge && outside(kr)) u = make_uint4(0u, 0u, 0u, 0u);
              v[i][0] = u.x, v[i][1] = u.y, v[i][2] = u.z, v[i][3] = u.w;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {   // elements 64 c + 8 g + 2 i and the next
              const uint32_t a0 = __byte_perm(v[0][i], v[1][i], 0x5410u), a1 = __byte_perm(v[0][i], v[1][i], 0x7632u);
              const uint32_t a2 = __byte_perm(v[2][i], v[3][i], 0x5410u), a3 = __byte_perm(v[2][i], v[3][i], 0x7632u);
#pragma unroll
              for (int n = 0; n < NT; ++n) mma16816<false>(o[n][4 * c + i], a0, a1, a2, a3, pb[0][n][0], pb[0][n][1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(empty + st);
    }
    // Every compute warp gets here in every run, one whose wait gave up too,
    // so that they leave together.
    if (!compute_barrier_all<C::WARPS * 32>(ok)) break;
    // ------------------------------------------------------------ join the four key groups
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int k = 4; k <= 16; k *= 2) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], k);
    auto put = [&](int slot) {   // this warp's state into slot 0 or 1 of its row tile
      float* dst = join + (rt * 2 + slot) * C::RW * (C::LDO + 2);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float* p = dst + (8 * n + 2 * t + e) * (C::LDO + 2);
#pragma unroll
          for (int i = 0; i < HD / 16; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) p[col_of(i, h)] = o[n][i][2 * h + e];
          if (g == 0) {
            p[C::LDO] = m[n][e];
            p[C::LDO + 1] = l[n][e];
          }
        }
    };
    auto take = [&](int slot) {   // adds a slot's state to this warp's
      const float* src = join + (rt * 2 + slot) * C::RW * (C::LDO + 2);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float* p = src + (8 * n + 2 * t + e) * (C::LDO + 2);
          const float m2 = p[C::LDO], mn = fmaxf(m[n][e], m2);
          const float ref = mn == -CUDART_INF_F ? 0.f : mn;
          const float wa = ptx::ex2(m[n][e] - ref), wb = ptx::ex2(m2 - ref);
          m[n][e] = mn;
          l[n][e] = l[n][e] * wa + p[C::LDO + 1] * wb;
#pragma unroll
          for (int i = 0; i < HD / 16; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) o[n][i][2 * h + e] = o[n][i][2 * h + e] * wa + p[col_of(i, h)] * wb;
        }
    };
    if (kg >= 2) put(kg - 2);
    compute_barrier<C::WARPS * 32>();
    if (kg < 2) take(kg);
    if (kg == 1) put(1);   // (only this warp read slot 1)
    compute_barrier<C::WARPS * 32>();
    if (kg == 0) take(1);
    if (CLUSTER && kg == 0) put(0);   // (only this warp read slot 0)
    if (!CLUSTER && kg == 0) {
      const bool whole = wk.run == wk.n;
      const int which = wk.s0 > 0 ? 0 : 1;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = 8 * n + 2 * t + e;
          if (row >= R) continue;
          const bool none = l[n][e] == 0.f;   // no key seen (a NaN among the row's scores goes through)
          const float inv = 1.f / l[n][e];
          const float lse = none ? -CUDART_INF_F : (m[n][e] - SHIFT + log2f(l[n][e])) * 0.69314718055994530942f;
          const long long at = whole ? static_cast<long long>(bh) * P.p.R + r0 + row
                                     : (static_cast<long long>(blockIdx.x) * 2 + which) * RB + rt * C::RW + row;
          if (g == 0) (whole ? P.LSE : P.LSEpart)[at] = lse;
#pragma unroll
          for (int c = 0; c < HD / 16; c += 4) {   // 8 adjacent columns
            const int col = col_of(c, 0);
            if (col >= dv) continue;
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = none ? 0.f : o[n][c + (i >> 1)][2 * (i & 1) + e] * inv;
            if (!SPLIT && whole) {
              *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(P.O) + at * dv + col) =
                  make_uint4(ptx::pack_bf16(f[0], f[1]), ptx::pack_bf16(f[2], f[3]), ptx::pack_bf16(f[4], f[5]),
                             ptx::pack_bf16(f[6], f[7]));
            } else {
              float4* dst = reinterpret_cast<float4*>((whole ? static_cast<float*>(P.O) : P.Opart) + at * dv + col);
              dst[0] = make_float4(f[0], f[1], f[2], f[3]);
              dst[1] = make_float4(f[4], f[5], f[6], f[7]);
            }
          }
        }
    }
    // (slot 1 is written again after the next run's first barrier)
  } while (wk.next(P));
}

// The end of a cluster, whose CTAs hold the stages of one pair: their states of
// a row added in order, a warp a row, from each other's shared memory.
template <typename E, bool SPLIT, int HD, int NT, int RT>
__device__ __forceinline__ void cluster_end(const Params& P, const uint8_t* smem) {
  using C = Cfg<E, SPLIT, HD, NT, RT>;
  constexpr int MAX = 8;   // CTAs
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncwarp();
  ptx::cluster_sync();
  if (warp < C::WARPS) {
    const int log2 = 31 - __clz(P.direct), pair = blockIdx.x >> log2, part = blockIdx.x & (P.direct - 1);
    const int e = pair / P.p.Hkv, h = pair - e * P.p.Hkv;
    const int b = e / P.groups, r0 = (e - b * P.groups) * C::RB, R = min(C::RB, P.p.R - r0);
    const int n = reinterpret_cast<const int*>(smem + C::OFF_MISC + 16)[2];
    // the CTAs that have stages
    const bool has = lane < P.direct && lane * n >> log2 < (lane + 1) * n >> log2;
    const unsigned written = __ballot_sync(0xffffffffu, has);
    for (int row = part + P.direct * warp; row < R; row += P.direct * C::WARPS) {
      const int in_tile = row % C::RW;
      const uint32_t at = ptx::smem_u32(smem) + C::OFF_JOIN +
                          4 * ((row / C::RW * 2 * C::RW + in_tile) * (C::LDO + 2));
      float2 ml = make_float2(-CUDART_INF_F, 0.f);
      if (has) ml = ptx::load_cluster(ptx::mapa_shared(at + 4 * C::LDO, lane));
      float2 v[MAX][HD / 64];
#pragma unroll
      for (int r = 0; r < MAX; ++r)
#pragma unroll
        for (int c = 0; c < HD / 64; ++c) {
          v[r][c] = make_float2(0.f, 0.f);
          if (written >> r & 1u) v[r][c] = ptx::load_cluster(ptx::mapa_shared(at + 4 * (64 * c + 2 * lane), r));
        }
      float mx = ml.x;
#pragma unroll
      for (int s = 1; s < MAX; s *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
      mx = __shfl_sync(0xffffffffu, mx, 0);
      const float weight = ptx::ex2(ml.x - (mx == -CUDART_INF_F ? 0.f : mx));
      float sum = 0.f;
      float2 acc[HD / 64] = {};
#pragma unroll
      for (int r = 0; r < MAX; ++r) {
        const float x = __shfl_sync(0xffffffffu, weight, r);
        sum = fmaf(x, __shfl_sync(0xffffffffu, ml.y, r), sum);
#pragma unroll
        for (int c = 0; c < HD / 64; ++c) {
          acc[c].x = fmaf(x, v[r][c].x, acc[c].x);
          acc[c].y = fmaf(x, v[r][c].y, acc[c].y);
        }
      }
      const bool none = sum == 0.f;   // no key seen (a NaN among the row's scores goes through)
      const float inv = none ? 0.f : 1.f / sum;
      const long long to = (static_cast<long long>(b) * P.p.Hkv + h) * P.p.R + r0 + row;
      if (lane == 0) P.LSE[to] = none ? -CUDART_INF_F : (mx - C::SHIFT + log2f(sum)) * 0.69314718055994530942f;
#pragma unroll
      for (int c = 0; c < HD / 64; ++c) {
        const int col = 64 * c + 2 * lane;
        if (col >= P.p.dv) continue;
        const float x = none ? 0.f : acc[c].x * inv, y = none ? 0.f : acc[c].y * inv;
        if constexpr (SPLIT)
          *reinterpret_cast<float2*>(static_cast<float*>(P.O) + to * P.p.dv + col) = make_float2(x, y);
        else
          *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(P.O) + to * P.p.dv + col) = ptx::pack_bf16(x, y);
      }
    }
  }
  __syncwarp();
  ptx::cluster_sync();   // the others have read this CTA's states
}

// (Two kernels: with the cluster's end behind a branch the loop of the other
// lost 4 to 9 % at 16 and 32 rows.)
template <typename E, bool SPLIT, int HD, int NT, int RT, bool CLUSTER>
__global__ void __launch_bounds__(Cfg<E, SPLIT, HD, NT, RT>::THREADS, Cfg<E, SPLIT, HD, NT, RT>::CTAS)
    tokens_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const __grid_constant__ Params P) {
  extern __shared__ __align__(1024) uint8_t smem[];
  attend<E, SPLIT, HD, NT, RT, CLUSTER>(tmK, tmV, P, smem);
  if constexpr (CLUSTER) cluster_end<E, SPLIT, HD, NT, RT>(P, smem);
}

template <typename E, bool SPLIT, int HD, int NT, int RT, bool CLUSTER>
cudaError_t launch_kernel(const CacheTokens& a, const Params& P) {
  using C = Cfg<E, SPLIT, HD, NT, RT>;
  static_assert(C::NST >= 2 && (C::SMEM + 1024) * C::CTAS <= 228 * 1024, "shared memory");
  auto kern = tokens_kernel<E, SPLIT, HD, NT, RT, CLUSTER>;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem(kern, C::SMEM, done);
  if (e != cudaSuccess) return e;
  return launch_clusters(kern, CLUSTER ? a.direct : 1, a.grid, C::THREADS, C::SMEM, a.stream, *a.tmK, *a.tmV, P);
}
template <typename E, bool SPLIT, int HD, int NT, int RT>
cudaError_t launch(const CacheTokens& a, Params& P) {
  if (a.direct > 1) return launch_kernel<E, SPLIT, HD, NT, RT, true>(a, P);
  const cudaError_t e = launch_kernel<E, SPLIT, HD, NT, RT, false>(a, P);
  return e != cudaSuccess ? e : cache_walk::launch_join<SPLIT>(P, a.grid, Cfg<E, SPLIT, HD, NT, RT>::RB, a.stream);
}

template <typename E, bool SPLIT, int HD>
cudaError_t rows(const CacheTokens& a, Params& P) {
  if (a.p.R <= 8) return launch<E, SPLIT, HD, 1, 1>(a, P);
  return a.p.R <= 16 ? launch<E, SPLIT, HD, 2, 1>(a, P) : launch<E, SPLIT, HD, 2, 2>(a, P);
}

}  // namespace cache_tokens

cudaError_t launch_cache_tokens(const CacheTokens& a) {
  cache_walk::Params P = cache_walk::params(a);
  using cache_tokens::rows;
  const bool narrow = a.p.d <= 64 && a.p.dv <= 64;
  if (!a.c.codes) return narrow ? rows<__nv_bfloat16, false, 64>(a, P) : rows<__nv_bfloat16, false, 128>(a, P);
  if (a.f32) return narrow ? rows<uint8_t, true, 64>(a, P) : rows<uint8_t, true, 128>(a, P);
  return narrow ? rows<uint8_t, false, 64>(a, P) : rows<uint8_t, false, 128>(a, P);
}

}  // namespace attn
