// bf16 scored attention of few query rows (single tokens) against a long
// cache (d, dv <= 128, at most 32 packed rows per key head).
//
// Reads every seen key and value once: bound by memory. The keys that the
// rows of a (batch entry, key head) see - the hull of their ranges - are cut
// into stages of 64; all stages of the launch form one list, of which every
// CTA takes an equal contiguous share, so sequences of any lengths load the
// SMs evenly. A CTA that holds all stages of a pair writes its rows' results;
// the others leave partial results, which a second kernel joins in order.
// The hulls are formed from the ranges in the kernel: there is no plan
// launch before it.
//
// A producer warp fills a ring of stages by TMA (128-byte swizzle); 4 warps
// per 16-row tile each take 16 of a stage's 64 keys and keep a running
// maximum, sum and accumulator of their own, joined at the end of the pair.
// The products run on mma.m16n8k16: with 16 rows or fewer per key head the
// tcgen05 tile of 128 rows would be mostly empty, and at this intensity (at
// most 32 rows) the memory is what counts: 32 sequences of 32768 keys, H=32
// Hkv=8 d=128, 2.6 GB, 357 us or 7.2 TB/s; 87 us of 79 with 16 rows at B=8
// Hkv=8 Tk=16384. Four row tiles of 16 were tried too: 338 us there with 64
// rows, where the 128-row tiles take 112. Fragments are read as 16-byte
// vectors: the columns of Q and K are permuted alike, so that a thread's
// fragments of K are 8 adjacent elements of a row; keys are numbered so that
// the accumulator layout of S is the operand layout of P, and V's pairs are
// formed from the rows of two keys by byte permutes. Within a 16-key group
// fragment column g stands for key g (g even) or g ^ 4 (g odd): the eight
// threads of one shared-memory phase then touch eight different 16-byte
// columns in both reads.
#include <cuda.h>
#include <cuda_bf16.h>
#include <math_constants.h>
#include <stdint.h>

#include "common.cuh"
#include "ptx.cuh"
#include "scored.h"
#include "scored_math.cuh"

namespace attn {
namespace scored_tokens {

using scored::Cap;

constexpr int BK = 64;              // keys per stage
constexpr int BOX = BK * 64 * 2;    // one TMA box: 64 rows x 64 columns
constexpr float TAU = 8.0f;

struct Params {
  ScoredProblem p;
  ScoredMask mask;
  const __nv_bfloat16* Q;
  __nv_bfloat16* O;
  float* LSE;
  int* start;       // [B + 1]: stages before a batch entry's first pair (written for the second kernel)
  float* Opart;     // [grid][2][R][dv]: a CTA's first and last pair where they go on in another CTA
  float* LSEpart;   // [grid][2][R]
  uint32_t* status;
  float sc2;
  Cap cap;
};

template <int HD, int RT>
struct Cfg {
  static constexpr int KB = HD / 64;
  static constexpr int STAGE = 2 * KB * BOX;
  static constexpr int WARPS = 4 * RT;            // compute warps
  static constexpr int THREADS = 32 * (WARPS + 1);
  static constexpr int CTAS = RT == 1 ? 2 : 1;    // per SM
  static constexpr int LDO = HD + 4;
  static constexpr int JOIN = RT * 2 * 16 * (LDO + 2) * 4;   // rows, maxima and sums of two key groups
  static constexpr int BUDGET = (RT == 1 ? 112 : 226) * 1024 - JOIN - 1024;
  static constexpr int NST = BUDGET / STAGE < 8 ? BUDGET / STAGE : 8;
  static constexpr int OFF_JOIN = NST * STAGE;
  static constexpr int OFF_BAR = OFF_JOIN + JOIN;
  static constexpr int OFF_MISC = OFF_BAR + 2 * NST * 8;
  static constexpr int OFF_HULL = OFF_MISC + 64 + 128;   // after the scan: [THREADS] hulls
  static constexpr int SMEM = OFF_HULL + 8 * THREADS;
};

// Hull of the ranges of batch entry b's tokens: [lo, hi), (0, 0) when no
// token sees a key. By one thread.
__device__ __forceinline__ int2 hull_of(const Params& P, int b) {
  int lo = 0x7fffffff, hi = 0;
  for (int t = 0; t < P.p.Tq; ++t) {
    int pos, a, z;
    scored::row_range(P.p, P.mask, b, t, &a, &z, &pos);
    if (a < z) {
      lo = min(lo, a);
      hi = max(hi, z);
    }
  }
  return hi > 0 ? make_int2(lo, hi) : make_int2(0, 0);
}
__device__ __forceinline__ int stages_of(int2 hull) { return (hull.y - hull.x + BK - 1) / BK; }

// The runs of stages a CTA works through, one pair (batch entry, key head)
// after another. Every warp walks them itself. `hulls`: those of all batch
// entries in shared memory, or null where there are more than threads.
struct Walk {
  const int2* hulls;
  int b, h, n;        // the pair, and the stages of each pair of b
  int s0, run;        // this run: stages [s0, s0 + run) of the pair
  int2 hull;
  int left;           // stages after this run

  __device__ __forceinline__ int2 hull_at(const Params& P, int e) const { return hulls ? hulls[e] : hull_of(P, e); }
  __device__ __forceinline__ void begin(const Params& P, const int2* all, int b0, int off, int count) {
    hulls = all;
    b = b0;
    hull = hull_at(P, b);
    n = stages_of(hull);
    h = off / n;
    s0 = off - h * n;
    run = min(n - s0, count);
    left = count - run;
  }
  __device__ __forceinline__ bool next(const Params& P) {
    if (left == 0) return false;
    if (++h == P.p.Hkv) {
      h = 0;
      do {   // entries without a key have no stages
        ++b;
        hull = hull_at(P, b);
      } while (hull.y == 0);
      n = stages_of(hull);
    }
    s0 = 0;
    run = min(n, left);
    left -= run;
    return true;
  }
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }

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

template <int HD, int RT>
__global__ void __launch_bounds__(Cfg<HD, RT>::THREADS, Cfg<HD, RT>::CTAS)
    tokens_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const __grid_constant__ Params P) {
  using C = Cfg<HD, RT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if ((ptx::smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicOr(P.status, ATTN_DEV_BAD_SMEM);
    return;
  }
  float* join = reinterpret_cast<float*>(smem + C::OFF_JOIN);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + C::NST;
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC);
  int* found = reinterpret_cast<int*>(smem + C::OFF_MISC + 16);   // {b, offset, count}
  int* scan = reinterpret_cast<int*>(smem + C::OFF_MISC + 64);
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NST; ++s) {
      ptx::mbar_init(full + s, 1);
      ptx::mbar_init(empty + s, C::WARPS);
    }
    *abort_flag = 0u;
    ptx::fence_mbar_init();
    ptx::tma_prefetch_desc(&tmK);
    ptx::tma_prefetch_desc(&tmV);
  }
  // This CTA's share of the launch's stages: every thread counts the stages
  // of a run of batch entries.
  const int B = P.p.B;
  const int per = (B + C::THREADS - 1) / C::THREADS;
  const int b_lo = min(B, static_cast<int>(threadIdx.x) * per), b_hi = min(B, b_lo + per);
  int2* hulls = reinterpret_cast<int2*>(smem + C::OFF_HULL);
  const bool one = per == 1;   // an entry per thread: its hull is kept
  int mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const int2 hull = hull_of(P, b);
    if (one) hulls[b] = hull;
    mine += stages_of(hull) * P.p.Hkv;
  }
  int before = mine;   // inclusive scan over the warp, then over the warps
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  if (lane == 31) scan[warp] = before;
  __syncthreads();
  int total = 0, base = 0;
  for (int i = 0; i < C::WARPS + 1; ++i) {
    if (i < warp) base += scan[i];
    total += scan[i];
  }
  before += base - mine;   // exclusive
  const long long grid = gridDim.x, cta = blockIdx.x;
  const int first = static_cast<int>(cta * total / grid), last = static_cast<int>((cta + 1) * total / grid);
  if (before <= first && first < before + mine) {
    int at = before, b = b_lo;
    for (; !one; ++b) {
      const int n = stages_of(hull_of(P, b)) * P.p.Hkv;
      if (first < at + n) break;
      at += n;
    }
    found[0] = b;
    found[1] = first - at;
  }
  if (blockIdx.x == 0) {
    int at = before;
    for (int b = b_lo; b < b_hi; ++b) {
      P.start[b] = at;
      if (!one) at += stages_of(hull_of(P, b)) * P.p.Hkv;
    }
    if (threadIdx.x == 0) P.start[B] = total;
  }
  __syncthreads();
  if (last <= first) return;
  Walk wk;
  wk.begin(P, one ? hulls : nullptr, found[0], found[1], last - first);

  if (warp == C::WARPS) {
    // ------------------------------------------------------------ producer
    ptx::WaitCtx w{abort_flag, P.status, 1u};
    bool ok = true;
    uint32_t it = 0;
    do {
      const int bh = wk.b * P.p.Hkv + wk.h;
      if (lane == 0) {
        for (int s = wk.s0; ok && s < wk.s0 + wk.run; ++s, ++it) {
          const int st = it % C::NST;
          if (!(ok = ptx::mbar_wait(empty + st, ((it / C::NST) & 1u) ^ 1u, w))) break;
          ptx::mbar_arrive_expect_tx(full + st, C::STAGE);
          uint8_t* dst = smem + st * C::STAGE;
          for (int c = 0; c < C::KB; ++c)
            ptx::tma_load_3d(dst + c * BOX, &tmK, full + st, c * 64, wk.hull.x + s * BK, bh);
          for (int c = 0; c < C::KB; ++c)
            ptx::tma_load_3d(dst + (C::KB + c) * BOX, &tmV, full + st, c * 64, wk.hull.x + s * BK, bh);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
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
  const int R = P.p.R, Tq = P.p.Tq, d = P.p.d, dv = P.p.dv;
  const int krow = (g & 1) ? g ^ 4 : g;                 // key of fragment column g within 8
  const int k_lo = 2 * t, k_hi = (2 * t + 1) ^ 4;       // keys of accumulator columns 2t, 2t + 1 within 8
  const int row[2] = {16 * rt + g, 16 * rt + g + 8};
  uint32_t it = 0;
  bool ok = true;
  uint4 q[2][HD / 32];      // rows g and g + 8, elements 32 c + 8 t .. + 7
  float o[HD / 8][4];
  do {
    const int bh = wk.b * P.p.Hkv + wk.h;
    int lo[2], hi[2], pos[2];
    float slope2[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      lo[i] = 0x7fffffff, hi[i] = 0, pos[i] = 0;
      if (row[i] < R) {
        scored::row_range(P.p, P.mask, wk.b, row[i] % Tq, &lo[i], &hi[i], &pos[i]);
        if (P.p.slopes) slope2[i] = __ldg(P.p.slopes + wk.h * P.p.G + row[i] / Tq) * scored::kLog2e;
      }
#pragma unroll
      for (int c = 0; c < HD / 32; ++c) {
        const int col = 32 * c + 8 * t;
        q[i][c] = row[i] < R && col < d
                      ? __ldg(reinterpret_cast<const uint4*>(P.Q + (static_cast<long long>(bh) * R + row[i]) * d + col))
                      : make_uint4(0u, 0u, 0u, 0u);
      }
    }
    float m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < HD / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

    for (int s = wk.s0; s < wk.s0 + wk.run; ++s, ++it) {
      const int st = it % C::NST;
      if (!(ok = __all_sync(0xffffffffu, ptx::mbar_wait(full + st, (it / C::NST) & 1u, w)))) break;
      const int key0 = wk.hull.x + s * BK + 16 * kg;   // of this warp's 16
      if (key0 < wk.hull.y) {
        const uint8_t* sK = smem + st * C::STAGE + 16 * kg * 128;
        const uint8_t* sV = sK + C::KB * BOX;
        float x[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int c = 0; c < HD / 32; ++c) {
          const uint8_t* p = sK + (c >> 1) * BOX + (((4 * (c & 1) + t) ^ krow) << 4) + krow * 128;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint4 k = lds(p + i * 1024);
            mma16816(x[i], q[0][c].x, q[1][c].x, q[0][c].y, q[1][c].y, k.x, k.y);
            mma16816(x[i], q[0][c].z, q[1][c].z, q[0][c].w, q[1][c].w, k.z, k.w);
          }
        }
        // changed and masked scores, in log2 units; x[i][2 r + e] is row g + 8 r, key 8 i + (e ? k_hi : k_lo)
        if (P.p.softcap > 0.f) {   // the cap's form by the warp's scores; degree 4 holds where degree 2 does
          float top = 0.f;
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(x[i][e]));
          if (__all_sync(0xffffffffu, !(top > P.cap.limit4))) {
            const scored::CapPoly<scored::kCapPoly4> poly(P.cap);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < 4; e += 2) {
                const scored::F2 v = scored::f2(x[i][e], x[i][e + 1]), y = scored::mul2(v, poly(v));
                x[i][e] = y.x, x[i][e + 1] = y.y;
              }
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) x[i][e] = scored::cap_any(x[i][e], P.cap);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[i][e] *= P.sc2;
        }
        float mx[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = e >> 1, key = key0 + 8 * i + ((e & 1) ? k_hi : k_lo);
            const float y = fmaf(-slope2[r], fabsf(static_cast<float>(key - pos[r])), x[i][e]);
            x[i][e] = key >= lo[r] && key < hi[r] ? y : -CUDART_INF_F;
            mx[r] = fmaxf(mx[r], x[i][e]);
          }
        bool need = false;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
          mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
          need = need || mx[r] > m[r] + TAU;   // (from -inf: any score)
        }
        if (__any_sync(0xffffffffu, need)) {
          // the running references move to the maxima
          float corr[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float mn = fmaxf(m[r], mx[r]);
            corr[r] = m[r] == mn ? 1.f : ptx::ex2(m[r] - mn);
            m[r] = mn;
            l[r] *= corr[r];
          }
#pragma unroll
          for (int i = 0; i < HD / 8; ++i) {
            o[i][0] *= corr[0], o[i][1] *= corr[0];
            o[i][2] *= corr[1], o[i][3] *= corr[1];
          }
        }
        const float ref[2] = {m[0] == -CUDART_INF_F ? 0.f : m[0], m[1] == -CUDART_INF_F ? 0.f : m[1]};
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[i][e] = ptx::ex2(x[i][e] - ref[e >> 1]);
            l[e >> 1] += x[i][e];
          }
        const uint32_t a0 = ptx::pack_bf16(x[0][0], x[0][1]), a1 = ptx::pack_bf16(x[0][2], x[0][3]);
        const uint32_t a2 = ptx::pack_bf16(x[1][0], x[1][1]), a3 = ptx::pack_bf16(x[1][2], x[1][3]);
        // rows of V behind the hull may hold anything: P is 0 there, 0 * NaN is not
        const bool tail = key0 + 16 > wk.hull.y;
#pragma unroll
        for (int c = 0; c < C::KB; ++c) {
          uint4 v[4];   // keys k_lo, k_hi, 8 + k_lo, 8 + k_hi; elements 64 c + 8 g .. + 7
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int kr = (i & 1) ? k_hi : k_lo;
            v[i] = lds(sV + c * BOX + ((i >> 1) * 8 + kr) * 128 + ((g ^ kr) << 4));
            if (tail && key0 + (i >> 1) * 8 + kr >= wk.hull.y) v[i] = make_uint4(0u, 0u, 0u, 0u);
          }
          const uint32_t* v0 = reinterpret_cast<const uint32_t*>(&v[0]);
          const uint32_t* v1 = reinterpret_cast<const uint32_t*>(&v[1]);
          const uint32_t* v2 = reinterpret_cast<const uint32_t*>(&v[2]);
          const uint32_t* v3 = reinterpret_cast<const uint32_t*>(&v[3]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {   // column g of tile i: element 64 c + 8 g + i
            const uint32_t sel = (i & 1) ? 0x7632u : 0x5410u;
            mma16816(o[8 * c + i], a0, a1, a2, a3, __byte_perm(v0[i >> 1], v1[i >> 1], sel),
                     __byte_perm(v2[i >> 1], v3[i >> 1], sel));
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
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    }
    auto put = [&](int slot) {   // this warp's state into slot 0 or 1 of its row tile
      float* dst = join + (rt * 2 + slot) * 16 * (C::LDO + 2);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float* p = dst + (g + 8 * r) * (C::LDO + 2);
#pragma unroll
        for (int i = 0; i < HD / 8; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) p[(i >> 3) * 64 + 16 * t + 8 * e + (i & 7)] = o[i][2 * r + e];
        if (t == 0) {
          p[C::LDO] = m[r];
          p[C::LDO + 1] = l[r];
        }
      }
    };
    auto take = [&](int slot) {   // adds a slot's state to this warp's
      const float* src = join + (rt * 2 + slot) * 16 * (C::LDO + 2);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float* p = src + (g + 8 * r) * (C::LDO + 2);
        const float m2 = p[C::LDO], mn = fmaxf(m[r], m2);
        const float ref = mn == -CUDART_INF_F ? 0.f : mn;
        const float wa = ptx::ex2(m[r] - ref), wb = ptx::ex2(m2 - ref);
        m[r] = mn;
        l[r] = l[r] * wa + p[C::LDO + 1] * wb;
#pragma unroll
        for (int i = 0; i < HD / 8; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            o[i][2 * r + e] = o[i][2 * r + e] * wa + p[(i >> 3) * 64 + 16 * t + 8 * e + (i & 7)] * wb;
      }
    };
    if (kg >= 2) put(kg - 2);
    compute_barrier<C::WARPS * 32>();
    if (kg < 2) take(kg);
    if (kg == 1) put(1);   // (only this warp read slot 1)
    compute_barrier<C::WARPS * 32>();
    if (kg == 0) {
      take(1);
      const bool whole = wk.run == wk.n;
      const int part = wk.s0 > 0 ? 0 : 1;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (row[r] >= R) continue;
        const bool none = l[r] == 0.f;   // no key seen (a NaN among the row's scores goes through)
        const float inv = 1.f / l[r];
        const float lse = none ? -CUDART_INF_F : (m[r] + log2f(l[r])) * 0.69314718055994530942f;
        const long long at = whole ? static_cast<long long>(bh) * R + row[r]
                                   : (static_cast<long long>(blockIdx.x) * 2 + part) * R + row[r];
        if (t == 0) (whole ? P.LSE : P.LSEpart)[at] = lse;
#pragma unroll
        for (int c = 0; c < C::KB; ++c)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int col = 64 * c + 16 * t + 8 * e;
            if (col >= dv) continue;
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = none ? 0.f : o[8 * c + i][2 * r + e] * inv;
            if (whole) {
              *reinterpret_cast<uint4*>(P.O + at * dv + col) =
                  make_uint4(ptx::pack_bf16(f[0], f[1]), ptx::pack_bf16(f[2], f[3]), ptx::pack_bf16(f[4], f[5]),
                             ptx::pack_bf16(f[6], f[7]));
            } else {
              float4* dst = reinterpret_cast<float4*>(P.Opart + at * dv + col);
              dst[0] = make_float4(f[0], f[1], f[2], f[3]);
              dst[1] = make_float4(f[4], f[5], f[6], f[7]);
            }
          }
      }
    }
    // (slot 1 is written again after the next run's first barrier)
  } while (wk.next(P));
}

// Rows whose pair is spread over several CTAs: their partial results joined
// in a fixed order. Rows of pairs without a key: zeros. WPR warps per row,
// warp w of them adding parts w, w + WPR, ... (a float4 of the row per lane):
// eight for rows of many parts, whose loads would otherwise wait for one
// another (38 parts with one warp: 29 us, three times the main kernel), one
// for many rows of few parts. The launch overlaps the main kernel's end.
constexpr int JOIN_THREADS = 256, JOIN_WARPS = JOIN_THREADS / 32;
constexpr int MAX_GRID = 304;   // CTAs of the main kernel

template <int WPR>
__global__ void __launch_bounds__(JOIN_THREADS) join_kernel(const __grid_constant__ Params P, int grid) {
  constexpr int ROWS = JOIN_WARPS / WPR;   // of a block
  __shared__ float red[JOIN_WARPS];
  __shared__ float4 part[WPR > 1 ? JOIN_WARPS : 1][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int own = warp / WPR, w = warp - own * WPR;   // row of the block, and warp of the row
  const int R = P.p.R, dv = P.p.dv;
  const long long n = static_cast<long long>(blockIdx.x) * ROWS + own;
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the main kernel's results
  int c0 = 0, c1 = -1, r = 0;
  long long tot = 1;
  const long long g = grid;
  auto begin = [&](int c) { return static_cast<int>(c * tot / g); };   // CTA c's first stage
  if (n < static_cast<long long>(P.p.B) * P.p.Hkv * R) {
    const int bh = static_cast<int>(n / R);
    r = static_cast<int>(n - static_cast<long long>(bh) * R);
    const int b = bh / P.p.Hkv, h = bh - b * P.p.Hkv;
    tot = P.start[P.p.B];
    const int s0 = P.start[b], stages = (P.start[b + 1] - s0) / P.p.Hkv;
    if (stages == 0) {
      if (w == 0) {
        for (int c = lane; c < dv; c += 32) P.O[n * dv + c] = __float2bfloat16_rn(0.f);
        if (lane == 0) P.LSE[n] = -CUDART_INF_F;
      }
    } else {
      auto cta_of = [&](int x) {   // the largest c with begin(c) <= x
        int c = static_cast<int>(x * g / tot);
        while (c + 1 < grid && begin(c + 1) <= x) ++c;
        return c;
      };
      c0 = cta_of(s0 + h * stages);
      c1 = cta_of(s0 + (h + 1) * stages - 1);
    }
  }
  const int parts = c1 > c0 ? c1 - c0 + 1 : 0;   // (one CTA: written by it)
  // the pair starts in c0 (its last part) and goes on in the others (their first part)
  auto at = [&](int i) { return ((c0 + i) * 2LL + (i == 0 ? 1 : 0)) * R + r; };
  auto lse_of = [&](int i) {   // a CTA without stages wrote nothing
    return begin(c0 + i) < begin(c0 + i + 1) ? P.LSEpart[at(i)] : -CUDART_INF_F;
  };
  float mx = -CUDART_INF_F;   // every warp of a row forms it
  for (int i = lane; i < parts; i += 32) mx = fmaxf(mx, lse_of(i));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float ref = mx == -CUDART_INF_F ? 0.f : mx;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  const int col = 4 * lane;
  for (int i0 = w; i0 < parts; i0 += 32 * WPR) {   // lane k: the weight of part i0 + k WPR
    const int mine = i0 + lane * WPR;
    const float lse = mine < parts ? lse_of(mine) : -CUDART_INF_F;
    const float weight = expf(lse - ref);
    // parts whose CTA wrote them; the weight of one may underflow, and a NaN in it still shows
    const unsigned written = __ballot_sync(0xffffffffu, lse != -CUDART_INF_F);
    const int count = min(32, (parts - i0 + WPR - 1) / WPR);
#pragma unroll 4
    for (int k = 0; k < count; ++k) {
      const float x = __shfl_sync(0xffffffffu, weight, k);
      if ((written >> k & 1u) && col < dv) {
        const float4 v = *reinterpret_cast<const float4*>(P.Opart + at(i0 + k * WPR) * dv + col);
        acc.x = fmaf(x, v.x, acc.x);
        acc.y = fmaf(x, v.y, acc.y);
        acc.z = fmaf(x, v.z, acc.z);
        acc.w = fmaf(x, v.w, acc.w);
      }
      sum += x;
    }
  }
  if constexpr (WPR > 1) {
    part[warp][lane] = acc;
    if (lane == 0) red[warp] = sum;
    __syncthreads();
    if (w > 0) return;
#pragma unroll
    for (int i = 1; i < WPR; ++i) {
      const float4 v = part[warp + i][lane];
      acc.x += v.x;
      acc.y += v.y;
      acc.z += v.z;
      acc.w += v.w;
      sum += red[warp + i];
    }
  }
  if (parts == 0) return;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if (col < dv)
    *reinterpret_cast<uint2*>(P.O + n * dv + col) =
        make_uint2(ptx::pack_bf16(acc.x * inv, acc.y * inv), ptx::pack_bf16(acc.z * inv, acc.w * inv));
  if (lane == 0) P.LSE[n] = sum == 0.f ? -CUDART_INF_F : ref + logf(sum);
}

template <int HD, int RT>
cudaError_t launch(const ScoredFwd& a) {
  using C = Cfg<HD, RT>;
  static_assert(C::NST >= 2 && C::SMEM <= 227 * 1024, "shared memory");
  if (a.grid > MAX_GRID) return cudaErrorInvalidValue;
  Params P;
  P.p = a.p;
  P.mask = a.mask;
  P.Q = static_cast<const __nv_bfloat16*>(a.Q);
  P.O = static_cast<__nv_bfloat16*>(a.O);
  P.LSE = a.LSE;
  P.start = a.start;
  P.Opart = a.Opart;
  P.LSEpart = a.LSEpart;
  P.status = a.status;
  P.sc2 = a.p.scale * scored::kLog2e;
  P.cap = scored::make_cap(a.p.scale, a.p.softcap);
  auto kern = tokens_kernel<HD, RT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  kern<<<a.grid, C::THREADS, C::SMEM, a.stream>>>(*a.tmK, *a.tmV, P);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // (rows fit int: the host checks)
  const int rows = a.p.B * a.p.Hkv * a.p.R;
  const bool few = a.grid <= 8 * a.p.B * a.p.Hkv;   // parts of a row, on average
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = few ? (rows + JOIN_WARPS - 1) / JOIN_WARPS : rows;
  cfg.blockDim = JOIN_THREADS;
  cfg.stream = a.stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few ? join_kernel<1> : join_kernel<JOIN_WARPS>, P, a.grid);
}

template <int HD>
cudaError_t rows(const ScoredFwd& a) {
  if (a.p.R <= 16) return launch<HD, 1>(a);
  return launch<HD, 2>(a);
}

}  // namespace scored_tokens

cudaError_t launch_scored_tokens_bf16(const ScoredFwd& a) {
  return a.p.d <= 64 && a.p.dv <= 64 ? scored_tokens::rows<64>(a) : scored_tokens::rows<128>(a);
}

}  // namespace attn
