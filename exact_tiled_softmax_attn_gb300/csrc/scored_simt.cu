// fp32 scored attention on CUDA cores, forward and backward.
//
// The forward and the dQ kernel take 32 rows by 64 keys a step, the dK/dV
// kernel 64 rows by 32 keys: 128 threads, each with a 4 x 4 piece of the
// scores and 4 rows (keys) by 4 columns per 64 of the accumulators. Small
// tiles, so that problems of a thousand rows fill the GPU and several CTAs of
// an SM cover one another's loads and barriers (with 64 x 64 tiles and 256
// threads a training step of B=2 H=8 T=1000 d=64 took 440 us, one CTA per SM
// waiting for itself most of the time). Per 16 products a thread reads 8
// floats of shared memory as float4; rows of a tile lie 64 * NC + 4 floats
// apart, an odd number of float4, so the rows a warp reads at one column fall
// into different banks. Scores use two-lane FMAs over even and odd columns.
// Bound by the FMA rate and those reads. Row tiles visit only the key tiles
// their ranges' hull meets, and key tiles only the row tiles whose hull meets
// them; hulls of 32 rows: those of 128 meet more tiles where documents are
// short (B=2 H=8 Hkv=4 T=1000 d=64, documents of about 300 tokens, cap and
// bias: forward 59 in place of 71 us, dQ 80 of 88, dK/dV 101 of 110).
#include <limits.h>
#include <math_constants.h>
#include <stdint.h>

#include "ptx.cuh"
#include "scored.h"

namespace attn {
namespace scored_simt {

constexpr int NT = 128;
constexpr int BM = 32, BN = 64;     // rows and keys of a step: forward, dQ
constexpr int KM = 64, KN = 32;     // rows and keys of a step: dK/dV
constexpr int LDP = BN + 4;         // pitch of a tile of weights, 64 keys wide
constexpr int LDK = KN + 4;         // and 32 keys wide

template <int NC>
struct Pitch {
  static constexpr int v = 64 * NC + 4;
};

// ROWS rows of `d` elements from row r0 into a tile of pitch 64 * NC + 4,
// zeros past column d and outside rows [lo, hi). The copies are asynchronous
// (loaded() waits for them); 16 bytes each where rows and base allow.
template <int NC, int ROWS>
__device__ __forceinline__ void load_tile(float* s, const float* g, int r0, int lo, int hi, int d) {
  const uint32_t dst = ptx::smem_u32(s);
  if (d % 4 == 0 && reinterpret_cast<uintptr_t>(g) % 16 == 0) {
    for (int i = threadIdx.x; i < ROWS * 16 * NC; i += NT) {
      const int r = i / (16 * NC), k = 4 * (i % (16 * NC)), row = r0 + r;
      const bool in = row >= lo && row < hi && k < d;
      const float* src = g + (in ? static_cast<long long>(row) * d + k : 0);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + (r * Pitch<NC>::v + k) * 4), "l"(src),
                   "r"(in ? 16 : 0)
                   : "memory");
    }
  } else {
    for (int i = threadIdx.x; i < ROWS * 64 * NC; i += NT) {
      const int r = i / (64 * NC), k = i % (64 * NC), row = r0 + r;
      const bool in = row >= lo && row < hi && k < d;
      const float* src = g + (in ? static_cast<long long>(row) * d + k : 0);
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst + (r * Pitch<NC>::v + k) * 4), "l"(src),
                   "r"(in ? 4 : 0)
                   : "memory");
    }
  }
}
__device__ __forceinline__ void loaded() {   // every thread's copies
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
}

// x[i][j] = row (4 ty + i) of a . row (tx + TX j) of b over d columns, with
// the threads as rows of TX
template <int NC, int TX>
__device__ __forceinline__ void dot_tile(float (&x)[4][4], const float* a, const float* b, int d) {
  const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
  constexpr int P = Pitch<NC>::v;
  float2 y[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) y[i][j] = make_float2(0.f, 0.f);
  const float* ar = a + 4 * ty * P;
  const float* br = b + tx * P;
#pragma unroll 2
  for (int k = 0; k < d; k += 4) {   // (columns past d are zeros)
    float4 u[4], v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = *reinterpret_cast<const float4*>(ar + i * P + k);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const float4*>(br + TX * j * P + k);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[i][j] = ptx::ffma2(make_float2(u[i].x, u[i].y), make_float2(v[j].x, v[j].y), y[i][j]);
        y[i][j] = ptx::ffma2(make_float2(u[i].z, u[i].w), make_float2(v[j].z, v[j].w), y[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) x[i][j] = y[i][j].x + y[i][j].y;
}

template <int NC>
__device__ __forceinline__ void add_products(float (&acc)[4][4 * NC], const float (&u)[4], const float* b) {
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const float4 v = *reinterpret_cast<const float4*>(b + 64 * c);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[i][4 * c] = fmaf(u[i], v.x, acc[i][4 * c]);
      acc[i][4 * c + 1] = fmaf(u[i], v.y, acc[i][4 * c + 1]);
      acc[i][4 * c + 2] = fmaf(u[i], v.z, acc[i][4 * c + 2]);
      acc[i][4 * c + 3] = fmaf(u[i], v.w, acc[i][4 * c + 3]);
    }
  }
}

// acc[i][4 c + e] += sum_k w[4 ty + i][k] * b[k][4 tx + 64 c + e] over BN keys
template <int NC>
__device__ __forceinline__ void acc_rows(float (&acc)[4][4 * NC], const float* w, const float* b) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  constexpr int P = Pitch<NC>::v;
#pragma unroll 2
  for (int k = 0; k < BN; k += 4) {
    float4 t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = *reinterpret_cast<const float4*>(w + (4 * ty + i) * LDP + k);
    const float* row = b + k * P + 4 * tx;
    add_products<NC>(acc, {t[0].x, t[1].x, t[2].x, t[3].x}, row);
    add_products<NC>(acc, {t[0].y, t[1].y, t[2].y, t[3].y}, row + P);
    add_products<NC>(acc, {t[0].z, t[1].z, t[2].z, t[3].z}, row + 2 * P);
    add_products<NC>(acc, {t[0].w, t[1].w, t[2].w, t[3].w}, row + 3 * P);
  }
}

// acc[i][4 c + e] += sum_r w[r][4 ty + i] * b[r][4 tx + 64 c + e] over KM rows
template <int NC>
__device__ __forceinline__ void acc_cols(float (&acc)[4][4 * NC], const float* w, const float* b) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  constexpr int P = Pitch<NC>::v;
#pragma unroll 4
  for (int r = 0; r < KM; ++r) {
    const float4 t = *reinterpret_cast<const float4*>(w + r * LDK + 4 * ty);
    add_products<NC>(acc, {t.x, t.y, t.z, t.w}, b + r * P + 4 * tx);
  }
}

template <int N>
__device__ __forceinline__ void zero_row(float (&acc)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) acc[e] = 0.f;
}

template <int NC>
__device__ __forceinline__ void store_row(float* row, const float (&acc)[4 * NC], float mul, int d) {
  const int tx = threadIdx.x & 15;
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (4 * tx + 64 * c + e < d) row[4 * tx + 64 * c + e] = acc[4 * c + e] * mul;
}

// The changed score of raw product x, and its derivative by scale * x.
__device__ __forceinline__ float score(float x, const ScoredProblem& p, float slope, int pos, int key, float* grad) {
  float s = x * p.scale;
  *grad = 1.f;
  if (p.softcap > 0.f) {
    const float t = tanhf(s / p.softcap);
    s = p.softcap * t;
    *grad = 1.f - t * t;
  }
  if (p.slopes) s -= slope * fabsf(static_cast<float>(pos - key));
  return s;
}

struct RowInfo {
  int lo[4], hi[4], pos[4];
  float slope[4];
};

template <int TX>
__device__ __forceinline__ RowInfo row_info(const ScoredProblem& p, const ScoredPlan& plan, int bh, int r0) {
  RowInfo ri;
  const int b = bh / p.Hkv, kvh = bh - b * p.Hkv, ty = threadIdx.x / TX;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + 4 * ty + i;   // (rows up to rpad have entries)
    const int4 w = plan.rows[static_cast<long long>(b) * p.rpad() + r];
    ri.lo[i] = w.x, ri.hi[i] = w.y, ri.pos[i] = w.z;
    ri.slope[i] = p.slopes && r < p.R ? p.slopes[kvh * p.G + r / p.Tq] : 0.f;
  }
  return ri;
}

__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int NCK, int NCV>
__global__ void __launch_bounds__(NT) fwd_kernel(const ScoredProblem p, const ScoredPlan plan, const float* __restrict__ Q,
                                                  const float* __restrict__ K, const float* __restrict__ V,
                                                  float* __restrict__ O, float* __restrict__ LSE, int n_splits,
                                                  int split_keys, float* __restrict__ Opart,
                                                  float* __restrict__ LSEpart) {
  extern __shared__ __align__(16) float smem[];
  float* sQ = smem;
  float* sK = sQ + BM * Pitch<NCK>::v;
  float* sV = sK + BN * Pitch<NCK>::v;
  float* sP = sV + BN * Pitch<NCV>::v;
  const int nt = (p.R + BM - 1) / BM;
  const int bh = blockIdx.x / nt, split = blockIdx.y;
  const int r0 = (nt - 1 - (blockIdx.x - bh * nt)) * BM;   // causal: the longest rows first
  const int b = bh / p.Hkv;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const RowInfo ri = row_info<16>(p, plan, bh, r0);
  const int2 hull = plan.fine[static_cast<long long>(b) * (p.rpad() / 32) + r0 / BM];
  const int k_lo = max(hull.x, split * split_keys), k_hi = min(hull.y, (split + 1) * split_keys);
  load_tile<NCK, BM>(sQ, Q + static_cast<long long>(bh) * p.R * p.d, r0, 0, p.R, p.d);
  const float* Kh = K + static_cast<long long>(bh) * p.Tk * p.d;
  const float* Vh = V + static_cast<long long>(bh) * p.Tk * p.dv;
  float acc[4][4 * NCV], m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -CUDART_INF_F;
    l[i] = 0.f;
#pragma unroll
    for (int e = 0; e < 4 * NCV; ++e) acc[i][e] = 0.f;
  }
  for (int k0 = k_lo / BN * BN; k0 < k_hi; k0 += BN) {
    __syncthreads();
    load_tile<NCK, BN>(sK, Kh, k0, k_lo, k_hi, p.d);
    load_tile<NCV, BN>(sV, Vh, k0, k_lo, k_hi, p.dv);
    loaded();
    float x[4][4];
    dot_tile<NCK, 16>(x, sQ, sK, p.d);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mx = -CUDART_INF_F, g;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = k0 + tx + 16 * j;
        const float s = score(x[i][j], p, ri.slope[i], ri.pos[i], key, &g);
        x[i][j] = key >= max(ri.lo[i], k_lo) && key < min(ri.hi[i], k_hi) ? s : -CUDART_INF_F;
        mx = fmaxf(mx, x[i][j]);
      }
      const float mn = fmaxf(m[i], row_max(mx));
      const float ref = mn == -CUDART_INF_F ? 0.f : mn;   // no key seen yet: every exponential is exp(-inf)
      const float corr = expf(m[i] - ref);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = expf(x[i][j] - ref);
        sum += e;
        sP[(4 * ty + i) * LDP + tx + 16 * j] = e;
      }
      l[i] = l[i] * corr + row_sum(sum);
      m[i] = mn;
#pragma unroll
      for (int e = 0; e < 4 * NCV; ++e) acc[i][e] *= corr;
    }
    __syncthreads();
    acc_rows<NCV>(acc, sP, sV);
  }
  const long long rows = static_cast<long long>(p.B) * p.Hkv * p.R;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + 4 * ty + i;
    if (r >= p.R) continue;
    const long long row = static_cast<long long>(bh) * p.R + r;
    const bool none = l[i] == 0.f;   // no key seen (a NaN among the row's scores goes through)
    const float inv = none ? 0.f : 1.f / l[i];
    const float lse = none ? -CUDART_INF_F : m[i] + logf(l[i]);
    if (none) zero_row(acc[i]);   // (0 times what other rows see may be NaN)
    if (n_splits > 1) {
      store_row<NCV>(Opart + (split * rows + row) * p.dv, acc[i], inv, p.dv);
      if (tx == 0) LSEpart[split * rows + row] = lse;
    } else {
      store_row<NCV>(O + row * p.dv, acc[i], inv, p.dv);
      if (tx == 0) LSE[row] = lse;
    }
  }
}

// dQ of a 32-row tile, and D = rowsum(dO o O) of its rows for the dK/dV kernel.
template <int NCK, int NCV>
__global__ void __launch_bounds__(NT) dq_kernel(const ScoredProblem p, const ScoredPlan plan, const float* __restrict__ Q,
                                                 const float* __restrict__ K, const float* __restrict__ V,
                                                 const float* __restrict__ O, const float* __restrict__ LSE,
                                                 const float* __restrict__ dO, float* __restrict__ dQ,
                                                 float* __restrict__ D) {
  extern __shared__ __align__(16) float smem[];
  float* sQ = smem;
  float* sK = sQ + BM * Pitch<NCK>::v;
  float* sdO = sK + BN * Pitch<NCK>::v;
  float* sV = sdO + BM * Pitch<NCV>::v;
  float* sW = sV + BN * Pitch<NCV>::v;
  const int nt = (p.R + BM - 1) / BM;
  const int bh = blockIdx.x / nt;
  const int r0 = (nt - 1 - (blockIdx.x - bh * nt)) * BM;
  const int b = bh / p.Hkv;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const RowInfo ri = row_info<16>(p, plan, bh, r0);
  const int2 hull = plan.fine[static_cast<long long>(b) * (p.rpad() / 32) + r0 / BM];
  load_tile<NCK, BM>(sQ, Q + static_cast<long long>(bh) * p.R * p.d, r0, 0, p.R, p.d);
  load_tile<NCV, BM>(sdO, dO + static_cast<long long>(bh) * p.R * p.dv, r0, 0, p.R, p.dv);
  load_tile<NCV, BM>(sV, O + static_cast<long long>(bh) * p.R * p.dv, r0, 0, p.R, p.dv);   // O, until the loop
  loaded();
  float lse[4], dd[4], acc[4][4 * NCK];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + 4 * ty + i;
    lse[i] = r < p.R ? LSE[static_cast<long long>(bh) * p.R + r] : -CUDART_INF_F;
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < 4 * NCV; ++c)
      s = fmaf(sdO[(4 * ty + i) * Pitch<NCV>::v + tx + 16 * c], sV[(4 * ty + i) * Pitch<NCV>::v + tx + 16 * c], s);
    dd[i] = row_sum(s);
    if (tx == 0) D[static_cast<long long>(bh) * p.rpad() + r] = dd[i];
#pragma unroll
    for (int e = 0; e < 4 * NCK; ++e) acc[i][e] = 0.f;
  }
  const float* Kh = K + static_cast<long long>(bh) * p.Tk * p.d;
  const float* Vh = V + static_cast<long long>(bh) * p.Tk * p.dv;
  for (int k0 = hull.x / BN * BN; k0 < hull.y; k0 += BN) {
    __syncthreads();
    load_tile<NCK, BN>(sK, Kh, k0, hull.x, hull.y, p.d);
    load_tile<NCV, BN>(sV, Vh, k0, hull.x, hull.y, p.dv);
    loaded();
    float x[4][4], y[4][4];
    dot_tile<NCK, 16>(x, sQ, sK, p.d);
    dot_tile<NCV, 16>(y, sdO, sV, p.dv);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = k0 + tx + 16 * j;
        float g;
        const float s = score(x[i][j], p, ri.slope[i], ri.pos[i], key, &g);
        const bool in = key >= ri.lo[i] && key < ri.hi[i];
        sW[(4 * ty + i) * LDP + tx + 16 * j] = in ? expf(s - lse[i]) * (y[i][j] - dd[i]) * g : 0.f;
      }
    __syncthreads();
    acc_rows<NCK>(acc, sW, sK);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + 4 * ty + i;
    if (ri.hi[i] == 0) zero_row(acc[i]);   // (as in the forward)
    if (r < p.R)
      store_row<NCK>(dQ + (static_cast<long long>(bh) * p.R + r) * p.d, acc[i], p.scale, p.d);
  }
}

template <int NCK, int NCV>
__global__ void __launch_bounds__(NT) dkdv_kernel(const ScoredProblem p, const ScoredPlan plan,
                                                   const float* __restrict__ Q, const float* __restrict__ K,
                                                   const float* __restrict__ V, const float* __restrict__ LSE,
                                                   const float* __restrict__ dO, const float* __restrict__ D,
                                                   float* __restrict__ dK, float* __restrict__ dV) {
  // (dK and dV: those of the parts where there are several)
  extern __shared__ __align__(16) float smem[];
  float* sQ = smem;
  float* sK = sQ + KM * Pitch<NCK>::v;
  float* sdO = sK + KN * Pitch<NCK>::v;
  float* sV = sdO + KM * Pitch<NCV>::v;
  float* sP = sV + KN * Pitch<NCV>::v;
  float* sW = sP + KM * LDK;
  const int nt = (p.Tk + KN - 1) / KN;
  const int bh = blockIdx.x / nt, k0 = (blockIdx.x - bh * nt) * KN;
  const int b = bh / p.Hkv;
  const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3;     // scores: rows 4 ty + i, keys tx + 8 j
  const int ky = threadIdx.x >> 4;                            // accumulators: keys 4 ky + i
  load_tile<NCK, KN>(sK, K + static_cast<long long>(bh) * p.Tk * p.d, k0, 0, p.Tk, p.d);
  load_tile<NCV, KN>(sV, V + static_cast<long long>(bh) * p.Tk * p.dv, k0, 0, p.Tk, p.dv);
  float ak[4][4 * NCK], av[4][4 * NCV];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int e = 0; e < 4 * NCK; ++e) ak[i][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 4 * NCV; ++e) av[i][e] = 0.f;
  }
  const int4 hull = plan.khull[static_cast<long long>(b) * p.n_kt + k0 / kScoredTile];
  const uint32_t* list = plan.kbits + (static_cast<long long>(b) * p.n_kt + k0 / kScoredTile) * p.n_words();
  const int rows = p.kv_split_tiles * kScoredTile, part = blockIdx.y;
  for (int r0 = part * rows; r0 < min(p.R, (part + 1) * rows); r0 += KM) {
    const int rt = r0 / kScoredTile;
    if (!(list[rt / 32] >> (rt % 32) & 1u)) continue;
    const int2* fine = plan.fine + static_cast<long long>(b) * (p.rpad() / 32) + r0 / 32;
    const int2 u = fine[0], v = fine[1];
    if ((u.x >= k0 + KN || u.y <= k0) && (v.x >= k0 + KN || v.y <= k0)) continue;
    const bool blank = plan.tiles[static_cast<long long>(b) * p.n_rt + rt].z == INT_MAX;
    __syncthreads();
    load_tile<NCK, KM>(sQ, Q + static_cast<long long>(bh) * p.R * p.d, r0, 0, p.R, p.d);
    load_tile<NCV, KM>(sdO, dO + static_cast<long long>(bh) * p.R * p.dv, r0, 0, p.R, p.dv);
    const RowInfo ri = row_info<8>(p, plan, bh, r0);
    float lse[4], dd[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + 4 * ty + i;
      lse[i] = r < p.R ? LSE[static_cast<long long>(bh) * p.R + r] : 0.f;
      dd[i] = D[static_cast<long long>(bh) * p.rpad() + r];
    }
    loaded();
    if (blank) {   // some row of the 128 sees no key: it may hold anything, and its weights of 0 must stay 0
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (ri.hi[i] > 0) continue;
        for (int c = tx; c < Pitch<NCK>::v; c += 8) sQ[(4 * ty + i) * Pitch<NCK>::v + c] = 0.f;
        for (int c = tx; c < Pitch<NCV>::v; c += 8) sdO[(4 * ty + i) * Pitch<NCV>::v + c] = 0.f;
      }
      __syncthreads();
    }
    float x[4][4], y[4][4];
    dot_tile<NCK, 8>(x, sQ, sK, p.d);
    dot_tile<NCV, 8>(y, sdO, sV, p.dv);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = k0 + tx + 8 * j;
        float g;
        const float s = score(x[i][j], p, ri.slope[i], ri.pos[i], key, &g);
        const bool in = key >= ri.lo[i] && key < ri.hi[i];
        const float e = in ? expf(s - lse[i]) : 0.f;
        sP[(4 * ty + i) * LDK + tx + 8 * j] = e;
        sW[(4 * ty + i) * LDK + tx + 8 * j] = in ? e * (y[i][j] - dd[i]) * g : 0.f;
      }
    __syncthreads();
    acc_cols<NCV>(av, sP, sdO);
    acc_cols<NCK>(ak, sW, sQ);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int key = k0 + 4 * ky + i;
    if (key < hull.x || key >= hull.y) {   // seen by no row
      zero_row(ak[i]);
      zero_row(av[i]);
    }
    if (key < p.Tk) {
      const long long at = (static_cast<long long>(part) * p.B * p.Hkv + bh) * p.Tk + key;
      store_row<NCK>(dK + at * p.d, ak[i], p.scale, p.d);
      store_row<NCV>(dV + at * p.dv, av[i], 1.f, p.dv);
    }
  }
}

template <int NCK, int NCV>
cudaError_t fwd(const ScoredFwd& a) {
  const ScoredProblem& p = a.p;
  const int smem = (BM * Pitch<NCK>::v + BN * Pitch<NCK>::v + BN * Pitch<NCV>::v + BM * LDP) * 4;
  auto kern = fwd_kernel<NCK, NCV>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((p.R + BM - 1) / BM * p.B * p.Hkv, a.n_splits);
  kern<<<grid, NT, smem, a.stream>>>(p, a.plan, static_cast<const float*>(a.Q), static_cast<const float*>(a.K),
                                     static_cast<const float*>(a.V), static_cast<float*>(a.O), a.LSE, a.n_splits,
                                     a.split_keys, a.Opart, a.LSEpart);
  return cudaGetLastError();
}

template <int NCK, int NCV>
cudaError_t bwd(const ScoredBwd& a) {
  const ScoredProblem& p = a.p;
  const int smem_q = ((BM + BN) * (Pitch<NCK>::v + Pitch<NCV>::v) + BM * LDP) * 4;
  const int smem_kv = ((KM + KN) * (Pitch<NCK>::v + Pitch<NCV>::v) + 2 * KM * LDK) * 4;
  auto kq = dq_kernel<NCK, NCV>;
  auto kk = dkdv_kernel<NCK, NCV>;
  cudaError_t e = cudaFuncSetAttribute(kq, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_q);
  if (e != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(kk, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_kv)) != cudaSuccess) return e;
  const float *Q = static_cast<const float*>(a.Q), *K = static_cast<const float*>(a.K), *V = static_cast<const float*>(a.V),
          *dO = static_cast<const float*>(a.dO);
  kq<<<(p.R + BM - 1) / BM * p.B * p.Hkv, NT, smem_q, a.stream>>>(p, a.plan, Q, K, V, static_cast<const float*>(a.O),
                                                                        a.LSE, dO, static_cast<float*>(a.dQ), a.D);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const bool parts = p.kv_splits > 1;
  kk<<<dim3((p.Tk + KN - 1) / KN * p.B * p.Hkv, p.kv_splits), NT, smem_kv, a.stream>>>(
      p, a.plan, Q, K, V, a.LSE, dO, a.D, parts ? a.dKpart : static_cast<float*>(a.dK),
      parts ? a.dVpart : static_cast<float*>(a.dV));
  return cudaGetLastError();
}

cudaError_t fwd_any(const ScoredFwd& a) {
  if (a.p.d <= 64) return a.p.dv <= 64 ? fwd<1, 1>(a) : fwd<1, 2>(a);
  return a.p.dv <= 64 ? fwd<2, 1>(a) : fwd<2, 2>(a);
}
cudaError_t bwd_any(const ScoredBwd& a) {
  if (a.p.d <= 64) return a.p.dv <= 64 ? bwd<1, 1>(a) : bwd<1, 2>(a);
  return a.p.dv <= 64 ? bwd<2, 1>(a) : bwd<2, 2>(a);
}

}  // namespace scored_simt

cudaError_t launch_scored_fwd_simt(const ScoredFwd& a) { return scored_simt::fwd_any(a); }
cudaError_t launch_scored_bwd_simt(const ScoredBwd& a) { return scored_simt::bwd_any(a); }

}  // namespace attn
