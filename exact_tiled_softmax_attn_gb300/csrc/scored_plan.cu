// Plan of a scored-attention call: the key range of every packed query row,
// the hull of the ranges of each 128-row tile, and the row tiles that each
// 128-key tile meets. Also the sums of partial results.
#include <cuda_bf16.h>
#include <limits.h>
#include <math_constants.h>

#include "scored.h"
#include "scored_math.cuh"

namespace attn {
namespace scored {

// bf16 elements [first, first + n) of x, multiples of 8, by the block.
__device__ __forceinline__ void zero_rows(void* x, long long first, int n) {
  uint4* p = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(x) + first);
  for (int i = threadIdx.x; i < n / 8; i += blockDim.x) p[i] = make_uint4(0u, 0u, 0u, 0u);
}

// One block per (row tile, batch entry), one thread per row.
__global__ void __launch_bounds__(kScoredTile) plan_rows_kernel(const ScoredProblem p, const ScoredMask m,
                                                                 const ScoredPlan out, const ScoredIdle idle) {
  const int b = blockIdx.x / p.n_rt, tile = blockIdx.x - b * p.n_rt;
  const int row = tile * kScoredTile + threadIdx.x;
  const bool valid = row < p.R;
  int lo = INT_MAX, hi = 0, pos = 0;
  if (valid) {
    row_range(p, m, b, row % p.Tq, &lo, &hi, &pos);
    if (lo >= hi) {
      lo = INT_MAX;
      hi = 0;
    }
  }
  const long long n = static_cast<long long>(b) * p.rpad() + row;
  out.rows[n] = make_int4(lo, hi, pos, 0);
  if (out.slope2 && b == 0)
    for (int k = 0; k < p.Hkv; ++k)
      out.slope2[static_cast<long long>(k) * p.rpad() + row] = valid ? p.slopes[k * p.G + row / p.Tq] * kLog2e : 0.f;
  if (out.even) {
    __shared__ int first;
    if (threadIdx.x == 0) first = pos;
    __syncthreads();
    const int head0 = tile * kScoredTile / p.Tq;
    const bool same = !valid || (pos == first + static_cast<int>(threadIdx.x) && row / p.Tq == head0);
    const bool all = __syncthreads_and(same);
    if (threadIdx.x == 0) out.even[b * static_cast<long long>(p.n_rt) + tile] = make_int4(all ? first : kScoredUneven, 0, 0, 0);
  }
  // hull over the rows that see keys; the keys that every row sees
  int v[4] = {lo, -hi, valid ? -lo : -INT_MAX, valid ? hi : INT_MAX};   // minima of all four
  if (!valid) v[2] = INT_MAX;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = min(v[i], __shfl_xor_sync(0xffffffffu, v[i], o));
  if (out.fine && (threadIdx.x & 31) == 0)
    out.fine[n / 32] = v[1] < 0 ? make_int2(v[0], -v[1]) : make_int2(0, 0);
  __shared__ int s[4][4];
  __shared__ int hull;
  if ((threadIdx.x & 31) == 0)
    for (int i = 0; i < 4; ++i) s[i][threadIdx.x >> 5] = v[i];
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 0; i < 4; ++i) v[i] = min(min(s[i][0], s[i][1]), min(s[i][2], s[i][3]));
    const int hull_hi = -v[1];
    out.tiles[static_cast<long long>(b) * p.n_rt + tile] =
        make_int4(hull_hi > 0 ? v[0] : 0, hull_hi, -v[2], v[3]);
    if (tile == 0 && b == 0) out.counters[0] = out.counters[1] = 0u;
    hull = hull_hi;
  }
  if (idle.O == nullptr && idle.dQ == nullptr) return;
  __syncthreads();
  if (hull > 0) return;
  // no row of the tile sees a key
  for (int k = 0; k < p.Hkv; ++k) {
    const long long head = static_cast<long long>(b) * p.Hkv + k;
    const int n = min(kScoredTile, p.R - tile * kScoredTile);
    const long long at = head * p.R + tile * kScoredTile;
    if (idle.O) {
      zero_rows(idle.O, at * p.dv, n * p.dv);
      if (valid) idle.LSE[head * p.R + row] = -CUDART_INF_F;
    } else {
      zero_rows(idle.dQ, at * p.d, n * p.d);
      idle.D[head * p.rpad() + row] = 0.f;
      idle.NL[head * p.rpad() + row] = -CUDART_INF_F;
    }
  }
}

// One warp per (key tile, batch entry).
__global__ void __launch_bounds__(128) plan_keys_kernel(const ScoredProblem p, const ScoredPlan out,
                                                        const ScoredIdle idle) {
  const long long w = (static_cast<long long>(blockIdx.x) * 128 + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (w >= static_cast<long long>(p.B) * p.n_kt) return;
  const int b = static_cast<int>(w / p.n_kt), kt = static_cast<int>(w % p.n_kt);
  const int k0 = kt * kScoredTile, k1 = k0 + kScoredTile;
  int count = 0;   // lane i: of part i
  bool any = false;
  int lo = INT_MAX, hi = 0;
  bool blank = false;
  for (int t0 = 0; t0 < p.n_rt; t0 += 32) {
    const int t = t0 + lane;
    bool meets = false;
    if (t < p.n_rt) {
      const int4 h = out.tiles[static_cast<long long>(b) * p.n_rt + t];
      meets = h.x < k1 && h.y > k0;
      if (meets) {
        lo = min(lo, h.x);
        hi = max(hi, h.y);
        blank = blank || h.z == INT_MAX;
      }
    }
    const unsigned word = __ballot_sync(0xffffffffu, meets);
    const int first = lane * p.kv_split_tiles - t0;
    count += __popc(word & bit_range(first, first + p.kv_split_tiles));
    any = any || word != 0u;
    if (lane == 0) out.kbits[w * p.n_words() + t0 / 32] = word;
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  blank = __any_sync(0xffffffffu, blank);
  if (lane == 0) out.khull[w] = make_int4(lo, hi, blank, 0);
  if (lane < p.kv_splits) out.kcount[w * p.kv_splits + lane] = count;
  if (any || idle.dK == nullptr) return;
  // no row sees a key of the tile
  for (int k = 0; k < p.Hkv; ++k) {
    const long long row = (static_cast<long long>(b) * p.Hkv + k) * p.Tk + k0;
    const int n = min(kScoredTile, p.Tk - k0);
    uint4* dk = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(idle.dK) + row * p.d);
    uint4* dv = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(idle.dV) + row * p.dv);
    for (int i = lane; i < n * p.d / 8; i += 32) dk[i] = make_uint4(0u, 0u, 0u, 0u);
    for (int i = lane; i < n * p.dv / 8; i += 32) dv[i] = make_uint4(0u, 0u, 0u, 0u);
  }
}

// dK and dV rows from their parts, in part order; one warp per key of a head.
// A part without row tiles for the key's tile was not written.
template <typename T>
__global__ void __launch_bounds__(256) kv_sum_kernel(const ScoredProblem p, const ScoredPlan plan,
                                                     const float* __restrict__ kpart, const float* __restrict__ vpart,
                                                     T* __restrict__ dK, T* __restrict__ dV) {
  const int lane = threadIdx.x & 31;
  const long long rows = static_cast<long long>(p.B) * p.Hkv * p.Tk;
  const long long row = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) >> 5;
  if (row >= rows) return;
  const int bh = static_cast<int>(row / p.Tk), key = static_cast<int>(row - static_cast<long long>(bh) * p.Tk);
  const long long kt = static_cast<long long>(bh / p.Hkv) * p.n_kt + key / kScoredTile;
  const unsigned some =
      __ballot_sync(0xffffffffu, lane < p.kv_splits && plan.kcount[kt * p.kv_splits + min(lane, p.kv_splits - 1)] > 0);
  float k[4] = {0.f, 0.f, 0.f, 0.f}, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
  for (int s = 0; s < p.kv_splits; ++s) {
    if (!(some >> s & 1u)) continue;
    const float* kr = kpart + (s * rows + row) * p.d;
    const float* vr = vpart + (s * rows + row) * p.dv;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (lane + 32 * c < p.d) k[c] += kr[lane + 32 * c];
      if (lane + 32 * c < p.dv) v[c] += vr[lane + 32 * c];
    }
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if (lane + 32 * c < p.d) dK[row * p.d + lane + 32 * c] = static_cast<T>(k[c]);
    if (lane + 32 * c < p.dv) dV[row * p.dv + lane + 32 * c] = static_cast<T>(v[c]);
  }
}

// O and LSE from the key ranges' partial results, in range order; one warp
// per row. TENSOR: the ranges of the tensor-core kernel, which writes a
// range's results only where the row's pair of row tiles has keys in it.
template <typename T, bool TENSOR>
__global__ void __launch_bounds__(256) merge_kernel(const ScoredProblem p, const int4* __restrict__ tiles,
                                                    const float* __restrict__ Opart,
                                                    const float* __restrict__ LSEpart, T* __restrict__ O,
                                                    float* __restrict__ LSE, int n_splits, int split_keys) {
  const int lane = threadIdx.x & 31;
  const long long rows = static_cast<long long>(p.B) * p.Hkv * p.R;
  const long long r = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) >> 5;
  if (r >= rows) return;
  int first = 0, last = n_splits - 1;   // ranges with results
  if constexpr (TENSOR) {
    const int bh = static_cast<int>(r / p.R), pair = static_cast<int>(r - static_cast<long long>(bh) * p.R) / 256;
    const int4* t = tiles + static_cast<long long>(bh / p.Hkv) * p.n_rt + 2 * pair;
    int4 a = t[0];
    if (2 * pair + 1 < p.n_rt) {
      const int4 b = t[1];
      if (a.y == 0 || (b.y > 0 && b.x < a.x)) a.x = b.x;
      a.y = max(a.y, b.y);
    }
    first = a.x / split_keys;
    last = a.y > 0 ? (a.y - 1) / split_keys : -1;
  }
  float mx = -CUDART_INF_F;
  for (int s = first + lane; s <= last; s += 32) mx = fmaxf(mx, LSEpart[s * rows + r]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  float lse = -CUDART_INF_F, wsum = 0.f;
  const float ref = mx == -CUDART_INF_F ? 0.f : mx;
#pragma unroll 4
  for (int s = first; s <= last; ++s) {
    // 0 for a range without keys, whose row is zeros; where the weight of one with keys underflows, a NaN in it shows
    const float w = expf(LSEpart[s * rows + r] - ref);
    wsum += w;
    const float* o = Opart + (s * rows + r) * p.dv;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (lane + 32 * c < p.dv) acc[c] = fmaf(w, o[lane + 32 * c], acc[c]);
  }
  if (wsum != 0.f) {   // (NaN too)
    const float inv = 1.0f / wsum;
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[c] *= inv;
    lse = ref + logf(wsum);
  }
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (lane + 32 * c < p.dv) O[r * p.dv + lane + 32 * c] = static_cast<T>(acc[c]);
  if (lane == 0) LSE[r] = lse;
}

}  // namespace scored

cudaError_t launch_scored_plan(const ScoredProblem& p, const ScoredMask& m, const ScoredPlan& plan,
                               const ScoredIdle& idle, cudaStream_t s) {
  scored::plan_rows_kernel<<<p.n_rt * p.B, kScoredTile, 0, s>>>(p, m, plan, idle);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || plan.kcount == nullptr) return e;
  const long long warps = static_cast<long long>(p.B) * p.n_kt;
  scored::plan_keys_kernel<<<static_cast<unsigned>((warps + 3) / 4), 128, 0, s>>>(p, plan, idle);
  return cudaGetLastError();
}

cudaError_t launch_scored_kv_sum(const ScoredBwd& a, bool bf16) {
  const long long rows = static_cast<long long>(a.p.B) * a.p.Hkv * a.p.Tk;
  const unsigned grid = static_cast<unsigned>((rows + 7) / 8);
  if (bf16)
    scored::kv_sum_kernel<<<grid, 256, 0, a.stream>>>(a.p, a.plan, a.dKpart, a.dVpart,
                                                      static_cast<__nv_bfloat16*>(a.dK),
                                                      static_cast<__nv_bfloat16*>(a.dV));
  else
    scored::kv_sum_kernel<<<grid, 256, 0, a.stream>>>(a.p, a.plan, a.dKpart, a.dVpart, static_cast<float*>(a.dK),
                                                      static_cast<float*>(a.dV));
  return cudaGetLastError();
}

cudaError_t launch_scored_merge(const ScoredFwd& a, bool bf16) {
  const long long rows = static_cast<long long>(a.p.B) * a.p.Hkv * a.p.R;
  const unsigned grid = static_cast<unsigned>((rows + 7) / 8);
  if (bf16)
    scored::merge_kernel<__nv_bfloat16, true><<<grid, 256, 0, a.stream>>>(
        a.p, a.plan.tiles, a.Opart, a.LSEpart, static_cast<__nv_bfloat16*>(a.O), a.LSE, a.n_splits, a.split_keys);
  else
    scored::merge_kernel<float, false><<<grid, 256, 0, a.stream>>>(a.p, a.plan.tiles, a.Opart, a.LSEpart,
                                                                   static_cast<float*>(a.O), a.LSE, a.n_splits,
                                                                   a.split_keys);
  return cudaGetLastError();
}

}  // namespace attn
