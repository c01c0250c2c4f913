// Reading a paged key-value cache back as contiguous rows, and the row ranges
// of an attention call over a cache. Bound by memory: every code is read and
// every element written once. 8 x 16384 tokens, 8 heads, d=128, e4m3 to bf16,
// 678 MB: 103 us, 6.6 TB/s (168 with one 8-code piece a thread and its place
// found by 64-bit divisions).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cache.h"
#include "ptx.cuh"

namespace attn {
namespace cache {
namespace {

constexpr int NT = 256;

// 32 bytes: in one store (sm_100 and later) where they are aligned to 32, else in two.
__device__ __forceinline__ void store32(void* p, const uint32_t (&x)[8], bool one) {
  if (!one) {
    static_cast<uint4*>(p)[0] = make_uint4(x[0], x[1], x[2], x[3]);
    static_cast<uint4*>(p)[1] = make_uint4(x[4], x[5], x[6], x[7]);
    return;
  }
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]), "r"(x[1]), "r"(x[2]),
               "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}

// 16 codes times s, to 16 elements at p.
template <typename T>
__device__ __forceinline__ void put16(T* p, uint4 x, float s, bool one) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t y[sizeof(T) * 4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint32_t h = codes_to_half2(static_cast<uint16_t>(w[i] >> 16 * half));
      const float2 v = ptx::fmul2(half2_to_float2(h), make_float2(s, s));
      const int at = 2 * i + half;
      if constexpr (sizeof(T) == 2) {
        y[at] = ptx::pack_bf16(v.x, v.y);
      } else {
        y[2 * at] = __float_as_uint(v.x);
        y[2 * at + 1] = __float_as_uint(v.y);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) {
    const uint32_t* q = y + 8 * i;
    const uint32_t z[8] = {q[0], q[1], q[2], q[3], q[4], q[5], q[6], q[7]};
    store32(reinterpret_cast<uint32_t*>(p) + 8 * i, z, one);
  }
}

// A block takes `tile` tokens of one head's keys or values, a thread 16 codes
// (V elements of a plain cache) of every step-th of them, the loads of U on
// their way together: pages and scales are looked up per row, from the
// first-level cache after the first.
constexpr int U = 4;

template <typename T, int V, bool CODES>
__global__ void __launch_bounds__(NT) read_kernel(const __grid_constant__ CacheRead P, int tile) {
  using In = rope::Vec<T, V>;
  const int side = blockIdx.y;
  const int w = P.w[side], per = w / V;
  const int tiles = (P.Tk + tile - 1) / tile;
  const int bh = static_cast<int>(blockIdx.x / tiles);
  const int t0 = static_cast<int>(blockIdx.x - static_cast<unsigned>(bh) * tiles) * tile;
  const int b = bh / P.Hkv, h = bh - b * P.Hkv;
  int from = t0, to = min(P.Tk, t0 + tile);
  const int last = tokens_of(P.c, b);
  if (P.hull) {
    const int2 hull = P.hull[b];
    from = max(from, hull.x);
    to = min(to, hull.y);
  }
  const int step = NT / per;   // (rows have at most NT pieces)
  const int lane = threadIdx.x / per;
  if (lane >= step) return;
  const int col = (static_cast<int>(threadIdx.x) - lane * per) * V, mask = (1 << P.c.shift) - 1;
  T* out = static_cast<T*>(P.out[side]) + static_cast<long long>(bh) * P.Tk * w;
  const bool one = reinterpret_cast<uintptr_t>(out) % 32 == 0;   // (rows are whole 32 bytes)
  for (int r0 = from + lane; r0 < to; r0 += U * step) {
    uint4 x[CODES ? U : 1];
    In y[CODES ? 1 : U];
    float s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = r0 + u * step;
      const int at = t < to && t < last ? page_of(P.c, b, t >> P.c.shift) : -1;
      const long long head = static_cast<long long>(at) * P.Hkv + h;
      const long long row = ((head << P.c.shift) + (t & mask)) * w + col;
      if constexpr (CODES) {
        x[u] = at >= 0 ? *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(P.c.pool[side]) + row)
                       : make_uint4(0u, 0u, 0u, 0u);
        s[u] = at >= 0 ? clamp_scale(__ldg(P.c.scale[side] + head)) : 1.f;
      } else {
        y[u] = at >= 0 ? *reinterpret_cast<const In*>(static_cast<const T*>(P.c.pool[side]) + row) : In{};
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = r0 + u * step;
      if (t >= to) break;
      T* p = out + static_cast<long long>(t) * w + col;
      if constexpr (CODES)
        put16(p, x[u], s[u], one);
      else
        *reinterpret_cast<In*>(p) = y[u];
    }
  }
}

template <typename T, int V, bool CODES>
cudaError_t read(const CacheRead& a) {
  // tokens of a block: 128, fewer where that leaves less than eight blocks an SM
  int tile = 128;
  const long long heads = static_cast<long long>(a.B) * a.Hkv * 2;
  while (tile > 16 && heads * ((a.Tk + tile - 1) / tile) < a.num_sms * 8LL) tile /= 2;
  const long long tiles = heads / 2 * ((a.Tk + tile - 1) / tile);
  if (tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
  read_kernel<T, V, CODES><<<dim3(static_cast<unsigned>(tiles), 2), NT, 0, a.stream>>>(a, tile);
  return cudaGetLastError();
}

// The rows of a sequence: one block.
__global__ void __launch_bounds__(NT) rows_kernel(const __grid_constant__ CacheRows P) {
  __shared__ int lo_s[NT / 32], hi_s[NT / 32];
  const int b = blockIdx.x;
  const int len = tokens_of(P.c, b), n = new_of(P.c, b, P.Tq);
  int most_hi = 0, least_lo = 0x7fffffff;
  for (int t = threadIdx.x; t < P.Tq; t += NT) {
    const long long at = static_cast<long long>(b) * P.Tq + t;
    int lo, hi, pos;
    cache::row_range(P.mask, at, t, len, n, P.Tk, P.window, &lo, &hi, &pos);
    const bool some = lo < hi;
    P.q_pos[at] = pos;
    P.key_begin[at] = some ? lo : 0;
    P.key_end[at] = some ? hi : 0;
    if (some) {
      least_lo = min(least_lo, lo);
      most_hi = max(most_hi, hi);
    }
  }
  least_lo = __reduce_min_sync(0xffffffffu, least_lo);
  most_hi = __reduce_max_sync(0xffffffffu, most_hi);
  if ((threadIdx.x & 31) == 0) lo_s[threadIdx.x >> 5] = least_lo, hi_s[threadIdx.x >> 5] = most_hi;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < NT / 32; ++i) least_lo = min(least_lo, lo_s[i]), most_hi = max(most_hi, hi_s[i]);
    P.hull[b] = most_hi > 0 ? make_int2(least_lo, most_hi) : make_int2(0, 0);
  }
}

}  // namespace
}  // namespace cache

cudaError_t launch_cache_read(const CacheRead& a) {
  if (a.c.codes) return a.bf16 ? cache::read<__nv_bfloat16, 16, true>(a) : cache::read<float, 16, true>(a);
  if (a.bf16) return cache::read<__nv_bfloat16, 8, false>(a);
  const bool wide = a.w[0] % 4 == 0 && a.w[1] % 4 == 0 &&
                    (reinterpret_cast<uintptr_t>(a.c.pool[0]) | reinterpret_cast<uintptr_t>(a.c.pool[1]) |
                     reinterpret_cast<uintptr_t>(a.out[0]) | reinterpret_cast<uintptr_t>(a.out[1])) % 16 == 0;
  return wide ? cache::read<float, 4, false>(a) : cache::read<float, 1, false>(a);
}

cudaError_t launch_cache_rows(const CacheRows& a) {
  cache::rows_kernel<<<a.B, cache::NT, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace attn
