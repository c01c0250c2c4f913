// Appending to a paged key-value cache: keys rotated by position and values,
// as they are or in e4m3 with a scale per page and head, and the rotation of
// the queries in the same launch.
//
// A unit is what one call adds to one page of one head, keys or values. Small
// ones (single tokens) are a warp's work each: it finds the largest element
// first, which fixes the page's scale, and reads its rows a second time (from
// the first-level cache) to rotate, round and store them. Where a page takes
// more, a block holds a unit in registers between the two, and goes through the
// heads of a page one after another: the sines and cosines, a third of the
// instructions if formed for every head, are formed once and kept in shared
// memory, and a head's rows are on their way while the one before is worked on.
// 2 x 8192 tokens, H=32 Hkv=8 d=128, bf16 to e4m3 in pages of 64, 369 MB: 62 us,
// 6.0 TB/s (91 with rows read twice and sines per head; 73 with the queries'
// blocks before the pages' instead of between them: the queries' alone are 42.5
// us of waiting for memory, the pages' 28 of arithmetic and barriers).
// The scale is a power of two, so that codes move between scales without a
// second rounding unless they reach the subnormal range, and it is taken from
// the keys before their rotation, times the most a rotation makes of them: it
// then follows from the inputs alone, not from the last bits of a sine.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "cache.h"
#include "ptx.cuh"

namespace attn {
namespace cache {
namespace {

constexpr int NT = rope::NT;
using rope::Vec;
using rope::to_f;
using rope::from_f;

struct Params {
  rope::Params q;
  CacheView c;
  const void* x[2];
  View s[2];
  const int* pos;
  int B, Hkv, T, w[2];
  int touch;            // pages of a sequence that a call may touch
  int rot_chunks;       // chunks of V rotated pairs of a key (0: none)
  int per[2];           // chunks of a key and of a value
  int rot;              // rotated elements of a key (0: none)
  float top[2];         // what the size of a rotated and of another element is multiplied by
  unsigned q_blocks;
  long long units;
};

// The least e with a <= 448 * 2^e (448 = 1.75 * 2^8), within the scales' range; exact.
__device__ __forceinline__ int scale_exponent(float a) {
  const uint32_t u = __float_as_uint(a);
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);   // (subnormal: below -100)
  return min(max(e, kScaleLeast), kScaleMost);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// LANES threads of a block: the largest of their values, in all of them.
template <int LANES>
__device__ __forceinline__ float group_max(float x, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  if constexpr (LANES > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < LANES / 32; ++i) x = fmaxf(x, red[i]);
  }
  return x;
}

__device__ __forceinline__ float finite_size(float x) {
  const float a = fabsf(x);
  return a <= 3.4028234e38f ? a : 0.f;
}
__device__ __forceinline__ float or_nan(float x) { return fabsf(x) <= 3.4028234e38f ? x : CUDART_NAN_F; }

// V numbers times `inv` as codes (CHECK: not finite as NaN).
template <int V, bool CHECK = true>
__device__ __forceinline__ void store_codes(uint8_t* dst, const float (&y)[V], float inv) {
  auto at = [&](int i) { return (CHECK ? or_nan(y[i]) : y[i]) * inv; };
  if constexpr (V == 1) {
    *dst = static_cast<uint8_t>(float2_to_codes(at(0), 0.f));
  } else {
    uint32_t r[V / 4];
#pragma unroll
    for (int i = 0; i < V / 4; ++i)
      r[i] = static_cast<uint32_t>(float2_to_codes(at(4 * i), at(4 * i + 1))) |
             static_cast<uint32_t>(float2_to_codes(at(4 * i + 2), at(4 * i + 3))) << 16;
    if constexpr (V == 8)
      *reinterpret_cast<uint2*>(dst) = make_uint2(r[0], r[1]);
    else
      *reinterpret_cast<uint32_t*>(dst) = r[0];
  }
}

// n codes (a multiple of 16) times `ratio`: the tokens that a page holds, at its new scale. By `lanes` threads.
__device__ __forceinline__ void requantise(uint8_t* codes, int n, float ratio, int lane, int lanes) {
  uint4* old = reinterpret_cast<uint4*>(codes);
  for (int i = lane; i < n / 16; i += lanes) {
    uint4 v = old[i];
    uint32_t* q = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 lo = half2_to_float2(codes_to_half2(static_cast<uint16_t>(q[e])));
      const float2 hi = half2_to_float2(codes_to_half2(static_cast<uint16_t>(q[e] >> 16)));
      q[e] = static_cast<uint32_t>(float2_to_codes(lo.x * ratio, lo.y * ratio)) |
             static_cast<uint32_t>(float2_to_codes(hi.x * ratio, hi.y * ratio)) << 16;
    }
    old[i] = v;
  }
}

template <typename T, int V, bool INTER, bool CODES, int LANES>
__global__ void __launch_bounds__(NT) append_kernel(const __grid_constant__ Params P) {
  ptx::grid_wait();          // (the launch overlaps the end of the kernel before)
  ptx::grid_launch_next();   // (and the next one's this)
  if (blockIdx.x < P.q_blocks) {
    __shared__ __align__(16) uint8_t room[V > 1 ? rope::STAGE_BYTES : 16];
    rope::turn_rows<T, V, INTER, true>(P.q, blockIdx.x, room);
    return;
  }
  using W = Vec<T, V>;
  __shared__ float red[NT / 32];
  const int lane = threadIdx.x % LANES;
  long long u = static_cast<long long>(blockIdx.x - P.q_blocks) * (NT / LANES) + threadIdx.x / LANES;
  if (u >= P.units) return;
  const int side = static_cast<int>(u & 1);
  u >>= 1;
  const int h = static_cast<int>(u % P.Hkv);
  u /= P.Hkv;
  const int j = static_cast<int>(u % P.touch), b = static_cast<int>(u / P.touch);
  // the unit's tokens [a, z), of the page's [p0, p0 + page)
  const int len = tokens_of(P.c, b), first = len - new_of(P.c, b, P.T);
  const int shift = P.c.shift;
  const int index = (max(first, 0) >> shift) + j, p0 = index << shift;
  const int a = max(max(first, 0), p0), z = min(len, p0 + (1 << shift));
  if (a >= z) return;
  const int at = page_of(P.c, b, index);
  if (at < 0) return;
  const int w = P.w[side], per = P.per[side];
  const int n = (z - a) * per;
  const T* x = static_cast<const T*>(P.x[side]) + b * P.s[side].b + h * P.s[side].h + (a - first) * P.s[side].t;
  const long long tile = ((static_cast<long long>(at) * P.Hkv + h) << shift) * w;   // the page's rows of the head
  const long long dst = tile + static_cast<long long>(a - p0) * w;
  const int rot_chunks = side == 0 ? P.rot_chunks : 0, rot = side == 0 ? P.rot : 0;

  auto places = [&](int c, int* o0, int* o1) {
    const bool turn = c < rot_chunks;
    *o0 = !turn ? rot + V * (c - rot_chunks) : INTER ? 2 * V * c : V * c;
    *o1 = !turn ? *o0 : INTER ? *o0 + V : *o0 + rot / 2;
    return turn;
  };
  float inv = 1.f;
  if constexpr (CODES) {
    float most = 0.f;
    for (int i = lane; i < n; i += LANES) {
      const int r = i / per, c = i - r * per;
      int o0, o1;
      const bool turn = places(c, &o0, &o1);
      const T* row = x + r * P.s[side].t;
      const W p = *reinterpret_cast<const W*>(row + o0);
      const W q = turn ? *reinterpret_cast<const W*>(row + o1) : p;
      float m = 0.f;
#pragma unroll
      for (int e = 0; e < V; ++e) m = fmaxf(m, fmaxf(finite_size(to_f(p.e[e])), finite_size(to_f(q.e[e]))));
      most = fmaxf(most, m * P.top[turn ? 0 : 1]);
    }
    float* place = P.c.scale[side] + static_cast<long long>(at) * P.Hkv + h;
    const float held = a > p0 ? clamp_scale(*place) : 0.f;
    // (the reduction is also the barrier between this read of the scale and its write)
    const float s = fmaxf(pow2(scale_exponent(group_max<LANES>(most, red))), held);
    __syncwarp();
    if (lane == 0) *place = s;
    inv = 1.f / s;   // (exact: all but a scale from elsewhere are powers of two)
    if (a > p0 && s > held)
      requantise(static_cast<uint8_t*>(P.c.pool[side]) + tile, (a - p0) * w, held * inv, lane, LANES);
  }
  for (int i = lane; i < n; i += LANES) {
    const int r = i / per, c = i - r * per;
    int o0, o1;
    const bool turn = places(c, &o0, &o1);
    const T* row = x + r * P.s[side].t;
    const W p = *reinterpret_cast<const W*>(row + o0);
    float y0[V], y1[V];
#pragma unroll
    for (int e = 0; e < V; ++e) y0[e] = to_f(p.e[e]);
    if (turn) {
      const W q = *reinterpret_cast<const W*>(row + o1);
#pragma unroll
      for (int e = 0; e < V; ++e) y1[e] = to_f(q.e[e]);
      const int t = a - first + r;
      const long long pos = P.pos ? P.pos[static_cast<long long>(b) * P.T + t] : a + r;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const unsigned long long turns = static_cast<unsigned long long>(pos) * P.q.plan.turns[V * c + e];
        float sn, cs;
        sincospif(static_cast<float>(static_cast<int>(turns >> 32)) * 0x1p-31f, &sn, &cs);
        sn *= P.q.plan.mscale;
        cs *= P.q.plan.mscale;
        float& pu = INTER ? (2 * e < V ? y0[(2 * e) % V] : y1[(2 * e) % V]) : y0[e];
        float& pv = INTER ? (2 * e + 1 < V ? y0[(2 * e + 1) % V] : y1[(2 * e + 1) % V]) : y1[e];
        const float f = pu, g = pv;
        pu = f * cs - g * sn;
        pv = g * cs + f * sn;
      }
    }
    const long long o = dst + static_cast<long long>(r) * w;
    if constexpr (CODES) {
      uint8_t* out = static_cast<uint8_t*>(P.c.pool[side]) + o;
      store_codes<V>(out + o0, y0, inv);
      if (turn) store_codes<V>(out + o1, y1, inv);
    } else {
      T* out = static_cast<T*>(P.c.pool[side]) + o;
      W k;
#pragma unroll
      for (int e = 0; e < V; ++e) k.e[e] = from_f<T>(y0[e]);
      *reinterpret_cast<W*>(out + o0) = k;
      if (turn) {
#pragma unroll
        for (int e = 0; e < V; ++e) k.e[e] = from_f<T>(y1[e]);
        *reinterpret_cast<W*>(out + o1) = k;
      }
    }
  }
}

// ---------------------------------------------------------------- units in registers

// The larger of the sizes in m and of V elements, as the bits of their
// magnitudes: two 16-bit numbers for bf16, whose order is that of the bits.
__device__ __forceinline__ void larger(uint32_t& m, uint32_t x, __nv_bfloat16) {
  const uint32_t a = x & 0x7fff7fffu;
  asm("max.u16x2 %0, %0, %1;" : "+r"(m) : "r"(a));
}
__device__ __forceinline__ void larger(uint32_t& m, uint32_t x, float) { m = max(m, x & 0x7fffffffu); }
__device__ __forceinline__ float size_of(uint32_t m, __nv_bfloat16) {
  return __uint_as_float(max(m >> 16, m & 0xffffu) << 16);
}
__device__ __forceinline__ float size_of(uint32_t m, float) { return __uint_as_float(m); }

// 16 bytes as V numbers.
template <typename T>
__device__ __forceinline__ void numbers(float (&y)[16 / sizeof(T)], uint4 x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      y[2 * i] = __uint_as_float(w[i] << 16);
      y[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      y[i] = __uint_as_float(w[i]);
    }
  }
}

// A page of one sequence, keys or values of `group` heads: a block, of up to NI
// pieces a thread. A piece is two 16-byte vectors of a row: both sides of V
// rotated pairs, or 2 V adjacent elements (the last of an odd number: one
// vector, twice). The blocks that rotate the queries, which wait for memory
// more, are spread between them.
template <typename T, bool INTER, bool CODES, int NI>
__global__ void __launch_bounds__(NT, 8 / NI) pages_kernel(const __grid_constant__ Params P, int group, unsigned blocks) {
  constexpr int V = 16 / sizeof(T), TH = NT;
  extern __shared__ float4 turns_of[];   // [NI][2][V / 4][TH]: a thread's cosines and sines, in its own slots
  __shared__ float red[2][TH / 32];
  const int groups = (P.Hkv + group - 1) / group;
  ptx::grid_wait();          // (the launch overlaps the end of the kernel before)
  ptx::grid_launch_next();   // (and the next one's this)
  // `blocks` of the launch's are pages': those at which this share of the index steps up
  const unsigned before = static_cast<unsigned>(static_cast<unsigned long long>(blockIdx.x) * blocks / gridDim.x);
  if (static_cast<unsigned>((blockIdx.x + 1ull) * blocks / gridDim.x) == before) {
    rope::turn_rows<T, V, INTER, true>(P.q, blockIdx.x - before, turns_of);
    return;
  }
  int u = static_cast<int>(before);
  const int side = u & 1;
  u >>= 1;
  const int h0 = u % groups * group;
  u /= groups;
  const int j = u % P.touch, b = u / P.touch;
  // the unit's tokens [a, z), of the page's [p0, p0 + page)
  const int len = tokens_of(P.c, b), first = len - new_of(P.c, b, P.T);
  const int shift = P.c.shift;
  const int index = (max(first, 0) >> shift) + j, p0 = index << shift;
  const int a = max(max(first, 0), p0), z = min(len, p0 + (1 << shift));
  if (a >= z) return;
  const int at = page_of(P.c, b, index);
  if (at < 0) return;
  const int w = P.w[side], rot = side == 0 ? P.rot : 0;
  const int turned = rot / 2 / V, per = turned + ((w - rot) / V + 1) / 2;   // pieces of a row
  const int n = (z - a) * per;
  const T* x = static_cast<const T*>(P.x[side]) + b * P.s[side].b + static_cast<long long>(a - first) * P.s[side].t;
  const int heads = min(group, P.Hkv - h0);

  const T* src[NI];
  int o0[NI], o1[NI];      // of the piece's vectors behind the page's first new row of a head; o0 < 0: no piece
  auto slot = [&](int i, int k, int v) -> float4& { return turns_of[((i * 2 + k) * (V / 4) + v) * TH + threadIdx.x]; };
  unsigned turn = 0;       // bit i: piece i is rotated
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int at_i = threadIdx.x + i * TH;
    o0[i] = -1, o1[i] = 0;
    src[i] = x;
    if (at_i >= n) continue;
    const int r = at_i / per, c = at_i - r * per;
    const bool t = c < turned;
    const int e0 = t ? (INTER ? 2 * V * c : V * c) : rot + 2 * V * (c - turned);
    const int e1 = t ? (INTER ? e0 + V : e0 + rot / 2) : (e0 + V < w ? e0 + V : e0);
    src[i] = x + r * P.s[side].t + e0;
    o0[i] = r * w + e0;
    o1[i] = e1 - e0;
    if (!t) continue;
    turn |= 1u << i;
    const long long pos = P.pos ? P.pos[static_cast<long long>(b) * P.T + (a - first) + r] : a + r;
    for (int v = 0; v < V / 4; ++v) {
      float sn[4], cs[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const unsigned long long turns = static_cast<unsigned long long>(pos) * P.q.plan.turns[V * c + 4 * v + e];
        sincospif(static_cast<float>(static_cast<int>(turns >> 32)) * 0x1p-31f, &sn[e], &cs[e]);
        sn[e] *= P.q.plan.mscale;
        cs[e] *= P.q.plan.mscale;
      }
      slot(i, 0, v) = make_float4(cs[0], cs[1], cs[2], cs[3]);
      slot(i, 1, v) = make_float4(sn[0], sn[1], sn[2], sn[3]);
    }
  }
  uint4 raw[NI][2];
  auto fetch = [&](int h) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (o0[i] < 0) continue;
      const T* p = src[i] + h * P.s[side].h;
      raw[i][0] = *reinterpret_cast<const uint4*>(p);
      raw[i][1] = *reinterpret_cast<const uint4*>(p + o1[i]);
    }
  };
  fetch(h0);
  for (int h = h0; h < h0 + heads; ++h) {
    const long long head = static_cast<long long>(at) * P.Hkv + h;
    const long long tile = (head << shift) * w;   // the page's rows of the head
    const long long dst = tile + static_cast<long long>(a - p0) * w;
    uint4 now[NI][2];
#pragma unroll
    for (int i = 0; i < NI; ++i) now[i][0] = raw[i][0], now[i][1] = raw[i][1];
    if (h + 1 < h0 + heads) fetch(h + 1);
    float inv = 1.f;
    bool safe = true;   // no element that is not finite, or that the rotation may leave not finite
    if constexpr (CODES) {
      float* place = P.c.scale[side] + head;
      const float held = a > p0 ? clamp_scale(*place) : 0.f;
      uint32_t m[2] = {0u, 0u};   // of rotated elements, and of others
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        if (o0[i] < 0) continue;
        uint32_t k = 0u;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          larger(k, now[i][v].x, T{});
          larger(k, now[i][v].y, T{});
          larger(k, now[i][v].z, T{});
          larger(k, now[i][v].w, T{});
        }
        larger(m[turn >> i & 1u ? 0 : 1], k, T{});
      }
      float most = fmaxf(size_of(m[0], T{}) * P.top[0], size_of(m[1], T{}) * P.top[1]);
      safe = size_of(m[0], T{}) * P.top[0] < 1.7e38f && size_of(m[1], T{}) < 1.7e38f;   // (a NaN's bits are a NaN here)
      if (!safe) {
        most = 0.f;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          if (o0[i] < 0) continue;
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            float y[V];
            numbers<T>(y, now[i][v]);
#pragma unroll
            for (int e = 0; e < V; ++e) most = fmaxf(most, finite_size(y[e]) * P.top[turn >> i & 1u ? 0 : 1]);
          }
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
      float* mine = red[(h - h0) & 1];
      if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = most;
      __syncthreads();   // (also between the reads of the old scale and its write)
#pragma unroll
      for (int i = 0; i < TH / 32; ++i) most = fmaxf(most, mine[i]);
      const float s = fmaxf(pow2(scale_exponent(most)), held);
      if (threadIdx.x == 0) *place = s;
      inv = 1.f / s;   // (exact: all but a scale from elsewhere are powers of two)
      if (a > p0 && s > held)
        requantise(static_cast<uint8_t*>(P.c.pool[side]) + tile, (a - p0) * w, held * inv, threadIdx.x, TH);
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (o0[i] < 0) continue;
      float y0[V], y1[V];
      numbers<T>(y0, now[i][0]);
      numbers<T>(y1, now[i][1]);
      if (turn >> i & 1u) {
        float cs[V], sn[V];
#pragma unroll
        for (int v = 0; v < V / 4; ++v) {
          const float4 f = slot(i, 0, v), g = slot(i, 1, v);
          cs[4 * v] = f.x, cs[4 * v + 1] = f.y, cs[4 * v + 2] = f.z, cs[4 * v + 3] = f.w;
          sn[4 * v] = g.x, sn[4 * v + 1] = g.y, sn[4 * v + 2] = g.z, sn[4 * v + 3] = g.w;
        }
        if constexpr (INTER) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            float& pu = 2 * e < V ? y0[(2 * e) % V] : y1[(2 * e) % V];
            float& pv = 2 * e + 1 < V ? y0[(2 * e + 1) % V] : y1[(2 * e + 1) % V];
            const float f = pu, g = pv;
            pu = f * cs[e] - g * sn[e];
            pv = g * cs[e] + f * sn[e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float f = y0[e], g = y1[e];
            y0[e] = f * cs[e] - g * sn[e];
            y1[e] = g * cs[e] + f * sn[e];
          }
        }
      }
      if constexpr (CODES) {
        uint8_t* out = static_cast<uint8_t*>(P.c.pool[side]) + dst + o0[i];
        if (!safe) {
#pragma unroll
          for (int e = 0; e < V; ++e) y0[e] = or_nan(y0[e]), y1[e] = or_nan(y1[e]);
        }
        store_codes<V, false>(out, y0, inv);
        store_codes<V, false>(out + o1[i], y1, inv);
      } else {
        T* out = static_cast<T*>(P.c.pool[side]) + dst + o0[i];
        Vec<T, V> k0, k1;
#pragma unroll
        for (int e = 0; e < V; ++e) k0.e[e] = from_f<T>(y0[e]), k1.e[e] = from_f<T>(y1[e]);
        *reinterpret_cast<Vec<T, V>*>(out) = k0;
        *reinterpret_cast<Vec<T, V>*>(out + o1[i]) = k1;
      }
    }
  }
}

template <typename T, bool CODES, int NI>
cudaError_t launch_pages(const CacheAppend& a, const Params& P) {
  const long long pages = static_cast<long long>(P.B) * P.touch * 2;
  // heads of a block: up to 8, fewer where that leaves less than four blocks an SM
  int group = P.Hkv < 8 ? P.Hkv : 8;
  while (group > 1 && pages * ((P.Hkv + group - 1) / group) < a.num_sms * 4LL) group = (group + 1) / 2;
  const long long blocks = pages * ((P.Hkv + group - 1) / group), grid = blocks + P.q_blocks;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  constexpr int SINES = NI * 2 * static_cast<int>(16 / sizeof(T)) * 4 * NT;
  constexpr int SMEM = SINES > rope::STAGE_BYTES ? SINES : rope::STAGE_BYTES;
  auto kern = a.q.plan.interleaved ? pages_kernel<T, true, CODES, NI> : pages_kernel<T, false, CODES, NI>;
  static std::atomic<unsigned long long> done[2];   // of the two kernels
  const cudaError_t e = SMEM > 47 * 1024 ? allow_smem(kern, SMEM, done[a.q.plan.interleaved ? 1 : 0]) : cudaSuccess;
  if (e != cudaSuccess) return e;
  return launch_over(kern, static_cast<unsigned>(grid), NT, SMEM, a.stream, P, group, static_cast<unsigned>(blocks));
}

// Pieces of a unit, at most.
int pieces(const CacheAppend& a, int rot, int V) {
  const int page = 1 << a.c.shift;
  const int k = rot / 2 / V + ((a.w[0] - rot) / V + 1) / 2, v = (a.w[1] / V + 1) / 2;
  return (a.T < page ? a.T : page) * (k > v ? k : v);
}

template <typename T, bool CODES>
cudaError_t launch_pages(const CacheAppend& a, const Params& P, int n) {
  if (n <= 2 * NT) return launch_pages<T, CODES, 2>(a, P);
  if (n <= 4 * NT) return launch_pages<T, CODES, 4>(a, P);
  return launch_pages<T, CODES, 8>(a, P);
}

int touched(int T, int shift) { return (T + (1 << shift) - 2) / (1 << shift) + 1; }

template <typename T, int V>
cudaError_t launch(const CacheAppend& a) {
  Params P{};
  P.q = a.q;
  P.c = a.c;
  for (int k = 0; k < 2; ++k) {
    P.x[k] = a.x[k];
    P.s[k] = a.s[k];
    P.w[k] = a.w[k];
  }
  P.pos = a.pos;
  P.B = a.B;
  P.Hkv = a.Hkv;
  P.T = a.T;
  P.touch = touched(a.T, a.c.shift);
  P.rot = a.turn ? a.q.plan.rot : 0;
  P.rot_chunks = P.rot / 2 / V;
  P.per[0] = P.rot_chunks + (a.w[0] - P.rot) / V;
  P.per[1] = a.w[1] / V;
  P.top[0] = kTurned * fabsf(a.q.plan.mscale);
  P.top[1] = 1.f;
  P.units = cache_append_units(a.B, a.Hkv, a.T, a.c.shift);
  long long q_blocks = 0;
  if (a.q.heads[0] > 0) q_blocks = rope::shape_launch<T, V>(P.q, a.num_sms);
  if (q_blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  P.q_blocks = static_cast<unsigned>(q_blocks);
  const bool inter = a.q.plan.interleaved;
  auto go = [&](auto kern, long long blocks) {
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_over(kern, static_cast<unsigned>(blocks), NT, 0, a.stream, P);
  };
  // a warp per unit up to 512 elements (16 tokens of d = 128, 2 sequences: 8.3 us by warps, 4.0 by blocks; 4 tokens of
  // 64 sequences: 6.4 us either way)
  const int most = a.T < (1 << a.c.shift) ? a.T : 1 << a.c.shift;
  if (most * (a.w[0] > a.w[1] ? a.w[0] : a.w[1]) <= 512) {
    const long long blocks = q_blocks + (P.units + NT / 32 - 1) / (NT / 32);
    if (a.c.codes)
      return inter ? go(append_kernel<T, V, true, true, 32>, blocks) : go(append_kernel<T, V, false, true, 32>, blocks);
    return inter ? go(append_kernel<T, V, true, false, 32>, blocks) : go(append_kernel<T, V, false, false, 32>, blocks);
  }
  if constexpr (V > 1) {
    const int n = pieces(a, P.rot, V);
    if (n <= 8 * NT) return a.c.codes ? launch_pages<T, true>(a, P, n) : launch_pages<T, false>(a, P, n);
  }
  const long long blocks = q_blocks + P.units;
  if (a.c.codes)
    return inter ? go(append_kernel<T, V, true, true, NT>, blocks) : go(append_kernel<T, V, false, true, NT>, blocks);
  return inter ? go(append_kernel<T, V, true, false, NT>, blocks) : go(append_kernel<T, V, false, false, NT>, blocks);
}

}  // namespace
}  // namespace cache

long long cache_append_units(int B, int Hkv, int T, int shift) {
  return static_cast<long long>(B) * cache::touched(T, shift) * Hkv * 2;
}

cudaError_t launch_cache_append(const CacheAppend& a) {
  if (a.bf16) return a.wide ? cache::launch<__nv_bfloat16, 8>(a) : cache::launch<__nv_bfloat16, 1>(a);
  return a.wide ? cache::launch<float, 4>(a) : cache::launch<float, 1>(a);
}

}  // namespace attn
