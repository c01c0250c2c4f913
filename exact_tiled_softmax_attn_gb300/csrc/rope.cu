// Rotary positions of queries and keys.
//
// Pair (u, v) of a token at position p is turned by p * f_i. The plan holds
// f_i / (2 pi), rounded to F_i * 2^-64, so that p * F_i modulo 2^64 is the
// angle as a fraction of a turn, off by |p| * 2^-65 at most; an int32 position
// leaves its upper 32 bits right, to one of them. They, as a signed
// number, times 2^-31 is the angle in half turns within [-1, 1), which
// sincospi takes. (An fp32 product p * f_i would be off by 0.03 radians at p
// = 10^6.) One thread does one chunk of pairs of one token for several heads
// and so computes each sine and cosine once for all of them; the rest of a
// head (from rot on) is copied in chunks of its own. Bound by memory: every
// element is read and written once, in 16-byte accesses where rows, strides
// and pointers allow. What a load waits for must not hold the next one back
// (a store in between may be to the same memory, so the compiler keeps the
// order): four heads ahead are copied to the thread's own slots in shared
// memory, which costs no registers.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attn.h"
#include "host.h"
#include "views.h"

namespace attn {
namespace rope {

constexpr int NT = 256;

struct Params {
  attn_rope_t plan;
  const void* x[2];   // Q, K
  void* y[2];
  View xs[2], ys[2];
  const int* pos;
  int heads[2];       // H, Hkv
  int B, T, d;
  int slots;          // threads that share a token's chunk, each with every slots-th head
  int rot_chunks;     // chunks of V pairs
  int chunks;         // and of V copied elements behind them
  int tokens_per_block;
  float sign;         // -1: inverse
};

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T e[V];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

constexpr int STAGES = 4;   // heads a thread has in flight

__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {   // all but the last N groups of this thread
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// V pairs (or V copied elements) a chunk; INTER: the pairs of a chunk are 2 V
// adjacent elements, otherwise V elements at i and V at i + rot / 2.
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(NT) rope_kernel(const __grid_constant__ Params P) {
  using W = Vec<T, V>;
  constexpr bool WIDE = sizeof(W) == 16;
  __shared__ __align__(16) W stage[WIDE ? STAGES : 1][2][WIDE ? NT : 1];
  const int per_token = P.slots * P.chunks;
  const long long tokens = static_cast<long long>(P.B) * P.T;
  const int n = P.tokens_per_block * per_token;
  const int total = P.heads[0] + P.heads[1];
  for (int i = threadIdx.x; i < n; i += NT) {
    const int tok = i / per_token, rest = i - tok * per_token;
    const int slot = rest / P.chunks, c = rest - slot * P.chunks;
    const long long bt = static_cast<long long>(blockIdx.x) * P.tokens_per_block + tok;
    if (bt >= tokens) return;
    const int b = static_cast<int>(bt / P.T), t = static_cast<int>(bt - static_cast<long long>(b) * P.T);
    const bool turn = c < P.rot_chunks;
    // the chunk's two places in a row
    const int o0 = !turn ? P.plan.rot + V * (c - P.rot_chunks) : INTER ? 2 * V * c : V * c;
    const int o1 = !turn ? o0 : INTER ? o0 + V : o0 + P.plan.rot / 2;
    const long long pos = !turn ? 0 : P.pos ? P.pos[bt] : t;
    // this token's rows of head 0, less the heads before K's for K
    const T* x[2];
    T* y[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      x[k] = static_cast<const T*>(P.x[k]) + b * P.xs[k].b + t * P.xs[k].t - (k ? P.heads[0] * P.xs[k].h : 0);
      y[k] = static_cast<T*>(P.y[k]) + b * P.ys[k].b + t * P.ys[k].t - (k ? P.heads[0] * P.ys[k].h : 0);
    }
    auto row = [&](int h) { return h < P.heads[0] ? x[0] + h * P.xs[0].h : x[1] + h * P.xs[1].h; };
    auto fetch = [&](int h, int s) {
      if constexpr (WIDE) {
        if (h < total) {
          const T* p = row(h);
          copy16(&stage[s][0][threadIdx.x], p + o0);
          if (turn) copy16(&stage[s][1][threadIdx.x], p + o1);
        }
        copy_commit();   // (an empty group past the end keeps the count)
      }
    };
    if constexpr (WIDE) {
#pragma unroll
      for (int s = 0; s < STAGES - 1; ++s) fetch(slot + s * P.slots, s);
    }
    float cs[V], sn[V];
    if (turn) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const unsigned long long turns = static_cast<unsigned long long>(pos) * P.plan.turns[V * c + e];
        const float half_turns = static_cast<float>(static_cast<int>(turns >> 32)) * 0x1p-31f;
        sincospif(half_turns, &sn[e], &cs[e]);
        sn[e] *= P.sign * P.plan.mscale;
        cs[e] *= P.plan.mscale;
      }
    }
    int s = 0;
    for (int h = slot; h < total; h += P.slots) {
      W u, v;
      if constexpr (WIDE) {
        fetch(h + (STAGES - 1) * P.slots, s == 0 ? STAGES - 1 : s - 1);   // (the slot read in the last step)
        copy_wait<STAGES - 1>();
        u = stage[s][0][threadIdx.x];
        v = stage[s][1][threadIdx.x];
        s = s == STAGES - 1 ? 0 : s + 1;
      } else {
        u = *reinterpret_cast<const W*>(row(h) + o0);
        v = *reinterpret_cast<const W*>(row(h) + o1);
      }
      T* out = h < P.heads[0] ? y[0] + h * P.ys[0].h : y[1] + h * P.ys[1].h;
      if (turn) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          // pair e of the chunk: (u_e, v_e), or elements 2e, 2e + 1 of the 2 V adjacent ones
          T& pu = INTER ? (2 * e < V ? u.e[(2 * e) % V] : v.e[(2 * e) % V]) : u.e[e];
          T& pv = INTER ? (2 * e + 1 < V ? u.e[(2 * e + 1) % V] : v.e[(2 * e + 1) % V]) : v.e[e];
          const float a = to_f(pu), w = to_f(pv);
          pu = from_f<T>(a * cs[e] - w * sn[e]);
          pv = from_f<T>(w * cs[e] + a * sn[e]);
        }
        *reinterpret_cast<W*>(out + o1) = v;
      }
      *reinterpret_cast<W*>(out + o0) = u;
    }
    if constexpr (WIDE) copy_wait<0>();
  }
}

// Sums of two doubles, x + y with |y| at most half a step of x (Dekker;
// Knuth): some 100 bits for the plan, whose entries have 64 behind the point.
struct Two {
  double x, y;
};
Two sum(double a, double b) {
  const double s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
Two operator+(Two a, Two b) {
  const Two s = sum(a.x, b.x), t = sum(a.y, b.y);
  const Two u = sum(s.x, s.y + t.x);
  return sum(u.x, u.y + t.y);
}
Two operator*(Two a, Two b) {
  const double p = a.x * b.x;
  return sum(p, fma(a.x, b.x, -p) + (a.x * b.y + a.y * b.x));
}
Two operator-(Two a) { return {-a.x, -a.y}; }
Two operator/(Two a, Two b) {
  const double q = a.x / b.x;
  const Two r = a + -(Two{q, 0.0} * b);
  return sum(q, r.x / b.x);
}

// theta^(-1/n): the double nearest to it, or nearly, corrected by one step of
// Newton's method on theta * f^n = 1.
Two root(double theta, int n) {
  const double f = pow(theta, -1.0 / n);
  Two r{theta, 0.0};
  for (int i = 0; i < n; ++i) r = r * Two{f, 0.0};
  const Two off = r + Two{-1.0, 0.0};
  return sum(f, -f * off.x / n);
}

template <typename T, int V>
cudaError_t launch(Params& P, cudaStream_t st, int num_sms) {
  const long long tokens = static_cast<long long>(P.B) * P.T;
  P.rot_chunks = P.plan.rot / 2 / V;
  P.chunks = P.rot_chunks + (P.d - P.plan.rot) / V;
  const int total = P.heads[0] + P.heads[1];
  // heads per thread: up to 8, as long as at least 1024 threads an SM are left
  int per = 8;
  while (per > 1 && tokens * P.chunks * ((total + per - 1) / per) < num_sms * 1024LL) per /= 2;
  P.slots = (total + per - 1) / per;
  const int per_token = P.slots * P.chunks;
  P.tokens_per_block = per_token >= NT ? 1 : NT / per_token;
  const long long grid = (tokens + P.tokens_per_block - 1) / P.tokens_per_block;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (P.plan.interleaved)
    rope_kernel<T, V, true><<<static_cast<unsigned>(grid), NT, 0, st>>>(P);
  else
    rope_kernel<T, V, false><<<static_cast<unsigned>(grid), NT, 0, st>>>(P);
  return cudaGetLastError();
}

}  // namespace rope
}  // namespace attn

using namespace attn;

extern "C" {

attn_status_t attn_rope_init(attn_rope_t* plan, int rot, int interleaved, double theta, double factor,
                             double original_length, double low_turns, double high_turns, double mscale) {
  if (plan == nullptr || rot < 2 || rot > 2 * ATTN_ROPE_MAX_PAIRS || rot % 2) return ATTN_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return ATTN_ERR_INVALID_ARG;
  if (!(theta > 1.0) || !isfinite(theta) || !(factor >= 1.0) || !isfinite(factor)) return ATTN_ERR_INVALID_ARG;
  if (!(original_length >= 0.0) || !isfinite(original_length)) return ATTN_ERR_INVALID_ARG;
  if (original_length > 0.0 && !(low_turns >= 0.0 && low_turns < high_turns && isfinite(high_turns)))
    return ATTN_ERR_INVALID_ARG;
  if (!(mscale > 0.0) || !isfinite(static_cast<float>(mscale)) || !(static_cast<float>(mscale) > 0.f))
    return ATTN_ERR_INVALID_ARG;
  *plan = attn_rope_t{};
  plan->rot = rot;
  plan->interleaved = interleaved;
  plan->mscale = static_cast<float>(mscale);
  // f_i = f_1^i, as turns: f_i / (2 pi)
  using rope::Two;
  const Two per_turn{0.15915494309189535, -9.839338337591243e-18};   // 1 / (2 pi)
  const Two f1 = rope::root(theta, rot / 2), one{1.0, 0.0};
  Two f = one;
  for (int i = 0; i < rot / 2; ++i, f = f * f1) {
    const Two t = f * per_turn;
    Two keep{0.0, 0.0};   // the share of f_i that is not divided by the factor
    if (original_length > 0.0) {
      keep = (Two{original_length, 0.0} * t + Two{-low_turns, 0.0}) / rope::sum(high_turns, -low_turns);
      keep = keep.x < 0.0 ? Two{0.0, 0.0} : keep.x >= 1.0 ? one : keep;
    }
    const Two g = t * keep + t / Two{factor, 0.0} * (one + -keep);
    const double units = ldexp(g.x, 64), whole = rint(units);   // below 2^62
    plan->turns[i] = static_cast<unsigned long long>(static_cast<long long>(whole) +
                                                     static_cast<long long>(rint(units - whole + ldexp(g.y, 64))));
  }
  return ATTN_OK;
}

attn_status_t attn_rope(const attn_rope_t* plan, const void* Q, void* Qout, const void* K, void* Kout,
                        const long long* strides, const int* pos, int B, int H, int Hkv, int T, int d, int inverse,
                        attn_dtype_t dtype, void* stream) {
  if (plan == nullptr || strides == nullptr || B < 0 || H < 0 || Hkv < 0 || T < 0 || d <= 0)
    return ATTN_ERR_INVALID_ARG;
  if (inverse != 0 && inverse != 1) return ATTN_ERR_INVALID_ARG;
  if (dtype != ATTN_F32 && dtype != ATTN_BF16) return ATTN_ERR_INVALID_ARG;
  if (plan->rot < 2 || plan->rot % 2 || plan->rot > d || (plan->interleaved != 0 && plan->interleaved != 1))
    return ATTN_ERR_INVALID_ARG;
  if (d > 2 * ATTN_ROPE_MAX_PAIRS) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(H) + Hkv > 0x7fffffff / 256) return ATTN_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(pos) % 4) return ATTN_ERR_MISALIGNED;
  const size_t es = elem_size(dtype);
  const void* in[2] = {Q, K};
  void* out[2] = {Qout, Kout};
  const int heads[2] = {H, Hkv};
  const bool some = B > 0 && T > 0;
  rope::Params P{};
  bool wide = true;   // 16-byte accesses everywhere
  const int V = 16 / static_cast<int>(es);
  Rows from[2], to[2];
  for (int k = 0; k < 2; ++k) {
    const long long* s = strides + 6 * k;
    P.xs[k] = View{s[0], s[1], s[2]};
    P.ys[k] = View{s[3], s[4], s[5]};
    P.heads[k] = some ? heads[k] : 0;
    if (P.heads[k] == 0) continue;
    for (int i = 0; i < 6; ++i) {
      if (s[i] < 0 || s[i] > (1LL << 50)) return ATTN_ERR_INVALID_ARG;
      wide = wide && s[i] % V == 0;
    }
    for (const void* p : {in[k], static_cast<const void*>(out[k])}) {
      if (p == nullptr) return ATTN_ERR_INVALID_ARG;
      if (reinterpret_cast<uintptr_t>(p) % es) return ATTN_ERR_MISALIGNED;
      wide = wide && reinterpret_cast<uintptr_t>(p) % 16 == 0;
    }
    if (static_cast<double>(s[0]) * B + static_cast<double>(s[1]) * heads[k] + static_cast<double>(s[2]) * T > 9e15 ||
        static_cast<double>(s[3]) * B + static_cast<double>(s[4]) * heads[k] + static_cast<double>(s[5]) * T > 9e15)
      return ATTN_ERR_INVALID_ARG;
    from[k] = rows_of(in[k], P.xs[k], B, heads[k], T, d, es);
    to[k] = rows_of(out[k], P.ys[k], B, heads[k], T, d, es);
    if (!distinct(to[k])) return ATTN_ERR_INVALID_ARG;
    P.x[k] = in[k];
    P.y[k] = out[k];
  }
  for (int k = 0; k < 2; ++k) {   // output k against the inputs and the other output
    if (P.heads[k] == 0) continue;
    for (int j = 0; j < 2; ++j) {
      if (P.heads[j] == 0) continue;
      // in place: the same rows (a stride of a single row does not count)
      bool in_place = j == k && in[k] == out[k];
      for (int i = 0; i < 3; ++i) in_place = in_place && (to[k].n[i] <= 1 || to[k].step[i] == from[k].step[i]);
      if (!in_place && !apart(to[k], from[j])) return ATTN_ERR_INVALID_ARG;
      if (j > k && !apart(to[k], to[j])) return ATTN_ERR_INVALID_ARG;
    }
    if (pos && !apart(to[k], Rows{reinterpret_cast<uintptr_t>(pos), 4LL * B * T, {}, {}})) return ATTN_ERR_INVALID_ARG;
  }
  if (!some || (H == 0 && Hkv == 0)) return ATTN_OK;
  DeviceInfo* di;
  attn_status_t s = device_info(&di);
  if (s != ATTN_OK) return s;
  P.plan = *plan;
  P.pos = pos;
  P.B = B;
  P.T = T;
  P.d = d;
  P.sign = inverse ? -1.f : 1.f;
  wide = wide && (plan->rot / 2) % V == 0 && (d - plan->rot) % V == 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == ATTN_BF16)
    e = wide ? rope::launch<__nv_bfloat16, 8>(P, st, di->num_sms) : rope::launch<__nv_bfloat16, 1>(P, st, di->num_sms);
  else
    e = wide ? rope::launch<float, 4>(P, st, di->num_sms) : rope::launch<float, 1>(P, st, di->num_sms);
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
}

}  // extern "C"
