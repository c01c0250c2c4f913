// Arithmetic of the scored attention shared by its tensor-core kernels: the
// tanh cap and the launch-wide constants of the changed scores, all in log2
// units (scores times log2(e)), as the exponentials take them.
#pragma once

#include <stdint.h>

#include "ptx.cuh"
#include "scored.h"

namespace attn {
namespace scored {

constexpr float kLog2e = 1.4426950408889634f;

// y = cap2 * tanh(k s), s the raw product q.k, k = scale / softcap, cap2 =
// softcap * log2(e). For |k s| <= kPolyMax: s times a polynomial in s^2 with
// k and cap2 in its coefficients. tanh(x) / x is fitted by a degree-4
// polynomial in x^2 on |x| <= 0.6 (least squares with Lawson's reweighting);
// |x * poly - tanh(x)| <= 2.0e-8, 8e-8 as evaluated in fp32, the size of
// fp32's own rounding there. It costs 6 two-lane FMA-pipe instructions per
// pair of scores, against 2 special-function instructions a score for the
// formula 1 - 2 / (1 + e^(2x)) that every other |x| takes. Scores of a
// trained layer lie well inside the cap, so nearly all tiles take the first.
struct Cap {
  float k2;        // 2 k log2(e): e^(2 k s) = 2^(k2 s)
  float cap2;      // softcap * log2(e)
  float ninv2;     // -1 / cap2^2
  float limit;     // kPolyMax / k, or -1 where k^8 leaves fp32's range
  float c[5];      // polynomial in s^2
};

constexpr float kPolyMax = 0.6f;

inline Cap make_cap(float scale, float softcap) {
  Cap r{};
  if (!(softcap > 0.f)) return r;
  const double c[5] = {0.9999996274092242, -0.333312085910721, 0.13299210221337304, -0.05169674295522158,
                       0.014976960081731636};
  const double k = static_cast<double>(scale) / softcap, cap2 = softcap * 1.4426950408889634;
  const double k2 = 2.0 * k * 1.4426950408889634;
  r.k2 = k2 < 1e30 ? static_cast<float>(k2) : 1e30f;   // (any score but 0 is at the cap there)
  r.cap2 = static_cast<float>(cap2);
  r.ninv2 = static_cast<float>(-1.0 / (cap2 * cap2));
  const double k8 = k * k * k * k * k * k * k * k;
  r.limit = k8 > 1e-30 && k8 < 1e30 ? static_cast<float>(kPolyMax / k) : -1.f;
  double kk = k * cap2;
  for (int i = 0; i < 5; ++i, kk *= k * k) r.c[i] = static_cast<float>(c[i] * kk);
  return r;
}

constexpr int kPosLimit = 1 << 30;

// The keys [lo, hi) token t of batch entry b sees (lo >= hi: none) and its position.
__device__ __forceinline__ void row_range(const ScoredProblem& p, const ScoredMask& m, int b, int t, int* lo, int* hi,
                                          int* pos) {
  const long long at = static_cast<long long>(b) * p.Tq + t;
  *pos = m.q_pos ? min(max(__ldg(m.q_pos + at), -kPosLimit), kPosLimit) : t;
  *lo = m.key_begin ? max(__ldg(m.key_begin + at), 0) : 0;
  *hi = m.key_end ? min(__ldg(m.key_end + at), p.Tk) : p.Tk;
  if (m.causal) *hi = min(*hi, *pos + 1);
}

// Two fp32 lanes (ptx::ffma2 and its kin).
using F2 = float2;
__device__ __forceinline__ F2 f2(float x, float y) { return make_float2(x, y); }
__device__ __forceinline__ F2 dup(float x) { return make_float2(x, x); }
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) { return ptx::ffma2(a, b, c); }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) { return ptx::fmul2(a, b); }
__device__ __forceinline__ F2 add2(F2 a, F2 b) { return ptx::fadd2(a, b); }
__device__ __forceinline__ F2 ex2(F2 a) {
  return f2(ptx::ex2(a.x), ptx::ex2(a.y));
}
__device__ __forceinline__ uint32_t pack_bf16(F2 a) {
  return ptx::pack_bf16(a.x, a.y);
}

// The polynomial's value at a pair of scores, the factor of s. Its
// coefficients are held as register pairs: read as constants they cost two
// moves per use, more than the arithmetic (1629 instructions per 128 x 32
// scores, 600 of them moves, before).
struct CapPoly {
  F2 c0, c1, c2, c3, c4;
  __device__ __forceinline__ explicit CapPoly(const Cap& c)
      : c0(pin(c.c[0])), c1(pin(c.c[1])), c2(pin(c.c[2])), c3(pin(c.c[3])), c4(pin(c.c[4])) {}
  static __device__ __forceinline__ F2 pin(float x) {
    F2 r;
    asm volatile("mov.b32 %0, %2;\n\tmov.b32 %1, %2;" : "=f"(r.x), "=f"(r.y) : "f"(x));
    return r;
  }
  __device__ __forceinline__ F2 operator()(F2 s) const {
    const F2 u = mul2(s, s);
    F2 g = fma2(c4, u, c3);
    g = fma2(g, u, c2);
    g = fma2(g, u, c1);
    return fma2(g, u, c0);
  }
};

// Bits [lo, hi) of a word, both any integers.
__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {
  const int a = max(lo, 0), b = min(hi, 32);
  if (b <= a) return 0u;
  return (b == 32 ? 0xffffffffu : (1u << b) - 1u) & ~((1u << a) - 1u);
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// cap2 * tanh(k s) for any s: -cap2 and cap2 at the infinities.
__device__ __forceinline__ float cap_any(float s, const Cap& c) {
  return fmaf(-2.f * c.cap2, rcp_approx(1.f + ptx::ex2(s * c.k2)), c.cap2);
}
__device__ __forceinline__ F2 cap_any(F2 s, const Cap& c) {
  return f2(cap_any(s.x, c), cap_any(s.y, c));
}

}  // namespace scored
}  // namespace attn
