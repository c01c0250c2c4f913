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
// softcap * log2(e). Three forms, chosen per warp and tile by the largest
// |k s|: s times a polynomial in s^2 that has k and cap2 in its coefficients,
// of degree 2 up to 0.25 and of degree 4 up to 0.6, and beyond cap_any, which
// chooses per score: that polynomial of degree 4 in (k s)^2 up to 0.6, else
// the formula 1 - 2 / (1 + e^(2x)). The formula alone would be off by a few
// 2^-24 of the cap, whatever the score: 0.1 at a cap of 10^6. A form is left
// out where a coefficient of it leaves fp32's range (degree 4 from a cap of
// about 2000 on at d = 128; degree 2 only for scales far from 1/sqrt(d)). The
// polynomials are fits of tanh(x) / x in x^2 (least squares with Lawson's
// reweighting) in the relative error, 4.0e-7 and 7.4e-8 at most, which is what
// scores far inside the cap need. Per pair of scores they cost 4 and 6
// two-lane FMA-pipe instructions (2 issue cycles each); the formula costs 2
// special-function instructions a score more than the uncapped exponential.
// Scores of a trained layer lie well inside the cap.
constexpr float kCapLimit2 = 0.25f, kCapLimit4 = 0.6f;
constexpr double kCapPoly2Fit[3] = {0.9999996043350667, -0.33321908145397344, 0.12841612166110375};
constexpr double kCapPoly4Fit[5] = {0.9999999268660169, -0.3333230996151517, 0.13310173509714307,
                                    -0.05210147391716534, 0.015475418969482619};
struct Cap {
  float k;         // scale / softcap
  float cap2;      // softcap * log2(e)
  float ninv2;     // -1 / cap2^2
  float limit2;    // |s| up to which the polynomial of degree 2 holds, or -1
  float limit4;    // and that of degree 4
  float c2[3];     // polynomials in s^2
  float c4[5];
  float n4[5];     // that of degree 4 in (k s)^2
};

inline Cap make_cap(float scale, float softcap) {
  Cap r{};
  if (!(softcap > 0.f)) return r;
  constexpr double kLeast = 1.2e-38, kMost = 1e38;   // within fp32's normal numbers
  const double k = static_cast<double>(scale) / softcap, cap2 = softcap * 1.4426950408889634;
  const double sc2 = scale * 1.4426950408889634;
  r.k = k < 1e30 ? static_cast<float>(k) : 1e30f;   // (any score but 0 is at the cap there)
  r.cap2 = static_cast<float>(cap2);
  r.ninv2 = static_cast<float>(-1.0 / (cap2 * cap2));
  bool fits2 = kCapLimit2 < k * 1e19, fits4 = kCapLimit4 < k * 1e19;   // (s^2 within range)
  double p = sc2;
  for (int i = 0; i < 5; ++i, p *= k * k) {
    const double a4 = kCapPoly4Fit[i] * p, size4 = a4 < 0 ? -a4 : a4;
    fits4 = fits4 && size4 > kLeast && size4 < kMost;
    r.c4[i] = static_cast<float>(a4);
    const double n4 = kCapPoly4Fit[i] * sc2;
    r.n4[i] = static_cast<float>(n4 > kMost ? kMost : n4 < -kMost ? -kMost : n4);
    if (i > 2) continue;
    const double a2 = kCapPoly2Fit[i] * p, size2 = a2 < 0 ? -a2 : a2;
    fits2 = fits2 && size2 > kLeast && size2 < kMost;
    r.c2[i] = static_cast<float>(a2);
  }
  r.limit2 = fits2 ? static_cast<float>(kCapLimit2 / k) : -1.f;
  r.limit4 = fits4 ? static_cast<float>(kCapLimit4 / k) : r.limit2;
  if (!fits4)   // where a kernel takes degree 4 for degree 2's range
    for (int i = 0; i < 5; ++i) r.c4[i] = i < 3 ? r.c2[i] : 0.f;
  return r;
}

// Which form a warp takes for scores within [lo, hi] (of this thread; NaN, of
// a thread whose scores are all NaN, goes through any).
enum { kCapPoly2 = 1, kCapPoly4 = 2, kCapFormula = 3 };
__device__ __forceinline__ int cap_form(const Cap& c, float lo, float hi) {
  const float a = fmaxf(hi, -lo);
  if (__all_sync(0xffffffffu, !(a > c.limit2))) return kCapPoly2;
  return __all_sync(0xffffffffu, !(a > c.limit4)) ? kCapPoly4 : kCapFormula;
}

// The order of a key head's blocks of packed rows (or pairs of row tiles): a
// block's length under a causal mask goes by its place within its query head,
// so the blocks at one place of all G heads follow one another, and a
// sequence that runs backwards over the numbers gives the longest first. The
// last head may lack a place: blocks past the last one have nothing to do.
__host__ __device__ __forceinline__ int packed_blocks(int n, int G) { return (n + G - 1) / G * G; }
__device__ __forceinline__ int packed_block(int i, int n_padded, int G) {
  const int per = n_padded / G;
  return (i % G) * per + i / G;
}

// A descriptor that exists from here on: the compiler would otherwise form it
// behind the wait before the product that uses it, where its latency counts.
__device__ __forceinline__ uint64_t formed(uint64_t desc) {
  asm volatile("" : "+l"(desc));
  return desc;
}

// Zeroes row r of a swizzled box of 64 bf16 columns in shared memory. The
// swizzle moves 16-byte pieces within a row only; taken in its order, eight
// rows' pieces are in different banks.
__device__ __forceinline__ void zero_box_row(uint8_t* box, int r) {
  uint4* p = reinterpret_cast<uint4*>(box + r * 128);
#pragma unroll
  for (int e = 0; e < 8; ++e) p[e ^ (r & 7)] = make_uint4(0u, 0u, 0u, 0u);
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

// A polynomial's value at a pair of scores, the factor of s. Its coefficients
// are held as register pairs from the construction on: read as constants they
// cost two moves per use, more than the arithmetic (1629 instructions per 128
// x 32 scores, 600 of them moves). Constructed where a tile's form is known,
// they are live no longer than needed.
__device__ __forceinline__ F2 pin(float x) {
  F2 r;
  asm volatile("mov.b32 %0, %2;\n\tmov.b32 %1, %2;" : "=f"(r.x), "=f"(r.y) : "f"(x));
  return r;
}
template <int FORM>
struct CapPoly {
  static constexpr int N = FORM == kCapPoly2 ? 3 : 5;
  F2 c[N];
  __device__ __forceinline__ explicit CapPoly(const Cap& cap) {
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = pin(FORM == kCapPoly2 ? cap.c2[i % 3] : cap.c4[i]);
  }
  __device__ __forceinline__ F2 operator()(F2 s) const {
    const F2 u = mul2(s, s);
    F2 g = fma2(c[N - 1], u, c[N - 2]);
#pragma unroll
    for (int i = N - 3; i >= 0; --i) g = fma2(g, u, c[i]);
    return g;
  }
};

// Piece i of lane q's four 16-byte pieces of its row for piece q of row i of
// its quad: rows of a warp, one per lane, then go to memory as 64 contiguous
// bytes per row and instruction. As 16 bytes per row, 32 rows at a time, the
// stores took a 128-row tile of 256-byte rows about 5000 cycles.
__device__ __forceinline__ void quad_transpose(uint4 (&v)[4], int lane) {
#pragma unroll
  for (int step = 1; step <= 2; step *= 2) {
    const bool up = lane & step;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & step) continue;
      uint32_t* a = reinterpret_cast<uint32_t*>(&v[i]);
      uint32_t* b = reinterpret_cast<uint32_t*>(&v[i + step]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {   // the piece that belongs to the other lane crosses over
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? a[e] : b[e], step);
        if (up) a[e] = got; else b[e] = got;
      }
    }
  }
}

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

// cap2 * tanh(k s) to within a few 2^-24 of cap2: enough for the references
// that exponentials and sums share.
__device__ __forceinline__ float cap_rough(float s, const Cap& c) {
  return fmaf(-2.f * c.cap2, rcp_approx(1.f + ptx::ex2(s * c.k * (2.f * kLog2e))), c.cap2);
}
// cap2 * tanh(k s) for any s: -cap2 and cap2 at the infinities. (Two-lane FMAs
// would hold the coefficients in registers, and the kernels' frequent forms
// would spill for it: 569 in place of 560 us for a training step of B=2 H=16
// T=4096 d=128 whose scores stay far inside the cap.)
__device__ __forceinline__ float cap_any(float s, const Cap& c) {
  const float x = s * c.k, u = x * x;
  float g = fmaf(c.n4[4], u, c.n4[3]);
#pragma unroll
  for (int i = 2; i >= 0; --i) g = fmaf(g, u, c.n4[i]);
  const float far = fmaf(-2.f * c.cap2, rcp_approx(1.f + ptx::ex2(x * (2.f * kLog2e))), c.cap2);
  return fabsf(x) <= kCapLimit4 ? s * g : far;
}
__device__ __forceinline__ F2 cap_any(F2 s, const Cap& c) { return f2(cap_any(s.x, c), cap_any(s.y, c)); }

}  // namespace scored
}  // namespace attn
