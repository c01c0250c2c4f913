// Internal interface of the paged key-value cache (include/attn.h, attn_cache_t)
// between its C-ABI layer and its kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "rope.cuh"
#include "scored.h"

namespace attn {

constexpr float kCodeMost = 448.f;                              // the largest e4m3 value
constexpr int kScaleLeast = -40, kScaleMost = 40;               // exponents of scales
constexpr float kTurned = 1.4142137f;   // a little over sqrt(2): |u cos a - v sin a| <= sqrt(2) max(|u|, |v|)

struct CacheView {
  void* pool[2];       // K, V
  float* scale[2];     // e4m3
  const int* table;
  const int* seq_len;
  const int* new_len;
  int pages, shift, max_pages;   // page = 1 << shift tokens
  bool codes;
};

namespace cache {

constexpr int kMostTokens = rope::kMostTokens;

#ifdef __CUDACC__
// An element of the call's arrays, by an ordinary load, as all that is read by
// kernels launched over the end of the kernel before: that may write lengths,
// table, scales, ranges or rows while they are resident, and a load through the
// read-only path is right only for what nobody writes in a kernel's life.
// (volatile: not moved before the wait for that kernel, and not made twice.)
__device__ __forceinline__ int load(const int* p) {
  int r;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(r) : "l"(p));
  return r;
}

// Tokens of sequence b, and how many of them are the call's new ones (of T at most).
__device__ __forceinline__ int tokens_of(const CacheView& c, int b) {
  return min(max(load(c.seq_len + b), 0), kMostTokens);
}
__device__ __forceinline__ int new_of(const CacheView& c, int b, int T) {
  return c.new_len ? min(max(load(c.new_len + b), 0), T) : T;
}
// The page that holds tokens [i * page, (i + 1) * page) of sequence b, or -1.
__device__ __forceinline__ int page_of(const CacheView& c, int b, int i) {
  if (i < 0 || i >= c.max_pages) return -1;
  const int at = load(c.table + static_cast<long long>(b) * c.max_pages + i);
  return at >= 0 && at < c.pages ? at : -1;
}
// (a NaN reads as the least)
__device__ __forceinline__ float clamp_scale(float s) { return fminf(fmaxf(s, 0x1p-40f), 0x1p40f); }

// The keys [lo, hi) (lo >= hi: none) that row t of a call sees, and its
// position; at: its place in the caller's arrays; of a sequence of len tokens,
// the last n of them new.
__device__ __forceinline__ void row_range(const ScoredMask& m, long long at, int t, int len, int n, int Tk, int window,
                                          int* lo, int* hi, int* pos) {
  *pos = m.q_pos ? min(max(load(m.q_pos + at), -kMostTokens), kMostTokens) : len - n + t;
  *lo = m.key_begin ? max(load(m.key_begin + at), 0) : 0;
  *hi = min(m.key_end ? load(m.key_end + at) : len, min(len, Tk));
  if (m.causal) *hi = min(*hi, *pos + 1);
  if (window > 0) *lo = max(*lo, *pos - window + 1);
  *hi = t < n ? max(*hi, 0) : 0;   // (an end far below 0 less a key would wrap around)
}

// Two e4m3 codes as fp16 (exact), and two fp32 numbers as codes: to the
// nearest, 448 beyond it; NaN stays.
__device__ __forceinline__ uint32_t codes_to_half2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
__device__ __forceinline__ float2 half2_to_float2(uint32_t h) {
  float2 r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(h));
  return r;
}
__device__ __forceinline__ uint16_t float2_to_codes(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
#endif

}  // namespace cache

// Gives a kernel `bytes` of dynamic shared memory on the current device, once:
// the call costs the host 1 to 3 us. `done`: the kernel's own, a bit per device.
template <typename K>
cudaError_t allow_smem(K kern, int bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Launches a kernel over the end of the one before it in the stream: it waits
// by ptx::grid_wait() before it touches memory. In clusters of `cluster` CTAs.
template <typename K, typename... A>
cudaError_t launch_clusters(K kern, unsigned cluster, unsigned grid, unsigned threads, size_t smem, cudaStream_t stream,
                            const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = threads;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}
template <typename K, typename... A>
cudaError_t launch_over(K kern, unsigned grid, unsigned threads, size_t smem, cudaStream_t stream, const A&... args) {
  return launch_clusters(kern, 1u, grid, threads, smem, stream, args...);
}

struct CacheAppend {
  CacheView c;
  rope::Params q;      // the queries' rotation; heads[0] == 0: none
  bool turn;           // rotate the keys by q.plan
  const void* x[2];    // K, V
  View s[2];
  const int* pos;
  int B, Hkv, T, w[2];   // w: d, dv
  bool wide;             // 16-byte accesses of the queries, K and V
  bool bf16;
  int num_sms;
  cudaStream_t stream;
};
cudaError_t launch_cache_append(const CacheAppend& a);

// Units of the append: (sequence, touched page, head, side).
long long cache_append_units(int B, int Hkv, int T, int shift);

struct CacheRead {
  CacheView c;
  void* out[2];        // K, V: [B, Hkv, Tk, w]
  int B, Hkv, Tk, w[2];
  bool bf16;
  const int2* hull;    // [B]: read only these tokens and write no others; null: all of [0, Tk), zeros behind the last
  int num_sms;
  cudaStream_t stream;
};
cudaError_t launch_cache_read(const CacheRead& a);

// The rows' ranges and positions as attn_score_t's arrays [B, Tq], and the
// hull of each sequence's ranges, in which it sees keys.
struct CacheRows {
  CacheView c;
  ScoredMask mask;
  int B, Tq, Tk, window;
  int* q_pos;
  int* key_begin;
  int* key_end;
  int2* hull;
  cudaStream_t stream;
};
cudaError_t launch_cache_rows(const CacheRows& a);

// Attention of few rows, which reads the pages where they lie: bf16 over any
// pages, fp32 over e4m3; tmK, tmV by make_map_bytes.
constexpr int kCacheTokenRows = 128;   // packed rows of a key head, at most
inline int cache_token_rows(int R) { return R <= 8 ? 8 : R <= 16 ? 16 : 32; }   // of a group
// CTAs of an SM, by the rows of a group: as many as registers and shared memory hold.
constexpr int cache_token_ctas(int rows, bool codes) { return rows == 32 ? 1 : rows == 8 && codes ? 3 : 2; }
inline int cache_token_groups(int R) { return (R + cache_token_rows(R) - 1) / cache_token_rows(R); }
struct CacheTokens {
  CacheView c;
  ScoredProblem p;
  ScoredMask mask;
  int window;
  const void* Q;
  void* O;
  float* LSE;
  bool f32;
  int grid;          // CTAs
  int groups;        // row groups of a key head
  int direct;        // not 0: so many CTAs, a cluster, per sequence, row group and key head
  int* start;        // [B * groups + 1]
  float* Opart;      // [grid][2][rows of a group][dv]
  float* LSEpart;    // [grid][2][rows of a group]
  const CUtensorMap* tmK;
  const CUtensorMap* tmV;
  uint32_t* status;
  cudaStream_t stream;
};
cudaError_t launch_cache_tokens(const CacheTokens& a);
// The same in tiles of 128 rows on tcgen05: bf16 over e4m3 (no tensor maps).
constexpr int kCacheTileRows = 128;
cudaError_t launch_cache_tiles(const CacheTokens& a);

}  // namespace attn
