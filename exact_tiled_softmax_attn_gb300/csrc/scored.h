// Internal interface of the scored attention (include/attn.h, attn_fwd_scored
// and attn_bwd_scored) between its C-ABI layer and its kernels.
//
// The query heads that share a key head are adjacent in memory, so their rows
// form one packed list of R = G * Tq rows per key head (G = H / Hkv): Q is
// [B * Hkv, R, d] and row r belongs to query head hkv * G + r / Tq at token
// r % Tq. Every kernel works on packed rows. Heads that share keys then also
// share key tiles, and the sums of dK and dV over a group are sums over rows.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace attn {

constexpr int kScoredTile = 128;   // rows of the plan's row tiles, keys of its key tiles

struct ScoredProblem {
  int B, Hkv, G, Tq, Tk, d, dv;
  int R;         // packed query rows of a key head: G * Tq
  int n_rt;      // 128-row tiles of R
  int n_kt;      // 128-key tiles of Tk
  int kv_splits;   // dK/dV: parts the row tiles of a key tile are cut into, as units of their own
  int kv_split_tiles;   // row tiles of a part
  float scale;
  float softcap;          // 0: none
  const float* slopes;    // [H] or null
  __host__ __device__ int n_words() const { return (n_rt + 31) / 32; }   // of a bit list of row tiles
  __host__ __device__ int rpad() const { return n_rt * kScoredTile; }
};

// What the plan kernel makes of the ranges of a call (all in the workspace).
struct ScoredPlan {
  int4* rows;      // [B][rpad]: {key begin, key end, position, 0}; begin = INT_MAX, end = 0 for rows that see nothing
  int4* tiles;     // [B][n_rt]: {min begin, max end over the rows that see keys, max begin, min end over all rows}
  int2* fine;      // [B][rpad / 32]: {min begin, max end} of 32 rows, (0, 0) where none sees a key (fp32 only), or null
  int* kcount;     // [B][n_kt][kv_splits]: row tiles of the part whose hull meets the key tile (backward only), or null
  int4* khull;     // [B][n_kt]: hull of the row tiles that meet the key tile, whether a row of theirs sees no key, 0; or null
  uint32_t* kbits; // [B][n_kt][n_words]: which they are, one bit each
  int4* even;      // [B][n_rt]: in .x, the position of a row tile's first row where its rows are of one head and at
                   // consecutive positions, else kScoredUneven (backward with a bias only), or null
  float* slope2;   // [Hkv][rpad]: slope * log2(e) of each packed row (backward with a bias only), or null
  uint32_t* counters;   // two unit counters, zeroed
};

constexpr int kScoredUneven = -0x7fffffff;

struct ScoredMask {   // the caller's arrays
  const int* q_pos;
  const int* key_begin;
  const int* key_end;
  int causal;
};

// Results of what has nothing to do, which the tensor-core kernels leave out
// (bf16; null pointers: none): rows of row tiles that see no key, and keys of
// key tiles that no row sees.
struct ScoredIdle {
  void* O;
  float* LSE;
  void* dQ;
  float* D;
  float* NL;
  void* dK;   // (with one part; the sum of several leaves empty ones out)
  void* dV;
};

cudaError_t launch_scored_plan(const ScoredProblem& p, const ScoredMask& m, const ScoredPlan& plan,
                               const ScoredIdle& idle, cudaStream_t s);

struct ScoredFwd {
  ScoredProblem p;
  ScoredPlan plan;
  ScoredMask mask;
  const void* Q;
  const void* K;
  const void* V;
  void* O;
  float* LSE;
  int* start;         // few-row kernel: [B + 1]
  int grid;           // few-row kernel: its CTAs
  int n_splits;       // key ranges of split_keys keys (a multiple of 128) each, as units of their own
  int split_keys;
  float* Opart;       // [n_splits][B * Hkv * R][dv] fp32, n_splits > 1
  float* LSEpart;     // [n_splits][B * Hkv * R]
  const CUtensorMap* tmQ;   // bf16 only
  const CUtensorMap* tmK;
  const CUtensorMap* tmV;
  uint32_t* status;
  int num_sms;
  size_t l2_bytes;
  cudaStream_t stream;
};

struct ScoredBwd {
  ScoredProblem p;
  ScoredPlan plan;
  const void* Q;
  const void* K;
  const void* V;
  const void* O;
  const float* LSE;
  const void* dO;
  void* dQ;
  void* dK;
  void* dV;
  float* D;         // [B * Hkv][rpad]: rowsum(dO o O), 0 behind row R
  float* dKpart;    // [kv_splits][B * Hkv * Tk][d] fp32, kv_splits > 1
  float* dVpart;    // [kv_splits][B * Hkv * Tk][dv]
  float* NL;        // [B * Hkv][rpad]: -LSE * log2(e), -inf for rows that see nothing and behind row R
  const CUtensorMap* tmQ;   // bf16 only
  const CUtensorMap* tmK;
  const CUtensorMap* tmV;
  const CUtensorMap* tmdO;
  const CUtensorMap* tmO;
  uint32_t* status;
  int num_sms;
  size_t l2_bytes;
  cudaStream_t stream;
};

// CUDA cores (fp32 problems)
cudaError_t launch_scored_fwd_simt(const ScoredFwd& a);
cudaError_t launch_scored_bwd_simt(const ScoredBwd& a);

// bf16 on the tensor cores; tmQ, tmK, tmV with 128-row boxes
cudaError_t launch_scored_fwd_bf16(const ScoredFwd& a);
// bf16, at most 32 packed rows a key head; tmK, tmV with 64-row boxes
constexpr int kScoredTokenRows = 32;
cudaError_t launch_scored_tokens_bf16(const ScoredFwd& a);
cudaError_t launch_scored_bwd_bf16(const ScoredBwd& a);

// dK and dV from the parts of their row tiles, in order
cudaError_t launch_scored_kv_sum(const ScoredBwd& a, bool bf16);

// O and LSE from the partial results of the key ranges, in range order
cudaError_t launch_scored_merge(const ScoredFwd& a, bool bf16);

}  // namespace attn
