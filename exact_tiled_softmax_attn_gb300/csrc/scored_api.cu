// C-ABI layer of the scored attention: argument validation, workspace
// layout and dispatch.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attn.h"
#include "host.h"
#include "launch.h"
#include "scored.h"

namespace attn {
namespace {

constexpr int kMaxRows = 1 << 30;
// Workspace sizes are rules of the shapes alone, so counts that aim at
// filling the GPU use GB300's SM count.
constexpr int kSms = 152;

attn_status_t check_scored(int B, int H, int Hkv, int Tq, int Tk, int d, int dv, attn_dtype_t dt) {
  if (B < 0 || H < 0 || Tq < 0 || Tk < 0 || d <= 0 || dv <= 0) return ATTN_ERR_INVALID_ARG;
  if (Hkv < 1 || H % Hkv) return ATTN_ERR_INVALID_ARG;
  if (dt != ATTN_F32 && dt != ATTN_BF16) return ATTN_ERR_INVALID_ARG;
  if (Tq > kMaxRows || Tk > kMaxRows || static_cast<long long>(H / Hkv) * Tq > kMaxRows) return ATTN_ERR_INVALID_ARG;
  // work units (32-row or 32-key tiles of every head) are counted in int
  const double heads = static_cast<double>(B) * Hkv;
  const double rows = static_cast<double>(H / Hkv) * Tq;
  // (and 128-row tiles with a place for every query head)
  if (heads * ((rows > Tk ? rows : Tk) / 32.0 + 2.0 + H / Hkv) > 2147483647.0 || heads * rows > 2147483647.0)
    return ATTN_ERR_INVALID_ARG;
  if (d > 128 || dv > 128) return ATTN_ERR_UNSUPPORTED;
  if (dt == ATTN_BF16 && (d % 8 || dv % 8)) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

attn_status_t check_score(const attn_score_t& sc, float scale) {
  if (!(scale > 0.f) || !isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if (sc.softcap != 0.f && !(sc.softcap >= 1e-4f && sc.softcap <= 1e6f)) return ATTN_ERR_INVALID_ARG;
  if (sc.causal != 0 && sc.causal != 1) return ATTN_ERR_INVALID_ARG;
  for (const void* x : {static_cast<const void*>(sc.slopes), static_cast<const void*>(sc.q_pos),
                        static_cast<const void*>(sc.key_begin), static_cast<const void*>(sc.key_end)})
    if (reinterpret_cast<uintptr_t>(x) % 4) return ATTN_ERR_MISALIGNED;
  return ATTN_OK;
}

// Parts of the row tiles of each key tile in the dK/dV kernel. A key head's
// query heads are all in one list of row tiles, so few key heads or keys mean
// few units with long lists: they are cut so that there are about two units
// per SM (fp32: four, of its 32-key tiles), at least four row tiles each, at
// most 16 parts. B=1 Hkv=1 H=8 T=4096 d=128 (32 key tiles, 10 parts each): the
// backward pass takes 129 us in place of 442; B=2 H=16 Hkv=2 T=4096: 370, 533.
void kv_split(ScoredProblem* p, attn_dtype_t dt) {
  const long long heads = static_cast<long long>(p->B) * p->Hkv;
  const long long units = dt == ATTN_BF16 ? heads * p->n_kt : heads * ((p->Tk + 31) / 32);
  const long long target = dt == ATTN_BF16 ? 2 * kSms : 4 * kSms;
  long long S = units > 0 ? (target + units - 1) / units : 1;
  if (S > p->n_rt / 4) S = p->n_rt / 4;
  if (S > 16) S = 16;
  if (S < 1) S = 1;
  p->kv_split_tiles = p->n_rt > 0 ? (p->n_rt + static_cast<int>(S) - 1) / static_cast<int>(S) : 1;
  p->kv_splits = p->n_rt > 0 ? (p->n_rt + p->kv_split_tiles - 1) / p->kv_split_tiles : 1;
}

ScoredProblem problem(int B, int H, int Hkv, int Tq, int Tk, int d, int dv, attn_dtype_t dt) {
  ScoredProblem p{};
  p.B = B;
  p.Hkv = Hkv;
  p.G = H / Hkv;
  p.Tq = Tq;
  p.Tk = Tk;
  p.d = d;
  p.dv = dv;
  p.R = p.G * Tq;
  p.n_rt = (p.R + kScoredTile - 1) / kScoredTile;
  p.n_kt = (Tk + kScoredTile - 1) / kScoredTile;
  kv_split(&p, dt);
  return p;
}

// Key ranges of the forward, for problems with few units: the fp32 kernel
// runs about four 32-row tiles per SM at a time, the tensor-core kernel one
// pair of 128-row tiles, and splits only where the pairs do not fill the SMs.
// B=1 H=4 Hkv=2, 300 rows against 8192 keys, d=128: 23.5 us with the plan and
// the merge; its six pairs alone would keep six of 152 SMs at work.
void fwd_splits(const ScoredProblem& p, attn_dtype_t dt, int* S, int* keys) {
  const long long heads = static_cast<long long>(p.B) * p.Hkv;
  int want = 1;
  if (dt == ATTN_F32)
    want = wave_splits(heads * ((p.R + 31) / 32), p.n_kt, 4 * kSms);
  else if (heads * ((p.R + 255) / 256) < kSms)
    want = wave_splits(heads * ((p.R + 255) / 256), p.n_kt, kSms);
  const int tiles = want > 1 ? (p.n_kt + want - 1) / want : p.n_kt;
  *S = want > 1 ? (p.n_kt + tiles - 1) / tiles : 1;
  *keys = tiles * kScoredTile;
}

// bf16 with at most 32 packed rows per key head: the few-row kernel, which
// streams the keys with every SM; more rows go to the 128-row tcgen05 tiles.
// 32 rows of B=8 Hkv=8 Tk=16384: 105 us against 110 at d=128 and 76 against 88
// at d=64 (at B=32 Tk=4096 d=128, 110 against 100); 16 rows: 87 and 52.
bool fwd_tokens(const ScoredProblem& p, attn_dtype_t dt) { return dt == ATTN_BF16 && p.R <= kScoredTokenRows; }

struct Layout {
  size_t start, rows, tiles, fine, counters, kcount, khull, kbits, even, slope2, D, NL, dkpart, dvpart, opart, lsepart, total;
  int n_splits, split_keys, grid;
};

// Forward: rows | tiles | fine (fp32) | counters | Opart | LSEpart, with few rows in bf16
// start | Opart | LSEpart. Backward: rows | tiles | fine |
// counters | kcount | khull | kbits | even | slope2 | D | NL | dKpart | dVpart. Each part starts on 256 bytes.
Layout layout(const ScoredProblem& p, attn_dtype_t dt, bool bwd) {
  Layout L{};
  L.n_splits = 1;
  L.split_keys = p.n_kt * kScoredTile;
  if (p.B == 0 || p.R == 0 || p.Tk == 0) return L;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = round_up(off + bytes, 256);
    return at;
  };
  const size_t B = p.B, rpad = p.rpad(), heads = B * p.Hkv;
  if (!bwd && fwd_tokens(p, dt)) {
    // one CTA per SM, two where 16 rows are enough, and at least a 64-key stage each
    const long long stages = static_cast<long long>(heads) * ((p.Tk + 63) / 64), want = p.R <= 16 ? 2 * kSms : kSms;
    L.grid = static_cast<int>(stages < want ? stages : want);
    L.start = take((B + 1) * sizeof(int));
    L.opart = take(static_cast<size_t>(L.grid) * 2 * p.R * p.dv * sizeof(float));
    L.lsepart = take(static_cast<size_t>(L.grid) * 2 * p.R * sizeof(float));
    L.total = off;
    return L;
  }
  L.rows = take(B * rpad * sizeof(int4));
  L.tiles = take(B * p.n_rt * sizeof(int4));
  if (dt == ATTN_F32) L.fine = take(B * rpad / 32 * sizeof(int2));
  L.counters = take(256);
  if (bwd) {
    L.kcount = take(B * p.n_kt * p.kv_splits * sizeof(int));
    L.khull = take(B * p.n_kt * sizeof(int4));
    L.kbits = take(B * p.n_kt * p.n_words() * sizeof(uint32_t));
    L.even = take(B * p.n_rt * sizeof(int4));
    L.slope2 = take(p.Hkv * rpad * sizeof(float));
    L.D = take(heads * rpad * sizeof(float));
    L.NL = take(heads * rpad * sizeof(float));
    if (p.kv_splits > 1) {
      L.dkpart = take(p.kv_splits * heads * p.Tk * p.d * sizeof(float));
      L.dvpart = take(p.kv_splits * heads * p.Tk * p.dv * sizeof(float));
    }
  } else {
    fwd_splits(p, dt, &L.n_splits, &L.split_keys);
    if (L.n_splits > 1) {
      L.opart = take(L.n_splits * heads * p.R * p.dv * sizeof(float));
      L.lsepart = take(L.n_splits * heads * p.R * sizeof(float));
    }
  }
  L.total = off;
  return L;
}

ScoredPlan plan_at(const Layout& L, void* ws, attn_dtype_t dt, bool bwd, bool bias) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  ScoredPlan s{};
  s.rows = reinterpret_cast<int4*>(w + L.rows);
  s.tiles = reinterpret_cast<int4*>(w + L.tiles);
  s.counters = reinterpret_cast<uint32_t*>(w + L.counters);
  if (dt == ATTN_F32) s.fine = reinterpret_cast<int2*>(w + L.fine);
  if (bwd) {
    s.kcount = reinterpret_cast<int*>(w + L.kcount);
    s.khull = reinterpret_cast<int4*>(w + L.khull);
    s.kbits = reinterpret_cast<uint32_t*>(w + L.kbits);
    if (bias) {
      s.even = reinterpret_cast<int4*>(w + L.even);
      s.slope2 = reinterpret_cast<float*>(w + L.slope2);
    }
  }
  return s;
}

struct Arrays {   // the caller's device arrays of attn_score_t as ranges
  Range r[4];
};
Arrays arrays(const attn_score_t& sc, int B, int H, int Tq) {
  const size_t n = static_cast<size_t>(B) * Tq * 4;
  return {{range(sc.slopes, sc.slopes ? static_cast<size_t>(H) * 4 : 0), range(sc.q_pos, sc.q_pos ? n : 0),
           range(sc.key_begin, sc.key_begin ? n : 0), range(sc.key_end, sc.key_end ? n : 0)}};
}

attn_status_t check_ws(const void* ws, size_t bytes, size_t need) {
  if (need == 0) return ATTN_OK;
  if (ws == nullptr || bytes < need || reinterpret_cast<uintptr_t>(ws) % 256) return ATTN_ERR_WORKSPACE;
  return ATTN_OK;
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" {

size_t attn_fwd_scored_workspace_size(int B, int H, int Hkv, int Tq, int Tk, int d, int dv, attn_dtype_t dtype) {
  if (check_scored(B, H, Hkv, Tq, Tk, d, dv, dtype) != ATTN_OK) return 0;
  return layout(problem(B, H, Hkv, Tq, Tk, d, dv, dtype), dtype, false).total;
}

size_t attn_bwd_scored_workspace_size(int B, int H, int Hkv, int Tq, int Tk, int d, int dv, attn_dtype_t dtype) {
  if (check_scored(B, H, Hkv, Tq, Tk, d, dv, dtype) != ATTN_OK) return 0;
  return layout(problem(B, H, Hkv, Tq, Tk, d, dv, dtype), dtype, true).total;
}

attn_status_t attn_fwd_scored(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H, int Hkv,
                              int Tq, int Tk, int d, int dv, float scale, const attn_score_t* score,
                              attn_dtype_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
  attn_status_t s = check_scored(B, H, Hkv, Tq, Tk, d, dv, dtype);
  const attn_score_t sc = score ? *score : attn_score_t{};
  if (s == ATTN_OK) s = check_score(sc, scale);
  if (s != ATTN_OK) return s;
  const bool bf16 = dtype == ATTN_BF16;
  const size_t es = elem_size(dtype), align = bf16 ? 16 : 4;
  const size_t nq = static_cast<size_t>(B) * H * Tq, nk = static_cast<size_t>(B) * Hkv * Tk;
  const void* ins[3] = {Q, K, V};
  const size_t in_bytes[3] = {nq * d * es, nk * d * es, nk * dv * es};
  for (int i = 0; i < 3; ++i)
    if ((s = check_ptr(ins[i], in_bytes[i], align)) != ATTN_OK) return s;
  if ((s = check_ptr(O, nq * dv * es, align)) != ATTN_OK) return s;
  if ((s = check_ptr(LSE, nq * 4, 4)) != ATTN_OK) return s;
  ScoredFwd a{};
  a.p = problem(B, H, Hkv, Tq, Tk, d, dv, dtype);
  a.p.scale = scale;
  a.p.softcap = sc.softcap;
  a.p.slopes = sc.slopes;
  const Layout L = layout(a.p, dtype, false);
  if ((s = check_ws(workspace, workspace_bytes, L.total)) != ATTN_OK) return s;
  const Arrays ar = arrays(sc, B, H, Tq);
  const Range ro = range(O, nq * dv * es), rl = range(LSE, nq * 4), rw = range(workspace, L.total);
  if (overlap(ro, rl)) return ATTN_ERR_INVALID_ARG;
  if (overlap(rw, ro) || overlap(rw, rl)) return ATTN_ERR_WORKSPACE;
  const Range in[7] = {range(Q, in_bytes[0]), range(K, in_bytes[1]), range(V, in_bytes[2]),
                       ar.r[0], ar.r[1], ar.r[2], ar.r[3]};
  for (const Range& x : in) {
    if (overlap(ro, x) || overlap(rl, x)) return ATTN_ERR_INVALID_ARG;
    if (overlap(rw, x)) return ATTN_ERR_WORKSPACE;
  }
  if (nq == 0) return ATTN_OK;
  DeviceInfo* di;
  if ((s = device_info(&di)) != ATTN_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (Tk == 0) {
    e = launch_fill_empty_fwd(Problem{B, H, Tq, Tk, d, dv, scale, 0}, O, LSE, static_cast<int>(es), st);
    return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
  }
  a.mask = ScoredMask{sc.q_pos, sc.key_begin, sc.key_end, sc.causal};
  a.plan = plan_at(L, workspace, dtype, false, sc.slopes != nullptr);
  a.Q = Q;
  a.K = K;
  a.V = V;
  a.O = O;
  a.LSE = LSE;
  a.n_splits = L.n_splits;
  a.grid = L.grid;
  a.split_keys = L.split_keys;
  a.Opart = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + L.opart);
  a.LSEpart = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + L.lsepart);
  a.status = di->status;
  a.num_sms = di->num_sms;
  a.l2_bytes = static_cast<size_t>(di->l2_bytes);
  a.stream = st;
  a.start = reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) + L.start);
  const bool tokens = fwd_tokens(a.p, dtype);
  CUtensorMap mq, mk, mv;
  if (bf16) {
    const int heads = B * Hkv;
    const unsigned key_rows = tokens ? 64u : 128u;
    if (!tokens && (s = make_map(&mq, Q, d, a.p.R, heads)) != ATTN_OK) return s;
    if ((s = make_map(&mk, K, d, Tk, heads, false, key_rows)) != ATTN_OK) return s;
    if ((s = make_map(&mv, V, dv, Tk, heads, false, key_rows)) != ATTN_OK) return s;
    a.tmQ = &mq;
    a.tmK = &mk;
    a.tmV = &mv;
  }
  if (tokens) {
    e = launch_scored_tokens_bf16(a);
  } else if ((e = launch_scored_plan(a.p, a.mask, a.plan, bf16 && L.n_splits == 1 ? ScoredIdle{O, LSE} : ScoredIdle{}, st)) ==
             cudaSuccess) {
    e = bf16 ? launch_scored_fwd_bf16(a) : launch_scored_fwd_simt(a);
    if (e == cudaSuccess && a.n_splits > 1) e = launch_scored_merge(a, bf16);
  }
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
}

attn_status_t attn_bwd_scored(const void* Q, const void* K, const void* V, const void* O, const float* LSE,
                              const void* dO, void* dQ, void* dK, void* dV, int B, int H, int Hkv, int Tq, int Tk,
                              int d, int dv, float scale, const attn_score_t* score, attn_dtype_t dtype,
                              void* workspace, size_t workspace_bytes, void* stream) {
  attn_status_t s = check_scored(B, H, Hkv, Tq, Tk, d, dv, dtype);
  const attn_score_t sc = score ? *score : attn_score_t{};
  if (s == ATTN_OK) s = check_score(sc, scale);
  if (s != ATTN_OK) return s;
  const bool bf16 = dtype == ATTN_BF16;
  const size_t es = elem_size(dtype), align = bf16 ? 16 : 4;
  const size_t nq = static_cast<size_t>(B) * H * Tq, nk = static_cast<size_t>(B) * Hkv * Tk;
  const void* ins[6] = {Q, K, V, O, LSE, dO};
  const size_t in_bytes[6] = {nq * d * es, nk * d * es, nk * dv * es, nq * dv * es, nq * 4, nq * dv * es};
  for (int i = 0; i < 6; ++i)
    if ((s = check_ptr(ins[i], in_bytes[i], i == 4 ? 4 : align)) != ATTN_OK) return s;
  void* outs[3] = {dQ, dK, dV};
  const size_t out_bytes[3] = {nq * d * es, nk * d * es, nk * dv * es};
  for (int i = 0; i < 3; ++i)
    if ((s = check_ptr(outs[i], out_bytes[i], align)) != ATTN_OK) return s;
  ScoredBwd a{};
  a.p = problem(B, H, Hkv, Tq, Tk, d, dv, dtype);
  a.p.scale = scale;
  a.p.softcap = sc.softcap;
  a.p.slopes = sc.slopes;
  const Layout L = layout(a.p, dtype, true);
  if ((s = check_ws(workspace, workspace_bytes, L.total)) != ATTN_OK) return s;
  const Arrays ar = arrays(sc, B, H, Tq);
  const Range ro[4] = {range(dQ, out_bytes[0]), range(dK, out_bytes[1]), range(dV, out_bytes[2]),
                       range(workspace, L.total)};
  for (int i = 0; i < 4; ++i) {
    const attn_status_t bad = i == 3 ? ATTN_ERR_WORKSPACE : ATTN_ERR_INVALID_ARG;
    for (int j = 0; j < 6; ++j)
      if (overlap(ro[i], range(ins[j], in_bytes[j]))) return bad;
    for (const Range& x : ar.r)
      if (overlap(ro[i], x)) return bad;
    for (int j = 0; j < i; ++j)
      if (overlap(ro[i], ro[j])) return bad;
  }
  if (nq == 0 && nk == 0) return ATTN_OK;
  DeviceInfo* di;
  if ((s = device_info(&di)) != ATTN_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (nq == 0 || nk == 0) {   // no query-key pair
    e = cudaSuccess;
    for (int i = 0; i < 3 && e == cudaSuccess; ++i) e = launch_zero(outs[i], out_bytes[i], st);
    return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
  }
  a.plan = plan_at(L, workspace, dtype, true, sc.slopes != nullptr);
  a.Q = Q;
  a.K = K;
  a.V = V;
  a.O = O;
  a.LSE = LSE;
  a.dO = dO;
  a.dQ = dQ;
  a.dK = dK;
  a.dV = dV;
  a.D = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + L.D);
  a.NL = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + L.NL);
  a.dKpart = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + L.dkpart);
  a.dVpart = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + L.dvpart);
  a.status = di->status;
  a.num_sms = di->num_sms;
  a.l2_bytes = static_cast<size_t>(di->l2_bytes);
  a.stream = st;
  CUtensorMap mq, mk, mv, mdo, mo;
  if (bf16) {
    const int heads = B * Hkv;
    if ((s = make_map(&mq, Q, d, a.p.R, heads)) != ATTN_OK) return s;
    if ((s = make_map(&mk, K, d, Tk, heads)) != ATTN_OK) return s;
    if ((s = make_map(&mv, V, dv, Tk, heads)) != ATTN_OK) return s;
    if ((s = make_map(&mdo, dO, dv, a.p.R, heads)) != ATTN_OK) return s;
    if ((s = make_map(&mo, O, dv, a.p.R, heads)) != ATTN_OK) return s;
    a.tmQ = &mq;
    a.tmK = &mk;
    a.tmV = &mv;
    a.tmdO = &mdo;
    a.tmO = &mo;
  }
  ScoredIdle idle{};
  if (bf16) {
    idle = ScoredIdle{nullptr, nullptr, dQ, a.D, a.NL, nullptr, nullptr};
    if (a.p.kv_splits == 1) {
      idle.dK = dK;
      idle.dV = dV;
    }
  }
  e = launch_scored_plan(a.p, ScoredMask{sc.q_pos, sc.key_begin, sc.key_end, sc.causal}, a.plan, idle, st);
  if (e == cudaSuccess) e = bf16 ? launch_scored_bwd_bf16(a) : launch_scored_bwd_simt(a);
  if (e == cudaSuccess && a.p.kv_splits > 1) e = launch_scored_kv_sum(a, bf16);
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
}

}  // extern "C"
