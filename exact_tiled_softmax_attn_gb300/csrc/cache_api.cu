// C-ABI layer of the paged key-value cache: argument validation, workspace
// layout and dispatch.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attn.h"
#include "cache.h"
#include "host.h"

namespace attn {
namespace {

constexpr int kMostRows = 1 << 29;   // tokens of a call
// Workspace sizes are rules of the shapes alone, so counts that aim at
// filling the GPU use GB300's SM count.
constexpr int kSms = 152;
// Packed rows of a key head above which the 128-row tiles take over. us by the
// few-row kernel and by the tiles, Hkv=4 d=128: 16 sequences of up to 12000 keys,
// 24 rows 65 and 58, 32 rows 66 and 58 (d=64: 45 and 43), 64 rows 113 and 60; 32
// rows of 8 pairs of 1024 keys 10 and 16, of 4096 15 and 20, of 64 pairs of 1024
// 16 and 16, of 4096 34 and 33, of 16384 86 and 70. Up to 32 rows it is the
// number of keys that decides: short sequences have clusters in the few-row
// kernel only, and they are what this limit is right for.
constexpr int kTilesFrom = 32;

// Sizes, widths and the pool's pointers; fills the view.
attn_status_t check_cache(const attn_cache_t* c, int B, int Hkv, int d, int dv, attn_dtype_t dt, int widest,
                          CacheView* view) {
  if (c == nullptr || B < 0 || Hkv < 1 || d <= 0 || dv <= 0) return ATTN_ERR_INVALID_ARG;
  if (dt != ATTN_F32 && dt != ATTN_BF16) return ATTN_ERR_INVALID_ARG;
  if (c->type != ATTN_CACHE_PLAIN && c->type != ATTN_CACHE_E4M3) return ATTN_ERR_INVALID_ARG;
  if (c->pages < 1 || c->max_pages < 0) return ATTN_ERR_INVALID_ARG;
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return ATTN_ERR_UNSUPPORTED;
  const bool codes = c->type == ATTN_CACHE_E4M3;
  const int step = codes ? 16 : dt == ATTN_BF16 ? 8 : 1;
  if (d > widest || dv > widest || d % step || dv % step) return ATTN_ERR_UNSUPPORTED;
  // pages of every head are counted in int
  if (static_cast<double>(c->pages) * Hkv > 2147483646.0 || static_cast<double>(B) * c->max_pages > 9e15 ||
      static_cast<double>(B) * Hkv > 2147483647.0)
    return ATTN_ERR_INVALID_ARG;
  if (B == 0) return ATTN_OK;
  const size_t align = codes || dt == ATTN_BF16 ? 16 : 4;
  for (const void* p : {c->k, c->v})
    if (p == nullptr) return ATTN_ERR_INVALID_ARG;
  if (c->seq_len == nullptr || (c->table == nullptr && c->max_pages > 0)) return ATTN_ERR_INVALID_ARG;
  if (codes && (c->k_scale == nullptr || c->v_scale == nullptr)) return ATTN_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(c->k) % align || reinterpret_cast<uintptr_t>(c->v) % align) return ATTN_ERR_MISALIGNED;
  for (const void* p : {static_cast<const void*>(c->table), static_cast<const void*>(c->seq_len),
                        static_cast<const void*>(c->new_len), static_cast<const void*>(codes ? c->k_scale : nullptr),
                        static_cast<const void*>(codes ? c->v_scale : nullptr)})
    if (reinterpret_cast<uintptr_t>(p) % 4) return ATTN_ERR_MISALIGNED;
  view->pool[0] = c->k;
  view->pool[1] = c->v;
  view->scale[0] = codes ? c->k_scale : nullptr;
  view->scale[1] = codes ? c->v_scale : nullptr;
  view->table = c->table;
  view->seq_len = c->seq_len;
  view->new_len = c->new_len;
  view->pages = c->pages;
  view->shift = c->page == 16 ? 4 : c->page == 32 ? 5 : c->page == 64 ? 6 : 7;
  view->max_pages = c->max_pages;
  view->codes = codes;
  return ATTN_OK;
}

struct CacheRanges {   // k, v, k_scale, v_scale | table, seq_len, new_len
  Range r[7];
};
CacheRanges ranges(const attn_cache_t& c, int B, int Hkv, int d, int dv, attn_dtype_t dt) {
  const size_t es = c.type == ATTN_CACHE_E4M3 ? 1 : elem_size(dt);
  const size_t heads = static_cast<size_t>(c.pages) * Hkv, rows = heads * c.page;
  const size_t scales = c.type == ATTN_CACHE_E4M3 ? heads * 4 : 0, n = static_cast<size_t>(B) * 4;
  return {{range(c.k, rows * d * es), range(c.v, rows * dv * es), range(c.k_scale, scales), range(c.v_scale, scales),
           range(c.table, n * c.max_pages), range(c.seq_len, n), range(c.new_len, c.new_len ? n : 0)}};
}

Rows flat(Range r) { return Rows{r.lo, static_cast<long long>(r.hi - r.lo), {0, 0, 0}, {1, 1, 1}}; }

attn_status_t check_ws(const void* ws, size_t bytes, size_t need) {
  if (need == 0) return ATTN_OK;
  if (ws == nullptr || bytes < need || reinterpret_cast<uintptr_t>(ws) % 256) return ATTN_ERR_WORKSPACE;
  return ATTN_OK;
}

// The workspace of an attention call that reads the pages first:
// q_pos | key_begin | key_end | hull | K | V | the scored attention's.
struct Gather {
  size_t q_pos, begin, end, hull, k, v, inner, inner_bytes, total;
};
Gather gather_layout(int B, int H, int Hkv, int Tq, int Tk, int d, int dv, attn_dtype_t dt) {
  Gather g{};
  if (B == 0 || H == 0 || Tq == 0) return g;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = round_up(off + bytes, 256);
    return at;
  };
  const size_t rows = static_cast<size_t>(B) * Tq * 4, es = elem_size(dt);
  const size_t keys = static_cast<size_t>(B) * Hkv * Tk;
  g.q_pos = take(rows);
  g.begin = take(rows);
  g.end = take(rows);
  g.hull = take(static_cast<size_t>(B) * 8);
  g.k = take(keys * d * es);
  g.v = take(keys * dv * es);
  g.inner_bytes = attn_fwd_scored_workspace_size(B, H, Hkv, Tq, Tk, d, dv, dt);
  g.inner = take(g.inner_bytes);
  g.total = off;
  return g;
}

// How a call reads the pages: where they lie, in groups of a few rows or (bf16
// over e4m3) in tiles of 128, or into the workspace first. fp32 pages take the
// last: their products need more than the tensor cores hold.
enum Way { kGather, kTokens, kTiles };
Way way_of(int B, int H, int Hkv, int Tq, int Tk, int type, attn_dtype_t dt) {
  const long long R = static_cast<long long>(H / Hkv) * Tq;
  if (R > kCacheTokenRows || (dt != ATTN_BF16 && type != ATTN_CACHE_E4M3)) return kGather;
  const Way way = R > kTilesFrom && dt == ATTN_BF16 && type == ATTN_CACHE_E4M3 ? kTiles : kTokens;
  // stages of 64 keys are counted in int
  const double groups = way == kTiles ? 1.0 : cache_token_groups(static_cast<int>(R));
  return static_cast<double>(B) * Hkv * groups * (Tk / 64 + 1.0) < 2e9 ? way : kGather;
}

// The workspace of such a call: start | Opart | LSEpart.
struct Few {
  size_t start, opart, lsepart, total;
  int grid, groups, want;   // want: CTAs that are resident at a time
  double pairs;             // of a sequence's row group and a key head
  int most;                 // CTAs of a cluster
  // CTAs per pair, a cluster, with which ranges of at most `keys` keys go without
  // the list of stages, or 0: the list costs a second kernel and, at every
  // pair's end inside a share, some microseconds, but loads the SMs evenly.
  // As many as have two stages each and are resident at a time. (A cluster lies
  // within a GPC, and what is left of one holds none: of eight CTAs, one to an
  // SM, 12 are resident but not 16 - 32 rows of 1024 keys 19.6 us, with four to
  // a cluster 12.3 - and of two to an SM 32.) Codes, d=128, 4 and 16 rows, us by
  // list, by one CTA per pair and by clusters: 8 pairs of 512 keys 8.3 8.2 6.6,
  // 10.8 11.5 8.6, of 2048 9.1 19.7 7.8, 11.4 27.5 10.1, of 4096 10.2 35.4 9.8,
  // 13.2 48.2 12.9, of 8192 13.5 - 14.0, 15.8 - 18.9; 64 pairs of 1024 11.8 12.1
  // 8.4, 19.0 16.9 11.3, of 4096 15.3 36.1 15.1, 24.4 49.5 21.2; 192 pairs of
  // 1024 15.3 14.0 13.1, of 4096 24.1 42.7 30.5; 512 pairs (no clusters) of 1024
  // 24.8 20.5, 49.2 33.5, of 4096 61.1 62.7, 92.6 88.7, of 16384 202 240, 247 320.
  int direct(long long keys) const {
    int s = 1;
    while (s < most && pairs * 2 * s <= want - 6 * (2 * s - 1) && keys >= 256 * s) s *= 2;
    const double ctas = pairs * s;
    return keys <= 512 * s + 2048 * (ctas < want ? ctas / want : 1.0) && ctas <= 2147483647.0 ? s : 0;
  }
};
Few few_layout(Way way, int B, int H, int Hkv, int Tq, int Tk, int dv, int type) {
  Few f{};
  if (B == 0 || H == 0 || Tq == 0) return f;
  const int R = H / Hkv * Tq, rows = way == kTiles ? kCacheTileRows : cache_token_rows(R);
  f.groups = way == kTiles ? 1 : cache_token_groups(R);   // (a tile holds all of kCacheTokenRows)
  const size_t entries = static_cast<size_t>(B) * f.groups;
  // All the CTAs that are resident at a time, and at least two stages each in
  // the few-row kernel: 8 pairs of 4096 keys, us with two and with one (fewer
  // parts to join, against a longer share), codes 10.2 and 12.6, bf16 10.4 and
  // 11.5; 32 pairs of 1024 11.2 and 10.3, 11.3 and 11.4. In tiles a stage: 2
  // pairs of 8000 keys with 64 rows 19.5 with two, 18.8 with one.
  const int keys = way == kTiles ? 128 : 64;
  const double stages = static_cast<double>(entries) * Hkv * ((Tk + keys - 1) / keys);
  const int want = way == kTiles ? kSms : cache_token_ctas(rows, type == ATTN_CACHE_E4M3) * kSms;
  f.pairs = static_cast<double>(entries) * Hkv;
  f.want = want;
  f.most = way == kTiles ? 1 : 8;
  if (const int s = f.direct(Tk)) {
    f.grid = static_cast<int>(f.pairs) * s;
    return f;
  }
  const double shares = way != kTiles ? stages / 2 : stages;
  f.grid = shares < want ? (shares < 1.0 ? 1 : static_cast<int>(shares)) : want;
  f.start = 0;
  f.opart = round_up((entries + 1) * sizeof(int), 256);
  f.lsepart = f.opart + round_up(static_cast<size_t>(f.grid) * 2 * rows * dv * sizeof(float), 256);
  f.total = f.lsepart + round_up(static_cast<size_t>(f.grid) * 2 * rows * sizeof(float), 256);
  return f;
}

// Sizes of an attention call; as attn_fwd_scored's, which runs where rows are many.
attn_status_t check_attend(int B, int H, int Hkv, int Tq, int Tk, int d, int dv, attn_dtype_t dt) {
  if (B < 0 || H < 0 || Tq < 0 || Tk < 0 || d <= 0 || dv <= 0 || Hkv < 1 || H % Hkv) return ATTN_ERR_INVALID_ARG;
  if (dt != ATTN_F32 && dt != ATTN_BF16) return ATTN_ERR_INVALID_ARG;
  if (Tq > kMostRows || Tk > (1 << 30) || static_cast<long long>(H / Hkv) * Tq > (1 << 30)) return ATTN_ERR_INVALID_ARG;
  const double heads = static_cast<double>(B) * Hkv, rows = static_cast<double>(H / Hkv) * Tq;
  if (heads * ((rows > Tk ? rows : Tk) / 32.0 + 2.0 + H / Hkv) > 2147483647.0 || heads * rows > 2147483647.0)
    return ATTN_ERR_INVALID_ARG;
  if (d > 128 || dv > 128) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}
bool widths_fit(int d, int dv, int type, attn_dtype_t dt) {
  const int step = type == ATTN_CACHE_E4M3 ? 16 : dt == ATTN_BF16 ? 8 : 1;
  return d % step == 0 && dv % step == 0;
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" {

attn_status_t attn_cache_append(const attn_cache_t* cache, const attn_rope_t* plan, const void* Q, void* Qout,
                                const void* K, const void* V, const long long* strides, const int* pos, int B, int H,
                                int Hkv, int T, int d, int dv, attn_dtype_t dtype, void* stream) {
  CacheAppend a{};
  attn_status_t s = check_cache(cache, B, Hkv, d, dv, dtype, 256, &a.c);
  if (s != ATTN_OK) return s;
  if (strides == nullptr || H < 0 || T < 0 || T > kMostRows || (H > 0 && plan == nullptr)) return ATTN_ERR_INVALID_ARG;
  if (plan && (plan->rot < 2 || plan->rot % 2 || plan->rot > d || (plan->interleaved != 0 && plan->interleaved != 1)))
    return ATTN_ERR_INVALID_ARG;
  if (H > 0x7fffffff / 512) return ATTN_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(pos) % 4) return ATTN_ERR_MISALIGNED;
  const size_t es = elem_size(dtype);
  const bool some = B > 0 && T > 0;
  const int v_elems = 16 / static_cast<int>(es);
  bool wide = d % v_elems == 0 && dv % v_elems == 0;
  if (plan) wide = wide && (plan->rot / 2) % v_elems == 0 && (d - plan->rot) % v_elems == 0;
  // Q, Qout, K, V
  const void* ptr[4] = {Q, Qout, K, V};
  const int heads[4] = {H, H, Hkv, Hkv}, width[4] = {d, d, d, dv};
  View view[4];
  Rows rows[4];
  for (int k = 0; k < 4; ++k) {
    const long long* t = strides + 3 * k;
    view[k] = View{t[0], t[1], t[2]};
    if (!some || heads[k] == 0) continue;
    for (int i = 0; i < 3; ++i) {
      if (t[i] < 0 || t[i] > (1LL << 50)) return ATTN_ERR_INVALID_ARG;
      wide = wide && t[i] % v_elems == 0;
    }
    if (static_cast<double>(t[0]) * B + static_cast<double>(t[1]) * heads[k] + static_cast<double>(t[2]) * T > 9e15)
      return ATTN_ERR_INVALID_ARG;
    if (ptr[k] == nullptr) return ATTN_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(ptr[k]) % es) return ATTN_ERR_MISALIGNED;
    wide = wide && reinterpret_cast<uintptr_t>(ptr[k]) % 16 == 0;
    rows[k] = rows_of(ptr[k], view[k], B, heads[k], T, width[k], static_cast<long long>(es));
  }
  if (!some) return ATTN_OK;
  if (cache->type == ATTN_CACHE_PLAIN)
    wide = wide && (reinterpret_cast<uintptr_t>(cache->k) | reinterpret_cast<uintptr_t>(cache->v)) % 16 == 0;
  // what is written (Qout, the pools and scales) against all else
  const Range at_pos = range(pos, pos ? static_cast<size_t>(B) * T * 4 : 0);
  const CacheRanges cr = ranges(*cache, B, Hkv, d, dv, dtype);
  for (int i = 0; i < 4; ++i) {
    if (cr.r[i].lo == cr.r[i].hi) continue;
    for (int j = 0; j < 7; ++j)
      if (j != i && overlap(cr.r[i], cr.r[j])) return ATTN_ERR_INVALID_ARG;
    if (overlap(cr.r[i], at_pos)) return ATTN_ERR_INVALID_ARG;
    for (int k = 0; k < 4; ++k)
      if (heads[k] > 0 && !apart(flat(cr.r[i]), rows[k])) return ATTN_ERR_INVALID_ARG;
  }
  if (H > 0) {
    if (!distinct(rows[1])) return ATTN_ERR_INVALID_ARG;
    bool in_place = Q == Qout;
    for (int i = 0; i < 3; ++i) in_place = in_place && (rows[1].n[i] <= 1 || rows[1].step[i] == rows[0].step[i]);
    if (!in_place && !apart(rows[1], rows[0])) return ATTN_ERR_INVALID_ARG;
    for (int k = 2; k < 4; ++k)
      if (heads[k] > 0 && !apart(rows[1], rows[k])) return ATTN_ERR_INVALID_ARG;
    if (pos && !apart(rows[1], flat(at_pos))) return ATTN_ERR_INVALID_ARG;
    for (int j = 4; j < 7; ++j)
      if (cr.r[j].lo != cr.r[j].hi && !apart(rows[1], flat(cr.r[j]))) return ATTN_ERR_INVALID_ARG;
  }
  if (static_cast<double>(B) * (T / static_cast<double>(cache->page) + 2.0) * Hkv * 2.0 > 2e9 ||
      static_cast<double>(B) * T > 2e9)
    return ATTN_ERR_INVALID_ARG;
  DeviceInfo* di;
  if ((s = device_info(&di)) != ATTN_OK) return s;
  if (plan)
    a.q.plan = *plan;
  else
    a.q.plan.mscale = 1.f;
  a.q.x[0] = Q;
  a.q.y[0] = Qout;
  a.q.xs[0] = view[0];
  a.q.ys[0] = view[1];
  a.q.pos = pos;
  a.q.seq_len = cache->seq_len;
  a.q.new_len = cache->new_len;
  a.q.heads[0] = H;
  a.q.B = B;
  a.q.T = T;
  a.q.d = d;
  a.q.sign = 1.f;
  a.turn = plan != nullptr;
  a.x[0] = K;
  a.x[1] = V;
  a.s[0] = view[2];
  a.s[1] = view[3];
  a.pos = pos;
  a.B = B;
  a.Hkv = Hkv;
  a.T = T;
  a.w[0] = d;
  a.w[1] = dv;
  a.wide = wide;
  a.bf16 = dtype == ATTN_BF16;
  a.num_sms = di->num_sms;
  a.stream = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_cache_append(a);
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
}

attn_status_t attn_cache_read(const attn_cache_t* cache, void* K, void* V, int B, int Hkv, int Tk, int d, int dv,
                              attn_dtype_t dtype, void* stream) {
  CacheRead a{};
  attn_status_t s = check_cache(cache, B, Hkv, d, dv, dtype, 256, &a.c);
  if (s != ATTN_OK) return s;
  // (blocks of 128 tokens of a head are counted in int)
  if (Tk < 0 || Tk > (1 << 30) || static_cast<double>(B) * Hkv * (Tk / 128.0 + 1.0) > 2147483647.0)
    return ATTN_ERR_INVALID_ARG;
  const size_t es = elem_size(dtype), align = dtype == ATTN_BF16 || cache->type == ATTN_CACHE_E4M3 ? 16 : 4;
  const size_t n = static_cast<size_t>(B) * Hkv * Tk;
  if ((s = check_ptr(K, n * d * es, align)) != ATTN_OK || (s = check_ptr(V, n * dv * es, align)) != ATTN_OK) return s;
  if (n == 0) return ATTN_OK;
  const Range out[2] = {range(K, n * d * es), range(V, n * dv * es)};
  if (overlap(out[0], out[1])) return ATTN_ERR_INVALID_ARG;
  const CacheRanges cr = ranges(*cache, B, Hkv, d, dv, dtype);
  for (const Range& o : out)
    for (const Range& r : cr.r)
      if (overlap(o, r)) return ATTN_ERR_INVALID_ARG;
  DeviceInfo* di;
  if ((s = device_info(&di)) != ATTN_OK) return s;
  a.out[0] = K;
  a.out[1] = V;
  a.B = B;
  a.Hkv = Hkv;
  a.Tk = Tk;
  a.w[0] = d;
  a.w[1] = dv;
  a.bf16 = dtype == ATTN_BF16;
  a.num_sms = di->num_sms;
  a.stream = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_cache_read(a);
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
}

size_t attn_fwd_cached_workspace_size(int B, int H, int Hkv, int Tq, int Tk, int d, int dv, int cache_type,
                                      attn_dtype_t dtype) {
  if (check_attend(B, H, Hkv, Tq, Tk, d, dv, dtype) != ATTN_OK) return 0;
  if ((cache_type != ATTN_CACHE_PLAIN && cache_type != ATTN_CACHE_E4M3) || !widths_fit(d, dv, cache_type, dtype)) return 0;
  const Way way = way_of(B, H, Hkv, Tq, Tk, cache_type, dtype);
  if (way != kGather) return few_layout(way, B, H, Hkv, Tq, Tk, dv, cache_type).total;
  return gather_layout(B, H, Hkv, Tq, Tk, d, dv, dtype).total;
}

attn_status_t attn_fwd_cached(const void* Q, const attn_cache_t* cache, void* O, float* LSE, int B, int H, int Hkv,
                              int Tq, int Tk, int d, int dv, float scale, int window, const attn_score_t* score,
                              attn_dtype_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
  attn_status_t s = check_attend(B, H, Hkv, Tq, Tk, d, dv, dtype);
  if (s != ATTN_OK) return s;
  CacheView view{};
  if ((s = check_cache(cache, B, Hkv, d, dv, dtype, 128, &view)) != ATTN_OK) return s;
  if (window < 0 || window > (1 << 30) || Tk > static_cast<long long>(cache->max_pages) * cache->page)
    return ATTN_ERR_INVALID_ARG;
  const attn_score_t sc = score ? *score : attn_score_t{};
  if (!(scale > 0.f) || !isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if (sc.softcap != 0.f && !(sc.softcap >= 1e-4f && sc.softcap <= 1e6f)) return ATTN_ERR_INVALID_ARG;
  if (sc.causal != 0 && sc.causal != 1) return ATTN_ERR_INVALID_ARG;
  for (const void* x : {static_cast<const void*>(sc.slopes), static_cast<const void*>(sc.q_pos),
                        static_cast<const void*>(sc.key_begin), static_cast<const void*>(sc.key_end)})
    if (reinterpret_cast<uintptr_t>(x) % 4) return ATTN_ERR_MISALIGNED;
  const bool bf16 = dtype == ATTN_BF16;
  const size_t es = elem_size(dtype), align = bf16 || view.codes ? 16 : 4;
  const size_t nq = static_cast<size_t>(B) * H * Tq;
  if ((s = check_ptr(Q, nq * d * es, align)) != ATTN_OK || (s = check_ptr(O, nq * dv * es, align)) != ATTN_OK ||
      (s = check_ptr(LSE, nq * 4, 4)) != ATTN_OK)
    return s;
  const Way way = way_of(B, H, Hkv, Tq, Tk, cache->type, dtype);
  const bool few = way != kGather;
  const Few f = few ? few_layout(way, B, H, Hkv, Tq, Tk, dv, cache->type) : Few{};
  const Gather g = few ? Gather{} : gather_layout(B, H, Hkv, Tq, Tk, d, dv, dtype);
  const size_t need = few ? f.total : g.total;
  if ((s = check_ws(workspace, workspace_bytes, need)) != ATTN_OK) return s;
  if (nq == 0) return ATTN_OK;
  const Range ro = range(O, nq * dv * es), rl = range(LSE, nq * 4), rw = range(workspace, need);
  if (overlap(ro, rl)) return ATTN_ERR_INVALID_ARG;
  if (overlap(rw, ro) || overlap(rw, rl)) return ATTN_ERR_WORKSPACE;
  const size_t nr = static_cast<size_t>(B) * Tq * 4;
  const CacheRanges cr = ranges(*cache, B, Hkv, d, dv, dtype);
  const Range in[12] = {range(Q, nq * d * es), range(sc.slopes, sc.slopes ? static_cast<size_t>(H) * 4 : 0),
                        range(sc.q_pos, sc.q_pos ? nr : 0), range(sc.key_begin, sc.key_begin ? nr : 0),
                        range(sc.key_end, sc.key_end ? nr : 0), cr.r[0], cr.r[1], cr.r[2], cr.r[3], cr.r[4], cr.r[5],
                        cr.r[6]};
  for (const Range& x : in) {
    if (overlap(ro, x) || overlap(rl, x)) return ATTN_ERR_INVALID_ARG;
    if (overlap(rw, x)) return ATTN_ERR_WORKSPACE;
  }
  DeviceInfo* di;
  if ((s = device_info(&di)) != ATTN_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* w = static_cast<uint8_t*>(workspace);
  if (few) {
    CacheTokens t{};
    t.c = view;
    t.p.B = B;
    t.p.Hkv = Hkv;
    t.p.G = H / Hkv;
    t.p.Tq = Tq;
    t.p.Tk = Tk;
    t.p.d = d;
    t.p.dv = dv;
    t.p.R = t.p.G * Tq;
    t.p.scale = scale;
    t.p.softcap = sc.softcap;
    t.p.slopes = sc.slopes;
    t.mask = ScoredMask{sc.q_pos, sc.key_begin, sc.key_end, sc.causal};
    t.window = window;
    t.Q = Q;
    t.O = O;
    t.LSE = LSE;
    t.f32 = !bf16;
    // a causal window at the sequence's end: no more keys than it and the tokens before the last one
    const long long in_window = window + static_cast<long long>(Tq);
    const long long keys = window > 0 && sc.causal && !sc.q_pos && in_window < Tk ? in_window : Tk;
    t.direct = f.direct(keys);
    t.grid = t.direct ? static_cast<int>(f.pairs) * t.direct : f.grid;
    t.groups = f.groups;
    t.start = reinterpret_cast<int*>(w + f.start);
    t.Opart = reinterpret_cast<float*>(w + f.opart);
    t.LSEpart = reinterpret_cast<float*>(w + f.lsepart);
    t.status = di->status;
    t.stream = st;
    if (way == kTiles) {
      const cudaError_t e = launch_cache_tiles(t);
      return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
    }
    CUtensorMap mk, mv;
    const unsigned width = view.codes && d <= 64 && dv <= 64 ? 64u : 128u, box_rows = cache->page < 64 ? cache->page : 64;
    const int planes = cache->pages * Hkv;
    if ((s = make_map_bytes(&mk, cache->k, d, cache->page, planes, view.codes, width, box_rows)) != ATTN_OK) return s;
    if ((s = make_map_bytes(&mv, cache->v, dv, cache->page, planes, view.codes, width, box_rows)) != ATTN_OK) return s;
    t.tmK = &mk;
    t.tmV = &mv;
    const cudaError_t e = launch_cache_tokens(t);
    return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
  }
  CacheRows r{};
  r.c = view;
  r.mask = ScoredMask{sc.q_pos, sc.key_begin, sc.key_end, sc.causal};
  r.B = B;
  r.Tq = Tq;
  r.Tk = Tk;
  r.window = window;
  r.q_pos = reinterpret_cast<int*>(w + g.q_pos);
  r.key_begin = reinterpret_cast<int*>(w + g.begin);
  r.key_end = reinterpret_cast<int*>(w + g.end);
  r.hull = reinterpret_cast<int2*>(w + g.hull);
  r.stream = st;
  cudaError_t e = launch_cache_rows(r);
  if (e == cudaSuccess && Tk > 0) {
    CacheRead a{};
    a.c = view;
    a.out[0] = w + g.k;
    a.out[1] = w + g.v;
    a.B = B;
    a.Hkv = Hkv;
    a.Tk = Tk;
    a.w[0] = d;
    a.w[1] = dv;
    a.bf16 = bf16;
    a.hull = r.hull;
    a.num_sms = di->num_sms;
    a.stream = st;
    e = launch_cache_read(a);
  }
  if (e != cudaSuccess) return cuda_fail(e);
  const attn_score_t rows{sc.softcap, 0, sc.slopes, r.q_pos, r.key_begin, r.key_end};
  return attn_fwd_scored(Q, w + g.k, w + g.v, O, LSE, B, H, Hkv, Tq, Tk, d, dv, scale, &rows, dtype,
                         g.inner_bytes ? w + g.inner : nullptr, g.inner_bytes, stream);
}

}  // extern "C"
