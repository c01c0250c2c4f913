/*
 * attn.h -- C ABI of the exact tiled softmax attention library (libattn.so).
 *
 * Exact scaled-dot-product softmax attention, forward and backward, computed
 * one key tile at a time with an online softmax, so the Tq x Tk score matrix
 * is never stored. Kernels are written for NVIDIA sm_103a (GB300).
 *
 * Definitions (sources are the pages this library restates):
 *   S   = scale * Q K^T, with S_ij = -inf where the mask blocks key j for
 *         query i. causal = 1 blocks j > i with global row indices
 *         ("Tiled attention with an online softmax", section "Task").
 *   O   = softmax(S) V                ("The Hidden Recurrence in Softmax
 *         Attention", section "Standard Attention / Forward Pass";
 *         "attention_backprop", section "Forward Pass")
 *   LSE = log sum_j exp(S_ij)         (natural log; the page's m_i + log l_i)
 *   D   = rowsum(dO o O)
 *   dV  = P^T dO,  dS = P o (dO V^T - D),  dQ = scale * dS K,
 *   dK  = scale * dS^T Q              ("attention_backprop", sections
 *         "Gradient of V and P", "Gradient of S", "Gradient of Q and K";
 *         the factor scale comes from S = scale * Q K^T)
 *
 * Layout: every tensor is a contiguous row-major device array.
 *   Q [B,H,Tq,d]  K [B,H,Tk,d]  V [B,H,Tk,dv]  O, dO [B,H,Tq,dv]
 *   dQ [B,H,Tq,d] dK [B,H,Tk,d] dV [B,H,Tk,dv] LSE, D [B,H,Tq] (fp32)
 * Q, K, V, O, dO, dQ, dK, dV use the element type `dtype`; LSE is always fp32.
 *
 * Ownership: the caller allocates and owns every buffer, including the
 * backward workspace. The library never allocates device memory in these
 * calls and never writes its inputs. Outputs must not overlap inputs.
 *
 * Asynchrony: every call validates its arguments on the host, then enqueues
 * kernels on `stream` (a cudaStream_t passed as void*; NULL = legacy default
 * stream) and returns without synchronising. A nonzero status from the host
 * checks means nothing was enqueued.
 *
 * Supported shapes:
 *   ATTN_F32 : 1 <= d, dv <= 256, any B, H, Tq, Tk >= 0 (attn_fwd_f32_blocked
 *              with block_n = 128 returns ATTN_ERR_UNSUPPORTED when its key
 *              tile does not fit in shared memory: d or dv above 128)
 *   ATTN_BF16: forward (attn_fwd, attn_fwd_splitkv): d and dv multiples
 *              of 8 from 8 to 256, independently (the page's task takes V
 *              with its own head dimension); a width below 64, 128 or 256
 *              runs on the next of those tile widths with zero columns, so
 *              64, 128 and 256 are the efficient sizes. Backward (attn_bwd):
 *              d and dv multiples of 8 up to 256, independently. The
 *              kernels take d, dv in {64, 128}, and d = 256 with dv in {64,
 *              128, 256}; other widths run on zero-padded copies of the
 *              inputs held in the workspace (rows wider than 128 on either
 *              side pad d to 256), and attn_bwd_phase takes only the
 *              kernels' own widths. Any B, H, Tq, Tk >= 0.
 * Zero-sized problems are valid: Tk == 0 gives O = 0 and LSE = -inf (a row
 * with no allowed key), and empty gradients are written as zeros.
 */
#ifndef ATTN_H_
#define ATTN_H_

#include <stddef.h>

#if defined(__GNUC__)
#define ATTN_API __attribute__((visibility("default")))
#else
#define ATTN_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  ATTN_OK = 0,
  ATTN_ERR_INVALID_ARG = 1,  /* null pointer, negative size, non-finite or non-positive scale, overlap */
  ATTN_ERR_UNSUPPORTED = 2,  /* valid request the library does not implement (e.g. bf16 with d = 96) */
  ATTN_ERR_MISALIGNED = 3,   /* a pointer breaks the alignment rule of its dtype (bf16: 16 B, f32: 4 B) */
  ATTN_ERR_CUDA = 4,         /* a CUDA runtime/driver call failed; see attn_last_cuda_error() */
  ATTN_ERR_TIMEOUT = 5,      /* a kernel's bounded pipeline wait gave up (reported by attn_device_status) */
  ATTN_ERR_WORKSPACE = 6     /* workspace missing, too small or not 256-byte aligned */
} attn_status_t;

typedef enum { ATTN_F32 = 0, ATTN_BF16 = 1 } attn_dtype_t;

/*
 * Forward pass: O and LSE from Q, K, V.
 * Restates flash_attention of "Tiled attention with an online softmax"
 * (sections "Task", "Input and output") for a batch of heads: returns the
 * attention output and the log-sum-exp of each query row. `scale` multiplies
 * Q K^T (the page uses 1/sqrt(d); pass that for the same result) and must be
 * finite and > 0. `causal` is 0 (no mask) or 1.
 * Errors: ATTN_ERR_INVALID_ARG, ATTN_ERR_UNSUPPORTED, ATTN_ERR_MISALIGNED,
 * ATTN_ERR_CUDA (launch failure).
 */
ATTN_API attn_status_t attn_fwd(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H, int Tq,
                       int Tk, int d, int dv, float scale, int causal, attn_dtype_t dtype, void* stream);

/*
 * Forward pass of the fp32 path with an explicit key-tile size (keys per
 * online-softmax step): block_n in {32, 64, 128}. The result must not depend
 * on it ("Tiled attention with an online softmax", section "Constraints":
 * equal to standard attention for every block size). attn_fwd uses 64.
 * Same arguments and errors as attn_fwd with dtype ATTN_F32.
 */
ATTN_API attn_status_t attn_fwd_f32_blocked(const float* Q, const float* K, const float* V, float* O, float* LSE, int B,
                                   int H, int Tq, int Tk, int d, int dv, float scale, int causal, int block_n,
                                   void* stream);

/*
 * Split-KV forward for problems with few query tiles per SM (small B*H*Tq,
 * long Tk): the key tiles of every query-tile unit (bf16: a pair of 128-row
 * query tiles, one tile for d = 256, 128-key tiles; fp32: one 64-row query
 * tile, 64-key tiles) are divided into S contiguous ranges ("splits") that
 * run as separate work units; each
 * writes its partial softmax state for its keys (O_s = A_s / l_s and LSE_s,
 * fp32) to `workspace`, and a merge kernel combines the splits with the
 * associative rescale of the running max, sum and accumulator ("The Hidden
 * Recurrence in Softmax Attention", section "Chunk-wise Mode with Online
 * Softmax Re-scale": chunk states rescaled to a common maximum and added):
 *   M = max_s LSE_s, w_s = exp(LSE_s - M), O = sum_s w_s O_s / sum_s w_s,
 *   LSE = M + log sum_s w_s.
 * Same inputs, outputs, layout and mask as attn_fwd; O and LSE agree with
 * attn_fwd up to fp32 rounding order. num_splits = 0 picks S from the
 * current device's SM count: the smallest S whose time (the waves of units
 * x S work units over the SMs, times the key tiles of a split) is within 5 %
 * of the best, at least two key tiles per split; a bf16 problem with at
 * least as many units as SMs keeps S = 1. num_splits >= 1 asks for that
 * many, clamped to the number of key tiles and 64. S = 1 is attn_fwd itself (no workspace). `workspace`
 * (256-byte aligned, at least attn_fwd_splitkv_workspace_size bytes, not
 * overlapping any other argument; may be NULL when that is 0) holds Opart
 * [S][B*H*Tq][dv] fp32 then LSEpart [S][B*H*Tq] (fp32 for bf16 problems;
 * fp64 for fp32 ones, whose merge weights exp(LSE_s - max) must keep fp32
 * accuracy at logits in the thousands); else ATTN_ERR_WORKSPACE. Other
 * errors as attn_fwd; asynchronous on `stream`.
 */
ATTN_API attn_status_t attn_fwd_splitkv(const void* Q, const void* K, const void* V, void* O, float* LSE, int B,
                                        int H, int Tq, int Tk, int d, int dv, float scale, int causal,
                                        attn_dtype_t dtype, int num_splits, void* workspace,
                                        size_t workspace_bytes, void* stream);

/*
 * The number of splits S attn_fwd_splitkv uses for these arguments (>= 1;
 * num_splits = 0 consults the current device's SM count), or -1 for invalid
 * arguments.
 */
ATTN_API int attn_fwd_splitkv_splits(int B, int H, int Tq, int Tk, int d, int dv, attn_dtype_t dtype,
                                     int num_splits);

/*
 * Bytes of workspace attn_fwd_splitkv needs (0 when S = 1 or the arguments
 * are invalid).
 */
ATTN_API size_t attn_fwd_splitkv_workspace_size(int B, int H, int Tq, int Tk, int d, int dv, attn_dtype_t dtype,
                                                int num_splits);

/*
 * Bytes of device workspace attn_bwd needs for this problem (0 is possible).
 * Holds -LSE * log2(e) and D = rowsum(dO o O), each [B*H, Tq_pad] fp32 with
 * Tq_pad = Tq rounded up to a multiple of 128, and, for bf16 with d <= 128
 * and deterministic == 0, the fp32 dQ accumulator [B,H,Tq,d], or, with
 * deterministic == 1 and S = attn_bwd_dq_splits(...) > 1 (either dtype), S
 * fp32 partial dQ arrays [S][B,H,Tq,d], and, for bf16 with d <= 128, 256 bytes of counters
 * through which the dQ and dK/dV kernels hand out their work units at run
 * time (reset by each call); each part starts on a 256-byte boundary. For bf16
 * widths other than 64 and 128 it first holds zero-padded bf16 copies of Q,
 * K, V, O, dO and of the three gradients, in rows of the next tile width (64,
 * 128 or 256 columns), then the workspace above for the padded widths; the
 * padded problem's dQ splits are the ones attn_bwd_dq_splits reports.
 * Returns 0 for invalid arguments as well.
 */
ATTN_API size_t attn_bwd_workspace_size(int B, int H, int Tq, int Tk, int d, int dv, attn_dtype_t dtype,
                               int deterministic);

/*
 * Number of key splits S the deterministic backward uses for dQ (1 when it
 * does not split; -1 for invalid arguments). Each query tile's keys are cut
 * into S ranges whose partial dQ go to the workspace and are then added in
 * split order, so the result stays bitwise reproducible. bf16: the dQ kernel
 * runs one unit per 128-row query tile; when there are fewer such units than
 * 76 (half of a GB300's 152 SMs) and at least 8 key tiles, S ranges of at
 * least 4 key tiles each, at most 152 units in all, S <= 64. fp32: with at
 * most 1 GiB of partials (S x B*H*Tq*d*4 bytes for S the number of 64-key
 * tiles), every key tile is a range of its own (S = the number of key tiles):
 * the dK/dV kernel writes each key tile's partial dQ (with one key tile, dQ
 * itself) and no separate dQ pass runs. Otherwise the dQ pass runs one unit
 * per 64-row query tile over ranges of 64-key tiles; S is the smallest count
 * whose time (the waves of units x S on 152 SMs, times the key tiles of a
 * range) is within 5 % of the best, at least two key tiles per range, S <=
 * 64. Rules of the shapes only, so that the workspace size needs no device:
 * the 152 is GB300's SM count, and on a device with another SM count the
 * split stays correct but fills the SMs less evenly.
 */
ATTN_API int attn_bwd_dq_splits(int B, int H, int Tq, int Tk, int d, int dv, attn_dtype_t dtype,
                                int deterministic);

/*
 * Backward pass: dQ, dK, dV from Q, K, V, the forward's O and LSE, and dO.
 * Recomputes P tile by tile from LSE instead of storing it ("The Hidden
 * Recurrence in Softmax Attention", section "Flash Attention Backward Pass":
 * store the row statistics, recompute the attention matrix per tile), forms
 * D = rowsum(dO o O), and accumulates the per-tile gradient terms of
 * "attention_backprop" (sections "Gradient of V and P" through "Gradient of
 * Q and K"). `O` and `LSE` must be the outputs of attn_fwd on the same
 * inputs, scale and mask. deterministic = 1 sums the key tiles' shares of
 * dQ in a fixed order (bitwise reproducible): bf16 in a separate dQ pass;
 * fp32 from one partial per 64-key tile that the dK/dV pass writes, added in
 * key-tile order, or, above 1 GiB of such partials, in a separate dQ pass
 * (attn_bwd_dq_splits). 0 adds each key tile's share with fp32 atomics. For
 * bf16 rows of 256 columns both
 * values run the fixed-order pass: there a dQ kernel, a dV kernel and a dK
 * kernel each hold one 256-column accumulator (tensor memory has room for
 * one next to the score tiles), all bitwise reproducible. `workspace` (256-byte aligned, at least
 * attn_bwd_workspace_size bytes; may be NULL when that is 0) is scratch
 * owned by the caller and overwritten.
 * Errors: as attn_fwd, plus ATTN_ERR_WORKSPACE.
 */
ATTN_API attn_status_t attn_bwd(const void* Q, const void* K, const void* V, const void* O, const float* LSE,
                       const void* dO, void* dQ, void* dK, void* dV, int B, int H, int Tq, int Tk, int d, int dv,
                       float scale, int causal, attn_dtype_t dtype, int deterministic, void* workspace,
                       size_t workspace_bytes, void* stream);

/*
 * The backward split into its launch groups, for measurement: the same
 * arguments as attn_bwd plus `phase`:
 *   1  preprocess: D = rowsum(dO o O) and -LSE * log2(e) (and zeroing of the
 *      fp32 dQ accumulator when deterministic == 0); a no-op for bf16 with
 *      deterministic == 1 and for bf16 rows wider than 128 columns, where
 *      the dQ kernel forms D itself
 *   2  main kernels: phases 5 and 4 in this order
 *   3  dQ conversion from the fp32 accumulator (bf16 with deterministic
 *      == 0), or the in-order sum of the split dQ partials (bf16 with
 *      deterministic == 1 and attn_bwd_dq_splits(...) > 1); a no-op otherwise
 *   4  the dK/dV kernel alone (with deterministic == 0 it also accumulates dQ;
 *      bf16 rows wider than 128 columns: the dV and the dK kernel)
 *   5  the separate dQ kernel alone (deterministic == 1, or bf16 rows wider
 *      than 128 columns; a no-op otherwise); for bf16 it also writes the D
 *      and -LSE * log2(e) phase 4 reads
 *   6  in place of phase 5, the same dQ pass on CTA pairs: two 128-row query
 *      tiles per cluster of two CTAs, each tensor-core product computed for
 *      both at once with the K and V operands split between the two SMs
 *      (bf16, d = 128, deterministic == 1 only, else ATTN_ERR_UNSUPPORTED).
 *      Same results within rounding; attn_bwd does not use it (on GB300 at
 *      B=2 H=16 T=8192 it is slower than phase 5).
 * Calling phases 1, 2, 3 (or 1, 5, 4, 3, or 1, 6, 4, 3) in order on one
 * stream equals one attn_bwd call; phase 0 is attn_bwd itself. Other values
 * give ATTN_ERR_INVALID_ARG.
 */
ATTN_API attn_status_t attn_bwd_phase(const void* Q, const void* K, const void* V, const void* O, const float* LSE,
                                      const void* dO, void* dQ, void* dK, void* dV, int B, int H, int Tq, int Tk,
                                      int d, int dv, float scale, int causal, attn_dtype_t dtype, int deterministic,
                                      void* workspace, size_t workspace_bytes, int phase, void* stream);

/*
 * Size of the static scratch buffer behind attn_bwd_noalloc (64 MiB). A
 * device holds a buffer of this size from the moment the library's code is
 * loaded on it until the process exits. With CUDA's lazy module loading (the
 * default since CUDA 12.2) that moment is the first attn_bwd_noalloc call on
 * the device; with eager loading (CUDA_MODULE_LOADING=EAGER) it is the
 * library's first use of the device.
 */
#define ATTN_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

/*
 * attn_bwd for callers that cannot allocate device memory: a host without
 * its own CUDA allocator or memory pool, a plug-in that may not grow the
 * process's device footprint, or a loop where a cudaMalloc (which can
 * synchronise the device) is not acceptable. The pages have no counterpart
 * to this call; it exists only for such callers.
 *
 * Arguments, layout and results are those of attn_bwd, without the workspace
 * arguments: the workspace lives in a static device buffer of
 * ATTN_NOALLOC_SCRATCH_BYTES inside the library (static device data of the
 * library's module, not a cudaMalloc). The call calls no cudaMalloc,
 * cudaFree or other allocating routine. Problems whose attn_bwd_workspace_size
 * exceeds that size are rejected with ATTN_ERR_WORKSPACE before anything is
 * enqueued (for bf16 with deterministic == 0 the need is about
 * B*H*Tq*(d+2)*4 bytes; deterministic == 1 or fp32 needs about B*H*Tq*8).
 *
 * The first call on a device (with that device current) looks up the
 * buffer's device address, and under lazy module loading that lookup is
 * also what reserves the 64 MiB on the device, so it can fail with
 * ATTN_ERR_CUDA (for example while the device's memory is full). Only a
 * successful lookup is kept: after a failure the next call tries again.
 * Make the first call on each device before any stream capture begins.
 * All calls on a device share the one buffer and leave their data in it; each call overwrites everything it reads back (D, and the fp32
 * dQ accumulator, which it zeroes first). Calls whose kernels can overlap on
 * the GPU (different streams without ordering, or several host threads) race
 * on the buffer and corrupt each other's gradients: order them on one stream.
 */
ATTN_API attn_status_t attn_bwd_noalloc(const void* Q, const void* K, const void* V, const void* O,
                                        const float* LSE, const void* dO, void* dQ, void* dK, void* dV, int B,
                                        int H, int Tq, int Tk, int d, int dv, float scale, int causal,
                                        attn_dtype_t dtype, int deterministic, void* stream);

/*
 * Scored attention: softmax attention whose scores are changed before the
 * softmax and whose mask is one range of keys per query row, with query heads
 * that share key heads. With x = scale * q_i . k_j, for query row i of query
 * head h and key j of key head h / (H / Hkv):
 *   t    = softcap * tanh(x / softcap)            (x itself when softcap == 0)
 *   S_ij = t - slopes[h] * |q_pos[b,i] - j|       (t itself when slopes == NULL)
 *   S_ij = -inf unless key_begin[b,i] <= j < key_end[b,i], and, with
 *          causal = 1, j <= q_pos[b,i]
 * and O, LSE as above. Causal, document (rows see their own document's keys),
 * prefix (rows see a prefix and what precedes them), sliding-window and padding
 * masks are all of this form. A row whose range is empty gives O = 0, LSE =
 * -inf and zero gradients, whatever other rows see. The three arrays are shared
 * by the heads of a batch entry; ranges are clamped to [0, Tk] and positions to
 * +-2^30 on the device, so any values are safe. The struct is read during the
 * call; the arrays it points to are device memory read by the enqueued kernels.
 */
typedef struct {
  float softcap;        /* 0: none; otherwise from 1e-4 to 1e6 */
  int causal;           /* 0 or 1 */
  const float* slopes;  /* [H] fp32, or NULL: no bias; any sign, slope times distance within fp32's range */
  const int* q_pos;     /* [B,Tq] int32, or NULL: row i is at position i */
  const int* key_begin; /* [B,Tq] int32, or NULL: 0 */
  const int* key_end;   /* [B,Tq] int32, or NULL: Tk */
} attn_score_t;

/*
 * Forward pass of the scored attention: O and LSE.
 * Layout: Q [B,H,Tq,d], K [B,Hkv,Tk,d], V [B,Hkv,Tk,dv], O [B,H,Tq,dv], LSE
 * [B,H,Tq] fp32; H a multiple of Hkv >= 1, heads of a group adjacent (query
 * head h reads key head h / (H / Hkv)). score = NULL: plain scores, no mask.
 * ATTN_F32: 1 <= d, dv <= 128; ATTN_BF16: d and dv multiples of 8 up to 128;
 * else ATTN_ERR_UNSUPPORTED. Tq, Tk <= 2^30, and H / Hkv * Tq too.
 * What no query reads may hold anything, NaN included: K and V rows that lie
 * before every range or behind every range of their batch entry (unused
 * capacity of a cache), and Q rows whose range is empty (padding); K and V rows
 * in gaps between ranges have to be finite. (ATTN_BF16 with a cap: scores near
 * by, seen or not, decide which of several forms of tanh, equal to a few 2^-24
 * of a score, a row's scores go through, and so may its last bits.) A NaN among
 * the scores that a row sees makes its O and LSE NaN; one in a value that it
 * sees makes that element of its O NaN, whatever the weight.
 * `workspace`: as in attn_fwd_splitkv (256-byte aligned, at least
 * attn_fwd_scored_workspace_size bytes, not overlapping any argument), else
 * ATTN_ERR_WORKSPACE; it is scratch, overwritten by each call, so calls that
 * may overlap on the GPU need one each. Other errors as attn_fwd;
 * asynchronous on `stream`; equal calls give bitwise equal results.
 */
ATTN_API attn_status_t attn_fwd_scored(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H,
                                       int Hkv, int Tq, int Tk, int d, int dv, float scale, const attn_score_t* score,
                                       attn_dtype_t dtype, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Bytes of workspace attn_fwd_scored needs (0 is possible; 0 for invalid
 * arguments as well). A rule of the shapes only.
 */
ATTN_API size_t attn_fwd_scored_workspace_size(int B, int H, int Hkv, int Tq, int Tk, int d, int dv,
                                               attn_dtype_t dtype);

/*
 * Backward pass of the scored attention: dQ [B,H,Tq,d], dK [B,Hkv,Tk,d] and
 * dV [B,Hkv,Tk,dv], the last two summed over the query heads that share the
 * key head. With T_ij = 1 - (t_ij / softcap)^2 (1 without a cap):
 *   P = exp(S - LSE),  D = rowsum(dO o O),  dV = P^T dO,
 *   dS = P o (dO V^T - D) o T,  dQ = scale * dS K,  dK = scale * dS^T Q
 * (the bias and the ranges have no gradient). `O` and `LSE` must be the outputs
 * of attn_fwd_scored on the same inputs, scale and score. (Those of a row over
 * more keys than the call holds give that row's share of the gradients.)
 * ATTN_BF16: D is formed from the rounded O and corrected by rowsum(P o dP),
 * which it equals, where a row's P sums to 1. Shapes as attn_fwd_scored. What
 * no query reads may hold anything here too: K and V rows before every range or
 * behind every range of their batch entry, and Q, O and dO rows whose range is
 * empty; their gradients are 0. Sums run in a fixed order: equal calls give
 * bitwise equal results. Workspace and errors as attn_fwd_scored, with
 * attn_bwd_scored_workspace_size.
 */
ATTN_API attn_status_t attn_bwd_scored(const void* Q, const void* K, const void* V, const void* O, const float* LSE,
                                       const void* dO, void* dQ, void* dK, void* dV, int B, int H, int Hkv, int Tq,
                                       int Tk, int d, int dv, float scale, const attn_score_t* score,
                                       attn_dtype_t dtype, void* workspace, size_t workspace_bytes, void* stream);
ATTN_API size_t attn_bwd_scored_workspace_size(int B, int H, int Hkv, int Tq, int Tk, int d, int dv,
                                               attn_dtype_t dtype);

/*
 * Rotary positions. Pair i (of rot / 2) of a head's first rot elements, (u,
 * v) = (x[2i], x[2i + 1]) with interleaved = 1 and (x[i], x[i + rot / 2])
 * with interleaved = 0, is turned by the angle a = pos * f_i:
 *   u' = m (u cos a - v sin a),  v' = m (v cos a + u sin a)
 * and the elements from rot on are copied. The plan holds each f_i as a
 * 64-bit fraction of a turn, so pos * f_i modulo one turn is one integer
 * product, off by at most |pos| * 2^-65 turns at any int32 position; its
 * upper 32 bits go on (2^-32 turns: 1.5e-9 radians).
 */
#define ATTN_ROPE_MAX_PAIRS 128
typedef struct {
  int rot;                                        /* rotated elements of a head, even, 2..256 */
  int interleaved;                                /* 0: pairs (i, i + rot/2); 1: pairs (2i, 2i + 1) */
  float mscale;                                   /* m above */
  int reserved;
  unsigned long long turns[ATTN_ROPE_MAX_PAIRS];  /* f_i / (2 pi) * 2^64 */
} attn_rope_t;

/*
 * Fills a plan (host only). Base frequencies f_i = theta^(-2i / rot). A
 * context stretched by `factor` >= 1: with original_length == 0 every f_i is
 * divided by it (positions interpolated); otherwise, with r = original_length
 * * f_i / (2 pi) the turns a pair makes over the original context, pairs with
 * r >= high_turns keep f_i, pairs with r <= low_turns take f_i / factor, and
 * the ones between a mixture linear in r. Errors: ATTN_ERR_INVALID_ARG (rot
 * odd, < 2 or > 256; theta <= 1; factor < 1; original_length < 0; unless 0 <=
 * low_turns < high_turns with original_length > 0; mscale <= 0; anything not
 * finite; plan NULL).
 */
ATTN_API attn_status_t attn_rope_init(attn_rope_t* plan, int rot, int interleaved, double theta, double factor,
                                      double original_length, double low_turns, double high_turns, double mscale);

/*
 * Rotates the queries and keys of B * T tokens: Q [B,H,T,d] -> Qout and K
 * [B,Hkv,T,d] -> Kout, any H, Hkv >= 0 (0: none, pointers ignored). inverse
 * = 1 turns by -a: the transpose, which is the gradient (dQ from dQout).
 * strides: 12 element strides, those of batch, head and token for Q, Qout, K
 * and Kout in this order; rows of d elements are contiguous. Strides are >=
 * 0; Qout and Kout must place no two elements at one address. In place (Qout
 * == Q with equal strides) is allowed; otherwise a call is refused where a row
 * of an output shares a byte with a row of an input, of the other output or
 * with pos. Slices and permutations of one tensor are told apart; views so
 * tangled that 16384 steps do not decide are refused. pos: int32 [B,T] device
 * positions of any sign, or NULL: token t is at position t. rot <= d <= 256.
 * Pointers aligned to the element size. cos, sin and the products are fp32,
 * rounded once to the type. Errors: ATTN_ERR_INVALID_ARG,
 * ATTN_ERR_UNSUPPORTED (d > 256), ATTN_ERR_MISALIGNED, ATTN_ERR_CUDA.
 * Asynchronous on `stream`; the plan and the strides are read during the call.
 */
ATTN_API attn_status_t attn_rope(const attn_rope_t* plan, const void* Q, void* Qout, const void* K, void* Kout,
                                 const long long* strides, const int* pos, int B, int H, int Hkv, int T, int d,
                                 int inverse, attn_dtype_t dtype, void* stream);

/*
 * A paged key-value cache. The pool holds `pages` pages of `page` tokens for
 * every key head: k [pages, Hkv, page, d] and v [pages, Hkv, page, dv]. Token j
 * of sequence b is row j % page of page table[b][j / page]. Sequence b holds
 * seq_len[b] tokens, those of the current call included; the last n_b of them
 * are the call's new ones, n_b = new_len[b] or, with new_len NULL, all T (Tq)
 * tokens of the call. Token t < n_b of a call's tensors is then token
 * seq_len[b] - n_b + t of its sequence; the rows t >= n_b are padding, may hold
 * anything and are left out. All arrays are device memory, any values are safe:
 * lengths are clamped to [0, 2^30] and n_b to [0, T]; a token without a place
 * (a negative index, one behind max_pages, a page outside [0, pages)) is not
 * written, and reads as zeros.
 * Types: ATTN_CACHE_PLAIN: elements of the call's dtype, no scales.
 * ATTN_CACHE_E4M3: 8-bit floats (4 exponent and 3 mantissa bits, largest value
 * 448) that stand for their value times one scale per page and head, k_scale
 * and v_scale [pages, Hkv] fp32; scales read as clamped to [2^-40, 2^40].
 * Widths: ATTN_CACHE_E4M3 multiples of 16, ATTN_CACHE_PLAIN with ATTN_BF16
 * multiples of 8, with ATTN_F32 any. page: 16, 32, 64 or 128. Pools aligned to
 * 16 bytes (ATTN_CACHE_PLAIN with ATTN_F32: 4).
 */
typedef enum { ATTN_CACHE_PLAIN = 0, ATTN_CACHE_E4M3 = 1 } attn_cache_type_t;
typedef struct {
  void* k;
  void* v;
  float* k_scale;      /* ATTN_CACHE_E4M3 only */
  float* v_scale;
  const int* table;    /* [B, max_pages] */
  const int* seq_len;  /* [B] */
  const int* new_len;  /* [B], or NULL */
  int pages;           /* of the pool, >= 1 */
  int page;            /* tokens of a page */
  int max_pages;       /* of a sequence */
  int type;            /* attn_cache_type_t */
} attn_cache_t;

/*
 * Appends T tokens of each sequence: their keys, rotated by the plan (NULL: as
 * they are), and their values go to their places in the cache, and their
 * queries are rotated on the way (Q [B,H,T,d] -> Qout; H = 0: none, pointers
 * ignored; H > 0 needs a plan). K [B,Hkv,T,d], V [B,Hkv,T,dv]. strides: 12
 * element strides, those of batch, head and token for Q, Qout, K and V in this
 * order; rows are contiguous. pos: int32 [B,T] rotary positions, or NULL: a
 * token's index in its sequence. d, dv <= 256. Rows of Qout behind n_b are left
 * as they were, and so is all of the cache but the new tokens' rows (and what
 * the next paragraph says).
 * ATTN_CACHE_E4M3: the call's new tokens in a page ask for the scale 2^e, e the
 * least integer with a <= 448 * 2^e, at least -40 and at most 40, where a is
 * the largest of |v|, or of |k| before the rotation, the rotated elements times
 * 1.4142137 * mscale (which bounds what any rotation makes of them). A page
 * whose first token is new takes that scale; one that holds tokens keeps the
 * larger of the two, and where that is the new one, the tokens that it holds
 * are requantised. Elements are rounded once, to the nearest (ties to even; the
 * largest is 448; by a kept scale that is no power of two after the quotient's
 * own rounding to fp32). Those that are not finite do not count towards a and are
 * stored as NaN.
 * A page may be appended to for one sequence of a call only; where two append
 * to it, what it then holds is unspecified.
 * Overlap rules as attn_rope's (Qout may be Q with equal strides); the pools,
 * scales and Qout may share no byte with another argument. Errors:
 * ATTN_ERR_INVALID_ARG, ATTN_ERR_UNSUPPORTED, ATTN_ERR_MISALIGNED,
 * ATTN_ERR_CUDA. Asynchronous on `stream`; the structs and the strides are read
 * during the call.
 */
ATTN_API attn_status_t attn_cache_append(const attn_cache_t* cache, const attn_rope_t* plan, const void* Q, void* Qout,
                                         const void* K, const void* V, const long long* strides, const int* pos, int B,
                                         int H, int Hkv, int T, int d, int dv, attn_dtype_t dtype, void* stream);

/*
 * Reads tokens [0, Tk) of each sequence: K [B,Hkv,Tk,d] and V [B,Hkv,Tk,dv],
 * contiguous, zeros from seq_len[b] on. d, dv <= 256. ATTN_CACHE_E4M3: each
 * element is code times scale, rounded once to dtype (exact for scales that are
 * powers of two). Errors as attn_cache_append; asynchronous on `stream`.
 */
ATTN_API attn_status_t attn_cache_read(const attn_cache_t* cache, void* K, void* V, int B, int Hkv, int Tk, int d,
                                       int dv, attn_dtype_t dtype, void* stream);

/*
 * Scored attention (attn_fwd_scored) of each sequence's newest tokens over its
 * cache: Q [B,H,Tq,d], O [B,H,Tq,dv], LSE [B,H,Tq] contiguous, keys [0, Tk) of
 * the cache; Tk a bound of the lengths known on the host, at most max_pages *
 * page. As there, but: without score->q_pos, row i is at position seq_len[b] -
 * n_b + i, its place in the sequence; every range also ends at min(seq_len[b],
 * Tk); with window > 0 it also begins at position - window + 1 or later; rows i
 * >= n_b see nothing. score = NULL: plain scores, all of the sequence's keys.
 * d, dv <= 128. What no query reads may hold anything, as there: tokens behind
 * a sequence's length, before every range of its rows or behind every one, and
 * the scales and table entries of pages that lie wholly there.
 * Up to 128 packed rows a key head (H / Hkv * Tq) the pages are read where they
 * lie (with ATTN_F32, where they hold e4m3); with more rows the seen tokens are
 * read into the workspace first, as by attn_cache_read, so that scales that are
 * no powers of two cost a rounding to dtype; it then grows with B * Hkv * Tk. Q
 * and O aligned to 16 bytes (ATTN_CACHE_PLAIN with ATTN_F32: 4). Scales may lie
 * as far apart as they like: a page of zeros, or of tokens that no row sees,
 * does not cost the others' values their bits.
 * Workspace as attn_fwd_scored, with attn_fwd_cached_workspace_size: a rule of
 * the shapes and types only (0 is possible). Other errors as attn_cache_append and
 * attn_fwd_scored; asynchronous on `stream`; equal calls give bitwise equal
 * results.
 */
ATTN_API attn_status_t attn_fwd_cached(const void* Q, const attn_cache_t* cache, void* O, float* LSE, int B, int H,
                                       int Hkv, int Tq, int Tk, int d, int dv, float scale, int window,
                                       const attn_score_t* score, attn_dtype_t dtype, void* workspace,
                                       size_t workspace_bytes, void* stream);
ATTN_API size_t attn_fwd_cached_workspace_size(int B, int H, int Hkv, int Tq, int Tk, int d, int dv, int cache_type,
                                               attn_dtype_t dtype);

/*
 * One step of the online softmax, on the device: for each of the n query
 * rows, fold one block of bs keys into the running state ("Tiled attention
 * with an online softmax", section "Task": the online_softmax_step of the
 * page; "The Hidden Recurrence in Softmax Attention", section "Chunk-wise
 * Mode with Online Softmax Re-scale"):
 *   m' = max(m, max_j s_ij), with 0 used for m' inside the exponentials when
 *        m' = -inf (a row with no allowed key so far)
 *   l' = exp(m - m') l + sum_j exp(s_ij - m')
 *   acc' = exp(m - m') acc + sum_j exp(s_ij - m') v_j
 * m, l [n] and acc [n, dv] (row-major) are fp32 device buffers updated in
 * place; a fresh row is m = -inf, l = 0, acc = 0, and acc / l is its
 * attention output once every block has been folded in. scores [n, bs] fp32
 * (-inf marks a blocked key) and v_block [bs, dv] fp32 are read only. The
 * arithmetic runs in fp64. n, bs >= 0 and 1 <= dv <= 512; buffers 4-byte
 * aligned, the three outputs disjoint from each other and from the inputs,
 * else ATTN_ERR_INVALID_ARG / ATTN_ERR_MISALIGNED before any launch.
 * Asynchronous on `stream`.
 */
ATTN_API attn_status_t attn_online_softmax_step(float* m, float* l, float* acc, const float* scores,
                                                const float* v_block, int n, int bs, int dv, void* stream);

/*
 * Synchronises `stream`, then reads and clears the device status word that
 * the kernels set when a bounded wait gives up (ATTN_ERR_TIMEOUT) or a launch
 * precondition fails on the device (ATTN_ERR_CUDA). ATTN_OK otherwise.
 * Intended for tests and debugging; it blocks the host.
 */
ATTN_API attn_status_t attn_device_status(void* stream);

/*
 * Test hook for the bounded wait itself: launches one CTA that waits on an
 * mbarrier nobody arrives at, with a limit of `limit_ms` milliseconds
 * (1..5000). The kernel gives up, records ATTN_ERR_TIMEOUT in the device
 * status word and exits normally; the context stays usable. Returns the
 * launch status; read the outcome with attn_device_status().
 */
ATTN_API attn_status_t attn_selftest_wait_timeout(int limit_ms, void* stream);

/* Human-readable text for a status code (static storage). */
ATTN_API const char* attn_strerror(attn_status_t status);

/* The cudaError_t (as int) of the last ATTN_ERR_CUDA on this thread, else 0. */
ATTN_API int attn_last_cuda_error(void);

/* Library ABI version: (major << 16) | minor. */
ATTN_API int attn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_H_ */
