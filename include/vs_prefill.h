/*
 * vs_prefill.h -- C ABI of libvs, vertical-slash sparse prefill attention on
 * NVIDIA B200 (sm_100a).
 *
 * The method (VSPrefill summary pages, "VSPrefill: Vertical-Slash Sparse
 * Attention with Lightweight Indexing for Long-Context Prefilling"):
 *   - attention in long-context prefill concentrates on vertical lines (key
 *     columns that every later query attends to) and slash lines (diagonals at
 *     a fixed relative offset o = i - j)  -- Technical Summary, section 2,
 *     "Core Concept: Vertical-Slash Pattern";
 *   - a light indexer predicts one score per column and one per offset from
 *     concat(K with RoPE, V)  -- section 2, "VSIndexer";
 *   - a cumulative threshold on those scores picks the budgets (k_v, k_s)
 *     -- section 2, "Adaptive Inference Pipeline", "Dynamic Budgeting";
 *   - a fused FlashAttention-style kernel attends each query to the union of
 *     the selected columns and the keys at the selected offsets behind it,
 *     without a precomputed mask -- section 2, "Fused Kernel Execution".
 *
 * Conventions for every call:
 *   - Every pointer argument is a DEVICE pointer on the current CUDA device
 *     (except `flags` of vs_read_device_status); the caller owns every buffer (inputs,
 *     outputs, workspace) and the stream.  The library allocates nothing,
 *     keeps no mutable global state (vs_sparse_attn_fwd_static_scratch is the
 *     one documented exception), never writes its inputs and overwrites its
 *     outputs completely.
 *   - Calls are asynchronous on `stream`; selected counts stay on the device,
 *     so select -> attention needs no host synchronisation.
 *   - Host-side argument checks run before anything is launched and return
 *     VS_ERR_INVALID_ARG / VS_ERR_UNSUPPORTED / VS_ERR_WORKSPACE.  A failed
 *     launch returns VS_ERR_CUDA.  Device-side problems (an index outside
 *     [0, N), a count above its row length, a bounded wait that gave up) are
 *     OR-ed into a status word at the start of the workspace; read it with
 *     vs_read_device_status.  Kernels never trap, assert or print.
 *   - Tensors are token-major: element (t, h, c) of Q lives at
 *     Q[t * q_stride_tok + h * d + c]; K and V likewise with kv_stride_tok.
 *     Strides are in elements and must be multiples of 8 (16-byte rows).
 *   - GQA: query head h reads KV head h / (Hq / Hkv) and index-set head
 *     h * H_sel / Hq.
 */
#ifndef VS_PREFILL_H
#define VS_PREFILL_H

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  VS_OK = 0,
  VS_ERR_INVALID_ARG = 1,    /* null pointer, bad size, k/cap/tau out of range */
  VS_ERR_UNSUPPORTED = 2,    /* valid but not implemented (e.g. d not in {64,128}) */
  VS_ERR_WORKSPACE = 3,      /* workspace missing, misaligned or too small */
  VS_ERR_CUDA = 4,           /* a CUDA runtime call or launch failed */
  VS_ERR_DEVICE_TIMEOUT = 5, /* returned by vs_read_device_status */
  VS_ERR_DEVICE_BOUNDS = 6   /* returned by vs_read_device_status */
} vs_status;

typedef enum { VS_SELECT_TOPK = 0, VS_SELECT_THRESHOLD = 1, VS_SELECT_MAXFRAC = 2 } vs_select_mode;

typedef enum { VS_BF16 = 0, VS_FP32 = 1 } vs_dtype;

/* Device status bits (vs_read_device_status `flags`). */
#define VS_DEVFLAG_TIMEOUT 0x1
#define VS_DEVFLAG_BOUNDS 0x2

/* Static, human-readable name of a status code. */
const char* vs_status_string(vs_status s);

/* Library version as MAJOR*10000 + MINOR*100 + PATCH. */
int vs_version(void);

/*
 * vs_index_scores -- the indexer: a shared-weight two-layer linear map on
 * concat(K with RoPE, V) producing a vertical and a slash score per position
 * (Technical Summary, section 2, "VSIndexer": input concatenated K and V with
 * RoPE on K, a bilayer linear network with separate down-projection heads for
 * the vertical and slash scores, linear cost in n).  The pages do not fix the
 * exact form; this library reads it as
 *     x = [k_t ; v_t] (2d values, k first),  h = ReLU(W1 x),
 *     logits_v[g][t] = W2[0] . h,  logits_s[g][t] = W2[1] . h,
 * no biases, one weight set shared by all KV heads g.  logits_s[g][t] is the
 * score of slash offset o = t.
 *   K, V      [N, Hkv, d] in `dtype` (VS_BF16 or VS_FP32), token stride
 *             `stride_tok`, head stride `stride_head` (elements).
 *   W1        fp32 [hidden][2d] row-major (device).   W2  fp32 [2][hidden].
 *   hidden    1..1024.
 *   logits_v, logits_s   fp32 [Hkv][N] outputs (device), fully overwritten.
 * Arithmetic: bf16 K/V with d = 64 or 128, hidden = 128 or 256, stride_head
 * = d and 16-byte aligned rows run on the tensor cores.  There W1 is split
 * into two bf16 parts (hi = bf16(W1), lo = bf16(W1 - hi)), the products are
 * exact and the accumulation is fp32; the result is deterministic (at most
 * two partial sums per logit, added onto zero).  Other inputs run in fp32 on
 * the CUDA cores.  The tensor-core kernel's device waits are bounded; a wait
 * that runs out (never on a correct launch) leaves NaN in the logits of the
 * tiles it affects, since this call has no workspace status word.
 */
vs_status vs_index_scores(const void* K, const void* V, vs_dtype dtype, int N, int Hkv, int d,
                          int64_t stride_tok, int64_t stride_head, const float* W1,
                          const float* W2, int hidden, float* logits_v, float* logits_s,
                          cudaStream_t stream);

/*
 * vs_select -- per-head budget selection over a score vector (Technical
 * Summary, section 2, "Dynamic Budgeting": a cumulative-threshold strategy
 * sets the budgets from the predicted importance scores; the German page's
 * Inferenz-Pipeline adds the top-k reading).  One call handles H heads.
 *   scores   fp32 [H][ld_scores] (device), the first N entries of each row used.
 *            Scores are logits: the "mass" of entry r is softmax(scores)_r.
 *   Order    score descending, NaN after -inf, ties to the smaller index.
 *   TOPK     keeps the first k_or_cap entries in that order.
 *   THRESHOLD keeps the smallest prefix in that order whose mass reaches
 *            tau (0 < tau <= 1): p_r = exp(s_r - s_max) in fp64, k is the
 *            smallest k >= 1 with sum_{r<k} p_r >= tau * sum_r p_r; tau = 1
 *            keeps every entry with p_r > 0; then k = min(k, k_or_cap).
 *   MAXFRAC  FlashPrefill's max-based dynamic threshold (FlashPrefill summary
 *            page, section 2B: discard every candidate scoring below alpha
 *            times the best one; no sort, no cumulative sum).  `tau` carries
 *            alpha (0 < alpha <= 1); with the mass reading the rule is
 *            p_r >= alpha, decided in fp64 as
 *              s_r == s_max  or  (double)s_r - (double)s_max >= log(alpha)
 *            (log taken on the host); NaN is never kept, an all-NaN row
 *            keeps one entry; then k = min(k, k_or_cap) in the order above.
 *   idx      int32 [H][ld_idx] (device): for each head the kept indices in
 *            ascending order, then -1 up to k_or_cap (entries past k_or_cap
 *            untouched).  ld_idx >= k_or_cap.
 *   count    int32 [H] (device): kept entries per head.
 *   ws       device workspace of at least vs_select_workspace_size(H, N)
 *            bytes, 256-byte aligned (holds the device status word).
 * Requires 1 <= k_or_cap <= N <= 2^20; tau in (0, 1] for THRESHOLD and
 * MAXFRAC (else VS_ERR_INVALID_ARG).
 * The fp64 mass sums are added in a fixed order (no atomics), so repeated
 * calls with the same H and N on the same device give the same result bit
 * for bit.  That order follows the thread-block cluster the launcher picks,
 * which depends on H, N and the device's SM count: a row selected in a call
 * with another H or N, or on another device, may be summed in another order,
 * and where the decision lies within rounding of tau * sum_r p_r it may then
 * differ by one entry.
 */
size_t vs_select_workspace_size(int H, int N);
vs_status vs_select(const float* scores, int H, int N, int64_t ld_scores, vs_select_mode mode,
                    int k_or_cap, double tau, int32_t* idx, int64_t ld_idx, int32_t* count,
                    void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * vs_select_varlen -- vs_select for B sequences packed along the token axis,
 * in one launch (the budget step of a batched prefill: each sequence's
 * vertical or slash scores select that sequence's index set).
 *   scores     fp32 [H][total_tokens] (device): head h of sequence b is
 *              scores[h * total_tokens + cu_seqlens[b] + j], j < n_b.
 *   cu_seqlens int32 [B + 1] (device), as for vs_sparse_attn_fwd_varlen;
 *              max_seqlen >= every n_b (host; sizes the launch).
 *   caps       int32 [B] (device): k_or_cap of sequence b, 1 <= caps[b] <=
 *              n_b and <= cap_max; cap_max >= 1 and ld_idx >= cap_max.
 *   mode, tau  as for vs_select, applied to every row.
 *   idx        int32 [B * H][ld_idx] (device): row b * H + h as vs_select's
 *              row for that sequence and head (indices from the sequence's
 *              start, ascending, then -1 up to caps[b]; entries past caps[b]
 *              untouched) -- the layout vs_sparse_attn_fwd_varlen reads.
 *   count      int32 [B * H] (device).
 *   ws         device workspace of at least
 *              vs_select_workspace_size_varlen(B, H, max_seqlen) bytes,
 *              256-byte aligned (status word).
 * A sequence with n_b = 0 keeps nothing (count 0, its rows untouched).  A
 * malformed offset or cap empties that sequence the same way and sets
 * VS_DEVFLAG_BOUNDS.  B * H <= 65535; max_seqlen <= 2^20.  The fp64 sums
 * are in a fixed order for a given (B, H, max_seqlen) and device, as for
 * vs_select (the order follows the cluster the launcher picks for B * H rows
 * of max_seqlen, so it may differ from a single-sequence call's).
 */
size_t vs_select_workspace_size_varlen(int B, int H, int max_seqlen);
vs_status vs_select_varlen(const float* scores, int total_tokens, int B, const int32_t* cu_seqlens,
                           int max_seqlen, int H, vs_select_mode mode, const int32_t* caps,
                           int cap_max, double tau, int32_t* idx, int64_t ld_idx, int32_t* count,
                           void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * vs_sparse_attn_fwd -- causal vertical-slash sparse attention forward
 * (Technical Summary, section 2, "Fused Kernel Execution": the vertical and
 * slash index lists are merged on the fly inside a FlashAttention-style
 * kernel, with no precomputed mask).  For query i of query head h:
 *     K_i = { j in V : j <= i }  union  { i - o : o in S, o <= i }
 * (each key once), and O_i = softmax_j(scale * q_i . k_j) over K_i times V;
 * LSE_i = log sum_{j in K_i} exp(scale * q_i . k_j).  An empty K_i gives
 * O_i = 0 and LSE_i = -inf.
 *   Q        [N, Hq, d], K, V [N, Hkv, d], `dtype` (VS_BF16: tensor-core path;
 *            VS_FP32: fp32 CUDA-core path).  d in {64, 128}.  Hq % Hkv == 0.
 *            1 <= N <= 2^22 (dense: 2^24).
 *   softmax_scale   0 selects 1/sqrt(d).
 *   H_sel    number of index sets; Hq % H_sel == 0.
 *   v_idx    int32 [H_sel][v_ld] vertical columns, v_cnt int32 [H_sel];
 *   s_idx    int32 [H_sel][s_ld] slash offsets,   s_cnt int32 [H_sel]
 *            (device; as produced by vs_select: entries in [0, N), the first
 *            cnt entries of each row used; duplicates and order do not matter).
 *   O        [N, Hq, d] in `dtype` with token stride q_stride_tok (output).
 *   lse      fp32 [Hq][N] (output) or NULL.
 *   ws       device workspace, 256-byte aligned, of at least
 *            vs_attn_workspace_size(N, Hq, H_sel, d) bytes (the plan).  With
 *            vs_attn_workspace_size_ld(N, Hq, H_sel, d, v_ld) bytes or more the
 *            selected vertical K/V rows are first packed contiguously and then
 *            loaded as tiles (when every index set's query heads lie in one KV
 *            group); with less they are gathered row by row.  Results are the
 *            same either way.
 */
size_t vs_attn_workspace_size(int N, int Hq, int H_sel, int d);
size_t vs_attn_workspace_size_ld(int N, int Hq, int H_sel, int d, int64_t v_ld);
vs_status vs_sparse_attn_fwd(const void* Q, const void* K, const void* V, vs_dtype dtype, int N,
                             int Hq, int Hkv, int d, int64_t q_stride_tok, int64_t kv_stride_tok,
                             float softmax_scale, int H_sel, const int32_t* v_idx, int64_t v_ld,
                             const int32_t* v_cnt, const int32_t* s_idx, int64_t s_ld,
                             const int32_t* s_cnt, void* O, float* lse, void* ws,
                             size_t ws_bytes, cudaStream_t stream);

/*
 * vs_sparse_attn_fwd_varlen / vs_dense_attn_fwd_varlen -- the same attention
 * over a batch of B independent sequences packed along the token axis
 * (variable-length batched prefill; each sequence attends only to itself).
 *   total_tokens  rows of Q, K, V, O (and columns of lse: lse is fp32
 *            [Hq][total_tokens]); at most 2^31 - 1.
 *   cu_seqlens    int32 [B + 1] (DEVICE): sequence b is tokens
 *            [cu_seqlens[b], cu_seqlens[b + 1]); the offsets must not
 *            decrease, start at >= 0, end at <= total_tokens and give no
 *            sequence longer than max_seqlen.  A malformed entry makes that
 *            sequence empty (its O rows are not written) and sets
 *            VS_DEVFLAG_BOUNDS.
 *   max_seqlen    the longest sequence (sizes the plan; >= 1).
 *   Index sets (sparse): one per (sequence, index-set head): v_idx
 *            [B * H_sel][v_ld] with v_cnt [B * H_sel] (row b * H_sel + hs),
 *            likewise s_idx / s_cnt; positions are relative to the sequence
 *            start (columns and offsets in [0, that sequence's length)).
 *   ws       at least vs_attn_workspace_size_varlen(B, max_seqlen, H_sel, d,
 *            0) bytes (the plan; dense: 256); with v_ld in place of 0, room to
 *            pack the selected vertical rows, as for vs_sparse_attn_fwd.
 *   VS_BF16 only (else VS_ERR_UNSUPPORTED); B * H_sel <= 65535.
 * The pages prefill one sequence at a time; this batching follows their
 * per-sequence definition unchanged.
 */
size_t vs_attn_workspace_size_varlen(int B, int max_seqlen, int H_sel, int d, int64_t v_ld);
vs_status vs_sparse_attn_fwd_varlen(const void* Q, const void* K, const void* V, vs_dtype dtype,
                                    int total_tokens, int B, const int32_t* cu_seqlens,
                                    int max_seqlen, int Hq, int Hkv, int d, int64_t q_stride_tok,
                                    int64_t kv_stride_tok, float softmax_scale, int H_sel,
                                    const int32_t* v_idx, int64_t v_ld, const int32_t* v_cnt,
                                    const int32_t* s_idx, int64_t s_ld, const int32_t* s_cnt,
                                    void* O, float* lse, void* ws, size_t ws_bytes,
                                    cudaStream_t stream);
vs_status vs_dense_attn_fwd_varlen(const void* Q, const void* K, const void* V, vs_dtype dtype,
                                   int total_tokens, int B, const int32_t* cu_seqlens,
                                   int max_seqlen, int Hq, int Hkv, int d, int64_t q_stride_tok,
                                   int64_t kv_stride_tok, float softmax_scale, void* O, float* lse,
                                   void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * vs_block_select -- FlashPrefill's block pattern discovery (FlashPrefill
 * summary page, section 2A: a skeleton of uniformly spaced queries probes
 * every key block through the block's mean key, a proxy that is monotone in
 * the block's total attention weight; section 2B: keep key block J for query
 * block I when its score is at least alpha times the best block's -- no
 * sort, no cumulative sum).  Read as, with 128-row blocks and the probes of
 * block I at rows 128 I + 8 m (m = 0..15, below N):
 *     Score(I, J) = mean over probes q of softmax_{J' < I}(scale q . kbar_J')[J],
 *     J < I kept iff Score(I, J) >= alpha * max_J' Score(I, J'),
 * the diagonal block J = I always kept; computed in fp64.
 *   Q [N, Hq, d], K [N, Hkv, d] (VS_BF16 or VS_FP32; strides as for the
 *            attention calls).  1 <= N <= 2^18.  0 < alpha <= 1.
 *   mask     uint32 [Hq][T][W] output (device), T = ceil(N / 128),
 *            W = ceil(T / 32): bit J of row (h, I) set iff block J is kept.
 *   ws       at least vs_block_select_workspace_size(N, Hkv, d) bytes,
 *            256-byte aligned: status word and work counter, the fp64 block
 *            means, and one dot-product scratch per SM of the current device
 *            (the size depends on that device; a workspace sized on a device
 *            with fewer SMs fails the check with VS_ERR_WORKSPACE).
 */
size_t vs_block_select_workspace_size(int N, int Hkv, int d);
vs_status vs_block_select(const void* Q, const void* K, vs_dtype dtype, int N, int Hq, int Hkv,
                          int d, int64_t q_stride_tok, int64_t kv_stride_tok, float softmax_scale,
                          double alpha, uint32_t* mask, void* ws, size_t ws_bytes,
                          cudaStream_t stream);

/*
 * vs_block_sparse_attn_fwd -- causal attention over kept key blocks
 * (FlashPrefill summary page, section 3: a block-sparse kernel that jumps
 * directly to the next kept block by index).  Query i (block I = i / 128)
 * attends to every key j <= i of every block J kept in row (h, I) of
 * `block_mask` (the layout vs_block_select writes; bits J > I are ignored).
 * O and lse as for vs_sparse_attn_fwd; a row with no kept key gets O = 0 and
 * LSE = -inf.  VS_BF16 only; 1 <= N <= 2^18.
 *   ws       at least vs_block_attn_workspace_size(N, Hq) bytes, 256-byte
 *            aligned (status word and the per-pair block lists).
 */
size_t vs_block_attn_workspace_size(int N, int Hq);
vs_status vs_block_sparse_attn_fwd(const void* Q, const void* K, const void* V, vs_dtype dtype,
                                   int N, int Hq, int Hkv, int d, int64_t q_stride_tok,
                                   int64_t kv_stride_tok, float softmax_scale,
                                   const uint32_t* block_mask, void* O, float* lse, void* ws,
                                   size_t ws_bytes, cudaStream_t stream);

/*
 * vs_block_select_varlen / vs_block_sparse_attn_fwd_varlen -- the block
 * discovery and the block-sparse attention above for B sequences packed along
 * the token axis (batched prefill; FlashPrefill summary page, sections 2A,
 * 2B and 3, applied to each sequence on its own: blocks, probes and the
 * alpha-times-best rule are per sequence, and a sequence attends only to
 * itself).
 *   total_tokens, cu_seqlens, max_seqlen  as for vs_sparse_attn_fwd_varlen
 *            (cu_seqlens on the DEVICE; a malformed entry empties that
 *            sequence and sets VS_DEVFLAG_BOUNDS).
 *   mask / block_mask  uint32 [B][Hq][T][W] with T = ceil(max_seqlen / 128),
 *            W = ceil(T / 32): sequence b's rows of head h at (b * Hq + h) * T;
 *            vs_block_select_varlen writes rows I >= that sequence's block
 *            count as zeros.  Each sequence's rows equal what vs_block_select
 *            writes for that sequence alone (same arithmetic, same order).
 *   O, lse   as for vs_sparse_attn_fwd_varlen (lse fp32 [Hq][total_tokens]).
 *   ws       vs_block_select_workspace_size_varlen(B, max_seqlen, Hkv, d) and
 *            vs_block_attn_workspace_size_varlen(B, max_seqlen, Hq) bytes,
 *            256-byte aligned.
 * Requires 1 <= max_seqlen <= 2^18; VS_ERR_UNSUPPORTED when the batch's
 * per-(sequence, head) block lists would not fit 32-bit offsets.
 */
size_t vs_block_select_workspace_size_varlen(int B, int max_seqlen, int Hkv, int d);
vs_status vs_block_select_varlen(const void* Q, const void* K, vs_dtype dtype, int total_tokens,
                                 int B, const int32_t* cu_seqlens, int max_seqlen, int Hq,
                                 int Hkv, int d, int64_t q_stride_tok, int64_t kv_stride_tok,
                                 float softmax_scale, double alpha, uint32_t* mask, void* ws,
                                 size_t ws_bytes, cudaStream_t stream);
size_t vs_block_attn_workspace_size_varlen(int B, int max_seqlen, int Hq);
vs_status vs_block_sparse_attn_fwd_varlen(const void* Q, const void* K, const void* V,
                                          vs_dtype dtype, int total_tokens, int B,
                                          const int32_t* cu_seqlens, int max_seqlen, int Hq,
                                          int Hkv, int d, int64_t q_stride_tok,
                                          int64_t kv_stride_tok, float softmax_scale,
                                          const uint32_t* block_mask, void* O, float* lse,
                                          void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * vs_sparse_attn_fwd_static_scratch -- vs_sparse_attn_fwd without a
 * caller-provided workspace.  The summary pages have no counterpart to this
 * call; it exists for callers that cannot allocate device memory: plain-C
 * hosts with no device memory manager, and plug-ins inside engines that own
 * every byte of device memory through their own pool and forbid cudaMalloc
 * (which may also synchronise the device mid-prefill).
 *   Same arguments and results as vs_sparse_attn_fwd, minus ws / ws_bytes;
 *   the caller still passes every input and output buffer.
 *   Scratch: one 16 MiB static device array inside libvs, held on every GPU
 *   that loads the library until the process exits.  Calls needing more
 *   (vs_attn_workspace_size(N, Hq, H_sel, d) > 16 MiB) return
 *   VS_ERR_UNSUPPORTED before launching anything.
 *   The first call on a device resolves the array's device address with
 *   cudaGetSymbolAddress (with that device current), and so does the first
 *   call after the device's context has been replaced (cudaDeviceReset): the
 *   address is kept per device together with the ID of the context it was
 *   taken in.  Make the first call on a device (and the first after a reset)
 *   before any stream capture.  No cudaMalloc / cudaFree or other allocating
 *   routine is called.
 *   Every call shares the array, which keeps the last call's contents (the
 *   call clears what it needs to start at zero itself); calls that overlap on
 *   the GPU -- other streams, other host threads -- race on it and must be
 *   serialised by the caller.  The device status word of this call is not
 *   exposed (vs_read_device_status needs a caller-owned workspace).
 */
vs_status vs_sparse_attn_fwd_static_scratch(const void* Q, const void* K, const void* V,
                                            vs_dtype dtype, int N, int Hq, int Hkv, int d,
                                            int64_t q_stride_tok, int64_t kv_stride_tok,
                                            float softmax_scale, int H_sel, const int32_t* v_idx,
                                            int64_t v_ld, const int32_t* v_cnt,
                                            const int32_t* s_idx, int64_t s_ld,
                                            const int32_t* s_cnt, void* O, float* lse,
                                            cudaStream_t stream);

/*
 * vs_dense_attn_fwd -- dense causal attention with the same kernel
 * machinery: the "full attention" the pages measure their speed-ups against
 * (Technical Summary, section 4, Speedup).  Same arguments as
 * vs_sparse_attn_fwd without the index sets; K_i = [0, i].
 */
vs_status vs_dense_attn_fwd(const void* Q, const void* K, const void* V, vs_dtype dtype, int N,
                            int Hq, int Hkv, int d, int64_t q_stride_tok, int64_t kv_stride_tok,
                            float softmax_scale, void* O, float* lse, void* ws, size_t ws_bytes,
                            cudaStream_t stream);

/*
 * vs_window_attn_fwd / vs_window_attn_fwd_varlen -- causal sliding-window
 * attention in which the first keys stay visible: the local-attention layers
 * next to the vertical-slash ones (a window is every slash offset below
 * `window`, the first keys are the vertical columns below `sinks`), without
 * index sets, plan or bitmaps.  Query i of a sequence attends to
 *     K_i = { j <= i : i - j < window  or  j < sinks },
 * each key once; O and lse as for vs_sparse_attn_fwd (a row is never empty:
 * it sees itself).
 *   window   1 .. INT_MAX; at N or above the attention is dense causal.
 *   sinks    0 .. INT_MAX first keys of each sequence (0: none).
 *   Other arguments as for vs_dense_attn_fwd and vs_dense_attn_fwd_varlen
 *            (a malformed cu_seqlens entry leaves that sequence's O rows
 *            unwritten and sets VS_DEVFLAG_BOUNDS; rows of O and lse behind
 *            the last sequence are left as they were).
 *   ws       at least 256 bytes, 256-byte aligned (status word).
 * VS_BF16 only (else VS_ERR_UNSUPPORTED); 1 <= N <= 2^24.
 * Scores, maxima, sums and O are held in fp32; the weights are rounded to bf16
 * for their product with V (as in every bf16 attention of this library): O is
 * off by up to 2^-8 max |V| from that, and by 2^-8 of itself from its own
 * rounding.  lse does not depend on the rounded weights.
 * What lies outside a sequence never reaches its rows, whatever it holds.
 * Inside a sequence V must be finite: an infinity or NaN in V row j also
 * reaches rows that do not see j but share its 128-key block (its weight is
 * 0, and 0 * inf is NaN).  K may hold anything where it is not visible; a row
 * that sees a NaN has O = NaN and lse = NaN.
 */
vs_status vs_window_attn_fwd(const void* Q, const void* K, const void* V, vs_dtype dtype, int N,
                             int Hq, int Hkv, int d, int64_t q_stride_tok, int64_t kv_stride_tok,
                             float softmax_scale, int window, int sinks, void* O, float* lse,
                             void* ws, size_t ws_bytes, cudaStream_t stream);
vs_status vs_window_attn_fwd_varlen(const void* Q, const void* K, const void* V, vs_dtype dtype,
                                    int total_tokens, int B, const int32_t* cu_seqlens,
                                    int max_seqlen, int Hq, int Hkv, int d, int64_t q_stride_tok,
                                    int64_t kv_stride_tok, float softmax_scale, int window,
                                    int sinks, void* O, float* lse, void* ws, size_t ws_bytes,
                                    cudaStream_t stream);

/*
 * vs_attn_aggregate -- ground-truth aggregation of the full causal attention
 * weights along vertical columns and slash diagonals: the indexer's
 * distillation target (Technical Summary, section 2, "Distillation Training":
 * a kernel aggregates full attention weights along the columns and diagonals
 * online during block-wise computation, without the n x n matrix).  For query
 * head h, with p_ij = exp(scale * q_i . k_j - LSE_i) over j <= i:
 *     A_v[h][j] = sum_{i >= j} p_ij,    A_s[h][o] = sum_{i >= o} p_{i, i-o},
 * so each row of A_v and of A_s sums to N (normalise by N for the
 * distributions the distillation loss compares).
 *   Q [N, Hq, d], K [N, Hkv, d]: VS_BF16 only (else VS_ERR_UNSUPPORTED);
 *            d in {64, 128}; strides and GQA as for vs_sparse_attn_fwd.
 *   lse      fp32 [Hq][N] (device): the row log-sum-exp of the same dense
 *            causal attention with the same scale, as written by
 *            vs_dense_attn_fwd.  The weights are only as correct as lse.
 *   A_v, A_s fp32 [Hq][N] outputs (device).  A_s is zeroed by the call and
 *            accumulated with fp32 atomics, so its last bits may vary from
 *            run to run; A_v is written once per entry.
 *   ws       device workspace of at least 256 bytes, 256-byte aligned (status
 *            word).
 */
vs_status vs_attn_aggregate(const void* Q, const void* K, vs_dtype dtype, int N, int Hq, int Hkv,
                            int d, int64_t q_stride_tok, int64_t kv_stride_tok,
                            float softmax_scale, const float* lse, float* A_v, float* A_s,
                            void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * vs_attn_aggregate_varlen -- vs_attn_aggregate for B sequences packed along
 * the token axis (each sequence's weights are its own causal softmax; the
 * sums are per sequence, at positions relative to its start).
 *   total_tokens, cu_seqlens, max_seqlen  as for vs_sparse_attn_fwd_varlen
 *            (cu_seqlens on the DEVICE; a malformed entry leaves that
 *            sequence's entries of A_v unwritten and of A_s zero, and sets
 *            VS_DEVFLAG_BOUNDS).
 *   lse      fp32 [Hq][total_tokens] as written by vs_dense_attn_fwd_varlen.
 *   A_v, A_s fp32 [Hq][total_tokens]: sequence b's column j at
 *            h * total_tokens + cu_seqlens[b] + j, its offset o likewise.
 */
vs_status vs_attn_aggregate_varlen(const void* Q, const void* K, vs_dtype dtype, int total_tokens,
                                   int B, const int32_t* cu_seqlens, int max_seqlen, int Hq,
                                   int Hkv, int d, int64_t q_stride_tok, int64_t kv_stride_tok,
                                   float softmax_scale, const float* lse, float* A_v, float* A_s,
                                   void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * The 4-bit paged key/value cache -- where the keys and values of a prefill
 * go, and the attention of the tokens that follow.  (The summary pages stop at
 * prefill; these calls continue from what this library computes there: the
 * column sums of vs_attn_aggregate are the weights that eviction starts from.)
 *
 * Pool: `n_pages` pages of vs_kv4_page_bytes(Hkv, d) bytes (device, 16-byte
 * aligned; d in {64, 128}).  A page holds 64 slots of every KV head; the bytes
 * of one (page, head) are contiguous, with GR = d / 64:
 *     key codes   [GR][64 slots][32 bytes]    value codes  likewise
 *     key pairs   [GR][64 slots] (s, m) bf16  value pairs  likewise
 * 64 channels (a group) of a slot are eight 32-bit words; bits 4j .. 4j+3 of
 * word w are the code n of channel 8 w + j, which stands for s n + m.
 * Table: int32 [B][table_ld] (device); slots [64 i, 64 i + 64) of sequence b
 * are in page table[b * table_ld + i].  Entries of pages that a call need not
 * touch are not read and may hold anything.  An entry outside [0, n_pages)
 * that is touched sets VS_DEVFLAG_BOUNDS; its slots are not written, or count
 * as invisible.  Sequences may share pages that no call writes.
 * lens: int32 [B] (device), slots in use, the same for every head of a
 * sequence.  max_len (host) bounds them: 1 <= max_len <= 2^24, and at most
 * 64 table_ld.  A length outside [0, max_len] counts as 0 and sets
 * VS_DEVFLAG_BOUNDS.  B * Hkv <= 65535.
 * All calls are asynchronous and read lens, table and the other device
 * arguments when they run, so a captured graph follows their contents.  Calls
 * on one cache must be ordered by the caller (one stream, or events), and
 * calls that may overlap need workspaces of their own.
 */
#define VS_KV4_PAGE 64
size_t vs_kv4_page_bytes(int Hkv, int d); /* 0 for an unsupported d */

/*
 * vs_kv4_append -- quantises new keys and values and writes them behind what
 * the cache holds: sequence b's new tokens, rows [cu_seqlens[b],
 * cu_seqlens[b + 1]) of K and V, go to slots [lens[b] - n_b, lens[b]).
 * Per group of 64 channels x: m = min x, s = bf16((max x - min x) / 15),
 * n = clamp(rint((x - m) / s), 0, 15) with ties to even, decided exactly;
 * s = 0 gives n = 0; an infinity or NaN gives a group that reads as NaN.
 *   K, V     [total_tokens, Hkv, d], VS_BF16 (else VS_ERR_UNSUPPORTED),
 *            strides as for the attention calls.  Keys carry their rotary
 *            embedding already: slots have no positions of their own.
 *   cu_seqlens int32 [B + 1] (device), max_new >= every n_b, as for
 *            vs_sparse_attn_fwd_varlen; n_b = 0 leaves the sequence alone.
 *   lens     lengths INCLUDING the new tokens.
 *   n_tokens int32 [B] (device): tokens seen so far, the new ones included
 *            (larger than lens after an eviction), or NULL: lens.
 *   acc, pos fp32 and int32 [B][Hkv][ld] (device), each may be NULL: the
 *            accumulated attention weight and the position of every slot.
 *            Entries of the new slots are written: acc[b][g][slot] = sum of
 *            A_v[h][row] over the query heads h of KV head g (0 without A_v),
 *            pos[b][g][slot] = n_tokens[b] - n_b + i for the i-th new token.
 *   A_v      fp32 [Hq][total_tokens] as vs_attn_aggregate_varlen writes it, or
 *            NULL (needs acc).
 * A sequence that does not fit (a malformed offset, more new tokens than
 * lens[b], lens[b] above 64 table_ld or, with acc or pos, above ld) is not
 * written and sets VS_DEVFLAG_BOUNDS.  ws: 256 bytes, 256-byte aligned.
 * max_new * Hkv * d / 8 < 2^31 (else VS_ERR_UNSUPPORTED).
 */
vs_status vs_kv4_append(const void* K, const void* V, vs_dtype dtype, int total_tokens,
                        const int32_t* cu_seqlens, int max_new, int64_t kv_stride_tok, void* pool,
                        int n_pages, const int32_t* table, int64_t table_ld, const int32_t* lens,
                        const int32_t* n_tokens, int B, int max_len, int Hq, int Hkv, int d,
                        const float* A_v, float* acc, int32_t* pos, int64_t ld, void* ws,
                        size_t ws_bytes, cudaStream_t stream);

/*
 * vs_kv4_read -- reads slots [start[b], start[b] + n_b) of every sequence back
 * as bf16 (s n + m, rounded once), n_b = cu_seqlens[b + 1] - cu_seqlens[b],
 * into rows [cu_seqlens[b], cu_seqlens[b + 1]) of K and V [total_tokens, Hkv,
 * d]: a cached prefix for the packed prefill calls.
 *   start    int32 [B] (device) or NULL: 0.   max_read >= every n_b.
 * Rows of no sequence are left as they were.  A sequence whose slots do not
 * all lie in [0, lens[b]) is not written and sets VS_DEVFLAG_BOUNDS, as does a
 * malformed offset.  ws: 256 bytes, 256-byte aligned.
 * max_read * Hkv * d / 8 < 2^31 (else VS_ERR_UNSUPPORTED).
 */
vs_status vs_kv4_read(const void* pool, int n_pages, const int32_t* table, int64_t table_ld,
                      const int32_t* lens, const int32_t* start, int B, int max_len, int Hkv, int d,
                      const int32_t* cu_seqlens, int max_read, int total_tokens, void* K, void* V,
                      int64_t kv_stride_tok, void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * vs_kv4_decode_attn_fwd -- attention of one new token per sequence over its
 * cached slots (append the token first for it to see itself):
 *     O[b][h] = sum_t softmax_t(scale q . k_t) v_t over the visible slots t,
 *     LSE = log sum_t exp(scale q . k_t),   k_t, v_t = s n + m.
 *   Q        [B, Hq, d], VS_BF16 (else VS_ERR_UNSUPPORTED), row stride
 *            q_stride_tok; O alike (output).  Hq % Hkv == 0, any ratio.
 *   window, sinks  window 0 (and sinks 0): every slot t < lens[b].  Else slots
 *            t >= lens[b] - window and t < sinks, the window attention of the
 *            prefill at its last row (for caches whose slots are positions:
 *            after an eviction they are not).  Pages without a visible slot
 *            are not touched.
 *   acc_out  fp32 [B][Hkv][ld], or NULL: for t < lens[b]
 *            acc_out = acc_in + sum over the query heads of the KV head of the
 *            softmax weight of slot t (0 where it is invisible); acc_in may be
 *            acc_out itself, or NULL (zeros).  ld >= max_len.  Entries from
 *            lens[b] on are left as they were.
 *   lse      fp32 [Hq][B] (output) or NULL.
 * Scores, maxima, sums, weights (acc) and O are held in fp32; only the products
 * of a weight and a step s are rounded to bf16 for their product with the codes
 * (counted from 8): O is off by up to 2^-8 8 max s from that, and by 2^-8 of
 * itself from its own rounding.
 * The values' steps s are expected to be 0 or in [2^-40, 2^40] and their minima
 * m below 2^44 in size, |Q| below 2^113 and softmax_scale |Q| below 2^112;
 * beyond that results lose precision or overflow.
 * A sequence without slots gives O = 0 and LSE = -inf.  Results do not depend
 * on timing: repeated calls give the same bits on the same device.
 *   ws       vs_kv4_decode_workspace_size(B, Hq, Hkv, d, max_len, acc_out !=
 *            NULL) bytes, 256-byte aligned (the size depends on the current
 *            device's SM count; with weights it includes one float per query
 *            head and slot).
 * VS_ERR_UNSUPPORTED where the pages of all rows come within 2^16 of 2^31.
 */
size_t vs_kv4_decode_workspace_size(int B, int Hq, int Hkv, int d, int max_len, int with_weights);
vs_status vs_kv4_decode_attn_fwd(const void* Q, vs_dtype dtype, int64_t q_stride_tok,
                                 const void* pool, int n_pages, const int32_t* table,
                                 int64_t table_ld, const int32_t* lens, int B, int max_len, int Hq,
                                 int Hkv, int d, float softmax_scale, int window, int sinks,
                                 const float* acc_in, float* acc_out, int64_t ld, void* O,
                                 float* lse, void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * vs_kv4_evict -- cuts every (sequence, KV head) row to k = min(lens[b], keep)
 * slots.  What stays, in this order: slots of fixed tokens (pos < sinks or pos
 * >= n_tokens[b] - recent), then by acc descending (NaN after -inf), ties to
 * the lower slot.  Slots below k that stay keep their place; the i-th slot
 * below k that goes is overwritten by the i-th slot at or above k that stays.
 * Every head keeps its own tokens.
 *   lens, acc, pos   as vs_kv4_append and vs_kv4_decode_attn_fwd leave them,
 *            rows of length ld >= max_len; n_tokens as for vs_kv4_append, but
 *            not NULL.
 *   keep, sinks, recent   keep >= 1, sinks >= 0, recent >= 0, sinks + recent
 *            <= keep.
 *   lens_out int32 [B], acc_out, pos_out [B][Hkv][ld_out], ld_out >=
 *            min(keep, max_len): the new lengths, and the kept slots' entries
 *            ([0, k) of each row; the rest is left as it was).  They must not
 *            overlap the input buffers.
 * The pool is changed in place; pages that only held slots at or above k are
 * free afterwards.  The pages of a sequence that is cut must not be shared
 * with another sequence.  1 <= max_len <= 2^18.
 *   ws       vs_kv4_evict_workspace_size(B, Hkv, max_len, keep) bytes,
 *            256-byte aligned.
 */
size_t vs_kv4_evict_workspace_size(int B, int Hkv, int max_len, int keep);
vs_status vs_kv4_evict(void* pool, int n_pages, const int32_t* table, int64_t table_ld,
                       const int32_t* lens, const int32_t* n_tokens, int B, int max_len, int Hkv,
                       int d, const float* acc, const int32_t* pos, int64_t ld, int keep,
                       int sinks, int recent, int32_t* lens_out, float* acc_out,
                       int32_t* pos_out, int64_t ld_out, void* ws, size_t ws_bytes,
                       cudaStream_t stream);

/*
 * Device status of the last call that used `ws`: synchronises `stream`,
 * copies the status word to `*flags` (VS_DEVFLAG_* bits) and returns VS_OK,
 * VS_ERR_DEVICE_TIMEOUT or VS_ERR_DEVICE_BOUNDS accordingly.
 */
vs_status vs_read_device_status(const void* ws, cudaStream_t stream, int* flags);

/*
 * Self-test of the device-side wait limit: launches one CTA that waits on an
 * mbarrier nothing will ever arrive at, through the same bounded-wait code the
 * kernels use, giving up after `limit_ns` nanoseconds (1e3..1e10).  Afterwards
 * vs_read_device_status(ws) reports VS_ERR_DEVICE_TIMEOUT.  The CUDA context
 * stays usable.  `ws` needs 256 bytes.
 */
vs_status vs_selftest_wait_timeout(void* ws, uint64_t limit_ns, cudaStream_t stream);

/*
 * Self-test of the fp64 exponential the block discovery uses for e^x, x <= 0
 * (Tang's table-driven method; arguments below -700 give 0): y[i] = e^x[i]
 * for the n device doubles at x (each <= 0 or -inf), written to the device
 * array y.  Asynchronous on `stream`.  VS_ERR_INVALID_ARG for null pointers
 * or n < 1.
 */
vs_status vs_selftest_exp(const double* x, double* y, int n, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* VS_PREFILL_H */
