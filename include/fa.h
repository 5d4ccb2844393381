/*
 * Exact IO-aware attention on GB300 (sm_103a): the C ABI.
 *
 * What is computed (tonho.wtf "flash attention" entry, section "como
 * funciona"; "Atencao eficiente - FlashAttention, sparse e hibrida", sections
 * "Insight 1 - Tiling" and "Insight 2 - Online softmax"):
 *
 *   forward   O = softmax(tau * Q K^T [+ causal mask]) V, computed tile by tile
 *             with a running row max m and row sum l, so the N x N score
 *             matrix never reaches device memory; the per-row statistics are
 *             returned packed as LSE = m + ln l.
 *   backward  keeps only O and LSE, rebuilds S and P on chip, and uses
 *             D_i = dO_i . O_i (equal to sum_j P_ij dP_ij) to form
 *             dS = P o (dP - D); returns dQ, dK, dV.
 *
 * Conventions shared by every entry point
 *   - Q, K, V, O, dO, dQ, dK, dV: bf16, contiguous [B][H][N][d] (d fastest).
 *     LSE: fp32 [B][H][N], natural log of sum_j exp(tau q_i . k_j).
 *   - d must be 64 or 128.  N may be any value >= 1 (a ragged last tile is
 *     handled inside the kernels).  B, H, N, d are ints >= 0; B, H or N equal
 *     to 0 is an empty problem: FA_OK, nothing is launched, pointers unused.
 *   - causal = 1 hides key j from query i when j > i (query and key lengths
 *     are equal, so top-left and bottom-right alignment coincide); 0 = no mask.
 *   - tau is the score scale, finite and > 0 (usually 1/sqrt(d)).
 *   - Inputs are finite.  A masked key's weight is 0, and 0 times an infinity or NaN
 *     in its V is NaN; only what an entry point says it never reads may hold one.
 *   - Every pointer is a device pointer (cudaMalloc / PyTorch CUDA memory)
 *     aligned to 16 bytes, except the host buffers of fa_host_pipeline_step.
 *     The caller owns every buffer; apart from a host pipeline object's
 *     buffers and fa_bwd_noalloc's fixed scratch array, the library keeps no
 *     device allocation between calls.  Outputs must not overlap inputs.
 *   - stream is a cudaStream_t (NULL = the legacy default stream).  Calls only
 *     enqueue work on it and never synchronise the host.
 *   - Errors are returned, never printed: invalid arguments are caught before
 *     anything is launched.  A kernel whose internal pipeline wait exceeds the
 *     watchdog limit gives up cleanly and records FA_ERR_TIMEOUT in a device
 *     word that fa_last_device_error() reads.
 */
#ifndef FA_GB300_FA_H
#define FA_GB300_FA_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define FA_API __attribute__((visibility("default")))
#else
#define FA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum fa_status {
    FA_OK = 0,
    FA_ERR_INVALID_ARG = 1,  /* null/misaligned pointer, negative size, bad tau, overlap */
    FA_ERR_UNSUPPORTED = 2,  /* d not in {64, 128}, a size limit, or no sm_103a device */
    FA_ERR_WORKSPACE = 3,    /* workspace given but smaller than fa_bwd_workspace_size */
    FA_ERR_CUDA = 4,         /* a CUDA runtime call or kernel launch failed */
    FA_ERR_TIMEOUT = 5,      /* a kernel's bounded pipeline wait ran out */
    FA_ERR_PAGE = 6          /* a cache length, token count or page number out of bounds */
} fa_status;

/*
 * Forward pass.  Reads Q, K, V; writes O (bf16) and LSE (fp32).
 * Source: tonho.wtf "flash attention", section "como funciona" (scores
 * tau*Q_i K_j^T, running max and sum, store of O and the statistics).
 */
FA_API fa_status fa_fwd(const void* Q, const void* K, const void* V, void* O, float* LSE,
                 int B, int H, int N, int d, float tau, int causal, void* stream);

/*
 * Forward pass with an fp32 O output (same kernel; only the final store
 * differs).  For checks whose tolerance is below the bf16 rounding of O.
 * O: fp32 [B][H][N][d].  Same source as fa_fwd.
 */
FA_API fa_status fa_fwd_o32(const void* Q, const void* K, const void* V, float* O, float* LSE,
                     int B, int H, int N, int d, float tau, int causal, void* stream);

/*
 * Bytes of device scratch fa_bwd needs: D (fp32 [B][H][N]) and the fp32 dQ
 * accumulator ([B][H][N][d]), each padded to 256 bytes.  0 for an empty or
 * unsupported problem.
 */
FA_API size_t fa_bwd_workspace_size(int B, int H, int N, int d);

/*
 * Backward pass.  Reads Q, K, V, O, dO (bf16) and LSE (fp32, as written by
 * fa_fwd for the same Q, K, V, tau, causal); writes dQ, dK, dV (bf16; every
 * element is written, nothing is accumulated into them).
 * workspace: device scratch of at least fa_bwd_workspace_size() bytes, owned
 * by the caller and free for the duration of the call on this stream; NULL
 * asks the library to take it with cudaMallocAsync on the stream and give it
 * back with cudaFreeAsync after the last kernel.
 * Arithmetic: S, dP and every product accumulate in fp32. P and dS enter the
 * tensor-core products as bf16. dS is the bf16 product of the bf16 P and
 * dP - D, which is formed in fp32 and rounded to bf16. dQ is summed over the
 * key tiles in an fp32 accumulator in the workspace.
 * Source: tonho.wtf "flash attention", section "como funciona", backward
 * paragraph (keep O and the statistics, rebuild S and P, D_i = dO_i . O_i);
 * "FlashAttention: O Que E e Como Acelera LLMs na Pratica", pillar 2
 * (recomputation in the backward pass).
 */
FA_API fa_status fa_bwd(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                 const float* LSE, void* dQ, void* dK, void* dV,
                 void* workspace, size_t workspace_bytes,
                 int B, int H, int N, int d, float tau, int causal, void* stream);

/* Static, human-readable name of a status code. */
FA_API const char* fa_status_string(fa_status s);

/*
 * Synchronises `stream`, then reads and clears the library's device error
 * words for the current device.  FA_ERR_TIMEOUT if some kernel launched since
 * the last call gave up on a bounded wait, FA_ERR_PAGE if one met a cache
 * length, token count or page number out of bounds (see fa_paged_cache),
 * FA_ERR_CUDA if the stream reports an error, else FA_OK.  Where both happened, the
 * timeout first and the page at the next call.
 */
FA_API fa_status fa_last_device_error(void* stream);

/*
 * Sets how long (nanoseconds) one pipeline wait inside a kernel may take
 * before the kernel gives up (default 2e9 = 2 s).  Applies to launches made
 * after the call, from any thread.  0 restores the default.
 */
FA_API fa_status fa_set_wait_limit_ns(unsigned long long ns);

/*
 * Watchdog self-test: launches one small kernel whose barrier wait is never
 * satisfied, so it times out after `limit_ns` and exits cleanly.  The caller
 * then sees FA_ERR_TIMEOUT from fa_last_device_error().  No fault, trap or
 * unbounded wait is involved.
 */
FA_API fa_status fa_watchdog_selftest(unsigned long long limit_ns, void* stream);

/*
 * Sliding-window (local) causal attention, forward.  Key j is visible from
 * query i iff i - window < j <= i: each query attends to its `window` most
 * recent keys, itself included ("Atencao eficiente - FlashAttention, sparse e
 * hibrida", section "Atencao hibrida: local + global intercalados": local
 * layers with windows of 4096 or 128 tokens).  Same buffers and conventions
 * as fa_fwd with causal = 1; key blocks outside every row's window are never
 * loaded.  window >= 1 (else FA_ERR_INVALID_ARG); window >= N is plain causal
 * attention.
 */
FA_API fa_status fa_fwd_window(const void* Q, const void* K, const void* V, void* O, float* LSE,
                               int B, int H, int N, int d, float tau, int window, void* stream);

/*
 * Sliding-window backward: fa_bwd for the mask of fa_fwd_window (LSE must come
 * from fa_fwd_window with the same window).  Same workspace rules as fa_bwd.
 */
FA_API fa_status fa_bwd_window(const void* Q, const void* K, const void* V, const void* O,
                               const void* dO, const float* LSE, void* dQ, void* dK, void* dV,
                               void* workspace, size_t workspace_bytes, int B, int H, int N, int d,
                               float tau, int window, void* stream);

/*
 * Sliding-window attention with sinks, forward: a causal window beside the first
 * `sinks` keys of the sequence, which every later query goes on seeing ("Atencao
 * eficiente - FlashAttention, sparse e hibrida", section "Sparse e hibrida": a
 * local window plus global anchor tokens; here element by element).  Key j is
 * visible from query i iff j <= i and (j > i - window or j < sinks).  Same buffers
 * and conventions as fa_fwd_window; key blocks that hold neither a sink nor a key
 * of some row's window are never loaded.  window >= 1 and sinks >= 0 (else
 * FA_ERR_INVALID_ARG); sinks = 0 is fa_fwd_window, and window + sinks >= N plain
 * causal attention (fa_fwd's bits).
 */
FA_API fa_status fa_fwd_sinks(const void* Q, const void* K, const void* V, void* O, float* LSE,
                              int B, int H, int N, int d, float tau, int window, int sinks,
                              void* stream);

/*
 * Backward for the mask of fa_fwd_sinks (LSE must come from fa_fwd_sinks with the
 * same window and sinks).  Same workspace rules as fa_bwd.  Until its last kernel
 * writes dQ, the call keeps in dQ's memory the partial dK, dV of the key tiles that
 * hold sinks, whose query lists extra CTAs share.
 */
FA_API fa_status fa_bwd_sinks(const void* Q, const void* K, const void* V, const void* O,
                              const void* dO, const float* LSE, void* dQ, void* dK, void* dV,
                              void* workspace, size_t workspace_bytes, int B, int H, int N, int d,
                              float tau, int window, int sinks, void* stream);

/*
 * Block-sparse attention, forward ("FlashAttention e o gargalo real de
 * inferencia", section "o que isso custou": the block-sparse variant skips
 * blocks, an approximation by design; "Atencao eficiente - FlashAttention,
 * sparse e hibrida", section "Sparse e hibrida": each token attends to a
 * subset, e.g. a local window plus global anchor tokens).
 *
 * block_mask: DEVICE pointer to bytes [mask_heads][nb][nb], nb = ceil(N / 128)
 * (FA_BLOCK_MASK_EDGE), row-major: entry [h][i][j] nonzero means the queries
 * of 128-row block i of head h see the keys of 128-key block j.  mask_heads
 * is 1 (one mask for every batch and head) or B*H (head bh = b*H + h uses
 * mask bh); anything else is FA_ERR_INVALID_ARG.  With causal = 1 a key is
 * visible only if it is also at or before the query.  Blocks that are not set
 * are never loaded.  A row that sees no key is the empty sum: O = 0 and
 * LSE = -inf.  The mask is read on the stream; it must stay valid until the
 * call's work is done and must not overlap O or LSE.  N <= FA_BLOCK_MASK_MAX_N
 * (else FA_ERR_UNSUPPORTED).  Other buffers and conventions as fa_fwd.
 */
#define FA_BLOCK_MASK_EDGE 128
#define FA_BLOCK_MASK_MAX_N 131072
FA_API fa_status fa_fwd_blocks(const void* Q, const void* K, const void* V, void* O, float* LSE,
                               int B, int H, int N, int d, float tau, int causal,
                               const unsigned char* block_mask, int mask_heads, void* stream);

/*
 * Block-sparse backward: fa_bwd for the mask of fa_fwd_blocks (LSE must come
 * from fa_fwd_blocks with the same mask).  Rows that see no key get dQ = 0;
 * keys that no query sees get dK = dV = 0.  Same workspace rules as fa_bwd;
 * the mask must not overlap dQ, dK, dV or the workspace.  Until its last
 * kernel writes dQ, the call keeps in dQ's memory the plan that splits key
 * tiles seen by many query tiles over extra CTAs, and their partial dK, dV.
 */
FA_API fa_status fa_bwd_blocks(const void* Q, const void* K, const void* V, const void* O,
                               const void* dO, const float* LSE, void* dQ, void* dK, void* dV,
                               void* workspace, size_t workspace_bytes, int B, int H, int N, int d,
                               float tau, int causal, const unsigned char* block_mask,
                               int mask_heads, void* stream);

/*
 * What changes the scores of fa_fwd_score and the entry points beside it, and which keys they
 * hide.  Fields left 0 or NULL change nothing; device pointers.
 *   softcap       x = tau q.k becomes softcap * tanh(x / softcap).  0, or 2^-20 to 2^60.
 *   slopes        fp32 [H]: then - slopes[h] |i - j| is added, i the query's position and j the
 *                 key's.
 *   bias, buckets a learned bias by buckets of distance: bias[e][h] is added, e =
 *                 buckets[max_distance + cut(i - j)], cut to +-max_distance; bias is
 *                 [num_buckets][H], bf16 or (bias_f32 = 1) fp32, buckets int
 *                 [2 max_distance + 1].  An entry outside [0, num_buckets) adds nothing.
 *                 num_buckets and max_distance from 1 to 1024 (above: FA_ERR_UNSUPPORTED).  Not
 *                 together with slopes.  The cap comes first, then the bias.
 *   docs          int [B][N]: a document is a run of equal numbers, and tokens see their own
 *                 document only; a token whose number is below 0 is in none (padding): it sees
 *                 nothing, O = 0 and LSE = -inf, and nothing sees it.
 *   prefix        int [B], with causal: the first prefix[b] positions (cut to [0, N]) are
 *                 visible from before them, too: j <= i or j < prefix[b].
 *   window        with causal: j > i - window only (>= 1; 0: none).
 * What hides a key hides it, whatever else shows it.  Values are finite.
 */
typedef struct fa_score {
    float softcap;
    const float* slopes;
    const void* bias;
    const int* buckets;
    int bias_f32, num_buckets, max_distance;
    const int* docs;
    const int* prefix;
    int window;
} fa_score;

/*
 * Attention with such scores, forward ("Atencao eficiente - FlashAttention, sparse e hibrida",
 * section "Sparse e hibrida": which tokens a token attends to; the scores' cap and bias have no
 * counterpart in the pages).  Q, O: bf16 [B][H][N][d] and K, V: bf16 [B][H_kv][N][d], H a
 * multiple of H_kv: query head h reads key head h / (H / H_kv).  LSE: fp32 [B][H][N], of the
 * changed scores; a row that sees nothing gives 0 and -inf.  Key blocks that no row of a
 * tile sees are not loaded.  score may not be NULL (all fields 0: plain attention with grouped
 * heads); it is host memory, only read during the call.  workspace:
 * fa_fwd_score_workspace_size bytes (0 without docs); NULL: taken with cudaMallocAsync and
 * given back.  Two calls that may run at the same time need two workspaces.  Other buffers and
 * conventions as fa_fwd.
 */
FA_API size_t fa_fwd_score_workspace_size(int B, int N, const fa_score* score);
FA_API fa_status fa_fwd_score(const void* Q, const void* K, const void* V, void* O, float* LSE,
                              int B, int H, int H_kv, int N, int d, float tau, int causal,
                              const fa_score* score, void* workspace, size_t workspace_bytes,
                              void* stream);

/*
 * Backward of fa_fwd_score (LSE as it wrote it for the same inputs; O is checked but not read: its
 * product with dO is summed anew from the weights, unrounded): dQ [B][H][N][d], dK,
 * dV [B][H_kv][N][d], summed over the query heads that share a key head; every element is
 * written (without query heads, H = 0, dK and dV are zeros).  dBias: with a bias its gradient [num_buckets][H], of its type (every element
 * written; buckets of no visible pair get 0), or NULL: not computed.  It is summed in fp32 in a
 * fixed order and rounded once, of weights in fp32 or, with a cap, off by at most 2^-11 of
 * themselves down to 2^-29.  (dQ's order of summation is not fixed, as in fa_bwd.)
 * workspace: fa_bwd_score_workspace_size bytes, or fa_bwd_score_frozen_workspace_size where
 * dBias is NULL (the same without a bias); NULL as in fa_fwd_score.
 */
FA_API size_t fa_bwd_score_workspace_size(int B, int H, int N, int d, int causal,
                                          const fa_score* score);
FA_API size_t fa_bwd_score_frozen_workspace_size(int B, int H, int N, int d, int causal,
                                                 const fa_score* score);
FA_API fa_status fa_bwd_score(const void* Q, const void* K, const void* V, const void* O,
                              const void* dO, const float* LSE, void* dQ, void* dK, void* dV,
                              void* dBias, int B, int H, int H_kv, int N, int d, float tau,
                              int causal, const fa_score* score, void* workspace,
                              size_t workspace_bytes, void* stream);

/*
 * Decode forward: Nq new query rows per (batch, head) against a KV cache of Nk
 * keys ("Atencao eficiente - FlashAttention, sparse e hibrida", box
 * "FlashAttention nao acelera o decode token a token": each decode step brings
 * one new query row that reads the whole KV cache, so the step is bound by
 * memory bandwidth).  Same result as the forward on the rectangular problem:
 *   O_i = sum_j softmax_j(tau q_i . k_j) v_j,  LSE_i = ln sum_j exp(tau q_i . k_j),
 * over the visible keys j: all Nk, or with causal = 1 (the queries being the
 * last Nq positions of the sequence) j <= i + Nk - Nq.
 *
 * Q, O: bf16 [B,H,Nq,d]; K, V: bf16 [B,H,Nk,d]; LSE: fp32 [B,H,Nq]; all device
 * pointers, contiguous, 16-byte aligned.  1 <= Nq <= 8 (else
 * FA_ERR_UNSUPPORTED); Nk >= 1, and Nq <= Nk when causal (else
 * FA_ERR_INVALID_ARG); d in {64, 128}.  The KV cache is cut into chunks
 * processed in parallel; their partial results go to `workspace`, which needs
 * fa_decode_workspace_size(B, H, Nq, Nk, d) bytes (0 when one chunk suffices;
 * NULL: the call takes it with cudaMallocAsync on `stream` and frees it with
 * cudaFreeAsync).  Asynchronous on `stream`.
 */
FA_API size_t fa_decode_workspace_size(int B, int H, int Nq, int Nk, int d);
FA_API fa_status fa_fwd_decode(const void* Q, const void* K, const void* V, void* O, float* LSE,
                               int B, int H, int Nq, int Nk, int d, float tau, int causal,
                               void* workspace, size_t workspace_bytes, void* stream);

/*
 * A paged key/value cache: sequence b's key j lies in page
 * page_table[b][j / page_size], row j % page_size ("Atencao eficiente -
 * FlashAttention, sparse e hibrida", box "FlashAttention nao acelera o decode
 * token a token": the cache that each decode step reads and extends).
 *   K, V            [num_pages][H_kv][page_size][d], bf16, or e4m3 bytes for the
 *                   _fp8 entry points; 16-byte aligned, contiguous
 *   k_scale,v_scale fp32 [num_pages][H_kv], from 2^-110 to 2^125 (appending sets 2^-100
 *                   to 2^121): the value of a code is code * scale of its page and
 *                   head.  NULL for a bf16 cache.
 *   page_table      int [B][max_pages]; lens: int [B] (4-byte aligned)
 * page_size is a power of two from 16 to 256, max_pages * page_size at most 2^30 and
 * d 64 or 128 (else FA_ERR_UNSUPPORTED).  Table and lengths are device data, read on the
 * stream, so a captured call can be replayed after they have changed.  Entries behind a
 * sequence's pages are not read; sequences may share pages that none of them appends to.
 * A length below 0 or above max_pages * page_size, a page number
 * outside [0, num_pages) that is needed, and a sequence's token counts that do not
 * ascend within [0, T] are not followed: fa_last_device_error then returns FA_ERR_PAGE,
 * and each entry point says what it did instead.  The description itself is host memory and
 * only read during the call; the caller owns all buffers.
 */
typedef struct fa_paged_cache {
    void* K;
    void* V;
    float* k_scale;
    float* v_scale;
    const int* page_table;
    const int* lens;
    int B, H_kv, d, num_pages, page_size, max_pages;
} fa_paged_cache;

/*
 * Appends the keys and values of T new tokens to a bf16 paged cache, rotating the
 * keys (and, given q, the same tokens' queries) by their position on the way.
 * Sequence b brings the rows cu_new[b] <= t < cu_new[b + 1] (device int [B + 1],
 * ascending; NULL: T / B rows each, T a multiple of B); row t stands at position
 * p = lens[b] + t - cu_new[b], where lens[b] keys are in the cache already (the
 * caller adds the new tokens to lens afterwards).  Rows before cu_new[0] and from
 * cu_new[B] on belong to no sequence: nothing of them is written, q_out included.
 *
 * k, v: bf16 [T][H_kv][d] and q, q_out: bf16 [T][H][d] with the given token (_st) and
 * head (_sh) strides in elements, columns contiguous, 16-byte aligned, strides multiples
 * of 8 and not negative: slices of one projection's output pass as they are.  q_out may be
 * q itself with the same strides.  q NULL: H = 0, no queries.
 * The first rot columns (a multiple of 16, at most d) turn: pair c, columns (c,
 * c + rot / 2) or with interleaved = 1 (2c, 2c + 1), goes from (x, y) to
 * (x cos a - y sin a, y cos a + x sin a), a = p * inv_freq[c] (device double
 * [rot / 2], radians per position), exact at any position and rounded once to bf16.
 * rot = 0 with inv_freq NULL (and no q): nothing turns.
 * A token whose position, page or sequence's counts are out of bounds is not stored
 * (FA_ERR_PAGE); its query is rotated all the same.  Counts that descend give FA_ERR_PAGE
 * too: rows that they leave to no sequence are left alone, rows that they give to two are
 * unspecified.  No page may be appended to twice in a call, by two sequences or by one
 * whose table names it twice.  K, V, the scales and q_out must not overlap what else the call reads or
 * writes (q_out = q aside).
 */
FA_API fa_status fa_kv_append(const fa_paged_cache* cache, const void* k, long long k_st,
                              long long k_sh, const void* v, long long v_st, long long v_sh, int T,
                              const int* cu_new, const void* q, long long q_st, long long q_sh,
                              void* q_out, long long qo_st, long long qo_sh, int H,
                              const double* inv_freq, int rot, int interleaved, void* stream);

/*
 * fa_kv_append into an e4m3 cache.  Each page has one scale per head for K and one
 * for V, set here: the smallest power of two s (2^-100 at least) with bound <= 448 s,
 * where bound is the largest magnitude of the page's new values, and for rotated keys
 * 1.5 times their largest magnitude before the rotation (a turned pair is at most
 * sqrt(2) times its larger half).  Values are rounded once, from fp32, to the nearest
 * e4m3 (ties to even; infinities become +-448 s, NaN stays NaN).  A page that held
 * keys before the call keeps the larger of its scale and the new one, and where that
 * grows its codes are rescaled, rounded to nearest even.  A page whose first row is
 * new takes the new scale.
 */
FA_API fa_status fa_kv_append_fp8(const fa_paged_cache* cache, const void* k, long long k_st,
                                  long long k_sh, const void* v, long long v_st, long long v_sh,
                                  int T, const int* cu_new, const void* q, long long q_st,
                                  long long q_sh, void* q_out, long long qo_st, long long qo_sh,
                                  int H, const double* inv_freq, int rot, int interleaved,
                                  void* stream);

/*
 * Attention of a decode step over a bf16 paged cache: fa_fwd_decode for sequences of
 * uneven length in pages, with grouped heads and, if asked for, a window with sinks.
 * The Nq (1..8, else FA_ERR_UNSUPPORTED) query rows of sequence b are the last Nq of
 * its lens[b] positions (lens counts them): row i sees key j iff
 *   j <= lens[b] - Nq + i, and with window > 0 also
 *   j > lens[b] - Nq + i - window or j < sinks.
 * Query head h reads key head h / (H / H_kv); H is a multiple of H_kv.  A row that
 * sees no key (lens[b] < Nq, or 0) is the empty sum: O = 0 and LSE = -inf.
 * Q, O: bf16 [B][H][Nq][d] with the given sequence (_sb), head (_sh) and row (_sn)
 * strides in elements, columns contiguous, 16-byte aligned, strides multiples of 8 and
 * not negative; O's rows must not overlap.  LSE: fp32 [B][H][Nq] contiguous.
 * window = 0: none; sinks > 0 needs a window.  Rows of a page behind a sequence's end,
 * and keys hidden from every row of the call, are never read.
 * workspace: fa_paged_workspace_size bytes (from the sizes alone, not the lengths; 0 for
 * small tables); NULL: taken with cudaMallocAsync and given back.  Two calls that may run
 * at the same time need two workspaces.  A length out of bounds is cut to the table's,
 * and keys on a page out of bounds are hidden (FA_ERR_PAGE).  More than 2^31 16-key tiles in full
 * tables (of all sequences, key heads and 64 query rows) are FA_ERR_UNSUPPORTED.
 */
FA_API size_t fa_paged_workspace_size(const fa_paged_cache* cache, int H, int Nq, int window,
                                      int sinks);
FA_API fa_status fa_fwd_paged(const fa_paged_cache* cache, const void* Q, long long q_sb,
                              long long q_sh, long long q_sn, void* O, long long o_sb, long long o_sh,
                              long long o_sn, float* LSE, int H, int Nq, float tau, int window,
                              int sinks, void* workspace, size_t workspace_bytes, void* stream);

/*
 * fa_fwd_paged over an e4m3 cache.  A weight (times its page's V scale) is held to 2^-11 of
 * itself down to 2^-28 of a row's largest, below that to 2^-39 of the largest.
 */
FA_API fa_status fa_fwd_paged_fp8(const fa_paged_cache* cache, const void* Q, long long q_sb,
                                  long long q_sh, long long q_sn, void* O, long long o_sb,
                                  long long o_sh, long long o_sn, float* LSE, int H, int Nq,
                                  float tau, int window, int sinks, void* workspace,
                                  size_t workspace_bytes, void* stream);

/*
 * fa_fwd_paged and fa_fwd_paged_fp8 with capped or biased scores: softcap, slopes, bias and
 * buckets of score; its docs, prefix and window must be unset (sequences are apart in the
 * cache, and window is an argument).  i - j counts positions of the sequence.  Same
 * workspace.
 */
FA_API fa_status fa_fwd_paged_score(const fa_paged_cache* cache, const void* Q, long long q_sb,
                                    long long q_sh, long long q_sn, void* O, long long o_sb,
                                    long long o_sh, long long o_sn, float* LSE, int H, int Nq,
                                    float tau, int window, int sinks, const fa_score* score,
                                    void* workspace, size_t workspace_bytes, void* stream);
FA_API fa_status fa_fwd_paged_score_fp8(const fa_paged_cache* cache, const void* Q, long long q_sb,
                                        long long q_sh, long long q_sn, void* O, long long o_sb,
                                        long long o_sh, long long o_sn, float* LSE, int H, int Nq,
                                        float tau, int window, int sinks, const fa_score* score,
                                        void* workspace, size_t workspace_bytes, void* stream);

/*
 * FP8 forward ("Atencao eficiente - FlashAttention, sparse e hibrida", the
 * FlashAttention-4 note: FlashAttention-3 added FP8 for Hopper).  Q, K, V are
 * e4m3 (OCP FP8 E4M3: 1 sign, 4 exponent bits with bias 7, 3 mantissa bits,
 * no infinities, max 448) stored one byte per element, [B,H,N,d] contiguous,
 * with one scale per tensor: the value of element x is x * scale.  Computes
 * the attention of those values, O = softmax(tau (sq Q)(sk K)^T [causal])
 * (sv V), with both products on FP8 tensor cores; the softmax numerator is
 * rounded to e4m3 before the second product, which is what limits accuracy
 * (O agrees with the exact result to about 1e-2 relative; LSE, computed from
 * the unrounded numerator, to about 1e-3).  O: bf16 [B,H,N,d]; LSE: fp32
 * [B,H,N], natural log.  d = 128 only (else FA_ERR_UNSUPPORTED); scales finite
 * and > 0 (else FA_ERR_INVALID_ARG).  Other conventions as fa_fwd.
 */
FA_API fa_status fa_fwd_fp8(const void* Q, const void* K, const void* V, void* O, float* LSE,
                            int B, int H, int N, int d, float tau, int causal, float q_scale,
                            float k_scale, float v_scale, void* stream);

/*
 * Kernel timing hook.  With both events non-NULL (cudaEvent_t created by the
 * caller), every later forward or backward call made from the
 * calling host thread records `start` on its stream right before the
 * attention kernel proper (the forward kernel; the backward's main kernel,
 * after its D/zeroing pre-kernel) and `stop` right after it, so the caller
 * can read that kernel's duration with cudaEventElapsedTime.  NULL, NULL
 * turns it off.  The events stay owned by the caller.  Not part of the
 * method: a measurement aid.
 */
FA_API fa_status fa_set_timing_events(void* start, void* stop);

/*
 * Backward pass that allocates nothing.
 *
 * The pages have no counterpart for this entry point; it exists for callers
 * that are not allowed to allocate device memory while they run: hosts that
 * reserve a fixed memory budget up front and forbid libraries from calling
 * cudaMalloc or cudaMallocAsync later (inference servers, plugins inside a
 * framework that owns every allocation, latency-bound loops where an
 * allocation could stall or fail).  Such a caller cannot pass a NULL
 * workspace to fa_bwd, and may have no spare buffer to lend it either.
 *
 * It computes exactly what fa_bwd computes (same arguments, minus the
 * workspace), using as scratch a fixed array of FA_NOALLOC_SCRATCH_BYTES that
 * lives in the library's device image.  Every GPU on which the library is
 * used holds that array until the process exits.  The problem must satisfy
 * fa_bwd_workspace_size(B, H, N, d) <= FA_NOALLOC_SCRATCH_BYTES, otherwise
 * the call returns FA_ERR_WORKSPACE before doing anything.  The call makes no
 * cudaMalloc/cudaFree (or any other allocating) call.
 *
 * The first call on a device looks up the array's device address (with that
 * device current) and keeps it; make that first call before any stream
 * capture begins.  A lookup that fails returns FA_ERR_CUDA and is retried on
 * the next call.  On a device other than sm_103 the call returns
 * FA_ERR_UNSUPPORTED, as every other entry point does.  All calls share the one array and it keeps the previous
 * call's contents (the kernels clear what must start at zero), so two calls
 * whose work overlaps on the GPU (different streams, or different host
 * threads, on the same device) race on it and give wrong results: order them.
 */
#define FA_NOALLOC_SCRATCH_BYTES (32u * 1024u * 1024u)
FA_API fa_status fa_bwd_noalloc(const void* Q, const void* K, const void* V, const void* O,
                                const void* dO, const float* LSE, void* dQ, void* dK, void* dV,
                                int B, int H, int N, int d, float tau, int causal, void* stream);

/*
 * Host-buffer pipeline: forward + backward steps on tensors that live in host
 * memory.  Not part of the method (the pages describe device-resident
 * tensors); it is the runtime a caller with host-resident batches uses, and
 * the library's end-to-end measurement goes through it.
 *
 * fa_host_pipeline_create allocates `depth` (1..8) device buffer sets for one
 * problem shape (Q, K, V, dO, O, LSE, dQ, dK, dV and the backward workspace,
 * on the current device; the only allocations the library makes on its own,
 * owned by the object until fa_host_pipeline_destroy) and two copy streams.
 * The kernels run on `stream` (NULL = the legacy default stream).
 *
 * fa_host_pipeline_step enqueues one step and returns: copy hQ, hK, hV, hdO
 * (host, bf16 [B][H][N][d]) in; fa_fwd and fa_bwd on the next buffer set; copy
 * O, LSE (fp32 [B][H][N]), dQ, dK, dV out to hO, hLSE, hdQ, hdK, hdV.  Events
 * order each set's reuse, so with depth >= 2 the copies of neighbouring steps
 * overlap the kernels.  Host buffers should be page-locked (cudaHostAlloc /
 * pinned): pageable memory works but its copies do not overlap.  The caller
 * must not touch a step's host buffers until that step has finished
 * (fa_host_pipeline_sync, or an event from fa_host_pipeline_mark).
 *
 * fa_host_pipeline_mark records `event` (a cudaEvent_t) on `stream` at a point
 * after everything enqueued so far, copies included, and makes every copy
 * enqueued later wait for it: two marks bracket whole steps for timing.
 * fa_host_pipeline_sync blocks the host until all enqueued work is done.
 * fa_host_pipeline_destroy synchronises, then frees everything (NULL is a
 * no-op).  An object is not thread-safe; use one per host thread.
 * Errors: FA_ERR_INVALID_ARG (null pointers, bad sizes or depth),
 * FA_ERR_UNSUPPORTED (d not 64 or 128), FA_ERR_CUDA (an allocation or CUDA
 * call failed), and whatever fa_fwd / fa_bwd return.
 */
typedef struct fa_host_pipeline fa_host_pipeline;
FA_API fa_status fa_host_pipeline_create(int B, int H, int N, int d, float tau, int causal,
                                         int depth, void* stream, fa_host_pipeline** out);
FA_API fa_status fa_host_pipeline_step(fa_host_pipeline* p, const void* hQ, const void* hK,
                                       const void* hV, const void* hdO, void* hO, float* hLSE,
                                       void* hdQ, void* hdK, void* hdV);
FA_API fa_status fa_host_pipeline_mark(fa_host_pipeline* p, void* event);
FA_API fa_status fa_host_pipeline_sync(fa_host_pipeline* p);
FA_API fa_status fa_host_pipeline_destroy(fa_host_pipeline* p);

#ifdef __cplusplus
}
#endif

#endif /* FA_GB300_FA_H */
