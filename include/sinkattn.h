/*
 * sinkattn.h -- C ABI of libsinkattn: grouped-query attention with a
 * per-head learned sink logit, for one NVIDIA GB300 (sm_103a).
 *
 * The method (source: "GPT-OSS on day 0", Perplexity blog, sections
 * "Attention: GQA with attention sinks" and "Kernels for GPT-OSS / Sink
 * Attention"):  every query head h owns a learned logit sink[h] that joins
 * the softmax normaliser beside the scaled scores s_j = scale * <q, k_j> and
 * has no value row.  For one query row with visible keys J:
 *     M   = max(sink[h], max_j s_j)
 *     Z   = exp(sink[h] - M) + sum_j exp(s_j - M)
 *     out = sum_j exp(s_j - M) / Z * v_j,      lse = M + ln Z.
 * sink[h] is compared with the scaled scores as it is (it is not multiplied
 * by `scale`).  Query head h reads key/value head h / (Hq / Hkv).
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers owned by the caller, dense and
 *     row-major in the layout stated beside each argument.  bf16 tensors and
 *     `out` must be 16-byte aligned; int32/f32 tensors 4-byte aligned.
 *   - The library allocates no device memory, frees nothing and never
 *     synchronises on the call path: the work is enqueued on `stream` (a
 *     cudaStream_t passed as void*; NULL = the legacy default stream) on the
 *     CUDA device that is current for the calling thread.
 *   - The return value reports host-side validation and launch errors only.
 *     Problems found on the device (an out-of-range page id or length, a
 *     pipeline wait that ran out) are recorded in a per-device error word
 *     that sinkattn_get_error() reads; the kernels never trap.
 *   - head_dim must be 64 and the KV page size 16; anything else returns
 *     SINKATTN_ERR_UNSUPPORTED.
 */
#ifndef SINKATTN_H_
#define SINKATTN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SINKATTN_OK = 0,
    SINKATTN_ERR_INVALID_ARG = 1,  /* null pointer, bad size, misaligned pointer */
    SINKATTN_ERR_UNSUPPORTED = 2,  /* head_dim != 64, page size != 16, group size > 16, ... */
    SINKATTN_ERR_WORKSPACE = 3,    /* workspace missing or smaller than required */
    SINKATTN_ERR_BAD_PAGE = 4,     /* device: a page id outside [0, num_pages) was met */
    SINKATTN_ERR_TIMEOUT = 5,      /* device: a pipeline wait gave up; results are invalid */
    SINKATTN_ERR_CUDA = 6,         /* a CUDA runtime call failed */
    SINKATTN_ERR_BAD_LENGTH = 7,   /* device: a kv_len outside [0, max_pages*16] was met */
    SINKATTN_ERR_NO_PAGES = 8,     /* device: the pool had fewer free pages than were needed */
    SINKATTN_ERR_BAD_VALUE = 9,    /* device: a NaN or +infinity where a finite value is needed */
    SINKATTN_ERR_BAD_INDEX = 10    /* device: a row or token index out of range */
} sinkattn_status_t;

/* Element types of the tensors that may have more than one. */
typedef enum {
    SINKATTN_DTYPE_F32 = 0,
    SINKATTN_DTYPE_BF16 = 1,
    SINKATTN_DTYPE_F16 = 2
} sinkattn_dtype_t;

/* Sizes of a paged decode call. */
typedef struct {
    int32_t batch;             /* B >= 0 requests, one query token each (B <= 32768)    */
    int32_t num_q_heads;       /* Hq                                                     */
    int32_t num_kv_heads;      /* Hkv; Hq % Hkv == 0 and Hq / Hkv <= 16                  */
    int32_t head_dim;          /* must be 64                                             */
    int32_t page_size;         /* must be 16                                             */
    int32_t num_pages;         /* P, pages in the K/V pools                              */
    int32_t max_pages;         /* row length of page_table (>= 1)                        */
    int32_t num_workers;       /* 0 = automatic (one share per resident CTA, up to four per SM);
                                  otherwise the number of equal shares the flattened
                                  (request, KV head, page) work is cut into, one CTA each.
                                  A request whose pages span several shares is split and
                                  merged; the result does not depend on this value.  Two
                                  shares per SM leave room for a prefill with share_sms
                                  on another stream.                                     */
} sinkattn_decode_dims_t;

/* Sizes of a packed variable-length prefill call. */
typedef struct {
    int32_t num_seqs;          /* N >= 0 sequences                                       */
    int32_t total_tokens;      /* T = cu_seqlens[N]                                      */
    int32_t max_seqlen;        /* an upper bound of every sequence length                */
    int32_t num_q_heads;       /* Hq                                                     */
    int32_t num_kv_heads;      /* Hkv; Hq % Hkv == 0                                     */
    int32_t head_dim;          /* must be 64                                             */
    int32_t share_sms;         /* 0: the fastest kernel for a prefill that has the GPU to
                                  itself (two query heads per CTA, a whole SM each, when
                                  Hq / Hkv is even); 1: a kernel that leaves room on every
                                  SM for another kernel on another stream (one head per CTA,
                                  two CTAs per SM at 32 K registers, ~100 KB of shared
                                  memory and 256 TMEM columns each), so that a decode
                                  launched just before it with two shares per SM
                                  (num_workers = 2 x SMs) runs beside it; other values:
                                  SINKATTN_ERR_INVALID_ARG                              */
} sinkattn_prefill_dims_t;

/* Sizes of a merge call. */
typedef struct {
    int32_t num_splits;        /* S partial results per row (>= 0)                       */
    int32_t num_rows;          /* R                                                      */
    int32_t num_heads;         /* H                                                      */
    int32_t head_dim;          /* must be 64                                             */
} sinkattn_merge_dims_t;

/*
 * Bytes of device workspace sinkattn_decode needs for `dims` on the current
 * device.  0 on invalid dims.  The workspace holds the split-KV partial
 * results and a small per-(request, KV head) table; it needs no
 * initialisation and its contents are dead after the call completes.
 */
size_t sinkattn_decode_workspace_size(const sinkattn_decode_dims_t *dims);

/*
 * Paged decode with split-KV and a merge that counts the sink once.
 * Source: "GPT-OSS on day 0", section "Kernels for GPT-OSS / Sink Attention"
 * (parallelism over heads and along the KV length; online softmax whose
 * running max is seeded from the head's sink in the first block only), and
 * "Accelerating Sonar through speculation", section "Inference with
 * speculative decoding" (KV pages allocated per request; page metadata copied
 * to the GPU before the attention kernel).
 *
 *   q          [B, Hq, 64]        bf16   one query token per request
 *   k_pages    [P, Hkv, 16, 64]   bf16   page p, KV head g, slot t: key of one token
 *   v_pages    [P, Hkv, 16, 64]   bf16   same layout for values
 *   page_table [B, max_pages]     int32  token t of request b lives in page
 *                                        page_table[b][t/16], slot t%16; entries past
 *                                        the request's last page are never read
 *   kv_lens    [B]                int32  cached tokens per request, 0..max_pages*16
 *   sinks      [Hq]               f32    learned sink logit of each query head
 *   scale      softmax scale applied to q.k (usually 1/sqrt(64))
 *   out        [B, Hq, 64]        bf16   attention output
 *   lse        [B, Hq]            f32    natural-log log-sum-exp including the sink,
 *                                        or NULL
 *   workspace  device scratch of at least sinkattn_decode_workspace_size(dims) bytes,
 *              256-byte aligned; it must not be shared by calls that may overlap.
 *
 * A request with kv_len 0 gives out = 0 and lse = sink[h].  Page ids outside
 * [0, P) are skipped (their tokens count as absent) and raise
 * SINKATTN_ERR_BAD_PAGE in the error word; kv_len outside [0, max_pages*16] is
 * clamped and raises SINKATTN_ERR_BAD_LENGTH.
 */
sinkattn_status_t sinkattn_decode(const void *q, const void *k_pages, const void *v_pages,
                                  const int32_t *page_table, const int32_t *kv_lens,
                                  const float *sinks, float scale, void *out, float *lse,
                                  const sinkattn_decode_dims_t *dims, void *workspace,
                                  size_t workspace_bytes, void *stream);

/* Shapes of a verification call. */
typedef struct {
    int32_t batch;             /* B requests, 0..32768                                     */
    int32_t q_len;             /* drafted query tokens per request, 1..16, and
                                  q_len * (num_q_heads / num_kv_heads) <= 64              */
    int32_t num_q_heads;       /* Hq                                                      */
    int32_t num_kv_heads;      /* Hkv, divides Hq                                         */
    int32_t head_dim;          /* must be 64                                              */
    int32_t page_size;         /* must be 16                                              */
    int32_t num_pages;         /* P, pages in the K/V pools                               */
    int32_t max_pages;         /* row length of page_table (>= 1)                         */
    int32_t num_workers;       /* as in sinkattn_decode_dims_t (0 = automatic)            */
} sinkattn_verify_dims_t;

/* Bytes of device workspace sinkattn_verify needs for `dims`; 0 on invalid dims. */
size_t sinkattn_verify_workspace_size(const sinkattn_verify_dims_t *dims);

/*
 * Attention of drafted tokens over the paged cache: the verification step of
 * speculative decoding.  Source: "Accelerating Sonar through speculation",
 * sections "Speculative decoding" (the target model runs over the drafted
 * tokens and produces logits for each of them) and "Inference with
 * speculative decoding" (verification batches over the paged KV cache); the
 * attention of every token is the sink attention of sinkattn_decode.
 *
 * The q_len query tokens of request b are its last q_len cached tokens, whose
 * K and V are already in the pages: token i sits at cache position
 * kv_lens[b] - q_len + i and attends to cache tokens 0 .. that position
 * (the whole prefix and the draft up to itself).  All q_len tokens of a
 * request share one pass over its pages.  q_len = 1 is sinkattn_decode.
 *
 *   q          [B, q_len, Hq, 64]  bf16
 *   k_pages, v_pages, page_table, sinks, scale: as sinkattn_decode
 *   kv_lens    [B] int32   cached tokens per request, the q_len drafted ones included;
 *                          a request shorter than q_len leaves its earliest tokens
 *                          without keys (out = 0, lse = sink)
 *   out        [B, q_len, Hq, 64]  bf16
 *   lse        [B, q_len, Hq]      f32 natural log, or NULL
 *   workspace  at least sinkattn_verify_workspace_size(dims) bytes, 256-byte aligned;
 *              it needs no initialisation and must not be shared by overlapping calls.
 *
 * Errors and the handling of bad page ids and lengths are those of sinkattn_decode.
 */
sinkattn_status_t sinkattn_verify(const void *q, const void *k_pages, const void *v_pages,
                                  const int32_t *page_table, const int32_t *kv_lens,
                                  const float *sinks, float scale, void *out, float *lse,
                                  const sinkattn_verify_dims_t *dims, void *workspace,
                                  size_t workspace_bytes, void *stream);

/*
 * sinkattn_verify for a TREE of drafted tokens.  Source: "Accelerating Sonar
 * through speculation", section "EAGLE": the drafter explores a tree of
 * candidate continuations and the target checks the whole tree at once with a
 * custom attention mask.
 *
 * The q_len drafted tokens of request b are its last q_len cached tokens, in
 * any order that puts parents before children: token i sits at cache position
 * kv_lens[b] - q_len + i, sees every cache token before the draft, and sees
 * drafted token j iff bit j of tree_mask[b][i] is set (its ancestors and
 * itself).  A mask with bits 0..i for token i is the linear draft of
 * sinkattn_verify.
 *
 *   tree_mask  [B, q_len] uint64, 8-byte aligned, device memory (q_len <= 64)
 *   everything else as sinkattn_verify (same workspace size).
 */
sinkattn_status_t sinkattn_verify_tree(const void *q, const void *k_pages, const void *v_pages,
                                       const int32_t *page_table, const int32_t *kv_lens,
                                       const uint64_t *tree_mask, const float *sinks, float scale,
                                       void *out, float *lse, const sinkattn_verify_dims_t *dims,
                                       void *workspace, size_t workspace_bytes, void *stream);

/* Shapes of the calls over a paged cache that take new tokens packed by cu_seqlens. */
typedef struct {
    int32_t num_seqs;          /* N sequences (requests), 0..16384                        */
    int32_t total_tokens;      /* T new tokens, packed by cu_seqlens                      */
    int32_t max_seqlen;        /* >= the largest number of new tokens of one sequence     */
    int32_t num_q_heads;       /* Hq (read by sinkattn_prefill_paged only)                */
    int32_t num_kv_heads;      /* Hkv, divides Hq                                         */
    int32_t head_dim;          /* must be 64                                              */
    int32_t page_size;         /* must be 16                                              */
    int32_t num_pages;         /* P, pages in the K/V pools                               */
    int32_t max_pages;         /* row length of page_table (>= 1)                         */
    int32_t share_sms;         /* sinkattn_prefill_paged only: as in sinkattn_prefill_dims_t
                                  (0 or 1; the other calls ignore it)                      */
} sinkattn_paged_dims_t;

/*
 * Writes the keys and values of new tokens into their requests' pages.
 * Source: "Accelerating Sonar through speculation", section "Inference with
 * speculative decoding": slots for the next tokens are allocated in the
 * per-request KV pages before the batch runs.
 *
 *   k, v        [T, Hkv, 64]     bf16   new tokens of N sequences, packed by cu_seqlens
 *   cu_seqlens  [N + 1]          int32  cu_seqlens[0] = 0, non-decreasing, cu_seqlens[N] = T
 *   start_pos   [N]              int32  cache position of each sequence's first new token
 *                                       (the number of tokens already cached)
 *   page_table  [N, max_pages]   int32  token at cache position p of sequence n goes to page
 *                                       page_table[n][p / 16], slot p % 16
 *   k_pages, v_pages [P, Hkv, 16, 64] bf16, written in place (only the new tokens' slots)
 *
 * A page id outside [0, P) skips its tokens and raises SINKATTN_ERR_BAD_PAGE; a
 * position past max_pages * 16 skips the token and raises SINKATTN_ERR_BAD_LENGTH.
 */
sinkattn_status_t sinkattn_kv_append(const void *k, const void *v, const int32_t *cu_seqlens,
                                     const int32_t *start_pos, const int32_t *page_table,
                                     void *k_pages, void *v_pages, const sinkattn_paged_dims_t *dims,
                                     void *stream);

/*
 * Chunked prefill over the paged cache: new tokens of N sequences attend to
 * everything cached before them and to the new tokens up to themselves.
 * Source: "Accelerating Sonar through speculation", section "Inference with
 * speculative decoding" (batches of prefill, decode or verification run over
 * the per-request KV pages); the attention is the sink attention of
 * sinkattn_prefill ("GPT-OSS on day 0", section "Kernels for GPT-OSS / Sink
 * Attention").
 *
 * The new tokens' keys and values must already be in the pages
 * (sinkattn_kv_append): new token i of sequence n sits at cache position
 * start_pos[n] + i and sees cache tokens 0 .. start_pos[n] + i.
 *
 *   q           [T, Hq, 64]   bf16   new tokens packed by cu_seqlens
 *   k_pages, v_pages [P, Hkv, 16, 64] bf16 (P >= 1), page_table [N, max_pages] int32,
 *   cu_seqlens [N + 1], start_pos [N]: as sinkattn_kv_append
 *   sinks [Hq] f32, scale: as sinkattn_prefill
 *   out         [T, Hq, 64]   bf16;  lse [T, Hq] f32 natural log, or NULL
 *
 * dims->max_seqlen bounds the new tokens of one sequence (a longer one is cut and
 * raises SINKATTN_ERR_BAD_LENGTH, as does start_pos[n] + len_n > max_pages * 16).
 * A page id outside [0, P) raises SINKATTN_ERR_BAD_PAGE; its tokens then read as
 * zero vectors and that sequence's result is not meaningful.  Slots past a
 * sequence's last cached token may hold anything.
 */
sinkattn_status_t sinkattn_prefill_paged(const void *q, const void *k_pages, const void *v_pages,
                                         const int32_t *page_table, const int32_t *cu_seqlens,
                                         const int32_t *start_pos, const float *sinks, float scale,
                                         void *out, float *lse, const sinkattn_paged_dims_t *dims,
                                         void *stream);

/* YaRN rotary embedding parameters (sinkattn_qkv_prologue). */
typedef struct {
    float theta;                    /* base of the rotary frequencies: theta^(-2d/64) for pair d  */
    float factor;                   /* context extension factor s (>= 1; 1 = plain rotary)        */
    int32_t original_max_position;  /* context length L the model was trained with               */
    float beta_fast;                /* pairs turning more than beta_fast times over L keep their
                                       frequency ...                                             */
    float beta_slow;                /* ... pairs turning fewer than beta_slow times are slowed by s;
                                       linear in between (beta_fast > beta_slow > 0)              */
    float attn_factor;              /* multiplier of rotated q and k; 0 = 0.1 ln(s) + 1 (1 if s = 1) */
    int32_t interleaved;            /* 0: pairs (d, d + 32); 1: pairs (2d, 2d + 1)                */
} sinkattn_rope_t;

/*
 * The pre-attention step of new tokens, fused: QKV bias, YaRN rotary embedding
 * of q and k, q to `q_out`, and k / v written straight into the tokens' page
 * slots (what sinkattn_kv_append does for ready keys and values).  Source:
 * "GPT-OSS on day 0", section "Attention: GQA with attention sinks" (QKV
 * projections with a bias; YaRN positional encoding as in DeepSeek-V3).  The
 * page gives no formulas; these follow the published YaRN method: for pair d,
 * theta_d = theta^(-2d/64) and r_d = L theta_d / (2 pi) (turns over the
 * original context); gamma = clamp((r_d - beta_slow) / (beta_fast - beta_slow),
 * 0, 1); the angle per position is ((1 - gamma) / s + gamma) theta_d; rotated q
 * and k are multiplied by attn_factor.
 *
 *   qkv        [T, (Hq + 2 Hkv) * 64] bf16  projected new tokens: Hq q heads, then Hkv k
 *                                           heads, then Hkv v heads
 *   bias       [(Hq + 2 Hkv) * 64]    bf16  added before the rotation, or NULL
 *   cu_seqlens [N + 1], start_pos [N], page_table [N, max_pages]: as sinkattn_kv_append
 *                                           (new token i of sequence n is at position
 *                                           start_pos[n] + i)
 *   q_out      [T, Hq, 64]            bf16
 *   k_pages, v_pages [P, Hkv, 16, 64] bf16  the new tokens' slots are written
 *
 * bf16 buffers 16-byte aligned.  Bad page ids and positions are reported as in
 * sinkattn_kv_append (q_out is still written).
 */
sinkattn_status_t sinkattn_qkv_prologue(const void *qkv, const void *bias, const int32_t *cu_seqlens,
                                        const int32_t *start_pos, const int32_t *page_table,
                                        const sinkattn_rope_t *rope, void *q_out, void *k_pages,
                                        void *v_pages, const sinkattn_paged_dims_t *dims, void *stream);

/*
 * Causal (or full) prefill over packed variable-length sequences.
 * Source: "GPT-OSS on day 0", section "Kernels for GPT-OSS / Sink Attention"
 * (the same sink-aware kernel template serves prefill and decode).
 *
 *   q          [T, Hq, 64]   bf16   query rows of all sequences, packed
 *   k, v       [T, Hkv, 64]  bf16   keys / values, packed the same way
 *   cu_seqlens [N+1]         int32  sequence n is rows cu_seqlens[n] .. cu_seqlens[n+1]-1;
 *                                   cu_seqlens[0] = 0, non-decreasing, cu_seqlens[N] = T
 *   sinks      [Hq]          f32
 *   causal     1: row i of a sequence sees keys 0..i of that sequence;
 *              0: it sees the whole sequence
 *   out        [T, Hq, 64]   bf16
 *   lse        [T, Hq]       f32    natural log, or NULL
 *
 * A sequence longer than dims->max_seqlen is computed only up to
 * max_seqlen rows; its remaining rows are left untouched and
 * SINKATTN_ERR_BAD_LENGTH is raised in the error word.
 */
sinkattn_status_t sinkattn_prefill(const void *q, const void *k, const void *v,
                                   const int32_t *cu_seqlens, const float *sinks, float scale,
                                   int32_t causal, void *out, float *lse,
                                   const sinkattn_prefill_dims_t *dims, void *stream);

/*
 * Log-sum-exp merge of split partial results.
 * Source: "GPT-OSS on day 0", section "Kernels for GPT-OSS / Sink Attention"
 * (when attention is split into blocks along the sequence, the sink belongs to
 * one block only).
 *
 *   partial_o   [S, R, H, 64] f32   o_c = normalised output of split c
 *   partial_lse [S, R, H]     f32   natural-log lse_c of split c; -inf marks an
 *                                   empty split (its o_c is ignored)
 *   sinks       [H] f32, or NULL.  NULL: the sink is already inside one split.
 *               Given: the splits hold no sink and the merge adds exp(sink[h])
 *               exactly once.
 *   out         [R, H, 64]    bf16  sum_c exp(lse_c - L) o_c
 *   lse         [R, H]        f32   L = log(sum_c exp(lse_c) [+ exp(sink[h])]), or NULL
 * A row with no live split and no sink gives out = 0 and lse = -inf.
 */
sinkattn_status_t sinkattn_merge(const float *partial_o, const float *partial_lse,
                                 const float *sinks, void *out, float *lse,
                                 const sinkattn_merge_dims_t *dims, void *stream);

/*
 * sinkattn_decode without a workspace argument, for callers that cannot
 * allocate device memory: a framework that has reserved the whole device for
 * its own pool, a plugin interface that passes only input and output buffers,
 * or a serving loop that must not call cudaMalloc / cudaFree because they can
 * synchronise the device.  The blog posts describing the method have no
 * counterpart to this call; it is a deployment convenience.
 *
 * Arguments, layouts and results are those of sinkattn_decode.  The split-KV
 * scratch lives in a fixed array inside the library, of
 * SINKATTN_DECODE_NOALLOC_SCRATCH_BYTES, held by every device that loads the
 * library until the process exits.  The call allocates and frees nothing.
 *   - A problem needing more scratch than that (see
 *     sinkattn_decode_workspace_size) returns SINKATTN_ERR_WORKSPACE and
 *     launches nothing.
 *   - The first call on a device looks up the array's device address; make it
 *     before any stream capture begins.
 *   - Every call shares the one array, which keeps the last call's contents;
 *     no value in it needs to start at zero.  Calls that can overlap on the
 *     GPU race on the array: order them (one stream, or events).
 */
#define SINKATTN_DECODE_NOALLOC_SCRATCH_BYTES (16u << 20)
sinkattn_status_t sinkattn_decode_noalloc(const void *q, const void *k_pages, const void *v_pages,
                                          const int32_t *page_table, const int32_t *kv_lens,
                                          const float *sinks, float scale, void *out, float *lse,
                                          const sinkattn_decode_dims_t *dims, void *stream);

/* ------------------------------------------------------------------------------------------------
 * A beam step over the paged cache.  N groups (requests) of K rows (beams of a beam search, or samples
 * of one prompt) each have a page table of their own, and rows share the pages of their common past.
 * One step of decoding is
 *   sinkattn_beam_select   the best continuations of each group over its beams and the vocabulary,
 *   sinkattn_pages_fork    page tables and page counts follow the chosen beams; new pages from the pool,
 *   sinkattn_kv_copy       copies the last pages that more than one row is about to write (each layer),
 *   sinkattn_kv_append     the new tokens' keys and values (each layer),
 *   sinkattn_decode_beams  one query token per row, shared pages read once per group (each layer).
 * The blog posts describing the method have no counterpart to these calls beyond the per-request KV
 * pages ("Accelerating Sonar through speculation", section "Inference with speculative decoding").
 * ------------------------------------------------------------------------------------------------ */

/* Shapes of a beam selection. */
typedef struct {
    int32_t num_groups;        /* N groups, 0..65535                                      */
    int32_t num_beams;         /* K beams per group, 1..32                                */
    int32_t vocab;             /* V tokens, 1..2^30                                       */
    int32_t num_select;        /* M continuations chosen per group, 1..64                 */
    int32_t dtype;             /* sinkattn_dtype_t of the logits                          */
    int32_t pad_token;         /* the token of a finished beam's continuation, 0..V-1     */
    int64_t row_stride;        /* elements from one beam's logits to the next's (>= V)    */
} sinkattn_beam_dims_t;

/* Bytes of device workspace sinkattn_beam_select needs for `dims` on the current device; 0 on invalid dims. */
size_t sinkattn_beam_select_workspace_size(const sinkattn_beam_dims_t *dims);

/*
 * Beam search's selection: of the K x V continuations of each group, the M of the highest score
 *     score(k, v) = scores[n][k] + logits[n][k][v] - ln sum_u exp(logits[n][k][u]),
 * in descending order; equal scores go to the lower beam, then the lower token.  Sums of exponentials are
 * held in 32 bits per thread (of at most 1024 tokens); everything above that, and the scores that are
 * compared, in pairs of floats (48 bits); out_scores are those rounded to f32.  A row's logarithm of the sum is
 * off by at most 8e-6 (3.1e-5 where its largest logit is beyond +-2^20), and beams whose scores lie closer than
 * twice that may come in either order.
 *
 *   logits    [N, K, V]  f32, bf16 or f16; row (n, k) starts row_stride elements after row (n, k - 1)
 *   scores    [N, K]     f32   running log-probability of each beam; -inf: the beam is not in use, its
 *                              logits are not read and it has no continuation
 *   finished  [N, K]     uint8 or NULL: a beam with a non-zero flag has one continuation, pad_token at its
 *                              unchanged score; its logits are not read
 *   out_scores  [N, M]   f32   may be scores itself where M = K
 *   out_parents [N, M]   int32 row n * K + k of the beam continued (as sinkattn_pages_fork takes it)
 *   out_tokens  [N, M]   int32
 *   workspace  at least sinkattn_beam_select_workspace_size(dims) bytes, 256-byte aligned; it needs no
 *              initialisation and must not be shared by calls that may overlap.
 *
 * A logit of -inf is no continuation.  A score below f32's range is returned as -inf, after all that are within
 * it (its beam is out of use in the next step).  Where a group has fewer than M continuations, the rest of its
 * row is score -inf, parent -1, token -1.  A beam in use whose score is NaN or +inf, or whose logits hold a NaN or +inf, has
 * no continuation and raises SINKATTN_ERR_BAD_VALUE.
 * K * M * ceil(V / 262144) above 4096 (candidates of a group that meet in one block) is
 * SINKATTN_ERR_UNSUPPORTED.
 */
sinkattn_status_t sinkattn_beam_select(const void *logits, const float *scores, const uint8_t *finished,
                                       float *out_scores, int32_t *out_parents, int32_t *out_tokens,
                                       const sinkattn_beam_dims_t *dims, void *workspace,
                                       size_t workspace_bytes, void *stream);

/* Shapes of a fork of page tables. */
typedef struct {
    int32_t num_rows_in;       /* rows of the present page table, 0..2^20                 */
    int32_t num_rows_out;      /* rows of the new page table, 0..2^20                     */
    int32_t num_pages;         /* P, pages of the pool, 0..2^30                           */
    int32_t max_pages;         /* row length of both page tables (>= 1)                   */
    int32_t page_size;         /* must be 16                                              */
    int32_t grow;              /* room for new tokens per row where room_lens is NULL (>= 0) */
} sinkattn_fork_dims_t;

/* Bytes of device workspace sinkattn_pages_fork needs for `dims`; 0 on invalid dims. */
size_t sinkattn_pages_fork_workspace_size(const sinkattn_fork_dims_t *dims);

/*
 * Page tables after a step: forks, drops, trims and grows rows, and counts the holders of every page.
 * A page of the pool is free while its count is 0.  Row r of the new table continues row p = parents[r] of
 * the present one with its first keep_lens[r] tokens and has room for room_lens[r]; every row of the
 * present table ends.  So a parent named by several rows is forked, one named by none is freed, and
 * parents[r] = -1 starts an empty row (a new request: keep 0, room = its prompt).
 *   - Pages of kept tokens are shared: the new row holds the parent's pages.
 *   - A row that keeps part of its last page and has room for more is going to write that page.  It stays
 *     in it only if the parent's row is its one holder (count 1), every row that continues this parent
 *     keeps the same number of tokens and has room for more, and r is the first of them.  Otherwise it
 *     gets a new page in its place, and copies[r] tells sinkattn_kv_copy what to bring there.
 *   - New pages are the lowest-numbered pages that are free when the call begins, dealt to the rows in
 *     order (first the replaced page, then the following columns).
 * Every result is a whole number and the same however the call is scheduled.
 *
 *   page_table  [R_in, max_pages]   int32   present table; columns past a row's held tokens are not read
 *   held_lens   [R_in]              int32   tokens that each present row has pages for
 *   parents     [R_out]             int32   -1 or a row of the present table
 *   keep_lens   [R_out]             int32   tokens kept of the parent (0..held), or NULL: all of them
 *   room_lens   [R_out]             int32   tokens the new row needs pages for (keep..max_pages*16), or
 *                                           NULL: keep + dims->grow (0 for a row without parent)
 *   page_refs   [P]                 int32   holders of each page
 *   out_table   [R_out, max_pages]  int32   the new table, -1 in unused columns
 *   out_lens    [R_out]             int32   room of each new row (held_lens of the next call)
 *   out_refs    [P]                 int32   the new counts; may be page_refs itself
 *   copies      [R_out, 3]          int32   (source page, destination page, tokens), or (-1, -1, 0)
 *   workspace   at least sinkattn_pages_fork_workspace_size(dims) bytes, 256-byte aligned; it needs no
 *               initialisation and must not be shared by calls that may overlap.
 * out_table, out_lens and copies must not overlap the inputs.  Either table may have no rows.
 *
 * With fewer free pages than needed nothing is done: counts stay, out_table is -1, out_lens 0, copies empty
 * and SINKATTN_ERR_NO_PAGES is raised (the present table stays valid).  A parent outside [-1, R_in) counts
 * as -1 (SINKATTN_ERR_BAD_INDEX); lengths outside their range are clamped (SINKATTN_ERR_BAD_LENGTH); a
 * held page id outside [0, P) is carried along uncounted (SINKATTN_ERR_BAD_PAGE).
 */
sinkattn_status_t sinkattn_pages_fork(const int32_t *page_table, const int32_t *held_lens,
                                      const int32_t *parents, const int32_t *keep_lens,
                                      const int32_t *room_lens, const int32_t *page_refs,
                                      int32_t *out_table, int32_t *out_lens, int32_t *out_refs,
                                      int32_t *copies, const sinkattn_fork_dims_t *dims, void *workspace,
                                      size_t workspace_bytes, void *stream);

/* Shapes of the calls that move cached tokens inside the pools of one or several layers. */
typedef struct {
    int32_t num_layers;        /* L pools one behind the other: [L, P, Hkv, 16, 64] (>= 1) */
    int32_t num_rows;          /* copies (kv_copy) or requests (kv_compact), 0..2^20      */
    int32_t num_kv_heads;      /* Hkv                                                     */
    int32_t head_dim;          /* must be 64                                              */
    int32_t page_size;         /* must be 16                                              */
    int32_t num_pages;         /* P, pages of one layer's pool                            */
    int32_t max_pages;         /* kv_compact: row length of page_table (>= 1)             */
    int32_t max_accepted;      /* kv_compact: row length of accepted, 1..16               */
} sinkattn_move_dims_t;

/*
 * Copies pages: the first `tokens` slots of every KV head of page src to page dst, keys and values, in
 * every layer.  Slots of dst past them keep what they held.
 *
 *   k_pages, v_pages  [L, P, Hkv, 16, 64]  bf16, in place
 *   copies            [num_rows, 3] int32  (src, dst, tokens), tokens 0..16; (-1, -1, any) is skipped
 *
 * No destination may be another entry's source or destination (sinkattn_pages_fork's copies are such);
 * entries that break this leave one or the other in the page.  A page id outside [0, P) skips the entry
 * (SINKATTN_ERR_BAD_PAGE), tokens outside [0, 16] are clamped (SINKATTN_ERR_BAD_LENGTH).
 */
sinkattn_status_t sinkattn_kv_copy(void *k_pages, void *v_pages, const int32_t *copies,
                                   const sinkattn_move_dims_t *dims, void *stream);

/*
 * After the verification of drafted tokens: moves the accepted ones together.  The keys and values at
 * cache position start_pos[b] + accepted[b][i] go to start_pos[b] + i for i < num_accepted[b], in every
 * KV head and layer, as if all were read before any is written.
 *
 *   k_pages, v_pages  [L, P, Hkv, 16, 64]  bf16, in place
 *   page_table    [B, max_pages]     int32 (B = num_rows)
 *   start_pos     [B]                int32 cache position of drafted token 0
 *   accepted      [B, max_accepted]  int32 drafted tokens kept, in their new order (entries past
 *                                          num_accepted are not read)
 *   num_accepted  [B]                int32 0..max_accepted
 *
 * The pages written must be held by one request only.  A position outside [0, max_pages * 16) skips its token
 * and raises SINKATTN_ERR_BAD_LENGTH, as does a num_accepted out of range (clamped); a page id outside
 * [0, P) skips its token and raises SINKATTN_ERR_BAD_PAGE; an accepted index below 0 skips its token and
 * raises SINKATTN_ERR_BAD_INDEX.
 */
sinkattn_status_t sinkattn_kv_compact(void *k_pages, void *v_pages, const int32_t *page_table,
                                      const int32_t *start_pos, const int32_t *accepted,
                                      const int32_t *num_accepted, const sinkattn_move_dims_t *dims,
                                      void *stream);

/* Shapes of a decode of groups of rows that share pages. */
typedef struct {
    int32_t num_groups;        /* N groups, 0..32768                                      */
    int32_t num_beams;         /* K rows per group, 1..32, and K * Hq / Hkv <= 128        */
    int32_t num_q_heads;       /* Hq                                                      */
    int32_t num_kv_heads;      /* Hkv, divides Hq                                         */
    int32_t head_dim;          /* must be 64                                              */
    int32_t page_size;         /* must be 16                                              */
    int32_t num_pages;         /* P, pages in the K/V pools                               */
    int32_t max_pages;         /* row length of page_table (>= 1)                         */
    int32_t num_workers;       /* as in sinkattn_decode_dims_t (0 = automatic)            */
} sinkattn_beams_dims_t;

/* Bytes of device workspace sinkattn_decode_beams needs for `dims` on the current device; 0 on invalid dims. */
size_t sinkattn_decode_beams_workspace_size(const sinkattn_beams_dims_t *dims);

/*
 * sinkattn_decode for groups of rows that share pages: every row attends to its own cached tokens, and a
 * page that several rows of a group hold in the same column is read once for all of them.  The result is
 * that of sinkattn_decode on the N * K rows.
 *
 *   q          [N, K, Hq, 64]          bf16   one query token per row
 *   k_pages, v_pages [P, Hkv, 16, 64]  bf16
 *   page_table [N, K, max_pages]       int32  entries past a row's last page are never read
 *   kv_lens    [N, K]                  int32  cached tokens per row, 0..max_pages*16 (rows of a group may
 *                                             differ)
 *   sinks      [Hq]                    f32
 *   out        [N, K, Hq, 64]          bf16
 *   lse        [N, K, Hq]              f32 natural log, or NULL
 *   workspace  at least sinkattn_decode_beams_workspace_size(dims) bytes, 256-byte aligned; it needs no
 *              initialisation and must not be shared by calls that may overlap.  Most of it is 16 bytes for
 *              every entry of page_table (a list of distinct pages has room for all of them), whatever
 *              the rows hold: 256 groups of 8 rows of 8192 columns need 268 MB.
 *
 * Errors and the handling of bad page ids and lengths are those of sinkattn_decode.
 */
sinkattn_status_t sinkattn_decode_beams(const void *q, const void *k_pages, const void *v_pages,
                                        const int32_t *page_table, const int32_t *kv_lens,
                                        const float *sinks, float scale, void *out, float *lse,
                                        const sinkattn_beams_dims_t *dims, void *workspace,
                                        size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------------------------------
 * A paged cache held in 8 bits, with a scale for each page of 16 tokens and KV head.  It takes half the
 * memory and, in a decode, half the traffic of the bf16 cache.  The blog posts describing the method hold
 * their cache in 16 bits and have no counterpart to these calls beyond the per-request KV pages
 * ("Accelerating Sonar through speculation", section "Inference with speculative decoding").
 *
 *   k_pages, v_pages [P, Hkv, 16, 64]  e4m3 codes (4 bits of exponent, 3 of mantissa, largest 448)
 *   kv_scales        [P, Hkv, 2]       uint8: the exponents, + 127, of the scales of the page's keys and values
 *                                      (E8M0).  A cached value is code * 2^(byte - 127).
 * Exponents are within -40..40: values up to 4.9e14, steps down to 2^-49.  A byte outside 87..167 is read as
 * the nearest in that range and raises SINKATTN_ERR_BAD_VALUE where tokens of its page are read.
 *
 * A scale that is a power of two costs no precision beside one that is not (a code's precision is relative),
 * and makes code * scale exact in bf16: sinkattn_kv_unpack_q8 loses nothing.
 * ------------------------------------------------------------------------------------------------ */

/*
 * sinkattn_kv_append into an 8-bit cache.  For each page and KV head that gets new tokens, and for keys and
 * values apart: e is the smallest exponent with max |x| <= 448 * 2^e over the new tokens' values x in that page;
 * if the page holds tokens of the same sequence before the first new one, not less than the exponent it has.
 * The new tokens' codes are x * 2^-e rounded to nearest even; where e has risen, the codes of the tokens before
 * are rounded again under the new scale (exact but for those below the least normal code).  Slots behind the
 * last new token keep their codes.
 *
 *   k, v, cu_seqlens, start_pos, page_table: as sinkattn_kv_append
 *   k_pages, v_pages, kv_scales: written in place; 16-byte, 16-byte and 2-byte aligned
 *
 * The pages written must be held by one sequence only.  Bad page ids and positions are reported as in
 * sinkattn_kv_append and skip their tokens.  A packing that is not 0 <= cu_seqlens[n] <= cu_seqlens[n + 1] <= T raises
 * SINKATTN_ERR_BAD_LENGTH; tokens of any sequence may then be left out, a page at a time.  A NaN or infinity is held as a NaN (its page's scale goes by the
 * finite values), a value beyond 448 * 2^40 as that, and both raise SINKATTN_ERR_BAD_VALUE.
 */
sinkattn_status_t sinkattn_kv_append_q8(const void *k, const void *v, const int32_t *cu_seqlens,
                                        const int32_t *start_pos, const int32_t *page_table, void *k_pages,
                                        void *v_pages, uint8_t *kv_scales, const sinkattn_paged_dims_t *dims,
                                        void *stream);

/*
 * sinkattn_qkv_prologue into an 8-bit cache: bias and rotation in 32 bits, q rounded to bf16, keys and values
 * rounded once, from 32 bits to 8, as sinkattn_kv_append_q8 does.  Arguments as those two calls'.  Where a bad packing
 * leaves tokens out of the pages, their rows of q_out are not written either.
 */
sinkattn_status_t sinkattn_qkv_prologue_q8(const void *qkv, const void *bias, const int32_t *cu_seqlens,
                                           const int32_t *start_pos, const int32_t *page_table,
                                           const sinkattn_rope_t *rope, void *q_out, void *k_pages, void *v_pages,
                                           uint8_t *kv_scales, const sinkattn_paged_dims_t *dims, void *stream);

/* Shapes of an unpack of 8-bit pages. */
typedef struct {
    int32_t num_rows;          /* entries of copies, 0..2^20                              */
    int32_t num_kv_heads;      /* Hkv                                                     */
    int32_t head_dim;          /* must be 64                                              */
    int32_t page_size;         /* must be 16                                              */
    int32_t num_pages;         /* P, pages of the 8-bit pools                             */
    int32_t num_pages_out;     /* P_out, pages of the bf16 pools                          */
} sinkattn_unpack_dims_t;

/*
 * Pages of an 8-bit cache as bf16 pages, exactly: the first `tokens` slots of every KV head of 8-bit page src to
 * bf16 page dst, keys and values; for the calls that take a bf16 cache (draft trees, shared pages) or to hand a
 * cache on.  Slots of dst past them keep what they held.
 *
 *   copies        [num_rows, 3] int32  (src, dst, tokens), tokens 0..16; (-1, -1, any) is skipped
 *   k_out, v_out  [P_out, Hkv, 16, 64] bf16, 16-byte aligned
 *
 * Entries with the same destination leave one or the other in it.  A page id outside its pool skips the entry
 * (SINKATTN_ERR_BAD_PAGE), tokens outside [0, 16] are clamped (SINKATTN_ERR_BAD_LENGTH).
 */
sinkattn_status_t sinkattn_kv_unpack_q8(const void *k_pages, const void *v_pages, const uint8_t *kv_scales,
                                        const int32_t *copies, void *k_out, void *v_out,
                                        const sinkattn_unpack_dims_t *dims, void *stream);

/* Bytes of device workspace sinkattn_decode_q8 needs for `dims` on the current device; 0 on invalid dims. */
size_t sinkattn_decode_q8_workspace_size(const sinkattn_decode_dims_t *dims);

/*
 * sinkattn_decode over an 8-bit cache.  The queries and weights are multiplied with the codes in f16 (11 bits), sums
 * are held in 32 bits.  Weights keep their 11 bits down to 2^-21 of a row's largest and are off by at most 2^-32 of it
 * below; those of a page whose values' scale is more than 2^6 above another's are taken relative to the page's own
 * largest.  Arguments, workspace rules and errors are those of sinkattn_decode, and kv_scales.
 */
sinkattn_status_t sinkattn_decode_q8(const void *q, const void *k_pages, const void *v_pages,
                                     const uint8_t *kv_scales, const int32_t *page_table, const int32_t *kv_lens,
                                     const float *sinks, float scale, void *out, float *lse,
                                     const sinkattn_decode_dims_t *dims, void *workspace, size_t workspace_bytes,
                                     void *stream);

/* Bytes of device workspace sinkattn_prefill_paged_q8 needs for `dims`; 0 on invalid dims. */
size_t sinkattn_prefill_paged_q8_workspace_size(const sinkattn_paged_dims_t *dims);

/*
 * sinkattn_prefill_paged over an 8-bit cache (chunks of a prompt, drafted tokens): the sequences' pages are first
 * widened to bf16, exactly, in the workspace, and read from there.  Arguments and errors are those of
 * sinkattn_prefill_paged, and kv_scales.
 *
 *   workspace  at least sinkattn_prefill_paged_q8_workspace_size(dims) bytes, 256-byte aligned: 4 KiB for each KV
 *              head of min(P, N * max_pages) pages (the pages of one layer; layers can share it), and N * max_pages
 *              integers where that is the lesser.  It needs no initialisation and must not be shared by calls that
 *              may overlap.
 */
sinkattn_status_t sinkattn_prefill_paged_q8(const void *q, const void *k_pages, const void *v_pages,
                                            const uint8_t *kv_scales, const int32_t *page_table,
                                            const int32_t *cu_seqlens, const int32_t *start_pos, const float *sinks,
                                            float scale, void *out, float *lse, const sinkattn_paged_dims_t *dims,
                                            void *workspace, size_t workspace_bytes, void *stream);

/* Shapes of a sampling of tokens. */
typedef struct {
    int32_t num_rows;          /* N rows, 0..2^20                                         */
    int32_t vocab;             /* V tokens, 1..2^30                                       */
    int32_t dtype;             /* sinkattn_dtype_t of the logits                          */
    int32_t reserved;          /* 0                                                       */
    int64_t row_stride;        /* elements from one row's logits to the next's (>= V)     */
} sinkattn_sample_dims_t;

/*
 * The next token of each row, from its logits and a random number.  With t the row's temperature and z_1 the
 * largest logit, a token's weight is e^((z - z_1) / t); tokens are ordered by falling logit, equal ones by rising
 * index.  Of this order
 *   top_k  keeps the first top_k tokens,
 *   top_p  of those the shortest start whose weights reach top_p of their sum (those before which the sum is
 *          below it; at least one),
 *   min_p  of those the ones whose weight is at least min_p.
 * With Z the sum of the kept weights the token chosen is the first, in the order of the vocabulary, up to and
 * with which the kept weights sum to more than uniform * Z.  Weights are off by at most 2^-28.5 of themselves, equal
 * logits' alike, and sums are held in 46 bits, so that the choice is that of exact arithmetic but for a chance of about
 * 1e-7 a row with 10^5 tokens of like weight and as many values; where few values are held by many tokens each (ties,
 * 16-bit logits) of about 1e-5 with 10^5 tokens of 50 values, and never more than 2^-29 times the number of kept
 * tokens.  The blog posts describing the method have no counterpart to this call.
 *
 *   logits       [N, V]  f32, bf16 or f16; row n starts row_stride elements after row n - 1
 *   uniform      [N]     f32 in [0, 1)
 *   temperature  [N]     f32 >= 0, or NULL: 1.  0: the token of the largest logit, the lowest of several
 *   top_k        [N]     int32, or NULL; off where it is <= 0 or >= V
 *   top_p        [N]     f32, or NULL; off where it is >= 1; <= 0 keeps one token
 *   min_p        [N]     f32, or NULL; off where it is <= 0; above 1 it counts as 1
 *   out_tokens   [N]     int32
 *   out_logprobs [N]     f32 or NULL: ln(weight / Z) of the token chosen (0 at temperature 0)
 *
 * A logit of -inf has no weight and is never chosen; a row of nothing else gives token -1 and log-probability
 * -inf, as does a row with a NaN or +inf among its logits, a NaN among its settings, a negative temperature or a
 * uniform outside [0, 1), all of which raise SINKATTN_ERR_BAD_VALUE.
 */
sinkattn_status_t sinkattn_sample(const void *logits, const float *uniform, const float *temperature,
                                  const int32_t *top_k, const float *top_p, const float *min_p,
                                  int32_t *out_tokens, float *out_logprobs, const sinkattn_sample_dims_t *dims,
                                  void *stream);

/*
 * Takes and clears the current device's error word in one atomic step ordered
 * on `stream` (after everything enqueued on it before), synchronises `stream`
 * and returns what it took (SINKATTN_OK when no kernel reported a problem).
 * If several problems were recorded, the one with the lowest status code is
 * returned.  A problem raised by a kernel on another stream after the step
 * stays in the word for the next call.
 */
sinkattn_status_t sinkattn_get_error(void *stream);

/*
 * Diagnostic for the failure path of the kernels' bounded waits (not for the hot path): enqueues on
 * `stream` one thread that waits, with the same bounded wait as every pipeline stage of the
 * attention kernels, on an mbarrier that nothing completes.  The wait gives up after its poll limit
 * (seconds) and raises SINKATTN_ERR_TIMEOUT in the device error word -- read it with
 * sinkattn_get_error -- and the kernel returns: no trap, and the context stays usable.  Returns
 * the status of the launch itself.
 */
sinkattn_status_t sinkattn_selftest_wait_timeout(void *stream);

/* Static English text for a status code. */
const char *sinkattn_status_string(sinkattn_status_t status);

/* Library version, major * 10000 + minor * 100 + patch. */
int32_t sinkattn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SINKATTN_H_ */
