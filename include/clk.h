/*
 * clk.h -- C ABI of the GB300 (sm_103a) hot path of context-lookup
 * speculative decoding ("lookup drafting").
 *
 * The method (HyperQwen 上下文复述加速：lookup 草稿如何把 25k 文档复读推到
 * 381 tok/s, section "lookup 草稿的原理：三步走"): before every decode step,
 * each request looks up the most recent earlier occurrence of the longest
 * 4-12-token suffix of its own token history and proposes the tokens that
 * follow it (Step 1); that draft is fused with a draft model's 7 head
 * proposals into a verify block of 8 or 16 tokens (Step 2); a per-request
 * scheduler uses the 16-token block only while a copy is in progress, with a
 * sticky exit (Step 3); the target's logits over the block are verified
 * greedily.  The history lookup runs over an index that is maintained
 * incrementally as tokens are committed (the forum thread 单卡 RTX 3090 跑
 * Qwen3.8-27B 381 tok/s？HyperQwen 的思路其实比数字更有意思, the reply's
 * point ①: a full rescan per step backfires on long contexts).
 *
 * Conventions for every entry point
 * ---------------------------------
 * - Return value: CLK_OK (0) or a negative CLK_E* code.  Host-side argument
 *   checks return CLK_EINVAL and launch nothing.  A failed kernel launch
 *   returns CLK_ECUDA.  No C++ exception crosses this boundary.
 * - Asynchrony: every call that takes a clk_stream_t (a cudaStream_t) only
 *   enqueues work on that stream; none synchronises, except clk_status,
 *   clk_cache_status, clk_attend_status, clk_read_counters,
 *   clk_read_slot_info, clk_lookup_read_history and
 *   clk_lookup_restore_state, which say so.
 * - Device errors: problems that can only be seen on the device (a history
 *   capacity overflow, a token outside [0, vocab), a bad slot index, a bad
 *   block length) are latched into a status word inside the lookup
 *   workspace; the first one wins; clk_status reads it.  The work item that
 *   hit the error is skipped; the rest of the batch proceeds.
 * - Memory: the library never allocates device memory.  Every buffer is
 *   owned by the caller (e.g. PyTorch tensors) and passed as a plain device
 *   pointer ("d_" prefix) or host pointer ("h_" prefix).  Integer arrays are
 *   int32, C-contiguous, 4-byte aligned, with the shapes given below.
 * - Logits: d_logits of the verify entry points may also point into
 *   page-locked host memory (cudaHostAlloc / cudaMallocHost, or
 *   cudaHostRegister'ed), which unified addressing lets kernels load from
 *   with the same pointer.  The kernels then read the rows they verify in
 *   place over the host link, and only those rows: no staging copy of the
 *   whole [B, rows, V] array.  Results are identical to device logits.
 * - Requests are addressed by slot (0 <= slot < max_slots).  A batch is a
 *   device array d_slots[B] of distinct slots; per-request arrays of the
 *   call are indexed by batch position b, not by slot.
 * - Threading: one lookup handle is used from one stream at a time.
 * - Sentinel: CLK_SENT (-1) marks an empty draft or output slot.  It never
 *   equals an argmax, so verification always stops on it.
 */
#ifndef CLK_H
#define CLK_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* clk_stream_t; /* the same type as cudaStream_t */

#if defined(__GNUC__)
#define CLK_API __attribute__((visibility("default")))
#else
#define CLK_API
#endif

enum {
    CLK_OK = 0,
    CLK_EINVAL = -1,    /* bad argument */
    CLK_ECAPACITY = -2, /* history or index capacity exceeded */
    CLK_ECUDA = -3,     /* CUDA runtime error */
    CLK_ENOTIMPL = -4,  /* not supported by the compiled library */
    CLK_ESTATE = -5     /* call out of order (e.g. handle not set up) */
};

enum {
    CLK_DTYPE_BF16 = 0,
    CLK_DTYPE_F32 = 1,
    CLK_DTYPE_F16 = 2, /* pools and attention only */
    CLK_DTYPE_E4M3 = 3 /* pools with scales only: 8 bits, 4 of exponent and 3 of fraction, no infinities, at most 448 */
};

#define CLK_SENT (-1)
#define CLK_BLOCK 16        /* slots in a verify block and in a lookup draft */
#define CLK_MAX_K 16        /* upper limit of max_k */
#define CLK_MAX_BATCH 8192  /* upper limit of B in one call */

/* Method constants (defaults in brackets).  Step 2 and Step 3 of the
 * article's "三步走" section fix the defaults; the block is 1 committed
 * token + head + tail drafts. */
typedef struct clk_params {
    int32_t min_k;           /* [4]  shortest suffix match that counts (Step 1: 4-12) */
    int32_t max_k;           /* [12] longest suffix searched (<= CLK_MAX_K) */
    int32_t head;            /* [7]  draft-model head slots 1..head (Step 2) */
    int32_t tail;            /* [8]  lookup-only tail slots (Step 2; DFLASH_TOKENS=15) */
    int32_t head_replace_k;  /* [8]  match that replaces the head outright */
    int32_t head_agree_k;    /* [6]  match that replaces it if the drafter agrees */
    int32_t head_agree_n;    /* [2]  leading proposals that must agree */
    int32_t tail_k;          /* [4]  match that fills the tail (and raises the flag) */
    int32_t enter_streak;    /* [2]  consecutive qualifying steps to enter the long block */
    int32_t sticky;          /* [3]  flag-down steps kept in the long block (STICKY=3) */
    int32_t near_full_slack; /* [1]  rejected drafts that still count as nearly full */
} clk_params;

/* Per-slot counters (clk_read_counters).  accept_hist[x][a] counts steps with
 * block class x (0 = short, 1 = long) that accepted a drafts. */
typedef struct clk_counters {
    int64_t steps;      /* scheduler steps */
    int64_t hits;       /* steps whose lookup matched (k >= min_k) */
    int64_t long_steps; /* steps that used the long block */
    int64_t drafted;    /* non-sentinel drafts placed in verify blocks */
    int64_t accepted;   /* drafts accepted (sum of a) */
    int64_t emitted;    /* tokens committed by steps (sum of a + 1) */
    int64_t accept_hist[2][16];
} clk_counters;

/* Scheduler and history state of one slot (clk_read_slot_info). */
typedef struct clk_slot_info {
    int32_t n;        /* history length */
    int32_t mode;     /* 0 = short block, 1 = long block */
    int32_t streak;   /* consecutive qualifying steps while short */
    int32_t miss;     /* consecutive flag-down steps while long */
    int32_t has_prev; /* a scheduler step has run since the slot was set up */
    int32_t cur_len;  /* block length chosen by the last scheduler step, 0 after append */
    int32_t n_indexed; /* the index holds every k-gram ending before position n_indexed - 1; the
                          positions committed since are indexed by the next proposal launches, and
                          n_indexed is raised by the launch after the one that indexed them */
} clk_slot_info;

typedef struct clk_lookup clk_lookup; /* opaque host handle */

/* Fills *p with the defaults above. */
CLK_API void clk_params_default(clk_params* p);

/* CLK_OK if *p is usable: 1 <= min_k <= max_k <= CLK_MAX_K,
 * 1 + head + tail <= CLK_BLOCK, head_agree_n <= head, enter_streak >= 1,
 * and the other fields >= 0; CLK_EINVAL otherwise. */
CLK_API int clk_params_check(const clk_params* p);

/* Text for a status code (static storage). */
CLK_API const char* clk_status_string(int code);

/* ---------------------------------------------------------------------- */
/* Lookup state: histories, the incremental index, scheduler state.        */
/* ---------------------------------------------------------------------- */

/* Bytes of device workspace for `max_slots` requests whose histories hold up
 * to `max_hist` tokens each (prompt plus every committed token).  The
 * workspace holds the histories, the per-request k-gram index (one
 * open-addressing table of 2^ceil(log2(2*max_hist)) 4-byte entries per match
 * length min_k..max_k: 8 * 9 = 72 bytes of index per history token at the
 * defaults, before each table is rounded up to a power of two), the
 * scheduler state with a copy of each history's last 64 tokens, the
 * counters, the fused verify's scratch and the status word.  Returns
 * CLK_EINVAL for bad sizes. */
CLK_API int clk_lookup_workspace_bytes(const clk_params* p, int32_t max_slots, int64_t max_hist, size_t* bytes);

/* Creates a host handle over a caller-owned device workspace of at least
 * clk_lookup_workspace_bytes bytes, 256-byte aligned.  Allocates only the
 * host handle (freed by clk_lookup_destroy).  Tokens must lie in
 * [0, vocab) (vocab <= 0: any token >= 0).  The workspace content is
 * undefined until clk_lookup_reset has run on it. */
CLK_API int clk_lookup_create(clk_lookup** h, const clk_params* p, int32_t max_slots, int64_t max_hist,
                              int32_t vocab, void* d_workspace, size_t bytes);

/* Zeroes the whole workspace (every slot empty, status clear). */
CLK_API int clk_lookup_reset(clk_lookup* h, clk_stream_t s);

/* Sets up the B slots d_slots[B] with the prompts given in CSR layout:
 * request b's prompt is d_prompt[d_prompt_off[b] .. d_prompt_off[b+1]) (int64
 * offsets, device).  Each slot's history becomes its prompt, its scheduler
 * state and counters are cleared, and its k-gram index is rebuilt from the
 * prompt (the 4-gram level and the longer levels, each mapping a k-gram to
 * its most recent end position, so that the lookup never rescans the
 * history).  A prompt must hold 1 .. max_hist tokens; otherwise the slot is
 * left empty and CLK_ECAPACITY (too long) or CLK_EINVAL (empty) is latched. */
CLK_API int clk_lookup_init(clk_lookup* h, const int32_t* d_slots, int32_t B, const int32_t* d_prompt,
                            const int64_t* d_prompt_off, clk_stream_t s);

/* Commits tokens: appends d_tok[b][0 .. d_count[b]) (d_tok is [B,16]) to slot
 * d_slots[b]'s history and inserts every k-gram that the new tokens complete
 * into its index.  A count of 0 is allowed.  A count outside [0, 16], a
 * token outside [0, vocab) or an overflow of max_hist latches an error and
 * skips that request.  If the slot's last scheduler step has not been
 * committed yet, the append counts as that step's commit (a = count - 1)
 * in the counters.  (Article, "三步走" Step 1: the lookup runs over the
 * request's own history, which grows by the committed tokens.) */
CLK_API int clk_lookup_append(clk_lookup* h, const int32_t* d_slots, int32_t B, const int32_t* d_tok,
                              const int32_t* d_count, clk_stream_t s);

/* Step 1 of "三步走": for each request, k = the longest suffix length in
 * [min_k, max_k] of its history h[0..n) that occurred earlier, overlap
 * allowed, and j = the largest position with h[j-k .. j) == h[n-k .. n) and
 * k <= j <= n-1 (the most recent occurrence of that suffix); k = 0, j = -1
 * when none.  The draft is d_draft[b][i] = h[j + (i mod (n - j))] for
 * i = 0..15: the tokens that followed the occurrence, continued as an LZ77
 * copy at distance n - j past the end of the history (all CLK_SENT when
 * k = 0).  Outputs: d_draft [B,16], d_k [B], d_j [B].  The launch also
 * indexes tokens committed by clk_verify_append since the slot's earlier
 * proposals: all of them when more than 16 are pending or B > 32; else it
 * may leave up to 16 to the next proposal launch on the handle (which runs
 * them before its own wait when a clk_verify_append came in between).  The
 * answers never depend on which launch indexes a position: pending
 * positions are checked directly. */
CLK_API int clk_lookup_propose(clk_lookup* h, const int32_t* d_slots, int32_t B, int32_t* d_draft, int32_t* d_k,
                               int32_t* d_j, clk_stream_t s);

/* The same proposal as clk_lookup_propose, by the pages' own method: a scan
 * of the whole history h[0..n) for every earlier occurrence of the suffix
 * ("三步走", Step 1: one scan per request; most candidates fail on their first
 * tokens, the survivors are extended up to max_k), without the index.  Cost
 * O(n) per request per call; kept as the ablation of the incremental index.
 * ctas_per_request: 1 scans each request's history in one CTA, the pages'
 * form (one program per request); n > 1 splits it over n CTAs; 0 takes one
 * CTA per 4,096 positions of the workspace's history capacity.  Any value
 * gives the same answers.  Outputs and errors as clk_lookup_propose
 * (CLK_EINVAL for a negative ctas_per_request); the index is not touched. */
CLK_API int clk_lookup_propose_scan(clk_lookup* h, const int32_t* d_slots, int32_t B, int32_t ctas_per_request,
                                    int32_t* d_draft, int32_t* d_k, int32_t* d_j, clk_stream_t s);

/* Step 3 of "三步走" (the long-block scheduler), one step per request.  The
 * flag is k >= tail_k (the lookup can fill the tail); nearly full means the
 * previous step accepted prev_accept >= prev_len - 1 - near_full_slack
 * drafts (there is no previous step right after clk_lookup_init).  A short
 * request enters the long block when the flag and the nearly-full signal
 * held on enter_streak consecutive steps; a long request leaves it when the
 * flag has been down on more than `sticky` consecutive steps.  Writes
 * d_len[b] = 1 + head + tail (long) or 1 + head (short).  d_len may alias
 * d_prev_len, and d_prev_accept may alias an output of the previous step.
 * Updates the slot's steps / hits / long_steps / drafted counters. */
CLK_API int clk_sched_step(clk_lookup* h, const int32_t* d_slots, int32_t B, const int32_t* d_k,
                           const int32_t* d_prev_accept, const int32_t* d_prev_len, int32_t* d_len, clk_stream_t s);

/* Step 2 of "三步走" (fusion), stateless.  d_block[b][0] = d_last_tok[b];
 * head slots 1..head take the lookup draft d_draft[b][0..head) when
 * k >= head_replace_k, or when k >= head_agree_k and the draft model's first
 * head_agree_n proposals d_head[b][..] equal the lookup's; otherwise they
 * take d_head[b][0..head).  Tail slots head+1 .. head+tail take
 * d_draft[b][head ..] when d_len[b] is the long length and k >= tail_k;
 * otherwise, and beyond the block, CLK_SENT.  d_head is [B, head]. */
CLK_API int clk_fuse(const clk_params* p, int32_t B, const int32_t* d_last_tok, const int32_t* d_draft, const int32_t* d_k,
                     const int32_t* d_head, const int32_t* d_len, int32_t* d_block, clk_stream_t s);

/* clk_sched_step followed by clk_fuse in one launch, with the last token read
 * from the slot's history.  Bit-identical to the two calls. */
CLK_API int clk_fuse_sched(clk_lookup* h, const int32_t* d_slots, int32_t B, const int32_t* d_draft, const int32_t* d_k,
                           const int32_t* d_head, const int32_t* d_prev_accept, const int32_t* d_prev_len, int32_t* d_len,
                           int32_t* d_block, clk_stream_t s);

/* clk_lookup_propose, clk_sched_step and clk_fuse in one launch (one CTA per
 * request).  Bit-identical to the three calls.  Like clk_lookup_propose it
 * first waits for the preceding launch on the stream (programmatic dependent
 * launch) and indexes the tokens that clk_verify_append committed since the
 * slot's earlier proposals (some of them possibly left to the next
 * proposal, as there).  When the handle's last fused verify was
 * clk_verify_append, the launch lets the next launch on the stream (the
 * step's clk_verify_append, which starts streaming its predicted rows) begin
 * before that wait; otherwise only after it. */
CLK_API int clk_propose_fuse_sched(clk_lookup* h, const int32_t* d_slots, int32_t B, const int32_t* d_head,
                                   const int32_t* d_prev_accept, const int32_t* d_prev_len, int32_t* d_draft,
                                   int32_t* d_k, int32_t* d_j, int32_t* d_len, int32_t* d_block, clk_stream_t s);

/* ---------------------------------------------------------------------- */
/* Greedy verification                                                     */
/* ---------------------------------------------------------------------- */

/* Scratch bytes for clk_verify_greedy with up to B requests. */
CLK_API int clk_verify_scratch_bytes(int32_t B, size_t* bytes);

/* Zeroes a verify scratch buffer; required once before its first use (each
 * call leaves it zeroed again; re-run it after any failed call). */
CLK_API int clk_verify_scratch_init(void* d_scratch, size_t bytes, clk_stream_t s);

/* Greedy verification (article, "三步走", last paragraph: greedy
 * verification never reads the draft distribution; the Polish page "Jak
 * DFlash2 przyspiesza Qwen3.8 i skraca kontekst": the first rejected
 * proposal ends the run).  For request b with block length L = d_len[b]
 * (1..16) and block d_block[b][0..16):
 *   g_r = argmax_v logits[b, r, v] for r < L (values compared as float32,
 *         the lowest index wins ties, +0 == -0, the first NaN wins);
 *   a   = the largest a <= L-1 with d_block[b][r+1] == g_r for all r < a;
 *   emitted = a + 1: the accepted drafts and the target's token after them.
 * Logits element (b, r, v) is at d_logits + b*req_stride + r*row_stride + v
 * (element strides), dtype CLK_DTYPE_BF16 or CLK_DTYPE_F32; rows r >= L are
 * never read.  Outputs: d_argmax [B,16] (g_r, CLK_SENT for r >= L),
 * d_accept [B], d_emitted [B], d_out_tok [B,16] (g_0..g_a, then CLK_SENT).
 * A request whose L is outside 1..16 gets a = 0, emitted = 0 and all-SENT
 * rows.  d_scratch: clk_verify_scratch_bytes(B) bytes, zeroed once by
 * clk_verify_scratch_init; calls that share a scratch buffer must not
 * overlap.  Runs as one grid sized to fill every SM. */
CLK_API int clk_verify_greedy(const void* d_logits, int32_t dtype, int64_t row_stride, int64_t req_stride, int32_t V,
                              int32_t B, const int32_t* d_block, const int32_t* d_len, int32_t* d_argmax,
                              int32_t* d_accept, int32_t* d_emitted, int32_t* d_out_tok, void* d_scratch,
                              size_t scratch_bytes, clk_stream_t s);

/* clk_verify_greedy for callers that cannot allocate device memory at all:
 * for example a plugin that is handed only its input and output pointers,
 * or a serving engine whose free HBM is already committed to its own pools
 * and which has no way to give this library a scratch buffer.  It takes
 * the same arguments minus the scratch and computes the same outputs.  It
 * allocates nothing: its scratch is a fixed array of
 * CLK_STATIC_VERIFY_MAX_BATCH * 17 * 8 bytes (139,264 bytes) inside the
 * library, which every GPU that loads the library keeps until the process
 * exits.  B above CLK_STATIC_VERIFY_MAX_BATCH returns CLK_ECAPACITY (any such
 * B, also beyond CLK_MAX_BATCH) and launches nothing.  The first call on
 * each device looks up the array's device address (cudaGetSymbolAddress),
 * and so does the first call after the device's context changed (after
 * cudaDeviceReset, say); make that first call before any stream capture.  Each call clears the part of the array it uses on its
 * stream and then launches the verify kernel.  All calls share the one
 * array, so calls whose executions overlap on the GPU (other streams, other
 * threads) race and corrupt each other's results: serialise them.  The
 * pages describe no counterpart; this entry point exists for such callers. */
#define CLK_STATIC_VERIFY_MAX_BATCH 1024
CLK_API int clk_verify_greedy_static(const void* d_logits, int32_t dtype, int64_t row_stride, int64_t req_stride,
                                     int32_t V, int32_t B, const int32_t* d_block, const int32_t* d_len,
                                     int32_t* d_argmax, int32_t* d_accept, int32_t* d_emitted, int32_t* d_out_tok,
                                     clk_stream_t s);

/* clk_verify_greedy followed by clk_lookup_append of its d_out_tok /
 * d_emitted, in one launch: each request's tokens are committed to its
 * history as soon as its rows are verified; the k-grams they complete are
 * indexed by the following clk_lookup_propose / clk_propose_fuse_sched /
 * clk_lookup_append calls on the slot (which see the same answers as with an
 * immediate index update).  Uses the scratch inside the lookup workspace.
 * Results are bit-identical to the two calls.
 * Launch order: the launch is a programmatic dependent of the preceding
 * launch on the stream, and d_block / d_len may come from that launch
 * (clk_propose_fuse_sched).  Before it waits for it, it reads the rows of a
 * predicted length of every request: max(1 + head, d_len_hint[b]) when the
 * hint is a valid length, else 1 + head (the short block, which every block
 * covers); after the wait it reads the rows the prediction missed.
 * d_len_hint (nullable) is only a prediction, e.g. the previous step's
 * lengths in a buffer the preceding launch does not write: any value gives
 * the same results, a good one saves a second pass.  So the logits must
 * already be complete when this call is made (as after any ordinary kernel
 * or copy on the stream) and must hold every predicted row (16 rows per
 * request serve any hint).  Consecutive calls on a handle alternate between
 * two halves of the scratch in the workspace, so that a call may start
 * streaming while the previous one finishes (clk_propose_fuse_sched between
 * them lets it); a call lets the next launch on the stream start only after
 * its own wait. */
CLK_API int clk_verify_append(clk_lookup* h, const int32_t* d_slots, const void* d_logits, int32_t dtype,
                              int64_t row_stride, int64_t req_stride, int32_t V, int32_t B, const int32_t* d_block,
                              const int32_t* d_len, const int32_t* d_len_hint, int32_t* d_argmax,
                              int32_t* d_accept, int32_t* d_emitted, int32_t* d_out_tok, clk_stream_t s);

/* Sampling verification with point-mass drafts (HyperQwen context-lookup
 * article, closing paragraph of "lookup 草稿的原理：三步走": for sampled
 * requests every drafted position is a point mass on its proposed token,
 * a proposal the standard speculative rejection sampler accepts, so the
 * emitted tokens follow plain sampling from the target).
 *
 * For request b, row r < L_b of the logits gives the target distribution
 * p_r = softmax(x_r * inv_temp[b]).  The draft c = block[b][r + 1] is
 * accepted iff u[b][r][0] < p_r(c).  At the first rejected row the emitted
 * token is drawn from p_r with c removed (renormalised) using u[b][r][1]; if
 * all L_b - 1 drafts are accepted, the bonus token is drawn from p_{L_b - 1}
 * using u[b][L_b - 1][1].  A draw with uniform u is the first token whose
 * running probability sum exceeds u.  A draft outside [0, V) (CLK_SENT) is
 * rejected and its row's whole distribution is drawn from.
 *
 * Layouts are those of clk_verify_greedy: logits [B, rows >= L_b, V] with
 * element strides, block [B, 16], len [B].  inv_temp: float32 [B], 1 /
 * temperature, > 0 and finite.  uniform: float32 [B, 16, 2] in [0, 1), the
 * acceptance and the draw uniform of every row (the caller's random
 * numbers; rows past L_b are not read).  Outputs: d_accept [B] (accepted
 * drafts a), d_emitted [B] (a + 1), d_out_tok [B, 16] (the a accepted drafts,
 * the drawn token, then CLK_SENT).  A request with L_b outside 1..16 or an
 * invalid inv_temp gets accept 0, emitted 0 and all CLK_SENT.  Logits must
 * be finite (-inf entries have weight 0).
 *
 * Computation is in float32; the results do not depend on the launch
 * configuration or on timing.  Only the L_b rows are read, once, plus one
 * 16,384-element segment of the drawn row.
 *
 * Scratch: a caller-owned device buffer of at least
 * clk_verify_sample_scratch_bytes(dtype, V, B) bytes, 16-byte aligned,
 * zeroed once before its first use (e.g. clk_verify_scratch_init); every
 * call leaves it ready for the next.  Calls sharing a scratch buffer must
 * not overlap on the GPU.  Errors: CLK_EINVAL for a bad dtype, size,
 * stride, pointer or scratch size (nothing is launched); CLK_ECUDA for a
 * launch failure. */
CLK_API int clk_verify_sample_scratch_bytes(int32_t dtype, int32_t V, int32_t B, size_t* bytes);
CLK_API int clk_verify_sample(const void* d_logits, int32_t dtype, int64_t row_stride, int64_t req_stride,
                              int32_t V, int32_t B, const int32_t* d_block, const int32_t* d_len,
                              const float* d_inv_temp, const float* d_uniform, int32_t* d_accept,
                              int32_t* d_emitted, int32_t* d_out_tok, void* d_scratch, size_t scratch_bytes,
                              clk_stream_t s);

/* clk_verify_sample with the target's weights defined as integers, so that
 * every acceptance and every draw is an integer comparison: the results are
 * a fixed function of the logits, drafts, lengths, temperatures and
 * uniforms, which another implementation of the same definition reproduces
 * bit for bit.  The rule (accept iff u_acc < p_r(c), draw from the residual
 * or the last row, inverse CDF) is clk_verify_sample's; only p_r changes:
 *
 *   s = fl32(inv_temp * fl32(log2 e)); each row is cut into chunks of 1024
 *   entries (the last one ragged).  Chunk k's reference is
 *   R_k = ceil(fl32(M_k * s)), M_k its largest entry.  An entry x of chunk k
 *   weighs q = Q(fma(x, s, -R_k)) with, for d >= -32, n = rint(d) (ties to
 *   even), r = d - n, f = P(r) the degree-6 Taylor polynomial of
 *   2^(r + 1/2) (coefficients sqrt(2) (ln 2)^j / j! rounded to float,
 *   evaluated by Horner's rule with fused multiply-adds) and
 *   Q(d) = floor(64 (bits(f) - bits(0.5f)) / 2^-n + 1/2), about
 *   2^(d + 29.5); Q(d) = 0 below -32.  S_k = the chunk's sum of q.  Row
 *   units are 2^-12 of a unit of the row's reference R = max_k R_k: a chunk
 *   quantity v counts U(v, e) = floor(v * 2^(12 - e)), e = R - R_k, and the
 *   row's total is T = sum_k U(S_k, e_k).
 *   A draft c in chunk kc is accepted iff floor(k(u_acc) T / 2^24) <
 *   U(q_c, e_kc), with k(u) = floor(u * 2^24) clamped to [0, 2^24 - 1].
 *   The draw with u_smp takes t = floor(k(u_smp) T' / 2^24), T' the sum of
 *   the chunks' totals with c's weight taken out of its chunk (nothing taken
 *   out after a full acceptance or a sentinel draft); the chunk is the
 *   first whose running total exceeds t, and the token the first entry of
 *   it (c skipped) whose running sum of q exceeds the remainder of t taken
 *   back to chunk units (times 2^(e - 12), rounded down).
 *
 * p_r differs from the float softmax by about 2^-22 relative per weight
 * (the polynomial and float rounding) plus half a unit of each weight;
 * entries more than about 30 binades below their chunk's largest entry
 * weigh 0.  A request any of whose L_b rows has a chunk with
 * |fl32(M_k * s)| > 2^22, or only -inf entries, gets the empty result, as
 * does an invalid length or temperature.  V is at most 4,194,304
 * (CLK_EINVAL above).  Logits must be finite or -inf (NaN entries:
 * unspecified result, no fault).
 *
 * Arguments, layouts, outputs and errors are those of clk_verify_sample;
 * the scratch must hold clk_verify_sample_exact_scratch_bytes(dtype, V, B)
 * bytes (16-byte aligned, zeroed once before its first use, left ready for
 * the next call; calls sharing it must not overlap on the GPU).  Every row
 * is read once, plus one 1024-entry chunk of the drawn row. */
CLK_API int clk_verify_sample_exact_scratch_bytes(int32_t dtype, int32_t V, int32_t B, size_t* bytes);
CLK_API int clk_verify_sample_exact(const void* d_logits, int32_t dtype, int64_t row_stride, int64_t req_stride,
                                    int32_t V, int32_t B, const int32_t* d_block, const int32_t* d_len,
                                    const float* d_inv_temp, const float* d_uniform, int32_t* d_accept,
                                    int32_t* d_emitted, int32_t* d_out_tok, void* d_scratch, size_t scratch_bytes,
                                    clk_stream_t s);

/* clk_verify_sample followed by clk_lookup_append of its d_out_tok /
 * d_emitted, in one launch: the sampled step of a decode loop.  Each
 * request's emitted tokens are committed to the history of d_slots[b] as
 * soon as its draw is made; the k-grams they complete are indexed by the
 * next proposal call on the slot.  The results equal those of the two
 * calls.  The launch is a programmatic dependent of the preceding launch on
 * the stream, and d_block / d_len may come from that launch
 * (clk_propose_fuse_sched).  As in clk_verify_append, it first reads the
 * rows of a predicted length of every request with a valid temperature:
 * max(1 + head, d_len_hint[b]) when the hint is a valid length, else
 * 1 + head; after waiting for that launch it reads the rows the prediction
 * missed.  d_len_hint (nullable, e.g. the previous step's lengths in a
 * buffer the preceding launch does not write) is only a prediction: any
 * value gives the same results.  So the logits (every predicted row; 16
 * rows per request serve any hint), the inverse temperatures and the
 * uniforms must be complete when the call is made.  A request with an
 * invalid length or temperature gets the empty result, commits nothing and
 * latches CLK_EINVAL in the handle's status (as do a bad slot, an
 * out-of-vocabulary token or a full history, which clk_lookup_append would
 * reject).  Scratch as for clk_verify_sample; calls sharing it must not
 * overlap on the GPU.  A scratch whose halves (each half of its size,
 * rounded down to a multiple of 256 bytes) each hold the needed size is used
 * as two halves that consecutive calls on the handle alternate (all of it
 * zeroed before the first use; the halves do not move with the batch): then,
 * as after
 * clk_verify_append, the next clk_propose_fuse_sched lets the next call
 * start streaming before its own wait, and a call lets the next launch on
 * the stream start only after its own wait.  With a smaller scratch the next
 * proposal lets the next call start only after that wait. */
CLK_API int clk_verify_sample_append(clk_lookup* h, const int32_t* d_slots, const void* d_logits, int32_t dtype,
                                     int64_t row_stride, int64_t req_stride, int32_t V, int32_t B,
                                     const int32_t* d_block, const int32_t* d_len, const int32_t* d_len_hint,
                                     const float* d_inv_temp, const float* d_uniform, int32_t* d_accept,
                                     int32_t* d_emitted, int32_t* d_out_tok, void* d_scratch, size_t scratch_bytes,
                                     clk_stream_t s);

/* clk_verify_sample_exact followed by clk_lookup_append of its d_out_tok /
 * d_emitted, in one launch: the sampled step of a decode loop on the exact
 * (fixed-point) weights.  Everything else is as for
 * clk_verify_sample_append: a programmatic dependent of the preceding launch,
 * the rows of a predicted length read before the wait (d_len_hint only a
 * prediction), the empty result, no commit and CLK_EINVAL latched for an
 * invalid length, temperature, slot or token, and the two scratch halves;
 * the scratch holds clk_verify_sample_exact_scratch_bytes(dtype, V, B) (or
 * twice that, rounded up to 256 bytes, for the halves).  A request with a row
 * that cannot be weighed (clk_verify_sample_exact) also gets the empty
 * result, commits nothing and latches CLK_EINVAL.  The results equal those
 * of clk_verify_sample_exact and clk_lookup_append. */
CLK_API int clk_verify_sample_exact_append(clk_lookup* h, const int32_t* d_slots, const void* d_logits, int32_t dtype,
                                           int64_t row_stride, int64_t req_stride, int32_t V, int32_t B,
                                           const int32_t* d_block, const int32_t* d_len, const int32_t* d_len_hint,
                                           const float* d_inv_temp, const float* d_uniform, int32_t* d_accept,
                                           int32_t* d_emitted, int32_t* d_out_tok, void* d_scratch,
                                           size_t scratch_bytes, clk_stream_t s);

/* ---------------------------------------------------------------------- */
/* The target's paged K/V cache                                            */
/* ---------------------------------------------------------------------- */
/* Verification asks the target for every drafted position's logits; its
 * attention reads the K and V rows of the tokens that were committed.  They
 * lie in pages of `page_tokens` rows that the caller owns (a clk_pool).  A
 * clk_cache keeps, in a caller-owned device workspace, which pages each slot
 * holds (a page table and a length per slot) and how many slots hold each
 * page.  Drafted tokens' K and V are not written to pages: they stay in the
 * caller's block buffers until the accepted ones are known
 * (clk_cache_append), so a rejected draft costs no page and no clean-up.
 *
 * Free pages are handed out lowest number first, request by request in batch
 * order, so that page tables depend on the calls alone and not on timing.
 * Only whole pages are shared between slots (clk_cache_fork): the page that a
 * slot still writes to is its own.  All entry points enqueue on the stream;
 * only clk_cache_status synchronises.  Device-side problems are latched in
 * the workspace as clk_lookup's are (first one wins, with the slot, or the
 * batch position where the slot itself is bad).  A handle is used from one
 * stream at a time. */
typedef struct clk_cache clk_cache; /* opaque host handle */

/* The pages of every plane: element (plane, page, head, token, d) lies at
 * d_base + plane*plane_stride + page*page_stride + head*head_stride +
 * token*tok_stride + d (strides in elements, >= 0; any order of the four).
 * Layer l's K is plane 2l and its V plane 2l + 1.  Rows of one page must not
 * overlap. */
typedef struct clk_pool {
    void* d_base;
    int32_t dtype;  /* CLK_DTYPE_BF16, CLK_DTYPE_F16 or CLK_DTYPE_F32 */
    int32_t planes; /* 2 * layers */
    int32_t heads;  /* K/V heads */
    int32_t dim;    /* elements of a row, 1 .. 256 */
    int64_t plane_stride, page_stride, head_stride, tok_stride;
} clk_pool;

/* Bytes of workspace for max_slots page tables of up to max_pages pages each
 * over num_pages pages (each of the three at least 1; num_pages and
 * max_slots * max_pages at most 2^30). */
CLK_API int clk_cache_workspace_bytes(int32_t max_slots, int32_t max_pages, int32_t num_pages, size_t* bytes);

/* Creates a host handle over a caller-owned workspace (256-byte aligned).
 * page_tokens: 16, 32, 64 or 128 rows a page; max_pages * page_tokens at most
 * 2^30.  The content is undefined until clk_cache_reset has run on it. */
CLK_API int clk_cache_create(clk_cache** h, int32_t max_slots, int32_t max_pages, int32_t num_pages,
                             int32_t page_tokens, void* d_workspace, size_t bytes);

/* Every slot empty, every page free, status clear. */
CLK_API int clk_cache_reset(clk_cache* h, clk_stream_t s);

/* Device arrays of the workspace, for the caller to read (in stream order):
 * d_len [max_slots] tokens held, d_table [max_slots, max_pages] page numbers
 * (-1 past the last one held), d_refs [num_pages] slots that hold the page.
 * Any of the three may be NULL. */
CLK_API int clk_cache_buffers(clk_cache* h, int32_t** d_len, int32_t** d_table, int32_t** d_refs);

/* Makes room: slot d_slots[b] grows by d_count[b] tokens, and takes the free
 * pages that this needs.  The rows' content is what clk_cache_append writes.
 * A request that its table (max_pages) cannot hold, or whose pages and those
 * of the requests before it in the batch outnumber the free pages, is left
 * as it was and latches CLK_ECAPACITY; a negative count or a bad slot
 * latches CLK_EINVAL. */
CLK_API int clk_cache_grow(clk_cache* h, const int32_t* d_slots, int32_t B, const int32_t* d_count, clk_stream_t s);

/* Writes K and V rows of `layers` layers from `layer0` on: request b's rows
 * i < d_count[b] go to its slot's last d_count[b] positions, len - count + i.
 * Only rows that clk_cache_grow made room for are written, and none that
 * another slot holds: d_count[b] is at most the slot's rows after those it had
 * when a grow of it last failed (such a grow leaves nothing to write until one
 * succeeds) and after the whole pages it has shared by clk_cache_fork, so that
 * a source's rows are written before it is forked.  Within that, rows of
 * several grows go in one call, and a call may be repeated or go layer by layer.
 * Row i is source row r = d_path[b*N + i] of request b, or r = i where d_path
 * is NULL (d_path: the accepted nodes of a tree, clk_tree_accept); 0 <= r <
 * the request's rows.  The request's rows start at row b*N of the source (N
 * rows each), or at d_off[b] where d_off is given (int64 [B+1], N is then
 * the total number of rows, d_path must be NULL and request b has
 * d_off[b+1] - d_off[b] rows).  Source element (layer l, row, head, d) lies
 * at d_k + l*layer_stride + row*row_stride + head*head_stride + d, and the
 * same for d_v (elements of the pool's type).  A count outside 0 .. min(rows
 * that may be written, the request's rows), offsets outside 0 .. N or falling,
 * a path entry out of range or a bad slot latches CLK_EINVAL; the rows
 * concerned are not written.  Source and pool must not overlap. */
CLK_API int clk_cache_append(clk_cache* h, const int32_t* d_slots, int32_t B, const clk_pool* pool, int32_t layer0,
                             int32_t layers, const void* d_k, const void* d_v, int64_t layer_stride,
                             int64_t row_stride, int64_t head_stride, int64_t N, const int64_t* d_off,
                             const int32_t* d_path, const int32_t* d_count, clk_stream_t s);

/* Slot d_dst[b] (empty) becomes a copy of slot d_src[b]: it shares the whole
 * pages, and the rows of a last page that is not full are copied to a page
 * of its own, in every plane.  One source may be forked into several slots
 * of a batch; no slot is both a source and a destination of it.  A bad slot
 * or a destination that is not empty latches CLK_EINVAL, a lack of pages
 * CLK_ECAPACITY (as in clk_cache_grow), and that destination stays as it
 * was: an empty slot, which a clk_cache_grow then fills as one, without the
 * source's rows. */
CLK_API int clk_cache_fork(clk_cache* h, const int32_t* d_src, const int32_t* d_dst, int32_t B, const clk_pool* pool,
                           clk_stream_t s);

/* Empties the slots; pages that no slot holds any more are free again.  A bad
 * slot latches CLK_EINVAL. */
CLK_API int clk_cache_free(clk_cache* h, const int32_t* d_slots, int32_t B, clk_stream_t s);

/* Moves the pages in use to the lowest numbers: with L pages in use, those
 * numbered L and above move, in ascending order, to the free ones below L, in
 * ascending order; their rows are copied in every plane (the rows that hold
 * tokens), and tables and counts follow.  Afterwards pages 0 .. L-1 are in
 * use, and the pool's end can be given back.  d_moved (nullable) receives the
 * number of pages moved. */
CLK_API int clk_cache_compact(clk_cache* h, const clk_pool* pool, int32_t* d_moved, clk_stream_t s);

/* A cache in 8 bits.  Its pool has dtype CLK_DTYPE_E4M3 and comes with scales,
 * one float32 for each block of `tokens` rows of a page and head: that of
 * (plane, page, head, block) lies at d_base + plane*plane_stride +
 * page*page_stride + head*head_stride + block*block_stride (strides in
 * floats, >= 0, any order), and token t of a page belongs to block t /
 * tokens.  An element stands for its value times its block's scale.  Blocks
 * do not span pages, so a page's scales go wherever the page goes. */
typedef struct clk_scales {
    float* d_base;
    int32_t tokens; /* 16, 32, 64 or 128, at most the cache's page_tokens */
    int64_t plane_stride, page_stride, head_stride, block_stride;
} clk_scales;

/* clk_cache_fork and clk_cache_compact of a pool with scales: those of the
 * copied pages are copied too.  (The calls without scales refuse such a
 * pool.) */
CLK_API int clk_cache_fork_scaled(clk_cache* h, const int32_t* d_src, const int32_t* d_dst, int32_t B, const clk_pool* pool,
                                  const clk_scales* scales, clk_stream_t s);
CLK_API int clk_cache_compact_scaled(clk_cache* h, const clk_pool* pool, const clk_scales* scales, int32_t* d_moved,
                                     clk_stream_t s);

/* ---------------------------------------------------------------------- */
/* Position rotation                                                       */
/* ---------------------------------------------------------------------- */
/* Pair i of a row at position p turns by an angle whose cosine and sine are
 * c = d_table[p][0][i] and s = d_table[p][1][i] (float32 [positions, 2,
 * pairs]; a factor of the model's own on cosines and sines goes into the
 * table).  The pair is elements (i, i + pairs), or (2i, 2i + 1) where
 * neighbours is 1; 2 * pairs is at most the rows' dim, and the elements past
 * 2 * pairs stay as they are.  (x, y) becomes (x c - y s, y c + x s) in
 * float32, every product and sum rounded, and is rounded once to where it
 * goes: the results are a fixed function of the inputs. */
typedef struct clk_rotary {
    const float* d_table;
    int64_t positions;
    int32_t pairs;
    int32_t neighbours;
} clk_rotary;

/* Queries and keys that a rotation reads and writes beside the pages.  Row r
 * of request b: q head h at d_q + b*q_req + r*q_row + h*q_head, its result at
 * d_q_out + b*qo_req + r*qo_row + h*qo_head, and k alike (element strides >=
 * 0, rows of `dim` elements of type dtype: CLK_DTYPE_BF16, CLK_DTYPE_F16 or
 * CLK_DTYPE_F32).  A result may lie in its source's place (same pointer and
 * strides); else results overlap no input. */
typedef struct clk_turn {
    int32_t dtype, q_heads, kv_heads, dim; /* dim 1 .. 256 */
    const void *d_q, *d_k;
    void *d_q_out, *d_k_out;
    int64_t q_req, q_row, q_head, k_req, k_row, k_head;
    int64_t qo_req, qo_row, qo_head, ko_req, ko_row, ko_head;
} clk_turn;

/* Rotates the queries and keys of a step's trees: node n of request b stands
 * at position ctx + (bits of d_mask[b*N + n] below d_nodes[b]) - 1 (its depth
 * behind the cached rows; at least ctx), with ctx = d_ctx[b], or the slot's
 * length where d_ctx is NULL, as in clk_tree_attend.  Rows n >= d_nodes[b]
 * are not written.  A bad slot, ctx or node count latches CLK_EINVAL, and the
 * request's rows are not written; nor is a row whose position is not below
 * `positions` (CLK_EINVAL).  B <= CLK_MAX_BATCH. */
CLK_API int clk_tree_rotate(clk_cache* h, const int32_t* d_slots, int32_t B, const clk_turn* t, int32_t N,
                            const int32_t* d_nodes, const int64_t* d_mask, const int32_t* d_ctx, const clk_rotary* rotary,
                            clk_stream_t s);

/* clk_cache_append with the keys rotated on the way, into a pool of the rows'
 * type or of 8 bits.  Everything that it says of rows, counts, offsets and
 * paths holds here.  B <= CLK_MAX_BATCH; 2 * layers * heads of the pool plus
 * the query heads are at most 2^30.
 *
 * rotary (nullable: no rotation): K's row for the slot's position p is turned
 * by position p, which has to be below `positions`, or the request is left
 * out (CLK_EINVAL).  V's rows are not turned.
 *
 * scales: NULL for a pool of type `dtype` (the rows'); else the pool is
 * CLK_DTYPE_E4M3, rows of any of the three types.  A row's values (keys after
 * their rotation, in float32) are divided by their block's scale and rounded
 * once to 8 bits; values beyond the range become the largest, a NaN stays
 * one.  The scale of a block (per layer, K or V, and head) that the call
 * writes to is 2^e with the least e >= -120 for which the largest finite
 * magnitude among the call's rows in it is at most 448 * 2^e; where the block
 * holds rows before the call's first one, it is the larger of that and the
 * scale that it had (one that is not finite or not positive counts as none),
 * and if it grows, those rows become value * old / new, rounded.  So a
 * repeated call changes nothing, and rows are rounded again only when larger
 * ones join their block.
 *
 * turn (nullable): where d_q is not NULL, the same rows of q are turned too
 * (by the same positions, into d_q_out), and where d_k_out is not NULL, the
 * turned keys are also written there, rounded to `dtype`: what the attention
 * of the same tokens reads.  Its d_k and its *_req and k strides are not
 * used: source row x of the call is row x of q and of the results.  layers
 * must be 1 and d_path NULL for it, and rotary given; rows that are not
 * appended are not written. */
CLK_API int clk_cache_append_rotary(clk_cache* h, const int32_t* d_slots, int32_t B, const clk_pool* pool,
                                    const clk_scales* scales, int32_t layer0, int32_t layers, int32_t dtype, const void* d_k,
                                    const void* d_v, int64_t layer_stride, int64_t row_stride, int64_t head_stride, int64_t N,
                                    const int64_t* d_off, const int32_t* d_path, const int32_t* d_count,
                                    const clk_rotary* rotary, const clk_turn* turn, clk_stream_t s);

/* As clk_status and clk_status_clear, for the cache's status word. */
CLK_API int clk_cache_status(clk_cache* h, int32_t* dev_status, int32_t* detail, clk_stream_t s);
CLK_API int clk_cache_status_clear(clk_cache* h, clk_stream_t s);

/* Frees the host handle (not the workspace). */
CLK_API void clk_cache_destroy(clk_cache* h);

/* ---------------------------------------------------------------------- */
/* Trees of drafted tokens                                                 */
/* ---------------------------------------------------------------------- */
#define CLK_TREE_MAX 64 /* nodes of a tree */

/* A request's tree has d_nodes[b] nodes (0 .. N, N <= CLK_TREE_MAX).  Node 0 is the
 * last committed token; node n > 0 is a drafted token that follows node
 * d_parent[b*N + n], which is below n.  A chain (the verify block of
 * clk_fuse) has parents n - 1.  d_parent[b*N] is not read. */

/* Ancestor masks: bit m of d_mask[b*N + n] is set where m is n or one of its
 * ancestors; 0 for n >= d_nodes[b].  A node whose parent is not in 0 .. n-1
 * starts a tree of its own (it sees itself and no node above it).  A node
 * count outside 0 .. N gives masks of 0. */
CLK_API int clk_tree_masks(int32_t B, int32_t N, const int32_t* d_parent, const int32_t* d_nodes, int64_t* d_mask,
                           clk_stream_t s);

/* Greedy verification of a tree, from the target's answers d_argmax [B,N] at
 * every node.  clk_verify_greedy, which writes [B,16], makes them: with N = 16
 * in one block a request, with N a multiple of 16 in N / 16 blocks (logits and
 * argmax [B,N,..] seen as [B*N/16,16,..]; its other outputs do not count
 * then).  Node 0 is accepted; node n is
 * accepted where its parent is and its token d_tok[b*N + n] (>= 0) is the
 * target's answer at the parent; of siblings that both match, the lowest.
 * Outputs: d_path [B,N] the accepted nodes from node 0 on, then -1; d_accept
 * [B] accepted drafts a; d_emitted [B] a + 1; d_out_tok [B,N] the target's
 * answers at the path's nodes (a accepted drafts and the token after them),
 * then CLK_SENT.  A node count of 0 or outside 0 .. N gives accept 0, emitted
 * 0, and -1 / CLK_SENT. */
CLK_API int clk_tree_accept(int32_t B, int32_t N, const int32_t* d_tok, const int32_t* d_parent,
                            const int32_t* d_nodes, const int32_t* d_argmax, int32_t* d_accept, int32_t* d_path,
                            int32_t* d_emitted, int32_t* d_out_tok, clk_stream_t s);

/* ---------------------------------------------------------------------- */
/* Attention over the cache                                                */
/* ---------------------------------------------------------------------- */
/* What both attentions read and write for the new tokens: q [.., q_heads,
 * dim], k and v [.., kv_heads, dim], out [.., q_heads, dim] contiguous.  Query
 * head h reads K/V head h / (q_heads / kv_heads).  Row r of request b lies at
 * d_q + b*q_req + r*q_row + head*q_head + d (element strides >= 0; k and v
 * alike).  dtype: CLK_DTYPE_BF16, CLK_DTYPE_F16 or CLK_DTYPE_F32; dim 1 ..
 * 256.
 *
 *   out[r, h] = sum_j p_j v_j,  p = softmax over the visible j of
 *   scale * <q[r, h], k_j>
 *
 * over the slot's first ctx cached rows and the visible new rows.  A row that
 * sees nothing gives 0.  What is not visible does not count, whatever it holds
 * (rows of a page past ctx, nodes off the mask, other requests): with one
 * rule, a row that does see a new token with an infinity or a NaN in its v
 * may be NaN in every element.  Scores, the softmax's maximum and sum and
 * the accumulators are float32; on the tensor cores (16-bit types, dim a
 * multiple of 8 up to 128) each weight is rounded to the inputs' type for the product with v, and
 * the sum of weights is of the unrounded ones.  out must not overlap an input.
 * There a call is a cooperative launch of one CTA per SM of the device: a
 * process that is given fewer SMs gets CLK_ECUDA. */
typedef struct clk_attn {
    int32_t dtype, q_heads, kv_heads, dim;
    float scale; /* finite */
    const void *d_q, *d_k, *d_v;
    void* d_out;
    int64_t q_req, q_row, q_head;
    int64_t k_req, k_row, k_head;
    int64_t v_req, v_row, v_head;
} clk_attn;

/* Scratch bytes for clk_tree_attend / clk_prompt_attend with these heads and
 * this dim on the current device, for any batch.  16-byte aligned; zeroed once
 * before its first use (e.g. clk_verify_scratch_init) and left ready by every
 * call; calls that share it must not overlap on the GPU.  Zero it again after
 * a call that failed (clk_attend_status). */
CLK_API int clk_attend_scratch_bytes(int32_t q_heads, int32_t kv_heads, int32_t dim, size_t* bytes);

/* Synchronises `s` and returns in *dev_status CLK_ECUDA where a wait inside an
 * attention on this scratch has run out since it was zeroed (the CTAs of a
 * launch wait for one another, at most about two seconds longer than their
 * own share took; the rows of that call are not whole), else CLK_OK.  A call with a cache latches it there too. */
CLK_API int clk_attend_status(const void* d_scratch, int32_t* dev_status, clk_stream_t s);

/* Attention of a step's block: request b has d_nodes[b] new tokens (0 .. N,
 * N <= CLK_TREE_MAX), of which token n sees the slot's first ctx rows (plane
 * 2*layer and 2*layer + 1 of the pool) and the new tokens m < d_nodes[b] whose
 * bit m of d_mask[b*N + n] is set (clk_tree_masks, or any other mask).
 * d_ctx [B] (nullable): ctx per request, 0 .. the slot's length; NULL: the
 * slot's length.  Rows n >= d_nodes[b] of out are 0.  N = 1 is plain decoding
 * by single tokens.  A bad slot, ctx or node count latches CLK_EINVAL in the
 * cache's status, and the request's rows are 0. */
CLK_API int clk_tree_attend(clk_cache* h, const int32_t* d_slots, int32_t B, const clk_pool* pool, int32_t layer,
                            const clk_attn* a, int32_t N, const int32_t* d_nodes, const int64_t* d_mask,
                            const int32_t* d_ctx, void* d_scratch, size_t scratch_bytes, clk_stream_t s);

/* Causal attention of packed prompts: request b's new tokens are rows
 * d_off[b] .. d_off[b+1] - 1 of q, k, v and out (T rows in all; the *_req
 * strides are not used); its token t sees the slot's first ctx rows and its
 * own new tokens 0 .. t.  d_ctx [B]: cached rows before the prompt (0 .. the
 * slot's length); NULL: none.  h, d_slots and pool may be NULL where d_ctx is
 * NULL.  Offsets that fall or leave 0 .. T, a bad slot or a bad ctx: the
 * request's rows are not written, and CLK_EINVAL is latched where h is given.
 * Rows of no request are not written. */
CLK_API int clk_prompt_attend(const clk_attn* a, const int64_t* d_off, int32_t B, int64_t T, clk_cache* h,
                              const int32_t* d_slots, const clk_pool* pool, int32_t layer, const int32_t* d_ctx,
                              void* d_scratch, size_t scratch_bytes, clk_stream_t s);

/* The two attentions over a pool of 8 bits: a->dtype is q's, the new tokens' and
 * out's type, the pool is CLK_DTYPE_E4M3, and each cached element is its
 * value times its block's scale (a product beyond float32's largest is an
 * infinity).  float32, rows of more than 128 elements and whatever else the
 * tensor cores do not take: that product in float32.  On the tensor cores
 * (16-bit types, dim a multiple of 8 up to 128, the pool's strides multiples
 * of 16):
 *   Prompts round it to a->dtype for the products.  bfloat16 holds it exactly
 * where scales are powers of two, as clk_cache_append_rotary makes them.  For
 * float16, K and V are divided by a power of two each where a request's scales
 * reach beyond 2^7, so that rows at the top of the type's range and beyond it
 * are read as what they stand for; what is below 2^-14 of the type, so divided,
 * is rounded to a multiple of 2^-24.
 *   Trees multiply the values as they are: q's elements are held to 9 bits
 * (bfloat16; its own are 8) or 14 (float16; 11), or to 2^-18 of the row's
 * largest where that is more, and weights of cached tokens, times V's scales,
 * to float16, their largest at 2^5 or more; V's scales may be any from 2^-100
 * to 2^90.
 * Everything else is as without scales. */
CLK_API int clk_tree_attend_scaled(clk_cache* h, const int32_t* d_slots, int32_t B, const clk_pool* pool,
                                   const clk_scales* scales, int32_t layer, const clk_attn* a, int32_t N,
                                   const int32_t* d_nodes, const int64_t* d_mask, const int32_t* d_ctx, void* d_scratch,
                                   size_t scratch_bytes, clk_stream_t s);
CLK_API int clk_prompt_attend_scaled(const clk_attn* a, const int64_t* d_off, int32_t B, int64_t T, clk_cache* h,
                                     const int32_t* d_slots, const clk_pool* pool, const clk_scales* scales, int32_t layer,
                                     const int32_t* d_ctx, void* d_scratch, size_t scratch_bytes, clk_stream_t s);

/* ---------------------------------------------------------------------- */
/* Status, counters, inspection (these synchronise the stream)             */
/* ---------------------------------------------------------------------- */

/* Synchronises `s`, returns the latched device status in *dev_status (CLK_OK
 * if none) and, if detail != NULL, the slot (or batch position) it came
 * from.  The status stays latched until clk_status_clear. */
CLK_API int clk_status(clk_lookup* h, int32_t* dev_status, int32_t* detail, clk_stream_t s);
CLK_API int clk_status_clear(clk_lookup* h, clk_stream_t s);

/* Synchronises `s` and copies slot `slot`'s counters (slot = -1: the sum
 * over all slots) into *out. */
CLK_API int clk_read_counters(clk_lookup* h, int32_t slot, clk_counters* out, clk_stream_t s);

/* Synchronises `s` and copies slot `slot`'s scheduler/history state. */
CLK_API int clk_read_slot_info(clk_lookup* h, int32_t slot, clk_slot_info* out, clk_stream_t s);

/* Synchronises `s` and copies up to `cap` tokens of slot `slot`'s history
 * into host memory h_out; *n_out receives the history length. */
CLK_API int clk_lookup_read_history(clk_lookup* h, int32_t slot, int32_t* h_out, int64_t cap, int64_t* n_out,
                                    clk_stream_t s);

/* Checkpoint / resume of one request.  A snapshot is three reads:
 * clk_lookup_read_history, clk_read_slot_info and clk_read_counters (the
 * slot's own).  To resume it, in the same or another workspace with the same
 * parameters: clk_lookup_init(slot, history) rebuilds the history and its
 * index, then this call writes back the scheduler state (mode, streak, miss,
 * has_prev, cur_len) and the counters.  info->n must equal the slot's
 * history length; mode must be 0 or 1, streak and miss >= 0, has_prev 0 or
 * 1, cur_len 0 or a block length 1..16; else CLK_EINVAL and nothing is
 * written.  n_indexed and the index itself stay as clk_lookup_init left
 * them.  The caller keeps the previous step's accepted count and block
 * length (the inputs of the next scheduler step) with the snapshot.
 * Synchronises `s`. */
CLK_API int clk_lookup_restore_state(clk_lookup* h, int32_t slot, const clk_slot_info* info,
                                     const clk_counters* counters, clk_stream_t s);

/* Launch setting of the handle's fused verify calls (clk_verify_append,
 * clk_verify_sample_append).  alone = 0 (the default): a call expects to
 * follow the step's proposal launch directly on the stream and to overlap
 * it, so it gives its CTAs that will be dispatched behind the proposal's
 * CTAs a smaller share of the rows.  alone = 1: each call is launched with
 * nothing to overlap (e.g. other work or event records between the
 * launches), and every CTA gets an even share.  Results do not depend on it;
 * only the timing does.  Host-side only: affects the calls made after it.
 * CLK_ESTATE for a bad handle. */
CLK_API int clk_lookup_set_alone(clk_lookup* h, int32_t alone);

/* Frees the host handle (not the workspace). */
CLK_API void clk_lookup_destroy(clk_lookup* h);

#ifdef __cplusplus
}
#endif

#endif /* CLK_H */
