/*
 * detint — C ABI of the GB300 (sm_103a) integer-only LLM decoder.
 *
 * The library runs the integer-only decoder forward pass of a Qwen3- or
 * Llama-shaped model: every operation from input ids to int32 logits is
 * exact integer arithmetic, so logits and greedy tokens are bit-identical
 * across batch composition, prefill vs decode and backends ("DetLLM — Fully
 * Deterministic LLM Inference", intro; DetLLM blog "Eliminating
 * Nondeterminism in LLM Inference with Integer-Only Arithmetic", section
 * "DetLLM"). The user-level API of the pages is
 * `IntQwen3(path, backend).generate(ids, max_new, use_graph)` (README,
 * "Usage"); its C counterpart is detint_load + detint_prefill +
 * detint_decode_step.
 *
 * Conventions
 *  - Streams are `cudaStream_t` values passed as `detint_stream_t`. All
 *    compute calls are stream-ordered and asynchronous; they return after
 *    enqueueing work. The legacy default stream (NULL) is accepted but CUDA
 *    graphs are only used on a non-default stream.
 *  - Device pointers are owned by the caller unless stated. The model owns
 *    its weights, KV cache and scratch, released by detint_free.
 *  - Every call returns 0 (DETINT_OK) or a positive DETINT_E_* code; nothing
 *    aborts. detint_strerror names a code; detint_last_error gives the
 *    detail of the last failure in this process.
 *  - Conditions only the device can see (a token id >= vocab, a saturated
 *    residual/logit) are recorded in a status word read by detint_status.
 */
#ifndef DETINT_H
#define DETINT_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct detint_model detint_model;
typedef struct CUstream_st* detint_stream_t;   /* == cudaStream_t */

enum {
    DETINT_OK = 0,
    DETINT_E_ARG = 1,       /* null pointer, bad count or option */
    DETINT_E_SHAPE = 2,     /* unsupported sizes (e.g. K not a multiple of 16) */
    DETINT_E_TOKEN = 3,     /* status: a token id outside [0, vocab) */
    DETINT_E_CTX = 4,       /* a sequence would exceed max_ctx */
    DETINT_E_ARTIFACT = 5,  /* unreadable or malformed artifact file */
    DETINT_E_SHA = 6,       /* artifact SHA-256 differs from its .sha256 file */
    DETINT_E_CUDA = 7,      /* a CUDA call failed */
    DETINT_E_OOM = 8,       /* device allocation failed */
    DETINT_E_SEQ = 9,       /* sequence id outside [0, max_batch) or repeated */
    DETINT_E_SAT = 10       /* status: a saturation was recorded */
};

/* Load an artifact (format: the artifact section of the arithmetic
 * specification; header, int8 weights, dyadic channel scales, int16 gammas,
 * int16 Q14 RoPE tables, per-kv-head fixed K/V scales) after checking its
 * SHA-256 against `<path>.sha256` (README, "Demo": comparisons are valid only
 * for the same artifact hash). Allocates the weights, a paged int8 KV cache
 * for `max_batch` sequences of up to `max_ctx` positions, and scratch.
 * `max_ctx` <= the artifact's RoPE table length. Synchronous.
 * Errors: ARG, ARTIFACT, SHA, OOM, CUDA, SHAPE. */
int detint_load(const char* artifact_path, int max_batch, int max_ctx, detint_stream_t s,
                detint_model** out);

/* The same with a choice of the K/V cache's width: kv_bits 8 (detint_load) or
 * 4, the 4-bit paged cache below, at (head_dim + 2) / (2 head_dim) of the
 * bytes and with contexts up to 524288. The 4-bit cache's units are 1/14 of
 * the artifact's int8 steps (arithmetic specification, section 16); logits
 * differ from the 8-bit model's, and are as invariant over batches, splits
 * and kernels as they are there. Its decode steps run one kernel per phase,
 * so the one-launch and staged-attention options have no effect.
 * Errors: as detint_load, and ARTIFACT for K/V parameters outside that
 * section's domain. */
int detint_load_kv(const char* artifact_path, int max_batch, int max_ctx, int kv_bits, detint_stream_t s,
                   detint_model** out);

/* Prefill: append a ragged batch of prompts to the KV caches of `n_seq`
 * distinct sequences and return the logits of each sequence's last new
 * position (DetLLM blog, "DetLLM": prefill and decode see the same cached
 * bits). seq_ids: host int32[n_seq], each in [0, max_batch), distinct.
 * cu_lens: host int32[n_seq + 1] (a host array, not a device one: the
 * library plans KV blocks and attention query blocks from the lengths
 * before it enqueues any kernel), cu_lens[0] = 0, non-decreasing, each
 * length >= 1; tokens of sequence i are tokens[cu_lens[i] .. cu_lens[i+1]).
 * tokens: device int32[cu_lens[n_seq]]. logits: device int32[n_seq][vocab]
 * or NULL. next_tok: device int32[n_seq] (argmax, ties to the lowest id).
 * Positions continue from each sequence's current length, so a prompt may
 * be split across calls (split prefill) with identical results.
 * Errors: ARG, SEQ, CTX, CUDA, OOM. */
int detint_prefill(detint_model* m, int n_seq, const int32_t* seq_ids, const int32_t* cu_lens,
                   const int32_t* tokens, int32_t* logits, int32_t* next_tok, detint_stream_t s);

/* One greedy decode step: one new token per sequence, appended to its KV
 * cache, then int32 logits and the tie-low argmax of the new position
 * (DetLLM blog, "DetLLM": decode reads the same cached integers a prefill
 * writes, and argmax prefers the smallest token id on ties; README, "Usage":
 * generate(ids, max_new, use_graph) is a prefill followed by such steps).
 * seq_ids: host int32[n_seq]; tok: device int32[n_seq]; logits: device
 * int32[n_seq][vocab] or NULL; next_tok: device int32[n_seq] (may alias
 * tok). With graphs enabled (default) the step is one CUDA-graph launch,
 * re-captured when the sequence set or a pointer changes.
 * Errors: ARG, SEQ, CTX, CUDA. */
int detint_decode_step(detint_model* m, int n_seq, const int32_t* seq_ids, const int32_t* tok,
                       int32_t* logits, int32_t* next_tok, detint_stream_t s);

/* Exact int8 x int8 -> int32 GEMM: C[m][n] = sum_k A[m][k] * B[n][k].
 * A: device int8 [M][K] row-major; B: device int8 [N][K] row-major (the
 * weight layout); C: device int32 [M][N]. M, N >= 1; K >= 16 and a multiple
 * of 16; A, B 16-byte aligned. The integer GEMM is the one operation the
 * pages dispatch per device (README, "Layout": int_gemm). Errors: ARG,
 * SHAPE, CUDA. */
int detint_gemm_i8(const int8_t* A, const int8_t* B, int32_t* C, int M, int N, int K,
                   detint_stream_t s);

/* Tie-low argmax of `rows` int32 rows of length `n` (device, row-major) into
 * out[rows] (device int32), for callers that cannot allocate device memory:
 * code running inside a stream capture that must stay allocation-free, in a
 * host callback, or under an application that owns every allocation. This
 * entry point calls no cudaMalloc/cudaFree or allocating library routine;
 * its per-block partial results live in one fixed device array of 128 KB
 * that every GPU loading this library holds until the process exits.
 * Limits: rows <= DETINT_ARGMAX_NOALLOC_MAX_ROWS, n <=
 * DETINT_ARGMAX_NOALLOC_MAX_COLS; larger sizes return DETINT_E_SHAPE.
 * The first call on a device looks up that array's device address (with the
 * device current), so make it before any stream capture. All calls share the
 * one array: calls that overlap on the GPU (different streams, no ordering)
 * race and give wrong results; calls ordered on one stream are safe. Each
 * call writes every partial slot it reads, so no clearing is needed.
 * Ties go to the lowest column, as in the decode steps' token choice. The
 * pages have no counterpart to this entry point.
 * Errors: ARG, SHAPE, CUDA. */
#define DETINT_ARGMAX_NOALLOC_MAX_ROWS 64
#define DETINT_ARGMAX_NOALLOC_MAX_COLS 1048576
int detint_argmax_noalloc(const int32_t* logits, int rows, int n, int32_t* out, detint_stream_t s);

/* Forget a sequence's cached context (length back to 0) and return its KV
 * blocks to the pool. No passage of the pages defines this: it is library
 * housekeeping for reusing a sequence slot (the scheduler cases of the
 * BitExact LLM post, "What the checks actually compare": preemption then
 * recomputation, start from an emptied slot). Synchronises the device
 * first. Errors: ARG, SEQ, CUDA. */
int detint_reset_seq(detint_model* m, int seq_id);

/* Current length of a sequence (host-side bookkeeping). */
int detint_seq_len(detint_model* m, int seq_id, int32_t* len);

/* Read and clear the device status word after synchronising `s`.
 * flags: host int32[8] or NULL; slots 0 token id out of range, 1 context
 * clamp, 2 residual saturation, 3 gate/up saturation, 4 logit saturation,
 * 5 q/k/v saturation, 6 a bounded wait of a kernel timed out (its results
 * are invalid). Returns DETINT_E_TOKEN if slot 0 is set, else
 * DETINT_E_CTX if slot 1 is set, else DETINT_OK. */
int detint_status(detint_model* m, int32_t* flags, detint_stream_t s);

/* Enable (1, default) or disable (0) CUDA-graph replay of decode steps
 * (README, "Usage": use_graph). */
int detint_set_graph(detint_model* m, int enable);

/* Exact int8 x int16 GEMM for wide-weight ("exact mode") linear layers:
 * C[m][n] = sum_k A[m][k] W[n][k] in int64, with int8 activations A
 * [M][K] and int16 weights W [N][K] given as two int8 limbs,
 * W = 256 * w_hi + w_lo (w_hi int8, w_lo uint8; detint_split_w16 makes them).
 * Both limb products run on the int8 tensor pipe in one pass and are
 * combined exactly (BitExact LLM post, "Fix the arithmetic, not just the
 * random seed": products of split integer limbs combined in wider
 * accumulators; its exact mode keeps wide weights). Device pointers, all
 * 16-byte aligned, caller-owned; K % 16 == 0 and K <= 65536. Asynchronous
 * on s. Errors: ARG, SHAPE, CUDA. */
int detint_gemm_w16(const int8_t* A, const int8_t* w_hi, const uint8_t* w_lo, int64_t* C, int M, int N,
                    int K, detint_stream_t s);
/* w_hi[i] = W[i] >> 8 (floor), w_lo[i] = W[i] & 255, for count elements
 * (device pointers). Errors: ARG, CUDA. */
int detint_split_w16(const int16_t* W, int8_t* w_hi, uint8_t* w_lo, long long count, detint_stream_t s);

/* Start sequence dst (which must be empty) with the first n_tokens positions
 * of sequence src, without recomputing them: whole 64-token KV blocks are
 * shared by reference count, the partial last block is copied, and later
 * appends to either sequence go to blocks of its own. Continuing dst gives
 * the same logits, bit for bit, as prefilling the same tokens afresh
 * (scheduler invariance: BitExact LLM post, "What the checks actually
 * compare" lists shared prefixes among the tested scheduler changes).
 * Stream-ordered on s. Errors: ARG, SEQ (ids out of range or equal, dst not
 * empty), CTX (block pool exhausted), CUDA. */
int detint_fork_seq(detint_model* m, int src, int dst, int n_tokens, detint_stream_t s);

/* Reorder sequences, as beam search does between steps: sequence seq_ids[i]
 * (host int32[n], distinct) becomes what sequence seq_ids[parents[i]] was (host
 * int32[n], values 0..n - 1), several of them the same one where parents
 * repeat. Whole blocks are shared by reference count, as detint_fork_seq shares
 * them; a block that is still being filled goes to the first of its sequence's
 * children and is copied for the others, in every layer, into blocks that
 * sequences without children give back: a beam search needs no more of them.
 * Continuing a sequence gives the same logits, bit for bit, as prefilling its
 * tokens afresh. ARG, SEQ, CTX and OOM change nothing. Stream-ordered on s. Errors:
 * ARG, SEQ, CTX (block pool exhausted), OOM (host memory), CUDA. */
int detint_reorder_seqs(detint_model* m, int n, const int32_t* seq_ids, const int32_t* parents, detint_stream_t s);

/* Integer sampling parameters of one row (see detint_sample). */
typedef struct {
    uint64_t seed;      /* SplitMix64 seed */
    uint64_t counter;   /* draw index: output counter + 1 of the generator */
    int32_t inv_temp;   /* Q16 of 1/temperature, 0 .. 2^20 (65536: T = 1; 0: uniform) */
    int32_t top_k;      /* keep the top_k largest logits (0 or >= n: off) */
    int32_t top_p;      /* Q16 nucleus mass, 1 .. 65536 (65536: off) */
    int32_t reserved;   /* set to 0 */
} detint_sampling_t;

/* Draw one token per logits row with integer arithmetic only: weights
 * E_i = exp2q(u_i - max u), u = the logit in base-2 Q10 at the temperature;
 * the top_k largest logits (ties by lower index), then the shortest prefix
 * of them (logit order) holding top_p of their weight plus its boundary ties;
 * then t = floor(r S / 2^64) with r = SplitMix64(seed, counter) and S the
 * kept weight, and the token is the first index (index order) whose
 * cumulative kept weight exceeds t. The pages ask for integer sampling rules
 * and deterministic sampling (BitExact LLM post, "Fix the arithmetic, not
 * just the random seed"; "Reproducibility has a cost") without an algorithm;
 * this is the reading in the arithmetic specification, section "Integer
 * sampling". top_k = 1 gives the tie-low argmax for every seed.
 * logits: device int32 [rows][n] (caller-owned); params: host [rows];
 * out: device int32 [rows]. Asynchronous on s; allocates nothing.
 * Errors: ARG (null pointer, rows or n < 1, a parameter out of range), CUDA. */
int detint_sample(const int32_t* logits, int rows, int n, const detint_sampling_t* params,
                  int32_t* out, detint_stream_t s);

/* Options: DETINT_OPT_GRAPH (1 = replay decode steps as CUDA graphs, the
 * default; same as detint_set_graph), DETINT_OPT_FUSED_DECODE (1 = decode
 * batches of up to 8 sequences through the fused streaming kernels, the
 * default; 0 = through the separate row kernels) and DETINT_OPT_TC_PREFILL
 * (1 = prefill attention on the int8 tensor pipe in two sweeps over the keys,
 * the default where head_dim is 64 or 128; 0 = the per-token attention
 * kernel) and DETINT_OPT_STAGED_DECODE (1 = fused decode attention with the
 * sequence's cached K/V copied into shared memory before the step's data is
 * ready, the default while every context fits that copy; 0 = the attention
 * kernel that reads the cache from global memory) and DETINT_OPT_PERSISTENT
 * (1 = a fused decode step of up to 8 sequences runs as one cooperative
 * launch of one CTA per SM whose phases hand rows to one another as tagged
 * words, where the shape fits; 0 = one kernel per phase). Every setting gives
 * bit-identical results.
 * DETINT_OPT_WAIT_TEST (value >= 0) exercises the failure path of the
 * one-launch step's bounded waits: while it is positive, the step's final
 * wait expects a tag that no CTA writes and gives up after `value` polls,
 * so the step ends with status slot 6 (a wait timed out) set and an invalid
 * token, without hanging; 0 (the default) turns it off. No passage of the
 * pages: a test hook of the library's failure detection.
 * Errors: ARG. */
enum { DETINT_OPT_GRAPH = 0, DETINT_OPT_FUSED_DECODE = 1, DETINT_OPT_TC_PREFILL = 2,
       DETINT_OPT_STAGED_DECODE = 3, DETINT_OPT_PERSISTENT = 4, DETINT_OPT_WAIT_TEST = 5 };
int detint_set_option(detint_model* m, int option, int value);

/* Integer-pipe peak loop, the measured denominator of the int8 GEMM and
 * prefill roofline fractions (no passage of the pages: a measurement
 * routine). kind 0: blocks x 256 threads of independent mma.sync m16n8k32
 * s8 operations on register operands; kind 1: the same with dp4a. Each
 * thread runs `iters` rounds and stores its 8 accumulators' checksums
 * into sink (device int32[blocks * 256 * 8], caller-owned); *ops (host) receives the integer
 * operations the launch performs (2 per multiply-add). Time it with events
 * on `s`. Asynchronous; allocates nothing. Errors: ARG, CUDA. */
int detint_int8_peak_loop(int kind, int blocks, int iters, int32_t* sink, long long* ops,
                          detint_stream_t s);

/* Shape of the loaded model: info[0..9] = n_layers, hidden, n_q, n_kv,
 * head_dim, ffn, vocab, max_pos, qk_norm, max_batch; info[10] = max_ctx. */
int detint_model_info(detint_model* m, int32_t* info);

/* ---- The 4-bit paged key/value cache (arithmetic specification, section 16).
 * The pages keep K and V in int8 with fixed scales (DetLLM blog, "DetLLM");
 * no passage of them defines a narrower cache. Here a cached integer is a
 * 4-bit code in -7..7 times the scale code (1..255) of its token and kv head,
 * so a token takes head_dim + 2 bytes per kv head for K and V together.
 *
 * Every call works on the caller's device memory and allocates nothing. The
 * tokens of a call are given by device arrays, so that a captured call can be
 * replayed after they changed: tok_seq[t] is a row of the block table,
 * tok_pos[t] the token's position in its sequence. A negative position marks
 * a padding token: nothing is appended for it, its query codes are zero and
 * its attention output is a zero row. What is outside its range sets slot 1
 * of `status`: for a position past the rotation's max_pos append does as for
 * padding; where the sequence, the position or the page is outside the block
 * table or the pool it leaves the token's keys and values out and quantises
 * its query all the same. Attention gives a zero row for a token outside the
 * table or past max_len; the keys of a page outside the pool are
 * masked. All three operators are exact integer arithmetic: the same inputs
 * give the same bits whatever the batch, the split or the kernel. */
typedef struct {
    int32_t n_q, n_kv;           /* heads; n_q = n_kv times 1..64, at most 1024 */
    int32_t head_dim;            /* 64 or 128 */
    int32_t n_blocks;            /* pages; a page holds 64 tokens of every kv head */
    int32_t n_seq, max_blocks;   /* block_table [n_seq][max_blocks] */
    uint8_t* k;                  /* [n_blocks][n_kv][64 * head_dim / 2] codes, 16-byte aligned */
    uint8_t* v;                  /* the same size; layout in the specification */
    uint8_t* k_scale;            /* [n_blocks][n_kv][64] scale codes */
    uint8_t* v_scale;
    const int32_t* block_table;  /* page of each 64 positions of a sequence */
    const int32_t* params;       /* [n_kv][8 + head_dim]: KQM KQS VQM VQS MV KV CSTM CSTK, then the
                                    key exponent 0..3 of every channel */
    int32_t* status;             /* device int32[8] (the slots of detint_status), or NULL */
} detint_kv4_t;

/* Rotation and normalisation of the query and key heads. The first rot_dim
 * channels rotate, in pairs (i, i + rot_dim / 2) or, interleaved, (2i, 2i+1),
 * by row tok_pos of the Q14 tables; the others pass. The tables are data
 * (README, "Layout": precomputed int16 sin/cos tables): positions scaled for
 * long contexts are scaled when they are made. q_gamma and k_gamma (Q12,
 * magnitudes up to 2^14) ask for the per-head RMS norm; without them the Q12
 * inputs are used as they are. */
typedef struct {
    const int16_t *cos, *sin;            /* [max_pos][rot_dim / 2], 8-byte aligned */
    int32_t max_pos;
    int32_t rot_dim;                     /* a multiple of 8, 0 (none) .. head_dim */
    int32_t interleaved;                 /* 0 or 1 */
    int32_t eps;                         /* round(eps 2^24), 0 .. 32767 */
    const int16_t *q_gamma, *k_gamma;    /* [head_dim] both, or NULL both */
} detint_rope_t;

/* Norm, rotate and quantise the projections of n_tok tokens, and append their
 * keys and values to the pages. qkv: device int32 rows (Q12) of n_q query,
 * n_kv key and n_kv value heads, qkv_stride elements apart (a multiple of 4).
 * q8 [n_tok][n_q][head_dim] and mq, kq [n_tok][n_q] receive the query codes
 * and their dyadic scales; k_val, v_val [n_tok][n_kv][head_dim], where given,
 * the integers the cache now holds for these tokens (zeros for a token that
 * was not appended). No two tokens of a call may fall on the same place of a
 * page: the codes there would be undefined.
 * Errors: ARG, SHAPE, CUDA. */
int detint_kv4_append(const detint_kv4_t* c, const detint_rope_t* r, const int32_t* qkv, long long qkv_stride,
                      const int32_t* tok_seq, const int32_t* tok_pos, int n_tok, int8_t* q8, int32_t* mq,
                      int32_t* kq, int16_t* k_val, int16_t* v_val, detint_stream_t s);

/* Bytes of workspace (16-byte aligned) that are enough for every
 * detint_kv4_decode of up to n_tok tokens with a max_len up to this one, with
 * any window; 0 for most sizes. A buffer sized for the largest batch and
 * context serves all calls below them. Two calls that may
 * overlap on the GPU, captured ones included, need a workspace each.
 * Errors: ARG, SHAPE, CUDA. */
int detint_kv4_workspace(const detint_kv4_t* c, int n_tok, int max_len, long long* bytes);

/* Attention of single tokens over the cache: token t sees the keys 0..tok_pos[t]
 * of its sequence, or the last `window` of them where window > 0. o: int32
 * Q12 rows [n_tok], o_stride elements apart (even). max_len (1..524288) is a
 * bound of every tok_pos + 1 of the call; a token beyond it is flagged and
 * gets a zero row. Each token is a unit of its own whose keys are split over
 * CTAs, so this is the call for one or a few tokens of each sequence.
 * Errors: ARG, SHAPE, CUDA. */
int detint_kv4_decode(const detint_kv4_t* c, const int8_t* q8, const int32_t* mq, const int32_t* kq,
                      const int32_t* tok_seq, const int32_t* tok_pos, int n_tok, int max_len, int window,
                      int32_t* o, long long o_stride, void* workspace, long long workspace_bytes,
                      detint_stream_t s);

/* The same attention with the same result, bit for bit, for many tokens of a
 * sequence: blocks of consecutive tokens of the call share one sweep over
 * their keys on the int8 tensor pipe. Tokens of one sequence should stand
 * together. No workspace: so few tokens that one wave of the single-token form
 * takes them are handed to it. Errors: ARG, SHAPE, CUDA. */
int detint_kv4_prefill(const detint_kv4_t* c, const int8_t* q8, const int32_t* mq, const int32_t* kq,
                       const int32_t* tok_seq, const int32_t* tok_pos, int n_tok, int max_len, int window,
                       int32_t* o, long long o_stride, detint_stream_t s);

/* Append with rotary positions of their own: tok_pos[t] is the token's place in
 * the cache, as everywhere, and rope_pos [n_axes][n_tok] (device int32) the rows
 * of the rotation tables, one for each axis. axis [rot_dim / 2] (device uint8,
 * values 0..n_axes - 1, larger ones count as the last) names the axis of each
 * pair; NULL for a single axis. n_axes is 1..4: time, height and width of a
 * picture's patches, in sections of the head or interleaved, or one axis for a
 * token whose place is not its position any more because keys before it were
 * evicted. A token with a rope_pos outside [0, max_pos) is treated as padding
 * and sets slot 1 of `status`; everything else is detint_kv4_append's.
 * Errors: ARG, SHAPE, CUDA. */
int detint_kv4_append_axes(const detint_kv4_t* c, const detint_rope_t* r, const int32_t* rope_pos, const uint8_t* axis,
                           int n_axes, const int32_t* qkv, long long qkv_stride, const int32_t* tok_seq,
                           const int32_t* tok_pos, int n_tok, int8_t* q8, int32_t* mq, int32_t* kq, int16_t* k_val,
                           int16_t* v_val, detint_stream_t s);

/* ---- What a context's keys are worth, and eviction (arithmetic specification,
 * sections 18 and 19). No passage of the pages: they keep every key. */

/* Add to the weight of every key that a token sees the probabilities (Q24) that
 * the q heads of the key's kv head give it: weight is device int64
 * [n_blocks][n_kv][64], in the order of the scale codes, 16-byte aligned and
 * owned by the caller, who clears it. Tokens, max_len and window are
 * detint_kv4_decode's; a token without keys adds nothing. Sums are exact, so
 * neither the order of the tokens nor pages that sequences share change them.
 * Each token is a unit of its own whose keys are split over CTAs. No
 * workspace. Errors: ARG, SHAPE, CUDA. */
int detint_kv4_weigh(const detint_kv4_t* c, const int8_t* q8, const int32_t* mq, const int32_t* kq, const int32_t* tok_seq,
                     const int32_t* tok_pos, int n_tok, int max_len, int window, int64_t* weight, detint_stream_t s);

/* The same weights, bit for bit, for many tokens of a sequence, which should
 * stand together: blocks of consecutive tokens of the call share a sweep over
 * their keys on the int8 tensor pipe. Few tokens, and all of a call that allows a
 * token more than 32768 keys (by max_len, or by window where there is one), are
 * weighed one by one as by detint_kv4_weigh, so a max_len far above the tokens'
 * contexts costs time. Errors: ARG, SHAPE, CUDA. */
int detint_kv4_weigh_block(const detint_kv4_t* c, const int8_t* q8, const int32_t* mq, const int32_t* kq,
                           const int32_t* tok_seq, const int32_t* tok_pos, int n_tok, int max_len, int window,
                           int64_t* weight, detint_stream_t s);

/* Keep `keep` tokens of each of n sequences and move them to new pages. seq,
 * lens: device int32 [n], rows of the block table and the tokens that they hold
 * now, at most max_len. For every kv head by itself the first `sinks` and the
 * last `recent` tokens stay, and of those between them the keep - sinks -
 * recent of the largest weights (the lower place first among equal ones). They
 * go, in their order, to places 0, 1, ... of the pages new_table [n][ceil(keep /
 * 64)] (device int32), with codes, scale codes and weights; a sequence of keep
 * tokens or fewer is moved whole. kept: device int32 [n][n_kv][keep], the old
 * places, -1 behind the last. The new pages must be in no sequence's use;
 * places behind the last kept token are left as they were. The caller puts the
 * new pages into the block table, appends from place min(lens, keep) on with
 * detint_kv4_append_axes, and may free the old pages. A token on a page outside
 * the pool weighs 0 and moves as a zero key and value; it, a sequence outside
 * the table, a length outside 0..max_len and a new page outside the pool (which
 * is skipped) set slot 1 of `status`. Weights that another stream changes during
 * the call may give any choice, even of fewer than keep tokens, and nothing
 * worse; the other inputs must not change. Errors: ARG, SHAPE, CUDA. */
int detint_kv4_evict(const detint_kv4_t* c, int64_t* weight, const int32_t* seq, const int32_t* lens, int n, int max_len,
                     int keep, int sinks, int recent, const int32_t* new_table, int32_t* kept, detint_stream_t s);

/* Copy whole pages of every kv head, src[i] to dst[i] (device int32 [n]): codes,
 * scale codes and, where weight is given, weights. A negative entry copies
 * nothing; one past the pool sets slot 1 of `status`. No page may be copied to
 * twice or be both copied from and to in a call. Errors: ARG, SHAPE, CUDA. */
int detint_kv4_copy(const detint_kv4_t* c, const int32_t* src, const int32_t* dst, int n, int64_t* weight,
                    detint_stream_t s);

/* ---- Beam search (arithmetic specification, section 17). The pages decode
 * greedily (DetLLM blog, "DetLLM"); no passage of them defines beams. */

/* The n_out (1..64) best continuations of each group of `beams` (1..64) rows.
 * logits: device int32 Q16 rows of n elements, `stride` apart, group after
 * group; -2^31 masks a token. scores: device int64 [groups][beams], the beams'
 * log-probabilities in Q16; below -2^62 the beam is not there (the first step of
 * a group has one beam). done: device int32 [groups][beams] or NULL: a beam with
 * a nonzero entry is finished and continues with end_id alone at its score.
 * Continuation i of a row scores score + l_i - lse(l), in whole units of Q16;
 * the larger score comes first, then the lower beam, then the lower token.
 * Outputs [groups][n_out], best first: parent (the beam in its group), token,
 * score, and done_out (1 where the parent was finished or the token is end_id);
 * where there are fewer continuations, parent and token -1, score -2^63 and
 * done 0. scores and done may be the outputs of the call before but not of this
 * one: outputs or a workspace that overlap another array are refused. end_id -1:
 * no token ends a beam. workspace: detint_beam_workspace bytes, 16-byte aligned;
 * calls that may overlap on the GPU, captured ones included, need one each. Up to
 * 65535 rows of up to 2^24 logits.
 * Errors: ARG, SHAPE, CUDA. */
int detint_beam_select(const int32_t* logits, long long stride, int n, const int64_t* scores, const int32_t* done,
                       int groups, int beams, int end_id, int n_out, int32_t* parent, int32_t* token, int64_t* score,
                       int32_t* done_out, void* workspace, long long workspace_bytes, detint_stream_t s);

/* Bytes of workspace for detint_beam_select of `rows` rows (groups times beams)
 * of n logits; enough for fewer rows and any n and n_out. Errors: ARG. */
int detint_beam_workspace(int rows, int n, int n_out, long long* bytes);

/* The block tables of the chosen beams. block_table: device int32 [groups *
 * beams][max_blocks]; parent: device int32 [groups][beams], as detint_beam_select
 * gives it; lens: device int32 [groups], the tokens that every beam of the group
 * holds. A beam that goes on as it is names itself. Row b of out (which may be
 * block_table itself) gets its parent's whole pages, shared. Of the page that is
 * still being filled, a beam's first child becomes the owner;
 * each other child gets the page of a beam that has no child, and an entry of
 * src and dst (device int32 [groups][beams], -1: none) that detint_kv4_copy
 * takes, once per layer, before the next append. So a group needs no page that it
 * does not have; its beams' growing pages and the entries behind them must be
 * distinct from the start. Later columns stay. A parent outside 0..beams - 1 (-1
 * where continuations ran out) means that the row holds no beam from now on: its
 * whole pages stay, but the page that is still being filled is dealt out with
 * those of the beams that have no child, so the row may end with the last tokens
 * of another beam, and nothing is copied for it. src, dst and an out that is not
 * block_table may overlap no other array. Errors: ARG, CUDA. */
int detint_beam_reorder(const int32_t* block_table, int32_t* out, int max_blocks, const int32_t* parent, const int32_t* lens,
                        int groups, int beams, int32_t* src, int32_t* dst, detint_stream_t s);

/* Release everything the model owns. NULL is a no-op. No passage of the
 * pages: library housekeeping. */
void detint_free(detint_model* m);

/* A static English name of an error code ("unknown error" for other
 * values); detint_last_error gives the detail of this thread's last
 * failure. No passage of the pages: library housekeeping. */
const char* detint_strerror(int code);
const char* detint_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* DETINT_H */
