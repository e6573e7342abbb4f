/*
 * ember.h -- C ABI of the GB300 (sm_103a) decoder forward library.
 *
 * One forward pass of a Llama/Qwen2-style decoder-only transformer: embedding
 * gather; per layer RMSNorm, q/k/v projections (optional biases, optional
 * per-head q/k RMSNorm), rotate-half RoPE (plain or llama3-scaled),
 * grouped-query attention over a causal bf16 KV cache (or unmasked, for the
 * bidirectional encoder variant), o_proj and a SwiGLU MLP; then a final
 * RMSNorm, a tied LM head (or a linear label head) and greedy argmax.  It runs
 * as one prefill followed by one cached decode step per new token.
 *
 * Where each operation is defined (page title, section / function):
 *   ember, scripts/reference_forward.py: forward() -- rmsnorm, q/k/v + bias,
 *     rope() rotate-half, KV append, per-head GQA loop, o_proj, SwiGLU, tied
 *     head; main() -- the greedy loop; load_safetensors() -- bf16 decode.
 *   LowLlamaBasic, reference.py: predict() -- rotary_cos_sin() with llama3
 *     scaling, self_attn() causal whole-sequence attention.
 *   PII-Tracer-vLLM, serving/reference_forward.py: forward() -- per-head q/k
 *     RMSNorm before RoPE, bidirectional attention, token_cls_head (+ bias).
 *   Falcon-H1-0.5B-Rust, src/lib.rs: Config::validate and logits()/generate()
 *     -- the argument errors mirrored by EMBER_ERR_INVALID_ARG / _TOKEN.
 *   ember internals: "ForwardModel trait" -- create_cache(max_seq_len) and
 *     forward_with_cache(ids, cache, start_pos), the shape of this ABI;
 *     "kv cache" -- one contiguous block per layer, a cursor that advances once
 *     per token after all layers, explicit positions (the prefill bug);
 *     "qk_scratch" -- no allocation on the hot path.
 *
 * Conventions for every call:
 *   - Pointers named ids / seqs / positions / logits / argmax / hidden / out and
 *     every weight pointer are DEVICE pointers (cudaMalloc'd or equivalent);
 *     every other pointer is a host pointer.
 *   - Calls that take a stream are asynchronous on it: the library enqueues
 *     kernels and returns.  Argument errors detectable on the host return at
 *     once; errors that depend on device data (a token id >= vocab, a position
 *     that disagrees with the cache cursor) raise a device-side status that
 *     ember_sync_status() reports.  The kernels never read or write outside
 *     their buffers on such errors: the offending token is skipped.
 *   - Nothing allocates device memory after ember_model_create / ember_kv_alloc
 *     except the first decode call of a new (batch, pointer) signature, which
 *     instantiates a CUDA graph for it.
 *   - ember_last_error() returns a thread-local message for the last failure.
 *   - Only one stream may use a given model at a time: the model owns one
 *     activation workspace.
 */
#ifndef EMBER_H
#define EMBER_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st;
/* A cudaStream_t; NULL means the legacy default stream. */
typedef struct CUstream_st *ember_stream_t;

typedef enum ember_status {
    EMBER_OK = 0,
    EMBER_ERR_INVALID_ARG = 1, /* bad dims, null pointer, n == 0, bad seq index       */
    EMBER_ERR_CAPACITY = 2,    /* start_pos + n > max_len, n > max_tokens, batch too big */
    EMBER_ERR_STATE = 3,       /* a position disagrees with the sequence's cursor        */
    EMBER_ERR_TOKEN = 4,       /* a token id outside [0, vocab) (found on the device)    */
    EMBER_ERR_TIMEOUT = 5,     /* a bounded device wait gave up                          */
    EMBER_ERR_CUDA = 6,        /* a CUDA runtime / driver call failed                    */
    EMBER_ERR_OOM = 7,         /* device allocation failed                               */
    EMBER_ERR_UNSUPPORTED = 8, /* a valid request this build does not serve              */
    EMBER_ERR_RANGE = 9        /* an activation outside the f16 range of the tensor-core
                                  operands (|v| > 65504 or NaN; found on the device)     */
} ember_status;

/* Model hyper-parameters.  Field names follow the HuggingFace config.json
 * fields the pages read (ember reference_forward.py main(); LowLlamaBasic
 * predict(); PII-Tracer forward(): head_dim is explicit, not hidden/heads).
 * Validation (Falcon-H1 Config::validate): every dimension > 0,
 * n_heads % n_kv_heads == 0, head_dim even; this build additionally needs
 * hidden and ff to be multiples of 8 (16-byte weight rows), head_dim one of
 * 16, 32, 64, 128, n_heads/n_kv_heads <= 16, hidden <= 8192, ff <= 16384. */
typedef struct ember_config {
    int32_t vocab, hidden, layers, n_heads, n_kv_heads, head_dim, ff;
    double rope_theta;       /* RoPE base                                         */
    double rms_eps;          /* RMSNorm epsilon                                   */
    int32_t rope_llama3;     /* 1: llama3 frequency scaling (LowLlamaBasic)       */
    double rs_factor, rs_low, rs_high; /* llama3 factor, low/high freq factors   */
    int32_t rs_orig_max_pos; /* llama3 original_max_position_embeddings           */
    int32_t qkv_bias;        /* 1: q/k/v projections carry biases (Qwen2)         */
    int32_t qk_norm;         /* 1: per-head RMSNorm of q and k before RoPE (Qwen3)*/
    int32_t causal;          /* 1: causal decoder; 0: bidirectional encoder       */
    int32_t n_labels;        /* 0: tied LM head over vocab; >0: linear head       */
    int32_t max_tokens;      /* capacity of one prefill / encode / decode call in
                                tokens (0 -> 4096); sizes the workspace           */
    int32_t max_positions;   /* RoPE table length for encode (0 -> max_tokens)    */
    int32_t weights_q8;      /* 1: the layer matrices (q/k/v, o, gate/up, down)
                                are quantized to q8_0 blocks at model creation
                                (ember internals, q8_0: 32 int8 codes per f16
                                scale d, value = code * d; codes = the nearest
                                integer to w / (amax/127), d = f16(amax/127)) and
                                every later product uses the decoded values, not
                                the bf16 inputs.  Needs hidden, ff and
                                n_heads*head_dim to be multiples of 32 and every
                                |w| / 127 within the f16 range (else
                                UNSUPPORTED).  Embedding, head and norms stay as
                                given.                                           */
} ember_config;

/* One layer's weights: device pointers to bf16 bit patterns, HuggingFace
 * [out_features, in_features] row-major.  Biases / q_norm / k_norm may be NULL
 * when the config disables them. */
typedef struct ember_layer_weights {
    const uint16_t *attn_norm;          /* [hidden]                          */
    const uint16_t *wq, *wk, *wv;       /* [NH*D, hidden], [NKV*D, hidden] x2 */
    const uint16_t *bq, *bk, *bv;       /* [NH*D], [NKV*D], [NKV*D]          */
    const uint16_t *q_norm, *k_norm;    /* [head_dim]                        */
    const uint16_t *wo;                 /* [hidden, NH*D]                    */
    const uint16_t *mlp_norm;           /* [hidden]                          */
    const uint16_t *w_gate, *w_up;      /* [ff, hidden]                      */
    const uint16_t *w_down;             /* [hidden, ff]                      */
} ember_layer_weights;

typedef struct ember_weights {
    const uint16_t *embed;              /* [vocab, hidden]; tied LM head     */
    const uint16_t *final_norm;         /* [hidden]                          */
    const uint16_t *cls_w, *cls_b;      /* [n_labels, hidden], [n_labels]    */
    const ember_layer_weights *layers;  /* HOST array of `layers` entries    */
} ember_weights;

typedef struct ember_model ember_model;
typedef struct ember_kv ember_kv;

/* Validate the config, repack the weights into the library's device layout
 * (fused [q;k;v] rows, interleaved gate/up rows, f32 norms and biases) and
 * allocate the activation workspace for cfg->max_tokens tokens.  The caller
 * keeps ownership of its weight buffers and may free them once this returns
 * (the call synchronises the device).  Errors: INVALID_ARG, OOM, CUDA. */
ember_status ember_model_create(const ember_config *cfg, const ember_weights *w,
                                ember_model **out);
void ember_model_destroy(ember_model *m);

/* Bytes of one bf16 KV cache for max_seqs sequences of max_len positions:
 * layers * 2 (K and V) * n_kv_heads * max_len * head_dim * 2 bytes * max_seqs
 * (ember internals, "kv cache": one contiguous block per layer). */
size_t ember_kv_bytes(const ember_config *cfg, int32_t max_seqs, int32_t max_len);

/* Allocate a zeroed bf16 KV cache ([seq][layer][kv_head][pos][head_dim] for
 * K and for V) and zeroed cursors, plus the RoPE tables for max_len
 * positions.  Errors: INVALID_ARG (max_seqs or max_len <= 0, encoder model),
 * OOM, CUDA. */
ember_status ember_kv_alloc(ember_model *m, int32_t max_seqs, int32_t max_len, ember_kv **out);
/* Synchronises the device, frees the cache and drops the decode graphs
 * captured against it.  A cache may outlive its model (it is then only good
 * for ember_kv_free; ember_kv_layout returns STATE). */
void ember_kv_free(ember_kv *kv);

/* Set sequence seq's cursor to 0 (its rows are left as they are and are
 * overwritten by the next prefill).  Asynchronous on stream. */
ember_status ember_kv_reset(ember_kv *kv, int32_t seq, ember_stream_t stream);

/* Set sequence seq's cursor to pos (0 <= pos <= max_len): rewinds a sequence
 * to an earlier length, keeping rows [0, pos).  Asynchronous on stream.
 * Errors: INVALID_ARG (seq out of range), CAPACITY (pos out of range). */
ember_status ember_kv_set_cursor(ember_kv *kv, int32_t seq, int32_t pos, ember_stream_t stream);

/* Read-only view of the cache for inspection: device base pointers of K and
 * V (bf16 bits) and the element strides of [seq, layer, kv_head, pos]; the
 * head_dim stride is 1. */
ember_status ember_kv_layout(const ember_kv *kv, const uint16_t **k_base,
                             const uint16_t **v_base, int64_t strides[4]);

/* Prefill: run n tokens ids[0..n) of sequence seq at positions
 * start_pos .. start_pos+n-1 through every layer, appending their K/V rows,
 * then advance the cursor to start_pos + n (ember internals, ForwardModel
 * forward_with_cache(ids, cache, start_pos)).
 *   logits  [vocab]   f32, logits of the last position (nullable)
 *   argmax  [1]       int32, greedy token of the last position, lowest index
 *                     among equal maxima (nullable)
 *   hidden  [n,hidden] f32, final-RMSNorm'd states of every position (nullable)
 * Host errors: INVALID_ARG (n <= 0, seq out of range, null ids), CAPACITY
 * (start_pos + n > max_len or n > max_tokens).  Device status: STATE when
 * start_pos != the cursor, TOKEN for an id >= vocab. */
ember_status ember_prefill(ember_model *m, ember_kv *kv, int32_t seq, const int32_t *ids,
                           int32_t n, int32_t start_pos, float *logits, int32_t *argmax,
                           float *hidden, ember_stream_t stream);

/* One cached decode step for `batch` sequences: token ids[b] of sequence
 * seqs[b] at position positions[b] (ember reference_forward.py forward(tok,
 * pos)); afterwards the cursor of seqs[b] is positions[b] + 1.  All arrays are
 * device arrays of `batch` entries; the sequences must be distinct.
 * positions may be NULL: each token then goes at its sequence's cursor, so
 * repeated calls with the same buffers (argmax fed back as ids) replay one
 * CUDA graph.
 *   logits [batch, vocab] f32 (nullable); argmax [batch] int32 (nullable).
 * argmax may be the next call's ids, so a greedy loop needs no host sync.
 * Host errors: INVALID_ARG, CAPACITY (batch > max_tokens or > max_seqs).
 * Device status: STATE (position != cursor), CAPACITY (position >= max_len),
 * INVALID_ARG (seq out of range), TOKEN. */
ember_status ember_decode_step(ember_model *m, ember_kv *kv, int32_t batch, const int32_t *seqs,
                               const int32_t *ids, const int32_t *positions, float *logits,
                               int32_t *argmax, ember_stream_t stream);

/* One decode step exactly as ember_decode_step computes it, run for
 * profiling: each kernel starts only after the previous one has finished (no
 * programmatic launch overlap), with a CUDA event recorded on `stream` before
 * every launch and after the last; the sequence runs as a one-off CUDA graph
 * so that host launch latency leaves no gaps.  Waits for the stream.
 *   launch_us [cap]  device time of launch i (its event to the next event)
 *   names     [cap]  launch i's kernel name as the CUDA runtime reports it
 *                    (mangled; static strings owned by the runtime)
 *   n                the step's number of launches (may exceed cap; entries
 *                    i >= cap are not written)
 * The times are those of serialised launches (each kernel's weight loads no
 * longer overlap its predecessor), an upper bound on a launch's share of a
 * graph-replayed step.  Errors as ember_decode_step, plus INVALID_ARG for a
 * stream that is being captured or NULL trace buffers with cap > 0, and CUDA
 * when an event cannot be created or timed. */
ember_status ember_decode_step_traced(ember_model *m, ember_kv *kv, int32_t batch, const int32_t *seqs,
                                      const int32_t *ids, const int32_t *positions, float *logits,
                                      int32_t *argmax, ember_stream_t stream, float *launch_us,
                                      const char **names, int32_t cap, int32_t *n);

/* Bidirectional (or causal, per the config) forward of B independent
 * sequences of T tokens each, positions restarting at 0 per sequence, no KV
 * cache (PII-Tracer forward()).
 *   out    [B*T, n_labels] f32 label logits (n_labels > 0), or
 *          [B*T, vocab] f32 tied-head logits (n_labels == 0)   (nullable)
 *   hidden [B*T, hidden] f32 final-RMSNorm'd states              (nullable)
 * Host errors: INVALID_ARG, CAPACITY (B*T > max_tokens, T > max_positions). */
ember_status ember_encode(ember_model *m, const int32_t *ids, int32_t B, int32_t T, float *out,
                          float *hidden, ember_stream_t stream);

/* ember_prefill that also records, after every decoder block, the residual
 * stream at the last of the n positions ("ember internals" ForwardModel
 * forward_with_activations: hidden states after each transformer block at
 * the last token, the input of the probe mode).
 *   acts [layers, hidden] f32 (device, required); logits / argmax as in
 *   ember_prefill (nullable).  The cache and its cursor advance as in
 *   ember_prefill.  Errors as ember_prefill, plus INVALID_ARG for NULL acts. */
ember_status ember_prefill_activations(ember_model *m, ember_kv *kv, int32_t seq, const int32_t *ids,
                                       int32_t n, int32_t start_pos, float *acts, float *logits,
                                       int32_t *argmax, ember_stream_t stream);

/* The mean-pooled sensitivity head of the bidirectional encoder
 * (PII-Tracer-vLLM serving/reference_forward.py forward(): the mean over
 * positions of the final-normed states, times the head's weight, plus its
 * bias): out[b][j] = (1/T sum_t hidden[b*T + t]) . w[j] + bias[j].
 *   hidden [B*T, H] f32 (device): the `hidden` output of ember_encode
 *   w      [n_out, H] bf16 bits, bias [n_out] bf16 bits or NULL (device;
 *          the caller's, not copied)
 *   out    [B, n_out] f32 (device)
 * Each column's sum runs in position order.  H <= 12288.  Asynchronous on
 * `stream`.  Errors: INVALID_ARG, CUDA. */
ember_status ember_mean_pooled_head(const float *hidden, int32_t B, int32_t T, int32_t H,
                                    const uint16_t *w, const uint16_t *bias, int32_t n_out,
                                    float *out, ember_stream_t stream);

/* Synchronise the stream, read and clear the device status word.  Returns
 * the first device-side error raised since the last call, else EMBER_OK. */
ember_status ember_sync_status(ember_model *m, ember_stream_t stream);

const char *ember_last_error(void);

/* ---- token sampler ------------------------------------------------------- */

/* One token per row of logits, the five stages of "ember internals" §sampler
 * in order: (1) temperature -- x = logit / temperature when temperature > 0;
 * temperature <= 0 is greedy and returns the first maximal logit (NaN counts
 * as maximal); (2) top-k -- for 0 < top_k < V every x below the top_k-th
 * largest is masked (ties with it are kept; 0 or >= V: no-op); (3) top-p --
 * for 0 < top_p < 1 the x whose softmax probability lies below the smallest
 * probability of the shortest most-probable set holding more than top_p of
 * the mass are masked (otherwise no-op); (4) softmax over the survivors
 * (uniform when every logit is -inf); (5) the first index whose running sum
 * of probabilities, in index order, exceeds r[b] (the last maximal index
 * when rounding leaves r[b] above the total).
 *   logits [B, ldl] f32, the first V columns used      (device)
 *   r      [B] f32 draws in [0, 1), one per row         (device; unused and
 *                                                        nullable when greedy)
 *   out    [B] int32 token ids                          (device)
 * Arithmetic: the division of stage 1 is IEEE f32; stages 2-3 select by exact
 * comparisons of x; the masses of stages 3-5 are exp(x - max) in f32 rounded
 * to multiples of 2^-40 and summed exactly (64-bit integers), so a call is
 * deterministic and its decisions differ from exact arithmetic only for draws
 * (or top_p) within ~1e-6 of a boundary.  Asynchronous on `stream`; reads
 * nothing else and allocates nothing.  Errors: INVALID_ARG (NULL pointers,
 * B or V <= 0, ldl < V, top_k < 0, NaN temperature or top_p), CUDA. */
ember_status ember_sample(const float *logits, int32_t B, int32_t V, int32_t ldl, float temperature,
                          int32_t top_k, float top_p, const float *r, int32_t *out,
                          ember_stream_t stream);

/* Element types of the operators below. */
typedef enum ember_dtype { EMBER_F32 = 0, EMBER_BF16 = 1, EMBER_F16 = 2 } ember_dtype;

/* ---- log probabilities ---------------------------------------------------- */

/* What a row of logits l says of its tokens, with x = l / temperature and
 * log p_i = x_i - log sum_j exp(x_j) (ember reference_forward.py forward()'s
 * logits; "ember internals", softmax):
 *   logprob [n]       log p of ids[r]
 *   rank    [n]       how many tokens stand before it: larger logits, and equal
 *                     ones of a lower index (0: it is the greedy token)
 *   entropy [n]       -sum_i p_i log p_i
 *   top_ids, top_logprobs [n][top]  the first `top` tokens in that order and
 *                     their log p; top at most EMBER_LOGPROBS_MAX_TOP
 *   logits [n] rows of V elements of `dtype` (F32, BF16, F16), ldl elements apart,
 *   aligned to their elements; ids [n] int32.  logprob, rank and entropy may be
 *   NULL, ids too (logprob and rank must then be); top may be 0.
 * An id outside [0, V) gives logprob NaN and rank -1.  A logit of -inf has no
 * weight; a row of nothing else is uniform, as in ember_sample.  In a row with a
 * NaN or +inf every log probability and the entropy are NaN; NaN counts as the
 * largest logit.  The order is that of the logits themselves, whatever the
 * temperature (1e-6 to 1e6) rounds together.  For the entropy distances between
 * logits beyond 1e30 count as 1e30; a log probability beyond f32's range is -inf.
 * Arithmetic is f32; equal calls give equal bits.  Asynchronous on `stream`; allocates nothing.
 * Host errors: INVALID_ARG, UNSUPPORTED (top), CUDA. */
#define EMBER_LOGPROBS_MAX_TOP 32
ember_status ember_logprobs(const void *logits, int32_t dtype, int32_t n, int32_t V, int64_t ldl,
                            float temperature, const int32_t *ids, int32_t top, float *logprob,
                            int32_t *rank, float *entropy, int32_t *top_ids, float *top_logprobs,
                            ember_stream_t stream);

/* ---- projections with adapters -------------------------------------------- */

/* A projection that all rows share (ember reference_forward.py forward(): q = Wq x
 * and the others) with a low-rank adapter of each row's own beside it:
 *   out_i = W x_i + bias + s_a B_a (A_a x_i),   a = ids[i]   (negative: W x_i + bias)
 * for a batch whose rows belong to requests with different adapters, in any order.
 *   x    [n] rows of K elements of `dtype` (BF16 or F16), ld_x apart
 *   w    [N][K], bias [N] or NULL, of dtype;  ids [n] int32
 *   a    [n_adapters][rank][K], b [n_adapters][N][rank] of dtype, scale
 *        [n_adapters] f32 or NULL (1).  Adapters of a lower rank are filled up with
 *        zeros.  rank is a multiple of 8 up to 128; N and K are multiples of 8.
 *   out  [n] rows of N elements of out_dtype (dtype or F32), ld_out apart
 *   workspace: ember_adapter_workspace(n, rank) bytes, 16-byte aligned, of any
 *        content; used until the call's kernels end, so calls that may overlap need
 *        one each.
 *   status: as for the paged operators below; INVALID_ARG for an id >= n_adapters
 *        (the row then goes without adapter), RANGE for f16 where an element of
 *        s_a A_a x lies beyond the type's range (its row is then not finite), TIMEOUT.
 * Products are taken on the type and summed in f32 by the tensor cores, which cut off;
 * for f32 outputs at most 48 of their steps, whose sums are added rounded to nearest
 * (W x, and A_a x, off by 0.8e-6 of their norms at most, whatever n and K; sums all
 * rounded to nearest are by 0.3e-6 to 1e-6); s_a A_a x is held as the sum of two values of the type (2^-17 relative for bf16, 2^-22 or
 * 2^-25 absolute for f16).
 * Element pointers are 16-byte aligned, scale, ids and status 4-byte; row strides
 * multiples of 8 elements; buffers may not overlap.  Values of an x, a, b or scale
 * that are not finite reach the rows that read them and no others; outputs next to
 * such a b's are taken again one by one, which is slow (0.6 ms instead of 22 us for
 * 64 rows of 40 adapters of which one is infinite all over).  No
 * atomics on results: equal calls give equal bits.  Asynchronous on `stream`; no gradient.
 * Host errors: INVALID_ARG, UNSUPPORTED, CAPACITY (workspace), CUDA. */
typedef struct ember_adapters {
    const void *a, *b;
    const float *scale;
    int32_t n_adapters, rank;
} ember_adapters;
size_t ember_adapter_workspace(int32_t n, int32_t rank);
ember_status ember_adapter_project(const ember_adapters *ad, const void *x, int64_t ld_x,
                                   const void *w, const void *bias, int32_t dtype, int32_t n,
                                   int32_t N, int32_t K, const int32_t *ids, void *out,
                                   int32_t out_dtype, int64_t ld_out, void *workspace,
                                   size_t workspace_bytes, int32_t *status,
                                   ember_stream_t stream);

/* ---- paged key/value cache ------------------------------------------------ */

/* Four operators on one pool of K/V pages that many sequences share, for a
 * serving loop whose sequences grow, end and are replaced: new tokens' rows go
 * in with ember_paged_append, and ember_paged_decode, ember_paged_decode_shared
 * (for sequences that share a prefix) and ember_paged_prefill attend over them.  They are stateless like ember_sample: the pool, the page
 * table and every other buffer are the caller's, nothing is kept, and they
 * compose on one stream with any other call.  (The cache of ember_kv_alloc --
 * "ember internals", "kv cache" -- is one block of max_len rows per sequence;
 * the same operations on it are inside ember_prefill / ember_decode_step.)
 *
 * Common rules:
 *   - Row r of page p of kv head g starts at k + p*page_stride +
 *     g*head_stride + r*row_stride elements, the same for v, and holds
 *     head_dim elements; so pages may hold a head's rows together or a row's
 *     heads together.  Position i of sequence s lies in page
 *     table[s*table_width + i / page_size], row i % page_size.
 *   - head_dim is 16, 32, 64 or 128; page_size a power of two from 16 to 1024;
 *     n_heads / n_kv_heads at most 16; table_width * page_size at most 2^30;
 *     n_heads * head_dim (and n_kv_heads * head_dim) at most 2^20; in decode
 *     B * n_kv_heads * table_width * page_size at most 2^34.
 *   - All element pointers are 16-byte aligned, lse and pointers to int32
 *     4-byte; strides and row lengths (ld_*, in elements) are multiples of 8.
 *     q / out rows hold the heads side by side, head_dim apart.
 *   - seqs[i] < 0 marks a padding token or row: it is skipped and what it
 *     would write stays as it was.
 *   - Errors that depend on device data raise the first code into *status (a
 *     device int32 that the caller zeroes and reads; NULL: not reported):
 *     INVALID_ARG for a seqs entry >= n_seqs, a cu entry out of order or a page
 *     outside [0, n_pages); CAPACITY for a position or length outside
 *     [0, table_width*page_size] or, in append, beyond the RoPE table.  The token,
 *     or the sequence's rows, are then skipped; of a bad page met by attention
 *     the keys read as zeros.  Nothing outside the buffers is touched.
 *   - Table entries of pages that hold no visible key are not read, nor are
 *     rows of a page that no query of the call sees: they may hold anything.
 *   - Products are taken on the cache's type and summed in f32.  Softmax weights
 *     are taken against a maximum that may lag behind the true one, so that a
 *     row's weights sum to at most 2^9 for each of its keys (their number rounded
 *     up to 64) before the division: bf16 values stay below 3.4e38 / (2^9 (keys +
 *     63)) in magnitude, 1e32 at 5000 keys, 5e30 at 131072 (f16 always does).  A
 *     score whose products sum beyond f32 counts as infinite; one below -3e38 /
 *     log2(e) has no weight.
 *   - A weight's rounding for the second product: decode, and prefill of short
 *     sequences (tables of at most 128 keys, at most 64 rows a sequence on average)
 *     or with a scale that is not positive, take it as the sum of two values of the
 *     cache's type (2^-16 relative for bf16, 2^-22 for f16), other prefill as one
 *     (2^-8, 2^-11: about the output's own rounding); f16's is at least 2^-32 of the
 *     largest weight of its row.  decode_shared: two terms, as decode.
 *   - B is at most 65535.  No operator has a gradient.
 *   - Buffers and the stream belong to the current device; buffers may not
 *     overlap, except that pages may be shared by the tables of sequences
 *     that only read them.  What a call reads is not to be written by others
 *     until its kernels have ended (page rows that it does not see may be). */
typedef struct ember_paged_kv {
    void *k, *v;                 /* the pages, elements of `dtype`              */
    const int32_t *table;        /* [n_seqs][table_width] page numbers          */
    int32_t dtype;               /* EMBER_BF16 or EMBER_F16                     */
    int32_t n_pages, page_size;  /* pages of the pool, rows of a page           */
    int32_t n_kv_heads, head_dim;
    int32_t n_seqs, table_width;
    int64_t page_stride, head_stride, row_stride; /* elements                   */
} ember_paged_kv;

/* Append n tokens: token t of sequence seqs[t] at position positions[t].  Per
 * head, q and k are RMS-normed over head_dim (q_norm / k_norm, bf16 bits
 * [head_dim], NULL: not normed; PII-Tracer forward(): before RoPE), rotated by
 * row positions[t] of the f32 tables cos_t / sin_t [n_pos][head_dim/2] (ember
 * reference_forward.py rope(), rotate-half) and rounded once to the cache's
 * type; k and v go to their page row, q to q_out.  All arithmetic is f32; the
 * rotation is that of ember_rope_store, bit for bit.
 *   q [n] rows of n_heads*head_dim, k, v [n] rows of n_kv_heads*head_dim, of
 *   src_dtype (F32, BF16 or F16), ld_* apart; slices of one fused q|k|v buffer
 *   fit.  q and q_out may both be NULL (n_heads is then not used).
 *   q_out [n] rows of n_heads*head_dim elements of the cache's type.
 * The (sequence, position) pairs of a call must be distinct: of two tokens at
 * one place each 16-byte piece is one or the other's.
 * Host errors: INVALID_ARG, UNSUPPORTED, CUDA. */
ember_status ember_paged_append(const ember_paged_kv *kv, const void *q, const void *k,
                                const void *v, int32_t src_dtype, int64_t ld_q, int64_t ld_k,
                                int64_t ld_v, int32_t n, int32_t n_heads, const int32_t *seqs,
                                const int32_t *positions, const uint16_t *q_norm,
                                const uint16_t *k_norm, float eps, const float *cos_t,
                                const float *sin_t, int32_t n_pos, void *q_out, int64_t ld_out,
                                int32_t *status, ember_stream_t stream);

/* Attention of one token per sequence, its last: row b stands at position
 * lens[b] - 1 of sequence seqs[b] (NULL: sequence b) and sees key j when
 * j < lens[b] and, for window > 0, j >= lens[b] - window or j < sinks.
 *   out[b] = sum_j p_j v_j,  p = softmax over the visible j of scale q . k_j
 *   (ember reference_forward.py forward(), the grouped-query head loop)
 *   lse[b][h] = log sum_j exp(scale q . k_j)   (f32 [B][n_heads], nullable)
 * lens[b] == 0 gives out 0 and lse -inf.  q, out: [B] rows of
 * n_heads*head_dim elements of the cache's type.
 *   workspace: ember_paged_decode_workspace bytes (which may be 0: then NULL
 *   will do), 16-byte aligned, of any content; used until the call's kernels
 *   end, so calls that may overlap (other streams, graphs that run at once) need
 *   one each: sharing it makes their outputs wrong (nothing else is touched).
 * How the keys are split, and with it the rounding, depends on B, the head
 * counts, the window, lens, the table's width and the device; there are no
 * atomics, so equal calls give equal bits.
 * Host errors: INVALID_ARG, UNSUPPORTED, CAPACITY (workspace too small), CUDA. */
size_t ember_paged_decode_workspace(const ember_paged_kv *kv, int32_t B, int32_t n_heads);
ember_status ember_paged_decode(const ember_paged_kv *kv, const void *q, int64_t ld_q, int32_t B,
                                int32_t n_heads, const int32_t *seqs, const int32_t *lens,
                                int32_t window, int32_t sinks, float scale, void *out,
                                int64_t ld_out, float *lse, void *workspace,
                                size_t workspace_bytes, int32_t *status, ember_stream_t stream);

/* ember_paged_decode for groups of sequences that share a long prefix (a system
 * prompt, a document), held once: rows groups[i] .. groups[i+1] - 1 (device int32
 * [n_groups+1], groups[0] = 0, groups[n_groups] = B) find their keys j < shared[i] in
 * the pages of table row prefixes[i] and the others, up to lens[b], in their own
 * row's (seqs[b]).  shared [n_groups] is any number, whole pages or not, and may
 * exceed a row's lens[b]: beyond the longest of a group's, rows of padding among them,
 * its prefix may hold anything; entries of a row's own pages that hold only shared keys
 * are not read.  Every key is seen: there is no window.  What the rows of a group
 * read together is read once for all of them; n_groups is at most B.  Calls of few
 * keys (by the table's width), of fewer than three rows a group on average or with a
 * scale that is not positive read a row's keys for each row, with the same result up
 * to rounding.  As in prefill, a K or V value of a prefix that is not finite, and that
 * some row of a group sees, may make the whole group not finite.
 * A row outside every group, a prefixes entry outside [0, n_seqs) and a shared entry
 * outside [0, table_width*page_size] raise INVALID_ARG and CAPACITY, and the rows
 * are skipped.  All else as in ember_paged_decode, with
 * ember_paged_decode_shared_workspace bytes of workspace. */
size_t ember_paged_decode_shared_workspace(const ember_paged_kv *kv, int32_t B, int32_t n_heads,
                                           int32_t n_groups);
ember_status ember_paged_decode_shared(const ember_paged_kv *kv, const void *q, int64_t ld_q,
                                       int32_t B, int32_t n_heads, const int32_t *seqs,
                                       const int32_t *lens, const int32_t *groups,
                                       const int32_t *shared, const int32_t *prefixes,
                                       int32_t n_groups, float scale, void *out, int64_t ld_out,
                                       float *lse, void *workspace, size_t workspace_bytes,
                                       int32_t *status, ember_stream_t stream);

/* Attention of several tokens per sequence: rows cu[b] .. cu[b+1] - 1 of q
 * (device int32 [B+1], 0 <= cu[b] <= cu[b+1] <= n) are the last positions of
 * sequence seqs[b] (NULL: sequence b), which holds lens[b] keys with theirs: row
 * cu[b] + i stands at p = lens[b] - (cu[b+1] - cu[b]) + i and sees key j when
 * j <= p and, for window > 0, j > p - window or j < sinks.  A row with p < 0
 * gives out 0 and lse -inf; rows outside every sequence stay as they were.
 * out, lse [n][n_heads], window, sinks and scale as in ember_paged_decode.
 * A K or V value that is not finite makes not only the rows that see its key
 * but also others of their tile not finite, as a product with zero does.
 * Host errors: INVALID_ARG, UNSUPPORTED, CUDA. */
ember_status ember_paged_prefill(const ember_paged_kv *kv, const void *q, int64_t ld_q, int32_t n,
                                 int32_t B, int32_t n_heads, const int32_t *seqs,
                                 const int32_t *cu, const int32_t *lens, int32_t window,
                                 int32_t sinks, float scale, void *out, int64_t ld_out, float *lse,
                                 int32_t *status, ember_stream_t stream);

/* Takes the status word of the operators above: *taken = *status and *status = 0
 * (device int32s) in one atomic step on the stream, so that an error which a call on
 * another stream raises meanwhile is either taken or kept for the next time.
 * Host errors: INVALID_ARG (NULL or not 4-byte aligned), CUDA. */
ember_status ember_paged_take_status(int32_t *status, int32_t *taken, ember_stream_t stream);

/* ---- kernel-level entry points used by the parity tests ------------------ */

/* The RoPE-and-store step of the K cache write, alone: for each of n_tok rows
 * of n_heads*head_dim f32 values x (already q/k-normed where the model does
 * so), rotate-half by the f32 tables cos_t/sin_t [n_tok, head_dim/2] and
 * round to bf16 (nearest even) into out [n_tok, n_heads*head_dim].  It is the
 * same device code the fused cache write runs; every product and sum is
 * rounded separately, so identical f32 inputs give identical bits on any
 * correct f32 implementation (ember reference_forward.py rope()). */
ember_status ember_rope_store(const float *x, int32_t n_tok, int32_t n_heads, int32_t head_dim,
                              const float *cos_t, const float *sin_t, uint16_t *out,
                              ember_stream_t stream);

/* D[M,N] = A[M,K] . B[N,K]^T with bf16 A, B and f32 D (row-major, K
 * contiguous), on the tcgen05 tensor-core GEMM the projections use.  K and
 * the row strides must be multiples of 8 elements.  Errors: INVALID_ARG. */
ember_status ember_gemm_bf16(const uint16_t *A, const uint16_t *B, float *D, int32_t M,
                             int32_t N, int32_t K, ember_stream_t stream);

/* y[b][n] = sum_k W[n][k] * x[b][k] for b < nb (nb <= 8), on the split GEMV
 * the batch-1..8 decode projections run (W bf16 [N][K], x and y f32, row
 * strides K and N; K a multiple of 8, K <= 16384).  The projections of
 * ember reference_forward.py forward() (q = Wq xb, ...) without their fused
 * prologue / epilogue.  Errors: INVALID_ARG. */
ember_status ember_gemv_bf16(const uint16_t *W, int32_t N, int32_t K, const float *x, int32_t nb,
                             float *y, ember_stream_t stream);

/* q8_0 block quantization (ember internals, q8_0 block format; the encoder
 * the pages leave implicit, read as: per block of 32 values amax = max |w|,
 * codes = w / (amax / 127) in f32 rounded to the nearest integer, ties to
 * even, clamped to [-127, 127], zero for a zero block; scale = amax / 127
 * rounded to f16, nearest even) of n bf16 values w (n a positive multiple of
 * 32).  Writes the int8 codes q[n] and the f16 scales d[n/32] (bit patterns):
 * the planar form of the pages' 34-byte blocks (scale, then 32 codes), which
 * this library keeps as two arrays so that the codes stay 8-byte aligned.
 * It is the quantizer ember_model_create runs for weights_q8.  All pointers
 * are device pointers owned by the caller.  Errors: INVALID_ARG. */
ember_status ember_q8_0_quantize(const uint16_t *w, int64_t n, int8_t *q, uint16_t *d,
                                 ember_stream_t stream);

/* y[b][n] = sum_k (q[n][k] * d[n][k/32]) * x[b][k] for b < nb (nb <= 8): the
 * split GEMV of ember_gemv_bf16 reading q8_0 weights (codes q int8 [N][K],
 * f16 scales d [N][K/32] as ember_q8_0_quantize writes them), the decode
 * projections of a weights_q8 model.  K a multiple of 32, K <= 16384; q
 * 8-byte and x 16-byte aligned.  Errors: INVALID_ARG. */
ember_status ember_gemv_q8_0(const int8_t *q, const uint16_t *d, int32_t N, int32_t K,
                             const float *x, int32_t nb, float *y, ember_stream_t stream);

/* ---- greedy LM head with no allocation ----------------------------------- */

/* The method this library implements has no counterpart to this entry point;
 * it serves callers that may not allocate device memory at all -- a serving
 * loop whose HBM is already handed out (to a KV pool, say), or a latency path
 * that cannot take the device-wide stall a cudaMalloc / cudaFree can cause.
 *
 * argmax[b] = the first index n of the largest y[b][n] = sum_k W[n][k] x[b][k]
 * for b < nb: the split GEMV of ember_gemv_bf16 (same arguments, same
 * arithmetic, bf16 W [N][K], f32 x [nb][K]; K a multiple of 8, K <= 16384, W
 * and x 16-byte aligned) with its argmax epilogue, the greedy step of the tied
 * LM head.  y (f32 [nb][N]) receives the logits when non-NULL.  argmax is a
 * device int32 [nb].  All pointers are the caller's; nothing is kept.
 *
 * Scratch: the per-row argmax keys sit in a fixed device array inside the
 * library (EMBER_NOALLOC_MAX_ROWS u64 keys, 64 bytes per device); no call
 * allocates, frees or calls an allocating library routine.  The keys must be
 * zero when a call starts: the set-up clears them once and each call clears
 * them again after use, in its second kernel.
 *
 * Set-up: the first call on each device (with that device current) resolves
 * the array's address and clears it on the given stream.  Make that first
 * call before any stream capture begins on the device.
 *
 * Concurrency: every call on one device shares that one array.  Two calls
 * whose kernels may overlap (different streams without an ordering between
 * them, or different host threads) race on it and may return wrong indices:
 * order them on one stream or with events.
 *
 * Errors: CAPACITY when nb > EMBER_NOALLOC_MAX_ROWS; INVALID_ARG for NULL or
 * misaligned pointers and bad sizes; UNSUPPORTED for device ordinals >= 64;
 * CUDA for a failed set-up or launch.  Returns once the two kernels are
 * queued on `stream`. */
#define EMBER_NOALLOC_MAX_ROWS 8
ember_status ember_gemv_argmax_noalloc(const uint16_t *W, int32_t N, int32_t K, const float *x,
                                       int32_t nb, float *y, int32_t *argmax,
                                       ember_stream_t stream);

/* Test-only (failure detection): runs one of the library's bounded device
 * waits -- which = 0 the shared-memory mbarrier wait of the TMA / tensor-core
 * kernels, 1 the cluster-scope wait of the fused batch-1 decode -- on an
 * mbarrier that nothing completes, with a budget of budget_cycles SM cycles
 * (<= 2e8) instead of the kernels' ~1 s.  The wait gives up and the kernel
 * raises EMBER_ERR_TIMEOUT in m's status word, which the next
 * ember_sync_status returns (and clears); nothing else is touched.  The
 * method this library implements has no counterpart to it. */
ember_status ember_test_bounded_wait(ember_model *m, int32_t which, int64_t budget_cycles,
                                     ember_stream_t stream);

/* Number of kernels this library has launched in this process so far (a
 * CUDA-graph replay counts each kernel node it runs).  For accounting. */
uint64_t ember_kernel_launches(void);

#ifdef __cplusplus
}
#endif
#endif /* EMBER_H */
