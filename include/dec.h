/*
 * dec.h -- C ABI of the GB300 persistent MoE decode engine.
 *
 * One call of dec_step runs a whole decode step (every layer, the LM head and the greedy
 * argmax) as ONE launch of one persistent, warp-specialised kernel, instead of a chain of
 * per-operator kernels. This is the execution model described on the page "Ultra-High
 * Interactivity on NVIDIA GPUs? TileRT on InferenceX", section "But What Exactly is TileRT?"
 * (the host launches once, warp groups specialise on data movement and compute, stages overlap
 * at tile granularity and intermediates stay in registers, shared memory and L2), applied to the
 * per-layer decode recipe of "vLLM's Kimi K3 Backend Hits 842 Tokens per Second", section "Four
 * changes drive the gains" (shape-aware small-N GEMV, split-K at larger batches, the shared
 * expert overlapped with routing, weight prefetch ahead of use).
 *
 * Conventions for every entry point:
 *  - Pointers marked "device" are CUDA device pointers; "host" pointers are CPU memory.
 *  - bf16 tensors are passed as 16-bit bit patterns (any type with that layout).
 *  - FP8 matrices are OCP E4M3 codes, row-major [rows][cols], with fp32 block scales
 *    [ceil(rows/128)][ceil(cols/128)]; element (r, c) means scale[r/128][c/128] * e4m3(W[r][c]).
 *  - A `stream` argument is a cudaStream_t; NULL means the engine's own (non-blocking) stream,
 *    so the legacy default stream must be passed as cudaStreamLegacy. Consecutive steps of one
 *    engine share its counters, exchange buffers and KV cache, so they must not overlap: when a
 *    call queues work on a different stream than the engine's previous work, the library makes
 *    the new stream wait for the old one (an event), so calls of one engine run in call order
 *    whatever streams they are given. Work of other engines and other libraries is never waited
 *    for: no entry point synchronises the whole device.
 *    Calls without a `stream` argument run on the engine's own stream: what the caller has queued
 *    elsewhere on their buffers has to be done before (the Python wrapper waits for it).
 *  - Entry points that queue device work require the engine's device to be the current CUDA
 *    device (DEC_ERR_ARG otherwise).
 *  - Every call returns a dec_status. Errors found on the device (a wait that ran out of time,
 *    a failed bounds check) are reported by the next call that synchronises (dec_sync,
 *    dec_generate, dec_prefill_kv, dec_export_kv) and POISON the engine: later calls return
 *    DEC_ERR_POISONED. dec_last_error() gives a human-readable reason.
 *  - No call falls back to a CPU path: shapes the kernel does not handle give
 *    DEC_ERR_UNSUPPORTED.
 *  - The engine is not thread-safe; use one engine per host thread.
 */
#ifndef DEC_H
#define DEC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct dec_engine dec_engine; /* opaque, owned by the library */

typedef enum {
  DEC_OK = 0,
  DEC_ERR_ARG = -1,         /* bad argument (NULL, out of range, batch > max_batch, ...) */
  DEC_ERR_CUDA = -2,        /* a CUDA runtime call failed */
  DEC_ERR_OOM = -3,         /* device allocation failed */
  DEC_ERR_TIMEOUT = -4,     /* a device-side wait ran out of time; engine poisoned */
  DEC_ERR_UNSUPPORTED = -5, /* model shape or batch the kernel does not implement */
  DEC_ERR_POISONED = -6,    /* an earlier device error made the engine unusable */
  DEC_ERR_DEVICE = -7,      /* a device-side consistency check failed; engine poisoned */
  DEC_ERR_CAPACITY = -8     /* a sequence would exceed max_ctx */
} dec_status;

/* Model shape. The layer is a pre-norm decoder: RMSNorm -> q/k/v projection -> RoPE (half-split
   pairing) -> GQA attention over a bf16 KV cache -> output projection + residual -> RMSNorm ->
   FFN + residual. The FFN is either a dense SwiGLU of width dense_ffn (n_experts == 0), or a
   sigmoid-routed MoE: top_k of n_experts SwiGLU experts of width moe_inter with gates normalised
   over the selected scores, plus n_shared (0 or 1) always-on experts of the same width.
   ("Kimi K3: The Manos, The Mythos, The Legendos": GQA; the expert as SwiGLU; top-k over router
   scores; the residual x_{l+1} = x_l + f(x_l).) vocab == 0 builds a headless stack that maps a
   bf16 hidden state to a bf16 hidden state (no embedding, LM head or argmax). */
typedef struct {
  int32_t n_layers;   /* >= 1 */
  int32_t hidden;     /* multiple of 128 */
  int32_t n_heads;    /* query heads */
  int32_t n_kv_heads; /* KV heads; n_heads / n_kv_heads must be 2 or 4 */
  int32_t head_dim;   /* 64 or 128 */
  int32_t n_experts;  /* 0 for a dense FFN, else <= 128 */
  int32_t top_k;      /* 1..16, <= n_experts */
  int32_t moe_inter;  /* expert SwiGLU width, multiple of 128 */
  int32_t n_shared;   /* 0 or 1 */
  int32_t dense_ffn;  /* dense SwiGLU width (multiple of 128) when n_experts == 0, else 0 */
  int32_t vocab;      /* 0: headless stack */
  int32_t max_ctx;    /* KV positions per sequence */
  int32_t max_batch;  /* sequences decoded together, 1..64 (8 and more: the wide kernels) */
  float rms_eps;
  float rope_theta;
} dec_model_cfg;

/* An FP8-E4M3 matrix with its fp32 block scales (both device pointers, borrowed). */
typedef struct {
  const void* w;
  const float* scale;
} dec_fp8_mat;

/* One layer's weights. Matrix shapes (rows x cols): wq [n_heads*head_dim x hidden],
   wk/wv [n_kv_heads*head_dim x hidden], wo [hidden x n_heads*head_dim],
   router [n_experts x hidden], gate/up [inter x hidden], down [hidden x inter].
   The expert and shared arrays are HOST arrays of device matrices. */
typedef struct {
  const void* attn_norm; /* device bf16 [hidden] */
  dec_fp8_mat wq, wk, wv, wo;
  const void* ffn_norm; /* device bf16 [hidden] */
  dec_fp8_mat router;
  const dec_fp8_mat* expert_gate; /* host array [n_experts] */
  const dec_fp8_mat* expert_up;
  const dec_fp8_mat* expert_down;
  const dec_fp8_mat* shared_gate; /* host array [n_shared] */
  const dec_fp8_mat* shared_up;
  const dec_fp8_mat* shared_down;
  dec_fp8_mat ffn_gate, ffn_up, ffn_down; /* dense FFN */
} dec_layer_weights;

typedef struct {
  const void* embed;      /* device bf16 [vocab][hidden] (vocab > 0) */
  const void* final_norm; /* device bf16 [hidden] (vocab > 0) */
  dec_fp8_mat lm_head;    /* [vocab x hidden] (vocab > 0) */
  const dec_layer_weights* layers; /* host array [n_layers] */
} dec_weights;

/* Host-only check of a model shape (no CUDA needed). DEC_OK, DEC_ERR_ARG (inconsistent) or
   DEC_ERR_UNSUPPORTED (consistent but not implemented by the kernel). */
dec_status dec_validate_cfg(const dec_model_cfg* cfg);

/* Build an engine on the current CUDA device: validates the shape, copies every weight into
   library-owned memory (repacked into the kernel's tile order; the caller may free its buffers
   once the call returns), builds the RoPE table (angles in double on the host), allocates the
   KV cache [n_layers][max_batch][n_kv_heads][max_ctx][head_dim] bf16 x2 and the workspace, and
   checks that one CTA per SM can be co-resident. An engine of max_batch >= 5 also builds the
   wide kernel's buffers and two tensor maps over the K and V caches (the driver's
   cuTensorMapEncodeTiled, reached through the runtime; DEC_ERR_CUDA if it is missing). All
   sequence lengths start at 0. Work is queued on `stream` and synchronised before return. *out
   receives the engine (NULL on failure).
   Environment, read here: DEC_TIMEOUT_MS bounds every device-side wait (default 1000);
   DEC_INFLIGHT / DEC_WIDE_INFLIGHT set how many ring slots one CTA keeps in flight (defaults 2
   and 4; tuning only); DEC_WIDE_MIN_BATCH (2..9, default 5) is the smallest decode batch that
   runs the wide kernel (tuning and tests);
   DEC_TEST_SKIP_ARRIVAL=1 (tests of the failure path only) makes the CTA holding the first
   q/k/v tile withhold that partial sum's arrival in layer 0 (in a step of 5 tokens or more:
   CTA 0 its arrival at the first grid barrier), so the waits for it run out after
   DEC_TIMEOUT_MS and the step ends with DEC_ERR_TIMEOUT instead of hanging;
   DEC_EPOCH_LIMIT lowers the number of steps after which a step first zeroes the engine's
   cross-step counters and flags (a cudaMemsetAsync on the step's stream) and restarts its epoch
   (default 2^30 / the largest number of k blocks of a row block), so tests can make it happen. */
dec_status dec_init(const dec_model_cfg* cfg, const dec_weights* weights, void* stream,
                    dec_engine** out);

/* Fill the KV cache of sequence slots [seq, seq + n_seq).
   Token mode (k_import == NULL): token_ids is device int32 [n_seq][n_tokens]; appending to each
   slot's current length, the engine runs the decode kernel over the prompt and discards the
   logits: for one slot (n_seq == 1) in launches of up to DEC_MAX_STEP_TOKENS consecutive
   positions each (as dec_step_positions: every launch streams the weights once for all of its
   positions), for several slots one launch per position with the slots side by side. This is
   decode-engine prefill as on the pages' prefill/decode split, not a compute-bound prefill
   engine.
   Import mode (k_import != NULL): copies an external KV state, device bf16
   [n_layers][n_kv_heads][n_tokens][head_dim] for K (post-RoPE) and V, into positions
   0..n_tokens of every slot in the range and sets their length to n_tokens (the handoff of a KV
   cache produced elsewhere, as in the TileRT page's section "PD Disaggregated Engine with vLLM
   and TileRT"). n_tokens == 0 is a no-op in both modes. Synchronises. */
typedef struct {
  int32_t seq;
  int32_t n_seq;
  const int32_t* token_ids; /* device, token mode */
  int32_t n_tokens;
  const void* k_import; /* device, import mode */
  const void* v_import;
} dec_ctx;
dec_status dec_prefill_kv(dec_engine* eng, const dec_ctx* ctx);

/* Token-mode prefill that allocates no device memory. The pages have no counterpart: this is a
   property of the library boundary, not of the method. dec_prefill_kv's token mode stages the
   step-major token ids in a buffer it takes with cudaMalloc and returns with cudaFree; a caller
   that may not allocate device memory while serving (a framework whose caching allocator holds
   the device's free memory, or a loop in which cudaFree's implicit device-wide synchronisation
   would stall other streams) calls this instead. The ids are staged in a file-scope device
   array of DEC_NOALLOC_PREFILL_MAX_IDS int32 (256 KiB), one per device.
   - ctx must be token mode (k_import and v_import NULL); anything else is DEC_ERR_ARG.
   - n_seq * n_tokens > DEC_NOALLOC_PREFILL_MAX_IDS returns DEC_ERR_ARG, with the sizes in
     dec_last_error(), before any work is queued; split longer prompts into several calls.
   - The first call on a device does a one-time setup: with that device current it looks up the
     array's device address (cudaGetSymbolAddress) and caches it. Make that first call before
     any stream capture begins.
   - Nothing needs to start at zero: a call writes every id it reads before reading it.
   - The array is shared by all engines on a device: overlapping calls (two host threads, or two
     engines on one device) race on it; the caller must serialise them. Within one engine the
     call is stream-ordered after the engine's earlier work (no device-wide synchronisation).
   - The engine's device must be the current device (DEC_ERR_ARG otherwise).
   Results, capacity checks and synchronisation are those of dec_prefill_kv's token mode. */
#define DEC_NOALLOC_PREFILL_MAX_IDS 65536
dec_status dec_prefill_kv_noalloc(dec_engine* eng, const dec_ctx* ctx);

/* One decode step of `batch` sequences in slots [seq0, seq0 + batch). Token b is written at
   position length[seq0 + b] and attends over positions 0..length (inclusive); the lengths grow
   by one. Exactly one kernel launch on `stream`; nothing is synchronised.
     tokens      device int32 [batch]         input ids (vocab > 0)
     hidden_in   device bf16 [batch][hidden]  input hidden states (vocab == 0; also accepted
                                              with vocab > 0 in place of tokens)
     logits      device fp32 [batch][vocab]   caller-owned output, may be NULL
     next_tokens device int32 [batch]         greedy argmax (lowest id on ties), may be NULL
     hidden_out  device bf16 [batch][hidden]  final residual stream (before the final norm),
                                              may be NULL
   batch == 0 is a no-op. Errors: DEC_ERR_ARG, DEC_ERR_CAPACITY (a length would pass max_ctx),
   DEC_ERR_POISONED, DEC_ERR_CUDA (launch failure).
   Batches of 5 .. 64 (engines built with max_batch >= 5) run the wide kernel: every GEMV on the
   tensor cores with all of the step's tokens as the N dimension, tokens grouped per routed expert
   (an expert's products kept for the tokens routed to it), attention as bf16 tensor-core products
   on KV tiles loaded by tensor-map copies, phases separated by grid barriers
   ("vLLM's Kimi K3 Backend Hits 842 Tokens per Second", section "A narrow deployment lane":
   decode batches up to 64). Same arguments, results and errors. */
typedef struct {
  const int32_t* tokens;
  const void* hidden_in;
  int32_t batch;
  int32_t seq0;
  float* logits;
  int32_t* next_tokens;
  void* hidden_out;
  void* stream;
} dec_step_args;
dec_status dec_step_ex(dec_engine* eng, const dec_step_args* args);

/* The most tokens one launch takes (sequences side by side, or positions of one sequence). */
#define DEC_MAX_STEP_TOKENS 8

/* Several consecutive positions of ONE sequence in one launch ("vLLM's Kimi K3 Backend Hits 842
   Tokens per Second", section "Throughput holds across the tested range": verifying speculative
   drafts; also chunked prefill). tokens is device int32 [n], 1 <= n <= DEC_MAX_STEP_TOKENS;
   token j is written at position length[seq] + j and attends over positions 0 .. length + j
   (causal: the keys and values of the earlier tokens of the same launch included); the slot's
   length grows by n. logits device fp32 [n][vocab] and next_tokens device int32 [n] (the argmax
   after each position) are optional. One launch on `stream`; nothing is synchronised.
   Requires vocab > 0. Errors: DEC_ERR_ARG, DEC_ERR_CAPACITY, DEC_ERR_POISONED, DEC_ERR_CUDA. */
dec_status dec_step_positions(dec_engine* eng, int32_t seq, const int32_t* tokens, int32_t n,
                              float* logits, int32_t* next_tokens, void* stream);

/* Speculative-decoding verify step: as dec_step_positions with tokens = [t0, d1, .., d(n-1)], t0
   the sequence's next input token and d the draft. The kernel accepts draft d(j+1) while it equals
   the argmax after position length + j, writes the accepted count m (0 <= m < n) to the host
   int *n_accepted, and keeps the positions length .. length + m in the cache: the slot's length
   becomes length + m + 1, and next_tokens[m] (if given) is the next input token. Synchronises
   with `stream` (the caller needs m to go on). */
dec_status dec_verify(dec_engine* eng, int32_t seq, const int32_t* tokens, int32_t n, float* logits,
                      int32_t* next_tokens, int32_t* n_accepted, void* stream);

/* The plain form: slots [0, batch), token input, logits/next_tokens outputs (may be NULL). */
dec_status dec_step(dec_engine* eng, const int32_t* token_ids, int32_t batch, float* logits,
                    int32_t* next_tokens, void* stream);

/* Greedy generation from HOST buffers: copies first_tokens (host int32 [batch]) to the device,
   runs n_steps greedy decode steps of slots [0, batch) in ONE launch of a resident kernel ("Ultra-
   High Interactivity on NVIDIA GPUs? TileRT on InferenceX", section "But What Exactly is
   TileRT?": the host launches once and execution stays on the GPU for the decode lifecycle):
   step i's argmax becomes step i+1's input through device memory and a flag, and the producer
   warps stream the next step's first weights while the LM head finishes. Copies the generated
   tokens back to out_tokens (host int32 [n_steps][batch]) and synchronises. Requires vocab > 0
   and length + n_steps <= max_ctx for every slot (DEC_ERR_CAPACITY otherwise). (A generation of
   more steps than the engine's epoch period takes one launch per period; batches of 5 and more
   take one wide-kernel launch per step, the tokens still chained on the device.) */
dec_status dec_generate(dec_engine* eng, const int32_t* first_tokens, int32_t batch,
                        int32_t n_steps, int32_t* out_tokens, void* stream);

/* The same resident generation with DEVICE buffers (first_tokens device int32 [batch],
   out_tokens device int32 [n_steps][batch]); queued on `stream`, nothing synchronised. */
dec_status dec_generate_device(dec_engine* eng, const int32_t* first_tokens, int32_t batch,
                               int32_t n_steps, int32_t* out_tokens, void* stream);

/* Sequence lengths (positions already in the cache). Setting a length rewinds or advances a
   slot without touching the cache contents. */
dec_status dec_set_length(dec_engine* eng, int32_t seq, int32_t length);
dec_status dec_get_length(dec_engine* eng, int32_t seq, int32_t* length);

/* Copy positions [pos0, pos0 + n) of one slot and layer out of the KV cache into device bf16
   buffers k_out/v_out [n_kv_heads][n][head_dim]. Synchronises. */
dec_status dec_export_kv(dec_engine* eng, int32_t seq, int32_t layer, int32_t pos0, int32_t n,
                         void* k_out, void* v_out);

/* Wait for all queued engine work and read the device status word. */
dec_status dec_sync(dec_engine* eng);

/* Engine facts for tools and benchmarks. */
typedef struct {
  int32_t grid;           /* persistent CTAs (one per SM) */
  int32_t threads;        /* threads per CTA */
  int32_t smem_bytes;     /* dynamic shared memory per CTA */
  int32_t ring_slots;     /* stages of the shared-memory weight ring */
  int32_t stages_per_layer;
  int64_t weight_bytes;   /* repacked weight bytes held by the engine */
  int64_t kv_bytes;       /* KV cache bytes */
  int64_t workspace_bytes;
  int64_t launches;       /* kernel launches issued by this engine so far */
  int32_t wide_min_batch; /* decode steps of at least this many tokens run the wide kernel
                             (a value above max_batch: none does) */
} dec_info;
dec_status dec_get_info(dec_engine* eng, dec_info* out);

/* Routing of the most recent step at one layer (MoE models): copies the selected experts
   (score-descending) into host idx [R][top_k] and their normalised gates into host gates
   [R][top_k], R = max(DEC_MAX_STEP_TOKENS, max_batch), one row per token of the step; rows >=
   the step's token count are stale. Synchronises. */
dec_status dec_get_routing(dec_engine* eng, int32_t layer, int32_t* idx, float* gates);

/* The router logits (fp32, before the sigmoid) the most recent step selected from at one layer
   (MoE models): host logits [R][n_experts], R = max(DEC_MAX_STEP_TOKENS, max_batch); rows >=
   the step's token count are stale. With
   dec_get_routing this lets a caller check that a selection is the top_k of its own logits
   (ties to the lower expert index). Synchronises. */
dec_status dec_get_router_logits(dec_engine* eng, int32_t layer, float* logits);

/* Diagnostics of the last step, recorded only by a library built with DEC_TRACE=1 /
   DEC_STAMPS=1 (`DEC_DIAG=1` when running latency_moe_decode_gb300/build.py; the default build
   records nothing, its words stay zero: the stores cost the step ~4% in instruction fetch).
   Per-step trace written by CTA 0: (event code, %globaltimer ns) pairs in host_buf[2i], [2i+1].
   code = what << 4 | event; what: 0 q/k/v GEMV, 1 output projection, 2 router, 3 shared-expert
   (or dense FFN) gate/up, 4 routed gate/up, 5 down projections, 6 LM head, 7 attention, 8 grid
   barrier, 9 routing wait, 10 step; event: 0 begin, 1 last tile consumed, 2 finalisers done
   (barrier: its site). Words [512 - 128, 512) hold CTA 0's producer trace in the same format.
   With DEC_STAMPS=1, words from 512 on hold per-CTA %globaltimer stamps of the first 8 layers:
   word
   512 + (layer * 16 + point) * grid + cta, for the points q/k/v tiles consumed (0), q/k/v done
   (1), attention merged (2), attention outputs ready (3), output-projection tiles consumed (4)
   and done (5), x_mid ready (6), router partials published (7), routing known (8), gate/up
   tiles consumed (9) and done (10), SwiGLU rows ready (11), down tiles consumed (12) and done
   (13), layer barrier passed (14). Copies up to n words and returns the count in *n_written.
   Synchronises. */
dec_status dec_get_trace(dec_engine* eng, uint64_t* host_buf, int32_t n, int32_t* n_written);

/* Per-layer timing of the most recent step, recorded in every build by one thread of the first
   CTA: host_buf[l] is the %globaltimer time (ns) at which the input of layer l was final, as
   that CTA saw it (l = 0: the step start; l = n_layers: the final norm's input), and
   host_buf[n_layers + 1] the time that CTA finished the step. So host_buf[l + 1] - host_buf[l]
   is layer l's time on the critical path and the last difference the LM head's tail (in a step over 4-bit
   caches the launches between included). Copies
   min(n, n_layers + 2) words and returns the count in *n_written. Synchronises with the
   engine's work. */
dec_status dec_get_layer_times(dec_engine* eng, uint64_t* host_buf, int32_t n, int32_t* n_written);

/* Reason for the last failing call on this engine ("" if none). Valid until the next call. */
const char* dec_last_error(const dec_engine* eng);

/* Fixed string naming a status code. */
const char* dec_status_string(dec_status s);

/* Release every device buffer of the engine (synchronises first). NULL is a no-op. */
void dec_destroy(dec_engine* eng);

/* ------------------------------------------------------------------------------------------
   Operators beside the engine: a paged KV cache held in 4 bits, attention over it (for trees of drafted
   tokens too), what keeps it within a bound, log-probabilities, and the verification of drafts. They keep no state of
   their own: the caller owns every buffer. Unlike the engine's entry points they take no engine, so:
    - stream == NULL is the legacy default stream; work is queued on `stream`, nothing is
      synchronised, no call allocates device memory, and every call may be captured into a graph;
    - the buffers must live on the current CUDA device (DEC_ERR_ARG when the cache's or the
      logits' buffer does not);
    - the reason of a failing call is dec_op_error(), one per host thread;
    - calls that share no buffer they write may run at the same time on several streams. Calls
      sharing a workspace, a status word's meaning or pages they write must be ordered by the
      caller. */

/* Reason for the last failing operator call of this host thread ("" if none). */
const char* dec_op_error(void);

/* A paged KV cache of one layer. pages is n_pages consecutive pages of dec_kvq_page_bytes()
   bytes, 16-byte aligned; their content is the library's, and no page has to be initialised
   before it is appended to. A page holds page_tokens positions of every KV head. Each run of 16
   consecutive values x of a (position, KV head) row is kept as one scale s and 16 codes c:
   s = max|x| / 7 rounded to nearest even among the values with 3 mantissa and 5 exponent bits
   (steps of 2^-14 below 2^-11, at most 480), c = x / s rounded to nearest even and clamped to
   -8 .. 7 (0 where s = 0), the value held is c * s, which bf16 represents exactly. A run with an
   infinity or NaN is held as NaNs.
   status (device int32, may be NULL; zero it once) receives DEC_ERR_ARG when a kernel meets a
   page id outside 0 .. n_pages - 1 or a negative position, and DEC_ERR_CAPACITY when a position
   lies beyond the page table or the rotation table (the first one met stays), and DEC_ERR_TIMEOUT
   if a kernel gave up waiting for its own copies. The kernel skips such a row or such positions
   and touches nothing out of range (an append whose page is bad still gives the row's queries). */
typedef struct {
  void* pages;
  int32_t n_pages;
  int32_t page_tokens; /* 16, 32, 64, 128 or 256 */
  int32_t n_kv_heads;  /* 1 .. 1024 */
  int32_t head_dim;    /* 64 or 128 */
  int32_t* status;
} dec_kvq_cache;

/* The sequences of a call. Token rows are numbered 0 .. n_tokens - 1; sequence b's are
   cu_tokens[b] .. cu_tokens[b + 1] - 1 (device int32 [batch + 1]; NULL: one row per sequence and
   n_tokens == batch). Its row j stands at position lengths[b] + j (device int32 [batch]), and
   position p is in page table[b * table_stride + p / page_tokens] (device int32; max_pages
   entries of each row are valid). cu_tokens must ascend (where they do not, the attention records
   DEC_ERR_ARG and computes none of the up to 256 neighbouring sequences of a launch). Rows before
   cu_tokens[0] or from cu_tokens[batch] on belong to no sequence: outputs leave them as they were. */
typedef struct {
  int32_t batch;
  int32_t n_tokens;
  const int32_t* cu_tokens;
  const int32_t* lengths;
  const int32_t* table;
  int32_t max_pages;
  int64_t table_stride;
} dec_kvq_seqs;

typedef enum { DEC_BF16 = 0, DEC_F32 = 1 } dec_dtype;

/* Rows of heads: element (row, head, d) at p[row * token_stride + head * head_stride + d]; p
   16-byte aligned, strides multiples of 16 bytes. */
typedef struct {
  void* p;
  int64_t token_stride;
  int64_t head_stride;
} dec_rows;

/* Bytes of one page (0 for a shape the cache does not have). */
int64_t dec_kvq_page_bytes(int32_t page_tokens, int32_t n_kv_heads, int32_t head_dim);

/* Append the call's keys and values to the cache, in one pass with the per-head RMSNorm and the
   rotation of queries and keys:
     q, k, v    rows of n_heads, n_kv_heads, n_kv_heads heads of `dtype` (q.p NULL: none)
     q_norm, k_norm  device bf16 [head_dim], NULL: no norm. x -> x / sqrt(mean(x^2) + eps) * w
     rope       device fp32 [rope_len][rotary_dim / 2][2]: cos, sin of position p's angles; NULL
                (rotary_dim 0): no rotation. The first rotary_dim (a multiple of 16) values of a
                head are rotated: pair i is (i, i + rotary_dim / 2), or with interleaved != 0
                (2i, 2i + 1): (a, b) -> (a cos - b sin, a sin + b cos)
     q_out      bf16 rows (may be q.p itself when that is bf16 with the same strides)
   Everything is computed in fp32 and rounded once, to bf16 or to the cache's codes; keys whose fp32
   value lies within five standard deviations of its roundings of the border between two codes or scales are
   computed again with twice the bits (so a code beside the formula's is not excluded, but would take
   roundings that all but agree). Inputs above 1e18 overflow the norm's squares. The same position must not be
   appended twice in one call. */
typedef struct {
  dec_dtype dtype;
  int32_t n_heads;
  dec_rows q, k, v, q_out;
  const void* q_norm;
  const void* k_norm;
  float eps;
  const float* rope;
  int32_t rope_len;
  int32_t rotary_dim;
  int32_t interleaved;
  const int32_t* positions; /* device [n_tokens], may be NULL: the rotary position of each row, where that is not
                               where the row stands in the cache (a token of a tree, a sequence that gave positions
                               up). A negative one is DEC_ERR_ARG, one beyond the rotation table DEC_ERR_CAPACITY, in
                               status; the row is skipped */
} dec_kvq_append_args;
dec_status dec_kvq_append(const dec_kvq_cache* cache, const dec_kvq_seqs* seqs, const dec_kvq_append_args* args,
                          void* stream);

/* Read positions back: row j of sequence b receives position lengths[b] + j as bf16 (exact). */
dec_status dec_kvq_gather(const dec_kvq_cache* cache, const dec_kvq_seqs* seqs, const dec_rows* k_out,
                          const dec_rows* v_out, void* stream);

/* Attention over the cache. Row j of sequence b attends to positions 0 .. lengths[b] + j (causal:
   its own included, as dec_kvq_append of the same sequences has written it) or 0 ..
   lengths[b] - 1 (causal == 0: a stored prefix; lse lets the caller join it with attention over
   other keys). Query head h reads KV head h / (n_heads / n_kv_heads).
     q, out     bf16 rows of n_heads heads (out may be q)
     lse        device fp32 [n_tokens][n_heads], may be NULL: natural log of the sum of
                exp(scale q.k) over the row's positions
     scale      0: 1 / sqrt(head_dim)
     max_tokens an upper bound of the rows of one sequence (host); rows beyond it are not computed
     likely_tokens  how many rows most sequences have (host; 0: max_tokens), where max_tokens is far above it:
                it chooses among kernels for few and for many rows, each of which takes any number
     tree_mask  device, NULL or the sequences' trees (causal != 0): row j of sequence b attends to positions 0 ..
                lengths[b] - 1 and, of the sequence's own rows, to those i (position lengths[b] + i) whose bit i % 32 of
                word tree_mask[row * tree_stride + i / 32] is set, i < 32 tree_words. tree_words: 1 .. DEC_MAX_TREE / 32;
                rows numbered from 32 tree_words on are seen by none. As dec_draft_tree writes them, or any other set
     workspace  16-byte aligned device memory of dec_kvq_attention_workspace() bytes; its content
                is of no interest before or after the call
   A row with no position gives out = 0 and lse = -infinity. Scores, softmax statistics and the
   output sum are fp32; queries enter the products exactly (values below 2^-17 of their head's
   largest: to 2^-25 of it). Probabilities enter the second product with 11 bits, down to 2^-29 of the row's
   largest, and below that to steps of 2^-40 of it; in the kernel for many rows (more than 16 query rows
   per KV head and sequence, 32 for heads of 64) down to 2^-21 and to steps of 2^-32. Their sum is of
   fp32 terms. Rows that meet a bad page or a position
   beyond the page table hold nothing of use, the other sequences' are right. A call repeated
   gives the same bits; a sequence in another batch may be cut and joined elsewhere. A call of 2^31 query
   rows or of a page table of 2^31 positions is DEC_ERR_UNSUPPORTED. */
#define DEC_MAX_TREE 1024 /* rows of one sequence's tree */
typedef struct {
  int32_t n_heads;
  dec_rows q, out;
  float* lse;
  float scale;
  int32_t causal;
  int32_t max_tokens;
  void* workspace;
  int64_t workspace_bytes;
  int32_t likely_tokens;
  const uint32_t* tree_mask;
  int64_t tree_stride;
  int32_t tree_words;
} dec_kvq_attention_args;
dec_status dec_kvq_attention(const dec_kvq_cache* cache, const dec_kvq_seqs* seqs, const dec_kvq_attention_args* args,
                             void* stream);
/* Workspace bytes for calls with these sizes on the current device (-1 for a refused shape); any batch
   needs the same. */
int64_t dec_kvq_attention_workspace(const dec_kvq_cache* cache, int32_t n_heads, int32_t batch, int32_t max_tokens);

/* Trees of drafted tokens. Row j of a sequence has the row parents[j] (an index within the sequence, below j) as
   its parent; row 0 is the sequence's last known token. A row whose parent is not an earlier row begins a path of
   its own.
     parents    device int32 [n_tokens]
     lengths    device int32 [batch]: position of row 0 (NULL: no positions)
     max_tokens an upper bound of the rows of one sequence (host), at most DEC_MAX_TREE: a sequence's rows beyond it
                are not computed
     mask       [n_tokens][mask_stride] words, of which the first (max_tokens + 31) / 32 of each row are written: bit i
                where row i of the sequence is the row itself or above it
     positions  device int32 [n_tokens], may be NULL: lengths[b] + how many rows are above the row
   Rows of no sequence are left as they are. A cu_tokens that does not ascend makes sequences of no rows. */
typedef struct {
  int32_t batch;
  int32_t n_tokens;
  const int32_t* cu_tokens; /* device [batch + 1] */
  const int32_t* parents;
  const int32_t* lengths;
  int32_t max_tokens;
  uint32_t* mask;
  int64_t mask_stride;
  int32_t* positions;
} dec_draft_tree_args;
dec_status dec_draft_tree(const dec_draft_tree_args* args, void* stream);

/* Attention weight that cached positions receive, added up: for every position p that a row of the call attends to
   (causal and lengths as in dec_kvq_attention) and every KV head h
     mass_out[p] = decay * mass[p] + sum over the rows that attend to p and the heads of h's group of exp(scale q.k - lse)
   where mass and mass_out are fp32 [n_pages][n_kv_heads][page_tokens], 16-byte aligned, laid out as the cache's pages
   (mass_out may be mass, or share nothing with it). Positions that the call's rows stand at (causal) have had nothing
   before, and where decay is 0 nothing is read. Positions that no row could attend to are left as they are.
     q          bf16 rows of n_heads heads, lse device fp32 [n_tokens][n_heads], both as the attention had and gave them;
                a row whose lse is not finite adds nothing. A tree's rows see less than causal says: after a step of
                drafts it is the accepted rows' queries and lse that go in, as a chain at the same lengths, once
                dec_kvq_move has brought their path into place
     max_tokens an upper bound of the rows of one sequence (host); rows beyond it add nothing. With n_tokens, where that
                is less, it chooses among kernels for up to 8, up to 16 and more query rows a KV head
   Scores and sums are fp32; queries enter the products exactly (in the kernels for up to 16 query rows values below
   2^-17 of their head's largest: to 2^-25 of it). A call repeated gives the same bits, and no sum's order depends on the
   call's other sequences but by the kernel that they choose. Bad pages, and positions beyond the page table, are
   skipped and recorded in the cache's status. What a page that several sequences of one call share is left with
   depends on their order, which is not fixed: sequences that share pages take calls of their own, one after the other.
   Calls of 2^30 query rows or 2^31 positions or cache groups are DEC_ERR_UNSUPPORTED, and so are those for which
   n_kv_heads * (max_pages * page_tokens + n_tokens) / 16 * (min(batch, 256) + n_tokens * n_heads / n_kv_heads / 128)
   passes 2^32. */
typedef struct {
  int32_t n_heads;
  dec_rows q;
  const float* lse;
  float scale; /* 0: 1 / sqrt(head_dim) */
  int32_t causal;
  int32_t max_tokens;
  float decay;
  const float* mass; /* may be NULL where decay is 0 */
  float* mass_out;
} dec_kvq_mass_args;
dec_status dec_kvq_mass(const dec_kvq_cache* cache, const dec_kvq_seqs* seqs, const dec_kvq_mass_args* args, void* stream);

/* The positions that a cache bounded to `budget` a sequence keeps, for every sequence b and KV head: the first `sinks`
   and the last `recent` of its lengths[b] positions and, of those between, the ones of the largest mass (equal masses:
   the lower position first; a NaN orders below everything), budget in all. A sequence of budget positions and fewer
   keeps all.
     kept       device int32 [batch][n_kv_heads][budget]: the positions, ascending; -1 behind the last
     count      device int32 [batch]: how many
   seqs: n_tokens is of no interest, cu_tokens NULL and n_tokens == batch. Positions in bad pages (recorded in the
   cache's status) weigh nothing; a sequence whose length is negative (DEC_ERR_ARG) or beyond the page table
   (DEC_ERR_CAPACITY) keeps none. sinks + recent <= budget.
   Keys keep the angles of the positions that they had. Rows that are appended behind a list that was moved together
   need theirs from dec_kvq_append's positions; the engine's steps, which turn a row by its place (dec_step_kvq,
   and any after dec_kvq_load), must not follow. */
typedef struct {
  const float* mass; /* fp32 [n_pages][n_kv_heads][page_tokens] */
  int32_t budget;
  int32_t sinks;
  int32_t recent;
  int32_t* kept;
  int32_t* count;
} dec_kvq_heaviest_args;
dec_status dec_kvq_heaviest(const dec_kvq_cache* cache, const dec_kvq_seqs* seqs, const dec_kvq_heaviest_args* args,
                            void* stream);

/* Move positions as they are held (codes and scales, nothing is rounded again): for every sequence b, KV head h and
   i < min(count[b], max_count) position lengths[b] + i receives what position lengths[b] + index[i] holds, index being
   the list at index + b * index_stride + h * head_stride (head_stride 0: one list for all heads).
     index      device int32. Within a list it ascends and index[i] >= i: positions move down, into room that others
                have left, or stay. A negative entry moves nothing. A list that does not ascend, or moves up, leaves
                anything in the sequence's positions
     count      device int32 [batch]
     to         device int32, NULL or the page table to write to, in place of seqs' own: [batch][to_stride], to_pages of
                each row valid. It shares no page with the table that is read
     mass       NULL, or fp32 [n_pages][n_kv_heads][page_tokens], moved alongside
   In place (to NULL), positions that stay are not written: pages at a sequence's beginning that others share may be
   part of it as long as nothing moves in them. Other pages belong to one sequence of the call.
   seqs: cu_tokens NULL and n_tokens == batch; lengths is where a sequence's moves begin (its committed length; NULL: 0).
   Pages and positions out of range are skipped and recorded in status. */
typedef struct {
  const int32_t* index;
  int64_t index_stride;
  int64_t head_stride;
  const int32_t* count;
  int32_t max_count;
  const int32_t* to;
  int32_t to_pages;
  int64_t to_stride;
  float* mass;
} dec_kvq_move_args;
dec_status dec_kvq_move(const dec_kvq_cache* cache, const dec_kvq_seqs* seqs, const dec_kvq_move_args* args, void* stream);

/* Log-probabilities of rows of logits (fp32 or bf16; row r at logits + r * row_stride elements):
     targets      device int32 [rows], may be NULL; a target outside 0 .. vocab - 1 gives
                  logprob NaN and rank -1
     logprob      fp32 [rows]: x[target] - lse, lse = log(sum(exp(x)))
     rank         int32 [rows]: how many ids come before the target in the order by logit, larger
                  first, equal logits by lower id
     entropy      fp32 [rows], nats
     top_ids, top_logprobs  int32, fp32 [rows][top_n]: the first top_n ids of that order (0 <=
                  top_n <= DEC_MAX_TOP, <= vocab) and their log-probabilities
   Each output may be NULL (logprob and rank need targets). Logits of -infinity have probability
   0; a row with nothing else gives log-probabilities of -infinity and entropy 0. A row with a
   NaN or +infinity gives NaN log-probabilities and entropy; a NaN orders as -infinity.
   Log-probabilities are at most 0 and entropies at least 0, and their error does not grow with a
   common offset of the logits. (Rows whose largest logit is 8192 and more in magnitude are read twice.) Sums are
   fp32: a call repeated gives the same bits, a row in a call of other sizes or at another
   alignment may be summed in another order. */
#define DEC_MAX_TOP 32
typedef struct {
  const void* logits;
  dec_dtype dtype;
  int32_t rows;
  int32_t vocab;
  int64_t row_stride;
  const int32_t* targets;
  float* logprob;
  int32_t* rank;
  float* entropy;
  int32_t top_n;
  int32_t* top_ids;
  float* top_logprobs;
} dec_logprobs_args;
dec_status dec_logprobs(const dec_logprobs_args* args, void* stream);

/* Verification of drafted tokens against the target's probabilities, so that the tokens that come out are
   distributed as the target's own ("vLLM's Kimi K3 Backend Hits 842 Tokens per Second", section "Throughput holds
   across the tested range": verifying speculative drafts). Sequence b's rows are cu_tokens[b] .. cu_tokens[b + 1] - 1:
   row 0 its last known token, every other one a draft with a parent as in dec_draft_tree (parents NULL: each row's
   parent is the row before, a chain). cu_tokens ascend; where they do not, nothing that comes out is of use.
   p_j = softmax(logits of row j / temperature[b]) is the target's distribution after row j, q_j the one that the children of row j were drawn from, independently of one another: row j of
   draft_probs, or (draft_probs NULL) certainty of the child's token. From row 0 on, at row j with p = p_j, its
   children c in ascending order:
     uniforms[c] q(tokens[c]) < p(tokens[c]): c is accepted, and it goes on at row c;
     otherwise p becomes max(p - q, 0) over its sum (where that is 0, p stays) for the next child.
   Where no child is accepted (or there is none) the next token is the first id, in ascending order, up to which p sums
   to more than uniforms[row 0] times its whole sum. temperature NULL: 1; one that is not above 0: greedily, p_j and q
   are certainty of the first of the largest logits, and of the child's token.
     logits     [n_tokens] rows of vocab, fp32 or bf16, row_stride elements apart; -infinity has probability 0. A row
                with a NaN or +infinity, or nothing but -infinity, has no distribution: no child of it is accepted, and
                the next token after it is -1
     draft_probs  device fp32, prob_stride elements apart, or NULL; read only for rows with children. Not renormalised
     tokens, parents  device int32 [n_tokens]. A draft outside the vocabulary is refused and changes nothing
     uniforms   device fp32 [n_tokens], in 0 <= u < 1: row 0's for the next token, a draft's for its acceptance
     max_tokens an upper bound of the rows of one sequence (host), at most DEC_MAX_TREE; rows beyond it are not looked at
     path       device int32 [batch][max_tokens]: the accepted rows, 0 first; -1 behind the last (dec_kvq_move's list)
     count      device int32 [batch]: how many (1 + the accepted drafts; 0 for a sequence of no rows)
     next_tokens  device int32 [batch] (-1 for a sequence of no rows)
     workspace  16-byte aligned, of dec_verify_drafts_workspace() bytes
   More than 2^24 ids or 2^26 rows are DEC_ERR_UNSUPPORTED.
   Acceptance is decided on fp32 sums where they leave no doubt, and like the next token on sums of some 36 bits where
   they do (temperatures from 1e-37 to 1e30). Probabilities below 2^-120 of the row's largest count as 0. A call
   repeated gives the same. */
typedef struct {
  const void* logits;
  dec_dtype dtype;
  int32_t vocab;
  int64_t row_stride;
  const float* draft_probs;
  int64_t prob_stride;
  int32_t batch;
  int32_t n_tokens;
  const int32_t* cu_tokens;
  const int32_t* tokens;
  const int32_t* parents;
  const float* uniforms;
  const float* temperature; /* device [batch] */
  int32_t max_tokens;
  int32_t* path;
  int32_t* count;
  int32_t* next_tokens;
  void* workspace;
  int64_t workspace_bytes;
} dec_verify_drafts_args;
dec_status dec_verify_drafts(const dec_verify_drafts_args* args, void* stream);
/* Workspace bytes for n_tokens rows on any device (-1: negative). */
int64_t dec_verify_drafts_workspace(int32_t n_tokens);

/* ------------------------------------------------------------------------------------------
   The engine over these operators. Conventions are the engine's again (errors in
   dec_last_error(), stream == NULL is the engine's stream, work ordered after its earlier work). */

/* One decode step of `batch` sequences whose keys and values live in paged 4-bit caches, one cache
   per layer, in place of the engine's own bf16 cache (which it neither reads nor writes; an engine
   used only this way can have max_ctx 1 and a rotation table of its caller's). Token b stands at
   position lengths[b] of seqs, is appended there in every layer, and attends to positions 0 ..
   lengths[b]. lengths are the caller's: add 1 before the next step. Its rotary position is its place (or lengths[b]
   and its depth in a tree): sequences that positions were taken from (dec_kvq_heaviest) are not for these steps.
     caches       host array [n_layers] of the engine's KV heads and head_dim
     seqs         cu_tokens NULL, n_tokens == batch <= max_batch. Or, to verify drafts, several token rows a sequence
                  (cu_tokens given): batch counts the rows, n_tokens == batch, max_tokens bounds the rows of one
                  sequence, and row j of sequence b is appended at lengths[b] + j
     parents      with cu_tokens: NULL (the rows of a sequence follow one another), or device int32 [batch], each row's
                  parent in its sequence's tree of drafts (dec_draft_tree): the row then attends to positions 0 ..
                  lengths[b] - 1 and to its own path, and its rotary position goes by its depth. dec_verify_drafts
                  takes the step's logits, dec_kvq_move its path, once for each layer's cache
     rope         device fp32 [rope_len][head_dim / 2][2] (as dec_kvq_append's, full heads, half
                  split); NULL: the engine's table of max_ctx positions
     the others   as dec_step_args'
   The step runs in n_layers + 1 cooperative launches (the wide kernel cut at each layer's attention)
   and the cache's append and attention launches between them; nothing is synchronised. The first
   call of an engine allocates its buffers for these steps, and so does its first one with cu_tokens (make them before
   a stream capture begins). Rows of no sequence (before cu_tokens[0], behind the last) give nothing of use.
   Page ids, lengths and table bounds that are wrong are recorded in the caches' status words.
   Errors: DEC_ERR_ARG, DEC_ERR_UNSUPPORTED (an engine without the wide kernels: max_batch below
   dec_info.wide_min_batch, or a shape they do not take), DEC_ERR_POISONED, DEC_ERR_OOM,
   DEC_ERR_CUDA. */
typedef struct {
  const int32_t* tokens;
  const void* hidden_in;
  int32_t batch;
  const dec_kvq_cache* caches;
  const dec_kvq_seqs* seqs;
  const float* rope;
  int32_t rope_len;
  float* logits;
  int32_t* next_tokens;
  void* hidden_out;
  void* stream;
  const int32_t* parents;
  int32_t max_tokens;
} dec_step_kvq_args;
dec_status dec_step_kvq(dec_engine* eng, const dec_step_kvq_args* args);

/* Move a sequence between the engine's bf16 cache and pages: store writes positions 0 .. length - 1
   of slot seq into the pages of `table` (device int32 [max_pages], page p holding positions p *
   page_tokens on) of every layer's cache; load reads `length` positions back into a slot and sets
   its length. Keys are stored as the engine holds them, rotated. Queued on `stream`, behind what the
   caller has queued there on the pages and the table; synchronised before return (what the
   kernels found wrong is reported only in the caches' status words). Without a stream they are queued on
   the engine's own: nothing of the caller's is waited for then, so the table has to be written and
   other work on the pages done before the call. */
dec_status dec_kvq_store_ex(dec_engine* eng, int32_t seq, const dec_kvq_cache* caches, const int32_t* table,
                            int32_t max_pages, void* stream);
dec_status dec_kvq_load_ex(dec_engine* eng, int32_t seq, const dec_kvq_cache* caches, const int32_t* table,
                           int32_t max_pages, int32_t length, void* stream);
/* The same with stream = NULL. */
dec_status dec_kvq_store(dec_engine* eng, int32_t seq, const dec_kvq_cache* caches, const int32_t* table,
                         int32_t max_pages);
dec_status dec_kvq_load(dec_engine* eng, int32_t seq, const dec_kvq_cache* caches, const int32_t* table,
                        int32_t max_pages, int32_t length);

/* Score a text: append tokens[0 .. n - 1] (device int32) to slot seq as dec_prefill_kv's token mode
   does (launches of up to DEC_MAX_STEP_TOKENS positions) and give, after each position i, the
   log-probability and rank of targets[i] (device int32 [n], usually tokens[i + 1]; may be NULL), the
   entropy and the top_n ids, as dec_logprobs (outputs device arrays of n rows, each may be NULL).
   Queued on `stream`, nothing is synchronised. Requires vocab > 0. Errors: DEC_ERR_ARG,
   DEC_ERR_CAPACITY, DEC_ERR_POISONED, DEC_ERR_CUDA. */
typedef struct {
  int32_t seq;
  const int32_t* tokens;
  int32_t n;
  const int32_t* targets;
  float* logprob;
  int32_t* rank;
  float* entropy;
  int32_t top_n;
  int32_t* top_ids;
  float* top_logprobs;
  void* stream;
} dec_score_args;
dec_status dec_score(dec_engine* eng, const dec_score_args* args);

#ifdef __cplusplus
}
#endif
#endif /* DEC_H */
