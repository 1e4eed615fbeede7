/*
 * mfs.h -- C ABI of the GB300 lockstep frame step of a Moshi-class
 * full-duplex speech model (PersonaPlex / Moshi RQ-Transformer).
 *
 * One frame step (80 ms of audio per session) for B concurrent sessions
 * ("slots") runs, on one GPU:
 *   - the 17-stream delayed embedding sum (1 text row + 16 audio codebooks,
 *     delays [0, 0, 1 x 7, 0, 1 x 7]: mobius PR #368 "Add PersonaPlex / Moshi
 *     full-duplex S2S support", section "P3 - ONNX Runtime example"; token
 *     column layout: vLLM-Omni PersonaPlex recipe, section "Architecture");
 *   - one decode step of the temporal transformer (RMSNorm, RoPE, sliding-
 *     window causal attention over a per-slot ring of keys/values, SwiGLU:
 *     mobius PR #368, "P2 - Moshi LM"; 3000-frame ring window: vLLM-Omni
 *     PersonaPlex recipe, "Architecture" and "Notes") and a greedy text argmax;
 *   - the 16-substep autoregressive depformer with per-substep weights and a
 *     greedy code argmax per substep (mobius PR #368, "P2 - Moshi LM");
 *     optionally temperature + top-k sampling instead of the argmaxes.
 *
 * Conventions for every entry point:
 *   - Return value: MFS_OK (0) or a negative MFS_E_* status.  An argument
 *     error is detected on the host before anything is launched and leaves
 *     every slot's state unchanged; mfs_last_error() gives a one-line reason.
 *   - Host pointers are read or written only during the call; the library
 *     keeps no reference to them.  Device pointers must be device memory of
 *     the context's GPU.
 *   - All GPU work runs on the stream given to mfs_create().
 *   - A context is not thread-safe: one host thread at a time.
 */
#ifndef MFS_H
#define MFS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MFS_OK 0
#define MFS_E_ARG (-1)     /* null pointer, n out of range, duplicate slot, bad config */
#define MFS_E_SLOT (-2)    /* slot id outside [0, max_slots) */
#define MFS_E_TOKEN (-3)   /* token outside [-1, vocab) (text) or [-1, card) (audio) */
#define MFS_E_RANGE (-4)   /* a slot would pass max_pos frames (context limit) */
#define MFS_E_STATE (-5)   /* weights missing, unknown tensor name or wrong size */
#define MFS_E_CUDA (-6)    /* a CUDA runtime call failed */
#define MFS_E_DEVICE (-7)  /* a device-side wait gave up (bounded spin); state undefined */
#define MFS_E_NOMEM (-8)   /* device or host allocation failed */

#define MFS_DTYPE_F32 0
#define MFS_DTYPE_BF16 1
#define MFS_DTYPE_E4M3 2 /* only the codes of mfs_quant_kv */

#define MFS_MAX_SLOTS 64
#define MFS_N_STREAMS 17

typedef struct mfs_ctx mfs_ctx;

/* Model shape and limits.  Stream 0 is the text row; streams 1..16 are the
 * audio codebooks (1..8 agent, 9..16 user); delays[k] is stream k's delay in
 * frames.  window = ring length W (keys of positions p-W+1..p are attended);
 * max_pos = largest frame count a slot may reach (RoPE range).  n_q and
 * dep_steps must be 16.  Limits: head_dim in {64, 128}, dep_head_dim = 64,
 * every K dimension (d, ffn, dep_d, dep_ffn) a multiple of 8 and at most
 * 12288, max_slots <= MFS_MAX_SLOTS. */
typedef struct {
    int d, n_layers, n_heads, head_dim, ffn, text_vocab, card, n_q, window, max_pos;
    int dep_d, dep_layers, dep_heads, dep_head_dim, dep_ffn, dep_steps;
    int delays[MFS_N_STREAMS];
    double rope_theta, eps;
    int weight_dtype; /* MFS_DTYPE_F32 | MFS_DTYPE_BF16: linears and embedding tables */
    int kv_dtype;     /* MFS_DTYPE_F32 | MFS_DTYPE_BF16: the ring of keys/values */
    int max_slots;
} mfs_config;

/* Create a context on the current CUDA device: allocates the weight arena,
 * the per-slot key/value rings (max_slots x n_layers x window x d, for keys
 * and for values), the token histories and the activations.  cuda_stream is a
 * cudaStream_t (NULL: the library creates its own).  Every slot starts fresh
 * (position 0, empty history).  On success *out owns all of it. */
int mfs_create(const mfs_config* cfg, void* cuda_stream, mfs_ctx** out);

/* Synchronize and free everything the context owns. NULL is accepted. */
void mfs_destroy(mfs_ctx* ctx);

/* Reason for the last non-OK status of this context (never NULL); with a
 * NULL context, the reason the last mfs_create() on this thread failed. */
const char* mfs_last_error(const mfs_ctx* ctx);

/* Copy one named tensor into the weight arena (the caller keeps ownership).
 * src: host memory (on_device = 0) or device memory (on_device = 1); bytes
 * must equal the tensor's size.  Names and row-major shapes (W = weight
 * dtype, gains always fp32; V = text_vocab, C = card, S = dep_steps,
 * d' = dep_d, F' = dep_ffn):
 *   emb.text [V+1, d] W        emb.audio [16, C+1, d] W   (row V / C = INIT)
 *   layers.{l}.attn_norm [d]   layers.{l}.wqkv [3d, d] W   (rows q | k | v)
 *   layers.{l}.wo [d, d] W     layers.{l}.ffn_norm [d]
 *   layers.{l}.wgu [2F, d] W   (rows: gate then up)      layers.{l}.wdown [d, F] W
 *   out_norm [d]               text_head [V, d] W
 *   dep.in [S, d', d] W        dep.emb.text [V, d'] W      dep.emb.audio [S-1, C, d'] W
 *   dep.layers.{l}.attn_norm [d']   dep.layers.{l}.wqkv [S, 3d', d'] W
 *   dep.layers.{l}.wo [S, d', d'] W dep.layers.{l}.ffn_norm [d']
 *   dep.layers.{l}.wgu [S, 2F', d'] W   dep.layers.{l}.wdown [S, d', F'] W
 *   dep.out_norm [d']          dep.head [S, C, d'] W
 * Blocking.  Returns MFS_E_STATE for an unknown name or a size mismatch. */
int mfs_load_weights(mfs_ctx* ctx, const char* name, const void* src, size_t bytes, int on_device);

/* One frame step for n slots (1 <= n <= max_slots): the lockstep step with
 * per-codebook delays and delayed output collection (mobius PR #368, "P3 -
 * ONNX Runtime example"), all listed sessions advancing together in one 80 ms
 * tick (vLLM-Omni PersonaPlex recipe, "Notes": batched ticks).
 *   slots    [n]      distinct slot ids (host)
 *   in_codes [n, 17]  frame p's tokens for each slot (host): -1 = generate,
 *                     else the token is forced (text < text_vocab, audio < card)
 *   text_tok [n]      out (host): text token of frame p
 *   codes    [n, 16]  out (host): code of stream k (k = 1..16) for frame
 *                     p - delays[k], or -1 when that frame is before 0
 * Slots not listed are untouched.  Each listed slot advances by one frame.
 * Blocks until the results are on the host. */
int mfs_step(mfs_ctx* ctx, int n, const int32_t* slots, const int32_t* in_codes,
             int32_t* text_tok, int32_t* codes);

/* Same step with device-resident tokens; returns without waiting.
 *   slots (host) [n]; d_in_codes [n, 17], d_text_tok [n], d_codes [n, 16]
 *   (device; may be NULL for outputs that are not wanted).
 * Token ranges are checked on the device: a bad token makes the whole step
 * (and any later step enqueued before the next mfs_sync) a no-op, and the
 * next mfs_sync (or blocking call) returns MFS_E_TOKEN with the positions of
 * those steps rolled back. */
int mfs_step_device(mfs_ctx* ctx, int n, const int32_t* slots, const int32_t* d_in_codes,
                    int32_t* d_text_tok, int32_t* d_codes);

/* Wait for enqueued steps; report a deferred device-side error (see above). */
int mfs_sync(mfs_ctx* ctx);

/* Teacher-forced prompt of T frames for n slots: codes [n, T, 17] (host), every
 * token >= 0 (persona and voice go in through the same lockstep step with their
 * rows supplied: vLLM-Omni PersonaPlex recipe, "Architecture").  Runs the temporal stack only (the text head and depformer
 * cannot change a slot whose every stream is supplied) and advances each slot
 * by T frames.  Blocking. */
int mfs_prefill(mfs_ctx* ctx, int n, const int32_t* slots, int T, const int32_t* codes);

/* Return a slot to the fresh state: position 0, empty history, so that a new
 * session can take it (vLLM-Omni PersonaPlex recipe, "Notes": a recycled slot
 * matches a fresh engine for the same inputs).  Its ring is not cleared:
 * positions are only ever read after being rewritten. */
int mfs_reset_slot(mfs_ctx* ctx, int slot);

/* Frame count of a slot (its next position), or a negative status. */
int mfs_position(const mfs_ctx* ctx, int slot);

/* ---------------------------------------------------------------- slot state
 * A slot's whole decode state as one host buffer, so that a session can be
 * checkpointed, moved to another context, or checked against an independent
 * implementation without replaying its history (SGLang-Omni cookbook,
 * PersonaPlex, "Known limitations": decode states are resident per request).
 * Layout, little-endian, MFS_SLOT_HEADER_BYTES of header then the ring:
 *   int32 version (1), position p, window W, kv dtype (MFS_DTYPE_*),
 *   int32 hist[17][3]: token of stream k for frame f at [k][f mod 3], -1 = none,
 *   zero padding to MFS_SLOT_HEADER_BYTES,
 *   keys [n_layers][W][d] then values [n_layers][W][d] in the kv dtype; row r
 *   holds the position q < p with q mod W == r among the last W positions
 *   (rows of positions never written are unspecified).
 * mfs_slot_state_bytes: the buffer size for this context.  Export copies the
 * slot's state out (waits for the stream); import replaces it after checking
 * the header (version, window, dtype, 0 <= p <= max_pos, every history token
 * -1 or inside its stream's vocabulary), else MFS_E_ARG and nothing changes. */
#define MFS_SLOT_HEADER_BYTES 256
size_t mfs_slot_state_bytes(const mfs_ctx* ctx);
int mfs_export_slot(mfs_ctx* ctx, int slot, void* buf, size_t bytes);
int mfs_import_slot(mfs_ctx* ctx, int slot, const void* buf, size_t bytes);

/* Diagnostics of the last step, rows in that step's slot order (any pointer
 * may be NULL): text logits [n, V], depformer logits [n, 16, C] (fp32), and
 * the raw argmaxes before forcing, text [n] and per substep [n, 16]. */
int mfs_read_debug(mfs_ctx* ctx, float* text_logits, float* dep_logits,
                   int32_t* text_argmax, int32_t* code_argmax);

/* Ring window variant (SGLang-Omni cookbook, PersonaPlex, "Known limitations":
 * the window follows the streaming ring, including the masked oldest slot once
 * the ring fills).  on = 1: a step at position p attends to positions
 * max(0, p - W + 2) .. p, i.e. W - 1 keys once the ring holds W; the ring keeps
 * its capacity W.  on = 0 (default): positions max(0, p - W + 1) .. p.  Applies
 * from the next step on; waits for the context's stream.  MFS_E_ARG if on is not
 * 0 or 1, or W < 2. */
int mfs_set_ring_mask_oldest(mfs_ctx* ctx, int on);

/* Testing: the next step (or prompt launch) takes sequence number seq + 1.
 * Phases hand values over as words tagged (sequence << 10) | phase in 32 bits,
 * so tags repeat every 2^22 steps; before the step whose sequence number is a
 * multiple of 2^22 the library sets every tagged word to a value no step
 * writes.  This call lets a test cross that point without 4 million steps.
 * Waits for the context's stream first; MFS_E_ARG on a null context. */
int mfs_debug_set_seq(mfs_ctx* ctx, uint32_t seq);

/* Execution mode: 0 (default) = one persistent cooperative launch per step,
 * in which a phase waits for the tagged outputs of the phases it reads (no
 * grid-wide barrier); 1 = one launch per phase (same arithmetic, bit for bit,
 * for diagnosis). */
int mfs_set_mode(mfs_ctx* ctx, int mode);

/* Sampling heads (mobius PR #368, commit note replacing greedy argmax with
 * temperature + top-k sampling: text 0.7 / 25, audio 0.8 / 250; SGLang-Omni
 * cookbook, PersonaPlex, "Stage sampling": every request draws from its own
 * generator).  mfs_set_sampling sets a slot's temperatures and top-k (k <= 1
 * or temperature 0: greedy, the default for every slot).  mfs_step_sampled is
 * mfs_step plus uniforms [n, 17] in [0, 1) from the caller's per-session
 * generator: row i's token of stream k (0: text) that is not supplied is drawn
 * with uniforms[i][k] as follows.  The candidates are the k largest logits
 * (ties: lower index first), weighted exp((logit - max) / temperature); the
 * token is the first candidate, in ascending index order, at which the running
 * sum of weights exceeds u times their total.  A drawn token feeds the next
 * substep like a greedy one.  mfs_read_debug still reports the raw argmaxes.
 * Uniforms outside [0, 1) give MFS_E_ARG.  mfs_step and mfs_step_device stay
 * greedy. */
int mfs_set_sampling(mfs_ctx* ctx, int slot, float text_temp, int text_topk, float audio_temp, int audio_topk);
int mfs_step_sampled(mfs_ctx* ctx, int n, const int32_t* slots, const int32_t* in_codes, const float* uniforms,
                     int32_t* text_tok, int32_t* codes);

/* Depformer substeps whose every output is settled without them (mobius PR
 * #368, "P3 - ONNX Runtime example": substep j yields the code of stream j+1;
 * SGLang-Omni cookbook, PersonaPlex, "Known limitations": the depformer steps
 * run after the backbone each frame).  With on = 1, a step skips the trailing
 * substeps j..15 when, for every slot, the tokens of streams j+1..16 are
 * supplied (or belong to frames before 0): the substeps are causal, so the
 * earlier substeps and every output are unchanged.  In decode with the user
 * streams supplied this skips substeps 8..15 (about 1.3 GB of weights per
 * step).  Skipped substeps leave no logits and report argmax -1 in
 * mfs_read_debug.  Default 0: all 16 substeps run. */
int mfs_set_skip_settled(mfs_ctx* ctx, int on);

/* Failure detection (the pages detect failures on the host only, e.g. sessions
 * beyond the batch size are refused: vLLM-Omni PersonaPlex recipe, "Notes";
 * the device-side limit below has no counterpart there).  Every wait inside the step kernel (on another CTA's
 * tagged output, on a weight stage) gives up after a limit, records where,
 * and the call returns MFS_E_DEVICE with that place in mfs_last_error; the
 * context stays usable, the state of the step's slots is undefined (reset or
 * import them).  mfs_set_wait_limit sets the limit (1 .. 60000 ms; default
 * 2000).  mfs_debug_stall checks the mechanism: it launches the slot's first
 * attention-projection phase alone, whose input is never produced, so its
 * waits run out; it returns MFS_E_DEVICE (or MFS_E_STATE if nothing gave up)
 * and leaves the slot's state undefined. */
int mfs_set_wait_limit(mfs_ctx* ctx, int ms);
int mfs_debug_stall(mfs_ctx* ctx, int slot);

/* Kernel launches made by the last step (for accounting). */
int mfs_launches_per_step(const mfs_ctx* ctx);

/* Kernel timing.  flags bit 0: every step records a CUDA event pair on the
 * context's stream around its kernel launch(es); mfs_kernel_time waits for
 * the stream, returns the summed device time (ms) and the number of steps
 * timed since the previous call, and starts a new sum.  flags bit 1: CTA 0
 * records, per phase, 8 values: GPU timer stamps (ns) at the start, when the
 * inputs are ready, when the last weight stage is consumed, at the end (0
 * where a point does not apply), then the ns spent waiting for weight stages
 * and the number of stages, summed since the last read, then the latest end
 * of the phase over all CTAs (timer ns, the maximum since the last read); mfs_phase_times
 * copies [phases + 1][8] values into ns, restarts the sums and returns the
 * count, or a negative status. */
int mfs_set_timing(mfs_ctx* ctx, int flags);
int mfs_kernel_time(mfs_ctx* ctx, double* total_ms, int* steps);
int mfs_phase_times(mfs_ctx* ctx, uint64_t* ns, int cap);

/* ---------------------------------------------------------------- Mimi RVQ
 * Encoder-side argmin quantizer of Mimi's split residual vector quantizer
 * (mobius PR #368, "P1 - Mimi": SplitResidualVectorQuantizer and the
 * encoder-side argmin quantizer, 8 codes per 80 ms frame; kyutai-labs/moshi,
 * "Mimi": the first codebook is semantic).  For each of T frames: codebook 0
 * takes the nearest codeword to z_sem[t]; codebooks 1..7 quantize z_ac[t] and
 * then, in turn, the residual the stage before leaves (r -= chosen codeword).
 * Nearest = least squared Euclidean distance (fp32), ties to the lower index.
 *   z_sem, z_ac  device, [T][D] fp32, 16-byte aligned (the quantizer's input
 *                latents; the codec's trained projections are not part of it)
 *   codebooks    device, [8][Cb][D] fp32, 16-byte aligned
 *   codes        device, [T][8] int32 out
 *   D            multiple of 4 in [4, MFS_RVQ_MAX_DIM]; stream as elsewhere
 * D a multiple of 8: the distances' cross terms r.c run on the tensor cores
 * (bf16 high/low parts of r and c, fp32 accumulation, about 16 significant
 * bits); per frame, the best 2 codewords by that score of each class of
 * indices mod 8 are candidates, and those within a band of four times the
 * score's error bound (2^-14 |r| |c|) of the best score are re-ranked by their
 * fp32 distance (a fixed summation order), so the code is the exhaustive fp32
 * argmin (up to that order's rounding) unless two codewords of the nearest's
 * class score within that error of it.  Up to D of about 520, CTAs work in
 * pairs (32 frames per pair, every other codeword tile per CTA) that exchange
 * each frame's winner through global memory, in cooperative launches of at
 * most the device's co-resident grid (2432 frames per launch on 152 SMs); a
 * larger D takes one CTA per 16 frames.  Codebooks of 2^24 or more codewords
 * use the CUDA-core form.  The tensor-core form takes about 4 * 8 * Cb * D +
 * 32 * Cb bytes of scratch (plus 1 KB per CTA pair) from the device's
 * stream-ordered pool and frees it on the stream.  Otherwise every distance is
 * computed exactly in fp32 on the CUDA cores.
 * Enqueues and returns; MFS_E_ARG on bad sizes, alignment or NULL pointers;
 * MFS_E_CUDA if the scratch or a launch fails (mfs_last_error(NULL) gives the
 * reason).  A frame whose distances are all NaN gets code 0x7fffffff; on the
 * tensor-core form, if one of the kernel's internal waits gives up (about 2 s:
 * a stalled device), the frames of the groups that saw it get code -1. */
#define MFS_RVQ_MAX_DIM 1024
int mfs_rvq_encode(const float* z_sem, const float* z_ac, int T, int D, const float* codebooks, int Cb,
                   int32_t* codes, void* cuda_stream);

/* ---------------------------------------------------------------- no-alloc
 * Greedy argmax over rows of fp32 logits that allocates no device memory.
 * The pages describe no such call: it exists for callers that cannot call
 * cudaMalloc at the point where they pick tokens, for example code running
 * inside a serving engine whose allocator has already reserved all free
 * device memory (a cudaMalloc there fails or takes memory the engine counts
 * on), or a real-time loop that must not block on the allocator.
 *
 * It is the frame step's argmax stage as a stand-alone kernel: blocks of 4096
 * columns leave partial maxima in scratch memory and the last block of each
 * row reduces them.  That scratch is a fixed static array of
 * MFS_ARGMAX_SCRATCH_BYTES (528 KiB) inside this library, held on every GPU
 * that loads the library until the process exits.
 *
 *   logits  device pointer, row r at logits + r * ld (fp32, read only)
 *   rows    0 .. MFS_ARGMAX_MAX_ROWS; 0 returns MFS_OK and launches nothing
 *   cols    >= 1, with rows * ceil(cols / 4096) <= MFS_ARGMAX_MAX_PARTIALS
 *   ld      row stride in elements, >= cols
 *   out     device pointer to rows int32: the lowest column holding the
 *           row's maximum (NaN never wins; a row of only NaN gives 0), the
 *           same rule as the step's text and code argmax
 *   stream  cudaStream_t (NULL = legacy default stream); the call only
 *           enqueues work and returns without waiting
 * Returns MFS_OK, MFS_E_ARG (bad sizes or NULL pointers), MFS_E_RANGE (sizes
 * beyond the fixed scratch), or MFS_E_CUDA; mfs_last_error(NULL) then gives
 * the reason.  MFS_E_ARG and MFS_E_RANGE are found before anything is
 * enqueued.  MFS_E_CUDA from the launch itself can come after the clear of the
 * row counters (a memset of the scratch) was already enqueued on the stream;
 * the argmax kernel then did not run and `out` is unchanged.
 *
 * The first call on each device looks up the device address of the scratch
 * array (cudaGetSymbolAddress) with that device current: make that first call
 * before any stream capture on the device.  The address is cached per device
 * for the life of the process and is not looked up again: after a
 * cudaDeviceReset of that device the cached address is stale, so do not call
 * this entry point on a device that was reset.  Every call on a device shares the
 * one array; each call first clears the per-row counters that must start at
 * zero.  Calls whose work overlaps on the GPU (other streams, other host
 * threads) race on the array and may return wrong indices: order them on one
 * stream or synchronise between them. */
#define MFS_ARGMAX_MAX_ROWS 4096
#define MFS_ARGMAX_MAX_PARTIALS 65536
#define MFS_ARGMAX_SCRATCH_BYTES (MFS_ARGMAX_MAX_ROWS * 4 + MFS_ARGMAX_MAX_PARTIALS * 8)
int mfs_argmax_rows_noalloc(const float* logits, int rows, int cols, long long ld, int32_t* out,
                            void* cuda_stream);

/* ---------------------------------------------------------------- sampling rows
 * Draws one token from each row of logits, from uniforms that the caller gives:
 * the sampling heads of mfs_step_sampled as a stand-alone call on device memory
 * (SGLang-Omni cookbook, PersonaPlex, "Stage sampling"), with min-p and top-p
 * beside temperature and top-k, and settings of its own for every row.
 *
 *   logits  device, row r at logits + r * ld (elements); dtype MFS_DTYPE_F32 or
 *           MFS_DTYPE_BF16; any alignment of an element; read only
 *   rows    >= 0 (0 returns MFS_OK); cols 1 .. MFS_SAMPLE_MAX_COLS; ld >= cols
 *   temperature, top_k, top_p, min_p
 *           device, [rows] each, or NULL: no temperature array means 1 for every
 *           row, no other array means that filter is off for every row
 *   uniforms device [rows], in [0, 1)
 *   tokens   device [rows], out
 * Row r, with T = temperature[r] and l_i its logits, m their maximum:
 *   - T <= 0 or NaN: the lowest column of the maximum (mfs_argmax_rows_noalloc's
 *     rule: NaN never wins, a row of only NaN gives 0).  The same where the
 *     maximum is -inf.
 *   - weights w_i = exp((l_i - m) / T) (1 where l_i = m; a T below 1.5e-30 counts as
 *     that, a difference past the largest fp32 number as infinite); a NaN logit is
 *     never a candidate.  Order the columns by logit, largest first, equal logits by
 *     column.  The candidates are the longest prefix of that order with
 *     w_i >= min_p[r] (min_p <= 0: every column; above 1 it counts as 1), cut to
 *     top_k[r] columns (<= 0: not cut), then cut to the shortest prefix whose
 *     weights sum to at least top_p[r] times the sum of the whole (>= 1: not
 *     cut; never less than one column).
 *   - The token is the first candidate, in ascending column order, at which the
 *     running sum of weights exceeds uniforms[r] times their sum (a uniform below
 *     0 or NaN acts as 0, one of 1 or more takes the last candidate).
 * Weights and sums are exact enough that the token is the one that the
 * definition gives in real numbers, unless a sum lies within 2^-40 + cols 2^-60
 * of the total from a border.  The same inputs always give the same tokens.
 * Enqueues on `stream` and returns; no memory is allocated, so it can be captured.
 * MFS_E_ARG on bad sizes or NULL pointers, before anything is enqueued. */
#define MFS_SAMPLE_MAX_COLS (1 << 22)
int mfs_sample_rows(const void* logits, int dtype, int rows, int cols, long long ld, const float* temperature,
                    const int32_t* top_k, const float* top_p, const float* min_p, const float* uniforms,
                    int32_t* tokens, void* cuda_stream);

/* ---------------------------------------------------------------- paged cache
 * Keys and values of many sequences in pages of a shared pool, for callers whose
 * sessions should hold only the memory of the frames they have seen, instead of
 * a whole ring each (SGLang-Omni cookbook, PersonaPlex, "Known limitations": the
 * windowed pool of keys and values).  One descriptor is one layer's cache.
 *
 *   k, v     device, dtype MFS_DTYPE_F32 or MFS_DTYPE_BF16; element e of head h
 *            at row r of page g lies at g * page_stride + h * head_stride +
 *            r * row_stride + e (strides in elements, of k and v alike, >= 0;
 *            k, v and every stride a multiple of 16 bytes)
 *   table    device int32: the page that holds positions j * page_size ..
 *            (j + 1) * page_size - 1 of sequence s is table[s * table_stride + j],
 *            j < table_width.
 *            Entries that a call does not need are not read as pages (they may
 *            hold anything); sequences may share pages they only read.
 *   head_dim 64 or 128; page_size 1 .. MFS_MAX_PAGE_SIZE; at most MFS_MAX_HEADS heads, of
 *            queries in the calls below too
 * A needed entry outside [0, n_pages), or a position at or past
 * table_width * page_size, never touches memory outside the pool: the append
 * skips that token's row, the attention gives NaN for that sequence. */
#define MFS_MAX_PAGE_SIZE 65536
#define MFS_MAX_HEADS 65535
typedef struct {
    void* k;
    void* v;
    const int32_t* table;
    int table_width;          /* entries of a sequence, >= 1 */
    long long table_stride;   /* entries from one sequence to the next, >= 0 */
    int n_pages, page_size, n_kv_heads, head_dim, dtype;
    long long page_stride, head_stride, row_stride;
} mfs_paged_kv;

#define MFS_ROPE_NONE 0
#define MFS_ROPE_INTERLEAVED 1 /* pairs (2 i, 2 i + 1): the frame step's layout */
#define MFS_ROPE_HALF 2        /* pairs (i, i + head_dim / 2) */

/* A rotation of part of each head, or one slowed down for contexts longer than the model's own:
 *   layout    MFS_ROPE_*
 *   dims      elements of each head that are rotated, from its first: pairs (2 i, 2 i + 1) or
 *             (i, i + dims / 2); a multiple of 16, at most head_dim; 0: all.  The others pass unchanged.
 *   theta     base, > 0: pair i turns by position * f_i, f_i = theta^(-2 i / dims)
 *   factor, original, low, high
 *             f_i becomes f_i (c_i + (1 - c_i) / factor), with c_i the clamp to [0, 1] of
 *             (r_i - low) / (high - low), r_i = original * f_i / (2 pi) the turns that pair i makes
 *             over `original` positions: pairs that turn often keep their speed, slow ones are
 *             interpolated, those between are blended.  original = 0: c_i = 0, every pair is
 *             slowed by factor.  factor = 1: no change.  factor > 0, original >= 0, and with
 *             original > 0 0 <= low < high.
 *   magnitude the rotated elements are multiplied by it, > 0 */
typedef struct {
    int layout, dims;
    double theta, factor, original, low, high, magnitude;
} mfs_rope;

/* Append new tokens' keys and values to the paged cache, rotated by their
 * positions on the way, and rotate their queries (mobius PR #368, "P2 - Moshi
 * LM": RoPE at the absolute position, offset by the cached length).
 *   cu       device [n_seqs + 1]: tokens cu[s] .. cu[s + 1] - 1 belong to sequence
 *            s (ascending, cu[0] = 0; a sequence may have none; tokens from
 *            cu[n_seqs] on belong to none and their rows are left as they are)
 *   kv_len   device [n_seqs]: the sequence's length with the new tokens, so the
 *            i-th of its c new tokens has position kv_len[s] - c + i (a negative
 *            position, like a bad page, is rotated but not written to the cache)
 *   q        [n_tokens][n_q_heads][head_dim] or NULL, out to q_out (may be q)
 *   k, v     [n_tokens][n_kv_heads][head_dim]; k_out: NULL, or the rotated keys
 *            (may be k), for mfs_prompt_attention
 *            *_stride: elements from one token to the next (heads are dense);
 *            pointers and strides multiples of 16 bytes; the cache's dtype
 *   theta    RoPE base, > 0: pair i turns by position * theta^(-2 i / head_dim);
 *            the angle is reduced in 64 bits, the rotation runs in 32 bits and is
 *            rounded once; ignored with MFS_ROPE_NONE
 * Outputs overlap inputs only where one is the other's array (same pointer and
 * stride).  Where two tokens of a call reach the same row of the same page, that
 * row is left with parts of both, its key and value not of one token; no other
 * row is touched.
 * Enqueues and returns; MFS_E_ARG on bad sizes, strides, alignment or NULL. */
int mfs_kv_append(const mfs_paged_kv* cache, int n_tokens, int n_seqs, const int32_t* cu, const int32_t* kv_len,
                  const void* q, long long q_stride, int n_q_heads, void* q_out, long long q_out_stride,
                  const void* k, long long k_stride, void* k_out, long long k_out_stride, const void* v,
                  long long v_stride, int rope, double theta, void* cuda_stream);

/* mfs_kv_append with a rotation as above (NULL: none). */
int mfs_kv_append_rope(const mfs_paged_kv* cache, int n_tokens, int n_seqs, const int32_t* cu, const int32_t* kv_len,
                       const void* q, long long q_stride, int n_q_heads, void* q_out, long long q_out_stride,
                       const void* k, long long k_stride, void* k_out, long long k_out_stride, const void* v,
                       long long v_stride, const mfs_rope* rope, void* cuda_stream);

/* Read the last rows of sequences back: row i of the c = cu[s + 1] - cu[s] rows of
 * sequence s is position kv_len[s] - c + i, as in mfs_kv_append.
 *   k_out, v_out  [n_tokens][n_kv_heads][head_dim], the cache's dtype, strides as above;
 *                 rows from cu[n_seqs] on are left as they are
 * A negative position or one without a valid page gives NaN. */
int mfs_kv_read(const mfs_paged_kv* cache, int n_tokens, int n_seqs, const int32_t* cu, const int32_t* kv_len, void* k_out,
                long long k_stride, void* v_out, long long v_stride, void* cuda_stream);

/* Attention of one new token per sequence over the paged cache:
 *   out[s][h] = sum_j softmax_j(scale * q[s][h] . k_j) v_j,  j in [max(0, L - window), L)
 * with L = kv_len[s] (the new token is already appended), the keys and values of
 * kv head h / (n_q_heads / n_kv_heads).  window = 0: every position.  The work is
 * split over the cache's length into equal shares and joined in a fixed order, so
 * the same inputs give the same bits.  L <= 0 gives zeros.
 *   q, out   [n_seqs][n_q_heads][head_dim], the cache's dtype, strides as above
 *            (out may be q); n_q_heads a multiple of n_kv_heads
 *   scale    > 0, finite
 *   workspace device memory of mfs_paged_attention_workspace() bytes, 16-byte
 *            aligned, its contents need not be kept or set between calls.  Calls whose work
 *            can overlap on the GPU (other streams, two captured graphs) need one each.
 * A score of -infinity is a weight of 0; a sequence that has no other gives NaN.
 * Rows of the cache at or past L, or before the window, are not read.  Sums and
 * softmax statistics are fp32; with a bf16 cache the softmax weights are rounded
 * to bf16 for the product with the values.  Enqueues and returns; MFS_E_ARG on
 * bad sizes, strides, alignment or NULL. */
size_t mfs_paged_attention_workspace(const mfs_paged_kv* cache, int n_q_heads);
int mfs_paged_attention(const mfs_paged_kv* cache, int n_seqs, const int32_t* kv_len, const void* q,
                        long long q_stride, int n_q_heads, void* out, long long out_stride, float scale, int window,
                        void* workspace, size_t workspace_bytes, void* cuda_stream);

/* ---------------------------------------------------------------- 8-bit cache
 * A paged cache whose rows (one position of one head, of keys or of values) are
 * held as e4m3 codes with one power of two each: half the memory, and half the
 * bytes that attention reads, of bf16 (SGLang-Omni cookbook, PersonaPlex, "Known
 * limitations": the pool's memory bounds the sessions).
 *
 *   kv       as above with dtype MFS_DTYPE_E4M3: k and v hold codes, strides in
 *            elements are bytes (multiples of 16)
 *   k_exp, v_exp
 *            device: the exponent byte b of head h at row r of page g lies at
 *            g * exp_page_stride + h * exp_head_stride + r * exp_row_stride (bytes, >= 0)
 * Code c of a row with exponent b stands for c * 2^(b - 127), 1 <= b <= 254; b = 0: the
 * row is zeros, whatever its codes (NaN among them).  The append writes the least b
 * that keeps the row's largest value within 448 (at least 1; 0 for a row of zeros)
 * and rounds to nearest, ties to even: off by at most 2^-4 of a value, or 2^-17 of
 * the row's largest, or 2^-136 (where b is at its least: rows below 448 * 2^-126) (a
 * value above 1.9375 * 2^127 becomes 2^128, which reads as infinite).  A row with an
 * element that is not finite becomes codes of NaN. */
typedef struct {
    mfs_paged_kv kv;
    uint8_t* k_exp;
    uint8_t* v_exp;
    long long exp_page_stride, exp_head_stride, exp_row_stride;
} mfs_quant_kv;

/* mfs_kv_append_rope into an 8-bit cache; q, k, v, q_out and k_out have `dtype`
 * (MFS_DTYPE_F32 or MFS_DTYPE_BF16).  A key is quantised as rotated in 32 bits;
 * k_out gets it rounded to dtype, not quantised. */
int mfs_quant_append(const mfs_quant_kv* cache, int dtype, int n_tokens, int n_seqs, const int32_t* cu, const int32_t* kv_len,
                     const void* q, long long q_stride, int n_q_heads, void* q_out, long long q_out_stride,
                     const void* k, long long k_stride, void* k_out, long long k_out_stride, const void* v,
                     long long v_stride, const mfs_rope* rope, void* cuda_stream);

/* mfs_kv_read from an 8-bit cache, to `dtype` (fp32 holds every value; bf16 rounds only below 2^-126). */
int mfs_quant_read(const mfs_quant_kv* cache, int dtype, int n_tokens, int n_seqs, const int32_t* cu, const int32_t* kv_len,
                   void* k_out, long long k_stride, void* v_out, long long v_stride, void* cuda_stream);

/* mfs_paged_attention over an 8-bit cache; q and out have `dtype`.  Products run on
 * the codes, scores, statistics and sums in fp32.  With bf16 queries the softmax
 * weights are rounded to 11 bits for the product with the values, with fp32 queries
 * queries and weights are held in two such parts.  A code of NaN in a row that is seen gives NaN. */
size_t mfs_quant_attention_workspace(const mfs_quant_kv* cache, int dtype, int n_q_heads);
int mfs_quant_attention(const mfs_quant_kv* cache, int dtype, int n_seqs, const int32_t* kv_len, const void* q,
                        long long q_stride, int n_q_heads, void* out, long long out_stride, float scale, int window,
                        void* workspace, size_t workspace_bytes, void* cuda_stream);

/* ------------------------------------------------------------ shared prefixes
 * mfs_paged_attention for a batch in groups of sequences that begin alike (one
 * persona's or one system prompt's frames): the keys and values of a group's
 * prefix are read and multiplied once for all its sequences.
 *   groups     device [n_groups + 1]: sequences groups[i] .. groups[i + 1] - 1 are group
 *              i (ascending; sequences outside every group are attended to by themselves)
 *   prefix_len device [n_groups]: positions that the group's sequences have in common.
 *              Their tables name the pages of all their positions, the shared
 *              ones among them, and positions count from the prefix's first, as for
 *              mfs_paged_attention: the result is that call's.  A prefix is
 *              read by way of the table of one of the group's sequences that see it whole.
 * A sequence that does not see its whole prefix (kv_len shorter than it, or a window
 * that begins inside it) is attended to by itself, as is one that is alone in its
 * group.  A bad page in a prefix gives NaN for those that share it.  Where all that
 * sharing could save is little by the table's width and the window (lengths are not
 * known on the host: give a table no wider than they need, as a view of a wider one),
 * or the queries are fp32 over an 8-bit cache, the call is the one-token attention's.  bf16 queries: prefix products
 * on the tensor cores, keys and values in bf16 (an 8-bit cache's values are exact in
 * it), softmax weights rounded to bf16, over an 8-bit cache held in two such parts (16
 * bits); if one of that kernel's internal waits gives up (about 2 s: a stalled device),
 * what it could not compute is NaN.  fp32: on the CUDA cores in fp32.
 *   workspace  of mfs_shared_attention_workspace() bytes for n_seqs sequences or more,
 *              else as for mfs_paged_attention */
size_t mfs_shared_attention_workspace(const mfs_paged_kv* cache, int n_q_heads, int n_seqs);
int mfs_shared_attention(const mfs_paged_kv* cache, int n_seqs, const int32_t* kv_len, int n_groups, const int32_t* groups,
                         const int32_t* prefix_len, const void* q, long long q_stride, int n_q_heads, void* out,
                         long long out_stride, float scale, int window, void* workspace, size_t workspace_bytes, void* cuda_stream);
size_t mfs_quant_shared_attention_workspace(const mfs_quant_kv* cache, int dtype, int n_q_heads, int n_seqs);
int mfs_quant_shared_attention(const mfs_quant_kv* cache, int dtype, int n_seqs, const int32_t* kv_len, int n_groups,
                               const int32_t* groups, const int32_t* prefix_len, const void* q, long long q_stride, int n_q_heads,
                               void* out, long long out_stride, float scale, int window, void* workspace, size_t workspace_bytes,
                               void* cuda_stream);

/* Causal attention over whole prompts, packed one behind the other:
 *   out[t][h] = sum_j softmax_j(scale * q[t][h] . k_j) v_j,  j in [max(b, t - window + 1), t]
 * with b the first token of t's sequence (mobius PR #368, "P2 - Moshi LM":
 * sliding-window causal attention); window = 0: from b on.
 *   cu       device [n_seqs + 1] as for mfs_kv_append; rows from cu[n_seqs] on
 *            are left as they are
 *   q, out   [n_tokens][n_q_heads][head_dim]; k, v [n_tokens][n_kv_heads][head_dim];
 *            dtype MFS_DTYPE_F32 or MFS_DTYPE_BF16; head_dim 64 or 128; n_q_heads a
 *            multiple of n_kv_heads, at most MFS_MAX_HEADS; strides as above; out overlaps no
 *            input
 * bf16 runs on the tensor cores (fp32 scores, statistics and sums; the softmax
 * weights are rounded to bf16 for the product with the values); fp32 runs on the
 * CUDA cores in fp32.  A key or value outside a row's range (another sequence's,
 * a later token's) has no influence on it, NaN and infinities included.  If one
 * of the bf16 kernel's internal waits gives up (about 2 s: a stalled device), the
 * rows that it had still to write are NaN.
 * Enqueues and returns; MFS_E_ARG on bad sizes, strides, alignment or NULL. */
int mfs_prompt_attention(int dtype, int n_tokens, int n_seqs, const int32_t* cu, const void* q, long long q_stride,
                         int n_q_heads, const void* k, long long k_stride, const void* v, long long v_stride,
                         int n_kv_heads, int head_dim, void* out, long long out_stride, float scale, int window,
                         void* cuda_stream);

#ifdef __cplusplus
}
#endif
#endif /* MFS_H */
