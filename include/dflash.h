/*
 * dflash.h - C ABI of the DFlash drafter block step on one GB300 (sm_103a).
 *
 * The drafter is the block-diffusion draft model of DFlash speculative decoding
 * as the dflash-ops model card describes it (sections "Usage" and "Method") and
 * as dflash_head.rs lays out its weights (struct DflashLayer, struct
 * BlockDiffusionDraftHead): a few Qwen3-style layers that denoise a 16-token
 * block [anchor, mask x 15] in one non-causal forward, attending a per-layer
 * sliding-window ring of K/V injected from fused target-model features.
 *
 * Conventions for every entry point:
 *   - Pointers marked "device" are CUDA device pointers; "host" pointers are
 *     ordinary process memory.  All device memory is owned by the caller and
 *     only borrowed by the library: weights, the ring, the scratch area and
 *     every input and output buffer must stay alive while a handle or a
 *     captured graph that names them can run.
 *   - `stream` is a cudaStream_t passed as void*; NULL means the legacy default
 *     stream.  Every call except dflash_create, dflash_read_status and
 *     dflash_step_host is asynchronous on that stream.
 *   - Matrices are row-major.  A weight W[out][in] computes y = x W^T.
 *   - Return value: DFLASH_OK (0) or a negative dflash_status.  Host-side
 *     checks run before anything is enqueued, so an error return means no
 *     work was launched.  DFLASH_ERR_CUDA keeps the CUDA error text in the
 *     handle (dflash_last_error).  No C++ exception crosses this boundary.
 *   - dflash_step and dflash_accept never allocate memory, never synchronise
 *     and never read device data on the host, so they can be captured in a
 *     CUDA graph (dflash_capture does exactly that).
 */
#ifndef DFLASH_H
#define DFLASH_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Symbols of the library are exported explicitly (it is built with hidden
 * default visibility). */
#if defined(__GNUC__)
#define DFLASH_API __attribute__((visibility("default")))
#else
#define DFLASH_API
#endif

/* Rows of one noise block: the anchor token then 15 mask tokens
 * (dflash-ops model card, Method; the block size of the shipped drafter). */
#define DFLASH_BLOCK 16
/* Largest number of drafter layers a handle accepts (the shipped drafter has 5). */
#define DFLASH_MAX_LAYERS 16

typedef enum {
  DFLASH_OK = 0,
  DFLASH_ERR_INVALID_ARG = -1,   /* null pointer, negative size, bad enum value */
  DFLASH_ERR_UNSUPPORTED = -2,   /* geometry or dtype mix the library does not run */
  DFLASH_ERR_TOO_MANY_ROWS = -3, /* T > window, or T > max_inject */
  DFLASH_ERR_SEQ_RANGE = -4,     /* sequence index or n_seq outside [0, max_seq) */
  DFLASH_ERR_CUDA = -5,          /* a CUDA runtime call failed; see dflash_last_error */
  DFLASH_ERR_NOT_CAPTURED = -6,  /* dflash_replay before dflash_capture */
  DFLASH_ERR_DEVICE = -7         /* device status word non-zero (dflash_read_status) */
} dflash_status;

typedef enum {
  DFLASH_DTYPE_F32 = 0,
  DFLASH_DTYPE_BF16 = 1,
  DFLASH_DTYPE_FP8_E4M3 = 2,     /* E4M3 "fn" codes + one f32 scale per output row */
  /* E2M1 codes with one E4M3 scale per 16 weights of a row and one f32 scale per
   * row: w[n][k] = s[n] * e4m3(b[n][k/16]) * e2m1(q[n][k]).  A matrix [N][K] is
   * one buffer of N*K/2 code bytes (row-major) followed by N*K/16 block-scale
   * bytes; the row scales use the *_scale pointer.  Within each 16-byte group of
   * a row (32 weights) byte 4t + j holds the codes of k = 2(t + 4j) (low nibble)
   * and k + 1 (high nibble), t, j = 0..3.  Projection weights only
   * (q/k/v/o/gate/up/down, lm_head); every K (n_embd, n_head*head_dim, n_ff) a
   * multiple of 256.  The products run in fp16 against an fp16 hi/lo activation
   * pair (exact weights, activations to 2^-22 relative), so projection inputs
   * must stay below 65504 in magnitude.  dflash_head.rs (field lm_head_nvfp4)
   * names an NVFP4 LM head but not its layout: this one is the library's own. */
  DFLASH_DTYPE_FP4_E2M1 = 3
} dflash_dtype;

/* Bits of the device status word (dflash_read_status). */
#define DFLASH_DEV_BAD_TOKEN 0x1u     /* an id_last outside [0, n_vocab): clamped */
#define DFLASH_DEV_BAD_POSITION 0x2u  /* a negative inject position or n_past: row skipped */
#define DFLASH_DEV_TIMEOUT 0x4u       /* a pipeline wait gave up after ~2 s: outputs invalid */
/* Bits of a cache handle's status word (dflash_cache_read_status; with BAD_POSITION
 * and TIMEOUT above). */
#define DFLASH_DEV_BAD_ROWS 0x8u      /* row_start, a row count or a length out of range: sequence skipped */
#define DFLASH_DEV_BAD_PAGE 0x10u     /* a page that is missing, out of range or (for a write) shared */
#define DFLASH_DEV_BAD_TREE 0x20u     /* a parent that is not an earlier node, or a path that is not ascending */
#define DFLASH_DEV_BAD_SEQ 0x40u      /* a sequence out of range, listed twice, or not empty where it has to be */
#define DFLASH_DEV_NO_PAGES 0x80u     /* dflash_cache_reserve found too few pages: nothing was changed */

/*
 * Drafter geometry and storage formats.
 *   n_layer <= DFLASH_MAX_LAYERS; n_head % n_head_kv == 0;
 *   head_dim in {32, 64, 128} (a multiple of 32 as the model card requires, and
 *   a divisor of the 128-row output tile of the projection kernels);
 *   n_embd, n_head*head_dim, n_ff and n_target_layers*target_embd multiples of 32.
 *   weight_dtype: q/k/v/o/gate/up/down and lm_head (F32, BF16 or FP8_E4M3);
 *   dense_dtype: tok_embd, fc, every norm weight and the target features
 *   (F32 or BF16); ring_dtype: ring K/V (F32 or BF16).
 *   max_seq: sequences (rings) the handle serves; max_inject: the largest row
 *   count of one dflash_encode / dflash_inject call (inject also needs
 *   T <= window: slots are pos % window, dflash-ops model card, Requirements).
 *   mask_token_id: token of block rows 1..15 (dflash_head.rs field mask_token_id).
 *   eps: RMSNorm epsilon (1e-6 in dflash_head.rs); rope_theta: rope base.
 */
typedef struct {
  int32_t n_layer;
  int32_t n_embd;
  int32_t n_head;
  int32_t n_head_kv;
  int32_t head_dim;
  int32_t n_ff;
  int32_t window;
  int32_t n_vocab;
  int32_t n_target_layers;
  int32_t target_embd;
  int32_t max_seq;
  int32_t max_inject;
  int32_t mask_token_id;
  int32_t weight_dtype;
  int32_t dense_dtype;
  int32_t ring_dtype;
  float eps;
  int32_t reserved0;
  double rope_theta;
} dflash_config;

/* One layer's device weights (dflash_head.rs, struct DflashLayer):
 *   attn_norm [n_embd], q_norm [head_dim], k_norm [head_dim], ffn_norm [n_embd]
 *     in dense_dtype;
 *   wq [n_head*head_dim][n_embd], wk and wv [n_head_kv*head_dim][n_embd],
 *   wo [n_embd][n_head*head_dim], gate and up [n_ff][n_embd], down [n_embd][n_ff]
 *     in weight_dtype;
 *   *_scale: f32 per output row, read only when weight_dtype is FP8_E4M3. */
typedef struct {
  const void* attn_norm;
  const void* wq;
  const void* wk;
  const void* wv;
  const void* wo;
  const void* q_norm;
  const void* k_norm;
  const void* ffn_norm;
  const void* gate;
  const void* up;
  const void* down;
  const float* wq_scale;
  const float* wk_scale;
  const float* wv_scale;
  const float* wo_scale;
  const float* gate_scale;
  const float* up_scale;
  const float* down_scale;
} dflash_layer_weights;

/* Model-level device weights:
 *   tok_embd [n_vocab][n_embd] dense_dtype and lm_head [n_vocab][n_embd]
 *     weight_dtype, both borrowed from the target model (dflash-ops model card,
 *     Usage); lm_head_scale f32 [n_vocab] for FP8;
 *   fc [n_embd][n_target_layers*target_embd], hidden_norm [n_embd],
 *   out_norm [n_embd] in dense_dtype (dflash_head.rs fields fc, hidden_norm, norm). */
typedef struct {
  const void* tok_embd;
  const void* lm_head;
  const float* lm_head_scale;
  const void* fc;
  const void* hidden_norm;
  const void* out_norm;
  dflash_layer_weights layers[DFLASH_MAX_LAYERS];
} dflash_weights;

typedef struct dflash_handle dflash_handle;

/*
 * Sizes of the two caller-owned device areas a handle needs.
 *   ring_bytes: K and V rings, [max_seq][n_layer][2][n_head_kv][window][head_dim]
 *     in ring_dtype, followed by ring_pos int32 [max_seq][window] (the position
 *     each slot holds, -1 when empty; one array per sequence, shared by layers).
 *   scratch_bytes: every intermediate of inject and step (activations, split-K
 *     partial sums, rope tables, counters, the status word).
 * Both areas must be 256-byte aligned.  Returns INVALID_ARG / UNSUPPORTED for a
 * bad configuration.
 */
DFLASH_API int dflash_workspace_size(const dflash_config* cfg, size_t* ring_bytes, size_t* scratch_bytes);

/*
 * Build a handle: validate the configuration, compute the host fp64 rope
 * inverse-frequency table theta^(-2j/head_dim) (dflash-ops model card, Method),
 * copy it into scratch, clear counters and the status word, zero the ring K/V
 * and mark every ring slot empty (ring_pos = -1).  Synchronous.  `w` is copied (the pointer
 * values, not the weights).  ring_mem and scratch_mem are device areas of at
 * least the dflash_workspace_size sizes.  On success *out receives the handle.
 */
DFLASH_API int dflash_create(const dflash_config* cfg, const dflash_weights* w, void* ring_mem,
                  void* scratch_mem, dflash_handle** out);

/* Free the handle's host state and its captured graph (not the borrowed memory). */
DFLASH_API void dflash_destroy(dflash_handle* h);

/*
 * Encode target features (dflash-ops model card, Usage: m.encode(target_features);
 * dflash_engine.py, class TargetContextFeatureFuser):
 *   H_t = RMSNorm(feats fc^T) * hidden_norm.
 *   feats: device [T][n_target_layers*target_embd] in dense_dtype;
 *   H_t:   device f32 [T][n_embd] (caller buffer, written).
 *   0 <= T <= max_inject (TOO_MANY_ROWS otherwise); T = 0 is a no-op.
 */
DFLASH_API int dflash_encode(dflash_handle* h, const void* feats, int32_t T, float* H_t, void* stream);

/*
 * dflash_encode for callers that cannot allocate device memory.  No page
 * defines this call; it exists for code that may not call cudaMalloc (an
 * allocator-free runtime, a plug-in limited to the buffers it is handed, a host
 * whose device memory is all owned by a pool) and therefore cannot provide the
 * scratch area dflash_create needs.  It computes exactly what dflash_encode
 * computes with the same kernels, without a handle:
 *   cfg:        geometry (n_embd, n_target_layers, target_embd, dense_dtype, eps;
 *               other fields are not read);
 *   fc:         device [n_embd][n_target_layers*target_embd], dense_dtype;
 *   hidden_norm: device [n_embd], dense_dtype;
 *   feats:      device [T][n_target_layers*target_embd], dense_dtype;
 *   H_t:        device f32 [T][n_embd], written (it also holds the intermediate
 *               un-normalised projection during the call).
 * Its intermediate memory is one 8 MiB file-scope __device__ array that every
 * GPU loading this library holds until the process exits.  Limits: with
 * tiles = ceil(n_embd / 128), tiles * ceil(T / 16) <= 16384 and
 * tiles * T <= 835,584 (T <= 5040 at n_embd 6656); larger calls return
 * DFLASH_ERR_TOO_MANY_ROWS and launch nothing.  The first call on a device looks
 * up the array's device address and sets kernel attributes for that device
 * (the device current at the call); make that first call before any stream
 * capture.  Nothing is allocated or freed, by this library or any library it
 * calls.  All calls share the array: calls that overlap on the GPU (on
 * different streams, or from different threads) race; it is cleared where it
 * must start at zero at the start of every call.  Asynchronous on `stream`.
 * There is no handle to hold an error text: DFLASH_ERR_CUDA from this call
 * carries no further detail (the runtime's own cudaGetLastError does).  The
 * runtime's last-error slot is cleared on entry, so an error left by earlier
 * unrelated work is not reported as this call's.
 */
DFLASH_API int dflash_encode_noalloc(const dflash_config* cfg, const void* fc, const void* hidden_norm,
                                     const void* feats, int32_t T, float* H_t, void* stream);

/*
 * Inject encoded rows into sequence `seq`'s ring (dflash-ops model card, Method
 * and Requirements): for every layer l and row t,
 *   K = rope(RMSNorm_head(H_t[t] wk_l^T) * k_norm_l, pos[t]),  V = H_t[t] wv_l^T,
 *   both rounded once to ring_dtype and stored at slot pos[t] % window, and
 *   ring_pos[slot] = pos[t].  No attn_norm is applied to H_t.
 *   H_t: device f32 [T][n_embd]; pos: device int32 [T], non-negative and
 *   distinct modulo window (contiguous positions are).  0 <= T <= min(window,
 *   max_inject); seq in [0, max_seq).  A negative position sets
 *   DFLASH_DEV_BAD_POSITION and its row is skipped.
 */
DFLASH_API int dflash_inject(dflash_handle* h, int32_t seq, const float* H_t, const int32_t* pos,
                  int32_t T, void* stream);

/*
 * Block width of the following steps, accepts, loop turns and captures
 * (dflash_head.rs, set_block_g: the scheduler's narrower block of the anchor
 * plus num_drafts mask rows, clamped to 2..16; its propose graphs are keyed by
 * width because a capture bakes its row count).  With width B the block holds
 * rows 0..B-1 at positions n_past .. n_past+B-1 ([id_last, mask x (B-1)]),
 * every row attends to the B block keys (and the ring); drafts j >= B-1 are
 * written as -1; logits rows >= B are computed but are not part of the result;
 * accept and advance count at most B-1 drafts.  dflash_capture and
 * dflash_capture_loop store one graph per width, and dflash_replay launches
 * the current width's graph.  2 <= width <= 16 (INVALID_ARG otherwise, or
 * while a capture is running).  Default 16.
 */
DFLASH_API int dflash_set_block_width(dflash_handle* h, int32_t width);

/*
 * Projection chains (off by default).  With chains on, a step of fewer than
 * 128 block rows with bf16, fp32 or E4M3 weights runs, per layer, one
 * persistent launch for o, gate/up, down and the next layer's q/k/v (the LM
 * head after the last layer) instead of four (dflash-ops model card,
 * Requirements and limits: the whole-block megakernel is the named next step;
 * this is its projection part).  Its CTAs wait for one another's output tiles
 * (bounded waits that end in DFLASH_DEV_TIMEOUT), which needs the whole grid
 * resident at once: keep chains off when other work may hold SMs for the
 * duration of a step (a GPU shared through MPS or partitioned contexts).
 * Results are bitwise identical either way; on a GB300 the chained step is not
 * faster (every tile of a stream-K phase completes near the phase's end, so the
 * next phase starts no earlier than after a kernel boundary with programmatic
 * dependent launch).  enable = 0 or 1; UNSUPPORTED when enabling on a handle
 * without chains (FP4 or E4M3 weights, or a device that cannot hold the grid);
 * INVALID_ARG during a capture.  Takes effect for later steps and captures.
 */
DFLASH_API int dflash_set_chain(dflash_handle* h, int32_t enable);

/*
 * The attention kernel a step of n_seq sequences runs (the choice is
 * automatic; this reports it for tests and benchmarks): 0 = split window (the
 * window of every (sequence, kv head) in 128-slot CTAs that the GPU holds at
 * once, merged through global scratch), 1 = clusters (a kv head's window over
 * up to 8 CTAs of a cluster, merged through distributed shared memory), 2 =
 * stream-K (one CTA per SM streaming equal ranges of all windows through a
 * double-buffered TMA pipeline; windows cut by a range merge their partials).
 * Returns the kind, INVALID_ARG for a null handle, SEQ_RANGE for n_seq outside
 * 1..max_seq.
 */
DFLASH_API int dflash_attention_kernel(const dflash_handle* h, int32_t n_seq);

/*
 * One block step for sequences 0..n_seq-1 (dflash-ops model card, Usage:
 * step(id_last, n_past) -> logits [16, n_vocab]; drafts = argmax of rows 1..15).
 *   id_last: device int32 [n_seq], the anchor token of each block;
 *   n_past:  device int32 [n_seq], position of block row 0 (rows sit at
 *            n_past .. n_past+15; ring slots holding positions p with
 *            0 <= p < n_past and n_past + i - p < window are row i's keys;
 *            all 16 block rows are keys of every row);
 *   logits:  device f32 [n_seq][16][n_vocab] (written), or NULL to skip storing
 *            them (drafts are still computed);
 *   drafts:  device int32 [n_seq][15], argmax of block rows 1..15, ties to the
 *            lowest token id (written).
 * 1 <= n_seq <= max_seq.  Scalars are read on the device, so a captured graph
 * replays with new id_last / n_past contents.
 */
DFLASH_API int dflash_step(dflash_handle* h, int32_t n_seq, const int32_t* id_last, const int32_t* n_past,
                float* logits, int32_t* drafts, void* stream);

/*
 * First-mismatch acceptance scan on the device (dflash-ops model card, Usage:
 * n_ok = m.accept(drafts, target_tokens); dflash_engine.py,
 * DFlashSpeculativeVerifier.verify_block): n_ok[s] = the number of leading
 * j in 0..14 with drafts[s][j] == targets[s][j] (15 when all agree).
 *   drafts, targets: device int32 [n_seq][15]; n_ok: device int32 [n_seq].
 */
DFLASH_API int dflash_accept(dflash_handle* h, int32_t n_seq, const int32_t* drafts, const int32_t* targets,
                  int32_t* n_ok, void* stream);

/*
 * Capture dflash_step (and dflash_accept when targets and n_ok are non-NULL)
 * with these exact pointers into a CUDA graph owned by the handle (dflash-ops
 * model card, Method: the captured step allocates nothing, so eager work may
 * run between replays).  Capture runs on an internal stream; nothing is
 * launched.  `stream` orders the capture after earlier work on it.
 * Replaces a previous dflash_capture of the current block width (a loop-turn
 * graph of dflash_capture_loop is kept separately and is not affected).
 */
DFLASH_API int dflash_capture(dflash_handle* h, int32_t n_seq, const int32_t* id_last, const int32_t* n_past,
                   float* logits, int32_t* drafts, const int32_t* targets, int32_t* n_ok,
                   void* stream);

/* Launch the current width's dflash_capture graph on `stream` (NOT_CAPTURED if there is none). */
DFLASH_API int dflash_replay(dflash_handle* h, void* stream);

/*
 * Node counts of the current width's captured graph (loop = 0: dflash_capture,
 * loop != 0: dflash_capture_loop), host int32 outputs: kernel launches, memory
 * allocation or free nodes (always 0: nothing in a step allocates), and every
 * other node (memset nodes of profiling captures).  NOT_CAPTURED if there is no
 * such graph.
 */
DFLASH_API int dflash_graph_nodes(dflash_handle* h, int32_t loop, int32_t* kernels,
                                  int32_t* mem_alloc, int32_t* other);

/*
 * One turn of the speculative loop on the device, after the target model has
 * verified the block that the last dflash_step drafted (dflash_engine.py,
 * DFlashSpeculativeVerifier.verify_block: accepted prefix + one bonus token;
 * dflash-ops model card, Usage: inject(encode(features), positions) of the
 * verified positions, then the next step(id_last, n_past)).  Per sequence s:
 *   m = number of leading j in 0..14 with drafts[s][j] == targets[s][j];
 *   the target features of block rows 0..m (positions n_past[s] .. n_past[s]+m)
 *   are encoded and injected into sequence s's ring (rows m+1..15 are encoded
 *   but not written: their slots may still hold keys inside the window);
 *   n_ok[s] = m; id_last[s] = targets[s][m] (the target's own token after the
 *   accepted drafts: the correction, or the bonus token when m = 15);
 *   n_past[s] += m + 1.
 *   drafts:  device int32 [n_seq][15] (the previous step's drafts);
 *   targets: device int32 [n_seq][16], the target's greedy token at block rows
 *            0..15 (row j predicts position n_past + j + 1);
 *   feats:   device [n_seq][16][n_target_layers*target_embd] in dense_dtype,
 *            the target's features at block rows 0..15;
 *   id_last, n_past: device int32 [n_seq], read and updated in place;
 *   n_ok:    device int32 [n_seq], written.
 * Requires 16 * n_seq <= max_inject and window >= 16 (TOO_MANY_ROWS
 * otherwise).  Nothing is read back to the host, so the call can be captured
 * (dflash_capture_loop).  Asynchronous on `stream`.
 */
DFLASH_API int dflash_advance(dflash_handle* h, int32_t n_seq, const int32_t* drafts,
                              const int32_t* targets, const void* feats, int32_t* id_last,
                              int32_t* n_past, int32_t* n_ok, void* stream);

/*
 * Capture one whole loop turn - dflash_advance followed by dflash_step with
 * the updated id_last / n_past - into the handle's loop graph of the current
 * block width (replacing a previous loop capture of that width; a dflash_capture
 * graph is kept separately; dflash_replay_loop launches it).  With these exact pointers,
 * each replay consumes the target's tokens and features for the block drafted
 * by the previous replay (or step) and leaves the next block's logits and
 * drafts in `logits` / `drafts`.  Capture runs on an internal stream; nothing
 * is launched; `stream` orders the capture after earlier work on it.
 */
DFLASH_API int dflash_capture_loop(dflash_handle* h, int32_t n_seq, const int32_t* targets,
                                   const void* feats, int32_t* id_last, int32_t* n_past,
                                   int32_t* n_ok, float* logits, int32_t* drafts, void* stream);

/* Launch the current width's dflash_capture_loop graph on `stream` (NOT_CAPTURED if there is none). */
DFLASH_API int dflash_replay_loop(dflash_handle* h, void* stream);

/*
 * The same step as dflash_step, driven from host memory: copies id_last and
 * n_past (host int32 [n_seq]) to the device, runs the step into internal
 * scratch buffers, copies the drafts back to host int32 [n_seq][15] (and the
 * logits to host f32 [n_seq][16][n_vocab] when `logits` is non-NULL), and waits
 * for `stream`.  Host buffers may be pageable or pinned.
 */
DFLASH_API int dflash_step_host(dflash_handle* h, int32_t n_seq, const int32_t* id_last,
                     const int32_t* n_past, float* logits, int32_t* drafts, void* stream);

/* Zero sequence `seq`'s ring K/V and mark every slot empty (ring_pos = -1), on `stream`. */
DFLASH_API int dflash_ring_reset(dflash_handle* h, int32_t seq, void* stream);

/*
 * Read and clear the device status word (DFLASH_DEV_* bits) after waiting for
 * `stream`.  Synchronous.  Returns DFLASH_ERR_DEVICE when a bit was set.
 */
DFLASH_API int dflash_read_status(dflash_handle* h, uint32_t* status, void* stream);

/*
 * Profiling.  dflash_profile_enable(h, mode): 0 off; 1 launch-class events on
 * eager calls; 2 device timestamps of every step launch.
 *
 * Mode 1 (eager calls, not captured graphs): every kernel launch of
 * dflash_step / dflash_encode / dflash_inject / dflash_accept is bracketed by
 * CUDA events recorded on the launching stream.
 * dflash_profile_read waits for those events, writes the summed device time in
 * milliseconds and the launch count of each class (arrays of DFLASH_PROF_N
 * entries, host memory) and clears the record.  Classes: 0 embedding + rope
 * table, 1 q/k/v projection, 2 attention chunks, 3 attention merge, 4 o
 * projection, 5 gate/up projection, 6 down projection, 7 LM head + drafts,
 * 8 encode (fc + norm), 9 injection (rope table + wk/wv + ring scatter),
 * 10 acceptance scan, 11 projection chain (one launch of o, gate/up, down and
 * the next layer's q/k/v or the LM head: steps of fewer than 128 block rows
 * with bf16, fp32 or E4M3 weights).  Enabling while a capture is in progress
 * is refused.
 */
#define DFLASH_PROF_N 12
DFLASH_API int dflash_profile_enable(dflash_handle* h, int enable);
DFLASH_API int dflash_profile_read(dflash_handle* h, double* ms, int32_t* launches);

/*
 * Mode 2: every kernel of a step (and of the acceptance scan of dflash_capture)
 * records the %globaltimer of its first CTA's start and of its last CTA's end
 * in a scratch slot, from eager calls and from graphs captured while mode 2 is
 * on (such a graph also zeroes the slots with one memset node ahead of the
 * step); the kernels, their order and their launch attributes are those of the
 * unprofiled step.  dflash_profile_stamps waits for `stream`, then writes, for
 * the launches of the last recorded step in launch order (at most `max`), the
 * class (as in mode 1) and the start and end in microseconds relative to the
 * earliest start (-1 for a launch that has not run), and their count to *n
 * (host arrays).  Synchronous.
 */
DFLASH_API int dflash_profile_stamps(dflash_handle* h, int32_t max, int32_t* cls, double* start_us,
                                     double* end_us, int32_t* n, void* stream);

/* Text of a dflash_status code (static storage). */
DFLASH_API const char* dflash_status_string(int status);

/* Text of the last CUDA error recorded in the handle ("" if none). */
DFLASH_API const char* dflash_last_error(const dflash_handle* h);

/* ------------------------------------------------------------------------- *
 * The target model's side: rotary positions, attention of a tree of drafted
 * tokens over a paged cache, acceptance along the tree, and the cache's pages.
 *
 * The drafter's block (or a tree made of several drafts) is verified by the
 * target model in one forward (dflash_engine.py, DFlashSpeculativeVerifier;
 * dflash_head.rs names the engine's paged K/V cache and its block tables).
 * One turn of a layer stack over a batch of trees:
 *
 *   dflash_cache_reserve    room for the trees behind each sequence
 *   dflash_tree_mask        parents -> ancestor masks and depths (once a turn)
 *   per layer: dflash_cache_append   rotate q and k, put k and v into the pages
 *              dflash_tree_attend    every node over its sequence and ancestors
 *   dflash_tree_accept      the path the target agrees with, and its next token
 *   dflash_cache_commit     the path's keys and values moved together
 *
 * and dflash_cache_fork / dflash_cache_trim share and release pages.  None of
 * these calls (dflash_cache_create, _destroy and _read_status apart) allocates,
 * synchronises or reads device data on the host, so all can be captured in a
 * CUDA graph; lengths and the page table live on the device.
 *
 * Rows.  A call works on T rows of n_seq sequences: rows row_start[s] ..
 * row_start[s+1] - 1 (device int32 [n_seq + 1], ascending, within 0..T) are
 * nodes 0.. of entry s.  Entry s is sequence seqs[s] of the cache (device int32
 * [n_seq]; NULL: sequence s).  Node i of a sequence of length n occupies slot
 * n + i.  Rows outside every range are not written, and what they hold (of q, k
 * and v, which a call may load whole) does not matter.  An entry whose range is
 * not within 0..T, or whose sequence is out of range, is skipped and sets a status
 * bit, as does every other fault that only the device can see; no such fault makes
 * a kernel read or write outside the handle's memory and the buffers of the call.
 * Where a call changes the cache (append, commit, trim, reserve), only the first
 * entry of a sequence that is listed twice is used (BAD_SEQ).
 *
 * The calls of one handle share its scratch area and change its state: they
 * must not overlap on the GPU (one stream, or streams ordered by events; the
 * same holds for two graphs captured from one handle).  Different handles are
 * independent.  A call uses the device its pages lie on, whichever is current.
 * ------------------------------------------------------------------------- */

/* Most nodes of a tree that has a mask, and most entries of one call. */
#define DFLASH_MAX_TREE 1024
#define DFLASH_MAX_CALL_SEQ 1024

typedef enum {
  DFLASH_ROPE_HALF = 0,         /* pair j: dims j and rotary_dim / 2 + j of a head */
  DFLASH_ROPE_INTERLEAVED = 1   /* pair j: dims 2j and 2j + 1 */
} dflash_rope_layout;

/* Angle of pair j at position p is p f_j with, for r = rotary_dim and F =
 * rope_factor:
 *   NONE    f_j = theta^(-2j/r)
 *   LINEAR  f_j = theta^(-2j/r) / F
 *   NTK     f_j = (theta F^(r/(r-2)))^(-2j/r)                         (r > 2)
 *   YARN    f_j = theta^(-2j/r) (w_j / F + 1 - w_j), w_j a ramp from 0 to 1
 *           between pairs lo and hi: w_j = clamp((j - lo) / max(hi - lo, 1e-3)),
 *           lo = max(floor(d(beta_fast)), 0), hi = min(ceil(d(beta_slow)), r - 1),
 *           d(b) = r ln(orig_positions / (2 pi b)) / (2 ln theta).
 * Rotated values are multiplied by rope_mscale (0: 0.1 ln F + 1 for YARN with
 * F > 1, else 1). */
typedef enum {
  DFLASH_ROPE_NONE = 0,
  DFLASH_ROPE_LINEAR = 1,
  DFLASH_ROPE_NTK = 2,
  DFLASH_ROPE_YARN = 3
} dflash_rope_scaling;

/*
 * Geometry of a cache handle.
 *   head_dim in {32, 64, 128}; n_head % n_head_kv == 0; page_size a power of two
 *   in 16..256; max_seq <= 4096 sequences, each of at most max_pages pages
 *   (max_pages * page_size <= 2^31 - 1024); n_pages * n_layer * 2 * n_head_kv < 2^31;
 *   dtype F32 or BF16: pages, queries, keys, values and outputs;
 *   rotary_dim: rotated dims of each head, a multiple of 8 in 0..head_dim;
 *   rope_theta > 1, rope_factor >= 1 (both read only with rotary_dim > 0);
 *   attn_scale >= 0: factor of the scores (0: 1 / sqrt(head_dim)).
 */
typedef struct {
  int32_t n_layer;
  int32_t n_head;
  int32_t n_head_kv;
  int32_t head_dim;
  int32_t page_size;
  int32_t n_pages;
  int32_t max_seq;
  int32_t max_pages;
  int32_t dtype;
  int32_t rope_layout;
  int32_t rotary_dim;
  int32_t rope_scaling;
  int32_t rope_orig_positions;
  float rope_factor;
  float rope_beta_fast;
  float rope_beta_slow;
  float rope_mscale;
  float attn_scale;
  double rope_theta;
} dflash_cache_config;

typedef struct dflash_cache dflash_cache;

/*
 * Sizes of the three caller-owned device areas of a cache handle (256-byte
 * aligned):
 *   page_bytes: pages[n_pages][n_layer][k, v][n_head_kv][page_size][head_dim] in
 *     dtype (slot p of a sequence: row p % page_size of its page p / page_size);
 *   state_bytes: int32 table[max_seq][max_pages] (-1: no page), then int32
 *     length[max_seq], then int32 refs[n_pages] (sequences that hold the page;
 *     0: free), each starting at a multiple of 256 bytes.  A caller may read and
 *     set them between calls;
 *   scratch_bytes: the library's own.
 */
DFLASH_API int dflash_cache_workspace_size(const dflash_cache_config* cfg, size_t* page_bytes,
                                           size_t* state_bytes, size_t* scratch_bytes);

/* Build a cache handle over those areas: every sequence empty, every page free
 * (the pages' contents are left as they are).  Synchronous, after all work that the
 * device has so far: the areas may be memory that some of it still uses. */
DFLASH_API int dflash_cache_create(const dflash_cache_config* cfg, void* page_mem, void* state_mem,
                                   void* scratch_mem, dflash_cache** out);

/* Free the handle's host state (not the borrowed memory). */
DFLASH_API void dflash_cache_destroy(dflash_cache* c);

/*
 * Rotary positions of n_heads heads per row, or their gradient:
 *   out[t][h] = R(pos[t]) x[t][h], or R(pos[t])^T x[t][h] when backward != 0
 * (with out = R x, dx = R^T dout), dims from rotary_dim on copied.
 *   x, out: device [T][n_heads][head_dim] in dtype with row strides x_stride and
 *   out_stride in elements (a head's dims and a row's heads are contiguous), both
 *   16-byte aligned with strides that are multiples of 16 bytes; out may be x.
 *   pos: device int32 [T].  A negative position sets DFLASH_DEV_BAD_POSITION and
 *   its row is not written.
 */
DFLASH_API int dflash_rope(dflash_cache* c, int32_t T, int32_t n_heads, const void* x, int64_t x_stride,
                           const int32_t* pos, void* out, int64_t out_stride, int32_t backward,
                           void* stream);

/*
 * Put T rows' keys and values of one layer into the pages, keys rotated, and
 * rotate their queries: row i of entry s has position n + depth (depth NULL: n +
 * i), n the sequence's length, and goes to slot n + i.  Lengths do not change
 * (dflash_cache_commit adds the rows that stay).
 *   k, v: device [T][n_head_kv][head_dim]; q, q_out: device [T][n_head][head_dim],
 *   or both NULL; q_out may be q.  Strides and alignment as for dflash_rope.
 *   depth: device int32 [T] (dflash_tree_mask) or NULL.
 * A slot without a page, or whose page other sequences hold too
 * (dflash_cache_reserve makes it private), sets DFLASH_DEV_BAD_PAGE and its key
 * and value are not written; a negative position is skipped with
 * DFLASH_DEV_BAD_POSITION.
 */
DFLASH_API int dflash_cache_append(dflash_cache* c, int32_t layer, int32_t n_seq, const int32_t* seqs,
                                   const int32_t* row_start, int32_t T, const int32_t* depth,
                                   const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride,
                                   const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                   void* stream);

/*
 * Ancestor masks of trees given by parents: bit j of mask[t] is set when node j
 * is row t's node or one of its ancestors; depth[t] counts the proper ancestors.
 *   parents: device int32 [T], the parent's node index within the row's own tree
 *   (an earlier node), or -1 for a root: a chain of B tokens has parents i - 1;
 *   mask: device uint32 [T][mask_words], mask_words in 1..32 (bits from the
 *   entry's node count on are zero); depth: device int32 [T] or NULL.
 * A parent that is neither -1 nor an earlier node counts as -1 and sets
 * DFLASH_DEV_BAD_TREE; an entry of more than 32 mask_words nodes is skipped with
 * DFLASH_DEV_BAD_ROWS.
 */
DFLASH_API int dflash_tree_mask(dflash_cache* c, int32_t n_seq, const int32_t* row_start, int32_t T,
                                const int32_t* parents, uint32_t* mask, int32_t mask_words,
                                int32_t* depth, void* stream);

/*
 * Attention of T rows over their sequences' pages: node i of an entry of length
 * n attends to slots 0 .. n-1 and to those slots n + j, j < the entry's node
 * count, whose bit j of mask is set (mask NULL: j <= i, a causal chain of any
 * length, e.g. a prompt):
 *   out[t][h] = sum_p w_p V[p], w = softmax over the attended slots of
 *   attn_scale q[t][h] . K[p], head h reading key/value head h / (n_head / n_head_kv);
 *   lse[t][h] = ln of the sum of exp of the scores.
 * A row that attends to nothing gets out 0 and lse -inf.  What slots past the
 * last node hold does not matter; an infinite or NaN value of a node may reach
 * every row of its entry, whether the row attends to it or not.
 * Weighted values are summed in fp32 relative to a reference that need not be the
 * largest score: values of magnitude up to 2^56 give finite results.  Scores, weights
 * and their sum are fp32; for the product with V bf16 heads of 64 and 128 round each
 * weight to bf16 once more (up to 2^-8 of it, independently of one another), bf16 heads
 * of 32 keep 16 bits of it, f32 all.
 *   max_tree: an upper bound of the entries' node counts (<= 32 mask_words with a
 *   mask); an entry of more is skipped with DFLASH_DEV_BAD_ROWS.
 *   q, out: device [T][n_head][head_dim], strides and alignment as for
 *   dflash_rope (out must not overlap q); lse: device f32 [T][n_head] or NULL.
 * A missing page sets DFLASH_DEV_BAD_PAGE; the entry's outputs are then
 * unspecified.
 */
DFLASH_API int dflash_tree_attend(dflash_cache* c, int32_t layer, int32_t n_seq, const int32_t* seqs,
                                  const int32_t* row_start, int32_t T, int32_t max_tree,
                                  const uint32_t* mask, int32_t mask_words, const void* q,
                                  int64_t q_stride, void* out, int64_t out_stride, float* lse,
                                  void* stream);

/*
 * Greedy acceptance along trees (the tree form of dflash_accept): node 0 is the
 * anchor, always accepted; after an accepted node i follows its child of lowest
 * index whose token equals targets[row of i], until there is none or the path
 * holds max_path nodes.
 *   parents (as for dflash_tree_mask; a bad one is never reached), tokens (the
 *   nodes' drafted tokens), targets (the target model's greedy token after each
 *   node): device int32 [T];
 *   path: device int32 [n_seq][max_path], the accepted nodes, ascending, -1 behind
 *   them; n_path: device int32 [n_seq], their number (0 for an entry without
 *   rows); id_last: device int32 [n_seq], the target's token after the last
 *   accepted node (unchanged for an entry without rows).
 */
DFLASH_API int dflash_tree_accept(dflash_cache* c, int32_t n_seq, const int32_t* row_start, int32_t T,
                                  const int32_t* parents, const int32_t* tokens, const int32_t* targets,
                                  int32_t* path, int32_t max_path, int32_t* n_path, int32_t* id_last,
                                  void* stream);

/*
 * Keep an accepted path: in every layer the keys and values of slots n +
 * path[s][j] move to slots n + j, j < n_path[s] (all read before they are
 * overwritten), and the sequence's length becomes n + n_path[s].
 *   path: device int32 [n_seq][max_path], strictly ascending node indices (entry j
 *   at least j), or NULL: nodes 0 .. n_path[s] - 1 stay where they are (a prompt
 *   or a chain).  An entry with a path that is not so, or with slots that have no
 *   private page (a fork after the reserve shares the part-filled one), is skipped
 *   (BAD_TREE, BAD_PAGE).
 */
DFLASH_API int dflash_cache_commit(dflash_cache* c, int32_t n_seq, const int32_t* seqs,
                                   const int32_t* path, int32_t max_path, const int32_t* n_path,
                                   void* stream);

/*
 * Make slots n .. n + count[s] - 1 of every entry ready to write: missing pages
 * are given out, and a part-filled last page that other sequences hold too is
 * replaced by a private copy of its slots below n (the last of its holders keeps
 * it).  Free pages are given out in ascending order to the entries in their
 * order.  If there are too few, or an entry would pass max_pages, nothing is
 * changed and DFLASH_DEV_NO_PAGES is set.  A negative count counts as 0
 * (BAD_ROWS).
 */
DFLASH_API int dflash_cache_reserve(dflash_cache* c, int32_t n_seq, const int32_t* seqs,
                                    const int32_t* count, void* stream);

/*
 * Fork: sequence dst[i] becomes a copy of sequence src[i] that shares its pages
 * (nothing is copied until dflash_cache_reserve).  src, dst: device int32 [n].
 * An entry whose dst is not empty (dflash_cache_trim to 0), is listed twice or is
 * a source of the same call is skipped (BAD_SEQ).
 */
DFLASH_API int dflash_cache_fork(dflash_cache* c, int32_t n, const int32_t* src, const int32_t* dst,
                                 void* stream);

/*
 * Cut every entry's sequence to at most new_len[s] tokens and release its pages
 * behind slot new_len[s] - 1, reserved ones too; 0 frees the sequence.  A page is
 * free once no sequence holds it.  A negative new_len is skipped (BAD_ROWS).
 */
DFLASH_API int dflash_cache_trim(dflash_cache* c, int32_t n_seq, const int32_t* seqs,
                                 const int32_t* new_len, void* stream);

/* Read and clear the handle's device status word after waiting for `stream`.
 * Synchronous.  Returns DFLASH_ERR_DEVICE when a bit was set. */
DFLASH_API int dflash_cache_read_status(dflash_cache* c, uint32_t* status, void* stream);

/* Text of the last CUDA error recorded in the handle ("" if none). */
DFLASH_API const char* dflash_cache_last_error(const dflash_cache* c);

#ifdef __cplusplus
}
#endif

#endif /* DFLASH_H */
