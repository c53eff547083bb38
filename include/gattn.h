/*
 * gattn.h -- C ABI of the GB300 (sm_103a) gated full-attention layer library.
 *
 * One thing runs here: the Qwen3.5-family full-attention decoder layer at
 * decode and speculative-verify time, for B sequences of R new rows each
 * (R = q_len: 1..4 for decode and the pages' verify rows, up to 32 for wider
 * verify rows and short prefill chunks, with B*R <= 32):
 *
 *   q_full = Wq x  (doubled q_proj: per head h the rows [h*2d, h*2d+d) are the
 *                   query and [h*2d+d, (h+1)*2d) the output gate)
 *   k = Wk x,  v = Wv x
 *   q = RoPE(RMSNorm(query, q_norm)),  k = RoPE(RMSNorm(k, k_norm))
 *   cache[cache_pos + r] = bf16(k), bf16(v)
 *   attn = causal GQA softmax(q k^T / sqrt(d)) v over t <= cache_pos + r
 *   out = Wo (attn * sigmoid(gate))
 *
 * Sources: "feat(engine): stage D6 - qwen3_5 dense full-attn deltas" (Summary:
 * doubled q_proj -> split queries/gate -> o_proj(attn * sigmoid(gate)); Audit
 * table: partial_rotary_factor, has_qk_norm); Atlas "spark_model/forward/
 * qwen3_5/mod.rs" (Qwen35ForwardConfig, q_total = num_heads*head_dim*2,
 * LayerKvCache: caller pre-allocates, KV-append at cache_pos, attention over
 * cache_pos+1); DS4Server issue 113 "Reproduction and boundary" (the verify
 * head-chunk plan); TensorFold issue 503 "Option C" (generic affine row decoder,
 * 2-8 bit, groups 32/64/128).
 *
 * Optional parts, each on the same kernels: the decoder block around the layer
 * (input RMSNorm, residual add, post-attention RMSNorm: gattn_layer_step_block;
 * Atlas mod.rs module doc, FullAttentionLayer input_ln / post_ln), Turbo4
 * quantized caches (Bf16KTurbo4V and symmetric Turbo4: gattn_kv_register_turbo4v,
 * gattn_kv_register_turbo4; Atlas mod.rs MetalKvDtype, LayerKvCache) and
 * attention masks (gattn_layer_set_mask; DS4Server issue 113, broadcast and
 * head-specific masks of the verify route).
 *
 * Beside the layer stand operators without a handle, described where they are declared:
 * packed sequences (prompts and the gated delta rule) and caches in pages.
 *
 * Conventions for every entry point:
 *   - Pointers marked (device) are CUDA device addresses, (host) host memory.
 *   - Weights, caches, x, out and cache_pos are BORROWED: the library never
 *     frees them.  The library OWNS its handles, its repacked weights, its
 *     scratch and its TMA descriptors (freed by the matching destroy call).
 *   - A status other than GATTN_OK leaves a message for gattn_last_error()
 *     (thread-local, valid until the next call on the same thread).
 *   - Streams are cudaStream_t values passed as gattn_stream (0 = legacy default).
 *   - Inadmissible configurations are rejected at create time, never silently
 *     at step time.
 */
#ifndef GATTN_H
#define GATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *gattn_stream; /* same type as cudaStream_t */

typedef enum gattn_status {
    GATTN_OK = 0,
    GATTN_E_INVALID_ARG = 1,   /* null pointer, bad size, misaligned buffer */
    GATTN_E_UNSUPPORTED = 2,   /* admissible on the pages but not built here */
    GATTN_E_CUDA = 3,          /* a CUDA runtime/driver call failed */
    GATTN_E_DEVICE_RANGE = 4,  /* a kernel saw cache_pos + q_len > capacity */
    GATTN_E_STATE = 5,         /* call out of order (e.g. step before set_weights) */
    GATTN_E_DEVICE_TIMEOUT = 6 /* a bounded device wait gave up (kernel returned early) */
} gattn_status;

enum { GATTN_DTYPE_F32 = 0, GATTN_DTYPE_BF16 = 1 };
enum { GATTN_PROJ_Q = 0, GATTN_PROJ_K = 1, GATTN_PROJ_V = 2, GATTN_PROJ_O = 3 };

/*
 * Layer configuration (mirrors the config fields of Qwen35ForwardConfig).
 *   hidden                 Hd, width of x and out; Hd % 128 == 0 and Hd <= 16384
 *   num_heads, num_kv_heads H, Hk (H % Hk == 0, gqa = H / Hk; query head h uses KV head h / gqa);
 *                          H * d % 128 == 0 and H * d <= 16384
 *   head_dim               d; d % 64 == 0 and d <= 256 in this library
 *   partial_rotary_factor  prf in (0, 1]; rotary dims rd = trunc(d * prf), even and >= 2
 *   rope_theta             base of inv_freq_i = theta^(-2i/rd)
 *   rms_eps                QK-RMSNorm epsilon (inside the square root)
 *   bits, group_size       default code width {2,3,4,5,6,8} and group {32,64,128}
 *   proj_bits[4], proj_group[4]  per projection q,k,v,o; 0 = the default
 *   x_dtype                GATTN_DTYPE_F32 or GATTN_DTYPE_BF16 (out is always bf16)
 *   max_batch, max_q_len   upper bounds for step(); max_batch*max_q_len <= 32 (<= 16 for
 *                          fp32 x)
 *   head_chunk             1 = the verify head-chunk plan is on (the pages'
 *                          default), 0 = off; both routes give the same result
 */
typedef struct gattn_cfg {
    int32_t hidden;
    int32_t num_heads;
    int32_t num_kv_heads;
    int32_t head_dim;
    float partial_rotary_factor;
    float rope_theta;
    float rms_eps;
    int32_t bits;
    int32_t group_size;
    int32_t proj_bits[4];
    int32_t proj_group[4];
    int32_t x_dtype;
    int32_t max_batch;
    int32_t max_q_len;
    int32_t head_chunk;
} gattn_cfg;

/*
 * Packed affine weights of one projection in the interchange layout, all (device):
 *   packed  uint32 [N][K*bits/32]: row n is an LSB-first bitstream, code k at
 *           bits [k*bits, (k+1)*bits) of the row's little-endian words
 *   scales  bf16   [N][K/group]
 *   biases  bf16   [N][K/group]      weight = scale * code + bias
 * N x K: q = (2*H*d) x Hd, k = v = (Hk*d) x Hd, o = Hd x (H*d).
 */
typedef struct gattn_proj {
    const uint32_t *packed;
    const uint16_t *scales;
    const uint16_t *biases;
} gattn_proj;

typedef struct gattn_weights {
    gattn_proj proj[4];        /* q, k, v, o */
    const uint16_t *q_norm;    /* bf16 [d] (device) */
    const uint16_t *k_norm;    /* bf16 [d] (device) */
} gattn_weights;

/*
 * A caller-owned bf16 KV cache (device), element (b, kv_head, token, j) of K at
 *   k + b*stride_batch + kv_head*stride_head + token*stride_token + j
 * and the same for V (same strides).  Strides are in elements; each must be a
 * multiple of 8 (16 bytes) and the base pointers 16-byte aligned.
 * [B][Hk][cap][d] is stride_token = d, stride_head = cap*d, stride_batch = Hk*cap*d;
 * the token-major [B][cap][Hk*d] layout is stride_token = Hk*d, stride_head = d.
 */
typedef struct gattn_kv_desc {
    void *k;
    void *v;
    int32_t batch;       /* sequences held */
    int32_t capacity;    /* tokens per sequence */
    int64_t stride_token;
    int64_t stride_head;
    int64_t stride_batch;
} gattn_kv_desc;

/* Intermediate taps of the last step (device, fp32), each may be NULL:
 *   y     [B*R][2*H*d + 2*Hk*d]  projection outputs q_full | k | v before the norm
 *   attn  [B*R][H*d]             attention output before the gate */
typedef struct gattn_taps {
    float *y;
    float *attn;
} gattn_taps;

typedef struct gattn_layer gattn_layer;
typedef struct gattn_kv gattn_kv;

/* Validate a configuration without touching a GPU.  Same rules as create(). */
gattn_status gattn_cfg_validate(const gattn_cfg *cfg);

/* Rotary dims the layer uses: trunc(head_dim * partial_rotary_factor), computed
 * in double ("rope dims" of the qwen3_5 deltas page); -1 if cfg is NULL. */
int32_t gattn_rotary_dims(const gattn_cfg *cfg);

/* Create a layer on the current CUDA device: validates cfg, allocates scratch
 * (sized by max_batch/max_q_len) and the repacked-weight buffers.  *out owned
 * by the caller, release with gattn_layer_destroy.  Errors: those of
 * gattn_cfg_validate (GATTN_E_INVALID_ARG, GATTN_E_UNSUPPORTED; *out = NULL),
 * GATTN_E_CUDA when an allocation or device query fails (nothing leaks). */
gattn_status gattn_layer_create(const gattn_cfg *cfg, gattn_layer **out);

/* Repack the interchange weights (TensorFold issue 503 "Option C" affine rows,
 * layout of gattn_proj) into the library's device tile layout (same bytes per
 * step); copies q_norm and k_norm.  Runs and synchronizes on `stream`; the
 * caller may free the interchange buffers after it returns.  Errors:
 * GATTN_E_INVALID_ARG for a NULL layer, weights or buffer; GATTN_E_CUDA when a
 * launch or copy fails.  May be called again to replace the weights. */
gattn_status gattn_layer_set_weights(gattn_layer *layer, const gattn_weights *w, gattn_stream stream);

/* Register a cache for this layer (Atlas qwen3_5 forward page, LayerKvCache:
 * the caller pre-allocates, the step appends at cache_pos): checks sizes and
 * alignment and encodes the TMA tensor maps once.  *out is owned by the
 * caller (gattn_kv_destroy); the cache memory is borrowed and must outlive the
 * registration, and the registration must not outlive the layer.  Errors:
 * GATTN_E_INVALID_ARG for a NULL or misaligned pointer, batch <= 0, capacity
 * < 16, a stride that is not a positive multiple of 8, or a layout the TMA
 * encoder rejects; GATTN_E_CUDA when the encoder cannot be found. */
gattn_status gattn_kv_register(gattn_layer *layer, const gattn_kv_desc *desc, gattn_kv **out);

/*
 * A caller-owned Bf16KTurbo4V cache (device): the "safer-asym" format of the
 * Atlas qwen3_5 forward page (MetalKvDtype::Bf16KTurbo4V, LayerKvCache with a
 * V-side scale buffer): K raw bf16, V in a Walsh-Hadamard-rotated basis as
 * 4-bit Lloyd-Max codebook indices plus one FP8 E4M3 scale per group of 16.
 *   K       bf16, element (b, kv_head, token, j) at
 *           k + b*k_stride_batch + kv_head*k_stride_head + token*k_stride_token + j
 *           (strides in elements, multiples of 8)
 *   v_codes uint8, the row of (b, kv_head, token) -- d/2 bytes, code j in the
 *           low (j even) or high (j odd) nibble of byte j/2 -- at
 *           v_codes + b*code_stride_batch + kv_head*code_stride_head + token*(d/2)
 *   v_scales uint8 E4M3, d/16 bytes per row, at
 *           v_scales + b*scale_stride_batch + kv_head*scale_stride_head + token*(d/16)
 * Code and scale strides are in bytes, multiples of 16; rows of one
 * (b, kv_head) are consecutive.  Pointers 16-byte aligned; capacity a
 * multiple of 16; head_dim a power of two from 64 to 256.  A V row is
 * dequantized as H (s * c(code)) / sqrt(d) (H the Sylvester Hadamard matrix,
 * c the levels of gattn_turbo4_codebook); the step quantizes its new V rows
 * from their bf16 values (gattn_turbo4_quantize_device states how) and
 * applies the inverse rotation once to each attention output row.
 */
typedef struct gattn_kv_turbo4v_desc {
    void *k;
    void *v_codes;
    void *v_scales;
    int32_t batch;
    int32_t capacity;
    int64_t k_stride_token, k_stride_head, k_stride_batch;
    int64_t code_stride_head, code_stride_batch;
    int64_t scale_stride_head, scale_stride_batch;
} gattn_kv_turbo4v_desc;

/* Register a Bf16KTurbo4V cache (as gattn_kv_register).  GATTN_E_INVALID_ARG
 * for a bad pointer, stride, capacity or head_dim. */
gattn_status gattn_kv_register_turbo4v(gattn_layer *layer, const gattn_kv_turbo4v_desc *desc,
                                       gattn_kv **out);

/*
 * A caller-owned symmetric Turbo4 cache (device; MetalKvDtype::Turbo4 of the
 * Atlas qwen3_5 forward page: K and V both WHT-rotated 4-bit Lloyd-Max codes
 * with E4M3 group-of-16 scales).  K and V planes have the layout of the V
 * planes of gattn_kv_turbo4v_desc (one set of code and scale strides for
 * both).  The step quantizes its new K rows from the bf16 values of the
 * normed, rotary-embedded keys, and its new V rows as for Bf16KTurbo4V; the
 * attention rotates each q row once (q' = H q / sqrt(d)) so the scores are
 * q' . dequantized key rows in the rotated basis.  Same rules as
 * gattn_kv_register_turbo4v (no bf16 K).
 */
typedef struct gattn_kv_turbo4_desc {
    void *k_codes;
    void *k_scales;
    void *v_codes;
    void *v_scales;
    int32_t batch;
    int32_t capacity;
    int64_t code_stride_head, code_stride_batch;
    int64_t scale_stride_head, scale_stride_batch;
} gattn_kv_turbo4_desc;

gattn_status gattn_kv_register_turbo4(gattn_layer *layer, const gattn_kv_turbo4_desc *desc,
                                      gattn_kv **out);

/* The Turbo4 codebook as the kernels use it (host, no GPU): the 16 levels of
 * the Lloyd-Max quantizer of N(0, 1), ascending, rounded to fp32, and the 15
 * decision thresholds between them (midpoints taken in double, then rounded;
 * the middle one is 0).  Computed once per process by Lloyd's iteration (the
 * pages name the codebook, Atlas MetalKvDtype::Turbo4, but print no values).
 * GATTN_E_INVALID_ARG for a NULL array. */
gattn_status gattn_turbo4_codebook(float levels[16], float thresholds[15]);

/*
 * Quantize `rows` bf16 rows of `d` values (device, [rows][d]) into Turbo4
 * codes (device, [rows][d/2]) and E4M3 scales (device, [rows][d/16]), as the
 * step does for its new V rows; enqueued on `stream`, no synchronization.
 * Per row: y = H v * fp32(1/sqrt(d)) (butterfly stages h = 1, 2, 4, ... in
 * fp32); per group of 16: ss = pairwise fp32 sum of y_i^2, u_i = y_i /
 * sqrt(ss/16), code_i = number of thresholds below u_i, scale = E4M3 (nearest,
 * ties to even, saturating at 448) of sqrt(ss / pairwise sum of level^2); a
 * zero group gets codes 0 and scale 0.  d a power of two from 64 to 256.
 * GATTN_E_INVALID_ARG for rows < 0, a NULL pointer with rows > 0 or another
 * d; GATTN_E_CUDA when the launch fails.  rows == 0 launches nothing.
 */
gattn_status gattn_turbo4_quantize_device(const void *v_bf16, int64_t rows, int32_t d,
                                          void *codes, void *scales, gattn_stream stream);

/*
 * One layer step, enqueued on `stream` with no host synchronization and no
 * allocation (capturable into a CUDA graph).
 *   x          (device) [batch][q_len][hidden], cfg.x_dtype
 *   kv         registered cache holding sequences 0..batch-1
 *   cache_pos  (device) int32 [batch]: first new position of each sequence;
 *              the new rows go to cache_pos[b] .. cache_pos[b]+q_len-1 and
 *              row r attends positions 0 .. cache_pos[b]+r
 *   out        (device) bf16 [batch][q_len][hidden]
 * A sequence with cache_pos < 0 or cache_pos + q_len > capacity is skipped on
 * the device (its cache is untouched and its out rows are zero) and the next
 * gattn_layer_poll_status() returns GATTN_E_DEVICE_RANGE.  One step at a time
 * per layer handle: steps of one handle on different streams race on its scratch.
 * Errors (nothing is launched): GATTN_E_INVALID_ARG for a NULL argument, a
 * cache registered with another layer, batch outside [1, min(max_batch, cache
 * batch)] or q_len outside [1, max_q_len]; GATTN_E_STATE before
 * gattn_layer_set_weights; GATTN_E_UNSUPPORTED for a step the set mask does not
 * take (gattn_layer_set_mask);
 * GATTN_E_CUDA when a launch fails.
 */
gattn_status gattn_layer_step(gattn_layer *layer, const void *x, gattn_kv *kv,
                              const int32_t *cache_pos, int32_t batch, int32_t q_len,
                              void *out, gattn_stream stream);

/*
 * gattn_layer_step from host buffers: copies x and cache_pos into the layer's
 * own device staging buffers, enqueues the step on `stream` after those
 * copies, and the copy of its output rows into out_host after the step, then
 * returns (no host synchronization: out_host holds the result once `stream`
 * has reached it).
 *   x_host          (host) [batch][q_len][hidden], cfg.x_dtype
 *   cache_pos_host  (host) int32 [batch], as cache_pos of gattn_layer_step
 *   out_host        (host) bf16 [batch][q_len][hidden]
 * The input copies run on a stream of the layer's own, ordered before the
 * step but not after earlier work on `stream`: x_host and cache_pos_host must
 * hold the step's inputs when the call is made (not be written by work still
 * pending on `stream`), and stay unchanged until the stream has passed the
 * step.  out_host is written by a copy on `stream` after the step.  Pinned
 * (page-locked) memory makes the copies asynchronous.  The staging buffers
 * (two input slots used in turn, allocated with the layer for the largest
 * step it admits) belong to the handle, like its scratch.  Errors: those of
 * gattn_layer_step, checked before anything is enqueued; GATTN_E_CUDA when a
 * copy or a launch fails.
 */
gattn_status gattn_layer_step_host(gattn_layer *layer, const void *x_host, gattn_kv *kv,
                                   const int32_t *cache_pos_host, int32_t batch, int32_t q_len,
                                   void *out_host, gattn_stream stream);

/* Synchronize `stream`, then read and clear the layer's device status word:
 * GATTN_OK, GATTN_E_DEVICE_RANGE or GATTN_E_DEVICE_TIMEOUT (GATTN_E_INVALID_ARG
 * for a NULL layer, GATTN_E_CUDA when the synchronization or read fails). */
gattn_status gattn_layer_poll_status(gattn_layer *layer, gattn_stream stream);

/* Ask the next steps to also write the taps (layout of gattn_taps; borrowed
 * device buffers; NULL or all-NULL turns them off).  GATTN_E_INVALID_ARG for a
 * NULL layer.  Test instrumentation, not part of the layer's computation. */
gattn_status gattn_layer_set_taps(gattn_layer *layer, const gattn_taps *taps);

/*
 * An attention mask for the following steps (DS4Server issue 113: the verify
 * route's broadcast and head-specific masks), device bytes, borrowed:
 *   byte mask[b*stride_batch + hm*stride_head + r*stride_row + t]
 * nonzero = row r of sequence b may attend cache position t; hm = 0 for a
 * broadcast mask (heads == 1), the query head for a head-specific one
 * (heads == num_heads).  A mask replaces the causal rule: row r attends the
 * marked positions t < cache_pos[b] + q_len (positions >= `positions` are not
 * attended and never read); a row with no position left gives a zero attention
 * row.  Strides in bytes; stride_row >= positions.  The step refuses
 * (GATTN_E_UNSUPPORTED) a head-specific mask when the head-chunked verify route
 * applies (it hands the mask unchanged to every head chunk, where only a
 * broadcast mask fits).  The contents may
 * change between steps (read at run time, graph-capturable).
 */
typedef struct gattn_mask {
    const uint8_t *mask;
    int32_t heads;
    int32_t positions;
    int64_t stride_row, stride_head, stride_batch;
} gattn_mask;

/* Set (or with NULL / mask->mask == NULL clear) the attention mask of the
 * following steps.  GATTN_E_INVALID_ARG for a NULL layer, heads other than 1
 * or num_heads, positions <= 0, stride_row < positions or a negative stride. */
gattn_status gattn_layer_set_mask(gattn_layer *layer, const gattn_mask *mask);

/* Free a layer and everything it owns (NULL is a no-op).  Call it after the
 * layer's last step has finished on the GPU and after destroying the caches
 * registered with it; borrowed buffers are left alone. */
void gattn_layer_destroy(gattn_layer *layer);
/* Free a cache registration (NULL is a no-op); the cache memory is the
 * caller's and is left alone. */
void gattn_kv_destroy(gattn_kv *kv);

/* Thread-local message of the last failed call on this thread ("" if none). */
const char *gattn_last_error(void);

/*
 * Host quantizer + packer for synthetic weights (host): per (row, group)
 *   bias = bf16(min w), scale = bf16((max w - min w)/(2^bits - 1)),
 *   code = clamp(nearest-even((w - bias)/scale), 0, 2^bits - 1), code = 0 if scale == 0,
 * all arithmetic in double with ties-to-even bf16 rounding, written into the
 * interchange layout above.  w float [N][K]; packed [N][K*bits/32];
 * scales/biases [N][K/group].  Requires K % group == 0 and K*bits % 32 == 0.
 */
gattn_status gattn_pack_affine_host(const float *w, int64_t N, int64_t K, int32_t bits,
                                    int32_t group, uint32_t *packed, uint16_t *scales,
                                    uint16_t *biases);

/* Decode interchange codes on the GPU (device in/out): codes uint8 [N][K],
 * enqueued on `stream`.  GATTN_E_INVALID_ARG for a NULL pointer, negative
 * sizes, bits outside 1..8 or K*bits not a multiple of 32. */
gattn_status gattn_unpack_codes_device(const uint32_t *packed, int64_t N, int64_t K, int32_t bits,
                                       uint8_t *codes, gattn_stream stream);

/* Dequantize one projection of a layer FROM ITS REPACKED DEVICE LAYOUT with the
 * same register unpack the projection kernels use: w (device) float [N][K],
 * w = fp32(scale*code + bias) (exact: scale*code has <= 16 significant bits).
 * Allocates a temporary device buffer and synchronizes `stream`.  Errors:
 * GATTN_E_INVALID_ARG (NULL, proj outside 0..3), GATTN_E_STATE before
 * gattn_layer_set_weights, GATTN_E_CUDA. */
gattn_status gattn_layer_dequant_device(gattn_layer *layer, int32_t proj, float *w,
                                        gattn_stream stream);

/*
 * Same result as gattn_layer_dequant_device (bit for bit), for callers that
 * cannot allocate device memory or synchronize at the point of the call: code
 * recording a CUDA graph in global capture mode, code whose framework owns the
 * whole device memory budget, latency-sensitive paths.  It allocates nothing:
 * its staging buffer is a fixed 16 MiB device array inside the library (held
 * on every GPU that loads it, until exit), and it returns without waiting for
 * the GPU (w is ready once `stream` reaches that point).
 *   - Limit: the 128-row blocks spanning the projection times K must fit in
 *     4 Mi floats; larger projections fail with GATTN_E_UNSUPPORTED and a
 *     message naming the sizes.
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress), and so does the first call after the device's
 *     context was created anew (e.g. after cudaDeviceReset); make those
 *     calls before any stream capture.
 *   - A sticky CUDA error of the context is returned as GATTN_E_CUDA; an
 *     error left by an earlier, unrelated launch is neither reported nor
 *     cleared.
 *   - Every call shares the one array: calls that can overlap on the GPU (on
 *     different streams, or different layers at once) race on it.
 * The pages have no counterpart of this entry point (it is a library utility).
 */
gattn_status gattn_layer_dequant_device_static(gattn_layer *layer, int32_t proj, float *w,
                                               gattn_stream stream);

/*
 * The verify head-chunk plan (DS4Server issue 113, "Reproduction and boundary"):
 * when enabled and q_len*gqa > 32 and q_len <= 32, the query heads of each KV
 * group are split into chunks of max(1, min(gqa, 32/q_len)) heads (the last
 * chunk of a group holds the remainder), in head order; otherwise each KV
 * group is one chunk.  Writes up to `cap` chunks (first head, head count) and
 * returns the chunk count, or -1 for bad arguments.
 */
int32_t gattn_head_chunk_plan(int32_t q_len, int32_t num_heads, int32_t num_kv_heads,
                              int32_t enabled, int32_t *chunk_first_head, int32_t *chunk_len,
                              int32_t cap);


/*
 * Decoder-block variant of gattn_layer_step: the steps on either side of the
 * layer in forward_full_attention (Atlas spark_model/forward/qwen3_5/mod.rs,
 * module doc and FullAttentionLayer: input_ln, post_ln, norm -> projections ->
 * attention -> residual + post-norm -> MLP).  Per row of x:
 *   h          = x / sqrt(mean(x^2) + rms_eps) * input_ln     (RMSNorm)
 *   out        = bf16(x + layer(h))                           (residual stream)
 *   out_normed = bf16(RMSNorm(out) * post_ln)                 (the MLP's input;
 *                computed from the stored bf16 row of out)
 * Arguments: x is the raw hidden state [batch][q_len][hidden] in the layer's x
 * dtype (device); input_ln and post_ln are bf16 [hidden] device vectors,
 * borrowed; out is bf16 [batch][q_len][hidden]; out_normed (may be NULL, then
 * post_ln may be NULL too) is bf16 of the same shape and must not alias out.
 * Cache, position, launch and error behaviour as gattn_layer_step.  The
 * post-norm runs inside the o_proj launch (its last CTA to finish normalizes
 * every row) when batch * q_len * hidden <= 16384 and out, out_normed and
 * post_ln are 16-byte aligned, else in one more launch.  The norm of the
 * input is rounded to bf16 for a bf16 layer (kept fp32 for an fp32 one)
 * before the projections.  GATTN_E_INVALID_ARG for a NULL input_ln,
 * out_normed without post_ln or aliasing out.
 */
gattn_status gattn_layer_step_block(gattn_layer *layer, const void *x, gattn_kv *kv,
                                    const int32_t *cache_pos, int32_t batch, int32_t q_len,
                                    const void *input_ln, const void *post_ln, void *out,
                                    void *out_normed, gattn_stream stream);

/* Per-step launch report of the layer's last step: number of kernel launches
 * it enqueued, all of them this library's own kernels: 4 (q|k|v projection,
 * attention, the merge of its chunk partials with the output gate, o_proj)
 * when the q|k|v kernel converts x itself, else 5 with the x prep launch, one
 * more for a decoder-block step whose post-norm takes its own launch. */
int32_t gattn_layer_launches_per_step(const gattn_layer *layer);

/* The kernels of the layer's last step, in launch order. */
enum {
    GATTN_KERNEL_XPREP = 1,     /* x -> tensor-core operand (+ input RMSNorm of the block) */
    GATTN_KERNEL_PROJ_QKV = 2,  /* q|k|v dequant projection + norm / rotary / KV append */
    GATTN_KERNEL_ATTN = 3,      /* causal GQA attention over key chunks (one-chunk segments:
                                   output gate -> o_proj operand) */
    GATTN_KERNEL_MERGE = 4,     /* merge of the attention chunk partials, output gate -> o_proj
                                   operand */
    GATTN_KERNEL_PROJ_O = 5,    /* o_proj (+ residual and fused post-norm of the block) */
    GATTN_KERNEL_POSTNORM = 6   /* post-attention RMSNorm of the block, own launch */
};
/* Writes up to `cap` GATTN_KERNEL_* values (host array) and returns the launch
 * count of the last step (0 before any step), or -1 for bad arguments. */
int32_t gattn_layer_step_kernels(const gattn_layer *layer, int32_t *kinds, int32_t cap);

/* Instrumentation: with n >= 2 cudaEvent_t handles, each following step
 * records events[i] on its stream right before its i-th kernel launch (for
 * i < n - 1) and events[n-1] after its last launch, so per-kernel durations
 * can be read with cudaEventElapsedTime (use n = launches_per_step + 1).
 * n == 0 (or events == NULL) turns it off.  The events are borrowed.
 * Recording between kernels serializes them (no programmatic overlap), so use
 * it for per-kernel timing passes only. */
gattn_status gattn_layer_set_events(gattn_layer *layer, void *const *events, int32_t n);

/* Failure-detection test hook for the bounded device waits.
 *
 * Every wait of the projection kernels (a weight stage landing in shared
 * memory, a stage slot being released, partial sums arriving from the other
 * CTAs of a cluster) gives up after a time limit; the kernel then skips the
 * remaining work of that CTA, still reaches every barrier, and returns; the
 * layer's status word gets the timeout bit, so the next
 * gattn_layer_poll_status() returns GATTN_E_DEVICE_TIMEOUT and the context
 * stays usable.
 *
 * wait_limit_ns: the limit of those waits for the following steps, in ns;
 *   0 restores the default (2 s).  Negative: GATTN_E_INVALID_ARG.
 * withhold_stage: nonzero makes CTA 0 of every following q|k|v projection
 *   launch skip the copy of its last weight stage, so that the wait for it
 *   runs out after wait_limit_ns (the outputs of such a step are garbage);
 *   0 turns that off.
 *
 * Meant for tests of the timeout path; a layer that never calls it keeps the
 * default limit and withholds nothing. */
gattn_status gattn_layer_set_test_wait(gattn_layer *layer, int64_t wait_limit_ns,
                                       int32_t withhold_stage);

/*
 * ---------------------------------------------------------------------------
 * Packed sequences: the prompt pass of a gated full-attention layer and the
 * gated delta-rule layers that stand beside it in the hybrid stack (Atlas
 * spark_model/forward/qwen3_5/mod.rs: forward_full_attention, and the
 * linear-attention layer's gated_delta_rule_decode).
 *
 * Conventions shared by the four entry points below:
 *   - Sequences of different lengths are packed along one row axis: sequence s
 *     owns rows cu_rows[s] .. cu_rows[s+1]-1 of every row tensor.  cu_rows is
 *     (device) int32 [num_seqs + 1], non-decreasing, its last entry at most
 *     total_rows, the rows that the tensors hold.  Rows before cu_rows[0] and
 *     at or past cu_rows[num_seqs] are not written and reach no result, whatever
 *     they hold; like all total_rows they have to be readable memory (tiles and
 *     early loads may take them along).  A sequence may have no rows.
 *   - Tensors are described by a base pointer and element strides of the row
 *     ("token") and of the head; the elements of a head are contiguous.  bf16
 *     and fp32 rows: base 16-byte aligned, strides positive multiples of 8
 *     elements.  Slices of a wider projection output are such tensors.  An
 *     output's strides, those of a cache that is written among them, must keep
 *     its rows apart: in order of size, each spans all steps of the smaller ones.
 *   - Offsets, positions, slots and status are 4-byte aligned.
 *   - Outputs must not overlap inputs unless an entry point says so.
 *   - `status` (device) uint32 [1], may be NULL: the kernels OR GATTN_STATUS_*
 *     bits into it (never clear it), so that a caller can read it when it
 *     likes.  GATTN_STATUS_RANGE: a sequence was skipped because its rows,
 *     positions or slot lie outside what the descriptor holds.
 *     GATTN_STATUS_TIMEOUT: a wait inside a kernel gave up after two seconds, and
 *     rows or states of the call are missing.  Without a status word a skipped
 *     sequence shows in its zero rows only, and a time-out not at all.
 *   - No handle, no allocation, no synchronization, no workspace: calls on
 *     different streams share nothing, and every call can be captured into a
 *     CUDA graph.  The launches go to the current device, which must be the
 *     one the pointers belong to.
 *   - total_rows and kv_rows are at most 2^30, num_seqs 2^24.
 *   - num_seqs == 0 or total_rows == 0 launches nothing (but see gattn_delta_*).
 * Errors of every entry point, before anything is launched: GATTN_E_INVALID_ARG
 * for a NULL pointer, a size, stride or alignment outside these rules, and
 * GATTN_E_UNSUPPORTED for shapes stated there; GATTN_E_CUDA when a launch fails.
 * ---------------------------------------------------------------------------
 */
enum { GATTN_STATUS_RANGE = 1, GATTN_STATUS_TIMEOUT = 2 };

/*
 * The rows of a prompt between the projections and the attention: per-head QK
 * RMSNorm, partial RoPE and the KV append, as steps 3 to 6 of gattn_layer_step
 * do them, for any number of rows.  Row i of sequence s has position
 * p = cache_pos[s] + i:
 *   q_out[row][h]           = bf16(RoPE_p(RMSNorm(q[row][h]) * q_norm))
 *   k_cache[slot][hk][p]    = bf16(RoPE_p(RMSNorm(k[row][hk]) * k_norm))
 *   v_cache[slot][hk][p]    = bf16(v[row][hk])
 * The gate half of a doubled q_proj stays where it is: q is the projection
 * output with q_stride_head = 2 * head_dim.
 *   x_dtype       GATTN_DTYPE_F32 or GATTN_DTYPE_BF16: type of q, k and v
 *   slots         (device) int32 [num_seqs] or NULL (slot = s): the cache row of
 *                 each sequence.  A slot may appear once; a later sequence that
 *                 names it again is skipped.
 *   q_out         bf16 [total_rows][num_heads][head_dim] by strides
 *   k_cache, v_cache  bf16, element (slot, hk, p, j) at base + slot*stride_batch +
 *                 hk*stride_head + p*stride_token + j, as gattn_kv_desc, each
 *                 with strides of its own
 * A sequence is skipped (its q_out rows zero, its cache untouched,
 * GATTN_STATUS_RANGE) when cache_pos < 0, cache_pos + rows > cache_capacity, or
 * its slot is outside [0, cache_batch) or taken.  head_dim: a multiple of 64 up
 * to 256; cache_capacity up to 2^24, where positions are exact in fp32 (else
 * GATTN_E_UNSUPPORTED).  Rotary dims, theta and eps as in gattn_cfg; q_norm and
 * k_norm are 16-byte aligned.
 */
typedef struct gattn_prompt_rows_desc {
    int32_t num_heads, num_kv_heads, head_dim;
    float partial_rotary_factor, rope_theta, rms_eps;
    int32_t x_dtype;
    int32_t num_seqs;
    int32_t total_rows;
    const int32_t *cu_rows;
    const int32_t *cache_pos;
    const int32_t *slots;
    const void *q, *k, *v;
    int64_t q_stride_token, q_stride_head;
    int64_t k_stride_token, k_stride_head;
    int64_t v_stride_token, v_stride_head;
    const uint16_t *q_norm, *k_norm;      /* bf16 [head_dim] (device) */
    void *q_out;
    int64_t o_stride_token, o_stride_head;
    void *k_cache, *v_cache;
    int32_t cache_batch, cache_capacity;
    int64_t kc_stride_token, kc_stride_head, kc_stride_batch;
    int64_t vc_stride_token, vc_stride_head, vc_stride_batch;
    uint32_t *status;
} gattn_prompt_rows_desc;

gattn_status gattn_prompt_rows(const gattn_prompt_rows_desc *desc, gattn_stream stream);

/*
 * Causal attention of packed prompt rows with grouped heads and the output
 * gate:
 *   out[row][h] = bf16( sum_j softmax_j(scale * q[row][h] . k_j) v_j  *  sigmoid(gate[row][h]) )
 * over the keys j of the row's sequence that it may see; query head h reads KV
 * head h / (num_heads / num_kv_heads).  Scores, sums and out up to its one rounding
 * are fp32; 2^(score - the row's reference) is rounded to bf16 before it meets its
 * value, and those rounded numbers are what the softmax divides by the sum of.
 * Where the keys come from:
 *   cache_pos != NULL  a cache [kv_batch][num_kv_heads][kv_rows] by strides:
 *                      sequence s reads cache row slots[s] (NULL: s), and its
 *                      row i sees positions 0 .. cache_pos[s] + i (the new
 *                      rows' keys are in the cache, see gattn_prompt_rows).
 *                      Slots may repeat: nothing is written there.
 *   cache_pos == NULL  packed keys of kv_rows rows (kv_batch 1): sequence s owns
 *                      key rows cu_kv[s] .. cu_kv[s+1]-1 (cu_kv NULL: cu_rows),
 *                      and its row i sees the first i + 1 + (keys - rows) of
 *                      them: the last row sees all.
 * k and v NULL with kv_rows 0: a tensor without keys; only sequences that ask for
 * none are within it.  A row that sees no key gives zeros.  Values and keys that a row does not see
 * do not reach it, whatever they hold (NaN and infinities included).
 *   q, k, v       bf16
 *   gate          gate_dtype (GATTN_DTYPE_F32 or _BF16), or NULL for no gate
 *   out           bf16
 *   scale         finite, > 0
 *   max_kv        a hint: the most keys of any sequence (0: unknown).  It only
 *                 chooses how the work is split, never the result's validity.
 * A sequence is skipped (out rows zero, GATTN_STATUS_RANGE) when its slot,
 * positions or key rows lie outside the keys' tensor.  head_dim: a multiple of
 * 64 up to 256; num_heads * head_dim <= 65536 (else GATTN_E_UNSUPPORTED).
 */
typedef struct gattn_prompt_attention_desc {
    int32_t num_heads, num_kv_heads, head_dim;
    float scale;
    int32_t num_seqs;
    int32_t total_rows;
    const int32_t *cu_rows;
    const int32_t *cu_kv;
    const int32_t *cache_pos;
    const int32_t *slots;
    const void *q;
    int64_t q_stride_token, q_stride_head;
    const void *k, *v;
    int32_t kv_batch, kv_rows;
    int64_t k_stride_token, k_stride_head, k_stride_batch;
    int64_t v_stride_token, v_stride_head, v_stride_batch;
    const void *gate;
    int32_t gate_dtype;
    int32_t max_kv;
    int64_t g_stride_token, g_stride_head;
    void *out;
    int64_t o_stride_token, o_stride_head;
    uint32_t *status;
} gattn_prompt_attention_desc;

gattn_status gattn_prompt_attention(const gattn_prompt_attention_desc *desc, gattn_stream stream);

/*
 * The gated delta rule.  Per value head h (key head h / (num_v_heads /
 * num_k_heads)) a state S of k_dim x v_dim, and per row of a sequence, in order:
 *   S <- exp(g) S
 *   w  = beta (v - S^T k)
 *   S <- S + k w^T
 *   out = bf16(scale S^T q)
 * with q and k divided by sqrt(sum x^2 + l2_eps) first when qk_l2norm is set
 * (l2_eps >= 0; the sum is an fp32 number: with l2_eps 0 its square root must not
 * vanish).
 *   q, k          bf16 [total_rows][num_k_heads][k_dim] by strides
 *   v, out        bf16 [total_rows][num_v_heads][v_dim] by strides
 *   g, beta       fp32 [total_rows][num_v_heads], row strides >= num_v_heads; g is
 *                 the natural logarithm of the decay
 *   cu_rows       NULL: every sequence has total_rows / num_seqs rows
 *   state         fp32 [num_slots][num_v_heads][k_dim][v_dim], slot stride
 *                 state_stride (elements, a multiple of 4); the state before
 *                 the first row; NULL: zeros
 *   state_out     the state after the last row, same layout; equal to state
 *                 (in place), a buffer of its own, or NULL (not kept: drafted
 *                 rows that may be rejected).  A sequence without rows copies
 *                 its state.
 *   slots         (device) int32 [num_seqs] or NULL (slot = s).  A slot may appear
 *                 once; a later sequence that names it again is skipped, as is
 *                 one outside [0, num_slots) (out rows zero, state untouched,
 *                 GATTN_STATUS_RANGE).
 * gattn_delta_prompt is for prompts: it works through the rows in chunks.
 * gattn_delta_step is for one to a few new rows of many sequences: it works
 * row by row.  Both take any lengths and differ in rounding only: the step
 * computes in fp32; the prompt multiplies operands of 22 bits into fp32 sums,
 * and both round out once, to bf16.  Rows that stretch the state (beta |k|^2 above
 * 2.25, or g above 1/256) and columns of it whose size changes by orders of
 * magnitude within 32 rows are within the rule: a prompt takes such rows one by
 * one, in a multiple of the time.  Errors are those of fp32 sums relative to norms (|q|
 * times that of a column of S), in a prompt plus 2^-24 of the largest that the column
 * held or was written within the same 32 rows, counted from the sequence's first.
 * num_seqs > 0 with total_rows == 0 copies the states.  k_dim 64 or 128; v_dim a
 * multiple of 32 up to 256 (else GATTN_E_UNSUPPORTED).
 */
typedef struct gattn_delta_desc {
    int32_t num_k_heads, num_v_heads, k_dim, v_dim;
    float scale;
    int32_t qk_l2norm;
    float l2_eps;
    int32_t num_seqs;
    int32_t total_rows;
    int32_t num_slots;
    const int32_t *cu_rows;
    const int32_t *slots;
    const void *q, *k, *v;
    int64_t q_stride_token, q_stride_head;
    int64_t k_stride_token, k_stride_head;
    int64_t v_stride_token, v_stride_head;
    const float *g, *beta;
    int64_t g_stride_token, beta_stride_token;
    const float *state;
    float *state_out;
    int64_t state_stride;
    void *out;
    int64_t o_stride_token, o_stride_head;
    uint32_t *status;
} gattn_delta_desc;

gattn_status gattn_delta_prompt(const gattn_delta_desc *desc, gattn_stream stream);
gattn_status gattn_delta_step(const gattn_delta_desc *desc, gattn_stream stream);

/*
 * ---------------------------------------------------------------------------
 * A key-value cache in pages: decoding for a server that hands out cache memory in
 * pages, beside the contiguous caches above.  (The reference has one contiguous cache
 * a layer, Atlas LayerKvCache: a cache in pages, scaled frequencies and eviction have no
 * counterpart there.)
 *
 * Position p of sequence s is row p % page_size of page table[s][p / page_size] of two
 * pools; element (page, hk, row, j) of the keys at
 *   k_pages + page*k_stride_page + hk*k_stride_head + row*k_stride_token + j
 * and the values likewise with strides of their own (bf16; base 16-byte aligned, strides
 * positive multiples of 8 elements; a call that writes the pools needs their rows apart).
 *   table        (device) int32 [num_seqs][table_width], row stride table_stride.  Only
 *                entries of positions that a call touches are read.
 *   page_size    a multiple of 16; table_width * page_size <= 2^24 (else
 *                GATTN_E_UNSUPPORTED)
 * The conventions of packed sequences hold, and these:
 *   - A sequence with rows whose positions, cache_pos[s] .. cache_pos[s] + rows - 1, do
 *     not fit its table row is skipped: GATTN_STATUS_RANGE.
 *   - An entry outside [0, num_pages) is no page: its positions hold no keys (none is
 *     attended, written or moved), GATTN_STATUS_RANGE; the rest of the sequence counts.
 *   - Reading calls may name a page twice, for prefixes that sequences share.  No page
 *     and row may be written by two rows of a call.
 *   - Rows are read by whoever comes later on the same stream; nothing else orders
 *     calls that share a pool.
 * ---------------------------------------------------------------------------
 */
typedef struct gattn_pages {
    void *k_pages, *v_pages;
    int32_t num_pages, page_size;
    int64_t k_stride_token, k_stride_head, k_stride_page;
    int64_t v_stride_token, v_stride_head, v_stride_page;
    const int32_t *table;
    int32_t table_width;
    int64_t table_stride;
} gattn_pages;

enum { GATTN_ROPE_PLAIN = 0, GATTN_ROPE_LINEAR = 1, GATTN_ROPE_YARN = 2 };

/*
 * New rows between the projections and the attention, as gattn_prompt_rows, into pages:
 * per-head RMSNorm, rotary embedding and append.  Row i of sequence s goes to position
 * cache_pos[s] + i and is turned by the angles of positions[row] (NULL: the same
 * position; after gattn_paged_evict a sequence's next token is further on than its next
 * place).
 *   q_norm, k_norm  bf16 [head_dim], 16-byte aligned; NULL: no norm
 *   rotary_dims     even, 2 .. head_dim: the first elements of a head, turned in pairs
 *   rope_pairs      0: (y_i, y_{i + rotary_dims/2});  else neighbours (y_2i, y_{2i+1})
 *   frequencies     f_i = rope_theta^(-2i / rotary_dims), angle = position * f_i;
 *     GATTN_ROPE_LINEAR: f_i / rope_factor
 *     GATTN_ROPE_YARN: f_i (1 - c_i) + f_i / rope_factor * c_i, c_i rising from 0 to 1 between
 *       pair floor(b(rope_beta_fast)) and ceil(b(rope_beta_slow)), kept within 0 and
 *       rotary_dims - 1; b(t) = rotary_dims ln(rope_original / (2 pi t)) / (2 ln rope_theta)
 *       (Peng et al., "YaRN: Efficient Context Window Extension of Large Language Models")
 *     rope_factor >= 1
 *   rope_size       factor of cos and sin; 0: 0.1 ln(rope_factor) + 1 for YaRN, else 1
 *   positions       (device) int32 [total_rows], 0 .. 2^24.  A row outside is skipped alone
 *                   (q_out zero, nothing written, GATTN_STATUS_RANGE).
 * A skipped sequence's q_out rows are zero; a row whose page does not exist has its q_out
 * all the same.  head_dim: a multiple of 64 up to 256 (else GATTN_E_UNSUPPORTED).
 */
typedef struct gattn_paged_rows_desc {
    int32_t num_heads, num_kv_heads, head_dim;
    int32_t rotary_dims, rope_pairs, rope_scaling;
    float rope_theta, rope_factor;
    int32_t rope_original;
    float rope_beta_fast, rope_beta_slow, rope_size, rms_eps;
    int32_t x_dtype;
    int32_t num_seqs;
    int32_t total_rows;
    const int32_t *cu_rows;
    const int32_t *cache_pos;
    const int32_t *positions;
    const void *q, *k, *v;
    int64_t q_stride_token, q_stride_head;
    int64_t k_stride_token, k_stride_head;
    int64_t v_stride_token, v_stride_head;
    const uint16_t *q_norm, *k_norm;
    void *q_out;
    int64_t o_stride_token, o_stride_head;
    gattn_pages pages;
    uint32_t *status;
} gattn_paged_rows_desc;

gattn_status gattn_paged_rows(const gattn_paged_rows_desc *desc, gattn_stream stream);

/*
 * Causal attention of new rows over pages, with grouped heads and the output gate:
 *   out[row][h] = bf16( sum_p softmax_p(scale * q[row][h] . k_p) v_p  *  sigmoid(gate[row][h]) )
 * Row i of sequence s sees positions 0 .. cache_pos[s] + i (its own key is in the pages,
 * see gattn_paged_rows).  Made for one to a few new rows of each sequence (decoding,
 * drafted rows to verify), any number is taken; a prompt is faster through
 * gattn_prompt_attention.  Scores, sums and out up to its one rounding are fp32;
 * the softmax's numerators meet the values with 16 bits.
 *   q             bf16
 *   gate          gate_dtype (GATTN_DTYPE_F32 or _BF16), or NULL for no gate
 *   lse           fp32 [total_rows][num_heads] or NULL: ln sum_p exp(scale * q . k_p)
 *   workspace     (device) at least gattn_paged_attention_workspace(...) bytes, 16-byte
 *                 aligned, for the parts of sequences that several CTAs share.  Its
 *                 contents need not be set and mean nothing afterwards.  Calls that may
 *                 run at once (other streams, graphs replayed side by side, other
 *                 threads: a call is two launches) need one each.
 * A row that sees no position (its sequence is skipped, or none of its pages exists) gives
 * zeros and lse -infinity.  What a row does not see does not reach it, whatever it holds.
 * A value that it does see and that is infinite or NaN makes its output infinite or NaN.
 * Scores of -infinity add nothing; a row that has no others is one that sees nothing.
 * head_dim: a multiple of 64 up to 256; num_heads * head_dim <= 65536; total_rows *
 * num_heads below 2^31 (else GATTN_E_UNSUPPORTED).
 */
typedef struct gattn_paged_attention_desc {
    int32_t num_heads, num_kv_heads, head_dim;
    float scale;
    int32_t num_seqs;
    int32_t total_rows;
    const int32_t *cu_rows;
    const int32_t *cache_pos;
    const void *q;
    int64_t q_stride_token, q_stride_head;
    gattn_pages pages;
    const void *gate;
    int32_t gate_dtype;
    int64_t g_stride_token, g_stride_head;
    void *out;
    int64_t o_stride_token, o_stride_head;
    float *lse;
    void *workspace;
    int64_t workspace_bytes;
    uint32_t *status;
} gattn_paged_attention_desc;

/* Bytes of workspace for calls of these heads with up to num_seqs sequences and up to
 * total_rows rows, -1 for shapes that gattn_paged_attention refuses.  No GPU is needed. */
int64_t gattn_paged_attention_workspace(int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                                        int32_t num_seqs, int32_t total_rows);
gattn_status gattn_paged_attention(const gattn_paged_attention_desc *desc, gattn_stream stream);

/*
 * The softmax weight that each position received from a call's rows, per KV head:
 *   weights_out[s][hk][p] = weights[s][hk][p]
 *                         + sum_{rows i that see p} sum_{h of hk's group} exp(scale * q_ih . k_p - lse_ih)
 * for the positions p < cache_pos[s] + rows of each sequence with rows; others are left as
 * they are.  Positions from cache_pos[s] on are new: they had nothing, whatever `weights`
 * holds there.
 *   attention     shapes, rows, q, scale, pages and status as gattn_paged_attention got
 *                 them, lse what it left there; v_pages, gate, out and workspace are not read.
 *                 A row whose lse is -infinity gives nothing.
 *   weights       fp32, element (s, hk, p) at s*w_stride_seq + hk*w_stride_head + p, or
 *                 NULL for zeros
 *   weights_out   fp32, the same strides (which keep weights_width positions apart);
 *                 may be weights, else shares no memory with them
 * A sequence with more positions than weights_width is skipped (GATTN_STATUS_RANGE).
 * The sums have one order: equal inputs give equal bits.
 */
typedef struct gattn_paged_weights_desc {
    gattn_paged_attention_desc attention;
    const float *weights;
    float *weights_out;
    int32_t weights_width;
    int64_t w_stride_seq, w_stride_head;
} gattn_paged_weights_desc;

gattn_status gattn_paged_weights(const gattn_paged_weights_desc *desc, gattn_stream stream);

/*
 * Shortens sequences: of the lengths[s] positions of sequence s and each KV head, the
 * newest min(recent, .) and those of the others with the largest weights, m =
 * min(lengths[s], keep) in all, move to positions 0 .. m-1 in their order.  Among equal
 * weights the lowest position is kept; a NaN counts as -infinity.
 *   lengths       (device) int32 [num_seqs]
 *   weights       fp32, element (s, hk, p) at s*w_stride_seq + hk*w_stride_head + p
 *   weights_out   fp32 with strides of its own, or NULL: weights of the kept positions,
 *                 in their new places; may be weights (equal strides over what there is more
 *                 than one of), else shares no memory with them
 *   kept          int32 [num_seqs][num_kv_heads][keep]: the positions that were kept, in
 *                 order; -1 behind them
 *   lengths_out   int32 [num_seqs]: m; not in lengths' memory
 *   out_table     the pages that the kept positions move to, of the same pools; NULL or
 *                 pages.table: in place.  Other pages must not be among those that the
 *                 call reads.  A sequence that keeps everything is copied to them too.
 * Heads move on their own: a position's keys are those of different tokens for different
 * heads afterwards, which attention does not mind (rotary positions are in the keys).
 * Pages that are written must belong to one sequence.  A sequence whose length is
 * negative or beyond its table row or weights_width, or whose m does not fit out_table
 * or weights_out_width, is skipped: kept -1, its length as it was, GATTN_STATUS_RANGE.
 */
typedef struct gattn_paged_evict_desc {
    int32_t num_kv_heads, head_dim;
    int32_t num_seqs;
    int32_t keep, recent;
    gattn_pages pages;
    const int32_t *out_table;
    int32_t out_table_width;
    int64_t out_table_stride;
    const int32_t *lengths;
    int32_t *lengths_out;
    const float *weights;
    int32_t weights_width;
    int64_t w_stride_seq, w_stride_head;
    float *weights_out;
    int32_t weights_out_width;
    int64_t wo_stride_seq, wo_stride_head;
    int32_t *kept;
    uint32_t *status;
} gattn_paged_evict_desc;

gattn_status gattn_paged_evict(const gattn_paged_evict_desc *desc, gattn_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* GATTN_H */
