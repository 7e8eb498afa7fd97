/*
 * gqa.h -- C ABI of the GB300 (sm_103a) GroupQueryAttention forward pass.
 *
 * The operation is com.microsoft.GroupQueryAttention as its README states it
 * (sections Description, Inputs, Outputs, Attributes, Type constraints):
 * grouped-query attention over BSH query/key/value and a BNSH key/value cache,
 * with optional paired Q/K RMS normalisation, NeoX rotary embedding, causal
 * and local-window masks, additive attention bias, softcap, head sink /
 * smooth softmax, an int8 (per-tensor or per-channel) or, for prompts, a
 * packed 4-bit quantised cache, a sliding-window (window-shift) cache, and a
 * prompt's float cache in the other float dtype.
 *
 * Conventions for every entry point:
 *   - All tensors are dense, row-major (C-contiguous) and live in device
 *     memory of the current CUDA device, except where a field says "host".
 *     Pointers must be 16-byte aligned.
 *   - The caller owns every buffer and the stream. No entry point allocates
 *     device memory; scratch space is the caller's workspace
 *     (gqa_workspace_size).
 *   - Work is enqueued asynchronously on the given stream (a cudaStream_t
 *     passed as void*; NULL is the legacy default stream).
 *   - Failures return a gqa_status; gqa_last_error() gives a one-line reason
 *     (per calling thread). Nothing is launched when a check fails.
 */
#ifndef GQA_GB300_H
#define GQA_GB300_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define GQA_API __attribute__((visibility("default")))
#else
#define GQA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum gqa_status {
  GQA_OK = 0,
  GQA_ERR_INVALID_ARGUMENT = 1, /* shapes, dtypes, attributes or pointers break the contract */
  GQA_ERR_UNSUPPORTED = 2,      /* allowed by the operator but not implemented here */
  GQA_ERR_CUDA = 3,             /* a CUDA runtime/driver call or a launch failed */
  GQA_ERR_DEVICE_STATUS = 4,    /* a kernel flagged bad data (see gqa_read_device_status) */
  GQA_ERR_WORKSPACE = 5         /* workspace NULL, misaligned or smaller than required */
} gqa_status;

/* Element types (section Type constraints: T in {float32, float16},
 * T_CACHE in {float32, float16, uint8, int8}, T_KV_SCALE float32, M int32).
 * GQA_BF16 exists only so that such a tensor is rejected as UNSUPPORTED. */
typedef enum gqa_dtype {
  GQA_DTYPE_NONE = 0,
  GQA_F32 = 1,
  GQA_F16 = 2,
  GQA_I8 = 3,
  GQA_U8 = 4,
  GQA_I32 = 5,
  GQA_BF16 = 6
} gqa_dtype;

/* k_quant_type / v_quant_type (section Attributes). */
typedef enum gqa_quant {
  GQA_QUANT_NONE = 0,
  GQA_QUANT_PER_TENSOR = 1,
  GQA_QUANT_PER_CHANNEL = 2
} gqa_quant;

/* One tensor: data == NULL means "input absent". shape[0..ndim-1] are used. */
typedef struct gqa_tensor {
  void* data;
  int32_t dtype; /* gqa_dtype */
  int32_t ndim;
  int64_t shape[4];
} gqa_tensor;

/* Attributes, section Attributes of the operator page; gqa_attrs_default()
 * fills the page's defaults (num_heads / kv_num_heads have none). */
typedef struct gqa_attrs {
  int32_t num_heads;            /* N, query heads */
  int32_t kv_num_heads;         /* N_kv, key/value heads; N % N_kv == 0 */
  int32_t causal;               /* 1 (default) causal; 0 bidirectional (needs local_window_size == -1) */
  int32_t do_rotary;            /* 0 (default) or 1: NeoX rotary on Q and on K before it is cached */
  int32_t local_window_size;    /* -1 (default) disables; W >= 0: key j visible from p iff p-W <= j <= p */
  float scale;                  /* 0 (default) selects 1/sqrt(head_size) */
  float softcap;                /* 0 (default) disables; c > 0: score -> c*tanh(score/c) before the bias */
  float qk_norm_epsilon;        /* 1e-6 (default) */
  int32_t smooth_softmax;       /* -1 (default); 1 adds exp(0 - max) to the denominator when no head_sink */
  int32_t k_quant_type;         /* gqa_quant; NONE (default) */
  int32_t v_quant_type;         /* gqa_quant; NONE (default) */
  int32_t kv_cache_bit_width;   /* 8: int8 cache; 4: packed 4-bit cache (prompt only); ignored when not quantised */
  int32_t sliding_window_cache; /* 0 (default); 1: past/present are window buffers (see gqa_outputs) */
} gqa_attrs;

/* Inputs, section Inputs of the operator page (same names, same shapes):
 *   query          T      (B, S, N*H)
 *   key, value     T      (B, S, N_kv*H)            -- kv_sequence_length == S
 *   past_key/value T_CACHE (B, N_kv, L, H) or absent. L is the capacity when
 *                  past and present are one buffer (past.data == present.data),
 *                  else the past length (copy mode). Absent for a 4-bit cache.
 *   seqlens_k      int32  (B): total length of batch b minus one (device)
 *   cos/sin_cache  T      (R, H/2), R > largest position; required iff do_rotary
 *   attention_bias T      (B or 1, N or 1, S, total_sequence_length) or absent
 *   head_sink      T      (N) or absent
 *   k/v_scale      float32 (1) for PER_TENSOR or (N_kv*H) for PER_CHANNEL
 *   q/k_norm_weight T     (H), both or neither
 * total_sequence_length is a HOST scalar: the largest seqlens_k[b] + 1. */
typedef struct gqa_inputs {
  gqa_tensor query, key, value;
  gqa_tensor past_key, past_value;
  gqa_tensor seqlens_k;
  gqa_tensor cos_cache, sin_cache;
  gqa_tensor attention_bias;
  gqa_tensor head_sink;
  gqa_tensor k_scale, v_scale;
  gqa_tensor q_norm_weight, k_norm_weight;
  int32_t total_sequence_length;
} gqa_inputs;

/* Outputs, section Outputs: output T (B, S, N*H); present_key/value T_CACHE
 * (B, N_kv, C, H). Shared buffer: present.data == past.data and C == L.
 * Copy mode: C == L + S. No past: C >= S (a capacity buffer).
 * sliding_window_cache == 1 with a past cache (section Attributes): the past
 * buffer (capacity L) holds the most recent n_old = min(past_b, L) rows of
 * the sequence, oldest first; the present keeps the last n_new - S of them at
 * rows 0 .. n_new-S-1 (older rows are evicted from the front) and appends the
 * S new rows after them, n_new = min(n_old + S, C); row r holds absolute
 * position total_b - n_new + r (masks and bias columns use it; rotary uses
 * the absolute position). Needs causal = 1, local_window_size W > 0,
 * C >= S + W and, for a separate past, L >= W; C need not equal L + S and
 * total_sequence_length may exceed C. Without a past the flag changes nothing.
 * 4-bit cache (kv_cache_bit_width == 4, section Inputs past_key / present_key):
 * GQA_U8 of shape (B, N_kv, C, H/2); byte k of a row holds code(2k) + 8 in
 * its low nibble and code(2k+1) + 8 in its high nibble, code =
 * clamp(rint(x / scale), -7, 7) with the fp32 division of the int8 code. */
typedef struct gqa_outputs {
  gqa_tensor output;
  gqa_tensor present_key, present_value;
} gqa_outputs;

typedef struct gqa_handle gqa_handle;

/* Fill *attrs with the defaults of section Attributes. */
GQA_API void gqa_attrs_default(gqa_attrs* attrs);

/* Create a handle holding a copy of the attributes (host memory only).
 * Returns INVALID_ARGUMENT for a NULL pointer, non-positive head counts,
 * num_heads % kv_num_heads != 0, causal == 0 with local_window_size != -1,
 * local_window_size < -1, softcap < 0, a non-finite scale or epsilon, or a
 * quant type outside gqa_quant, or a quantised cache whose kv_cache_bit_width
 * is neither 8 nor 4, or sliding_window_cache not 0 / 1, or 1 without causal
 * attention and local_window_size > 0. */
GQA_API gqa_status gqa_create(const gqa_attrs* attrs, gqa_handle** out);

/* Bytes of device workspace gqa_forward needs for these shapes (host-only;
 * makes no CUDA call). Runs every host-side check of gqa_forward, so it is
 * also the way to validate a call without a GPU. */
GQA_API gqa_status gqa_workspace_size(const gqa_handle* handle, const gqa_inputs* in,
                              const gqa_outputs* out, size_t* bytes);

/* Forward pass (whole operator) on `stream`:
 *   1. append the S new K/V rows of every (batch, KV head) at positions
 *      past_b .. past_b+S-1 of the present cache, past_b = seqlens_k[b]+1-S
 *      with a past cache and 0 without (K: RMS norm, then rotary at the
 *      absolute position, then cast, int8-quantise or pack 4-bit codes;
 *      V: the same store without norm or rotary);
 *      in copy mode the live past rows 0 .. past_b-1 are copied first;
 *   2. output[b, i, h] = softmax over the visible cache rows of
 *      scale * q_h . k (softcapped, plus bias), with query head h reading KV
 *      head h / (N/N_kv), the head-sink logit in the denominator, times V.
 * Operator page sections Description, Inputs, Outputs, Attributes and
 * Implementation variants (share_append / new_kv_past / quant_int8 decode and
 * flash prefill: append first, then attend over the cache as stored, with
 * causal bounds right-aligned at the live length from seqlens_k).
 * Present rows that are not appended (or copied) keep their bytes. Output
 * rows i >= total_b of a prompt without past (padding) are written as 0.
 * workspace: device buffer of at least gqa_workspace_size bytes, 256-byte
 * aligned, owned by the caller, not used concurrently by another call. Its
 * contents need not survive between calls: every call first clears the
 * workspace header (status word and split-merge tickets) on `stream`, so the
 * caller may use the buffer for anything else in between.
 * Host-side checks as in gqa_workspace_size. Data errors found on the device
 * (seqlens_k[b]+1 outside [S or 1, min(C, total_sequence_length)], a rotary
 * position beyond the cos/sin rows) skip that batch entry without any write
 * out of bounds and set a bit of the workspace's status word, which then
 * describes this call until the next call on the same workspace clears it. */
GQA_API gqa_status gqa_forward(gqa_handle* handle, const gqa_inputs* in, const gqa_outputs* out,
                       void* workspace, size_t workspace_bytes, void* stream);

/* Forward pass without any workspace, for callers that cannot allocate device
 * memory: a plugin inside a host runtime that hands it only its input and output
 * buffers and exposes no allocator, or code on a latency-critical path where
 * cudaMalloc / cudaFree (which may synchronise the device) are not acceptable.
 * The operator's pages have no counterpart: this is a deployment variant of
 * gqa_forward's decode regime, with the same inputs, outputs and results.
 *   - Scratch (status word, merge tickets, split partials) comes from one
 *     fixed array of 16 MiB compiled into the library; every GPU that loads
 *     the library holds it until the process exits. Nothing is allocated:
 *     no cudaMalloc, cudaFree or allocating library routine is called.
 *   - Only the decode regime (gqa_describe_plan reports GQA_REGIME_DECODE);
 *     other calls return GQA_ERR_UNSUPPORTED. A call that needs more than
 *     16 MiB of scratch returns GQA_ERR_WORKSPACE with the size it needs.
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress) with that device current; make that first call
 *     before any stream capture.
 *   - Every call shares the one array and it keeps the last call's contents;
 *     each call clears the status word and tickets on its stream first. Calls
 *     that overlap on the GPU (other streams, threads or handles) race and give
 *     wrong results: serialise them.
 *   - Data errors found on the device skip that batch entry as in gqa_forward,
 *     but are not reported: no entry point reads this status word. */
GQA_API gqa_status gqa_forward_noalloc(gqa_handle* handle, const gqa_inputs* in, const gqa_outputs* out,
                                       void* stream);

/* Bound of the pipeline waits of the tensor-core kernels, for callers that
 * want a data-dependent stall reported sooner, and a switch to test the
 * timeout path (no counterpart on the operator's pages).
 *   cycles: every barrier wait of a tensor-core CTA gives up after this many
 *     SM clock cycles (0 restores the default, 4e9 cycles, about 2 s at the
 *     maximum clock; otherwise at least 1000). A CTA whose wait gives up sets
 *     GQA_DEVICE_TIMEOUT, stops its pipeline, waits for its own copies and
 *     MMAs in flight, frees its tensor memory and returns; the call's outputs
 *     are then undefined. The next call on the handle and workspace is
 *     unaffected (each call clears the workspace header).
 *   withhold_copy: -1 (default) off; k >= 0 makes the TMA warp of every
 *     tensor-core CTA stop before the copy of its k-th key tile (in the
 *     prefill over an int8 / 4-bit cache: the converter warps before its
 *     conversion), so the waits for that tile expire: a test of the timeout
 *     path that faults nothing.
 * Applies to the following gqa_forward / gqa_forward_noalloc calls on the
 * handle. Host-only; INVALID_ARGUMENT for a NULL handle or a value out of range. */
GQA_API gqa_status gqa_set_wait_limit(gqa_handle* handle, int64_t cycles, int32_t withhold_copy);

/* Synchronise `stream`, read and clear the status word that the kernels of
 * the most recent gqa_forward call on `workspace` set (each call clears it
 * first). *status receives the OR of GQA_DEVICE_* bits (0 = no data error).
 * Returns DEVICE_STATUS if it is non-zero, CUDA on a runtime failure. */
#define GQA_DEVICE_BAD_SEQLEN 1u  /* seqlens_k out of range for the cache / total length / S */
#define GQA_DEVICE_BAD_ROTARY 2u  /* a rotary position is not covered by cos/sin_cache rows */
#define GQA_DEVICE_TIMEOUT 4u     /* a bounded pipeline wait gave up (kernel returned early) */
GQA_API gqa_status gqa_read_device_status(gqa_handle* handle, void* workspace, void* stream, uint32_t* status);

/* Host-only description of how gqa_forward would run a call: the regime
 * (GQA_REGIME_DECODE: one fused split-KV launch; GQA_REGIME_PREFILL: pre-pass
 * then flash prefill), the number of kernel launches per call, the decode
 * split length / split count (0 for prefill) and the workspace bytes. Same
 * checks and status codes as gqa_workspace_size.
 * Decode regime: up to 8 query rows per KV head (S * num_heads / kv_num_heads)
 * with head size 64 or 128 on the CUDA-core kernel (split_len = keys per
 * split, max_splits = splits per (batch, KV head)), or, for fp16 inputs and
 * cache with head size 128, up to 16 rows on the tensor-core kernel
 * (split_len = 128 keys per work unit, max_splits = partial-result slots). */
#define GQA_REGIME_DECODE 1
#define GQA_REGIME_PREFILL 2
typedef struct gqa_plan_info {
  int32_t regime;
  int32_t launches;
  int32_t split_len;
  int32_t max_splits;
  uint64_t workspace_bytes;
} gqa_plan_info;
GQA_API gqa_status gqa_describe_plan(const gqa_handle* handle, const gqa_inputs* in, const gqa_outputs* out,
                                     gqa_plan_info* info);

/* ---- Rotary embedding with several position axes -------------------------
 * Adjacent to section Attributes, do_rotary, whose single position is a row's
 * place in its sequence. Here every token has one position on each of
 * num_axes axes (time, height, width, ...), and each rotated pair takes its
 * angle from one of them:
 *   y[d]     = x[d] c - x[d+D] s,   y[d+D] = x[d+D] c + x[d] s,   d < D,
 *   c = cos_cache[p][d], s = sin_cache[p][d], p = positions[axis(d)][b][i],
 * D = sum of sections (2 D <= head size; coordinates from 2 D on pass through).
 * axis(d): interleaved == 0: the first sections[0] pairs take axis 0, the next
 * sections[1] axis 1, and so on. interleaved == 1: pair d takes axis
 * r = d % num_axes while d < num_axes * sections[r], else axis 0 (sections[0]
 * is then the number of pairs left for axis 0).
 * With norm weights x is first RMS normalised, x / sqrt(mean(x^2) + eps) * w
 * (qk_norm_epsilon of the handle). Computed in fp32, rounded once; for head
 * sizes 64, 128 and 256 the operation order is that of the rows gqa_forward
 * stores (equal bytes at equal positions). Positions are explicit, so rows of
 * a cache that gqa_block_evict has compacted keep their own.
 *   query      T (B, S, N*H);  key T (B, S, N_kv*H) or absent
 *   positions  int32 (num_axes, B, S), each in [0, R); a token with another
 *              position is not written and sets GQA_DEVICE_BAD_ROTARY
 *   cos/sin_cache  T or float32 (R, D)
 *   q/k_norm_weight T (H): both or neither (without key: q only)
 * Outputs have the inputs' shapes; each may be its input (in place) and may
 * not overlap another tensor. D is a multiple of 8, num_axes 1 .. 8, N*H at
 * most 2^30. */
#define GQA_MAX_ROTARY_AXES 8
typedef struct gqa_rotary_inputs {
  gqa_tensor query, key;
  gqa_tensor positions;
  gqa_tensor cos_cache, sin_cache;
  gqa_tensor q_norm_weight, k_norm_weight;
  int32_t sections[GQA_MAX_ROTARY_AXES]; /* pairs of each axis (host values) */
  int32_t num_axes;
  int32_t interleaved;
} gqa_rotary_inputs;

typedef struct gqa_rotary_outputs {
  gqa_tensor query, key;
} gqa_rotary_outputs;

/* One launch on `stream`. Of the handle's attributes only the head counts and
 * qk_norm_epsilon apply. status: see gqa_block_forward. */
GQA_API gqa_status gqa_rotary_axes(gqa_handle* handle, const gqa_rotary_inputs* in, const gqa_rotary_outputs* out,
                                   void* status, void* stream);

/* ---- int8 cache with a scale for each block of tokens and KV head ---------
 * Beside the per-tensor and per-channel scales of section Inputs (k_scale,
 * v_scale), which are fixed by the caller, these belong to the cache and
 * follow the data. Row r of head g of sequence b is
 *   value[d] = code[b][g][r][d] * scale[b][g][r / block_size],  scale >= 0.
 *   key/value_codes   int8 (B, N_kv, C, H)
 *   key/value_scales  float32 (B, N_kv, ceil(C / block_size))
 *   block_size        16, 32, 64, 128 or 256 tokens */
typedef struct gqa_block_cache {
  gqa_tensor key_codes, value_codes;
  gqa_tensor key_scales, value_scales;
  int32_t block_size;
} gqa_block_cache;

/* Inputs of one step. total_b = seqlens_k[b] + 1 is the number of live cache
 * rows of sequence b after the step; the last n_b = new_lens[b] (S without
 * new_lens; 0 <= n_b <= min(S, total_b)) of them belong to the first n_b rows
 * of query (key, value); rows n_b .. S-1 are padding. seqlens_k[b] may be -1
 * with n_b = 0 (an empty slot).
 *   query            T (B, S, N*H), prepared (see gqa_rotary_axes)
 *   key, value       T (B, S, N_kv*H), or both absent: the rows are in the cache already
 *   seqlens_k        int32 (B);  new_lens int32 (B) or absent
 *   head_sink        T (N) or absent
 *   past_weights     float32 (B, N_kv, C) or absent (read as zeros)
 *   total_sequence_length  HOST scalar, at least the largest total_b, at most C */
typedef struct gqa_block_inputs {
  gqa_tensor query, key, value;
  gqa_tensor seqlens_k, new_lens;
  gqa_tensor head_sink;
  gqa_tensor past_weights;
  int32_t total_sequence_length;
} gqa_block_inputs;

/*   output           T (B, S, N*H); padding rows are written as 0
 *   present_weights  float32 (B, N_kv, C) or absent; may be past_weights itself */
typedef struct gqa_block_outputs {
  gqa_tensor output;
  gqa_tensor present_weights;
} gqa_block_outputs;

/* Bytes of workspace gqa_block_forward needs for these shapes (host-only; runs
 * every host-side check). May be 0. */
GQA_API gqa_status gqa_block_workspace_size(const gqa_handle* handle, const gqa_block_cache* cache,
                                            const gqa_block_inputs* in, const gqa_block_outputs* out, size_t* bytes);

/* One step over a block-scaled cache, on `stream`:
 *   1. with key / value, store the new rows at cache rows total_b - n_b ..
 *      total_b - 1. The scale of a block is max|x| over the rows stored in
 *      it times fp32(1/127), rounded to fp32; a block that already holds rows keeps its
 *      scale when the new rows need no larger one, else it takes the larger
 *      one and its old codes are rounded anew. A code is the integer nearest
 *      to the exact quotient x / scale, ties to even, within +-127. An
 *      infinite x becomes +-127 and a NaN 0, and neither enters the scale.
 *   2. output[b, i, h] = softmax over the visible rows j of scale * q . k_j
 *      (softcap c: c tanh(s / c)), times the values; query row i stands at
 *      cache row p = total_b - n_b + i and sees rows max(0, p - W) .. p, W =
 *      local_window_size (all rows up to p without a window); query head h
 *      reads KV head h / (N / N_kv). head_sink / smooth_softmax add a logit to
 *      the denominator as in gqa_forward.
 *   3. with present_weights: present_weights[b, g, j] = past_weights[b, g, j]
 *      (0 for j >= total_b - n_b) + the sum over the n_b rows and the heads of
 *      group g of the probability of row j, for j < total_b. Other entries
 *      keep their values. No atomics: a call's result does not vary.
 * Rows of the cache behind total_b keep their bytes. Attributes used:
 * num_heads, kv_num_heads, local_window_size, scale, softcap, smooth_softmax;
 * causal must be 1 and do_rotary, the quant types and sliding_window_cache off.
 * workspace: at least gqa_block_workspace_size bytes, 256-byte aligned, not
 * used concurrently by another call; its contents need not survive.
 * status: one device uint32 (4-byte aligned) or NULL. Data errors (lengths out
 * of range: that sequence is skipped, nothing of it is written) OR
 * GQA_DEVICE_* bits into it; it is never cleared here: clear it once before
 * its first use, and read and clear it with gqa_read_device_status. */
GQA_API gqa_status gqa_block_forward(gqa_handle* handle, const gqa_block_cache* cache, const gqa_block_inputs* in,
                                     const gqa_block_outputs* out, void* workspace, size_t workspace_bytes,
                                     void* status, void* stream);

/* Host-only description of how gqa_block_forward would run a call (same checks):
 * regime GQA_REGIME_DECODE: the keys of every KV head split over the warps of the
 * GPU (split_len keys a unit, max_splits workers); GQA_REGIME_PREFILL: the
 * tensor-core prefill over whole key ranges. launches counts the kernels. */
GQA_API gqa_status gqa_block_describe_plan(const gqa_handle* handle, const gqa_block_cache* cache,
                                           const gqa_block_inputs* in, const gqa_block_outputs* out,
                                           gqa_plan_info* info);

/* Eviction from a block-scaled cache by accumulated attention weight: the live
 * rows of every (sequence, KV head) are reduced to at most `keep`, copied in
 * their order to rows 0 .. of another cache. Sequences with total_b <= keep
 * keep all rows. Otherwise rows [0, first) and the `recent` last ones stay,
 * and of the rows between them the keep - first - recent with the largest
 * weights (equal weights: the lower row first; a NaN counts as the lowest).
 *   from, into       caches of the same B, N_kv, H and block_size; into has
 *                    C >= min(keep, total_sequence_length) and shares no memory with `from`
 *   weights          float32 (B, N_kv, from C);  seqlens_k int32 (B)
 *   into_weights     float32 (B, N_kv, into C) or absent: the kept rows' weights
 *   kept             int32 (B, N_kv, keep): source row of each kept row, -1 behind the last
 *   into_seqlens_k   int32 (B): min(total_b, keep) - 1
 * A block of `into` takes the largest scale among its rows' source blocks;
 * rows of a block with that scale keep their codes, the others are rounded
 * anew (nearest, ties to even). Rows and blocks behind the last kept row keep
 * their bytes. A sequence with total_b outside [0, min(C, total_sequence_length)]
 * is skipped and sets GQA_DEVICE_BAD_SEQLEN; its entries of kept and
 * into_seqlens_k keep their values, or become -1 (no row, an empty slot) with
 * GQA_FILL_KEPT and GQA_FILL_SEQLENS in fill_skipped.
 * 0 <= first, 0 <= recent, 1 <= keep, first + recent <= keep. */
#define GQA_FILL_KEPT 1
#define GQA_FILL_SEQLENS 2
typedef struct gqa_evict_args {
  gqa_block_cache from, into;
  gqa_tensor weights, seqlens_k;
  gqa_tensor into_weights, kept, into_seqlens_k;
  int32_t total_sequence_length;
  int32_t keep, recent, first;
  int32_t fill_skipped; /* 0, or GQA_FILL_* bits */
} gqa_evict_args;

/* Two launches on `stream`, no workspace; of the handle's attributes only
 * kv_num_heads applies. */
GQA_API gqa_status gqa_block_evict(gqa_handle* handle, const gqa_evict_args* args, void* status, void* stream);

/* Per-launch timing for measurement tools. gqa_profile_begin creates
 * 2*max_launches CUDA events (host-side driver objects, no device memory);
 * while profiling is on, every call on this handle that launches kernels
 * records an event pair around each kernel it launches (up to
 * max_launches launches in total). gqa_profile_end synchronises the events,
 * writes up to `capacity` (kind, milliseconds) pairs in launch order, sets
 * *count to the number of launches recorded, releases the events and turns
 * profiling off. Kinds: */
#define GQA_KERNEL_COPY_PAST 1
#define GQA_KERNEL_PREPASS 2
#define GQA_KERNEL_DECODE 3
#define GQA_KERNEL_PREFILL_CUDA_CORE 4
#define GQA_KERNEL_PREFILL_TENSOR_CORE 5
#define GQA_KERNEL_DECODE_TENSOR_CORE 6
#define GQA_KERNEL_WINDOW_SHIFT 7
#define GQA_KERNEL_BIAS_STAGE 8
#define GQA_KERNEL_ROTARY_AXES 9
#define GQA_KERNEL_BLOCK_APPEND 10
#define GQA_KERNEL_BLOCK_ATTENTION 11
#define GQA_KERNEL_BLOCK_MERGE 12
#define GQA_KERNEL_BLOCK_PREFILL 13
#define GQA_KERNEL_BLOCK_WEIGHTS 14
#define GQA_KERNEL_EVICT_SELECT 15
#define GQA_KERNEL_EVICT_GATHER 16
GQA_API gqa_status gqa_profile_begin(gqa_handle* handle, int32_t max_launches);
GQA_API gqa_status gqa_profile_end(gqa_handle* handle, int32_t* kinds, float* ms, int32_t capacity, int32_t* count);

/* Release the handle (host memory only). NULL is a no-op. */
GQA_API void gqa_destroy(gqa_handle* handle);

/* Static name of a status code. */
GQA_API const char* gqa_status_string(gqa_status status);

/* One-line reason of the last non-OK status returned on this thread. */
GQA_API const char* gqa_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* GQA_GB300_H */
