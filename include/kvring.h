/*
 * kvring -- a rolling FP8 attention cache for one GPU (sm_103a).
 *
 * One kvring_t holds one transformer layer's attention cache, as described
 * in "Runway Characters: Serving a 57B Video Diffusion Transformer for
 * Real-Time Conversation" (Runway research post):
 *
 *   - section "Do It Once, at Write Time": each new frame's keys get rotary
 *     position embeddings (RoPE) once, as they enter the cache, and keys and
 *     values are quantised to FP8 with per-head scales calibrated once per
 *     session; the cache is a ring, so the window advances by overwriting
 *     the oldest slots with no copy; at each periodic position reset a
 *     single delta rotation is applied to the cached keys in place; after
 *     wrap-around slot order is not time order, so every slot keeps its own
 *     position;
 *   - section "Where the Time Went": every attention call reads its layer's
 *     cache (5,788 slots, 757 of them new);
 *   - sections "What Broke in Production" and "Blackwell and Beyond Four
 *     GPUs": no host/device synchronisation on the steady path, no buffer
 *     per input shape, calls that chain correctly inside CUDA graphs, and an
 *     FP8 attention kernel that takes per-head scales.
 *
 * Formats.  FP8 is OCP OFP8 E4M3 ("fn": bias 7, no infinities, largest
 * finite 448), rounded to nearest even with saturation to +-448.  RoPE is
 * the adjacent-pair form: pair (x[2i], x[2i+1]) rotates by p * base^(-2i/d).
 *
 * Conventions for every entry point.
 *   - Tensors are device pointers, row-major and contiguous, 16-byte
 *     aligned.  Token inputs are bf16 [n][num_heads][head_dim] (what a QKV
 *     projection emits).  Positions are int32 [n] on the device.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Every
 *     call only enqueues work on that stream; none synchronises with the
 *     host, none allocates memory.  Calls on one ring must be ordered (one
 *     stream, or the caller's events); two rings are independent.
 *   - A ring belongs to the device that was current at kvring_create; every
 *     call that takes a ring returns KVRING_ERR_INVALID_ARG unless that
 *     device is current (the kernels would otherwise run on another GPU
 *     against this one's memory).  Its tensors and stream must be on that
 *     device too, which the library cannot check.
 *   - Arguments are checked on the host before anything is enqueued; a
 *     failed check enqueues nothing and returns an error status.  CUDA
 *     launch failures return KVRING_ERR_CUDA.  Problems only the device can
 *     see (a position outside the RoPE table, a timed-out wait) set bits in
 *     an error word that kvring_export() returns in state[KVRING_STATE_ERROR];
 *     the kernels then skip the offending element instead of faulting.
 *   - The ring's head, fill level and next position live in device memory,
 *     so a CUDA graph that captured a write or an attention call advances
 *     the ring correctly on every replay.
 *   - Kernels overlap their predecessor on the stream (programmatic
 *     dependent launch): each may start before the kernel enqueued just
 *     before it has finished, and waits for it before touching anything
 *     that kernel may write.  kvring_write_frame reads its frame, and
 *     kvring_attention its queries, before that wait, except when a library
 *     kernel that may still be running writes a caller buffer overlapping
 *     them (kvring_project_write's q_out or kv_out, an attention output,
 *     the legacy window): the library records those buffers per stream and
 *     the call then reads after the wait.  A caller's own kernel launched
 *     with programmatic stream serialisation that triggers its dependents
 *     before it has written these inputs must not precede the library call
 *     that reads them.
 */
#ifndef KVRING_H
#define KVRING_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct kvring kvring_t;   /* opaque host handle, one per layer */

typedef enum {
  KVRING_OK = 0,
  KVRING_ERR_INVALID_ARG = 1,     /* null/misaligned pointer, bad size or config */
  KVRING_ERR_NOT_CALIBRATED = 2,  /* write or attention before calibration */
  KVRING_ERR_CAPACITY = 3,        /* more tokens than the ring or config allows */
  KVRING_ERR_UNSUPPORTED = 4,     /* head_dim or device not supported */
  KVRING_ERR_CUDA = 5             /* a CUDA runtime call or launch failed */
} kvring_status;

typedef struct {
  int32_t num_heads;      /* H >= 1 */
  int32_t head_dim;       /* d: 64 or 128 */
  int32_t capacity;       /* C ring slots, 1 .. 2^24 */
  int32_t max_tokens;     /* most tokens per write / calibration / attention call */
  int32_t max_position;   /* RoPE table rows: positions lie in [0, max_position) */
  int32_t max_kv_splits;  /* most key/value partitions one attention call may use (1..32) */
  int32_t attn_precision; /* 0 = automatic per tile; 1..4 = fixed precision level */
  int32_t pinned_prefix;  /* P, 0 .. capacity - 1: slots [0, P) keep the first P tokens ever
                             written and are never overwritten; later tokens cycle over the
                             other capacity - P slots.  0 = the plain ring.  (The pages give
                             5,788 = 7 x 757 + 489 slots and do not say whether a part is
                             never evicted; P = 489 reads the remainder as such a part.) */
  int32_t rope_pairs_t;   /* 0 = 1-D RoPE (one position per token).  Else the 3-D variant: of
                             the head_dim/2 rotation pairs, [0, T) turn with the frame index t,
                             [T, T + Y) with the row y and the rest with the column x, each
                             section a RoPE of its own (local pair j of a section of 2m dims
                             turns by coordinate * base^(-2j/(2m))).  T >= 8; T, Y and the
                             column pairs are multiples of 8.  Positions are then int32
                             [n][3] = (t, y, x), required by every call that takes them;
                             slot positions hold t, and a reset turns only the temporal
                             pairs.  (The pages give one position per token; a video model's
                             tokens have three coordinates.) */
  int32_t rope_pairs_y;   /* Y, the row pairs of the 3-D variant (0 with 1-D RoPE) */
  double rope_base;       /* RoPE base, e.g. 10000 */
} kvring_config;

#define KVRING_DELTA_TO_OLDEST (-1)
#define KVRING_OUT_F32 0
#define KVRING_OUT_BF16 1

/* Layout of the int32 state[] array returned by kvring_export(). */
#define KVRING_STATE_HEAD 0        /* next slot to be written */
#define KVRING_STATE_NVALID 1      /* filled slots: min(capacity, tokens written) */
#define KVRING_STATE_TOTAL_LO 2    /* tokens written, low 32 bits */
#define KVRING_STATE_TOTAL_HI 3    /* tokens written, high 32 bits */
#define KVRING_STATE_NEXT_POS 4    /* position given to the next token by default */
#define KVRING_STATE_CALIBRATED 5  /* 1 once scales are set */
#define KVRING_STATE_ERROR 6       /* device error bits, see KVRING_DEVERR_* */
#define KVRING_STATE_LAST_DELTA 7  /* delta used by the last delta rotation */
#define KVRING_STATE_WORDS 8

#define KVRING_DEVERR_POSITION 1u  /* a position outside [0, max_position) was skipped */
#define KVRING_DEVERR_TIMEOUT 2u   /* a pipeline wait in the attention kernel gave up */
#define KVRING_DEVERR_DELTA 4u     /* delta outside [0, max_position): rotation skipped */

/* Bytes of device memory one ring needs (cache, scales, positions, state,
 * RoPE table, attention workspace).  0 if the config is invalid. */
size_t kvring_required_bytes(const kvring_config* cfg);

/* Create a ring inside `dev_buf` (device memory of at least
 * kvring_required_bytes(cfg) bytes, 256-byte aligned, owned by the caller,
 * which must keep it alive until kvring_destroy and free it afterwards).
 * Clears the ring, uploads the RoPE table and builds the TMA descriptors.
 * This is the only call that synchronises (it waits for its own upload on
 * `stream`).  On success *out receives the handle. */
kvring_status kvring_create(const kvring_config* cfg, void* dev_buf, size_t bytes,
                            void* stream, kvring_t** out);

/* Free the host handle.  The device buffer stays the caller's. */
kvring_status kvring_destroy(kvring_t* ring);

/* Once per session ("Do It Once, at Write Time": per-head scales calibrated
 * once per session).  k, v: bf16 [n][H][d]; pos: int32 [n] device positions
 * of the keys, or NULL for next_pos + i (3-D RoPE: int32 [n][3], required).  For each head h:
 *   scale_k[h] = max |rope(k)[., h, .]| / 448, scale_v[h] = max |v[., h, .]| / 448
 * (IEEE single division; a result below 2^-126, e.g. an all-zero head,
 * becomes 1), and the reciprocals used for quantisation.  Writes nothing
 * into the ring; usually followed by kvring_write_frame of the same frame.
 * Errors: INVALID_ARG (n < 1, bad pointers), CAPACITY (n > max_tokens). */
kvring_status kvring_calibrate_scales(kvring_t* ring, const void* k_bf16, const void* v_bf16,
                                      const int32_t* pos, int32_t n, void* stream);

/* Write one frame of n new tokens ("Do It Once, at Write Time").
 * Token t goes to slot (head + t) mod capacity (with a pinned prefix P:
 * the g-th token ever written goes to slot g while g < P, else to slot
 * P + (g - P) mod (capacity - P)):
 *   K[h][slot][:] = e4m3(rope(k[t,h,:], pos[t]) * inv_scale_k[h])
 *   V[h][slot][:] = e4m3(v[t,h,:] * inv_scale_v[h])
 *   slot_pos[slot] = pos[t]
 * then head advances by n slots, n_valid = min(capacity, n_valid + n),
 * total += n, next_pos += n.  RoPE is computed in fp32 from the fp32
 * cos/sin table with every product and sum rounded separately.
 * pos: int32 [n] device positions, or NULL for next_pos + t (3-D RoPE:
 * int32 [n][3] = (t, y, x), required; slot_pos[slot] = t).
 * Errors: NOT_CALIBRATED, CAPACITY (n > capacity, n > capacity - P when
 * P > 0, or n > max_tokens), INVALID_ARG. */
kvring_status kvring_write_frame(kvring_t* ring, const void* k_bf16, const void* v_bf16,
                                 const int32_t* pos, int32_t n, void* stream);

/* Position reset ("Do It Once, at Write Time": one delta rotation of the
 * cached window at each reset).  Every filled slot's key is rotated by
 * -delta in place, in the FP8 code units (no rescaling): for each pair
 * (a, b) of decoded codes and the table row (c, s) of delta,
 *   a' = a*c + b*s,  b' = b*c - a*s   (fp32, each step rounded), then e4m3.
 * slot_pos -= delta for filled slots, next_pos -= delta.  Values are not
 * touched.  delta = KVRING_DELTA_TO_OLDEST reads, on the device, the
 * position of the oldest slot (the next slot to be overwritten once the
 * ring is full, slot 0 before), so the window restarts at position 0.
 * With a pinned prefix P only the rolling slots [P, n_valid) are rotated
 * and have their positions lowered (prefix keys are never re-rounded), and
 * KVRING_DELTA_TO_OLDEST takes delta = position of the oldest rolling slot -
 * (position of slot P - 1 + 1), at least 0, so the window continues right
 * after the prefix.
 * Errors: INVALID_ARG (delta < -1 or >= max_position). */
kvring_status kvring_delta_rotate(kvring_t* ring, int32_t delta, void* stream);

/* ------------------------------------------------------------------------
 * QKV projection with the cache write in its epilogue ("fused pre-attention
 * kernels", section "Judging Quality When Pixels Can't": the projection,
 * RoPE and FP8 quantisation in front of the attention, fused).
 *
 * y = x W^T for one frame: x bf16 [n][d_model] (the block's input rows), W
 * bf16 [3 * num_heads * head_dim][d_model] (a linear layer's weight: output
 * rows by input columns; rows [0, H*d) make the queries, [H*d, 2*H*d) the
 * keys, [2*H*d, 3*H*d) the values).  Summed in fp32 on the tensor cores and
 * rounded once to bf16 (the projection's output format); then
 *   - queries: stored to q_out bf16 [n][num_heads][head_dim] (NULL = not
 *     stored), what kvring_attention takes;
 *   - with KVRING_PROJECT_WRITE: keys and values written into the ring
 *     exactly as kvring_write_frame(k, v, pos, n) writes those bf16 values
 *     (same positions, slots, state advance, error word); needs a
 *     calibrated ring and n <= capacity - pinned_prefix;
 *   - with KVRING_PROJECT_STORE_KV: keys and values also stored to kv_out
 *     bf16 [2][n][num_heads][head_dim] (keys first), e.g. to calibrate a new
 *     session's scales from its first frame.
 * d_model is a multiple of 64 (at least 64); n <= max_tokens.  An fp32
 * tensor-core sum may round to a bf16 one step away from the exactly rounded
 * sum when that sum lies that close to a rounding midpoint.
 * ------------------------------------------------------------------------ */
#define KVRING_PROJECT_WRITE 1
#define KVRING_PROJECT_STORE_KV 2
kvring_status kvring_project_write(kvring_t* ring, const void* x, const void* w, int32_t d_model,
                                   const int32_t* pos, int32_t n, void* q_out, void* kv_out,
                                   int32_t flags, void* stream);

/* ------------------------------------------------------------------------
 * Between two blocks: a block's output joins the residual stream, and the
 * stream's norm, modulated, is the next block's input (kvring_project_write's
 * x, for instance).  For every token t, with r its row of the modulation tables:
 *   u        = y[t], or norm(y[t]) * post_weight
 *   h_out[t] = h[t] + residual_scale * gate[r] * u
 *   x_out[t] = norm(h_out[t]) * weight * (1 + scale[r]) + shift[r]
 *   KVRING_NORM_RMS    z / sqrt(mean(z^2) + eps)
 *   KVRING_NORM_LAYER  (z - mean(z)) / sqrt(var(z) + eps), var over all `width` values
 * h, h_out: [num_tokens][width] fp32 or bf16 (stream_dtype); y, x_out: bf16;
 * gate, scale, shift: [mod_rows][width], fp32 or bf16 (mod_dtype), each NULL
 * for none (1, 0, 0); weight, post_weight: bf16 [width] or NULL (ones).
 * mod_index: int32 [num_tokens] rows, or NULL: row 0 of one, or row t of
 * num_tokens; a token whose row is outside [0, mod_rows) gets NaN.
 * Rows lie stride elements apart (multiples of 8, at most 2^28, at least width where
 * there is more than one row), so slices of packed tensors can be passed.
 * y NULL: h is normed as it is (h_out, gate, post_weight NULL, post_norm none).
 * x_out NULL and norm KVRING_NORM_NONE: the sum alone.  h_out may be NULL when x_out
 * is not.  h_out may be h (with its stride); no other result's span, first row to
 * last, may lie over that of an argument or the other result.  Everything between
 * reading and the one rounding of each result is fp32, squares included; x_out comes from the unrounded sum.
 * Works on the current device, and keeps no state.
 * ------------------------------------------------------------------------ */
#define KVRING_NORM_NONE 0
#define KVRING_NORM_RMS 1
#define KVRING_NORM_LAYER 2
#define KVRING_NORM_MAX_WIDTH 16384

typedef struct {
  int32_t num_tokens;     /* n >= 1 */
  int32_t width;          /* a multiple of 8, 8 .. KVRING_NORM_MAX_WIDTH */
  int32_t stream_dtype;   /* KVRING_OUT_F32 or KVRING_OUT_BF16 */
  int32_t mod_dtype;      /* the same, of gate, scale and shift */
  int32_t mod_rows;       /* rows of gate, scale and shift (ignored without them) */
  int32_t post_norm;      /* KVRING_NORM_*: of y */
  int32_t norm;           /* KVRING_NORM_*: of the stream */
  int32_t reserved;       /* 0 */
  int64_t h_stride, y_stride, mod_stride, h_out_stride, x_out_stride;
  float eps, residual_scale;
} kvring_norm_config;

kvring_status kvring_residual_norm(const kvring_norm_config* cfg, const void* h, const void* y, const void* gate,
                                   const void* scale, const void* shift, const int32_t* mod_index,
                                   const void* post_weight, const void* weight, void* h_out, void* x_out,
                                   void* stream);

/* The cache upkeep the ring replaced, kept as the comparison path ("Where
 * the Time Went": before the ring, every attention call re-applied RoPE to
 * every cached key, re-quantised the cache to FP8 and shifted the window by
 * copying it).  The caller keeps the window of the last `capacity` tokens,
 * unrotated bf16 [capacity][H][d] in time order, in two buffer pairs and
 * alternates them: this call copies wk_in/wv_in shifted by the n new tokens
 * (the n oldest leave once the window is full) plus the frame k/v (bf16
 * [n][H][d]) into wk_out/wv_out, takes per-head scales from the whole new
 * window (amax of the rotated keys, of the values, over 448), and rewrites
 * the ring's FP8 cache from it: window slot i -> ring slot i, key rotated at
 * position base + i (base = position of the oldest token in the window,
 * positions counting the tokens given so far from 0), same pinned fp32 RoPE
 * and E4M3 conversion as kvring_write_frame.  Afterwards kvring_attention
 * reads the ring as usual.  Do not mix with kvring_write_frame on one ring.
 * Errors: INVALID_ARG (NULL, unaligned or aliased buffers), CAPACITY
 * (n > capacity or n > max_tokens), UNSUPPORTED (a ring with a pinned
 * prefix or 3-D RoPE: the original upkeep had neither). */
kvring_status kvring_legacy_upkeep(kvring_t* ring, const void* wk_in, const void* wv_in, void* wk_out,
                                   void* wv_out, const void* k_bf16, const void* v_bf16, int32_t n,
                                   void* stream);

/* Largest number of rings one batched call takes (a model's layers). */
#define KVRING_MAX_BATCH 64

/* kvring_write_frame on num_rings rings at once, in one launch: ring i gets
 * k_bf16[i], v_bf16[i] and pos[i] (pos may be NULL, or any pos[i] NULL, for
 * next_pos + t of that ring).  Every ring must have the same num_heads,
 * head_dim, capacity and pinned_prefix; n applies to all.  The result on each ring is
 * byte-for-byte that of kvring_write_frame.  The reset of the page
 * ("Do It Once, at Write Time") and the per-step upkeep touch every layer,
 * and one launch over all of them moves hundreds of megabytes instead of a
 * few per launch.  `rings`, `k_bf16`, `v_bf16` and `pos` are host arrays of
 * num_rings entries (the pointers in them are device pointers); rings must
 * be distinct.
 * Errors: INVALID_ARG (num_rings outside 1..KVRING_MAX_BATCH, a NULL or
 * repeated ring, mismatched shapes, unaligned pointers), NOT_CALIBRATED,
 * CAPACITY; nothing is launched on an error. */
kvring_status kvring_write_frames_many(kvring_t* const* rings, int32_t num_rings,
                                       const void* const* k_bf16, const void* const* v_bf16,
                                       const int32_t* const* pos, int32_t n, void* stream);

/* kvring_delta_rotate on num_rings rings of the same num_heads, head_dim,
 * capacity and pinned_prefix in one launch (delta, or KVRING_DELTA_TO_OLDEST read per ring on
 * the device).  Each ring ends byte-for-byte as after kvring_delta_rotate.
 * Errors: INVALID_ARG (as above, or delta < -1 or >= a ring's max_position);
 * nothing is launched on an error. */
kvring_status kvring_delta_rotate_many(kvring_t* const* rings, int32_t num_rings, int32_t delta,
                                       void* stream);

/* FP8 attention of n_q queries over the ring ("Where the Time Went";
 * "Blackwell and Beyond Four GPUs": FP8 attention with per-head scales).
 *   out[t,h,:] = sum_j softmax_j(rope(q[t,h,:], qpos[t]) . Kdeq[h,j,:] / sqrt(d)) Vdeq[h,j,:]
 * over the filled slots j, with Kdeq = code * scale_k[h], Vdeq = code *
 * scale_v[h].  Slot order does not matter: keys carry their rotation.
 * Queries are split into 1 to 4 FP8 terms with a per-row scale; the
 * probabilities multiply V in half precision (V widened exactly from its
 * E4M3 codes), as one f16 term at levels 1-3 and as two (the f16 value and
 * the f16 rounding of what it left) at level 4; products accumulate in fp32
 * on the tensor cores.  The level (1-4 query terms) is chosen per 128-query
 * tile from L = max|rotated q| * max|k| and V = max|v| of the head, unless
 * attn_precision fixes it: 4 when V > 128 or L*V > 4800, else 1 when L <= 4
 * and V <= 0.5, else 2 while L*V <= 435, else 3.
 * q: bf16 [n_q][H][d]; qpos: int32 [n_q] device positions (3-D RoPE:
 * int32 [n_q][3], required), or NULL for
 * next_pos - n_q + t (the positions of the last n_q tokens written with
 * default positions).  out: [n_q][H][d], fp32 (KVRING_OUT_F32) or bf16
 * (KVRING_OUT_BF16).  An empty ring gives zeros.
 * Errors: NOT_CALIBRATED, CAPACITY (n_q > max_tokens), INVALID_ARG. */
kvring_status kvring_attention(kvring_t* ring, const void* q_bf16, const int32_t* qpos,
                               int32_t n_q, void* out, int32_t out_dtype, void* stream);

/* Attention that allocates nothing, for callers that cannot hand the library
 * device memory.  Some callers cannot allocate device memory at all: a
 * plugin living inside a host program that owns the whole device memory
 * pool, or a real-time loop where an allocation would stall the device or
 * break its memory budget.  This entry point computes exactly what
 * kvring_attention computes, with the same arguments and errors, but its
 * scratch (the precision level chosen for each 128-query tile and head)
 * lives in a fixed 128 KiB static device array inside the library rather
 * than in the ring's buffer.  Every GPU that loads the library holds that
 * array until the process exits.
 *   - It calls no cudaMalloc, cudaFree or allocating library routine.
 *   - The first call on a device looks up the array's device address
 *     (once per device, with that device current); make that first call
 *     before any stream capture.
 *   - The array is shared by every call: calls that overlap on the GPU
 *     (other streams, other rings) race and must be ordered by the caller.
 *     Nothing in it needs to start at zero (each call writes every level
 *     it uses before reading it).
 *   - It uses at most 8 key/value splits, which merge inside their
 *     thread-block cluster, so it needs no split partials.  A call with more
 *     than 32,768 (128-query tile, head) units, i.e. more than 4 bytes of
 *     levels per unit beyond 128 KiB, returns KVRING_ERR_CAPACITY.
 * The paper has no counterpart: this is a deployment variant. */
kvring_status kvring_attention_noalloc(kvring_t* ring, const void* q_bf16, const int32_t* qpos,
                                       int32_t n_q, void* out, int32_t out_dtype, void* stream);

/* ------------------------------------------------------------------------
 * A paged cache for many requests (sessions of different lengths on one
 * GPU), beside the ring: kvring_pages_t holds, for every layer of a model,
 * a pool of pages, each page holding `page_size` tokens' keys and values
 * of all key/value heads, and one set of block tables that all layers
 * share.  A step is
 *   kvring_pages_plan        where the step's new tokens go
 *   for every layer:
 *     kvring_pages_write     head norms, RoPE, keys and values into the pages
 *     kvring_pages_attention the new tokens' queries over their requests
 *   kvring_pages_commit      the new lengths and the taken pages become final
 * and nothing in it needs the host: lengths, tables, the free list and the
 * plan live in device memory, so a captured step replays with whatever
 * lengths the device then holds.  The conventions at the top of this file
 * hold (alignment, streams, checks, device); calls on one kvring_pages_t
 * must be ordered (one stream, or the caller's events), captured graphs
 * that use one included, since its plan and workspace are shared by them.
 *
 * Requests live in rows 0 .. max_requests - 1 of the block tables.  A row
 * is free when its length is 0.  Pages are taken from a stack of free page
 * ids, the last id first, in the order of the plan's requests and of their
 * pages; kvring_pages_release puts a request's pages back, first page first.
 * ------------------------------------------------------------------------ */
typedef struct kvring_pages kvring_pages_t;

#define KVRING_CACHE_E4M3 0
#define KVRING_CACHE_BF16 1
#define KVRING_ROPE_ADJACENT 0   /* pairs (x[2i], x[2i+1]), as the ring's */
#define KVRING_ROPE_HALVES 1     /* pairs (x[i], x[i + d/2]) */

typedef struct {
  int32_t num_q_heads;   /* Hq, a multiple of num_kv_heads */
  int32_t num_kv_heads;  /* Hkv; query head h reads key/value head h / (Hq / Hkv).  Hq / Hkv <= 64 */
  int32_t head_dim;      /* d: 64 or 128 */
  int32_t num_layers;    /* 1 .. 1024 */
  int32_t page_size;     /* tokens per page: 16, 32, 64, 128 or 256 */
  int32_t num_pages;     /* pages per layer; num_pages * Hkv * page_size < 2^31 */
  int32_t max_requests;  /* rows of the block tables, 1 .. 4096 */
  int32_t max_pages_per_request;  /* W, entries per row; W * page_size <= 2^24 */
  int32_t max_tokens;    /* most new tokens of one step, 1 .. 2^20 */
  int32_t cache_dtype;   /* KVRING_CACHE_* */
  int32_t rope_pairing;  /* KVRING_ROPE_* */
  int32_t reserved;      /* 0 */
  double rope_base;
} kvring_pages_config;

/* What a cache may have besides; a structure of its own, so that programs
 * that know nothing of it hold kvring_pages_config and kvring_pages_layout at
 * the sizes that they always had.  All zeros, but for `size`: nothing. */
typedef struct {
  int32_t size;          /* sizeof(kvring_pages_options) */
  int32_t scale_block;   /* E4M3: 0 = a scale per layer and head (kvring_pages_set_scales), or
                            KVRING_SCALE_BLOCK = a scale for every 16 tokens of a page and head, set by
                            kvring_pages_write */
  int32_t rope_pairs_t;  /* 0 = 1-D RoPE by a token's position in its request.  Else 3-D: of the
                            head_dim/2 pairs, [0, T) turn with t, [T, T + Y) with y, the rest with x
                            (any sizes, T >= 1), the coordinates being given to
                            kvring_pages_write_3d */
  int32_t rope_pairs_y;  /* Y (0 with 1-D RoPE) */
  int32_t rope_frequencies; /* KVRING_FREQ_* of 3-D RoPE (0 with 1-D) */
  int32_t max_position;  /* 3-D: coordinates lie in [0, max_position), at most 2^24; 0 = W * page_size
                            (0 with 1-D) */
  int32_t reserved;      /* 0 */
} kvring_pages_options;

#define KVRING_SCALE_BLOCK 16
#define KVRING_FREQ_SECTION 0    /* each section a RoPE of its own: its j-th of m pairs turns by
                                    coordinate * base^(-j/m), as the ring's */
#define KVRING_FREQ_HEAD 1       /* pair i turns by coordinate * base^(-2i/d), so equal coordinates turn
                                    a head as the 1-D position does */

/* Where things lie in the buffer given to kvring_pages_create (byte
 * offsets), for a caller's own kernels, snapshots and tests. */
typedef struct {
  size_t k_cache;      /* [L][num_pages][Hkv][page_size][d] cache_dtype */
  size_t v_cache;      /* the same */
  size_t scales;       /* float [L][4][Hkv]: scale_k, scale_v, 1/scale_k, 1/scale_v (1 at create) */
  size_t lengths;      /* int32 [max_requests]: committed lengths */
  size_t tables;       /* int32 [max_requests][W]: page ids, -1 where never set */
  size_t free_pages;   /* int32 [num_pages]: the stack of free page ids */
  size_t state;        /* int32 [KVRING_PAGES_STATE_WORDS] */
  size_t step_rows;    /* int32 [max_requests]: the planned requests' rows */
  size_t step_cu;      /* int32 [max_requests + 1]: first new token of each planned request */
  size_t step_lengths; /* int32 [max_requests]: their lengths with the new tokens */
  size_t positions;    /* int32 [max_tokens]: position of each new token in its request */
  size_t slots;        /* int32 [max_tokens]: page * page_size + offset, -1 for padding */
  size_t total;        /* bytes of the whole buffer */
} kvring_pages_layout;

#define KVRING_PAGES_STATE_FREE 0       /* free pages */
#define KVRING_PAGES_STATE_ERROR 1      /* KVRING_PAGES_ERR_* bits, never cleared by the library */
#define KVRING_PAGES_STATE_PLANNED 2    /* 1 while a plan awaits its commit */
#define KVRING_PAGES_STATE_REQUESTS 3   /* requests of the last plan */
#define KVRING_PAGES_STATE_TOKENS 4     /* its new tokens */
#define KVRING_PAGES_STATE_TAKEN 5      /* pages it takes */
#define KVRING_PAGES_STATE_WORDS 8

#define KVRING_PAGES_ERR_ROW 1u      /* a row outside [0, max_requests), or twice in one call */
#define KVRING_PAGES_ERR_TOKENS 2u   /* negative or more than max_new tokens, or more than num_tokens in all */
#define KVRING_PAGES_ERR_LENGTH 4u   /* a request longer than W pages */
#define KVRING_PAGES_ERR_PAGES 8u    /* not enough free pages */
#define KVRING_PAGES_ERR_COMMIT 16u  /* a commit with no plan before it */
#define KVRING_PAGES_ERR_TABLE 32u   /* a page id outside [0, num_pages) in a table or the free list */
#define KVRING_PAGES_ERR_TIMEOUT 64u /* a wait in the attention kernel gave up */
#define KVRING_PAGES_ERR_POSITION 128u /* a coordinate outside [0, max_position): the token was skipped */

/* The layout for a config; INVALID_ARG if the config is invalid (*out is
 * then zeroed).  layout.total is what kvring_pages_create needs. */
kvring_status kvring_pages_get_layout(const kvring_pages_config* cfg, kvring_pages_layout* out);

/* The same of a cache with options (NULL: none).  k_block_scales, v_block_scales (each may be
 * NULL): where the exponents of block scales lie, uint8 [L][num_pages][Hkv][page_size / 16], a
 * block's scale being 2^(byte - 127), E8M0 (127 at create); of no bytes without scale_block. */
kvring_status kvring_pages_get_layout_with(const kvring_pages_config* cfg, const kvring_pages_options* options,
                                           kvring_pages_layout* out, size_t* k_block_scales, size_t* v_block_scales);

/* Create a paged cache inside `dev_buf` (device memory of at least
 * layout.total bytes, 256-byte aligned, the caller's until after
 * kvring_pages_destroy).  Every row is empty, every page free (the stack
 * holds num_pages - 1 .. 0, so page 0 is taken first), scales are 1; cached
 * keys and values are not cleared.  Waits for its own set-up on `stream`. */
kvring_status kvring_pages_create(const kvring_pages_config* cfg, void* dev_buf, size_t bytes, void* stream,
                                  kvring_pages_t** out);
/* The same with options (NULL: none). */
kvring_status kvring_pages_create_with(const kvring_pages_config* cfg, const kvring_pages_options* options,
                                       void* dev_buf, size_t bytes, void* stream, kvring_pages_t** out);
kvring_status kvring_pages_destroy(kvring_pages_t* pages);

/* Take over a state: lengths int32 [max_requests], tables int32
 * [max_requests][W], free_pages int32 [n_free] (the stack, bottom first).
 * Device pointers, each either outside the cache's buffer or its own array,
 * which then stays as it is.  Drops a plan that awaits its commit. */
kvring_status kvring_pages_restore(kvring_pages_t* pages, const int32_t* lengths, const int32_t* tables,
                                   const int32_t* free_pages, int32_t n_free, void* stream);

/* Per-head scales of one layer of an E4M3 cache (device, float [Hkv] each):
 * a cached value is code * scale.  Must be positive and finite. */
kvring_status kvring_pages_set_scales(kvring_pages_t* pages, int32_t layer, const float* scale_k,
                                      const float* scale_v, void* stream);

/* Plan a step: request i (of num_requests) is row rows[i] of the tables
 * (rows NULL: row i) and gets new_tokens[i] >= 0 new tokens, positions
 * len .. len + new - 1.  Both are device int32 arrays, outside the step's own.
 * On the device:
 *   step_cu       exclusive sums of new_tokens (num_requests + 1 entries)
 *   step_lengths  length + new
 *   tables        entries of the pages the new tokens need beyond those the
 *                 request has, taken from the free stack
 *   positions, slots  for tokens 0 .. num_tokens - 1; those past the last
 *                 request's get slot -1, position 0
 * num_tokens (<= max_tokens) is the token count of the step's tensors, at
 * least the sum of new_tokens; max_new bounds every new_tokens[i] and lets
 * kvring_pages_attention pick its kernels (num_tokens if unknown).
 * Lengths and the free list change only with kvring_pages_commit: a plan
 * that is not committed is dropped by the next one and costs nothing.
 * A plan that cannot be made (rows, tokens, length or pages: see the error
 * bits) sets its error bit and plans no token for any request.  A page id
 * outside the pool does not stop a plan: it sets KVRING_PAGES_ERR_TABLE, its
 * tokens get slot -1 and are not written, and attention reads zeros there. */
kvring_status kvring_pages_plan(kvring_pages_t* pages, const int32_t* rows, const int32_t* new_tokens,
                                int32_t num_requests, int32_t num_tokens, int32_t max_new, void* stream);

/* Make the last plan final: row lengths and the free list. */
kvring_status kvring_pages_commit(kvring_pages_t* pages, void* stream);

/* End num_requests requests: their pages go back to the free stack (in the
 * order of `rows` (device int32), each request's first page first) and
 * their lengths to 0.  Rows that are already empty are allowed; a row out
 * of range or given twice sets KVRING_PAGES_ERR_ROW and nothing is
 * released.  A table entry that is no page of the pool sets
 * KVRING_PAGES_ERR_TABLE and does not go back; the other pages do.  Drops a plan that awaits its commit, and empties the step. */
kvring_status kvring_pages_release(kvring_pages_t* pages, const int32_t* rows, int32_t num_requests, void* stream);

/* Keys, values and queries of the planned tokens, for one layer:
 *   y = x * rsqrt(mean(x^2) + eps) * weight   per head row (q_weight,
 *       k_weight: bf16 [d]; NULL leaves q or k as it is)
 *   q_out[t] = rope(y_q, positions[t]), bf16 [num_tokens][Hq][d] contiguous
 *   K page   = rope(y_k, positions[t]), V page = v
 * at slots[t].  An E4M3 cache stores e4m3(value * (1/scale)).  Everything
 * between reading bf16 and the one rounding of the result is fp32, the squares
 * too: a normed row whose mean square leaves fp32's range (values of 2^63 and
 * more) comes out as zeros, and with eps 0 one of 2^-60 and less has no meaning.
 * q, k, v: bf16, row (t, h) at base + t * token_stride + h * d (elements;
 * strides a multiple of 8, at least that of heads * d), so slices of one
 * packed projection output can be passed.  q_out must not overlap them, the
 * weights or the cache's buffer.
 * q, k and v hold num_tokens (<= max_tokens) tokens: rows past the plan's may be
 * read, whatever they hold has no effect, and those of q_out stay as they were. */
kvring_status kvring_pages_write(kvring_pages_t* pages, int32_t layer, const void* q, const void* k, const void* v,
                                 int64_t q_stride, int64_t k_stride, int64_t v_stride, const void* q_weight,
                                 const void* k_weight, float eps, void* q_out, int32_t num_tokens, void* stream);

/* kvring_pages_write for a cache with 3-D RoPE: coords int32 [num_tokens][3] = (t, y, x)
 * of every token (device; outside q_out and the cache's buffer).  Where tokens
 * go and what attention lets them see stays with their places in the request.  A
 * token with a coordinate outside [0, max_position) sets
 * KVRING_PAGES_ERR_POSITION; its row of q_out and its place in the cache stay as
 * they were (with block scales its codes do, and the block's scale where the step has
 * no other token in it; once committed, the place counts as one that holds a token).
 * kvring_pages_write refuses such a cache, and this call a 1-D one.
 *
 * In a cache with block scales (either call) 16 tokens at places 16 b .. 16 b + 15
 * of a request share a scale per head, of keys and of values:
 *   need  = least 2^e with |value| <= 448 2^e for the step's tokens in the block,
 *           e in [-40, 40] (beyond, values saturate or vanish)
 *   scale = need, or max(need, the scale so far) where the block holds tokens
 *           from before; these are then rounded to the new scale,
 *           code = e4m3(code * (old / new))
 *   code  = e4m3(value / scale)
 * Values that are not finite have no part in `need`: infinities saturate, NaN stays.
 * A scale raised by a write whose plan is then dropped stays raised, and the
 * tokens rounded to it.  A block that two rows of the tables share must not be
 * appended to. */
kvring_status kvring_pages_write_3d(kvring_pages_t* pages, int32_t layer, const void* q, const void* k, const void* v,
                                    int64_t q_stride, int64_t k_stride, int64_t v_stride, const void* q_weight,
                                    const void* k_weight, float eps, const int32_t* coords, void* q_out,
                                    int32_t num_tokens, void* stream);

/* Attention of the planned tokens' queries over their requests' cached
 * tokens, the new ones included:
 *   out[t,h] = sum_j softmax_j(scale * q[t,h] . K[j,h/G]) V[j,h/G]
 * causal != 0: j <= position of t, and with window > 0 also
 * j > position - window; causal == 0: every cached and new token of the
 * request (window must be 0).  scale 0 means 1/sqrt(d).  q (rotated) and
 * out: bf16 [num_tokens][Hq][d], q with a token stride (elements, a multiple
 * of 8), out contiguous, overlapping neither q nor the cache's buffer; rows
 * past the plan's tokens stay as they were.  Scores, softmax statistics and sums are fp32; probabilities
 * are rounded once, to bf16 (f16 over an E4M3 cache; over block scales what is
 * rounded is the probability with its value's scale).  Block scales' bytes outside 87 .. 167
 * (2^-40 .. 2^40) are read as the nearest of these, and a row of queries whose factor, 2^e scale
 * log2(e) with 2^e the power of two at or below its largest size, is beyond 2^69 as one of 2^69
 * (its scores keep their order).  Finite cached values
 * of any size give finite results at any length.  Cached tokens that
 * a query's mask hides do not affect it, whatever they hold. */
kvring_status kvring_pages_attention(kvring_pages_t* pages, int32_t layer, const void* q, int64_t q_stride, void* out,
                                     int32_t num_tokens, int32_t causal, int32_t window, float scale, void* stream);

/* Test support for the bounded waits of the attention kernels: as
 * kvring_debug_set_attention_wait (limit_ns in [1000, 6e10], stall 0 or 1).
 * A call whose waits gave up sets KVRING_PAGES_ERR_TIMEOUT and leaves `out`
 * undefined; plan again before the next call. */
kvring_status kvring_pages_debug_set_wait(kvring_pages_t* pages, int64_t limit_ns, int32_t stall);

/* Copy the ring out for inspection (tests, snapshots).  Any pointer may be
 * NULL to skip that part.  k_out, v_out: uint8 [H][capacity][d] codes;
 * scales: float [4H] = scale_k, scale_v, inv_scale_k, inv_scale_v;
 * slot_pos: int32 [capacity] (INT32_MIN = empty); state: int32
 * [KVRING_STATE_WORDS].  Destinations may be device or pinned host memory;
 * the copies are enqueued on `stream` (the caller synchronises). */
kvring_status kvring_export(kvring_t* ring, void* k_out, void* v_out, float* scales,
                            int32_t* slot_pos, int32_t* state, void* stream);

/* Test support, not part of the cache: encode n fp32 values to E4M3 codes
 * with the same conversion the kernels use (device pointers). */
kvring_status kvring_debug_encode_e4m3(const float* in, uint8_t* out, int64_t n, void* stream);

/* Measurement support: the fixed cost of kvring_write_frame for n tokens.
 * Launches a kernel with the write's grid, launch mode (a programmatic
 * dependent of the preceding kernel), wait, ring-state read, completion
 * ticket and state publication, but no data: nothing is read from the
 * frame, nothing written to the cache, and the ring state is rewritten with
 * its current values.  (The delta rotation's counterpart is
 * kvring_delta_rotate with delta 0, which moves no rows.)
 * Errors: INVALID_ARG, CAPACITY (as kvring_write_frame). */
kvring_status kvring_debug_write_floor(kvring_t* ring, int32_t n, void* stream);

/* Test support for the attention kernel's bounded waits.  Every wait in the
 * kernel gives up after limit_ns of wall time (default one second); a wait
 * that gives up sets KVRING_DEVERR_TIMEOUT in the ring's error word and the
 * kernel drains its copies and MMAs, frees its tensor memory and returns, so
 * the context stays usable.  With stall = 1 the kernel's first QK waits on a
 * barrier that nothing ever completes, so every following attention call on
 * this ring takes that path on purpose (its output is not the attention);
 * stall = 0 restores normal calls.  Host-side setting only: takes effect on
 * calls enqueued afterwards.
 * Errors: INVALID_ARG (limit_ns outside [1000, 6e10], stall not 0 or 1). */
kvring_status kvring_debug_set_attention_wait(kvring_t* ring, int64_t limit_ns, int32_t stall);

/* Test support for the attention's early query preparation.  With default
 * positions the kernel prepares its queries before waiting for the
 * preceding kernel, for the positions implied by a next-position hint that
 * every write leaves as it starts, and after the wait redoes the
 * preparation if the ring's next position turned out different.  With
 * wrong = 1 the guess of every following attention call on this ring is
 * off by max_position (so also outside the RoPE table, which must not be
 * reported), which exercises the redo; wrong = 0 restores normal calls.
 * Host-side setting only: takes effect on calls enqueued afterwards.
 * Errors: INVALID_ARG (wrong not 0 or 1). */
kvring_status kvring_debug_attention_guess(kvring_t* ring, int32_t wrong);

/* Test support: the precision level (1..4) each attention tile used in the
 * last kvring_attention call, int32 [ceil(n_q/128)][H], copied to `levels`
 * (device or pinned host) on `stream`. */
kvring_status kvring_debug_attention_levels(kvring_t* ring, int32_t* levels, void* stream);

/* Test support: how many kvring_write_frame and kvring_attention calls so
 * far (in this process, all rings and streams) found that the previous
 * library kernel on their stream may write their frame or queries, and so
 * read them only after waiting for it. */
int64_t kvring_debug_late_reads(void);

/* Static text for a status code. */
const char* kvring_status_string(kvring_status s);

#ifdef __cplusplus
}
#endif
#endif /* KVRING_H */
