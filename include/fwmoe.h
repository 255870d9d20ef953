/*
 * fwmoe — the routed mixture-of-experts feed-forward step over Q8_0 weights,
 * on one NVIDIA GB300 (sm_103a). C ABI.
 *
 * The step (the Flyweight README, "flyweight-llm" 0.2.0, §Features: "sparse
 * MoE execution"; §Quantization: grouped routed-expert GPU kernels for Q8_0
 * among other formats; the pages print no formula, and the reading used here
 * is the standard top-k softmax router):
 *
 *   z[t,e]   = sum_h x[t,h] * router_w[e,h] + router_bias[e]        (fp32)
 *   ids[t,:] = the k largest z[t,.]; ties go to the lower expert id; ordered
 *              by descending z (equal z: lower id first)
 *   gates    = softmax of z[t,.] restricted to ids[t,:], renormalised to sum 1
 *   y_e(x)   = W_down,e ( SiLU(W_gate,e x) * (W_up,e x) ),  SiLU(a) = a/(1+e^-a)
 *   out[t]   = sum_j gates[t,j] * y_{ids[t,j]}(x_t)  (+ y_shared(x_t), weight 1)
 *
 * There is no residual add: out is the MoE output only.
 *
 * Q8_0 weight layout accepted by fw_moe_init (GGUF convention; the pages name
 * the format, §Quantization): each matrix row is cut along its input dimension
 * into blocks of 32 values, each block 34 bytes: a little-endian IEEE binary16
 * scale d, then 32 int8 codes q; the weight is d*q. Expert matrices are stored
 * back to back, expert-major: w_gate / w_up are E x [I rows x H/32 blocks],
 * w_down is E x [H rows x I/32 blocks].
 *
 * Conventions for every call:
 *  - Pointers named "device" are CUDA device pointers owned by the caller.
 *  - `stream` is a cudaStream_t (NULL = legacy default stream). Calls enqueue
 *    asynchronously; none synchronises except fw_moe_init, fw_moe_free,
 *    fw_moe_status and fw_moe_forward_host.
 *  - Argument errors are reported before anything is enqueued. A failed call
 *    returns a negative fw_status and fw_moe_last_error() describes it.
 *  - There is no CPU fallback: without an sm_103 device, fw_moe_init fails
 *    with FW_EUNSUPPORTED.
 */
#ifndef FWMOE_H
#define FWMOE_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FW_OK = 0,
  FW_EINVAL = -1,       /* bad argument (null pointer, size, alignment) */
  FW_ENOMEM = -2,       /* device allocation failed */
  FW_ECUDA = -3,        /* a CUDA call or launch failed */
  FW_EUNSUPPORTED = -4, /* no sm_103 device, or a shape this build does not handle */
  FW_ESTATE = -5,       /* call order broken (e.g. ffn with a T other than the last route's) */
  FW_ETIMEOUT = -6,     /* a kernel gave up a bounded wait (see fw_moe_status) */
  FW_EDEVICE = -7       /* a kernel reported a failed index or layout check */
} fw_status;

typedef struct fw_moe_handle fw_moe_handle; /* opaque; one handle = one MoE layer */

/* Layer shape. H and I must be multiples of 64, not only of the Q8_0 block
 * length 32: the prefill GEMMs step K by 64 (two Q8_0 blocks per 128-byte
 * swizzled shared-memory row). Every Qwen/DeepSeek-shaped MoE layer the pages
 * speak of meets this. */
typedef struct {
  int32_t H;            /* hidden size; multiple of 64 */
  int32_t I;            /* per-expert intermediate size; multiple of 64 */
  int32_t E;            /* routed experts, 1..256 */
  int32_t k;            /* experts per token, 1..min(E, 16) */
  int32_t n_shared;     /* always-on shared experts: 0 or 1 */
  int32_t T_max;        /* largest T any call on this handle may pass (sizes the workspace) */
  int32_t decode_T_max; /* T <= this takes the decode (grouped GEMV) path; 0 = 16; at most 16.
                         * The decode kernel holds a call's x in shared memory: one token
                         * up to H = 14336, several up to H = 2048; calls past that take
                         * the prefill path whatever their T. */
  int32_t act_q8;       /* 0: bf16 activations (the default step). 1: Q8 activations on the
                         * decode path (the Flyweight README, §Quantization: Q8-activation
                         * dp4a decode kernels): each token's x quantised per 32-block and
                         * each expert's h = SiLU(g)*u per 16-block by the Q8_0 rule in fp32
                         * (d = amax/127, codes round-half-away(v/d)), integer dot products
                         * with the Q8_0 weights, scales applied per block. The prefill path
                         * keeps bf16 activations (sm_103a has no int8 tensor-core MMA). */
} fw_moe_config;

typedef struct { /* all DEVICE pointers, read only during fw_moe_init */
  const float *router_w;       /* [E, H] fp32 row-major */
  const float *router_bias;    /* [E] fp32 or NULL; added to the logits (selection and gates) */
  const uint8_t *w_gate;       /* E x [I x H/32] Q8_0 blocks */
  const uint8_t *w_up;         /* E x [I x H/32] Q8_0 blocks */
  const uint8_t *w_down;       /* E x [H x I/32] Q8_0 blocks */
  const uint8_t *shared_gate;  /* [I x H/32] Q8_0, or NULL when n_shared == 0 */
  const uint8_t *shared_up;    /* [I x H/32] Q8_0, or NULL when n_shared == 0 */
  const uint8_t *shared_down;  /* [H x I/32] Q8_0, or NULL when n_shared == 0 */
} fw_moe_weights;

/* How a layer's router chooses and weights its experts. The default (until
 * fw_moe_set_routing) is the step above. Under a rule:
 *   s[t,e]   = softmax of z[t,.] over all E, or 1 / (1 + e^-z[t,e])
 *   c[t,e]   = s[t,e] + select_bias[e]
 *   groups   : n_group runs of E / n_group neighbouring experts; a group's score is
 *              the sum of its two largest c (its only one); the top_group groups of
 *              largest score stay, ties to the lower group
 *   ids[t,:] = the k largest c of the groups that stay, descending, ties to the lower id
 *   gates    = scale * s[t,ids], divided by (their sum of s + 1e-20) when renorm
 * (The vOOM README speaks of DeepSeek-shaped experts and routers, the Flyweight
 * README's served families name that MoE too; the pages print no formula, and this
 * is the reading used.) A NaN among a token's logits is no score: the softmax is over the
 * others, a group's score is made of the others' c, and its expert ranks below every number;
 * where it is chosen all the same, its gate is NaN, and under renorm all of the token's. Infinite
 * logits have the scores' limits (several of +infinity share a softmax evenly). */
typedef struct {
  int32_t score;               /* 0 softmax over all experts, 1 sigmoid */
  int32_t n_group, top_group;  /* 1..32, dividing E; 1..n_group, with k experts at least in that many groups. 1, 1: no groups */
  int32_t renorm;              /* 0 or 1 */
  float scale;                 /* positive, finite */
  const float *select_bias;    /* DEVICE [E] or NULL (zeros); only moves the choice */
} fw_moe_routing;

/* Create a layer (the pages' runtime loads routed experts of GGUF Q8_0 models
 * onto the GPU for its grouped kernels: Flyweight README, §Quantization and
 * §Features): validates the shapes, copies the router and repacks every
 * Q8_0 matrix into the handle's own device memory (a byte-preserving change of
 * layout: int8 code planes plus binary16 scale planes), allocates the
 * workspace for T_max tokens and synchronises `stream` once. The caller may
 * free its weight buffers afterwards. *out receives the handle. */
fw_status fw_moe_init(const fw_moe_config *cfg, const fw_moe_weights *w, void *stream, fw_moe_handle **out);

/* Set the layer's routing rule (NULL: back to the default step) for the routes and
 * forwards from here on; a route made before is no longer valid for fw_moe_ffn.
 * select_bias is copied into the handle in stream order (the first rule of a handle
 * also allocates for it: not inside a stream capture). A captured graph keeps the
 * rule that it was captured with, and reads the bias set last. */
fw_status fw_moe_set_routing(fw_moe_handle *h, const fw_moe_routing *routing, void *stream);

/* The router step (Flyweight README, §Current limitations: dynamic MoE routing;
 * vOOM README, router/top-k substeps; the reading: fp32 logits, top-k with ties
 * to the lower id, softmax restricted to the k and renormalised).
 * Routing for T tokens (0 <= T <= T_max): x is DEVICE bf16 [T, H] row-major.
 * Writes expert_ids (DEVICE int32 [T, k]) and gates (DEVICE fp32 [T, k], may be
 * NULL), and keeps the routing and the token-to-expert grouping in the handle
 * for the next fw_moe_ffn. T == 0 is a no-op. */
fw_status fw_moe_route(fw_moe_handle *h, const void *x, int32_t T, int32_t *expert_ids, float *gates,
                       void *stream);

/* The routed-expert step (Flyweight README, §Features "sparse MoE execution",
 * §Quantization: grouped routed-expert kernels over Q8_0; vOOM README: SwiGLU
 * experts, shared experts): each selected expert's SiLU(gate) * up then down
 * projection, gate-weighted and summed in slot order (+ the shared expert).
 * Experts and combine for the routing made by the last fw_moe_route on this
 * handle: same x, same T, same stream. out is DEVICE bf16 [T, H] row-major.
 * A T different from the last route's returns FW_ESTATE. */
fw_status fw_moe_ffn(fw_moe_handle *h, const void *x, int32_t T, void *out, void *stream);

/* fw_moe_route followed by fw_moe_ffn (expert_ids may not be NULL; gates may). */
fw_status fw_moe_forward(fw_moe_handle *h, const void *x, int32_t T, int32_t *expert_ids, float *gates, void *out,
                         void *stream);

/* The whole step from and to HOST memory: copies x (bf16 [T, H]) to the device,
 * runs fw_moe_forward on the handle's own device buffers, copies expert_ids
 * (int32 [T, k]) and out (bf16 [T, H]) back and synchronises `stream`. Host
 * buffers should be pinned for the copies to be asynchronous. */
fw_status fw_moe_forward_host(fw_moe_handle *h, const void *x_host, int32_t T, int32_t *expert_ids_host,
                              void *out_host, void *stream);

/* The token-to-expert permutation the grouped kernels run on (Flyweight
 * README, §Runtime controls: block-table kernels for routed experts).
 * Token-to-expert grouping of the last route (for tests and tools): offsets
 * DEVICE int32 [E + 1], the exclusive prefix sum of the per-expert counts;
 * perm DEVICE int32 [T*k], the slot ids s = t*k + j grouped by ascending expert
 * and, within an expert, by ascending token; inv DEVICE int32 [T*k] (may be
 * NULL), inv[perm[p]] = p. */
fw_status fw_moe_get_permutation(fw_moe_handle *h, int32_t *offsets, int32_t *perm, int32_t *inv, void *stream);

/* Copy one repacked matrix of one expert back out in the GGUF Q8_0 layout
 * (which: 0 gate, 1 up, 2 down; expert E is the shared expert). blocks is
 * DEVICE memory of rows x K/32 x 34 bytes. Round-trips fw_moe_init's input. */
fw_status fw_moe_export_q8_0(fw_moe_handle *h, int32_t expert, int32_t which, uint8_t *blocks, void *stream);

/* A chain of layer calls captured once as one CUDA graph and replayed by a
 * single launch (Flyweight README, §Current limitations: host
 * synchronisation points of dynamic MoE routing, persistent layer kernels
 * listed as incomplete; §Features: CUDA-graph replay of decode). No call of
 * fw_moe_forward synchronises with the host -- routing, grouping and tile
 * lists stay on the device for both paths -- so n of them capture into one
 * graph. Call i runs fw_moe_forward(layers[i], x[i], T, expert_ids[i], NULL,
 * out[i]): x[i] and out[i] DEVICE bf16 [T, H_i], 16-byte aligned (out[i] may be
 * x[i + 1], chaining the layers); expert_ids[i] DEVICE int32 [T, k_i]. The
 * handles, T and every pointer are fixed at capture; the buffers' contents
 * are read at each launch. Capture runs on a stream of its own on the current
 * device, which must be every layer's. Replays of one graph, and other work
 * on its layers, must not overlap (they share each handle's workspace).
 * Errors: FW_EINVAL for arguments (before any CUDA call), FW_ESTATE if a layer
 * is profiling, else what a capture or instantiation reports. */
typedef struct fw_moe_graph fw_moe_graph;
fw_status fw_moe_graph_create(fw_moe_handle *const *layers, int32_t n, int32_t T, const void *const *x,
                              void *const *out, int32_t *const *expert_ids, fw_moe_graph **graph);
/* Enqueue one replay of the chain on `stream`. */
fw_status fw_moe_graph_launch(fw_moe_graph *graph, void *stream);
/* Release the graph (not its layers). NULL is a no-op. */
fw_status fw_moe_graph_destroy(fw_moe_graph *graph);

/* Synchronise `stream`, read and clear the handle's device status word.
 * FW_OK, FW_ETIMEOUT or FW_EDEVICE. */
fw_status fw_moe_status(fw_moe_handle *h, void *stream);

/* Kernel kinds reported by fw_moe_profile_end. */
enum {
  FW_KERNEL_ROUTE_DECODE = 0, /* decode router: GEMV, top-k, gates, grouping */
  FW_KERNEL_ROUTE_TILES = 1,  /* prefill router: tiled GEMM, top-k, per-tile counts */
  FW_KERNEL_ROUTE_SCAN = 2,   /* prefill grouping: offsets, tile lists */
  FW_KERNEL_ROUTE_SCATTER = 3,/* prefill grouping: stable scatter */
  FW_KERNEL_DECODE_EXPERTS = 4, /* decode experts: gate/up GEMV + SiLU, grid barrier, down GEMV + combine */
  FW_KERNEL_RESERVED_5 = 5,
  FW_KERNEL_PREFILL_GATEUP = 6,  /* prefill gate/up grouped GEMM (tcgen05) + SiLU */
  FW_KERNEL_PREFILL_DOWN = 7,    /* prefill down grouped GEMM (tcgen05) x gate */
  FW_KERNEL_PREFILL_COMBINE = 8, /* prefill un-permute and sum */
  FW_KERNEL_PREFILL_GATHER = 9, /* prefill: x rows gathered into grouped order */
  FW_KERNEL_PREFILL_GATEUP_SMALL = 10, /* prefill gate/up GEMM over the tiles of at most 64 rows */
  FW_KERNEL_PREFILL_DOWN_SMALL = 11,   /* prefill down GEMM over the tiles of at most 64 rows */
  FW_KERNEL_PREFILL_GATEUP_MID = 12,   /* prefill gate/up GEMM over the tiles of 65 to 96 rows */
  FW_KERNEL_PREFILL_DOWN_MID = 13,     /* prefill down GEMM over the tiles of 65 to 96 rows */
  FW_KERNEL_KINDS = 16
};

/* Optional per-kernel timing, for measurement tools. After
 * fw_moe_profile_begin, every kernel this handle launches (up to max_launches)
 * is bracketed by CUDA events recorded on its own stream; this serialises the
 * kernels (no programmatic overlap), so profile in a pass of its own.
 * fw_moe_profile_end synchronises, writes per kind (arrays of n_kinds, at most
 * FW_KERNEL_KINDS) the summed milliseconds and the launch count, and stops
 * recording. Creating the events happens in begin, not on the launch path. */
fw_status fw_moe_profile_begin(fw_moe_handle *h, int32_t max_launches);
fw_status fw_moe_profile_end(fw_moe_handle *h, int32_t n_kinds, float *total_ms, int32_t *launches);

/* Release the handle (no counterpart on the pages: resource management of
 * this library). Synchronises its device first. NULL is a no-op; a
 * handle already freed is detected (FW_EINVAL) as long as its memory has not
 * been reused. */
fw_status fw_moe_free(fw_moe_handle *h);

/* Text of the last failed call on this thread ("" if none). No counterpart
 * on the pages. */
const char *fw_moe_last_error(void);

/* Routing only (logits, top-k with ties to the lower id, renormalised gates)
 * for callers that must not allocate device memory: code that runs inside a
 * framework whose memory manager owns every byte of the device (a serving
 * engine's pool or a fixed arena), or on a latency path where cudaMalloc's
 * implicit synchronisation is not acceptable. It needs no handle: x is DEVICE
 * bf16 [T, H], router_w DEVICE fp32 [E, H] (16-byte aligned), router_bias
 * DEVICE fp32 [E] or NULL; writes expert_ids DEVICE int32 [T, k] and gates
 * DEVICE fp32 [T, k] (may be NULL), the same values fw_moe_route writes.
 * The pages have no counterpart: this is a convenience of this library.
 *
 * Its only scratch (the T x E logits and a ticket counter, 16.25 KiB) is a
 * file-scope __device__ array that every GPU loading this library holds until
 * process exit; limits: T <= 16, E <= 256, k <= min(E, 16), H % 4 == 0, beyond
 * which it returns FW_EINVAL with text. The first call on a device looks the
 * array's device address up (cudaGetSymbolAddress, with that device
 * current); make that first call before any stream capture. Each call clears
 * the ticket in stream order. All calls share the one array and it keeps the
 * last call's contents: calls that can overlap on the GPU (other streams, or
 * other threads' streams) race and must be serialised by the caller. It calls
 * no cudaMalloc, cudaFree or allocating library routine. `stream` must belong
 * to the current device (checked: FW_EINVAL otherwise); the looked-up address
 * is kept for the life of the process, so after a cudaDeviceReset of the
 * device this entry point (like every handle) may no longer be used. */
fw_status fw_moe_route_noalloc(const void *x, int32_t T, int32_t H, const float *router_w, const float *router_bias,
                               int32_t E, int32_t k, int32_t *expert_ids, float *gates, void *stream);

/* A tool for preparing inputs, not a step of the MoE layer (the pages name
 * the GGUF Q8_0 format, Flyweight README §Quantization; the layer itself
 * never quantises). Quantise fp32 weights to Q8_0 on the GPU: w DEVICE [rows, K] row-major fp32,
 * K % 32 == 0; blocks DEVICE rows x K/32 x 34 bytes. Per block of 32:
 * amax = max|w|, d = amax/127 (fp64), q = round-half-away-from-zero(w/d)
 * clamped to +-127 (fp64), d stored as binary16 (round to nearest even);
 * an all-zero block stores zeros. */
fw_status fw_q8_0_quantize(const float *w, int64_t rows, int64_t K, uint8_t *blocks, void *stream);

/* ------------------------------------------------------------------------
 * The attention side of the same layer (the Flyweight README, §Features:
 * attention with tensor-core prefill, sliding window; §Quantization:
 * KV-cache codecs; the pages print no formula or layout, and the readings
 * below are this library's own): the step's plan, the norms and rotation of
 * queries and keys, and attention over a paged key/value cache held in 4 bits.
 * These calls need no handle: the caller owns every buffer, the cache among
 * them. They never synchronise and allocate nothing, so they capture into
 * CUDA graphs. Bad values that only the device sees (a slot or position out of
 * range) are skipped and reported as FW_KV_* bits in a caller's status word.
 *
 * Page format. A page holds P positions (16, 32, 64 or 128) of one request for
 * every key/value head; the cache is n_pages x n_kv blocks of P * D * 9 / 8
 * bytes, 16-byte aligned, D = 64 or 128 dims a head, NB = D / 32:
 *   K codes  [P][4 q][NB b] 32-bit words: dims 32 b + 8 q + i; nibbles 0..3
 *            hold i = 0, 2, 4, 6 and nibbles 4..7 hold i = 1, 3, 5, 7
 *   K scales [P][NB] bf16
 *   V codes  [P / 2][8 g][NB b] 32-bit words: dims 32 b + 4 g + i; nibbles
 *            0..3 hold i = 0..3 of the even position, 4..7 of the odd one
 *   V scales [P / 2][NB][2] bf16: the even position's, the odd position's
 * The value of a code c in 0..15 is d * (c - 8). A block of 32 values x takes
 * d = its element of largest magnitude (of a tie the positive one) / -8 and
 * c = round-half-even(x / d) + 8 clamped to 0..15 (d = 0: c = 8); d is exact in
 * bf16 for the bf16 keys and values stored here (of blocks with a largest
 * magnitude below 2^-123 rounded to a multiple of 2^-133). A block holding an infinity
 * or NaN stands for non-finite values. A slot is page * P + place in the page. */
enum {
  FW_KV_POOL_EMPTY = 1,   /* the plan ran out of free pages */
  FW_KV_TABLE_FULL = 2,   /* a request needs more than max_blocks pages */
  FW_KV_TOKENS_FULL = 4,  /* more new tokens than T_cap */
  FW_KV_BAD_LENGTH = 8,   /* a negative length, or one above 2^30 (taken as 0) */
  FW_KV_BAD_SLOT = 16,    /* a slot or page id outside the cache */
  FW_KV_BAD_POSITION = 32, /* a position outside the cos_sin table */
  FW_KV_TIMEOUT = 64,     /* a kernel gave up a bounded wait; its outputs mean nothing */
  FW_KV_BAD_QUERIES = 128 /* a request's q_start entries decrease, leave 0..T or bring more than max_q */
};

/* The plan of a step, made on the GPU from the requests' lengths: all DEVICE
 * int32. Request r has cached_lens[r] positions in the cache and brings
 * new_lens[r] more (0 is allowed for both). Its pages are block_table[r][0 ..];
 * the first ceil(cached / page) entries are read, the entries of the pages its
 * new positions open are WRITTEN, taken from free_pages in request order,
 * starting at entry *free_used (NULL: 0). Outputs: q_start [R + 1], the
 * exclusive sum of new_lens; seq_lens [R] = cached + new; for each of T_cap
 * token places requests, positions and slots (-1 past the last token); counts
 * [3] = {tokens, free-list entries used, *free_used included, FW_KV_* bits}.
 * Without a page for it a token's slot, and its table entry, is -1; of a page id
 * that no cache can have the slot is 2^31 - 1; tokens past
 * T_cap are not placed and the entries of pages they open not written. The next
 * step may pass this call's counts + 1 as free_used, with other counts. */
fw_status fw_kv_plan(const int32_t *cached_lens, const int32_t *new_lens, int32_t R, int32_t page,
                     int32_t *block_table, int32_t max_blocks, const int32_t *free_pages, int32_t n_free,
                     const int32_t *free_used, int32_t T_cap, int32_t *q_start, int32_t *seq_lens,
                     int32_t *requests, int32_t *positions, int32_t *slots, int32_t *counts, void *stream);

/* Norms of queries and keys for each head with the position rotation in the
 * same pass, and the store into the cache: per head row x of D bf16 values
 *   y = x / sqrt(mean(x^2) + eps) * norm           (norm NULL: y = x)
 *   (a, b) -> (a cos - b sin, b cos + a sin)       over rot dims, the rest as is
 * in fp32, rounded once to bf16. The pairs (a, b) are dims (i, i + rot / 2), or
 * (2 i, 2 i + 1) when interleaved. cos_sin [n_pos][rot] fp32 holds a position's
 * rot / 2 cosines, then its sines. With a cache, the rotated keys (as rounded
 * to bf16) and the values v are quantised into the tokens' slots; a slot of -1
 * stores nothing, and a position of -1 (padding) is rotated as position 0.
 * Two tokens of a call may not share a slot. Outputs may be their inputs. */
typedef struct {
  int32_t T, n_q, n_kv, D;   /* tokens, query heads, key/value heads, dims a head (64 or 128) */
  int32_t rot;               /* dims rotated: a multiple of 16, 0..D */
  int32_t interleaved;       /* 0 or 1 */
  float eps;
  int32_t n_pos;             /* rows of cos_sin */
  const void *q, *k, *v;     /* DEVICE bf16 [T][heads][D]; v read only with a cache */
  int64_t q_stride, k_stride, v_stride; /* elements between tokens; multiples of 8 */
  const float *q_norm, *k_norm;         /* DEVICE fp32 [D] or NULL */
  const float *cos_sin;      /* DEVICE fp32 [n_pos][rot] */
  const int32_t *positions;  /* DEVICE [T] */
  void *q_out, *k_out;       /* DEVICE bf16; k_out may be NULL with a cache */
  int64_t q_out_stride, k_out_stride;
  void *cache;               /* DEVICE, or NULL */
  const int32_t *slots;      /* DEVICE [T], with a cache */
  int32_t page, n_pages;
  int32_t *status;           /* DEVICE, FW_KV_* bits are OR-ed in; or NULL */
} fw_qk_norm_rope_args;
fw_status fw_qk_norm_rope(const fw_qk_norm_rope_args *args, void *stream);

/* The keys and values that slots hold, as bf16 [T][n_kv][D] (d * (c - 8)
 * rounded; zeros for a slot of -1): for tests and for moving a cache. */
fw_status fw_kv_export(const void *cache, int32_t n_pages, int32_t n_kv, int32_t D, int32_t page,
                       const int32_t *slots, int32_t T, void *k, void *v, int32_t *status, void *stream);

/* Causal attention of a step's new tokens over the cache, which already holds
 * their own keys and values. Tokens q_start[r] .. q_start[r + 1] - 1 belong to
 * request r and are its last positions: the i-th of n stands at
 * p = seq_lens[r] - n + i and sees position j when
 *   j <= p and (window == 0 or j > p - window or j < sinks)
 * Query head h reads key/value head h / (n_q / n_kv). A row that sees nothing
 * gives zeros; what is masked is never part of a result, whatever it holds.
 * Softmax statistics and sums are fp32. Besides the output, what is rounded:
 * for requests of up to 16 query rows (new tokens x n_q / n_kv) a probability times
 * its value block's scale, to bf16; for others a probability alone, to f16 (2^-11,
 * and 2^-28 of the row's largest), but a probability and a value, to bf16, in 128
 * neighbouring positions with a block of values whose largest magnitude is neither
 * zero nor within 2^-7 .. 2^7. Sums of values past 2^100 may be infinite. Keys and queries are exact
 * (for requests of more than 16 rows but for what is below 2^-37 of the largest key
 * of 128 neighbours, or 2^-25 of the largest element of a query row; a row with
 * none above 2^-100 is taken to have that). max_q is the largest number of new
 * tokens of a request, or more, up to T. A request that brings more than max_q, or whose
 * q_start entries decrease or leave 0..T, is reported and its rows are not written.
 * Rows of q past q_start[R] are neither read nor written.
 * workspace: DEVICE, 16-byte aligned, at least fw_attn_q4_workspace bytes; its
 * contents mean nothing between calls, and calls that may overlap need one each. */
typedef struct {
  int32_t R, T, max_q;       /* requests, rows of q, most new tokens of a request */
  int32_t n_q, n_kv, D;
  int32_t page, n_pages, max_blocks; /* max_blocks: entries of a block_table row */
  int32_t window, sinks;
  float scale;               /* > 0; usually 1 / sqrt(D) */
  const void *q;             /* DEVICE bf16 [T][n_q][D] */
  void *out;                 /* DEVICE bf16 [T][n_q][D] */
  int64_t q_stride, out_stride; /* elements between tokens; multiples of 8 */
  const void *cache;         /* DEVICE */
  const int32_t *block_table, *q_start, *seq_lens; /* DEVICE [R][max_blocks], [R + 1], [R] */
  int32_t *status;           /* DEVICE, FW_KV_BAD_SLOT, _BAD_QUERIES and _TIMEOUT are OR-ed in; or NULL */
} fw_attn_q4_args;
fw_status fw_attn_q4_workspace(const fw_attn_q4_args *args, int64_t *bytes);
fw_status fw_attn_q4(const fw_attn_q4_args *args, void *workspace, int64_t bytes, void *stream);

/* ------------------------------------------------------------------------
 * What a layer needs between its attention and its experts: linear layers in 8
 * bits and the norms at the residual stream. (The Flyweight README, §Quantization,
 * names kernels with quantised activations for dense projections and the LM head;
 * the pages name neither this format nor a formula, and the readings below are this
 * library's own.) Like the attention side these calls need no handle, never
 * synchronise and allocate nothing.
 *
 * 8-bit blocks. A block of values x has m = max(its largest magnitude, 2^-96),
 * scale = m / 448 and codes e4m3(x * (448 / m)); quotients and product are
 * fp32, rounded to nearest, the codes to nearest even. A block with an
 * infinity or NaN stands for non-finite values. Activations: a block is 128
 * neighbours of one token (the last one of a token may be shorter); codes
 * [T][K], scales fp32 [ceil(K / 128)] rows of T, scale_stride elements apart (a
 * multiple of 4, 16-byte aligned: rows are copied in bulk). Weights: a block is 128 x 128 of
 * [N][K] (smaller at the edges); codes [N][K], scales fp32
 * [ceil(N / 128)][ceil(K / 128)], as checkpoints of 8-bit block-scaled models
 * hold them. */

/* x DEVICE bf16 [T][K], x_stride elements between tokens (a multiple of 8), K a
 * multiple of 16; codes DEVICE e4m3 [T][K] and scales DEVICE fp32, 16-byte aligned. */
fw_status fw_fp8_quantize(const void *x, int64_t x_stride, int32_t T, int32_t K, void *codes, float *scales, int64_t scale_stride,
                          void *stream);

/* w DEVICE [N][K] bf16 (w_fp32 == 0) or fp32 (1), K a multiple of 16. */
fw_status fw_fp8_quantize_weight(const void *w, int32_t w_fp32, int32_t N, int32_t K, void *codes, float *scales, void *stream);

/* A linear layer: out[t][n] = sum over k of x[t][k] w[n][k], both as their codes and
 * scales stand for. Products of codes are exact, the sum over the at most 128 of a
 * block is the tensor core's (fp32), and blocks are scaled and added in fp32, also where the
 * product of the two scales would leave fp32's range (of scales that the rule gives, from
 * 2^-105 to 2^120, and of weights to 2^103; smaller ones may cost precision, larger ones of
 * weights may overflow before a token's small scale is applied); out is rounded once. x may be bf16: it is then quantised by the rule above, with the same
 * result as fw_fp8_quantize before the call. out may not overlap x or w.
 * workspace: DEVICE, 16-byte aligned, at least fw_linear_fp8_workspace bytes (0 with
 * codes, and with bf16 up to 16 tokens; it may then be NULL); its contents mean nothing
 * between calls, and calls that may overlap need one each. */
typedef struct {
  int32_t T, K, N;           /* 0 <= T <= 2^22; K a multiple of 16; 1 <= N <= 2^26 */
  int32_t out_fp32;          /* 0: out is bf16, 1: fp32 */
  const void *x;             /* DEVICE, 16-byte aligned: bf16 [T][K], or with x_scale e4m3 codes */
  const float *x_scale;      /* DEVICE fp32 [ceil(K / 128)] rows of T, 16-byte aligned, or NULL */
  int64_t x_stride;          /* elements between tokens: a multiple of 8 (bf16) or 16 (codes) */
  int64_t x_scale_stride;    /* elements between rows of x_scale: at least T, a multiple of 4 */
  const void *w;             /* DEVICE e4m3 [N][K], 16-byte aligned */
  const float *w_scale;      /* DEVICE fp32 [ceil(N / 128)][ceil(K / 128)] */
  void *out;                 /* DEVICE [T][N] */
  int64_t out_stride;        /* elements between tokens, at least N */
  int32_t *status;           /* DEVICE, FW_KV_TIMEOUT is OR-ed in; or NULL */
} fw_linear_fp8_args;
fw_status fw_linear_fp8_workspace(const fw_linear_fp8_args *args, int64_t *bytes);
fw_status fw_linear_fp8(const fw_linear_fp8_args *args, void *workspace, int64_t bytes, void *stream);

/* The norms after a block and before the next one, with the block's gate, the
 * residual scale and the sum between them:
 *   r = residual + scale * gate * y / sqrt(mean(y^2) + eps) * post_norm
 *       (post_norm NULL: y as it is; gate NULL: 1; residual NULL: 0)
 *   h = r / sqrt(mean(r^2) + eps) * norm           (norm NULL: h = r)
 * in fp32, r and h each rounded once (h is made of r before it is rounded). h is
 * written as bf16, as 8-bit codes (of the bf16 values, by the rule above) or both.
 * residual_out may be residual, and h may be y, with the same strides. */
typedef struct {
  int32_t T, H;              /* H a multiple of 8 (of 16 with h_codes), at most 32768 */
  int32_t residual_fp32;     /* residual and residual_out: 0 bf16, 1 fp32 */
  int32_t gate_fp32;         /* gate: 0 bf16, 1 fp32 */
  int32_t gate_per_token;    /* 1: gate is one value a token, gate_stride elements apart; 0: H values,
                              * gate_stride elements between tokens (0: the same for every token) */
  float eps, scale;
  const void *y;             /* DEVICE bf16 [T][H] */
  const void *residual;      /* DEVICE [T][H], or NULL */
  const void *gate;          /* DEVICE, or NULL */
  int64_t y_stride, residual_stride, gate_stride; /* elements between tokens; multiples of 8 (gate_stride: unless per token) */
  const float *post_norm, *norm; /* DEVICE fp32 [H] or NULL */
  void *residual_out;        /* DEVICE [T][H], or NULL */
  void *h;                   /* DEVICE bf16 [T][H], or NULL */
  int64_t residual_out_stride, h_stride;
  void *h_codes;             /* DEVICE e4m3 [T][H], or NULL */
  float *h_scale;            /* DEVICE fp32 [ceil(H / 128)] rows of T, 16-byte aligned, with h_codes */
  int64_t h_scale_stride;    /* elements between its rows: at least T, a multiple of 4 */
} fw_norm_residual_args;
fw_status fw_norm_residual(const fw_norm_residual_args *args, void *stream);

#ifdef __cplusplus
}
#endif
#endif
