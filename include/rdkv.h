/*
 * rdkv.h — C ABI of the RDKV hot path on one GPU (sm_103a).
 *
 * RDKV ("RDKV - KV 캐시 공동 추방 및 양자화를 위한 왜곡-비트 할당",
 * gist.science/ko/paper/2605.08317) compresses a KV cache after prefill by
 *   section 2.1  distortion weights: w_t (attention mass a token receives) for
 *                V tokens, w_c = |Q_:,c| |K_:,c| / sqrt(d) for K channels;
 *   section 2.2  discrete reverse water-filling (Lagrangian relaxation of a
 *                multiple-choice knapsack) over widths {0,2,4,8,16}: V tokens
 *                first, then K channels of the kept tokens;
 *   section 2.3  the TriZone layout: zone A packed 2/4/8-bit rows grouped by
 *                width, zone B fp16 V rows of 16-bit tokens, zone C fp16 rows
 *                of new tokens; decode attention dequantises inside the
 *                products and reads the three zones in one pass.
 * The quantiser is the asymmetric min-max formula of "Matematika KV Cache
 * Compression" (aistudio.id), section "Solusi 3".
 *
 * Conventions for every call:
 *   - All tensor pointers are DEVICE pointers owned by the caller; the library
 *     allocates no device memory.  Scratch memory is passed in as `ws` with
 *     the size the matching *_workspace_bytes() call returns.
 *   - `stream` is a cudaStream_t (NULL = legacy default stream).  Calls are
 *     asynchronous on that stream unless stated otherwise.
 *   - Tensors are dense, row-major, little-endian.  fp16 = IEEE binary16.
 *   - Shapes: B = batch, N = prompt tokens, H_q, H_kv query/KV heads
 *     (G = H_q / H_kv), D = head_dim (64 or 128), W = window,
 *     N_p = N - W allocatable prefix tokens.
 *   - Errors: a call that returns anything but RDKV_OK launched nothing
 *     (argument errors) or hit a CUDA error (RDKV_ERR_CUDA); the message is
 *     in rdkv_last_error_string() (thread-local).
 */
#ifndef RDKV_H
#define RDKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum rdkv_status {
  RDKV_OK = 0,
  RDKV_ERR_INVALID_ARG = 1,   /* bad pointer, size, budget or (device-side) gain */
  RDKV_ERR_UNSUPPORTED = 2,   /* dtype / head_dim / group size outside the supported set */
  RDKV_ERR_CAPACITY = 3,      /* zone C is full (rdkv_append) */
  RDKV_ERR_CUDA = 4,          /* a CUDA runtime error */
  RDKV_ERR_TIMEOUT = 5,       /* a bounded device-side wait ran out */
  RDKV_ERR_WORKSPACE = 6      /* ws too small */
} rdkv_status;

enum { RDKV_F16 = 0, RDKV_F32 = 1 };

/* Problem shape.  Q, K, V of the prefill are [B][N][H][D] in `dtype`. */
typedef struct rdkv_shape {
  int32_t batch, n_tokens, h_q, h_kv, head_dim, window, dtype;
} rdkv_shape;

/* One (sequence, KV head) of the plan, written by rdkv_allocate (device memory).
 * Token classes are V widths 2,4,8,16; K segments are widths 16,8,4,2. */
typedef struct rdkv_head_plan {
  int32_t n_v[4];        /* kept prefix tokens of each V width */
  int32_t tiles[4];      /* 32-token tiles of each V width: ceil(n_v / 32) */
  int32_t n_k[5];        /* channels of K width 16, 8, 4, 2, 0 */
  int32_t k_words[4];    /* 32-bit words per K row in the 16/8/4/2-bit segments */
  int32_t row_words;     /* sum of k_words */
  int32_t k_slots;       /* channel slots of a K row (kept channels + pads) */
  int32_t meta_slots;    /* slots of the 8/4/2-bit segments (those carry scale/zero) */
  int32_t tile_bytes[4]; /* zone-A bytes of one tile of each V width */
  int64_t a_off;         /* byte offset of this head's first tile in zone A */
  int64_t a_bytes;       /* zone-A bytes of this head */
  int64_t b_row;         /* first zone-B row of this head */
  int64_t slot_off;      /* first index-map slot of this head */
} rdkv_head_plan;        /* 128 bytes */

/* Head of the device plan buffer.  The buffer continues with
 *   rdkv_head_plan heads[n_heads]                 (heads in (b, j) order)
 *   int16_t slot_channel[n_heads][slot_stride]    (channel of each K slot, -1 = pad)
 *   float levels[2][batch * h_kv]                 (water levels found; see rdkv_allocate_mode)
 * at the offsets given by the fields below. */
typedef struct rdkv_plan_header {
  int32_t status;          /* RDKV_OK, or RDKV_ERR_INVALID_ARG if a gain was NaN/inf/negative */
  int32_t n_heads;         /* batch * h_kv */
  int32_t batch, h_kv, head_dim, slot_stride;
  int64_t heads_off, slots_off, lambda_off;   /* byte offsets inside the plan buffer */
  int64_t zone_a_bytes;    /* zone-A bytes of the whole batch */
  int64_t zone_b_rows;     /* zone-B rows (each D fp16) */
  int64_t index_slots;     /* index-map entries */
  int64_t kept_tokens;     /* kept prefix tokens over all heads */
  int64_t max_tile_bytes;  /* largest zone-A tile present */
  int64_t max_stage_bytes; /* largest tile plus the zone-B rows it carries (decode staging) */
} rdkv_plan_header;

/* Heads whose decode work rdkv_plan_sizes estimates for the host (see rdkv_sizes). */
#define RDKV_COST_HEADS 64

/* Host copy of the totals, from rdkv_plan_sizes.  head_cost[h], for the first
 * min(n_heads, RDKV_COST_HEADS) (sequence, KV head) pairs in plan order, is an
 * estimate (> 0, arbitrary units) of the zone-A decode work of that head; the
 * decode calls deal their blocks to the heads in proportion to it on the host.
 * When it is not filled (zeros: more than RDKV_COST_HEADS heads, or a record
 * built by hand) the decode kernel deals the blocks itself from the plan.  Only
 * the speed of the decode depends on these numbers, never its result. */
typedef struct rdkv_sizes {
  int64_t zone_a_bytes, zone_b_rows, index_slots, kept_tokens, max_tile_bytes, max_stage_bytes;
  int32_t status, n_heads;
  int32_t head_cost[RDKV_COST_HEADS];
} rdkv_sizes;

/* Rows of one zone-C page when zone C is paged (see rdkv_cache). */
#define RDKV_ZONE_C_PAGE_ROWS 16
/* Bytes of one zone-A page and rows of one zone-B page when zones A and B are
 * paged (see rdkv_cache). */
#define RDKV_ZONE_A_PAGE_BYTES 65536
#define RDKV_ZONE_B_PAGE_ROWS 16

/* A packed TriZone cache.  All pointers are caller-owned device memory.
 * zone_c_k / zone_c_v are fp16 [batch][h_kv][cap_c][D], or, when
 * zone_c_pages is not NULL, pools of pages [n_pages][RDKV_ZONE_C_PAGE_ROWS][D]
 * (the PagedAttention block table of "Matematika KV Cache Compression",
 * "Solusi 1"): row r of head h = b * h_kv + j is row
 * r % 16 of page zone_c_pages[h * zone_c_page_stride + r / 16].  The table
 * (int32, device) must name a distinct page for every 16-row block a head may
 * use (up to cap_c rows, so zone_c_page_stride >= ceil(cap_c / 16)); the
 * kernels read it when they touch zone C.  The number of zone-C
 * rows in use (same for every sequence) is kept twice: len_dev (one device
 * int32) is what the kernels read and advance, so a captured CUDA graph of
 * append + decode calls stays correct when replayed; len_c is the host mirror
 * the host-side capacity check uses.  rdkv_pack sets both to the window W;
 * rdkv_append advances both.  Replaying captured appends advances only
 * len_dev; a device-side append past cap_c writes nothing.
 *
 * Zones A and B may live in pages of pools shared by several caches (the same
 * block table idea, applied to the zones the pack writes): when zone_a_pages is
 * not NULL, byte o of the cache's zone A (the plan's offsets, a_off and up) is
 * byte o % RDKV_ZONE_A_PAGE_BYTES of page zone_a_pages[o / RDKV_ZONE_A_PAGE_BYTES]
 * of the pool at zone_a (pages of RDKV_ZONE_A_PAGE_BYTES bytes); when
 * zone_b_pages is not NULL, zone-B row r is row r % 16 of page
 * zone_b_pages[r / 16] of the pool at zone_b ([n_pages][16][D] fp16).  The
 * tables (int32, device) name a distinct page for every page the cache's sizes
 * need (ceil(zone_a_bytes / RDKV_ZONE_A_PAGE_BYTES), ceil(zone_b_rows / 16));
 * rdkv_pack writes through them and the decode calls read through them.
 * Caches of sequences with different prompt lengths can so share one pool and
 * be attended in one launch (rdkv_decode_ragged). */
typedef struct rdkv_cache {
  rdkv_shape shape;
  const void* plan;
  uint8_t* zone_a;
  uint16_t* zone_b;
  uint16_t* zone_c_k;
  uint16_t* zone_c_v;
  int32_t* index_map;
  int32_t* len_dev;
  int32_t cap_c;
  int32_t len_c;
  rdkv_sizes sizes;
  const int32_t* zone_c_pages;  /* NULL: contiguous zone C; else its page table */
  int32_t zone_c_page_stride;   /* table entries per head */
  const int32_t* zone_a_pages;  /* NULL: contiguous zone A; else its page table */
  const int32_t* zone_b_pages;  /* NULL: contiguous zone B; else its page table */
} rdkv_cache;

/* ---------------------------------------------------------------- misc */
const char* rdkv_last_error_string(void);
int32_t rdkv_version(void);
/* Number of CUDA kernels this library has launched (or recorded into a graph
 * being captured) in this process, over all threads. */
uint64_t rdkv_launch_count(void);

/* ---------------------------------------------------------------- workspace sizes
 * One workspace query for the calls that take a shape (no counterpart in the
 * paper).  which_call:
 *   RDKV_CALL_SCORE     the same value as rdkv_score_workspace_bytes(shape);
 *   RDKV_CALL_ALLOCATE  the same value as rdkv_allocate_workspace_bytes(shape)
 *                       (also enough for rdkv_allocate_mode and
 *                       rdkv_allocate_at_levels on that shape);
 *   RDKV_CALL_DECODE    an upper bound of rdkv_decode_workspace_bytes(cache)
 *                       for every single cache of this shape on the current
 *                       device (the exact value depends on the cache's plan:
 *                       query it once the plan's sizes are known).
 * Returns 0 for an invalid shape or an unknown call.  Host only. */
enum { RDKV_CALL_SCORE = 0, RDKV_CALL_ALLOCATE = 1, RDKV_CALL_DECODE = 2 };
size_t rdkv_workspace_bytes(const rdkv_shape* shape, int32_t which_call);

/* ---------------------------------------------------------------- step 1: weights
 * RDKV section 2.1 (and section 2.2 step 1: computed once after prefill on the
 * full cache).  For each sequence b and KV head j (query heads h of group j):
 *   w_tok[b][j][t]  = sum_{h in j} sum_{tau >= t} softmax_t(q_tau,h . k_t / sqrt(D))   (causal)
 *   w_chan[b][j][c] = sqrt(sum_{tau, h in j} q_tau,h,c^2) * sqrt(sum_t k_t,j,c^2) / sqrt(D)
 *   sigma_tok[b][j][t] = population std of v_t,j over its D elements
 *   g_tok[b][j][t]  = fl32(w_tok * sigma_tok) for t < N_p
 * q [B][N][H_q][D], k, v [B][N][H_kv][D] in shape->dtype.  Outputs fp32:
 * w_tok, sigma_tok [B][H_kv][N], w_chan [B][H_kv][D], g_tok [B][H_kv][N_p].
 * Supported: D in {64, 128}, 1 <= G <= 8.  fp16 inputs use tensor cores with
 * fp32 accumulation; fp32 inputs use fp32 CUDA-core arithmetic.  q, k, v must
 * be 16-byte aligned (RDKV_ERR_INVALID_ARG otherwise). */
size_t rdkv_score_workspace_bytes(const rdkv_shape* shape);
rdkv_status rdkv_score(const rdkv_shape* shape, const void* q, const void* k, const void* v,
                       float* w_tok, float* w_chan, float* sigma_tok, float* g_tok,
                       void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------- step 2/3: allocation
 * Discrete reverse water-filling (RDKV section 2.2) on n_inst independent
 * instances of n_units gains each: g [n_inst][n_units] fp32 (finite, >= 0).
 * Per instance, with B = floor((double)avg_bits * n_units):
 *   beta_{u,k} = fl32(g_u * s_k), s = (0.375, 0.09375, 0.0146484375, 255/524288)
 *   lambda*    = smallest float32 >= 0 with sum_u b_u(lambda*) <= B
 *   b_u        = width after every upgrade k with beta_{u,k} > lambda*
 * bits [n_inst][n_units] uint8 in {0,2,4,8,16}; lambda_out [n_inst] fp32 (may be NULL).
 * lambda* is found by an 8-bit-per-level bisection of the float32 bit pattern.
 * status_out (device int32, may be NULL) is set to RDKV_ERR_INVALID_ARG if a
 * gain is NaN, infinite or negative (that unit gets 0 bits). */
size_t rdkv_waterfill_workspace_bytes(int32_t n_inst, int64_t n_units);
rdkv_status rdkv_waterfill(int32_t n_inst, int64_t n_units, const float* g, float avg_bits,
                           uint8_t* bits, float* lambda_out, int32_t* status_out,
                           void* ws, size_t ws_bytes, void* stream);

/* Full allocation of a batch (RDKV section 2.2 steps 2 and 3) and the TriZone plan:
 *   V: water-filling of g_tok [B][H_kv][N_p] per sequence (pooled over heads)
 *      with avg_bits_v -> bits_tok [B][H_kv][N_p];
 *   K: sigma_chan [B][H_kv][D] = population std of K over the kept prefix
 *      tokens of the head (0 if none); g_chan = fl32(w_chan * sigma_chan);
 *      water-filling per sequence with avg_bits_k -> bits_chan [B][H_kv][D];
 *   plan: counts, orders and zone offsets (layout above) in `plan`
 *      (rdkv_plan_bytes(shape) bytes of device memory).
 * k is the prefill K [B][N][H_kv][D], 16-byte aligned (RDKV_ERR_INVALID_ARG
 * otherwise; the same holds for rdkv_allocate_mode and rdkv_allocate_at_levels). */
size_t rdkv_plan_bytes(const rdkv_shape* shape);
size_t rdkv_allocate_workspace_bytes(const rdkv_shape* shape);
rdkv_status rdkv_allocate(const rdkv_shape* shape, const float* g_tok, const float* w_chan,
                          const void* k, float avg_bits_v, float avg_bits_k,
                          uint8_t* bits_tok, float* sigma_chan, float* g_chan, uint8_t* bits_chan,
                          void* plan, void* ws, size_t ws_bytes, void* stream);

/* Allocation variants on the same plan, pack and decode (the RDKV page's
 * section 2.2 is the method; the others are a different reading of its scope
 * and two eviction-only baselines the pages compare against).
 *   RDKV_ALLOC_POOLED    the method, as rdkv_allocate (one water level per
 *                        sequence for V and one for K);
 *   RDKV_ALLOC_PER_HEAD  one water level per (sequence, KV head) for V (budget
 *                        floor(avg_bits_v * N_p) per head) and for K (budget
 *                        floor(avg_bits_k * D) per head);
 *   RDKV_ALLOC_TOPK      heavy-hitter eviction (H2O-style): per (sequence, KV
 *                        head), k = floor(floor(avg_bits_v * N_p) / 16) tokens
 *                        are affordable at 16 bits; every prefix token whose
 *                        w_t exceeds lambda, the smallest non-negative level
 *                        at most k weights exceed, is kept at 16 bits (equal
 *                        weights at lambda are all dropped); every K channel
 *                        16 bits;
 *   RDKV_ALLOC_THRESHOLD eviction by a threshold on the weight (KVzap-style):
 *                        prefix tokens with w_t > param kept at 16 bits; every
 *                        K channel 16 bits.
 * w_tok [B][H_kv][N] (rdkv_score's output; used by TOPK and THRESHOLD),
 * g_tok [B][H_kv][N_p] (used by POOLED and PER_HEAD); the other arguments as
 * rdkv_allocate (sigma_chan, g_chan are computed over the kept tokens in every
 * mode).  Levels in the plan: POOLED: V [B] then K [B]; the other modes:
 * V [B*H_kv] then K [B*H_kv] (0 for the K stage of TOPK and THRESHOLD, param
 * for the V stage of THRESHOLD). */
typedef enum rdkv_alloc_mode {
  RDKV_ALLOC_POOLED = 0,
  RDKV_ALLOC_PER_HEAD = 1,
  RDKV_ALLOC_TOPK = 2,
  RDKV_ALLOC_THRESHOLD = 3
} rdkv_alloc_mode;
rdkv_status rdkv_allocate_mode(const rdkv_shape* shape, int mode, float param, const float* w_tok,
                               const float* g_tok, const float* w_chan, const void* k,
                               float avg_bits_v, float avg_bits_k, uint8_t* bits_tok,
                               float* sigma_chan, float* g_chan, uint8_t* bits_chan,
                               void* plan, void* ws, size_t ws_bytes, void* stream);

/* Copies the plan totals to the host.  SYNCHRONISES `stream`.  Returns the
 * plan's device status (RDKV_ERR_INVALID_ARG if a gain was invalid). */
rdkv_status rdkv_plan_sizes(const void* plan, rdkv_sizes* out, void* stream);

/* Upper bounds of the plan totals rdkv_allocate (pooled or per-head levels)
 * can produce for this shape and these budgets, from the budgets alone: no
 * device access, no synchronisation.  Zones sized from them let the whole
 * compression (rdkv_score, rdkv_allocate, rdkv_pack with cache->sizes = the
 * bounds) run as one stream-ordered sequence, capturable in a CUDA graph;
 * rdkv_plan_sizes afterwards gives the exact totals (and the head costs) for
 * the decode.  Not a bound for the eviction baselines of rdkv_allocate_mode
 * (top-k, threshold), nor for the levels of rdkv_allocate_at_levels. */
rdkv_status rdkv_zone_bounds(const rdkv_shape* shape, float avg_bits_v, float avg_bits_k, rdkv_sizes* out);

/* ---------------------------------------------------------------- TriZone pack
 * RDKV section 2.3.  Writes zone A (sizes.zone_a_bytes), zone B
 * (sizes.zone_b_rows x D fp16), the index map (sizes.index_slots int32) and
 * the window rows [0, W) of zone C from the prefill k, v [B][N][H_kv][D];
 * sets cache->len_c = W.  cache->plan must be the plan bits_tok/bits_chan came
 * with; cap_c >= W; cache->sizes the plan's totals or upper bounds of them
 * (rdkv_zone_bounds); k and v 16-byte aligned (else RDKV_ERR_INVALID_ARG).  Bytes are bit-exact with the layout rules:
 * asymmetric min-max codes (aistudio.id "Solusi 3") with fp16 scale/zero. */
rdkv_status rdkv_pack(rdkv_cache* cache, const void* k, const void* v,
                      const uint8_t* bits_tok, const uint8_t* bits_chan, void* stream);

/* ---------------------------------------------------------------- allocation and pack in one launch
 * RDKV section 2.2 steps 2 and 3, then section 2.3, as ONE persistent
 * (cooperative) kernel whose phases are separated by grid-wide barriers: the
 * V water level and widths, the K channel spreads over the kept tokens, the K
 * water level and widths, the plan, the index map, the head K metadata, the
 * zone-A tiles and zone-B rows, the zone-C window and *len_dev = W.  Every
 * output (bits_tok, sigma_chan, g_chan, bits_chan, the plan with its levels
 * and channel statistics, zones A and B, the index map, zone C rows [0, W))
 * is byte-identical to rdkv_allocate (per_head = 0; rdkv_allocate_mode with
 * RDKV_ALLOC_PER_HEAD for per_head = 1) followed by rdkv_pack.
 *
 * cache: as for rdkv_pack, except that cache->plan is the plan buffer this
 *   call WRITES (rdkv_plan_bytes(shape) bytes) and cache->sizes holds the
 *   zones' capacities (zone_a_bytes, zone_b_rows, index_slots; normally
 *   rdkv_zone_bounds for these budgets).  The exact totals (and the head
 *   costs the decode deals its blocks by) come afterwards from
 *   rdkv_plan_sizes; the call itself does not synchronise, so it can be
 *   captured in a CUDA graph.  Sets cache->len_c = W.
 * g_tok, w_chan: rdkv_score's outputs; k, v: the prefill [B][N][H_kv][D],
 *   16-byte aligned.  Outputs as for rdkv_allocate.
 * ws: rdkv_allocate_pack_workspace_bytes(shape, per_head) bytes of device
 *   memory (the call clears the part it needs cleared, asynchronously on
 *   `stream`).
 * Errors: the host checks of rdkv_allocate and rdkv_pack (nothing launched);
 *   RDKV_ERR_UNSUPPORTED when fewer blocks stay resident than there are
 *   water-filling instances.  Device-side outcomes land in the plan status
 *   (read by rdkv_plan_sizes): RDKV_ERR_INVALID_ARG for an invalid gain (the
 *   pack still runs, as rdkv_pack would), RDKV_ERR_CAPACITY when the plan
 *   needs more than a capacity (then nothing is packed), RDKV_ERR_TIMEOUT when
 *   a grid barrier waited past its bound (about two seconds; the outputs are
 *   then not valid). */
size_t rdkv_allocate_pack_workspace_bytes(const rdkv_shape* shape, int32_t per_head);
rdkv_status rdkv_allocate_pack(rdkv_cache* cache, int32_t per_head, const float* g_tok,
                               const float* w_chan, const void* k, const void* v,
                               float avg_bits_v, float avg_bits_k, uint8_t* bits_tok,
                               float* sigma_chan, float* g_chan, uint8_t* bits_chan,
                               void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------- append
 * RDKV section 2.3 zone C: writes the new token's k_new, v_new [B][H_kv][D]
 * (shape->dtype) as fp16 rows at row *len_dev of zone C and advances *len_dev
 * and len_c.  Returns RDKV_ERR_CAPACITY (nothing launched) when the host
 * mirror len_c == cap_c. */
rdkv_status rdkv_append(rdkv_cache* cache, const void* k_new, const void* v_new, void* stream);

/* ---------------------------------------------------------------- decode attention
 * RDKV section 2.3: for every sequence b and query head h (KV head h / G),
 *   out[b][h] = sum_t softmax_t(q[b][h] . k^_t / sqrt(D)) v^_t
 * over the kept tokens of zones A (dequantised K and V) and B (fp16 V) and the
 * *len_dev rows of zone C.  q [B][H_q][D] in shape->dtype, out [B][H_q][D]
 * fp32.  Split-K over tiles with an fp32 online softmax; the partial results
 * and per-head tickets live in ws, which must be ZERO-FILLED before its first
 * use: every call leaves the tickets at zero again, so the same ws serves any
 * number of calls (and CUDA-graph replays) without a reset. */
size_t rdkv_decode_workspace_bytes(const rdkv_cache* cache);
rdkv_status rdkv_decode_attn(const rdkv_cache* cache, const void* q, float* out,
                             void* ws, size_t ws_bytes, void* stream);

/* Launch order (rdkv_decode_attn and rdkv_decode_step): the kernel is launched
 * as a programmatic dependent of the kernel before it on `stream`.  Before it
 * waits for that kernel it reads only the plan and zone A (dealing the work,
 * staging tile copies); the query, the new token, zone C and *len_dev are read
 * after the wait.  So the plan and zone A must not be written by the kernel
 * launched immediately before a decode call on the same stream (rdkv_pack ends
 * with a kernel that writes neither); anything else may be. */

/* ---------------------------------------------------------------- decode step
 * RDKV section 2.3, one decode step in one launch: rdkv_append(k_new, v_new)
 * followed by rdkv_decode_attn(q), computed together.  The new token's row
 * enters the attention straight from k_new/v_new; once every block of a head
 * has read zone C, that head's row is stored at row *len_dev, and the last
 * head to finish advances *len_dev (and the call advances the host mirror
 * len_c).  Same q/out layout and workspace (same size, same zero-filled
 * contract) as rdkv_decode_attn.  Returns RDKV_ERR_CAPACITY (nothing
 * launched) when the host mirror len_c == cap_c; a replayed step that finds
 * *len_dev == cap_c attends with the new token but stores nothing and leaves
 * RDKV_ERR_CAPACITY in the status word. */
rdkv_status rdkv_decode_step(rdkv_cache* cache, const void* q, const void* k_new, const void* v_new,
                             float* out, void* ws, size_t ws_bytes, void* stream);

/* Reads the status word the rdkv_decode_attn / rdkv_decode_step calls on this
 * cache and ws left behind since the last read, and clears it.  SYNCHRONISES
 * `stream`.  RDKV_ERR_TIMEOUT means a bounded wait for a tile copy ran out in
 * one of those calls (its output is not valid); RDKV_ERR_CAPACITY means a
 * step found zone C full and did not store its token. */
rdkv_status rdkv_decode_status(const rdkv_cache* cache, const void* ws, void* stream);

/* Failure-detection self-test of the decode (no counterpart in the paper).
 * Runs the rdkv_decode_attn kernel on `cache`, `q`, `out` and `ws` (same
 * layouts and workspace contract) with every stage's barrier armed for 16
 * bytes that no copy delivers, and no copy issued: each warp's bounded wait
 * runs out after `wait_cycles` SM clock cycles (clamped to [1e5, 4e9]; 2e6
 * is about 1 ms), the kernel records RDKV_ERR_TIMEOUT in the status word and
 * returns, as it would if a tile copy never completed.  Nothing faults or
 * hangs and the context stays usable; `out` holds no attention result.
 * rdkv_decode_status then returns RDKV_ERR_TIMEOUT and clears the word.
 * Returns RDKV_ERR_INVALID_ARG for wait_cycles <= 0, else as rdkv_decode_attn
 * for the launch itself.  Asynchronous on `stream`. */
rdkv_status rdkv_decode_timeout_selftest(const rdkv_cache* cache, const void* q, float* out, void* ws,
                                         size_t ws_bytes, int64_t wait_cycles, void* stream);

/* ---------------------------------------------------------------- decode without a workspace
 * No counterpart in the paper: a deployment variant of rdkv_decode_attn.
 * Some callers cannot allocate device memory themselves: a plugin hosted by
 * an engine that owns every device allocation, or code that must not call the
 * allocator on its serving path.  This entry point computes the same output as
 * rdkv_decode_attn, but keeps its scratch (split partials, per-head tickets and
 * the status word) in a fixed 4 MiB array built into the library, which every
 * GPU that loads the library holds until the process exits; it allocates
 * nothing.
 *   - Returns RDKV_ERR_WORKSPACE (nothing launched) when the cache needs more
 *     than 4 MiB of scratch (rdkv_decode_workspace_bytes tells how much).
 *   - The first call on a device looks up the array's device address (and
 *     raises the kernel's shared-memory limit); make that first call before
 *     any stream capture.  The lookup is cached per device for the CUDA
 *     runtime's primary context of that device (the context every call of
 *     this library runs in); host threads may make their first calls at the
 *     same time.
 *   - All calls share the one array and each clears the counters it needs, so
 *     calls that overlap on the GPU (other streams, other threads) race and
 *     must be serialised by the caller.
 *   - The status word of a call lives in that shared array and is not exposed:
 *     if a bounded wait for a tile copy runs out inside this call, nothing
 *     reports it, the call still returns RDKV_OK and its output is undefined.
 *     Callers that need the timeout report use rdkv_decode_attn. */
rdkv_status rdkv_decode_attn_noalloc(const rdkv_cache* cache, const void* q, float* out, void* stream);

/* ---------------------------------------------------------------- zone-C re-compression
 * New tokens start in zone C (RDKV section 2.3); the pages do not say how
 * they later join zones A and B.  These calls move the oldest zone-C rows into
 * a new SEGMENT: a TriZone cache of their own (window 0) packed by rdkv_pack,
 * with token weights from the attention the recent decode queries gave them
 * and widths at the prefill's water levels (section 2.2, the levels kept
 * instead of found again).  The attention over the segments and the live
 * cache is merged from each part's output and log-sum-exp. */

/* rdkv_decode_attn / rdkv_decode_step that also write lse [B][H_q] fp32: the
 * natural log of the softmax denominator, ln sum_t exp(q . k^_t / sqrt(D)),
 * over the same keys (-inf when there are none; out is then 0).  lse is
 * caller-owned device memory; everything else as in the calls without it. */
rdkv_status rdkv_decode_attn_lse(const rdkv_cache* cache, const void* q, float* out, float* lse,
                                 void* ws, size_t ws_bytes, void* stream);
rdkv_status rdkv_decode_step_lse(rdkv_cache* cache, const void* q, const void* k_new, const void* v_new,
                                 float* out, float* lse, void* ws, size_t ws_bytes, void* stream);

/* Attention over the union of disjoint key sets from its parts:
 *   out = sum_i e^(lse_i) out_i / sum_i e^(lse_i),  lse = ln sum_i e^(lse_i)
 * per row.  outs [n_parts][rows][head_dim], lses [n_parts][rows] fp32 device
 * (rows = B * H_q for decode outputs); out [rows][head_dim] and lse_out
 * [rows] (may be NULL) fp32 device.  Parts with lse = -inf weigh 0; a row with
 * no keys in any part gets out 0, lse -inf; one with a NaN lse gets NaN.  out may alias outs[0]; lse_out
 * must not alias lses. */
rdkv_status rdkv_merge_attn(int32_t n_parts, const float* outs, const float* lses, int64_t rows,
                            int32_t head_dim, float* out, float* lse_out, void* stream);

/* One launch over several caches sharing the query: the softmax over the union
 * of their keys (zones A and B of each, and each one's zone-C rows), the same
 * output rdkv_merge_attn gives from one call per cache, without the extra
 * launches.  parts[0 .. n_parts) (1 <= n_parts <= 8) must share batch, h_q,
 * h_kv, head_dim and dtype; typically the segments moved out of zone C and
 * then the live cache.  q, out, lse (may be NULL) and the workspace contract
 * as rdkv_decode_attn_lse, the workspace sized by
 * rdkv_decode_multi_workspace_bytes for the same list (0 if the list is
 * invalid).  With more than one cache, every cache's sizes must carry its
 * plan costs (rdkv_plan_sizes) and the batch at most RDKV_COST_HEADS heads,
 * else RDKV_ERR_UNSUPPORTED.  rdkv_decode_multi_status reads and clears the
 * status word as rdkv_decode_status does. */
size_t rdkv_decode_multi_workspace_bytes(const rdkv_cache* const* parts, int32_t n_parts);
rdkv_status rdkv_decode_attn_multi(const rdkv_cache* const* parts, int32_t n_parts, const void* q, float* out,
                                   float* lse, void* ws, size_t ws_bytes, void* stream);
rdkv_status rdkv_decode_multi_status(const rdkv_cache* const* parts, int32_t n_parts, const void* ws, void* stream);

/* ---------------------------------------------------------------- ragged batch
 * RDKV section 2.3 for a batch of independent sequences with different prompt
 * lengths (the batching of "Matematika KV Cache Compression", "Solusi 1"): each
 * sequence is its own cache (batch 1, its own n_tokens, plan and zones, often
 * in pages of shared pools), and ONE launch attends all of them:
 *   out[s][h] = sum_t softmax_t(q[s][h] . k^_t / sqrt(D)) v^_t over the keys of
 *   sequence s only (zones A and B and the *len_dev rows of its zone C).
 * seqs[0 .. n_seq) (1 <= n_seq <= 8) must share h_q, h_kv, head_dim and dtype,
 * have batch 1, carry their plan costs (rdkv_plan_sizes), and n_seq * h_kv
 * must be at most RDKV_COST_HEADS, else RDKV_ERR_INVALID_ARG or
 * RDKV_ERR_UNSUPPORTED.  q [n_seq][H_q][D] in the caches' dtype, out
 * [n_seq][H_q][D] fp32, lse [n_seq][H_q] fp32 or NULL; the workspace sized by
 * rdkv_decode_ragged_workspace_bytes for the same list (0 if it is invalid),
 * with the zero-filled contract of rdkv_decode_attn.  rdkv_decode_ragged_status
 * reads and clears the status word as rdkv_decode_status does.  (Append the new
 * tokens with rdkv_append before the call.) */
size_t rdkv_decode_ragged_workspace_bytes(const rdkv_cache* const* seqs, int32_t n_seq);
rdkv_status rdkv_decode_ragged(const rdkv_cache* const* seqs, int32_t n_seq, const void* q, float* out, float* lse,
                               void* ws, size_t ws_bytes, void* stream);
rdkv_status rdkv_decode_ragged_status(const rdkv_cache* const* seqs, int32_t n_seq, const void* ws, void* stream);

/* Takes rows [0, n_move) of every head's zone C out of the cache: copies them
 * to k_out, v_out [B][n_move][H_kv][D] in the cache's dtype (the fp16 values
 * of zone C, widened for fp32 caches; the prefill layout, ready for
 * rdkv_recompress_score, rdkv_allocate_at_levels and rdkv_pack with a shape
 * of n_move tokens, window 0 and the cache's dtype, whose queries are then
 * the model's), moves rows [n_move, len_c) to the front and
 * lowers len_c and *len_dev by n_move.  Requires 0 < n_move <= len_c and
 * len_c - n_move <= n_move (the rows that stay fit in the rows that leave, so
 * the move never overlaps itself), else RDKV_ERR_INVALID_ARG with nothing
 * launched.  Uses the host mirror len_c: do not call it while captured
 * decode steps are pending replay. */
rdkv_status rdkv_zone_c_take(rdkv_cache* cache, int32_t n_move, void* k_out, void* v_out, void* stream);

/* Token weights and gains of moved tokens (reading of section 2.1 for tokens
 * that entered after the prefill): for sequence b, KV head j and moved token t
 *   w_tok[b][j][t] = weight_scale * sum over r < n_recent and the G query heads
 *                    h of group j of
 *                    exp(q_recent[b][r][h] . k[b][t][j] / sqrt(D) - lse_recent[b][r][h])
 * i.e. the attention the recent decode steps gave the token (their lse from
 * rdkv_decode_*_lse), scaled: a prefill weight sums the attention of up to N
 * query rows, so weight_scale = N / n_recent puts the moved tokens on the scale
 * the prefill's water levels were found for.  sigma_tok = population std of
 * the token's V row and g_tok = fl32(w_tok * sigma_tok).  seg: the segment's shape (n_tokens =
 * moved rows, window 0, dtype of k, v); k, v [B][n][H_kv][D]; q_recent
 * [B][n_recent][H_q][D] in q_dtype; lse_recent [B][n_recent][H_q] fp32;
 * outputs [B][H_kv][n] fp32.  All device memory; 1 <= n_recent. */
rdkv_status rdkv_recompress_score(const rdkv_shape* seg, const void* k, const void* v, const void* q_recent,
                                  int32_t q_dtype, const float* lse_recent, int32_t n_recent, float weight_scale,
                                  float* w_tok, float* sigma_tok, float* g_tok, void* stream);

/* Section 2.2 steps 2 and 3 at given water levels: V widths are the
 * Lagrangian choice at lam_v, then sigma_c of each K channel over the kept
 * moved tokens, g_chan = fl32(w_chan * sigma_c) and K widths at lam_k; then
 * the plan, as rdkv_allocate.  levels [2][n_inst] fp32 device: lam_v of every
 * instance, then lam_k; an instance is a sequence (per_head = 0, the pooled
 * levels of rdkv_allocate) or a (sequence, KV head) pair (per_head = 1).  The
 * plan's own levels are set to these.  w_chan is the prefill's [B][H_kv][D];
 * other arguments, outputs and the workspace as rdkv_allocate for the
 * segment's shape. */
rdkv_status rdkv_allocate_at_levels(const rdkv_shape* seg, int32_t per_head, const float* levels,
                                    const float* g_tok, const float* w_chan, const void* k, uint8_t* bits_tok,
                                    float* sigma_chan, float* g_chan, uint8_t* bits_chan, void* plan, void* ws,
                                    size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------- 4-bit cache, quantised as it is written
 * No counterpart in the paper: a cache for the tokens that no prefill
 * statistics exist for (new tokens, or whole prompts when the prefill's
 * attention is not scored).  Every row is quantised on its own when it is
 * written, by the quantiser of the TriZone pack: per KV head and group of 32
 * channels of one token, K and V alike,
 *   zero = fp16(min), scale = fp16(fl32(max - min) / 15),
 *   code = clamp(rint((x - zero) / scale), 0, 15)   (IEEE fp32, ties to even; scale 0: code 0)
 * and stands for x^ = fl32(zero + scale * code).  Values past +-65504
 * (infinities too) are held as +-65504; a NaN takes no part in min and max
 * and gets code 0.
 *
 * Layout.  Pages of RDKV_Q4_PAGE_TOKENS tokens of one sequence, each with all
 * KV heads: pages [n_pages][h_kv][rdkv_q4_page_bytes(head_dim)], position p of
 * sequence b is slot p % 64 of page page_table[b * page_stride + p / 64].  With
 * NG = head_dim / 32 groups, the 80 * head_dim bytes of a (page, head) are
 *   K codes   uint32 [64 tokens][4 q][NG]: word q of a token and group holds its channels 8q .. 8q+7,
 *             element e at bit 16 (e mod 2) + 4 (e / 2);
 *   K scales  fp16 [32 token pairs][NG][2 tokens];
 *   K zeros   fp16 [64 tokens][NG];
 *   V codes   uint32 [32 token pairs][8 g][NG]: channels 4g .. 4g+3 of the group at bits 0, 4, 8, 12 for
 *             the even token and 16 above for the odd one;
 *   V scales, V zeros  fp16 [32 token pairs][NG][2 tokens].
 * `bounds` (may be NULL: no rdkv_q4_select) is fp16 [n_pages][h_kv][2][head_dim]:
 * the smallest and the largest value fp16(x^) of each K channel over the
 * page's tokens (all the tokens written since the page's slot 0 was).
 *
 * `lens` [batch] (int32, device) is the number of tokens each sequence holds,
 * kept by the caller: raise it BEFORE rdkv_q4_write, which writes the last rows
 * of each sequence, and call rdkv_q4_attn with the same values.  A slot without
 * a sequence has length 0.  Nothing in these calls changes it, so captured
 * graphs replay with whatever it then holds.
 *
 * Entries of `page_table` that no held token needs are not read, and may be
 * anything.  Pages may be shared between sequences (a common prefix) as long as
 * no call writes them.
 * `status` is one device int32, zero before the first call: a call that finds
 * RDKV_ERR_INVALID_ARG (a page outside [0, n_pages), row counts or positions
 * that do not fit), RDKV_ERR_CAPACITY (a length past 64 * page_stride) or
 * RDKV_ERR_TIMEOUT (a bounded wait) on the device leaves out what it concerns
 * and raises *status to that code; rdkv_q4_status reads and clears it.
 *
 * Supported: head_dim 64 or 128, 1 <= h_q / h_kv <= 8, rows and queries in
 * RDKV_F16, RDKV_F32 or RDKV_BF16 (beside these calls and the 8-bit cache's, the
 * calls of this library take no RDKV_BF16).  pages and bounds 16-byte aligned. */
enum { RDKV_BF16 = 2 };
#define RDKV_Q4_PAGE_TOKENS 64
/* Most query tokens of a sequence in one rdkv_q4_attn or rdkv_q4_select; batch *
 * n_q * h_kv is at most 65,535 in both (else RDKV_ERR_UNSUPPORTED). */
#define RDKV_Q4_MAX_QUERIES 64
/* Bytes at the start of their workspaces that hold counters. */
#define RDKV_Q4_COUNTER_BYTES 262144
typedef struct rdkv_q4_cache {
  int32_t batch, h_kv, head_dim;
  int32_t n_pages;            /* pages of the pool */
  int32_t page_stride;        /* page-table entries of a sequence */
  uint8_t* pages;
  uint16_t* bounds;           /* or NULL */
  const int32_t* page_table;  /* [batch][page_stride] */
  const int32_t* lens;        /* [batch] */
  int32_t* status;            /* [1] */
} rdkv_q4_cache;

/* Bytes of one (page, KV head): 80 * head_dim; 0 for an unsupported head_dim. */
size_t rdkv_q4_page_bytes(int32_t head_dim);

/* Writes new rows k, v [rows][h_kv][head_dim] in `dtype`, consecutive rows
 * row_stride elements apart (>= h_kv * head_dim).  rows counts them all: a
 * sequence whose rows end past it gets none (RDKV_ERR_INVALID_ARG in *status).  Sequence b's rows are
 * [row_start[b], row_start[b + 1]) (int32 [batch + 1], device), at most
 * max_rows of them, or, with row_start NULL, max_rows rows each, sequence after
 * sequence.  They are its LAST tokens: row i of n goes to position
 * lens[b] - n + i.  A sequence with more rows than lens[b] (or, with row_start,
 * than max_rows) gets none written (RDKV_ERR_INVALID_ARG in *status); but
 * with row_start NULL a sequence of length 0 is an empty slot: its rows are
 * skipped.  Rows past row_start[batch] are not read.  k, v 16-byte aligned, row_stride a
 * multiple of 16 bytes. */
rdkv_status rdkv_q4_write(const rdkv_q4_cache* cache, int32_t dtype, const void* k, const void* v, int64_t rows,
                          int64_t row_stride, const int32_t* row_start, int32_t max_rows, void* stream);

/* Reads rows back, x^ rounded to `dtype` (fp16 saturates at +-65504): k, v as for rdkv_q4_write,
 * row i of sequence b from position first[b] + i (int32 [batch], device; NULL:
 * 0).  Rows at positions past lens[b] are left as they were, and so are rows
 * of k, v that belong to no sequence. */
rdkv_status rdkv_q4_read(const rdkv_q4_cache* cache, int32_t dtype, void* k, void* v, int64_t rows,
                         int64_t row_stride, const int32_t* row_start, const int32_t* first, int32_t max_rows, void* stream);

/* Attention of the n_q (1 .. RDKV_Q4_MAX_QUERIES) newest tokens of every
 * sequence over its cache: query token i of sequence b sees positions
 * [0, lens[b] - n_q + i + 1), and for query head h (KV head h / G)
 *   out = sum_t softmax_t(q . k^_t / sqrt(head_dim)) v^_t,
 *   lse = ln sum_t exp(q . k^_t / sqrt(head_dim))
 * (no position seen: out 0, lse -inf; a query that holds a NaN and sees a
 * position: out and lse NaN, the other queries' as they are).  q
 * [batch][n_q][h_q][head_dim] in
 * `dtype`, consecutive tokens q_stride elements apart (16-byte aligned,
 * q_stride a multiple of 16 bytes); out [batch][n_q][h_q][head_dim] dense in
 * out_dtype, which is dtype or RDKV_F32.  Sums are fp32.  For fp32 outputs every
 * operand is held in 22 bits or more; for 16-bit outputs the weights, weight
 * times scale and the groups' middles are rounded to fp16, which together adds
 * less to an output's error than its own rounding does.  lse [batch][n_q][h_q] fp32 or NULL.
 * fp32 out and lse join other caches' attention through rdkv_merge_attn.
 *
 * sel NULL: every position.  Else sel [batch][n_q][h_kv][n_sel] (int32, device;
 * rdkv_q4_select's output, or the caller's own choice): query token i's heads of
 * KV head j see only the positions that also lie in one of those pages (indices
 * into the sequence's pages, position / 64; entries < 0 or past its last page
 * are left out; an index must not occur twice), n_sel >= 1 (none to be seen:
 * entries of -1).
 *
 * ws: rdkv_q4_attn_workspace_bytes bytes, 16-byte aligned, its first
 * RDKV_Q4_COUNTER_BYTES zero before its first use; every call leaves them zero
 * again, one that reports RDKV_ERR_TIMEOUT too, so calls of any
 * shape that need no more bytes, of rdkv_q4_select too, may follow one another
 * on it.  Calls that may run at the same time (two streams, two captured
 * graphs) need one each.  batch * n_q * h_kv * page_stride (with sel: * n_sel)
 * is at most 2^31 - 1 (else RDKV_ERR_UNSUPPORTED). */
size_t rdkv_q4_attn_workspace_bytes(const rdkv_q4_cache* cache, int32_t h_q, int32_t n_q);
rdkv_status rdkv_q4_attn(const rdkv_q4_cache* cache, int32_t dtype, const void* q, int64_t q_stride, int32_t h_q,
                         int32_t n_q, const int32_t* sel, int32_t n_sel, void* out, int32_t out_dtype, float* lse,
                         void* ws, size_t ws_bytes, void* stream);

/* Failure-detection self-test of rdkv_q4_attn: its kernel on the same arguments,
 * but the pages of a sequence whose index plus KV head is a multiple of
 * `withhold` (>= 1; 1: all) are waited for and never copied.  Each warp that
 * meets one waits for `wait_cycles` SM clock cycles (clamped to [1e5, 4e9]; 2e6
 * is about 1 ms), reports RDKV_ERR_TIMEOUT in *status and leaves out what was
 * left of its pages, as if a copy never completed.  Nothing faults or hangs;
 * out and lse hold no attention result where a page was left out (all rows are
 * written), and ws serves the next call.  RDKV_ERR_INVALID_ARG for withhold or
 * wait_cycles <= 0, else as rdkv_q4_attn. */
rdkv_status rdkv_q4_timeout_selftest(const rdkv_q4_cache* cache, int32_t dtype, const void* q, int64_t q_stride,
                                     int32_t h_q, int32_t n_q, const int32_t* sel, int32_t n_sel, void* out,
                                     int32_t out_dtype, float* lse, void* ws, size_t ws_bytes, int32_t withhold,
                                     int64_t wait_cycles, void* stream);

/* Chooses n_keep pages for every (sequence, query token, KV head): sel
 * [batch][n_q][h_kv][n_keep] int32, ascending, -1 behind the last.  Of the P
 * pages that hold a position the query token sees, all when P <= n_keep; else
 * the first n_first, the last n_last and the best others by
 *   score(page) = max over the G query heads of sum_c max(q_c lo_c, q_c hi_c),
 * lo and hi the page's `bounds`: no logit of the page's keys (up to the bounds'
 * fp16 rounding) is larger than score / sqrt(head_dim).  Equal scores: the lower
 * page first; the order is that of sums carried to twice fp32's precision.  A
 * query head that holds a NaN or an infinity takes no part in the maximum; with
 * no other head, and for pages outside the pool (RDKV_ERR_INVALID_ARG in
 * *status), there is no score: such pages come last, the lower first.
 * q, q_stride, h_q, n_q as for rdkv_q4_attn; 0 <= n_first, 0 <= n_last,
 * n_first + n_last <= n_keep, 1 <= n_keep; cache->bounds not NULL; ws as for
 * rdkv_q4_attn, sized by rdkv_q4_select_workspace_bytes. */
size_t rdkv_q4_select_workspace_bytes(const rdkv_q4_cache* cache, int32_t h_q, int32_t n_q);
rdkv_status rdkv_q4_select(const rdkv_q4_cache* cache, int32_t dtype, const void* q, int64_t q_stride, int32_t h_q,
                           int32_t n_q, int32_t n_keep, int32_t n_first, int32_t n_last, int32_t* sel, void* ws,
                           size_t ws_bytes, void* stream);

/* Reads *status and clears it.  SYNCHRONISES `stream`. */
rdkv_status rdkv_q4_status(const rdkv_q4_cache* cache, void* stream);

/* ---------------------------------------------------------------- 8-bit cache, kept at a budget by attention weight
 * A cache of fp8 codes beside the 4-bit one, with the same pages, page table,
 * lengths, status and rules for them (above); where its calls say nothing else,
 * what the rdkv_q4_* calls say of sharing, streams and errors holds.  The keys of
 * a (page, KV head), 64 tokens by head_dim channels, share one scale, and so do
 * its values.  A scale is a power of two and a code is an e4m3 number:
 *   scale = 2^e, e the smallest of -24 .. 7 with max |x| <= 448 2^e,
 *   code = e4m3(x / scale) (nearest, ties to even),   x^ = scale * code.
 * Values past +-57344 (infinities too) are held as +-57344, a NaN as 0.  A code's
 * precision does not depend on the scale until x falls below 2^-6 scale, so rows
 * that meet in one block, or whose block takes another scale, keep their values
 * down to there: rows written behind others in a page raise its scales where
 * they need more, the earlier codes are taken in the new scale (rounded once
 * more where they are that small), and no write lowers a scale but the one that
 * begins a page (slot 0).
 *
 * Layout.  pages [n_pages][h_kv][rdkv_q8_page_bytes(head_dim)]: 64 D bytes of
 * key codes, then 64 D of value codes (D = head_dim),
 *   keys    uint8 [32 token pairs][D / 64][2 tokens][64 channels];
 *   values  uint8 [8 runs of 8 tokens][D / 64][8 g][4 token pairs][8 c][2 tokens]: channel
 *           64 j + 8 g + c of run [..][j].
 * scales [n_pages][h_kv][2] fp32: the keys' scale, the values'.
 *
 * Supported: head_dim, heads and types as for the 4-bit cache; pages 16-byte
 * aligned, scales 8-byte aligned. */
#define RDKV_Q8_PAGE_TOKENS 64
#define RDKV_Q8_MAX_QUERIES 64
#define RDKV_Q8_COUNTER_BYTES 262144
typedef struct rdkv_q8_cache {
  int32_t batch, h_kv, head_dim;
  int32_t n_pages;            /* pages of the pool */
  int32_t page_stride;        /* page-table entries of a sequence */
  uint8_t* pages;
  float* scales;
  const int32_t* page_table;  /* [batch][page_stride] */
  const int32_t* lens;        /* [batch] */
  int32_t* status;            /* [1] */
} rdkv_q8_cache;

/* Bytes of one (page, KV head): 128 * head_dim; 0 for an unsupported head_dim. */
size_t rdkv_q8_page_bytes(int32_t head_dim);

/* Rows into the cache and back: arguments, positions and errors as
 * rdkv_q4_write and rdkv_q4_read. */
rdkv_status rdkv_q8_write(const rdkv_q8_cache* cache, int32_t dtype, const void* k, const void* v, int64_t rows,
                          int64_t row_stride, const int32_t* row_start, int32_t max_rows, void* stream);
rdkv_status rdkv_q8_read(const rdkv_q8_cache* cache, int32_t dtype, void* k, void* v, int64_t rows,
                         int64_t row_stride, const int32_t* row_start, const int32_t* first, int32_t max_rows, void* stream);

/* Attention of the n_q newest tokens of every sequence over its cache, q, out,
 * lse and ws as for rdkv_q4_attn without a selection (the bytes from
 * rdkv_q8_attn_workspace_bytes, the first RDKV_Q8_COUNTER_BYTES zero before the
 * first use).  Sums are fp32; for 16-bit outputs the weights are rounded to
 * fp16, for fp32 outputs every operand is held in 22 bits or more.
 *
 * mass NULL, or fp32 [batch][h_kv][mass_stride] (8-byte aligned, mass_stride an even
 * number >= 64 * page_stride): the weight that each held position p has received so far,
 *   mass[b][j][p] += sum over query tokens i that see p and the G heads h of
 *                    KV head j of exp(q_i,h . k^_p / sqrt(head_dim) - lse_i,h),
 * summed in this order for every p, so that equal calls give equal bits.
 * rdkv_score's w_tok of a prompt is the same sum over the prompt's queries: copied in, it is
 * where the decode goes on.  A query head whose lse is not finite (it holds a NaN) adds
 * nothing, and neither does a call that reports RDKV_ERR_TIMEOUT, nor one after it before the
 * status is read.  Positions that are not
 * held are not touched: rows that are written over (rejected drafts) start with what mass
 * holds at their positions, so zero it there.  What a query token gave the positions before it stays
 * when that token is rejected: mass keeps no account by query, so a caller who does not want it there
 * copies mass before a call of drafts.  with_mass of the workspace query: 1 for calls with mass (it
 * then holds the logits too, 4 bytes for every query row and position that the page TABLE has room
 * for: some 256 * batch * n_q * h_q * page_stride), and such calls add one launch, which also grows with the table. */
size_t rdkv_q8_attn_workspace_bytes(const rdkv_q8_cache* cache, int32_t h_q, int32_t n_q, int32_t with_mass);
rdkv_status rdkv_q8_attn(const rdkv_q8_cache* cache, int32_t dtype, const void* q, int64_t q_stride, int32_t h_q,
                         int32_t n_q, float* mass, int64_t mass_stride, void* out, int32_t out_dtype, float* lse,
                         void* ws, size_t ws_bytes, void* stream);

/* Failure-detection self-test of rdkv_q8_attn, as rdkv_q4_timeout_selftest is
 * of rdkv_q4_attn (a page is withheld where its index plus the KV head is a
 * multiple of `withhold`); takes no mass. */
rdkv_status rdkv_q8_timeout_selftest(const rdkv_q8_cache* cache, int32_t dtype, const void* q, int64_t q_stride,
                                     int32_t h_q, int32_t n_q, void* out, int32_t out_dtype, float* lse, void* ws,
                                     size_t ws_bytes, int32_t withhold, int64_t wait_cycles, void* stream);

/* Brings every sequence that holds more than n_keep tokens down to n_keep, in
 * every KV head on its own: kept are the first n_first and the last n_last
 * positions and, of the others, those with the most mass (equal mass: the
 * lower position; a NaN counts as more than any number).  The kept rows move to positions
 * 0 .. n_keep - 1 in their order, within the sequence's own pages, and their
 * mass with them; the mass of positions n_keep .. lens[b] - 1 becomes 0, and so do
 * the codes behind position n_keep - 1 in its page.
 * kept [batch][h_kv][n_keep] int32: the position each row came from,
 * ascending; -1 behind the last.  A sequence of at most n_keep tokens stays as
 * it is (kept: its positions).  Pages whose rows all stay where they are stay as they
 * are; another page takes the scales that its rows need, by the rule of a page written
 * whole (values that fall below 2^-6 of their new scale are rounded once more).
 *
 * The caller lowers lens afterwards (min(lens[b], n_keep)), in place and on the
 * stream, as it raises it before a write; pages past it are then free.
 * 0 <= n_first, 0 <= n_last, n_first + n_last <= n_keep, 1 <= n_keep.  No page of
 * a sequence that is brought down may be shared with another sequence.  A
 * sequence with a page outside the pool (RDKV_ERR_INVALID_ARG in *status) is left as
 * it is, rows and mass, and its kept are -1.  ws as for rdkv_q8_attn, of
 * rdkv_q8_evict_workspace_bytes bytes: calls of both may follow one another on it.
 * Two launches.
 *
 * Rows move in place, so a wait that ran out cannot be taken back: after
 * RDKV_ERR_TIMEOUT from this call the rows, the scales, the mass and kept of the
 * sequences that held more than n_keep tokens are undefined, at the old length and
 * at the new one, and such a sequence has to be written anew.  Sequences of at
 * most n_keep tokens and pages that hold no token of the others are as they were,
 * and ws serves the next call.  (The wait is for another block of the same launch,
 * of some microseconds; its limit is some two seconds.) */
size_t rdkv_q8_evict_workspace_bytes(const rdkv_q8_cache* cache);
rdkv_status rdkv_q8_evict(const rdkv_q8_cache* cache, float* mass, int64_t mass_stride, int32_t n_keep, int32_t n_first,
                          int32_t n_last, int32_t* kept, void* ws, size_t ws_bytes, void* stream);

/* Failure-detection self-test of rdkv_q8_evict: its kernels on the same
 * arguments, but a page of a sequence whose index plus KV head is a multiple of
 * `withhold` (>= 1; 1: all) does not tell that its rows have been read, and a block
 * that waits for it gives up after `wait_cycles` SM clock cycles (clamped to [1e5,
 * 4e9]) and reports RDKV_ERR_TIMEOUT, as above: for a cache whose contents are not
 * needed.  RDKV_ERR_INVALID_ARG for withhold or wait_cycles <= 0, else as
 * rdkv_q8_evict. */
rdkv_status rdkv_q8_evict_timeout_selftest(const rdkv_q8_cache* cache, float* mass, int64_t mass_stride, int32_t n_keep,
                                           int32_t n_first, int32_t n_last, int32_t* kept, void* ws, size_t ws_bytes,
                                           int32_t withhold, int64_t wait_cycles, void* stream);

/* Reads *status and clears it.  SYNCHRONISES `stream`. */
rdkv_status rdkv_q8_status(const rdkv_q8_cache* cache, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* RDKV_H */
