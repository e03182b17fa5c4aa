/*
 * bsp.h - C ABI of the GB300 shared-prefix (cascade) beam decode attention
 * library (libbsp.so).
 *
 * One decode step of wide beam search over a paged KV cache, per layer:
 *   bsp_plan        host planning: validates lengths and beam 0's prompt page
 *                   tables, splits the prompt attention into work units and
 *                   stages the plan to the device without a stream sync;
 *   bsp_append_kv   writes each beam's new token K/V at its flat cache slot;
 *   bsp_decode_attn attends each request's shared prompt once for all of its
 *                   beams (tensor cores), each beam's own tail through
 *                   cache_indirection, and merges the two by log-sum-exp,
 *                   returning O and LSE.
 * Around it: bsp_process_logits, bsp_beam_select and bsp_beam_advance take the
 * step's logits to the next step's beams; bsp_key_weights and bsp_evict_prefix
 * shorten the prompts' cache to the rows that the attention looked at. For the
 * cache itself: appends that normalise and rotate, E4M3 pools with block scales
 * and their attention, and pages forked, given back, compacted and copied.
 * The method: TensorRT-LLM PR #21738, "Add opt-in cascade attention for wide
 * beam search on KVCM V2" (description, "Solution"); the valid-prefix bound:
 * TensorRT-Model-Connect PR #2202, "prefill and decode over the cached prefix,
 * not the whole KV allocation"; the append: TensorRT-LLM PR #18614, "Fuse
 * MiniMax-M3 MSA per-layer KV-cache writes into one kernel".
 *
 * Conventions for every call
 *  - Memory: all device and host memory is owned by the caller. The library
 *    allocates nothing and keeps no state between calls beyond what it writes
 *    into the caller's workspace.
 *  - Streams: `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *    stream). Every device effect of a call is enqueued on that stream; no call
 *    synchronises the stream unless documented (BSP_FLAG_CHECK,
 *    bsp_read_device_status).
 *  - Errors: arguments are validated on the host before anything is enqueued;
 *    on any error nothing is launched and pools/outputs are left unchanged.
 *    Indices that live in device memory (beam_pages, cache_indirection,
 *    out_cache_loc) cannot be validated without a sync: kernels bounds-check
 *    them, skip the access and set a flag in the workspace's device status
 *    word, which bsp_read_device_status (or BSP_FLAG_CHECK) reports as
 *    BSP_ERR_PAGE_INDEX. Kernels never trap.
 *  - Layouts (row-major, innermost last, 16-bit elements unless stated):
 *      q, o            [R = batch * beam_width][num_q_heads][head_dim], row r = b*W + w
 *      lse             [R][num_q_heads] float32
 *      k_pool, v_pool  [num_pages][num_kv_heads][page_size][head_dim]
 *      beam_pages      [R][beam_pages_stride] int32 page ids of each beam's sequence
 *      cache_indirection [batch][beam_width][max_seq] int32 source beam per position
 *    Query head h uses kv head h / (num_q_heads / num_kv_heads).
 *    Device pointers must be 16-byte aligned.
 */
#ifndef BSP_H_
#define BSP_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define BSP_API __attribute__((visibility("default")))
#else
#define BSP_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum bsp_status {
    BSP_OK = 0,
    BSP_ERR_INVALID_ARG = 1,  /* null/misaligned/host pointer, bad length or stride */
    BSP_ERR_UNSUPPORTED = 2,  /* dtype, head_dim, group size, page size or tail outside the supported set */
    BSP_ERR_PAGE_INDEX = 3,   /* a page id, slot, indirection value or RoPE position out of range */
    BSP_ERR_CAPACITY = 4,     /* workspace or staging buffer too small */
    BSP_ERR_STALE_PLAN = 5,   /* plan superseded by a newer bsp_plan on the same workspace */
    BSP_ERR_CUDA = 6,         /* a CUDA runtime/driver call failed */
    BSP_ERR_DEVICE_TIMEOUT = 7 /* a kernel's bounded wait gave up (reported by status reads) */
} bsp_status;

enum { BSP_DTYPE_BF16 = 0, BSP_DTYPE_FP16 = 1 };
/* What the K/V pools hold (bsp_geometry.kv_dtype): elements of `dtype`, or one-byte FP8 E4M3 values
   ("e4m3fn": 4 exponent bits with bias 7, 3 fraction bits, no infinities, max 448) in the same
   [page][kv head][slot][head_dim] layout */
enum { BSP_KV_DTYPE_SAME = 0, BSP_KV_DTYPE_E4M3 = 1 };

/* Launch flags (bsp_decode_attn, bsp_prefill_attn; bsp_key_weights takes LSE_BASE2, CHECK and ACCUMULATE) */
enum {
    BSP_FLAG_LSE_BASE2 = 1, /* write LSE as log2-sum-exp2 instead of the natural log */
    BSP_FLAG_CHECK = 2,     /* synchronise after the launches and report device status */
    BSP_FLAG_ACCUMULATE = 8, /* bsp_key_weights only: add to `weights` instead of writing it */
    BSP_FLAG_GRAPH = 4      /* bsp_decode_attn only, not with BSP_FLAG_CHECK: launch shapes that do not
                               depend on the plan's lengths, so that the launches may be captured in a
                               CUDA graph once and replayed after every later bsp_plan on the same
                               workspace with the same batch, beam_width, max_tail, geometry, SM count,
                               page-table stride and buffers (the CUDA-graph serving mode: TensorRT-LLM
                               PR #21738, description: the host plan of a step is made before capture and
                               before every replay; the tail bound caps the tail under graphs). The
                               prompt kernel runs one CTA per SM of the plan and the tail kernel is
                               always launched for max_tail tail rows; a replay whose staged plan has
                               another shape writes nothing and sets BSP_DEVFLAG_GRAPH */
};

#define BSP_MAX_TAIL 8   /* tail positions per beam (TensorRT-LLM PR #21738, description: correctness and limits) */
#define BSP_MAX_GROUP 8  /* query heads per kv head */

/* Bits of the device status word. */
#define BSP_DEVFLAG_PAGE_INDEX 1
#define BSP_DEVFLAG_TIMEOUT 2
#define BSP_DEVFLAG_POSITION 4  /* a RoPE position outside [0, max_position) (bsp_rope_append_kv) */
#define BSP_DEVFLAG_PAGES 16    /* bsp_fork_tables: not enough free pages for every row; reported as BSP_ERR_CAPACITY */
#define BSP_DEVFLAG_GRAPH 8     /* a replayed graph-mode launch found a plan of another shape (nothing
                                   written); reported as BSP_ERR_STALE_PLAN */

typedef struct bsp_geometry {
    int32_t num_q_heads;  /* Hq */
    int32_t num_kv_heads; /* Hkv; Hq % Hkv == 0, Hq / Hkv <= BSP_MAX_GROUP */
    int32_t head_dim;     /* 64, 128 or 256 */
    int32_t page_size;    /* tokens per page: 8, 16, 32, 64 or 128 */
    int32_t num_pages;    /* pages in each pool */
    int32_t dtype;        /* BSP_DTYPE_*; q, o and new K/V share it, and the pools unless kv_dtype says */
    int32_t kv_dtype;     /* BSP_KV_DTYPE_*: 0 (the pools hold `dtype`), or E4M3 pools, which decode
                             plans at head_dim 64 and 128 support (bsp_decode_attn_fp8; the writes:
                             bsp_append_kv_fp8, bsp_rope_append_kv_fp8); any other use returns
                             BSP_ERR_UNSUPPORTED */
} bsp_geometry;

/*
 * Plan of one decode step, filled by bsp_plan / bsp_plan_build. Caller-owned
 * plain data; the fields below `generation` describe the staged device image
 * and are read by the launches. A plan refers to the workspace it was staged
 * into; it stays valid until the next bsp_plan on that workspace.
 */
typedef struct bsp_plan_t {
    bsp_geometry geo;
    int32_t batch;               /* B */
    int32_t beam_width;          /* W (a prefill plan: the rows of a partial slot, the largest prompt) */
    int32_t max_tail;            /* bound on every tail_len, <= BSP_MAX_TAIL */
    int32_t prefix_pages_stride; /* row stride of the prefix_pages table given to the plan */
    int32_t num_units;           /* prompt-attention work units (CTAs) */
    int32_t num_parts;           /* (request, key split) prompt partial states */
    int32_t row_blocks;          /* query-row blocks per (request, kv head) */
    int32_t beams_per_block;     /* beams in one query-row block */
    int32_t tile_keys;           /* keys per prompt tile */
    int32_t max_prefix_len;      /* max_b P_b */
    int32_t max_total_len;       /* max_b P_b + T_b */
    int32_t num_sms;             /* SM count the units were balanced for */
    int32_t max_tail_len;        /* max_b T_b */
    int32_t prefix_ctas;         /* persistent CTAs of the prompt kernel (<= num_sms) */
    uint64_t generation;         /* staging generation of this plan (0: built only, not staged) */
    void* ws_device;             /* device workspace the plan was staged into */
    uint64_t ws_device_bytes;
    void* ws_host;               /* host staging buffer paired with ws_device */
    uint64_t image_bytes;        /* bytes of the staged plan image */
    uint64_t off_req;            /* byte offsets into ws_device */
    uint64_t off_units;
    uint64_t off_pages;
    uint64_t off_part_lse;
    uint64_t off_part_o;
    uint64_t device_bytes_used;
    int32_t tail_requests;       /* requests the tail kernel finishes (no prompt, a prompt split over
                                    several partial states, or more tail keys per row block than one
                                    tile holds); the prompt kernel finishes the others. No tail launch
                                    when 0 */
    int32_t total_rows;          /* query rows of the step: batch * beam_width (decode) or the prompt
                                    tokens of all requests (prefill) */
    int32_t kind;                /* 0: a decode-step plan (bsp_plan); 1: a prefill plan (bsp_plan_prefill) */
    int32_t layout;              /* prompt kernel of the plan: 0 one softmax warp set (head_dim 256, and
                                    decode row blocks of <= 64 query rows, two threads per row); 2 two
                                    MMA blocks in one CTA sharing every K/V tile: all 129-256 query rows
                                    of a (request, kv head) of a decode step (the prompt read once), or
                                    a prefill's prompt tokens at head_dim <= 128 in units of two blocks
                                    of beams_per_block = 4 * floor(32 / G) tokens; 1 two softmax warp
                                    sets taking a unit's key tiles alternately (other decode steps at
                                    head_dim <= 128) */
    uint64_t off_cta;            /* byte offset of the per-CTA unit table */
    int32_t max_splits;          /* the most prompt partial states of a request */
    int32_t reserved;
} bsp_plan_t;

/* Human-readable name of a bsp_status value. Never NULL. */
BSP_API const char* bsp_status_string(int32_t status);

/*
 * Rows to bind for a cached prefix of `valid_rows` rows in an allocation of
 * `capacity` rows: the next multiple of 256 rows, or a single row when nothing
 * is cached, at most the allocation (TensorRT-Model-Connect PR #2202,
 * Implementation: kv_cache.{h,cpp}, kCacheRowBucket). The kernels themselves
 * read only the valid rows; this is the bound a caller binds when it needs a
 * shape that changes once per 256 tokens. Returns -1 if capacity < 1.
 */
BSP_API int32_t bsp_bucket_rows(int32_t valid_rows, int32_t capacity);

/*
 * Upper bounds of the device workspace and the host staging buffer for plans
 * with batch <= max_batch, beam_width <= max_beam and prompt page tables of at
 * most max_prefix_pages pages (TensorRT-LLM PR #21738: the fp32 workspace is
 * sized once from the engine's largest row counts). The host staging buffer should
 * be pinned (page-locked) for the copy to be asynchronous.
 */
BSP_API bsp_status bsp_workspace_size(const bsp_geometry* geo, int32_t max_batch, int32_t max_beam,
                              int32_t max_prefix_pages, size_t* device_bytes, size_t* host_bytes);

/*
 * Host-only planning: validates the step and writes the device plan image into
 * `image` (host memory, `image_bytes` capacity) without touching CUDA. Used by
 * bsp_plan; exposed for tests and for callers that stage the image themselves.
 *   prefix_len[b]   valid prompt rows P_b >= 0 of request b (host)
 *   tail_len[b]     tail positions T_b in [0, max_tail] (host); the tail
 *                   includes the current token once it is appended
 *   prefix_pages    host [batch][prefix_pages_stride]: beam 0's page ids of the
 *                   prompt; the first ceil(P_b / page_size) entries of row b
 *                   are read and each must lie in [0, num_pages), else
 *                   BSP_ERR_PAGE_INDEX (never clamped) (TensorRT-LLM PR #21738,
 *                   the commit that makes an invalid prompt page id an error)
 *   max_tail        <= BSP_MAX_TAIL (the same PR's limit on the generated
 *                   positions a beam may hold in graph mode)
 *   num_sms         SMs to balance the prompt work units for (> 0)
 * `plan_out->generation` is 0 and the workspace fields are left NULL.
 */
BSP_API bsp_status bsp_plan_build(const bsp_geometry* geo, int32_t batch, int32_t beam_width,
                          const int32_t* prefix_len, const int32_t* tail_len, const int32_t* prefix_pages,
                          int32_t prefix_pages_stride, int32_t max_tail, int32_t num_sms, void* image,
                          size_t image_bytes, bsp_plan_t* plan_out);

/*
 * Plans one decode step (per-step host planning, TensorRT-LLM PR #21738: the
 * plan is made on the host before graph capture and before each replay, and its
 * inputs are staged in pinned memory so that planning every step never
 * synchronises the stream).
 * Builds the image (bsp_plan_build, balanced for the current device's SM
 * count), writes it into one of two slots of `ws_host` and enqueues its copy
 * into `ws_device` on `stream`. The workspace pair (ws_device, ws_host) must
 * have at least the sizes bsp_workspace_size reports; ws_host should be pinned.
 * A slot is rewritten only after the stream has finished copying the plan
 * that used it two plans earlier (the stream echoes a generation number back
 * into ws_host); if that has not happened the call waits for it, up to 10 s,
 * then returns BSP_ERR_CUDA. Planning again makes every earlier plan of this
 * workspace stale (BSP_ERR_STALE_PLAN from the launches) (TensorRT-LLM PR
 * #21738, the commit that discards the previous step's plan).
 */
BSP_API bsp_status bsp_plan(const bsp_geometry* geo, int32_t batch, int32_t beam_width, const int32_t* prefix_len,
                    const int32_t* tail_len, const int32_t* prefix_pages, int32_t prefix_pages_stride,
                    int32_t max_tail, void* ws_device, size_t ws_device_bytes, void* ws_host,
                    size_t ws_host_bytes, void* stream, bsp_plan_t* plan_out);

/*
 * Per-step update of a staged decode plan: the same batch, beam width, prompt
 * lengths and prompt pages, new tail lengths. Beam search keeps a request's
 * prompt fixed while its tail grows by one position a step, so the work units,
 * the CTA table and the prompt page list of the plan (the dealing, which costs
 * the planner O(units log units) and more) stay as they are; only the request
 * records change: T_b, and whether the prompt kernel or the tail kernel
 * finishes request b (the same rule bsp_plan applies). O(batch) host work and
 * one copy of the image header and request records (64 + 48 * batch bytes)
 * through the next staging slot, with the slot protocol of bsp_plan (TensorRT-
 * LLM PR #21738: per-step host planning with pinned staging and no stream
 * synchronisation). The units stay balanced for the tails the plan was built
 * with; re-plan with bsp_plan when the batch or a prompt changes.
 *   plan       in/out: a current decode plan of its workspace (from bsp_plan or
 *              an earlier update); on success its generation, max_tail_len,
 *              max_total_len and tail_requests describe the new step and
 *              every earlier plan of the workspace is stale
 *   tail_len   host [batch]: T_b in [0, plan->max_tail] (BSP_ERR_CAPACITY
 *              above it, BSP_ERR_INVALID_ARG below 0); nothing is changed on
 *              error
 *   stream     the stream of the step's launches (the copy is enqueued on it)
 * A CUDA graph captured with BSP_FLAG_GRAPH from a plan of this workspace
 * replays correctly after updates: the header it checks does not change.
 */
BSP_API bsp_status bsp_plan_update_tails(bsp_plan_t* plan, const int32_t* tail_len, void* stream);

/*
 * Paged KV append: for every new token i < n and kv head h, copies the
 * head_dim elements of k_new / v_new row i, head h to
 * pool[out_cache_loc[i] / page_size][h][out_cache_loc[i] % page_size][:],
 * bit for bit, in one launch (TensorRT-LLM PR #18614, description: one launch
 * per layer computes each slot's page and in-page row from out_cache_loc in
 * registers and writes K and V in the same pass).
 *   k_new, v_new    device [n] rows of num_kv_heads * head_dim contiguous
 *                   elements, rows `src_row_stride` elements apart
 *                   (>= num_kv_heads * head_dim, a multiple of 8), so that K
 *                   and V may be column slices of one projection output
 *   out_cache_loc   device int32 [n] flat slots; a slot outside
 *                   [0, num_pages * page_size) is skipped and flagged
 *   n               0 is a no-op returning BSP_OK; must be <= batch * beam_width
 *   events          NULL, or 2 cudaEvent_t (as void*) recorded on `stream`
 *                   before and after the append kernel (timing only; under
 *                   stream capture they become external event-record nodes)
 * Duplicate slots are a caller error (the surviving row is unspecified).
 */
BSP_API bsp_status bsp_append_kv(const bsp_plan_t* plan, const void* k_new, const void* v_new, int64_t src_row_stride,
                         const int32_t* out_cache_loc, int32_t n, void* k_pool, void* v_pool,
                         void* const* events, void* stream);

/*
 * Paged append into FP8 E4M3 pools (a KV cache kept in 8 bits; TensorRT-LLM
 * PR #18614, the review follow-up commit on the fused KV write: the
 * case of an fp8 source written to an fp8 cache, and the review of msa_scatter.py: the
 * write converts the source dtype to the cache's). Same slots, layout and
 * error behaviour as bsp_append_kv, with pools of one byte per element,
 * uint8 [num_pages][num_kv_heads][page_size][head_dim]:
 *   src_dtype = BSP_FP8_SRC_16BIT: k_new / v_new hold the geometry's dtype
 *                   (bf16 or fp16); element x is stored as the E4M3 value
 *                   nearest to fp32(x) * k_mul (v_mul for V), the product
 *                   rounded once to fp32, ties to even, values past +-448
 *                   saturated to +-448 (k_mul, v_mul finite and > 0: a cache's
 *                   per-tensor quantisation multipliers, 1 for a plain cast)
 *   src_dtype = BSP_FP8_SRC_E4M3: k_new / v_new hold E4M3 bytes, copied bit
 *                   for bit (the multipliers are not used)
 *   src_row_stride  elements of the source type between rows, >= num_kv_heads
 *                   * head_dim, rows 16-byte aligned (a multiple of 8 for a
 *                   16-bit source, of 16 for E4M3)
 * The plan may have either kv_dtype (the pools passed here are E4M3 either way);
 * bsp_decode_attn_fp8 reads such pools.
 */
enum { BSP_FP8_SRC_16BIT = 0, BSP_FP8_SRC_E4M3 = 1 };
BSP_API bsp_status bsp_append_kv_fp8(const bsp_plan_t* plan, const void* k_new, const void* v_new,
                                     int64_t src_row_stride, int32_t src_dtype, float k_mul, float v_mul,
                                     const int32_t* out_cache_loc, int32_t n, void* k_pool, void* v_pool,
                                     void* const* events, void* stream);

/*
 * Rotary position embedding (RoPE) on the paged append. The pages apply RoPE to
 * K before it is written to the paged cache (TensorRT-LLM PR #21738: the model
 * applies it itself, per the description; the review of flash_attn4_kernels.py
 * names the rope_write_kv_paged helper and its partial-RoPE partner lookup) but
 * do not define it; the definition is the published one (Su et al., RoFormer,
 * section 3.2): the first rotary_dim dims of a head row form rotary_dim/2 pairs,
 * pair j turns by the angle p * theta_j, theta_j = base^(-2j / rotary_dim),
 * (x, y) -> (x cos - y sin, y cos + x sin); the other dims pass unchanged.
 *
 * The caller-owned table of cos/sin values, device fp32
 *   cos_sin[p][j]                  = cos(p * theta_j),  j < rotary_dim / 2
 *   cos_sin[p][rotary_dim / 2 + j] = sin(p * theta_j),
 * p in [0, max_position), is filled once by bsp_rope_cos_sin.
 */
typedef struct bsp_rope_config {
    const float* cos_sin;   /* device [max_position][rotary_dim], 16-byte aligned */
    int32_t max_position;   /* rows of cos_sin */
    int32_t rotary_dim;     /* rotated leading dims of a head row: a multiple of 16, 16 .. head_dim */
    int32_t interleaved;    /* 0: pair j = dims (j, j + rotary_dim/2) (rotate-half, e.g. Qwen3);
                               1: pair j = dims (2j, 2j + 1) */
    int32_t reserved;       /* 0 */
} bsp_rope_config;

/*
 * Fills the cos/sin table of a bsp_rope_config: angles and their cos/sin in
 * fp64 on the device, each value rounded once to fp32. One launch on `stream`,
 * no sync.
 *   max_position   > 0 rows;  rotary_dim even, 2 .. 1024;  base > 1, finite
 *   cos_sin        device fp32 [max_position][rotary_dim], 16-byte aligned
 * Argument errors: BSP_ERR_INVALID_ARG before any launch.
 */
BSP_API bsp_status bsp_rope_cos_sin(int32_t max_position, int32_t rotary_dim, double base, float* cos_sin,
                                    void* stream);

/*
 * Paged append with RoPE, one launch: for every new token i < n at position
 * positions[i] and slot out_cache_loc[i], the kv head rows of k_new are rotated
 * and written, the rows of v_new copied, to
 * pool[slot / page_size][h][slot % page_size][:] (as bsp_append_kv); when q is
 * non-NULL, the token's num_q_heads query rows are rotated in place. Rotation
 * in fp32 from the fp32 table (one fused multiply-add per output after one
 * product), rounded to nearest even into the pools' dtype; V rows and dims past
 * rotary_dim are copied bit for bit.
 *   plan            a decode or prefill plan (geometry, status word, n bound)
 *   rope            table and layout (bsp_rope_config)
 *   positions       device int32 [n]: the token's logical position (a decode
 *                   step: P_b + T_b - 1 for every beam of request b; a
 *                   prefill: C_b + t)
 *   q               NULL, or device [n] rows of num_q_heads * head_dim elements
 *                   q_row_stride elements apart (>= that, a multiple of 8)
 *   k_new, v_new, src_row_stride, out_cache_loc, n, k_pool, v_pool, events:
 *                   as bsp_append_kv
 * A token whose slot is outside [0, num_pages * page_size) or whose position is
 * outside [0, max_position) is skipped entirely (no pool row written, its q rows
 * left as they were) and sets BSP_DEVFLAG_PAGE_INDEX or BSP_DEVFLAG_POSITION;
 * bsp_read_device_status reports either as BSP_ERR_PAGE_INDEX. Host-checkable
 * errors return before any launch with nothing written.
 */
BSP_API bsp_status bsp_rope_append_kv(const bsp_plan_t* plan, const bsp_rope_config* rope, const int32_t* positions,
                                      void* q, int64_t q_row_stride, const void* k_new, const void* v_new,
                                      int64_t src_row_stride, const int32_t* out_cache_loc, int32_t n,
                                      void* k_pool, void* v_pool, void* const* events, void* stream);

/*
 * RoPE on the append into FP8 E4M3 pools (the fused write of the FP8 KV path:
 * TensorRT-LLM PR #18614, the review follow-up commit on the fused KV
 * write, where the RoPE kernel writes K and V as E4M3). As bsp_rope_append_kv, except that
 * k_pool / v_pool are uint8 E4M3 pools: each rotated K value (fp32, not rounded
 * to 16 bits first) times k_mul and each V value times v_mul, the product
 * rounded to fp32, is stored as the nearest E4M3 value (ties to even,
 * saturating at +-448); q (if given) is rotated in place in its 16-bit dtype.
 * k_mul, v_mul finite and > 0. Errors as bsp_rope_append_kv.
 */
BSP_API bsp_status bsp_rope_append_kv_fp8(const bsp_plan_t* plan, const bsp_rope_config* rope, const int32_t* positions,
                                          void* q, int64_t q_row_stride, const void* k_new, const void* v_new,
                                          int64_t src_row_stride, float k_mul, float v_mul,
                                          const int32_t* out_cache_loc, int32_t n, void* k_pool, void* v_pool,
                                          void* const* events, void* stream);

/*
 * Rotary tables of a model stretched beyond the length it was trained for: bsp_rope_cos_sin with scaled frequencies,
 * theta_j = base^(-2j / rotary_dim) before, and both halves of the table times `amplitude`. fp64 on the device, each
 * value rounded once. Kinds:
 *   BSP_ROPE_LINEAR  theta_j / factor (position interpolation)
 *   BSP_ROPE_BASE    a base of base * factor^(rotary_dim / (rotary_dim - 2)); rotary_dim > 2
 *   BSP_ROPE_BANDS   by the turns t_j = original_positions * theta_j / (2 pi) that a pair makes over the trained length
 *                    (as Peng et al., YaRN, section 3.2): theta_j * ((1 - s) / factor + s),
 *                    s = clamp((t_j - low) / (high - low), 0, 1)
 *   BSP_ROPE_RAMP    by the pair's index, linear between the indices of the two turns, rounded outwards (the form that
 *                    implementations of YaRN use): theta_j / factor * s + theta_j * (1 - s),
 *                    s = clamp((j - lo) / max(hi - lo, 0.001), 0, 1) with i(t) = rotary_dim * ln(original_positions /
 *                    (2 pi t)) / (2 ln base), lo = max(floor(i(high)), 0), hi = min(ceil(i(low)), rotary_dim - 1)
 * factor > 0, amplitude > 0 finite; BANDS and RAMP: original_positions > 0 and 0 < low < high, finite (not read
 * otherwise). Errors as bsp_rope_cos_sin. (No counterpart on the pages the method comes from.)
 */
enum { BSP_ROPE_LINEAR = 1, BSP_ROPE_BASE = 2, BSP_ROPE_BANDS = 3, BSP_ROPE_RAMP = 4 };
typedef struct bsp_rope_scaling {
    int32_t kind;                /* BSP_ROPE_* */
    int32_t original_positions;
    double factor;
    double low, high;            /* turns */
    double amplitude;            /* 1: plain cos and sin */
} bsp_rope_scaling;
BSP_API bsp_status bsp_rope_cos_sin_scaled(int32_t max_position, int32_t rotary_dim, double base,
                                           const bsp_rope_scaling* scaling, float* cos_sin, void* stream);

/*
 * The append of a layer that normalises its queries and keys per head, one launch: every K row and query row x of
 * head_dim elements becomes
 *   y = x / sqrt(mean(x^2) + eps) * (w + weight_offset)
 * in fp32 (sum of squares too: rows with elements beyond about 1e18 leave its range), is rotated by its token's
 * position as in bsp_rope_append_kv (rope NULL: not), and is rounded once; K goes to the pool, the query row to q_out.
 * V rows are copied bit for bit (E4M3 pools: quantised as in bsp_append_kv_fp8).
 *   norm            weights and eps; q_weight, k_weight device [head_dim], 16-byte aligned, in the geometry's dtype or
 *                   fp32 (weight_fp32 = 1), or NULL: ones (weight_offset is then not added); eps >= 0, finite
 *   q, q_row_stride NULL, or device [n] rows of num_q_heads * head_dim elements q_row_stride apart
 *   q_out, q_out_stride  where the query rows go (with q): q itself with its stride, or memory that overlaps none of the
 *                   call's inputs (BSP_ERR_INVALID_ARG; rows of q_out's stride are compared as they lie, so a column
 *                   slice of the buffer that holds the inputs will do, rows of another stride by all that they span);
 *                   rows of decode_attn's q when q_out_stride = num_q_heads * head_dim
 *   positions       device int32 [n]; NULL without rope
 *   other arguments, skipped tokens and errors: as bsp_rope_append_kv (events too)
 * The _fp8 form writes E4M3 pools with one multiplier per tensor. (No counterpart on the pages the method comes from.)
 */
typedef struct bsp_qk_norm {
    const void* q_weight;
    const void* k_weight;
    float eps;
    float weight_offset;   /* 0, or 1 for weights stored as their distance from one */
    int32_t weight_fp32;
    int32_t reserved;      /* 0 */
} bsp_qk_norm;
BSP_API bsp_status bsp_norm_rope_append_kv(const bsp_plan_t* plan, const bsp_qk_norm* norm, const bsp_rope_config* rope,
                                           const int32_t* positions, const void* q, int64_t q_row_stride, void* q_out,
                                           int64_t q_out_stride, const void* k_new, const void* v_new,
                                           int64_t src_row_stride, const int32_t* out_cache_loc, int32_t n, void* k_pool,
                                           void* v_pool, void* const* events, void* stream);
BSP_API bsp_status bsp_norm_rope_append_kv_fp8(const bsp_plan_t* plan, const bsp_qk_norm* norm,
                                               const bsp_rope_config* rope, const int32_t* positions, const void* q,
                                               int64_t q_row_stride, void* q_out, int64_t q_out_stride,
                                               const void* k_new, const void* v_new, int64_t src_row_stride, float k_mul,
                                               float v_mul, const int32_t* out_cache_loc, int32_t n, void* k_pool,
                                               void* v_pool, void* const* events, void* stream);

/*
 * Cascade decode attention (TensorRT-LLM PR #21738, description, "Solution"):
 * for every row r = b*W + w and query head h,
 *   O[r][h] = softmax(scale * q K^T) V over the beam's logical sequence:
 *             prompt positions j < P_b read through beam 0's prompt pages
 *             (the plan's prefix_pages), tail positions j in [P_b, P_b + T_b)
 *             read through beam_pages[b*W + cache_indirection[b][w][j]];
 *   LSE[r][h] = log-sum-exp of the scaled scores (natural log, or base 2 with
 *             BSP_FLAG_LSE_BASE2); an empty sequence gives O = 0, LSE = -inf.
 * Each (request, kv head) reads its prompt keys a single time for all beams and query
 * heads (tensor cores), the tail per beam, and the two merge exactly by
 * log-sum-exp. Only the valid P_b prompt rows are read, never the allocation.
 * Values are finite numbers: an infinity or NaN in a beam's tail may reach the
 * outputs of the request's other beams, for which its probability is 0. In a
 * key it stays with the rows that attend it.
 *   beam_pages_stride  entries per beam_pages row, >= ceil(max(P_b+T_b)/page_size)
 *   max_seq            innermost extent of cache_indirection, >= max(P_b + T_b)
 *   softmax_scale      > 0, typically 1/sqrt(head_dim)
 *   flags              BSP_FLAG_* bits
 *   events             NULL, or 3 cudaEvent_t (as void*) recorded on `stream`
 *                      before the prompt kernel, between the prompt and the
 *                      tail kernels, and after the tail kernel (timing only;
 *                      under stream capture they become external event-record
 *                      nodes)
 * The plan must be the latest one staged into its workspace.
 */
BSP_API bsp_status bsp_decode_attn(const bsp_plan_t* plan, const void* q, const void* k_pool, const void* v_pool,
                           const int32_t* beam_pages, int32_t beam_pages_stride, const int32_t* cache_indirection,
                           int32_t max_seq, float softmax_scale, int32_t flags, void* o, float* lse,
                           void* const* events, void* stream);

/*
 * bsp_decode_attn over FP8 E4M3 pools (TensorRT-LLM PR #18614, the review
 * follow-up commit on the fused KV write: a KV cache kept in 8 bits, written by
 * bsp_append_kv_fp8). The plan's geometry has kv_dtype = BSP_KV_DTYPE_E4M3 (and
 * head_dim 64 or 128); k_pool and v_pool hold one byte per element. Key and
 * value element x of the pools stand for e4m3(x) * k_scale and
 * e4m3(x) * v_scale (per-tensor scales, finite and > 0; 1 and 1 read the codes
 * as they are). The result is the decode attention of bsp_decode_attn over
 * those keys and values:
 *   O   = softmax(softmax_scale * k_scale * q . e4m3(K)) e4m3(V) * v_scale
 *   LSE = log-sum-exp of softmax_scale * k_scale * q . e4m3(K)
 * The kernels read the E4M3 tiles (half the bytes of the 16-bit pools) and
 * widen them exactly to the q dtype in shared memory (every E4M3 value is a
 * bf16 and a binary16 value), so the tensor-core products are those of the
 * 16-bit path. A NaN code (0x7f, 0xff) in a key that a row of q attends makes
 * the row's output and LSE NaN, one in a value the output's element of that
 * column (in a tail row it may be all of the row's output and its LSE); rows
 * that do not attend it are what they are without it. Other arguments, flags,
 * events and errors as bsp_decode_attn; a plan whose pools are not E4M3 is BSP_ERR_INVALID_ARG here,
 * and an E4M3 plan is BSP_ERR_INVALID_ARG for bsp_decode_attn, bsp_append_kv
 * and bsp_rope_append_kv.
 */
BSP_API bsp_status bsp_decode_attn_fp8(const bsp_plan_t* plan, const void* q, const void* k_pool, const void* v_pool,
                               const int32_t* beam_pages, int32_t beam_pages_stride,
                               const int32_t* cache_indirection, int32_t max_seq, float softmax_scale,
                               float k_scale, float v_scale, int32_t flags, void* o, float* lse,
                               void* const* events, void* stream);

/*
 * E4M3 pools with block scales: each block of `block` consecutive slots of a (page, kv head) has a scale of its own
 * for K and for V, a power of two kept as its exponent byte E: element x of the block stands for
 * e4m3(x) * 2^(E - 127). E = 0 means that nothing has been written to the block (its codes are read as 0, those of
 * NaN as NaN). An 8-bit float loses nothing by a power of two, so the scale only places its range; it can be changed
 * without rounding the codes again (but for those that leave the range below), and the product is exact in 16 bits:
 * bf16 takes exponents E - 127 up to 15, fp16 those in [-15, 7]; larger ones (fp16: smaller ones too) are read as the
 * nearest of these.
 * Only calls that take a bsp_block_scales know of the scales, and no call can tell such pools from others:
 * bsp_decode_attn_fp8, bsp_key_weights_fp8 and the appends with one multiplier per tensor pass the exponents over,
 * bsp_evict_prefix moves codes between blocks without them, and so do bsp_fork_rows and bsp_copy_pages with scales NULL.
 * Their results over such pools are wrong.
 * (These entry points have no counterpart on the pages the method comes from.)
 */
#define BSP_MAX_SCALE_BLOCK 32
typedef struct bsp_block_scales {
    uint8_t* k;        /* device [num_pages][num_kv_heads][page_size / block], 16-byte aligned; zeroed once */
    uint8_t* v;        /* the same for V */
    int32_t block;     /* slots of a block: a power of two, at most the page size and BSP_MAX_SCALE_BLOCK */
    int32_t reserved;  /* 0 */
} bsp_block_scales;

/*
 * The append into such pools, one launch: K rows (normalised with norm, rotated with rope; each may be NULL) and V rows
 * of the geometry's dtype become codes and scales, query rows go to q_out as in bsp_norm_rope_append_kv. The tokens of
 * a call whose slots are in one block form a run and must stand next to one another in ascending order of their slots,
 * as a prompt's or a beam's do; otherwise, and where a skipped token (which is flagged) parts a run, the codes and scale
 * that the block ends up with are unspecified. With top the largest finite or infinite magnitude of the run's rows (of
 * one head, of K or of V):
 *  - E is the smallest exponent byte with top <= 448 * 2^(E - 127), within 27 .. 142 (fp16: 112 .. 134): for all but
 *    the largest values nothing saturates; 0 if top is 0;
 *  - a run that begins at the block's first slot starts the block anew with E. Another keeps the rows before it: the
 *    block's exponent becomes the larger of E and its own (as it is read, see above), and if it grew, the codes of the
 *    slots before the run are brought to it (times a power of two, rounded to nearest even). So a page that is taken
 *    from another sequence and not written from a block's first slot on has its exponents cleared, or copied with its
 *    rows, first. An exponent of 0 has no rows to keep: codes of slots that nothing was written to stay, and are read
 *    as 0 no longer but at the new scale (no sequence reads such slots);
 *  - x is stored as the E4M3 value nearest to x * 2^(127 - E), ties to even, saturated to +-448; a NaN as a NaN code.
 * The plan may have either kv_dtype and any head_dim. Other arguments and errors as bsp_norm_rope_append_kv.
 */
BSP_API bsp_status bsp_append_kv_fp8_blocks(const bsp_plan_t* plan, const bsp_qk_norm* norm, const bsp_rope_config* rope,
                                            const int32_t* positions, const void* q, int64_t q_row_stride, void* q_out,
                                            int64_t q_out_stride, const void* k_new, const void* v_new,
                                            int64_t src_row_stride, const int32_t* out_cache_loc, int32_t n, void* k_pool,
                                            void* v_pool, const bsp_block_scales* scales, void* const* events,
                                            void* stream);

/*
 * bsp_decode_attn over E4M3 pools with block scales (the plan's geometry has kv_dtype = BSP_KV_DTYPE_E4M3 and head_dim
 * 64 or 128): bsp_decode_attn over the keys and values that the codes and scales stand for, prompt and tail alike. A
 * tile's codes are widened together with their scales, exactly, so the scales cost one byte read per row and no product
 * of their own. Other arguments, flags, events and errors as bsp_decode_attn_fp8.
 */
BSP_API bsp_status bsp_decode_attn_fp8_blocks(const bsp_plan_t* plan, const void* q, const void* k_pool,
                                              const void* v_pool, const bsp_block_scales* scales,
                                              const int32_t* beam_pages, int32_t beam_pages_stride,
                                              const int32_t* cache_indirection, int32_t max_seq, float softmax_scale,
                                              int32_t flags, void* o, float* lse, void* const* events, void* stream);

/*
 * Prefill over the cached prefix (TensorRT-Model-Connect PR #2202, "prefill and
 * decode over the cached prefix, not the whole KV allocation", Implementation:
 * the prompt rows attend the bound cache rows and then the prompt rows, with
 * only the valid cached prefix bound). Request b holds cached_len[b] >= 0 valid
 * cached rows and prompt_len[b] >= 0 prompt tokens, whose K/V the caller has
 * already written (bsp_append_kv) at logical positions cached_len[b] ..
 * cached_len[b] + prompt_len[b] - 1; every position p of request b is read
 * through its page table: page = pages[b * pages_stride + p / page_size],
 * slot = p % page_size (the first ceil((cached + prompt) / page_size) entries
 * must lie in [0, num_pages), else BSP_ERR_PAGE_INDEX). With `causal` != 0,
 * prompt token i sees positions 0 .. cached_len[b] + i, else all
 * cached_len[b] + prompt_len[b] positions. Positions past those are never
 * read. Values are finite numbers: an infinity or NaN in one prompt token's may
 * reach the outputs of tokens before it. The query rows are the prompt tokens of all requests in order (request
 * b's tokens start at the sum of the earlier prompt_len), `total_rows` in all.
 * A request whose longest work unit is above the launch's mean load per SM has
 * its cached rows cut into key ranges (every cut inside the cached rows, so
 * that each prompt row has keys in each range); the prompt kernel writes one
 * partial state per range and the tail kernel merges them (the plan's
 * tail_requests counts such requests, its beam_width is then the rows of a
 * partial slot: the largest prompt_len). bsp_plan_prefill_build writes the host
 * image only (as bsp_plan_build); bsp_plan_prefill stages it without a sync (as
 * bsp_plan); the workspace must hold a plan of max_batch = batch and max_beam =
 * 1 (bsp_workspace_size), and with max_beam = the largest prompt_len it also
 * holds the partial states of key splits: bsp_plan_prefill plans without them
 * when they do not fit.
 */
BSP_API bsp_status bsp_plan_prefill_build(const bsp_geometry* geo, int32_t batch, const int32_t* cached_len,
                                  const int32_t* prompt_len, const int32_t* pages, int32_t pages_stride,
                                  int32_t causal, int32_t num_sms, void* image, size_t image_bytes,
                                  bsp_plan_t* plan_out);
BSP_API bsp_status bsp_plan_prefill(const bsp_geometry* geo, int32_t batch, const int32_t* cached_len,
                            const int32_t* prompt_len, const int32_t* pages, int32_t pages_stride,
                            int32_t causal, void* ws_device, size_t ws_device_bytes, void* ws_host,
                            size_t ws_host_bytes, void* stream, bsp_plan_t* plan_out);

/*
 * The prefill attention of a bsp_plan_prefill plan: for every prompt row r and
 * query head h, O[r][h] = softmax(scale * q K^T) V and LSE[r][h] over the keys
 * the plan gives that row, on the tensor cores (the prompt kernel: at head_dim
 * <= 128 each (request, kv head, two blocks of 4 * floor(32 / G) prompt tokens,
 * key range) a work unit of the two-block kernel, at 256 each (request, kv
 * head, block of floor(128 / G) tokens, key range) one of the one-set kernel; a
 * causal unit reads keys only up to its last token; then the tail kernel for
 * the requests whose keys were split). q, o [total_rows][Hq][head_dim]
 * in the pools' dtype, lse [total_rows][Hq] fp32 (natural log, or base 2 with
 * BSP_FLAG_LSE_BASE2). A decode plan is BSP_ERR_INVALID_ARG here (and a prefill
 * plan in bsp_decode_attn). events: NULL or 3 cudaEvent_t, as bsp_decode_attn.
 */
BSP_API bsp_status bsp_prefill_attn(const bsp_plan_t* plan, const void* q, const void* k_pool, const void* v_pool,
                            float softmax_scale, int32_t flags, void* o, float* lse, void* const* events,
                            void* stream);

/*
 * Synchronises `stream`, then reads the workspace's device status word into
 * *flags_out (BSP_DEVFLAG_* bits set by kernels since the last clear) and
 * clears it when `clear` is non-zero. Returns, for the bits that are set, the
 * first of BSP_ERR_PAGE_INDEX, BSP_ERR_STALE_PLAN (BSP_DEVFLAG_GRAPH),
 * BSP_ERR_CAPACITY (BSP_DEVFLAG_PAGES) and BSP_ERR_DEVICE_TIMEOUT; BSP_OK when
 * there are none.
 */
BSP_API bsp_status bsp_read_device_status(const bsp_plan_t* plan, void* stream, int32_t clear, int32_t* flags_out);

/* Size, in MiB, of the fixed device scratch array of bsp_decode_attn_noalloc (one per GPU). */
#define BSP_NOALLOC_SCRATCH_MIB 32

/*
 * bsp_decode_attn_noalloc - the same cascade decode attention as
 * bsp_decode_attn, for callers that cannot allocate device memory.
 * (This entry point has no counterpart on the pages the method comes from.)
 *
 * Some callers cannot call cudaMalloc on the decode path: serving engines that
 * give the whole GPU to their KV-cache pools at start-up and forbid later
 * allocations, plugins whose host runtime owns every device allocation, and
 * code that must not take the allocator's locks while it decodes. This call
 * takes no workspace: it plans the step itself (the arguments of bsp_plan) and
 * keeps its scratch (plan image, status word, prompt partial states) in one
 * fixed device array of BSP_NOALLOC_SCRATCH_MIB MiB compiled into the library.
 * It calls no cudaMalloc, cudaFree or other allocating routine.
 *  - Set-up: CUDA loads a library's device code lazily by default
 *    (CUDA_MODULE_LOADING=LAZY), and the array is placed on a device when this
 *    call first looks it up there. So call it once per device with batch = 0
 *    (and a valid geometry; nothing else is read) before allocating the KV
 *    pools: that call only looks the array up, with the device current, and
 *    returns BSP_OK. (With CUDA_MODULE_LOADING=EAGER the array is placed when
 *    the library is loaded.) From then on the device holds the array until the
 *    process exits. Every call looks the address up again, so no address
 *    outlives a device reset.
 *  - All calls share the array, which keeps the last call's contents; the call
 *    clears the status word itself. Calls whose GPU work overlaps (different
 *    streams or host threads) race on the array: serialise them.
 *  - A call on a stream that is being captured into a CUDA graph returns
 *    BSP_ERR_INVALID_ARG before anything is looked up or enqueued: each call
 *    copies its plan from one shared host array, so a captured copy would
 *    replay a later call's plan.
 *  - Indices in device memory (cache_indirection, beam_pages) are checked by
 *    the kernels as in bsp_decode_attn, and a bad one sets a bit in the array's
 *    status word; only BSP_FLAG_CHECK (which synchronises the stream) reads it
 *    back, as BSP_ERR_PAGE_INDEX. Without that flag such errors go unreported.
 *  - A step whose plan image and prompt partials need more than the array is
 *    rejected with BSP_ERR_CAPACITY before anything is enqueued.
 * Inputs, outputs, layouts, flags (BSP_FLAG_LSE_BASE2, BSP_FLAG_CHECK) and
 * errors are otherwise those of bsp_plan and bsp_decode_attn; the plan arrays
 * are host memory, every other pointer device memory. The plan image is copied
 * from host memory that is not page-locked. 16-bit pools only: a geometry with
 * E4M3 pools is BSP_ERR_UNSUPPORTED here.
 */
BSP_API bsp_status bsp_decode_attn_noalloc(const bsp_geometry* geo, int32_t batch, int32_t beam_width,
                                           const int32_t* prefix_len, const int32_t* tail_len,
                                           const int32_t* prefix_pages, int32_t prefix_pages_stride,
                                           int32_t max_tail, const void* q, const void* k_pool,
                                           const void* v_pool, const int32_t* beam_pages, int32_t beam_pages_stride,
                                           const int32_t* cache_indirection, int32_t max_seq, float softmax_scale,
                                           int32_t flags, void* o, float* lse, void* stream);

/* ------------------------------------------------------------------------------------------------------
 * Around the attention of a step: from logits to beams, and from attention weights to a shorter cache.
 * (These entry points have no counterpart on the pages the method comes from.)
 *
 * These calls take the plan of the step for its batch, beam width, lengths, prompt pages and status word.
 * They follow the conventions above: host-checkable errors return before any launch; nothing is allocated or
 * synchronised; indices in device memory are checked by the kernels. Their logits, scores, lists and tables
 * need the alignment of their element only (q, the pools and workspaces: 16 bytes), and every pointer, the plan's
 * workspace too, must be memory of the current device (or managed memory). They may be captured into a CUDA graph
 * (without BSP_FLAG_CHECK, which synchronises). bsp_process_logits and bsp_beam_select take only the batch, the beam
 * width and the status word of the plan, at the call. The others read the lengths from the staged plan, so that a replay
 * follows later decode plans of the same batch, beam width and (bsp_key_weights, bsp_evict_prefix) geometry; a replay
 * that finds any other plan, after a capture on a prefill plan any but that very one, or lengths past the tables it was
 * captured with, leaves what it would write and sets BSP_DEVFLAG_GRAPH.
 */

enum { BSP_LOGITS_BF16 = 0, BSP_LOGITS_FP16 = 1, BSP_LOGITS_FP32 = 2 };

#define BSP_MAX_VOCAB (1 << 21)
#define BSP_MAX_LISTED 8192          /* token_cols (with frequency or presence penalties) + bias_cols */
#define BSP_MAX_CANDIDATES 512       /* continuations per request of bsp_beam_select */
#define BSP_MAX_ADVANCE_BEAMS 16384
#define BSP_MAX_STEP_BATCH 65535     /* requests of bsp_beam_select and bsp_evict_prefix */
#define BSP_MAX_WEIGHTS_BATCH 4096
#define BSP_MAX_EVICT_ROWS (1 << 19) /* prompt rows per request of bsp_evict_prefix */

/* Grammar masks, packed: token t is allowed by state s when bit t % 32 of bits[s * stride + t / 32] is set.
   index[r] is beam row r's state; -1 leaves the row unmasked (so does an index >= rows, which is flagged as
   BSP_DEVFLAG_PAGE_INDEX). bits NULL: no masks. */
typedef struct bsp_token_mask {
    const uint32_t* bits;   /* device [rows][stride] */
    int64_t stride;         /* words, >= ceil(vocab / 32) */
    const int32_t* index;   /* device [batch * beam_width] */
    int32_t rows;
    int32_t reserved;       /* 0 */
} bsp_token_mask;

/* What bsp_process_logits does to a row. All device pointers; NULL leaves the step out. Tokens outside
   [0, vocab) in the lists are padding and are passed over; lengths are cut to [0, cols]. */
typedef struct bsp_logits_params {
    const int32_t* prompt_tokens;   /* [batch][prompt_stride]: the request's prompt, shared by its beams */
    const int32_t* prompt_len;      /* [batch] */
    int64_t prompt_stride;
    const int32_t* tokens;          /* [batch * beam_width][token_stride]: what the beam generated */
    const int32_t* token_len;       /* [batch * beam_width] */
    int64_t token_stride;
    const int32_t* bias_tokens;     /* [batch][bias_stride]; an id given twice: its first value counts */
    const float* bias_values;       /* [batch][bias_stride] */
    const int32_t* bias_len;        /* [batch], or NULL: bias_cols entries each */
    int64_t bias_stride;
    const float* repetition_penalty; /* [batch], > 0 */
    const float* frequency_penalty;  /* [batch] */
    const float* presence_penalty;   /* [batch] */
    const float* temperature;        /* [batch], > 0 and large enough for a finite reciprocal (from 2^-127 on) */
    bsp_token_mask mask;
    int32_t prompt_cols, token_cols, bias_cols; /* columns of the lists */
    int32_t reserved;               /* 0 */
} bsp_logits_params;

/*
 * Penalties, biases, temperature and grammar masks on the logits of every beam row, with the log-sum-exp of
 * each processed row, in one pass. In fp32, in this order, for token t of row r of request b:
 *   1. t in the prompt or in the row's generated tokens: x = x > 0 ? x / repetition : x * repetition;
 *   2. t generated c > 0 times: x = x - frequency * c, then x = x - presence;
 *   3. t in the bias list: x = x + bias;
 *   4. x = x / temperature (as the product with its rounded reciprocal);
 *   5. t not allowed by the row's grammar state: x = -inf, whatever it was (NaN and infinities included).
 * The result is rounded once to the logits' type. lse[r] (fp32, natural log; may be NULL) is that of the stored
 * values: -inf for a row without a finite one, +inf with +inf in the row, NaN with a NaN.
 *   logits, out     [batch * beam_width] rows of vocab elements, logits_stride / out_stride elements apart
 *                   (>= vocab). out may be logits itself (same stride): only vectors that change are written
 *                   then; any other overlap of the two address ranges (first row's start to last row's end) is
 *                   BSP_ERR_INVALID_ARG
 * A tensor-parallel or padded head's columns past vocab are neither read nor written.
 */
BSP_API bsp_status bsp_process_logits(const bsp_plan_t* plan, const void* logits, int32_t logits_dtype,
                                      int64_t logits_stride, int32_t vocab, const bsp_logits_params* params,
                                      void* out, int64_t out_stride, float* lse, void* stream);

/*
 * The best continuations of each request over the vocabularies of all of its beams: the num_candidates largest
 * of
 *   score(w, t) = fl(fl(x[b * W + w][t] - lse[b * W + w]) + cum_scores[b][w])
 * (two fp32 operations, so the choice is exactly reproducible), in descending order; equal scores (-0 and +0
 * among them) go by the lower beam, then the lower token. A token the mask rejects, and a score of -inf or
 * NaN, is no candidate; a beam whose cumulative score is -inf or NaN is not read. Places without a candidate
 * get score -inf, parent -1 and token -1.
 *   cum_scores      device [batch] rows of beam_width fp32, cum_stride apart (the scores of the step before)
 *   mask            NULL, or the grammar masks: rejected logits are then not read. Logits that
 *                   bsp_process_logits has masked need none
 *   scores, parents, tokens   device [batch][num_candidates]; may not overlap the inputs
 *   workspace       16-byte aligned device memory of bsp_beam_select_workspace_size bytes; its contents need not
 *                   be kept or cleared. Calls whose GPU work overlaps (two graphs too) need one each
 * beam_width * vocab must be below 2^32.
 */
BSP_API bsp_status bsp_beam_select_workspace_size(int32_t batch, int32_t beam_width, int32_t vocab,
                                                  int32_t num_candidates, size_t* device_bytes);
BSP_API bsp_status bsp_beam_select(const bsp_plan_t* plan, const void* logits, int32_t logits_dtype,
                                   int64_t logits_stride, int32_t vocab, const float* lse, const float* cum_scores,
                                   int64_t cum_stride, const bsp_token_mask* mask, int32_t num_candidates,
                                   float* scores, int32_t* parents, int32_t* tokens, void* workspace,
                                   size_t workspace_bytes, void* stream);

/*
 * The beams' tables after a step's choice, for the step that follows: with p = parents[b][w], P = P_b and
 * T = T_b of the plan (the tail positions that exist),
 *   ci_out[b][w][P + j]      = ci_in[b][p][P + j], j < T;     ci_out[b][w][P + T] = w
 *   tokens_out[b * W + w][j] = tokens_in[b * W + p][j], j < T; tokens_out[b * W + w][T] = chosen[b][w]
 *   token_len[b * W + w]     = T + 1
 * Other entries stay as they were. Each output may be its input (no other overlap). A parent of -1 (a place
 * without a candidate) keeps the beam's own rows; one outside [-1, beam_width) does so too and is flagged as
 * BSP_DEVFLAG_PAGE_INDEX.
 *   parents, chosen  device [batch] rows, cand_stride (>= beam_width) apart, the first beam_width of each read
 *   ci_in, ci_out    device [batch][beam_width][max_seq], max_seq > max(P_b + T_b); both NULL: left out
 *   tokens_in, tokens_out  device [batch * beam_width] rows of token_cols (> max T_b) entries, token_stride
 *                    apart; both NULL: left out
 *   token_len        device [batch * beam_width] or NULL
 */
BSP_API bsp_status bsp_beam_advance(const bsp_plan_t* plan, const int32_t* parents, const int32_t* chosen,
                                    int64_t cand_stride, const int32_t* ci_in, int32_t* ci_out, int32_t max_seq,
                                    const int32_t* tokens_in, int32_t* tokens_out, int64_t token_stride,
                                    int32_t token_cols, int32_t* token_len, void* stream);

/*
 * The attention weight that each prompt key received from the plan's query rows: for request b, kv head g and
 * key j of its prompt (a decode plan: j < P_b; a prefill plan: j < cached + prompt rows),
 *   weights[b][g][j] = sum over rows r of b and query heads h of g of exp(softmax_scale * q[r][h] . k[j] - lse[r][h])
 * with lse from the attention of the same rows (bsp_decode_attn: the whole sequence's, tail included; base 2
 * with BSP_FLAG_LSE_BASE2). A row with lse -inf adds nothing, whatever its q holds (padding; over finite keys). A
 * causal prefill's row adds to the keys it sees.
 *   window        a prefill plan: only the last `window` prompt rows of each request are summed (0: all);
 *                 a decode plan: 0
 *   flags         BSP_FLAG_LSE_BASE2, BSP_FLAG_CHECK, BSP_FLAG_ACCUMULATE (add to weights)
 *   weights       device fp32 [batch][num_kv_heads][weights_stride], weights_stride >= the plan's longest
 *                 prompt; entries past a request's keys (all entries of one without rows) stay as they were
 * One pass over K on the tensor cores; each sum is taken in one order, so repeated calls agree bit for bit.
 * The _fp8 form reads E4M3 pools with one scale per tensor (key = code * k_scale; head_dim 64 or 128, decode plans);
 * of pools with block scales it would read the codes alone.
 */
BSP_API bsp_status bsp_key_weights(const bsp_plan_t* plan, const void* q, const void* k_pool, const float* lse,
                                   float softmax_scale, int32_t window, int32_t flags, float* weights,
                                   int64_t weights_stride, void* stream);
BSP_API bsp_status bsp_key_weights_fp8(const bsp_plan_t* plan, const void* q, const void* k_pool, const float* lse,
                                       float softmax_scale, float k_scale, int32_t window, int32_t flags,
                                       float* weights, int64_t weights_stride, void* stream);

/*
 * Evicts prompt rows from the cache, per (request, kv head): the keep = clamp(keep_len[b], 0, P_b) slots of
 * largest weight stay, and those of them behind the first `keep` slots move, K and V, into the evicted slots
 * before them (the i-th evicted slot takes the i-th such row), within the request's own prompt pages and the
 * pools' element size. Attention does not depend on the order of its keys, so a plan with prompt length keep
 * over the first ceil(keep / page_size) of the same pages reads exactly the rows kept; the other pages are
 * free. Equal weights (-0 and +0 among them) go by the lower slot; a NaN counts below every number. Slots whose
 * position is < sinks or among the last `recent` (>= the highest position held + 1 - recent) rank above all
 * weights.
 *   plan           a decode plan without tail rows (they would follow the old length: BSP_ERR_INVALID_ARG) or
 *                  a prefill plan (a request without prompt rows is left as it is), whose requests share no
 *                  page with one another and hold none twice
 *   positions      device int32 [batch][num_kv_heads][weights_stride]: the slots' logical positions, or NULL:
 *                  the slot numbers (a cache that nothing was evicted from)
 *   keep_len       device int32 [batch]
 *   kept           device int32 [batch][num_kv_heads][out_stride] out: slot i < keep now holds the row that
 *                  was in slot kept[i]
 *   weights_out, positions_out   NULL, or [batch][num_kv_heads][out_stride]: the kept slots' weights and
 *                  positions (each may be its input when the strides agree)
 * Not for pools with block scales (bsp_block_scales): a row moved to another block would be read at that block's scale.
 * Entries of the outputs from `keep` on stay as they were. weights_stride, out_stride >= the longest prompt. A replay
 * that finds a page id past the pools it was captured with does not copy that row and sets BSP_DEVFLAG_PAGE_INDEX.
 */
BSP_API bsp_status bsp_evict_prefix(const bsp_plan_t* plan, const float* weights, int64_t weights_stride,
                                    const int32_t* positions, const int32_t* keep_len, int32_t sinks, int32_t recent,
                                    void* k_pool, void* v_pool, int32_t* kept, float* weights_out,
                                    int32_t* positions_out, int64_t out_stride, void* stream);

/* ------------------------------------------------------------------------------------------------------
 * Pages of the cache. (These entry points have no counterpart on the pages the method comes from.)
 *
 * What is known of a pool's pages is one count per page, device int32 refs[num_pages]: how many sequences hold it. A
 * page with a count of 0 is free. The calls take the plan for its geometry (num_pages, the page's heads, slots and
 * element type) and status word, and follow the conventions of the operators around a step; the tables' calls run once
 * for all layers, the rows' calls once per layer. Counts and tables need the alignment of their element. Where a call has
 * refs_in and refs_out, or tables_in and tables_out, the second may be the first (no other overlap). Free pages are
 * taken lowest id first and live pages keep their order, so repeated calls agree.
 */

#define BSP_MAX_PAGES (1 << 28)      /* pages of a pool, for these calls */
#define BSP_MAX_FORK_ROWS (1 << 20)  /* batch * num_forks of bsp_fork_tables and bsp_fork_rows */

/*
 * Beams that go on as sequences of their own. Row i = b * num_forks + j is the fork of beam w = beams[b][j] of request
 * b, with the L = P_b + T_b positions of the plan (a decode plan): its table is the full prompt pages, shared (the first
 * floor(P_b / page_size) of the plan's; each gains a reference per row), and then fresh pages up to
 * ceil(L / page_size) in all, the lowest free ones in the order of the rows, with a count of 1.
 * bsp_fork_rows writes what belongs there.
 *   beams          device int32 [batch] rows, beams_stride (>= num_forks) apart: beams in [0, beam_width), or -1: none
 *                  (others are taken as -1 and flagged as BSP_DEVFLAG_PAGE_INDEX). A beam may be forked several times
 *   refs_in, refs_out  the counts before and after
 *   pages_out      device int32 [batch * num_forks] rows of pages_out_cols (>= ceil(max L / page_size)) entries,
 *                  pages_out_stride apart: the first ceil(L / page_size) are written, the others stay as they were
 *   workspace      4-byte aligned device memory of bsp_fork_workspace_size bytes, contents not kept; calls whose GPU
 *                  work overlaps (two graphs too) need one each
 * A row without a beam gets -1 entries and no pages. When the free pages do not suffice, the rows from the first that
 * finds too few on get -1 entries and hold nothing, whatever they need, and BSP_DEVFLAG_PAGES is set.
 */
BSP_API bsp_status bsp_fork_workspace_size(int32_t batch, int32_t num_forks, size_t* device_bytes);
BSP_API bsp_status bsp_fork_tables(const bsp_plan_t* plan, const int32_t* beams, int64_t beams_stride, int32_t num_forks,
                                   const int32_t* refs_in, int32_t* refs_out, int32_t* pages_out,
                                   int64_t pages_out_stride, int32_t pages_out_cols, void* workspace,
                                   size_t workspace_bytes, void* stream);
/*
 * The rows of the forks' fresh pages, K and V: positions from floor(P_b / page_size) * page_size to P_b - 1 out of the
 * plan's prompt page, the tail's out of beam_pages[b * W + cache_indirection[b][w][pos]], as bsp_decode_attn reads them.
 * Rows whose table holds -1 are left out. The fresh pages' other slots keep what they held.
 *   beam_pages, cache_indirection  as bsp_decode_attn (both may be NULL for a plan without tails)
 *   scales         NULL, or the block scales of E4M3 pools: a block takes the largest exponent among those of the blocks
 *                  that its rows come from (as they are read), rows of a smaller one are brought to it (times a power of
 *                  two, rounded to nearest even), and blocks without rows are cleared
 */
BSP_API bsp_status bsp_fork_rows(const bsp_plan_t* plan, const int32_t* beams, int64_t beams_stride, int32_t num_forks,
                                 const int32_t* pages_out, int64_t pages_out_stride, int32_t pages_out_cols,
                                 const int32_t* beam_pages, int32_t beam_pages_stride,
                                 const int32_t* cache_indirection, int32_t max_seq, void* k_pool, void* v_pool,
                                 const bsp_block_scales* scales, void* stream);

/*
 * References given back: refs_out[p] = refs_in[p] less the number of times that page p stands in the tables. -1 entries
 * are passed over; an entry outside the pool, and one more reference given back than there are (the count stays 0),
 * set BSP_DEVFLAG_PAGE_INDEX.
 *   tables   device int32 [rows] rows of cols entries, stride (>= cols) apart
 */
BSP_API bsp_status bsp_free_pages(const bsp_plan_t* plan, const int32_t* tables, int64_t stride, int32_t rows,
                                  int32_t cols, const int32_t* refs_in, int32_t* refs_out, void* stream);

/*
 * Compaction: with L pages live, the i-th live page whose id is at least L takes the place of the i-th free page below
 * L, so that afterwards the pages 0 .. L - 1 are the live ones and the rest of the pool is free.
 *   pairs    device int32 [num_pages / 2][2] out: (from, to) of the pages that move, in ascending order
 *   count    device int32 [2] out: the number of pairs, and L
 *   remap    device int32 [num_pages] out: where each page is now
 *   tables_in, tables_out  device int32 [rows] rows of cols entries, stride apart: every live sequence's table, with the
 *            new ids in tables_out (-1 entries, and others outside the pool, which are flagged, as they are); NULL with
 *            rows = 0 (remap then serves to update what else names pages)
 * bsp_copy_pages moves the rows of each layer.
 */
BSP_API bsp_status bsp_compact_tables(const bsp_plan_t* plan, const int32_t* refs_in, int32_t* refs_out, int32_t* pairs,
                                      int32_t* count, int32_t* remap, const int32_t* tables_in, int32_t* tables_out,
                                      int64_t stride, int32_t rows, int32_t cols, void* stream);

/*
 * Whole pages copied, K and V (and their exponents with `scales`): page pairs[i][1] becomes a copy of pairs[i][0], for
 * i < min(count[0], max_pairs). No page is both a source and a target, or a target twice. A pair of -1 is passed over;
 * others outside the pool are skipped and flagged as BSP_DEVFLAG_PAGE_INDEX.
 *   pairs, count   device int32 [max_pairs][2], [1] (of bsp_compact_tables, or the caller's own)
 */
BSP_API bsp_status bsp_copy_pages(const bsp_plan_t* plan, const int32_t* pairs, const int32_t* count, int32_t max_pairs,
                                  void* k_pool, void* v_pool, const bsp_block_scales* scales, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BSP_H_ */
