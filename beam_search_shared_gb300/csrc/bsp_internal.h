// Internal contract between the host library (bsp_host.cpp) and the kernels:
// the staged plan image layout and the launch parameter blocks.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/bsp.h"

namespace bsp {

// Prompt-attention tiling.
constexpr int kTileKeys = 64;      // keys per prompt tile (MMA N of Q*K^T, MMA K of P*V)
constexpr int kRowsPerBlock = 128; // query rows per CTA (MMA M)
constexpr int kExtraParts = 64;    // key splits beyond one per request the workspace holds

// Device workspace: [status words | plan image | partial LSE | partial O].
constexpr size_t kStatusBytes = 256;
constexpr size_t kAlign = 256;

// Plan image (int32 fields, offsets relative to the image start).
constexpr int kImageHeaderBytes = 64;  // u64 generation, then int32 fields:
// kHdrRows: query rows of the plan; kHdrPages: bytes from the image's start to the page table; the heads, page
// size and head_dim the plan was made for.
enum HeaderField { kHdrBatch = 2, kHdrUnits = 3, kHdrWidth = 4, kHdrSms = 5, kHdrKind = 6, kHdrMaxTail = 7, kHdrRows = 8,
                   kHdrPages = 9, kHdrQHeads = 10, kHdrKvHeads = 11, kHdrPageSize = 12, kHdrHeadDim = 13 };
// Per-request record.
// kReqFused: the prompt kernel finishes the request (one prompt partial state, and every unit's tail keys
// fit the prompt kernel's tail tiles); the tail kernel skips it.
// kReqRows: the request's query rows per (kv head, head in group) - beams for a decode step, prompt
// tokens for a prefill; kReqRowOff: its first row of q / o (b * W, or the tokens of earlier requests);
// kReqCausal: -1, or the cached rows C of a causal prefill (row t sees keys 0 .. C + t).
enum ReqField { kReqPrefix = 0, kReqTail = 1, kReqSplits = 2, kReqPartOff = 3, kReqPageOff = 4, kReqFused = 5,
                kReqRows = 8, kReqCausal = 9, kReqRowOff = 10, kReqFields = 12 };
// keys per tile of the prompt kernel, which bounds a row block's tail keys for the fused tail
constexpr int prefix_tile_keys(int head_dim) { return head_dim <= 128 ? 128 : 64; }
// tail tiles of prefix_tile_keys(head_dim) keys the one-set prompt kernel may gather for a unit (the
// request is finished by the tail kernel beyond)
constexpr int kPrefixMaxTailTiles = 4;
// Beams per TMEM lane quadrant when the prompt kernel places a row block's query rows in lanes
// 0-15 of each quadrant and gives each row two softmax threads (half of the keys each): the
// block's beams spread over the four quadrants, at most 16 rows each, with 128-key tiles. 0 when
// the block does not fit that way (the rows then fill the lanes densely, one thread per row).
constexpr int prefix_quad_beams(int head_dim, int beams_per_block, int group) {
    const int bq = (beams_per_block + 3) / 4;
    return (prefix_tile_keys(head_dim) == 128 && bq * group <= 16) ? bq : 0;
}
// The wide layout of a decode step (bsp_wide.cu): when a (request, kv head) has more query rows than
// one MMA holds (W * G in (128, 256]) at head_dim <= 128, one unit holds all of them as two M = 128
// blocks (beams [0, Wb) and [Wb, W), Wb = ceil(W / 2)) that share every K/V tile, so the prompt is read
// once. Each block's beams spread over the four TMEM lane quadrants, bq = ceil(Wb / 4) beams (bq * G
// rows) per quadrant. 0 when the beams do not fit that way.
constexpr int wide_quad_beams(int head_dim, int beam_width, int group) {
    const int wb = (beam_width + 1) / 2;
    const int bq = (wb + 3) / 4;
    return (head_dim <= 128 && beam_width * group > kRowsPerBlock && beam_width * group <= 2 * kRowsPerBlock &&
            bq * group <= 32)
               ? bq
               : 0;
}
// tail tiles of 128 keys a wide unit may gather (the request is finished by the tail kernel beyond)
constexpr int kWideMaxTailTiles = 4;
// The alternating-tile layout of a decode step (bsp_alt.cu), at head_dim <= 128: a unit is one query-row
// block (W_blk beams x G heads <= 128 rows) whose key tiles go alternately to two softmax warp sets;
// the block's beams spread over the four TMEM lane quadrants, bq = ceil(W_blk / 4) beams (bq * G rows)
// per quadrant. 0 when the beams do not fit that way.
constexpr int alt_quad_beams(int head_dim, int beams_per_block, int group) {
    const int bq = (beams_per_block + 3) / 4;
    return (head_dim <= 128 && beams_per_block * group <= kRowsPerBlock && bq * group <= 32) ? bq : 0;
}
// tail tiles of 128 keys an alternating-tile unit may gather (the request is finished by the tail
// kernel beyond)
constexpr int kAltMaxTailTiles = 4;
// Per-work-unit record: request, kv head, query-row block, key tiles [kt0, kt1), partial slot, and
// the cost the host dealt it by (eighths of a prompt-kernel key tile; not read by the kernels).
enum UnitField { kUnitReq = 0, kUnitKvHead = 1, kUnitRowBlock = 2, kUnitTile0 = 3, kUnitTile1 = 4, kUnitPart = 5,
                 kUnitCost = 6, kUnitFields = 8 };

struct PrefixParams {
    // fused requests: tail keys gathered by the prompt kernel, final O / LSE written by it
    const void* k_pool;
    const void* v_pool;
    const int32_t* beam_pages;
    const int32_t* ci;
    void* o;
    float* lse;
    int beam_pages_stride, max_seq, lse_base2;
    const int32_t* units;    // [num_units][kUnitFields], grouped by CTA
    const int32_t* cta_off;  // [gridDim.x + 1]: CTA c runs units cta_off[c] .. cta_off[c+1]-1
    const int32_t* req;
    const int32_t* pages;
    float* part_o;    // [part][W][Hq][D]   (normalised partial output)
    float* part_lse;  // [part][W][Hq]      (log2-sum-exp2 of the scaled scores)
    int32_t* status;
    int W, Hq, Hkv, G, ps_log2, Wblk, num_pages;
    int bq;            // > 0: half-row softmax, bq beams of the block per TMEM lane quadrant (prefix_quad_beams)
    int num_units;     // units in the list
    float v_scale;     // E4M3 pools: the values' per-tensor scale, applied to O (1 for 16-bit pools)
    // graph mode (else null): the staged plan's header, checked at the start against the launch
    // (batch, beam width, one CTA per SM of the plan, a decode plan)
    const int32_t* graph_hdr;
    int graph_batch;
    float scale_log2;  // softmax_scale * log2(e)
};

struct TailParams {
    const void* q;
    const void* k_pool;
    const void* v_pool;
    const int32_t* beam_pages;
    const int32_t* ci;
    const int32_t* req;
    const float* part_o;
    const float* part_lse;
    void* o;
    float* lse;
    int32_t* status;
    int B, W, Hq, Hkv, G, ps_log2, num_pages, beam_pages_stride, max_seq;
    float scale_log2;
    int lse_base2;
    float v_scale;     // E4M3 pools: the values' per-tensor scale, applied to the tail's O (1 otherwise)
    // graph mode (else null): the staged plan's header, checked against the launch (batch, beam width,
    // a decode plan, a tail bound within the one the launch was made for)
    const int32_t* graph_hdr;
    int graph_max_tail;
};

struct AppendParams {
    const void* k_new;
    const void* v_new;
    int64_t src_row_stride;  // elements
    const int32_t* loc;
    void* k_pool;
    void* v_pool;
    int32_t* status;
    int n, Hkv, D, ps_log2, num_pages;
};

cudaError_t launch_prefix(int head_dim, bool bf16, int ctas, const CUtensorMap& tq, const CUtensorMap& tk,
                          const CUtensorMap& tv, const PrefixParams& p, cudaStream_t stream);
// Kernel attributes (shared-memory size and split) are set by the prepare_* calls, once before
// the launches, so that timing events recorded around a launch bracket the launch alone.
cudaError_t prepare_prefix(int head_dim, bool bf16);
cudaError_t prepare_tail(int head_dim, bool bf16, int max_tail_len, int num_q_heads, bool fp8 = false);
// after_prefix: the prompt kernel was the last launch on `stream`; the tail kernel is then a
// programmatic dependent launch of it (it starts on SMs the prompt kernel has left, resolves and
// prefetches its tail rows, and waits for the prompt kernel's partials before merging).
cudaError_t launch_tail(int head_dim, bool bf16, int max_tail_len, const TailParams& p, bool after_prefix,
                        cudaStream_t stream, bool fp8 = false);
// The alternating-tile prompt kernel (p.Wblk = beams per row block, p.bq = beams per quadrant). fp8: E4M3
// pools (tk, tv map one-byte elements without swizzle, boxes of min(page, 64) rows x head_dim bytes).
cudaError_t prepare_alt(int head_dim, bool bf16, bool fp8 = false);
cudaError_t launch_alt(int head_dim, bool bf16, int ctas, const CUtensorMap& tq, const CUtensorMap& tk,
                       const CUtensorMap& tv, const PrefixParams& p, cudaStream_t stream, bool fp8 = false);
// The wide-layout prompt kernel (p.Wblk = beams per block, p.bq = beams per quadrant); fp8 as above.
cudaError_t prepare_wide(int head_dim, bool bf16, bool fp8 = false);
cudaError_t launch_wide(int head_dim, bool bf16, int ctas, const CUtensorMap& tq, const CUtensorMap& tk,
                        const CUtensorMap& tv, const PrefixParams& p, cudaStream_t stream, bool fp8 = false);
// ---------------------------------------------------------------- the operators around a step (bsp_step.cpp)

// The plan a launch was made for, as far as what the launch fixes (addresses in the image, tensor maps, sizes of its
// other tensors) depends on it.
struct PlanShape {
    int32_t gen[2];  // of a prefill plan
    int32_t batch, w, kind, rows, pages_at, q_heads, kv_heads, page_size, head_dim;
};

// Whether the plan staged now is one the launch may follow: a launch replayed from a CUDA graph reads the lengths and
// pages of the latest plan. hdr: its image's header.
#ifdef __CUDACC__
// For the requests' records alone, which stand at the same place in every image.
__device__ __forceinline__ bool plan_matches(const int32_t* hdr, int batch, int w, int kind) {
    return __ldg(hdr + kHdrBatch) == batch && __ldg(hdr + kHdrWidth) == w && __ldg(hdr + kHdrKind) == kind;
}
// For the page table, q and lse too. A decode plan's image has one layout for its batch, beam width and geometry. A
// prefill plan's is packed and its rows are the prompts' tokens: only the very plan of the launch will do.
__device__ __forceinline__ bool plan_matches(const int32_t* hdr, const PlanShape& s) {
    const int4* h = reinterpret_cast<const int4*>(hdr);
    const int4 a = __ldg(h), b = __ldg(h + 1), c = __ldg(h + 2), d = __ldg(h + 3);
    static_assert(kHdrBatch == 2 && kHdrWidth == 4 && kHdrKind == 6 && kHdrRows == 8 && kHdrPages == 9 && kHdrQHeads == 10 &&
                      kHdrKvHeads == 11 && kHdrPageSize == 12 && kHdrHeadDim == 13, "the fields read as vectors");
    return a.z == s.batch && b.x == s.w && b.z == s.kind && c.x == s.rows && c.y == s.pages_at && c.z == s.q_heads &&
           c.w == s.kv_heads && d.x == s.page_size && d.y == s.head_dim &&
           (s.kind == 0 || (a.x == s.gen[0] && a.y == s.gen[1]));
}
#endif

constexpr size_t kMaxSmem = 227 * 1024;  // shared memory of a CTA, static and dynamic

// Lets a kernel of at most 16 KB of static shared memory have `smem` bytes of dynamic; within the 48 KB that every
// kernel has, the call is saved (0.5 us of a launch's host time). The limit belongs to the function, not to the launch:
// it is set to `most`, the most that any call of the kernel asks for, so that threads whose calls differ in size set the
// same value and none lowers it between another's setting and launch.
inline cudaError_t allow_smem(const void* kernel, size_t smem, size_t most) {
    if (smem <= 32 * 1024) return cudaSuccess;
    if (smem > most) return cudaErrorInvalidValue;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
}

struct TokenMask {
    const uint32_t* bits;  // [rows][stride]: bit t of a row: token t is allowed; null: no masks
    long long stride;      // words
    const int32_t* index;  // [query rows]: row of `bits`, -1: none
    int rows;
};

struct ProcessParams {
    const void* x;
    void* out;
    long long x_stride, out_stride;  // elements
    float* lse;
    const int32_t* prompt_tokens;
    const int32_t* prompt_len;
    const int32_t* tokens;
    const int32_t* token_len;
    const int32_t* bias_tokens;
    const float* bias_values;
    const int32_t* bias_len;
    long long prompt_stride, token_stride, bias_stride;
    const float *repetition, *frequency, *presence, *temperature;
    TokenMask mask;
    int32_t* status;
    int vocab, W, rows, prompt_cols, token_cols, bias_cols;
    int hot_at, mask_at, table_at;  // words before the bitmaps of named and of allowed tokens, and before the table
    int hash_slots;    // slots of the table of counts and biases (a power of two), 0: none
};
constexpr int kProcessSlotBytes = 12;
constexpr size_t kProcessSmem = kMaxSmem - 16 * 1024;  // dynamic, beside the kernel's own
cudaError_t launch_process(int dtype, const ProcessParams& p, int cluster, size_t smem, cudaStream_t stream);

struct SelectParams {
    const void* x;
    long long x_stride;  // elements
    const float* lse;
    const float* cum;
    long long cum_stride;
    TokenMask mask;
    uint64_t* part_keys;   // [ctas + batch][K]: the list of (scanning CTA, request) at their sum
    uint64_t* part_head;   // [ctas + batch][2]: its length, and a bound below the request's best K or 0
    float* scores;
    int32_t* parents;
    int32_t* tokens;
    int32_t* status;
    int batch, W, vocab, K;
    int ctas;      // scanning CTAs
    int segments;  // scanning units of a row
    int cap;       // keys of a scanning CTA's buffer
};
constexpr int64_t kMergeKeys = 16384;  // candidates one merging CTA holds (128 KB of its shared memory)
int select_unit_elems(int dtype, bool masked);
int select_unit_warps();
int select_sm_ctas(bool masked);
int select_buffer(int K);
cudaError_t launch_select(int dtype, const SelectParams& p, int most_lists, cudaStream_t stream);

struct AdvanceParams {
    const int32_t* req;
    const int32_t* plan_hdr;
    const int32_t* parents;
    const int32_t* chosen;
    long long cand_stride;
    const int32_t* ci_in;
    int32_t* ci_out;
    const int32_t* tok_in;
    int32_t* tok_out;
    int32_t* token_len;
    int32_t* status;
    long long tok_stride;
    int batch, W, max_seq, tok_cols;
    int cols;  // tail columns of both tables staged at a time
};
constexpr size_t kAdvanceSmem = 160 * 1024;
cudaError_t launch_advance(const AdvanceParams& p, cudaStream_t stream);

struct WeightsParams {
    const void* q;
    const int32_t* req;
    const int32_t* pages;
    const int32_t* plan_hdr;
    const float* lse;
    float* weights;
    long long stride;
    int32_t* status;
    PlanShape shape;
    int batch, Hq, Hkv, G, ps_log2, num_pages, max_keys, window, accumulate;
    int block_rows;  // beams (prompt tokens) of a Q block
    int mma_n;       // its rows for the MMA: block_rows * G rounded up to 16
    int q_slots, k_slots;
    float scale_log2, lse_mul;
};
constexpr int kWeightsBarBytes = 384;
constexpr int kWeightsTableBytes = (8 * 132 + 4 * 128) * 4;  // -lse and partial sums
// Before the tensor maps: their encoder needs a current context, and on a host thread that has made no CUDA call yet
// the kernel's attribute is the first call to make one so.
cudaError_t prepare_weights(int head_dim, bool bf16, bool fp8);
cudaError_t launch_weights(int head_dim, bool bf16, bool fp8, const CUtensorMap& tq, const CUtensorMap& tk,
                           const WeightsParams& p, int ctas, size_t smem, cudaStream_t stream);

struct EvictParams {
    const int32_t* req;
    const int32_t* pages;
    const int32_t* plan_hdr;
    const float* weights;
    const int32_t* positions;
    const int32_t* keep;
    uint8_t* k_pool;
    uint8_t* v_pool;
    int32_t* kept;
    float* weights_out;
    int32_t* positions_out;
    long long stride, out_stride;
    int32_t* status;
    PlanShape shape;
    int batch, Hkv, num_pages, ps_log2, row_bytes, max_keys, sinks, recent;
    int cached_keys, cluster;  // set by launch_evict
};
// longest: the plan's longest prompt
cudaError_t launch_evict(EvictParams p, int longest, int num_sms, cudaStream_t stream);

// bsp_host.cpp, for bsp_step.cpp
bsp_status check_plan(const bsp_plan_t* plan);
bool encode_map(CUtensorMap* m, int dtype, int rank, const void* base, const cuuint64_t* dims,
                const cuuint64_t* strides_bytes, const cuuint32_t* box, bool e4m3 = false);

cudaError_t prepare_append();
cudaError_t launch_append(const AppendParams& p, cudaStream_t stream);

// bsp_host.cpp: the attention of a plan whose status word, image and partial states sit at `ws`
// (the caller's workspace, or the fixed scratch of the no-allocation entry point). attn_check_args
// checks what the host can check and enqueues nothing; attn_launches enqueues the launches.
// fp8: the caller is the E4M3 entry point (the plan's pools must then be E4M3, and 16-bit otherwise);
// k_scale and v_scale are the E4M3 pools' per-tensor scales (1 for 16-bit pools).
bsp_status attn_check_args(const bsp_plan_t* plan, const void* q, const void* k_pool, const void* v_pool,
                           const int32_t* beam_pages, int32_t beam_pages_stride, const int32_t* cache_indirection,
                           int32_t max_seq, float softmax_scale, int32_t flags, void* o, float* lse, bool prefill,
                           bool fp8 = false, float k_scale = 1.f, float v_scale = 1.f);
bsp_status attn_launches(const bsp_plan_t* plan, uint8_t* ws, const void* q, const void* k_pool, const void* v_pool,
                         const int32_t* beam_pages, int32_t beam_pages_stride, const int32_t* cache_indirection,
                         int32_t max_seq, float softmax_scale, int32_t flags, void* o, float* lse,
                         void* const* events, cudaStream_t s, bool prefill, float k_scale = 1.f, float v_scale = 1.f);
// A decode plan with the packed layout (sections and partial states sized by the plan's own units and
// splits), for a caller that never replays it from a CUDA graph.
bsp_status plan_build_packed(const bsp_geometry* geo, int32_t batch, int32_t beam_width, const int32_t* prefix_len,
                             const int32_t* tail_len, const int32_t* prefix_pages, int32_t prefix_pages_stride,
                             int32_t max_tail, int32_t num_sms, void* image, size_t image_bytes, bsp_plan_t* out);

}  // namespace bsp
