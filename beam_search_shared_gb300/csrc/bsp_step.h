// Contract between the host entries of the operators around a step (bsp_step.cpp), their kernels, and the planner:
// the fields of a plan image's header and the launch parameter blocks. Apart from bsp_internal.h, which the attention
// kernels are built from.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/bsp.h"
#include "bsp_internal.h"

namespace bsp {

// Image header: u64 generation, then int32 fields.
// kHdrRows: query rows of the plan; kHdrPages: bytes from the image's start to the page table; the heads, page
// size and head_dim the plan was made for.
enum HeaderField { kHdrBatch = 2, kHdrUnits = 3, kHdrWidth = 4, kHdrSms = 5, kHdrKind = 6, kHdrMaxTail = 7, kHdrRows = 8,
                   kHdrPages = 9, kHdrQHeads = 10, kHdrKvHeads = 11, kHdrPageSize = 12, kHdrHeadDim = 13 };

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
constexpr int kWeightsBarBytes = 512;
constexpr int kWeightsTableBytes = (8 * 128 + 4 * 128) * 4;  // -lse and partial sums
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

}  // namespace bsp
