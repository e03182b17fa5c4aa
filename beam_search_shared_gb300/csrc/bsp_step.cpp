// Host side of the operators around a beam step: argument validation and launches of the logits'
// processing, the choice of the beams, their bookkeeping, the keys' attention weights and the eviction of
// cached rows. Declared in include/bsp.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/bsp.h"
#include "bsp_check.h"
#include "bsp_step.h"

namespace {

using namespace bsp;

int logits_bytes(int dtype) { return dtype == BSP_LOGITS_FP32 ? 4 : 2; }

// The decode plan, logits type, vocabulary and row stride that the logits' calls share.
bsp_status check_logits(const bsp_plan_t* plan, int32_t dtype, int32_t vocab, int64_t stride) {
    bsp_status st = check_plan(plan);
    if (st != BSP_OK) return st;
    if (plan->kind != 0) return BSP_ERR_INVALID_ARG;
    if (dtype != BSP_LOGITS_BF16 && dtype != BSP_LOGITS_FP16 && dtype != BSP_LOGITS_FP32) return BSP_ERR_UNSUPPORTED;
    if (vocab < 1 || stride < vocab) return BSP_ERR_INVALID_ARG;
    if (vocab > BSP_MAX_VOCAB) return BSP_ERR_UNSUPPORTED;
    return BSP_OK;
}

bsp_status check_mask(const bsp_token_mask* m, int32_t vocab, TokenMask* out) {
    *out = TokenMask{nullptr, 0, nullptr, 0};
    if (!m || !m->bits) return BSP_OK;
    if (m->rows < 1 || m->stride < ceil_div(vocab, 32)) return BSP_ERR_INVALID_ARG;
    if (!device_ptr(m->bits, 4) || !device_ptr(m->index, 4)) return BSP_ERR_INVALID_ARG;
    *out = TokenMask{m->bits, m->stride, m->index, m->rows};
    return BSP_OK;
}

// How a selection is cut: units of a row, scanning CTAs, and the most CTAs that meet one request.
struct SelectSplit {
    int segments, ctas, lists;
};
SelectSplit select_split(int batch, int W, int vocab, int K, int dtype, bool masked, int sms) {
    SelectSplit s;
    s.segments = static_cast<int>(ceil_div(vocab, select_unit_elems(dtype, masked)));
    const int64_t requests = std::max(1, batch), warps = select_unit_warps();
    const int64_t u = static_cast<int64_t>(W) * s.segments;  // units of a request
    const int64_t most = static_cast<int64_t>(select_sm_ctas(masked)) * sms;
    // a request's lists fit its merging CTA (an even cut of n CTAs over the batch gives a request at most
    // ceil(n / requests) + 1 of them)
    const int64_t room = std::max<int64_t>(1, kMergeKeys / K - 1);
    // Few units: n CTAs for a request take about 3 us for each of a warp's ceil(u / 8n) units and 0.8 ns for each of
    // the merge's n K keys, which is least near n^2 = 468 u / K; then as few as do with the same units per warp, and no
    // CTA between two requests (1 x 30 rows of 128000, K = 60: 237 CTAs of 8 units 30.5 us, 118 of 16 25.5, 86 of 22
    // 30.1, 59 of 32 27.3; 8 x 30 of 32000: 30 a request 23, 38 a request 29.5). Many, from 8 a warp on: all that are
    // resident, on an even cut of the whole batch.
    const int64_t best = static_cast<int64_t>(std::sqrt(468.0 * static_cast<double>(u) / K)) + 1;
    const int64_t n = std::max<int64_t>(1, std::min({best, room, most / requests, ceil_div(u, warps)}));
    const int64_t each = ceil_div(u, warps * n);  // units of a warp
    s.ctas = static_cast<int>(each < 8 ? requests * ceil_div(u, warps * each) : std::min(most, room * requests));
    s.lists = static_cast<int>(ceil_div(s.ctas, requests) + 1);
    return s;
}

bool device_sms(int* sms) {
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess &&
           cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess;
}

}  // namespace

extern "C" {

bsp_status bsp_process_logits(const bsp_plan_t* plan, const void* logits, int32_t logits_dtype, int64_t logits_stride,
                              int32_t vocab, const bsp_logits_params* params, void* out, int64_t out_stride, float* lse,
                              void* stream) {
    bsp_status st = check_logits(plan, logits_dtype, vocab, logits_stride);
    if (st != BSP_OK) return st;
    if (!params || out_stride < vocab) return BSP_ERR_INVALID_ARG;
    const int es = logits_bytes(logits_dtype);
    const bsp_logits_params& q = *params;
    ProcessParams p{};
    p.rows = plan->total_rows;
    if (p.rows == 0) return BSP_OK;
    if (!plan_here(plan)) return BSP_ERR_INVALID_ARG;
    if (!device_ptr(logits, es) || !device_ptr(out, es) || !optional_ptr(lse, 4)) return BSP_ERR_INVALID_ARG;
    if (out == logits && out_stride != logits_stride) return BSP_ERR_INVALID_ARG;
    if (out != logits) {
        // rows of the output may not overlap logits that are still to be read
        const uint8_t* a = static_cast<const uint8_t*>(logits);
        const uint8_t* c = static_cast<const uint8_t*>(out);
        const int64_t na = ((p.rows - 1) * logits_stride + vocab) * es, nc = ((p.rows - 1) * out_stride + vocab) * es;
        if (a < c + nc && c < a + na) return BSP_ERR_INVALID_ARG;
    }
    const bool lists = q.repetition_penalty || q.frequency_penalty || q.presence_penalty;
    const bool counts = q.frequency_penalty || q.presence_penalty;
    if (q.prompt_tokens) {
        if (q.prompt_cols < 0 || q.prompt_stride < q.prompt_cols) return BSP_ERR_INVALID_ARG;
        if (!device_ptr(q.prompt_tokens, 4) || !device_ptr(q.prompt_len, 4)) return BSP_ERR_INVALID_ARG;
    }
    if (q.tokens) {
        if (q.token_cols < 0 || q.token_stride < q.token_cols) return BSP_ERR_INVALID_ARG;
        if (!device_ptr(q.tokens, 4) || !device_ptr(q.token_len, 4)) return BSP_ERR_INVALID_ARG;
    }
    if (q.bias_tokens) {
        if (q.bias_cols < 0 || q.bias_stride < q.bias_cols) return BSP_ERR_INVALID_ARG;
        if (!device_ptr(q.bias_tokens, 4) || !device_ptr(q.bias_values, 4) || !optional_ptr(q.bias_len, 4))
            return BSP_ERR_INVALID_ARG;
    }
    if (!optional_ptr(q.repetition_penalty, 4) || !optional_ptr(q.frequency_penalty, 4) ||
        !optional_ptr(q.presence_penalty, 4) || !optional_ptr(q.temperature, 4))
        return BSP_ERR_INVALID_ARG;
    st = check_mask(&q.mask, vocab, &p.mask);
    if (st != BSP_OK) return st;
    p.x = logits;
    p.out = out;
    p.x_stride = logits_stride;
    p.out_stride = out_stride;
    p.lse = lse;
    if (lists && q.prompt_tokens && q.prompt_cols > 0) {
        p.prompt_tokens = q.prompt_tokens;
        p.prompt_len = q.prompt_len;
        p.prompt_stride = q.prompt_stride;
        p.prompt_cols = q.prompt_cols;
    }
    if (lists && q.tokens && q.token_cols > 0) {
        p.tokens = q.tokens;
        p.token_len = q.token_len;
        p.token_stride = q.token_stride;
        p.token_cols = q.token_cols;
    }
    if (q.bias_tokens && q.bias_cols > 0) {
        p.bias_tokens = q.bias_tokens;
        p.bias_values = q.bias_values;
        p.bias_len = q.bias_len;
        p.bias_stride = q.bias_stride;
        p.bias_cols = q.bias_cols;
    }
    p.repetition = q.repetition_penalty;
    p.frequency = q.frequency_penalty;
    p.presence = q.presence_penalty;
    p.temperature = q.temperature;
    p.status = status_word(plan);
    p.vocab = vocab;
    p.W = plan->beam_width;
    const int64_t named = (counts ? p.token_cols : 0) + static_cast<int64_t>(p.bias_cols);
    if (named > BSP_MAX_LISTED) return BSP_ERR_UNSUPPORTED;
    p.hash_slots = named ? std::max(4, 1 << ilog2(static_cast<int>(2 * named))) : 0;

    // A cluster per row, its CTAs slices of the vocabulary. Few rows are cut while the CTAs are all resident at
    // once (four per SM) and a slice keeps 4 KB: 4 rows of 256 KB 55 us whole, 31 / 18 / 12 in 2 / 4 / 8; 240 rows
    // of 64 KB 16.7 whole, 14.9 / 19.5 in 2 / 4. Rows beyond that stay whole (960 rows of 256 KB 121, in two 126;
    // 1920 of 64 KB 78 and 90), unless the bitmaps of a slice would leave fewer than four CTAs to an SM
    // (3840 rows of 512 KB: 1028 whole, 751 in two, 814 in four).
    int cluster = 1;
    const int64_t row_bytes = static_cast<int64_t>(vocab) * es;
    while (cluster < 8 && static_cast<int64_t>(p.rows) * cluster * 2 <= 4 * plan->num_sms && row_bytes / (2 * cluster) >= 4096)
        cluster *= 2;
    size_t smem = 0;
    for (;; cluster *= 2) {
        // bitmaps of a slice: penalised tokens, tokens in the table, allowed tokens; each as far as it is needed
        const int words = static_cast<int>(((ceil_div(vocab, cluster) + 48) / 32 + 2 + 3) / 4 * 4);
        p.hot_at = q.repetition_penalty && (p.prompt_tokens || p.tokens) ? words : 0;
        p.mask_at = p.hot_at + (p.hash_slots ? words : 0);
        p.table_at = p.mask_at + (p.mask.bits ? words : 0);
        smem = static_cast<size_t>(p.table_at) * 4 + static_cast<size_t>(p.hash_slots) * kProcessSlotBytes;
        if (smem <= 40 * 1024) break;  // (with the kernel's own 16 KB, four times in an SM)
        if (cluster == 8) {
            if (smem > kProcessSmem) {
                // More than 4096 named tokens beside the bitmaps of a large vocabulary: a table that they may fill, with
                // longer walks to a slot (V = 2^21, all 8192 in one slice).
                p.hash_slots = 1 << ilog2(static_cast<int>(named));
                smem = static_cast<size_t>(p.table_at) * 4 + static_cast<size_t>(p.hash_slots) * kProcessSlotBytes;
                static_assert(3 * ((BSP_MAX_VOCAB / 8 + 48) / 32 + 8) * 4 + BSP_MAX_LISTED * kProcessSlotBytes <= kProcessSmem &&
                                  (BSP_MAX_LISTED & (BSP_MAX_LISTED - 1)) == 0,
                              "the largest vocabulary with the longest lists");
            }
            break;
        }
    }
    return launched(launch_process(logits_dtype, p, cluster, smem, static_cast<cudaStream_t>(stream)));
}

bsp_status bsp_beam_select_workspace_size(int32_t batch, int32_t beam_width, int32_t vocab, int32_t num_candidates,
                                          size_t* device_bytes) {
    if (!device_bytes || batch < 0 || beam_width < 1 || vocab < 1 || num_candidates < 1) return BSP_ERR_INVALID_ARG;
    if (vocab > BSP_MAX_VOCAB || num_candidates > BSP_MAX_CANDIDATES) return BSP_ERR_UNSUPPORTED;
    // No cut has more CTAs than one per request, or than are resident (up to 512 SMs), fit the merge and have a unit
    // for every warp: of the smallest units, fp32 under masks.
    const int64_t requests = std::max(1, batch), warps = select_unit_warps();
    const int64_t u = static_cast<int64_t>(beam_width) * ceil_div(vocab, select_unit_elems(BSP_LOGITS_FP32, true));
    const int64_t room = std::max<int64_t>(1, kMergeKeys / num_candidates - 1);
    const int64_t ctas = std::max(requests, std::min({int64_t(select_sm_ctas(true)) * 512, room * requests, requests * ceil_div(u, warps)}));
    const int64_t lists = ctas + batch;
    *device_bytes = static_cast<size_t>(lists) * (static_cast<size_t>(num_candidates) + 2) * 8;
    return BSP_OK;
}

bsp_status bsp_beam_select(const bsp_plan_t* plan, const void* logits, int32_t logits_dtype, int64_t logits_stride,
                           int32_t vocab, const float* lse, const float* cum_scores, int64_t cum_stride,
                           const bsp_token_mask* mask, int32_t num_candidates, float* scores, int32_t* parents,
                           int32_t* tokens, void* workspace, size_t workspace_bytes, void* stream) {
    bsp_status st = check_logits(plan, logits_dtype, vocab, logits_stride);
    if (st != BSP_OK) return st;
    if (num_candidates < 1 || cum_stride < plan->beam_width) return BSP_ERR_INVALID_ARG;
    if (num_candidates > BSP_MAX_CANDIDATES) return BSP_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(plan->beam_width) * vocab > (int64_t(1) << 32) - 1) return BSP_ERR_UNSUPPORTED;
    if (plan->batch > BSP_MAX_STEP_BATCH) return BSP_ERR_UNSUPPORTED;
    if (plan->total_rows == 0) return BSP_OK;
    if (!plan_here(plan)) return BSP_ERR_INVALID_ARG;
    const int es = logits_bytes(logits_dtype);
    if (!device_ptr(logits, es) || !device_ptr(lse, 4) || !device_ptr(cum_scores, 4) || !device_ptr(scores, 4) ||
        !device_ptr(parents, 4) || !device_ptr(tokens, 4) || !device_ptr(workspace, 16))
        return BSP_ERR_INVALID_ARG;
    SelectParams p{};
    st = check_mask(mask, vocab, &p.mask);
    if (st != BSP_OK) return st;
    int sms = 0;
    if (!device_sms(&sms)) return BSP_ERR_CUDA;
    const SelectSplit s = select_split(plan->batch, plan->beam_width, vocab, num_candidates, logits_dtype, p.mask.bits != nullptr, std::min(sms, 512));
    if (static_cast<int64_t>(plan->beam_width) * s.segments > (int64_t(1) << 30)) return BSP_ERR_UNSUPPORTED;
    const int64_t lists = static_cast<int64_t>(s.ctas) + plan->batch;
    if (static_cast<size_t>(lists) * (static_cast<size_t>(num_candidates) + 2) * 8 > workspace_bytes) return BSP_ERR_CAPACITY;
    p.x = logits;
    p.x_stride = logits_stride;
    p.lse = lse;
    p.cum = cum_scores;
    p.cum_stride = cum_stride;
    p.part_keys = static_cast<uint64_t*>(workspace);
    p.part_head = p.part_keys + lists * num_candidates;
    p.scores = scores;
    p.parents = parents;
    p.tokens = tokens;
    p.status = status_word(plan);
    p.batch = plan->batch;
    p.W = plan->beam_width;
    p.vocab = vocab;
    p.K = num_candidates;
    p.ctas = s.ctas;
    p.segments = s.segments;
    p.cap = select_buffer(num_candidates);
    return launched(launch_select(logits_dtype, p, s.lists, static_cast<cudaStream_t>(stream)));
}

bsp_status bsp_beam_advance(const bsp_plan_t* plan, const int32_t* parents, const int32_t* chosen, int64_t cand_stride,
                            const int32_t* ci_in, int32_t* ci_out, int32_t max_seq, const int32_t* tokens_in,
                            int32_t* tokens_out, int64_t token_stride, int32_t token_cols, int32_t* token_len,
                            void* stream) {
    bsp_status st = check_plan(plan);
    if (st != BSP_OK) return st;
    if (plan->kind != 0 || cand_stride < plan->beam_width) return BSP_ERR_INVALID_ARG;
    if ((ci_in == nullptr) != (ci_out == nullptr) || (tokens_in == nullptr) != (tokens_out == nullptr))
        return BSP_ERR_INVALID_ARG;
    if (plan->beam_width > BSP_MAX_ADVANCE_BEAMS) return BSP_ERR_UNSUPPORTED;
    if (plan->total_rows == 0) return BSP_OK;
    if (!plan_here(plan)) return BSP_ERR_INVALID_ARG;
    if (!device_ptr(parents, 4) || !device_ptr(chosen, 4) || !optional_ptr(ci_in, 4) || !optional_ptr(ci_out, 4) ||
        !optional_ptr(tokens_in, 4) || !optional_ptr(tokens_out, 4) || !optional_ptr(token_len, 4))
        return BSP_ERR_INVALID_ARG;
    if (ci_in && max_seq <= plan->max_total_len) return BSP_ERR_INVALID_ARG;
    if (tokens_in && (token_cols <= plan->max_tail_len || token_stride < token_cols)) return BSP_ERR_INVALID_ARG;
    AdvanceParams p{};
    p.req = section(plan, plan->off_req);
    p.plan_hdr = image_header(plan);
    p.parents = parents;
    p.chosen = chosen;
    p.cand_stride = cand_stride;
    p.ci_in = ci_in;
    p.ci_out = ci_out;
    p.tok_in = tokens_in;
    p.tok_out = tokens_out;
    p.token_len = token_len;
    p.status = status_word(plan);
    p.batch = plan->batch;
    p.W = plan->beam_width;
    p.max_seq = max_seq;
    p.tok_stride = token_stride;
    p.tok_cols = token_cols;
    p.cols = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(BSP_MAX_TAIL, int64_t(kAdvanceSmem) / (8 * int64_t(plan->beam_width)))));
    return launched(launch_advance(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

bsp_status key_weights_impl(const bsp_plan_t* plan, const void* q, const void* k_pool, const float* lse,
                            float softmax_scale, float k_scale, int32_t window, int32_t flags, float* weights,
                            int64_t weights_stride, void* stream, bool fp8) {
    bsp_status st = check_plan(plan);
    if (st != BSP_OK) return st;
    const bsp_geometry& geo = plan->geo;
    if ((geo.kv_dtype == BSP_KV_DTYPE_E4M3) != fp8) return BSP_ERR_INVALID_ARG;
    if (flags & ~(BSP_FLAG_LSE_BASE2 | BSP_FLAG_CHECK | BSP_FLAG_ACCUMULATE)) return BSP_ERR_INVALID_ARG;
    if (!(softmax_scale > 0.f) || !std::isfinite(softmax_scale) || !(k_scale > 0.f) || !std::isfinite(k_scale))
        return BSP_ERR_INVALID_ARG;
    if (window < 0 || (window > 0 && plan->kind != 1)) return BSP_ERR_INVALID_ARG;
    if (weights_stride < plan->max_prefix_len) return BSP_ERR_INVALID_ARG;
    if (plan->batch > BSP_MAX_WEIGHTS_BATCH) return BSP_ERR_UNSUPPORTED;
    if (plan->total_rows == 0) return BSP_OK;
    if (!plan_here(plan)) return BSP_ERR_INVALID_ARG;
    if (!device_ptr(q, 16) || !device_ptr(k_pool, 16) || !device_ptr(lse, 4) || !device_ptr(weights, 4))
        return BSP_ERR_INVALID_ARG;
    const int D = geo.head_dim, Hq = geo.num_q_heads, Hkv = geo.num_kv_heads, G = Hq / Hkv, ps = geo.page_size;
    WeightsParams p{};
    // query rows of a block: one MMA's N (at head_dim 256 half of that, so that a K ring fits beside it). A
    // decode step's rows are the beams; a prefill's at most its rows, or the window.
    const int nmax = D == 256 ? 128 : 256;
    const int rows = plan->kind == 0 ? plan->beam_width
                     : window > 0    ? std::min(window, plan->total_rows)
                                     : plan->total_rows;
    p.block_rows = std::min(rows, nmax / G);
    p.mma_n = static_cast<int>(ceil_div(p.block_rows * G, 16) * 16);
    const size_t q_bytes = static_cast<size_t>(D) * 2 * p.mma_n, k_bytes = static_cast<size_t>(D) * 2 * 128;
    const size_t fixed = 1024 + kWeightsTableBytes + kWeightsBarBytes + (static_cast<size_t>(plan->batch) + 1) * 4;
    const size_t room = kMaxSmem - fixed;
    // A second Q slot hides the change of (request, kv head), a deeper K ring the latency of every tile: two slots
    // where three K slots remain (30 beams, D = 128: group 2, 500 keys, 20.8 us and 23.0 with one; group 4, 2000
    // keys, 55 and 58). With fewer the K ring is worth more (D = 256, group 4: one K slot left, 142 and 100).
    p.q_slots = 2 * q_bytes + 3 * k_bytes <= room ? 2 : 1;
    p.k_slots = static_cast<int>(std::min<size_t>(8, (room - p.q_slots * q_bytes) / k_bytes));
    if (p.k_slots < 1) return BSP_ERR_UNSUPPORTED;
    p.req = section(plan, plan->off_req);
    p.pages = section(plan, plan->off_pages);
    p.plan_hdr = image_header(plan);
    p.q = q;
    p.lse = lse;
    p.weights = weights;
    p.stride = weights_stride;
    p.status = status_word(plan);
    p.batch = plan->batch;
    p.shape = plan_shape(plan);
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = G;
    p.ps_log2 = ilog2(ps);
    p.num_pages = geo.num_pages;
    p.max_keys = static_cast<int>(std::min<int64_t>(weights_stride, 1 << 30));
    p.window = window;
    p.accumulate = (flags & BSP_FLAG_ACCUMULATE) != 0;
    const float log2e = 1.4426950408889634f;
    p.scale_log2 = softmax_scale * k_scale * log2e;
    p.lse_mul = (flags & BSP_FLAG_LSE_BASE2) ? 1.f : log2e;
    const size_t smem = fixed + p.q_slots * q_bytes + p.k_slots * k_bytes;
    const bool bf16 = geo.dtype == BSP_DTYPE_BF16;
    st = launched(prepare_weights(D, bf16, fp8));
    if (st != BSP_OK) return st;
    CUtensorMap tq, tk;
    cuuint64_t qdims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(Hq), static_cast<cuuint64_t>(plan->total_rows)};
    cuuint64_t qstr[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(Hq) * D * 2};
    cuuint32_t qbox[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(p.block_rows)};
    cuuint64_t kdims[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(geo.num_pages) * Hkv * ps};
    cuuint64_t kstr[1] = {static_cast<cuuint64_t>(D) * (fp8 ? 1 : 2)};
    cuuint32_t kbox[2] = {static_cast<cuuint32_t>(fp8 ? D : 64), static_cast<cuuint32_t>(std::min(ps, 64))};
    if (!encode_map(&tq, geo.dtype, 3, q, qdims, qstr, qbox) || !encode_map(&tk, geo.dtype, 2, k_pool, kdims, kstr, kbox, fp8))
        return BSP_ERR_CUDA;
    st = launched(launch_weights(D, bf16, fp8, tq, tk, p, plan->num_sms, smem, static_cast<cudaStream_t>(stream)));
    if (st != BSP_OK) return st;
    return (flags & BSP_FLAG_CHECK) ? bsp_read_device_status(plan, stream, 1, nullptr) : BSP_OK;
}

}  // namespace

extern "C" {

bsp_status bsp_key_weights(const bsp_plan_t* plan, const void* q, const void* k_pool, const float* lse,
                           float softmax_scale, int32_t window, int32_t flags, float* weights, int64_t weights_stride,
                           void* stream) {
    return key_weights_impl(plan, q, k_pool, lse, softmax_scale, 1.f, window, flags, weights, weights_stride, stream, false);
}

bsp_status bsp_key_weights_fp8(const bsp_plan_t* plan, const void* q, const void* k_pool, const float* lse,
                               float softmax_scale, float k_scale, int32_t window, int32_t flags, float* weights,
                               int64_t weights_stride, void* stream) {
    return key_weights_impl(plan, q, k_pool, lse, softmax_scale, k_scale, window, flags, weights, weights_stride, stream, true);
}

bsp_status bsp_evict_prefix(const bsp_plan_t* plan, const float* weights, int64_t weights_stride,
                            const int32_t* positions, const int32_t* keep_len, int32_t sinks, int32_t recent,
                            void* k_pool, void* v_pool, int32_t* kept, float* weights_out, int32_t* positions_out,
                            int64_t out_stride, void* stream) {
    bsp_status st = check_plan(plan);
    if (st != BSP_OK) return st;
    const bsp_geometry& geo = plan->geo;
    if (sinks < 0 || recent < 0) return BSP_ERR_INVALID_ARG;
    if (plan->max_tail_len > 0) return BSP_ERR_INVALID_ARG;  // tail rows follow the prompt: evict before there are any
    if (weights_stride < plan->max_prefix_len || out_stride < plan->max_prefix_len) return BSP_ERR_INVALID_ARG;
    if (plan->max_prefix_len > BSP_MAX_EVICT_ROWS || plan->batch > BSP_MAX_STEP_BATCH) return BSP_ERR_UNSUPPORTED;
    if (plan->total_rows == 0) return BSP_OK;
    if (!plan_here(plan)) return BSP_ERR_INVALID_ARG;
    if (!device_ptr(weights, 4) || !optional_ptr(positions, 4) || !device_ptr(keep_len, 4) || !device_ptr(k_pool, 16) ||
        !device_ptr(v_pool, 16) || !device_ptr(kept, 4) || !optional_ptr(weights_out, 4) || !optional_ptr(positions_out, 4))
        return BSP_ERR_INVALID_ARG;
    // in place only where every slot keeps its address
    if ((weights_out == weights || (positions && positions_out == positions)) && weights_stride != out_stride)
        return BSP_ERR_INVALID_ARG;
    EvictParams p{};
    p.req = section(plan, plan->off_req);
    p.pages = section(plan, plan->off_pages);
    p.plan_hdr = image_header(plan);
    p.weights = weights;
    p.positions = positions;
    p.keep = keep_len;
    p.k_pool = static_cast<uint8_t*>(k_pool);
    p.v_pool = static_cast<uint8_t*>(v_pool);
    p.kept = kept;
    p.weights_out = weights_out;
    p.positions_out = positions_out;
    p.stride = weights_stride;
    p.out_stride = out_stride;
    p.status = status_word(plan);
    p.batch = plan->batch;
    p.shape = plan_shape(plan);
    p.Hkv = geo.num_kv_heads;
    p.num_pages = geo.num_pages;
    p.ps_log2 = ilog2(geo.page_size);
    p.row_bytes = geo.head_dim * (geo.kv_dtype == BSP_KV_DTYPE_E4M3 ? 1 : 2);
    // lengths of a replayed plan are checked against this, the tables' room
    p.max_keys = static_cast<int>(std::min<int64_t>({weights_stride, out_stride, BSP_MAX_EVICT_ROWS}));
    p.sinks = sinks;
    p.recent = recent;
    return launched(launch_evict(p, plan->max_prefix_len, plan->num_sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
