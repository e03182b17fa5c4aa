// Host side of the cache's other entries: appends of normalised rows, of blocks with scales, tables of stretched
// rotations, and the page bookkeeping. Declared in include/bsp.h.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/bsp.h"
#include "bsp_check.h"
#include "bsp_pages.h"
#include "bsp_write.h"

namespace {

using namespace bsp;

bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
    const uint8_t* x = static_cast<const uint8_t*>(a);
    const uint8_t* y = static_cast<const uint8_t*>(b);
    return x < y + nb && y < x + na;
}

// Whether one of n rows of na bytes, sa apart from a on, shares a byte with one of n rows of nb bytes, sb apart from b
// on. Rows of one stride are compared as they lie, so that column slices of one buffer pass; others by what they span.
bool rows_overlap(const void* a, int64_t na, int64_t sa, const void* b, int64_t nb, int64_t sb, int64_t n) {
    if (sa != sb) return overlap(a, (n - 1) * sa + na, b, (n - 1) * sb + nb);
    // row i + k of b begins d + k sa behind row i of a: of the k within n rows, the largest that begins before a's row ends
    const int64_t d = static_cast<int64_t>(reinterpret_cast<intptr_t>(b) - reinterpret_cast<intptr_t>(a));
    const int64_t room = na - 1 - d;
    const int64_t k = std::min(room >= 0 ? room / sa : -((-room + sa - 1) / sa), n - 1);
    return k > -n && d + k * sa + nb > 0;
}

// What the three appends share: the arguments but for the pools' own, checked, in *a. BSP_OK with a->n = 0: nothing
// to do.
bsp_status check_norm_append(const bsp_plan_t* plan, const bsp_qk_norm* norm, const bsp_rope_config* rope,
                             const int32_t* positions, const void* q, int64_t q_row_stride, void* q_out,
                             int64_t q_out_stride, const void* k_new, const void* v_new, int64_t src_row_stride,
                             const int32_t* loc, int32_t n, const void* k_pool, const void* v_pool, NormRope* a) {
    *a = NormRope{};
    const bsp_geometry& geo = plan->geo;
    const int D = geo.head_dim;
    if (n < 0) return BSP_ERR_INVALID_ARG;
    if (norm) {
        if (!(norm->eps >= 0.f) || !std::isfinite(norm->eps) || !std::isfinite(norm->weight_offset) ||
            norm->reserved != 0 ||
            (norm->weight_fp32 != 0 && norm->weight_fp32 != 1))
            return BSP_ERR_INVALID_ARG;
    }
    if (rope) {
        if (rope->rotary_dim < 16 || rope->rotary_dim > D || (rope->rotary_dim & 15) || rope->max_position <= 0 ||
            (rope->interleaved != 0 && rope->interleaved != 1) || rope->reserved != 0)
            return BSP_ERR_INVALID_ARG;
    }
    if (n == 0) return BSP_OK;
    if (n > plan->total_rows) return BSP_ERR_INVALID_ARG;
    const int64_t kv_row = static_cast<int64_t>(geo.num_kv_heads) * D;
    const int64_t q_row = static_cast<int64_t>(geo.num_q_heads) * D;
    if (src_row_stride < kv_row || (src_row_stride & 7)) return BSP_ERR_INVALID_ARG;
    if (q && (q_row_stride < q_row || (q_row_stride & 7) || q_out_stride < q_row || (q_out_stride & 7)))
        return BSP_ERR_INVALID_ARG;
    if (!plan_here(plan)) return BSP_ERR_INVALID_ARG;
    if (!device_ptr(k_new, 16) || !device_ptr(v_new, 16) || !device_ptr(loc, 4) || !device_ptr(k_pool, 16) ||
        !device_ptr(v_pool, 16))
        return BSP_ERR_INVALID_ARG;
    if (q && (!device_ptr(q, 16) || !device_ptr(q_out, 16))) return BSP_ERR_INVALID_ARG;
    if (rope && (!device_ptr(rope->cos_sin, 16) || !device_ptr(positions, 4))) return BSP_ERR_INVALID_ARG;
    if (norm && (!optional_ptr(norm->q_weight, 16) || !optional_ptr(norm->k_weight, 16))) return BSP_ERR_INVALID_ARG;
    if (q && q_out == q && q_out_stride != q_row_stride) return BSP_ERR_INVALID_ARG;
    if (q && q_out != q) {
        auto over_rows = [&](const void* x, int64_t row, int64_t stride) {
            return rows_overlap(q_out, 2 * q_row, 2 * q_out_stride, x, 2 * row, 2 * stride, n);
        };
        auto over = [&](const void* x, int64_t bytes) {
            return x && overlap(q_out, 2 * ((n - 1) * q_out_stride + q_row), x, bytes);
        };
        if (over_rows(q, q_row, q_row_stride) || over_rows(k_new, kv_row, src_row_stride) ||
            over_rows(v_new, kv_row, src_row_stride) || over(loc, 4ll * n))
            return BSP_ERR_INVALID_ARG;
        if (rope && (over(positions, 4ll * n) ||
                     over(rope->cos_sin, 4ll * rope->max_position * rope->rotary_dim)))
            return BSP_ERR_INVALID_ARG;
        const int64_t weight = static_cast<int64_t>(D) * (norm && norm->weight_fp32 ? 4 : 2);
        if (norm && (over(norm->q_weight, weight) || over(norm->k_weight, weight))) return BSP_ERR_INVALID_ARG;
    }
    a->loc = loc;
    if (rope) {
        a->pos = positions;
        a->cos_sin = rope->cos_sin;
        a->rot = rope->rotary_dim;
        a->interleaved = rope->interleaved;
        a->max_pos = rope->max_position;
    }
    a->q = q;
    a->q_out = q ? q_out : nullptr;
    a->q_stride = q_row_stride;
    a->q_out_stride = q_out_stride;
    if (norm) {
        a->norm = 1;
        a->q_weight = norm->q_weight;
        a->k_weight = norm->k_weight;
        a->eps = norm->eps;
        a->weight_offset = norm->weight_offset;
        a->weight_fp32 = norm->weight_fp32;
    }
    a->Hq = q ? geo.num_q_heads : 0;  // (without query rows the last CTA's spare warps find none)
    a->n = n;
    return BSP_OK;
}

bsp_status norm_append_impl(const bsp_plan_t* plan, const bsp_qk_norm* norm, const bsp_rope_config* rope,
                            const int32_t* positions, const void* q, int64_t q_row_stride, void* q_out,
                            int64_t q_out_stride, const void* k_new, const void* v_new, int64_t src_row_stride,
                            bool fp8, float k_mul, float v_mul, const int32_t* loc, int32_t n, void* k_pool,
                            void* v_pool, void* const* events, void* stream) {
    bsp_status st = check_plan(plan);
    if (st != BSP_OK) return st;
    if (!norm) return BSP_ERR_INVALID_ARG;
    if (!fp8 && plan->geo.kv_dtype != BSP_KV_DTYPE_SAME) return BSP_ERR_INVALID_ARG;  // 16-bit pools only
    if (fp8 && (!std::isfinite(k_mul) || !std::isfinite(v_mul) || !(k_mul > 0.f) || !(v_mul > 0.f)))
        return BSP_ERR_INVALID_ARG;
    NormAppendParams p{};
    st = check_norm_append(plan, norm, rope, positions, q, q_row_stride, q_out, q_out_stride, k_new, v_new,
                           src_row_stride, loc, n, k_pool, v_pool, &p.a);
    if (st != BSP_OK || p.a.n == 0) return st;
    const bsp_geometry& geo = plan->geo;
    p.k_new = k_new;
    p.v_new = v_new;
    p.src_stride = src_row_stride;
    p.k_pool = k_pool;
    p.v_pool = v_pool;
    p.status = status_word(plan);
    p.Hkv = geo.num_kv_heads;
    p.ps_log2 = ilog2(geo.page_size);
    p.num_pages = geo.num_pages;
    p.k_mul = k_mul;
    p.v_mul = v_mul;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!record_event(events, 0, s)) return BSP_ERR_CUDA;
    st = launched(launch_norm_append(geo.head_dim, geo.dtype == BSP_DTYPE_BF16, fp8 ? kPoolE4m3 : kPool16, false, p,
                                     plan->num_sms, s));
    if (st != BSP_OK) return st;
    return record_event(events, 1, s) ? BSP_OK : BSP_ERR_CUDA;
}

// The geometry of a page call: its pools' bytes per row, and that its pages can be counted.
bsp_status check_pages(const bsp_plan_t* plan) {
    bsp_status st = check_plan(plan);
    if (st != BSP_OK) return st;
    if (plan->geo.num_pages > BSP_MAX_PAGES) return BSP_ERR_UNSUPPORTED;
    return BSP_OK;
}
int row_bytes(const bsp_geometry& geo) { return geo.head_dim * (geo.kv_dtype == BSP_KV_DTYPE_E4M3 ? 1 : 2); }

bsp_status check_forks(const bsp_plan_t* plan, int64_t beams_stride, int32_t num_forks, int64_t out_stride,
                       int32_t out_cols) {
    if (plan->kind != 0 || num_forks < 1 || beams_stride < num_forks) return BSP_ERR_INVALID_ARG;
    if (static_cast<int64_t>(plan->batch) * num_forks > BSP_MAX_FORK_ROWS) return BSP_ERR_UNSUPPORTED;
    if (out_cols < 0 || out_stride < out_cols || out_cols < ceil_div(plan->max_total_len, plan->geo.page_size))
        return BSP_ERR_INVALID_ARG;
    return BSP_OK;
}

}  // namespace

extern "C" {

bsp_status bsp_norm_rope_append_kv(const bsp_plan_t* plan, const bsp_qk_norm* norm, const bsp_rope_config* rope,
                                   const int32_t* positions, const void* q, int64_t q_row_stride, void* q_out,
                                   int64_t q_out_stride, const void* k_new, const void* v_new, int64_t src_row_stride,
                                   const int32_t* out_cache_loc, int32_t n, void* k_pool, void* v_pool,
                                   void* const* events, void* stream) {
    return norm_append_impl(plan, norm, rope, positions, q, q_row_stride, q_out, q_out_stride, k_new, v_new,
                            src_row_stride, false, 1.f, 1.f, out_cache_loc, n, k_pool, v_pool, events, stream);
}

bsp_status bsp_norm_rope_append_kv_fp8(const bsp_plan_t* plan, const bsp_qk_norm* norm, const bsp_rope_config* rope,
                                       const int32_t* positions, const void* q, int64_t q_row_stride, void* q_out,
                                       int64_t q_out_stride, const void* k_new, const void* v_new,
                                       int64_t src_row_stride, float k_mul, float v_mul, const int32_t* out_cache_loc,
                                       int32_t n, void* k_pool, void* v_pool, void* const* events, void* stream) {
    return norm_append_impl(plan, norm, rope, positions, q, q_row_stride, q_out, q_out_stride, k_new, v_new,
                            src_row_stride, true, k_mul, v_mul, out_cache_loc, n, k_pool, v_pool, events, stream);
}

bsp_status bsp_append_kv_fp8_blocks(const bsp_plan_t* plan, const bsp_qk_norm* norm, const bsp_rope_config* rope,
                                    const int32_t* positions, const void* q, int64_t q_row_stride, void* q_out,
                                    int64_t q_out_stride, const void* k_new, const void* v_new, int64_t src_row_stride,
                                    const int32_t* out_cache_loc, int32_t n, void* k_pool, void* v_pool,
                                    const bsp_block_scales* scales, void* const* events, void* stream) {
    bsp_status st = check_plan(plan);
    if (st != BSP_OK) return st;
    const bsp_geometry& geo = plan->geo;
    st = check_block_scales(scales, geo.page_size, n > 0);
    if (st != BSP_OK) return st;
    NormAppendParams p{};
    st = check_norm_append(plan, norm, rope, positions, q, q_row_stride, q_out, q_out_stride, k_new, v_new,
                           src_row_stride, out_cache_loc, n, k_pool, v_pool, &p.a);
    if (st != BSP_OK || p.a.n == 0) return st;
    if (!device_ptr(scales->k, 16) || !device_ptr(scales->v, 16)) return BSP_ERR_INVALID_ARG;
    const bool bf16 = geo.dtype == BSP_DTYPE_BF16;
    p.k_new = k_new;
    p.v_new = v_new;
    p.src_stride = src_row_stride;
    p.k_pool = k_pool;
    p.v_pool = v_pool;
    p.k_exp = scales->k;
    p.v_exp = scales->v;
    p.status = status_word(plan);
    p.Hkv = geo.num_kv_heads;
    p.ps_log2 = ilog2(geo.page_size);
    p.num_pages = geo.num_pages;
    p.block_log2 = ilog2(scales->block);
    p.exp_lo = bf16 ? 27 : kReadLo<false>;  // 2^-100 .. 2^15, 2^-15 .. 2^7
    p.exp_hi = bf16 ? kReadHi<true> : kReadHi<false>;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!record_event(events, 0, s)) return BSP_ERR_CUDA;
    st = launched(launch_norm_append(geo.head_dim, bf16, kPoolBlocks, plan->kind == 1, p, plan->num_sms, s));
    if (st != BSP_OK) return st;
    return record_event(events, 1, s) ? BSP_OK : BSP_ERR_CUDA;
}

bsp_status bsp_rope_cos_sin_scaled(int32_t max_position, int32_t rotary_dim, double base,
                                   const bsp_rope_scaling* scaling, float* cos_sin, void* stream) {
    if (max_position <= 0 || rotary_dim < 2 || rotary_dim > 1024 || (rotary_dim & 1)) return BSP_ERR_INVALID_ARG;
    if (!(base > 1.0) || !std::isfinite(base) || !scaling) return BSP_ERR_INVALID_ARG;
    const bsp_rope_scaling& c = *scaling;
    if (c.kind < BSP_ROPE_LINEAR || c.kind > BSP_ROPE_RAMP) return BSP_ERR_UNSUPPORTED;
    if (!(c.factor > 0) || !std::isfinite(c.factor) || !(c.amplitude > 0) || !std::isfinite(c.amplitude))
        return BSP_ERR_INVALID_ARG;
    if (c.kind == BSP_ROPE_BASE && rotary_dim == 2) return BSP_ERR_INVALID_ARG;
    if (c.kind >= BSP_ROPE_BANDS &&
        (c.original_positions <= 0 || !(c.low > 0) || !(c.high > c.low) || !std::isfinite(c.high)))
        return BSP_ERR_INVALID_ARG;
    if (!device_ptr(cos_sin, 16)) return BSP_ERR_INVALID_ARG;
    return launched(launch_rope_scaled(max_position, rotary_dim, base, c, cos_sin, static_cast<cudaStream_t>(stream)));
}

bsp_status bsp_fork_workspace_size(int32_t batch, int32_t num_forks, size_t* device_bytes) {
    if (!device_bytes || batch < 0 || num_forks < 1) return BSP_ERR_INVALID_ARG;
    if (static_cast<int64_t>(batch) * num_forks > BSP_MAX_FORK_ROWS) return BSP_ERR_UNSUPPORTED;
    // a row's first fresh page, and its fresh pages: the rest of a page and a tail fill two at most
    static_assert(BSP_MAX_TAIL <= 8, "the smallest page holds a whole tail");
    *device_bytes = static_cast<size_t>(batch) * num_forks * 12;
    return BSP_OK;
}

bsp_status bsp_fork_tables(const bsp_plan_t* plan, const int32_t* beams, int64_t beams_stride, int32_t num_forks,
                           const int32_t* refs_in, int32_t* refs_out, int32_t* pages_out, int64_t pages_out_stride,
                           int32_t pages_out_cols, void* workspace, size_t workspace_bytes, void* stream) {
    bsp_status st = check_pages(plan);
    if (st != BSP_OK) return st;
    st = check_forks(plan, beams_stride, num_forks, pages_out_stride, pages_out_cols);
    if (st != BSP_OK) return st;
    if (!plan_here(plan) || !device_ptr(refs_in, 4) || !device_ptr(refs_out, 4)) return BSP_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bsp_geometry& geo = plan->geo;
    if (plan->batch == 0) {  // nothing forks
        if (refs_in == refs_out) return BSP_OK;
        return launched(cudaMemcpyAsync(refs_out, refs_in, static_cast<size_t>(geo.num_pages) * 4,
                                        cudaMemcpyDeviceToDevice, s));
    }
    const int64_t rows = static_cast<int64_t>(plan->batch) * num_forks;
    if (!device_ptr(beams, 4) || (pages_out_cols > 0 && !device_ptr(pages_out, 4)) || !device_ptr(workspace, 4))
        return BSP_ERR_INVALID_ARG;
    if (static_cast<size_t>(rows) * 12 > workspace_bytes) return BSP_ERR_CAPACITY;
    ForkParams p{};
    p.req = section(plan, plan->off_req);
    p.pages = section(plan, plan->off_pages);
    p.plan_hdr = image_header(plan);
    p.beams = beams;
    p.beams_stride = beams_stride;
    p.refs_in = refs_in;
    p.refs_out = refs_out;
    p.pages_out = pages_out;
    p.out_stride = pages_out_stride;
    p.out_cols = pages_out_cols;
    p.base = static_cast<int32_t*>(workspace);
    p.fresh = p.base + rows;
    p.status = status_word(plan);
    p.shape = plan_shape(plan);
    p.batch = plan->batch;
    p.W = plan->beam_width;
    p.num_forks = num_forks;
    p.rows = static_cast<int>(rows);
    p.num_pages = geo.num_pages;
    p.ps_log2 = ilog2(geo.page_size);
    return launched(launch_fork_tables(p, s));
}

bsp_status bsp_fork_rows(const bsp_plan_t* plan, const int32_t* beams, int64_t beams_stride, int32_t num_forks,
                         const int32_t* pages_out, int64_t pages_out_stride, int32_t pages_out_cols,
                         const int32_t* beam_pages, int32_t beam_pages_stride, const int32_t* cache_indirection,
                         int32_t max_seq, void* k_pool, void* v_pool, const bsp_block_scales* scales, void* stream) {
    bsp_status st = check_pages(plan);
    if (st != BSP_OK) return st;
    st = check_forks(plan, beams_stride, num_forks, pages_out_stride, pages_out_cols);
    if (st != BSP_OK) return st;
    const bsp_geometry& geo = plan->geo;
    if (scales) {
        if (geo.kv_dtype != BSP_KV_DTYPE_E4M3) return BSP_ERR_INVALID_ARG;
        st = check_block_scales(scales, geo.page_size, true);
        if (st != BSP_OK) return st;
    }
    if (static_cast<int64_t>(geo.num_kv_heads) * geo.page_size * row_bytes(geo) > INT32_MAX) return BSP_ERR_UNSUPPORTED;
    if (plan->batch == 0) return BSP_OK;
    if (!plan_here(plan) || !device_ptr(beams, 4) || !device_ptr(pages_out, 4) || !device_ptr(k_pool, 16) ||
        !device_ptr(v_pool, 16) ||
        !optional_ptr(beam_pages, 4) || !optional_ptr(cache_indirection, 4))
        return BSP_ERR_INVALID_ARG;
    if ((beam_pages == nullptr) != (cache_indirection == nullptr)) return BSP_ERR_INVALID_ARG;
    if (plan->max_tail_len > 0 && (!beam_pages || max_seq < plan->max_total_len ||
                                   beam_pages_stride < ceil_div(plan->max_total_len, geo.page_size)))
        return BSP_ERR_INVALID_ARG;
    ForkRowsParams p{};
    p.req = section(plan, plan->off_req);
    p.pages = section(plan, plan->off_pages);
    p.plan_hdr = image_header(plan);
    p.beams = beams;
    p.beams_stride = beams_stride;
    p.pages_out = pages_out;
    p.out_stride = pages_out_stride;
    p.out_cols = pages_out_cols;
    p.beam_pages = beam_pages;
    p.beam_cols = beam_pages ? beam_pages_stride : 0;
    p.ci = cache_indirection;
    p.max_seq = beam_pages ? max_seq : 0;
    p.k_pool = static_cast<uint8_t*>(k_pool);
    p.v_pool = static_cast<uint8_t*>(v_pool);
    if (scales) {
        p.k_exp = scales->k;
        p.v_exp = scales->v;
        p.block_log2 = ilog2(scales->block);
        p.read_lo = geo.dtype == BSP_DTYPE_BF16 ? kReadLo<true> : kReadLo<false>;
        p.read_hi = geo.dtype == BSP_DTYPE_BF16 ? kReadHi<true> : kReadHi<false>;
    }
    p.status = status_word(plan);
    p.shape = plan_shape(plan);
    p.W = plan->beam_width;
    p.num_forks = num_forks;
    p.rows = plan->batch * num_forks;
    p.num_pages = geo.num_pages;
    p.Hkv = geo.num_kv_heads;
    p.ps_log2 = ilog2(geo.page_size);
    p.row_bytes = row_bytes(geo);
    return launched(launch_fork_rows(p, plan->num_sms, static_cast<cudaStream_t>(stream)));
}

bsp_status bsp_free_pages(const bsp_plan_t* plan, const int32_t* tables, int64_t stride, int32_t rows, int32_t cols,
                          const int32_t* refs_in, int32_t* refs_out, void* stream) {
    bsp_status st = check_pages(plan);
    if (st != BSP_OK) return st;
    if (rows < 0 || cols < 0 || stride < cols) return BSP_ERR_INVALID_ARG;
    if (!plan_here(plan) || !device_ptr(refs_in, 4) || !device_ptr(refs_out, 4)) return BSP_ERR_INVALID_ARG;
    if (rows > 0 && cols > 0 && !device_ptr(tables, 4)) return BSP_ERR_INVALID_ARG;
    FreeParams p{};
    p.tables = tables;
    p.stride = stride;
    p.refs_out = refs_out;
    p.status = status_word(plan);
    p.rows = rows;
    p.cols = cols;
    p.num_pages = plan->geo.num_pages;
    return launched(launch_free_pages(p, refs_in, plan->num_sms, static_cast<cudaStream_t>(stream)));
}

bsp_status bsp_compact_tables(const bsp_plan_t* plan, const int32_t* refs_in, int32_t* refs_out, int32_t* pairs,
                              int32_t* count, int32_t* remap, const int32_t* tables_in, int32_t* tables_out,
                              int64_t stride, int32_t rows, int32_t cols, void* stream) {
    bsp_status st = check_pages(plan);
    if (st != BSP_OK) return st;
    if (rows < 0 || cols < 0 || stride < cols) return BSP_ERR_INVALID_ARG;
    if (!plan_here(plan) || !device_ptr(refs_in, 4) || !device_ptr(refs_out, 4) || !device_ptr(count, 4) ||
        !device_ptr(remap, 4))
        return BSP_ERR_INVALID_ARG;
    if (plan->geo.num_pages > 1 && !device_ptr(pairs, 4)) return BSP_ERR_INVALID_ARG;
    if (rows > 0 && cols > 0 && (!device_ptr(tables_in, 4) || !device_ptr(tables_out, 4))) return BSP_ERR_INVALID_ARG;
    CompactParams p{};
    p.refs_in = refs_in;
    p.refs_out = refs_out;
    p.pairs = pairs;
    p.count = count;
    p.remap = remap;
    p.tables_in = tables_in;
    p.tables_out = tables_out;
    p.stride = stride;
    p.status = status_word(plan);
    p.rows = rows;
    p.cols = cols;
    p.num_pages = plan->geo.num_pages;
    return launched(launch_compact_tables(p, plan->num_sms, static_cast<cudaStream_t>(stream)));
}

bsp_status bsp_copy_pages(const bsp_plan_t* plan, const int32_t* pairs, const int32_t* count, int32_t max_pairs,
                          void* k_pool, void* v_pool, const bsp_block_scales* scales, void* stream) {
    bsp_status st = check_pages(plan);
    if (st != BSP_OK) return st;
    const bsp_geometry& geo = plan->geo;
    if (max_pairs < 0) return BSP_ERR_INVALID_ARG;
    if (scales) {
        if (geo.kv_dtype != BSP_KV_DTYPE_E4M3) return BSP_ERR_INVALID_ARG;
        st = check_block_scales(scales, geo.page_size, true);
        if (st != BSP_OK) return st;
    }
    if (max_pairs == 0) return BSP_OK;
    if (!plan_here(plan) || !device_ptr(pairs, 4) || !device_ptr(count, 4) || !device_ptr(k_pool, 16) ||
        !device_ptr(v_pool, 16))
        return BSP_ERR_INVALID_ARG;
    CopyParams p{};
    p.pairs = pairs;
    p.count = count;
    p.max_pairs = max_pairs;
    p.k_pool = static_cast<uint8_t*>(k_pool);
    p.v_pool = static_cast<uint8_t*>(v_pool);
    if (scales) {
        p.k_exp = scales->k;
        p.v_exp = scales->v;
        p.exp_bytes = geo.num_kv_heads * (geo.page_size / scales->block);
    }
    p.status = status_word(plan);
    p.page_bytes = static_cast<long long>(geo.num_kv_heads) * geo.page_size * row_bytes(geo);
    p.num_pages = geo.num_pages;
    return launched(launch_copy_pages(p, plan->num_sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
