// Page bookkeeping of the paged cache: tables of forked beams and their rows, references given back, live pages moved
// to the lowest ids, pages copied. The state is one count of references per page; a page without any is free. Free
// pages are always taken lowest first and live ones keep their order, so every choice is a rank among the pages, found
// by a running count, and nothing depends on the order of arrival.
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/bsp.h"
#include "bsp_pages.h"

namespace cg = cooperative_groups;

namespace bsp {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kScanThreads = 1024;
constexpr int kScanCtas = 8;  // of the cluster that scans
// A pool of up to kSmallPool pages is scanned by a single CTA, a count a thread, without the cluster's barriers:
// compaction of 96 pages 3.3 us for 6.8, of 1024 3.9 for 7.7 (4096 with four a thread 10.8 for 8.0); forks' tables over
// 512 pages 4.9 for 7.5 (2048: 7.4 for 7.2).
constexpr int kSmallPool = kScanThreads;
// counts of a thread in a round of a scan by CTAS CTAs
template <int CTAS>
constexpr int kCounts = CTAS == 1 ? 1 : 4;

template <int CTAS>
__device__ __forceinline__ void scan_sync() {
    if constexpr (CTAS == 1) __syncthreads();
    else cg::this_cluster().sync();
}
template <int CTAS>
__device__ __forceinline__ int scan_rank() {
    return CTAS == 1 ? 0 : static_cast<int>(cg::this_cluster().block_rank());
}

// Exclusive running sum over the CTA's threads and the total, in s_warp[33] of shared memory.
__device__ __forceinline__ int cta_scan(int x, int* s_warp, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int v = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += y;
    }
    __syncthreads();  // (the last round's sums have been read)
    if (lane == 31) s_warp[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int w = s_warp[lane], s = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, s, o);
            if (lane >= o) s += y;
        }
        s_warp[lane] = s - w;
        if (lane == 31) s_warp[32] = s;
    }
    __syncthreads();
    *total = s_warp[32];
    return s_warp[warp] + v - x;
}

// The sum over the CTA's threads.
__device__ __forceinline__ int cta_sum(int x, int* s_warp) {
    x = __reduce_add_sync(kFull, x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = x;
    __syncthreads();
    if (threadIdx.x < 32) {
        const int s = __reduce_add_sync(kFull, s_warp[threadIdx.x]);
        if (threadIdx.x == 0) s_warp[32] = s;
    }
    __syncthreads();
    return s_warp[32];
}

// The sum of what the cluster's CTAs hold in `mine` (shared memory, the same variable in each), of those before this
// one and of all. Every CTA's value is set before and stays until the cluster's next barrier.
template <int CTAS>
__device__ __forceinline__ int cluster_sum(int* mine, int* all) {
    if constexpr (CTAS == 1) {
        *all = *mine;
        return 0;
    }
    cg::cluster_group cl = cg::this_cluster();
    int before = 0, sum = 0;
    const unsigned me = cl.block_rank();
#pragma unroll
    for (unsigned r = 0; r < CTAS; ++r) {
        const int x = *cl.map_shared_rank(mine, r);
        if (r < me) before += x;
        sum += x;
    }
    *all = sum;
    return before;
}

// A CTA's share of n items, [lo, hi): even shares in whole vectors of four.
template <int CTAS>
__device__ __forceinline__ void share_of(int n, int rank, int* lo, int* hi) {
    const int per = ((n + CTAS - 1) / CTAS + 3) & ~3;
    *lo = min(n, rank * per);
    *hi = min(n, *lo + per);
}

__device__ __forceinline__ int valid_beam(const ForkParams& p, int b, int j) {
    const int w = __ldg(p.beams + b * p.beams_stride + j);
    if (w < -1 || w >= p.W) atomicOr(p.status, BSP_DEVFLAG_PAGE_INDEX);
    return w >= 0 && w < p.W ? w : -1;
}
// fresh pages of a row of request b, and its full prompt pages
__device__ __forceinline__ int fresh_pages(const ForkParams& p, int b, int* full) {
    const int32_t* rec = p.req + static_cast<long long>(b) * kReqFields;
    const int P = __ldg(rec + kReqPrefix), T = __ldg(rec + kReqTail);
    *full = P >> p.ps_log2;
    return ((P + T + (1 << p.ps_log2) - 1) >> p.ps_log2) - *full;
}

// The entries of a forked row's table and its fresh pages' counts, by `lanes` threads.
__device__ __forceinline__ void fork_row_table(const ForkParams& p, int i, int lane, int lanes) {
    const int b = i / p.num_forks;
    int full;
    const int need = fresh_pages(p, b, &full);
    if (full + need > p.out_cols) {  // a replayed plan that outgrew the table
        if (lane == 0) atomicOr(p.status, BSP_DEVFLAG_GRAPH);
        return;
    }
    const int32_t* prompt = p.pages + __ldg(p.req + static_cast<long long>(b) * kReqFields + kReqPageOff);
    const int base = p.base[i];
    int32_t* out = p.pages_out + static_cast<long long>(i) * p.out_stride;
    for (int c = lane; c < full + need; c += lanes) {
        int page = -1;
        if (base >= 0) {
            page = c < full ? __ldg(prompt + c) : p.fresh[base + c - full];
            if (c >= full) p.refs_out[page] = 1;
        }
        out[c] = page;
    }
}
// The references that a request's served forks add to its full prompt pages, by a warp.
__device__ __forceinline__ void fork_request_refs(const ForkParams& p, int b, int lane) {
    int full;
    if (fresh_pages(p, b, &full) + full > p.out_cols) return;
    const int32_t* prompt = p.pages + __ldg(p.req + static_cast<long long>(b) * kReqFields + kReqPageOff);
    int n = 0;
    for (int j = lane; j < p.num_forks; j += 32) n += p.base[b * p.num_forks + j] >= 0;
    n = __reduce_add_sync(kFull, n);
    for (int c = lane; n > 0 && c < full; c += 32) {
        const int page = __ldg(prompt + c);
        if (static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages)) atomicAdd(p.refs_out + page, n);
    }
}

// Fork: one cluster (or CTA). The rows' needs are summed in order, row i = b * num_forks + j, into base[i] (-1: a row
// without a beam, or one for which the free pages do not suffice); the free pages, lowest first, are listed as far as
// they are needed. Where the rows are few (`whole`) it goes on to their tables, else fork_tables_kernel does.
// A few passes over one int per page and per row, bound by their latency: 9 us for 1920 rows of 64 requests.
template <int CTAS>
__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(kScanThreads)
    fork_scan_kernel(const ForkParams p, bool whole) {
    __shared__ int s_warp[33], s_free, s_need;
    constexpr int PER = kCounts<CTAS>;
    const int rank = scan_rank<CTAS>(), tid = threadIdx.x;
    const bool ok = plan_matches(p.plan_hdr, p.shape);
    if (!ok) {
        if (tid == 0 && rank == 0) atomicOr(p.status, BSP_DEVFLAG_GRAPH);
        return;  // (uniform in the cluster)
    }
    int lo, hi, rlo, rhi;
    share_of<CTAS>(p.num_pages, rank, &lo, &hi);
    share_of<CTAS>(p.rows, rank, &rlo, &rhi);
    int free = 0, need = 0, full;
    // a thread's counts of the share's first round are kept for the second pass
    int first[PER];
    for (int i0 = lo; i0 < hi; i0 += PER * kScanThreads) {
        const int i = i0 + PER * tid;
        int r[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            r[e] = i + e < hi ? p.refs_in[i + e] : 1;
            free += r[e] == 0;
            if (i0 == lo) first[e] = r[e];
        }
        if (p.refs_out != p.refs_in) {
#pragma unroll
            for (int e = 0; e < PER; ++e)
                if (i + e < hi) p.refs_out[i + e] = r[e];
        }
    }
    for (int i = rlo + tid; i < rhi; i += kScanThreads) {
        const int b = i / p.num_forks;
        if (valid_beam(p, b, i - b * p.num_forks) >= 0) need += fresh_pages(p, b, &full);
    }
    free = cta_sum(free, s_warp);
    need = cta_sum(need, s_warp);
    if (tid == 0) {
        s_free = free;
        s_need = need;
    }
    scan_sync<CTAS>();
    int available, wanted;
    int at = cluster_sum<CTAS>(&s_free, &available);
    int row_at = cluster_sum<CTAS>(&s_need, &wanted);
    for (int i0 = rlo; i0 < rhi; i0 += kScanThreads) {
        const int i = i0 + tid;
        int n = 0, total;
        bool on = false;
        if (i < rhi) {
            const int b = i / p.num_forks;
            on = valid_beam(p, b, i - b * p.num_forks) >= 0;
            if (on) n = fresh_pages(p, b, &full);
        }
        const int base = row_at + cta_scan(n, s_warp, &total);
        if (i < rhi) {
            const bool served = on && base + n <= available;
            if (on && !served) atomicOr(p.status, BSP_DEVFLAG_PAGES);
            p.base[i] = served ? base : -1;
        }
        row_at += total;
    }
    const int most = min(wanted, available);  // (pages listed beyond the last served row's stay free)
    for (int i0 = lo; i0 < hi && at < most; i0 += PER * kScanThreads) {
        const int i = i0 + PER * tid;
        int n = 0, total;
        bool f[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            f[e] = (i0 == lo ? first[e] : i + e < hi ? p.refs_in[i + e] : 1) == 0;
            n += f[e];
        }
        int k = at + cta_scan(n, s_warp, &total);
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            if (f[e]) {
                if (k < most) p.fresh[k] = i + e;
                ++k;
            }
        }
        at += total;
    }
    scan_sync<CTAS>();  // base, fresh and the counts are complete, and no CTA leaves while another reads its sums
    if (!whole) return;
    const int warps = CTAS * kScanThreads / 32, lane = tid & 31;
    for (int x = rank * (kScanThreads / 32) + (tid >> 5); x < p.rows + p.batch; x += warps) {
        if (x < p.rows) fork_row_table(p, x, lane, 32);
        else fork_request_refs(p, x - p.rows, lane);
    }
}

// A warp per row writes its table and takes its fresh pages; a warp per request counts its forks and adds them to the
// references of the full prompt pages.
__global__ void __launch_bounds__(256) fork_tables_kernel(const ForkParams p) {
    if (!plan_matches(p.plan_hdr, p.shape)) return;  // (flagged by the scan)
    const int lane = threadIdx.x & 31;
    const int x = static_cast<int>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (x < p.rows) fork_row_table(p, x, lane, 32);
    else if (x < p.rows + p.batch) fork_request_refs(p, x - p.rows, lane);
}

// 8 E4M3 codes times a power of two, rounded to the nearest code
__device__ __forceinline__ uint2 rescale8(uint2 v, float mul) {
    const uint32_t two[4] = {v.x & 0xffffu, v.x >> 16, v.y & 0xffffu, v.y >> 16};
    uint32_t q[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two[e]), __NV_E4M3);
        const float2 u = __half22float2(*reinterpret_cast<const __half2*>(&hr));
        q[e] = __nv_cvt_float2_to_fp8x2(make_float2(u.x * mul, u.y * mul), __NV_SATFINITE, __NV_E4M3);
    }
    return make_uint2((q[0] & 0xffffu) | (q[1] << 16), (q[2] & 0xffffu) | (q[3] << 16));
}

// The rows of one forked row's fresh pages: a CTA per (row, fresh page, group of heads). The slots' source rows (the
// page of the prompt's last rows, then the tail's through the indirection) are resolved into shared memory, then the
// CTA's threads copy K and V, 16 bytes a thread and four in flight.
// Bound by the rows' traffic, 2 x (K, V) x row bytes: 1920 forks of 8 heads x 128 in 16 bits 44 us, 60 a call with the
// tables before them (50 for the bytes); 80 with divisions in place of the shifts and the product below.
// SCALES: blocks of the fresh page take the largest exponent among their rows' blocks, and rows of a smaller one are
// brought to it; blocks without rows are cleared.
template <bool SCALES>
__global__ void __launch_bounds__(256) fork_rows_kernel(const ForkRowsParams p) {
    __shared__ int s_src[128];  // source page of a slot, -1: none
    __shared__ uint8_t s_exp[2][8][128], s_new[2][8][128];
    const int i = static_cast<int>(blockIdx.x / p.per_row);
    const int of = static_cast<int>(blockIdx.x - static_cast<unsigned>(i) * p.per_row);
    const int k = of & 1, h0 = (of >> 1) * p.heads;  // fresh page of the row, first head
    const int tid = threadIdx.x, ps = 1 << p.ps_log2;
    if (!plan_matches(p.plan_hdr, p.shape)) {
        if (tid == 0 && blockIdx.x == 0) atomicOr(p.status, BSP_DEVFLAG_GRAPH);
        return;
    }
    const int b = i / p.num_forks;
    const int32_t* rec = p.req + static_cast<long long>(b) * kReqFields;
    const int P = __ldg(rec + kReqPrefix), T = __ldg(rec + kReqTail);
    const int col = (P >> p.ps_log2) + k, first = col << p.ps_log2;
    const int n = min(ps, P + T - first);  // rows of the page
    if (n <= 0) return;
    // a replayed plan that outgrew the tables
    if (col >= p.out_cols || (T > 0 && (P + T > p.max_seq || col >= p.beam_cols))) {
        if (tid == 0) atomicOr(p.status, BSP_DEVFLAG_GRAPH);
        return;
    }
    const int to = p.pages_out[static_cast<long long>(i) * p.out_stride + col];
    const int w = __ldg(p.beams + b * p.beams_stride + (i - b * p.num_forks));
    if (to < 0 || w < 0 || w >= p.W) return;  // a row without a beam or without pages
    if (to >= p.num_pages) {
        if (tid == 0) atomicOr(p.status, BSP_DEVFLAG_PAGE_INDEX);
        return;
    }
    for (int s = tid; s < n; s += 256) {
        const int pos = first + s;
        int page = -1;
        if (pos < P) {
            page = __ldg(p.pages + __ldg(rec + kReqPageOff) + col);
        } else {
            const int src = __ldg(p.ci + (static_cast<long long>(b) * p.W + w) * p.max_seq + pos);
            if (static_cast<unsigned>(src) < static_cast<unsigned>(p.W))
                page = __ldg(p.beam_pages + (static_cast<long long>(b) * p.W + src) * p.beam_cols + col);
        }
        if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.num_pages)) {
            atomicOr(p.status, BSP_DEVFLAG_PAGE_INDEX);
            page = -1;
        }
        s_src[s] = page;
    }
    __syncthreads();
    const int heads = min(p.heads, p.Hkv - h0);
    if constexpr (SCALES) {
        // per (tensor, head): the slots' exponents and, a warp at a time, their blocks' largest
        const int lane = tid & 31;
        for (int x = tid >> 5; x < 2 * heads; x += 8) {
            const int t = x / heads, h = x - t * heads;
            uint8_t* exps = t ? p.v_exp : p.k_exp;
            for (int s = lane; s < max(ps, 32); s += 32) {
                int e = 0;
                if (s < n && s_src[s] >= 0)
                    e = exps[(((static_cast<long long>(s_src[s]) * p.Hkv + h0 + h) << p.ps_log2) + s) >> p.block_log2];
                if (e != 0) e = min(max(e, p.read_lo), p.read_hi);  // (as the attention reads it)
                int m = e;
                for (int o = 1; o < 1 << p.block_log2; o <<= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
                if (s < ps) {
                    s_exp[t][h][s] = static_cast<uint8_t>(e);
                    s_new[t][h][s] = static_cast<uint8_t>(m);
                }
            }
        }
        // (a fresh page is no other row's source: its exponents may be written at once)
        __syncthreads();
        for (int x = tid; x < 2 * heads * (ps >> p.block_log2); x += 256) {
            const int blocks = ps >> p.block_log2, t = x / (heads * blocks);
            const int y = x - t * heads * blocks, h = y / blocks, q = y - h * blocks;
            const long long row = (static_cast<long long>(to) * p.Hkv + h0 + h) << (p.ps_log2 - p.block_log2);
            (t ? p.v_exp : p.k_exp)[row + q] = s_new[t][h][q << p.block_log2];
        }
    }
    const int cl2 = __ffs(p.row_bytes) - 5, chunks = 1 << cl2;  // 16-byte chunks of a row
    const int total = 2 * heads * n * chunks;
    // y / n for y < 2 * 8 * 128 as a product: y (n - 1) < 2^20
    const uint32_t inv = ((1u << 20) + n - 1) / n;
    // (below 2^31: 128 slots of 512 bytes, and heads to match)
    const int page_bytes = (p.Hkv << p.ps_log2) * p.row_bytes;
    const int first_off = ((h0 << p.ps_log2) * p.row_bytes), row_bytes = p.row_bytes;
    for (int x0 = tid; x0 < total; x0 += 4 * 256) {
        uint4 v[4];
        int off[4], at[4];  // bytes from a page's start (-1: nothing to copy), place in the exponents' tables
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int x = x0 + u * 256;
            off[u] = -1;
            if (x >= total) continue;
            const int c = x & (chunks - 1), y = x >> cl2;  // y: (tensor, head, slot)
            const int z = static_cast<int>((static_cast<uint32_t>(y) * inv) >> 20), s = y - z * n;
            const int t = z >= heads, h = t ? z - heads : z;
            const int src = s_src[s];
            if (src < 0) continue;
            off[u] = first_off + ((h << p.ps_log2) + s) * row_bytes + 16 * c;
            at[u] = (t * 8 + h) * 128 + s;
            const uint8_t* pool = t ? p.v_pool : p.k_pool;
            v[u] = *reinterpret_cast<const uint4*>(pool + static_cast<long long>(src) * page_bytes + off[u]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (off[u] < 0) continue;
            if constexpr (SCALES) {
                const int eo = (&s_exp[0][0][0])[at[u]], en = (&s_new[0][0][0])[at[u]];
                if (eo != en) {
                    const uint32_t ratio = static_cast<uint32_t>(max(1, 127 + eo - en)) << 23;
                    const float mul = eo == 0 ? 0.f : __uint_as_float(ratio);
                    const uint2 lo = rescale8(make_uint2(v[u].x, v[u].y), mul);
                    const uint2 hi = rescale8(make_uint2(v[u].z, v[u].w), mul);
                    v[u] = make_uint4(lo.x, lo.y, hi.x, hi.y);
                }
            }
            uint8_t* pool = at[u] >= 8 * 128 ? p.v_pool : p.k_pool;
            *reinterpret_cast<uint4*>(pool + static_cast<long long>(to) * page_bytes + off[u]) = v[u];
        }
    }
}

// One reference less for the page of entry x of the tables. A page whose count would fall below zero keeps zero and is
// flagged.
__device__ __forceinline__ void free_entry(const FreeParams& p, long long x) {
    const long long r = x / p.cols;
    const int page = __ldg(p.tables + r * p.stride + (x - r * p.cols));
    if (page == -1) return;
    if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.num_pages)) {
        atomicOr(p.status, BSP_DEVFLAG_PAGE_INDEX);
    } else if (atomicSub(p.refs_out + page, 1) <= 0) {
        atomicAdd(p.refs_out + page, 1);
        atomicOr(p.status, BSP_DEVFLAG_PAGE_INDEX);
    }
}
__global__ void __launch_bounds__(256) free_pages_kernel(const FreeParams p) {
    const long long total = static_cast<long long>(p.rows) * p.cols;
    const long long step = static_cast<long long>(gridDim.x) * 256;
    for (long long x = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; x < total; x += step)
        free_entry(p, x);
}
// The same for few pages and entries, with the copy of the counts before it: one cluster (or CTA).
template <int CTAS>
__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(kScanThreads)
    free_few_kernel(const FreeParams p, const int32_t* refs_in) {
    const int at = static_cast<int>(blockIdx.x * kScanThreads + threadIdx.x);
    for (int i = at; i < p.num_pages; i += CTAS * kScanThreads) p.refs_out[i] = refs_in[i];
    scan_sync<CTAS>();
    const int total = p.rows * p.cols;
    for (int x = at; x < total; x += CTAS * kScanThreads) free_entry(p, x);
}

// The new id of entry x of the tables. -1 and entries outside the pool are copied as they are.
__device__ __forceinline__ void remap_entry(const CompactParams& p, long long x) {
    const long long r = x / p.cols, c = x - r * p.cols;
    const int page = p.tables_in[r * p.stride + c];
    const bool inside = static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages);
    if (!inside && page != -1) atomicOr(p.status, BSP_DEVFLAG_PAGE_INDEX);
    p.tables_out[r * p.stride + c] = inside ? p.remap[page] : page;
}

// Compaction: one cluster (or CTA), which goes on to the tables where they are short (`whole`). L pages are live; the
// i-th live page with an id of at least L goes to the i-th free page below L. With before(p) the live pages below p, a
// free page p < L is hole p - before(p), and a live page p >= L is mover before(p) - before(L): one running count
// ranks both.
// Bound by its latency, two sums and a scan: 3.3 us for 96 pages on one CTA, 8.5 for 8192 on the cluster.
template <int CTAS>
__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(kScanThreads)
    compact_scan_kernel(const CompactParams p, bool whole) {
    __shared__ int s_warp[33], s_live, s_front;
    constexpr int PER = kCounts<CTAS>;
    const int rank = scan_rank<CTAS>(), tid = threadIdx.x;
    int lo, hi;
    share_of<CTAS>(p.num_pages, rank, &lo, &hi);
    int live = 0, kept[PER] = {};  // a thread's counts of the share's first round stay for the later passes
    for (int i0 = lo; i0 < hi; i0 += PER * kScanThreads) {
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int i = i0 + PER * tid + e, r = i < hi ? p.refs_in[i] : 0;
            live += r > 0;
            if (i0 == lo) kept[e] = r;
        }
    }
    live = cta_sum(live, s_warp);
    if (tid == 0) s_live = live;
    scan_sync<CTAS>();
    int L;
    int at = cluster_sum<CTAS>(&s_live, &L);
    int front = 0;  // of the CTA's live pages, those below L
    for (int i0 = lo; i0 < min(hi, L); i0 += PER * kScanThreads) {
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int i = i0 + PER * tid + e;
            if (i < min(hi, L)) front += (i0 == lo ? kept[e] : p.refs_in[i]) > 0;
        }
    }
    front = cta_sum(front, s_warp);
    if (tid == 0) s_front = front;
    scan_sync<CTAS>();
    int A;  // before(L)
    cluster_sum<CTAS>(&s_front, &A);
    for (int i0 = lo; i0 < hi; i0 += PER * kScanThreads) {
        const int i = i0 + PER * tid;
        int n = 0, total;
        int r[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            r[e] = i0 == lo ? kept[e] : i + e < hi ? p.refs_in[i + e] : 0;
            n += r[e] > 0;
        }
        int before = at + cta_scan(n, s_warp, &total);
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int page = i + e;
            if (page < hi) {
                p.remap[page] = page;
                if (p.refs_out != p.refs_in) p.refs_out[page] = max(r[e], 0);
                if (r[e] > 0) {
                    if (page >= L) p.pairs[2ll * (before - A)] = page;
                    ++before;
                } else if (page < L) {
                    p.pairs[2ll * (page - before) + 1] = page;
                }
            }
        }
        at += total;
    }
    if (rank == 0 && tid == 0) {
        p.count[0] = L - A;
        p.count[1] = L;
    }
    scan_sync<CTAS>();  // the pairs are complete, and no CTA leaves while another reads its sums
    for (int k = rank * kScanThreads + tid; k < L - A; k += CTAS * kScanThreads) {
        const int from = p.pairs[2ll * k], to = p.pairs[2ll * k + 1];
        p.remap[from] = to;
        p.refs_out[to] = p.refs_in[from];
        p.refs_out[from] = 0;
    }
    if (!whole) return;  // (uniform)
    scan_sync<CTAS>();  // remap is complete
    for (int x = rank * kScanThreads + tid; x < p.rows * p.cols; x += CTAS * kScanThreads) remap_entry(p, x);
}

// The entries of longer tables.
__global__ void __launch_bounds__(256) remap_tables_kernel(const CompactParams p) {
    const long long total = static_cast<long long>(p.rows) * p.cols;
    const long long step = static_cast<long long>(gridDim.x) * 256;
    for (long long x = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; x < total; x += step)
        remap_entry(p, x);
}

// Pages copied pair by pair, (from, to), K and V and their exponents. CTAs share the 16-byte vectors of all pages in
// parts of kPart: loads of a part are in flight together, and the stores follow.
// Bound by the pages' traffic, 2 x (K, V) x page bytes: 1500 pages of 128 KB moved in 57 us, 6.8 TB/s.
constexpr int kPart = 256 * 8;  // vectors

__global__ void __launch_bounds__(256) copy_pages_kernel(const CopyParams p) {
    const int n = min(max(__ldg(p.count), 0), p.max_pairs);
    const int tid = threadIdx.x;
    const long long vectors = p.page_bytes >> 4;
    const long long parts = (vectors + kPart - 1) / kPart;
    const long long total = 2 * parts * n;
    for (long long x = blockIdx.x; x < total; x += gridDim.x) {
        const long long pair = x / (2 * parts);
        const int y = static_cast<int>(x - pair * 2 * parts);
        const bool is_v = y >= parts;
        const long long part = is_v ? y - parts : y;
        const int from = __ldg(p.pairs + 2 * pair), to = __ldg(p.pairs + 2 * pair + 1);
        if (static_cast<unsigned>(from) >= static_cast<unsigned>(p.num_pages) ||
            static_cast<unsigned>(to) >= static_cast<unsigned>(p.num_pages)) {
            if (tid == 0 && (from != -1 || to != -1)) atomicOr(p.status, BSP_DEVFLAG_PAGE_INDEX);
            continue;
        }
        uint8_t* pool = is_v ? p.v_pool : p.k_pool;
        const uint4* src = reinterpret_cast<const uint4*>(pool + from * p.page_bytes);
        uint4* dst = reinterpret_cast<uint4*>(pool + to * p.page_bytes);
        const long long v0 = part * kPart + tid;
        uint4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (v0 + 256 * u < vectors) v[u] = __ldcs(src + v0 + 256 * u);
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (v0 + 256 * u < vectors) __stcs(dst + v0 + 256 * u, v[u]);
        if (part == 0 && p.exp_bytes) {
            uint8_t* exps = is_v ? p.v_exp : p.k_exp;
            for (int e = tid; e < p.exp_bytes; e += 256)
                exps[static_cast<long long>(to) * p.exp_bytes + e] =
                    exps[static_cast<long long>(from) * p.exp_bytes + e];
        }
    }
}

unsigned grid_for(long long items, int sms) {
    const long long n = (items + 255) / 256;
    return static_cast<unsigned>(n < 1 ? 1 : n < 8ll * sms ? n : 8ll * sms);
}

}  // namespace

cudaError_t launch_fork_tables(const ForkParams& p, cudaStream_t stream) {
    // up to four rows (or requests) for each of the scan's warps: one launch instead of two (two beams of one
    // request forked, rows too, 24.6 -> 18.3 us a call); 1920 rows are served better by a grid of their own
    const int all = p.rows + p.batch, warps = kScanThreads / 32;
    const bool small = p.num_pages <= kSmallPool && all <= 4 * warps, whole = all <= 4 * kScanCtas * warps;
    if (small) fork_scan_kernel<1><<<1, kScanThreads, 0, stream>>>(p, true);
    else fork_scan_kernel<kScanCtas><<<kScanCtas, kScanThreads, 0, stream>>>(p, whole);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || whole) return e;
    fork_tables_kernel<<<(p.rows + p.batch + 7) / 8, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_fork_rows(ForkRowsParams p, int num_sms, cudaStream_t stream) {
    // A CTA takes up to 8 heads of a fresh page; fewer while all CTAs are resident at once
    p.heads = p.Hkv < 8 ? p.Hkv : 8;
    auto per_row = [&] { return 2 * ((p.Hkv + p.heads - 1) / p.heads); };
    while (p.heads > 1 && static_cast<long long>(p.rows) * per_row() * 2 <= 8ll * num_sms) p.heads = (p.heads + 1) / 2;
    p.per_row = per_row();
    const long long ctas = static_cast<long long>(p.rows) * p.per_row;
    if (ctas > INT32_MAX) return cudaErrorInvalidValue;
    if (p.k_exp) fork_rows_kernel<true><<<static_cast<unsigned>(ctas), 256, 0, stream>>>(p);
    else fork_rows_kernel<false><<<static_cast<unsigned>(ctas), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_free_pages(const FreeParams& p, const int32_t* refs_in, int num_sms, cudaStream_t stream) {
    const long long total = static_cast<long long>(p.rows) * p.cols;
    // eight for each of the cluster's threads: one launch instead of a copy and a kernel (freed and compacted, 96
    // pages: 28.3 -> 21.3 us)
    const int few = 8 * kScanCtas * kScanThreads;
    if (refs_in != p.refs_out && p.num_pages <= few && total <= few) {
        if (p.num_pages <= kSmallPool && total <= 8 * kScanThreads)
            free_few_kernel<1><<<1, kScanThreads, 0, stream>>>(p, refs_in);
        else
            free_few_kernel<kScanCtas><<<kScanCtas, kScanThreads, 0, stream>>>(p, refs_in);
        return cudaGetLastError();
    }
    if (refs_in != p.refs_out) {
        const cudaError_t e = cudaMemcpyAsync(p.refs_out, refs_in, static_cast<size_t>(p.num_pages) * 4,
                                              cudaMemcpyDeviceToDevice, stream);
        if (e != cudaSuccess) return e;
    }
    if (total == 0) return cudaSuccess;
    free_pages_kernel<<<grid_for(total, num_sms), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_compact_tables(const CompactParams& p, int num_sms, cudaStream_t stream) {
    const long long total = static_cast<long long>(p.rows) * p.cols;
    // (eight entries for each of the scan's threads)
    const bool small = p.num_pages <= kSmallPool && total <= 8 * kScanThreads;
    const bool whole = total <= 8 * kScanCtas * kScanThreads;
    if (small) compact_scan_kernel<1><<<1, kScanThreads, 0, stream>>>(p, true);
    else compact_scan_kernel<kScanCtas><<<kScanCtas, kScanThreads, 0, stream>>>(p, whole);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || whole) return e;
    remap_tables_kernel<<<grid_for(total, num_sms), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_copy_pages(const CopyParams& p, int num_sms, cudaStream_t stream) {
    const long long parts = 2 * ((p.page_bytes / 16 + kPart - 1) / kPart) * p.max_pairs;
    const long long most = 4ll * num_sms;
    copy_pages_kernel<<<static_cast<unsigned>(parts < most ? parts : most), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace bsp
