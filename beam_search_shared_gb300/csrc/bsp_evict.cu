// Eviction from a request's cached rows (bsp_evict_prefix): per (request, kv head) the keep_b rows of highest
// weight stay; those of them that stand behind the first keep_b slots move into the evicted slots before
// them, in place.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/bsp.h"
#include "bsp_step.h"
#include "bsp_topk.cuh"

namespace bsp {
namespace {

// position of the n-th (from 0) set bit of m, which has more than n
__device__ __forceinline__ int nth_bit(uint32_t m, int n) {
    int at = 0;
#pragma unroll
    for (int s = 16; s; s >>= 1) {
        const int c = __popc(m & ((1u << s) - 1));
        if (n >= c) {
            n -= c;
            m >>= s;
            at += s;
        }
    }
    return at;
}

// One cluster per (request, kv head). Each of its CTAs finds the keep-th best key by narrowing ranges
// (bsp_topk.cuh; the keys' order is kept in shared memory where it fits) and a bitmap of the kept slots with
// running counts per word: the r-th evicted slot before keep takes the r-th kept row behind it, found by a
// binary search of the counts, so nothing is sorted. The choice is made by every CTA for itself, which costs a
// cluster no time; then its warps share the slots before keep, 32 at a time: a lane reads a slot's source and
// page ids, and the warp copies the rows that move, 16 bytes a lane and four slots in flight. Sources stand at
// or behind keep and targets before it, so the order of the copies does not matter; outputs that are the
// inputs are written once all CTAs of the cluster have read them.
// Bound by the scattered rows' traffic, 2 x (K, V) x row bytes each; few heads: by the passes over the keys.
// Measured, 8 kv heads, D = 128, 16 bits: batch 128, about 3000 rows cut to 1024: 161 us, 4.7 TB/s, 0.69 of what a
// copy reaches (choosing in one kernel and moving in another: 246 us); one request of 10000 rows cut to 2048: 18.4 us.
template <int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) evict_kernel(const EvictParams p) {
    extern __shared__ uint32_t s_dyn[];  // [3][words]: kept bits, movers and holes before the word; then the orders
    __shared__ TopkScratch<NT> s_top;
    __shared__ int s_warp[2][32];
    __shared__ int s_last, s_fixed;  // the last position held; protected slots
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = p.cluster;
    const long long head = blockIdx.x / C;
    const int rank = blockIdx.x % C;
    const int b = static_cast<int>(head / p.Hkv), h = static_cast<int>(head - static_cast<long long>(b) * p.Hkv);
    if (!plan_matches(p.plan_hdr, p.shape)) {
        if (tid == 0 && blockIdx.x == 0) atomicOr(p.status, BSP_DEVFLAG_GRAPH);
        return;
    }
    const int32_t* rec = p.req + static_cast<long long>(b) * kReqFields;
    const int P = __ldg(rec + kReqPrefix);
    if (P > p.max_keys || __ldg(rec + kReqTail) > 0) {  // a replayed plan that outgrew the tables, or with tail rows
        if (tid == 0 && h == 0) atomicOr(p.status, BSP_DEVFLAG_GRAPH);
        return;
    }
    const int keep = max(0, min(__ldg(p.keep + b), P));
    if (keep == 0) return;  // (uniform in the cluster, like the returns above)
    const float* wt = p.weights + head * p.stride;
    const int32_t* pos = p.positions ? p.positions + head * p.stride : nullptr;

    // ---- the keys: protected slots above all weights, NaN below them, equal weights by the lower slot
    int last = P - 1;  // the last position held
    if (tid == 0) {
        s_last = INT32_MIN;
        s_fixed = 0;
    }
    __syncthreads();
    if (pos) {
        int m = INT32_MIN;
        for (int i = tid; i < P; i += NT) m = max(m, __ldcg(pos + i));
        m = __reduce_max_sync(~0u, m);
        if (lane == 0) atomicMax(&s_last, m);
        __syncthreads();
        last = s_last;
    }
    const long long recent0 = static_cast<long long>(last) + 1 - p.recent;
    auto order = [&](int i) -> uint32_t {
        const int at = pos ? __ldcg(pos + i) : i;
        const float w = __ldcg(wt + i);
        return at < p.sinks || at >= recent0 ? ~0u : isnan(w) ? 0u : float_order(w);
    };
    const int words = (P + 31) >> 5;
    uint32_t* s_kept = s_dyn;
    int* s_mov = reinterpret_cast<int*>(s_dyn + words);
    int* s_hol = s_mov + words;
    uint32_t* s_ord = s_dyn + 3 * words;
    const bool cached = P <= p.cached_keys;
    int fixed = 0;  // protected slots
#pragma unroll 4
    for (int i = tid; i < P; i += NT) {
        const uint32_t o = order(i);
        if (cached) s_ord[i] = o;
        fixed += o == ~0u;
    }
    fixed = __reduce_add_sync(~0u, fixed);
    if (lane == 0) atomicAdd(&s_fixed, fixed);
    __syncthreads();
    fixed = s_fixed;
    auto key = [&](int i) -> uint64_t {
        return (static_cast<uint64_t>(cached ? s_ord[i] : order(i)) << 32) | static_cast<uint32_t>(~i);
    };
    // the last of the protected slots that stay, or with all of them the last of the others: apart, since bins
    // over both would leave few to the weights
    const bool among_fixed = keep <= fixed;
    uint64_t edge = 0;
    if (keep < P)
        edge = topk_threshold<NT>(P, among_fixed ? keep : keep - fixed, 0, s_top, [&](int i) -> uint64_t {
            const uint64_t k = key(i);
            return (static_cast<uint32_t>(k >> 32) == ~0u) == among_fixed ? k : 0ull;
        });

    // ---- kept slots, and the counts of movers (kept, behind keep) and holes (evicted, before it)
    for (int i0 = warp * 32; i0 < P; i0 += NT) {
        const int i = i0 + lane;
        const uint32_t bits = __ballot_sync(~0u, i < P && key(i) >= edge);
        if (lane == 0) s_kept[i0 >> 5] = bits;
    }
    __syncthreads();
    // slots of word w before keep, as a bit mask
    auto front = [&](int w) -> uint32_t {
        const int n = keep - 32 * w;
        return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1;
    };
    const int per = (words + NT - 1) / NT;
    const int w0 = min(words, tid * per), w1 = min(words, w0 + per);
    int mov = 0, hol = 0;
    for (int w = w0; w < w1; ++w) {
        mov += __popc(s_kept[w] & ~front(w));
        hol += __popc(~s_kept[w] & front(w));
    }
    int mi = mov, hi = hol;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int a = __shfl_up_sync(~0u, mi, d), c = __shfl_up_sync(~0u, hi, d);
        if (lane >= d) {
            mi += a;
            hi += c;
        }
    }
    if (lane == 31) {
        s_warp[0][warp] = mi;
        s_warp[1][warp] = hi;
    }
    __syncthreads();
    int m0 = mi - mov, h0 = hi - hol;
    for (int i = 0; i < warp; ++i) {
        m0 += s_warp[0][i];
        h0 += s_warp[1][i];
    }
    for (int w = w0; w < w1; ++w) {
        s_mov[w] = m0;
        s_hol[w] = h0;
        m0 += __popc(s_kept[w] & ~front(w));
        h0 += __popc(~s_kept[w] & front(w));
    }
    if (C > 1)
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    else
        __syncthreads();

    // ---- the slots before keep
    const int chunks = p.row_bytes >> 4;       // 16-byte chunks of a row: 4, 8, 16 or 32
    const int two = 2 * chunks;                // of a slot's K and V rows
    const int slots = 32 / min(32, two);       // slots one pass of the warp copies
    const int ps_mask = (1 << p.ps_log2) - 1;
    const int32_t* pages = p.pages + __ldg(rec + kReqPageOff);
    constexpr int NW = NT / 32;
    // more warps than groups of 32 slots: up to 8 of them share a group's copies
    const int parts = max(1, min(8, C * NW / ((keep + 31) >> 5)));
    for (int g = rank * NW + warp; 32 * (g / parts) < keep; g += C * NW) {
        const int t = g / parts, part = g - t * parts;
        const int i = 32 * t + lane;
        int from = i;
        const uint32_t bits = s_kept[t];
        if (i < keep && !((bits >> lane) & 1u)) {
            const int r = s_hol[t] + __popc(~bits & ((1u << lane) - 1));
            // the last word with at most r movers before it holds mover r (there are as many movers as holes)
            int lo = 0, hi2 = words - 1;
            while (lo < hi2) {
                const int mid = (lo + hi2 + 1) >> 1;
                if (s_mov[mid] <= r) lo = mid; else hi2 = mid - 1;
            }
            from = 32 * lo + nth_bit(s_kept[lo] & ~front(lo), r - s_mov[lo]);
        }
        if (i < keep && part == 0) {
            p.kept[head * p.out_stride + i] = from;
            if (p.weights_out) p.weights_out[head * p.out_stride + i] = __ldcg(wt + from);
            if (p.positions_out) p.positions_out[head * p.out_stride + i] = pos ? __ldcg(pos + from) : from;
        }
        long long src = 0, dst = 0;  // byte offsets of the rows in either pool
        bool moves = from != i;
        if (moves) {
            const int here = __ldg(pages + (from >> p.ps_log2)), there = __ldg(pages + (i >> p.ps_log2));
            if (max(static_cast<unsigned>(here), static_cast<unsigned>(there)) >= static_cast<unsigned>(p.num_pages)) {
                atomicOr(p.status, BSP_DEVFLAG_PAGE_INDEX);  // a replayed plan whose pools are larger: the row stays
                moves = false;
            }
            src = (((static_cast<long long>(here) * p.Hkv + h) << p.ps_log2) + (from & ps_mask)) * p.row_bytes;
            dst = (((static_cast<long long>(there) * p.Hkv + h) << p.ps_log2) + (i & ps_mask)) * p.row_bytes;
        }
        // lane k takes over the k-th slot that moves
        const uint32_t todo = __ballot_sync(~0u, moves);
        const int n = __popc(todo);
        const int of = lane < n ? nth_bit(todo, lane) : 0;
        src = __shfl_sync(~0u, src, of);
        dst = __shfl_sync(~0u, dst, of);
        for (int k0 = part * 4 * slots; k0 < n; k0 += parts * 4 * slots) {
            uint4 val[8];
            long long to[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int k = k0 + u * slots + (two >= 32 ? 0 : lane / two);
                const long long s = __shfl_sync(~0u, src, k & 31);
                to[u] = __shfl_sync(~0u, dst, k & 31);
                if (k >= n) to[u] = -1;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int c = (two >= 32 ? lane : lane % two) + 32 * q;
                    if (to[u] >= 0 && c < two)
                        val[2 * u + q] = __ldcs(reinterpret_cast<const uint4*>((c >= chunks ? p.v_pool : p.k_pool) + s) +
                                                (c >= chunks ? c - chunks : c));
                }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int c = (two >= 32 ? lane : lane % two) + 32 * q;
                    if (to[u] >= 0 && c < two)
                        reinterpret_cast<uint4*>((c >= chunks ? p.v_pool : p.k_pool) + to[u])[c >= chunks ? c - chunks : c] = val[2 * u + q];
                }
        }
    }
}

constexpr size_t kStatic = 14 * 1024;  // the kernel's other shared memory
static_assert(sizeof(TopkScratch<1024>) + 1024 <= kStatic, "shared memory of the narrowing");

template <int NT>
cudaError_t launch_t(const EvictParams& p, size_t smem, cudaStream_t stream) {
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(evict_kernel<NT>), smem, kMaxSmem - kStatic);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(p.batch) * p.Hkv * p.cluster);
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = p.cluster;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, evict_kernel<NT>, p);
}

}  // namespace

cudaError_t launch_evict(EvictParams p, int longest, int num_sms, cudaStream_t stream) {
    // the orders of the longest prompt in shared memory beside the bitmap, as far as they fit
    const size_t bitmap = static_cast<size_t>((p.max_keys + 31) >> 5) * 12;
    const size_t room = kMaxSmem - kStatic - bitmap;
    p.cached_keys = static_cast<int>(static_cast<size_t>(longest) * 4 <= room ? longest : room / 4);
    const size_t smem = bitmap + static_cast<size_t>(p.cached_keys) * 4;
    // Many (request, kv head) pairs: small CTAs, so that some choose while others move rows. Few: clusters of
    // large ones, for the passes over the keys and for the copies. 3000 rows cut to 1024, small and large CTAs:
    // 240 pairs 60 and 53 us, 304 pairs 65 and 59, 384 pairs 73 and 80, 1024 pairs 160 and 193 (600 rows cut to
    // 300: 384 pairs 26 and 35). Above 10000 rows large ones stay ahead (512 pairs 337 and 311), by less.
    const long long heads = static_cast<long long>(p.batch) * p.Hkv;
    p.cluster = 1;
    if (heads > 2ll * num_sms) return launch_t<256>(p, smem, stream);
    while (p.cluster < 8 && heads * p.cluster * 2 <= 2ll * num_sms) p.cluster *= 2;
    return launch_t<1024>(p, smem, stream);
}

}  // namespace bsp
