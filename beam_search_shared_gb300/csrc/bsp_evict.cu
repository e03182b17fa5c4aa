// Eviction from a request's cached rows (bsp_evict_prefix): per (request, kv head) the keep_b rows of highest
// weight stay; those of them that stand behind the first keep_b slots move into the evicted slots before
// them, in place.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/bsp.h"
#include "bsp_internal.h"
#include "bsp_topk.cuh"

namespace bsp {
namespace {

constexpr int kPickThreads = 1024;
constexpr int kMoveThreads = 256;

// One CTA per (request, kv head). The keep-th best key by narrowing ranges (bsp_topk.cuh), then a bitmap of
// the kept slots in shared memory with running counts per word: the r-th evicted slot before keep takes
// the r-th kept row behind it, found by a binary search of the counts, so nothing is sorted and nothing
// is written but `kept`.
__global__ void __launch_bounds__(kPickThreads) evict_select_kernel(const EvictParams p) {
    extern __shared__ uint32_t s_dyn[];  // [3][words]: kept bits, movers before the word, holes before it
    __shared__ TopkScratch<kPickThreads> s_top;
    __shared__ int s_warp[2][32];
    __shared__ int s_max;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.x, b = blockIdx.y;
    if (!plan_matches(p.plan_hdr, p.batch, p.plan_w, p.plan_kind)) {
        if (tid == 0 && h == 0 && b == 0) atomicOr(p.status, BSP_DEVFLAG_GRAPH);
        return;
    }
    const int P = __ldg(p.req + static_cast<long long>(b) * kReqFields + kReqPrefix);
    const int T = __ldg(p.req + static_cast<long long>(b) * kReqFields + kReqTail);
    if (P > p.max_keys || T > 0) {  // a replayed plan that outgrew the tables, or that has tail rows
        if (tid == 0 && h == 0) atomicOr(p.status, BSP_DEVFLAG_GRAPH);
        return;
    }
    const int keep = max(0, min(__ldg(p.keep + b), P));
    if (keep == 0) return;
    const long long head = static_cast<long long>(b) * p.Hkv + h;
    const float* wt = p.weights + head * p.stride;
    const int32_t* pos = p.positions ? p.positions + head * p.stride : nullptr;
    int32_t* kept = p.kept + head * p.out_stride;

    int last = P - 1;  // the last position held
    if (pos) {
        if (tid == 0) s_max = INT32_MIN;
        __syncthreads();
        int m = INT32_MIN;
        for (int i = tid; i < P; i += kPickThreads) m = max(m, __ldg(pos + i));
        m = __reduce_max_sync(~0u, m);
        if (lane == 0) atomicMax(&s_max, m);
        __syncthreads();
        last = s_max;
    }
    const long long recent0 = static_cast<long long>(last) + 1 - p.recent;
    auto key = [&](int i) -> uint64_t {
        const int at = pos ? __ldg(pos + i) : i;
        const float w = __ldg(wt + i);
        const uint32_t o = at < p.sinks || at >= recent0 ? ~0u : isnan(w) ? 0u : float_order(w);
        return (static_cast<uint64_t>(o) << 32) | static_cast<uint32_t>(~i);
    };
    const uint64_t edge = keep < P ? topk_threshold<kPickThreads>(P, keep, 0, s_top, key) : 0;

    uint32_t* s_kept = s_dyn;
    const int words = (P + 31) >> 5;
    int* s_mov = reinterpret_cast<int*>(s_dyn + words);
    int* s_hol = s_mov + words;
    for (int i0 = warp * 32; i0 < P; i0 += kPickThreads) {
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
    // exclusive running counts over the words, a contiguous run of words per thread
    const int per = (words + kPickThreads - 1) / kPickThreads;
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
    __syncthreads();
    for (int i = tid; i < keep; i += kPickThreads) {
        const int w = i >> 5, bit = i & 31;
        int from = i;
        if (!((s_kept[w] >> bit) & 1u)) {
            const int r = s_hol[w] + __popc(~s_kept[w] & ((1u << bit) - 1));
            // the last word with at most r movers before it holds mover r (as many movers as holes)
            int lo = 0, hi2 = words - 1;
            while (lo < hi2) {
                const int mid = (lo + hi2 + 1) >> 1;
                if (s_mov[mid] <= r) lo = mid; else hi2 = mid - 1;
            }
            const uint32_t m = s_kept[lo] & ~front(lo);
            from = 32 * lo + __fns(m, 0, r - s_mov[lo] + 1);
        }
        kept[i] = from;
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Moves the K and V rows that `kept` names (and gathers weights and positions with them): a warp takes 32
// consecutive slots, reads their sources and page ids with one lane each, and copies the rows of the slots
// that change, 16 bytes a lane. Sources stand at or behind keep and targets before it, so the order of the
// copies does not matter. Bound by the scattered rows' traffic: 2 x (K, V) x row bytes for each.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!plan_matches(p.plan_hdr, p.batch, p.plan_w, p.plan_kind)) return;
    const int lane = threadIdx.x & 31;
    const int tiles = (p.max_keys + 31) >> 5;  // per (request, kv head)
    const long long total = static_cast<long long>(p.batch) * p.Hkv * tiles;
    const long long warps = static_cast<long long>(gridDim.x) * (kMoveThreads / 32);
    const int chunks = p.row_bytes >> 4;       // 16-byte chunks of a row: 4, 8, 16 or 32
    const int two = 2 * chunks;                // of a slot's K and V rows
    const int per = 32 / min(32, two);         // slots one pass of the warp copies
    const int ps_mask = (1 << p.ps_log2) - 1;
    for (long long t = static_cast<long long>(blockIdx.x) * (kMoveThreads / 32) + (threadIdx.x >> 5); t < total; t += warps) {
        const long long head = t / tiles;
        const int i0 = static_cast<int>(t - head * tiles) * 32, i = i0 + lane;
        const int b = static_cast<int>(head / p.Hkv), h = static_cast<int>(head - static_cast<long long>(b) * p.Hkv);
        const int32_t* rec = p.req + static_cast<long long>(b) * kReqFields;
        const int P = __ldg(rec + kReqPrefix);
        if (P > p.max_keys || __ldg(rec + kReqTail) > 0) continue;
        const int keep = max(0, min(__ldg(p.keep + b), P));
        if (i0 >= keep) continue;
        const int from = i < keep ? __ldcg(p.kept + head * p.out_stride + i) : i;
        if (i < keep) {
            if (p.weights_out) p.weights_out[head * p.out_stride + i] = p.weights[head * p.stride + from];
            if (p.positions_out)
                p.positions_out[head * p.out_stride + i] = p.positions ? p.positions[head * p.stride + from] : from;
        }
        long long src = 0, dst = 0;  // byte offsets of the rows in either pool
        const bool moves = from != i;
        if (moves) {
            const int32_t* pages = p.pages + __ldg(rec + kReqPageOff);
            src = (((static_cast<long long>(__ldg(pages + (from >> p.ps_log2))) * p.Hkv + h) << p.ps_log2) + (from & ps_mask)) * p.row_bytes;
            dst = (((static_cast<long long>(__ldg(pages + (i >> p.ps_log2))) * p.Hkv + h) << p.ps_log2) + (i & ps_mask)) * p.row_bytes;
        }
        const uint32_t todo = __ballot_sync(~0u, moves);
        const int n = __popc(todo);
        for (int k0 = 0; k0 < n; k0 += 4 * per) {
            uint4 val[8];
            long long to[8];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int k = k0 + u * per + (two >= 32 ? 0 : lane / two);
                const int bit = k < n ? __fns(todo, 0, k + 1) : 0;
                const long long s = __shfl_sync(~0u, src, bit), d = __shfl_sync(~0u, dst, bit);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int c = (two >= 32 ? lane : lane % two) + 32 * q;
                    to[2 * u + q] = -1;
                    if (k < n && c < two) {
                        const bool is_v = c >= chunks;
                        const int at = (is_v ? c - chunks : c) * 16;
                        val[2 * u + q] = __ldcs(reinterpret_cast<const uint4*>((is_v ? p.v_pool : p.k_pool) + s + at));
                        to[2 * u + q] = d + at;
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int c = (two >= 32 ? lane : lane % two) + 32 * (u & 1);
                if (to[u] >= 0) *reinterpret_cast<uint4*>((c >= chunks ? p.v_pool : p.k_pool) + to[u]) = val[u];
            }
        }
    }
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, int num_sms, cudaStream_t stream) {
    const size_t smem = static_cast<size_t>((p.max_keys + 31) >> 5) * 12;
    cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    evict_select_kernel<<<dim3(p.Hkv, p.batch), kPickThreads, smem, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const long long tiles = static_cast<long long>(p.batch) * p.Hkv * ((p.max_keys + 31) >> 5);
    const long long blocks = (tiles + kMoveThreads / 32 - 1) / (kMoveThreads / 32);
    if (blocks == 0) return cudaSuccess;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks < 8ll * num_sms ? blocks : 8ll * num_sms));
    cfg.blockDim = dim3(kMoveThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, evict_move_kernel, p);
}

}  // namespace bsp
