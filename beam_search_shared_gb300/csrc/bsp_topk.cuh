// The K largest of n distinct 64-bit keys, by one CTA.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace bsp {

// Order of fp32 values as unsigned integers (-0 counts as +0; NaN is the caller's to leave out), and back.
__device__ __forceinline__ uint32_t float_order(float v) {
    const uint32_t u = __float_as_uint(__fadd_rn(v, 0.f));
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float order_float(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

constexpr int kTopkBins = 1024;  // 32 x 32, so that two warp scans find a bin
// Up to so many keys are ranked against one another at once, without the histogram (a selection of K = 8 over 4 x 50257
// logits: up to 64, 128, 256 keys 11.6, 11.0, 11.6 us, never 14.0; K = 192 over 96 x 32000, 128 requests, masked: 212,
// 212, 217 and 212).
constexpr int kTopkRanked = 128;

template <int NT>
struct TopkScratch {
    uint32_t hist[kTopkBins];
    uint32_t coarse[32];
    uint64_t list[NT];
    uint64_t lo[NT / 32], hi[NT / 32];
    uint64_t range_lo, range_hi;  // the K-th largest key lies in [range_lo, range_hi]
    int need;                     // how many of the keys in it are wanted
    int state;                    // 0: narrow further, 1: found, 2: few enough to rank
    int count, listed;
};

// One bin per lane, higher lanes holding larger keys: the lane in which the count from above, which begins at
// `above`, reaches `need`. `above` becomes the count of the lanes behind it.
__device__ __forceinline__ int find_bin(uint32_t mine, uint32_t need, uint32_t& above) {
    const int lane = threadIdx.x & 31;
    uint32_t incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_down_sync(~0u, incl, d);
        if (lane + d < 32) incl += o;
    }
    const uint32_t ok = __ballot_sync(~0u, above + incl >= need);
    const int l = ok ? 31 - __clz(ok) : 0;
    above += __shfl_sync(~0u, incl - mine, l);
    return l;
}

// The K-th largest of the keys key(0) .. key(n - 1), which are distinct; 0 is no key, and K >= 1 of them are
// others. All NT threads call it, after a barrier if key() reads shared memory; key(i) may be evaluated
// several times. The keys of the present range are counted in 1024 bins, and the bin that holds the K-th
// largest becomes the range: if its lower edge has K to K + slack keys at or above it, the edge is the answer;
// if it holds at most NT keys they are ranked against one another; else the bin is divided again. Scattered keys
// take one pass to count and one to rank.
template <int NT, typename Key>
__device__ uint64_t topk_threshold(int n, int K, int slack, TopkScratch<NT>& s, Key key) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int NW = NT / 32;
    static_assert(kTopkRanked <= NT, "the keys ranked at once");
    if (n <= kTopkRanked) {
        if (tid < n) s.list[tid] = key(tid);
        __syncthreads();
        if (tid < n) {
            const uint64_t k = s.list[tid];
            int larger = 0;
#pragma unroll 8
            for (int j = 0; j < n; ++j) larger += s.list[j] > k;
            if (larger == K - 1) s.range_lo = k;  // (no absent one: at least K keys are larger than those)
        }
        __syncthreads();
        const uint64_t t = s.range_lo;
        __syncthreads();
        return t;
    }
    uint64_t lo = ~0ull, hi = 0;
    for (int i = tid; i < n; i += NT) {
        const uint64_t k = key(i);
        if (k) {
            lo = k < lo ? k : lo;
            hi = k > hi ? k : hi;
        }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const uint64_t a = __shfl_xor_sync(~0u, lo, d), c = __shfl_xor_sync(~0u, hi, d);
        lo = a < lo ? a : lo;
        hi = c > hi ? c : hi;
    }
    if (lane == 0) {
        s.lo[warp] = lo;
        s.hi[warp] = hi;
    }
    for (int i = tid; i < kTopkBins; i += NT) s.hist[i] = 0;
    __syncthreads();
    if (warp == 0) {
        lo = lane < NW ? s.lo[lane] : ~0ull;
        hi = lane < NW ? s.hi[lane] : 0ull;
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            const uint64_t a = __shfl_xor_sync(~0u, lo, d), c = __shfl_xor_sync(~0u, hi, d);
            lo = a < lo ? a : lo;
            hi = c > hi ? c : hi;
        }
        if (lane == 0) {
            s.range_lo = lo;
            s.range_hi = hi;
            s.need = K;
            s.state = 0;
            s.listed = 0;
        }
    }
    __syncthreads();
    // (a round takes 10 bits off the range: at most 7 of them)
    for (int round = 0; round < 8; ++round) {
        const uint64_t r0 = s.range_lo, r1 = s.range_hi;
        const uint32_t need = static_cast<uint32_t>(s.need);
        const int bits = 64 - __clzll(static_cast<long long>(r1 - r0));  // (r1 - r0) >> shift < 1024
        const int shift = bits > 10 ? bits - 10 : 0;
        for (int i = tid; i < n; i += NT) {
            const uint64_t k = key(i);
            if (k >= r0 && k <= r1) atomicAdd(&s.hist[(k - r0) >> shift], 1u);
        }
        __syncthreads();
        for (int c = warp; c < 32; c += NW) {
            const uint32_t sum = __reduce_add_sync(~0u, s.hist[32 * c + lane]);
            if (lane == 0) s.coarse[c] = sum;
        }
        __syncthreads();
        if (warp == 0) {
            // the coarse bin, then the fine one, in which the count from above reaches `need`
            uint32_t above = 0;
            const int c = find_bin(s.coarse[lane], need, above);
            const int bin = 32 * c + find_bin(s.hist[32 * c + lane], need, above);
            if (lane == 0) {
                const uint32_t in = s.hist[bin];
                const uint64_t e0 = r0 + (static_cast<uint64_t>(bin) << shift), width = (1ull << shift) - 1;
                s.range_lo = e0;
                s.range_hi = r1 - e0 > width ? e0 + width : r1;  // (e0 + width may pass 2^64)
                s.need = static_cast<int>(need - above);
                s.state = above + in <= need + slack || shift == 0 ? 1 : in <= NT ? 2 : 0;
            }
        }
        __syncthreads();
        if (s.state) break;
        for (int i = tid; i < kTopkBins; i += NT) s.hist[i] = 0;
        __syncthreads();
    }
    if (s.state == 2) {
        const uint64_t r0 = s.range_lo, r1 = s.range_hi;
        for (int i = tid; i < n; i += NT) {
            const uint64_t k = key(i);
            if (k >= r0 && k <= r1) s.list[atomicAdd(&s.listed, 1)] = k;
        }
        __syncthreads();
        const int m = s.listed, need = s.need;
        if (tid < m) {
            const uint64_t k = s.list[tid];
            int larger = 0;
            for (int j = 0; j < m; ++j) larger += s.list[j] > k;
            if (larger == need - 1) s.range_lo = k;
        }
        __syncthreads();
    }
    const uint64_t t = s.range_lo;
    __syncthreads();
    return t;
}

// Moves the K to K + slack largest of the n > K keys in buf to its front (in no order); their number is left in
// s.count. Returns a key that exactly these lie above, so that further candidates must too. All NT
// threads call it after a barrier; it ends with one. (Not inlined: its callers' loops stay in the
// instruction cache.)
template <int NT>
__device__ __noinline__ uint64_t topk_compact(uint64_t* buf, int n, int K, int slack, TopkScratch<NT>& s) {
    const uint64_t edge = topk_threshold<NT>(n, K, slack, s, [&](int i) { return buf[i]; });
    const int tid = threadIdx.x, lane = tid & 31;
    if (tid == 0) s.count = 0;
    __syncthreads();
    // a round reads its NT keys before it writes the ones that stay, which number no more than were read
    for (int i0 = 0; i0 < n; i0 += NT) {
        const int i = i0 + tid;
        const uint64_t k = i < n ? buf[i] : 0;
        const bool stay = i < n && k >= edge;
        const uint32_t who = __ballot_sync(~0u, stay);
        __syncthreads();
        int first = 0;
        if (lane == 0 && who) first = atomicAdd(&s.count, __popc(who));
        first = __shfl_sync(~0u, first, 0);
        if (stay) buf[first + __popc(who & ((1u << lane) - 1))] = k;
    }
    __syncthreads();
    return edge - 1;
}

}  // namespace bsp
