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

template <int NT>
struct TopkScratch {
    uint32_t hist[256];
    uint64_t lo[NT / 32], hi[NT / 32];
    uint64_t range_lo, range_hi;  // the K-th largest key lies in [range_lo, range_hi]
    int need;                     // how many of the keys in it are wanted
    int done;
    int count;
};

// The K-th largest of the n keys key(0) .. key(n - 1), n >= K >= 1, distinct. All NT threads call it; key(i)
// may be evaluated several times. Narrows a range of keys by 256 bins at a time: the bins of the present
// range are counted, and the one that holds the K-th largest becomes the range. It ends as soon as a bin's
// lower edge has K to K + slack keys at or above it, which for scattered keys and no slack takes two or three
// passes; the edge is returned.
template <int NT, typename Key>
__device__ uint64_t topk_threshold(int n, int K, int slack, TopkScratch<NT>& s, Key key) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint64_t lo = ~0ull, hi = 0;
    for (int i = tid; i < n; i += NT) {
        const uint64_t k = key(i);
        lo = k < lo ? k : lo;
        hi = k > hi ? k : hi;
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
    __syncthreads();
    if (tid == 0) {
        for (int i = 1; i < NT / 32; ++i) {
            lo = s.lo[i] < lo ? s.lo[i] : lo;
            hi = s.hi[i] > hi ? s.hi[i] : hi;
        }
        s.range_lo = lo;
        s.range_hi = hi;
        s.need = K;
        s.done = n <= K + slack;
    }
    for (int i = tid; i < 256; i += NT) s.hist[i] = 0;
    __syncthreads();
    // (a round takes 8 bits off the range: at most 8 of them)
    for (int round = 0; round < 9 && !s.done; ++round) {
        const uint64_t r0 = s.range_lo, r1 = s.range_hi;
        const int need = s.need;
        const int bits = 64 - __clzll(static_cast<long long>(r1 - r0));  // (r1 - r0) >> shift < 256
        const int shift = bits > 8 ? bits - 8 : 0;
        for (int i = tid; i < n; i += NT) {
            const uint64_t k = key(i);
            if (k >= r0 && k <= r1) atomicAdd(&s.hist[(k - r0) >> shift], 1u);
        }
        __syncthreads();
        if (warp == 0) {
            // lane l: bins 8 l .. 8 l + 7; `above`: keys in higher lanes' bins
            uint32_t c[8], sum = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                c[j] = s.hist[8 * lane + j];
                s.hist[8 * lane + j] = 0;
                sum += c[j];
            }
            uint32_t incl = sum;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t o = __shfl_down_sync(~0u, incl, d);
                if (lane + d < 32) incl += o;
            }
            uint32_t above = incl - sum;
            if (above < static_cast<uint32_t>(need) && incl >= static_cast<uint32_t>(need)) {
#pragma unroll
                for (int j = 7; j >= 0; --j) {
                    if (above < static_cast<uint32_t>(need) && above + c[j] >= static_cast<uint32_t>(need)) {
                        const uint64_t e0 = r0 + (static_cast<uint64_t>(8 * lane + j) << shift);
                        const uint64_t width = (1ull << shift) - 1;
                        s.range_lo = e0;
                        s.range_hi = r1 - e0 > width ? e0 + width : r1;  // (e0 + width may pass 2^64)
                        s.need = need - static_cast<int>(above);
                        s.done = above + c[j] <= static_cast<uint32_t>(need + slack) || shift == 0;
                        break;
                    }
                    above += c[j];
                }
            }
        }
        __syncthreads();
    }
    const uint64_t t = s.range_lo;
    __syncthreads();
    return t;
}

// Moves the K to K + slack largest of the n > K keys in buf to its front (in no order); their number is left in
// s.count. Returns a key above which every further candidate must lie: the smallest of them less one. All NT
// threads call it after a barrier; it ends with one. (Not inlined: its callers' loops stay in the
// instruction cache.)
template <int NT>
__device__ __noinline__ uint64_t topk_compact(uint64_t* buf, int n, int K, int slack, TopkScratch<NT>& s) {
    const uint64_t edge = topk_threshold<NT>(n, K, slack, s, [&](int i) { return buf[i]; });
    const int tid = threadIdx.x, lane = tid & 31;
    if (tid == 0) s.count = 0;
    __syncthreads();
    // a round reads its NT keys before it writes the ones that stay, which number no more than were read
    uint64_t least = ~0ull;
    for (int i0 = 0; i0 < n; i0 += NT) {
        const int i = i0 + tid;
        const uint64_t k = i < n ? buf[i] : 0;
        const bool stay = i < n && k >= edge;
        const uint32_t who = __ballot_sync(~0u, stay);
        __syncthreads();
        int first = 0;
        if (lane == 0 && who) first = atomicAdd(&s.count, __popc(who));
        first = __shfl_sync(~0u, first, 0);
        if (stay) {
            buf[first + __popc(who & ((1u << lane) - 1))] = k;
            least = k < least ? k : least;
        }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const uint64_t a = __shfl_xor_sync(~0u, least, d);
        least = a < least ? a : least;
    }
    if (lane == 0) s.lo[tid >> 5] = least;
    __syncthreads();
    least = s.lo[0];
    for (int i = 1; i < NT / 32; ++i) least = s.lo[i] < least ? s.lo[i] : least;
    __syncthreads();
    return least - 1;
}

}  // namespace bsp
