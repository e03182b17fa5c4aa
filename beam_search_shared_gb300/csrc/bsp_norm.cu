// Appends of normalised and rotated rows: per-head RMS norm of keys and queries, the rotary rotation, and the write
// into 16-bit pools or E4M3 pools with one scale per tensor or per block of slots, in one launch; and the tables of
// stretched rotations.
//
// A head row x of D elements becomes y = x / sqrt(mean(x^2) + eps) * (w + offset), in fp32, then its first rot dims
// turn by the position's angles (bsp_rope.cu has the rotation), and the result is rounded once, into the pools' type.
// Values are copied, or quantised as they are. A row lies on D / 8 consecutive lanes, 8 elements each: the sum of
// squares is log2(D / 8) shuffles, and the partner of the rotate-half layout comes by shuffle.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "../../include/bsp.h"
#include "bsp_ptx.cuh"
#include "bsp_write.h"

namespace bsp {
namespace {

constexpr unsigned kFull = 0xffffffffu;

// Pairs of fp32, one instruction for both: norm and rotation are 9 of the 45 us of the largest steps (norm_append_kernel).
using f2 = unsigned long long;
__device__ __forceinline__ f2 pair(float x, float y) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 halves(f2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 x, f2 y) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ f2 add2(f2 x, f2 y) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 x, f2 y, f2 z) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}

// 8 elements of a row as 4 pairs
template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& x, f2 (&f)[4]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 v;
        if constexpr (BF16) v = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        else v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        f[i] = pair(v.x, v.y);
    }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const f2 (&f)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = halves(f[i]);
        if constexpr (BF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __half2 h = __floats2half2_rn(v.x, v.y);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 8 values times a factor, each product rounded to fp32, then to the nearest E4M3 (ties to even, saturating)
__device__ __forceinline__ uint2 quant8(const f2 (&f)[4], float mul) {
    const f2 m = pair(mul, mul);
    uint32_t q[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) q[e] = __nv_cvt_float2_to_fp8x2(halves(mul2(f[e], m)), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(__byte_perm(q[0], q[1], 0x5410), __byte_perm(q[2], q[3], 0x5410));
}

// Chunk c (8 elements) of a norm's weights, in fp32 and with the offset added; weights NULL: ones.
template <bool BF16>
__device__ __forceinline__ void load_weight(const NormRope& a, const void* weight, int c, f2 (&w)[4]) {
    if (!weight) {
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = pair(1.f, 1.f);
        return;
    }
    if (a.weight_fp32) {
        const float4 lo = __ldg(static_cast<const float4*>(weight) + 2 * c);
        const float4 hi = __ldg(static_cast<const float4*>(weight) + 2 * c + 1);
        w[0] = pair(lo.x, lo.y), w[1] = pair(lo.z, lo.w), w[2] = pair(hi.x, hi.y), w[3] = pair(hi.z, hi.w);
    } else {
        unpack8<BF16>(__ldg(static_cast<const uint4*>(weight) + c), w);
    }
    const f2 o = pair(a.weight_offset, a.weight_offset);
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = add2(w[e], o);
}

// How a lane's 8 elements x of a head row become y = r * (x A + z B): r the row's 1 / sqrt(mean + eps), z the partners'
// elements in the rotation; A and B hold the norm's weights and the position's cos and sin, so that they are worked
// out once for all rows of a kind at a position.
struct Mix {
    f2 A[4], B[4];
};
template <int D, bool BF16>
__device__ __forceinline__ void load_mix(const NormRope& a, const void* weight, int pos, int lane, Mix& m) {
    const int c = lane & (D / 8 - 1);
    load_weight<BF16>(a, weight, c, m.A);
    if (!a.cos_sin) return;  // (uniform)
#pragma unroll
    for (int e = 0; e < 4; ++e) m.B[e] = 0ull;
    if (8 * c >= a.rot) return;
    const int half = a.rot >> 1;
    const float* row = a.cos_sin + static_cast<long long>(pos) * a.rot;
    if (a.interleaved) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(row + 4 * c));
        const float4 y = __ldg(reinterpret_cast<const float4*>(row + half + 4 * c));
        const float cs[4] = {x.x, x.y, x.z, x.w}, sn[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 w = halves(m.A[e]);
            m.B[e] = mul2(pair(-w.y, w.x), pair(sn[e], sn[e]));
            m.A[e] = mul2(m.A[e], pair(cs[e], cs[e]));
        }
    } else {
        const int hc = a.rot >> 4;  // the partner chunk is hc away
        const int pc = c < hc ? c + hc : c - hc, j = 8 * min(c, pc);
        const float4 c0 = __ldg(reinterpret_cast<const float4*>(row + j));
        const float4 c1 = __ldg(reinterpret_cast<const float4*>(row + j + 4));
        const float4 s0 = __ldg(reinterpret_cast<const float4*>(row + half + j));
        const float4 s1 = __ldg(reinterpret_cast<const float4*>(row + half + j + 4));
        const float sign = c < hc ? -1.f : 1.f;  // x cos - z sin in the first half, x cos + z sin in the second
        const f2 sg = pair(sign, sign);
        load_weight<BF16>(a, weight, pc, m.B);
        m.A[0] = mul2(m.A[0], pair(c0.x, c0.y)), m.A[1] = mul2(m.A[1], pair(c0.z, c0.w));
        m.A[2] = mul2(m.A[2], pair(c1.x, c1.y)), m.A[3] = mul2(m.A[3], pair(c1.z, c1.w));
        m.B[0] = mul2(mul2(m.B[0], sg), pair(s0.x, s0.y)), m.B[1] = mul2(mul2(m.B[1], sg), pair(s0.z, s0.w));
        m.B[2] = mul2(mul2(m.B[2], sg), pair(s1.x, s1.y)), m.B[3] = mul2(mul2(m.B[3], sg), pair(s1.z, s1.w));
    }
}

// 1 / sqrt(mean + eps) of N head rows (raw: a lane's 8 elements as read), on all lanes of a row. Every lane of the warp
// takes part. The rows' sums go side by side: one after another, each waits for its own shuffles.
template <int D, bool BF16, int N>
__device__ __forceinline__ void row_factors(const NormRope& a, const uint4 (&raw)[N], float (&r)[N]) {
#pragma unroll
    for (int k = 0; k < N; ++k) r[k] = 1.f;
    if (!a.norm) return;  // (uniform)
#pragma unroll
    for (int k = 0; k < N; ++k) {
        f2 x[4];
        unpack8<BF16>(raw[k], x);
        f2 s2 = mul2(x[0], x[0]);
#pragma unroll
        for (int e = 1; e < 4; ++e) s2 = fma2(x[e], x[e], s2);
        const float2 s = halves(s2);
        r[k] = s.x + s.y;
    }
#pragma unroll
    for (int o = D / 16; o >= 1; o >>= 1) {
#pragma unroll
        for (int k = 0; k < N; ++k) r[k] += __shfl_xor_sync(kFull, r[k], o);
    }
#pragma unroll
    for (int k = 0; k < N; ++k) r[k] = rsqrtf(fmaf(r[k], 1.f / D, a.eps));
}

// The lane's 8 elements of a head row with the factor r, normalised and rotated. Every lane of the warp takes part.
template <int D, bool BF16>
__device__ __forceinline__ void norm_rotate(const NormRope& a, const Mix& m, int lane, const uint4& raw, float r,
                                            f2 (&f)[4]) {
    constexpr int CPR = D / 8;
    const int c = lane & (CPR - 1);
    f2 x[4];
    unpack8<BF16>(raw, x);
    const f2 rr = pair(r, r);
    if (!a.cos_sin) {  // (uniform)
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = mul2(mul2(x[e], rr), m.A[e]);
        return;
    }
    f2 z[4];
    const bool turned = 8 * c < a.rot;
    if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 v = halves(x[e]);
            z[e] = turned ? pair(v.y, v.x) : 0ull;
        }
    } else {
        const int hc = a.rot >> 4;
        const int src = lane - c + (turned ? (c < hc ? c + hc : c - hc) : c);
        uint4 w;
        w.x = __shfl_sync(kFull, raw.x, src);
        w.y = __shfl_sync(kFull, raw.y, src);
        w.z = __shfl_sync(kFull, raw.z, src);
        w.w = __shfl_sync(kFull, raw.w, src);
        unpack8<BF16>(turned ? w : make_uint4(0, 0, 0, 0), z);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = mul2(rr, fma2(x[e], m.A[e], mul2(z[e], m.B[e])));
}

// The same for a row by itself.
template <int D, bool BF16>
__device__ __forceinline__ void norm_rotate_row(const NormRope& a, const Mix& m, int lane, const uint4& raw,
                                                f2 (&f)[4]) {
    const uint4 one[1] = {raw};
    float r[1];
    row_factors<D, BF16>(a, one, r);
    norm_rotate<D, BF16>(a, m, lane, raw, r[0], f);
}

// A token's rows of n elements into L2, by a warp.
__device__ __forceinline__ void prefetch_row(const uint16_t* row, int n, int lane) {
    for (int at = lane * 64; at < n; at += 32 * 64) prefetch_l2(row + at);
}

// A token's slot (-1: the token is skipped) and position; what is wrong with it is flagged where `tell`.
__device__ __forceinline__ int token_slot(const NormAppendParams& p, int i, bool tell, int* pos) {
    const NormRope& a = p.a;
    const int loc = __ldg(a.loc + i);
    *pos = a.cos_sin ? __ldg(a.pos + i) : 0;
    const bool pos_ok = !a.cos_sin || (*pos >= 0 && *pos < a.max_pos);
    if (pos_ok && loc >= 0 && loc < static_cast<long long>(p.num_pages) << p.ps_log2) return loc;
    if (tell) atomicOr(p.status, pos_ok ? BSP_DEVFLAG_PAGE_INDEX : BSP_DEVFLAG_POSITION);
    return -1;
}

// A slot's row of a kv head in the pools.
__device__ __forceinline__ long long pool_row(const NormAppendParams& p, int slot, int h) {
    return ((static_cast<long long>(slot >> p.ps_log2) * p.Hkv + h) << p.ps_log2) + (slot & ((1 << p.ps_log2) - 1));
}

// A block's exponent byte as the attention reads it: the nearest one of its range; 0 as it is.
template <bool BF16>
__device__ __forceinline__ int held_exponent(int e) {
    const int held = min(e, kReadHi<BF16>);
    return BF16 || e == 0 ? held : max(held, kReadLo<BF16>);
}
static_assert(kReadLo<true> == 1, "bf16: no byte below the range but 0");
// The exponent byte of a block whose new rows' largest magnitude has the bits `top` and whose own byte is `old` (0:
// starts anew): the smallest E with top <= 448 * 2^(E - 127), 448 = 1.75 * 2^8, within the written range.
__device__ __forceinline__ int block_exponent(const NormAppendParams& p, uint32_t top, int old) {
    int e = 0;
    if (top) e = min(max(static_cast<int>(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u), p.exp_lo), p.exp_hi);
    return max(e, old);
}
__device__ __forceinline__ float code_factor(int e) {  // 2^(127 - E)
    return e == 0 ? 0.f : __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
}

// The `off` leading rows of a block (from `row` on, D codes each) brought from exponent old to e, by one row's lanes.
template <int D>
__device__ __forceinline__ void raise_rows(uint8_t* row, int off, int old, int e, int c) {
    constexpr int CPR = D / 8;
    // (2^-126 brings every code to 0, as the smaller factors do)
    const float mul = __uint_as_float(static_cast<uint32_t>(max(1, 127 + old - e)) << 23);
    for (int r = 0; r < off; ++r) {
        uint2* at = reinterpret_cast<uint2*>(row + static_cast<long long>(r) * D) + c;
        const uint2 v = *at;
        const uint32_t two[4] = {v.x & 0xffffu, v.x >> 16, v.y & 0xffffu, v.y >> 16};
        f2 g[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two[k]), __NV_E4M3);
            const float2 u = __half22float2(*reinterpret_cast<const __half2*>(&hr));
            g[k] = pair(u.x, u.y);
        }
        *at = quant8(g, mul);
    }
    static_assert(CPR <= 32, "a row within a warp");
}

// The largest magnitude of a lane's 8 elements (a NaN is passed over), and of a row, on all of its lanes.
__device__ __forceinline__ float lane_top(const f2 (&f)[4]) {
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 v = halves(f[e]);
        m = fmaxf(m, fmaxf(fabsf(v.x), fabsf(v.y)));
    }
    return m;
}
template <int D, int N>
__device__ __forceinline__ void row_tops(float (&m)[N]) {  // (side by side, as row_factors)
#pragma unroll
    for (int o = D / 16; o >= 1; o >>= 1) {
#pragma unroll
        for (int k = 0; k < N; ++k) m[k] = fmaxf(m[k], __shfl_xor_sync(kFull, m[k], o));
    }
}

// The run of token i: the tokens next to it whose slots are in its block (block_log2); its place in the run and the
// run's length. A run has at most 32 tokens.
__device__ __forceinline__ void find_run(const NormAppendParams& p, int i, int slot, int lane, int* place,
                                         int* length) {
    const int block = slot >> p.block_log2;
    auto same = [&](int j) -> bool {
        if (j < 0 || j >= p.a.n) return false;
        int pos;
        const int s = token_slot(p, j, false, &pos);
        return s >= 0 && (s >> p.block_log2) == block;
    };
    const uint32_t before = __ballot_sync(kFull, same(i - 1 - lane)), after = __ballot_sync(kFull, same(i + 1 + lane));
    *place = before == ~0u ? 31 : __ffs(~before) - 1;  // (a run of 32 has 31 others at most)
    const int rest = after == ~0u ? 31 : __ffs(~after) - 1;
    *length = *place + 1 + rest;
}

constexpr int kItems = 4;  // rows that a lane has in flight
constexpr int kAbreast = 2;  // ... and works on without a branch between

// Batch b of a token's query rows: kItems groups of RPW heads side by side. m: the mix, made here once (`have`).
template <int D, bool BF16>
__device__ __forceinline__ void query_rows(const NormAppendParams& p, int i, int pos, int b, int lane, Mix& m,
                                           bool& have) {
    constexpr int CPR = D / 8, RPW = 32 / CPR;
    const NormRope& a = p.a;
    const int c = lane & (CPR - 1), seg = lane / CPR;
    const int h0 = b * kItems * RPW + seg;
    const uint16_t* src = static_cast<const uint16_t*>(a.q) + i * a.q_stride + h0 * D + 8 * c;
    uint4 x[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        x[k] = make_uint4(0, 0, 0, 0);
        if (h0 + k * RPW < a.Hq) x[k] = __ldcs(reinterpret_cast<const uint4*>(src + k * RPW * D));
    }
    if (!have) load_mix<D, BF16>(a, a.q_weight, pos, lane, m);
    have = true;
    float r[kItems];
    row_factors<D, BF16>(a, x, r);
    uint16_t* out = static_cast<uint16_t*>(a.q_out) + i * a.q_out_stride + h0 * D + 8 * c;
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        if (k % kAbreast == 0 && h0 - seg + k * RPW >= a.Hq) break;  // (uniform)
        f2 f[4];
        norm_rotate<D, BF16>(a, m, lane, x[k], r[k], f);
        if (h0 + k * RPW < a.Hq) *reinterpret_cast<uint4*>(out + k * RPW * D) = pack8<BF16>(f);
    }
}

// Batch b of a token's K (or V) rows, each by itself, to the slot whose row of kv head 0 is `base`.
template <int D, bool BF16, int POOL, bool IS_V>
__device__ __forceinline__ void kv_rows(const NormAppendParams& p, int i, int pos, int slot, long long base, int b,
                                        int lane, Mix& m, bool& have) {
    constexpr int CPR = D / 8, RPW = 32 / CPR;
    const NormRope& a = p.a;
    const int c = lane & (CPR - 1), seg = lane / CPR;
    const int h0 = b * kItems * RPW + seg;
    const uint16_t* src = static_cast<const uint16_t*>(IS_V ? p.v_new : p.k_new) + i * p.src_stride + h0 * D + 8 * c;
    void* pool = IS_V ? p.v_pool : p.k_pool;
    uint8_t* exps = IS_V ? p.v_exp : p.k_exp;
    const int off = slot & ((1 << p.block_log2) - 1);  // rows of the block before the token's
    uint4 x[kItems];
    int old[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const int h = h0 + k * RPW;
        x[k] = make_uint4(0, 0, 0, 0);
        old[k] = 0;
        if (h < p.Hkv) {
            x[k] = __ldcs(reinterpret_cast<const uint4*>(src + k * RPW * D));
            // the exponent that the block has, unless the token starts it anew
            if (POOL == kPoolBlocks && off != 0)
                old[k] = exps[(base + (static_cast<long long>(h) << p.ps_log2)) >> p.block_log2];
        }
    }
    if (!IS_V) {
        if (!have) load_mix<D, BF16>(a, a.k_weight, pos, lane, m);
        have = true;
    }
    float r[kItems];
    if constexpr (!IS_V) row_factors<D, BF16>(a, x, r);
#pragma unroll
    for (int k0 = 0; k0 < kItems; k0 += kAbreast) {
        if (h0 - seg + k0 * RPW >= p.Hkv) break;  // (uniform)
        f2 f[kAbreast][4];
        float top[kAbreast];
#pragma unroll
        for (int j = 0; j < kAbreast; ++j) {
            if constexpr (!IS_V) norm_rotate<D, BF16>(a, m, lane, x[k0 + j], r[k0 + j], f[j]);
            else if constexpr (POOL != kPool16) unpack8<BF16>(x[k0 + j], f[j]);
            if constexpr (POOL == kPoolBlocks) top[j] = lane_top(f[j]);
        }
        if constexpr (POOL == kPoolBlocks) row_tops<D>(top);
#pragma unroll
        for (int j = 0; j < kAbreast; ++j) {
            const int k = k0 + j, h = h0 + k * RPW;
            if (h >= p.Hkv) continue;
            const long long row = base + (static_cast<long long>(h) << p.ps_log2);
            if constexpr (POOL == kPool16) {
                uint4* to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(pool) + row * D) + c;
                if constexpr (IS_V) *to = x[k];
                else *to = pack8<BF16>(f[j]);
            } else if constexpr (POOL == kPoolE4m3) {
                const float mul = IS_V ? p.v_mul : p.k_mul;
                reinterpret_cast<uint2*>(static_cast<uint8_t*>(pool) + row * D)[c] = quant8(f[j], mul);
            } else {
                const int was = held_exponent<BF16>(old[k]), e = block_exponent(p, __float_as_uint(top[j]), was);
                reinterpret_cast<uint2*>(static_cast<uint8_t*>(pool) + row * D)[c] = quant8(f[j], code_factor(e));
                const long long head = row >> p.block_log2;
                // (0: zeros that start it anew)
                if (c == 0 && (e != old[k] || e == 0)) exps[head] = static_cast<uint8_t>(e);
                if (was != 0 && e != was)
                    raise_rows<D>(static_cast<uint8_t*>(pool) + (head << p.block_log2) * D, off, was, e, c);
            }
        }
    }
}

// One group of heads of K (or V) over the rows of a run of several tokens from `lead` on: once for the largest
// magnitude, once for the codes, the second time out of L1 or L2.
template <int D, bool BF16>
__device__ __forceinline__ void run_rows(const NormAppendParams& p, int lead, int length, int slot, int group,
                                         bool is_v, int lane) {
    constexpr int CPR = D / 8, RPW = 32 / CPR;
    const NormRope& a = p.a;
    const int c = lane & (CPR - 1), seg = lane / CPR;
    const int h = group * RPW + seg;
    const bool live = h < p.Hkv;
    uint8_t* pool = static_cast<uint8_t*>(is_v ? p.v_pool : p.k_pool);
    uint8_t* exps = is_v ? p.v_exp : p.k_exp;
    const int off = __ldg(a.loc + lead) & ((1 << p.block_log2) - 1);
    const long long head = live ? pool_row(p, slot, h) >> p.block_log2 : 0;  // the block's place in the table
    const int old = live && off != 0 ? held_exponent<BF16>(exps[head]) : 0;
    const uint16_t* src = static_cast<const uint16_t*>(is_v ? p.v_new : p.k_new);
    auto rows = [&](auto&& each) {
        for (int r = 0; r < length; ++r) {
            uint4 raw = make_uint4(0, 0, 0, 0);
            if (live) raw = __ldg(reinterpret_cast<const uint4*>(src + (lead + r) * p.src_stride + h * D) + c);
            f2 f[4];
            if (is_v) {
                unpack8<BF16>(raw, f);
            } else {
                Mix m;
                load_mix<D, BF16>(a, a.k_weight, a.cos_sin ? __ldg(a.pos + lead + r) : 0, lane, m);
                norm_rotate_row<D, BF16>(a, m, lane, raw, f);
            }
            each(r, f);
        }
    };
    float top = 0.f;
    rows([&](int, const f2(&f)[4]) { top = fmaxf(top, lane_top(f)); });
    float tops[1] = {top};
    row_tops<D>(tops);
    const int e = block_exponent(p, __float_as_uint(tops[0]), old);
    const float mul = code_factor(e);
    rows([&](int r, const f2(&f)[4]) {
        if (live) reinterpret_cast<uint2*>(pool + pool_row(p, __ldg(a.loc + lead + r), h) * D)[c] = quant8(f, mul);
    });
    if (!live) return;
    if (c == 0) exps[head] = static_cast<uint8_t>(e);
    if (old != 0 && e != old) raise_rows<D>(pool + (head << p.block_log2) * D, off, old, e, c);
}

}  // namespace

// One launch for the K, V and query rows of n tokens. A group is the 32 / (D / 8) heads side by side that fill a warp;
// a batch is kItems groups of a token's K, V or query rows, all in flight together. `units` warps take a token, one
// for all of its batches where there are tokens enough, so that its slot, position and angles are read once and the
// norm's weights are mixed with them once per kind; a warp per batch where there are few.
// POOL: what K and V become. kPool16, kPoolE4m3 (one multiplier per tensor): each row by itself. kPoolBlocks: the scale
// of a block has to cover the largest of the call's rows in it. Tokens next to one another in one block are a run. A
// run of one token (a decode step's) takes the same path, and finds its exponent by shuffles. The warps of a longer run
// share its groups (run_rows). Nothing is shared between warps. Where a block's exponent grows, its rows before the
// run are brought to the new one in place.
// Times in a replayed graph, 16 query and 8 K and V heads of 128. Bound by latency at a step's sizes: 4 tokens 2.6 us, the
// chain of slot, position, angles and rows; 1920 tokens into 16-bit pools 7.9 us where the bytes take 4.6, all CTAs
// resident at once: K and V alone 4.6 (the plain append 4.1), without the rotation 6.7. Large ones have two parts: 12288
// tokens into 8-bit blocks take 45 us, 26 for the bytes. K and V alone take 25, and the plain E4M3 append of the same
// rows 24 (bsp_append.cu): writes of 128 bytes to pages of their own run at half of the copy rate. The query rows add
// their bytes, and norm and rotation their instructions: without both it takes 35.5, K and V alone 21.
// E4M3 pools with one scale: 12288 tokens 36.6 us, 3540 prompt tokens (32 query heads) 19.4.
// Seven CTAs an SM: 1920 tokens 7.8 us, 12288 into blocks 44.8; six 9.0 and 45.3, eight 8.1 and 47.1 (spills).
template <int D, bool BF16, int POOL>
__global__ void __launch_bounds__(128, 7) norm_append_kernel(const NormAppendParams p) {
    const int lane = threadIdx.x & 31;
    const unsigned w = blockIdx.x * 4u + (threadIdx.x >> 5);
    const int i = static_cast<int>(w / p.units), u = static_cast<int>(w - static_cast<unsigned>(i) * p.units);
    if (i >= p.a.n) return;
    if (p.units == 1) {
        // all of the token's rows will be read here: those of the later batches come into L2 meanwhile
        prefetch_row(static_cast<const uint16_t*>(p.v_new) + i * p.src_stride, p.Hkv * D, lane);
        if (p.a.q) prefetch_row(static_cast<const uint16_t*>(p.a.q) + i * p.a.q_stride, p.a.Hq * D, lane);
    }
    // lanes 0 to 2 look at the token before, the token and the one behind (only a block's scale asks for the others)
    int pos = 0, slot = -1;
    {
        const int j = i - 1 + lane;
        const bool look = POOL == kPoolBlocks ? lane < 3 && j >= 0 && j < p.a.n : lane == 1;
        if (look) slot = token_slot(p, j, u == 0 && lane == 1, &pos);
    }
    const int before = __shfl_sync(kFull, slot, 0), behind = __shfl_sync(kFull, slot, 2);
    slot = __shfl_sync(kFull, slot, 1);
    pos = __shfl_sync(kFull, pos, 1);
    if (slot < 0) return;
    const long long base = pool_row(p, slot, 0);
    int first = u;  // the warp's first batch
    if constexpr (POOL == kPoolBlocks) {
        auto near = [&](int s) { return s >= 0 && (s >> p.block_log2) == (slot >> p.block_log2); };
        if (near(before) || near(behind)) {  // (uniform; a step's tokens stand alone)
            int place, length;
            find_run(p, i, slot, lane, &place, &length);
            for (int item = place * p.units + u; item < 2 * p.groups; item += length * p.units) {
                const bool is_v = item >= p.groups;
                run_rows<D, BF16>(p, i - place, length, slot, is_v ? item - p.groups : item, is_v, lane);
            }
            while (first < 2 * p.kv_batches) first += p.units;
        }
    }
    Mix m;
    bool have = false;
    int b = first;
    for (; b < p.kv_batches; b += p.units) kv_rows<D, BF16, POOL, false>(p, i, pos, slot, base, b, lane, m, have);
    for (; b < 2 * p.kv_batches; b += p.units)
        kv_rows<D, BF16, POOL, true>(p, i, pos, slot, base, b - p.kv_batches, lane, m, have);
    have = false;
    for (; b < p.batches; b += p.units) query_rows<D, BF16>(p, i, pos, b - 2 * p.kv_batches, lane, m, have);
}

// Block scales for tokens that come in runs, a prompt's: a CTA takes the runs that begin among kWindow tokens, of one
// group of heads, K or V. A run has at most kWindow tokens, so they end within the window behind. Its warps take the
// tokens piece by piece, normalise and rotate their rows into shared memory (fp32) and find each run's largest
// magnitude there; then the rows' codes follow. Each row is read and worked out once, and no CTA depends on another.
// The query rows' CTAs are dealt between the others', which wait more than they move.
// 3540 prompt tokens, 32 query and 8 K and V heads, blocks of 32: 27 us (12 for the bytes), K and V alone 18 (12 without
// norm and rotation, the plain E4M3 append 7), bound by the phases of a CTA one after another and a warp's chain for each
// of its tokens; runs by warps
// (norm_append_kernel), which read and normalise their rows twice, took 41. Windows of 16 tokens 34 us, four warps 38,
// sixteen 33.
constexpr int kWindow = 32;
constexpr int kSpan = kWindow + BSP_MAX_SCALE_BLOCK;         // tokens that the runs of a window reach over
constexpr size_t kWindowSmem = kSpan * 256 * sizeof(float);  // (a group of heads has 256 elements)
static_assert(kWindow == 32 && kSpan == 64, "two tokens a lane");

template <int D, bool BF16>
__global__ void __launch_bounds__(256, 3) block_window_kernel(const NormAppendParams p, unsigned kv_ctas,
                                                              unsigned ctas) {
    constexpr int CPR = D / 8, RPW = 32 / CPR, BATCH = 2;
    const NormRope& a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = lane & (CPR - 1), seg = lane / CPR;
    // CTA x is the y-th for K and V where the running share of those steps up at x
    const unsigned y = static_cast<unsigned>(static_cast<unsigned long long>(blockIdx.x) * kv_ctas / ctas);
    const bool kv = static_cast<unsigned>(static_cast<unsigned long long>(blockIdx.x + 1) * kv_ctas / ctas) != y;
    if (!kv) {
        const int i = static_cast<int>((blockIdx.x - y) * 8u + warp);  // a warp takes a token's query rows
        if (i >= a.n) return;
        prefetch_row(static_cast<const uint16_t*>(a.q) + i * a.q_stride, a.Hq * D, lane);
        int pos;
        if (token_slot(p, i, false, &pos) < 0) return;
        Mix m;
        bool have = false;
        for (int b = 0; b < p.batches - 2 * p.kv_batches; ++b) query_rows<D, BF16>(p, i, pos, b, lane, m, have);
        return;
    }
    extern __shared__ f2 s_rows[];                // [kSpan][4][32]: pair e of lane l's elements of a token
    __shared__ uint32_t s_top[kWindow][RPW];      // a run's largest magnitude, at its first token
    __shared__ ushort2 s_exp[kWindow][RPW];       // its block's exponent before and after
    const int items = 2 * p.groups;
    const int window = static_cast<int>(y / items), item = static_cast<int>(y - static_cast<unsigned>(window) * items);
    const bool is_v = item >= p.groups;
    const int h0 = (is_v ? item - p.groups : item) * RPW;  // the group's first head
    const bool live = h0 + seg < p.Hkv;
    const int i0 = window * kWindow;
    const uint16_t* src = static_cast<const uint16_t*>(is_v ? p.v_new : p.k_new) + i0 * p.src_stride + h0 * D;
    {
        // the rows come into L2 while the slots are looked up
        const int t = tid >> 2, at = 64 * (tid & 3);
        if (t < kSpan && i0 + t < a.n && h0 * D + at < p.Hkv * D) prefetch_l2(src + t * p.src_stride + at);
    }
    if (tid < kWindow * RPW) s_top[tid / RPW][tid % RPW] = 0u;
    // every warp looks at all of the tokens, two a lane: their slots, positions and runs stay in registers
    int slot[2], pos[2] = {0, 0}, run[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int i = i0 + 32 * j + lane;
        slot[j] = i < a.n ? token_slot(p, i, item == 0 && warp == 0 && j == 0, &pos[j]) : -1;
    }
    unsigned long long lead = 0;  // tokens at which a run begins
    {
        int before = -1, unused;
        if (lane == 0 && i0 > 0) before = token_slot(p, i0 - 1, false, &unused);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int up = __shfl_up_sync(kFull, slot[j], 1);
            if (lane != 0) before = up;
            else if (j == 1) before = run[0];
            run[0] = __shfl_sync(kFull, slot[j], 31);  // (for the next half's first lane)
            // (-1 >> n is -1: a token that is skipped is no run's)
            const bool leads = slot[j] >= 0 && (slot[j] >> p.block_log2) != (before >> p.block_log2);
            lead |= static_cast<unsigned long long>(__ballot_sync(kFull, leads)) << (32 * j);
        }
    }
    // the first token of a token's run; -1: of none, or of one that another CTA writes
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int first = 63 - __clzll(lead & (~0ull >> (63 - 32 * j - lane)));
        run[j] = slot[j] >= 0 && first < kWindow ? first : -1;
    }
    auto of = [&](const int (&x)[2], int t) -> int { return __shfl_sync(kFull, t < 32 ? x[0] : x[1], t & 31); };
    // the tokens from the first to the last of these runs, shared out among the warps piece by piece: a warp's tokens
    // are of few runs
    const unsigned long long mine = __ballot_sync(kFull, run[0] >= 0) |
                                    static_cast<unsigned long long>(__ballot_sync(kFull, run[1] >= 0)) << 32;
    if (mine == 0) return;  // (every warp finds the same)
    const int begin = __ffsll(mine) - 1, share = (63 - __clzll(mine) - begin) / 8 + 1;
    const int t_begin = min(kSpan, begin + warp * share), t_end = min(kSpan, t_begin + share);
    __syncthreads();
    int at_run = -1;  // the run that `top` is of
    float top[1] = {0.f};
    auto give = [&] {
        if (at_run < 0) return;
        row_tops<D>(top);
        if (c == 0) atomicMax(&s_top[at_run][seg], __float_as_uint(top[0]));  // (not negative: ordered as integers)
    };
#pragma unroll 1
    for (int t0 = t_begin; t0 < t_end; t0 += BATCH) {
        uint4 x[BATCH];
        int first[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int t = t0 + k;
            first[k] = t < t_end ? of(run, t) : -1;  // (uniform)
            x[k] = make_uint4(0, 0, 0, 0);
            if (first[k] >= 0 && live) x[k] = __ldcs(reinterpret_cast<const uint4*>(src + t * p.src_stride) + lane);
        }
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            if (first[k] < 0) continue;
            const int t = t0 + k;
            f2 f[4];
            if (is_v) {
                unpack8<BF16>(x[k], f);
            } else {
                Mix m;
                load_mix<D, BF16>(a, a.k_weight, of(pos, t), lane, m);
                norm_rotate_row<D, BF16>(a, m, lane, x[k], f);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) s_rows[(t * 4 + e) * 32 + lane] = f[e];
            if (first[k] != at_run) {
                give();
                at_run = first[k];
                top[0] = 0.f;
            }
            top[0] = fmaxf(top[0], lane_top(f));
        }
    }
    give();
    __syncthreads();
    uint8_t* pool = static_cast<uint8_t*>(is_v ? p.v_pool : p.k_pool);
    uint8_t* exps = is_v ? p.v_exp : p.k_exp;
    if (warp < RPW) {
        // a thread for each run and head
        const int hs = h0 + warp;
        int e = 0, old = 0;
        if ((lead >> lane & 1) && hs < p.Hkv) {
            uint8_t* at = exps + (pool_row(p, slot[0], hs) >> p.block_log2);
            if ((slot[0] & ((1 << p.block_log2) - 1)) != 0) old = held_exponent<BF16>(*at);
            e = block_exponent(p, s_top[lane][warp], old);
            *at = static_cast<uint8_t>(e);
        }
        s_exp[lane][warp] = make_ushort2(static_cast<unsigned short>(old), static_cast<unsigned short>(e));
    }
    __syncthreads();
    const long long head = static_cast<long long>(h0 + seg) << p.ps_log2;  // rows before the lane's head in a page
#pragma unroll 2
    for (int t = t_begin; t < t_end; ++t) {
        const int first = of(run, t), at = of(slot, t);
        if (first < 0 || !live) continue;
        f2 f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = s_rows[(t * 4 + e) * 32 + lane];
        uint2* to = reinterpret_cast<uint2*>(pool + (pool_row(p, at, 0) + head) * D) + c;
        *to = quant8(f, code_factor(s_exp[first][seg].y));
    }
    for (int t = warp; t < kWindow; t += 8) {
        const int at = of(slot, t);
        if (!(lead >> t & 1) || !live) continue;
        const int old = s_exp[t][seg].x, e = s_exp[t][seg].y, off = at & ((1 << p.block_log2) - 1);
        if (old != 0 && e != old) raise_rows<D>(pool + (pool_row(p, at, h0 + seg) - off) * D, off, old, e, c);
    }
}

namespace {

template <int D, bool BF16>
cudaError_t launch_norm_t(NormAppendParams p, PoolKind pools, bool runs, int num_sms, cudaStream_t stream) {
    constexpr int RPW = 32 / (D / 8);
    p.groups = (p.Hkv + RPW - 1) / RPW;
    p.kv_batches = (p.groups + kItems - 1) / kItems;
    p.batches = 2 * p.kv_batches + (p.a.q ? (p.a.Hq + RPW * kItems - 1) / (RPW * kItems) : 0);
    if (pools == kPoolBlocks && p.block_log2 > 0 && runs) {
        const long long kv = static_cast<long long>((p.a.n + kWindow - 1) / kWindow) * 2 * p.groups;
        const long long q = p.a.q ? (p.a.n + 7) / 8 : 0;
        if (kv + q > INT32_MAX) return cudaErrorInvalidValue;
        const cudaError_t e = cudaFuncSetAttribute(block_window_kernel<D, BF16>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, kWindowSmem);
        if (e != cudaSuccess) return e;
        const unsigned kv_ctas = static_cast<unsigned>(kv), ctas = static_cast<unsigned>(kv + q);
        block_window_kernel<D, BF16><<<ctas, 256, kWindowSmem, stream>>>(p, kv_ctas, ctas);
        return cudaGetLastError();
    }
    // warps of a token: as many as keep the SMs' resident warps (28 of each) busy. Twice as many: 1920 tokens 8.3 us
    // for 7.8, 3540 tokens 17.9 for 18.4; four times as many: 8.3 and 21.4. 4 tokens with one warp each: 2 us more
    p.units = std::max(1, std::min(p.batches, 28 * num_sms / p.a.n));
    const long long warps = static_cast<long long>(p.a.n) * p.units;
    if (warps > INT32_MAX) return cudaErrorInvalidValue;
    const unsigned blocks = static_cast<unsigned>((warps + 3) / 4);
    switch (pools) {
        case kPool16: norm_append_kernel<D, BF16, kPool16><<<blocks, 128, 0, stream>>>(p); break;
        case kPoolE4m3: norm_append_kernel<D, BF16, kPoolE4m3><<<blocks, 128, 0, stream>>>(p); break;
        case kPoolBlocks: norm_append_kernel<D, BF16, kPoolBlocks><<<blocks, 128, 0, stream>>>(p); break;
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_append(int head_dim, bool bf16, PoolKind pools, bool runs, const NormAppendParams& p,
                               int num_sms, cudaStream_t stream) {
    static_assert(BSP_MAX_SCALE_BLOCK <= 32, "a run within a warp's look around");
    auto by_type = [&](auto dim) {
        constexpr int D = decltype(dim)::value;
        return bf16 ? launch_norm_t<D, true>(p, pools, runs, num_sms, stream)
                    : launch_norm_t<D, false>(p, pools, runs, num_sms, stream);
    };
    switch (head_dim) {
        case 64: return by_type(std::integral_constant<int, 64>());
        case 128: return by_type(std::integral_constant<int, 128>());
        case 256: return by_type(std::integral_constant<int, 256>());
        default: return cudaErrorInvalidValue;
    }
}

// Table of a stretched rotation (bsp_rope_scaling): the pair's frequency by its kind, in fp64, then as
// rope_cos_sin_kernel (bsp_rope.cu).
__global__ void rope_scaled_kernel(int max_pos, int rot, double base, bsp_rope_scaling sc, float* cs) {
    const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    const int half = rot >> 1;
    if (i >= static_cast<long long>(max_pos) * half) return;
    const int pos = static_cast<int>(i / half), j = static_cast<int>(i % half);
    const double two_pi = 6.283185307179586476925286766559;
    if (sc.kind == BSP_ROPE_BASE) base *= pow(sc.factor, static_cast<double>(rot) / (rot - 2));
    double theta = pow(base, -2.0 * j / rot);
    if (sc.kind == BSP_ROPE_LINEAR) {
        theta /= sc.factor;
    } else if (sc.kind == BSP_ROPE_BANDS) {
        const double turns = sc.original_positions * theta / two_pi;
        const double s = fmin(fmax((turns - sc.low) / (sc.high - sc.low), 0.0), 1.0);
        theta = theta * ((1.0 - s) / sc.factor + s);
    } else if (sc.kind == BSP_ROPE_RAMP) {
        const double span = rot / (2.0 * log(base));
        const double lo = fmax(floor(span * log(sc.original_positions / (two_pi * sc.high))), 0.0);
        const double hi = fmin(ceil(span * log(sc.original_positions / (two_pi * sc.low))), rot - 1.0);
        const double s = fmin(fmax((j - lo) / fmax(hi - lo, 0.001), 0.0), 1.0);
        theta = theta / sc.factor * s + theta * (1.0 - s);
    }
    double sn, co;
    sincos(pos * theta, &sn, &co);
    cs[static_cast<long long>(pos) * rot + j] = __double2float_rn(co * sc.amplitude);
    cs[static_cast<long long>(pos) * rot + half + j] = __double2float_rn(sn * sc.amplitude);
}

cudaError_t launch_rope_scaled(int max_pos, int rot, double base, const bsp_rope_scaling& sc, float* cos_sin,
                               cudaStream_t stream) {
    const long long n = static_cast<long long>(max_pos) * (rot / 2), blocks = (n + 255) / 256;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    rope_scaled_kernel<<<static_cast<unsigned>(blocks), 256, 0, stream>>>(max_pos, rot, base, sc, cos_sin);
    return cudaGetLastError();
}

}  // namespace bsp
