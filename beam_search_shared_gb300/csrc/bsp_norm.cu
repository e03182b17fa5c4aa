// Appends of normalised and rotated rows: per-head RMS norm of keys and queries, the rotary rotation, and the write
// into 16-bit pools or E4M3 pools with one scale per tensor (norm_append_kernel) or with block scales
// (block_append_kernel), one launch each.
//
// A head row x of D elements becomes y = x / sqrt(mean(x^2) + eps) * (w + offset), in fp32, then its first rot dims
// turn by the position's angles (bsp_rope.cu has the rotation), and the result is rounded once, into the pools' type.
// Values are copied, or quantised as they are. A row lies on D / 8 consecutive lanes, 8 elements each: the sum of
// squares is log2(D / 8) shuffles, and the partner of the rotate-half layout comes by shuffle.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/bsp.h"
#include "bsp_write.h"

namespace bsp {
namespace {

constexpr unsigned kFull = 0xffffffffu;

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& x, float (&f)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 v;
        if constexpr (BF16) v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
        else v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
    }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (BF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 8 values times a factor, each product rounded to fp32, then to the nearest E4M3 (ties to even, saturating)
__device__ __forceinline__ uint2 quant8(const float (&f)[8], float mul) {
    uint32_t w[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const float2 a = make_float2(__fmul_rn(f[4 * e], mul), __fmul_rn(f[4 * e + 1], mul));
        const float2 b = make_float2(__fmul_rn(f[4 * e + 2], mul), __fmul_rn(f[4 * e + 3], mul));
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3);
        w[e] = (lo & 0xffffu) | (hi << 16);
    }
    return make_uint2(w[0], w[1]);
}

// Chunk c (8 elements) of a norm's weights, in fp32 and with the offset added; weights NULL: ones.
template <bool BF16>
__device__ __forceinline__ void load_weight(const NormRope& a, const void* weight, int c, float (&w)[8]) {
    if (!weight) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.f;
        return;
    }
    if (a.weight_fp32) {
        const float4 lo = __ldg(static_cast<const float4*>(weight) + 2 * c), hi = __ldg(static_cast<const float4*>(weight) + 2 * c + 1);
        w[0] = lo.x, w[1] = lo.y, w[2] = lo.z, w[3] = lo.w, w[4] = hi.x, w[5] = hi.y, w[6] = hi.z, w[7] = hi.w;
    } else {
        unpack8<BF16>(__ldg(static_cast<const uint4*>(weight) + c), w);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] += a.weight_offset;
}

// The lane's 8 elements f of a head row, chunk c of its D / 8, normalised (NORM and `on`) and rotated by table row t
// (`on` and t not null). Every lane of the warp takes part, rows of different kinds beside one another.
template <int D, bool BF16>
__device__ __forceinline__ void norm_rotate(const NormRope& a, const void* weight, bool on, const float* t, int lane,
                                            float (&f)[8]) {
    constexpr int CPR = D / 8;
    const int c = lane & (CPR - 1);
    if (a.norm) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
#pragma unroll
        for (int o = CPR / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
        if (on) {
            const float r = 1.f / sqrtf(fmaf(ss, 1.f / D, a.eps));
            float w[8];
            load_weight<BF16>(a, weight, c, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = f[e] * r * w[e];
        }
    }
    if (!a.cos_sin) return;  // (uniform)
    const int half = a.rot >> 1;
    const bool turned = on && t != nullptr && 8 * c < a.rot;
    if (!a.interleaved) {
        const int hc = a.rot >> 4;  // the partner chunk is hc away
        const bool first = c < hc;
        const int src = lane - c + (8 * c < a.rot ? (first ? c + hc : c - hc) : c);
        float z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = __shfl_sync(kFull, f[e], src);
        if (turned) {
            const int j0 = 8 * (first ? c : c - hc);
            const float4 c0 = __ldg(reinterpret_cast<const float4*>(t + j0)), c1 = __ldg(reinterpret_cast<const float4*>(t + j0 + 4));
            const float4 s0 = __ldg(reinterpret_cast<const float4*>(t + half + j0)), s1 = __ldg(reinterpret_cast<const float4*>(t + half + j0 + 4));
            const float cs[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
            const float sn[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
            const float sign = first ? -1.f : 1.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = __fmaf_rn(f[e], cs[e], sign * __fmul_rn(z[e], sn[e]));
        }
    } else if (turned) {
        const float4 c4 = __ldg(reinterpret_cast<const float4*>(t + 4 * c)), s4 = __ldg(reinterpret_cast<const float4*>(t + half + 4 * c));
        const float cs[4] = {c4.x, c4.y, c4.z, c4.w}, sn[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x = f[2 * e], y = f[2 * e + 1];
            f[2 * e] = __fmaf_rn(x, cs[e], -__fmul_rn(y, sn[e]));
            f[2 * e + 1] = __fmaf_rn(y, cs[e], __fmul_rn(x, sn[e]));
        }
    }
}

__device__ __forceinline__ const float* table_row(const NormRope& a, int pos) {
    return a.cos_sin ? a.cos_sin + static_cast<long long>(pos) * a.rot : nullptr;
}

// A token's slot (-1: the token is skipped) and position; what is wrong with it is flagged where `tell`.
__device__ __forceinline__ int token_slot(const NormRope& a, int i, int ps_log2, int num_pages, int32_t* status, bool tell, int* pos) {
    const int loc = __ldg(a.loc + i);
    *pos = a.cos_sin ? __ldg(a.pos + i) : 0;
    const bool pos_ok = !a.cos_sin || (*pos >= 0 && *pos < a.max_pos);
    if (pos_ok && loc >= 0 && loc < static_cast<long long>(num_pages) << ps_log2) return loc;
    if (tell) atomicOr(status, pos_ok ? BSP_DEVFLAG_PAGE_INDEX : BSP_DEVFLAG_POSITION);
    return -1;
}

// A lane's share of the tokens' query rows: row `r` of n * Hq.
template <int D, bool BF16>
__device__ __forceinline__ void query_row(const NormRope& a, long long r, int lane, int ps_log2, int num_pages, int32_t* status) {
    constexpr int CPR = D / 8;
    const int c = lane & (CPR - 1);
    const bool live = r < static_cast<long long>(a.n) * a.Hq;
    const int i = live ? static_cast<int>(r / a.Hq) : 0;
    const int h = live ? static_cast<int>(r - static_cast<long long>(i) * a.Hq) : 0;
    uint4 x = make_uint4(0, 0, 0, 0);
    int pos = 0, slot = -1;
    if (live) {
        x = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + i * a.q_stride + static_cast<long long>(h) * D) + c);
        slot = token_slot(a, i, ps_log2, num_pages, status, false, &pos);
    }
    float f[8];
    unpack8<BF16>(x, f);
    norm_rotate<D, BF16>(a, a.q_weight, slot >= 0, slot >= 0 ? table_row(a, pos) : nullptr, lane, f);
    if (slot >= 0)
        reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.q_out) + i * a.q_out_stride + static_cast<long long>(h) * D)[c] = pack8<BF16>(f);
}

}  // namespace

// 16-bit pools, or (FP8) E4M3 pools with one multiplier per tensor: one row a warp segment, the kinds of rows in
// order: K and V rows of all tokens, then their query rows.
// Bound by its traffic; small steps by the launch.
template <int D, bool BF16, bool FP8>
__global__ void __launch_bounds__(256) norm_append_kernel(const NormAppendParams p) {
    constexpr int CPR = D / 8, RPW = 32 / CPR;
    const NormRope& a = p.a;
    const int lane = threadIdx.x & 31, c = lane & (CPR - 1);
    const long long gr = (static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * RPW + lane / CPR;
    const long long kv_rows = static_cast<long long>(a.n) * 2 * p.Hkv;
    // (kv_rows is made a multiple of a warp's rows, so that a warp has one kind)
    const long long first_q = (kv_rows + RPW - 1) / RPW * RPW;
    if (gr - lane / CPR >= first_q) {
        query_row<D, BF16>(a, gr - first_q, lane, p.ps_log2, p.num_pages, p.status);
        return;
    }
    const bool live = gr < kv_rows;
    const int i = live ? static_cast<int>(gr / (2 * p.Hkv)) : 0;
    const int r = live ? static_cast<int>(gr - static_cast<long long>(i) * 2 * p.Hkv) : 0;
    const bool is_k = r < p.Hkv;
    const int h = is_k ? r : r - p.Hkv;
    uint4 x = make_uint4(0, 0, 0, 0);
    int pos = 0, slot = -1;
    if (live) {
        const uint16_t* src = static_cast<const uint16_t*>(is_k ? p.k_new : p.v_new) + i * p.src_stride + static_cast<long long>(h) * D;
        x = __ldcs(reinterpret_cast<const uint4*>(src) + c);
        slot = token_slot(a, i, p.ps_log2, p.num_pages, p.status, r == 0 && c == 0, &pos);
    }
    float f[8];
    unpack8<BF16>(x, f);
    norm_rotate<D, BF16>(a, a.k_weight, is_k && slot >= 0, slot >= 0 ? table_row(a, pos) : nullptr, lane, f);
    if (slot < 0) return;
    const long long page = slot >> p.ps_log2;
    const long long dst = (((page * p.Hkv + h) << p.ps_log2) + (slot & ((1 << p.ps_log2) - 1))) * D;
    if constexpr (FP8)
        reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_k ? p.k_pool : p.v_pool) + dst)[c] = quant8(f, is_k ? p.k_mul : p.v_mul);
    else
        reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_k ? p.k_pool : p.v_pool) + dst)[c] = is_k ? pack8<BF16>(f) : x;
}

// E4M3 pools with block scales. The scale of a block has to cover the largest of the call's rows in it, so the rows of
// a block are written by one CTA: a CTA takes the runs (tokens next to one another whose slots are in one block) that
// begin among its kWindow tokens, of one kv head and of K or V, holds their rows in registers, finds each run's largest
// magnitude in shared memory, and then quantises. A run has at most `block` <= kWindow tokens, so a CTA's last run ends
// within 2 kWindow - 1 tokens of its first. The exponent is the smallest with which that magnitude is at most 448 codes,
// but never below the block's own, unless the run begins at the block's first slot (what the block held is over then);
// where it grows, the leading rows of the block are brought to it, in place (a power of two: exact but for codes that
// fall below the format's smallest).
// The query rows are the CTAs behind (kv_ctas), as in norm_append_kernel.
constexpr int kWindow = 32;

template <int D, bool BF16>
__global__ void __launch_bounds__(256) block_append_kernel(const BlockAppendParams p) {
    constexpr int CPR = D / 8, RPW = 32 / CPR, RPP = 8 * RPW;      // rows of a warp, and of a pass of the CTA
    constexpr int PASSES = 2 * kWindow / RPP;
    const NormRope& a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = lane & (CPR - 1);
    if (blockIdx.x >= p.kv_ctas) {
        const long long r = (static_cast<long long>(blockIdx.x - p.kv_ctas) * 8 + warp) * RPW + lane / CPR;
        query_row<D, BF16>(a, r, lane, p.ps_log2, p.num_pages, p.status);
        return;
    }
    __shared__ int s_slot[2 * kWindow], s_pos[2 * kWindow];
    __shared__ uint32_t s_lead[2];              // tokens at which a run begins
    __shared__ uint32_t s_top[kWindow];         // a run's largest magnitude, at its first token
    __shared__ int s_new[kWindow], s_old[kWindow];
    const int per = 2 * p.Hkv;
    const int w = static_cast<int>(blockIdx.x / per), kind = static_cast<int>(blockIdx.x - static_cast<unsigned>(w) * per);
    const bool is_k = kind < p.Hkv;
    const int h = is_k ? kind : kind - p.Hkv;
    const long long i0 = static_cast<long long>(w) * kWindow;
    uint8_t* pool = is_k ? p.k_pool : p.v_pool;
    uint8_t* exps = is_k ? p.k_exp : p.v_exp;
    const int block = 1 << p.block_log2;
    auto pool_row = [&](int slot) -> long long {
        return ((static_cast<long long>(slot >> p.ps_log2) * p.Hkv + h) << p.ps_log2) + (slot & ((1 << p.ps_log2) - 1));
    };

    int old = 0;  // of the run that begins at token tid
    if (tid < 2 * kWindow) {
        const long long i = i0 + tid;
        int pos = 0, slot = -1, before = -1;
        if (i < a.n) slot = token_slot(a, static_cast<int>(i), p.ps_log2, p.num_pages, p.status, kind == 0 && tid < kWindow, &pos);
        if (i < a.n && i > 0) {
            int q;
            before = token_slot(a, static_cast<int>(i - 1), p.ps_log2, p.num_pages, p.status, false, &q);
        }
        s_slot[tid] = slot;
        s_pos[tid] = pos;
        // -1 >> n is -1: a token that is skipped is no run's, and the next one begins a run
        const bool lead = slot >= 0 && (slot >> p.block_log2) != (before >> p.block_log2);
        const uint32_t m = __ballot_sync(kFull, lead);
        if (lane == 0) s_lead[warp] = m;
        if (tid < kWindow) {
            s_top[tid] = 0u;
            if (lead && (slot & (block - 1)) != 0) old = exps[pool_row(slot) >> p.block_log2];
        }
    }
    __syncthreads();
    const uint32_t lead0 = s_lead[0], lead1 = s_lead[1];
    // the run that token t belongs to, by its first token; -1: none, or one that another CTA writes
    auto run_of = [&](int t) -> int {
        if (s_slot[t] < 0) return -1;
        if (t < kWindow) return 31 - __clz(lead0 & (~0u >> (31 - t)));
        return (lead1 & (~0u >> (63 - t))) ? -1 : 31 - __clz(lead0);
    };

    float f[PASSES][8];
    int run[PASSES];
#pragma unroll
    for (int s = 0; s < PASSES; ++s) {
        const int t = s * RPP + warp * RPW + lane / CPR;
        run[s] = run_of(t);
        uint4 x = make_uint4(0, 0, 0, 0);
        if (run[s] >= 0) {
            const uint16_t* src = static_cast<const uint16_t*>(is_k ? p.k_new : p.v_new) + (i0 + t) * p.src_stride + static_cast<long long>(h) * D;
            x = __ldcs(reinterpret_cast<const uint4*>(src) + c);
        }
        unpack8<BF16>(x, f[s]);
    }
#pragma unroll
    for (int s = 0; s < PASSES; ++s) {
        const int t = s * RPP + warp * RPW + lane / CPR;
        if (!__any_sync(kFull, run[s] >= 0)) continue;
        if (is_k) norm_rotate<D, BF16>(a, a.k_weight, run[s] >= 0, run[s] >= 0 ? table_row(a, s_pos[t]) : nullptr, lane, f[s]);
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f[s][e]));  // (a NaN is passed over)
#pragma unroll
        for (int o = CPR / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
        if (c == 0 && run[s] >= 0) atomicMax(&s_top[run[s]], __float_as_uint(m));  // (not negative: ordered as integers)
    }
    __syncthreads();
    if (tid < kWindow) {
        int e = 0;
        if (lead0 >> tid & 1) {
            const uint32_t top = s_top[tid];
            // 448 = 1.75 * 2^8
            if (top) e = min(max(static_cast<int>(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u), p.exp_lo), p.exp_hi);
            e = max(e, old);
            exps[pool_row(s_slot[tid]) >> p.block_log2] = static_cast<uint8_t>(e);
        }
        s_new[tid] = e;
        s_old[tid] = old;
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < PASSES; ++s) {
        if (run[s] < 0) continue;
        const int t = s * RPP + warp * RPW + lane / CPR;
        const int e = s_new[run[s]];
        const float mul = e == 0 ? 0.f : __uint_as_float(static_cast<uint32_t>(254 - e) << 23);  // 2^(127 - E)
        reinterpret_cast<uint2*>(pool + pool_row(s_slot[t]) * D)[c] = quant8(f[s], mul);
    }
    // leading rows of blocks whose scale grew
    for (int t = warp; t < kWindow; t += 8) {
        if (!(lead0 >> t & 1) || s_old[t] == 0 || s_new[t] == s_old[t]) continue;  // (uniform in the warp)
        const int slot = s_slot[t], off = slot & (block - 1);
        const float mul = __uint_as_float(static_cast<uint32_t>(127 + s_old[t] - s_new[t]) << 23);
        uint2* row = reinterpret_cast<uint2*>(pool + (pool_row(slot) - off) * D);
        for (int x = lane; x < off * CPR; x += 32) {
            const uint2 v = row[x];
            const uint32_t two[4] = {v.x & 0xffffu, v.x >> 16, v.y & 0xffffu, v.y >> 16};
            float g[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two[e]), __NV_E4M3);
                const float2 u = __half22float2(*reinterpret_cast<const __half2*>(&hr));
                g[2 * e] = u.x;
                g[2 * e + 1] = u.y;
            }
            row[x] = quant8(g, mul);
        }
    }
}

namespace {

template <int D, bool BF16>
cudaError_t launch_norm_t(const NormAppendParams& p, bool fp8, cudaStream_t stream) {
    constexpr int RPW = 32 / (D / 8);
    const long long kv = (static_cast<long long>(p.a.n) * 2 * p.Hkv + RPW - 1) / RPW;  // warps
    const long long q = p.a.q ? (static_cast<long long>(p.a.n) * p.a.Hq + RPW - 1) / RPW : 0;
    const unsigned blocks = static_cast<unsigned>((kv + q + 7) / 8);
    if (fp8) norm_append_kernel<D, BF16, true><<<blocks, 256, 0, stream>>>(p);
    else norm_append_kernel<D, BF16, false><<<blocks, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

template <int D, bool BF16>
cudaError_t launch_block_t(BlockAppendParams p, cudaStream_t stream) {
    constexpr int RPW = 32 / (D / 8);
    const long long windows = (p.a.n + kWindow - 1) / kWindow;
    const long long kv = windows * 2 * p.Hkv;
    const long long q = p.a.q ? (static_cast<long long>(p.a.n) * p.a.Hq + 8 * RPW - 1) / (8 * RPW) : 0;
    if (kv + q > INT32_MAX) return cudaErrorInvalidValue;
    p.kv_ctas = static_cast<unsigned>(kv);
    block_append_kernel<D, BF16><<<static_cast<unsigned>(kv + q), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_append(int head_dim, bool bf16, bool fp8, const NormAppendParams& p, cudaStream_t stream) {
    switch (head_dim) {
        case 64: return bf16 ? launch_norm_t<64, true>(p, fp8, stream) : launch_norm_t<64, false>(p, fp8, stream);
        case 128: return bf16 ? launch_norm_t<128, true>(p, fp8, stream) : launch_norm_t<128, false>(p, fp8, stream);
        case 256: return bf16 ? launch_norm_t<256, true>(p, fp8, stream) : launch_norm_t<256, false>(p, fp8, stream);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_block_append(int head_dim, bool bf16, const BlockAppendParams& p, cudaStream_t stream) {
    static_assert(kWindow >= BSP_MAX_SCALE_BLOCK, "a run ends within a second window");
    switch (head_dim) {
        case 64: return bf16 ? launch_block_t<64, true>(p, stream) : launch_block_t<64, false>(p, stream);
        case 128: return bf16 ? launch_block_t<128, true>(p, stream) : launch_block_t<128, false>(p, stream);
        case 256: return bf16 ? launch_block_t<256, true>(p, stream) : launch_block_t<256, false>(p, stream);
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

cudaError_t launch_rope_scaled(int max_pos, int rot, double base, const bsp_rope_scaling& sc, float* cos_sin, cudaStream_t stream) {
    const long long n = static_cast<long long>(max_pos) * (rot / 2), blocks = (n + 255) / 256;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    rope_scaled_kernel<<<static_cast<unsigned>(blocks), 256, 0, stream>>>(max_pos, rot, base, sc, cos_sin);
    return cudaGetLastError();
}

}  // namespace bsp
