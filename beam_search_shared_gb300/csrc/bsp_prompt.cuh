// Device-side pieces shared by the prompt-attention kernels (bsp_prefix.cu, bsp_wide.cu, bsp_alt.cu): the
// work unit as the plan image describes it, tile counts, 16-bit packing, and the widening of E4M3 tiles.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "bsp_internal.h"

namespace bsp {

struct UnitInfo {
    int b, g, rb, part, P, page_off;
    int key_begin, key_end;  // keys [key_begin, key_end) of the request's prompt
    int T;                   // tail positions of the request
    bool fused;              // this kernel finishes the request: tail tiles when T > 0, final O / LSE
    int rows;                // the request's query rows per head (beams, or prompt tokens of a prefill)
    int causal;              // -1, or the cached rows C of a causal prefill: row t sees keys 0 .. C + t
    int row_off;             // the request's first row of q and o
};

__device__ __forceinline__ UnitInfo load_unit(const PrefixParams& p, int u) {
    const int4 a = __ldg(reinterpret_cast<const int4*>(p.units + static_cast<long long>(u) * kUnitFields));
    const int4 c = __ldg(reinterpret_cast<const int4*>(p.units + static_cast<long long>(u) * kUnitFields + 4));
    const int4 r = __ldg(reinterpret_cast<const int4*>(p.req + a.x * kReqFields));
    const int4 r2 = __ldg(reinterpret_cast<const int4*>(p.req + a.x * kReqFields + 4));
    const int4 r3 = __ldg(reinterpret_cast<const int4*>(p.req + a.x * kReqFields + 8));
    UnitInfo ui;
    ui.b = a.x;
    ui.g = a.y;
    ui.rb = a.z;
    ui.part = c.y;
    ui.P = r.x;
    ui.page_off = r2.x;
    ui.key_begin = a.w * kTileKeys;                // plan tiles are kTileKeys keys
    ui.key_end = min(c.x * kTileKeys, ui.P);
    ui.T = r.y;
    ui.fused = r2.y != 0;                            // kReqFused
    ui.rows = r3.x;                                  // kReqRows
    ui.causal = r3.y;                                // kReqCausal
    ui.row_off = r3.z;                               // kReqRowOff
    return ui;
}

// prompt tiles of a unit
template <int TK>
__device__ __forceinline__ int prompt_tiles(const UnitInfo& ui) {
    return (ui.key_end - ui.key_begin + TK - 1) / TK;
}

// Two values as a 16-bit pair. Probabilities go to P*V this way: the MMA's operands have one type, V's. Each is off by
// half a step (bf16 2^-8 of the value, fp16 2^-11, or 2^-25 below 2^-14), so an output element by that share of
// sum p |v| beside its own rounding. Row sums add the fp32 values.
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (BF16) {
        __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t*>(&h);
    } else {
        __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<uint32_t*>(&h);
    }
}

// ---- E4M3 pools: the kernels load E4M3 tiles and widen them to the q dtype in shared memory

// Two E4M3 codes (bits 0-7 and 8-15 of `two`) as bfloat16 values times 2^-112, the first in the low half: the
// hardware conversion gives binary16, and the binary16 sign, exponent and fraction fields move into bfloat16
// fields (the exponent keeps its binary16 bias of 15 instead of 127). E4M3-derived binary16 values are zero or
// normal (the smallest, 2^-9, has exponent field 6) with the fraction's low 7 bits zero, so the shifted values
// are exact, zero or normal. A product with 0 gives each half's sign bit, and 0x7fff for a NaN code, whose
// exponent field would be that of a number once shifted; the mask cuts what the upper half's fraction (of a
// NaN) moves into the lower half. z: that product.
__device__ __forceinline__ uint32_t e4m3x2_shifted(uint32_t two, uint32_t& z) {
    uint32_t h;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(two));
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(z) : "r"(h), "r"(0u));
    return ((h >> 3) & 0x0fff0fffu) | z;
}

// Two E4M3 codes as a pair of 16-bit floats of the q dtype, exactly: every E4M3 value is a binary16 and a
// bfloat16 value, and one multiplication by 2^112 restores the shifted one. NaN codes give NaN.
template <bool BF16>
__device__ __forceinline__ uint32_t e4m3x2_to_16(uint32_t two) {
    uint32_t r, z;
    if constexpr (BF16)
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(e4m3x2_shifted(two, z)), "r"(0x77807780u));  // 2^112 in both halves
    else
        asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(two));
    return r;
}

// The factor, in both halves of a word, that scaled_e4m3x2 takes for a block's exponent byte E (scale 2^(E - 127)).
// bfloat16: 2^112 * 2^(E - 127), one exponent field of E + 112 (E up to 142, a scale of 2^15), so that the scale costs no
// multiplication of its own. binary16: 2^(E - 127) for exponents in [-15, 7], with which every product is a number of
// the type: |code| <= 448 * 2^7 < 2^16, and the smallest step of a code, 2^-9, gives a multiple of 2^-24.
// A block that nothing was written to (E = 0) reads as 0.
template <bool BF16>
__device__ __forceinline__ uint32_t block_factor(uint32_t e) {
    uint32_t f;
    if constexpr (BF16) {
        f = (e == 0 ? 0u : min(e, 142u) + 112u) << 7;
    } else {
        const uint32_t c = min(max(e, 112u), 134u);
        f = e == 0 ? 0u : c == 112u ? 0x0200u : (c - 112u) << 10;  // 2^-15 is half of the smallest normal number
    }
    return f | (f << 16);
}
// The same scale in fp32 (0 for a block that nothing was written to).
template <bool BF16>
__device__ __forceinline__ float block_scale(uint32_t e) {
    return e == 0 ? 0.f : __uint_as_float((BF16 ? min(e, 142u) : min(max(e, 112u), 134u)) << 23);
}
// e4m3x2_to_16 times a block's scale, exact where the product is a number of the type (bfloat16: all but the
// smallest scales' products below 2^-133). NaN codes give NaN under every factor, 0 among them.
template <bool BF16>
__device__ __forceinline__ uint32_t scaled_e4m3x2(uint32_t two, uint32_t factor) {
    uint32_t r, z;
    if constexpr (BF16) asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(e4m3x2_shifted(two, z)), "r"(factor));
    else asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(e4m3x2_to_16<false>(two)), "r"(factor));
    return r;
}
// 8 E4M3 codes (bytes in order) -> one 16-byte chunk of 8 16-bit values
template <bool BF16>
__device__ __forceinline__ uint4 e4m3x8_to_16(uint2 in) {
    return make_uint4(e4m3x2_to_16<BF16>(in.x & 0xffffu), e4m3x2_to_16<BF16>(in.x >> 16),
                      e4m3x2_to_16<BF16>(in.y & 0xffffu), e4m3x2_to_16<BF16>(in.y >> 16));
}

// The same with a block's scale (BLK).
template <bool BF16, bool BLK>
__device__ __forceinline__ uint4 widen_e4m3x8(uint2 in, uint32_t factor) {
    if constexpr (BLK)
        return make_uint4(scaled_e4m3x2<BF16>(in.x & 0xffffu, factor), scaled_e4m3x2<BF16>(in.x >> 16, factor),
                          scaled_e4m3x2<BF16>(in.y & 0xffffu, factor), scaled_e4m3x2<BF16>(in.y >> 16, factor));
    else
        return e4m3x8_to_16<BF16>(in);
}

// A gathered tail tile holds rows of all beams of its block, and a probability of 0 times a NaN is a NaN: a value's NaN
// would reach the beams that do not read it. So the gathering threads mark what they have seen in `nan` (widen_values,
// seen_nan), and go over their chunks of the tile once more if there was one: 8 values with a NaN among them become
// zeros, and the 8 elements of the key beside them NaNs (spread_nan). The mask keeps those from the other beams'
// scores, and the rows that read the key become NaN, output and log-sum-exp.
template <bool BF16, bool BLK>
__device__ __forceinline__ uint4 widen_values(uint2 in, uint32_t factor, uint32_t& nan) {
    if constexpr (BF16) {
        const uint32_t f = BLK ? factor : 0x77807780u;
        const uint32_t two[4] = {in.x & 0xffffu, in.x >> 16, in.y & 0xffffu, in.y >> 16};
        uint32_t r[4], z[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r[i]) : "r"(e4m3x2_shifted(two[i], z[i])), "r"(f));
        nan |= z[0] | z[1];
        nan |= z[2] | z[3];
        return make_uint4(r[0], r[1], r[2], r[3]);
    } else {
        // (a NaN code has all seven bits below its sign set: one more carries into the sign's place)
        nan |= ((in.x & 0x7f7f7f7fu) + 0x01010101u) | ((in.y & 0x7f7f7f7fu) + 0x01010101u);
        return widen_e4m3x8<BF16, BLK>(in, factor);
    }
}
template <bool BF16>
__device__ __forceinline__ bool seen_nan(uint32_t nan) {
    return (nan & (BF16 ? 0x7fff7fffu : 0x80808080u)) != 0u;
}
template <bool BF16>
__device__ __forceinline__ void spread_nan(uint8_t* key, uint8_t* value) {
    const uint4 v = *reinterpret_cast<const uint4*>(value);
    constexpr uint32_t inf = BF16 ? 0x7f80u : 0x7c00u;
    bool nan = false;
    for (uint32_t w : {v.x, v.y, v.z, v.w}) nan |= (w & 0x7fffu) > inf || (w >> 16 & 0x7fffu) > inf;
    if (!nan) return;
    *reinterpret_cast<uint4*>(key) = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
    *reinterpret_cast<uint4*>(value) = make_uint4(0u, 0u, 0u, 0u);
}

// The prompt tiles of a CTA's units in order, one ahead of the tile that is widened, so that the exponent bytes of the
// next tile's rows (a page id, then a byte: two loads from L2 or farther) arrive while this one waits for its codes.
// Run by the NT threads of a widening stream. Each holds the factors of TK / NT of the tile's rows: the LPR lanes that
// widen rows r0 + RS i hold row r0 + RS (j + LPR e) on lane j, and a row's factor comes from its lane by a shuffle.
template <int D, int TK, bool BF16, int NT>
struct BlockFactors {
    static constexpr int LPR = D / 16;       // lanes of a row
    static constexpr int RS = NT / LPR;      // rows one pass of the threads covers
    static constexpr int NE = TK / NT;       // rows whose factor a thread holds
    int k, t, tiles, key0, key_end, page_off, g;
    uint32_t f[NE];

    __device__ __forceinline__ void unit(const PrefixParams& p, int u_begin, int nunits) {
        for (tiles = 0; k < nunits; ++k) {
            const UnitInfo ui = load_unit(p, u_begin + k);
            tiles = prompt_tiles<TK>(ui);
            if (tiles <= 0) continue;
            t = 0;
            key0 = ui.key_begin;
            key_end = ui.key_end;
            page_off = ui.page_off;
            g = ui.g;
            return;
        }
    }
    __device__ __forceinline__ void fetch(const PrefixParams& p, const uint8_t* exps, int nunits, int gtid) {
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            const int key = key0 + gtid / LPR + RS * ((gtid & (LPR - 1)) + LPR * e);
            uint32_t x = 0;
            if (k < nunits && key < key_end) {
                const int page = __ldg(p.pages + page_off + (key >> p.ps_log2));
                if (static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages)) {
                    const int row = ((page * p.Hkv + g) << p.ps_log2) + (key & ((1 << p.ps_log2) - 1));  // (as the loads' rows)
                    x = __ldg(exps + (row >> p.block_log2));
                }
            }
            f[e] = x;
        }
    }
    __device__ __forceinline__ void begin(const PrefixParams& p, const uint8_t* exps, int u_begin, int nunits, int gtid) {
        k = 0;
        unit(p, u_begin, nunits);
        fetch(p, exps, nunits, gtid);
    }
    // the factors of the tile at hand into now[], and the next tile's bytes on their way
    __device__ __forceinline__ void next(const PrefixParams& p, const uint8_t* exps, int u_begin, int nunits, int gtid,
                                         uint32_t (&now)[NE]) {
#pragma unroll
        for (int e = 0; e < NE; ++e) now[e] = block_factor<BF16>(f[e]);
        key0 += TK;
        if (++t >= tiles && k < nunits) {
            ++k;
            unit(p, u_begin, nunits);
        }
        fetch(p, exps, nunits, gtid);
    }
};

// Byte offset of 16-byte chunk kc (8 elements) of key row r in a 16-bit K or V tile of TK rows laid out
// as a TMA box with 128-byte swizzle: column half kc / 8, then row r, then chunk (kc % 8) ^ (r % 8).
template <int TK>
__device__ __forceinline__ uint32_t sw128_chunk(int kc, int r) {
    return static_cast<uint32_t>((kc >> 3) * (TK * 128) + r * 128 + (((kc & 7) ^ (r & 7)) << 4));
}

// Widens the E4M3 K or V tile that a TMA load left in the upper half of a ring slot (TK rows of D codes,
// row r at slot + TK * D + r * D) into the slot's 16-bit layout (sw128_chunk); rows >= valid become zero
// rows. Run by the NT threads gtid = 0 .. NT - 1 (NT = 64 or 128) of NT / 32 warps, which synchronise on
// named barrier `bar` (NT threads) at head_dim 64. The 16-bit rows overwrite the E4M3 rows in place:
//  - D = 128: a 16-bit row's first column half lies below the E4M3 rows and its second half on the E4M3
//    row of the same key, so each key row belongs to one warp (rows r with r mod (NT / 8) in the warp's
//    four values), which reads all of it before writing it;
//  - D = 64: the 16-bit row r covers E4M3 rows 2r - TK and 2r - TK + 1, so all threads read the whole
//    tile into registers before any of them writes.
// The caller fences the writes for the tensor core and synchronises the NT threads afterwards.
// BLK: each row is widened with its block's scale, of the factors that the threads hold (BlockFactors).
template <int D, int TK, bool BF16, int NT = 64, bool BLK = false>
__device__ __forceinline__ void widen_e4m3_tile(uint8_t* slot, int valid, int gtid, int bar,
                                                const uint32_t (&factor)[TK / NT] = {}) {
    // the factor of the thread's i-th row, from the lane that holds it (every lane takes part)
    auto of_row = [&](int i) -> uint32_t {
        if constexpr (!BLK) return 0u;
        constexpr int LPR = D / 16;
        const uint32_t held = TK / NT > 1 && i >= LPR ? factor[TK / NT - 1] : factor[0];
        return __shfl_sync(0xffffffffu, held, (gtid & 31 & ~(LPR - 1)) | (i & (LPR - 1)));
    };
    static_assert(D == 64 || D == 128, "E4M3 tiles at head_dim 64 and 128");
    static_assert(NT == 64 || NT == 128, "64 or 128 threads");
    const uint8_t* src = slot + TK * D;
    if constexpr (D == 128) {
        constexpr int RS = NT / 8;  // rows one pass of the threads covers
        const int j = gtid & 7;     // codes 16j .. 16j + 15 of a row
        const int r0 = gtid >> 3;   // rows r0 + RS i: warp w holds r0 in [4w, 4w + 4)
#pragma unroll 1
        for (int i0 = 0; i0 < TK / RS; i0 += 4) {
            uint4 in[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int r = r0 + RS * (i0 + u);
                in[u] = r < valid ? *reinterpret_cast<const uint4*>(src + r * D + 16 * j) : make_uint4(0, 0, 0, 0);
            }
            __syncwarp();
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int r = r0 + RS * (i0 + u);
                uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
                const uint32_t fac = of_row(i0 + u);
                if (r < valid) {
                    lo = widen_e4m3x8<BF16, BLK>(make_uint2(in[u].x, in[u].y), fac);
                    hi = widen_e4m3x8<BF16, BLK>(make_uint2(in[u].z, in[u].w), fac);
                }
                *reinterpret_cast<uint4*>(slot + sw128_chunk<TK>(2 * j, r)) = lo;
                *reinterpret_cast<uint4*>(slot + sw128_chunk<TK>(2 * j + 1, r)) = hi;
            }
            __syncwarp();
        }
    } else {
        constexpr int RS = NT / 4;  // rows one pass of the threads covers
        const int j = gtid & 3;     // codes 16j .. 16j + 15 of a row
        const int r0 = gtid >> 2;   // rows r0 + RS i
        uint4 in[TK / RS];
#pragma unroll
        for (int i = 0; i < TK / RS; ++i) {
            const int r = r0 + RS * i;
            in[i] = r < valid ? *reinterpret_cast<const uint4*>(src + r * D + 16 * j) : make_uint4(0, 0, 0, 0);
        }
        asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(NT) : "memory");
#pragma unroll
        for (int i = 0; i < TK / RS; ++i) {
            const int r = r0 + RS * i;
            uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
            const uint32_t fac = of_row(i);
            if (r < valid) {
                lo = widen_e4m3x8<BF16, BLK>(make_uint2(in[i].x, in[i].y), fac);
                hi = widen_e4m3x8<BF16, BLK>(make_uint2(in[i].z, in[i].w), fac);
            }
            *reinterpret_cast<uint4*>(slot + sw128_chunk<TK>(2 * j, r)) = lo;
            *reinterpret_cast<uint4*>(slot + sw128_chunk<TK>(2 * j + 1, r)) = hi;
        }
    }
}

}  // namespace bsp
