// Launch contract of the write-side kernels beside the plain append (RoPE on the append in
// bsp_rope.cu, the append into FP8 E4M3 pools in bsp_append.cu) with the host library.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/bsp.h"
#include "bsp_internal.h"

namespace bsp {

// RoPE on the paged append (bsp_rope.cu).
struct RopeAppendParams {
    const void* k_new;
    const void* v_new;
    int64_t src_row_stride;  // elements
    void* q;                 // may be null: no query rows
    int64_t q_row_stride;    // elements
    const int32_t* loc;
    const int32_t* pos;
    const float* cos_sin;    // [max_pos][rot]
    void* k_pool;
    void* v_pool;
    int32_t* status;
    int n, Hq, Hkv, ps_log2, num_pages;
    int rot, interleaved, max_pos;
    float k_mul, v_mul;      // fp8 pools: quantisation multipliers of K (after the rotation) and V
};
// fp8: the pools are E4M3 bytes (K and V quantised), else the q dtype
cudaError_t launch_rope_append(int head_dim, bool bf16, bool fp8, const RopeAppendParams& p, cudaStream_t stream);
cudaError_t prepare_rope_append(int head_dim, bool bf16, bool fp8);
cudaError_t launch_rope_cos_sin(int max_pos, int rot, double base, float* cos_sin, cudaStream_t stream);

// Append into E4M3 pools (bsp_append.cu).
struct AppendFp8Params {
    const void* k_new;       // 16-bit (bf16 / fp16) or E4M3 rows
    const void* v_new;
    int64_t src_row_stride;  // elements of the source type
    const int32_t* loc;
    uint8_t* k_pool;         // [num_pages][Hkv][ps][D] bytes
    uint8_t* v_pool;
    int32_t* status;
    float k_mul, v_mul;      // quantisation multipliers of a 16-bit source
    int n, Hkv, D, ps_log2, num_pages;
};
// src: 0 bf16, 1 fp16, 2 E4M3 (copied)
cudaError_t launch_append_fp8(int src, const AppendFp8Params& p, cudaStream_t stream);
cudaError_t prepare_append_fp8(int src);

// Exponent bytes of block scales that the attention reads as they are; others, but 0, it takes as the nearest of them.
template <bool BF16>
constexpr int kReadLo = BF16 ? 1 : 112;
template <bool BF16>
constexpr int kReadHi = BF16 ? 142 : 134;

// Normalised and rotated appends (bsp_norm.cu): what K and query rows go through, and the query rows.
struct NormRope {
    const int32_t* loc;
    const int32_t* pos;        // with cos_sin
    const float* cos_sin;      // [max_pos][rot], or null: no rotation
    const void* q;             // may be null: no query rows
    void* q_out;
    int64_t q_stride, q_out_stride;  // elements
    const void* q_weight;      // may be null: ones
    const void* k_weight;
    float eps, weight_offset;
    int norm, weight_fp32;
    int n, Hq, rot, interleaved, max_pos;
};
struct NormAppendParams {
    NormRope a;
    const void* k_new;
    const void* v_new;
    int64_t src_stride;
    void* k_pool;
    void* v_pool;
    uint8_t* k_exp;            // block scales: exponent bytes, and the range that a write chooses from
    uint8_t* v_exp;
    int32_t* status;
    int Hkv, ps_log2, num_pages;
    int block_log2, exp_lo, exp_hi;
    float k_mul, v_mul;        // E4M3 pools with one multiplier per tensor
    // set by launch_norm_append: groups of heads that fill a warp, batches of K (and of V) of a token, all of its
    // batches, warps of a token
    int groups, kv_batches, batches, units;
};
// runs: the tokens are prompts', many of a block next to one another (the kernels differ in speed only)
cudaError_t launch_norm_append(int head_dim, bool bf16, PoolKind pools, bool runs, const NormAppendParams& p,
                               int num_sms, cudaStream_t stream);
cudaError_t launch_rope_scaled(int max_pos, int rot, double base, const bsp_rope_scaling& sc, float* cos_sin,
                               cudaStream_t stream);

}  // namespace bsp
