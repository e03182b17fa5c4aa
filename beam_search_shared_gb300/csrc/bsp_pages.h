// Contract between the host entries of the page bookkeeping (bsp_cache.cpp) and its kernels (bsp_pages.cu).
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "bsp_step.h"

namespace bsp {

struct ForkParams {
    const int32_t* req;
    const int32_t* pages;      // the plan's page table
    const int32_t* plan_hdr;
    const int32_t* beams;
    long long beams_stride;
    const int32_t* refs_in;
    int32_t* refs_out;
    int32_t* pages_out;
    long long out_stride;
    int32_t* base;             // workspace: [rows] first fresh page of a row, -1: none
    int32_t* fresh;            // workspace: [2 rows] fresh pages in order
    int32_t* status;
    PlanShape shape;
    int batch, W, num_forks, rows, num_pages, ps_log2, out_cols;
};
cudaError_t launch_fork_tables(const ForkParams& p, cudaStream_t stream);

struct ForkRowsParams {
    const int32_t* req;
    const int32_t* pages;
    const int32_t* plan_hdr;
    const int32_t* beams;
    long long beams_stride;
    const int32_t* pages_out;
    long long out_stride;
    const int32_t* beam_pages;
    const int32_t* ci;
    uint8_t* k_pool;
    uint8_t* v_pool;
    uint8_t* k_exp;            // null: no block scales
    uint8_t* v_exp;
    int32_t* status;
    PlanShape shape;
    int W, num_forks, rows, num_pages, Hkv, ps_log2, row_bytes, block_log2, out_cols, beam_cols, max_seq;
    int read_lo, read_hi;      // exponent bytes that the attention reads as they are
    int heads, per_row;        // set by launch_fork_rows: heads of a CTA, CTAs of a row
};
cudaError_t launch_fork_rows(ForkRowsParams p, int num_sms, cudaStream_t stream);

struct FreeParams {
    const int32_t* tables;
    long long stride;
    int32_t* refs_out;
    int32_t* status;
    int rows, cols, num_pages;
};
cudaError_t launch_free_pages(const FreeParams& p, const int32_t* refs_in, int num_sms, cudaStream_t stream);

struct CompactParams {
    const int32_t* refs_in;
    int32_t* refs_out;
    int32_t* pairs;
    int32_t* count;
    int32_t* remap;
    const int32_t* tables_in;
    int32_t* tables_out;
    long long stride;
    int32_t* status;
    int rows, cols, num_pages;
};
cudaError_t launch_compact_tables(const CompactParams& p, int num_sms, cudaStream_t stream);

struct CopyParams {
    const int32_t* pairs;
    const int32_t* count;
    uint8_t* k_pool;
    uint8_t* v_pool;
    uint8_t* k_exp;
    uint8_t* v_exp;
    int32_t* status;
    long long page_bytes;
    int max_pairs, num_pages, exp_bytes;
};
cudaError_t launch_copy_pages(const CopyParams& p, int num_sms, cudaStream_t stream);

}  // namespace bsp
