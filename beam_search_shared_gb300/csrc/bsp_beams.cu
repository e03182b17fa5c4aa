// Beam bookkeeping after the beams of a step are chosen (bsp_beam_advance).
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/bsp.h"
#include "bsp_step.h"

namespace bsp {
namespace {

constexpr int kAdvThreads = 512;

// One CTA per request. The tail columns of cache_indirection and of the generated tokens are gathered by
// parent through shared memory, `cols` columns of both at a time: everything a round overwrites has been
// read before, so the outputs may be the inputs. A few KB per request: the launch and two dependent loads
// bound it (one request of 4 beams 2.5 us, 128 requests of 96 beams 3.4 us, of which an empty launch is about 2).
__global__ void __launch_bounds__(kAdvThreads) beam_advance_kernel(const AdvanceParams p) {
    extern __shared__ int32_t s_buf[];  // [2][cols][W]
    const int b = blockIdx.x, tid = threadIdx.x, W = p.W;
    if (!plan_matches(p.plan_hdr, p.batch, p.W, 0)) {
        if (tid == 0 && b == 0) atomicOr(p.status, BSP_DEVFLAG_GRAPH);
        return;
    }
    const int P = __ldg(p.req + static_cast<long long>(b) * kReqFields + kReqPrefix);
    const int T = __ldg(p.req + static_cast<long long>(b) * kReqFields + kReqTail);
    const bool ci_on = p.ci_in != nullptr, tok_on = p.tok_out != nullptr;
    if ((ci_on && P + T >= p.max_seq) || (tok_on && T >= p.tok_cols)) {  // a replayed plan that outgrew the tables
        if (tid == 0) atomicOr(p.status, BSP_DEVFLAG_GRAPH);
        return;
    }
    const long long row0 = static_cast<long long>(b) * W;
    const int32_t* parent = p.parents + b * p.cand_stride;
    for (int c0 = 0; c0 < T; c0 += p.cols) {
        const int n = min(p.cols, T - c0);
        for (int i = tid; i < W * n; i += kAdvThreads) {
            const int w = i / n, c = i - w * n;
            int from = __ldg(parent + w);
            if (from < 0 || from >= W) from = w;
            if (ci_on) s_buf[i] = p.ci_in[(row0 + from) * p.max_seq + P + c0 + c];
            if (tok_on) s_buf[W * p.cols + i] = p.tok_in[(row0 + from) * p.tok_stride + c0 + c];
        }
        __syncthreads();
        for (int i = tid; i < W * n; i += kAdvThreads) {
            const int w = i / n, c = i - w * n;
            if (ci_on) p.ci_out[(row0 + w) * p.max_seq + P + c0 + c] = s_buf[i];
            if (tok_on) p.tok_out[(row0 + w) * p.tok_stride + c0 + c] = s_buf[W * p.cols + i];
        }
        __syncthreads();
    }
    for (int w = tid; w < W; w += kAdvThreads) {
        const int from = __ldg(parent + w);
        if (from < -1 || from >= W) atomicOr(p.status, BSP_DEVFLAG_PAGE_INDEX);
        if (ci_on) p.ci_out[(row0 + w) * p.max_seq + P + T] = w;  // the new token's row is the beam's own
        if (tok_on) p.tok_out[(row0 + w) * p.tok_stride + T] = __ldg(p.chosen + b * p.cand_stride + w);
        if (p.token_len) p.token_len[row0 + w] = T + 1;
    }
}

}  // namespace

cudaError_t launch_advance(const AdvanceParams& p, cudaStream_t stream) {
    const size_t smem = static_cast<size_t>(2) * p.cols * p.W * 4;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(beam_advance_kernel), smem, kAdvanceSmem);
    if (e != cudaSuccess) return e;
    beam_advance_kernel<<<p.batch, kAdvThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace bsp
