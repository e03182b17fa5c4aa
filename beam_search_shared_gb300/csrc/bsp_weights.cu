// Accumulated attention weight of cached keys (bsp_key_weights): for every (request b, kv head g, key j of its
// prompt)
//   weights[b][g][j] (+)= sum over query rows r of b and heads h of g of exp(scale * q[r][h] . k[j] - lse[r][h]),
// the mass that the rows' softmax gave the key. It is one contraction and a row sum, so the product is taken
// transposed, S^T = K Q^T: a tile of 128 keys is the MMA's M and up to 256 query rows its N. A key is then one
// TMEM lane, hence one thread, and the sum over query rows runs along the lane's columns in registers: no
// reduction across threads, no atomics, the same order on every run.
//
// Work item = (b, g, 128 keys). Its K tile is loaded once; the query rows pass in blocks of at most 256 (128
// at head_dim 256). A CTA takes a contiguous run of items when one block holds all rows of a (b, g), so that Q
// stays in shared memory from one tile to the next, and every gridDim-th item otherwise.
//
// Warps: 0 loads K tiles (TMA boxes of a page, or 64 rows of one) and Q blocks; 1 issues tcgen05.mma into two
// TMEM accumulators by turns; 2 stages the blocks' -lse; 4-11 sum, warps 4-7 the even and 8-11 the odd
// 32-column chunks; 12-15 (E4M3 pools) widen the K tiles to the q dtype. Bounds, at 192 rows per (b, g) and
// head_dim 128: K from HBM once, and one exp2 per (row, key, head) pair.
// Every wait is bounded (1 s without progress); on expiry the CTA flags BSP_DEVFLAG_TIMEOUT, drains its own
// copies and MMAs, frees TMEM and exits.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/bsp.h"
#include "bsp_internal.h"
#include "bsp_prompt.cuh"
#include "bsp_ptx.cuh"

namespace bsp {
namespace {

constexpr int TK = 128;                             // keys per tile (MMA M)
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr uint64_t kDrainWaitNs = 200000000ull;
constexpr uint32_t FULL = 0xffffffffu;

struct Bars {
    uint64_t k_full[8], k_ready[8], k_empty[8];
    uint64_t q_full[2], q_empty[2];
    uint64_t lse_full[2], lse_empty[2];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t part_full[4];
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(Bars) <= kWeightsBarBytes, "barrier area");

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// (d0, d1) = (a0, a1) * b + (c0, c1)
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b, float c0, float c1) {
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\t"
        "mov.b64 rb, {%4, %4};\n\t"
        "mov.b64 rc, {%5, %6};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rc;\n\t"
        "mov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b), "f"(c0), "f"(c1));
}

// The items of a CTA in order. Every role walks the same sequence.
struct Walk {
    const WeightsParams& p;
    const int* cum;       // [batch + 1] key tiles of the requests before b
    long long at, end, step;
    int b = 0, last_b = -1, last_g = -1;
    bool last_single = false;
    // the current item
    int g = 0, kt = 0, P = 0, page_off = 0, row0 = 0, seen = 0, cbase = 0, rb = 0, nrb = 0;
    bool causal = false, new_q = false;

    __device__ __forceinline__ Walk(const WeightsParams& p_, const int* cum_) : p(p_), cum(cum_) {
        const long long total = static_cast<long long>(cum[p.batch]) * p.Hkv;
        if (p.strided) {
            at = blockIdx.x;
            end = total;
            step = gridDim.x;
        } else {
            at = total * blockIdx.x / gridDim.x;
            end = total * (blockIdx.x + 1) / gridDim.x;
            step = 1;
        }
        if (at < end) {
            int lo = 0, hi = p.batch - 1;  // the last request whose tiles begin at or before the item
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (static_cast<long long>(cum[mid]) * p.Hkv <= at) lo = mid; else hi = mid - 1;
            }
            b = lo;
        }
    }
    __device__ __forceinline__ bool more() const { return at < end; }
    // reads the item at `at`; its query-row blocks are rb .. nrb - 1
    __device__ __forceinline__ void open() {
        while (static_cast<long long>(cum[b + 1]) * p.Hkv <= at) ++b;
        const int nt = cum[b + 1] - cum[b];
        const int rem = static_cast<int>(at - static_cast<long long>(cum[b]) * p.Hkv);
        g = rem / nt;
        kt = rem - g * nt;
        const int32_t* r = p.req + static_cast<long long>(b) * kReqFields;
        P = __ldg(r + kReqPrefix);
        page_off = __ldg(r + kReqPageOff);
        const int rows = __ldg(r + kReqRows), c = __ldg(r + kReqCausal);
        seen = p.window > 0 ? min(p.window, rows) : rows;
        row0 = __ldg(r + kReqRowOff) + rows - seen;
        causal = c >= 0;
        cbase = c + rows - seen;  // causal: row i of the seen ones sees keys 0 .. cbase + i
        nrb = (seen + p.block_rows - 1) / p.block_rows;
        rb = causal ? max(0, kt * TK - cbase) / p.block_rows : 0;
        new_q = !(nrb == 1 && last_single && b == last_b && g == last_g);
        last_b = b;
        last_g = g;
        last_single = nrb == 1;
    }
    __device__ __forceinline__ void next() { at += step; }
};

template <int D, bool BF16, bool FP8>
__global__ void __launch_bounds__(FP8 ? 512 : 384, 1)
key_weights_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const WeightsParams p) {
    constexpr int NC = D / 64;
    constexpr int K_BYTES = TK * D * 2;
    constexpr int THREADS = FP8 ? 512 : 384;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int NS = p.mma_n;                         // rows of a Q block as the MMA sees it
    const int q_bytes = NC * NS * 128;
    const int NQ = p.q_slots, KST = p.k_slots;
    auto q_buf = [&](int i) { return smem + (i % NQ) * q_bytes; };
    auto k_buf = [&](int i) { return smem + NQ * q_bytes + (i % KST) * K_BYTES; };
    uint8_t* rest = smem + NQ * q_bytes + KST * K_BYTES;
    float* s_nlse = reinterpret_cast<float*>(rest);                 // [2][256]
    float* s_part = s_nlse + 512;                                   // [4][128]
    Bars* bars = reinterpret_cast<Bars*>(s_part + 512);
    int* s_cum = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + kWeightsBarBytes);  // [batch + 1]
    volatile int* abort_flag = &bars->abort_flag;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (!plan_matches(p.plan_hdr, p.batch, p.plan_w, p.plan_kind)) {
        if (tid == 0 && blockIdx.x == 0) atomicOr(p.status, BSP_DEVFLAG_GRAPH);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < KST; ++i) {
            mbar_init(&bars->k_full[i], 1);
            mbar_init(&bars->k_ready[i], 4);   // one arrival per widening warp
            mbar_init(&bars->k_empty[i], 1);   // the first summing warp, when it sees the item's last product
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->q_full[i], 1);
            mbar_init(&bars->q_empty[i], 1);
            mbar_init(&bars->lse_full[i], 1);
            mbar_init(&bars->lse_empty[i], 8);
            mbar_init(&bars->acc_full[i], 1);
            mbar_init(&bars->acc_empty[i], 8);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&bars->part_full[i], 4);
        mbar_init(&bars->drain, 1);
        bars->abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
    }
    for (int b = tid; b < p.batch; b += THREADS) {
        const int P = __ldg(p.req + static_cast<long long>(b) * kReqFields + kReqPrefix);
        const bool fits = P <= p.max_keys;
        if (!fits && blockIdx.x == 0) atomicOr(p.status, BSP_DEVFLAG_GRAPH);  // a replayed plan that outgrew `weights`
        s_cum[b + 1] = fits ? (P + TK - 1) / TK : 0;
    }
    if (tid == 0) s_cum[0] = 0;
    if (warp == 1) tmem_alloc(&bars->tmem_base, 512);
    __syncthreads();
    if (warp == 0) {
        int before = 0;
        for (int b0 = 0; b0 < p.batch; b0 += 32) {
            int v = b0 + lane < p.batch ? s_cum[b0 + lane + 1] : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(FULL, v, d);
                if (lane >= d) v += o;
            }
            if (b0 + lane < p.batch) s_cum[b0 + lane + 1] = before + v;
            before += __shfl_sync(FULL, v, 31);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    const int ps = 1 << p.ps_log2;

    if (warp == 0) {
        // ================= loads
        const int BR = min(ps, 64);
        int kn = 0, qn = 0;
        bool ok = true;
        for (Walk w(p, s_cum); w.more() && ok; w.next(), ++kn) {
            w.open();
            // K of the item
            if (kn >= KST) ok = __all_sync(FULL, mbar_wait(&bars->k_empty[kn % KST], ((kn / KST) - 1) & 1, abort_flag, kWaitNs));
            if (!ok) break;
            const int key0 = w.kt * TK;
            const int valid = min(TK, w.P - key0);
            const int nchunks = (valid + BR - 1) / BR;
            uint64_t* full = &bars->k_full[kn % KST];
            if (lane == 0) mbar_arrive_expect_tx(full, nchunks * BR * D * (FP8 ? 1 : 2));
            __syncwarp();
            constexpr int NB = FP8 ? 1 : NC;  // boxes of a chunk: column halves (E4M3: whole rows)
            for (int bx = lane; bx < nchunks * NB; bx += 32) {
                const int ch = bx / NB, c = bx - ch * NB;
                const int key = key0 + ch * BR;
                int page = __ldg(p.pages + w.page_off + (key >> p.ps_log2));
                if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.num_pages)) {
                    atomicOr(p.status, BSP_DEVFLAG_PAGE_INDEX);
                    page = 0;
                }
                const int row = ((page * p.Hkv + w.g) << p.ps_log2) + (key & (ps - 1));
                if constexpr (FP8)
                    tma_load_2d(k_buf(kn) + TK * D + ch * BR * D, &tm_k, full, 0, row);
                else
                    tma_load_2d(k_buf(kn) + c * TK * 128 + ch * BR * 128, &tm_k, full, c * 64, row);
            }
            __syncwarp();
            for (int rb = w.rb; rb < w.nrb && w.new_q; ++rb, ++qn) {
                if (qn >= NQ) ok = __all_sync(FULL, mbar_wait(&bars->q_empty[qn % NQ], ((qn / NQ) - 1) & 1, abort_flag, kWaitNs));
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&bars->q_full[qn % NQ], NC * p.block_rows * p.G * 128);
                    for (int c = 0; c < NC; ++c)
                        tma_load_3d(q_buf(qn) + c * NS * 128, &tm_q, &bars->q_full[qn % NQ], c * 64, w.g * p.G,
                                    w.row0 + rb * p.block_rows);
                }
                __syncwarp();
            }
        }
        if (!ok) {
            if (lane == 0) {
                *abort_flag = 1;
                atomicOr(p.status, BSP_DEVFLAG_TIMEOUT);
            }
            // drain: this CTA's own copies land before it exits
            const uint64_t t0 = globaltimer_ns();
            for (int j = max(0, kn - KST); j <= kn; ++j)
                while (!mbar_try_wait(&bars->k_full[j % KST], (j / KST) & 1) && globaltimer_ns() - t0 < kDrainWaitNs) {
                }
            for (int j = max(0, qn - NQ); j <= qn; ++j)
                while (!mbar_try_wait(&bars->q_full[j % NQ], (j / NQ) & 1) && globaltimer_ns() - t0 < kDrainWaitNs) {
                }
        }
    } else if (warp == 1) {
        // ================= products
        if (lane == 0) {
            const uint32_t idesc = idesc_f16(TK, NS, BF16, false);
            int kn = 0, qn = -1, step = 0;
            bool ok = true;
            for (Walk w(p, s_cum); w.more() && ok; w.next(), ++kn) {
                w.open();
                ok = mbar_wait(FP8 ? &bars->k_ready[kn % KST] : &bars->k_full[kn % KST], (kn / KST) & 1, abort_flag, kWaitNs);
                if (!ok) break;
                const uint32_t k_addr = smem_u32(k_buf(kn));
                for (int rb = w.rb; rb < w.nrb; ++rb, ++step) {
                    if (w.new_q) {
                        ++qn;
                        ok = mbar_wait(&bars->q_full[qn % NQ], (qn / NQ) & 1, abort_flag, kWaitNs);
                        if (!ok) break;
                    }
                    const int a = step & 1;
                    if (step >= 2) ok = mbar_wait(&bars->acc_empty[a], ((step >> 1) - 1) & 1, abort_flag, kWaitNs);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t q_addr = smem_u32(q_buf(qn));
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint64_t ad = sdesc_sw128(k_addr + (kk >> 2) * (TK * 128) + (kk & 3) * 32, 16, 1024);
                        const uint64_t bd = sdesc_sw128(q_addr + (kk >> 2) * (NS * 128) + (kk & 3) * 32, 16, 1024);
                        mma_f16(tmem + a * 256, ad, bd, idesc, kk > 0 ? 1u : 0u);
                    }
                    mma_commit(&bars->acc_full[a]);
                }
            }
            if (!ok) {
                *abort_flag = 1;
                atomicOr(p.status, BSP_DEVFLAG_TIMEOUT);
            }
            // drain: every MMA issued by this thread completes before TMEM is freed
            mma_commit(&bars->drain);
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(&bars->drain, 0) && globaltimer_ns() - t0 < kDrainWaitNs) {
            }
        }
    } else if (warp == 2) {
        // ================= -lse of each Q block, in base 2; -inf for rows without one
        int qn = 0;
        bool ok = true;
        for (Walk w(p, s_cum); w.more() && ok; w.next()) {
            w.open();
            for (int rb = w.rb; rb < w.nrb && w.new_q; ++rb, ++qn) {
                const int i0 = rb * p.block_rows;
                const int n = min(p.block_rows, w.seen - i0) * p.G;
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int c = lane + 32 * j;
                    v[j] = -INFINITY;
                    if (c < n) {
                        const int i = c / p.G;
                        const float l = __ldg(p.lse + static_cast<long long>(w.row0 + i0 + i) * p.Hq + w.g * p.G + (c - i * p.G));
                        v[j] = l == -INFINITY ? -INFINITY : -l * p.lse_mul;
                    }
                }
                if (qn >= 2) ok = __all_sync(FULL, mbar_wait(&bars->lse_empty[qn & 1], ((qn >> 1) - 1) & 1, abort_flag, kWaitNs));
                if (!ok) break;
#pragma unroll
                for (int j = 0; j < 8; ++j) s_nlse[(qn & 1) * 256 + lane + 32 * j] = v[j];
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->lse_full[qn & 1]);
            }
        }
        if (!ok && lane == 0) {
            *abort_flag = 1;
            atomicOr(p.status, BSP_DEVFLAG_TIMEOUT);
        }
    } else if (warp >= 4 && warp < 12) {
        // ================= sums: thread <-> key <-> TMEM lane
        const int quad = warp & 3, odd = warp >= 8 ? 1 : 0;
        const int key_lane = quad * 32 + lane;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        const float c2 = p.scale_log2;
        int kn = 0, qn = -1, step = 0;
        bool ok = true;
        for (Walk w(p, s_cum); w.more() && ok; w.next(), ++kn) {
            w.open();
            const int key = w.kt * TK + key_lane;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
            for (int rb = w.rb; rb < w.nrb; ++rb, ++step) {
                const int a = step & 1;
                if (w.new_q) {
                    // the block before is done with: its products are complete and its -lse read
                    if (qn >= 0 && lane == 0) {
                        mbar_arrive(&bars->lse_empty[qn & 1]);
                        if (warp == 4) mbar_arrive(&bars->q_empty[qn % NQ]);
                    }
                    ++qn;
                    ok = mbar_wait(&bars->lse_full[qn & 1], (qn >> 1) & 1, abort_flag, kWaitNs);
                    ok = __all_sync(FULL, ok);
                    if (!ok) break;
                }
                ok = mbar_wait(&bars->acc_full[a], (step >> 1) & 1, abort_flag, kWaitNs);
                ok = __all_sync(FULL, ok);
                if (!ok) break;
                tc_fence_after();
                if (warp == 4 && lane == 0 && rb == w.nrb - 1) mbar_arrive(&bars->k_empty[kn % KST]);
                const int i0 = rb * p.block_rows;
                const int n = min(p.block_rows, w.seen - i0) * p.G;
                // columns below cmin are rows that do not see this thread's key
                const int cmin = w.causal ? max(0, key - w.cbase - i0) * p.G : 0;
                const bool all_see = !w.causal || w.kt * TK + TK - 1 <= w.cbase + i0;
                const float* nl = s_nlse + (qn & 1) * 256;
                for (int c0 = odd * 32; c0 < n; c0 += 64) {
                    uint32_t s[32];
                    tmem_ld32(lane_base + a * 256 + c0, s);
                    tmem_wait_ld();
                    if (all_see && c0 + 32 <= n) {
#pragma unroll
                        for (int c = 0; c < 32; c += 4) {
                            const float4 l = *reinterpret_cast<const float4*>(nl + c0 + c);
                            float e0, e1, e2, e3;
                            fma2(e0, e1, __uint_as_float(s[c]), __uint_as_float(s[c + 1]), c2, l.x, l.y);
                            fma2(e2, e3, __uint_as_float(s[c + 2]), __uint_as_float(s[c + 3]), c2, l.z, l.w);
                            add2_acc(sum[0], sum[1], ex2(e0), ex2(e1));
                            add2_acc(sum[2], sum[3], ex2(e2), ex2(e3));
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            const float e = ex2(fmaf(__uint_as_float(s[c]), c2, nl[c0 + c]));
                            sum[c & 3] += (c0 + c < n && c0 + c >= cmin) ? e : 0.f;
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->acc_empty[a]);
            }
            if (!ok) break;
            const float mine = (sum[0] + sum[1]) + (sum[2] + sum[3]);
            // The odd chunks' sums pass through shared memory, in four slots by turns: item kn + 4 is summed
            // only once both halves have left the accumulator of item kn + 2, so its slot has been read.
            if (odd) {
                s_part[(kn & 3) * 128 + key_lane] = mine;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->part_full[kn & 3]);
            } else {
                ok = mbar_wait(&bars->part_full[kn & 3], (kn >> 2) & 1, abort_flag, kWaitNs);
                ok = __all_sync(FULL, ok);
                if (!ok) break;
                if (key < w.P) {
                    float* out = p.weights + (static_cast<long long>(w.b) * p.Hkv + w.g) * p.stride + key;
                    const float v = mine + s_part[(kn & 3) * 128 + key_lane];
                    *out = p.accumulate ? *out + v : v;
                }
            }
        }
        if (!ok && lane == 0) {
            *abort_flag = 1;
            atomicOr(p.status, BSP_DEVFLAG_TIMEOUT);
        }
    } else if (FP8 && warp >= 12) {
        // ================= E4M3 tiles widened to the q dtype in their slots
        if constexpr (FP8) {
            int kn = 0;
            bool ok = true;
            for (Walk w(p, s_cum); w.more(); w.next(), ++kn) {
                w.open();
                ok = mbar_wait(&bars->k_full[kn % KST], (kn / KST) & 1, abort_flag, kWaitNs);
                // the four warps go on, or leave, together
                uint32_t all;
                asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                             "barrier.cta.red.and.pred q, 2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                             : "=r"(all) : "r"(ok ? 1u : 0u) : "memory");
                ok = all != 0;
                if (!ok) break;
                widen_e4m3_tile<D, TK, BF16, 128>(k_buf(kn), min(TK, w.P - w.kt * TK), tid - 384, 1);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->k_ready[kn % KST]);
            }
            if (!ok && lane == 0) {
                *abort_flag = 1;
                atomicOr(p.status, BSP_DEVFLAG_TIMEOUT);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, bool BF16, bool FP8>
cudaError_t launch_t(const CUtensorMap& tq, const CUtensorMap& tk, const WeightsParams& p, int ctas, size_t smem,
                     cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(key_weights_kernel<D, BF16, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    key_weights_kernel<D, BF16, FP8><<<ctas, FP8 ? 512 : 384, smem, stream>>>(tq, tk, p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_weights(int head_dim, bool bf16, bool fp8, const CUtensorMap& tq, const CUtensorMap& tk,
                           const WeightsParams& p, int ctas, size_t smem, cudaStream_t stream) {
    if (fp8) {
        if (head_dim == 64)
            return bf16 ? launch_t<64, true, true>(tq, tk, p, ctas, smem, stream) : launch_t<64, false, true>(tq, tk, p, ctas, smem, stream);
        if (head_dim == 128)
            return bf16 ? launch_t<128, true, true>(tq, tk, p, ctas, smem, stream) : launch_t<128, false, true>(tq, tk, p, ctas, smem, stream);
        return cudaErrorInvalidValue;
    }
    if (head_dim == 64)
        return bf16 ? launch_t<64, true, false>(tq, tk, p, ctas, smem, stream) : launch_t<64, false, false>(tq, tk, p, ctas, smem, stream);
    if (head_dim == 128)
        return bf16 ? launch_t<128, true, false>(tq, tk, p, ctas, smem, stream) : launch_t<128, false, false>(tq, tk, p, ctas, smem, stream);
    return bf16 ? launch_t<256, true, false>(tq, tk, p, ctas, smem, stream) : launch_t<256, false, false>(tq, tk, p, ctas, smem, stream);
}

}  // namespace bsp
