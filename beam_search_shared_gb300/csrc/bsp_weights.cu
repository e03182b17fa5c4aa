// Accumulated attention weight of cached keys (bsp_key_weights): for every (request b, kv head g, key j of its
// prompt)
//   weights[b][g][j] (+)= sum over query rows r of b and heads h of g of exp(scale * q[r][h] . k[j] - lse[r][h]),
// the mass that the rows' softmax gave the key. It is one contraction and a row sum, so the product is taken
// transposed, S^T = K Q^T: a tile of 128 keys is the MMA's M and up to 256 query rows its N. A key is then one
// TMEM lane, hence one thread, and the sum over query rows runs along the lane's columns in registers: no
// reduction across threads, no atomics, the same order on every run.
//
// Work item = (b, g, 128 keys). Its K tile is loaded once; the query rows pass in blocks of at most 256 (128
// at head_dim 256). A CTA takes a contiguous run of items: where one block holds all rows of a (b, g), Q stays in
// shared memory from one tile to the next, else its blocks in L2 (32 requests of 96 beams, group 4, D = 128, 2000
// keys, two blocks: 100 us, and 115 with every gridDim-th item to a CTA).
//
// Warps: 0 loads K tiles (TMA boxes of a page, or 64 rows of one), 2 the Q blocks; 1 issues tcgen05.mma into four
// TMEM accumulators of 128 columns, or two of 256; 4-19 sum: four sets of four warps (one per lane quadrant);
// 20-23 (E4M3 pools) widen the K tiles to the q dtype; 3 fills up the first warpgroup. Up to 128 rows, the sets
// take items by turns; above, two sets take the halves of an item's columns and two the next one's, and the
// second half's sums pass through shared memory. An item costs a summing warp some 200 instructions of its own,
// at latencies that the sets hide from one another.
//
// Measured at batch 128, 96 beams, 16/8 heads, D = 128, bf16, 2800-3200 keys (192 rows per (b, g); K is 0.79 GB
// and q, lse and the weights 0.06 GB): 165 us, 5.1 TB/s, 0.75 of what a copy reaches. The same kernel without the
// sums takes 157 us, with all warps on one tile and the columns dealt among them 237 us at the best warp
// count, with the halves as products of their own (K read twice from shared memory) 227 us. Per tile and SM:
// K from HBM 0.7 us, the products 0.5 us, one exp2 per (row, key, head) pair 0.4 us; K bounds it.
// A weight is good to some 2^-21: the hardware's exp2 is off by 2^-22, its argument, whose -lse log2(e) is one fp32 number
// so that a packed FMA does the whole, by 2^-23 of lse (itself fp32, off by as much), the fp32 product by less.
// Every wait is bounded (1 s without progress); on expiry the CTA flags BSP_DEVFLAG_TIMEOUT, drains its own
// copies and MMAs, frees TMEM and exits.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/bsp.h"
#include "bsp_step.h"
#include "bsp_prompt.cuh"
#include "bsp_ptx.cuh"

namespace bsp {
namespace {

constexpr int TK = 128;                             // keys per tile (MMA M)
constexpr int kSets = 4;                            // sets of four summing warps
constexpr int kSumWarps = 4 * kSets;
constexpr int kSetCols = 128;                       // TMEM columns of an accumulator
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr uint64_t kDrainWaitNs = 200000000ull;
constexpr uint32_t FULL = 0xffffffffu;

struct Bars {
    uint64_t k_full[8], k_ready[8], k_empty[8];
    uint64_t q_full[2], q_clean[2], q_empty[2];
    uint64_t lse_full[kSets];   // a set's -lse of a new block
    uint64_t acc_full[kSets], acc_empty[kSets];
    uint64_t part_full[2][2];   // the second half's sums of an item of the pair of sets, in either place
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
// a load that stays where it is written, before the waits that follow
__device__ __forceinline__ void ld_early(float& d, const float* p) {
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(d) : "l"(p));
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

// The items of a CTA in order: all of them, or from the `from`-th on every `every`-th. A request's record is read
// once, and an item that follows its predecessor costs no division.
struct Walk {
    const WeightsParams* pp;
    const int* cum;       // [batch + 1] key tiles of the requests before b
    long long at, end;
    int every;
    int b = -1, last_b = -1, last_g = -1;
    int nt = 0;           // key tiles of request b
    // the current item: kv head, key tile; its request's keys, pages, first row, rows, blocks of rows; the blocks
    // it takes are rb .. nrb - 1
    int g = 0, kt = 0, P = 0, page_off = 0, row0 = 0, seen = 0, cbase = 0, rb = 0, nrb = 0;
    bool causal = false, new_q = false;

    __device__ __forceinline__ Walk(const WeightsParams& p, const int* cum_, int from = 0, int every_ = 1) : pp(&p), cum(cum_), every(every_) {
        const long long total = static_cast<long long>(cum[p.batch]) * p.Hkv;
        at = total * blockIdx.x / gridDim.x + from;
        end = total * (blockIdx.x + 1) / gridDim.x;
    }
    __device__ __forceinline__ bool more() const { return at < end; }
    __device__ __forceinline__ void next() { at += every; }
    __device__ __forceinline__ void open() {
        if (b >= 0) {
            kt += every;
            while (kt >= nt) {
                kt -= nt;
                if (++g == pp->Hkv) {
                    g = 0;
                    int to = b + 1;
                    while (cum[to + 1] == cum[to]) ++to;  // (there is one: the item exists)
                    read(to);
                }
            }
        } else {
            int lo = 0, hi = pp->batch - 1;  // the last request whose tiles begin at or before the item
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (static_cast<long long>(cum[mid]) * pp->Hkv <= at) lo = mid; else hi = mid - 1;
            }
            if (lo != b) read(lo);
            const int rem = static_cast<int>(at - static_cast<long long>(cum[b]) * pp->Hkv);
            g = rem / nt;
            kt = rem - g * nt;
        }
        rb = causal ? max(0, kt * TK - cbase) / pp->block_rows : 0;
        new_q = nrb != 1 || b != last_b || g != last_g;
        last_b = nrb == 1 ? b : -1;
        last_g = g;
    }

private:
    __device__ __forceinline__ void read(int to) {
        b = to;
        nt = cum[b + 1] - cum[b];
        const int32_t* r = pp->req + static_cast<long long>(b) * kReqFields;
        P = __ldg(r + kReqPrefix);
        page_off = __ldg(r + kReqPageOff);
        const int rows = __ldg(r + kReqRows), c = __ldg(r + kReqCausal);
        seen = pp->window > 0 ? min(pp->window, rows) : rows;
        row0 = __ldg(r + kReqRowOff) + rows - seen;
        causal = c >= 0;
        cbase = c + rows - seen;  // causal: row i of the seen ones sees keys 0 .. cbase + i
        nrb = (seen + pp->block_rows - 1) / pp->block_rows;
    }
};

// A place in a ring of n slots and the parity of its present round. A consumer waits for `parity`, a producer for
// the other one (which a fresh barrier counts as passed).
struct Ring {
    int n, slot = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ explicit Ring(int n_) : n(n_) {}
    __device__ __forceinline__ void next() {
        if (++slot == n) {
            slot = 0;
            parity ^= 1;
        }
    }
};

__host__ __device__ constexpr int weights_threads(bool fp8) { return 32 * (4 + kSumWarps + (fp8 ? 4 : 0)); }

template <int D, bool BF16, bool FP8>
__global__ void __launch_bounds__(weights_threads(FP8), 1)
key_weights_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const WeightsParams p) {
    constexpr int NC = D / 64;
    constexpr int K_BYTES = TK * D * 2;
    constexpr int THREADS = weights_threads(FP8);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int NS = p.mma_n;                         // rows of a Q block as the MMA sees it
    const int q_bytes = NC * NS * 128;
    const int NQ = p.q_slots, KST = p.k_slots;
    const bool halves = NS > kSetCols;              // a block's columns go to two sets
    const int NU = halves ? (NS / 2 + 31) / 32 * 32 : NS;  // columns of the first
    const int accs = halves ? 2 : kSets;            // accumulators
    const int acc_cols = 4 * kSetCols / accs;
    auto q_buf = [&](int slot) { return smem + slot * q_bytes; };
    auto k_buf = [&](int slot) { return smem + NQ * q_bytes + slot * K_BYTES; };
    uint8_t* rest = smem + NQ * q_bytes + KST * K_BYTES;
    float* s_nlse = reinterpret_cast<float*>(rest);                 // [kSets][2][128]: -lse of the present block and the next
    float* s_part = s_nlse + kSets * 2 * kSetCols;                  // [2][2][128]: of each pair of sets, two items
    Bars* bars = reinterpret_cast<Bars*>(s_part + 2 * 2 * TK);
    int* s_cum = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + kWeightsBarBytes);  // [batch + 1]
    volatile int* abort_flag = &bars->abort_flag;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (!plan_matches(p.plan_hdr, p.shape)) {
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
            mbar_init(&bars->q_clean[i], 1);  // its rows without a log-sum-exp are 0
            mbar_init(&bars->q_empty[i], 1);  // the block's last product completed
            mbar_init(&bars->part_full[0][i], 4);
            mbar_init(&bars->part_full[1][i], 4);
        }
        for (int i = 0; i < kSets; ++i) {
            mbar_init(&bars->lse_full[i], 4);
            mbar_init(&bars->acc_full[i], 1);
            mbar_init(&bars->acc_empty[i], p.mma_n > kSetCols ? 8 : 4);
        }
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
        Ring k(KST);
        bool ok = true;
        Walk w(p, s_cum);
        // lane ch: the page of the tile's chunk ch (at most 16 chunks), fetched an item ahead
        auto page_of = [&](const Walk& at) -> int {
            const int key = at.kt * TK + lane * BR;
            return lane < TK / BR && key < at.P ? __ldg(p.pages + at.page_off + (key >> p.ps_log2)) : 0;
        };
        int page_next = 0;
        if (w.more()) {
            w.open();
            page_next = page_of(w);
        }
        while (w.more() && ok) {
            const int pages = page_next;
            Walk ahead = w;
            ahead.next();
            if (ahead.more()) {
                ahead.open();
                page_next = page_of(ahead);
            }
            // K of the item
            ok = __all_sync(FULL, mbar_wait(&bars->k_empty[k.slot], k.parity ^ 1, abort_flag, kWaitNs));
            if (!ok) break;
            const int key0 = w.kt * TK;
            const int valid = min(TK, w.P - key0);
            const int nchunks = (valid + BR - 1) / BR;
            uint64_t* full = &bars->k_full[k.slot];
            uint8_t* tile = k_buf(k.slot);
            if (lane == 0) mbar_arrive_expect_tx(full, nchunks * BR * D * (FP8 ? 1 : 2));
            __syncwarp();
            constexpr int NB = FP8 ? 1 : NC;  // boxes of a chunk: column halves (E4M3: whole rows)
            for (int b0 = 0; b0 < nchunks * NB; b0 += 32) {
                const int bx = b0 + lane, ch = min(bx / NB, nchunks - 1), c = bx % NB;
                int page = __shfl_sync(FULL, pages, ch);
                if (bx >= nchunks * NB) continue;
                if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.num_pages)) {
                    atomicOr(p.status, BSP_DEVFLAG_PAGE_INDEX);
                    page = 0;
                }
                const int row = ((page * p.Hkv + w.g) << p.ps_log2) + ((key0 + ch * BR) & (ps - 1));
                if constexpr (FP8)
                    tma_load_2d(tile + TK * D + ch * BR * D, &tm_k, full, 0, row);
                else
                    tma_load_2d(tile + c * TK * 128 + ch * BR * 128, &tm_k, full, c * 64, row);
            }
            __syncwarp();
            w = ahead;
            k.next();
        }
        if (!ok) {
            if (lane == 0) {
                *abort_flag = 1;
                atomicOr(p.status, BSP_DEVFLAG_TIMEOUT);
            }
            // drain: this CTA's own copies land before it exits
            const uint64_t t0 = globaltimer_ns();
            // (the round before in the slots from this one on, this round in the others)
            for (int j = 0; j < KST; ++j)
                while (!mbar_try_wait(&bars->k_full[j], j < k.slot ? k.parity : k.parity ^ 1) && globaltimer_ns() - t0 < kDrainWaitNs) {
                }
        }
    } else if (warp == 1) {
        // ================= products
        if (lane == 0) {
            const uint32_t idesc = idesc_f16(TK, NS, BF16, false);
            const uint64_t k_desc0 = sdesc_sw128(smem_u32(k_buf(0)), 16, 1024), q_desc0 = sdesc_sw128(smem_u32(q_buf(0)), 16, 1024);
            Ring k(KST), q(NQ);
            uint64_t q_desc = q_desc0;
            Ring acc(accs);
            uint32_t parities = 0;  // of the accumulators
            int q_slot = -1;        // the present block's
            bool ok = true;
            for (Walk w(p, s_cum); w.more() && ok; w.next(), k.next()) {
                w.open();
                ok = mbar_wait(FP8 ? &bars->k_ready[k.slot] : &bars->k_full[k.slot], k.parity, abort_flag, kWaitNs);
                if (!ok) break;
                const uint64_t k_desc = k_desc0 + static_cast<uint32_t>(k.slot * (K_BYTES >> 4));
                for (int rb = w.rb; rb < w.nrb && ok; ++rb) {
                    if (w.new_q) {
                        if (q_slot >= 0) mma_commit(&bars->q_empty[q_slot]);
                        ok = mbar_wait(&bars->q_full[q.slot], q.parity, abort_flag, kWaitNs) &&
                             mbar_wait(&bars->q_clean[q.slot], q.parity, abort_flag, kWaitNs);
                        if (!ok) break;
                        q_slot = q.slot;
                        q_desc = q_desc0 + static_cast<uint32_t>(q.slot * (q_bytes >> 4));
                        q.next();
                    }
                    // (the blocks of an item take its accumulator one after another)
                    const int a = acc.slot;
                    ok = mbar_wait(&bars->acc_empty[a], ((parities >> a) & 1u) ^ 1u, abort_flag, kWaitNs);
                    if (!ok) break;
                    parities ^= 1u << a;
                    tc_fence_after();
                    // (a k-step of 16 elements is 32 bytes on, a column region TK or NS rows of 128 bytes)
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        mma_f16(tmem + a * acc_cols, k_desc + ((kk >> 2) * (TK * 8) + (kk & 3) * 2),
                                q_desc + static_cast<uint32_t>((kk >> 2) * (NS * 8) + (kk & 3) * 2), idesc, kk > 0 ? 1u : 0u);
                    mma_commit(&bars->acc_full[a]);
                }
                acc.next();
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
        // ================= the Q blocks
        // A row with lse -inf (padding) adds nothing whatever its q holds: exp2 of a finite product less infinity is 0,
        // of a NaN or an infinite one it is a NaN. So such rows' q is cleared where it lies, between its load and the
        // products: 1 % of the kernel (E4M3 pools 2.5 %, the smallest calls 0.6 us), 3 to 6 % where a third of the rows
        // are such. (Leaving their columns out of the sums: 1 to 10 %, and 85 %. A warp of its own for the clearing: up to
        // 5 %.) lse is fetched before the wait for the slot, so that the look costs the block no time.
        const int line = p.G * D * 2 / 128;  // 128-byte lines of a row's heads
        // j / line and c / G as products: exact for the at most 512 lines and 256 rows of a block
        const int line_mul = 65536 / line + 1, g_mul = 65536 / p.G + 1;
        int at[8];  // where lse of the block's rows lane + 32 j stands, of at most 256
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = lane + 32 * j, i = (c * g_mul) >> 16;
            at[j] = i * p.Hq + (c - i * p.G);
        }
        Ring q(NQ);
        bool ok = true;
        for (Walk w(p, s_cum); w.more() && ok; w.next()) {
            w.open();
            for (int rb = w.rb; rb < w.nrb && w.new_q; ++rb, q.next()) {
                const int i0 = rb * p.block_rows;
                const int rows_here = min(p.block_rows, w.seen - i0), n = rows_here * p.G;
                const float* lse = p.lse + static_cast<long long>(w.row0 + i0) * p.Hq + w.g * p.G;
                float l[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    l[j] = 0.f;
                    if (lane + 32 * j < n) ld_early(l[j], lse + at[j]);
                }
                // the block on its way to L2: its shared-memory slot may be free only shortly before it is needed
                const uint8_t* rows = static_cast<const uint8_t*>(p.q) + (static_cast<long long>(w.row0 + i0) * p.Hq + w.g * p.G) * (D * 2);
                for (int j = lane; j < rows_here * line; j += 32) {
                    const int i = (j * line_mul) >> 16;
                    prefetch_l2(rows + static_cast<long long>(i) * p.Hq * (D * 2) + (j - i * line) * 128);
                }
                ok = __all_sync(FULL, mbar_wait(&bars->q_empty[q.slot], q.parity ^ 1, abort_flag, kWaitNs));
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&bars->q_full[q.slot], NC * p.block_rows * p.G * 128);
                    for (int c = 0; c < NC; ++c)
                        tma_load_3d(q_buf(q.slot) + c * NS * 128, &tm_q, &bars->q_full[q.slot], c * 64, w.g * p.G, w.row0 + i0);
                }
                __syncwarp();
                uint32_t none = 0;  // bit j: row lane + 32 j has no log-sum-exp
#pragma unroll
                for (int j = 0; j < 8; ++j) none |= l[j] == -INFINITY ? 1u << j : 0u;
                if (__any_sync(FULL, none != 0)) {
                    ok = __all_sync(FULL, mbar_wait(&bars->q_full[q.slot], q.parity, abort_flag, kWaitNs));
                    if (!ok) {
                        q.next();  // (this slot's copy is under way: it is drained with the round's)
                        break;
                    }
                    for (; none; none &= none - 1) {
                        // (a row is 128 bytes in each column region, whatever the order of their 16-byte chunks)
                        uint8_t* row = q_buf(q.slot) + (lane + 32 * (__ffs(none) - 1)) * 128;
                        for (int c = 0; c < NC; ++c)
#pragma unroll
                            for (int k = 0; k < 8; ++k) reinterpret_cast<uint4*>(row + c * NS * 128)[k] = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive(&bars->q_clean[q.slot]);
            }
        }
        if (!ok) {
            if (lane == 0) {
                *abort_flag = 1;
                atomicOr(p.status, BSP_DEVFLAG_TIMEOUT);
            }
            const uint64_t t0 = globaltimer_ns();
            for (int j = 0; j < NQ; ++j)
                while (!mbar_try_wait(&bars->q_full[j], j < q.slot ? q.parity : q.parity ^ 1) && globaltimer_ns() - t0 < kDrainWaitNs) {
                }
        }
    } else if (warp >= 4 && warp < 4 + kSumWarps) {
        // ================= sums: thread <-> key <-> TMEM lane
        const int quad = warp & 3, set = (warp - 4) >> 2;
        const int key_lane = quad * 32 + lane;
        const float c2 = p.scale_log2;
        const int every = halves ? 2 : 4, half = halves ? set & 1 : 0, pair = set >> 1;
        const int col0 = half * NU;                       // the set's first column of a block
        const int slot = halves ? pair : set;             // its accumulator
        const uint32_t acc = tmem + slot * acc_cols + col0 + (static_cast<uint32_t>(quad * 32) << 16);
        float* nlse = s_nlse + set * 2 * kSetCols;        // of the present block: by turns in either half
        int k_slot = slot % KST;
        uint32_t acc_parity = 0, lse_parity = 0;
        Ring part(2);                                     // places of the second half's sums
        bool ok = true;
        for (Walk w(p, s_cum, slot, every); w.more() && ok; w.next()) {
            w.open();
            const int key = w.kt * TK + key_lane;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
            for (int rb = w.rb; rb < w.nrb; ++rb) {
                const int i0 = rb * p.block_rows;
                const int n = min(p.block_rows, w.seen - i0) * p.G - col0;  // the block's columns for this set
                if (w.new_q) {
                    // -lse of the set's columns in base 2, a column per thread; -inf for rows without one. The other
                    // half of the buffer is still read by warps that are a block behind, but no further: they
                    // have arrived for the present block.
                    nlse = s_nlse + set * 2 * kSetCols + (lse_parity ? 0 : kSetCols);
                    float v = -INFINITY;
                    if (key_lane < min(n, NU)) {
                        const int i = (col0 + key_lane) / p.G;
                        const float l = __ldg(p.lse + static_cast<long long>(w.row0 + i0 + i) * p.Hq + w.g * p.G + (col0 + key_lane - i * p.G));
                        v = l == -INFINITY ? -INFINITY : -l * p.lse_mul;
                    }
                    nlse[key_lane] = v;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars->lse_full[set]);
                    ok = __all_sync(FULL, mbar_wait(&bars->lse_full[set], lse_parity, abort_flag, kWaitNs));
                    if (!ok) break;
                    lse_parity ^= 1;
                }
                ok = __all_sync(FULL, mbar_wait(&bars->acc_full[slot], acc_parity, abort_flag, kWaitNs));
                if (!ok) break;
                acc_parity ^= 1;
                tc_fence_after();
                // the K tile has been read when its last product is complete
                if (quad == 0 && lane == 0 && half == 0 && rb == w.nrb - 1) mbar_arrive(&bars->k_empty[k_slot]);
                const int cols = min(n, NU);
                // columns below cmin are rows that do not see this thread's key
                const int cmin = w.causal ? max(0, key - w.cbase - i0) * p.G - col0 : 0;
                const bool all_see = !w.causal || w.kt * TK + TK - 1 <= w.cbase + i0;
                for (int c0 = 0; c0 < cols; c0 += 32) {
                    uint32_t s[32];
                    tmem_ld32(acc + c0, s);
                    tmem_wait_ld();
                    if (all_see && c0 + 32 <= cols) {
#pragma unroll
                        for (int c = 0; c < 32; c += 4) {
                            const float4 l = *reinterpret_cast<const float4*>(nlse + c0 + c);
                            float e0, e1, e2, e3;
                            fma2(e0, e1, __uint_as_float(s[c]), __uint_as_float(s[c + 1]), c2, l.x, l.y);
                            fma2(e2, e3, __uint_as_float(s[c + 2]), __uint_as_float(s[c + 3]), c2, l.z, l.w);
                            add2_acc(sum[0], sum[1], ex2(e0), ex2(e1));
                            add2_acc(sum[2], sum[3], ex2(e2), ex2(e3));
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            const float e = ex2(fmaf(__uint_as_float(s[c]), c2, nlse[c0 + c]));
                            sum[c & 3] += (c0 + c < cols && c0 + c >= cmin) ? e : 0.f;
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->acc_empty[slot]);
            }
            if (!ok) break;
            k_slot += every;
            while (k_slot >= KST) k_slot -= KST;
            float v = (sum[0] + sum[1]) + (sum[2] + sum[3]);
            if (halves) {
                // The second half's sums, in two places by turns with a barrier each: the second half's set is at
                // most one item ahead, since the accumulator of the item after waits for both sets.
                float* place = s_part + (2 * pair + part.slot) * TK + key_lane;
                uint64_t* full = &bars->part_full[pair][part.slot];
                if (half) {
                    *place = v;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(full);
                } else {
                    ok = __all_sync(FULL, mbar_wait(full, part.parity, abort_flag, kWaitNs));
                    if (!ok) break;
                    v += *place;
                }
                part.next();
            }
            if (!half && key < w.P) {
                float* out = p.weights + (static_cast<long long>(w.b) * p.Hkv + w.g) * p.stride + key;
                *out = p.accumulate ? *out + v : v;
            }
        }
        if (!ok && lane == 0) {
            *abort_flag = 1;
            atomicOr(p.status, BSP_DEVFLAG_TIMEOUT);
        }
    } else if (FP8 && warp >= 4 + kSumWarps) {
        // ================= E4M3 tiles widened to the q dtype in their slots
        if constexpr (FP8) {
            Ring k(KST);
            bool ok = true;
            for (Walk w(p, s_cum); w.more(); w.next(), k.next()) {
                w.open();
                ok = mbar_wait(&bars->k_full[k.slot], k.parity, abort_flag, kWaitNs);
                // the four warps go on, or leave, together
                uint32_t all;
                asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                             "barrier.cta.red.and.pred q, 2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                             : "=r"(all) : "r"(ok ? 1u : 0u) : "memory");
                ok = all != 0;
                if (!ok) break;
                widen_e4m3_tile<D, TK, BF16, 128>(k_buf(k.slot), min(TK, w.P - w.kt * TK), tid - 32 * (4 + kSumWarps), 1);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->k_ready[k.slot]);
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

using Kernel = void (*)(CUtensorMap, CUtensorMap, WeightsParams);
template <int D>
Kernel kernel_of(bool bf16) {
    return bf16 ? key_weights_kernel<D, true, false> : key_weights_kernel<D, false, false>;
}
template <int D>
Kernel kernel_of_fp8(bool bf16) {
    return bf16 ? key_weights_kernel<D, true, true> : key_weights_kernel<D, false, true>;
}
Kernel kernel_of(int head_dim, bool bf16, bool fp8) {
    if (fp8) return head_dim == 64 ? kernel_of_fp8<64>(bf16) : head_dim == 128 ? kernel_of_fp8<128>(bf16) : nullptr;
    return head_dim == 64 ? kernel_of<64>(bf16) : head_dim == 128 ? kernel_of<128>(bf16) : kernel_of<256>(bf16);
}

}  // namespace

cudaError_t prepare_weights(int head_dim, bool bf16, bool fp8) {
    const Kernel kernel = kernel_of(head_dim, bf16, fp8);
    if (!kernel) return cudaErrorInvalidValue;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMaxSmem));
}

cudaError_t launch_weights(int head_dim, bool bf16, bool fp8, const CUtensorMap& tq, const CUtensorMap& tk,
                           const WeightsParams& p, int ctas, size_t smem, cudaStream_t stream) {
    const Kernel kernel = kernel_of(head_dim, bf16, fp8);
    if (!kernel) return cudaErrorInvalidValue;
    kernel<<<ctas, weights_threads(fp8), smem, stream>>>(tq, tk, p);
    return cudaGetLastError();
}

}  // namespace bsp
