// Logits of a beam step: penalties, biases, temperature and grammar masks with the row's log-sum-exp
// (bsp_process_logits), and the best continuations of each request (bsp_beam_select).
//
// Built without fast-math: stored logits and scores are single IEEE operations in a fixed order, so that
// the chosen beams do not depend on how a sum was contracted, and denormal logits keep their value.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/bsp.h"
#include "bsp_internal.h"
#include "bsp_topk.cuh"

namespace bsp {
namespace {

constexpr float kNegInf = -INFINITY;
constexpr float kLog2e = 1.4426950408889634f;

// ---- 16-byte vectors of logits

template <int DT>
struct Logit;
template <>
struct Logit<BSP_LOGITS_BF16> {
    using T = __nv_bfloat16;
    static constexpr int E = 8;
    static constexpr uint32_t kNegInfPair = 0xff80ff80u;
    static __device__ __forceinline__ float get(T v) { return __bfloat162float(v); }
    static __device__ __forceinline__ T put(float v) { return __float2bfloat16_rn(v); }
    static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Logit<BSP_LOGITS_FP16> {
    using T = __half;
    static constexpr int E = 8;
    static constexpr uint32_t kNegInfPair = 0xfc00fc00u;
    static __device__ __forceinline__ float get(T v) { return __half2float(v); }
    static __device__ __forceinline__ T put(float v) { return __float2half_rn(v); }
    static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[2 * i] = a.x;
            f[2 * i + 1] = a.y;
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Logit<BSP_LOGITS_FP32> {
    using T = float;
    static constexpr int E = 4;
    static constexpr uint32_t kNegInfPair = 0xff800000u;
    static __device__ __forceinline__ float get(T v) { return v; }
    static __device__ __forceinline__ T put(float v) { return v; }
    static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[4]) {
        f[0] = __uint_as_float(v.x);
        f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z);
        f[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};

// elements before the first 16-byte boundary at or after p (p is aligned to its element)
template <int E>
__device__ __forceinline__ int lead_elems(const void* p) {
    constexpr int es = 16 / E;
    return static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / es);
}

// 32 mask bits that start at token s (s may be negative: no tokens there) of a packed row of `words` words
__device__ __forceinline__ uint32_t mask_bits(const uint32_t* row, int words, int s) {
    const int g = s >> 5, sh = s & 31;
    const uint32_t lo = (g >= 0 && g < words) ? __ldg(row + g) : 0u;
    if (sh == 0) return lo;
    const uint32_t hi = (g + 1 >= 0 && g + 1 < words) ? __ldg(row + g + 1) : 0u;
    return __funnelshift_r(lo, hi, sh);
}

// the row's grammar state, or null: none (index -1), or an index out of range (flagged)
__device__ __forceinline__ const uint32_t* mask_row(const TokenMask& m, int r, int32_t* status, bool flag) {
    if (!m.bits) return nullptr;
    const int i = __ldg(m.index + r);
    if (i < 0) return nullptr;
    if (i >= m.rows) {
        if (flag) atomicOr(status, BSP_DEVFLAG_PAGE_INDEX);
        return nullptr;
    }
    return m.bits + static_cast<long long>(i) * m.stride;
}

// ---------------------------------------------------------------- log-sum-exp of a running row

// Running maximum and sum of exp(x - maximum). A maximum of +-infinity subtracts nothing, so that a row of
// -inf sums to 0 (log-sum-exp -inf), +inf gives +inf, and a NaN anywhere a NaN.
struct Running {
    float m, s;
};
__device__ __forceinline__ float shift_of(float m) { return isinf(m) ? 0.f : m; }
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ Running join(Running a, Running b) {
    Running r;
    r.m = fmaxf(a.m, b.m);
    const float sh = shift_of(r.m);
    // a part without any finite or infinite value has sum 0 (or NaN, which stays)
    const float fa = a.m == r.m ? 1.f : exp2_approx((shift_of(a.m) - sh) * kLog2e);
    const float fb = b.m == r.m ? 1.f : exp2_approx((shift_of(b.m) - sh) * kLog2e);
    r.s = (a.m == kNegInf && !isnan(a.s) ? 0.f : a.s * fa) + (b.m == kNegInf && !isnan(b.s) ? 0.f : b.s * fb);
    return r;
}
template <int N>
__device__ __forceinline__ void add_values(Running& a, const float (&f)[N]) {
    float top = f[0];
#pragma unroll
    for (int i = 1; i < N; ++i) top = fmaxf(top, f[i]);
    if (top > a.m) {
        a.s = a.m == kNegInf && !isnan(a.s) ? 0.f : a.s * exp2_approx((shift_of(a.m) - shift_of(top)) * kLog2e);
        a.m = top;
    }
    // (the difference first: x * log2(e) of a row of lowest values would overflow)
    const float c = shift_of(a.m);
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        s0 += exp2_approx((f[i] - c) * kLog2e);
        if (i + 1 < N) s1 += exp2_approx((f[i + 1] - c) * kLog2e);
    }
    a.s += s0 + s1;
}

// ---------------------------------------------------------------- process

constexpr int kProcThreads = 512;

struct HashSlot {
    uint32_t token;  // token + 1; 0: empty
    uint32_t count;  // occurrences in the row's generated tokens
    uint32_t bias;   // index of the first bias entry, or ~0
};
static_assert(sizeof(HashSlot) == kProcessSlotBytes, "table slot");

__device__ __forceinline__ uint32_t hash_of(uint32_t token, uint32_t mask) { return (token * 0x9E3779B1u >> 15) & mask; }

// The table's slot of a token, claimed if it is new. The table has at least twice as many slots as tokens.
__device__ __forceinline__ HashSlot* hash_claim(HashSlot* table, uint32_t mask, uint32_t token) {
    uint32_t h = hash_of(token, mask);
    for (uint32_t probe = 0; probe <= mask; ++probe, h = (h + 1) & mask) {
        const uint32_t old = atomicCAS(&table[h].token, 0u, token + 1);
        if (old == 0u || old == token + 1) return table + h;
    }
    return nullptr;
}
__device__ __forceinline__ const HashSlot* hash_find(const HashSlot* table, uint32_t mask, uint32_t token) {
    uint32_t h = hash_of(token, mask);
    for (uint32_t probe = 0; probe <= mask; ++probe, h = (h + 1) & mask) {
        if (table[h].token == token + 1) return table + h;
        if (table[h].token == 0u) return nullptr;
    }
    return nullptr;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void store_at_rank(const void* p, uint32_t rank, float v) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}

// One cluster per row, each CTA a slice of the vocabulary. Tokens that the lists name are marked in two
// bitmaps of the slice (penalised; in the table of counts and biases), so that a 16-byte vector without a
// marked token costs two shared-memory words; a vector whose tokens the grammar rejects is not read at all.
template <int DT>
__global__ void __launch_bounds__(kProcThreads) process_logits_kernel(const ProcessParams p) {
    using L = Logit<DT>;
    using T = typename L::T;
    constexpr int E = L::E;
    constexpr int U = 4;  // vectors in flight per thread
    extern __shared__ uint32_t smem[];
    __shared__ Running s_part[kProcThreads / 32];
    __shared__ float s_m[16], s_s[16];

    const int tid = threadIdx.x;
    const int rank = static_cast<int>(cluster_rank()), ranks = static_cast<int>(cluster_size());
    const int r = blockIdx.x / ranks;
    const int b = r / p.W;
    const T* x = static_cast<const T*>(p.x) + static_cast<long long>(r) * p.x_stride;
    T* out = static_cast<T*>(p.out) + static_cast<long long>(r) * p.out_stride;
    const bool in_place = p.x == p.out;
    const bool joined = p.lse && ranks > 1;
    if (joined) cluster_arrive();  // waited for before the first access to another CTA's shared memory

    // the slice: vectors [v0, v1) from element `head` on, plus the row's ragged ends for the first / last CTA
    const int head = min(lead_elems<E>(x), p.vocab);
    const int nv = (p.vocab - head) / E;
    const int v0 = static_cast<int>(static_cast<long long>(nv) * rank / ranks);
    const int v1 = static_cast<int>(static_cast<long long>(nv) * (rank + 1) / ranks);
    const int lo = rank == 0 ? 0 : head + v0 * E;
    const int hi = rank == ranks - 1 ? p.vocab : head + v1 * E;
    // bit i of the bitmaps is token base + i; vectors start at multiples of E bits
    const int base = rank == 0 && head > 0 ? head - E : lo;
    const bool vec_out = ((reinterpret_cast<uintptr_t>(out + head)) & 15) == 0;

    uint32_t* bm_pen = smem;
    uint32_t* bm_hot = bm_pen + p.bitmap_words;
    uint32_t* bm_mask = bm_hot + p.bitmap_words;
    HashSlot* table = reinterpret_cast<HashSlot*>(bm_mask + p.bitmap_words);
    const uint32_t hmask = p.hash_slots - 1;
    const int words = (hi - base + 31) >> 5;
    const bool counts = p.frequency || p.presence;

    const uint32_t* mrow = mask_row(p.mask, r, p.status, rank == 0 && tid == 0);
    for (int i = tid; i < words; i += kProcThreads) {
        bm_pen[i] = 0;
        bm_hot[i] = 0;
        if (mrow) bm_mask[i] = mask_bits(mrow, (p.vocab + 31) >> 5, base + 32 * i);
    }
    for (int i = tid; i < p.hash_slots; i += kProcThreads) table[i] = HashSlot{0u, 0u, ~0u};
    __syncthreads();
    auto mark = [&](uint32_t* bm, int t) { atomicOr(bm + ((t - base) >> 5), 1u << ((t - base) & 31)); };
    if (p.repetition && p.prompt_tokens) {
        const int n = max(0, min(__ldg(p.prompt_len + b), p.prompt_cols));
        const int32_t* list = p.prompt_tokens + static_cast<long long>(b) * p.prompt_stride;
        for (int i = tid; i < n; i += kProcThreads) {
            const int t = __ldg(list + i);
            if (t >= lo && t < hi) mark(bm_pen, t);
        }
    }
    if (p.tokens && (p.repetition || counts)) {
        const int n = max(0, min(__ldg(p.token_len + r), p.token_cols));
        const int32_t* list = p.tokens + static_cast<long long>(r) * p.token_stride;
        for (int i = tid; i < n; i += kProcThreads) {
            const int t = __ldg(list + i);
            if (t >= lo && t < hi) {
                if (p.repetition) mark(bm_pen, t);
                if (counts) {
                    mark(bm_hot, t);
                    if (HashSlot* s = hash_claim(table, hmask, t)) atomicAdd(&s->count, 1u);
                }
            }
        }
    }
    if (p.bias_tokens) {
        const int n = p.bias_len ? max(0, min(__ldg(p.bias_len + b), p.bias_cols)) : p.bias_cols;
        const int32_t* list = p.bias_tokens + static_cast<long long>(b) * p.bias_stride;
        for (int i = tid; i < n; i += kProcThreads) {
            const int t = __ldg(list + i);
            if (t >= lo && t < hi) {
                mark(bm_hot, t);
                // an id given twice: its first value counts
                if (HashSlot* s = hash_claim(table, hmask, t)) atomicMin(&s->bias, static_cast<uint32_t>(i));
            }
        }
    }
    const float rep = p.repetition ? __ldg(p.repetition + b) : 1.f;
    const float freq = p.frequency ? __ldg(p.frequency + b) : 0.f;
    const float pres = p.presence ? __ldg(p.presence + b) : 0.f;
    // the product with the rounded reciprocal: 1.5 half-steps of fp32 from the quotient, one multiplication
    // per logit in place of a division
    const float inv_t = p.temperature ? __frcp_rn(__ldg(p.temperature + b)) : 1.f;
    const float* bias = p.bias_values ? p.bias_values + static_cast<long long>(b) * p.bias_stride : nullptr;
    __syncthreads();

    auto change = [&](float v, int t) -> float {  // a marked token, before the temperature
        const int i = t - base;
        if ((bm_pen[i >> 5] >> (i & 31)) & 1u) v = v > 0.f ? __fdiv_rn(v, rep) : __fmul_rn(v, rep);
        if ((bm_hot[i >> 5] >> (i & 31)) & 1u) {
            const HashSlot* s = hash_find(table, hmask, static_cast<uint32_t>(t));
            if (s) {
                if (s->count) {
                    v = __fsub_rn(v, __fmul_rn(freq, static_cast<float>(s->count)));
                    v = __fsub_rn(v, pres);
                }
                if (s->bias != ~0u) v = __fadd_rn(v, __ldg(bias + s->bias));
            }
        }
        return v;
    };

    Running run{kNegInf, 0.f};
    const bool temp = p.temperature != nullptr;
    // the ragged ends, one element per thread
    {
        const int n_head = rank == 0 ? head : 0;
        const int tail0 = head + nv * E;
        const int n_tail = rank == ranks - 1 ? p.vocab - tail0 : 0;
        if (tid < n_head + n_tail) {
            const int t = tid < n_head ? tid : tail0 + tid - n_head;
            const int i = t - base;
            float f[1] = {kNegInf};
            if (!mrow || ((bm_mask[i >> 5] >> (i & 31)) & 1u)) {
                f[0] = change(L::get(x[t]), t);
                if (temp) f[0] = __fmul_rn(f[0], inv_t);
            }
            const T y = L::put(f[0]);
            out[t] = y;
            f[0] = L::get(y);
            add_values(run, f);
        }
    }
    const uint4* xv = reinterpret_cast<const uint4*>(x + head);
    constexpr uint32_t ALL = (1u << E) - 1;
    for (int vb = v0 + tid; vb < v1; vb += U * kProcThreads) {
        uint4 val[U];
        uint32_t keep[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int v = vb + u * kProcThreads;
            const int i = head + v * E - base;
            keep[u] = v >= v1 ? 0u : mrow ? (bm_mask[i >> 5] >> (i & 31)) & ALL : ALL;
            if (keep[u]) val[u] = __ldcs(xv + v);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int v = vb + u * kProcThreads;
            if (v >= v1) break;
            const int t0 = head + v * E, i = t0 - base;
            uint4 res = make_uint4(L::kNegInfPair, L::kNegInfPair, L::kNegInfPair, L::kNegInfPair);
            bool changed = true;
            if (keep[u]) {
                float f[E];
                L::unpack(val[u], f);
                const uint32_t marked = ((bm_pen[i >> 5] | bm_hot[i >> 5]) >> (i & 31)) & ALL & keep[u];
                changed = temp || marked || keep[u] != ALL;
                if (changed) {
                    if (marked) {
#pragma unroll
                        for (int e = 0; e < E; ++e)
                            if ((marked >> e) & 1u) f[e] = change(f[e], t0 + e);
                    }
                    if (temp) {
#pragma unroll
                        for (int e = 0; e < E; ++e) f[e] = __fmul_rn(f[e], inv_t);
                    }
                    if (keep[u] != ALL) {
#pragma unroll
                        for (int e = 0; e < E; ++e)
                            if (!((keep[u] >> e) & 1u)) f[e] = kNegInf;
                    }
                    res = L::pack(f);
                    L::unpack(res, f);  // the log-sum-exp is that of the stored values
                } else {
                    res = val[u];
                }
                add_values(run, f);
            }
            if (!in_place || changed) {
                if (vec_out) {
                    __stcs(reinterpret_cast<uint4*>(out + t0), res);
                } else {
                    const T* e = reinterpret_cast<const T*>(&res);
#pragma unroll
                    for (int k = 0; k < E; ++k) out[t0 + k] = e[k];
                }
            }
        }
    }

    // ---- the row's log-sum-exp: warp, CTA, cluster
    if (!p.lse) return;  // uniform
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        Running o;
        o.m = __shfl_xor_sync(~0u, run.m, d);
        o.s = __shfl_xor_sync(~0u, run.s, d);
        run = join(run, o);
    }
    if ((tid & 31) == 0) s_part[tid >> 5] = run;
    __syncthreads();
    if (joined) cluster_wait();
    if (tid == 0) {
        for (int i = 1; i < kProcThreads / 32; ++i) run = join(run, s_part[i]);
        if (joined) {
            store_at_rank(&s_m[rank], 0, run.m);
            store_at_rank(&s_s[rank], 0, run.s);
        }
    }
    if (joined) {
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        if (rank == 0 && tid == 0) {
            run = Running{s_m[0], s_s[0]};
            for (int i = 1; i < ranks; ++i) run = join(run, Running{s_m[i], s_s[i]});
        }
    }
    if (rank == 0 && tid == 0) p.lse[r] = logf(run.s) + shift_of(run.m);
}

template <int DT>
cudaError_t launch_process_t(const ProcessParams& p, int cluster, size_t smem, cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(process_logits_kernel<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(p.rows) * cluster);
    cfg.blockDim = dim3(kProcThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, process_logits_kernel<DT>, p);
}

// ---------------------------------------------------------------- select

constexpr int kSelThreads = 256;
constexpr int kSelU = 2;  // vectors per thread and unit

// Candidates as 64-bit keys: the score's order in the high half, the flat index (beam * vocab + token)
// complemented in the low half, so that the larger key is the better candidate and equal scores go by the
// lower index. Keys are distinct, hence the chosen set does not depend on the order of arrival.
__device__ __forceinline__ uint64_t candidate_key(float score, uint32_t flat) {
    return (static_cast<uint64_t>(float_order(score)) << 32) | static_cast<uint32_t>(~flat);
}

template <int DT>
__global__ void __launch_bounds__(kSelThreads) beam_scan_kernel(const SelectParams p) {
    using L = Logit<DT>;
    using T = typename L::T;
    constexpr int E = L::E, U = kSelU;
    // [limit + kSelThreads * U * E + 16]: the candidates held, and the most one unit can add (a row's ragged
    // ends: below 16)
    extern __shared__ uint64_t s_buf[];
    __shared__ TopkScratch<kSelThreads> s_top;
    __shared__ int s_count;

    const int tid = threadIdx.x, lane = tid & 31;
    const int b = blockIdx.y, S = gridDim.x;
    const int limit = p.limit;             // candidates held when a unit begins: at most this many (>= K)
    if (tid == 0) s_count = 0;
    __syncthreads();
    uint64_t floor_key = 0;                // only larger keys are candidates (a lower bound of the best K)
    float floor_score = kNegInf;
    bool have = false;                     // floor_key is set
    const int nseg = p.segments;           // units of a row

    for (int u = blockIdx.x; u < p.W * nseg; u += S) {
        const int w = u / nseg, seg = u - w * nseg;
        const int r = b * p.W + w;
        const float cum = __ldg(p.cum + static_cast<long long>(b) * p.cum_stride + w);
        const float lse = __ldg(p.lse + r);
        if (!(cum > kNegInf)) continue;    // uniform: a dead beam (or a NaN score) has no candidates
        const T* x = static_cast<const T*>(p.x) + static_cast<long long>(r) * p.x_stride;
        const int head = min(lead_elems<E>(x), p.vocab);
        const int nv = (p.vocab - head) / E;
        const int v0 = static_cast<int>(static_cast<long long>(nv) * seg / nseg);
        const int v1 = static_cast<int>(static_cast<long long>(nv) * (seg + 1) / nseg);
        const uint32_t* mrow = mask_row(p.mask, r, p.status, tid == 0 && seg == 0);
        const int mwords = (p.vocab + 31) >> 5;
        const uint4* xv = reinterpret_cast<const uint4*>(x + head);
        float f[U][E], g = kNegInf;        // scores (-inf: not a candidate); g: a ragged element
        int tg = -1;
        {
            uint4 val[U];
            uint32_t keep[U];
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int v = v0 + tid + k * kSelThreads;
                keep[k] = v >= v1 ? 0u : mrow ? mask_bits(mrow, mwords, head + v * E) & ((1u << E) - 1) : (1u << E) - 1;
                if (keep[k]) val[k] = __ldcs(xv + v);
            }
            const int n_head = seg == 0 ? head : 0;
            const int tail0 = head + nv * E;
            const int n_tail = seg == nseg - 1 ? p.vocab - tail0 : 0;
            if (tid < n_head + n_tail) {
                tg = tid < n_head ? tid : tail0 + tid - n_head;
                if (!mrow || (mask_bits(mrow, mwords, tg) & 1u)) g = __fadd_rn(__fsub_rn(L::get(x[tg]), lse), cum);
            }
#pragma unroll
            for (int k = 0; k < U; ++k) {
#pragma unroll
                for (int e = 0; e < E; ++e) f[k][e] = kNegInf;
                if (keep[k]) {
                    L::unpack(val[k], f[k]);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const float s = __fadd_rn(__fsub_rn(f[k][e], lse), cum);
                        f[k][e] = ((keep[k] >> e) & 1u) ? s : kNegInf;
                    }
                }
            }
        }
        // candidates: above the floor (before there is one: anything above -inf; NaN compares false)
        auto passes = [&](float s, int t) -> bool {
            if (!(s >= floor_score) || !(s > kNegInf)) return false;
            return !have || candidate_key(s, static_cast<uint32_t>(w) * p.vocab + t) > floor_key;
        };
        int mine = 0;
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
            for (int e = 0; e < E; ++e) mine += passes(f[k][e], head + (v0 + tid + k * kSelThreads) * E + e);
        mine += tg >= 0 && passes(g, tg);
        bool full = false;
        if (__any_sync(~0u, mine)) {
            int at = mine;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(~0u, at, d);
                if (lane >= d) at += o;
            }
            const int total = __shfl_sync(~0u, at, 31);
            int first = 0;
            if (lane == 0) first = atomicAdd(&s_count, total);
            first = __shfl_sync(~0u, first, 0);
            full = first + total > limit;
            at += first - mine;
            if (mine) {
#pragma unroll
                for (int k = 0; k < U; ++k)
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const int t = head + (v0 + tid + k * kSelThreads) * E + e;
                        if (passes(f[k][e], t)) s_buf[at++] = candidate_key(f[k][e], static_cast<uint32_t>(w) * p.vocab + t);
                    }
                if (tg >= 0 && passes(g, tg)) s_buf[at++] = candidate_key(g, static_cast<uint32_t>(w) * p.vocab + tg);
            }
        }
        if (__syncthreads_or(full)) {
            const int n = s_count;
            floor_key = topk_compact<kSelThreads>(s_buf, n, p.K, s_top);
            floor_score = order_float(static_cast<uint32_t>(floor_key >> 32));
            have = true;
            if (tid == 0) s_count = min(n, p.K);
            __syncthreads();
        }
    }
    __syncthreads();
    int n = s_count;
    if (n > p.K) {
        topk_compact<kSelThreads>(s_buf, n, p.K, s_top);
        n = p.K;
    }
    const long long list = static_cast<long long>(b) * S + blockIdx.x;
    if (tid == 0) p.part_count[list] = n;
    for (int i = tid; i < n; i += kSelThreads) p.part_keys[list * p.K + i] = s_buf[i];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

constexpr int kMergeThreads = 512;

// One CTA per request: the splits' lists, cut to the best K and put in order.
__global__ void __launch_bounds__(kMergeThreads) beam_merge_kernel(const SelectParams p) {
    extern __shared__ uint64_t s_buf[];  // [splits * K]
    __shared__ TopkScratch<kMergeThreads> s_top;
    __shared__ int s_count;
    const int tid = threadIdx.x, lane = tid & 31;
    const int b = blockIdx.x;
    if (tid == 0) s_count = 0;
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long list0 = static_cast<long long>(b) * p.splits;
    for (int i0 = 0; i0 < p.splits * p.K; i0 += kMergeThreads) {
        const int i = i0 + tid;
        const int s = i / p.K, j = i - s * p.K;
        const bool in = s < p.splits && j < __ldcg(p.part_count + list0 + s);
        uint64_t key = 0;
        if (in) key = __ldcg(reinterpret_cast<const unsigned long long*>(p.part_keys) + (list0 + s) * p.K + j);
        const uint32_t who = __ballot_sync(~0u, in);
        int first = 0;
        if (lane == 0 && who) first = atomicAdd(&s_count, __popc(who));
        first = __shfl_sync(~0u, first, 0);
        if (in) s_buf[first + __popc(who & ((1u << lane) - 1))] = key;
    }
    __syncthreads();
    int n = s_count;
    if (n > p.K) {
        topk_compact<kMergeThreads>(s_buf, n, p.K, s_top);
        n = p.K;
    }
    // rank = number of larger keys (distinct keys, K <= 512): the output place
    for (int i = tid; i < p.K; i += kMergeThreads) {
        const long long o = static_cast<long long>(b) * p.K;
        if (i < n) {
            const uint64_t key = s_buf[i];
            int place = 0;
            for (int j = 0; j < n; ++j) place += s_buf[j] > key;
            const uint32_t flat = ~static_cast<uint32_t>(key);
            p.scores[o + place] = order_float(static_cast<uint32_t>(key >> 32));
            p.parents[o + place] = static_cast<int32_t>(flat / static_cast<uint32_t>(p.vocab));
            p.tokens[o + place] = static_cast<int32_t>(flat % static_cast<uint32_t>(p.vocab));
        } else {
            p.scores[o + i] = kNegInf;
            p.parents[o + i] = -1;
            p.tokens[o + i] = -1;
        }
    }
}

template <int DT>
cudaError_t launch_scan(const SelectParams& p, cudaStream_t stream) {
    constexpr int E = Logit<DT>::E;
    const size_t smem = static_cast<size_t>(kSelThreads * kSelU * E + 16 + p.limit) * 8;
    cudaError_t e = cudaFuncSetAttribute(beam_scan_kernel<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    beam_scan_kernel<DT><<<dim3(p.splits, p.batch), kSelThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_process(int dtype, const ProcessParams& p, int cluster, size_t smem, cudaStream_t stream) {
    switch (dtype) {
        case BSP_LOGITS_BF16: return launch_process_t<BSP_LOGITS_BF16>(p, cluster, smem, stream);
        case BSP_LOGITS_FP16: return launch_process_t<BSP_LOGITS_FP16>(p, cluster, smem, stream);
        default: return launch_process_t<BSP_LOGITS_FP32>(p, cluster, smem, stream);
    }
}

int select_unit_elems(int dtype) { return kSelThreads * kSelU * (dtype == BSP_LOGITS_FP32 ? 4 : 8); }

cudaError_t launch_select(int dtype, const SelectParams& p, cudaStream_t stream) {
    cudaError_t e = dtype == BSP_LOGITS_BF16   ? launch_scan<BSP_LOGITS_BF16>(p, stream)
                    : dtype == BSP_LOGITS_FP16 ? launch_scan<BSP_LOGITS_FP16>(p, stream)
                                               : launch_scan<BSP_LOGITS_FP32>(p, stream);
    if (e != cudaSuccess) return e;
    const size_t smem = static_cast<size_t>(p.splits) * p.K * 8;
    e = cudaFuncSetAttribute(beam_merge_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(p.batch);
    cfg.blockDim = dim3(kMergeThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, beam_merge_kernel, p);
}

}  // namespace bsp
