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
#include "bsp_step.h"
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
    // the larger values of two words, and the largest value of a word (NaN passed over, unless there is
    // nothing else)
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
        return *reinterpret_cast<const uint32_t*>(&m);
    }
    static __device__ __forceinline__ float top(uint32_t a) {
        return fmaxf(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
    }
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
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        const __half2 m = __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
        return *reinterpret_cast<const uint32_t*>(&m);
    }
    static __device__ __forceinline__ float top(uint32_t a) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&a));
        return fmaxf(f.x, f.y);
    }
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
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }
    static __device__ __forceinline__ float top(uint32_t a) { return __uint_as_float(a); }
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
// (d0, d1) = (a0 * b + c, a1 * b + c); (s0, s1) += (a0, a1): two fp32 values an instruction
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b, float c) {
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %4};\n\tmov.b64 rc, {%5, %5};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b), "f"(c));
}
__device__ __forceinline__ void mul2(float& d0, float& d1, float b) {
    asm("{\n\t.reg .b64 ra, rb;\n\tmov.b64 ra, {%0, %1};\n\tmov.b64 rb, {%2, %2};\n\t"
        "mul.rn.f32x2 ra, ra, rb;\n\tmov.b64 {%0, %1}, ra;\n\t}"
        : "+f"(d0), "+f"(d1) : "f"(b));
}
__device__ __forceinline__ void add2(float& s0, float& s1, float a0, float a1) {
    asm("{\n\t.reg .b64 rs, ra;\n\tmov.b64 rs, {%0, %1};\n\tmov.b64 ra, {%2, %3};\n\t"
        "add.rn.f32x2 rs, rs, ra;\n\tmov.b64 {%0, %1}, rs;\n\t}"
        : "+f"(s0), "+f"(s1) : "f"(a0), "f"(a1));
}

// One thread's sum of exp(x - m), in two halves. m is a value of the row, at most 16 below the largest so far: it
// is raised only when one stands further above it, which after the first vector hardly happens, and
// exp(16) times a vocabulary is well inside fp32. Each term is good to about 2^-22 (the hardware's exp2; one instruction in
// place of some ten), and its argument to 2^-24 of |m| (-m log2(e) as one fp32 number, one packed FMA in place of a
// difference and a product), which moves the log-sum-exp, of m's size, by no more than the rounding of its own last sum.
struct RowSum {
    float m = kNegInf, limit = kNegInf, s0 = 0.f, s1 = 0.f;
    float c = 0.f;       // -shift * log2(e), where that is well inside fp32
    bool far = false;    // it is not: a row of lowest (or highest) values, whose x * log2(e) would overflow

    __device__ __noinline__ static RowSum raised(RowSum o, float top) {
        const float r = o.m == kNegInf ? 1.f : exp2_approx((shift_of(o.m) - shift_of(top)) * kLog2e);
        o.s0 = o.s0 == 0.f ? 0.f : o.s0 * r;  // (a sum of 0 stays 0, a NaN stays NaN)
        o.s1 = o.s1 == 0.f ? 0.f : o.s1 * r;
        o.m = top;
        o.limit = top + 16.f;
        o.far = fabsf(shift_of(top)) > 1e30f;
        o.c = -shift_of(top) * kLog2e;
        return o;
    }
    // values of which `top` is the largest
    template <int N>
    __device__ __forceinline__ void add(const float (&f)[N], float top) {
        if (top > limit) *this = raised(*this, top);
        if (far || N == 1) {
            const float sh = shift_of(m);
#pragma unroll
            for (int i = 0; i < N; ++i) s0 += exp2_approx((f[i] - sh) * kLog2e);
        } else {
#pragma unroll
            for (int i = 0; i + 1 < N; i += 2) {
                float d0, d1;
                fma2(d0, d1, f[i], f[i + 1], kLog2e, c);
                add2(s0, s1, exp2_approx(d0), exp2_approx(d1));
            }
        }
    }
};

// ---------------------------------------------------------------- process

constexpr int kProcThreads = 256;
constexpr int kProcListed = 96;  // marked vectors a warp puts aside

struct HashSlot {
    uint32_t token;  // token + 1; 0: empty
    uint32_t count;  // occurrences in the row's generated tokens
    uint32_t bias;   // index of the first bias entry, or ~0
};
static_assert(sizeof(HashSlot) == kProcessSlotBytes, "table slot");

__device__ __forceinline__ uint32_t hash_of(uint32_t token, uint32_t mask) { return (token * 0x9E3779B1u >> 15) & mask; }

// The table's slot of a token, claimed if it is new. The table has at least twice as many slots as tokens, or beside the
// largest vocabularies as many.
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
// marked token costs two shared-memory words; a vector whose tokens the grammar rejects is not read at all, and
// where no 32 tokens have more than 8 allowed ones only those are read, one by one.
// The lists, their lengths and the mask are fetched together, and with no mask the first logits before them:
// a row is short beside their latencies, which the four CTAs of an SM hide from one another.
//
// Bound by the logits' traffic, and then by the exponentials' instructions. Measured: 64 x 30 rows of 128000
// bf16 (0.98 GB), lists and temperature, 235 us, 4.2 TB/s, 0.61 of what a copy reaches; without lists and
// temperature 168 us, 0.86. (Five CTAs per SM at fewer registers 257 us, CTAs of 128 threads 271. One list of marked
// vectors for the CTA, filled by an atomic counter, 229 us, but then the order of the sums differs from run to run.)
// Sparse masks: 128 x 96 rows of 32000 fp16 with 1 / 3 / 6 / 12 % allowed take 220 / 271 / 307 / 393 us by their
// bits and 347 / 341 / 337 / 331 by vectors; 64 x 30 rows of 128000 bf16 166 / 205 / 213 / 235 and
// 197 / 204 / 205 / 204. Eight of 32 are reached somewhere in a row at about 6 %.
template <int DT>
__global__ void __launch_bounds__(kProcThreads, 4) process_logits_kernel(const ProcessParams p) {
    using L = Logit<DT>;
    using T = typename L::T;
    constexpr int E = L::E;
    constexpr int U = 4;  // vectors in flight per thread
    constexpr uint32_t ALL = (1u << E) - 1;
    extern __shared__ uint32_t smem[];
    __shared__ Running s_part[kProcThreads / 32];
    __shared__ float s_m[16], s_s[16];
    __shared__ uint4 s_vec[kProcThreads / 32 * kProcListed];  // marked vectors put aside, and their numbers
    __shared__ int s_list[kProcThreads / 32 * kProcListed];
    __shared__ int s_listed[kProcThreads / 32];

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
    const uint4* xv = reinterpret_cast<const uint4*>(x + head);

    const bool counts = p.frequency || p.presence;
    const bool pens = p.repetition && (p.prompt_tokens || p.tokens), hots = p.hash_slots > 0;
    uint32_t* bm_pen = smem;
    uint32_t* bm_hot = smem + p.hot_at;
    uint32_t* bm_mask = smem + p.mask_at;
    HashSlot* table = reinterpret_cast<HashSlot*>(smem + p.table_at);
    const uint32_t hmask = p.hash_slots - 1;
    const int words = (hi - base + 31) >> 5;

    uint4 val[U];
    if (!p.mask.bits) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (v0 + tid + u * kProcThreads < v1) val[u] = __ldcs(xv + v0 + tid + u * kProcThreads);
    }
    // the lists' first entries, whatever their lengths
    const int32_t* prompt = p.prompt_tokens + static_cast<long long>(b) * p.prompt_stride;
    const int32_t* made = p.tokens + static_cast<long long>(r) * p.token_stride;
    const int32_t* biased = p.bias_tokens + static_cast<long long>(b) * p.bias_stride;
    const int first_p = p.prompt_tokens && tid < p.prompt_cols ? __ldg(prompt + tid) : -1;
    const int first_t = p.tokens && tid < p.token_cols ? __ldg(made + tid) : -1;
    const int first_b = p.bias_tokens && tid < p.bias_cols ? __ldg(biased + tid) : -1;
    const int n_p = p.prompt_tokens ? min(__ldg(p.prompt_len + b), p.prompt_cols) : 0;
    const int n_t = p.tokens ? min(__ldg(p.token_len + r), p.token_cols) : 0;
    const int n_b = !p.bias_tokens ? 0 : p.bias_len ? min(__ldg(p.bias_len + b), p.bias_cols) : p.bias_cols;
    const float rep = p.repetition ? __ldg(p.repetition + b) : 1.f;
    const float freq = p.frequency ? __ldg(p.frequency + b) : 0.f;
    const float pres = p.presence ? __ldg(p.presence + b) : 0.f;
    const float temperature = p.temperature ? __ldg(p.temperature + b) : 1.f;
    const uint32_t* mrow = mask_row(p.mask, r, p.status, rank == 0 && tid == 0);
    if (pens)
        for (int i = tid; i < words; i += kProcThreads) bm_pen[i] = 0;
    if (hots) {
        for (int i = tid; i < words; i += kProcThreads) bm_hot[i] = 0;
        for (int i = tid; i < p.hash_slots; i += kProcThreads) table[i] = HashSlot{0u, 0u, ~0u};
    }
    bool dense = !mrow;  // or: some 32 tokens of the slice have more than 8 allowed ones
    if (mrow)
        for (int i = tid; i < words; i += kProcThreads) {
            const uint32_t m = mask_bits(mrow, (p.vocab + 31) >> 5, base + 32 * i);
            bm_mask[i] = m;
            dense |= __popc(m) > 8;
        }
    if (pens || hots || mrow) dense = __syncthreads_or(dense);
    if (pens || hots) {
        auto mark = [&](uint32_t* bm, int t) { atomicOr(bm + ((t - base) >> 5), 1u << ((t - base) & 31)); };
        if (pens)
            for (int i = tid, t = first_p; i < n_p; i += kProcThreads) {
                if (i != tid) t = __ldg(prompt + i);
                if (t >= lo && t < hi) mark(bm_pen, t);
            }
        for (int i = tid, t = first_t; i < n_t; i += kProcThreads) {
            if (i != tid) t = __ldg(made + i);
            if (t < lo || t >= hi) continue;
            if (pens) mark(bm_pen, t);
            if (counts) {
                mark(bm_hot, t);
                if (HashSlot* s = hash_claim(table, hmask, t)) atomicAdd(&s->count, 1u);
            }
        }
        for (int i = tid, t = first_b; i < n_b; i += kProcThreads) {
            if (i != tid) t = __ldg(biased + i);
            if (t < lo || t >= hi) continue;
            mark(bm_hot, t);
            // an id given twice: its first value counts
            if (HashSlot* s = hash_claim(table, hmask, t)) atomicMin(&s->bias, static_cast<uint32_t>(i));
        }
        __syncthreads();
    }
    // the product with the rounded reciprocal: 1.5 half-steps of fp32 from the quotient, one multiplication
    // per logit in place of a division
    const float inv_t = __frcp_rn(temperature);
    const float* bias = p.bias_values + static_cast<long long>(b) * p.bias_stride;

    auto marked_bits = [&](int i) -> uint32_t {
        return (pens ? bm_pen[i >> 5] >> (i & 31) : 0u) | (hots ? bm_hot[i >> 5] >> (i & 31) : 0u);
    };
    auto change = [&](float v, int t) -> float {  // a marked token, before the temperature
        const int i = t - base;
        if (pens && ((bm_pen[i >> 5] >> (i & 31)) & 1u)) v = v > 0.f ? __fdiv_rn(v, rep) : __fmul_rn(v, rep);
        if (hots && ((bm_hot[i >> 5] >> (i & 31)) & 1u)) {
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

    RowSum sum;
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
                f[0] = L::get(x[t]);
                if (marked_bits(i) & 1u) f[0] = change(f[0], t);
                if (temp) f[0] = __fmul_rn(f[0], inv_t);
            }
            const T y = L::put(f[0]);
            out[t] = y;
            f[0] = L::get(y);
            sum.add(f, f[0]);
        }
    }
    // one vector of the output
    auto store = [&](int v, const uint4& res) {
        if (vec_out) {
            __stcs(reinterpret_cast<uint4*>(out + head + v * E), res);
        } else {
            const T* e = reinterpret_cast<const T*>(&res);
#pragma unroll
            for (int q = 0; q < E; ++q) out[head + v * E + q] = e[q];
        }
    };
    if (!dense) {
        // A sparse mask: a warp takes 32 words of it at a time (1024 tokens), a lane a word, and lists the allowed
        // tokens of as many such chunks as give up to 256; reads their logits, 8 a lane at once; fills the chunks
        // with -inf; and puts the processed logits in their places.
        constexpr int R = 8;
        const int lane = tid & 31;
        int* list = reinterpret_cast<int*>(s_vec) + (tid >> 5) * (32 * R);
        const int first = rank == 0 && head > 0 ? 1 : 0;  // the ragged head stands in the first E bits
        constexpr int step = kProcThreads;                // words of all warps' chunks
        int j_from = (tid >> 5) * 32, n = 0;              // the first chunk of the list, and its tokens
        auto flush = [&](int j_to) {                      // chunks j_from, j_from + step, .. before j_to
            float f[R];
#pragma unroll
            for (int q = 0; q < R; ++q)
                if (lane + 32 * q < n) f[q] = L::get(x[list[lane + 32 * q]]);
            __syncwarp();
            const uint4 none = make_uint4(L::kNegInfPair, L::kNegInfPair, L::kNegInfPair, L::kNegInfPair);
            for (int j0 = j_from; j0 < j_to; j0 += step)
#pragma unroll
                for (int q = 0; q < 32 / E; ++q) {
                    const int v = v0 - first + 32 * j0 / E + lane + 32 * q;
                    if (v >= v0 && v < v1) store(v, none);
                }
            __syncwarp();
#pragma unroll
            for (int q = 0; q < R; ++q)
                if (lane + 32 * q < n) {
                    const int t = list[lane + 32 * q];
                    float y[1] = {f[q]};
                    if (marked_bits(t - base) & 1u) y[0] = change(y[0], t);
                    if (temp) y[0] = __fmul_rn(y[0], inv_t);
                    const T o = L::put(y[0]);
                    out[t] = o;
                    y[0] = L::get(o);
                    sum.add(y, y[0]);
                }
            __syncwarp();
            n = 0;
            j_from = j_to;
        };
        int j0 = j_from;
        for (; j0 < words; j0 += step) {
            uint32_t bits = j0 + lane < words ? bm_mask[j0 + lane] : 0u;
            const int t0 = base + 32 * (j0 + lane);  // token of the word's first bit
            // only the vectors' tokens
            const int skip = head + v0 * E - t0, left = head + v1 * E - t0;
            if (skip > 0) bits &= ~((1u << skip) - 1);
            if (left < 32) bits &= left > 0 ? (1u << left) - 1 : 0u;
            int at = __popc(bits);
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(~0u, at, d);
                if (lane >= d) at += o;
            }
            const int more = __shfl_sync(~0u, at, 31);
            if (n + more > 32 * R) flush(j0);
            at += n - __popc(bits);
            for (; bits; bits &= bits - 1) list[at++] = t0 + __ffs(bits) - 1;
            n += more;
            __syncwarp();
        }
        flush(j0);
    }

    // temperature, mask, rounding, the sum of the stored values, and the store
    auto finish = [&](int v, uint32_t k, float (&f)[E]) {
        if (temp) {
#pragma unroll
            for (int e = 0; e < E; e += 2) mul2(f[e], f[e + 1], inv_t);
        }
        if (k != ALL) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (!((k >> e) & 1u)) f[e] = kNegInf;
        }
        const uint4 res = L::pack(f);
        L::unpack(res, f);  // the log-sum-exp is that of the stored values
        sum.add(f, L::top(L::max2(L::max2(res.x, res.y), L::max2(res.z, res.w))));
        store(v, res);
    };
    // a vector with marked tokens
    auto finish_marked = [&](int v, const uint4& raw) {
        const int t0 = head + v * E, i = t0 - base;
        const uint32_t k = mrow ? (bm_mask[i >> 5] >> (i & 31)) & ALL : ALL;
        float f[E];
        L::unpack(raw, f);
        for (uint32_t todo = marked_bits(i) & k; todo; todo &= todo - 1) {
            const int e = __ffs(todo) - 1;
            float y = f[0];
#pragma unroll
            for (int q = 1; q < E; ++q) y = e == q ? f[q] : y;
            y = change(y, t0 + e);
#pragma unroll
            for (int q = 0; q < E; ++q) f[q] = e == q ? y : f[q];
        }
        finish(v, k, f);
    };
    if (dense) {
        // all vectors of the slice but those with a marked token: each warp lists its own, as far as the list goes,
        // so that afterwards all threads have one each; places in the order of the vectors, hence sums in the same
        // order on every run
        const int lane = tid & 31, warp = tid >> 5;
        int listed = 0;
        bool loaded = !p.mask.bits;  // the first vectors are there
        for (int vb = v0 + tid; vb - lane < v1; vb += U * kProcThreads) {
            uint32_t keep = 0;  // E bits per vector
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int v = vb + u * kProcThreads;
                const int i = head + v * E - base;
                const uint32_t k = v >= v1 ? 0u : mrow ? (bm_mask[i >> 5] >> (i & 31)) & ALL : ALL;
                if (k && !loaded) val[u] = __ldcs(xv + v);
                keep |= k << (E * u);
            }
            loaded = false;
            uint32_t late = 0, aside = 0;
            if (pens || hots) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int v = vb + u * kProcThreads;
                    const uint32_t k = (keep >> (E * u)) & ALL;
                    const bool marked = k && (marked_bits(head + v * E - base) & k);
                    const uint32_t who = __ballot_sync(~0u, marked);
                    if (marked) {
                        const int at = listed + __popc(who & ((1u << lane) - 1));
                        aside |= 1u << u;
                        if (at < kProcListed) {
                            s_list[warp * kProcListed + at] = v;
                            s_vec[warp * kProcListed + at] = val[u];
                        } else {
                            late |= 1u << u;
                        }
                    }
                    listed += __popc(who);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int v = vb + u * kProcThreads;
                if (v >= v1) break;
                if ((aside >> u) & 1u) continue;
                const uint32_t k = (keep >> (E * u)) & ALL;
                if (!k) {
                    store(v, make_uint4(L::kNegInfPair, L::kNegInfPair, L::kNegInfPair, L::kNegInfPair));
                    continue;
                }
                float f[E];
                L::unpack(val[u], f);
                if (temp || k != ALL) {
                    finish(v, k, f);
                } else {
                    sum.add(f, L::top(L::max2(L::max2(val[u].x, val[u].y), L::max2(val[u].z, val[u].w))));
                    if (!in_place) store(v, val[u]);
                }
            }
            for (; late; late &= late - 1) {
                const int v = vb + (__ffs(late) - 1) * kProcThreads;
                finish_marked(v, __ldcs(xv + v));
            }
        }
        if (pens || hots) {
            if (lane == 0) s_listed[warp] = min(listed, kProcListed);
            __syncthreads();
            for (int i = tid;; i += kProcThreads) {
                int w = 0, j = i;  // the j-th of warp w
                while (w < kProcThreads / 32 && j >= s_listed[w]) j -= s_listed[w++];
                if (w == kProcThreads / 32) break;
                finish_marked(s_list[w * kProcListed + j], s_vec[w * kProcListed + j]);
            }
        }
    }

    // ---- the row's log-sum-exp: warp, CTA, cluster
    if (!p.lse) return;  // uniform
    Running run{sum.m, sum.s0 + sum.s1};
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
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(process_logits_kernel<DT>), smem, kProcessSmem);
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
constexpr int kSelWarps = kSelThreads / 32;
// Vectors per lane and unit, and CTAs per SM at the registers that takes. Without masks eight in flight and 128
// registers (built for three or four CTAs the loop spills). With masks much of a unit is the wait for the mask, then
// for the tokens it leaves: more warps on smaller units (128 x 96 rows of 32000 bf16, K = 192, 1 / 3 / 12 % allowed:
// 4 CTAs 191 / 208 / 263 us, 3 200 / 211 / 266, 2 252 / 264 / 327; eight vectors and 2 CTAs 250 / 267 / 480).
template <bool MASKED>
constexpr int kSelVectors = MASKED ? 4 : 8;
template <bool MASKED>
constexpr int kSelCtas = MASKED ? 4 : 2;
// Allowed ones of any 32 tokens up to which they are read one by one (the rows above, 1 / 3 / 12 / 25 / 50 %: always
// one by one 190 / 207 / 259 / 306 / 377 us, always vectors 293 / 298 / 296 / 297 / 292).
constexpr int kByBits = 8;
constexpr int kSelRounds = 4;  // most units per warp of the sample that sets the first floor

// Candidates as 64-bit keys: the score's order in the high half, the flat index (beam * vocab + token)
// complemented in the low half, so that the larger key is the better candidate and equal scores go by the
// lower index. Keys are distinct, hence the chosen set does not depend on the order of arrival.
__device__ __forceinline__ uint64_t candidate_key(float score, uint32_t flat) {
    return (static_cast<uint64_t>(float_order(score)) << 32) | static_cast<uint32_t>(~flat);
}

// The best K of each request in one pass over the logits. The units of all requests (32 * kSelVectors vectors of a
// row) are one sequence, cut evenly among the CTAs, whatever the batch; a CTA that crosses into another
// request leaves its list and begins anew. Inside a CTA the warps scan on their own. A unit costs a packed
// maximum over the lane's vectors and one comparison with the logit below which the row cannot reach the
// floor; where a lane passes, its elements are tried and the candidates go to a buffer in shared memory, each
// lane's next one at a time. When that is full the warps meet, cut it to the best K and raise the floor to the
// K-th. Rows with a sparse mask are read by its bits.
//
// The first floor is guessed from a sample of units spread over the CTA's, hence over its rows, for beams differ in
// their scores: if K of n vectors hold a candidate of the best K, a share K / n of the sample's do, and the floor is
// the sample's vector maximum some four deviations further down. It lets through a few times K candidates in all. If
// fewer than K come through, the CTA scans its part of the request once more under the sample's K-th maximum, which is
// a sure bound.
// Bound by reading the logits, and by the candidates' way through the buffer: 64 x 30 rows of 128000 bf16, K = 60,
// 129 us, 3.8 TB/s, 0.56 of what a copy reaches; 128 x 96 rows of 32000, K = 192, 190 us (98 and 154 us with a floor
// that no logit reaches, which is the scan alone). A run of units per warp in place of every eighth one took 239 us for
// the latter, rings of bulk copies in shared memory 190-198 us.
template <int DT, bool MASKED>
__global__ void __launch_bounds__(kSelThreads, kSelCtas<MASKED>) beam_scan_kernel(const SelectParams p) {
    using L = Logit<DT>;
    using T = typename L::T;
    constexpr int E = L::E, U = kSelVectors<MASKED>;
    constexpr uint32_t ALL = (1u << E) - 1;
    extern __shared__ uint64_t s_buf[];  // [p.cap], cap >= the sample's keys (4 per thread) and > K
    __shared__ TopkScratch<kSelThreads> s_top;
    __shared__ int s_count;
    __shared__ volatile int s_full;      // a warp waits for the buffer to be cut

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nseg = p.segments;         // units of a row
    const long long per_request = static_cast<long long>(p.W) * nseg;
    const long long total = per_request * p.batch;
    long long at = total * blockIdx.x / gridDim.x;
    const long long end = total * (blockIdx.x + 1) / gridDim.x;
    const int mwords = (p.vocab + 31) >> 5;
    bool sure = false;                   // the floor is no guess

    while (at < end) {  // one request at a time
        const int b = static_cast<int>(at / per_request);
        const int u_begin = static_cast<int>(at - b * per_request);
        const int u_end = static_cast<int>(min(per_request, end - b * per_request));
        uint64_t floor_key = 0;  // only larger keys are candidates
        bool have = false;       // it is set
        if (tid == 0) {
            s_count = 0;
            s_full = 0;
        }
        __syncthreads();

        // the present row: beam, logits, mask, scores' terms, elements before the first 16-byte boundary, vectors,
        // and the logit below which its scores stay under the floor
        int w = -1, head = 0, nv = 0;
        const T* x = nullptr;     // null: a beam without candidates (a cumulative score of -inf or NaN)
        const uint32_t* mrow = nullptr;
        float cum = 0.f, lse = 0.f, reach = 0.f;
        auto set_reach = [&]() {
            // less a margin that covers the score's two roundings (2^-24 of |score| + |cum| + |lse| each)
            const float fl = have ? order_float(static_cast<uint32_t>(floor_key >> 32)) : kNegInf;
            const float room = (fabsf(fl) + fabsf(cum) + fabsf(lse)) * 0x1p-20f;
            reach = have && room < 1e30f ? fl - cum + lse - room : kNegInf;  // (room: false for NaN)
        };
        auto open_row = [&](int to, bool flag) {
            w = to;
            const int r = b * p.W + w;
            cum = __ldg(p.cum + static_cast<long long>(b) * p.cum_stride + w);
            lse = __ldg(p.lse + r);
            x = cum > kNegInf ? static_cast<const T*>(p.x) + static_cast<long long>(r) * p.x_stride : nullptr;
            head = min(lead_elems<E>(x), p.vocab);
            nv = (p.vocab - head) / E;
            if constexpr (MASKED) mrow = mask_row(p.mask, r, p.status, flag);
            set_reach();
        };
        auto score = [&](float v) { return __fadd_rn(__fsub_rn(v, lse), cum); };
        auto key_of = [&](float sc, int t) {
            return candidate_key(sc, static_cast<uint32_t>(w) * static_cast<uint32_t>(p.vocab) + t);
        };
        // All warps meet: a buffer of more than K is cut to the best K (and up to an eighth of the rest, which
        // saves passes). Returns whether all of them are done.
        auto meet = [&](bool done) -> bool {
            const bool all = __syncthreads_and(done);
            const int n = min(s_count, p.cap);
            int left = n;
            if (n > p.K) {
                floor_key = topk_compact<kSelThreads>(s_buf, n, p.K, all ? 0 : (p.cap - p.K) >> 3, s_top);
                have = true;
                left = s_top.count;
            }
            __syncthreads();
            if (tid == 0) {
                s_count = left;
                s_full = 0;
            }
            __syncthreads();
            set_reach();
            return all;
        };
        // Stores each lane's candidate (ok): places in the buffer by one atomic for the warp; when it is full the
        // warps meet, and what found no place is tried against the new floor. (A NaN score compares false.)
        auto put = [&](bool ok, float sc, int t) {
            const uint64_t key = key_of(sc, t);
            ok = ok && sc > kNegInf && (!have || key > floor_key);
            for (;;) {
                const uint32_t who = __ballot_sync(~0u, ok);
                if (!who) break;
                int to = 0;
                if (lane == 0) to = atomicAdd(&s_count, __popc(who));
                to = __shfl_sync(~0u, to, 0) + __popc(who & ((1u << lane) - 1));
                if (ok && to < p.cap) {
                    s_buf[to] = key;
                    ok = false;
                }
                if (!__any_sync(~0u, ok)) break;
                if (lane == 0) s_full = 1;
                meet(false);
                ok = ok && key > floor_key;
            }
        };
        // lane i: which of tokens 32 i .. 32 i + 31 of the unit that begins at vector v0 are allowed
        auto allowed = [&](int v0) -> uint32_t {
            static_assert(!MASKED || U * E <= 32, "a word of the mask per lane");
            const int t = head + v0 * E + 32 * lane, left = lane < U * E ? head + nv * E - t : 0;
            if (left <= 0) return 0u;
            return (mrow ? mask_bits(mrow, mwords, t) : ~0u) & (left < 32 ? (1u << left) - 1 : ~0u);
        };
        // the lane's vectors of the unit, those with an allowed token; their tokens that count, E bits each
        auto load = [&](int v0, uint32_t word, uint4 (&val)[U]) -> uint64_t {
            const uint4* xv = reinterpret_cast<const uint4*>(x + head) + v0 + lane;
            uint64_t keep = 0;
            if (!MASKED && v0 + 32 * U <= nv) {
#pragma unroll
                for (int k = 0; k < U; ++k) val[k] = __ldcs(xv + 32 * k);
                keep = E * U == 64 ? ~0ull : (1ull << (E * U & 63)) - 1;
            } else {
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    uint32_t m;
                    if constexpr (MASKED)
                        m = (__shfl_sync(~0u, word, lane * E / 32 + E * k) >> (lane * E & 31)) & ALL;
                    else
                        m = v0 + lane + 32 * k < nv ? ALL : 0u;
                    if (m) val[k] = __ldcs(xv + 32 * k);
                    keep |= static_cast<uint64_t>(m) << (E * k);
                }
            }
            return keep;
        };

        // ---- the first floor: from up to four units per warp, spread over the run
        {
            const int units = u_end - u_begin;
            const int rounds = max(1, min(kSelRounds, units / kSelWarps)), probes = min(units, rounds * kSelWarps);
            const float mean = static_cast<float>(p.K) * probes / units;
            const int rank = sure ? p.K : min(p.K, static_cast<int>(mean + 4.f * sqrtf(mean)) + 4);
            uint64_t best[4] = {0, 0, 0, 0};  // the lane's best candidates: of a round, or of a quarter of the unit
#pragma unroll
            for (int q = 0; q < kSelRounds; ++q) {
                const int probe = q * kSelWarps + warp;
                if (q >= rounds || probe >= probes) break;
                const int u = u_begin + static_cast<int>(static_cast<long long>(units) * (2 * probe + 1) / (2 * probes));
                open_row(u / nseg, false);
                if (!x) continue;
                const int v0 = (u - w * nseg) * (32 * U);
                uint4 val[U];
                const uint64_t keep = load(v0, MASKED ? allowed(v0) : 0u, val);
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const uint32_t m = static_cast<uint32_t>(keep >> (E * k)) & ALL;
                    if (!m) continue;
                    float f[E], top = kNegInf;
                    int e0 = 0;
                    L::unpack(val[k], f);
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        if (((m >> e) & 1u) && f[e] > top) {
                            top = f[e];
                            e0 = e;
                        }
                    const float sc = score(top);
                    const uint64_t key = sc > kNegInf ? key_of(sc, head + E * (v0 + lane + 32 * k) + e0) : 0;
                    const int slot = rounds > 1 ? q : k / (U / 4);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i == slot && key > best[i]) best[i] = key;
                }
            }
            if (rank <= 64) {  // a lane's best alone: few lanes hold two of so few
                best[0] = max(max(best[0], best[1]), max(best[2], best[3]));
                best[1] = best[2] = best[3] = 0;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t who = __ballot_sync(~0u, best[i] != 0);
                if (!who) continue;
                int to = 0;
                if (lane == 0) to = atomicAdd(&s_count, __popc(who));
                to = __shfl_sync(~0u, to, 0) + __popc(who & ((1u << lane) - 1));
                if (best[i]) s_buf[to] = best[i];
            }
            __syncthreads();
            const int n = s_count;
            sure = rank == p.K || n < rank;
            if (n >= rank) {
                floor_key = topk_threshold<kSelThreads>(n, rank, 0, s_top, [&](int i) { return s_buf[i]; }) - 1;
                have = true;
            }
            __syncthreads();
            if (tid == 0) s_count = 0;
            w = -1;
            __syncthreads();
        }

        // ---- the scan
        int to_w = (u_begin + warp) / nseg, seg = u_begin + warp - to_w * nseg;
        for (int u = u_begin + warp; u < u_end; u += kSelWarps, seg += kSelWarps) {
            while (seg >= nseg) {
                seg -= nseg;
                ++to_w;
            }
            if (to_w != w) open_row(to_w, lane == 0 && seg < kSelWarps);
            if (__any_sync(~0u, s_full)) meet(false);  // (the lanes' reads may differ: the warp goes together)
            if (!x) continue;
            const int v0 = seg * (32 * U);
            uint64_t pend = 0;  // the lane's elements that reach the floor
            float first = 0.f;  // the first one's logit: most units that have any hold one
            uint32_t word = 0;
            bool by_bits = false;
            if constexpr (MASKED) {
                // few allowed: those are read one by one
                word = allowed(v0);
                by_bits = __reduce_max_sync(~0u, __popc(word)) <= kByBits;
                if (by_bits) {
                    constexpr int R = 4;  // a lane's tokens in flight together
                    while (__any_sync(~0u, word != 0)) {
                        float v[R];
                        int t[R];
#pragma unroll
                        for (int q = 0; q < R; ++q) {
                            t[q] = word ? head + v0 * E + 32 * lane + __ffs(word) - 1 : -1;
                            v[q] = word ? L::get(x[t[q]]) : kNegInf;
                            word &= word - 1;
                        }
#pragma unroll
                        for (int q = 0; q < R; ++q) {
                            const bool ok = t[q] >= 0 && v[q] >= reach;
                            if (__any_sync(~0u, ok)) put(ok, score(v[q]), t[q]);
                        }
                    }
                }
            }
            if (!by_bits) {
                uint4 val[U];
                const uint64_t keep = load(v0, word, val);
                bool hit = true;
                if (!MASKED && v0 + 32 * U <= nv) {  // all vectors there: one maximum
                    uint4 m = val[0];
#pragma unroll
                    for (int k = 1; k < U; ++k) {
                        m.x = L::max2(m.x, val[k].x);
                        m.y = L::max2(m.y, val[k].y);
                        m.z = L::max2(m.z, val[k].z);
                        m.w = L::max2(m.w, val[k].w);
                    }
                    hit = L::top(L::max2(L::max2(m.x, m.y), L::max2(m.z, m.w))) >= reach;
                }
                if (__any_sync(~0u, hit)) {
#pragma unroll
                    for (int k = 0; k < U; ++k) {
                        const uint32_t m = static_cast<uint32_t>(keep >> (E * k)) & ALL;
                        const bool some = hit && m && (m != ALL || L::top(L::max2(L::max2(val[k].x, val[k].y), L::max2(val[k].z, val[k].w))) >= reach);
                        if (!__any_sync(~0u, some)) continue;
                        float f[E];
                        L::unpack(val[k], f);
                        uint32_t got = 0;
#pragma unroll
                        for (int e = 0; e < E; ++e) got |= f[e] >= reach ? 1u << e : 0u;
                        if (some && (got & m)) {
                            if (!pend) {
                                const int e0 = __ffs(got & m) - 1;
                                first = f[0];
#pragma unroll
                                for (int e = 1; e < E; ++e) first = e == e0 ? f[e] : first;
                            }
                            pend |= static_cast<uint64_t>(got & m) << (E * k);
                        }
                    }
                }
            }
            for (bool again = false; __any_sync(~0u, pend != 0); again = true) {
                const bool ok = pend != 0;
                const int bit = ok ? __ffsll(static_cast<long long>(pend)) - 1 : 0;
                pend &= pend - 1;
                const int t = head + E * (v0 + lane + 32 * (bit / E)) + bit % E;
                const float v = ok && again ? L::get(x[t]) : first;
                put(ok, score(v), t);
            }
            // the ragged ends of a row: with its first and its last unit
            const int n_head = seg == 0 ? head : 0;
            const int tail0 = head + nv * E;
            const int n_tail = seg == nseg - 1 ? p.vocab - tail0 : 0;
            if (n_head + n_tail > 0) {
                const int t = lane < n_head ? lane : tail0 + lane - n_head;
                const bool ok = lane < n_head + n_tail && (!mrow || (mask_bits(mrow, mwords, t) & 1u));
                put(ok, score(ok ? L::get(x[t]) : kNegInf), t);
            }
        }
        while (!meet(true)) {
        }
        const int n = s_count;
        if (n < p.K && !sure) {  // the guess was too high: once more under a sure floor
            sure = true;
            __syncthreads();
            continue;
        }
        sure = false;
        const long long list = static_cast<long long>(blockIdx.x) + b;
        if (tid == 0) {
            // the list's length, and for a full one a key that the request's best K exceed
            p.part_head[2 * list] = n;
            p.part_head[2 * list + 1] = n == p.K && have ? floor_key : 0;
        }
        for (int i = tid; i < n; i += kSelThreads) p.part_keys[list * p.K + i] = s_buf[i];
        at = b * per_request + u_end;
        __syncthreads();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

constexpr int kMergeThreads = 512;

// One CTA per request: the lists of the scanning CTAs that met it, cut to the best K and put in order. A list's
// place is CTA + request: going through the units, one of the two grows at every step. Every full list's
// K-th key is a bound for all, so most of the others' keys fall away as they are read.
__global__ void __launch_bounds__(kMergeThreads) beam_merge_kernel(const SelectParams p) {
    extern __shared__ uint64_t s_buf[];  // [most lists of a request * K]
    __shared__ TopkScratch<kMergeThreads> s_top;
    __shared__ int s_count;
    __shared__ unsigned long long s_floor;
    const int tid = threadIdx.x, lane = tid & 31;
    const int b = blockIdx.x;
    if (tid == 0) {
        s_count = 0;
        s_floor = 0;
    }
    const long long per_request = static_cast<long long>(p.W) * p.segments;
    const long long total = per_request * p.batch;
    // CTA c scans the units from total * c / ctas on: the last c whose first unit is not behind x
    auto cta_of = [&](long long x) { return static_cast<int>(((x + 1) * p.ctas - 1) / total); };
    const int c0 = cta_of(b * per_request), c1 = cta_of((b + 1) * per_request - 1);
    const int lists = c1 - c0 + 1;
    const unsigned long long* heads = reinterpret_cast<const unsigned long long*>(p.part_head) + 2 * (static_cast<long long>(c0) + b);
    const unsigned long long* keys = reinterpret_cast<const unsigned long long*>(p.part_keys) + (static_cast<long long>(c0) + b) * p.K;
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int s = tid; s < lists; s += kMergeThreads) atomicMax(&s_floor, __ldcg(heads + 2 * s + 1));
    __syncthreads();
    const unsigned long long floor = s_floor;
    constexpr int R = 4;
    const int slots = lists * p.K;
    for (int i0 = 0; i0 < slots; i0 += R * kMergeThreads) {
        unsigned long long key[R], len[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {  // (places behind a list's end hold anything, and are passed over)
            const int i = i0 + q * kMergeThreads + tid;
            key[q] = i < slots ? __ldcg(keys + i) : 0ull;
            len[q] = i < slots ? __ldcg(heads + 2 * (i / p.K)) : 0ull;
        }
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const int i = i0 + q * kMergeThreads + tid;
            const bool in = i < slots && static_cast<unsigned long long>(i % p.K) < len[q] && key[q] > floor;
            const uint32_t who = __ballot_sync(~0u, in);
            if (!who) continue;
            int first = 0;
            if (lane == 0) first = atomicAdd(&s_count, __popc(who));
            first = __shfl_sync(~0u, first, 0);
            if (in) s_buf[first + __popc(who & ((1u << lane) - 1))] = key[q];
        }
    }
    __syncthreads();
    int n = s_count;
    if (n > p.K && n > kTopkRanked) {
        topk_compact<kMergeThreads>(s_buf, n, p.K, 0, s_top);
        n = p.K;
    }
    // rank = number of larger keys (distinct keys): the output place
    const long long o = static_cast<long long>(b) * p.K;
    for (int i = tid; i < n; i += kMergeThreads) {
        const uint64_t key = s_buf[i];
        int place = 0;
#pragma unroll 8
        for (int j = 0; j < n; ++j) place += s_buf[j] > key;
        if (place >= p.K) continue;
        const uint32_t flat = ~static_cast<uint32_t>(key);
        p.scores[o + place] = order_float(static_cast<uint32_t>(key >> 32));
        p.parents[o + place] = static_cast<int32_t>(flat / static_cast<uint32_t>(p.vocab));
        p.tokens[o + place] = static_cast<int32_t>(flat % static_cast<uint32_t>(p.vocab));
    }
    for (int i = n + tid; i < p.K; i += kMergeThreads) {
        p.scores[o + i] = kNegInf;
        p.parents[o + i] = -1;
        p.tokens[o + i] = -1;
    }
}

template <int DT, bool MASKED>
cudaError_t launch_scan_t(const SelectParams& p, cudaStream_t stream) {
    const size_t smem = static_cast<size_t>(p.cap) * 8;  // at most 8 KB
    beam_scan_kernel<DT, MASKED><<<p.ctas, kSelThreads, smem, stream>>>(p);
    return cudaGetLastError();
}
template <int DT>
cudaError_t launch_scan(const SelectParams& p, cudaStream_t stream) {
    return p.mask.bits ? launch_scan_t<DT, true>(p, stream) : launch_scan_t<DT, false>(p, stream);
}

}  // namespace

cudaError_t launch_process(int dtype, const ProcessParams& p, int cluster, size_t smem, cudaStream_t stream) {
    switch (dtype) {
        case BSP_LOGITS_BF16: return launch_process_t<BSP_LOGITS_BF16>(p, cluster, smem, stream);
        case BSP_LOGITS_FP16: return launch_process_t<BSP_LOGITS_FP16>(p, cluster, smem, stream);
        default: return launch_process_t<BSP_LOGITS_FP32>(p, cluster, smem, stream);
    }
}

// Logits of a scanning unit, warps of a CTA, CTAs resident on an SM, and the least buffer of a CTA.
int select_unit_elems(int dtype, bool masked) { return 32 * (masked ? kSelVectors<true> : kSelVectors<false>) * (dtype == BSP_LOGITS_FP32 ? 4 : 8); }
int select_unit_warps() { return kSelWarps; }
int select_sm_ctas(bool masked) { return masked ? kSelCtas<true> : kSelCtas<false>; }
int select_buffer(int K) {
    const int sample = 4 * kSelThreads;
    return K + 256 > sample ? K + 256 : sample;
}

cudaError_t launch_select(int dtype, const SelectParams& p, int most_lists, cudaStream_t stream) {
    cudaError_t e = dtype == BSP_LOGITS_BF16   ? launch_scan<BSP_LOGITS_BF16>(p, stream)
                    : dtype == BSP_LOGITS_FP16 ? launch_scan<BSP_LOGITS_FP16>(p, stream)
                                               : launch_scan<BSP_LOGITS_FP32>(p, stream);
    if (e != cudaSuccess) return e;
    const size_t smem = static_cast<size_t>(most_lists) * p.K * 8;
    e = allow_smem(reinterpret_cast<const void*>(beam_merge_kernel), smem, kMergeKeys * 8);
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
