// Log probabilities of given tokens, with their place among the vocabulary, the entropy and the top alternatives.
//
// With M = max x and Z' = the sum of exp(x - M) over all entries but one that attains M,
//     log p(i) = (x_i - M) - log1p(Z'),     entropy = log1p(Z') - S / (1 + Z'),  S = sum exp(x - M) (x - M),
// so that a token of probability near one keeps the bits of its small log, and the entropy is a sum of terms of one
// sign.  One read of the logits from HBM: a warp copies a CTA's rows to a ring in shared memory, ahead into the next
// row; each thread keeps the running (M, Z, S) of its entries and counts those that come before the token, in packed
// bf16 or fp16.  Z is held in two parts, the chunk of 32 entries (fp32: 16) that holds the maximum and the rest; only the
// threads that hold the row's maximum read that chunk again and sum it without it.
//
// The terms are taken as 2^(x log2(e) - C) with C = M log2(e) rounded, one multiplication-addition each, and the sums
// corrected by 2^(C - M log2(e)), which is near one while M is of ordinary size.  A CTA whose maximum is beyond +-4096 (a
// row of masks, infinity) reads its entries once more and takes each as exp(x - M).
//
// The sums are kept against a reference that is at most 8 below the running maximum, so that they are scaled once or
// twice a row.
//
// The top alternatives are found by a threshold: of the maxima of 32 groups of threads the K-th largest is a lower
// bound of the K-th largest entry.  The vectors of threads whose maximum reaches it are searched again (from L2) by the
// whole CTA, which lists what reaches it, some 30 to 130 entries; those are ranked by counting.  Where the list
// overflows (many equal entries: masks), those above the bound and the first ones equal to it are listed instead; where
// that does not do either, K searches.  Order: larger first, equal ones by index, NaN below -inf.
//
// Bound: instructions, about 7 an entry of bf16 (packed maximum and count 1.5, conversions 1, exponential and sums 2.5),
// with the exponentials next: 2,048 rows of 151,936 take 125 us, 5.0 TB/s; 256 rows 27 us, where 104 of
// the SMs have two rows and the others one; 17 rows of fp32 17 us, mostly the chain from the first load to the result.
//
// A cluster of up to 8 CTAs shares a row where there are few rows: they write states and lists to the first one, which
// merges them in rank order.
#include <math.h>

#include <algorithm>

#include "va_convert.cuh"
#include "va_internal.h"

namespace va {

struct LogprobParams {
    const void *logits;
    int64_t stride;  // elements between rows
    const int32_t *tokens;
    float *logprobs, *entropy, *top_logprobs;
    int32_t *ranks, *top_tokens;
    int rows, vocab, top, cluster;
};

namespace {

constexpr int kMaxTop = 32;
constexpr int kMaxCluster = 8;
// Small CTAs, three of an SM, so that one's search at its row's end runs beside the others' sums: 2,048 rows of 151,936
// bf16 took 165 us with 2 x 512 threads, 129 with 3 x 256, 130 with 5 x 128 (whose 17 rows in fp32 took 23 us, not 17).
constexpr int kThreads = 256, kWarps = kThreads / 32;  // and a warp that loads
constexpr int kVecs = 4;                               // 16-byte vectors of a thread in a chunk
constexpr int kChunk = kThreads * kVecs;               // vectors
constexpr int kStages = 4;
constexpr int kCtas = 3;     // of an SM
constexpr int kList = 1024;  // candidates
constexpr int kFirst = 512;  // entries of a slice whose ties with the bound are taken where there are too many
constexpr int kTake = 16;    // chunks between takes of the packed counts
constexpr uint32_t kRingBytes = kStages * kChunk * 16;
// A wait that runs out leaves NaN.  The tests build a copy of this file in which a cluster's CTA of one rank loads only
// the first chunk of its first row, so that its waits run out, and soon.
#ifndef VA_LOGPROBS_WITHHELD
#define VA_LOGPROBS_WITHHELD -1
#define VA_LOGPROBS_WAIT_NS 2000000000ull
#endif
constexpr int kWithheld = VA_LOGPROBS_WITHHELD;
constexpr uint64_t kWaitNs = VA_LOGPROBS_WAIT_NS;
static_assert(kWarps * 32 <= kList && kTake * 4 * kVecs <= 256, "bounds go through the list; packed counts are exact");

// Beyond this a maximum has too few bits behind the point for C; see above.  Reference points below -4 kWide are
// replaced by 0: their entries have no weight then, and none beside a maximum that is not below -kWide either.
constexpr float kWide = 4096.f;

typedef unsigned long long u64;

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN stays
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Floats in an order of unsigned integers: NaN lowest (0), both zeros alike.
__device__ __forceinline__ uint32_t order_of(float x) {
    if (x != x) return 0u;
    const uint32_t b = __float_as_uint(x + 0.f);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
    if (o == 0u) return __uint_as_float(0x7FFFFFFFu);
    return __uint_as_float((o & 0x80000000u) ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ u64 key_of(float x, int i) { return (u64)order_of(x) << 32 | (0xFFFFFFFFu - (uint32_t)i); }

// exp(d) for d <= 0, |relative error| about 2^-22 + 2^-24 |d|: 0 for d of -1e30
__device__ __forceinline__ float exp_neg(float d) { return ex2_approx(d * 1.4426950408889634f); }

// The bits of the next value below (a type of `sign` + 1 bits; not -0).
__device__ __forceinline__ uint32_t next_below(uint32_t b, int sign) {
    return b >> sign ? b + 1 : b ? b - 1 : (1u << sign) + 1;
}

// What a type needs: kN entries in 16 bytes; the larger of packed entries, NaN left out, and the larger of a word's; a word
// with what is below a floor raised to it, which is finite; entries as floats; a bound, the next value below one (so
// that "at least x" is "greater than below(x)"), and a count of entries that are greater than a bound.
template <typename T>
struct Type;
template <>
struct Type<float> {
    static constexpr int kN = 4;
    static constexpr uint32_t kLowest = 0xFF800000u;
    static __device__ __forceinline__ float one(const float *p) { return __ldg(p); }
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }
    static __device__ __forceinline__ float top(uint32_t w) { return __uint_as_float(w); }
    static __device__ __forceinline__ uint32_t raise(uint32_t w) { return __float_as_uint(max_nan(__uint_as_float(w), -1e30f)); }
    static __device__ __forceinline__ void floats(const uint32_t (&w)[4], float *x) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(w[i]);
    }
    static __device__ __forceinline__ uint32_t bound(float x) { return __float_as_uint(x + 0.f); }
    static __device__ __forceinline__ uint32_t below(uint32_t b) { return next_below(b, 31); }
    struct Count {
        int n = 0;
        __device__ __forceinline__ void add(const uint32_t (&w)[4], uint32_t bound) {
#pragma unroll
            for (int i = 0; i < 4; ++i) n += __uint_as_float(w[i]) > __uint_as_float(bound);
        }
        __device__ __forceinline__ int take() {
            const int t = n;
            n = 0;
            return t;
        }
    };
};
template <>
struct Type<__nv_bfloat16> {
    static constexpr int kN = 8;
    static constexpr uint32_t kLowest = 0xFF80FF80u;
    static __device__ __forceinline__ float one(const __nv_bfloat16 *p) {
        return bf16_bits_to_float(__ldg(reinterpret_cast<const unsigned short *>(p)));
    }
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    static __device__ __forceinline__ float top(uint32_t w) {
        return fmaxf(bf16_bits_to_float(w & 0xFFFFu), __uint_as_float(w & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint32_t raise(uint32_t w) {
        uint32_t d;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(w), "r"(0xF14AF14Au));
        return d;
    }
    static __device__ __forceinline__ void floats(const uint32_t (&w)[4], float *x) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    static __device__ __forceinline__ uint32_t bound(float x) { return (__float_as_uint(x + 0.f) >> 16) * 0x10001u; }
    static __device__ __forceinline__ uint32_t below(uint32_t b) { return next_below(b & 0xFFFFu, 15) * 0x10001u; }
    struct Count {
        uint32_t n = 0;  // two counts in bf16, exact up to 256
        __device__ __forceinline__ void add(const uint32_t (&w)[4], uint32_t bound) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t m;
                asm("set.gt.bf16x2.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(w[i]), "r"(bound));
                asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(n) : "r"(m), "r"(0x3F803F80u));
            }
        }
        __device__ __forceinline__ int take() {
            const int t = (int)__uint_as_float(n << 16) + (int)__uint_as_float(n & 0xFFFF0000u);
            n = 0;
            return t;
        }
    };
};
template <>
struct Type<__half> {
    static constexpr int kN = 8;
    static constexpr uint32_t kLowest = 0xFC00FC00u;
    static __device__ __forceinline__ float one(const __half *p) { return __half2float(*p); }
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    static __device__ __forceinline__ float2 pair(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }
    static __device__ __forceinline__ float top(uint32_t w) { return fmaxf(pair(w).x, pair(w).y); }
    static __device__ __forceinline__ uint32_t raise(uint32_t w) {
        uint32_t d;
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(w), "r"(0xFBFFFBFFu));
        return d;
    }
    static __device__ __forceinline__ void floats(const uint32_t (&w)[4], float *x) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = pair(w[i]).x, x[2 * i + 1] = pair(w[i]).y;
    }
    static __device__ __forceinline__ uint32_t bound(float x) {
        const __half h = __float2half_rn(x + 0.f);  // it is one
        return *reinterpret_cast<const unsigned short *>(&h) * 0x10001u;
    }
    static __device__ __forceinline__ uint32_t below(uint32_t b) { return next_below(b & 0xFFFFu, 15) * 0x10001u; }
    struct Count {
        uint32_t n = 0;  // two counts in fp16
        __device__ __forceinline__ void add(const uint32_t (&w)[4], uint32_t bound) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t m;
                asm("set.gt.f16x2.f16x2 %0, %1, %2;" : "=r"(m) : "r"(w[i]), "r"(bound));
                asm("add.rn.f16x2 %0, %1, %0;" : "+r"(n) : "r"(m));
            }
        }
        __device__ __forceinline__ int take() {
            const int t = (int)pair(n).x + (int)pair(n).y;
            n = 0;
            return t;
        }
    };
};

// The entries of a row that a CTA has: the row's vectors [v0, v1), in chunks, each dealt to the threads one by one, and
// single entries: those before the row's first 16-byte boundary and those behind its last whole vector.
template <typename T>
struct Slice {
    static constexpr int kN = Type<T>::kN;
    const T *row;
    const uint4 *body;
    int lead;  // entries before the first vector
    int head, v0, v1, tail0, tail1;

    __device__ __forceinline__ Slice(const LogprobParams &p, int64_t n, int rank) {
        row = static_cast<const T *>(p.logits) + n * p.stride;
        const int skip = (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / (int)sizeof(T);
        lead = min(skip, p.vocab);
        body = reinterpret_cast<const uint4 *>(row + lead);
        const int vectors = (p.vocab - lead) / kN, per = (vectors + p.cluster - 1) / p.cluster;
        v0 = min(vectors, rank * per), v1 = min(vectors, v0 + per);
        head = rank == 0 ? lead : 0;
        tail0 = lead + vectors * kN, tail1 = rank == p.cluster - 1 ? p.vocab : 0;
    }
    __device__ __forceinline__ int chunks() const { return (v1 - v0 + kChunk - 1) / kChunk; }
    __device__ __forceinline__ int vector(int c, int i) const { return v0 + c * kChunk + i * kThreads + (int)threadIdx.x; }
    __device__ __forceinline__ int index(int v) const { return lead + v * kN; }  // of its first entry
    // calls f(words, vector) for each vector of this thread, from global memory
    template <typename F>
    __device__ __forceinline__ void vectors(F f) const {
#pragma unroll 1
        for (int v = v0 + (int)threadIdx.x; v < v1; v += kThreads) {
            const uint4 x = __ldg(body + v);
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
            f(w, v);
        }
    }
    // calls f(index) for each single entry of this thread
    template <typename F>
    __device__ __forceinline__ void singles(F f) const {
        if ((int)threadIdx.x < head) f((int)threadIdx.x);  // at most seven each
        if (tail0 + (int)threadIdx.x < tail1) f(tail0 + (int)threadIdx.x);
    }
};

struct State {
    float m, z, s;  // the maximum; the sum of exp(x - m) without one entry that attains it; sum of exp(x - m)(x - m)
};

__device__ __forceinline__ State merge(State a, State b) {
    if (b.m > a.m) {
        const State t = a;
        a = b, b = t;
    }
    const bool none = b.m == -INFINITY;
    const float d = none ? 0.f : max_nan(b.m - a.m, -1e30f), e = none ? 0.f : exp_neg(d);
    const float w = 1.f + b.z;
    a.s += none ? b.s * 0.f : e * (b.s + d * w);
    a.z += none ? b.z * 0.f : e * w;  // NaN stays
    return a;
}

// A thread's running state: the maximum m, and the sums of the entries against `ref`, which is at most kLag below it (so
// that they are rarely scaled), in two parts: the chunk that holds the maximum and the rest.
struct Running {
    float m = -INFINITY, ref = -INFINITY, rest = 0.f, held = 0.f, s = 0.f, s_held = 0.f;
    int chunk = 0;  // that chunk; ~i: the single entry i
    __device__ __forceinline__ void move(float to) {  // the reference
        const float d = ref == -INFINITY ? -1e30f : fmaxf(ref - to, -1e30f), e = exp_neg(d);
        s = e * (s + d * rest);
        s_held = e * (s_held + d * held);
        rest *= e;
        held *= e;
        ref = to;
    }
    __device__ __forceinline__ void hold(float top, int c, float z, float sum) {  // c has the maximum now
        rest += held, s += s_held;
        held = z, s_held = sum;
        m = top;
        chunk = c;
    }
};
constexpr float kLag = 8.f;

// An entry by itself.
__device__ __forceinline__ void take_one(Running &r, float x, int i) {
    if (x > r.m) {
        r.move(x);
        r.hold(x, ~i, 1.f, 0.f);
    } else {
        const float d = max_nan(x - (r.ref == -INFINITY ? 0.f : r.ref), -1e30f), e = exp_neg(d);
        r.rest += e;
        r.s += e * d;
    }
}

// What the CTAs of a cluster give to the first one.
struct Given {
    State state;
    int before;
    u64 best[kMaxTop];
};

__device__ __forceinline__ void sync_rows() { named_bar_sync(1, kThreads); }  // the threads that take entries

template <typename T>
__global__ void __launch_bounds__(kThreads + 32, kCtas) logprobs_kernel(const LogprobParams p) {
    using Ty = Type<T>;
    constexpr int kN = Ty::kN;
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ __align__(8) uint64_t bars[2 * kStages];
    __shared__ float red_m[kWarps], red_z[kWarps], red_s[kWarps];
    __shared__ int red_c[kWarps], red_w[kWarps], count, threads, broken;
    __shared__ u64 best_of[kWarps], list[kList];
    __shared__ unsigned short who[kThreads];
    __shared__ Given given[kMaxCluster];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ranks = p.cluster, rank = blockIdx.x % ranks, V = p.vocab, K = p.top;
    const int n0 = blockIdx.x / ranks, step = gridDim.x / ranks;
    auto full = [&](int i) { return smem_u32(&bars[i]); };
    auto empty = [&](int i) { return smem_u32(&bars[kStages + i]); };
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(full(i), 1), mbar_init(empty(i), kWarps);
        fence_barrier_init();
        broken = 0;
    }
    __syncthreads();
    if (ranks > 1) cluster_arrive();  // this CTA has begun: see cluster_wait below
    griddep_wait();

    if (warp == kWarps) {
        // ------------------------------------------------------------ loads, ahead into the next row
        int g = 0;
        if (lane == 0) {
            bool ok = true;
            for (int n = n0; n < p.rows && ok; n += step) {
                const Slice<T> sl(p, n, rank);
                for (int v = sl.v0; v < sl.v1 && ok; v += kChunk, ++g) {
                    if (rank == kWithheld && v > sl.v0) {
                        n = p.rows;
                        break;
                    }
                    const int st = g % kStages;
                    if (g >= kStages) ok = mbar_wait(empty(st), (g / kStages - 1) & 1, kWaitNs);
                    if (!ok) break;
                    const uint32_t bytes = 16u * min(kChunk, sl.v1 - v);
                    mbar_arrive_expect_tx(full(st), bytes);
                    bulk_load(smem_u32(ring) + 16u * kChunk * st, sl.body + v, bytes, full(st));
                }
            }
            // every issued copy lands before the CTA ends
            for (int i = max(0, g - kStages); i < g; ++i) ok &= mbar_wait(full(i % kStages), (i / kStages) & 1, kWaitNs);
            if (!ok) broken = 1;
        }
        __syncwarp();
        if (ranks > 1) {
            cluster_wait();
            cluster_sync();
        }
        return;
    }

    int g = 0;
    int token = n0 < p.rows ? __ldg(p.tokens + n0) : -1;
    float mine = token >= 0 && token < V ? Ty::one(static_cast<const T *>(p.logits) + n0 * p.stride + token) : 0.f;
    for (int n = n0; n < p.rows; n += step) {
        const Slice<T> sl(p, n, rank);
        const bool known = token >= 0 && token < V;
        const int after = n + step, next_token = after < p.rows ? __ldg(p.tokens + after) : -1;
        // entries before the token come before it where they are at least its logit, those behind it where they are
        // greater; beside the lowest and NaN by their order
        const bool by_order = known && !(mine > -INFINITY);
        const uint32_t bound_behind = Ty::bound(by_order || !known ? 0.f : mine), bound_before = Ty::below(bound_behind);
        const uint32_t mine_order = order_of(mine);
        auto precedes = [&](float x, int i) {
            const uint32_t o = order_of(x);
            return o > mine_order || (o == mine_order && i < token);
        };
        // vectors below this are before the token; its own counts as behind, but for the entries up to it
        const int token_vector = token < sl.lead ? -1 : (token - sl.lead) / kN;
        int before = 0;
        if (known && !by_order && tid < kN && token_vector >= sl.v0 && token_vector < sl.v1 && sl.index(token_vector) + tid < token)
            before = Ty::one(sl.row + sl.index(token_vector) + tid) == mine;
        if (tid == 0) count = threads = 0;

        Running r;
        typename Ty::Count counted;
        const int chunks = broken ? 0 : sl.chunks();  // a wait ran out in an earlier row
        auto take_chunk = [&](int c) {
            const uint32_t at = smem_u32(ring) + 16u * (kChunk * (g % kStages) + tid);
            const bool whole = sl.v1 - sl.v0 - c * kChunk >= kChunk;
            uint32_t w[kVecs][4], top[4] = {Ty::kLowest, Ty::kLowest, Ty::kLowest, Ty::kLowest};
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const bool has = whole || sl.vector(c, i) < sl.v1;
                const uint4 x = has ? lds_u4(at + 16u * kThreads * i) : make_uint4(Ty::kLowest, Ty::kLowest, Ty::kLowest, Ty::kLowest);
                w[i][0] = x.x, w[i][1] = x.y, w[i][2] = x.z, w[i][3] = x.w;
            }
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
#pragma unroll
                for (int k = 0; k < 4; ++k) top[k] = Ty::larger(top[k], w[i][k]);
                counted.add(w[i], sl.vector(c, i) < token_vector ? bound_before : bound_behind);
            }
            const float mb = Ty::top(Ty::larger(Ty::larger(top[0], top[1]), Ty::larger(top[2], top[3])));
            const bool moved = mb > r.m;
            if (mb > r.ref + kLag) r.move(mb);
            // 2^(x log2(e) - C) = exp(x - m) 2^off, off what C is below m log2(e)
            const float m = r.ref < -4.f * kWide ? 0.f : r.ref;
            const float l2e = 1.4426950408889634f, C = m * l2e;
            const float off = fmaf(m, l2e, -C);
            const uint64_t l2 = f2_pack(__float_as_uint(l2e), __float_as_uint(l2e));
            const uint64_t c2 = f2_pack(__float_as_uint(-C), __float_as_uint(-C));
            float z, s;
#pragma unroll 1
            for (bool again = false;; again = true) {
                uint64_t z2[2] = {0ull, 0ull}, s2[2] = {0ull, 0ull};
#pragma unroll
                for (int i = 0; i < kVecs; ++i) {
                    float x[kN];
                    Ty::floats(w[i], x);
#pragma unroll
                    for (int j = 0; j < kN; j += 2) {
                        const uint64_t t2 = f2_fma(f2_pack(__float_as_uint(x[j]), __float_as_uint(x[j + 1])), l2, c2);
                        uint32_t a, b;
                        f2_unpack(t2, a, b);
                        const uint64_t e2 = f2_pack(__float_as_uint(ex2_approx(__uint_as_float(a))),
                                                    __float_as_uint(ex2_approx(__uint_as_float(b))));
                        z2[(j / 2) & 1] = f2_add(z2[(j / 2) & 1], e2);
                        s2[(j / 2) & 1] = f2_fma(e2, t2, s2[(j / 2) & 1]);
                    }
                }
                uint32_t a, b;
                f2_unpack(f2_add(z2[0], z2[1]), a, b);
                z = __uint_as_float(a) + __uint_as_float(b);
                f2_unpack(f2_add(s2[0], s2[1]), a, b);
                s = __uint_as_float(a) + __uint_as_float(b);
                if (s == s || again) break;
                // 0 * -inf, or NaN
#pragma unroll
                for (int i = 0; i < kVecs; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[i][j] = Ty::raise(w[i][j]);
            }
            const float by = 1.f - 0.69314718f * off;  // 2^-off but for 2^-24: off is 2^-12 at most for kWide
            s = (s - off * z) * (0.69314718f * by), z *= by;
            if (moved)
                r.hold(mb, c, z, s);
            else
                r.rest += z, r.s += s;
        };
        for (int c = 0; c < chunks; ++c, ++g) {
            const int st = g % kStages;
            if (!mbar_wait(full(st), (g / kStages) & 1, kWaitNs)) {
                broken = 1;
                break;
            }
            take_chunk(c);
            if (c % kTake == kTake - 1) before += counted.take();
            fence_proxy_async_smem();  // the loads are done: the arrival by itself does not wait for their values
            __syncwarp();
            if (lane == 0) mbar_arrive(empty(st));
        }
        before += counted.take();
        if (by_order) {
            before = 0;
            sl.vectors([&](const uint32_t (&w)[4], int v) {
                float x[kN];
                Ty::floats(w, x);
#pragma unroll
                for (int j = 0; j < kN; ++j) before += precedes(x[j], sl.index(v) + j);
            });
        }
        sl.singles([&](int i) {
            const float x = Ty::one(sl.row + i);
            take_one(r, x, i);
            before += known && precedes(x, i);
        });

        // The CTA's maximum, and in `order_of`'s order the largest entry of each thread; without one above -inf it has
        // entries of -inf or NaN, or none (0).  Group i has lane i of each warp.
        float M = r.m;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        if (lane == 0) red_m[warp] = M;
        uint32_t *tops = reinterpret_cast<uint32_t *>(list);
        const uint32_t top = r.m > -INFINITY || (r.rest == r.rest && (sl.vector(0, 0) < sl.v1 || tid < sl.head || sl.tail0 + tid < sl.tail1))
                                 ? order_of(r.m) : 0u;
        if (K > 0) tops[tid] = top;
        sync_rows();
        M = red_m[0];
#pragma unroll
        for (int i = 1; i < kWarps; ++i) M = fmaxf(M, red_m[i]);
        uint32_t bound = 0;
        if (K > 0) {
            // the K-th largest of the groups' (0 where fewer groups have one: then everything is a candidate)
            uint32_t mine_g = tops[lane];
#pragma unroll
            for (int i = 1; i < kWarps; ++i) mine_g = max(mine_g, tops[32 * i + lane]);
            for (int k = 0;; ++k) {
                bound = __reduce_max_sync(0xffffffffu, mine_g);
                if (k == K - 1) break;
                const uint32_t has = __ballot_sync(0xffffffffu, mine_g == bound);
                if (lane == __ffs(has) - 1) mine_g = 0;
            }
            if (sl.vector(0, 0) < sl.v1 && (top >= bound || r.m == -INFINITY)) who[atomicAdd(&threads, 1)] = (unsigned short)tid;
            if (tid < kMaxTop) given[0].best[tid] = 0;
        }
        if (!(fabsf(M) <= kWide)) {  // alike in the CTA: every entry by itself
            r = Running();
            sl.vectors([&](const uint32_t (&w)[4], int v) {
                float x[kN];
                Ty::floats(w, x);
#pragma unroll
                for (int j = 0; j < kN; ++j) take_one(r, x[j], sl.index(v) + j);
            });
            sl.singles([&](int i) { take_one(r, Ty::one(sl.row + i), i); });
        }

        // sums against the CTA's maximum; those who hold it sum its chunk again without it
        const bool holds = r.m == M && M > -INFINITY;
        const float by = max_nan(r.ref - M, -1e30f), e0 = exp_neg(by);  // the reference's distance
        float z = r.rest, s = r.s;
        if (holds) {
            s = e0 * (s + by * z);
            z *= e0;
            if (r.chunk >= 0) {
                uint4 y[kVecs];
#pragma unroll
                for (int i = 0; i < kVecs; ++i)
                    if (sl.vector(r.chunk, i) < sl.v1) y[i] = __ldg(sl.body + sl.vector(r.chunk, i));
                bool out = false;
#pragma unroll
                for (int i = 0; i < kVecs; ++i) {
                    if (sl.vector(r.chunk, i) >= sl.v1) continue;
                    const uint32_t w[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
                    float x[kN];
                    Ty::floats(w, x);
#pragma unroll
                    for (int j = 0; j < kN; ++j) {
                        const bool it = !out && x[j] == M;
                        out |= it;
                        const float d = max_nan(x[j] - M, -1e30f), e = it ? 0.f : exp_neg(d);
                        z += e, s += e * d;
                    }
                }
            }
        } else if (r.m > -INFINITY) {
            const float w = z + r.held;
            s = e0 * (s + r.s_held + by * w);
            z = e0 * w;
        } else {
            z += r.held;  // nothing, or NaN
        }
        int c = before, w = holds;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            z += __shfl_xor_sync(0xffffffffu, z, o);
            s += __shfl_xor_sync(0xffffffffu, s, o);
            c += __shfl_xor_sync(0xffffffffu, c, o);
            w += __shfl_xor_sync(0xffffffffu, w, o);
        }
        if (lane == 0) red_z[warp] = z, red_s[warp] = s, red_c[warp] = c, red_w[warp] = w;
        if (after < p.rows && next_token >= 0 && next_token < V)
            mine = Ty::one(static_cast<const T *>(p.logits) + after * p.stride + next_token);
        const int this_token = token;
        token = next_token;
        sync_rows();

        // of `have` keys in `list`, in any order, the K largest to put(0 .. K-1, key), largest first: eight threads
        // count what is above a key
        auto rank_list = [&](int have, auto put) {
            for (int i0 = 0; i0 < have; i0 += kThreads / 8) {
                const int i = i0 + tid / 8;
                const u64 key = i < have ? list[i] : 0;
                int above = 0;
                for (int j = tid % 8; j < have; j += 8) above += list[j] > key;
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) above += __shfl_xor_sync(0xffffffffu, above, o);
                if (i < have && tid % 8 == 0 && above < K) put(above, key);
            }
        };
        if (K > 0) {
            const float least = value_of(bound);  // of a candidate; NaN: any
            const int found = threads, each = (sl.v1 - sl.v0 + kThreads - 1) / kThreads;
            int have = 0;
            bool above = false;
#pragma unroll 1
            for (;; above = true) {
                // `above`: of what lies above the bound everything, of what is equal to it the first entries
                const uint32_t from = bound + (above ? 1u : 0u);
                auto offer = [&](float x, int i) {
                    const uint32_t o = order_of(x);
                    if (o >= from && *static_cast<volatile int *>(&count) <= kList) {  // else it has overflowed
                        const int at = atomicAdd(&count, 1);
                        if (at < kList) list[at] = (u64)o << 32 | (0xFFFFFFFFu - (uint32_t)i);
                    }
                };
                for (int i = tid; i < found * each; i += kThreads) {
                    const int j = i / found, v = sl.v0 + j * kThreads + who[i - j * found];
                    if (v >= sl.v1) continue;
                    const uint4 y = __ldg(sl.body + v);
                    const uint32_t w[4] = {y.x, y.y, y.z, y.w};
                    if (Ty::top(Ty::larger(Ty::larger(y.x, y.y), Ty::larger(y.z, y.w))) < least) continue;
                    float x[kN];
                    Ty::floats(w, x);
#pragma unroll
                    for (int k = 0; k < kN; ++k) offer(x[k], sl.index(v) + k);
                }
                sl.singles([&](int i) { offer(Ty::one(sl.row + i), i); });
                if (above) {
                    const int first = rank == 0 ? 0 : sl.index(sl.v0);
                    for (int i = first + tid; i < min(first + kFirst, rank == 0 ? V : sl.index(sl.v1)); i += kThreads) {
                        const uint32_t o = order_of(Ty::one(sl.row + i));
                        if (o == bound) {
                            const int at = atomicAdd(&count, 1);
                            if (at < kList) list[at] = (u64)o << 32 | (0xFFFFFFFFu - (uint32_t)i);
                        }
                    }
                }
                sync_rows();
                have = count;
                if (above || have <= kList) break;
                sync_rows();  // it is read
                if (tid == 0) count = 0;
                sync_rows();
            }
            // (the second time the list holds the K largest if it holds as many)
            const bool search = have > kList || (above && have < K);
            if (search) {
                // too many reach the bound: the largest key below the last one found, K times
                u64 last = ~0ull;
                for (int k = 0; k < K; ++k) {
                    u64 best = 0;
                    auto look = [&](float x, int i) {
                        const u64 key = key_of(x, i);
                        if (key < last && key > best) best = key;
                    };
                    sl.vectors([&](const uint32_t (&w)[4], int v) {
                        float x[kN];
                        Ty::floats(w, x);
#pragma unroll
                        for (int j = 0; j < kN; ++j) look(x[j], sl.index(v) + j);
                    });
                    sl.singles([&](int i) { look(Ty::one(sl.row + i), i); });
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) best = max(best, (u64)__shfl_xor_sync(0xffffffffu, best, o));
                    sync_rows();
                    if (lane == 0) best_of[warp] = best;
                    sync_rows();
                    last = 0;
                    for (int i = 0; i < kWarps; ++i) last = max(last, best_of[i]);
                    if (tid == 0) given[0].best[k] = last;
                }
            } else {
                rank_list(have, [&](int at, u64 key) { given[0].best[at] = key; });
            }
        }
        if (tid == 0) {
            float zt = red_z[0], st = red_s[0];
            int ct = red_c[0], wt = red_w[0];
            for (int i = 1; i < kWarps; ++i) zt += red_z[i], st += red_s[i], ct += red_c[i], wt += red_w[i];
            // of several that attain the maximum one is left out
            given[0].state = {M, wt > 1 ? zt + (float)(wt - 1) : zt, st};
            const float none = __uint_as_float(0x7FFFFFFFu);
            if (broken) given[0].state = {none, none, none};  // a wait ran out: NaN through every merge
            given[0].before = ct;
        }
        sync_rows();
        if (ranks > 1) {
            cluster_wait();  // the first CTA has begun
            if (rank > 0) {
                constexpr int kWords = sizeof(Given) / 8;
                static_assert(sizeof(Given) % 8 == 0, "whole words");
                for (int i = tid; i < kWords; i += kThreads)
                    st_cluster_u64(reinterpret_cast<u64 *>(&given[rank]) + i, 0, reinterpret_cast<const u64 *>(&given[0])[i]);
            }
            cluster_sync();
            if (rank > 0) return;
        }
        State all = given[0].state;
        int ahead = given[0].before;
        for (int q = 1; q < ranks; ++q) {
            all = merge(all, given[q].state);
            ahead += given[q].before;
        }
        const bool empty_row = all.m == -INFINITY && all.z == all.z;  // nothing has any weight
        if (all.m == INFINITY) all.z = __uint_as_float(0x7FFFFFFFu);
        const float log_z = log1pf(all.z);
        auto log_prob = [&](float x) { return empty_row ? -INFINITY : (x - all.m) - log_z; };
        if (tid == 0) {
            const float x = known ? Ty::one(sl.row + this_token) : 0.f;
            if (p.logprobs) p.logprobs[n] = known ? log_prob(x) : -INFINITY;
            if (p.ranks) p.ranks[n] = known ? ahead : -1;
            if (p.entropy) p.entropy[n] = empty_row ? 0.f : log_z - all.s / (1.f + all.z);
        }
        if (K > 0) {
            auto put = [&](int at, u64 key) {
                if (key == 0) return;
                p.top_tokens[(int64_t)n * K + at] = (int32_t)(0xFFFFFFFFu - (uint32_t)key);
                p.top_logprobs[(int64_t)n * K + at] = log_prob(value_of((uint32_t)(key >> 32)));
            };
            if (ranks == 1) {
                if (tid < K) put(tid, given[0].best[tid]);
            } else {
                const int lists = ranks * K;
                for (int i = tid; i < lists; i += kThreads) list[i] = given[i / K].best[i % K];
                sync_rows();
                rank_list(lists, put);
            }
        }
    }
}

template <typename T>
cudaError_t launch_t(const LogprobParams &p, int sms, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(logprobs_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.cluster > 1 ? p.rows * p.cluster : std::min(p.rows, kCtas * sms)));
    cfg.blockDim = dim3(kThreads + 32);
    cfg.dynamicSmemBytes = kRingBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<T>, p);
}

}  // namespace
}  // namespace va

extern "C" int verify_attn_logprobs(const void *logits, int64_t stride, va_float_type type, const int32_t *tokens,
                                    int num_rows, int vocab, int num_top, float *logprobs, int32_t *ranks,
                                    float *entropy, int32_t *top_tokens, float *top_logprobs, void *stream) {
    if (num_rows < 0 || vocab < 1 || vocab > (1 << 30) || num_top < 0 || num_top > VA_LOGPROBS_MAX_TOP || num_top > vocab)
        return VA_ERR_INVALID_ARGUMENT;
    if (type != VA_FLOAT_BF16 && type != VA_FLOAT_FP16 && type != VA_FLOAT_FP32) return VA_ERR_UNSUPPORTED;
    const size_t size = type == VA_FLOAT_FP32 ? 4 : 2;
    if (!logits || !tokens || reinterpret_cast<uintptr_t>(logits) % size || (num_top > 0 && (!top_tokens || !top_logprobs)))
        return VA_ERR_INVALID_ARGUMENT;
    for (const void *x : {(const void *)tokens, (const void *)logprobs, (const void *)ranks, (const void *)entropy,
                          (const void *)top_tokens, (const void *)top_logprobs})
        if (reinterpret_cast<uintptr_t>(x) % 4) return VA_ERR_INVALID_ARGUMENT;
    if (num_rows > (1 << 27)) return VA_ERR_INVALID_ARGUMENT;
    if (num_rows == 0) return VA_OK;
    int device = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
    // a cluster of CTAs a row while the rows are fewer than the CTAs that the GPU holds
    int cluster = 1;
    while (cluster < va::kMaxCluster && (int64_t)num_rows * cluster * 2 <= va::kCtas * sms && vocab / (cluster * 2) >= 4096)
        cluster *= 2;
    const va::LogprobParams p = {logits, stride, tokens, logprobs, entropy, top_logprobs, ranks, top_tokens,
                                 num_rows, vocab, num_top, cluster};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (e == cudaSuccess)
        e = type == VA_FLOAT_FP32   ? va::launch_t<float>(p, sms, s)
            : type == VA_FLOAT_BF16 ? va::launch_t<__nv_bfloat16>(p, sms, s)
                                    : va::launch_t<__half>(p, sms, s);
    if (e == cudaSuccess) return VA_OK;
    va::note_cuda_error(e);
    cudaGetLastError();
    return VA_ERR_CUDA;
}
