// Log probabilities of given tokens, with their place among the vocabulary, the entropy and the top alternatives.
//
// With M = max x and Z' = the sum of exp(x - M) over all entries but one that attains M,
//     log p(i) = (x_i - M) - log1p(Z'),     entropy = log1p(Z') - S / (1 + Z'),  S = sum exp(x - M) (x - M),
// so that a token of probability near one keeps the bits of its small log, and the entropy is a sum of terms of one
// sign.  One read of the logits from HBM: each thread keeps the running (M, Z, S) of its entries and counts those that
// come before the token.  Z is held in two parts, the batch of 16 that holds the maximum and the rest; only the threads
// that hold the row's maximum read that batch again and sum it without it.
//
// The top alternatives are found by a threshold: of the maxima of 32 groups of threads the K-th largest is a lower
// bound of the K-th largest entry.  Threads whose maximum reaches it go through their entries again (from L2) and list
// what reaches it, some 30 to 130 entries; those are ranked by counting.  Rows whose list overflows (many equal
// entries) are searched K times instead.  Order: larger first, equal ones by index, NaN below -inf.
//
// A cluster of up to 8 CTAs shares a row where there are few rows; states and lists are merged in rank order.
#include <math.h>

#include <cstring>

#include "va_convert.cuh"
#include "va_internal.h"

namespace va {

struct LogprobParams {
    const void *logits;
    int64_t stride;  // elements between rows
    const int32_t *tokens;
    float *logprobs, *entropy, *top_logprobs;
    int32_t *ranks, *top_tokens;
    int vocab, top, cluster;
};

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 16;   // entries whose maximum is taken at once
constexpr int kList = 4096;  // candidates: more than a sorted row has (32 groups x 16 threads x 8 entries)
constexpr int kMaxTop = 32;

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

// 16 bytes of the row as floats.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int kN = 4;
    static __device__ __forceinline__ void unpack(const uint4 &v, float *x) {
        x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ float one(const float *p) { return __ldg(p); }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int kN = 8;
    static __device__ __forceinline__ void unpack(const uint4 &v, float *x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[2 * i] = bf16_bits_to_float(w[i] & 0xFFFFu), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    static __device__ __forceinline__ float one(const __nv_bfloat16 *p) {
        return bf16_bits_to_float(__ldg(reinterpret_cast<const unsigned short *>(p)));
    }
};
template <>
struct Vec<__half> {
    static constexpr int kN = 8;
    static __device__ __forceinline__ void unpack(const uint4 &v, float *x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
    }
    static __device__ __forceinline__ float one(const __half *p) { return __half2float(*p); }
};

// The entries of one CTA: the row's 16-byte vectors [v0, v1), dealt to the threads one by one, and single entries: of
// those before the first vector boundary the first `head`, from `tail0` on the last ones.
template <typename T>
struct Slice {
    static constexpr int kN = Vec<T>::kN;
    static constexpr int kVecs = kBatch / kN;  // vectors of a batch
    const T *row;
    const uint4 *body;
    int head, v0, v1, tail0, tail1;  // entries of vector v: head_all + v * kN ..
    int head_all;

    // calls f(x[16], first index of the batch's vectors, batch number, count) for each batch of this thread
    template <typename F>
    __device__ __forceinline__ void batches(F f) const {
        constexpr int kLoads = 64 / 16;  // vectors in flight
        for (int v = v0 + (int)threadIdx.x, n = 0; v < v1; v += kLoads * kThreads, n += kLoads / kVecs) {
            uint4 raw[kLoads];
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                if (v + i * kThreads < v1) raw[i] = __ldg(body + v + i * kThreads);
#pragma unroll
            for (int b = 0; b < kLoads / kVecs; ++b) {
                if (v + b * kVecs * kThreads >= v1) break;
                float x[kBatch];
#pragma unroll
                for (int i = 0; i < kVecs; ++i) {
                    if (v + (b * kVecs + i) * kThreads < v1) {
                        Vec<T>::unpack(raw[b * kVecs + i], x + i * kN);
                    } else {
#pragma unroll
                        for (int j = 0; j < kN; ++j) x[i * kN + j] = -INFINITY;
                    }
                }
                f(x, v + b * kVecs * kThreads, n + b);
            }
        }
    }
    // entry j of a batch whose first vector is v; kN-th vectors are kThreads apart.  A missing vector's entries: past v1
    __device__ __forceinline__ int index(int v, int j) const { return head_all + (v + j / kN * kThreads) * kN + j % kN; }
    __device__ __forceinline__ bool has(int v, int j) const { return v + j / kN * kThreads < v1; }
    // the first vector of batch n of this thread
    __device__ __forceinline__ int first_vector(int n) const { return v0 + (int)threadIdx.x + n * kVecs * kThreads; }
    // calls f(index) for each single entry of this thread
    template <typename F>
    __device__ __forceinline__ void singles(F f) const {
        for (int i = threadIdx.x; i < head; i += kThreads) f(i);
        for (int i = tail0 + (int)threadIdx.x; i < tail1; i += kThreads) f(i);
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
    const float d = none ? 0.f : b.m - a.m, e = none ? 0.f : exp_neg(max_nan(d, -1e30f));
    const float w = 1.f + b.z;
    a.s += none ? b.s * 0.f : e * (b.s + max_nan(d, -1e30f) * w);
    a.z += none ? b.z * 0.f : e * w;  // NaN stays
    return a;
}

template <typename F>
__device__ __forceinline__ float warp_sum(float x, F) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) logprobs_kernel(const LogprobParams p) {
    __shared__ float red_m[kWarps], red_z[kWarps], red_s[kWarps];
    __shared__ int red_c[kWarps], red_w[kWarps];
    __shared__ u64 group[32], list[kList], best[kMaxTop];
    __shared__ int count;
    __shared__ float out_m, out_z, out_s;
    __shared__ int out_c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ranks = p.cluster, rank = blockIdx.x % ranks, V = p.vocab, K = p.top;
    const int64_t n = blockIdx.x / ranks;
    griddep_wait();

    Slice<T> sl;
    constexpr int kN = Slice<T>::kN;
    sl.row = static_cast<const T *>(p.logits) + n * p.stride;
    const int skip = (int)((16 - (reinterpret_cast<uintptr_t>(sl.row) & 15)) & 15) / (int)sizeof(T);
    sl.head_all = min(skip, V);
    sl.body = reinterpret_cast<const uint4 *>(sl.row + sl.head_all);
    const int vectors = (V - sl.head_all) / kN, per = (vectors + ranks - 1) / ranks;
    sl.v0 = min(vectors, rank * per), sl.v1 = min(vectors, sl.v0 + per);
    sl.head = rank == 0 ? sl.head_all : 0;
    sl.tail0 = sl.head_all + vectors * kN, sl.tail1 = rank == ranks - 1 ? V : 0;

    const int token = p.tokens[n];
    const bool known = token >= 0 && token < V;
    const float mine = known ? Vec<T>::one(sl.row + token) : 0.f;
    const uint32_t mine_order = order_of(mine);
    // entries before the token count where they are not less, those behind it where they are greater; "not less than
    // mine" is "greater than the next float below"; NaN and -inf, which have none, by their order
    const bool by_order = !(mine > -INFINITY);
    const float below = by_order ? 0.f : mine == 0.f ? -__int_as_float(1) : value_of(mine_order - 1);  // 0 is both zeros
    auto precedes = [&](float x, int i) { const uint32_t o = order_of(x); return o > mine_order || (o == mine_order && i < token); };

    float m = -INFINITY, rest = 0.f, held = 0.f, s = 0.f;  // held: the sum of the batch with the maximum, which counts 1
    int held_batch = -1, held_at = 0, before = 0;          // and the vector of it that has the maximum; -1: entry held_at
    sl.batches([&](const float (&x)[kBatch], int v, int b) {
        constexpr int kVecs = Slice<T>::kVecs;
        float mx[kVecs];  // of each vector
        float mb = -INFINITY;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            mx[i] = x[i * kN];
#pragma unroll
            for (int j = 1; j + 1 < kN; j += 2) mx[i] = fmax3(mx[i], x[i * kN + j], x[i * kN + j + 1]);
            mx[i] = fmaxf(mx[i], x[i * kN + kN - 1]);
            mb = fmaxf(mb, mx[i]);
        }
        const bool moved = mb > m;
        if (moved) {
            const float d = m == -INFINITY ? -1e30f : fmaxf(m - mb, -1e30f), e = exp_neg(d);
            const float w = rest + held;
            s = e * (s + d * w);
            rest = e * w;
            m = mb;
            held_batch = b;
            held_at = 0;
#pragma unroll
            for (int i = kVecs - 1; i > 0; --i) held_at = mx[i] == mb ? i : held_at;
            if (mx[0] == mb) held_at = 0;
        }
        const float ref = m == -INFINITY ? 0.f : m;
        const uint64_t nm2 = f2_pack(__float_as_uint(-ref), __float_as_uint(-ref));
        const uint32_t l2e = __float_as_uint(1.4426950408889634f);
        const uint64_t l2 = f2_pack(l2e, l2e);
        uint64_t z2[2] = {0ull, 0ull}, s2[2] = {0ull, 0ull};
#pragma unroll
        for (int j = 0; j < kBatch; j += 2) {
            uint32_t a, c, ea, ec;
            f2_unpack(f2_add(f2_pack(__float_as_uint(x[j]), __float_as_uint(x[j + 1])), nm2), a, c);
            a = __float_as_uint(max_nan(__uint_as_float(a), -1e30f));  // -inf: 0 times it is to be 0
            c = __float_as_uint(max_nan(__uint_as_float(c), -1e30f));
            const uint64_t d2 = f2_pack(a, c);
            f2_unpack(f2_mul(d2, l2), ea, ec);
            const uint64_t e2 = f2_pack(__float_as_uint(ex2_approx(__uint_as_float(ea))),
                                        __float_as_uint(ex2_approx(__uint_as_float(ec))));
            z2[(j / 2) & 1] = f2_add(z2[(j / 2) & 1], e2);
            s2[(j / 2) & 1] = f2_fma(e2, d2, s2[(j / 2) & 1]);
        }
        uint32_t a, c;
        f2_unpack(f2_add(z2[0], z2[1]), a, c);
        const float zb = __uint_as_float(a) + __uint_as_float(c);
        if (moved)
            held = zb;
        else
            rest += zb;
        f2_unpack(f2_add(s2[0], s2[1]), a, c);
        s += __uint_as_float(a) + __uint_as_float(c);
        if (by_order) {
#pragma unroll 1
            for (int j = 0; j < kBatch; ++j) {
                float y = x[0];
#pragma unroll
                for (int q = 1; q < kBatch; ++q) y = q == j ? x[q] : y;
                before += known && sl.has(v, j) && precedes(y, sl.index(v, j));
            }
        } else {
#pragma unroll
            for (int i = 0; i < Slice<T>::kVecs; ++i) {
                const int first = sl.index(v, i * kN);
                if (first <= token && token < first + kN) {
#pragma unroll
                    for (int j = 0; j < kN; ++j) before += x[i * kN + j] > (first + j < token ? below : mine);
                } else {
                    const float t = first < token ? below : mine;
#pragma unroll
                    for (int j = 0; j < kN; ++j) before += x[i * kN + j] > t;
                }
            }
        }
    });
    sl.singles([&](int i) {
        const float x = Vec<T>::one(sl.row + i);
        if (x > m) {
            const float d = m == -INFINITY ? -1e30f : fmaxf(m - x, -1e30f), e = exp_neg(d);
            const float w = rest + held;
            s = e * (s + d * w);
            rest = e * w;
            held = 1.f;
            m = x;
            held_batch = -1, held_at = i;
        } else {
            const float d = max_nan(x - (m == -INFINITY ? 0.f : m), -1e30f), e = exp_neg(d);
            rest += e;
            s += e * d;
        }
        before += known && precedes(x, i);
    });

    // the CTA's maximum
    float M = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (lane == 0) red_m[warp] = M;
    if (tid == 0) count = 0;
    u64 top_key = 0, sure_key = 0;  // bounds of the key of the thread's maximum: its index is somewhere in the vector
    if (K > 0) {
        if (m > -INFINITY) {
            const int first = held_batch < 0 ? held_at : sl.index(sl.first_vector(held_batch), held_at * kN);
            top_key = key_of(m, first);
            sure_key = key_of(m, held_batch < 0 ? first : first + kN - 1);
        } else if (sl.has(sl.first_vector(0), 0)) {  // nothing but -inf, or NaN
            const int first = sl.index(sl.first_vector(0), 0);
            const float least = rest == rest ? -INFINITY : rest;
            top_key = key_of(-INFINITY, first);
            sure_key = key_of(least, first + kN - 1);
        }
        u64 g = sure_key;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
            const u64 other = __shfl_xor_sync(0xffffffffu, g, o);
            g = other > g ? other : g;
        }
        if ((lane & 15) == 0) group[tid / 16] = g;
    }
    __syncthreads();
    M = red_m[0];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) M = fmaxf(M, red_m[i]);

    // sums against the CTA's maximum; those who hold it sum its batch again without it
    const bool holds = m == M && M > -INFINITY;
    float z = rest;
    if (holds) {
        if (held_batch >= 0) {
            const int v = sl.first_vector(held_batch);
            bool out = false;
#pragma unroll 1
            for (int i = 0; i < Slice<T>::kVecs; ++i) {
                if (v + i * kThreads >= sl.v1) break;
                float x[kN];
                Vec<T>::unpack(__ldg(sl.body + v + i * kThreads), x);
#pragma unroll
                for (int j = 0; j < kN; ++j) {
                    if (!out && x[j] == m)
                        out = true;
                    else
                        z += exp_neg(max_nan(x[j] - m, -1e30f));
                }
            }
        }
    } else if (m > -INFINITY) {
        const float d = max_nan(m - M, -1e30f), e = exp_neg(d), w = rest + held;
        s = e * (s + d * w);
        z = e * w;
    } else {
        z += held;  // nothing, or NaN
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

    if (K > 0) {
        // the K-th largest of the groups' maxima (0 where fewer groups have one: then everything is a candidate)
        u64 mine_g = group[lane], bound = 0;
        int above = 0;
        for (int i = 0; i < 32; ++i) above += group[i] > mine_g || (group[i] == mine_g && i < lane);
        const uint32_t who = __ballot_sync(0xffffffffu, above == K - 1);
        bound = __shfl_sync(0xffffffffu, mine_g, __ffs(who) - 1);
        auto offer = [&](u64 key) {
            if (key >= bound) {
                const int at = atomicAdd(&count, 1);
                if (at < kList) list[at] = key;
            }
        };
        if (bound == 0 || top_key >= bound) {
            sl.batches([&](const float (&x)[kBatch], int v, int) {
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
                    if (sl.has(v, j)) offer(key_of(x[j], sl.index(v, j)));
            });
            sl.singles([&](int i) { offer(key_of(Vec<T>::one(sl.row + i), i)); });
        }
        __syncthreads();
        int have = count;
        if (have > kList) {
            // too many reach the bound: the largest key below the last one found, K times
            u64 last = ~0ull;
            for (int k = 0; k < K; ++k) {
                u64 g = 0;
                sl.batches([&](const float (&x)[kBatch], int v, int) {
#pragma unroll
                    for (int j = 0; j < kBatch; ++j) {
                        const u64 key = sl.has(v, j) ? key_of(x[j], sl.index(v, j)) : 0;
                        if (key < last && key > g) g = key;
                    }
                });
                sl.singles([&](int i) {
                    const u64 key = key_of(Vec<T>::one(sl.row + i), i);
                    if (key < last && key > g) g = key;
                });
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const u64 other = __shfl_xor_sync(0xffffffffu, g, o);
                    g = other > g ? other : g;
                }
                __syncthreads();
                if (lane == 0) group[warp] = g;
                __syncthreads();
                last = 0;
                for (int i = 0; i < kWarps; ++i) last = group[i] > last ? group[i] : last;
                if (tid == 0) best[k] = last;
            }
        } else {
            if (tid < kMaxTop) best[tid] = 0;
            __syncthreads();
            for (int i = tid; i < have; i += kThreads) {
                const u64 key = list[i];
                int at = 0;
                for (int j = 0; j < have && at < K; ++j) at += list[j] > key;
                if (at < K) best[at] = key;
            }
        }
    }
    __syncthreads();
    if (tid == 0) {
        float zt = red_z[0], st = red_s[0];
        int ct = red_c[0], wt = red_w[0];
        for (int i = 1; i < kWarps; ++i) zt += red_z[i], st += red_s[i], ct += red_c[i], wt += red_w[i];
        out_m = M, out_s = st, out_c = ct;
        out_z = wt > 1 ? zt + (float)(wt - 1) : zt;  // of several that attain the maximum one is left out
    }
    State all;
    if (ranks > 1) {
        cluster_sync();
        if (rank != 0) {
            cluster_sync();
            return;
        }
    } else {
        __syncthreads();
    }
    all = {out_m, out_z, out_s};
    int ahead = out_c;
    for (int r = 1; r < ranks; ++r) {
        all = merge(all, {ld_cluster_f32(&out_m, r), ld_cluster_f32(&out_z, r), ld_cluster_f32(&out_s, r)});
        ahead += __float_as_int(ld_cluster_f32(reinterpret_cast<const float *>(&out_c), r));
    }
    const bool empty = all.m == -INFINITY && all.z == all.z;  // nothing has any weight
    if (all.m == INFINITY) all.z = __uint_as_float(0x7FFFFFFFu);
    const float log_z = log1pf(all.z);
    auto log_prob = [&](float x) { return empty ? -INFINITY : (x - all.m) - log_z; };
    if (tid == 0) {
        if (p.logprobs) p.logprobs[n] = known ? log_prob(mine) : -INFINITY;
        if (p.ranks) p.ranks[n] = known ? ahead : -1;
        if (p.entropy) p.entropy[n] = empty ? 0.f : log_z - all.s / (1.f + all.z);
    }
    if (K > 0) {
        const int lists = ranks * K;
        for (int i = tid; i < lists; i += kThreads) list[i] = ld_cluster_u64(&best[i % K], i / K);
        __syncthreads();
        for (int i = tid; i < lists; i += kThreads) {
            const u64 key = list[i];
            if (key == 0) continue;
            int at = 0;
            for (int j = 0; j < lists && at < K; ++j) at += list[j] > key;
            if (at < K) {
                p.top_tokens[n * K + at] = (int32_t)(0xFFFFFFFFu - (uint32_t)key);
                p.top_logprobs[n * K + at] = log_prob(value_of((uint32_t)(key >> 32)));
            }
        }
    }
    if (ranks > 1) cluster_sync();  // the others' lists are read
}

template <typename T>
cudaError_t launch_t(const LogprobParams &p, int64_t rows, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * p.cluster));
    cfg.blockDim = dim3(kThreads);
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
    // a cluster of CTAs a row while the rows are fewer than the CTAs that the GPU holds
    int cluster = 1;
    while (cluster < 8 && (int64_t)num_rows * cluster * 2 <= 2 * 152 && vocab / (cluster * 2) >= 4096) cluster *= 2;
    const va::LogprobParams p = {logits, stride, tokens, logprobs, entropy, top_logprobs, ranks, top_tokens,
                                 vocab, num_top, cluster};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = type == VA_FLOAT_FP32   ? va::launch_t<float>(p, num_rows, s)
                    : type == VA_FLOAT_BF16 ? va::launch_t<__nv_bfloat16>(p, num_rows, s)
                                            : va::launch_t<__half>(p, num_rows, s);
    if (e == cudaSuccess) return VA_OK;
    va::note_cuda_error(e);
    cudaGetLastError();
    return VA_ERR_CUDA;
}
