// Speculative acceptance from given probabilities and random numbers.
// Definition in verify_attn.h.
//
// Mathematics.  The decisions u q < p are products of two binary32 numbers,
// exact in binary64.  The emitted token inverts the cumulative distribution of
// the weights, a whole number that must not depend on how the sum is split: so
// every p and q is rounded to a multiple of 2^-54, the residual max(0, p - q)
// is an exact integer subtraction and the sums are exact 128-bit integers.  The
// threshold u W is m W / 2^k for u = m 2^-k with m of 24 bits: exact in 128
// bits too, and sum > u W holds for integers exactly where sum > floor(m W /
// 2^k).  Rounding each of 152k entries by 2^-55 moves a sum by some 1e-14.
//
// The integers are read off binary32 additions.  x + 1.5 2^-9 lies where
// binary32 counts in steps of 2^-32: its last bits are x in those steps,
// rounded, and what the rounding left, x - ((x + 1.5 2^-9) - 1.5 2^-9), is
// exact.  Once more in steps of 2^-54, and x is n2 2^-32 + n3 2^-54 with two
// small signed integers, which are summed as they are (the constants cancel in
// p - q).  That holds for x below 2^-10; the few larger ones first go through
// steps of 2^-10.  Two numbers an instruction (add.f32x2, fma.f32x2), four or
// seven of them a number.  64 sequences at a vocabulary of 151,936 (two rows
// where a model's draft is rejected): 34.8 us with significands shifted into
// 64-bit integers, which takes about four times the instructions; binary64
// does two lanes a clock and SM here.
//
// One thread-block cluster per sequence.  Every CTA evaluates the (at most T)
// acceptance tests; each then sums its slice of the one row that decides, a
// contiguous run per warp, and the CTAs exchange their sums through
// distributed shared memory.  The CTA whose slice holds the threshold reads the
// one run that holds it again (from L2), eight entries a thread, and finds the
// entry (one warp alone took 4 us longer at 2,374 entries a run).  Bound: for one
// sequence (7.2 us) the chain of dependent reads, draft, its probabilities, the
// row, the run, with the cluster's barrier between them.  For 64 (18.5 us, 61 MB
// from DRAM) the rows: by stamps in a copy of the kernel a CTA's sums take 8 us
// where one row is read, 12 where two are (medians, all CTAs at once); before
// them 2 us of drafts and their probabilities, behind them 2.5 us of barriers
// and, in the CTA that holds the threshold, 2 to 3 us of search.
#include <cuda_fp16.h>

#include <algorithm>

#include "va_internal.h"
#include "va_sm100.cuh"

namespace va {
namespace {

using namespace sm100;
typedef unsigned __int128 u128;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
static_assert(kWarps <= 32, "a warp scans one number per warp of the block");
// CTAs of a sequence: the most, up to the portable cluster size, that keep all sequences' CTAs resident together (two of this
// size on each of 152 SMs) and kMinPerCta entries in each.  Measured with a model's drafts, fp32, the rule's choice first:
// 64 sequences of 152,064 entries 4 CTAs 20.8 us, 2 23.8, 8 (two waves) 26.2; one of them 8 CTAs 8.5 us, 4 10.9, 1 27.2; one
// of 8,000 entries 2 CTAs 6.6 us, 1 7.3, 4 6.2, 8 6.1; 64 of 8,000 2 CTAs 6.9 us, 1 7.4, 4 8.5.  It is not the best count
// everywhere: 64 of 16,000 get 4 CTAs (8.9 us) where 2 take 7.5, 16 of 32,000 get 8 (7.8 us) where 4 take 7.2.
constexpr int kMaxCluster = 8;
constexpr int kMinPerCta = 2048;
constexpr int kSlots = 304;

struct ProbsParams {
    const void *p, *q;  // q null: point mass
    int64_t p_seq, p_pos, q_seq, q_pos;  // elements
    const int32_t *drafts, *lens;
    const float *u_accept, *u_emit;
    int32_t *out, *nacc;
    int T, V;
};

template <int TYPE>
struct Prob;
template <>
struct Prob<VA_FLOAT_FP32> {
    using T = uint32_t;
    static constexpr int kVec = 4;
    static __device__ __forceinline__ uint32_t bits(uint32_t x) { return x; }
};
template <>
struct Prob<VA_FLOAT_BF16> {
    using T = uint16_t;
    static constexpr int kVec = 8;
    static __device__ __forceinline__ uint32_t bits(uint16_t x) { return (uint32_t)x << 16; }
};
template <>
struct Prob<VA_FLOAT_FP16> {
    using T = uint16_t;
    static constexpr int kVec = 8;
    static __device__ __forceinline__ uint32_t bits(uint16_t x) {
        return __float_as_uint(__half2float(__ushort_as_half(x)));
    }
};

// NaN and negative numbers count as 0, numbers above one as 1.
__device__ __forceinline__ uint32_t sane(uint32_t bits) {
    return bits <= 0x3F800000u ? bits : bits <= 0x7F800000u ? 0x3F800000u : 0u;
}

__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) { return ((uint64_t)hi << 32) | lo; }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
constexpr uint32_t kSign = 0x80000000u;
constexpr uint32_t kStep1 = 0x46400000u;  // 1.5 * 2^13: steps of 2^-10
constexpr uint32_t kStep2 = 0x3B400000u;  // 1.5 * 2^-9: steps of 2^-32
constexpr uint32_t kStep3 = 0x30400000u;  // 1.5 * 2^-31: steps of 2^-54
constexpr uint32_t kOne = 0x3F800000u;
constexpr uint32_t kSmall = 0x3A800000u;  // 2^-10: numbers below need no first step

// Two numbers in [0, 1] (binary32 bits) in the three steps, each plus the bits of its constant; FIRST = false where both are
// below 2^-10.
template <bool FIRST>
struct Steps {
    uint64_t n1, n2, n3;
    static __device__ __forceinline__ uint64_t left(uint64_t x, uint64_t n, uint32_t step) {  // x - (n - step), exact
        return fma2(add2(n, pack2(step | kSign, step | kSign)), pack2(kOne | kSign, kOne | kSign), x);
    }
    __device__ __forceinline__ explicit Steps(uint64_t x) {
        n1 = 0;
        if (FIRST) {
            n1 = add2(x, pack2(kStep1, kStep1));
            x = left(x, n1, kStep1);
        }
        n2 = add2(x, pack2(kStep2, kStep2));
        n3 = add2(left(x, n2, kStep2), pack2(kStep3, kStep3));
    }
};

// A sum of weights in the three steps.  One weight adds at most 2^10, 2^22 and 2^22 to them (the first step leaves at most
// 2^-11, the second 2^-33; without the first, numbers below 2^-10), so they hold kHeld weights before they have to go into
// wider integers.
constexpr int kHeld = 256;
struct Sum {
    int n1 = 0, n2 = 0, n3 = 0;
    template <bool FIRST, bool MODEL>
    __device__ __forceinline__ void add(const Steps<FIRST> &p, const Steps<FIRST> &q) {  // both halves of p - q, or of p
        if (FIRST) n1 += both<MODEL>(p.n1, q.n1, kStep1);
        n2 += both<MODEL>(p.n2, q.n2, kStep2);
        n3 += both<MODEL>(p.n3, q.n3, kStep3);
    }
    template <bool MODEL>
    static __device__ __forceinline__ int both(uint64_t p, uint64_t q, uint32_t step) {
        const int lo = (int)(uint32_t)p - (MODEL ? (int)(uint32_t)q : (int)step);
        return lo + (int)(uint32_t)(p >> 32) - (MODEL ? (int)(uint32_t)(q >> 32) : (int)step);
    }
    // in units of 2^-54: not negative, below 2^63
    __device__ __forceinline__ uint64_t value() const {
        return (uint64_t)(((int64_t)n1 << 44) + ((int64_t)n2 << 22) + n3);
    }
};

__device__ __forceinline__ u128 shfl_up(u128 v, int d) {
    const uint64_t lo = __shfl_up_sync(0xffffffffu, (uint64_t)v, d);
    const uint64_t hi = __shfl_up_sync(0xffffffffu, (uint64_t)(v >> 64), d);
    return ((u128)hi << 64) | lo;
}
__device__ __forceinline__ u128 shfl(u128 v, int from) {
    const uint64_t lo = __shfl_sync(0xffffffffu, (uint64_t)v, from);
    const uint64_t hi = __shfl_sync(0xffffffffu, (uint64_t)(v >> 64), from);
    return ((u128)hi << 64) | lo;
}
// inclusive sums over the lanes
__device__ __forceinline__ u128 warp_scan(u128 v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u128 x = shfl_up(v, o);
        if (lane >= o) v += x;
    }
    return v;
}

// The weights of one row: p alone, p without the point mass at `drop`, or max(0, p - q).
template <int TYPE>
struct Row {
    using E = typename Prob<TYPE>::T;
    static constexpr int kVec = Prob<TYPE>::kVec;
    union Vec {
        uint4 raw;
        E e[kVec];
    };
    const E *p, *q;
    int drop;
    bool vec;  // both rows start on a 16-byte boundary

    // entries i .. i + kVec - 1 (i a multiple of kVec) of a row that starts anywhere, or that ends among them (as 0)
    static __device__ __forceinline__ uint4 load_slowly(const E *row, int i, int hi) {
        Vec v;
        v.raw = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < kVec; ++k)
            if (i + k < hi) v.e[k] = row[i + k];
        return v.raw;
    }
    __device__ __forceinline__ uint4 load(const E *row, int i, int hi) const {
        if (i >= hi || !row) return make_uint4(0, 0, 0, 0);
        if (vec && i + kVec <= hi) return *reinterpret_cast<const uint4 *>(row + i);
        return load_slowly(row, i, hi);
    }
    template <bool MODEL>
    __device__ __forceinline__ void add(Sum &s, const uint4 &praw, const uint4 &qraw, int i) const {
        Vec pv, qv;
        pv.raw = praw;
        qv.raw = qraw;
        uint32_t a[kVec], b[kVec], most = 0;
#pragma unroll
        for (int k = 0; k < kVec; ++k) {
            a[k] = Prob<TYPE>::bits(pv.e[k]);
            b[k] = MODEL ? Prob<TYPE>::bits(qv.e[k]) : 0;
            most = max(most, max(a[k], b[k]));
        }
        if (!MODEL && (unsigned)(drop - i) < kVec) {
#pragma unroll
            for (int k = 0; k < kVec; ++k) a[k] = i + k == drop ? 0 : a[k];
        }
        if (most < kSmall) {
            add_steps<false, MODEL>(s, a, b);
        } else {
            if (most > kOne) {  // not probabilities: rare
#pragma unroll
                for (int k = 0; k < kVec; ++k) {
                    a[k] = sane(a[k]);
                    b[k] = sane(b[k]);
                }
            }
            add_steps<true, MODEL>(s, a, b);
        }
    }
    template <bool FIRST, bool MODEL>
    static __device__ __forceinline__ void add_steps(Sum &s, const uint32_t (&a)[kVec], const uint32_t (&b)[kVec]) {
#pragma unroll
        for (int k = 0; k < kVec; k += 2) {  // bits order as the numbers do: the smaller of the two as q leaves 0 where q >= p
            const Steps<FIRST> p2(pack2(a[k], a[k + 1]));
            if (MODEL) s.add<FIRST, true>(p2, Steps<FIRST>(pack2(min(a[k], b[k]), min(a[k + 1], b[k + 1]))));
            else s.add<FIRST, false>(p2, p2);
        }
    }
    __device__ __forceinline__ uint64_t one(int i) const {  // the weight of one entry
        const uint32_t a = sane(Prob<TYPE>::bits(p[i])), b = i == drop ? a : q ? sane(Prob<TYPE>::bits(q[i])) : 0;
        Sum s;
        s.add<true, true>(Steps<true>(a), Steps<true>(min(a, b)));
        return s.value();
    }

    // this lane's share of the sum over [lo, hi)
    template <bool MODEL>
    __device__ __forceinline__ u128 sum(int lo, int hi, int lane) const {
        constexpr int U = (MODEL ? 16 : 32) / kVec;  // 64 bytes (fp32) of each row in flight, 128 of one row
        u128 total = 0;
        int base = lo + lane * kVec;
        while (base < hi) {
            Sum s;
            for (int r = 0; r < kHeld / (kVec * U) && base < hi; ++r, base += 32 * kVec * U) {
                uint4 pv[U], qv[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    pv[u] = load(p, base + u * 32 * kVec, hi);
                    if (MODEL) qv[u] = load(q, base + u * 32 * kVec, hi);
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (base + u * 32 * kVec < hi) add<MODEL>(s, pv[u], MODEL ? qv[u] : pv[u], base + u * 32 * kVec);
            }
            total += s.value();
        }
        return total;
    }

    // The first entry of [lo, hi) where `before` plus the sum from lo passes the threshold, found by the whole CTA, kEach
    // neighbouring entries a thread.  One warp finds it (token >= 0 in all its lanes), the others get -1.
    __device__ __forceinline__ int pass(int lo, int hi, u128 before, u128 threshold, u128 *s_sums) const {
        constexpr int kEach = 8;
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        int token = -1;
        for (int base = lo; base < hi && before <= threshold; base += kThreads * kEach) {
            const int i = base + threadIdx.x * kEach;
            Sum s;
            uint4 pv[kEach / kVec], qv[kEach / kVec];
#pragma unroll
            for (int u = 0; u < kEach / kVec; ++u) {
                pv[u] = load(p, i + u * kVec, hi);
                qv[u] = load(q, i + u * kVec, hi);
            }
#pragma unroll
            for (int u = 0; u < kEach / kVec; ++u) {
                if (q) add<true>(s, pv[u], qv[u], i + u * kVec);
                else add<false>(s, pv[u], pv[u], i + u * kVec);
            }
            const u128 own = s.value(), inc = warp_scan(own, lane);
            __syncthreads();  // s_sums may still be read
            if (lane == 31) s_sums[warp] = inc;
            __syncthreads();
            const u128 sums = warp_scan(lane < kWarps ? s_sums[lane] : 0, lane);
            const u128 chunk = shfl(sums, 31), earlier = shfl(sums, max(warp - 1, 0));
            const u128 start = before + inc - own + (warp ? earlier : 0);
            before += chunk;
            const unsigned mine = __ballot_sync(0xffffffffu, start <= threshold && threshold < start + own);
            if (mine) {  // this warp: the lane's entries one to a lane
                const int who = __ffs(mine) - 1, first = base + (warp * 32 + who) * kEach;
                const u128 each = warp_scan(lane < kEach && first + lane < hi ? one(first + lane) : 0, lane);
                token = first + __ffs(__ballot_sync(0xffffffffu, shfl(start, who) + each > threshold)) - 1;
            }
        }
        return token;
    }
};

template <int TYPE>
__global__ void __launch_bounds__(kThreads, 2) accept_probs_kernel(const ProbsParams a) {
    using E = typename Prob<TYPE>::T;
    constexpr int kVec = Prob<TYPE>::kVec;
    __shared__ int s_first;
    __shared__ u128 s_warp[kWarps];  // sums of the warps' runs, then the sums before them
    __shared__ u128 s_sums[kWarps];
    __shared__ uint64_t s_ctas[2][kMaxCluster][2];  // the CTAs' sums in each pass, written by them
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = (int)cluster_rank(), ctas = (int)cluster_size();
    const int b = blockIdx.y;
    if (threadIdx.x == 0) s_first = 0x7FFFFFFF;
    __syncthreads();
    cluster_arrive();  // this CTA runs: its shared memory may be written
    griddep_wait();
    const int count = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
    const E *p0 = static_cast<const E *>(a.p) + b * a.p_seq;
    const E *q0 = a.q ? static_cast<const E *>(a.q) + b * a.q_seq : nullptr;
    const float u_emit = a.u_emit[b];
    int32_t *out = a.out + (int64_t)b * (a.T + 1);
    for (int t = threadIdx.x; t < count; t += kThreads) {
        const int d = a.drafts[(int64_t)b * a.T + t];
        const double u = (double)a.u_accept[(int64_t)b * a.T + t];
        bool ok = d >= 0 && d < a.V;
        if (ok) {
            const double p = (double)__uint_as_float(Prob<TYPE>::bits(p0[t * a.p_pos + d]));
            const double q = q0 ? (double)__uint_as_float(Prob<TYPE>::bits(q0[t * a.q_pos + d])) : 1.0;
            ok = u * q < p;
        }
        if (!ok) atomicMin(&s_first, t);
    }
    __syncthreads();
    const int n = min(s_first, count);
    const bool rejected = n < count;

    Row<TYPE> row;
    row.p = p0 + n * a.p_pos;
    row.q = rejected && q0 ? q0 + n * a.q_pos : nullptr;
    row.drop = rejected && !q0 ? a.drafts[(int64_t)b * a.T + n] : -1;
    const int per_warp = ((a.V + ctas * kWarps - 1) / (ctas * kWarps) + kVec - 1) / kVec * kVec;
    const int64_t start = (int64_t)(rank * kWarps + warp) * per_warp;
    const int lo = (int)min((int64_t)a.V, start), hi = (int)min((int64_t)a.V, start + per_warp);

    bool empty = false;
    for (int pass = 0; pass < 2; ++pass) {  // the second only where the residual is zero everywhere
        row.vec = ((reinterpret_cast<uintptr_t>(row.p) | reinterpret_cast<uintptr_t>(row.q)) & 15) == 0;
        const u128 sum = warp_scan(row.q ? row.template sum<true>(lo, hi, lane) : row.template sum<false>(lo, hi, lane), lane);
        if (lane == 31) s_warp[warp] = sum;
        __syncthreads();
        if (pass == 0) cluster_wait();
        if (warp == 0) {
            const u128 v = lane < kWarps ? s_warp[lane] : 0, inc = warp_scan(v, lane);
            if (lane < kWarps) s_warp[lane] = inc - v;
            const u128 own = shfl(inc, 31);
            if (lane < ctas) {
                st_cluster_u64(&s_ctas[pass][rank][0], lane, (uint64_t)own);
                st_cluster_u64(&s_ctas[pass][rank][1], lane, (uint64_t)(own >> 64));
            }
        }
        cluster_sync();  // all sums are here; nothing is written to another CTA after the last one
        const u128 cta = lane < ctas ? ((u128)s_ctas[pass][lane][1] << 64) | s_ctas[pass][lane][0] : 0;
        const u128 upto = warp_scan(cta, lane), own = shfl(cta, rank), total = shfl(upto, 31);
        u128 before = shfl(upto, rank) - own;
        if (total != 0) {
            const float u = u_emit > 0.f ? fminf(u_emit, 0.999999940395355224609375f) : 0.f;  // 1 - 2^-24; NaN: 0
            const uint32_t bits = __float_as_uint(u);
            const int e = (int)(bits >> 23);
            const uint32_t m = (bits & 0x7FFFFFu) | (e ? 0x800000u : 0u);
            const int k = 150 - max(e, 1);  // u = m 2^-k, 24 <= k <= 149
            const u128 threshold = k < 128 ? ((u128)m * total) >> k : 0;
            if (before <= threshold && threshold < before + own) {  // in this CTA's slice: in whose run?
                const int w = 31 - __clz(__ballot_sync(0xffffffffu, lane < kWarps && before + s_warp[lane % kWarps] <= threshold));
                before += s_warp[w];
                const int64_t from = (int64_t)(rank * kWarps + w) * per_warp;
                const int run_lo = (int)min((int64_t)a.V, from), run_hi = (int)min((int64_t)a.V, from + per_warp);
                const int token = row.pass(run_lo, run_hi, before, threshold, s_sums);
                if (token >= 0 && lane == 0) out[n] = token;
            }
            break;
        }
        empty = !row.q && row.drop < 0;  // p itself is zero
        if (empty) break;
        row.q = nullptr;
        row.drop = -1;
    }
    if (rank == 0) {
        for (int t = threadIdx.x; t <= a.T; t += kThreads)
            if (t != n || empty) out[t] = t < n ? a.drafts[(int64_t)b * a.T + t] : -1;
        if (threadIdx.x == 0) a.nacc[b] = n;
    }
}

template <int TYPE>
cudaError_t launch(const ProbsParams &p, int num_seqs, int cluster, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cluster, num_seqs);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, accept_probs_kernel<TYPE>, p);
}

}  // namespace
}  // namespace va

extern "C" int verify_attn_accept_probs(const va_rows *target_probs, const va_rows *draft_probs, va_float_type type,
                                        const int32_t *draft_tokens, const int32_t *draft_lens,
                                        const float *u_accept, const float *u_emit, int num_seqs, int T, int vocab,
                                        int32_t *out_tokens, int32_t *num_accepted, void *stream) {
    if (!target_probs || !target_probs->data || !u_emit || !out_tokens || !num_accepted) return VA_ERR_INVALID_ARGUMENT;
    if (num_seqs < 1 || num_seqs > 65535 || T < 0 || T > 65535 || vocab < 1 || vocab > (1 << 30))
        return VA_ERR_INVALID_ARGUMENT;
    if (T > 0 && (!draft_tokens || !u_accept)) return VA_ERR_INVALID_ARGUMENT;
    if (type != VA_FLOAT_BF16 && type != VA_FLOAT_FP16 && type != VA_FLOAT_FP32) return VA_ERR_UNSUPPORTED;
    const bool model = draft_probs && draft_probs->data && T > 0;
    const uintptr_t size = type == VA_FLOAT_FP32 ? 4 : 2;
    auto misaligned = [](const void *ptr, uintptr_t a) { return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) != 0; };
    if (misaligned(target_probs->data, size) || (model && misaligned(draft_probs->data, size)) ||
        misaligned(draft_tokens, 4) || misaligned(draft_lens, 4) || misaligned(u_accept, 4) || misaligned(u_emit, 4) ||
        misaligned(out_tokens, 4) || misaligned(num_accepted, 4))
        return VA_ERR_INVALID_ARGUMENT;
    if (target_probs->stride_seq < 0 || target_probs->stride_pos < 0 ||
        (model && (draft_probs->stride_seq < 0 || draft_probs->stride_pos < 0)))
        return VA_ERR_INVALID_ARGUMENT;
    va::ProbsParams p{};
    p.p = target_probs->data;
    p.p_seq = target_probs->stride_seq;
    p.p_pos = target_probs->stride_pos;
    if (model) {
        p.q = draft_probs->data;
        p.q_seq = draft_probs->stride_seq;
        p.q_pos = draft_probs->stride_pos;
    }
    p.drafts = draft_tokens;
    p.lens = draft_lens;
    p.u_accept = u_accept;
    p.u_emit = u_emit;
    p.out = out_tokens;
    p.nacc = num_accepted;
    p.T = T;
    p.V = vocab;
    int cluster = va::kMaxCluster;
    while (cluster > 1 && (num_seqs * cluster > va::kSlots || vocab < cluster * va::kMinPerCta)) cluster /= 2;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = type == VA_FLOAT_BF16   ? va::launch<VA_FLOAT_BF16>(p, num_seqs, cluster, s)
                          : type == VA_FLOAT_FP16 ? va::launch<VA_FLOAT_FP16>(p, num_seqs, cluster, s)
                                                  : va::launch<VA_FLOAT_FP32>(p, num_seqs, cluster, s);
    if (e != cudaSuccess) {
        va::note_cuda_error(e);
        return VA_ERR_CUDA;
    }
    return VA_OK;
}
