// Speculative acceptance from given probabilities and random numbers.
// Definition in verify_attn.h.
//
// Mathematics.  The decisions u q < p are products of two binary32 numbers,
// exact in binary64.  The emitted token inverts the cumulative distribution of
// the weights, an integer that must not depend on how the sum is split: so
// every p and q becomes a multiple of 2^-62 (an integer of 63 bits; what is
// cut off is below 2^-62 an entry, 2^-44 over a whole vocabulary), the
// residual max(0, p - q) is an exact integer subtraction and the sums are
// exact 128-bit integers.  The threshold u W is m W / 2^k for u = m 2^-k with
// m of 24 bits: exact in 128 bits too, and sum > u W holds for integers
// exactly where sum > floor(m W / 2^k).  The integers also keep the work off
// the FP64 pipe, which does two lanes a clock and SM here.
//
// One thread-block cluster per sequence.  Every CTA evaluates the (at most T)
// acceptance tests; each then sums its slice of the one row that decides, a
// contiguous run per warp, and the CTAs exchange their sums through
// distributed shared memory.  The one warp whose run holds the threshold reads
// it again (from L2) and finds the entry.  Bound: the bytes of one row of p
// (and one of q) per sequence for a large batch; for one sequence the chain of
// dependent reads (draft, its probabilities, the row) and two cluster barriers.
#include <cuda_fp16.h>

#include <algorithm>

#include "va_internal.h"
#include "va_sm100.cuh"

namespace va {
namespace {

using namespace sm100;
typedef unsigned __int128 u128;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;  // portable cluster size
constexpr int kMinPerCta = 8192;  // entries below which a row is not split further
constexpr int kSlots = 304;       // resident CTAs of this size: two on each of 152 SMs

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

// A binary32 probability as a multiple of 2^-62: NaN and negative numbers 0, above one 1.
__device__ __forceinline__ uint64_t fixed62(uint32_t bits) {
    const int e = (int)(bits >> 23);
    const uint64_t m = (bits & 0x7FFFFFu) | (e ? 0x800000u : 0u);  // value m 2^(e - 150)
    const int s = e - 88;
    uint64_t v = s >= 0 ? m << min(s, 39) : m >> min(-s, 31);
    if (bits > 0x3F800000u) v = bits <= 0x7F800000u ? (uint64_t)1 << 62 : 0;
    return v;
}

__device__ __forceinline__ uint64_t weight(uint32_t p_bits, uint32_t q_bits) {
    const uint64_t a = fixed62(p_bits), b = fixed62(q_bits);
    return a > b ? a - b : 0;
}

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
    const E *p, *q;
    int drop;
    bool vec;  // both rows start on a 16-byte boundary

    __device__ __forceinline__ uint64_t at(int i) const {
        const uint32_t pb = Prob<TYPE>::bits(p[i]);
        if (q) return weight(pb, Prob<TYPE>::bits(q[i]));
        return i == drop ? 0 : fixed62(pb);
    }
    // the weights of entries i .. i + kVec - 1 (i a multiple of kVec), those from `hi` on as 0
    __device__ __forceinline__ void load(int i, int hi, uint64_t (&w)[kVec]) const {
        if (vec && i + kVec <= hi) {
            const uint4 a = *reinterpret_cast<const uint4 *>(p + i);
            const E *pe = reinterpret_cast<const E *>(&a);
            if (q) {
                const uint4 b = *reinterpret_cast<const uint4 *>(q + i);
                const E *qe = reinterpret_cast<const E *>(&b);
#pragma unroll
                for (int k = 0; k < kVec; ++k) w[k] = weight(Prob<TYPE>::bits(pe[k]), Prob<TYPE>::bits(qe[k]));
            } else {
#pragma unroll
                for (int k = 0; k < kVec; ++k) w[k] = i + k == drop ? 0 : fixed62(Prob<TYPE>::bits(pe[k]));
            }
        } else {
#pragma unroll
            for (int k = 0; k < kVec; ++k) w[k] = i + k < hi ? at(i + k) : 0;
        }
    }
};

template <int TYPE>
__global__ void __launch_bounds__(kThreads) accept_probs_kernel(const ProbsParams a) {
    using E = typename Prob<TYPE>::T;
    constexpr int kVec = Prob<TYPE>::kVec;
    __shared__ int s_first;
    __shared__ u128 s_warp[kWarps];  // sums of the warps' runs, then the sums before them
    __shared__ uint64_t s_cta[2];    // this CTA's sum, read by the others
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = (int)cluster_rank(), ctas = (int)cluster_size();
    const int b = blockIdx.y;
    griddep_wait();
    const int count = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
    const E *p0 = static_cast<const E *>(a.p) + b * a.p_seq;
    const E *q0 = a.q ? static_cast<const E *>(a.q) + b * a.q_seq : nullptr;
    if (threadIdx.x == 0) s_first = count;
    __syncthreads();
    for (int t = threadIdx.x; t < count; t += kThreads) {
        const int d = a.drafts[(int64_t)b * a.T + t];
        bool ok = d >= 0 && d < a.V;
        if (ok) {
            const double p = (double)__uint_as_float(Prob<TYPE>::bits(p0[t * a.p_pos + d]));
            const double q = q0 ? (double)__uint_as_float(Prob<TYPE>::bits(q0[t * a.q_pos + d])) : 1.0;
            ok = (double)a.u_accept[(int64_t)b * a.T + t] * q < p;
        }
        if (!ok) atomicMin(&s_first, t);
    }
    __syncthreads();
    const int n = s_first;
    const int dn = n < count ? a.drafts[(int64_t)b * a.T + n] : -1;

    Row<TYPE> row;
    row.p = p0 + n * a.p_pos;
    row.q = n < count && q0 ? q0 + n * a.q_pos : nullptr;
    row.drop = n < count && !q0 ? dn : -1;
    const int per_warp = ((a.V + ctas * kWarps - 1) / (ctas * kWarps) + kVec - 1) / kVec * kVec;
    const int64_t start = (int64_t)(rank * kWarps + warp) * per_warp;
    const int lo = (int)min((int64_t)a.V, start), hi = (int)min((int64_t)a.V, start + per_warp);

    int token = -1;
    bool mine = false, empty = false;
    for (int pass = 0; pass < 2; ++pass) {  // the second only where the residual is zero everywhere
        row.vec = ((reinterpret_cast<uintptr_t>(row.p) | reinterpret_cast<uintptr_t>(row.q)) & 15) == 0;
        u128 sum = 0;
        for (int i = lo + lane * kVec; i < hi; i += 32 * kVec) {
            uint64_t w[kVec];
            row.load(i, hi, w);
#pragma unroll
            for (int k = 0; k < kVec; ++k) sum += w[k];
        }
        sum = warp_scan(sum, lane);
        if (lane == 31) s_warp[warp] = sum;
        __syncthreads();
        if (warp == 0) {
            const u128 v = s_warp[lane], inc = warp_scan(v, lane);
            s_warp[lane] = inc - v;
            if (lane == 31) {
                s_cta[0] = (uint64_t)inc;
                s_cta[1] = (uint64_t)(inc >> 64);
            }
        }
        cluster_sync();
        u128 before = 0, total = 0;
        for (int r = 0; r < ctas; ++r) {
            const u128 x = ((u128)ld_cluster_u64(&s_cta[1], r) << 64) | ld_cluster_u64(&s_cta[0], r);
            if (r < rank) before += x;
            total += x;
        }
        cluster_sync();  // s_cta may be rewritten, and the CTA may leave
        if (total != 0) {
            float u = a.u_emit[b];
            u = u > 0.f ? fminf(u, 0.999999940395355224609375f) : 0.f;  // 1 - 2^-24; NaN: 0
            const uint32_t bits = __float_as_uint(u);
            const int e = (int)(bits >> 23);
            const uint32_t m = (bits & 0x7FFFFFu) | (e ? 0x800000u : 0u);
            const int k = 150 - max(e, 1);  // u = m 2^-k, 24 <= k <= 149
            const u128 threshold = k < 128 ? ((u128)m * total) >> k : 0;
            before += s_warp[warp];
            const u128 own = shfl(sum, 31);
            mine = before <= threshold && threshold < before + own;
            if (mine) {
                for (int base = lo; base < hi; base += 32 * kVec) {
                    uint64_t w[kVec];
                    u128 s = 0;
                    const int i = base + lane * kVec;
                    if (i < hi) {
                        row.load(i, hi, w);
#pragma unroll
                        for (int j = 0; j < kVec; ++j) s += w[j];
                    }
                    const u128 inc = warp_scan(s, lane);
                    const unsigned past = __ballot_sync(0xffffffffu, before + inc > threshold);
                    if (past) {
                        const int who = __ffs(past) - 1;
                        if (lane == who) {
                            u128 c = before + inc - s;
#pragma unroll
                            for (int j = 0; j < kVec; ++j) {
                                c += w[j];
                                if (token < 0 && c > threshold) token = i + j;
                            }
                        }
                        token = __shfl_sync(0xffffffffu, token, who);
                        break;
                    }
                    before += shfl(inc, 31);
                }
            }
            break;
        }
        empty = !row.q && row.drop < 0;  // p itself is zero
        if (empty) break;
        row.q = nullptr;
        row.drop = -1;
    }
    int32_t *out = a.out + (int64_t)b * (a.T + 1);
    if (mine && lane == 0) out[n] = token;
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
    if (num_seqs < 1 || num_seqs > 65535 || T < 0 || T > 65535 || vocab < 1) return VA_ERR_INVALID_ARGUMENT;
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
