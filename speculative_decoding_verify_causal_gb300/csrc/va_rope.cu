// Rotary positions with several axes: q and k of a batch rotated in one
// launch (rope_kernel), or rotated and appended to the paged cache in one
// launch (rope_append_kernel).  Definitions in verify_attn.h.
//
// Angles.  A binary32 product position * frequency loses the angle: at
// position 200,000 its last bit is 1/64 of a radian.  turn[i] holds the part
// of a turn that one step makes as a 64-bit fraction, so position * turn[i]
// modulo 2^64 (one integer multiplication, negative positions included) is
// the angle's part of a turn to 2^-65 times the position, at most 2^-34.  Its top 32 bits
// give the nearest quarter turn and a signed remainder of at most 1/8 turn,
// which binary32 holds to 24 bits; sincospif of the remainder is then within
// a few ulps, and the quarter turn swaps and negates.
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include <algorithm>

#include "va_internal.h"

namespace va {
namespace {

// (cos, sin) of position pos * turn / 2^64 of a full turn, times scale
__device__ __forceinline__ float2 turned(uint64_t turn, int pos, float scale) {
    const uint64_t phase = turn * (uint64_t)(int64_t)pos;
    const uint32_t hi = (uint32_t)((phase + 0x80000000ull) >> 32);
    const uint32_t quarter = (hi + 0x20000000u) >> 30;
    const int rest = (int)(hi - (quarter << 30));  // in units of 2^-32 turn = 2^-31 pi
    float s, c;
    sincospif((float)rest * 4.656612873077392578125e-10f, &s, &c);  // 2^-31
    c *= scale;
    s *= scale;
    float2 r = (quarter & 1u) ? make_float2(-s, c) : make_float2(c, s);
    if (quarter & 2u) r = make_float2(-r.x, -r.y);
    return r;
}

// (cos, sin) of the N neighbouring pairs from `first` on (a multiple of N) for a token at the positions `at`.  The description
// is in the launch's arguments (16-byte aligned there), where reads that differ from lane to lane go one after the other: they
// are made as wide as they can be (16 tokens of 24 + 8 heads of 256, a quarter turned: 3.6 -> 2.9 us).
template <int N>
__device__ __forceinline__ void angles(const va_rope &r, int first, const int (&at)[VA_ROPE_MAX_AXES], float2 *cs) {
    uint64_t axes;
    if constexpr (N == 8) axes = *reinterpret_cast<const uint64_t *>(r.axis + first);
    else if constexpr (N == 4) axes = *reinterpret_cast<const uint32_t *>(r.axis + first);
    else if constexpr (N == 2) axes = *reinterpret_cast<const uint16_t *>(r.axis + first);
    else axes = r.axis[first];
    uint64_t turns[N];
    if constexpr (N == 1) {
        turns[0] = r.turn[first];
    } else {
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            const ulonglong2 two = *reinterpret_cast<const ulonglong2 *>(r.turn + first + j);
            turns[j] = two.x;
            turns[j + 1] = two.y;
        }
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int axis = (int)(axes >> (8 * j)) & 255;
        cs[j] = turned(turns[j], axis < 2 ? (axis ? at[1] : at[0]) : (axis == 2 ? at[2] : at[3]), r.scale);
    }
}

// The positions of one token.
__device__ __forceinline__ void positions(const va_rope &r, const int32_t *pos, int64_t stride, int (&at)[VA_ROPE_MAX_AXES]) {
#pragma unroll
    for (int a = 0; a < VA_ROPE_MAX_AXES; ++a) at[a] = a < r.num_axes ? pos[a * stride] : 0;
}

// n / d and n % d for 0 <= n < 2^31 with a multiplication (d >= 1)
struct FastDiv {
    uint32_t d, mul, shift;
};
FastDiv fast_div(uint32_t d) {
    FastDiv f{d, 0, 0};
    while (f.shift < 31 && (1u << f.shift) < d) ++f.shift;
    f.mul = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << f.shift) - d)) / d + 1);
    return f;
}
__device__ __forceinline__ uint32_t div(uint32_t n, const FastDiv &f) { return (__umulhi(n, f.mul) + n) >> f.shift; }

// ------------------------------------------------------------------------- rotary alone

constexpr int kThreads = 128;
constexpr int kInFlight = 64;   // bytes that a thread has in flight while it turns as many
// Heads of a thread: kHeadBytes of them where there is work enough (8 heads of a 16-byte vector, 32 of a 4-byte one, whose
// angles cost as much a pair: 46 us instead of 56 with 8 heads of 4-byte vectors, 16,384 tokens of 40 heads of 72), fewer
// while the grid is below kMinCtas, two CTAs for each of 152 SMs.
// Fewer heads share a thread's angles: with 912 and 2,432 CTAs wanted, 1,024 tokens of 40 heads of 128 took 6.4 and 8.1 us
// instead of 5.5, 256 tokens 4.7 instead of 3.3.  With 16 heads a thread the grid of an image tower's 4,110 tokens is 1.06 waves
// (16.5 us, with 8 heads 15.0); at 32,768 tokens 8 to 40 heads are within 1.5 %.
constexpr int kHeadBytes = 128;
constexpr int kMinCtas = 304;

struct Tensor {
    const char *in;
    char *out;
    int64_t in_seq, in_token, in_head, out_seq, out_token, out_head;  // bytes
};

struct alignas(16) RopeParams {
    va_rope rope;
    const int32_t *pos;
    int64_t pos_axis, pos_seq, pos_token;
    Tensor q, k;
    int q_heads, heads;      // heads of q, of q and k together
    int tokens;              // num_seqs * T
    int head_dim;
    int head_chunk;          // heads per thread
    int units;               // of a head: those of the pairs, then the unrotated vectors
    int pair_units;
    float inverse_sign;      // -1 for the inverse
    FastDiv by_T, by_units;
};

template <int BYTES>
struct Raw;
template <>
struct Raw<16> {
    using V = uint4;
};
template <>
struct Raw<8> {
    using V = uint2;
};
template <>
struct Raw<4> {
    using V = uint32_t;
};
template <>
struct Raw<2> {
    using V = uint16_t;
};

template <int TYPE>
struct Elem {
    static constexpr int kBytes = TYPE == VA_FLOAT_FP32 ? 4 : 2;
};

// W elements of a 16- or 32-bit type <-> fp32
template <int TYPE, int W, typename V>
__device__ __forceinline__ void unpack(const V &raw, float (&x)[W]) {
    if constexpr (TYPE == VA_FLOAT_FP32) {
        const float *f = reinterpret_cast<const float *>(&raw);
#pragma unroll
        for (int e = 0; e < W; ++e) x[e] = f[e];
    } else {
        const uint16_t *h = reinterpret_cast<const uint16_t *>(&raw);
#pragma unroll
        for (int e = 0; e < W; ++e)
            x[e] = TYPE == VA_FLOAT_BF16 ? __uint_as_float((uint32_t)h[e] << 16) : __half2float(__ushort_as_half(h[e]));
    }
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int TYPE, int W, typename V>
__device__ __forceinline__ V packed(const float (&x)[W]) {
    V raw;
    if constexpr (TYPE == VA_FLOAT_FP32) {
        float *f = reinterpret_cast<float *>(&raw);
#pragma unroll
        for (int e = 0; e < W; ++e) f[e] = x[e];
    } else if constexpr (W == 1) {
        raw = TYPE == VA_FLOAT_BF16 ? (V)(pack_bf16x2(x[0], 0.f) & 0xFFFFu) : (V)__half_as_ushort(__float2half_rn(x[0]));
    } else {
        uint32_t *h = reinterpret_cast<uint32_t *>(&raw);
#pragma unroll
        for (int e = 0; e < W; e += 2) {
            if constexpr (TYPE == VA_FLOAT_BF16) {
                h[e / 2] = pack_bf16x2(x[e], x[e + 1]);
            } else {
                const __half2 p = __floats2half2_rn(x[e], x[e + 1]);
                h[e / 2] = *reinterpret_cast<const uint32_t *>(&p);
            }
        }
    }
    return raw;
}

// A unit is a piece of one head whose pairs are whole: a vector of W elements of each half, or one vector of neighbours (two
// single elements where W is 1), or, past the pairs, as many vectors that are copied.  A thread has one unit of one token: it
// makes its (cos, sin) once, in registers, and turns that unit of head_chunk heads with them.  No shared memory and no barrier: a
// first form that made a token's (cos, sin) in shared memory for all its heads issued twice the instructions and waited on
// the table's bank conflicts (32,768 tokens, 40 heads of 128, bf16: 123.5 us; this one 104.2 us, 6.4 TB/s).
template <int TYPE, int W, bool ADJACENT>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
    using V = typename Raw<W * Elem<TYPE>::kBytes>::V;
    constexpr int kElem = Elem<TYPE>::kBytes;
    constexpr bool kOne = ADJACENT && W > 1;  // one vector holds the pairs; a unit is one vector, else two
    constexpr int kPairs = kOne ? W / 2 : W;
    const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
    const uint32_t n = div(i, p.by_units), unit = i - n * p.units;
    if (n >= (uint32_t)p.tokens) return;
    const int P = p.rope.num_pairs;
    const int b = (int)div(n, p.by_T), t = (int)n - b * (int)p.by_T.d;
    const bool pairs = (int)unit < p.pair_units;
    const int pair0 = kPairs * (int)unit;
    const int elem = pairs ? (ADJACENT ? 2 * pair0 : pair0) : 2 * P + (kOne ? W : 2 * W) * ((int)unit - p.pair_units);
    const int64_t off0 = (int64_t)elem * kElem, off1 = off0 + (pairs && !ADJACENT ? P : W) * kElem;
    const bool two = !kOne && (pairs || elem + W < p.head_dim);
    const int h0 = blockIdx.y * p.head_chunk, h1 = min(p.heads, h0 + p.head_chunk);
    griddep_wait();
    // heads h0 .. h1 - 1 of q and k, kAhead at a time: kInFlight bytes of each unit's vectors, eight heads at most
    constexpr int kBytes = (kOne ? 1 : 2) * W * kElem, kAhead = kInFlight / kBytes < 8 ? kInFlight / kBytes : 8;
    V lo[kAhead], hi[kAhead];
    char *to[kAhead];
    auto load = [&](int h) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u, ++h) {
            if (h >= h1) continue;
            const bool is_k = h >= p.q_heads;
            const Tensor &x = is_k ? p.k : p.q;
            const int g = is_k ? h - p.q_heads : h;
            const char *in = x.in + b * x.in_seq + t * x.in_token + g * x.in_head;
            to[u] = x.out + b * x.out_seq + t * x.out_token + g * x.out_head;
            lo[u] = *reinterpret_cast<const V *>(in + off0);
            if (two) hi[u] = *reinterpret_cast<const V *>(in + off1);
        }
    };
    load(h0);  // under way while the angles are computed
    float2 cs[kPairs];
    if (pairs) {
        int at[VA_ROPE_MAX_AXES];
        positions(p.rope, p.pos + b * p.pos_seq + t * p.pos_token, p.pos_axis, at);
        angles<kPairs>(p.rope, pair0, at, cs);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) cs[j].y *= p.inverse_sign;
    }
    for (int h = h0; h < h1; h += kAhead) {
        V x[kAhead], y[kAhead];
        char *out[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            x[u] = lo[u];
            y[u] = hi[u];
            out[u] = to[u];
        }
        load(h + kAhead);  // under way while these are turned
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (h + u >= h1) continue;
            if (pairs) {
                float x0[W], x1[W];
                unpack<TYPE, W>(x[u], x0);
                if (!kOne) unpack<TYPE, W>(y[u], x1);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
                    float &first = x0[kOne ? 2 * j : j], &second = kOne ? x0[(2 * j + 1) % W] : x1[j];
                    const float na = fmaf(first, cs[j].x, -second * cs[j].y), nb = fmaf(second, cs[j].x, first * cs[j].y);
                    first = na;
                    second = nb;
                }
                x[u] = packed<TYPE, W, V>(x0);
                if (!kOne) y[u] = packed<TYPE, W, V>(x1);
            }
            *reinterpret_cast<V *>(out[u] + off0) = x[u];
            if (two) *reinterpret_cast<V *>(out[u] + off1) = y[u];
        }
    }
}

template <int TYPE, int W>
cudaError_t launch_rope_w(const RopeParams &p, dim3 grid, cudaStream_t s) {
    return p.rope.adjacent ? launch_pdl(rope_kernel<TYPE, W, true>, grid, dim3(kThreads), 0, s, p)
                           : launch_pdl(rope_kernel<TYPE, W, false>, grid, dim3(kThreads), 0, s, p);
}

template <int TYPE>
cudaError_t launch_rope(const RopeParams &p, int w, dim3 grid, cudaStream_t s) {
    constexpr int kWide = 16 / Elem<TYPE>::kBytes;
    return w == kWide ? launch_rope_w<TYPE, kWide>(p, grid, s)
           : w == 4   ? launch_rope_w<TYPE, 4>(p, grid, s)
           : w == 2   ? launch_rope_w<TYPE, 2>(p, grid, s)
                      : launch_rope_w<TYPE, 1>(p, grid, s);
}

// ------------------------------------------------------------------------- rotary and append

struct alignas(16) RopeAppendParams {
    va_rope rope;
    const int32_t *pos;  // null: the token's place in its sequence
    int64_t pos_axis, pos_seq, pos_token;
    const uint16_t *q, *k, *v;
    int64_t q_seq, q_token, q_head, k_seq, k_token, k_head, v_seq, v_token, v_head;  // elements
    uint16_t *q_out;
    void *k_pages, *v_pages;
    float *k_scale, *v_scale;
    const int32_t *block_table;
    const int32_t *seq_lens;
    int *flags;
    int T, Hq, Hkv, bt_stride, num_pages;
    int tokens, chunk;  // num_seqs * T; rows of a token per thread
};

// Rows of a thread: kRowsEach where there is work enough, fewer while the grid is below kAppendCtas, six CTAs for each of 152
// SMs (320 tokens of 24 + 8 heads of 256, fp8: 5.9 us then; with 304 CTAs wanted 9.6, with 9,728 7.6).
constexpr int kRowsEach = 48;
constexpr int kAppendThreads = 64;
constexpr int kAppendCtas = 912;
constexpr int kE = 16;  // elements of a lane: two 16-byte vectors of bf16

// Where the two elements of a pair are, as the kernel is built for it.
enum Pairing : int {
    kHalves,    // P / 8 lanes hold 8 pairs each: 8 elements of either half (P a multiple of 8)
    kAdjacent,  // inside a lane's vectors
    kApart      // halves that begin inside a vector: the other element is read again, two bytes at a time, with one row in
                // flight (8,192 tokens of 32 + 16 heads of 128, 108 of it turned: bf16 73.8 us, fp8 78.5; all of it 34.4, 38.4)
};

__device__ __forceinline__ uint64_t pair2(float lo, float hi) {
    return ((uint64_t)__float_as_uint(hi) << 32) | __float_as_uint(lo);
}
__device__ __forceinline__ float low(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float high(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ uint64_t fma2_down(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rm.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// y = x / s, each rounded to nearest as IEEE division rounds it.  With the reciprocal correctly rounded, one correction by the
// exact remainder gives a quotient within an ulp and a second one the correctly rounded quotient (Markstein, IBM J. Res. Dev.
// 34, 1990), two elements an instruction: 8,192 tokens of 32 + 16 heads of 128 into an fp8 cache 41.0 us by divisions, 38.4
// so.  Remainders are exact where the scale is far from both ends of the exponents; else by divisions.  (A remainder that
// underflows all the same belongs to a quotient below 2^-10, whose code is 0 either way.)  The remainders are
// rounded down, which changes no exact one but those that are 0: -0 then, which added to a zero quotient leaves its sign
// (a +0 would make -0 a +0, whose e4m3 code is another).
__device__ __forceinline__ void quotients(const float (&x)[8], float s, float (&y)[8]) {
    if (s >= 8.67361737988403547e-19f && s <= 1.152921504606846976e18f) {  // 2^-60, 2^60
        const float r = __frcp_rn(s);
        const uint64_t r2 = pair2(r, r), minus = pair2(-s, -s);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const uint64_t x2 = pair2(x[e], x[e + 1]);
            uint64_t q = mul2(x2, r2);
            q = fma2(fma2_down(minus, q, x2), r2, q);
            q = fma2(fma2_down(minus, q, x2), r2, q);
            y[e] = low(q);
            y[e + 1] = high(q);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = __fdiv_rn(x[e], s);
    }
}

// Eight codes of the append's rule, element e at bit e * bits of the result.
template <int DT>
__device__ __forceinline__ uint64_t codes8(const float (&x)[8], float s) {
    constexpr int kBits = DT == VA_INT4 ? 4 : DT == VA_INT2 ? 2 : 8;
    constexpr int qm = DT == VA_INT8 ? 127 : DT == VA_INT4 ? 7 : 1, mask = (1 << kBits) - 1;
    float y[8];
    quotients(x, s, y);
    uint64_t codes = 0;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        uint32_t two;
        if constexpr (DT == VA_FP8_E4M3) {
            two = (uint32_t)__nv_cvt_float2_to_fp8x2(
                make_float2(fminf(fmaxf(y[e], -448.f), 448.f), fminf(fmaxf(y[e + 1], -448.f), 448.f)), __NV_SATFINITE, __NV_E4M3);
        } else {
            two = ((uint32_t)max(-qm, min(qm, __float2int_rn(y[e]))) & mask) |
                  (((uint32_t)max(-qm, min(qm, __float2int_rn(y[e + 1]))) & mask) << kBits);
        }
        codes |= (uint64_t)two << (e * kBits);
    }
    return codes;
}

// The append's rule (verify_attn_kv_append) on a row that D / 16 lanes hold: absmax over the lanes (exact), the scale an IEEE
// binary32 division, the quotients rounded as one, the codes rounded to nearest even.  x0 and x1 are 8 elements each, from e0 and e1.
template <int D, int DT>
__device__ __forceinline__ void store_quantised(const float (&x0)[8], const float (&x1)[8], int e0, int e1, void *pages,
                                                float *scales, size_t row, bool first, bool write) {
    float a = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) a = fmaxf(a, fmaxf(fabsf(x0[e]), fabsf(x1[e])));
#pragma unroll
    for (int o = D / kE / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    if (!write) return;  // a row that is not the cache's, in a warp with one that is
    constexpr float qmax = DT == VA_FP8_E4M3 ? 448.f : DT == VA_INT8 ? 127.f : DT == VA_INT4 ? 7.f : 1.f;
    constexpr int kBits = DT == VA_INT4 ? 4 : DT == VA_INT2 ? 2 : 8;
    const float s = a > 0.f ? __fdiv_rn(a, qmax) : 1.f;
    unsigned char *dst = static_cast<unsigned char *>(pages) + row * (D * kBits / 8);
    auto put = [&](int e, uint64_t codes) {
        unsigned char *to = dst + e * kBits / 8;
        if constexpr (kBits == 8) *reinterpret_cast<uint2 *>(to) = make_uint2((uint32_t)codes, (uint32_t)(codes >> 32));
        else if constexpr (kBits == 4) *reinterpret_cast<uint32_t *>(to) = (uint32_t)codes;
        else *reinterpret_cast<uint16_t *>(to) = (uint16_t)codes;
    };
    put(e0, codes8<DT>(x0, s));
    put(e1, codes8<DT>(x1, s));
    if (first) scales[row] = s;
}

// D / 16 lanes hold a row of one token, 16 elements each, and turn `chunk` rows of that token (its Hq + 2 Hkv rows: q, k, v)
// one after the other, kAhead of them with their loads in flight.  Both elements of a pair are in the lane, whose 8 (cos, sin)
// stay in registers: a rotation is two multiplications and two fused ones, two pairs an instruction, without shared memory,
// barriers or exchange.  8,192 tokens of 32 + 16 heads of 128, bf16: with pairs spread over lanes (the other element by a
// shuffle) 85 us, bound by its instructions; with a token's (cos, sin) in shared memory for all its rows 66 us; this one 34.4
// us, 5.8 TB/s, bound by the loads in flight: three rows ahead in eight CTAs an SM (two rows 38.4 us; four 36.4; nine CTAs,
// with fewer registers, 41.1).  In CTAs of 64 threads, since 128 leave a sixth of the SMs a CTA short here.
template <int D, int DT, int PAIRING>
__global__ void __launch_bounds__(kAppendThreads, 8) rope_append_kernel(const __grid_constant__ RopeAppendParams p) {
    constexpr int kLanes = D / kE, kAhead = PAIRING == kApart ? 1 : 3;
    const int P = p.rope.num_pairs;
    const int lane = threadIdx.x & 31, sub = lane % kLanes;
    const int n = (blockIdx.x * kAppendThreads + threadIdx.x) / kLanes;
    const bool here = n < p.tokens;  // whole rows of lanes, so that those past the end only take part in exchanges
    const int b = here ? n / p.T : 0, t = here ? n - b * p.T : 0;
    const int rows = p.Hq + 2 * p.Hkv;
    const int from = blockIdx.y * p.chunk, to = min(rows, from + p.chunk);
    // this lane's elements, 8 from e0 and 8 from e1: halves of the same 8 pairs (then the rest of the head, two vectors a
    // lane), or vectors of the head's own halves
    const int pair_lanes = P / 8;
    const bool tail = PAIRING == kHalves && sub >= pair_lanes;
    const int e0 = tail ? 2 * P + kE * (sub - pair_lanes) : 8 * sub;
    const int e1 = PAIRING != kHalves ? D / 2 + e0 : tail ? e0 + 8 : P + 8 * sub;
    auto pair_of = [&](int j) { return PAIRING == kHalves ? 8 * sub + j : (j < 4 ? e0 / 2 + j : e1 / 2 + j - 4); };
    griddep_wait();
    auto source = [&](int row) {
        return row < p.Hq           ? p.q + b * p.q_seq + t * p.q_token + row * p.q_head
               : row < p.Hq + p.Hkv ? p.k + b * p.k_seq + t * p.k_token + (row - p.Hq) * p.k_head
                                    : p.v + b * p.v_seq + t * p.v_token + (row - p.Hq - p.Hkv) * p.v_head;
    };
    const int place = p.seq_lens[b] - p.T + t;
    int at[VA_ROPE_MAX_AXES] = {place, place, place, place};
    if (p.pos) positions(p.rope, p.pos + b * p.pos_seq + t * p.pos_token, p.pos_axis, at);
    auto angle = [&](int pair) {
        float2 cs;
        angles<1>(p.rope, pair, at, &cs);
        return cs;
    };
    uint4 next0[kAhead], next1[kAhead];
    auto load = [&](int row) {
#pragma unroll
        for (int r = 0; r < kAhead; ++r) {
            next0[r] = next1[r] = make_uint4(0, 0, 0, 0);
            if (here && row + r < to) {
                const uint16_t *src = source(row + r);
                next0[r] = *reinterpret_cast<const uint4 *>(src + e0);
                next1[r] = *reinterpret_cast<const uint4 *>(src + e1);
            }
        }
    };
    load(from);  // under way while the angles are computed
    int page = -1;
    const int block = place / VA_PAGE_SIZE;
    if (to > p.Hq && place >= 0 && block < p.bt_stride) page = p.block_table[(size_t)b * p.bt_stride + block];
    const bool stored = here && page >= 0 && (p.num_pages == 0 || page < p.num_pages);
    float2 cs[8];
    if (PAIRING != kApart && from < p.Hq + p.Hkv && !tail) {
#pragma unroll
        for (int j = 0; j < 8; j += 4)
            if (pair_of(j) < P) angles<4>(p.rope, pair_of(j), at, cs + j);
    }
    float2 each[PAIRING == kApart ? kE : 1];  // of every element
    if (PAIRING == kApart) {
#pragma unroll
        for (int m = 0; m < kE; ++m) {
            const int i = m < 8 ? e0 + m : e1 + m - 8;
            each[PAIRING == kApart ? m : 0] = i < 2 * P ? angle(i < P ? i : i - P) : make_float2(1.f, 0.f);
        }
    }
    for (int base = from; base < to; base += kAhead) {
        uint4 raw0[kAhead], raw1[kAhead];
#pragma unroll
        for (int r = 0; r < kAhead; ++r) {
            raw0[r] = next0[r];
            raw1[r] = next1[r];
        }
        load(base + kAhead);  // under way while these are turned
#pragma unroll
        for (int r = 0; r < kAhead; ++r) {
            const int row = base + r;
            if (row >= to) break;
            const bool is_v = row >= p.Hq + p.Hkv;
            float x0[8], x1[8];
            unpack<VA_FLOAT_BF16, 8>(raw0[r], x0);
            unpack<VA_FLOAT_BF16, 8>(raw1[r], x1);
            if (!is_v) {
                if constexpr (PAIRING == kHalves) {
                    if (!tail) {
#pragma unroll
                        for (int j = 0; j < 8; j += 2) {
                            const uint64_t a2 = pair2(x0[j], x0[j + 1]), b2 = pair2(x1[j], x1[j + 1]);
                            const uint64_t c2 = pair2(cs[j].x, cs[j + 1].x), s2 = pair2(cs[j].y, cs[j + 1].y);
                            const uint64_t na = fma2(a2, c2, mul2(b2, pair2(-cs[j].y, -cs[j + 1].y)));
                            const uint64_t nb = fma2(b2, c2, mul2(a2, s2));
                            x0[j] = low(na), x0[j + 1] = high(na);
                            x1[j] = low(nb), x1[j + 1] = high(nb);
                        }
                    }
                } else if constexpr (PAIRING == kAdjacent) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float &u = j < 4 ? x0[2 * (j & 3)] : x1[2 * (j & 3)], &v = j < 4 ? x0[2 * (j & 3) + 1] : x1[2 * (j & 3) + 1];
                        const float nu = fmaf(u, cs[j].x, -v * cs[j].y), nv = fmaf(v, cs[j].x, u * cs[j].y);
                        if (pair_of(j) < P) u = nu, v = nv;
                    }
                } else {
                    const uint16_t *src = source(row);
#pragma unroll
                    for (int m = 0; m < kE; ++m) {
                        const int i = m < 8 ? e0 + m : e1 + m - 8;
                        if (i < 2 * P && here) {
                            const float2 r2 = each[m];
                            const float far = __uint_as_float((uint32_t)src[i < P ? i + P : i - P] << 16);
                            float &x = m < 8 ? x0[m & 7] : x1[m & 7];
                            x = fmaf(x, r2.x, i < P ? -far * r2.y : far * r2.y);
                        }
                    }
                    __syncwarp();  // every lane has read before q is written, where it is q_out itself
                }
            }
            if (row < p.Hq) {
                if (here) {
                    uint16_t *dst = p.q_out + ((size_t)n * p.Hq + row) * D;
                    *reinterpret_cast<uint4 *>(dst + e0) = packed<VA_FLOAT_BF16, 8, uint4>(x0);
                    *reinterpret_cast<uint4 *>(dst + e1) = packed<VA_FLOAT_BF16, 8, uint4>(x1);
                }
                continue;
            }
            if (here && !stored && sub == 0 && p.flags) atomicOr(p.flags, kFlagBadPage);
            const size_t dst_row = stored ? ((size_t)page * VA_PAGE_SIZE + place % VA_PAGE_SIZE) * p.Hkv + row - p.Hq - (is_v ? p.Hkv : 0) : 0;
            void *pages = is_v ? p.v_pages : p.k_pages;
            if constexpr (DT == VA_BF16) {  // v's bits unchanged, as in the append
                if (stored) {
                    uint16_t *dst = static_cast<uint16_t *>(pages) + dst_row * D;
                    *reinterpret_cast<uint4 *>(dst + e0) = is_v ? raw0[r] : packed<VA_FLOAT_BF16, 8, uint4>(x0);
                    *reinterpret_cast<uint4 *>(dst + e1) = is_v ? raw1[r] : packed<VA_FLOAT_BF16, 8, uint4>(x1);
                }
            } else {
                store_quantised<D, DT>(x0, x1, e0, e1, pages, is_v ? p.v_scale : p.k_scale, dst_row, sub == 0, stored);
            }
        }
    }
}

template <int D, int DT>
cudaError_t launch_append(RopeAppendParams p, cudaStream_t s) {
    const int rows = p.Hq + 2 * p.Hkv;
    const unsigned ctas = (unsigned)(((long long)p.tokens * (D / kE) + kAppendThreads - 1) / kAppendThreads);
    const int chunks = std::min(rows, std::max((rows + kRowsEach - 1) / kRowsEach, (int)((kAppendCtas + ctas - 1) / ctas)));
    p.chunk = (rows + chunks - 1) / chunks;
    const dim3 grid(ctas, (rows + p.chunk - 1) / p.chunk), block(kAppendThreads);
    if (p.rope.adjacent) return launch_pdl(rope_append_kernel<D, DT, kAdjacent>, grid, block, 0, s, p);
    return p.rope.num_pairs % 8 == 0 ? launch_pdl(rope_append_kernel<D, DT, kHalves>, grid, block, 0, s, p)
                                     : launch_pdl(rope_append_kernel<D, DT, kApart>, grid, block, 0, s, p);
}

template <int D>
cudaError_t launch_append_d(const RopeAppendParams &p, int dtype, cudaStream_t s) {
    switch (dtype) {
    case VA_BF16: return launch_append<D, VA_BF16>(p, s);
    case VA_FP8_E4M3: return launch_append<D, VA_FP8_E4M3>(p, s);
    case VA_INT8: return launch_append<D, VA_INT8>(p, s);
    case VA_INT4: return launch_append<D, VA_INT4>(p, s);
    default: return launch_append<D, VA_INT2>(p, s);
    }
}

bool rope_ok(const va_rope *r) {
    if (!r || r->num_pairs < 1 || r->num_pairs > VA_ROPE_MAX_PAIRS || r->num_axes < 1 || r->num_axes > VA_ROPE_MAX_AXES)
        return false;
    for (int i = 0; i < r->num_pairs; ++i)
        if (r->axis[i] >= r->num_axes) return false;
    return true;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Whether the elements of an output lie apart: each dimension's stride clears the extent of those inside it.
bool apart(const va_heads &x, int num_seqs, int T, int head_dim) {
    struct Dim {
        int64_t stride, size;
    } d[3] = {{x.stride_head, x.num_heads}, {x.stride_token, T}, {x.stride_seq, num_seqs}};
    std::sort(d, d + 3, [](const Dim &a, const Dim &b) { return a.stride < b.stride; });
    __int128 extent = head_dim;  // strides are any number of 63 bits
    for (const Dim &k : d) {
        if (k.size <= 1) continue;
        if (k.stride < extent) return false;
        extent += (__int128)(k.size - 1) * k.stride;
    }
    return true;
}

bool same_strides(const va_heads &a, const va_heads &b, int num_seqs, int T) {
    return (num_seqs <= 1 || a.stride_seq == b.stride_seq) && (T <= 1 || a.stride_token == b.stride_token) &&
           (a.num_heads <= 1 || a.stride_head == b.stride_head);
}

// The strides that matter (of a dimension of more than one) are multiples of w elements and not negative.
bool strides_ok(const va_heads &x, int num_seqs, int T, int64_t w) {
    return (num_seqs <= 1 || (x.stride_seq >= 0 && x.stride_seq % w == 0)) &&
           (T <= 1 || (x.stride_token >= 0 && x.stride_token % w == 0)) &&
           (x.num_heads <= 1 || (x.stride_head >= 0 && x.stride_head % w == 0));
}

}  // namespace
}  // namespace va

extern "C" int verify_attn_rope_init(va_rope *rope, const double *inv_freq, const int32_t *axis, int num_pairs,
                                     int num_axes, int adjacent, float scale) {
    if (!rope || !inv_freq || num_pairs < 1 || num_pairs > VA_ROPE_MAX_PAIRS || num_axes < 1 ||
        num_axes > VA_ROPE_MAX_AXES || !std::isfinite(scale))
        return VA_ERR_INVALID_ARGUMENT;
    for (int i = 0; i < num_pairs; ++i) {
        if (!std::isfinite(inv_freq[i]) || std::fabs(inv_freq[i]) > 1048576.0) return VA_ERR_INVALID_ARGUMENT;
        if (axis && (axis[i] < 0 || axis[i] >= num_axes)) return VA_ERR_INVALID_ARGUMENT;
    }
    // 1 / (2 pi) in units of 2^-130, in two words: cut there, it is off by less than 2^-130, an angle at any frequency up to
    // 2^20 and any int32 position by less than 2^-79 of a turn, so that the rounding of turn[i] to 2^-64 is all of its error.
    // (One word would cost 2^-21 of a turn at the largest of both.)
    constexpr uint64_t kTurnHigh = 0xA2F9836E4E441529ull, kTurnLow = 0xFC2757D1F534DDC0ull;
    *rope = va_rope{};
    for (int i = 0; i < num_pairs; ++i) {
        int e = 0;
        const double m = std::frexp(std::fabs(inv_freq[i]), &e);  // in [0.5, 1), or 0
        const uint64_t whole = (uint64_t)std::ldexp(m, 53);       // inv_freq = whole 2^(e - 53)
        // the product of 53 and 128 bits without its last word, which lies below every rounding
        const unsigned __int128 product = (unsigned __int128)whole * kTurnHigh + (((unsigned __int128)whole * kTurnLow) >> 64);
        // turns = product 2^(e - 53 - 66); as a multiple of 2^-64: product 2^(e - 55), rounded
        const int shift = 55 - e;
        const uint64_t turn =  // e <= 21, so shift >= 34
            shift > 120 ? 0 : (uint64_t)((product + ((unsigned __int128)1 << (shift - 1))) >> shift);
        rope->turn[i] = inv_freq[i] < 0 ? 0 - turn : turn;
        rope->axis[i] = (uint8_t)(axis ? axis[i] : 0);
    }
    rope->num_pairs = num_pairs;
    rope->num_axes = num_axes;
    rope->adjacent = adjacent != 0;
    rope->scale = scale;
    return VA_OK;
}

extern "C" int verify_attn_rope(const va_rope *rope, const va_positions *positions, va_float_type type, int num_seqs,
                                int T, int head_dim, const va_heads *q, const va_heads *q_out, const va_heads *k,
                                const va_heads *k_out, int inverse, void *stream) {
    if (!va::rope_ok(rope) || !positions || !q || !q_out || !k != !k_out) return VA_ERR_INVALID_ARGUMENT;
    if (type != VA_FLOAT_BF16 && type != VA_FLOAT_FP16 && type != VA_FLOAT_FP32) return VA_ERR_UNSUPPORTED;
    if (num_seqs < 0 || T < 0 || head_dim < 2 * rope->num_pairs || head_dim > 1024) return VA_ERR_INVALID_ARGUMENT;
    if (q->num_heads < 1 || q->num_heads != q_out->num_heads || (k && (k->num_heads < 1 || k->num_heads != k_out->num_heads)))
        return VA_ERR_INVALID_ARGUMENT;
    const long long tokens = (long long)num_seqs * T;
    if (tokens > (1LL << 30) || (long long)q->num_heads + (k ? k->num_heads : 0) > 65535) return VA_ERR_INVALID_ARGUMENT;
    const int heads = q->num_heads + (k ? k->num_heads : 0);
    if (tokens == 0) return VA_OK;
    const int bytes = type == VA_FLOAT_FP32 ? 4 : 2;
    if (!positions->data || !va::aligned(positions->data, 4)) return VA_ERR_INVALID_ARGUMENT;
    const va_heads *all[4] = {q, q_out, k, k_out};
    for (int i = 0; i < 4; ++i) {
        if (!all[i]) continue;
        if (!all[i]->data || !va::aligned(all[i]->data, bytes) || !va::strides_ok(*all[i], num_seqs, T, 1))
            return VA_ERR_INVALID_ARGUMENT;
        if ((i & 1) && !va::apart(*all[i], num_seqs, T, head_dim)) return VA_ERR_INVALID_ARGUMENT;
        if ((i & 1) && all[i]->data == all[i - 1]->data && !va::same_strides(*all[i], *all[i - 1], num_seqs, T))
            return VA_ERR_INVALID_ARGUMENT;
    }
    // the widest vector, up to 16 bytes, that every pointer, stride and part of the head is a multiple of (16,384 tokens of 40
    // heads, bf16: 16 bytes 84-99 % of the copy rate, 4 bytes (head_dim 72, 36 of it turned) 60 %, 2 bytes (34 turned) 40 %)
    const int P = rope->num_pairs;
    int w = 1;
    for (int cand : {16 / bytes, 4, 2}) {
        bool ok = (rope->adjacent ? 2 * P : P) % cand == 0 && (head_dim - 2 * P) % cand == 0;
        for (const va_heads *x : all)
            ok = ok && (!x || (va::aligned(x->data, (uintptr_t)cand * bytes) && va::strides_ok(*x, num_seqs, T, cand)));
        if (ok) {
            w = cand;
            break;
        }
    }
    va::RopeParams p{};
    p.rope = *rope;
    p.pos = positions->data;
    p.pos_axis = positions->stride_axis;
    p.pos_seq = positions->stride_seq;
    p.pos_token = positions->stride_token;
    auto tensor = [&](const va_heads *in, const va_heads *out) {
        return va::Tensor{static_cast<const char *>(in->data), static_cast<char *>(out->data),
                          in->stride_seq * bytes, in->stride_token * bytes, in->stride_head * bytes,
                          out->stride_seq * bytes, out->stride_token * bytes, out->stride_head * bytes};
    };
    p.q = tensor(q, q_out);
    if (k) p.k = tensor(k, k_out);
    p.q_heads = q->num_heads;
    p.heads = heads;
    p.tokens = (int)tokens;
    const bool one = rope->adjacent && w > 1;  // vectors of a unit: one, else two
    p.head_dim = head_dim;
    p.pair_units = one ? 2 * P / w : P / w;
    p.units = p.pair_units + ((head_dim - 2 * P) / w + (one ? 0 : 1)) / (one ? 1 : 2);
    p.inverse_sign = inverse ? -1.f : 1.f;
    if (tokens * p.units > (1LL << 30)) return VA_ERR_INVALID_ARGUMENT;
    const unsigned ctas = (unsigned)((tokens * p.units + va::kThreads - 1) / va::kThreads);
    const int each = va::kHeadBytes / (w * bytes);
    const int chunks = std::min<long long>(heads, std::max<long long>((heads + each - 1) / each,
                                                                      (va::kMinCtas + ctas - 1) / ctas));
    p.head_chunk = (heads + chunks - 1) / chunks;
    p.by_T = va::fast_div((uint32_t)T);
    p.by_units = va::fast_div((uint32_t)p.units);
    const dim3 grid(ctas, (unsigned)((heads + p.head_chunk - 1) / p.head_chunk));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = type == VA_FLOAT_BF16   ? va::launch_rope<VA_FLOAT_BF16>(p, w, grid, s)
                          : type == VA_FLOAT_FP16 ? va::launch_rope<VA_FLOAT_FP16>(p, w, grid, s)
                                                  : va::launch_rope<VA_FLOAT_FP32>(p, w, grid, s);
    if (e != cudaSuccess) {
        va::note_cuda_error(e);
        return VA_ERR_CUDA;
    }
    return VA_OK;
}

extern "C" int verify_attn_rope_append(const va_rope *rope, const va_positions *positions, int num_seqs, int T,
                                       int head_dim, const va_heads *q, void *q_out, const va_heads *k_new,
                                       const va_heads *v_new, va_kv_dtype kv_dtype, void *k_pages, void *v_pages,
                                       float *k_scale, float *v_scale, const int32_t *block_table,
                                       int block_table_stride, const int32_t *seq_lens, int num_pages, int *flags,
                                       void *stream) {
    if (!va::rope_ok(rope) || !q != !q_out || !k_new || !v_new || !k_pages || !v_pages || !block_table || !seq_lens)
        return VA_ERR_INVALID_ARGUMENT;
    if (num_seqs < 1 || T < 1 || block_table_stride < 1 || num_pages < 0) return VA_ERR_INVALID_ARGUMENT;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return VA_ERR_UNSUPPORTED;
    if (kv_dtype < VA_BF16 || kv_dtype > VA_INT2) return VA_ERR_UNSUPPORTED;
    if (kv_dtype != VA_BF16 && (!k_scale || !v_scale)) return VA_ERR_INVALID_ARGUMENT;
    if (2 * rope->num_pairs > head_dim) return VA_ERR_INVALID_ARGUMENT;
    if (k_new->num_heads < 1 || k_new->num_heads != v_new->num_heads || (q && q->num_heads < 1))
        return VA_ERR_INVALID_ARGUMENT;
    if (positions && (!positions->data || !va::aligned(positions->data, 4))) return VA_ERR_INVALID_ARGUMENT;
    // rows move as 16-byte (bf16 in) / 8-byte (codes out) units
    for (const va_heads *x : {q, k_new, v_new})
        if (x && (!x->data || !va::aligned(x->data, 16) || !va::strides_ok(*x, num_seqs, T, 8))) return VA_ERR_INVALID_ARGUMENT;
    if (q && q_out == q->data) {  // in place: q has to lie as q_out does
        const va_heads whole{q_out, (int64_t)T * q->num_heads * head_dim, (int64_t)q->num_heads * head_dim, head_dim, q->num_heads};
        if (!va::same_strides(*q, whole, num_seqs, T)) return VA_ERR_INVALID_ARGUMENT;
    }
    if (!va::aligned(k_pages, 16) || !va::aligned(v_pages, 16) || (q_out && !va::aligned(q_out, 16)) ||
        !va::aligned(block_table, 4) || !va::aligned(seq_lens, 4) || !va::aligned(k_scale, 4) ||
        !va::aligned(v_scale, 4) || !va::aligned(flags, 4))
        return VA_ERR_INVALID_ARGUMENT;
    const long long tokens = (long long)num_seqs * T;
    if (tokens > (1LL << 26) || (q && q->num_heads > 65535) || k_new->num_heads > 65535) return VA_ERR_INVALID_ARGUMENT;
    va::RopeAppendParams p{};
    p.rope = *rope;
    if (positions) {
        p.pos = positions->data;
        p.pos_axis = positions->stride_axis;
        p.pos_seq = positions->stride_seq;
        p.pos_token = positions->stride_token;
    }
    if (q) {
        p.q = static_cast<const uint16_t *>(q->data);
        p.q_seq = q->stride_seq;
        p.q_token = q->stride_token;
        p.q_head = q->stride_head;
        p.Hq = q->num_heads;
        p.q_out = static_cast<uint16_t *>(q_out);
    }
    p.k = static_cast<const uint16_t *>(k_new->data);
    p.k_seq = k_new->stride_seq;
    p.k_token = k_new->stride_token;
    p.k_head = k_new->stride_head;
    p.v = static_cast<const uint16_t *>(v_new->data);
    p.v_seq = v_new->stride_seq;
    p.v_token = v_new->stride_token;
    p.v_head = v_new->stride_head;
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.flags = flags;
    p.T = T;
    p.tokens = (int)tokens;
    p.Hkv = k_new->num_heads;
    p.bt_stride = block_table_stride;
    p.num_pages = num_pages;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (head_dim) {
    case 64: e = va::launch_append_d<64>(p, kv_dtype, s); break;
    case 128: e = va::launch_append_d<128>(p, kv_dtype, s); break;
    default: e = va::launch_append_d<256>(p, kv_dtype, s); break;
    }
    if (e != cudaSuccess) {
        va::note_cuda_error(e);
        return VA_ERR_CUDA;
    }
    return VA_OK;
}
