// One quantised row of the paged cache, written by one warp: the rule of
// verify_attn_kv_append, shared by the append kernels.  Lane l holds elements
// [l E, l E + E) of the D-long row in fp32 (E = D / 32).  The absmax is a warp
// max-reduction (exact); the scale and the quotients are IEEE fp32 divisions
// (__fdiv_rn), the e4m3 code is the hardware's round-to-nearest-even
// saturating conversion and the integer codes a round-half-even conversion, so
// every byte is the one the definition in verify_attn.h fixes.
#pragma once

#include <cuda_fp8.h>

#include "va_internal.h"

namespace va {

template <int E>
struct RowVec;  // the E 16-bit values of a lane as one load
template <>
struct RowVec<2> {
    using In = uint32_t;
};
template <>
struct RowVec<4> {
    using In = uint2;
};
template <>
struct RowVec<8> {
    using In = uint4;
};

// x -> codes and scale of cache row `dst_row` (= (page * 16 + slot) * Hkv + g)
template <int D, int DT>
__device__ __forceinline__ void store_quantised_row(const float (&x)[D / 32], void *pages, float *scales,
                                                    size_t dst_row, int lane) {
    constexpr int E = D / 32;
    static_assert(DT != VA_BF16, "bf16 rows are stored unquantised");
    float a = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) a = fmaxf(a, fabsf(x[e]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    if constexpr (DT == VA_INT4 || DT == VA_INT2) {
        // 4-bit / 2-bit codes: the int8 rule with qmax 7 / 1, each lane's E
        // codes packed into an F-bit field (element e at bit e * bits), then
        // the fields of 32 / F neighbouring lanes ORed into one 32-bit word
        // (lane order = element order, so the word is the row's little-endian
        // bit stream) that the first of them stores.
        constexpr int kBits = DT == VA_INT4 ? 4 : 2;
        constexpr int qm = (1 << (kBits - 1)) - 1;
        constexpr int F = E * kBits;          // 4 .. 32 bits per lane
        constexpr int kLanesPerWord = 32 / F;
        const float s = a > 0.f ? __fdiv_rn(a, (float)qm) : 1.f;
        uint32_t field = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = max(-qm, min(qm, __float2int_rn(__fdiv_rn(x[e], s))));
            field |= ((uint32_t)c & ((1u << kBits) - 1)) << (e * kBits);
        }
        uint32_t word = field;
#pragma unroll
        for (int k = 1; k < kLanesPerWord; ++k) {
            const uint32_t nb = __shfl_down_sync(0xffffffffu, field, k);
            if (lane + k < 32) word |= nb << (k * F);
        }
        unsigned char *dst = static_cast<unsigned char *>(pages) + dst_row * (D * kBits / 8);
        if (lane % kLanesPerWord == 0) *reinterpret_cast<uint32_t *>(dst + lane * F / 8) = word;
        if (lane == 0) scales[dst_row] = s;
    } else {
        const float qmax = DT == VA_FP8_E4M3 ? 448.f : 127.f;
        const float s = a > 0.f ? __fdiv_rn(a, qmax) : 1.f;
        // codes of elements e, e + 1 as one 16-bit pair, element e in the low byte
        uint32_t pair[E / 2];
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            float y0 = __fdiv_rn(x[e], s), y1 = __fdiv_rn(x[e + 1], s);
            if constexpr (DT == VA_FP8_E4M3) {
                y0 = fminf(fmaxf(y0, -448.f), 448.f);
                y1 = fminf(fmaxf(y1, -448.f), 448.f);
                pair[e / 2] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(y0, y1), __NV_SATFINITE, __NV_E4M3);
            } else {
                const uint32_t c0 = (uint32_t)(max(-127, min(127, __float2int_rn(y0))) & 0xFF);
                const uint32_t c1 = (uint32_t)(max(-127, min(127, __float2int_rn(y1))) & 0xFF);
                pair[e / 2] = c0 | (c1 << 8);
            }
        }
        unsigned char *dst = static_cast<unsigned char *>(pages) + dst_row * D + lane * E;
        if constexpr (E == 2) {
            *reinterpret_cast<uint16_t *>(dst) = (uint16_t)pair[0];
        } else if constexpr (E == 4) {
            *reinterpret_cast<uint32_t *>(dst) = pair[0] | (pair[1] << 16);
        } else {
            *reinterpret_cast<uint2 *>(dst) = make_uint2(pair[0] | (pair[1] << 16), pair[2] | (pair[3] << 16));
        }
        if (lane == 0) scales[dst_row] = s;
    }
}

}  // namespace va
