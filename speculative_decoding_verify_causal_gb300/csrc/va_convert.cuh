// Device helpers of the tensor-core kernels: packed fp32 arithmetic, the exact conversions of cached
// codes to fp16, the swizzle of a tile, and the driver's tensor-map encoder.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <mutex>

#include "va_internal.h"
#include "va_sm100.cuh"

namespace va {
namespace {

using namespace sm100;

__device__ __forceinline__ float bf16_bits_to_float(uint32_t b) { return __uint_as_float(b << 16); }

// 2^x with the hardware approximation (relative error ~2^-22; -inf -> +0).
__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Packed fp32 pairs (sm_100+): each lane of a pair is one IEEE-rounded fp32
// multiply / fused multiply-add / add, the same result as the scalar
// instruction, at half the issue cost.
__device__ __forceinline__ uint64_t f2_pack(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t r, uint32_t &lo, uint32_t &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(r));
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// max of three (one instruction on sm_100+)
__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&h);
}

__device__ __forceinline__ uint32_t pack_bf162(float lo, float hi) {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&h);
}

// int8 -> fp16, exact: bias each byte to u = b + 128, place it in the low
// mantissa bits of 1024.0 (0x6400 | u = 1024 + u) and subtract 1152.  This is
// the published "magic number" integer-to-float conversion (e.g. Kim et al.,
// "Who Says Elephants Can't Run", 2022); here it is written out for 4 bytes.
__device__ __forceinline__ void int8x4_to_half2x2(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const uint32_t x = w ^ 0x80808080u;
    uint32_t a, b;
    asm("prmt.b32 %0, %1, %2, 0x4140;" : "=r"(a) : "r"(x), "r"(0x64646464u));
    asm("prmt.b32 %0, %1, %2, 0x4342;" : "=r"(b) : "r"(x), "r"(0x64646464u));
    const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
    __half2 ha = __hsub2(*reinterpret_cast<__half2 *>(&a), bias);
    __half2 hb = __hsub2(*reinterpret_cast<__half2 *>(&b), bias);
    lo = *reinterpret_cast<uint32_t *>(&ha);
    hi = *reinterpret_cast<uint32_t *>(&hb);
}

__device__ __forceinline__ void e4m3x4_to_half2x2(uint32_t w, uint32_t &lo, uint32_t &hi) {
    __half2_raw a = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xFFFFu), __NV_E4M3);
    __half2_raw b = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), __NV_E4M3);
    lo = *reinterpret_cast<uint32_t *>(&a);
    hi = *reinterpret_cast<uint32_t *>(&b);
}

// 4-bit codes -> fp16, exact, the same magic-number idea: code k of w sits in
// bits [4k, 4k + 4); a nibble n of a two's-complement code c has n ^ 8 = c + 8
// in [0, 16), so (n ^ 8) | 0x6400 is the fp16 1024 + c + 8 and subtracting
// 1032 leaves c.  One mask-and-xor makes the pairs (c_s, c_s+4); byte
// permutes put them in element order.  h[j] = (c_2j, c_2j+1).
__device__ __forceinline__ void int4x8_to_half2x4(uint32_t w, uint32_t (&h)[4]) {
    uint32_t a[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) a[s] = ((w >> (4 * s)) & 0x000F000Fu) ^ 0x64086408u;
    asm("prmt.b32 %0, %1, %2, 0x5410;" : "=r"(h[0]) : "r"(a[0]), "r"(a[1]));
    asm("prmt.b32 %0, %1, %2, 0x5410;" : "=r"(h[1]) : "r"(a[2]), "r"(a[3]));
    asm("prmt.b32 %0, %1, %2, 0x7632;" : "=r"(h[2]) : "r"(a[0]), "r"(a[1]));
    asm("prmt.b32 %0, %1, %2, 0x7632;" : "=r"(h[3]) : "r"(a[2]), "r"(a[3]));
    const __half2 bias = __halves2half2(__ushort_as_half(0x6408), __ushort_as_half(0x6408));  // 1032
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        __half2 v = __hsub2(*reinterpret_cast<__half2 *>(&h[j]), bias);
        h[j] = *reinterpret_cast<uint32_t *>(&v);
    }
}

// 2-bit codes -> fp16, exact: code k of w in bits [2k, 2k + 2), (n ^ 2) = c + 2
// in [0, 4), bias 1026; pairs (c_s, c_s+8) permuted into element order.
__device__ __forceinline__ void int2x16_to_half2x8(uint32_t w, uint32_t (&h)[8]) {
    uint32_t a[8];
#pragma unroll
    for (int s = 0; s < 8; ++s) a[s] = ((w >> (2 * s)) & 0x00030003u) ^ 0x64026402u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        asm("prmt.b32 %0, %1, %2, 0x5410;" : "=r"(h[j]) : "r"(a[2 * j]), "r"(a[2 * j + 1]));
        asm("prmt.b32 %0, %1, %2, 0x7632;" : "=r"(h[4 + j]) : "r"(a[2 * j]), "r"(a[2 * j + 1]));
    }
    const __half2 bias = __halves2half2(__ushort_as_half(0x6402), __ushort_as_half(0x6402));  // 1026
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        __half2 v = __hsub2(*reinterpret_cast<__half2 *>(&h[j]), bias);
        h[j] = *reinterpret_cast<uint32_t *>(&v);
    }
}

// The 16 elements of one raw piece of a quantised cache row -> 8 fp16 pairs
// in element order.  A piece is 16 / 8 / 4 bytes (8-bit / 4-bit / 2-bit).
template <int DT>
struct RawPiece {
    static constexpr int kWords = DT == VA_INT4 ? 2 : DT == VA_INT2 ? 1 : 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(uint32_t a) {
        if constexpr (kWords == 4) {
            const uint4 v = lds_u4(a);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else if constexpr (kWords == 2) {
            const uint2 v = lds_u2(a);
            w[0] = v.x, w[1] = v.y;
        } else {
            w[0] = lds_u32(a);
        }
    }
    // the halves of the piece in the other order
    __device__ __forceinline__ void exchange(bool yes) {
        if constexpr (kWords == 1) {
            w[0] = __funnelshift_l(w[0], w[0], yes ? 16 : 0);
        } else {
#pragma unroll
            for (int i = 0; i < kWords / 2; ++i) {
                const uint32_t a = w[i], b = w[i + kWords / 2];
                w[i] = yes ? b : a, w[i + kWords / 2] = yes ? a : b;
            }
        }
    }
    __device__ __forceinline__ void to_half(uint32_t (&hw)[8]) const {
        if constexpr (DT == VA_INT2) {
            int2x16_to_half2x8(w[0], hw);
        } else if constexpr (DT == VA_INT4) {
            uint32_t a[4], b[4];
            int4x8_to_half2x4(w[0], a);
            int4x8_to_half2x4(w[1], b);
#pragma unroll
            for (int j = 0; j < 4; ++j) hw[j] = a[j], hw[4 + j] = b[j];
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (DT == VA_INT8)
                    int8x4_to_half2x2(w[k], hw[2 * k], hw[2 * k + 1]);
                else
                    e4m3x4_to_half2x2(w[k], hw[2 * k], hw[2 * k + 1]);
            }
        }
    }
};

// Byte offset of 16-byte unit u (0..7) of tile row `row` inside a 64-d chunk
// of a 128-byte-swizzled tile (rows of 128 bytes, 8-row / 1024-byte atoms).
__device__ __forceinline__ uint32_t sw128(int row, int u) { return row * 128 + ((u ^ (row & 7)) << 4); }

// ---------------------------------------------------------------- host side
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
    static std::once_flag once;
    static EncodeTiledFn fn = nullptr;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(f);
        else
            cudaGetLastError();
    });
    return fn;
}

// q [N, heads, D] by boxes of 64 elements x G heads x tpt tokens.
inline bool make_q_map(CUtensorMap *m, const va_heads &q, int N, int D, int G, int tpt) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)q.num_heads, (cuuint64_t)N};
    cuuint64_t strides[2] = {(cuuint64_t)q.stride_head * 2, (cuuint64_t)q.stride_token * 2};
    cuuint32_t box[3] = {64u, (cuuint32_t)G, (cuuint32_t)tpt};
    cuuint32_t one[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, q.data, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace va
