// The attention weight that each cached token gathers from a chunk of new tokens, for sm_103a (tcgen05 + TMEM + TMA).
//
//     w[b, g, j] = sum over tokens t with j <= L - n + t, and query heads h of kv head g, of exp(s_j - lse[t, h]),
//     s_j = <q[t, h], K_j> / sqrt(D),
// with the log-sum-exp of the attention itself, so that a token's weights over the keys sum to one.
//
// A CTA holds a block of keys in shared memory (one tile of 128 at head_dim 256, else two) and lets the packed rows of
// q (128 at a time, as chunk attention packs them) pass by: S^T = K Q^T, keys on the tensor memory's lanes.  The sums
// then run along lanes: four threads share a key until the end, and -lse of the rows is read from shared memory.
// Half of the attention's products, the same exponentials, no maximum, no second product.
// Where there are few blocks of keys, a cluster shares one: its CTAs take the tiles of rows in turn and their sums
// are added in rank order, so that the result does not depend on timing.  No atomics.
//
// Bound.  At head_dim 128 (two tiles of keys) a tile of rows is 1,024 clocks of the tensor pipe and 1,024 of the
// exponentials; it takes about 2,200, as the sums of a tile and its loads from the tensor memory come one after the other
// in a warp but for half a tile: 8,192 tokens of 32 heads, bf16, 297 us (389 with a row of scores to a lane).  At 256,
// where one tile of keys takes 1,024, about 1,350: 500 on 24,500 tokens, int8, 139 us (277 without clusters).  8 sequences
// of 16 on 2,048 tokens, fp8, 23 us: the CTAs' starts, half of the 5 us of each of three, which is why all of a thread's
// keys are asked for at once and q before they are there (26 us).
//
// Arithmetic: the keys' codes are exact in bf16, products exact, sums binary32; a thread adds a tile's exponentials
// first and the tiles' sums with a compensation, so that 32,768 rows cost no more bits than 128.
#include <math.h>

#include "va_chunk.h"
#include "va_convert.cuh"

namespace va {
namespace {

constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kRows = kMmaRows;  // packed rows of one tile of q
constexpr int kLseRing = 16;     // tiles whose lse is held: the stages of q, three tiles of scores, one being written

template <int D>
struct Cfg {
    static constexpr int kKeyTiles = weight_keys(D) / 128;
    static constexpr int kChunkBytes = 128 * 128;  // 64 elements of 128 rows
    static constexpr int kTileBytes = D / 64 * kChunkBytes;
    static constexpr int kStages = D == 64 ? 8 : D == 128 ? 4 : 2;
    static constexpr int kSumWarps = 8 * kKeyTiles;
    static constexpr int kProducerWarp = kSumWarps, kMmaWarp = kSumWarps + 1;  // one issuing warp for each tile of keys
    static constexpr int kThreads = (kMmaWarp + kKeyTiles) * 32;
    static constexpr int kK = 0;
    static constexpr int kQ = kKeyTiles * kTileBytes;
    static constexpr int kLse = kQ + kStages * kTileBytes;
    static constexpr int kSum = kLse + kLseRing * kRows * 4;
    static constexpr int kBars = kSum + kKeyTiles * 128 * 4;
    static constexpr int kSmem = kBars + 32 * 8 + 1024;
    static_assert(kSmem <= (int)kMaxSmemPerBlock && kLseRing >= kStages + 4, "shared memory");
};

enum Bar : int {
    kQFull = 0,              // stages
    kQEmpty = 8,             // stages
    kSFull = 16,             // key tile * 2 + buffer
    kSEmpty = kSFull + 4,
    kDone = kSEmpty + 4,
    kTmemSlot = 31,
};

struct Args {
    CUtensorMap tm_q;
    WeightParams p;
};

// 16 elements of a cached row as 8 words of two bf16, exact.
template <int DT>
struct KeyPiece {
    static constexpr int kBytes = DT == VA_BF16 ? 32 : DT == VA_INT4 ? 8 : DT == VA_INT2 ? 4 : 16;
    uint32_t w[kBytes / 4];
    // from `from`, or zeros: without a branch, so that a thread's loads are in flight together
    __device__ __forceinline__ void load(const void *from, bool there) {
#pragma unroll
        for (int i = 0; i < kBytes / 4; ++i) w[i] = 0;
#pragma unroll
        for (int i = 0; i < kBytes; i += 16) {
            const char *at = static_cast<const char *>(from) + i;
            if constexpr (kBytes >= 16)
                asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t@p ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
                             : "+r"(w[i / 4]), "+r"(w[i / 4 + 1]), "+r"(w[i / 4 + 2]), "+r"(w[i / 4 + 3])
                             : "l"(at), "r"((uint32_t)there));
            else if constexpr (kBytes == 8)
                asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %3, 0;\n\t@p ld.global.nc.v2.u32 {%0, %1}, [%2];\n\t}"
                             : "+r"(w[0]), "+r"(w[1])
                             : "l"(at), "r"((uint32_t)there));
            else
                asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p ld.global.nc.u32 %0, [%1];\n\t}"
                             : "+r"(w[0])
                             : "l"(at), "r"((uint32_t)there));
        }
    }
    __device__ __forceinline__ void store(uint32_t lo, uint32_t hi) const {
        uint32_t h[8];
        if constexpr (DT == VA_BF16) {
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] = w[i];
        } else {
            RawPiece<DT> raw;
#pragma unroll
            for (int i = 0; i < kBytes / 4; ++i) raw.w[i] = w[i];
            raw.to_half(h);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
                h[i] = pack_bf162(f.x, f.y);
            }
        }
        sts_u4(lo, make_uint4(h[0], h[1], h[2], h[3]));
        sts_u4(hi, make_uint4(h[4], h[5], h[6], h[7]));
    }
};

template <int D, int DT>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1) weights_kernel(const __grid_constant__ Args args) {
    using C = Cfg<D>;
    const WeightParams &p = args.p;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                            ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int i) { return sbase + C::kBars + 8u * i; };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ranks = p.cluster, rank = blockIdx.x % ranks;

    griddep_wait();
    const WeightItem it = p.items[blockIdx.x / ranks];
    const int G = p.G, tpt = p.tpt;
    const int before = it.L - it.n;                     // keys that every token of the chunk sees
    const int t_first = max(0, it.key0 - before);       // the first token that sees one of the block's keys
    const int all = (it.n - t_first + tpt - 1) / tpt;   // tiles of rows
    const int tiles = all > rank ? (all - rank + ranks - 1) / ranks : 0;
    auto tile_t0 = [&](int m) { return t_first + (m * ranks + rank) * tpt; };
    constexpr int kProducerWarp = C::kProducerWarp, kMmaWarp = C::kMmaWarp;

    // The producer's: rows of q, and their -lse in units of ln 2.
    int token[4];  // of a tile, of this lane's four rows; past every chunk where there is no such row
    int64_t place[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 32 * i + lane;
        token[i] = r < tpt * G ? r / G : 0x40000000;
        place[i] = (int64_t)(it.q0 + r / G) * p.Hq + it.kvh * G + r % G;
    }
    auto load_lse = [&](int m, float (&x)[4]) {
        const int t0 = tile_t0(m);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = m < tiles && token[i] < it.n - t0 ? __ldg(p.lse + place[i] + (int64_t)t0 * p.Hq) : INFINITY;
    };
    float next[4];
    auto load_tile = [&](int m) {
        const int st = m % C::kStages;
#pragma unroll
        for (int i = 0; i < 4; ++i)  // a row without keys, or none, gives nothing
            sts_f32(sbase + C::kLse + 4u * ((m % kLseRing) * kRows + 32 * i + lane),
                    fabsf(next[i]) == INFINITY ? -INFINITY : -next[i] * 1.4426950408889634f);
        __syncwarp();
        if (lane == 0) {
            mbar_arrive_expect_tx(bar(kQFull + st), (uint32_t)(D / 64 * G * tpt * 128));
            for (int c = 0; c < D / 64; ++c)
                tma_load_3d(sbase + C::kQ + st * C::kTileBytes + c * C::kChunkBytes, &args.tm_q, c * 64, it.kvh * G,
                            it.q0 + tile_t0(m), bar(kQFull + st));
        }
        __syncwarp();
        load_lse(m + 1, next);
    };
    int issued = 0;
    if (warp == kProducerWarp) {
        if (lane == 0) {
            prefetch_tensormap(&args.tm_q);
            for (int i = 0; i < C::kStages; ++i) {
                mbar_init(bar(kQFull + i), 1);
                mbar_init(bar(kQEmpty + i), C::kKeyTiles);
            }
            for (int i = 0; i < 2 * C::kKeyTiles; ++i) {
                mbar_init(bar(kSFull + i), 1);
                mbar_init(bar(kSEmpty + i), 8);
            }
            mbar_init(bar(kDone), C::kKeyTiles);
            fence_barrier_init();
        }
        __syncwarp();
        load_lse(0, next);
        for (; issued < min(tiles, C::kStages); ++issued) load_tile(issued);
    } else if (warp == kMmaWarp) {
        tmem_alloc(bar(kTmemSlot), 256 * C::kKeyTiles);
        tmem_relinquish();
    }
    const int32_t *bt = p.block_table + (size_t)it.b * p.bt_stride;
    auto page_of = [&](int key) -> int {  // -1: no such key
        const int page = __ldg(bt + min(key, it.L - 1) / VA_PAGE_SIZE);
        return key >= it.L || page < 0 || (p.num_pages > 0 && page >= p.num_pages) ? -1 : page;
    };
    // A sum warp has 16 keys; a thread two of them, row x (8 apart), in a quarter of the columns: c and c + 1 of each 8.
    const int kt = warp >> 3, h = (warp >> 2) & 1, c = 2 * (lane & 3);
    auto my_row = [&](int x) { return kt * 128 + (warp & 3) * 32 + 16 * h + 8 * x + (lane >> 2); };
    uint64_t c2[2];
    int key[2], page[2];
    if (warp < C::kSumWarps) {
        float scale[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            key[x] = it.key0 + my_row(x);
            page[x] = page_of(key[x]);
        }
        // what is not needed before the keys are there, is asked for before them
#pragma unroll
        for (int x = 0; x < 2; ++x)
            scale[x] = DT != VA_BF16 && page[x] >= 0
                           ? __ldg(p.k_scale + ((size_t)page[x] * VA_PAGE_SIZE + key[x] % VA_PAGE_SIZE) * p.Hkv + it.kvh)
                           : 1.f;
        // the block's keys, 16 elements a piece
        constexpr int kPieces = D / 16, kBatch = D == 64 ? 2 : D == 128 ? 4 : 8;  // all of a thread's: one trip
        constexpr int kTotal = C::kKeyTiles * 128 * kPieces, kStride = C::kSumWarps * 32;
        const unsigned char *pages = static_cast<const unsigned char *>(p.k_pages);
#pragma unroll 1
        for (int e0 = tid; e0 < kTotal; e0 += kBatch * kStride) {
            KeyPiece<DT> x[kBatch];
            int from[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) from[i] = page_of(it.key0 + (e0 + i * kStride) / kPieces);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int e = e0 + i * kStride, key = it.key0 + e / kPieces;
                x[i].load(pages + ((((int64_t)from[i] * VA_PAGE_SIZE + key % VA_PAGE_SIZE) * p.Hkv + it.kvh) * kPieces +
                                   e % kPieces) * KeyPiece<DT>::kBytes, from[i] >= 0);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int e = e0 + i * kStride, row = e / kPieces, u = e % kPieces * 2;
                const uint32_t at = sbase + C::kK + (row / 128) * C::kTileBytes + (u / 8) * C::kChunkBytes;
                x[i].store(at + sw128(row % 128, u % 8), at + sw128(row % 128, u % 8 + 1));
            }
        }
        static_assert(kTotal % (kBatch * kStride) == 0, "whole batches");
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const uint32_t by = __float_as_uint(p.sm_scale_log2 * scale[x]);
            c2[x] = f2_pack(by, by);
        }
        // rows of q's tiles that no box fills: with -lse of -inf they add nothing, as long as they are numbers
        const int full = tpt * G;
        for (int e = tid; e < C::kStages * (D / 8) * (kRows - full); e += kStride) {
            const int row = full + e % (kRows - full), u = e / (kRows - full) % (D / 8), st = e / (kRows - full) / (D / 8);
            sts_u4(sbase + C::kQ + st * C::kTileBytes + (u / 8) * C::kChunkBytes + sw128(row, u % 8), make_uint4(0, 0, 0, 0));
        }
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = lds_u32(bar(kTmemSlot));
    bool ok = true;

    if (warp == kProducerWarp) {
        // ------------------------------------------------------------ producer, once the first stages are on their way
        for (; issued < tiles; ++issued) {
            const int st = issued % C::kStages;
            ok = __all_sync(0xffffffffu, mbar_wait(bar(kQEmpty + st), ((issued / C::kStages) & 1) ^ 1, kWaitNs));
            if (!ok) break;
            load_tile(issued);
        }
        if (lane == 0)
            for (int m = max(0, issued - C::kStages); m < issued; ++m)
                if (!mbar_wait(bar(kQFull + m % C::kStages), (m / C::kStages) & 1, kWaitNs)) ok = false;
    } else if (warp >= kMmaWarp) {
        // ------------------------------------------------------------ MMA issue, by a whole warp: its tile of keys
        const int tile = warp - kMmaWarp;
        constexpr uint32_t id = idesc_f16(128, kRows, 1, 0, 0);
        constexpr uint32_t kHi = smem_desc_hi(1024, 2);
        const uint32_t klo = smem_desc_lo(sbase + C::kK + tile * C::kTileBytes, 16), qlo = smem_desc_lo(sbase + C::kQ, 16);
        for (int m = 0; m < tiles && ok; ++m) {
            const int st = m % C::kStages, s = tile * 2 + (m & 1);
            ok = __all_sync(0xffffffffu, m < 2 ? mbar_wait(bar(kQFull + st), (m / C::kStages) & 1, kWaitNs)
                                               : mbar_wait2(bar(kQFull + st), (m / C::kStages) & 1, bar(kSEmpty + s),
                                                            ((m >> 1) & 1) ^ 1, kWaitNs));
            tc_fence_after();
            if (!ok) break;
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = (kk / 4) * (C::kChunkBytes >> 4) + (kk % 4) * 2;
                    mma_ss_lo<kHi>(tmem + s * kRows, klo + off, qlo + st * (C::kTileBytes >> 4) + off, id, kk > 0);
                }
                mma_commit(bar(kSFull + s));
                mma_commit(bar(kQEmpty + st));
            }
            __syncwarp();
        }
        if (elect_one()) mma_commit(bar(kDone));
        __syncwarp();
        if (!__all_sync(0xffffffffu, mbar_wait(bar(kDone), 0, kWaitNs))) ok = false;
    } else {
        // ------------------------------------------------------------ sums
        const uint32_t half_tm = tmem + ((uint32_t)((warp & 3) * 32 + 16 * h) << 16);
        float sum[2] = {0.f, 0.f}, lost[2] = {0.f, 0.f};
        const int last_key = it.key0 + C::kKeyTiles * 128 - 1;  // of the block: both of a CTA's tiles take one view
        // Half a tile of columns at a time: while one half's exponentials run, the next one is on its way from the
        // tensor memory.
        uint64_t acc[2][2];
        auto add = [&](int m, int half, uint32_t (&x)[32]) {
            const int t0 = tile_t0(m);
            const uint32_t nl = sbase + C::kLse + 4u * ((m % kLseRing) * kRows + 64 * half + c);
            const int to = min(tpt, it.n - t0) * G;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const uint2 l = lds_u2(nl + 32u * u);
                const uint64_t l2 = f2_pack(l.x, l.y);
#pragma unroll
                for (int y = 0; y < 2; ++y)
                    f2_unpack(f2_fma(f2_pack(x[4 * u + 2 * y], x[4 * u + 2 * y + 1]), c2[y], l2), x[4 * u + 2 * y],
                              x[4 * u + 2 * y + 1]);
            }
            if (to < tpt * G || last_key > before + t0) {  // columns [from, to) are rows that see the key
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int from = max(0, key[y] - before - t0) * G;
#pragma unroll
                    for (int u = 0; u < 8; ++u)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int col = 64 * half + 8 * u + c + e;
                            if (col < from || col >= to) x[4 * u + 2 * y + e] = 0xFF800000u;
                        }
                }
            }
#pragma unroll
            for (int u = 0; u < 8; ++u)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const uint64_t e2 = f2_pack(__float_as_uint(ex2_approx(__uint_as_float(x[4 * u + 2 * y]))),
                                                __float_as_uint(ex2_approx(__uint_as_float(x[4 * u + 2 * y + 1]))));
                    acc[y][u & 1] = half == 0 && u < 2 ? e2 : f2_add(acc[y][u & 1], e2);
                }
        };
        auto scores_of = [&](int m) {
            const bool done = __all_sync(0xffffffffu, mbar_wait(bar(kSFull + kt * 2 + (m & 1)), (m >> 1) & 1, kWaitNs));
            tc_fence_after();
            return done;
        };
        uint32_t x0[32], x1[32];
        if (tiles > 0) {
            ok = scores_of(0);
            if (ok) tmem_ld_16x256b(half_tm + kt * 2 * kRows, x0);
        }
#pragma unroll 1
        for (int m = 0; m < tiles && ok; ++m) {
            const int s = kt * 2 + (m & 1);
            tmem_wait_ld();
            tmem_ld_16x256b(half_tm + s * kRows + 64, x1);
            add(m, 0, x0);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kSEmpty + s));
            if (m + 1 < tiles) {
                ok = scores_of(m + 1);
                if (ok) tmem_ld_16x256b(half_tm + (s ^ 1) * kRows, x0);
            }
            add(m, 1, x1);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                uint32_t a, b;
                f2_unpack(f2_add(acc[y][0], acc[y][1]), a, b);
                const float z = __fsub_rn(__fadd_rn(__uint_as_float(a), __uint_as_float(b)), lost[y]);
                const float t = __fadd_rn(sum[y], z);
                lost[y] = __fsub_rn(__fsub_rn(t, sum[y]), z);
                if (!(fabsf(lost[y]) < INFINITY)) lost[y] = 0.f;  // of a sum that is not finite
                sum[y] = t;
            }
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            float z = sum[y];
            z += __shfl_xor_sync(0xffffffffu, z, 1);
            z += __shfl_xor_sync(0xffffffffu, z, 2);
            if ((lane & 3) == 0) sts_f32(sbase + C::kSum + 4u * my_row(y), page[y] < 0 ? 0.f : z);
        }
    }
    if (!ok) atomicOr(p.flags, kFlagTimeoutBit);
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 256 * C::kKeyTiles);
    }
    if (ranks > 1) cluster_sync();
    if (rank == 0 && tid < C::kKeyTiles * 128) {
        const int key = it.key0 + tid;
        float sum = lds_f32(sbase + C::kSum + 4u * tid);
        for (int r = 1; r < ranks; ++r) sum += ld_cluster_f32(smem + C::kSum + 4 * tid, r);
        if (key < it.L) {
            const int64_t at = it.b * p.stride_seq + it.kvh * p.stride_head + key;
            if (p.accumulate && key < before) sum += p.weights[at];
            p.weights[at] = sum;
            if (p.slot_pos && key >= before) p.slot_pos[at] = p.positions[it.q0 + key - before];
            if (page_of(key) < 0) atomicOr(p.flags, kFlagBadPage);
        }
    }
    if (ranks > 1) cluster_sync();  // the sums are read
}

template <int D, int DT>
cudaError_t launch_one(const WeightParams &p, const va_heads &q, int N, int n, cudaStream_t s) {
    using C = Cfg<D>;
    Args a;
    a.p = p;
    if (!make_q_map(&a.tm_q, q, N, D, p.G, p.tpt)) return cudaErrorInvalidValue;
    auto k = weights_kernel<D, DT>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(n * p.cluster);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k, a);
}

template <int D>
cudaError_t launch_d(const WeightParams &p, const va_heads &q, int N, int dtype, int n, cudaStream_t s) {
    switch (dtype) {
    case VA_BF16: return launch_one<D, VA_BF16>(p, q, N, n, s);
    case VA_FP8_E4M3: return launch_one<D, VA_FP8_E4M3>(p, q, N, n, s);
    case VA_INT8: return launch_one<D, VA_INT8>(p, q, N, n, s);
    case VA_INT4: return launch_one<D, VA_INT4>(p, q, N, n, s);
    default: return launch_one<D, VA_INT2>(p, q, N, n, s);
    }
}

}  // namespace

cudaError_t launch_weights(const WeightParams &p, const va_heads &q, int N, int D, int dtype, int num_blocks, cudaStream_t s) {
    if (num_blocks <= 0) return cudaSuccess;
    switch (D) {
    case 64: return launch_d<64>(p, q, N, dtype, num_blocks, s);
    case 128: return launch_d<128>(p, q, N, dtype, num_blocks, s);
    default: return launch_d<256>(p, q, N, dtype, num_blocks, s);
    }
}

}  // namespace va
