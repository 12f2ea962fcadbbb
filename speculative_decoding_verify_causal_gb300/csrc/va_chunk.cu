// Attention of ragged chunks of new tokens over the paged cache, for sm_103a (tcgen05 + TMEM + TMA).
//
// For token t of a chunk of n that ends a sequence of L cached tokens, and query head h of kv head g:
//     s_j = <q, K_j> / sqrt(D), j <= L - n + t;   lse = ln sum_j exp(s_j);   out = sum_j exp(s_j - lse) V_j.
// A tile is 128 packed rows: `tpt` tokens of one sequence with all query heads of one kv head (row = token * G +
// head), so each key and value is read once for all of them.  A CTA takes one item: one tile of rows (head_dim 256)
// or up to two (64, 128) over a range of keys.
//
// Steps.  Step k of a two-tile item is (rows k % 2, keys k / 2); of a one-tile item it is (keys k).  Scores alternate
// between two tensor-memory slots of 80 columns, probabilities between two of 40: 2 x 128 columns (or 256) of O and
// these are all 512, so that the next scores need not wait for the product of these.  Of two tiles each has its slot
// and a warp that issues its instructions: S(i + 1) as soon as the softmax has read S(i), then P(i) V(i).  Of one tile
// one warp issues P(k) V(k), S(k + 2): while the softmax of one slot runs, the tensor pipe works on the other.
//   producer warps  page ids from the block table, then TMA boxes (16 slots of one page and head) into the ring
//   dequant warps   (quantised caches) raw panel -> fp16 panel, exact, in the MMA's swizzled layout; keys' scales
//   MMA warps       as above; panels are used in the order of the ring
//   softmax warps   eight per tile of rows: k scale, mask, running maximum (moved, and O rescaled, only when it grows by
//                   more than 2^8), P * v_scale * 2^beta; at the end O / l and lse
// A softmax warp has 16 rows, and a thread two of them in a quarter of the columns (the 16x256b layout of the tensor
// memory), so a key's scales are read from shared memory by 4 lanes for 16 rows; with a row per lane every lane reads
// every scale, and those reads alone were half of the shared memory's bandwidth.  Four such warps in each quarter of
// the SM hide each other's waits.
// A panel is one tile of keys by min(D, 128) elements: what one ring slot holds.
//
// P is rounded to the type of the values' tile: bf16 for a bf16 cache, fp16 for codes (with v_scale; 2^beta, a power
// of two by each row's largest v scale in the tile, keeps that product in fp16's normal range).  Scores, maxima,
// sums and O are binary32.
//
// Bound.  Two tiles of rows by 80 keys at head_dim 128 are 1,470 clocks of the tensor pipe.  bf16, 8,192 tokens of 32
// heads of 128: 365 us at 2,070 MHz, 78 % of the measured bf16 rate, 389 us in a long run under the power cap (1,912 MHz):
// the tensor pipe, less the tiles on the diagonal, items' starts and ends.  Codes: the warps' issue slots (74 % taken; a
// softmax warp about 400 instructions a tile, of which 20 each for the two scales) at head_dim 128, 48 sequences, 948 us;
// the shared memory's bandwidth at 256, where a tile has one of rows and so twice the panels a product, 2,000 on 23,000
// tokens, 1,520 us (951 with a bf16 cache, which needs no conversion).
// Why 80 keys: probabilities that take the place of their scores (64 keys, the first kernel) hold the next scores back
// until their product is done; with 80 keys both have slots of their own beside O, which with an issuing warp for each
// tile of rows took the prompt from 477 to 417 us and the 48 sequences from 1,498 to 1,145.  Sixteen softmax warps
// instead of eight: 417 to 384 and 1,145 to 1,110.  Registers shared out among the warpgroups: 1,228 to 1,001.  Two
// producer warps: one needs 38 clocks a box, 110 in a busy quarter of the SM, more than the tensor pipe takes for a panel.
//
// Keys that a row must not see: their scores are replaced, not multiplied, and elements of V that are not finite are
// taken out of the tiles that the mask cuts (0 times infinity is not 0); rows that do see them get them back at the
// end.  Waits give up after 2 s (flag bit 2).
#include <math.h>

#include <cstring>
#include <type_traits>

#include "va_chunk.h"
#include "va_convert.cuh"

namespace va {
namespace {

constexpr uint64_t kWaitNs = 2000000000ull;
constexpr float kRescaleLog2 = 8.0f;
// The largest power of two that the values' scales are brought up by: a thread adds 20 probabilities of up to 2^(8 + beta)
// before the sum is scaled back, and 20 x 2^123 is the last that binary32 holds.
constexpr int kMaxBeta = 115;
// A raise of beta looks at what O holds, and leaves it below 2^kHeld (the products to come add 2^49 at most: p vs 2^beta
// is below 2^10, codes below 2^9).  Products that beta does not bring into fp16's reach then are below 2^-90 of what O holds.
constexpr int kHeld = 120;
constexpr int kScaleRing = 4;
constexpr int kBadRing = 16;   // tiles whose bad pages are remembered: more than the ring holds ahead
constexpr int kMaxStages = 8;
constexpr int kProducers = 2;  // warps that issue panels in turn: one alone takes longer than the tensor pipe needs for them

template <int D, int DT>
struct Cfg {
    static constexpr bool kQuant = DT != VA_BF16;
    static constexpr int kTiles = chunk_tiles(D);
    static constexpr int kKeys = kChunkKeys;
    static constexpr int kPages = kKeys / VA_PAGE_SIZE;
    static constexpr int kPanelD = D < 128 ? D : 128;
    static constexpr int kPanels = D / kPanelD;       // panels of a K or V tile
    static constexpr int kChunks = kPanelD / 64;      // 64-element chunks of a panel
    static constexpr int kChunkBytes = kKeys * 128;
    static constexpr int kPanelBytes = kChunks * kChunkBytes;
    static constexpr int kBits = DT == VA_BF16 ? 16 : DT == VA_INT4 ? 4 : DT == VA_INT2 ? 2 : 8;
    static constexpr int kRawRow = kPanelD * kBits / 8;  // bytes of a row of a raw panel
    static constexpr int kRawBytes = kKeys * kRawRow;
    static constexpr int kQChunk = kMmaRows * 128;       // 64-element chunk of a tile of q
    static constexpr int kQBytes = D / 64 * kQChunk;
    static constexpr int kStages = kQuant ? (D == 64 ? 6 : 5) : (D == 128 ? 7 : 8);
    // Even, so that a raw slot belongs to one producer and one dequant group: a barrier's parity tells a phase from the
    // next, not from the one after that, and nothing holds two producers or two groups within a ring of each other.
    // (The ring of whole panels is given back by the MMA warps, in order, so there the others cannot be a phase ahead.)
    static constexpr int kRawStages = kQuant ? (D == 64 ? 6 : 4) : 0;
    static_assert(kRawStages % 2 == 0 && kProducers == 2, "a slot's owner");
    static constexpr int kScaleFloats = 2 * kKeys + 4;   // k scales, v scales, the largest v scale of each dequant warp
    static constexpr int kSoftmaxWarps = 8 * kTiles;
    static constexpr int kDequantWarps = kQuant ? 8 : 0;  // two groups, which take panels in turn
    static constexpr int kProducerWarp = kSoftmaxWarps + kDequantWarps;  // and the ones behind it
    static constexpr int kMmaWarp = kProducerWarp + kProducers;          // one for each tile of rows
    static constexpr int kThreads = (kMmaWarp + kTiles + 3) / 4 * 128;  // whole warpgroups
    // Registers of a thread.  With dequant warps and two tiles of rows the block's even share is too few for a softmax
    // thread's scores; its warpgroups take what the others give back.
    static constexpr bool kShare = kQuant && kTiles == 2;
    static constexpr int kLaunchRegs = 65536 / kThreads / 8 * 8;
    static constexpr int kSoftmaxRegs = 88, kDequantRegs = 56, kOtherRegs = 40;
    static_assert(!kShare || (kSoftmaxWarps * kSoftmaxRegs + kDequantWarps * kDequantRegs + 4 * kOtherRegs) * 32 <=
                                 kThreads * kLaunchRegs, "registers that the block was launched with");
    static constexpr uint32_t kPCol = 2 * kKeys;                  // S slots at 0 and kKeys, P slots behind them
    static constexpr uint32_t kOCol = 3 * kKeys;
    static_assert(kOCol + kTiles * D <= 512, "tensor memory");
    static constexpr int kQ = 0;
    static constexpr int kConv = kTiles * kQBytes;
    static constexpr int kRaw = kConv + kStages * kPanelBytes;
    static constexpr int kScale = kRaw + kRawStages * kRawBytes;
    static constexpr int kBad = kScale + (kQuant ? kScaleRing * kScaleFloats * 4 : 0);
    static constexpr int kStats = kQuant ? 4 : 2;      // values of each row that the softmax hands from thread to thread
    static constexpr int kStat = kBad + kBadRing * 4;
    static constexpr int kBars = kStat + kTiles * kStats * kMmaRows * 4;
    static constexpr int kSmem = kBars + 64 * 8 + 1024;  // and slack for the alignment
    static_assert(kSmem <= (int)kMaxSmemPerBlock, "shared memory");
};

enum Bar : int {
    kFull = 0,                       // panel in the MMA's layout
    kEmpty = kFull + kMaxStages,     // and read
    kRawFull = kEmpty + kMaxStages,
    kRawEmpty = kRawFull + kMaxStages,
    kSFull = kRawEmpty + kMaxStages,  // scores of a slot
    kSRead = kSFull + 2,              // the softmax has them in registers
    kPFull = kSRead + 2,              // its probabilities
    kODone = kPFull + 2,              // its product with V
    kOFinal = kODone + 2,
    kQFull = kOFinal + 1,             // q from memory
    kQReady = kQFull + 1,             // q as the MMA takes it
    kScaleFree = kQReady + 1,
    kSwept = kScaleFree + kScaleRing,  // the softmax warps have gone through an edge tile's values
    kNumBars = kSwept + 1,
    kTmemSlot = 62,
    kPoison = 63,
};
static_assert(kNumBars <= kTmemSlot, "barrier block");

struct Args {
    CUtensorMap tm_q, tm_k, tm_v;  // 64-byte aligned members first
    ChunkParams p;
};

// Place of a V tile in the order in which tiles are used, K0 K1 V0 K2 V1 .. (the next scores are issued before the
// product), n tiles of keys; and the reverse, which tile, and whether it is V.
__device__ __forceinline__ int v_entry(int i, int n) { return i == n - 1 ? 2 * n - 1 : 2 * i + 2; }
__device__ __forceinline__ int entry_tile(int e, int n, bool &v) {
    if (e == 0) return v = false, 0;
    if (e == 2 * n - 1) return v = true, n - 1;
    v = !(e & 1);
    return v ? (e - 2) >> 1 : (e + 1) >> 1;
}

__device__ __forceinline__ bool half_finite(uint32_t w, uint32_t exponent) {  // both 16-bit elements of a word
    return (w & exponent) != exponent && ((w >> 16) & exponent) != exponent;
}

// Element d of a cached row, as a number (the slow path of values that are not finite).
template <int D, int DT>
__device__ float cached_value(const void *pages, const float *scale, size_t row, int d) {
    if constexpr (DT == VA_BF16) {
        return bf16_bits_to_float(static_cast<const uint16_t *>(pages)[row * D + d]);
    } else if constexpr (DT == VA_FP8_E4M3) {
        const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<const __nv_fp8_storage_t *>(pages)[row * D + d], __NV_E4M3);
        return __half2float(*reinterpret_cast<const __half *>(&h)) * scale[row];
    } else {
        return 0.f;  // codes are always finite
    }
}

template <int D, int DT>
__global__ void __launch_bounds__(Cfg<D, DT>::kThreads, 1) chunk_kernel(const __grid_constant__ Args args) {
    using C = Cfg<D, DT>;
    constexpr int kKeys = C::kKeys, kPages = C::kPages;
    const ChunkParams &p = args.p;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                            ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int i) { return sbase + C::kBars + 8u * i; };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    griddep_wait();
    const ChunkItem it = p.items[blockIdx.x];
    const int G = p.G, tpt = p.tpt;
    const bool two = C::kTiles == 2 && it.nt > tpt;  // both tiles of rows hold something
    const int nq = two ? 2 : 1;
    const int ntiles = (it.k_end - it.k_begin + kKeys - 1) / kKeys;
    const int lp0 = it.k_begin / VA_PAGE_SIZE;  // k_begin is a multiple of a tile
    const int npages = (it.k_end + VA_PAGE_SIZE - 1) / VA_PAGE_SIZE - lp0;
    const int32_t *bt = p.block_table + (size_t)it.b * p.bt_stride + lp0;

    if (warp == C::kProducerWarp && lane == 0) {
        prefetch_tensormap(&args.tm_q);
        prefetch_tensormap(&args.tm_k);
        prefetch_tensormap(&args.tm_v);
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(bar(kFull + i), C::kQuant ? 4 : 1);
            mbar_init(bar(kEmpty + i), nq);
            mbar_init(bar(kRawFull + i), 1);
            mbar_init(bar(kRawEmpty + i), C::kQuant ? 4 : 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(kSFull + i), 1);
            mbar_init(bar(kSRead + i), 8);
            mbar_init(bar(kPFull + i), 8);
            mbar_init(bar(kODone + i), 1);
        }
        mbar_init(bar(kOFinal), nq);
        mbar_init(bar(kQFull), 1);
        mbar_init(bar(kQReady), (C::kQuant ? 8 : 4) * nq);
        mbar_init(bar(kSwept), 8 * nq);
        for (int i = 0; i < kScaleRing; ++i) mbar_init(bar(kScaleFree + i), 8 * nq);
        sts_u32(bar(kPoison), 0u);
        fence_barrier_init();
    } else if (warp == C::kMmaWarp) {
        tmem_alloc(bar(kTmemSlot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = lds_u32(bar(kTmemSlot));
    bool ok = true;

    if (warp >= C::kProducerWarp) {
        if constexpr (C::kShare) regs_down<C::kOtherRegs>();
        if (warp < C::kMmaWarp) {
            // ------------------------------------------------------------ producers
            const int pw = warp - C::kProducerWarp;
            // q: one box of 64 elements x G heads x tpt tokens per tile of rows and chunk; tokens past q's end read 0
            if (pw == 0) {
                if (lane == 0) mbar_arrive_expect_tx(bar(kQFull), (uint32_t)(nq * (D / 64) * G * tpt * 128));
                __syncwarp();
                if (lane < nq * (D / 64)) {
                    const int q = lane / (D / 64), c = lane % (D / 64);
                    tma_load_3d(sbase + C::kQ + q * C::kQBytes + c * C::kQChunk, &args.tm_q, c * 64, it.kvh * G,
                                it.q0 + q * tpt, bar(kQFull));
                }
                __syncwarp();
            }
            constexpr int kRing = C::kQuant ? C::kRawStages : C::kStages;
            constexpr int kFullBar = C::kQuant ? kRawFull : kFull, kEmptyBar = C::kQuant ? kRawEmpty : kEmpty;
            const int total = 2 * ntiles * C::kPanels;
            int end = total;
            // page ids of a panel, alike in all lanes: one panel ahead
            int ids[kPages];
            auto load_ids = [&](int e) {
                bool v;
                const int i = e < total ? entry_tile(e / C::kPanels, ntiles, v) : ntiles;
#pragma unroll
                for (int pg = 0; pg < kPages; ++pg) ids[pg] = i * kPages + pg < npages ? __ldg(bt + i * kPages + pg) : 0;
            };
            load_ids(pw);
            for (int e = pw; e < total; e += kProducers) {
                bool v;
                const int i = entry_tile(e / C::kPanels, ntiles, v);
                const int pp = e % C::kPanels;
                const int npg = min(kPages, npages - i * kPages);
                uint32_t bads = 0;
                int page[kPages];
#pragma unroll
                for (int pg = 0; pg < kPages; ++pg) {
                    const bool bad = p.num_pages > 0 && (uint32_t)ids[pg] >= (uint32_t)p.num_pages;
                    bads |= bad ? 1u << pg : 0u;
                    page[pg] = bad ? 0 : ids[pg];
                }
                load_ids(e + kProducers);
                const int slot = e % kRing, use = e / kRing;
                if (use > 0) {
                    ok = __all_sync(0xffffffffu, mbar_wait(bar(kEmptyBar + slot), (use & 1) ^ 1, kWaitNs));
                    if (!ok) {
                        end = e;
                        break;
                    }
                }
                const CUtensorMap *map = v ? &args.tm_v : &args.tm_k;
                const uint32_t full = bar(kFullBar + slot);
                if (elect_one()) {
                    if (!v && pp == 0) {
                        sts_u32(sbase + C::kBad + 4u * (i % kBadRing), bads);
                        if (bads) atomicOr(p.flags, kFlagBadPage);
                    }
                    mbar_arrive_expect_tx(full, (uint32_t)npg * (C::kQuant ? VA_PAGE_SIZE * C::kRawRow
                                                                           : VA_PAGE_SIZE * 128 * C::kChunks));
#pragma unroll
                    for (int pg = 0; pg < kPages; ++pg) {
                        if (pg >= npg) break;
                        if constexpr (C::kQuant) {
                            tma_load_4d(sbase + C::kRaw + slot * C::kRawBytes + pg * VA_PAGE_SIZE * C::kRawRow, map,
                                        pp * C::kRawRow, it.kvh, 0, page[pg], full);
                        } else {
#pragma unroll
                            for (int c = 0; c < C::kChunks; ++c)
                                tma_load_4d(sbase + C::kConv + slot * C::kPanelBytes + c * C::kChunkBytes +
                                                pg * VA_PAGE_SIZE * 128,
                                            map, pp * C::kPanelD + c * 64, it.kvh, 0, page[pg], full);
                        }
                    }
                }
                __syncwarp();
            }
            // every issued copy lands before the CTA ends
            for (int e = max(0, end - kRing); e < end; ++e)
                if (e % kProducers == pw && !mbar_wait(bar(kFullBar + e % kRing), (e / kRing) & 1, kWaitNs)) ok = false;
            if (pw == 0 && !mbar_wait(bar(kQFull), 0, kWaitNs)) ok = false;
        } else {
            // ------------------------------------------------------------ MMA issue, by a whole warp
            const int w = warp - C::kMmaWarp;  // of two tiles of rows, the one that this warp issues
            if (w < nq) {
                constexpr int kAB = C::kQuant ? 0 : 1;
                constexpr uint32_t idS = idesc_f16(128, kKeys, kAB, 0, 0);
                constexpr uint32_t idO = idesc_f16(128, C::kPanelD, kAB, 0, 1);
                // K-major operands: 8-row groups 1024 bytes apart; V is MN-major, its 64-element chunks kChunkBytes apart
                constexpr uint32_t kHi = smem_desc_hi(1024, 2);
                const uint32_t qlo = smem_desc_lo(sbase + C::kQ + w * C::kQBytes, 16);
                const uint32_t klo = smem_desc_lo(sbase + C::kConv, 16);
                const uint32_t vlo = smem_desc_lo(sbase + C::kConv, C::kChunkBytes);
                int stage = 0, phase = 0;  // of the next panel
                auto pass = [&] {
                    if (++stage == C::kStages) stage = 0, phase ^= 1;
                };
                auto here = [&]() -> bool {  // the next panel
                    return __all_sync(0xffffffffu, mbar_wait(bar(kFull + stage), phase, kWaitNs));
                };
                auto here_and = [&](int b, int parity) -> bool {  // and another barrier
                    const bool done = __all_sync(
                        0xffffffffu, mbar_wait2(bar(kFull + stage), phase, bar(b), parity, kWaitNs));
                    tc_fence_after();
                    return done;
                };
                auto scores = [&](int slot) -> bool {  // of the next tile of keys, whose first panel is here
#pragma unroll
                    for (int pp = 0; pp < C::kPanels; ++pp) {
                        if (pp > 0 && !here()) return false;
                        if (elect_one()) {
                            const uint32_t kd = klo + (uint32_t)(stage * (C::kPanelBytes >> 4));
                            const uint32_t qd = qlo + (uint32_t)(pp * (C::kPanelD / 64 * C::kQChunk) >> 4);
#pragma unroll
                            for (int kk = 0; kk < C::kPanelD / 16; ++kk)
                                mma_ss_lo<kHi>(tmem + slot * kKeys, qd + (kk / 4) * (C::kQChunk >> 4) + (kk % 4) * 2,
                                               kd + (kk / 4) * (C::kChunkBytes >> 4) + (kk % 4) * 2, idS, pp > 0 || kk > 0);
                            if (pp == C::kPanels - 1) mma_commit(bar(kSFull + slot));
                            mma_commit(bar(kEmpty + stage));
                        }
                        __syncwarp();
                        pass();
                    }
                    return true;
                };
                auto product = [&](int slot, bool first) -> bool {
                    const uint32_t from = tmem + C::kPCol + slot * (kKeys / 2);
#pragma unroll
                    for (int pp = 0; pp < C::kPanels; ++pp) {
                        if (pp > 0 && !here()) return false;
                        if (elect_one()) {
                            const uint32_t vd = vlo + (uint32_t)(stage * (C::kPanelBytes >> 4));
#pragma unroll
                            for (int kk = 0; kk < kKeys / 16; ++kk)
                                mma_ts_lo<kHi>(tmem + C::kOCol + w * D + pp * C::kPanelD, from + kk * 8,
                                               vd + kk * (16 * 128 >> 4), idO, !first || kk > 0);
                            if (pp == C::kPanels - 1) mma_commit(bar(kODone + slot));
                            mma_commit(bar(kEmpty + stage));
                        }
                        __syncwarp();
                        pass();
                    }
                    return true;
                };
                ok = here_and(kQReady, 0);
                if (two) {
                    ok = ok && scores(w);
                    for (int i = 0; i < ntiles && ok; ++i) {
                        if (i + 1 < ntiles) ok = here_and(kSRead + w, i & 1) && scores(w);
                        ok = ok && here_and(kPFull + w, i & 1) && product(w, i == 0);
                    }
                } else {
                    ok = ok && scores(0) && (ntiles < 2 || (here() && scores(1)));
                    for (int k = 0; k < ntiles && ok; ++k) {
                        ok = here_and(kPFull + (k & 1), (k >> 1) & 1) && product(k & 1, k == 0);
                        if (ok && k + 2 < ntiles) ok = here() && scores(k & 1);
                    }
                }
                if (elect_one()) mma_commit(bar(kOFinal));
                __syncwarp();
                if (!__all_sync(0xffffffffu, mbar_wait(bar(kOFinal), 0, kWaitNs))) ok = false;
            }
        }
    } else if (warp < C::kSoftmaxWarps) {
        // ------------------------------------------------------------ softmax
        if constexpr (C::kShare) regs_up<C::kSoftmaxRegs>();
        const int w = warp >> 3;         // tile of rows
        const int h = (warp >> 2) & 1;   // half of the 32 rows of this quarter; half of the elements at the end
        const int r = (warp & 3) * 32 + lane;
        const int nt = max(0, min(tpt, it.nt - w * tpt));
        const bool row_ok = r < nt * G;
        if (w < nq) {
            const int token = w * tpt + r / G;  // of the item
            const int head = it.kvh * G + r % G;
            const int vis = it.vis0 + token;
            const uint32_t lane_tm = tmem + ((uint32_t)((warp & 3) * 32) << 16);
            const uint32_t stat = sbase + C::kStat + w * (C::kStats * kMmaRows * 4);
            // q as the MMA takes it: rows without a token are zero; for a cache of codes, fp16 scaled by a power of
            // two that brings the row's largest element into [2^14, 2^15)
            ok = __all_sync(0xffffffffu, mbar_wait(bar(kQFull), 0, kWaitNs));
            // Codes: two threads of a row, each half of its elements; else one, for the rows without a token.
            float prescale = 1.f;
            const uint32_t row = sbase + C::kQ + w * C::kQBytes;
            constexpr int kUnits = C::kQuant ? D / 16 : D / 8;
            auto unit = [&](int u) { return row + ((h * kUnits + u) / 8) * C::kQChunk + sw128(r, (h * kUnits + u) % 8); };
            if constexpr (C::kQuant) {
                float amax = 0.f;
                if (row_ok) {
#pragma unroll 2
                    for (int u = 0; u < kUnits; ++u) {
                        const uint4 x = lds_u4(unit(u));
                        const uint32_t ws[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            amax = fmaxf(amax, fmaxf(fabsf(bf16_bits_to_float(ws[e] & 0xFFFFu)),
                                                     fabsf(__uint_as_float(ws[e] & 0xFFFF0000u))));
                    }
                }
                sts_f32(stat + 4u * ((2 + h) * kMmaRows + r), amax);
                named_bar_sync(2 + w, 256);
                amax = fmaxf(amax, lds_f32(stat + 4u * ((3 - h) * kMmaRows + r)));
                if (amax > 0.f && amax < INFINITY)
                    prescale = __uint_as_float(min(254u, 268u - (__float_as_uint(amax) >> 23)) << 23);
            }
            if (!row_ok && (C::kQuant || h == 0)) {
#pragma unroll 2
                for (int u = 0; u < kUnits; ++u) sts_u4(unit(u), make_uint4(0, 0, 0, 0));
            } else if (C::kQuant && row_ok) {
#pragma unroll 2
                for (int u = 0; u < kUnits; ++u) {
                    const uint4 x = lds_u4(unit(u));
                    const uint32_t ws[4] = {x.x, x.y, x.z, x.w};
                    uint32_t y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        y[e] = pack_half2(bf16_bits_to_float(ws[e] & 0xFFFFu) * prescale,
                                          __uint_as_float(ws[e] & 0xFFFF0000u) * prescale);
                    sts_u4(unit(u), make_uint4(y[0], y[1], y[2], y[3]));
                }
            }
            if (h == 0) {
                sts_f32(stat + 4u * r, p.sm_scale_log2 / prescale);
                sts_u32(stat + 4u * (kMmaRows + r), (uint32_t)(row_ok ? vis : -1));
            }
            if (C::kQuant || h == 0) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kQReady));
            }
            named_bar_sync(2 + w, 256);  // the rows' data
            // this thread's rows of the warp's 16: lane / 4 and 8 further, as row x; its columns of each 8: c, c + 1
            const int c = 2 * (lane & 3);
            auto my_row = [&](int x) { return (warp & 3) * 32 + 16 * h + 8 * x + (lane >> 2); };
            const uint32_t half_tm = lane_tm + ((uint32_t)(16 * h) << 16);
            float c_r[2], m_run[2], l_run[2];
            int beta[2], seen[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                c_r[x] = lds_f32(stat + 4u * my_row(x));
                seen[x] = (int)lds_u32(stat + 4u * (kMmaRows + my_row(x)));
                m_run[x] = -INFINITY, l_run[x] = 0.f, beta[x] = 0;
            }
            constexpr int kU = kKeys / 8;
            const int first_vis = it.vis0 + w * tpt;  // of the tile's first token
            int swept = 0;
            for (int i = 0; i < ntiles && ok; ++i) {
                const int sl = two ? w : i & 1, ph = two ? i : i >> 1;
                ok = __all_sync(0xffffffffu, ok && mbar_wait(bar(kSFull + sl), ph & 1, kWaitNs));
                if (!ok) break;
                tc_fence_after();
                const int key0 = it.k_begin + i * kKeys;
                const uint32_t bads = lds_u32(sbase + C::kBad + 4u * (i % kBadRing));
                // an edge tile hides some key from some row of the item; both tiles of rows take the same view of it
                const bool edge = key0 + kKeys > it.k_end || key0 + kKeys - 1 > it.vis0 || bads != 0;
                const bool cut = edge && (key0 + kKeys > it.k_end || key0 + kKeys - 1 > first_vis || bads != 0);
                const uint32_t s_tm = half_tm + sl * kKeys;
                const uint32_t ring = sbase + C::kScale + (i % kScaleRing) * C::kScaleFloats * 4;
                uint32_t s[4 * kU];  // row x, unit u of 8 columns: s[4 u + 2 x], s[4 u + 2 x + 1]
                static_assert(kU == 10, "80 columns in two loads");
                tmem_ld_16x256b(s_tm, reinterpret_cast<uint32_t(&)[32]>(s[0]));
                tmem_ld_16x256b(s_tm + 64, reinterpret_cast<uint32_t(&)[8]>(s[32]));
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kSRead + sl));
                // raw scores times k scale, hidden keys at -inf, and the rows' maxima
                if constexpr (C::kQuant) {
#pragma unroll
                    for (int u = 0; u < kU; ++u) {
                        const uint2 sc = lds_u2(ring + 4u * (8 * u + c));
                        const uint64_t ks = f2_pack(sc.x, sc.y);
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            uint32_t *y = &s[4 * u + 2 * x];
                            f2_unpack(f2_mul(f2_pack(y[0], y[1]), ks), y[0], y[1]);
                        }
                    }
                }
                float mx[2], mv[2];
                if (cut) {  // rows' own maxima of the value scales too: of the keys that they see
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int last = min(seen[x], it.k_end - 1) - key0;
                        mv[x] = 0.f;
#pragma unroll
                        for (int u = 0; u < kU; ++u) {
                            const bool bad = (bads >> (u / 2)) & 1u;  // a page is two units
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                uint32_t &y = s[4 * u + 2 * x + e];
                                if (bad || 8 * u + c + e > last)
                                    y = 0xFF800000u;
                                else if (C::kQuant)
                                    mv[x] = fmaxf(mv[x], fabsf(lds_f32(ring + 4u * (kKeys + 8 * u + c + e))));
                            }
                        }
#pragma unroll
                        for (int o = 1; o <= 2; o <<= 1) mv[x] = fmaxf(mv[x], __shfl_xor_sync(0xffffffffu, mv[x], o));
                    }
                } else if constexpr (C::kQuant) {
                    const float4 y = lds_f4(ring + 8u * kKeys);
                    mv[0] = mv[1] = fmaxf(fmaxf(y.x, y.y), fmaxf(y.z, y.w));
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) mx[x] = -INFINITY;
#pragma unroll
                for (int u = 0; u < kU; ++u) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t *y = &s[4 * u + 2 * x];
                        mx[x] = fmax3(mx[x], __uint_as_float(y[0]), __uint_as_float(y[1]));
                    }
                }
#pragma unroll
                for (int o = 1; o <= 2; o <<= 1) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], o));
                }
                // does a row's maximum, or its value scales' power of two, have to move?
                bool move = false;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    mx[x] *= c_r[x];
                    move |= mx[x] > m_run[x] + kRescaleLog2;
                    if constexpr (C::kQuant) {
                        const float rr = mv[x] * __uint_as_float((uint32_t)(127 + beta[x]) << 23);
                        move |= !(rr >= 0x1p-6f && rr < 4.f);
                    }
                }
                // the product before this one: P's slot is free and O holds it
                if (two ? i > 0 : i > 1) {
                    if (!__all_sync(0xffffffffu, mbar_wait(bar(kODone + sl), (ph - 1) & 1, kWaitNs))) ok = false;
                    tc_fence_after();
                }
                if (__any_sync(0xffffffffu, move)) {
                    float fo[2];  // what O is multiplied by
                    bool raise = false;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        fo[x] = 1.f;
                        if (mx[x] > m_run[x] + kRescaleLog2) {
                            if (m_run[x] != -INFINITY) fo[x] = ex2_approx(m_run[x] - mx[x]);
                            m_run[x] = mx[x];
                            l_run[x] *= fo[x];
                        }
                        if (C::kQuant && mv[x] > 0.f && mv[x] < INFINITY) {
                            const float rr = mv[x] * __uint_as_float((uint32_t)(127 + beta[x]) << 23);
                            if (!(rr >= 0x1p-6f && rr < 4.f)) {
                                // mv in [2^(E-127), 2^(E-126)); beta at least -100, so that the sums, which take it, lose
                                // no key above 2^-26 of the largest (scales up to 2^107 then are in fp16's reach)
                                const int E = max(127 - kMaxBeta, min(227, (int)((__float_as_uint(mv[x]) >> 23) & 0xFFu)));
                                const int up = min(kHeld, 127 - E - beta[x]);  // down to -215: in two factors
                                fo[x] = fo[x] * __uint_as_float((uint32_t)(127 + (up >> 1)) << 23) *
                                        __uint_as_float((uint32_t)(127 + up - (up >> 1)) << 23);
                                beta[x] += up;
                                raise |= up > 0;
                            }
                        }
                    }
                    if (i > 0 && __any_sync(0xffffffffu, fo[0] != 1.f || fo[1] != 1.f)) {
                        // (of one tile, the product before this one is the one of the other slot)
                        if (!two &&
                            !__all_sync(0xffffffffu, mbar_wait(bar(kODone + ((i - 1) & 1)), ((i - 1) >> 1) & 1, kWaitNs)))
                            ok = false;
                        tc_fence_after();
                        if (C::kQuant && __any_sync(0xffffffffu, raise)) {
                            float top[2] = {0.f, 0.f};
#pragma unroll 1
                            for (int c0 = 0; c0 < D; c0 += 32) {
                                uint32_t o[16];
                                tmem_ld_16x256b(half_tm + C::kOCol + w * D + c0, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int j = 0; j < 16; ++j)
                                    top[(j >> 1) & 1] = fmaxf(top[(j >> 1) & 1], fabsf(__uint_as_float(o[j])));
                            }
#pragma unroll
                            for (int x = 0; x < 2; ++x) {  // a row's four lanes: what it holds is below 2^held
#pragma unroll
                                for (int n = 1; n <= 2; n <<= 1) top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], n));
                                const int held = (int)(__float_as_uint(top[x]) >> 23) + (int)(__float_as_uint(fo[x]) >> 23) - 252;
                                const int cut = max(0, min(126, held - kHeld));
                                fo[x] *= __uint_as_float((uint32_t)(127 - cut) << 23);
                                beta[x] -= cut;
                            }
                        }
#pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 32) {
                            const uint32_t at = half_tm + C::kOCol + w * D + c0;
                            uint32_t o[16];
                            tmem_ld_16x256b(at, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                o[j] = __float_as_uint(__uint_as_float(o[j]) * fo[(j >> 1) & 1]);
                            tmem_st_16x256b(at, o);
                        }
                        tmem_wait_st();
                    }
                }
                const uint32_t p_tm = half_tm + C::kPCol + sl * (kKeys / 2);
                auto give = [&](auto cut_tile) {
                    constexpr bool kCut = decltype(cut_tile)::value;
                    uint32_t pk[4];  // of two units
                    uint64_t ls[2] = {0ull, 0ull}, c2[2], nm2[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float nm = (m_run[x] == -INFINITY ? 0.f : -m_run[x]) + (float)beta[x];
                        c2[x] = f2_pack(__float_as_uint(c_r[x]), __float_as_uint(c_r[x]));
                        nm2[x] = f2_pack(__float_as_uint(nm), __float_as_uint(nm));
                    }
#pragma unroll
                    for (int u = 0; u < kU; ++u) {
                        uint64_t vs = 0ull;
                        if constexpr (C::kQuant) {
                            const uint2 sc = lds_u2(ring + 4u * (kKeys + 8 * u + c));
                            vs = f2_pack(sc.x, sc.y);
                        }
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            uint32_t a, b;
                            f2_unpack(f2_fma(f2_pack(s[4 * u + 2 * x], s[4 * u + 2 * x + 1]), c2[x], nm2[x]), a, b);
                            a = __float_as_uint(ex2_approx(__uint_as_float(a)));
                            b = __float_as_uint(ex2_approx(__uint_as_float(b)));
                            const uint64_t pr = f2_pack(a, b);
                            ls[x] = f2_add(ls[x], pr);
                            if constexpr (C::kQuant) {
                                f2_unpack(f2_mul(pr, vs), a, b);
                                if (kCut) {  // a hidden key's scale may be anything
                                    const int last = min(seen[x], it.k_end - 1) - key0;
                                    const bool bad = (bads >> (u / 2)) & 1u;
                                    if (bad || 8 * u + c > last) a = 0u;
                                    if (bad || 8 * u + c + 1 > last) b = 0u;
                                }
                                pk[2 * (u & 1) + x] = pack_half2(__uint_as_float(a), __uint_as_float(b));
                            } else {
                                pk[2 * (u & 1) + x] = pack_bf162(__uint_as_float(a), __uint_as_float(b));
                            }
                        }
                        if (u & 1) tmem_st_16x128b(p_tm + 4 * (u - 1), pk);
                    }
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        uint32_t a, b;
                        f2_unpack(ls[x], a, b);
                        l_run[x] += (__uint_as_float(a) + __uint_as_float(b)) * __uint_as_float((uint32_t)(127 - beta[x]) << 23);
                    }
                };
                if (C::kQuant && cut)
                    give(std::true_type{});
                else
                    give(std::false_type{});
                if constexpr (C::kQuant) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kScaleFree + i % kScaleRing));
                }
                tmem_wait_st();
                if (edge && (DT == VA_BF16 || DT == VA_FP8_E4M3)) {
                    // values that are not finite, in a tile that the mask cuts: out of the product (0 * inf is not 0).
                    // All softmax threads share the sweep and leave it together.
                    const int valid = min(kKeys, it.k_end - key0);
                    bool found = false;
                    // With two panels a tile (one-tile items) and five stages a panel's slot may have held one of the tile
                    // before, which these scores do not show to be done: so that the wait's parity means this panel.
                    if (C::kPanels > 1 && i > 0 &&
                        !__all_sync(0xffffffffu, mbar_wait(bar(kODone + ((i - 1) & 1)), ((i - 1) >> 1) & 1, kWaitNs)))
                        ok = false;
                    for (int pp = 0; pp < C::kPanels; ++pp) {
                        const int e = v_entry(i, ntiles) * C::kPanels + pp, slot = e % C::kStages;
                        if (!__all_sync(0xffffffffu, mbar_wait(bar(kFull + slot), (e / C::kStages) & 1, kWaitNs))) ok = false;
                        const uint32_t panel = sbase + C::kConv + slot * C::kPanelBytes;
                        for (int u = w * 256 + h * 128 + r; u < kKeys * C::kPanelD / 8; u += nq * 256) {
                            const int row = u / (C::kPanelD / 8), cu = u % (C::kPanelD / 8);
                            const uint32_t a = panel + (cu / 8) * C::kChunkBytes + sw128(row, cu % 8);
                            constexpr uint32_t kExp = DT == VA_BF16 ? 0x7F80u : 0x7C00u;
                            uint4 x = lds_u4(a);
                            if (row >= valid) {
                                sts_u4(a, make_uint4(0, 0, 0, 0));
                            } else if (!(half_finite(x.x, kExp) && half_finite(x.y, kExp) && half_finite(x.z, kExp) &&
                                         half_finite(x.w, kExp))) {
                                uint32_t ws[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                                for (int n = 0; n < 4; ++n) {
                                    if ((ws[n] & kExp) == kExp) ws[n] &= 0xFFFF0000u;
                                    if (((ws[n] >> 16) & kExp) == kExp) ws[n] &= 0x0000FFFFu;
                                }
                                sts_u4(a, make_uint4(ws[0], ws[1], ws[2], ws[3]));
                                found = true;
                            }
                        }
                    }
                    if (found) sts_u32(bar(kPoison), 1u);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kSwept));
                    if (!__all_sync(0xffffffffu, mbar_wait(bar(kSwept), swept & 1, kWaitNs))) ok = false;
                    ++swept;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kPFull + sl));
            }
            // the rows' sums over the four lanes that share them, and all of a row to its own lane
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int o = 1; o <= 2; o <<= 1) l_run[x] += __shfl_xor_sync(0xffffffffu, l_run[x], o);
                if ((lane & 3) == 0) {
                    sts_f32(stat + 4u * my_row(x), m_run[x]);
                    sts_f32(stat + 4u * (kMmaRows + my_row(x)), l_run[x]);
                    if (C::kQuant) sts_u32(stat + 4u * (2 * kMmaRows + my_row(x)), (uint32_t)beta[x]);
                }
            }
            named_bar_sync(2 + w, 256);  // a row's lane is in another warp, or in two
            const float m_row = lds_f32(stat + 4u * r), l_row = lds_f32(stat + 4u * (kMmaRows + r));
            const int beta_row = !C::kQuant ? 0 : (int)lds_u32(stat + 4u * (2 * kMmaRows + r));
            // epilogue
            if (!__all_sync(0xffffffffu, mbar_wait(bar(kOFinal), 0, kWaitNs))) ok = false;
            tc_fence_after();
            const bool poison = lds_u32(bar(kPoison)) != 0;
            const float inv = l_row == 0.f ? 0.f : (1.f / l_row) * __uint_as_float((uint32_t)(127 - beta_row) << 23);
            const float lse = l_row == 0.f ? -INFINITY : (m_row + log2f(l_row)) * 0.69314718055994531f;
            const size_t orow = (size_t)(it.q0 + token) * p.Hq + head;
            if (row_ok && ok && h == 0) {
                if (it.part < 0) {
                    if (p.lse) p.lse[orow] = lse;
                } else {
                    p.lse_part[(size_t)(it.part + w) * kMmaRows + r] = lse;
                }
            }
            // what was taken out comes back to the rows that see it
            auto give_back = [&](int d) -> float {
                float add = 0.f;
                for (int i = 0; i < ntiles; ++i) {
                    const int key0 = it.k_begin + i * kKeys;
                    bool edge = key0 + kKeys > it.k_end || key0 + kKeys - 1 > it.vis0;
                    for (int n = 0; n < kPages && !edge; ++n) {
                        const int page = bt[i * kPages + n];
                        edge = p.num_pages > 0 && (page < 0 || page >= p.num_pages);
                    }
                    if (!edge) continue;
                    for (int key = key0; key < min(key0 + kKeys, min(it.k_end, vis + 1)); ++key) {
                        const int page = bt[key / VA_PAGE_SIZE - lp0];
                        if (page < 0 || (p.num_pages > 0 && page >= p.num_pages)) continue;
                        const float x = cached_value<D, DT>(
                            p.v_pages, p.v_scale, ((size_t)page * VA_PAGE_SIZE + key % VA_PAGE_SIZE) * p.Hkv + it.kvh, d);
                        if (!(fabsf(x) < INFINITY)) add += x;
                    }
                }
                return add;
            };
            if (it.part < 0) {
                // bf16 rows staged over this tile of q, units exchanged by row, then written 16 bytes a lane
                const uint32_t stage = sbase + C::kQ + w * C::kQBytes;
                auto unit = [&](int row, int u) { return stage + row * (D * 2) + (((u & ~7) | ((u ^ row) & 7)) << 4); };
#pragma unroll 1
                for (int c0 = h * (D / 2); c0 < (h + 1) * (D / 2); c0 += 32) {
                    uint32_t o[32];
                    tmem_ld32(lane_tm + C::kOCol + w * D + c0, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * inv);
                    if (poison && row_ok) {
#pragma unroll 1
                        for (int j = 0; j < 32; ++j) {
                            const float add = give_back(c0 + j);
                            if (add != 0.f) {
#pragma unroll
                                for (int n = 0; n < 32; ++n)
                                    if (n == j) o[n] = __float_as_uint(__uint_as_float(o[n]) + add);
                            }
                        }
                    }
#pragma unroll
                    for (int n = 0; n < 4; ++n)
                        sts_u4(unit(r, c0 / 8 + n),
                               make_uint4(pack_bf162(__uint_as_float(o[8 * n]), __uint_as_float(o[8 * n + 1])),
                                          pack_bf162(__uint_as_float(o[8 * n + 2]), __uint_as_float(o[8 * n + 3])),
                                          pack_bf162(__uint_as_float(o[8 * n + 4]), __uint_as_float(o[8 * n + 5])),
                                          pack_bf162(__uint_as_float(o[8 * n + 6]), __uint_as_float(o[8 * n + 7]))));
                }
                named_bar_sync(2 + w, 256);
                if (ok) {
                    for (int e = h * 128 + r; e < nt * G * (D / 8); e += 256) {
                        const int row = e / (D / 8), u = e % (D / 8);
                        const size_t to = (size_t)(it.q0 + w * tpt + row / G) * p.Hq + it.kvh * G + row % G;
                        reinterpret_cast<uint4 *>(p.out)[to * (D / 8) + u] = lds_u4(unit(row, u));
                    }
                }
            } else {
                float *o_part = p.o_part + (size_t)(it.part + w) * D * kMmaRows + r;
#pragma unroll 1
                for (int c0 = h * (D / 2); c0 < (h + 1) * (D / 2); c0 += 32) {
                    uint32_t o[32];
                    tmem_ld32(lane_tm + C::kOCol + w * D + c0, o);
                    tmem_wait_ld();
                    if (!row_ok || !ok) continue;
#pragma unroll
                    for (int j = 0; j < 32; ++j) o_part[(size_t)(c0 + j) * kMmaRows] = __uint_as_float(o[j]) * inv;
#pragma unroll 1
                    for (int j = 0; poison && j < 32; ++j) {
                        const float add = give_back(c0 + j);
                        if (add != 0.f) o_part[(size_t)(c0 + j) * kMmaRows] += add;
                    }
                }
            }
        }
    } else if constexpr (C::kQuant) {
        // ------------------------------------------------------------ dequant
        if constexpr (C::kShare) regs_down<C::kDequantRegs>();
        // A panel is 16-element pieces; each thread takes kPer of them, kStep rows (a multiple of the swizzle's 8) apart.
        constexpr int kPieces = C::kPanelD / 16;  // of a row
        constexpr int kPer = (kKeys * kPieces + 127) / 128;
        constexpr int kStep = 128 / kPieces;
        constexpr int kPieceBytes = C::kBits * 2;
        static_assert(kStep % 8 == 0, "rows apart");
        constexpr bool kEven = kKeys * kPieces % 128 == 0;  // else some threads have one less
        const int dt = (tid - C::kSoftmaxWarps * 32) & 127;  // in the group, also the key whose scales it carries
        const int group = (warp - C::kSoftmaxWarps) >> 2;
        const int n0 = dt / kPieces, d0 = (dt % kPieces) * 16;
        // In odd chunks the piece's second half goes first, so that a quarter of a warp hits no bank twice: the raw words
        // are exchanged, not the stores' order, which would be a branch within the warp and twice the stores.
        const bool odd = (d0 / 64) & 1;
        const uint32_t first_at = (d0 / 64) * C::kChunkBytes + sw128(n0, (d0 % 64) / 8 + (odd ? 1 : 0));
        const uint32_t second_at = (d0 / 64) * C::kChunkBytes + sw128(n0, (d0 % 64) / 8 + (odd ? 0 : 1));
        // The scales of a tile of keys go with its first K panel.  Of one panel a tile that is group 0 for tile 0 and
        // group 1 for the others (K0 K1 V0 K2 V1 ..), of two panels always group 0.
        const int first = C::kPanels == 1 ? group : 0;
        const int beyond = C::kPanels == 1 ? (group == 0 ? 1 : ntiles) : (group == 0 ? ntiles : 0);
        auto load_id = [&](int i) -> int {
            const int n = i * kPages + dt / VA_PAGE_SIZE;
            if (dt >= kKeys || i >= beyond || i >= ntiles || n >= npages || it.k_begin + i * kKeys + dt >= it.k_end) return -1;
            const int page = __ldg(bt + n);
            return p.num_pages > 0 && page >= p.num_pages ? -1 : page;
        };
        auto load_scale = [&](const float *from, int page) -> float {
            return page < 0 ? 0.f : __ldg(from + ((size_t)page * VA_PAGE_SIZE + dt % VA_PAGE_SIZE) * p.Hkv + it.kvh);
        };
        // scales two tiles ahead, page ids three
        int id0 = load_id(first), id1 = load_id(first + 1), id2 = load_id(first + 2);
        float ks0 = load_scale(p.k_scale, id0), vs0 = load_scale(p.v_scale, id0);
        float ks1 = load_scale(p.k_scale, id1), vs1 = load_scale(p.v_scale, id1);
        constexpr int kRawN = C::kRawStages ? C::kRawStages : 1;
        const int total = 2 * ntiles * C::kPanels;
        for (int e = group; e < total && ok; e += 2) {
            bool v;
            const int i = entry_tile(e / C::kPanels, ntiles, v);
            const int rs = e % kRawN, slot = e % C::kStages;
            if (!mbar_wait(bar(kRawFull + rs), (e / kRawN) & 1, kWaitNs)) { ok = false; break; }
            const uint32_t src = sbase + C::kRaw + rs * C::kRawBytes + dt * kPieceBytes;
            const uint32_t dst = sbase + C::kConv + slot * C::kPanelBytes;
            RawPiece<DT> raw[kPer];
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if (kEven || n0 + j * kStep < kKeys) raw[j].load(src + j * 128 * kPieceBytes);
            // The loads are done before the slot is given back: nothing below needs their values before the arrival, which
            // does not wait for them by itself, and with a cold TLB the copy of a later panel came first.
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kRawEmpty + rs));
            const int nvalid = it.k_end - (it.k_begin + i * kKeys);
            if (e / C::kStages > 0 &&
                !mbar_wait(bar(kEmpty + slot), ((e / C::kStages) & 1) ^ 1, kWaitNs)) { ok = false; break; }
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                if (!kEven && n0 + j * kStep >= kKeys) break;
                uint32_t h[8];
                raw[j].exchange(odd);
                raw[j].to_half(h);
                if (n0 + j * kStep >= nvalid) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) h[k] = 0;
                }
                const uint32_t at = dst + j * kStep * 128;
                sts_u4(at + first_at, make_uint4(h[0], h[1], h[2], h[3]));
                sts_u4(at + second_at, make_uint4(h[4], h[5], h[6], h[7]));
            }
            if (!v && e % C::kPanels == 0) {
                if (i >= kScaleRing &&
                    !mbar_wait(bar(kScaleFree + i % kScaleRing), ((i / kScaleRing) & 1) ^ 1, kWaitNs)) { ok = false; break; }
                const uint32_t ring = sbase + C::kScale + (i % kScaleRing) * C::kScaleFloats * 4;
                if (dt < kKeys) {
                    sts_f32(ring + 4u * dt, ks0);
                    sts_f32(ring + 4u * (kKeys + dt), vs0);
                }
                const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(vs0)));
                if (lane == 0) sts_u32(ring + 4u * (2 * kKeys + dt / 32), top);
                ks0 = ks1, vs0 = vs1;
                ks1 = load_scale(p.k_scale, id2), vs1 = load_scale(p.v_scale, id2);
                id2 = load_id(i + 3);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kFull + slot));
        }
    }

    if (!ok) atomicOr(p.flags, kFlagTimeoutBit);
    tc_fence_before();
    __syncthreads();
    if (warp == C::kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Log-sum-exp merge of a tile's partials.  A CTA takes kCols elements of all 128 rows: thread = row, so that the partials
// (rows innermost) are read in whole segments; the merged piece goes through shared memory, so that rows of `out` are
// written in pieces of kCols elements.  kWays threads share a row's partials: one after the other, each waiting for its
// loads, ten partials of a question of 45 tokens (24 heads of 256) took longer than the attention itself, 30 us in all
// against 22 with 8 x 4.  A merge that fills the GPU prefers wider pieces and fewer ways: 384 tiles' 5 partials, 2,000
// tokens on 23,000, took 1,523 us in all with 8 x 4, 1,495 with 16 x 1, 1,485 with 16 x 2.  The border is where the CTAs of
// the second are four to an SM.  Verify blocks of 16 on 6,000 tokens, whole calls, 8 x 4 against 16 x 2, by tiles times
// pieces of 16: head_dim 64, bf16: 32: 15 and 27 us, 320: 41 and 43, 512: 51.3 both, 768: 82 and 80; 128, int8: 64: 19 and 29,
// 256: 27 and 29, 512: 53.3 both, 768: 70 and 68, 1,408: 162 and 155; 256, int8: 64: 23 and 41, 512: 46 and 45, 640: 59.5 both,
// 1,024: 83 and 80, 2,048: 134 and 125.
template <int kCols, int kWays>
__global__ void __launch_bounds__(kMmaRows * kWays) chunk_combine_kernel(const ChunkCombineParams p) {
    __shared__ uint32_t tile[kMmaRows][kCols / 2 + 1];
    __shared__ float part[kWays - 1][kCols][kMmaRows], top[kWays][kMmaRows], sum[kWays][kMmaRows];
    griddep_wait();
    const ChunkGroup g = p.groups[blockIdx.x];
    const int r = threadIdx.x % kMmaRows, w = threadIdx.x / kMmaRows, d0 = blockIdx.y * kCols;
    const int rows = g.nt * p.G;
    const size_t step = (size_t)g.step * kMmaRows;
    float m = -INFINITY, z = 0.f, acc[kCols] = {};
    if (r < rows) {
        const float *lse = p.lse_part + (size_t)g.first_part * kMmaRows + r;
        const float *o = p.o_part + ((size_t)g.first_part * p.D + d0) * kMmaRows + r;
        for (int n = w; n < g.n; n += kWays) {
            const float l = lse[n * step];
            float x[kCols];
#pragma unroll
            for (int d = 0; d < kCols; ++d) x[d] = o[n * step * p.D + d * kMmaRows];
            if (l == -INFINITY) continue;  // no keys: the partial has zeros, or nothing
            const float to = fmaxf(m, l), e = expf(l - to), old = m == -INFINITY ? 0.f : expf(m - to);
            m = to;
            z = z * old + e;
#pragma unroll
            for (int d = 0; d < kCols; ++d) acc[d] = fmaf(acc[d], old, e * x[d]);
        }
    }
    top[w][r] = m;
    __syncthreads();
    float M = top[0][r];
#pragma unroll
    for (int i = 1; i < kWays; ++i) M = fmaxf(M, top[i][r]);
    const float e = m == -INFINITY ? 0.f : expf(m - M);
    sum[w][r] = z * e;
    if (w > 0) {
#pragma unroll
        for (int d = 0; d < kCols; ++d) part[w - 1][d][r] = acc[d] * e;
    }
    __syncthreads();
    if (w == 0 && r < rows) {
        z = sum[0][r];
#pragma unroll
        for (int i = 1; i < kWays; ++i) z += sum[i][r];
        const float inv = z == 0.f ? 0.f : 1.f / z;
#pragma unroll
        for (int d = 0; d < kCols; ++d) {
            acc[d] *= e;
#pragma unroll
            for (int i = 1; i < kWays; ++i) acc[d] += part[i - 1][d][r];
        }
#pragma unroll
        for (int d = 0; d < kCols / 2; ++d) tile[r][d] = pack_bf162(acc[2 * d] * inv, acc[2 * d + 1] * inv);
        if (blockIdx.y == 0 && p.lse)
            p.lse[(size_t)(g.q0 + r / p.G) * p.Hq + g.kvh * p.G + r % p.G] = z == 0.f ? -INFINITY : M + logf(z);
    }
    __syncthreads();
    constexpr int kUnits = kCols / 8;
    for (int i = threadIdx.x; i < rows * kUnits; i += kMmaRows * kWays) {
        const int row = i / kUnits, u = i % kUnits;
        const size_t to = (size_t)(g.q0 + row / p.G) * p.Hq + g.kvh * p.G + row % p.G;
        reinterpret_cast<uint4 *>(p.out)[(to * p.D + d0) / 8 + u] =
            make_uint4(tile[row][4 * u], tile[row][4 * u + 1], tile[row][4 * u + 2], tile[row][4 * u + 3]);
    }
}

// A page pool [pages, 16, Hkv, row] by boxes of one page and head: 64 elements (bf16, swizzled) or one panel's bytes.
bool make_cache_map(CUtensorMap *m, const void *base, int D, int bits, int box_row, int Hkv, int num_pages) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const bool bf16 = bits == 16;
    const cuuint64_t bytes = (cuuint64_t)D * bits / 8;
    const cuuint64_t pages = num_pages > 0 ? (cuuint64_t)num_pages : (cuuint64_t)1 << 30;
    cuuint64_t dims[4] = {bf16 ? (cuuint64_t)D : bytes, (cuuint64_t)Hkv, (cuuint64_t)VA_PAGE_SIZE, pages};
    cuuint64_t strides[3] = {bytes, bytes * Hkv, bytes * Hkv * VA_PAGE_SIZE};
    cuuint32_t box[4] = {(cuuint32_t)box_row, 1u, (cuuint32_t)VA_PAGE_SIZE, 1u};
    cuuint32_t one[4] = {1, 1, 1, 1};
    return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(base),
               dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               bf16 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int DT>
cudaError_t launch_one(const ChunkParams &p, const va_heads &q, int N, int n, cudaStream_t s) {
    using C = Cfg<D, DT>;
    Args a;
    a.p = p;
    const int box = C::kQuant ? C::kRawRow : 64;
    if (!make_q_map(&a.tm_q, q, N, D, p.G, p.tpt) ||
        !make_cache_map(&a.tm_k, p.k_pages, D, C::kBits, box, p.Hkv, p.num_pages) ||
        !make_cache_map(&a.tm_v, p.v_pages, D, C::kBits, box, p.Hkv, p.num_pages))
        return cudaErrorInvalidValue;
    auto k = chunk_kernel<D, DT>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(k, dim3(n), dim3(C::kThreads), C::kSmem, s, a);
}

template <int D>
cudaError_t launch_d(const ChunkParams &p, const va_heads &q, int N, int dtype, int n, cudaStream_t s) {
    switch (dtype) {
    case VA_BF16: return launch_one<D, VA_BF16>(p, q, N, n, s);
    case VA_FP8_E4M3: return launch_one<D, VA_FP8_E4M3>(p, q, N, n, s);
    case VA_INT8: return launch_one<D, VA_INT8>(p, q, N, n, s);
    case VA_INT4: return launch_one<D, VA_INT4>(p, q, N, n, s);
    default: return launch_one<D, VA_INT2>(p, q, N, n, s);
    }
}

}  // namespace

cudaError_t launch_chunk(const ChunkParams &p, const va_heads &q, int N, int D, int dtype, int num_items, cudaStream_t s) {
    if (num_items <= 0) return cudaSuccess;
    switch (D) {
    case 64: return launch_d<64>(p, q, N, dtype, num_items, s);
    case 128: return launch_d<128>(p, q, N, dtype, num_items, s);
    default: return launch_d<256>(p, q, N, dtype, num_items, s);
    }
}

cudaError_t launch_chunk_combine(const ChunkCombineParams &p, int num_groups, int num_sms, cudaStream_t s) {
    if (num_groups * (p.D / 16) <= 4 * num_sms)
        return launch_pdl(chunk_combine_kernel<8, 4>, dim3(num_groups, p.D / 8), dim3(kMmaRows * 4), 0, s, p);
    return launch_pdl(chunk_combine_kernel<16, 2>, dim3(num_groups, p.D / 16), dim3(kMmaRows * 2), 0, s, p);
}

}  // namespace va
