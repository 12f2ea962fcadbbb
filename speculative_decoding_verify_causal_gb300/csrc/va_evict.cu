// Eviction from the paged cache by the weight that its tokens have gathered.
//
// Every kv head of a sequence keeps the same number of tokens but chooses them for itself: first those that are
// protected (the oldest and the newest positions), then the heaviest, of equal ones the lower slot.  The kept tokens
// have to end up in the first `keep` slots.  Order does not matter to attention, so only as many rows move as must:
// the k-th kept slot from `keep` on goes to the k-th slot below it whose token goes.  Sources and destinations are
// disjoint, so all rows move at once and in place.
//
// Two kernels.  The first takes a cluster of up to 8 CTAs for each sequence and kv head: the weights as integers of
// the same order, three rounds of a histogram of 11, 11 and 10 bits give the keep-th largest, and counts before each
// CTA's and warp's slots give the places in the list of moves.  The second moves the rows.  Whole numbers throughout:
// the result does not depend on timing.
//
// Bound: latency.  4 sequences of 25,000 slots, 4 heads of 256, int8, cut to 4,096: 20 us for both kernels, 8.7 us of
// bytes at the copy rate; most is the chain of the first one: a read of the weights (kept in shared memory as integers),
// three rounds with two cluster barriers each, one exchange of counts (with the weights read again in each of six
// passes and two exchanges more: 36 us).  Each CTA adds up a share of the bins and tells the others: eight times fewer remote reads than all of them
// by all.  Two kernels, since eight CTAs of a head cannot move long lists of rows at the copy rate.
#include <math.h>

#include <algorithm>

#include "va_internal.h"
#include "va_sm100.cuh"

namespace va {

struct EvictParams {
    uint4 *k_pages, *v_pages;
    float *k_scale, *v_scale;
    const int32_t *block_table, *seq_lens, *keep, *recent_from, *ref_count;
    float *weights;
    int32_t *slot_pos, *new_lens, *flags;
    int64_t stride_seq, stride_head;
    int2 *moves;     // [num_seqs * Hkv][half]: from, to
    int32_t *count;  // [num_seqs * Hkv]
    int bt_stride, num_seqs, Hkv, num_pages, num_sinks, cluster, half, slots;
    int units;   // 16-byte units of a row
    int cached;  // slots of a CTA whose weights lie in shared memory
};

namespace {

using namespace sm100;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMoveThreads = 256;
constexpr int kMaxCluster = 8;
constexpr int kMaxCached = 40960;  // 160 KB

// Weights in an order of unsigned integers: NaN lowest, then -inf .. +inf; protected tokens above all.
__device__ __forceinline__ uint32_t weight_order(float x) {
    if (x != x) return 0u;
    const uint32_t b = __float_as_uint(x + 0.f);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ void st_cluster_u32(const void *local, uint32_t rank, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_map(local, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster_u32(const void *local, uint32_t rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_map(local, rank)) : "memory");
    return v;
}

// What a warp's slots hold: above the threshold from `keep` on and below it under `keep`, and at it on either side.
struct Counts {
    int up, down, tied_low, tied_high;
    __device__ __forceinline__ void add(const Counts &x) {
        up += x.up, down += x.down, tied_low += x.tied_low, tied_high += x.tied_high;
    }
};

__global__ void __launch_bounds__(kThreads) evict_select_kernel(const EvictParams p) {
    extern __shared__ uint32_t keys[];
    __shared__ uint32_t bins[kBins], total[kBins];
    __shared__ uint32_t warp_sum[kWarps], found[2];
    __shared__ Counts of_warp[kWarps], of_cta;
    __shared__ int bad;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ranks = p.cluster, rank = (int)(blockIdx.x % ranks);
    const int bg = blockIdx.x / ranks, b = bg / p.Hkv, g = bg % p.Hkv;
    griddep_wait();
    auto sync = [&] {
        if (ranks > 1)
            cluster_sync();
        else
            __syncthreads();
    };
    const int L = p.seq_lens[b], want = p.keep[b];
    const int32_t *bt = p.block_table + (size_t)b * p.bt_stride;
    // requests that are not carried out: the sequence stays as it is
    const int wrong = L < 0 || L > p.slots || (int64_t)L > (int64_t)p.bt_stride * VA_PAGE_SIZE ? VA_PAGES_BAD_REQUEST : 0;
    if (wrong || want < 0 || want >= L) {  // alike in all CTAs of the cluster
        if (rank == 0 && tid == 0) {
            if (wrong && p.flags) atomicOr(p.flags, wrong);
            p.new_lens[b] = L;  // the same from every head
            p.count[bg] = 0;
        }
        return;
    }

    const int64_t row = b * p.stride_seq + g * p.stride_head;
    const float *weights = p.weights + row;
    const int recent = p.recent_from ? p.recent_from[b] : 0x7FFFFFFF;
    // a CTA's slots, whole warps' worth
    const int per = ((L + ranks - 1) / ranks + 31) / 32 * 32;
    const int s0 = min(L, rank * per), s1 = min(L, s0 + per), cached = min(s1, s0 + p.cached);
    auto order = [&](int s) -> uint32_t {
        const int pos = p.slot_pos ? p.slot_pos[row + s] : s;
        const uint32_t o = weight_order(weights[s]);
        return pos < p.num_sinks || pos >= recent ? 0xFFFFFFFFu : o;
    };
    auto key = [&](int s) { return s < cached ? keys[s - s0] : order(s); };
#pragma unroll 8
    for (int s = s0 + tid; s < cached; s += kThreads) keys[s - s0] = order(s);
    if (tid == 0) bad = 0;
    for (int i = tid; i < kBins; i += kThreads) bins[i] = 0;
    __syncthreads();
    for (int i = rank * kThreads + tid; i < (L + VA_PAGE_SIZE - 1) / VA_PAGE_SIZE; i += ranks * kThreads) {
        const int page = bt[i];
        if (page < 0 || (p.num_pages > 0 && page >= p.num_pages))
            atomicOr(&bad, VA_PAGES_BAD_ENTRY);
        else if (p.ref_count && p.ref_count[page] > 1)
            atomicOr(&bad, VA_PAGES_BAD_REQUEST);
    }

    // the keep-th largest: from the top, the digit in which the count reaches `left`
    uint32_t prefix = 0, mask = 0;
    int left = want;
    for (int round = 0; round < 3 && want > 0; ++round) {
        const int shift = round == 0 ? 21 : round == 1 ? 10 : 0, width = round == 2 ? 10 : 11, n = 1 << width;
#pragma unroll 4
        for (int s = s0 + tid; s < s1; s += kThreads) {
            const uint32_t o = key(s);
            if ((o & mask) == prefix) atomicAdd(&bins[(o >> shift) & (n - 1)], 1u);
        }
        sync();
        const uint32_t *sums = bins;
        if (ranks > 1) {
            // each CTA adds up its share of the bins and tells all of them
            const int share = n / ranks;
            for (int i = tid; i < share; i += kThreads) {
                uint32_t t = 0;
#pragma unroll
                for (int q = 0; q < kMaxCluster; ++q)
                    if (q < ranks) t += ld_cluster_u32(&bins[rank * share + i], q);
#pragma unroll
                for (int q = 0; q < kMaxCluster; ++q)
                    if (q < ranks) st_cluster_u32(&total[rank * share + i], q, t);
            }
            cluster_sync();
            sums = total;
        }
        // from the top: thread t has bins n - 1 - each t ..
        const int each = n / kThreads;  // 4 or 2
        uint32_t mine = 0;
        for (int i = 0; i < each; ++i) mine += sums[n - 1 - (tid * each + i)];
        uint32_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        if (lane == 31) warp_sum[warp] = upto;
        __syncthreads();
        uint32_t before = upto - mine;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) before += i < warp ? warp_sum[i] : 0u;
        if (before < (uint32_t)left && before + mine >= (uint32_t)left) {
            uint32_t above = before;
            for (int i = 0; i < each; ++i) {
                const int bin = n - 1 - (tid * each + i);
                if (above + sums[bin] >= (uint32_t)left) {
                    found[0] = bin, found[1] = above;
                    break;
                }
                above += sums[bin];
            }
        }
        __syncthreads();
        prefix |= found[0] << shift;
        mask |= (uint32_t)(n - 1) << shift;
        left -= (int)found[1];
        for (int i = tid; i < kBins; i += kThreads) bins[i] = 0;
        __syncthreads();
    }
    // Kept: above the threshold, and of those at it the first `left`.  The places of a warp's moves and holes follow
    // from the counts before it: over the CTAs of lower rank and the warps of lower slots.
    const uint32_t threshold = prefix;
    const int each = ((s1 - s0 + kWarps - 1) / kWarps + 31) / 32 * 32;  // slots of a warp, one after the other
    const int w0 = min(s1, s0 + warp * each), w1 = min(s1, w0 + each);
    Counts mine = {0, 0, 0, 0};
    for (int s = w0 + lane; s < w1; s += 32) {
        const uint32_t o = key(s);
        const bool above = want > 0 && o > threshold, tie = want > 0 && o == threshold;
        mine.up += above && s >= want;
        mine.down += !above && !tie && s < want;
        mine.tied_low += tie && s < want;
        mine.tied_high += tie && s >= want;
    }
    mine.up = __reduce_add_sync(0xffffffffu, mine.up);
    mine.down = __reduce_add_sync(0xffffffffu, mine.down);
    mine.tied_low = __reduce_add_sync(0xffffffffu, mine.tied_low);
    mine.tied_high = __reduce_add_sync(0xffffffffu, mine.tied_high);
    if (lane == 0) of_warp[warp] = mine;
    __syncthreads();
    Counts before = {0, 0, 0, 0}, all = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        if (i < warp) before.add(of_warp[i]);
        all.add(of_warp[i]);
    }
    int refused = bad, low = all.tied_low;
    if (ranks > 1) {
        if (tid == 0) of_cta = all;
        cluster_sync();
#pragma unroll
        for (int q = 0; q < kMaxCluster; ++q) {
            if (q >= ranks || q == rank) continue;
            const int tied_low = ld_cluster_u32(&of_cta.tied_low, q);
            low += tied_low;
            refused |= ld_cluster_u32(&bad, q);
            if (q < rank)
                before.add({(int)ld_cluster_u32(&of_cta.up, q), (int)ld_cluster_u32(&of_cta.down, q), tied_low,
                            (int)ld_cluster_u32(&of_cta.tied_high, q)});
        }
        cluster_arrive();  // read: no CTA ends before cluster_wait
    }
    if (rank == 0 && tid == 0) {
        if (refused && p.flags) atomicOr(p.flags, refused);
        p.new_lens[b] = refused ? L : want;  // the same from every head
    }
    if (refused) {
        if (rank == 0 && tid == 0) p.count[bg] = 0;
    } else {
        const int high = max(0, left - low);  // kept of those at the threshold from `keep` on
        int ties_low = before.tied_low, ties_high = before.tied_high;
        int movers = before.up + min(ties_high, high), holes = before.down + ties_low - min(ties_low, left);
        for (int s = w0 + lane; s - lane < w1; s += 32) {
            const uint32_t o = s < w1 ? key(s) : 0u, lower = (1u << lane) - 1u;
            const bool tie = s < w1 && want > 0 && o == threshold;
            const uint32_t tl = __ballot_sync(0xffffffffu, tie && s < want), th = __ballot_sync(0xffffffffu, tie && s >= want);
            const bool kept = s < w1 && want > 0 &&
                              (o > threshold || (tie && (s < want ? ties_low + __popc(tl & lower) < left
                                                                  : ties_high + __popc(th & lower) < high)));
            const bool mover = kept && s >= want, hole = s < w1 && !kept && s < want;
            const uint32_t mv = __ballot_sync(0xffffffffu, mover), hl = __ballot_sync(0xffffffffu, hole);
            if (mover) p.moves[(size_t)bg * p.half + movers + __popc(mv & lower)].x = s;
            if (hole) p.moves[(size_t)bg * p.half + holes + __popc(hl & lower)].y = s;
            ties_low += __popc(tl), ties_high += __popc(th);
            movers += __popc(mv), holes += __popc(hl);
        }
        if (rank == ranks - 1 && warp == kWarps - 1 && lane == 0) p.count[bg] = movers;  // as many as holes
    }
    if (ranks > 1) cluster_wait();
}

// Rows of K and V: thread = 16 bytes of a row; scales, weights and positions with the row's first thread.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p) {
    griddep_wait();
    const int bg = blockIdx.y, b = bg / p.Hkv, g = bg % p.Hkv;
    const int n = p.count[bg];
    const int32_t *bt = p.block_table + (size_t)b * p.bt_stride;
    const int64_t row = b * p.stride_seq + g * p.stride_head;
    const int units = p.units;
    for (int64_t e = (int64_t)blockIdx.x * kMoveThreads + threadIdx.x; e < (int64_t)n * units;
         e += (int64_t)gridDim.x * kMoveThreads) {
        const int i = (int)(e / units), u = (int)(e % units);
        const int2 mv = p.moves[(size_t)bg * p.half + i];
        const size_t from = ((size_t)bt[mv.x / VA_PAGE_SIZE] * VA_PAGE_SIZE + mv.x % VA_PAGE_SIZE) * p.Hkv + g;
        const size_t to = ((size_t)bt[mv.y / VA_PAGE_SIZE] * VA_PAGE_SIZE + mv.y % VA_PAGE_SIZE) * p.Hkv + g;
        const uint4 k = p.k_pages[from * units + u], v = p.v_pages[from * units + u];
        p.k_pages[to * units + u] = k;
        p.v_pages[to * units + u] = v;
        if (u == 0) {
            if (p.k_scale) {
                p.k_scale[to] = p.k_scale[from];
                p.v_scale[to] = p.v_scale[from];
            }
            p.weights[row + mv.y] = p.weights[row + mv.x];
            if (p.slot_pos) p.slot_pos[row + mv.y] = p.slot_pos[row + mv.x];
        }
    }
}

}  // namespace
}  // namespace va

namespace {

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

}  // namespace

extern "C" {

size_t verify_attn_evict_workspace_bytes(int num_seqs, int num_kv_heads, int num_slots) {
    if (num_seqs < 1 || num_kv_heads < 1 || num_slots < 0 || num_slots > (1 << 30) ||
        (int64_t)num_seqs * num_kv_heads > 65535)
        return 0;
    const size_t heads = (size_t)num_seqs * num_kv_heads;
    return align_up(heads * 4) + heads * (num_slots / 2) * sizeof(int2) + 16;
}

int verify_attn_evict(void *k_pages, void *v_pages, float *k_scale, float *v_scale, va_kv_dtype kv_dtype,
                      const int32_t *block_table, int block_table_stride, const int32_t *seq_lens, int num_seqs,
                      int num_kv_heads, int head_dim, int num_pages, float *weights, int32_t *slot_pos,
                      int64_t stride_seq, int64_t stride_head, int num_slots, const int32_t *keep_lens, int num_sinks,
                      const int32_t *recent_from, const int32_t *ref_count, int32_t *new_lens, void *workspace,
                      int32_t *flags, void *stream) {
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return VA_ERR_UNSUPPORTED;
    if (kv_dtype < VA_BF16 || kv_dtype > VA_INT2) return VA_ERR_UNSUPPORTED;
    const size_t need = verify_attn_evict_workspace_bytes(num_seqs, num_kv_heads, num_slots);
    if (need == 0 || block_table_stride < 0 || num_pages < 0 || num_sinks < 0 || stride_seq < 0 || stride_head < 0 ||
        !k_pages || !v_pages || !block_table || !seq_lens || (!weights && num_slots > 0) || !keep_lens || !new_lens ||
        !workspace)
        return VA_ERR_INVALID_ARGUMENT;
    if (kv_dtype != VA_BF16 && (!k_scale || !v_scale)) return VA_ERR_INVALID_ARGUMENT;
    for (const void *x : {(const void *)k_pages, (const void *)v_pages, (const void *)workspace})
        if (reinterpret_cast<uintptr_t>(x) % 16) return VA_ERR_INVALID_ARGUMENT;
    for (const void *x : {(const void *)k_scale, (const void *)v_scale, (const void *)block_table, (const void *)seq_lens,
                          (const void *)weights, (const void *)slot_pos, (const void *)keep_lens, (const void *)recent_from,
                          (const void *)ref_count, (const void *)new_lens, (const void *)flags})
        if (reinterpret_cast<uintptr_t>(x) % 4) return VA_ERR_INVALID_ARGUMENT;
    if (va::rows_overlap(stride_seq, stride_head, num_seqs, num_kv_heads, num_slots))
        return VA_ERR_INVALID_ARGUMENT;
    // every head of a sequence reads these, and one writes new_lens
    for (const int32_t *x : {seq_lens, keep_lens, recent_from})
        if (x && x < new_lens + num_seqs && new_lens < x + num_seqs) return VA_ERR_INVALID_ARGUMENT;
    const int bits = kv_dtype == VA_BF16 ? 16 : kv_dtype == VA_INT4 ? 4 : kv_dtype == VA_INT2 ? 2 : 8;
    const int heads = num_seqs * num_kv_heads, row = head_dim * bits / 8;
    va::EvictParams p = {};
    p.k_pages = static_cast<uint4 *>(k_pages), p.v_pages = static_cast<uint4 *>(v_pages);
    if (kv_dtype != VA_BF16) p.k_scale = k_scale, p.v_scale = v_scale;
    p.block_table = block_table, p.seq_lens = seq_lens, p.keep = keep_lens, p.recent_from = recent_from;
    p.ref_count = ref_count, p.weights = weights, p.slot_pos = slot_pos, p.new_lens = new_lens, p.flags = flags;
    p.stride_seq = stride_seq, p.stride_head = stride_head;
    p.count = static_cast<int32_t *>(workspace);
    p.moves = reinterpret_cast<int2 *>(static_cast<char *>(workspace) + align_up((size_t)heads * 4));
    p.bt_stride = block_table_stride, p.num_seqs = num_seqs, p.Hkv = num_kv_heads, p.num_pages = num_pages;
    p.num_sinks = num_sinks, p.half = num_slots / 2, p.slots = num_slots;
    p.units = row / 16;
    int device = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
    // CTAs of a cluster: one for each 4,096 slots, as long as there are SMs for all
    p.cluster = 1;
    while (p.cluster < va::kMaxCluster && num_slots > 4096 * p.cluster && heads * p.cluster * 2 <= 2 * sms) p.cluster *= 2;
    p.cached = std::min(va::kMaxCached, ((num_slots + p.cluster - 1) / p.cluster + 31) / 32 * 32);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(heads * p.cluster));
    cfg.blockDim = dim3(va::kThreads);
    cfg.dynamicSmemBytes = p.cached * sizeof(uint32_t);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (e == cudaSuccess && p.cached > 4096)  // with the static part past 32 KB: it has to be asked for
        e = cudaFuncSetAttribute(va::evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 va::kMaxCached * (int)sizeof(uint32_t));
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, va::evict_select_kernel, p);
    if (e == cudaSuccess) {
        const int64_t most = (int64_t)p.half * p.units;  // threads' worth of work of a head, at most
        int64_t blocks = (most + va::kMoveThreads - 1) / va::kMoveThreads;
        const int64_t cap = (8 * sms + heads - 1) / heads;
        if (blocks > cap) blocks = cap;
        if (blocks < 1) blocks = 1;
        e = va::launch_pdl(va::evict_move_kernel, dim3((unsigned)blocks, heads), dim3(va::kMoveThreads), 0, s, p);
    }
    if (e == cudaSuccess) return VA_OK;
    va::note_cuda_error(e);
    cudaGetLastError();
    return VA_ERR_CUDA;
}

}  // extern "C"
