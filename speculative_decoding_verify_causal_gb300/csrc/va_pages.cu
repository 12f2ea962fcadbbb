// Care of a paged cache: resize (give pages back, take pages, copy on write),
// fork and compact.  Definitions in verify_attn.h.
//
// Each call is one bookkeeping kernel on one thread-block cluster, then one
// copy kernel over the list of (source, destination) pages that the first left
// in the workspace.  Which pages change hands is known on the device only, so
// nothing here asks the host.
//
// The bookkeeping is integer work whose results do not depend on timing.
// Counts go down and up by atomics (order-free).  The pages that a call frees
// are first marked in a bitmap, whose scan then pushes them in ascending
// order; requests are placed by prefix sums over the sequences, which every
// CTA computes for itself in shared memory, so that only the bitmap, the counts
// and the lists are shared (through L2, cluster barriers between the phases).
// Work is spread over table entries, not sequences: entry i belongs to the
// sequence whose prefix sum it falls into (a binary search in shared memory),
// so one long sequence is shared by all threads.  Bound: a chain of dependent
// L2 round trips and barriers, not bytes.
//
// The copy kernel is HBM-bound: every byte of a page is read and written once.
#include <algorithm>

#include "va_internal.h"
#include "va_sm100.cuh"

namespace va {
namespace {

using namespace sm100;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;  // portable cluster size

struct Header {
    int jobs;    // pages to copy
    int movers;  // compaction: pages that move
    int pad[14];
};

struct Pool {
    int32_t *table, *lens, *ref, *free_list, *num_free, *flags;
    int stride, B, P;
    // workspace
    Header *head;
    uint32_t *mask;   // two bitmaps over the pages
    int32_t *claim;   // [B]
    int32_t *map;     // [P]
    int32_t *movers;  // [P]
    int2 *jobs;       // [P] (source, destination)
};

__host__ __device__ inline int mask_words(int P) { return (P + 31) / 32; }
__device__ __forceinline__ int blocks_of(int len) { return (int)(((unsigned)len + VA_PAGE_SIZE - 1) / VA_PAGE_SIZE); }
__device__ __forceinline__ int cluster_thread() { return (int)cluster_rank() * kThreads + threadIdx.x; }
__device__ __forceinline__ int cluster_threads() { return (int)cluster_size() * kThreads; }
__device__ __forceinline__ void flag(const Pool &p, int bit) {
    if (p.flags) atomicOr(p.flags, bit);
}

__device__ __forceinline__ int warp_scan(int v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
    }
    return v;
}

// Exclusive sum over the block's threads; `total` gets the sum of all.
__device__ int block_scan(int v, int &total) {
    __shared__ int sums[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int inc = warp_scan(v, lane);
    __syncthreads();  // sums may still be read from the call before
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    const int w = sums[lane], winc = warp_scan(w, lane);
    total = __shfl_sync(0xffffffffu, winc, 31);
    return inc - v + (warp ? __shfl_sync(0xffffffffu, winc, warp - 1) : 0);
}

// a[0 .. n) -> its exclusive prefix sums, a[n] = the sum; all threads of the block.
__device__ void prefix_sums(int *a, int n) {
    const int per = (n + kThreads - 1) / kThreads;
    const int lo = min(n, (int)threadIdx.x * per), hi = min(n, lo + per);
    __syncthreads();
    int sum = 0;
    for (int i = lo; i < hi; ++i) sum += a[i];
    int total, at = block_scan(sum, total);
    for (int i = lo; i < hi; ++i) {
        const int v = a[i];
        a[i] = at;
        at += v;
    }
    if (threadIdx.x == 0) a[n] = total;
    __syncthreads();
}

// The b with pre[b] <= i < pre[b + 1].
__device__ __forceinline__ int find(const int *pre, int n, int i) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Exclusive sum over the cluster's CTAs of one number each; `total` gets the sum of all.
__device__ int cluster_scan(int v, int &total) {
    __shared__ unsigned long long slot;
    if (threadIdx.x == 0) slot = (unsigned long long)(unsigned)v;
    cluster_sync();
    int before = 0;
    total = 0;
    for (int r = 0; r < (int)cluster_size(); ++r) {
        const int x = (int)ld_cluster_u64(&slot, r);
        if (r < (int)cluster_rank()) before += x;
        total += x;
    }
    cluster_sync();
    return before;
}

// Push the pages marked in `mask` onto the free list, in ascending order, above its first nf entries.  Returns the new
// count.  The marks must be visible (a cluster barrier before); the entries are visible after the next one.
__device__ int push_marked(const Pool &p, const uint32_t *mask, int nf) {
    const int W = mask_words(p.P), n = (int)cluster_size();
    const int per = (W + n - 1) / n, lo = min(W, (int)cluster_rank() * per), hi = min(W, lo + per);
    int mine = 0;
    for (int w = lo + threadIdx.x; w < hi; w += kThreads) mine += __popc(__ldcg(mask + w));
    int sum, total;
    block_scan(mine, sum);
    int at = nf + cluster_scan(sum, total);
    for (int base = lo; base < hi && sum > 0; base += kThreads) {
        const int w = base + threadIdx.x;
        uint32_t bits = w < hi ? __ldcg(mask + w) : 0;
        int chunk, to = at + block_scan(__popc(bits), chunk);
        while (bits) {
            if (to < p.P) p.free_list[to] = 32 * w + __ffs(bits) - 1;
            ++to;
            bits &= bits - 1;
        }
        at += chunk;
    }
    if (nf + total > p.P && cluster_thread() == 0) flag(p, VA_PAGES_BAD_COUNT);
    return min(p.P, nf + total);
}

__device__ __forceinline__ void drop_reference(const Pool &p, int page, uint32_t *mask) {
    const int old = atomicSub(p.ref + page, 1);
    if (old == 1) {
        atomicOr(mask + (page >> 5), 1u << (page & 31));
    } else if (old <= 0) {
        atomicAdd(p.ref + page, 1);
        flag(p, VA_PAGES_BAD_COUNT);
    }
}

__device__ __forceinline__ int free_count(const Pool &p) {
    const int nf = __ldcg(p.num_free);
    if ((nf < 0 || nf > p.P) && cluster_thread() == 0) flag(p, VA_PAGES_BAD_COUNT);
    return min(max(nf, 0), p.P);
}

__global__ void __launch_bounds__(kThreads) resize_kernel(const Pool p, const int32_t *new_lens) {
    extern __shared__ int smem[];
    int *pre = smem, *len = smem + p.B + 1;
    unsigned char *own_copy = reinterpret_cast<unsigned char *>(len + p.B);
    __shared__ int s_taken, s_copies;
    const int me = cluster_thread(), all = cluster_threads();
    const bool first = cluster_rank() == 0;
    uint32_t *mask2 = p.mask + mask_words(p.P);
    const int64_t most = (int64_t)p.stride * VA_PAGE_SIZE;
    griddep_wait();
    for (int w = me; w < 2 * mask_words(p.P); w += all) __stcg(p.mask + w, 0u);
    if (me == 0) p.head->jobs = 0;
    for (int b = threadIdx.x; b < p.B; b += kThreads) {
        const int L = p.lens[b], N = new_lens[b];
        const bool ok = L >= 0 && L <= most && N <= most;
        if (!ok && first) flag(p, VA_PAGES_BAD_REQUEST);
        len[b] = ok && N >= 0 ? L : -1;  // -1: left alone
        pre[b] = ok && N >= 0 && N < L ? blocks_of(L) - blocks_of(N) : 0;
    }
    if (threadIdx.x == 0) s_taken = s_copies = 0;
    prefix_sums(pre, p.B);
    cluster_sync();  // the bitmaps are clear
    // 1. shrinking sequences drop their last pages
    for (int i = me; i < pre[p.B]; i += all) {
        const int b = find(pre, p.B, i);
        int32_t *entry = p.table + (size_t)b * p.stride + blocks_of(new_lens[b]) + (i - pre[b]);
        const int page = *entry;
        *entry = -1;
        if (page < 0 || page >= p.P) flag(p, VA_PAGES_BAD_ENTRY);
        else drop_reference(p, page, p.mask);
    }
    cluster_sync();
    int nf = push_marked(p, p.mask, free_count(p));
    // 2. what each growing sequence needs, and who can be served
    for (int b = threadIdx.x; b < p.B; b += kThreads) {
        const int L = len[b], N = new_lens[b];
        int need = 0;
        own_copy[b] = 0;
        if (L >= 0 && N > L) {
            need = blocks_of(N) - blocks_of(L);
            if (L % VA_PAGE_SIZE) {
                const int page = p.table[(size_t)b * p.stride + L / VA_PAGE_SIZE];
                if (page < 0 || page >= p.P) {
                    if (first) flag(p, VA_PAGES_BAD_ENTRY);
                } else if (__ldcg(p.ref + page) > 1) {
                    own_copy[b] = 1;
                    ++need;
                }
            }
        }
        pre[b] = need;
    }
    prefix_sums(pre, p.B);
    for (int b = threadIdx.x; b < p.B; b += kThreads) {
        const int need = pre[b + 1] - pre[b];
        if (need == 0) continue;
        if (pre[b + 1] <= nf) {
            atomicMax(&s_taken, pre[b + 1]);
            if (own_copy[b]) s_copies = 1;
        } else if (first) {
            flag(p, VA_PAGES_EXHAUSTED);
        }
    }
    cluster_sync();  // everybody has decided; the pushed entries are visible
    const int taken = s_taken;
    for (int i = me; i < taken; i += all) {
        const int b = find(pre, p.B, i), k = i - pre[b], L = len[b];
        const bool copy = own_copy[b] && k == 0;
        const int j = copy ? L / VA_PAGE_SIZE : blocks_of(L) + k - own_copy[b];
        int32_t *entry = p.table + (size_t)b * p.stride + j;
        int page = __ldcg(p.free_list + nf - 1 - i);
        if (page < 0 || page >= p.P) {
            flag(p, VA_PAGES_BAD_ENTRY);
            page = -1;
        } else {
            p.ref[page] = 1;
        }
        if (copy) {
            const int old = *entry;
            p.jobs[atomicAdd(&p.head->jobs, 1)] = make_int2(page < 0 ? -1 : old, page);
            drop_reference(p, old, mask2);
        }
        *entry = page;
    }
    if (first) {
        for (int b = threadIdx.x; b < p.B; b += kThreads)
            if (len[b] >= 0 && (pre[b + 1] == pre[b] || pre[b + 1] <= nf)) p.lens[b] = new_lens[b];
    }
    // 3. shared pages that all their holders replaced
    nf -= taken;
    if (s_copies) {
        cluster_sync();
        nf = push_marked(p, mask2, nf);
    }
    if (me == 0) *p.num_free = nf;
}

__global__ void __launch_bounds__(kThreads) fork_kernel(const Pool p, const int32_t *parents, const int32_t *children,
                                                        const int32_t *lens, int F, int share) {
    extern __shared__ int smem[];
    int *held = smem, *need = held + F + 1, *len = need + F + 1;
    __shared__ int s_taken;
    const int me = cluster_thread(), all = cluster_threads();
    const bool first = cluster_rank() == 0;
    const int64_t most = (int64_t)p.stride * VA_PAGE_SIZE;
    griddep_wait();
    for (int b = me; b < p.B; b += all) __stcg(p.claim + b, F);
    cluster_sync();
    for (int f = me; f < F; f += all) {
        const int c = children[f];
        if (c >= 0 && c < p.B) atomicMin(p.claim + c, f);
    }
    if (threadIdx.x == 0) s_taken = 0;
    cluster_sync();
    const int nf = free_count(p);
    for (int f = threadIdx.x; f < F; f += kThreads) {
        const int from = parents[f], to = children[f];
        int n = -1;
        if (from >= 0 && from < p.B && to >= 0 && to < p.B && p.lens[to] == 0 && __ldcg(p.claim + to) == f) {
            const int L = p.lens[from];
            n = lens ? lens[f] : L;
            if (L < 0 || L > most || n < 0 || n > L) n = -1;
        }
        if (n < 0 && first) flag(p, VA_PAGES_BAD_REQUEST);
        len[f] = n;
        held[f] = n < 0 ? 0 : blocks_of(n);
        need[f] = n < 0 ? 0 : share ? (n % VA_PAGE_SIZE != 0) : blocks_of(n);
    }
    prefix_sums(held, F);
    prefix_sums(need, F);
    for (int f = threadIdx.x; f < F; f += kThreads) {
        if (need[f + 1] == need[f]) continue;
        if (need[f + 1] <= nf) atomicMax(&s_taken, need[f + 1]);
        else if (first) flag(p, VA_PAGES_EXHAUSTED);
    }
    cluster_sync();  // everybody has decided
    for (int i = me; i < held[F]; i += all) {
        const int f = find(held, F, i), j = i - held[f];
        if (need[f + 1] > need[f] && need[f + 1] > nf) continue;  // refused
        int page = p.table[(size_t)parents[f] * p.stride + j];
        const bool bad = page < 0 || page >= p.P;
        if (bad) flag(p, VA_PAGES_BAD_ENTRY);
        const int fresh = share ? len[f] / VA_PAGE_SIZE : 0;  // the first block that is copied
        if (j < fresh) {
            if (bad) page = -1;
            else atomicAdd(p.ref + page, 1);
        } else {
            const int k = need[f] + j - fresh;
            int to = p.free_list[nf - 1 - k];
            if (to < 0 || to >= p.P) {
                flag(p, VA_PAGES_BAD_ENTRY);
                to = -1;
            } else {
                p.ref[to] = 1;
            }
            p.jobs[k] = make_int2(bad || to < 0 ? -1 : page, to);
            page = to;
        }
        p.table[(size_t)children[f] * p.stride + j] = page;
    }
    if (first) {
        for (int f = threadIdx.x; f < F; f += kThreads)
            if (len[f] >= 0 && (need[f + 1] == need[f] || need[f + 1] <= nf)) p.lens[children[f]] = len[f];
        if (threadIdx.x == 0) {
            *p.num_free = nf - s_taken;
            p.head->jobs = s_taken;
        }
    }
}

__global__ void __launch_bounds__(kThreads) compact_kernel(const Pool p) {
    extern __shared__ int smem[];
    __shared__ int word_pre[kThreads];
    const int me = cluster_thread(), all = cluster_threads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool first = cluster_rank() == 0;
    const int64_t most = (int64_t)p.stride * VA_PAGE_SIZE;
    griddep_wait();
    if (me == 0) p.head->movers = 0;
    // which pages are held, 32 to a word, and how many before each CTA's words
    const int W = mask_words(p.P), ncta = (int)cluster_size();
    const int per = (W + ncta - 1) / ncta, lo = min(W, (int)cluster_rank() * per), hi = min(W, lo + per);
    int mine = 0;
    for (int w = lo + warp; w < hi; w += kWarps) {
        const int page = 32 * w + lane;
        const uint32_t live = __ballot_sync(0xffffffffu, page < p.P && p.ref[page] > 0);
        if (lane == 0) {
            p.mask[w] = live;
            mine += __popc(live);
        }
    }
    int sum, n;
    block_scan(mine, sum);
    int before = cluster_scan(sum, n);  // n pages are held
    // free places below n, held pages from n on
    for (int base = lo; base < hi; base += kThreads) {
        const int w = base + threadIdx.x;
        int chunk;
        const int at = block_scan(w < hi ? __popc(p.mask[w]) : 0, chunk);
        word_pre[threadIdx.x] = before + at;
        before += chunk;
        __syncthreads();
        for (int v = base + warp; v < min(hi, base + kThreads); v += kWarps) {
            const uint32_t live = p.mask[v];
            const int page = 32 * v + lane;
            const int below = word_pre[v - base] + __popc(live & ((1u << lane) - 1));  // held pages below this one
            if (page == n) p.head->movers = page - below;
            if (page < p.P) {
                if (live >> lane & 1) {
                    p.map[page] = page;
                    if (page >= n) p.movers[n - 1 - below] = page;  // counted from the last held page
                } else {
                    p.map[page] = -1;
                    if (page < n) p.jobs[page - below].y = page;
                }
            }
        }
        __syncthreads();
    }
    cluster_sync();
    const int M = n < p.P ? __ldcg(&p.head->movers) : 0;
    for (int k = me; k < M; k += all) {
        const int src = __ldcg(p.movers + M - 1 - k), dst = __ldcg(&p.jobs[k].y);
        p.jobs[k].x = src;
        p.map[src] = dst;
        p.ref[dst] = p.ref[src];
        p.ref[src] = 0;
    }
    for (int i = me; i < p.P - n; i += all) p.free_list[i] = p.P - 1 - i;
    if (me == 0) {
        if (*p.num_free != p.P - n) flag(p, VA_PAGES_BAD_COUNT);
        *p.num_free = p.P - n;
        p.head->jobs = M;
    }
    for (int b = threadIdx.x; b < p.B; b += kThreads) {
        const int L = p.lens[b];
        const bool ok = L >= 0 && L <= most;
        if (!ok && first) flag(p, VA_PAGES_BAD_REQUEST);
        smem[b] = ok ? blocks_of(L) : 0;
    }
    prefix_sums(smem, p.B);
    cluster_sync();
    for (int i = me; i < smem[p.B]; i += all) {
        const int b = find(smem, p.B, i);
        int32_t *entry = p.table + (size_t)b * p.stride + (i - smem[b]);
        const int page = *entry;
        if (page < 0 || page >= p.P) {
            flag(p, VA_PAGES_BAD_ENTRY);
            continue;
        }
        const int to = __ldcg(p.map + page);
        if (to < 0) flag(p, VA_PAGES_BAD_COUNT);
        else if (to != page) *entry = to;
    }
}

// ------------------------------------------------------------------------- copies

constexpr int kCopyThreads = 1024;
constexpr int kCopyCtas = 304;      // two of 1,024 threads on each of 152 SMs
constexpr int kUnit = 2048;         // bytes a warp has in flight: four 16-byte loads a lane
constexpr int kMaxBuffers = 128;    // of one launch

struct CopyParams {
    const Header *head;
    const int2 *jobs;
    char *data[kMaxBuffers];
    uint32_t page_16[kMaxBuffers];         // page size in 16-byte pieces
    uint32_t unit_begin[kMaxBuffers + 1];  // units of one page in the buffers before
    int buffers;
};

// A warp copies one unit at a time: (page pair, buffer, 2 KB piece of the page).  Units are dealt round the CTAs, so that
// a few pages spread over all SMs.
__global__ void __launch_bounds__(kCopyThreads, 2) copy_kernel(const __grid_constant__ CopyParams p) {
    griddep_wait();
    const int jobs = p.head->jobs;
    const int lane = threadIdx.x & 31;
    const uint32_t units = p.unit_begin[p.buffers];
    const uint32_t warps = gridDim.x * (kCopyThreads / 32), mine = (threadIdx.x >> 5) * gridDim.x + blockIdx.x;
    const uint32_t step_job = warps / units, step_unit = warps % units;
    uint32_t job = mine / units, unit = mine % units;
    while (job < (uint32_t)jobs) {
        const int2 pages = p.jobs[job];
        int lo = 0, hi = p.buffers;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.unit_begin[mid] <= unit) lo = mid;
            else hi = mid;
        }
        const uint32_t at = (unit - p.unit_begin[lo]) * (kUnit / 16), size = p.page_16[lo];
        if (pages.x >= 0) {
            const uint4 *src = reinterpret_cast<const uint4 *>(p.data[lo]) + (size_t)pages.x * size + at;
            uint4 *dst = reinterpret_cast<uint4 *>(p.data[lo]) + (size_t)pages.y * size + at;
            const uint32_t left = size - at;
            uint4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (lane + 32 * k < left) v[k] = src[lane + 32 * k];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (lane + 32 * k < left) dst[lane + 32 * k] = v[k];
        }
        job += step_job;
        unit += step_unit;
        if (unit >= units) {
            unit -= units;
            ++job;
        }
    }
}

// ------------------------------------------------------------------------- host

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

struct Layout {
    size_t mask, claim, map, movers, jobs, total;
    Layout(int B, int P) {
        mask = align_up(sizeof(Header));
        claim = mask + align_up(2 * sizeof(uint32_t) * (size_t)mask_words(P));
        map = claim + align_up(sizeof(int32_t) * (size_t)B);
        movers = map + align_up(sizeof(int32_t) * (size_t)P);
        jobs = movers + align_up(sizeof(int32_t) * (size_t)P);
        total = jobs + align_up(sizeof(int2) * (size_t)P);
    }
};

bool sizes_ok(int B, int P) { return B >= 1 && B <= VA_PAGES_MAX_SEQS && P >= 1 && P <= (1 << 24); }

int check(const va_page_pool *v, Pool *p) {
    if (!v || !v->block_table || !v->seq_lens || !v->ref_count || !v->free_list || !v->num_free || !v->workspace)
        return VA_ERR_INVALID_ARGUMENT;
    if (!sizes_ok(v->num_seqs, v->num_pages) || v->block_table_stride < 1 ||
        (long long)v->num_seqs * v->block_table_stride >= (1LL << 31) ||
        (long long)v->block_table_stride * VA_PAGE_SIZE >= (1LL << 31) || v->num_buffers < 0 ||
        (v->num_buffers > 0 && !v->buffers))
        return VA_ERR_INVALID_ARGUMENT;
    auto aligned = [](const void *ptr, uintptr_t a) { return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) == 0; };
    for (const void *x : {(const void *)v->block_table, (const void *)v->seq_lens, (const void *)v->ref_count,
                          (const void *)v->free_list, (const void *)v->num_free, (const void *)v->flags})
        if (!aligned(x, 4)) return VA_ERR_INVALID_ARGUMENT;
    if (!aligned(v->workspace, 16)) return VA_ERR_INVALID_ARGUMENT;
    for (int i = 0; i < v->num_buffers; ++i)
        if (!v->buffers[i].data || !aligned(v->buffers[i].data, 16) || v->buffers[i].page_bytes == 0 ||
            v->buffers[i].page_bytes % 16 != 0 || v->buffers[i].page_bytes > (1u << 30))
            return VA_ERR_INVALID_ARGUMENT;
    *p = Pool{};
    p->table = v->block_table;
    p->lens = v->seq_lens;
    p->ref = v->ref_count;
    p->free_list = v->free_list;
    p->num_free = v->num_free;
    p->flags = v->flags;
    p->stride = v->block_table_stride;
    p->B = v->num_seqs;
    p->P = v->num_pages;
    const Layout at(p->B, p->P);
    char *ws = static_cast<char *>(v->workspace);
    p->head = reinterpret_cast<Header *>(ws);
    p->mask = reinterpret_cast<uint32_t *>(ws + at.mask);
    p->claim = reinterpret_cast<int32_t *>(ws + at.claim);
    p->map = reinterpret_cast<int32_t *>(ws + at.map);
    p->movers = reinterpret_cast<int32_t *>(ws + at.movers);
    p->jobs = reinterpret_cast<int2 *>(ws + at.jobs);
    return VA_OK;
}

// One cluster: a single CTA while the pool and the table are small (its barriers cost least), eight beyond.
int cluster_for(const Pool &p, long long entries) { return p.P <= 16384 && entries <= 16384 ? 1 : kMaxCluster; }

template <typename... KArgs, typename... Args>
cudaError_t launch_book(void (*kernel)(KArgs...), int cluster, size_t smem, cudaStream_t s, Args... args) {
    if (smem > 40 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
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
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

cudaError_t launch_copies(const va_page_pool *v, const Pool &p, cudaStream_t s) {
    for (int done = 0; done < v->num_buffers; done += kMaxBuffers) {
        CopyParams c{};
        c.head = p.head;
        c.jobs = p.jobs;
        c.buffers = std::min(kMaxBuffers, v->num_buffers - done);
        for (int i = 0; i < c.buffers; ++i) {
            const va_page_buffer &b = v->buffers[done + i];
            c.data[i] = static_cast<char *>(b.data);
            c.page_16[i] = (uint32_t)(b.page_bytes / 16);
            c.unit_begin[i + 1] = c.unit_begin[i] + (uint32_t)((b.page_bytes + kUnit - 1) / kUnit);
        }
        const cudaError_t e = launch_pdl(copy_kernel, dim3(kCopyCtas), dim3(kCopyThreads), 0, s, c);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

int done(cudaError_t e) {
    if (e == cudaSuccess) return VA_OK;
    note_cuda_error(e);
    return VA_ERR_CUDA;
}

}  // namespace
}  // namespace va

extern "C" size_t verify_attn_pages_workspace_bytes(int num_seqs, int num_pages) {
    return va::sizes_ok(num_seqs, num_pages) ? va::Layout(num_seqs, num_pages).total : 0;
}

extern "C" int verify_attn_pages_resize(const va_page_pool *pool, const int32_t *new_lens, void *stream) {
    va::Pool p;
    if (const int rc = va::check(pool, &p)) return rc;
    if (!new_lens || (reinterpret_cast<uintptr_t>(new_lens) & 3)) return VA_ERR_INVALID_ARGUMENT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t smem = sizeof(int) * (2 * (size_t)p.B + 1) + (size_t)p.B;
    cudaError_t e = va::launch_book(va::resize_kernel, va::cluster_for(p, (long long)p.B * p.stride), smem, s, p, new_lens);
    if (e == cudaSuccess) e = va::launch_copies(pool, p, s);
    return va::done(e);
}

extern "C" int verify_attn_pages_fork(const va_page_pool *pool, const int32_t *parents, const int32_t *children,
                                      const int32_t *lens, int num_forks, int share, void *stream) {
    va::Pool p;
    if (const int rc = va::check(pool, &p)) return rc;
    if (num_forks < 0 || num_forks > VA_PAGES_MAX_SEQS) return VA_ERR_INVALID_ARGUMENT;
    if (num_forks == 0) return VA_OK;
    if (!parents || !children || (long long)num_forks * p.stride >= (1LL << 31)) return VA_ERR_INVALID_ARGUMENT;
    for (const int32_t *x : {parents, children, lens})
        if (reinterpret_cast<uintptr_t>(x) & 3) return VA_ERR_INVALID_ARGUMENT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t smem = sizeof(int) * (3 * (size_t)num_forks + 2);
    cudaError_t e = va::launch_book(va::fork_kernel, va::cluster_for(p, (long long)num_forks * p.stride), smem, s, p,
                                    parents, children, lens, num_forks, share);
    if (e == cudaSuccess) e = va::launch_copies(pool, p, s);
    return va::done(e);
}

extern "C" int verify_attn_pages_compact(const va_page_pool *pool, void *stream) {
    va::Pool p;
    if (const int rc = va::check(pool, &p)) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t smem = sizeof(int) * ((size_t)p.B + 1);
    cudaError_t e = va::launch_book(va::compact_kernel, va::cluster_for(p, (long long)p.B * p.stride), smem, s, p);
    if (e == cudaSuccess) e = va::launch_copies(pool, p, s);
    return va::done(e);
}
