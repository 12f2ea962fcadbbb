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
// are first marked in a bitmap, which lies in the CTAs' shared memory, a slice
// each, and is marked there by all of them; its scan then pushes the pages in
// ascending order.  Requests are placed by prefix sums over the sequences,
// which every CTA computes for itself, so that only the bitmap, the counts and
// the lists are shared, with cluster barriers between the phases.  Work is
// spread over table entries, not sequences: entry i belongs to the sequence
// whose prefix sum it falls into (a binary search in shared memory), so one
// long sequence is shared by all threads, each with kBatch entries' loads in
// flight.  Bound: a chain of dependent L2 round trips and barriers, not bytes.
//
// The copy kernel is HBM-bound: every byte of a page is read and written once
// (0.95 GB of traffic in 144 us, 6.6 TB/s).
#include <algorithm>

#include "va_internal.h"
#include "va_sm100.cuh"

namespace va {
namespace {

using namespace sm100;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
static_assert(kWarps == 32, "a warp scans one number per warp of the block");
constexpr int kMaxCluster = 8;  // portable cluster size
constexpr int kBatch = 4;

// The kernel behind this one on the stream, the copies, may take its places on the other SMs now; it waits there for this
// one's end (griddep_wait), which then costs no launch.
__device__ __forceinline__ void griddep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

struct Header {
    int jobs;  // pages to copy
    int held;  // compaction: held pages
    int pad[14];
};

struct Pool {
    int32_t *table, *lens, *ref, *free_list, *num_free, *flags;
    int stride, B, P;
    int slice_bits;  // of the bitmap's 32-bit words: each CTA has 2^slice_bits of them
    // workspace
    Header *head;
    int32_t *map;     // [P] compaction: -1 for a free page, a moving page's place among the movers
    int32_t *movers;  // [P] compaction: the pages that move, the last one first
    int2 *jobs;       // [P] (source, destination); compaction: the destinations, in order
};

__host__ __device__ inline int mask_words(int P) { return (P + 31) / 32; }
__device__ __forceinline__ int blocks_of(int len) { return (int)(((unsigned)len + VA_PAGE_SIZE - 1) / VA_PAGE_SIZE); }
// Threads are counted warp by warp round the CTAs, so that what a round leaves over spreads over all of them.
__device__ __forceinline__ int spread_thread(int cta, int ctas) {
    return (((int)threadIdx.x >> 5) * ctas + cta) * 32 + ((int)threadIdx.x & 31);
}
__device__ __forceinline__ int cluster_thread() { return spread_thread((int)cluster_rank(), (int)cluster_size()); }
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

// load(i), then use(i, what it gave), for the items i = me, me + all, .. below `total`: kBatch loads in flight.
template <typename Load, typename Use>
__device__ __forceinline__ void for_items(int me, int all, int total, Load load, Use use) {
    for (int base = me; base < total; base += kBatch * all) {
        decltype(load(0)) v[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (base + u * all < total) v[u] = load(base + u * all);
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (base + u * all < total) use(base + u * all, v[u]);
    }
}

// Exclusive sum over the cluster's CTAs of one number each (v of thread 0 .. ctas - 1 of each CTA); `total` gets the sum of
// all.  One cluster barrier; `slots` of this CTA is written by the others and serves one call.
__device__ int cluster_scan(int v, int &total, unsigned long long *slots) {
    const int rank = (int)cluster_rank(), ctas = (int)cluster_size();
    if ((int)threadIdx.x < ctas) st_cluster_u64(slots + rank, threadIdx.x, (unsigned long long)(unsigned)v);
    cluster_sync();
    int before = 0;
    total = 0;
    for (int r = 0; r < ctas; ++r) {
        const int x = (int)slots[r];
        if (r < rank) before += x;
        total += x;
    }
    return before;
}

// Mark a page in the bitmap, in the shared memory of the CTA that has its word.
__device__ __forceinline__ void mark(const Pool &p, uint32_t *mask, int page) {
    const int w = page >> 5;
    asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(
                     cluster_map(mask + (w & ((1 << p.slice_bits) - 1)), w >> p.slice_bits)),
                 "r"(1u << (page & 31))
                 : "memory");
}

// Push the marked pages onto the free list, in ascending order, above its first nf entries, and clear the marks.  Returns
// the new count.  The marks must be complete (a cluster barrier before); the entries are visible after the next one.
__device__ int push_marked(const Pool &p, uint32_t *mask, int nf, unsigned long long *slots) {
    __shared__ int word_pre[kThreads];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int first = (int)cluster_rank() << p.slice_bits, words = max(0, min(1 << p.slice_bits, mask_words(p.P) - first));
    int mine = 0;
    for (int w = threadIdx.x; w < words; w += kThreads) mine += __popc(mask[w]);
    int sum, total;
    int before = block_scan(mine, sum);  // each word's own where a thread has one word
    int at = nf + cluster_scan(sum, total, slots), chunk = sum;
    for (int base = 0; base < words && sum > 0; base += kThreads) {
        const int w = base + threadIdx.x;
        if (words > kThreads) before = block_scan(w < words ? __popc(mask[w]) : 0, chunk);
        word_pre[threadIdx.x] = at + before;
        at += chunk;
        __syncthreads();
        for (int v = base + warp; v < min(words, base + kThreads); v += kWarps) {  // a warp per word, a lane per page
            const uint32_t bits = mask[v];
            const int to = word_pre[v - base] + __popc(bits & ((1u << lane) - 1));
            if ((bits >> lane & 1) && to < p.P) p.free_list[to] = 32 * (first + v) + lane;
            __syncwarp();
            if (lane == 0) mask[v] = 0;
        }
        __syncthreads();
    }
    if (nf + total > p.P && cluster_thread() == 0) flag(p, VA_PAGES_BAD_COUNT);
    return min(p.P, nf + total);
}

__device__ __forceinline__ int take_reference(const Pool &p, int page) { return atomicSub(p.ref + page, 1); }
__device__ __forceinline__ void dropped(const Pool &p, uint32_t *mask, int page, int old) {
    if (old == 1) {
        mark(p, mask, page);
    } else if (old <= 0) {
        atomicAdd(p.ref + page, 1);
        flag(p, VA_PAGES_BAD_COUNT);
    }
}

__device__ __forceinline__ bool in_pool(const Pool &p, int page) { return page >= 0 && page < p.P; }

__device__ __forceinline__ int free_count(const Pool &p) {
    const int nf = __ldcg(p.num_free);
    if ((nf < 0 || nf > p.P) && cluster_thread() == 0) flag(p, VA_PAGES_BAD_COUNT);
    return min(max(nf, 0), p.P);
}

__global__ void __launch_bounds__(kThreads) resize_kernel(const Pool p, const int32_t *kept_lens, const int32_t *new_lens) {
    extern __shared__ int smem[];
    int *pre = smem, *len = pre + p.B + 1, *want = len + p.B, *tail = want + p.B;
    uint32_t *mask = reinterpret_cast<uint32_t *>(tail + p.B);
    __shared__ unsigned long long slots[2][kMaxCluster];
    __shared__ int s_taken, s_copies;
    const int me = cluster_thread(), all = cluster_threads();
    const bool first = cluster_rank() == 0;
    const int64_t most = (int64_t)p.stride * VA_PAGE_SIZE;
    for (int w = threadIdx.x; w < (1 << p.slice_bits); w += kThreads) mask[w] = 0;
    if (threadIdx.x == 0) s_taken = s_copies = 0;
    cluster_arrive();  // the bitmap is clear, and this CTA runs
    griddep_launch();
    griddep_wait();
    if (me == 0) p.head->jobs = 0;
    int nf = free_count(p);
    for (int b = threadIdx.x; b < p.B; b += kThreads) {
        const int L = p.lens[b], N = new_lens[b], K = kept_lens && N >= 0 ? kept_lens[b] : L;
        const bool ok = L >= 0 && L <= most && N <= most && K >= 0 && K <= L;
        if (!ok && first) flag(p, VA_PAGES_BAD_REQUEST);
        const int cut = ok ? min(K, N) : -1;  // what stays of the sequence before it grows
        len[b] = cut;  // -1: left alone
        want[b] = N;
        pre[b] = cut >= 0 ? blocks_of(L) - blocks_of(cut) : 0;
        // the partly filled last page of a sequence that grows
        const bool part = cut >= 0 && N > cut && cut % VA_PAGE_SIZE;
        tail[b] = part ? p.table[(size_t)b * p.stride + cut / VA_PAGE_SIZE] : -1;
        if (part && !in_pool(p, tail[b])) {
            if (first) flag(p, VA_PAGES_BAD_ENTRY);
            tail[b] = -1;
        }
    }
    prefix_sums(pre, p.B);
    cluster_wait();
    // 1. sequences that are cut back drop their last pages
    const int drops = pre[p.B];
    if (drops) {
        struct Entry {
            int32_t *at;
            int page;
        };
        for (int base = me; base < drops; base += kBatch * all) {
            Entry v[kBatch];
            int old[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int i = base + u * all;
                v[u].page = -1;
                if (i >= drops) continue;
                const int b = find(pre, p.B, i);
                v[u].at = p.table + (size_t)b * p.stride + blocks_of(len[b]) + (i - pre[b]);
                v[u].page = *v[u].at;
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (base + u * all >= drops) continue;
                *v[u].at = -1;
                if (in_pool(p, v[u].page)) old[u] = take_reference(p, v[u].page);
                else flag(p, VA_PAGES_BAD_ENTRY);
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (base + u * all < drops && in_pool(p, v[u].page)) dropped(p, mask, v[u].page, old[u]);
        }
        cluster_sync();
        nf = push_marked(p, mask, nf, slots[0]);
    }
    // 2. what each growing sequence needs, and who can be served
    __syncthreads();  // pre is read no more
    for (int b = threadIdx.x; b < p.B; b += kThreads) {
        const int L = len[b], N = want[b];
        if (tail[b] >= 0 && __ldcg(p.ref + tail[b]) <= 1) tail[b] = -1;  // its own already
        pre[b] = L >= 0 && N > L ? blocks_of(N) - blocks_of(L) + (tail[b] >= 0) : 0;
    }
    prefix_sums(pre, p.B);
    for (int b = threadIdx.x; b < p.B; b += kThreads) {
        if (pre[b + 1] == pre[b]) continue;
        if (pre[b + 1] <= nf) {
            atomicMax(&s_taken, pre[b + 1]);
            if (tail[b] >= 0) s_copies = 1;
        } else if (first) {
            flag(p, VA_PAGES_EXHAUSTED);
        }
    }
    cluster_sync();  // everybody has decided; the pushed entries are visible
    const int taken = s_taken, copies = s_copies;
    for_items(me, all, taken, [&](int i) { return __ldcg(p.free_list + nf - 1 - i); }, [&](int i, int page) {
        const int b = find(pre, p.B, i), k = i - pre[b], L = len[b];
        const int own = tail[b] >= 0;
        const bool copy = own && k == 0;
        if (in_pool(p, page)) {
            p.ref[page] = 1;
        } else {
            flag(p, VA_PAGES_BAD_ENTRY);
            page = -1;
        }
        if (copy) {
            p.jobs[atomicAdd(&p.head->jobs, 1)] = make_int2(page < 0 ? -1 : tail[b], page);
            dropped(p, mask, tail[b], take_reference(p, tail[b]));
        }
        p.table[(size_t)b * p.stride + (copy ? L / VA_PAGE_SIZE : blocks_of(L) + k - own)] = page;
    });
    if (first) {
        for (int b = threadIdx.x; b < p.B; b += kThreads)
            if (len[b] >= 0) p.lens[b] = pre[b + 1] == pre[b] || pre[b + 1] <= nf ? want[b] : len[b];
    }
    // 3. shared pages that all their holders replaced
    nf -= taken;
    if (copies) {
        cluster_sync();
        nf = push_marked(p, mask, nf, slots[1]);
    }
    if (me == 0) *p.num_free = nf;
}

__global__ void __launch_bounds__(kThreads) fork_kernel(const Pool p, const int32_t *parents, const int32_t *children,
                                                        const int32_t *lens, int F, int share) {
    extern __shared__ int smem[];
    int *held = smem, *need = held + F + 1, *len = need + F + 1, *parent = len + F, *child = parent + F, *claim = child + F;
    __shared__ int s_taken;
    const int me = cluster_thread(), all = cluster_threads();
    const bool first = cluster_rank() == 0;
    const int64_t most = (int64_t)p.stride * VA_PAGE_SIZE;
    for (int b = threadIdx.x; b < p.B; b += kThreads) claim[b] = F;
    if (threadIdx.x == 0) s_taken = 0;
    __syncthreads();
    griddep_launch();
    griddep_wait();
    const int nf = free_count(p);
    // the first fork of the call that wants a slot has it
    for (int f = threadIdx.x; f < F; f += kThreads) {
        parent[f] = parents[f];
        child[f] = children[f];
        if (child[f] >= 0 && child[f] < p.B) atomicMin(claim + child[f], f);
    }
    __syncthreads();
    for (int f = threadIdx.x; f < F; f += kThreads) {
        const int from = parent[f], to = child[f];
        int n = -1;
        if (from >= 0 && from < p.B && to >= 0 && to < p.B && claim[to] == f) {
            const int L = p.lens[from], there = p.lens[to];
            n = lens ? lens[f] : L;
            if (there != 0 || L < 0 || L > most || n < 0 || n > L) n = -1;
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
    cluster_arrive();  // this CTA has read the lengths and the free count
    struct Entry {
        int f, j, page, to;
    };
    for_items(
        me, all, held[F],
        [&](int i) {
            Entry e;
            e.f = find(held, F, i);
            e.j = i - held[e.f];
            e.page = p.table[(size_t)parent[e.f] * p.stride + e.j];
            const int fresh = share ? len[e.f] / VA_PAGE_SIZE : 0, k = need[e.f] + e.j - fresh;
            e.to = e.j >= fresh && need[e.f + 1] <= nf ? p.free_list[nf - 1 - k] : -1;
            return e;
        },
        [&](int, const Entry &e) {
            if (need[e.f + 1] > need[e.f] && need[e.f + 1] > nf) return;  // refused
            const bool bad = !in_pool(p, e.page);
            if (bad) flag(p, VA_PAGES_BAD_ENTRY);
            const int fresh = share ? len[e.f] / VA_PAGE_SIZE : 0;  // the first block that is copied
            int page = bad ? -1 : e.page;
            if (e.j < fresh) {
                if (!bad) atomicAdd(p.ref + page, 1);
            } else {
                const bool good = in_pool(p, e.to);
                if (good) p.ref[e.to] = 1;
                else flag(p, VA_PAGES_BAD_ENTRY);
                p.jobs[need[e.f] + e.j - fresh] = make_int2(good ? page : -1, good ? e.to : -1);
                page = good ? e.to : -1;
            }
            p.table[(size_t)child[e.f] * p.stride + e.j] = page;
        });
    __syncthreads();
    cluster_wait();
    if (first) {
        for (int f = threadIdx.x; f < F; f += kThreads)
            if (len[f] >= 0 && (need[f + 1] == need[f] || need[f + 1] <= nf)) p.lens[child[f]] = len[f];
        if (threadIdx.x == 0) {
            *p.num_free = nf - s_taken;
            p.head->jobs = s_taken;
        }
    }
}

// Which pages move and where to.  What follows from that, counts, lists and tables, is done beside the copies.
__global__ void __launch_bounds__(kThreads) compact_kernel(const Pool p) {
    extern __shared__ int smem[];
    uint32_t *mask = reinterpret_cast<uint32_t *>(smem);
    __shared__ int word_pre[kThreads];
    __shared__ unsigned long long slots[kMaxCluster];
    const int me = cluster_thread();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    cluster_arrive();  // this CTA runs
    griddep_launch();
    griddep_wait();
    if (me == 0) p.head->jobs = 0;
    // which pages are held, 32 to a word, and how many before each CTA's words
    const int word0 = (int)cluster_rank() << p.slice_bits, words = max(0, min(1 << p.slice_bits, mask_words(p.P) - word0));
    int mine = 0;
    for (int base = warp; base < words; base += kWarps * kBatch) {
        int held[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int page = 32 * (word0 + base + u * kWarps) + lane;
            held[u] = base + u * kWarps < words && page < p.P ? p.ref[page] : 0;
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const uint32_t live = __ballot_sync(0xffffffffu, held[u] > 0);
            if (lane == 0 && base + u * kWarps < words) {
                mask[base + u * kWarps] = live;
                mine += __popc(live);
            }
        }
    }
    int sum, n;
    block_scan(mine, sum);
    cluster_wait();
    int before = cluster_scan(sum, n, slots);  // n pages are held
    if (me == 0) p.head->held = n;
    // free places below n, held pages from n on
    for (int base = 0; base < words; base += kThreads) {
        const int w = base + threadIdx.x;
        int chunk;
        const int at = block_scan(w < words ? __popc(mask[w]) : 0, chunk);
        word_pre[threadIdx.x] = before + at;
        before += chunk;
        __syncthreads();
        for (int v = base + warp; v < min(words, base + kThreads); v += kWarps) {
            const uint32_t live = mask[v];
            const int page = 32 * (word0 + v) + lane;
            const int below = word_pre[v - base] + __popc(live & ((1u << lane) - 1));  // held pages below this one
            if (page >= p.P) continue;
            if (page == n) p.head->jobs = page - below;  // as many move as there are free places below n
            if (live >> lane & 1) {
                const int last = n - 1 - below;  // counted from the last held page
                p.map[page] = page < n ? 0 : last;
                if (page >= n) p.movers[last] = page;
            } else {
                p.map[page] = -1;
                if (page < n) p.jobs[page - below].y = page;
            }
        }
        __syncthreads();
    }
}

// The rest of a compaction, by the first kSideCtas CTAs of the copy kernel: the k-th mover from below goes to destination k,
// and is the (M - 1 - k)-th from the last.
constexpr int kSideCtas = 8;
__device__ void compact_rest(const Pool &p, int *pre) {
    const int me = spread_thread(blockIdx.x, kSideCtas), all = kSideCtas * kThreads;
    const int64_t most = (int64_t)p.stride * VA_PAGE_SIZE;
    const int M = p.head->jobs, n = p.head->held;
    for_items(me, all, M, [&](int k) { return make_int2(p.movers[M - 1 - k], p.jobs[k].y); },
              [&](int, int2 move) {
                  p.ref[move.y] = p.ref[move.x];
                  p.ref[move.x] = 0;
              });
    for (int i = me; i < p.P - n; i += all) p.free_list[i] = p.P - 1 - i;
    if (me == 0) {
        if (*p.num_free != p.P - n) flag(p, VA_PAGES_BAD_COUNT);
        *p.num_free = p.P - n;
    }
    for (int b = threadIdx.x; b < p.B; b += kThreads) {
        const int L = p.lens[b];
        const bool ok = L >= 0 && L <= most;
        if (!ok && blockIdx.x == 0) flag(p, VA_PAGES_BAD_REQUEST);
        pre[b] = ok ? blocks_of(L) : 0;
    }
    prefix_sums(pre, p.B);
    const int entries = pre[p.B];
    for (int base = me; base < entries; base += kBatch * all) {
        int32_t *at[kBatch];
        int page[kBatch], to[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int i = base + u * all;
            if (i >= entries) continue;
            const int b = find(pre, p.B, i);
            at[u] = p.table + (size_t)b * p.stride + (i - pre[b]);
            page[u] = *at[u];
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (base + u * all < entries && in_pool(p, page[u])) to[u] = p.map[page[u]];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (base + u * all >= entries) continue;
            if (!in_pool(p, page[u])) flag(p, VA_PAGES_BAD_ENTRY);
            else if (to[u] < 0) flag(p, VA_PAGES_BAD_COUNT);
            else if (page[u] >= n) *at[u] = p.jobs[M - 1 - to[u]].y;
        }
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
    const int32_t *movers;  // compaction: the sources, the last one first
};

// A warp copies one unit at a time: (page pair, buffer, 2 KB piece of the page).  Units are dealt round the CTAs, so that
// a few pages spread over all SMs.
template <bool COMPACT>
__device__ __forceinline__ void copy_pages(const CopyParams &p, uint32_t cta, uint32_t ctas) {
    const int jobs = p.head->jobs;
    const int lane = threadIdx.x & 31;
    const uint32_t units = p.unit_begin[p.buffers];
    const uint32_t warps = ctas * (kCopyThreads / 32), mine = (threadIdx.x >> 5) * ctas + cta;
    const uint32_t step_job = warps / units, step_unit = warps % units;
    uint32_t job = mine / units, unit = mine % units;
    while (job < (uint32_t)jobs) {
        int2 pages = p.jobs[job];
        if (COMPACT) pages.x = p.movers[jobs - 1 - job];
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

__global__ void __launch_bounds__(kCopyThreads, 2) copy_kernel(const __grid_constant__ CopyParams p) {
    griddep_wait();
    copy_pages<false>(p, blockIdx.x, gridDim.x);
}

// A compaction's copies, and in the first CTAs its counts, lists and tables (not again in the launches of further buffers).
__global__ void __launch_bounds__(kCopyThreads, 2)
    compact_copy_kernel(const __grid_constant__ CopyParams p, const __grid_constant__ Pool pool, int side) {
    extern __shared__ int smem[];
    griddep_wait();
    if ((int)blockIdx.x < side) compact_rest(pool, smem);
    else if (p.buffers) copy_pages<true>(p, blockIdx.x - side, gridDim.x - side);
}

// ------------------------------------------------------------------------- host

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

struct Layout {
    size_t map, movers, jobs, total;
    explicit Layout(int P) {
        map = align_up(sizeof(Header));
        movers = map + align_up(sizeof(int32_t) * (size_t)P);
        jobs = movers + align_up(sizeof(int32_t) * (size_t)P);
        total = jobs + align_up(sizeof(int2) * (size_t)P);
    }
};

bool sizes_ok(int B, int P) { return B >= 1 && B <= VA_PAGES_MAX_SEQS && P >= 1 && P <= VA_PAGES_MAX_PAGES; }

int check(const va_page_pool *v, Pool *p) {
    if (!v || !v->block_table || !v->seq_lens || !v->ref_count || !v->free_list || !v->num_free || !v->workspace)
        return VA_ERR_INVALID_ARGUMENT;
    if (!sizes_ok(v->num_seqs, v->num_pages) || v->block_table_stride < 1 ||
        (long long)v->num_seqs * v->block_table_stride > (1LL << 30) ||
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
    const Layout at(p->P);
    char *ws = static_cast<char *>(v->workspace);
    p->head = reinterpret_cast<Header *>(ws);
    p->map = reinterpret_cast<int32_t *>(ws + at.map);
    p->movers = reinterpret_cast<int32_t *>(ws + at.movers);
    p->jobs = reinterpret_cast<int2 *>(ws + at.jobs);
    return VA_OK;
}

// One cluster of eight CTAs whatever the sizes (one CTA alone is 0.3 us faster on 16 sequences, 2 us slower on 45), with a
// slice of the bitmap each.
void set_slices(Pool &p) {
    while ((kMaxCluster << p.slice_bits) < mask_words(p.P)) ++p.slice_bits;
}

// The most dynamic shared memory that a bookkeeping kernel asks for: fork with all sequences and as many forks, or resize with
// all sequences and an eighth of the largest bitmap.
constexpr size_t kMaxBookSmem = sizeof(int) * (6 * (size_t)VA_PAGES_MAX_SEQS + 2);
static_assert(4 * (size_t)VA_PAGES_MAX_SEQS + 1 + VA_PAGES_MAX_PAGES / 32 / kMaxCluster <= kMaxBookSmem / sizeof(int),
              "resize's arrays and its slice of the bitmap");
static_assert(kMaxBookSmem + 16 * 1024 <= kMaxSmemPerBlock, "the kernels' own arrays lie beside it");

template <typename... KArgs, typename... Args>
cudaError_t launch_book(void (*kernel)(KArgs...), size_t smem, cudaStream_t s, Args... args) {
    if (smem > 40 * 1024) {  // always the same limit: it is the function's, and other host threads launch it too
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxBookSmem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kMaxCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kMaxCluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

CopyParams copy_params(const va_page_pool *v, const Pool &p, int done) {
    CopyParams c{};
    c.head = p.head;
    c.jobs = p.jobs;
    c.movers = p.movers;
    c.buffers = std::min(kMaxBuffers, v->num_buffers - done);
    for (int i = 0; i < c.buffers; ++i) {
        const va_page_buffer &b = v->buffers[done + i];
        c.data[i] = static_cast<char *>(b.data);
        c.page_16[i] = (uint32_t)(b.page_bytes / 16);
        c.unit_begin[i + 1] = c.unit_begin[i] + (uint32_t)((b.page_bytes + kUnit - 1) / kUnit);
    }
    return c;
}

cudaError_t launch_copies(const va_page_pool *v, const Pool &p, cudaStream_t s) {
    for (int done = 0; done < v->num_buffers; done += kMaxBuffers) {
        const cudaError_t e = launch_pdl(copy_kernel, dim3(kCopyCtas), dim3(kCopyThreads), 0, s, copy_params(v, p, done));
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_compact_copies(const va_page_pool *v, const Pool &p, cudaStream_t s) {
    const size_t smem = sizeof(int) * ((size_t)p.B + 1);
    for (int done = 0; done == 0 || done < v->num_buffers; done += kMaxBuffers) {
        const int side = done == 0 ? kSideCtas : 0;
        const cudaError_t e = launch_pdl(compact_copy_kernel, dim3(v->num_buffers ? kCopyCtas : side), dim3(kCopyThreads),
                                         side ? smem : 0, s, copy_params(v, p, done), p, side);
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
    return va::sizes_ok(num_seqs, num_pages) ? va::Layout(num_pages).total : 0;
}

extern "C" int verify_attn_pages_resize_ex(const va_page_pool *pool, const int32_t *kept_lens, const int32_t *new_lens,
                                           void *stream) {
    va::Pool p;
    if (const int rc = va::check(pool, &p)) return rc;
    if (!new_lens || (reinterpret_cast<uintptr_t>(new_lens) & 3) || (reinterpret_cast<uintptr_t>(kept_lens) & 3))
        return VA_ERR_INVALID_ARGUMENT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    va::set_slices(p);
    const size_t smem = sizeof(int) * (4 * (size_t)p.B + 1 + ((size_t)1 << p.slice_bits));
    cudaError_t e = va::launch_book(va::resize_kernel, smem, s, p, kept_lens, new_lens);
    if (e == cudaSuccess) e = va::launch_copies(pool, p, s);
    return va::done(e);
}

extern "C" int verify_attn_pages_resize(const va_page_pool *pool, const int32_t *new_lens, void *stream) {
    return verify_attn_pages_resize_ex(pool, nullptr, new_lens, stream);
}

extern "C" int verify_attn_pages_fork(const va_page_pool *pool, const int32_t *parents, const int32_t *children,
                                      const int32_t *lens, int num_forks, int share, void *stream) {
    va::Pool p;
    if (const int rc = va::check(pool, &p)) return rc;
    if (num_forks < 0 || num_forks > VA_PAGES_MAX_SEQS) return VA_ERR_INVALID_ARGUMENT;
    if (num_forks == 0) return VA_OK;
    if (!parents || !children || (long long)num_forks * p.stride > (1LL << 30)) return VA_ERR_INVALID_ARGUMENT;
    for (const int32_t *x : {parents, children, lens})
        if (reinterpret_cast<uintptr_t>(x) & 3) return VA_ERR_INVALID_ARGUMENT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    va::set_slices(p);
    const size_t smem = sizeof(int) * (5 * (size_t)num_forks + 2 + (size_t)p.B);
    cudaError_t e = va::launch_book(va::fork_kernel, smem, s, p, parents, children, lens, num_forks, share);
    if (e == cudaSuccess) e = va::launch_copies(pool, p, s);
    return va::done(e);
}

extern "C" int verify_attn_pages_compact(const va_page_pool *pool, void *stream) {
    va::Pool p;
    if (const int rc = va::check(pool, &p)) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    va::set_slices(p);
    const size_t smem = sizeof(int) * ((size_t)1 << p.slice_bits);
    cudaError_t e = va::launch_book(va::compact_kernel, smem, s, p);
    if (e == cudaSuccess) e = va::launch_compact_copies(pool, p, s);
    return va::done(e);
}
