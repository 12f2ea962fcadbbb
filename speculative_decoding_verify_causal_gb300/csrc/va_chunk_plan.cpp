// Host side of chunk attention and of the weights that cached tokens gather: planning from the live lengths,
// argument checks, launches.
#include <algorithm>
#include <cmath>
#include <exception>
#include <functional>
#include <new>
#include <queue>
#include <vector>

#include "va_chunk.h"

struct va_chunk_plan {
    int num_seqs, Hq, Hkv, G, D, kv_dtype, tpt, num_sms, device;
    int total;       // rows of q, out and lse that the chunks take
    int max_blocks;  // block-table entries of the longest sequence that takes part
    int max_len;     // and its length
    int num_items, num_groups, num_parts, max_tiles, num_blocks, cluster;
    void *dev_mem;
    va::ChunkItem *items;
    va::ChunkGroup *groups;
    va::WeightItem *blocks;
    int *flags;
    float *o_part, *lse_part;
    long long workspace_bytes;
};

namespace {

constexpr int kMaxLen = 1 << 30;

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

int validate(const int32_t *chunk_lens, const int32_t *seq_lens, int B, int Hq, int Hkv, int D, int dtype) {
    if (!chunk_lens || !seq_lens || B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return VA_ERR_INVALID_ARGUMENT;
    if (D != 64 && D != 128 && D != 256) return VA_ERR_UNSUPPORTED;
    if (dtype < VA_BF16 || dtype > VA_INT2 || Hq / Hkv > va::kMmaRows) return VA_ERR_UNSUPPORTED;
    long long total = 0;
    for (int b = 0; b < B; ++b) {
        if (chunk_lens[b] < 0 || seq_lens[b] < chunk_lens[b] || seq_lens[b] > kMaxLen) return VA_ERR_INVALID_ARGUMENT;
        total += chunk_lens[b];
    }
    return total > kMaxLen ? VA_ERR_INVALID_ARGUMENT : VA_OK;
}

// Time of `costs` (descending) handed to `slots` SMs one after the other; of many items the estimate that the last
// one begins when the others are done.
double makespan(const std::vector<double> &costs, int slots) {
    if (costs.empty()) return 0.0;
    if ((int)costs.size() <= slots) return costs.front();
    if (costs.size() > 4096) {
        double sum = 0.0;
        for (double c : costs) sum += c;
        return sum / slots + costs.back();
    }
    std::priority_queue<double, std::vector<double>, std::greater<double>> load;
    for (int i = 0; i < slots; ++i) load.push(0.0);
    double worst = 0.0;
    for (double c : costs) {
        const double l = load.top() + c;
        load.pop();
        load.push(l);
        worst = std::max(worst, l);
    }
    return worst;
}

struct Geometry {
    std::vector<va::ChunkItem> items;
    std::vector<va::ChunkGroup> groups;
    std::vector<va::WeightItem> blocks;
    int num_parts = 0, max_tiles = 0, cluster = 1;
};

// One row item of one kv head before it is split: `nt` tokens, `tiles` tiles of keys.
struct Rows {
    int b, q0, nt, vis0, k_end, tiles;
};

void plan_geometry(const int32_t *chunk_lens, const int32_t *seq_lens, int B, int Hkv, int G, int D, int num_sms,
                   Geometry &g) {
    const int tpt = va::kMmaRows / G, most = tpt * va::chunk_tiles(D), keys = va::kChunkKeys;
    std::vector<Rows> rows;
    int at = 0;
    for (int b = 0; b < B; ++b) {
        const int n = chunk_lens[b], L = seq_lens[b];
        for (int t = 0; t < n; t += most) {
            const int nt = std::min(most, n - t), vis0 = L - n + t;
            const int k_end = vis0 + nt;  // the last token of the item sees the keys below
            rows.push_back({b, at + t, nt, vis0, k_end, (k_end + keys - 1) / keys});
        }
        at += n;
    }
    // Costs in units of one tile of keys of a one-tile item: a second tile of rows nearly doubles a tile's work, an
    // item has a start and an end, a split writes partials and the merge is another launch.
    const double second = 0.8, start = 2.5, split_cost = 0.5, merge = 4.0;
    auto weight = [&](const Rows &r) { return r.nt > tpt ? 1.0 + second : 1.0; };
    auto cost_of = [&](int c) {
        std::vector<double> costs;
        bool any = false;
        for (const Rows &r : rows) {
            const int pieces = (r.tiles + c - 1) / c;
            any |= pieces > 1;
            for (int i = 0; i < pieces; ++i) {
                const int len = (int)((long long)r.tiles * (i + 1) / pieces - (long long)r.tiles * i / pieces);
                const double x = start + len * weight(r) + (pieces > 1 ? split_cost : 0.0);
                costs.insert(costs.end(), Hkv, x);
            }
        }
        std::sort(costs.begin(), costs.end(), std::greater<double>());
        return makespan(costs, num_sms) + (any ? merge : 0.0);
    };
    int longest = 1;
    double units = 0.0;
    for (const Rows &r : rows) {
        longest = std::max(longest, r.tiles);
        units += (double)r.tiles * weight(r) * Hkv;
    }
    int chosen = longest;
    double best = rows.empty() ? 0.0 : cost_of(longest);
    for (double waves : {0.5, 0.75, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, 8.0, 12.0}) {
        const int c = std::max(2, (int)std::ceil(units / (num_sms * waves)));
        if (c >= longest) continue;
        const double x = cost_of(c);
        if (x < best) best = x, chosen = c;
    }
    std::vector<std::pair<double, va::ChunkItem>> items;
    for (const Rows &r : rows) {
        const int pieces = (r.tiles + chosen - 1) / chosen, tiles = r.nt > tpt ? 2 : 1;
        for (int h = 0; h < Hkv; ++h) {
            const int first = g.num_parts;
            for (int i = 0; i < pieces; ++i) {
                const int t0 = (int)((long long)r.tiles * i / pieces), t1 = (int)((long long)r.tiles * (i + 1) / pieces);
                const va::ChunkItem it = {r.b, h, r.q0, r.nt, r.vis0, t0 * keys,
                                          std::min(t1 * keys, r.k_end), pieces > 1 ? first + i * tiles : -1};
                items.push_back({(t1 - t0) * weight(r), it});
            }
            if (pieces > 1) {
                g.num_parts += pieces * tiles;
                for (int w = 0; w < tiles; ++w)
                    g.groups.push_back({h, r.q0 + w * tpt, std::min(tpt, r.nt - w * tpt), first + w, pieces, tiles, 0, 0});
            }
        }
        g.max_tiles = std::max(g.max_tiles, (r.tiles + pieces - 1) / pieces);
    }
    std::stable_sort(items.begin(), items.end(), [](const auto &a, const auto &b) { return a.first > b.first; });
    for (const auto &x : items) g.items.push_back(x.second);
}

// Blocks of keys for the gathered weights, the ones that most tiles of rows pass by first, and how many CTAs share one.
void plan_blocks(const int32_t *chunk_lens, const int32_t *seq_lens, int B, int Hkv, int G, int D, int num_sms, Geometry &g) {
    const int tpt = va::kMmaRows / G, keys = va::weight_keys(D);
    std::vector<std::pair<int, va::WeightItem>> blocks;
    int at = 0;
    for (int b = 0; b < B; at += chunk_lens[b], ++b) {
        const int n = chunk_lens[b], L = seq_lens[b];
        for (int key0 = 0; n > 0 && key0 < L; key0 += keys) {
            const int tiles = (n - std::max(0, key0 - (L - n)) + tpt - 1) / tpt;
            for (int h = 0; h < Hkv; ++h) blocks.push_back({tiles, {b, h, key0, at, n, L, 0, 0}});
        }
    }
    std::stable_sort(blocks.begin(), blocks.end(), [](const auto &a, const auto &b) { return a.first > b.first; });
    for (const auto &x : blocks) g.blocks.push_back(x.second);
    // CTAs of a block: as many as leave the longest one half of an SM's share of all tiles, where they have several each
    // (the last CTAs to end then leave few SMs idle; a CTA's start costs about two tiles)
    long long tiles = 0;
    for (const auto &x : blocks) tiles += x.first;
    while (!blocks.empty() && g.cluster < va::kWeightClusters && blocks.front().first >= 8 * g.cluster &&
           2ll * blocks.front().first * num_sms > tiles * g.cluster)
        g.cluster *= 2;
}

// Everything of a plan but its device memory.
int plan_host(const int32_t *chunk_lens, const int32_t *seq_lens, int B, int Hq, int Hkv, int D, int dtype, int num_sms,
              va_chunk_plan &p, Geometry &g) {
    try {
        plan_geometry(chunk_lens, seq_lens, B, Hkv, Hq / Hkv, D, num_sms, g);
        plan_blocks(chunk_lens, seq_lens, B, Hkv, Hq / Hkv, D, num_sms, g);
    } catch (const std::exception &) {
        return VA_ERR_OUT_OF_MEMORY;
    }
    p = {};
    p.num_seqs = B, p.Hq = Hq, p.Hkv = Hkv, p.G = Hq / Hkv, p.D = D, p.kv_dtype = dtype;
    p.tpt = va::kMmaRows / p.G;
    p.num_sms = num_sms;
    for (int b = 0; b < B; ++b) {
        p.total += chunk_lens[b];
        if (chunk_lens[b] > 0) p.max_len = std::max(p.max_len, seq_lens[b]);
    }
    p.max_blocks = (p.max_len + VA_PAGE_SIZE - 1) / VA_PAGE_SIZE;
    p.num_items = (int)g.items.size();
    p.num_groups = (int)g.groups.size();
    p.num_parts = g.num_parts;
    p.max_tiles = g.max_tiles;
    p.num_blocks = (int)g.blocks.size();
    p.cluster = g.cluster;
    return VA_OK;
}

void fill_info(const va_chunk_plan &p, va_chunk_plan_info *info) {
    *info = {p.num_seqs, p.Hq, p.Hkv, p.D, p.kv_dtype, p.total, p.max_blocks, p.num_items, p.num_groups,
             p.max_tiles * va::kChunkKeys, p.num_sms, p.workspace_bytes};
}

int fail(cudaError_t e) {
    va::note_cuda_error(e);
    cudaGetLastError();
    return VA_ERR_CUDA;
}

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// The tensor maps are made by the driver, which needs a context; a host thread has one from its first runtime call
// on.  A question about the stream is one that is allowed while it is captured.
int bind_thread(cudaStream_t s) {
    thread_local bool bound = false;
    if (bound) return VA_OK;
    cudaStreamCaptureStatus capture;
    const cudaError_t e = cudaStreamIsCapturing(s, &capture);
    if (e != cudaSuccess) return fail(e);
    bound = true;
    return VA_OK;
}

// q as the kernels read it: strides that nothing is reached by are replaced by ones that a tensor map takes.
int check_q(const va_chunk_plan *p, const va_heads *q, va_heads &out) {
    if (!q || !q->data || q->num_heads != p->Hq || !aligned(q->data, 16)) return VA_ERR_INVALID_ARGUMENT;
    out = *q;
    if (p->Hq == 1) out.stride_head = p->D;
    if (p->total == 1) out.stride_token = (int64_t)p->Hq * p->D;
    for (int64_t s : {out.stride_head, out.stride_token})
        if (s <= 0 || s % 8 != 0 || s >= (1ll << 38)) return VA_ERR_INVALID_ARGUMENT;
    return VA_OK;
}

}  // namespace

extern "C" {

int verify_attn_chunk_plan(const int32_t *chunk_lens, const int32_t *seq_lens, int num_seqs, int num_q_heads,
                           int num_kv_heads, int head_dim, va_kv_dtype kv_dtype, int num_sms, va_chunk_plan **out_plan) {
    if (!out_plan) return VA_ERR_INVALID_ARGUMENT;
    *out_plan = nullptr;
    const int rc = validate(chunk_lens, seq_lens, num_seqs, num_q_heads, num_kv_heads, head_dim, kv_dtype);
    if (rc != VA_OK) return rc;
    if (num_sms < 0) return VA_ERR_INVALID_ARGUMENT;
    int device = 0, sms = 0;
    if (cudaGetDevice(&device) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) {
        cudaGetLastError();
        return VA_ERR_NO_DEVICE;
    }
    if (num_sms == 0) num_sms = sms;
    Geometry g;
    va_chunk_plan *p = new (std::nothrow) va_chunk_plan();
    if (!p) return VA_ERR_OUT_OF_MEMORY;
    const int made = plan_host(chunk_lens, seq_lens, num_seqs, num_q_heads, num_kv_heads, head_dim, kv_dtype, num_sms, *p, g);
    if (made != VA_OK) {
        delete p;
        return made;
    }
    p->device = device;
    const size_t items = align_up(sizeof(va::ChunkItem) * g.items.size());
    const size_t groups = align_up(sizeof(va::ChunkGroup) * g.groups.size());
    const size_t blocks = align_up(sizeof(va::WeightItem) * g.blocks.size());
    const size_t lse = align_up(sizeof(float) * g.num_parts * va::kMmaRows);
    const size_t total = 256 + items + groups + blocks + lse + sizeof(float) * g.num_parts * va::kMmaRows * (size_t)head_dim;
    if (cudaMalloc(&p->dev_mem, total) != cudaSuccess) {
        cudaGetLastError();
        delete p;
        return VA_ERR_OUT_OF_MEMORY;
    }
    char *at = static_cast<char *>(p->dev_mem);
    p->flags = reinterpret_cast<int *>(at);
    p->items = reinterpret_cast<va::ChunkItem *>(at += 256);
    p->groups = reinterpret_cast<va::ChunkGroup *>(at += items);
    p->blocks = reinterpret_cast<va::WeightItem *>(at += groups);
    p->lse_part = reinterpret_cast<float *>(at += blocks);
    p->o_part = reinterpret_cast<float *>(at += lse);
    p->workspace_bytes = (long long)total;
    auto copy = [](void *to, const void *from, size_t n) {
        return n == 0 ? cudaSuccess : cudaMemcpy(to, from, n, cudaMemcpyHostToDevice);
    };
    cudaError_t e = copy(p->items, g.items.data(), sizeof(va::ChunkItem) * g.items.size());
    if (e == cudaSuccess) e = copy(p->groups, g.groups.data(), sizeof(va::ChunkGroup) * g.groups.size());
    if (e == cudaSuccess) e = copy(p->blocks, g.blocks.data(), sizeof(va::WeightItem) * g.blocks.size());
    if (e == cudaSuccess) e = cudaMemset(p->flags, 0, 256);
    // copies and the memset may still be under way, and streams that do not wait for the legacy one come next
    if (e == cudaSuccess) e = cudaStreamSynchronize(cudaStreamLegacy);
    if (e != cudaSuccess) {
        cudaFree(p->dev_mem);
        delete p;
        return fail(e);
    }
    *out_plan = p;
    return VA_OK;
}

int verify_attn_chunk_plan_describe(const int32_t *chunk_lens, const int32_t *seq_lens, int num_seqs, int num_q_heads,
                                    int num_kv_heads, int head_dim, va_kv_dtype kv_dtype, int num_sms,
                                    va_chunk_plan_info *info, int32_t *out, int max_items) {
    const int rc = validate(chunk_lens, seq_lens, num_seqs, num_q_heads, num_kv_heads, head_dim, kv_dtype);
    if (rc != VA_OK) return rc;
    if (num_sms < 1 || !info || (out && max_items < 0)) return VA_ERR_INVALID_ARGUMENT;
    Geometry g;
    va_chunk_plan p;
    const int made = plan_host(chunk_lens, seq_lens, num_seqs, num_q_heads, num_kv_heads, head_dim, kv_dtype, num_sms, p, g);
    if (made != VA_OK) return made;
    fill_info(p, info);
    for (int i = 0; out && i < std::min(max_items, p.num_items); ++i) {
        const va::ChunkItem &it = g.items[i];
        const int32_t x[6] = {it.b, it.kvh, it.q0, it.nt, it.k_begin, it.k_end};
        std::copy(x, x + 6, out + 6 * i);
    }
    return VA_OK;
}

void verify_attn_chunk_plan_destroy(va_chunk_plan *p) {
    if (!p) return;
    cudaFree(p->dev_mem);
    delete p;
}

int verify_attn_chunk_plan_get_info(const va_chunk_plan *p, va_chunk_plan_info *info) {
    if (!p || !info) return VA_ERR_INVALID_ARGUMENT;
    fill_info(*p, info);
    return VA_OK;
}

int verify_attn_chunk_plan_device_flags(const va_chunk_plan *p, int clear, int *flags, void *stream) {
    if (!p || !flags) return VA_ERR_INVALID_ARGUMENT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int host = 0;
    cudaError_t e = cudaMemcpyAsync(&host, p->flags, sizeof(int), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess && clear) e = cudaMemsetAsync(p->flags, 0, sizeof(int), s);
    if (e != cudaSuccess) return fail(e);
    *flags = host;
    return VA_OK;
}

int verify_attn_chunk(const va_chunk_plan *p, const va_heads *q, const void *k_pages, const void *v_pages,
                      const float *k_scale, const float *v_scale, const int32_t *block_table, int block_table_stride,
                      int num_pages, void *out, float *lse, void *stream) {
    if (!p) return VA_ERR_NO_PLAN;
    if (p->total == 0) return VA_OK;  // tensors without elements have no addresses
    va_heads qv;
    int rc = check_q(p, q, qv);
    if (rc != VA_OK) return rc;
    if (!k_pages || !v_pages || !block_table || !out || num_pages < 0 || block_table_stride < p->max_blocks)
        return VA_ERR_INVALID_ARGUMENT;
    if (p->kv_dtype != VA_BF16 && (!k_scale || !v_scale)) return VA_ERR_INVALID_ARGUMENT;
    if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(out, 16) || !aligned(block_table, 4) ||
        !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(lse, 4))
        return VA_ERR_INVALID_ARGUMENT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    rc = bind_thread(s);
    if (rc != VA_OK) return rc;
    const float scale = (float)(1.4426950408889634 / std::sqrt((double)p->D));
    const va::ChunkParams cp = {k_pages, v_pages, k_scale, v_scale, block_table, p->items, static_cast<uint16_t *>(out),
                                lse, p->o_part, p->lse_part, p->flags, block_table_stride, p->Hq, p->Hkv, p->G, p->tpt,
                                num_pages, scale};
    cudaError_t e = va::launch_chunk(cp, qv, p->total, p->D, p->kv_dtype, p->num_items, s);
    if (e == cudaSuccess && p->num_groups > 0) {
        const va::ChunkCombineParams mp = {p->groups, p->o_part, p->lse_part, cp.out, lse, p->Hq, p->G, p->D};
        e = va::launch_chunk_combine(mp, p->num_groups, p->num_sms, s);
    }
    return e == cudaSuccess ? VA_OK : fail(e);
}

int verify_attn_chunk_weights(const va_chunk_plan *p, const va_heads *q, const void *k_pages, const float *k_scale,
                              const int32_t *block_table, int block_table_stride, int num_pages, const float *lse,
                              float *weights, int64_t weights_stride_seq, int64_t weights_stride_head, int accumulate,
                              int32_t *slot_pos, const int32_t *positions, void *stream) {
    if (!p) return VA_ERR_NO_PLAN;
    if (p->total == 0) return VA_OK;  // tensors without elements have no addresses
    va_heads qv;
    int rc = check_q(p, q, qv);
    if (rc != VA_OK) return rc;
    if (!k_pages || !block_table || !lse || !weights || num_pages < 0 || block_table_stride < p->max_blocks ||
        (slot_pos && !positions) || weights_stride_seq < 0 || weights_stride_head < 0 ||
        va::rows_overlap(weights_stride_seq, weights_stride_head, p->num_seqs, p->Hkv, p->max_len))
        return VA_ERR_INVALID_ARGUMENT;
    if (p->kv_dtype != VA_BF16 && !k_scale) return VA_ERR_INVALID_ARGUMENT;
    if (!aligned(k_pages, 16) || !aligned(block_table, 4) || !aligned(k_scale, 4) || !aligned(lse, 4) ||
        !aligned(weights, 4) || !aligned(slot_pos, 4) || !aligned(positions, 4))
        return VA_ERR_INVALID_ARGUMENT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    rc = bind_thread(s);
    if (rc != VA_OK) return rc;
    const float scale = (float)(1.4426950408889634 / std::sqrt((double)p->D));
    const va::WeightParams wp = {k_pages, k_scale, lse, block_table, p->blocks, weights, slot_pos, positions,
                                 weights_stride_seq, weights_stride_head, p->flags, block_table_stride, p->Hq, p->Hkv,
                                 p->G, p->tpt, num_pages, accumulate != 0, p->cluster, scale};
    const cudaError_t e = va::launch_weights(wp, qv, p->total, p->D, p->kv_dtype, p->num_blocks, s);
    return e == cudaSuccess ? VA_OK : fail(e);
}

}  // extern "C"
