// Host side of the paged key/value cache: argument checks and launches.  All
// state is the caller's; nothing here allocates, copies or waits, so every
// call may be captured into a CUDA graph.

#include <limits.h>
#include <math.h>

#include <algorithm>
#include <initializer_list>
#include <utility>

#include "tb_internal.h"
#include "tb_kv.h"

namespace {

using tb::fail;

int elem_bytes(int dtype)
{
    switch (dtype) {
    case TB_DTYPE_F16:
    case TB_DTYPE_BF16:
        return 2;
    case TB_DTYPE_F32:
        return 4;
    case TB_DTYPE_BYTE:
        return 1;
    default:
        return 0;
    }
}

bool unaligned(const void *p, uintptr_t to)
{
    return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0;
}

// Checks the sizes and, where asked, the pools and the page table of *cache.
int view_of(tb_ctx *ctx, const tb_kv_cache *cache, bool pools, bool table, const char *who,
            tb::KvView *out)
{
    if (!cache)
        return fail(ctx, TB_EINVAL, "%s: null cache", who);
    const tb_kv_cache &c = *cache;
    const int elem = elem_bytes(c.dtype);
    if (!elem || c.pages < 1 || c.page_tokens < 1)
        return fail(ctx, TB_EINVAL, "%s: dtype TB_DTYPE_*, pages >= 1, page_tokens >= 1", who);
    tb::KvView v{};
    v.pages = c.pages;
    v.page_tokens = c.page_tokens;
    if (pools) {
        if (!c.k || !c.v || c.layers < 1 || c.kv_heads < 1 || c.head_dim < 1)
            return fail(ctx, TB_EINVAL, "%s: null pool, or layers, kv_heads or head_dim < 1", who);
        const int64_t row = (int64_t)c.head_dim * elem;
        if (c.layers > 65535 || c.kv_heads > 65535)
            return fail(ctx, TB_ENOTSUP, "%s: more than 65535 layers or heads", who);
        if (row > (1 << 20) || (row | c.layer_stride | c.page_stride | c.token_stride | c.head_stride) & 15 ||
            unaligned(c.k, 16) || unaligned(c.v, 16))
            return fail(ctx, TB_EINVAL,
                        "%s: pools, strides and head_dim * element size must be multiples of 16 "
                        "bytes (head_dim * element size at most 1 MiB)",
                        who);
        // No two rows may share an address: with the strides in ascending
        // order each has to clear what the ones before it span.
        std::pair<int64_t, int64_t> dim[4] = {{c.layer_stride, c.layers},
                                              {c.page_stride, c.pages},
                                              {c.token_stride, c.page_tokens},
                                              {c.head_stride, c.kv_heads}};
        std::sort(dim, dim + 4);
        int64_t span = row;
        for (const auto &d : dim) {
            if (d.second == 1)
                continue;
            int64_t reach = 0;
            if (d.first < span || __builtin_mul_overflow(d.first, d.second - 1, &reach) ||
                __builtin_add_overflow(span, reach, &span))
                return fail(ctx, TB_EINVAL, "%s: two elements of a pool share an address, or its "
                                            "size overflows", who);
        }
        // Bytes of a page's rows of one layer: what the copies count in 32 bits.
        if ((int64_t)c.page_tokens * c.kv_heads > INT_MAX / row)
            return fail(ctx, TB_ENOTSUP, "%s: a page of a layer holds more than 2 GiB", who);
        v.pool[0] = static_cast<char *>(c.k);
        v.pool[1] = static_cast<char *>(c.v);
        v.layers = c.layers;
        v.heads = c.kv_heads;
        v.row_bytes = (int32_t)row;
        v.layer_stride = c.layer_stride;
        v.page_stride = c.page_stride;
        v.token_stride = c.token_stride;
        v.head_stride = c.head_stride;
    }
    if (table) {
        if (!c.table || !c.held || !c.lens || !c.refs || c.slots < 1 || c.table_width < 1)
            return fail(ctx, TB_EINVAL,
                        "%s: null table, held, lens or refs, or slots or table_width < 1", who);
        // Positions of a slot are counted in 32 bits.
        if (c.table_width > (1 << 30) / c.page_tokens)
            return fail(ctx, TB_ENOTSUP, "%s: table_width * page_tokens exceeds 2^30", who);
        if (c.pages > 1 << 30 || c.slots > INT_MAX / c.table_width)
            return fail(ctx, TB_ENOTSUP, "%s: more than 2^30 pages or 2^31 - 1 table entries", who);
        v.table = c.table;
        v.held = c.held;
        v.lens = c.lens;
        v.refs = c.refs;
        v.slots = c.slots;
        v.width = c.table_width;
    }
    *out = v;
    return TB_OK;
}

// Whether an element of the one pool lies on one of the other: whether some
// difference of two rows' places is within a row of the pools' distance.  As
// the strides are nested (view_of), the largest one's multiple has to be the
// one below or above what is left, and so on down.
bool pools_meet(const tb::KvView &v)
{
    std::pair<int64_t, int64_t> dim[4] = {{v.layer_stride, v.layers},
                                          {v.page_stride, v.pages},
                                          {v.token_stride, v.page_tokens},
                                          {v.head_stride, v.heads}};
    std::sort(dim, dim + 4);
    int64_t left[16] = {(int64_t)((uintptr_t)v.pool[1] - (uintptr_t)v.pool[0])};
    int n = 1;
    for (int d = 3; d >= 0; --d) {
        if (dim[d].second == 1)
            continue;
        for (int i = n - 1; i >= 0; --i) {
            const int64_t stride = dim[d].first, most = dim[d].second - 1;
            int64_t low = left[i] / stride;
            if (low * stride > left[i])
                --low;
            const int64_t a = std::min(std::max(low, -most), most);
            const int64_t b = std::min(std::max(low + 1, -most), most);
            left[i] -= a * stride;
            left[n + i] = left[i] + (a - b) * stride;
        }
        n *= 2;
    }
    return std::any_of(left, left + n, [&](int64_t x) { return x > -v.row_bytes && x < v.row_bytes; });
}

// An array of 32-bit words.
struct Words {
    const int32_t *at;
    uint64_t n;
};

// Whether two arrays share no word (an empty one shares none).
bool apart(const Words &a, const Words &b)
{
    return !a.n || !b.n || reinterpret_cast<uintptr_t>(a.at) + 4 * a.n <= reinterpret_cast<uintptr_t>(b.at) ||
           reinterpret_cast<uintptr_t>(b.at) + 4 * b.n <= reinterpret_cast<uintptr_t>(a.at);
}

bool apart(const Words &a, std::initializer_list<Words> others)
{
    return std::all_of(others.begin(), others.end(), [&](const Words &b) { return apart(a, b); });
}

int launched(tb_ctx *ctx, cudaError_t e, const char *what)
{
    return e == cudaSuccess ? TB_OK : tb::cuda_fail(ctx, e, what);
}

}  // namespace

extern "C" {

int tb_kv_copy_pages(tb_ctx *ctx, const tb_kv_cache *cache, const int32_t *src, const int32_t *dst,
                     const int32_t *tokens, int32_t n, tb_stream stream)
{
    if (!ctx)
        return TB_EINVAL;
    tb::KvView v;
    int rc = view_of(ctx, cache, true, false, "kv_copy_pages", &v);
    if (rc != TB_OK)
        return rc;
    if (n < 0 || (n > 0 && (!src || !dst)))
        return fail(ctx, TB_EINVAL, "kv_copy_pages: n < 0 or a null page list");
    if (n == 0)
        return TB_OK;
    tb::DeviceScope scope(tb::ctx_device(ctx));
    return launched(ctx,
                    tb::launch_copy_pages(v, src, dst, tokens, n, tb::ctx_options(ctx).use_pdl != 0,
                                          static_cast<cudaStream_t>(stream)),
                    "launch of the page copy");
}

int tb_kv_resize(tb_ctx *ctx, const tb_kv_cache *cache, const int32_t *capacity, int32_t *status,
                 tb_stream stream)
{
    if (!ctx)
        return TB_EINVAL;
    tb::KvView v;
    int rc = view_of(ctx, cache, false, true, "kv_resize", &v);
    if (rc != TB_OK)
        return rc;
    if (!capacity || !status)
        return fail(ctx, TB_EINVAL, "kv_resize: null capacity or status");
    if (v.slots > TB_KV_MAX_SLOTS)
        return fail(ctx, TB_ENOTSUP, "kv_resize: more than %d slots", TB_KV_MAX_SLOTS);
    const uint64_t slots = (uint64_t)v.slots;
    const Words table{v.table, slots * (uint64_t)v.width}, held{v.held, slots}, lens{v.lens, slots},
        refs{v.refs, (uint64_t)v.pages}, caps{capacity, slots};
    // (Capacities that are the lengths themselves stay what they are.)
    if (!apart(caps, {table, held, refs}) || !apart(Words{status, 1}, {table, held, lens, refs, caps}))
        return fail(ctx, TB_EINVAL, "kv_resize: capacity or status overlaps what the call changes, or "
                                    "status overlaps capacity");
    tb::DeviceScope scope(tb::ctx_device(ctx));
    return launched(ctx,
                    tb::launch_kv_resize(v, capacity, status, tb::ctx_options(ctx).use_pdl != 0,
                                         static_cast<cudaStream_t>(stream)),
                    "launch of the resize");
}

int tb_kv_fork(tb_ctx *ctx, const tb_kv_cache *cache, const int32_t *parents, int32_t *table_out,
               int32_t *held_out, int32_t *lens_out, int32_t *status, tb_stream stream)
{
    if (!ctx)
        return TB_EINVAL;
    tb::KvView v;
    int rc = view_of(ctx, cache, true, true, "kv_fork", &v);
    if (rc != TB_OK)
        return rc;
    if (!parents || !table_out || !held_out || !lens_out || !status)
        return fail(ctx, TB_EINVAL, "kv_fork: null parents, output or status");
    if (v.slots > TB_KV_MAX_SLOTS)
        return fail(ctx, TB_ENOTSUP, "kv_fork: more than %d slots", TB_KV_MAX_SLOTS);
    const uint64_t slots = (uint64_t)v.slots, rows = slots * (uint64_t)v.width;
    const Words table{v.table, rows}, held{v.held, slots}, lens{v.lens, slots}, refs{v.refs, (uint64_t)v.pages},
        list{parents, slots};
    const Words outs[] = {{table_out, rows}, {held_out, slots}, {lens_out, slots}, {status, 1}};
    for (int i = 0; i < 4; ++i) {
        bool fine = apart(outs[i], {table, held, lens, refs, list});
        for (int j = 0; j < i; ++j)
            fine = fine && apart(outs[i], outs[j]);
        if (!fine)
            return fail(ctx, TB_EINVAL, "kv_fork: an output or status overlaps an input or another output");
    }
    if (!apart(refs, list))
        return fail(ctx, TB_EINVAL, "kv_fork: parents overlaps refs");
    tb::DeviceScope scope(tb::ctx_device(ctx));
    return launched(ctx,
                    tb::launch_kv_fork(v, parents, table_out, held_out, lens_out, status,
                                       tb::ctx_options(ctx).use_pdl != 0,
                                       static_cast<cudaStream_t>(stream)),
                    "launch of the fork");
}

int tb_kv_compact(tb_ctx *ctx, const tb_kv_cache *cache, const int32_t *start, const int32_t *keep,
                  int32_t keep_stride, const int32_t *count, int32_t *status, tb_stream stream)
{
    if (!ctx)
        return TB_EINVAL;
    tb::KvView v;
    int rc = view_of(ctx, cache, true, true, "kv_compact", &v);
    if (rc != TB_OK)
        return rc;
    if (!start || !count || !status || keep_stride < 0 || (keep_stride > 0 && !keep))
        return fail(ctx, TB_EINVAL,
                    "kv_compact: null start, keep, count or status, or keep_stride < 0");
    if (pools_meet(v))
        return fail(ctx, TB_EINVAL, "kv_compact: the two pools share an element");
    const uint64_t slots = (uint64_t)v.slots;
    const Words table{v.table, slots * (uint64_t)v.width}, held{v.held, slots}, lens{v.lens, slots},
        refs{v.refs, (uint64_t)v.pages}, from{start, slots}, kept{keep, slots * (uint64_t)keep_stride},
        counts{count, slots};
    if (!apart(lens, {from, kept, counts}))
        return fail(ctx, TB_EINVAL, "kv_compact: start, keep or count overlaps the cache's lens");
    if (!apart(Words{status, slots}, {table, held, lens, refs, from, kept, counts}))
        return fail(ctx, TB_EINVAL, "kv_compact: status overlaps an input or the cache's arrays");
    if (v.slots > 65535)
        return fail(ctx, TB_ENOTSUP, "kv_compact: more than 65535 slots");
    tb::DeviceScope scope(tb::ctx_device(ctx));
    return launched(ctx,
                    tb::launch_kv_compact(v, start, keep, keep_stride, count, status,
                                          tb::ctx_options(ctx).use_pdl != 0,
                                          static_cast<cudaStream_t>(stream)),
                    "launch of the compaction");
}

int tb_tree_attention_workspace(tb_ctx *ctx, const tb_kv_cache *cache, int32_t q_heads,
                                uint64_t *bytes)
{
    if (!ctx)
        return TB_EINVAL;
    if (!cache || !bytes || cache->kv_heads < 1 || q_heads < 1 || q_heads % cache->kv_heads)
        return fail(ctx, TB_EINVAL, "tree_attention_workspace: null argument, or q_heads not a "
                                    "positive multiple of kv_heads");
    *bytes = tb::tree_workspace_bytes(tb::ctx_num_sms(ctx), cache->head_dim);
    return TB_OK;
}

int tb_tree_attention(tb_ctx *ctx, const tb_tree *t, tb_stream stream)
{
    if (!ctx)
        return TB_EINVAL;
    if (!t)
        return fail(ctx, TB_EINVAL, "tree_attention: null arguments");
    tb::TreePlan p{};
    volatile uint32_t *expired = tb::ctx_tree_status(ctx, &p.status);
    if (*expired != 0u) {
        *expired = 0u;
        return fail(ctx, TB_ETIMEOUT, "an earlier tree attention on this context stopped early: a "
                                      "bounded wait inside the kernel expired");
    }
    int rc = view_of(ctx, t->cache, true, true, "tree_attention", &p.c);
    if (rc != TB_OK)
        return rc;
    const tb_kv_cache &c = *t->cache;
    if (t->layer < 0 || t->layer >= c.layers || t->seqs < 0 || t->rows < 0 || t->mask_words < 0 ||
        t->q_heads < 1 || t->q_heads % c.kv_heads)
        return fail(ctx, TB_EINVAL, "tree_attention: layer in [0, layers), seqs, rows, mask_words "
                                    ">= 0, q_heads a positive multiple of kv_heads");
    if (c.dtype != TB_DTYPE_F16 && c.dtype != TB_DTYPE_BF16)
        return fail(ctx, TB_ENOTSUP, "tree_attention: the cache must be TB_DTYPE_F16 or _BF16");
    if (c.head_dim > 128)
        return fail(ctx, TB_ENOTSUP, "tree_attention: head_dim %d is more than 128", c.head_dim);
    if (t->seqs > TB_TREE_MAX_SEQS)
        return fail(ctx, TB_ENOTSUP, "tree_attention: more than %d sequences", TB_TREE_MAX_SEQS);
    if (t->rows > (1 << 29) || t->rows > (1 << 30) / t->q_heads)
        return fail(ctx, TB_ENOTSUP, "tree_attention: rows exceeds 2^29 or rows * q_heads 2^30");
    // Work is counted in 32 bits, in tiles of 128 positions: what the longest
    // rows of the table and all query rows could make of it.
    const int64_t tiles = (int64_t)c.table_width * c.page_tokens / 128 + t->rows / 128 + 8;
    const int64_t units = (int64_t)t->rows * (t->q_heads / c.kv_heads) / 128 + t->seqs;
    if (units * c.kv_heads > INT_MAX / tiles)
        return fail(ctx, TB_ENOTSUP, "tree_attention: rows, heads and table_width make more than 2^31 - 1 "
                                     "tiles of work");
    if (!t->seq_slots && t->seqs > c.slots)
        return fail(ctx, TB_EINVAL, "tree_attention: more sequences than slots");
    if (!isfinite(t->scale))
        return fail(ctx, TB_EINVAL, "tree_attention: scale is not finite");
    if (t->seqs == 0 || t->rows == 0)
        return TB_OK;
    if (!t->q_start || !t->q || !t->out || (t->mask_words > 0 && !t->mask))
        return fail(ctx, TB_EINVAL, "tree_attention: null q_start, q, out or mask");
    if ((t->q_row_stride | t->q_head_stride | t->out_row_stride | t->out_head_stride) & 15 ||
        unaligned(t->q, 16) || unaligned(t->out, 16))
        return fail(ctx, TB_EINVAL, "tree_attention: q, out and their strides must be multiples of "
                                    "16 bytes");
    if (!t->workspace || unaligned(t->workspace, 16) ||
        t->workspace_bytes < tb::tree_workspace_bytes(tb::ctx_num_sms(ctx), c.head_dim))
        return fail(ctx, TB_EINVAL, "tree_attention: workspace null, not 16-byte aligned or "
                                    "smaller than tb_tree_attention_workspace");
    p.c.pool[0] += (int64_t)t->layer * c.layer_stride;
    p.c.pool[1] += (int64_t)t->layer * c.layer_stride;
    p.bf16 = c.dtype == TB_DTYPE_BF16;
    p.head_dim = c.head_dim;
    p.seqs = t->seqs;
    p.rows = t->rows;
    p.q_heads = t->q_heads;
    p.group = t->q_heads / c.kv_heads;
    p.mask_words = t->mask_words;
    p.seq_slots = t->seq_slots;
    p.q_start = t->q_start;
    p.q = static_cast<const char *>(t->q);
    p.out = static_cast<char *>(t->out);
    p.q_row = t->q_row_stride;
    p.q_head = t->q_head_stride;
    p.o_row = t->out_row_stride;
    p.o_head = t->out_head_stride;
    p.lse = t->lse;
    p.mask = t->mask;
    p.workspace = t->workspace;
    p.scale = t->scale;
    p.wait_ns = tb::ctx_options(ctx).kernel_wait_ns;
    tb::DeviceScope scope(tb::ctx_device(ctx));
    return launched(ctx,
                    tb::launch_tree(p, tb::ctx_num_sms(ctx), tb::ctx_options(ctx).use_pdl != 0,
                                    static_cast<cudaStream_t>(stream)),
                    "launch of the tree attention");
}

}  // extern "C"
