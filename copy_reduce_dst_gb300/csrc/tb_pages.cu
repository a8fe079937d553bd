// Page operations of the paged key/value cache (sm_103a): pages copied, given
// to and taken from slots, forked between slots, and tokens squeezed together
// inside a slot.  All lists are read on the device.

#include <cuda_runtime.h>
#include <stdint.h>

#include "tb_device.cuh"
#include "tb_kv.h"

namespace tb {
namespace {

using namespace dev;

constexpr int kPageThreads = 256;
constexpr int kPlanThreads = 1024;

// The bytes that the first `tokens` tokens of a page cover in one layer:
// n1 x n2 runs of `bytes` contiguous bytes.  Rows that lie one after another
// join into longer runs.
struct Runs {
    uint32_t n1, n2, bytes;
    int64_t s1, s2;
};

__device__ __forceinline__ Runs page_runs(const KvView &c, uint32_t tokens)
{
    const uint32_t row = c.row_bytes, heads = c.heads;
    Runs r{1, 1, 0, 0, 0};
    if (c.heads == 1 || c.head_stride == row) {  // a token's heads are contiguous
        if (c.token_stride == (int64_t)heads * row) {
            r.bytes = tokens * heads * row;
        } else {
            r.n1 = tokens;
            r.s1 = c.token_stride;
            r.bytes = heads * row;
        }
    } else if (c.page_tokens == 1 || c.token_stride == row) {  // a head's tokens are contiguous
        r.bytes = tokens * row;
        if ((int32_t)tokens == c.page_tokens && c.head_stride == (int64_t)r.bytes) {
            r.bytes *= heads;
        } else {
            r.n1 = heads;
            r.s1 = c.head_stride;
        }
    } else {
        r.n1 = tokens;
        r.s1 = c.token_stride;
        r.n2 = heads;
        r.s2 = c.head_stride;
        r.bytes = row;
    }
    return r;
}

// One page of one layer by a whole CTA, 16 bytes a thread and step.
__device__ __forceinline__ void copy_page(const KvView &c, char *pool, int32_t src, int32_t dst,
                                          uint32_t tokens)
{
    const Runs r = page_runs(c, tokens);
    const uint32_t per_run = r.bytes / 16, total = r.n1 * r.n2 * per_run;
    const char *from = pool + src * c.page_stride;
    char *to = pool + dst * c.page_stride;
    for (uint32_t i = threadIdx.x; i < total; i += blockDim.x) {
        const uint32_t run = i / per_run;
        const int64_t at = (run / r.n2) * r.s1 + (run % r.n2) * r.s2 + (int64_t)(i % per_run) * 16;
        *reinterpret_cast<uint4 *>(to + at) = *reinterpret_cast<const uint4 *>(from + at);
    }
}

__device__ __forceinline__ bool is_page(const KvView &c, int32_t p)
{
    return p >= 0 && p < c.pages;
}

__global__ void __launch_bounds__(kPageThreads)
    k_copy_pages(const KvView c, const int32_t *src, const int32_t *dst, const int32_t *tokens,
                 int64_t jobs)
{
    pdl_launch_dependents();
    pdl_wait_prerequisite();
    for (int64_t j = blockIdx.x; j < jobs; j += gridDim.x) {
        const int64_t i = j / (2 * c.layers);
        const int32_t lane = (int32_t)(j % (2 * c.layers));
        const int32_t s = src[i], d = dst[i];
        const int32_t t = tokens ? min(max(tokens[i], 0), c.page_tokens) : c.page_tokens;
        if (is_page(c, s) && is_page(c, d) && s != d && t > 0)
            copy_page(c, c.pool[lane & 1] + (lane >> 1) * c.layer_stride, s, d, (uint32_t)t);
    }
}

// Sum over the CTA before this thread, and the CTA's total; warp_sums: 33 ints.
__device__ int scan_before(int v, int *warp_sums, int &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d)
            x += y;
    }
    __syncthreads();
    if (lane == 31)
        warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int w = lane < (int)(blockDim.x >> 5) ? warp_sums[lane] : 0;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int y = __shfl_up_sync(0xffffffffu, w, d);
            if (lane >= d)
                w += y;
        }
        warp_sums[lane] = w;
    }
    __syncthreads();
    total = warp_sums[31];
    return x - v + (warp ? warp_sums[warp - 1] : 0);
}

__device__ __forceinline__ int pages_for(int tokens, int page_tokens)
{
    return tokens / page_tokens + (tokens % page_tokens != 0);
}

// Free pages of the pool.
__device__ int count_free(const KvView &c, int *warp_sums)
{
    int mine = 0, total;
    for (int p = threadIdx.x; p < c.pages; p += blockDim.x)
        mine += c.refs[p] == 0;
    scan_before(mine, warp_sums, total);
    return total;
}

// Calls take(rank, page) for the `wanted` lowest free pages, in any order.
template <class Take>
__device__ void take_free(const KvView &c, int wanted, int *warp_sums, Take take)
{
    int rank = 0;
    for (int base = 0; base < c.pages && rank < wanted; base += blockDim.x) {
        const int p = base + (int)threadIdx.x;
        const int is_free = p < c.pages && c.refs[p] == 0;
        int total;
        const int mine = rank + scan_before(is_free, warp_sums, total);
        if (is_free && mine < wanted)
            take(mine, p);
        rank += total;
    }
}

__global__ void __launch_bounds__(kPlanThreads)
    k_kv_resize(const KvView c, const int32_t *capacity, int32_t *status)
{
    extern __shared__ int first_rank[];  // [slots]: rank of the first page each slot takes
    __shared__ int warp_sums[33];
    __shared__ int bad;
    pdl_launch_dependents();
    pdl_wait_prerequisite();
    if (threadIdx.x == 0)
        bad = 0;
    __syncthreads();
    int wanted = 0;
    for (int base = 0; base < c.slots; base += blockDim.x) {
        const int s = base + (int)threadIdx.x;
        int grow = 0;
        if (s < c.slots && capacity[s] >= 0) {
            const int cap = capacity[s], held = min(max(c.held[s], 0), c.width);
            const int need = pages_for(cap, c.page_tokens);
            if (need > c.width)
                bad = 1;
            // The last page kept is written again past the cut: not if it is shared.
            if (cap < c.lens[s] && cap % c.page_tokens && need <= held) {
                const int p = c.table[(int64_t)s * c.width + need - 1];
                if (is_page(c, p) && c.refs[p] > 1)
                    bad = 1;
            }
            grow = max(need - held, 0);
        }
        int total;
        const int before = scan_before(min(grow, c.width), warp_sums, total);
        if (s < c.slots)
            first_rank[s] = wanted + before;
        wanted += total;
    }
    const int missing = wanted ? max(wanted - count_free(c, warp_sums), 0) : 0;
    __syncthreads();
    const int verdict = bad ? -1 : missing;
    if (threadIdx.x == 0)
        *status = verdict;
    if (verdict)
        return;
    take_free(c, wanted, warp_sums, [&](int rank, int p) {
        int lo = 0, hi = c.slots;  // the last slot whose first rank is <= rank
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (first_rank[mid] <= rank)
                lo = mid;
            else
                hi = mid;
        }
        const int held = min(max(c.held[lo], 0), c.width);
        c.table[(int64_t)lo * c.width + held + rank - first_rank[lo]] = p;
        c.refs[p] = 1;
    });
    __syncthreads();
    for (int s = threadIdx.x >> 5; s < c.slots; s += blockDim.x >> 5) {
        const int cap = capacity[s];
        if (cap < 0)
            continue;
        const int held = min(max(c.held[s], 0), c.width), need = pages_for(cap, c.page_tokens);
        for (int j = need + (int)(threadIdx.x & 31); j < held; j += 32) {
            int32_t *entry = c.table + (int64_t)s * c.width + j;
            if (is_page(c, *entry))
                atomicSub(c.refs + *entry, 1);
            *entry = -1;
        }
        __syncwarp();
        if ((threadIdx.x & 31) == 0) {
            c.held[s] = need;
            c.lens[s] = min(c.lens[s], cap);
        }
    }
}

// ---------------------------------------------------------------------------
// Fork
// ---------------------------------------------------------------------------

// Decides which children take a fresh page for the part-filled one, takes
// those pages and enters them in the output table; the launch after it does
// the rest by what it finds there.
__global__ void __launch_bounds__(kPlanThreads)
    k_fork_plan(const KvView c, const int32_t *parents, int32_t *table_out, int32_t *status)
{
    extern __shared__ int shared[];
    int *heir = shared;               // [slots]: -1: the slot goes on; else its lowest child
    int *needy = shared + c.slots;    // slots that take a fresh page, in order
    __shared__ int warp_sums[33];
    __shared__ int bad;
    pdl_launch_dependents();
    pdl_wait_prerequisite();
    if (threadIdx.x == 0)
        bad = 0;
    for (int s = threadIdx.x; s < c.slots; s += blockDim.x)
        heir[s] = INT32_MAX;
    __syncthreads();
    for (int s = threadIdx.x; s < c.slots; s += blockDim.x) {
        const int p = parents[s];
        if (p >= c.slots)
            bad = 1;
        else if (p >= 0)
            atomicMin(heir + p, p == s ? -1 : s);
    }
    __syncthreads();
    int wanted = 0;
    for (int base = 0; base < c.slots; base += blockDim.x) {
        const int s = base + (int)threadIdx.x;
        int takes = 0;
        if (s < c.slots) {
            const int p = parents[s];
            takes = p >= 0 && p < c.slots && p != s && heir[p] != s && c.lens[p] > 0 &&
                    c.lens[p] % c.page_tokens != 0 && c.lens[p] / c.page_tokens < c.width;
        }
        int total;
        const int before = scan_before(takes, warp_sums, total);
        if (takes)
            needy[wanted + before] = s;
        wanted += total;
    }
    const int missing = wanted ? max(wanted - count_free(c, warp_sums), 0) : 0;
    __syncthreads();
    const int verdict = bad ? -1 : missing;
    if (threadIdx.x == 0)
        *status = verdict;
    if (verdict)
        return;
    take_free(c, wanted, warp_sums, [&](int rank, int page) {
        const int s = needy[rank], p = parents[s];
        table_out[(int64_t)s * c.width + c.lens[p] / c.page_tokens] = page;
        c.refs[page] = 1;
    });
}

// The rows, counts and lengths after the plan: CTA (x, s) does entries
// x * kPageThreads .. of slot s's old row and of its new one.
__global__ void __launch_bounds__(kPageThreads)
    k_fork_rows(const KvView c, const int32_t *parents, int32_t *table_out, int32_t *held_out,
                int32_t *lens_out, const int32_t *status)
{
    __shared__ int children, others;  // children of slot s; its parent's lowest child, -1: itself
    pdl_launch_dependents();
    pdl_wait_prerequisite();
    const int s = blockIdx.y, j = blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t row = (int64_t)s * c.width;
    const int p = parents[s];
    if (*status) {
        if (j < c.width)
            table_out[row + j] = c.table[row + j];
        if (j == 0) {
            held_out[s] = c.held[s];
            lens_out[s] = c.lens[s];
        }
        return;
    }
    if (threadIdx.x == 0) {
        children = 0;
        others = INT32_MAX;
    }
    __syncthreads();
    for (int k = threadIdx.x; k < c.slots; k += blockDim.x) {
        const int q = parents[k];
        if (q == s)
            atomicAdd(&children, 1);
        if (p >= 0 && q == p)
            atomicMin(&others, q == k ? -1 : k);
    }
    __syncthreads();
    if (j < c.width && j < c.held[s]) {
        const int page = c.table[row + j];
        const int change = j < c.lens[s] / c.page_tokens ? children - 1 : (children ? 0 : -1);
        if (change && is_page(c, page))
            atomicAdd(c.refs + page, change);
    }
    const bool inherits = p >= 0 && (p == s || others == s);
    const int length = p >= 0 ? c.lens[p] : 0, full = length / c.page_tokens;
    const bool tail = length % c.page_tokens != 0;
    const int keeps = p < 0 ? 0 : inherits ? min(c.held[p], c.width) : min(full + tail, c.width);
    if (j < c.width && !(p >= 0 && !inherits && tail && j == full))
        table_out[row + j] = j < keeps ? c.table[(int64_t)p * c.width + j] : -1;
    if (j == 0) {
        held_out[s] = keeps;
        lens_out[s] = length;
    }
}

// The part-filled pages of the children that took a fresh one.
__global__ void __launch_bounds__(kPageThreads)
    k_fork_tails(const KvView c, const int32_t *parents, const int32_t *table_out,
                 const int32_t *status)
{
    pdl_launch_dependents();
    pdl_wait_prerequisite();
    const int s = blockIdx.x / (2 * c.layers), lane = blockIdx.x % (2 * c.layers);
    const int p = parents[s];
    if (*status || p < 0 || p == s)
        return;
    const int length = c.lens[p], full = length / c.page_tokens, tail = length % c.page_tokens;
    if (length <= 0 || tail == 0 || full >= c.width)
        return;
    const int from = c.table[(int64_t)p * c.width + full];
    const int to = table_out[(int64_t)s * c.width + full];
    if (is_page(c, from) && is_page(c, to) && from != to)
        copy_page(c, c.pool[lane & 1] + (lane >> 1) * c.layer_stride, from, to, (uint32_t)tail);
}

// ---------------------------------------------------------------------------
// Compact
// ---------------------------------------------------------------------------
// A token's rows of one layer are split into 16-byte columns; a thread walks
// one column through the slot's list.  It reads kAhead tokens, then writes
// them: every later source lies past every destination written so far (keep
// ascends, so keep[i] >= i), so no column needs another's progress.
constexpr int kAhead = 8;

__global__ void __launch_bounds__(kPageThreads)
    k_kv_compact(const KvView c, const int32_t *start, const int32_t *keep, int32_t keep_stride,
                 const int32_t *count, int32_t *status)
{
    __shared__ int verdict, skip;
    __shared__ int64_t from[kPageThreads], to[kPageThreads];
    pdl_launch_dependents();
    pdl_wait_prerequisite();
    const int s = blockIdx.y, n = count[s], P = c.page_tokens;
    const int64_t first = start[s];
    const int32_t *list = keep + (int64_t)s * keep_stride, *row = c.table + (int64_t)s * c.width;
    if (n < 0) {
        if (blockIdx.x == 0 && threadIdx.x == 0)
            status[s] = 0;
        return;
    }
    if (threadIdx.x == 0) {
        verdict = 0;
        skip = n;
    }
    __syncthreads();
    const int held = min(max(c.held[s], 0), c.width);
    const int64_t room = (int64_t)held * P;
    if (n > keep_stride || first < 0 || first + n > room)
        verdict = 2;
    else
        for (int i = threadIdx.x; i < n; i += blockDim.x) {
            const int k = list[i];
            if (k < 0 || first + k >= room || (i > 0 && list[i - 1] >= k) ||
                !is_page(c, row[(first + k) / P]) || !is_page(c, row[(first + i) / P]))
                verdict = 2;
            if (k != i)
                atomicMin(&skip, i);  // tokens before the first that moves stay where they are
        }
    __syncthreads();
    if (verdict == 0) {
        // From the first page written, or the page of the new end, on: none shared.
        for (int64_t j = (first + skip) / P + threadIdx.x; j < held; j += blockDim.x)
            if (is_page(c, row[j]) && c.refs[row[j]] > 1)
                verdict = 1;
    }
    __syncthreads();
    if (blockIdx.x == 0 && threadIdx.x == 0)
        status[s] = verdict;
    if (verdict)
        return;
    if (blockIdx.x == 0 && threadIdx.x == 0)
        c.lens[s] = (int32_t)(first + n);
    const uint32_t cols = c.row_bytes / 16;
    const int64_t col = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t total = 2ll * c.layers * c.heads * cols;
    char *base = nullptr;
    if (col < total) {
        const int64_t pl = col / ((int64_t)c.heads * cols), in = col % ((int64_t)c.heads * cols);
        base = c.pool[pl & 1] + (pl >> 1) * c.layer_stride + in / cols * c.head_stride +
               in % cols * 16;
    }
    for (int b = skip; b < n; b += kPageThreads) {
        const int here = min(n - b, kPageThreads), i = b + (int)threadIdx.x;
        __syncthreads();
        if ((int)threadIdx.x < here) {
            const int64_t f = first + list[i], t = first + i;
            from[threadIdx.x] = row[f / P] * c.page_stride + f % P * c.token_stride;
            to[threadIdx.x] = row[t / P] * c.page_stride + t % P * c.token_stride;
        }
        __syncthreads();
        if (!base)
            continue;
        for (int k = 0; k < here; k += kAhead) {
            uint4 v[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (k + u < here)
                    v[u] = *reinterpret_cast<const uint4 *>(base + from[k + u]);
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (k + u < here)
                    *reinterpret_cast<uint4 *>(base + to[k + u]) = v[u];
        }
    }
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
template <class... Args>
cudaError_t launch(void (*kernel)(Args...), dim3 grid, int threads, size_t smem, bool pdl,
                   cudaStream_t stream, Args... args)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_copy_pages(const KvView &c, const int32_t *src, const int32_t *dst,
                              const int32_t *tokens, int32_t n, int num_sms, bool pdl,
                              cudaStream_t stream)
{
    (void)num_sms;
    const int64_t jobs = 2ll * c.layers * n;
    const unsigned grid = (unsigned)(jobs < (1 << 30) ? jobs : 1 << 30);
    return launch(k_copy_pages, dim3(grid), kPageThreads, 0, pdl, stream, c, src, dst, tokens, jobs);
}

cudaError_t launch_kv_resize(const KvView &c, const int32_t *capacity, int32_t *status, bool pdl,
                             cudaStream_t stream)
{
    return launch(k_kv_resize, dim3(1), kPlanThreads, c.slots * sizeof(int), pdl, stream, c,
                  capacity, status);
}

cudaError_t launch_kv_fork(const KvView &c, const int32_t *parents, int32_t *table_out,
                           int32_t *held_out, int32_t *lens_out, int32_t *status, int num_sms,
                           bool pdl, cudaStream_t stream)
{
    (void)num_sms;
    const size_t smem = 2 * c.slots * sizeof(int);
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(
            (const void *)k_fork_plan, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess)
            return e;
    }
    cudaError_t e = launch(k_fork_plan, dim3(1), kPlanThreads, smem, pdl, stream, c, parents,
                           table_out, status);
    if (e != cudaSuccess)
        return e;
    e = launch(k_fork_rows, dim3((c.width + kPageThreads - 1) / kPageThreads, c.slots),
               kPageThreads, 0, pdl, stream, c, parents, table_out, held_out, lens_out,
               (const int32_t *)status);
    if (e != cudaSuccess)
        return e;
    return launch(k_fork_tails, dim3((unsigned)(2ll * c.layers * c.slots)), kPageThreads, 0, pdl,
                  stream, c, parents, (const int32_t *)table_out, (const int32_t *)status);
}

cudaError_t launch_kv_compact(const KvView &c, const int32_t *start, const int32_t *keep,
                              int32_t keep_stride, const int32_t *count, int32_t *status,
                              bool pdl, cudaStream_t stream)
{
    const int64_t cols = 2ll * c.layers * c.heads * (c.row_bytes / 16);
    return launch(k_kv_compact, dim3((unsigned)((cols + kPageThreads - 1) / kPageThreads), c.slots),
                  kPageThreads, 0, pdl, stream, c, start, keep, keep_stride, count, status);
}

}  // namespace tb
