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

// One page of one layer by a whole CTA, four 16-byte loads a thread in flight.
__device__ __forceinline__ void copy_page(const KvView &c, char *pool, int32_t src, int32_t dst,
                                          uint32_t tokens)
{
    const Runs r = page_runs(c, tokens);
    const uint32_t per_run = r.bytes / 16, total = r.n1 * r.n2 * per_run;
    const char *from = pool + src * c.page_stride;
    char *to = pool + dst * c.page_stride;
    auto place = [&](uint32_t i) {
        if (r.n1 * r.n2 == 1)
            return (int64_t)i * 16;
        const uint32_t run = i / per_run;
        return (run / r.n2) * r.s1 + (run % r.n2) * r.s2 + (int64_t)(i - run * per_run) * 16;
    };
    for (uint32_t i = threadIdx.x; i < total; i += 4 * blockDim.x) {
        uint4 v[4];
        int64_t at[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (i + u * blockDim.x < total) {
                at[u] = place(i + u * blockDim.x);
                v[u] = *reinterpret_cast<const uint4 *>(from + at[u]);
            }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (i + u * blockDim.x < total)
                *reinterpret_cast<uint4 *>(to + at[u]) = v[u];
    }
}

__device__ __forceinline__ bool is_page(const KvView &c, int32_t p)
{
    return p >= 0 && p < c.pages;
}

// Pool of a layer's keys (even lanes) or values (odd).
__device__ __forceinline__ char *pool_of(const KvView &c, int32_t lane)
{
    return (lane & 1 ? c.pool[1] : c.pool[0]) + (lane >> 1) * c.layer_stride;
}

// A CTA per page, layer and pool.  Bound by HBM: 1000 pages of 32 KB in 16 layers
// 302 us (6.9 TB/s read and written; one load a thread in flight 319 us), 8
// pages in 2 layers 2.8 us, a launch's latency.
__global__ void __launch_bounds__(kPageThreads)
    k_copy_pages(const KvView c, const int32_t *src, const int32_t *dst, const int32_t *tokens,
                 int64_t jobs)
{
    pdl_launch_dependents();
    pdl_wait_prerequisite();
    for (int64_t j = blockIdx.x; j < jobs; j += gridDim.x) {
        const int64_t i = j >> 32 ? j / (2 * c.layers) : (uint32_t)j / (uint32_t)(2 * c.layers);
        const int32_t lane = (int32_t)(j - i * (2 * c.layers));
        const int32_t s = src[i], d = dst[i];
        const int32_t t = tokens ? min(max(tokens[i], 0), c.page_tokens) : c.page_tokens;
        if (is_page(c, s) && is_page(c, d) && s != d && t > 0)
            copy_page(c, pool_of(c, lane), s, d, (uint32_t)t);
    }
}

// Sums over the CTA before this thread, and the CTA's totals, of two counts at
// a time; sums: 32 words.
__device__ int2 scan_before(int2 v, int2 *sums, int2 &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int2 x = v;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int a = __shfl_up_sync(0xffffffffu, x.x, d), b = __shfl_up_sync(0xffffffffu, x.y, d);
        if (lane >= d) {
            x.x += a;
            x.y += b;
        }
    }
    __syncthreads();
    if (lane == 31)
        sums[warp] = x;
    __syncthreads();
    const int2 w = lane < (int)(blockDim.x >> 5) ? sums[lane] : int2{0, 0};
    total = int2{__reduce_add_sync(0xffffffffu, w.x), __reduce_add_sync(0xffffffffu, w.y)};
    const int2 before{__reduce_add_sync(0xffffffffu, lane < warp ? w.x : 0),
                      __reduce_add_sync(0xffffffffu, lane < warp ? w.y : 0)};
    return int2{x.x - v.x + before.x, x.y - v.y + before.y};
}

__device__ __forceinline__ int pages_for(int tokens, int page_tokens)
{
    return tokens / page_tokens + (tokens % page_tokens != 0);
}

// ---------------------------------------------------------------------------
// Handing out pages.  "The lowest free pages" needs a count of the free pages
// before each one: the pool's counts are split over the CTAs of one cluster
// (their SMs read together; totals meet in distributed shared memory, so no
// scratch memory is needed), and each warp counts, then hands out, a run of
// them: 32 neighbouring pages a lane, as bits of a word kept in a register from
// the first pass to the second.  A small call is bound by the chain of its steps (6
// us); a large one by the work of 16 SMs on the counts, entries and pages given
// back (512 slots, 1.17 million pages, 4.7 MB of counts, 109,000 entries: 24
// us a call; with one CTA 1670, a page a lane and every count read twice 65).
// ---------------------------------------------------------------------------
constexpr int kCluster = 16;
// Pools of more pages than this are looked through by the cluster, others by one
// CTA, which spares the cluster's start and barriers.  A call for 64 slots, one
// CTA and 16: 1024 pages 5.2 and 6.4 us, 8192 6.6 and 8.4, 16384 8.6 and 8.4,
// 65536 12.2 and 8.4, 1048576 51.2 and 12.2.
constexpr int kClusterPages = 12288;
constexpr int kPlanWarps = kPlanThreads / 32;

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

// All threads of the cluster; orders their memory accesses before and after.
__device__ __forceinline__ void cluster_sync()
{
    __syncwarp();  // the barrier is one for whole warps
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Writes a word of the same shared variable in CTA `rank`.
__device__ __forceinline__ void store_remote(int *local, uint32_t rank, int value)
{
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(remote)
                 : "r"(smem_u32(local)), "r"(rank));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote), "r"(value) : "memory");
}

// 1024 pages of a warp's share: a lane's word has the bits of 32 neighbouring
// ones, a set bit is a free page.
constexpr int kGroupPages = 1024;
constexpr int kHeldGroups = 4;  // groups kept in registers between the passes

struct FreePages {
    int from, to;                  // this warp's share
    uint32_t group[kHeldGroups];   // its first groups
};

struct FreeCount {
    int cta[kCluster];      // free pages in each CTA's share
    int warp[kPlanWarps];   // ... in each warp's, this CTA
};

__device__ __forceinline__ uint32_t free_group(const KvView &c, int from, int to)
{
    const int lane = threadIdx.x & 31;
    const bool wide = (reinterpret_cast<uintptr_t>(c.refs) & 15) == 0;
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < kGroupPages / 128; ++i) {
        const int p = from + 128 * i + 4 * lane;
        if (wide && p + 4 <= to) {
            const int4 r = *reinterpret_cast<const int4 *>(c.refs + p);
            bits |= (uint32_t)((r.x == 0) | (r.y == 0) << 1 | (r.z == 0) << 2 | (r.w == 0) << 3) << 4 * i;
        } else {
            for (int k = 0; k < 4; ++k)
                if (p + k < to && c.refs[p + k] == 0)
                    bits |= 1u << (4 * i + k);
        }
    }
    // Read four pages a lane, 128 a step; wanted 32 a lane: step lane / 4, and
    // eight lanes' four bits of it.
    uint32_t word = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t other = __shfl_sync(0xffffffffu, bits, 8 * (lane & 3) + k);
        word |= (other >> 4 * (lane >> 2) & 15u) << 4 * k;
    }
    return word;
}

// The first look at this warp's share: its loads depend on nothing else.
__device__ __forceinline__ void find_free(const KvView &c, FreePages &f)
{
    const int shares = (int)cluster_size() * kPlanWarps;
    const int mine = (int)cluster_rank() * kPlanWarps + (int)(threadIdx.x >> 5);
    const int blocks = c.pages / 128 + (c.pages % 128 != 0);
    const int each = blocks / shares, more = blocks % shares;
    const int first = each * mine + min(mine, more), count = each + (mine < more);
    f.from = min(first * 128, c.pages);  // pages <= 2^30
    f.to = min(f.from + count * 128, c.pages);
#pragma unroll
    for (int g = 0; g < kHeldGroups; ++g)
        f.group[g] = f.from + g * kGroupPages < f.to ? free_group(c, f.from + g * kGroupPages, f.to) : 0;
}

// All threads of the cluster; orders their memory accesses before and after.
template <bool CLUSTER>
__device__ __forceinline__ void plan_sync()
{
    if (CLUSTER)
        cluster_sync();
    else
        __syncthreads();
}

// Free pages of the pool; all threads of the cluster call it, after a
// plan_sync that says that every CTA runs.
template <bool CLUSTER>
__device__ int count_free(const KvView &c, const FreePages &pages, FreeCount &f)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int mine = 0;
#pragma unroll
    for (int g = 0; g < kHeldGroups; ++g)
        mine += __popc(pages.group[g]);
    for (int p = pages.from + kHeldGroups * kGroupPages; p < pages.to; p += kGroupPages)
        mine += __popc(free_group(c, p, pages.to));
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0)
        f.warp[warp] = mine;
    __syncthreads();
    const int sum = __reduce_add_sync(0xffffffffu, f.warp[lane]);
    if (!CLUSTER)
        return sum;
    if (warp == 0 && lane < (int)cluster_size())
        store_remote(&f.cta[cluster_rank()], lane, sum);
    cluster_sync();
    return __reduce_add_sync(0xffffffffu, lane < (int)cluster_size() ? f.cta[lane] : 0);
}

// Hands out the `wanted` lowest free pages, after count_free: take(rank, n, bits,
// page) gets the first n of the set bits of `bits`, pages page .. page + 31.
template <bool CLUSTER, class Take>
__device__ void take_free(const KvView &c, const FreePages &pages, const FreeCount &f, int wanted,
                          Take take)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int rank = __reduce_add_sync(0xffffffffu, lane < warp ? f.warp[lane] : 0);
    if (CLUSTER)
        rank += __reduce_add_sync(0xffffffffu, lane < (int)cluster_rank() ? f.cta[lane] : 0);
    const int end = min(rank + f.warp[warp], wanted);
    for (int g = 0; rank < end; ++g) {
        const int first = pages.from + g * kGroupPages;
        uint32_t bits = 0;
        if (g >= kHeldGroups)
            bits = free_group(c, first, pages.to);
#pragma unroll
        for (int k = 0; k < kHeldGroups; ++k)
            if (g == k)
                bits = pages.group[k];
        const int n = __popc(bits);
        int before = n;
        for (int d = 1; d < 32; d *= 2) {
            const int y = __shfl_up_sync(0xffffffffu, before, d);
            if (lane >= d)
                before += y;
        }
        const int total = __shfl_sync(0xffffffffu, before, 31), mine = rank + before - n;
        if (n && mine < end)
            take(mine, min(n, end - mine), bits, first + 32 * lane);
        rank += total;
    }
}

// The last of n ascending entries (the first is 0) that is <= x.
__device__ __forceinline__ int last_at_most(const int *v, int n, int x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (v[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// New pages for slot s: need - held where that is positive; a prefix sum over the
// slots turns a free page's rank into its slot and entry.  16 slots 6.3 us: two
// dependent reads, three scans of the block and the writes.
template <bool CLUSTER>
__global__ void __launch_bounds__(kPlanThreads, 1)
    k_kv_resize(const KvView c, const int32_t *capacity, int32_t *status)
{
    extern __shared__ int shared[];
    int *first_new = shared;              // [slots] pages that the slots before it take
    int *first_gone = shared + c.slots;   // [slots] ... give back
    int *held = shared + 2 * c.slots;     // [slots]
    __shared__ int2 warp_sums[32];
    __shared__ FreeCount found;
    __shared__ int bad;
    pdl_launch_dependents();
    pdl_wait_prerequisite();
    if (threadIdx.x == 0)
        bad = 0;
    FreePages pages;
    find_free(c, pages);
    plan_sync<CLUSTER>();
    int wanted = 0, gone = 0;
    for (int base = 0; base < c.slots; base += blockDim.x) {
        const int s = base + (int)threadIdx.x;
        int grow = 0, shrink = 0;
        if (s < c.slots) {
            const int cap = capacity[s], has = min(max(c.held[s], 0), c.width), length = c.lens[s];
            held[s] = has;
            if (cap >= 0) {
                const int need = pages_for(cap, c.page_tokens);
                if (need > c.width)
                    bad = 1;
                // The last page kept is written again past the cut: not if it is shared.
                if (cap < length && cap % c.page_tokens && need <= has) {
                    const int p = c.table[(int64_t)s * c.width + need - 1];
                    if (is_page(c, p) && c.refs[p] > 1)
                        bad = 1;
                }
                grow = min(max(need - has, 0), c.width);
                shrink = max(has - need, 0);
            }
        }
        int2 total;
        const int2 before = scan_before(int2{grow, shrink}, warp_sums, total);
        if (s < c.slots) {
            first_new[s] = wanted + before.x;
            first_gone[s] = gone + before.y;
        }
        wanted += total.x;
        gone += total.y;
    }
    __syncthreads();
    int missing = 0;
    if (wanted)
        missing = max(wanted - count_free<CLUSTER>(c, pages, found), 0);
    const int verdict = bad ? -1 : missing;
    if (cluster_rank() == 0 && threadIdx.x == 0)
        *status = verdict;
    if (!verdict && wanted)
        take_free<CLUSTER>(c, pages, found, wanted, [&](int rank, int n, uint32_t bits, int page) {
            int s = last_at_most(first_new, c.slots, rank);
            for (; n; --n, ++rank, bits &= bits - 1) {
                while (s + 1 < c.slots && first_new[s + 1] <= rank)
                    ++s;
                const int p = page + __ffs(bits) - 1;
                c.table[(int64_t)s * c.width + held[s] + rank - first_new[s]] = p;
                c.refs[p] = 1;
            }
        });
    // Pages are given back after every CTA has looked for free ones, and
    // nothing is written before all have read held and lens.
    plan_sync<CLUSTER>();
    if (verdict)
        return;
    const int threads = (int)cluster_size() * kPlanThreads;
    const int mine = (int)cluster_rank() * kPlanThreads + (int)threadIdx.x;
#pragma unroll 4
    for (int i = mine; i < gone; i += threads) {
        const int s = last_at_most(first_gone, c.slots, i);
        const int kept = pages_for(capacity[s], c.page_tokens);
        int32_t *entry = c.table + (int64_t)s * c.width + kept + i - first_gone[s];
        const int p = *entry;
        if (is_page(c, p))
            atomicSub(c.refs + p, 1);
        *entry = -1;
    }
    for (int s = mine; s < c.slots; s += threads) {
        const int cap = capacity[s];
        if (cap >= 0) {
            c.held[s] = pages_for(cap, c.page_tokens);
            c.lens[s] = min(c.lens[s], cap);
        }
    }
}

// ---------------------------------------------------------------------------
// Fork, in two launches: which slots take a fresh page has to be known for all
// before pages are handed out; the counts, rows and page tails then go to as many
// CTAs as there are.  Bound by the two launches' latency: 4 beams 6.6 us, 32 x 8
// beams of 4007 tokens 14.9 (20 MB of tails and rows, 6.1 us of HBM).
// ---------------------------------------------------------------------------

// Decides which children take a fresh page for the part-filled one and takes
// those pages.  It enters the page that holds the part-filled one's tokens in
// the output row of every slot that does not simply go on: the launch after it
// copies where that is another page, and leaves the entry alone.
template <bool CLUSTER>
__global__ void __launch_bounds__(kPlanThreads, 1)
    k_fork_plan(const KvView c, const int32_t *parents, int32_t *table_out, int32_t *status)
{
    extern __shared__ int shared[];
    int *heir = shared;               // [slots]: -1: the slot goes on; else its lowest child
    int *needy = shared + c.slots;    // slots that take a fresh page, in order
    __shared__ int2 warp_sums[32];
    __shared__ FreeCount found;
    __shared__ int bad;
    pdl_launch_dependents();
    pdl_wait_prerequisite();
    if (threadIdx.x == 0)
        bad = 0;
    for (int s = threadIdx.x; s < c.slots; s += blockDim.x)
        heir[s] = INT32_MAX;
    FreePages pages;
    find_free(c, pages);
    plan_sync<CLUSTER>();
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
            if (p >= 0 && p < c.slots && p != s) {
                const int length = c.lens[p], full = length / c.page_tokens;
                takes = length > 0 && length % c.page_tokens != 0 && full < c.width;
                if (takes && heir[p] == s) {
                    takes = 0;
                    if (cluster_rank() == 0)
                        table_out[(int64_t)s * c.width + full] = c.table[(int64_t)p * c.width + full];
                }
            }
        }
        int2 total;
        const int2 before = scan_before(int2{takes, 0}, warp_sums, total);
        if (takes)
            needy[wanted + before.x] = s;
        wanted += total.x;
    }
    __syncthreads();
    int missing = 0;
    if (wanted)
        missing = max(wanted - count_free<CLUSTER>(c, pages, found), 0);
    const int verdict = bad ? -1 : missing;
    if (cluster_rank() == 0 && threadIdx.x == 0)
        *status = verdict;
    if (!verdict && wanted)
        take_free<CLUSTER>(c, pages, found, wanted, [&](int rank, int n, uint32_t bits, int page) {
            for (; n; --n, ++rank, bits &= bits - 1) {
                const int s = needy[rank], p = page + __ffs(bits) - 1;
                table_out[(int64_t)s * c.width + c.lens[parents[s]] / c.page_tokens] = p;
                c.refs[p] = 1;
            }
        });
}

// The rest of the fork.  Blocks below row_blocks: entries of slot s's old row
// (counts) and of its new one; the others: the part-filled page of a child that
// took a fresh one, `each` of the layers' keys and values a CTA: one, for
// latency's sake, while all are on the SMs at once, else four, whose checks are
// then done once.  With 1 and 4 (half the slots copy): 4 slots of 2 layers 6.5
// and 8.7 us, 64 of 4 10.0 and 11.5, 256 of 4 14.5 and 15.9, 256 of 16 25.6 and
// 21.4.
__host__ __device__ constexpr int tail_lanes(int slots, int lanes)
{
    return (int64_t)slots * lanes > 2048 ? 4 : 1;
}

__global__ void __launch_bounds__(kPageThreads)
    k_fork_rest(const KvView c, const int32_t *parents, int32_t *table_out, int32_t *held_out,
                int32_t *lens_out, const int32_t *status, int row_blocks, int blocks_per_row)
{
    __shared__ int children, others;  // children of slot s; its parent's lowest child, -1: itself
    pdl_launch_dependents();
    pdl_wait_prerequisite();
    const bool refused = *status != 0;
    if ((int)blockIdx.x >= row_blocks) {
        const int lanes = 2 * c.layers, each = tail_lanes(c.slots, lanes);
        const int groups = (lanes + each - 1) / each;
        const int s = (blockIdx.x - row_blocks) / groups;
        const int first = (blockIdx.x - row_blocks) % groups * each;
        const int p = parents[s];
        if (refused || p < 0 || p == s)
            return;
        const int length = c.lens[p], full = length / c.page_tokens, tail = length % c.page_tokens;
        if (length <= 0 || tail == 0 || full >= c.width)
            return;
        const int from = c.table[(int64_t)p * c.width + full];
        const int to = table_out[(int64_t)s * c.width + full];
        if (is_page(c, from) && is_page(c, to) && from != to)
            for (int lane = first; lane < min(first + each, lanes); ++lane)
                copy_page(c, pool_of(c, lane), from, to, (uint32_t)tail);
        return;
    }
    const int s = blockIdx.x / blocks_per_row;
    const int j = blockIdx.x % blocks_per_row * blockDim.x + threadIdx.x;
    const int64_t row = (int64_t)s * c.width;
    const int p = parents[s];
    if (refused) {
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
    if (j < c.width && !(p >= 0 && p != s && tail && j == full))  // the plan's entry
        table_out[row + j] = j < keeps ? c.table[(int64_t)p * c.width + j] : -1;
    if (j == 0) {
        held_out[s] = keeps;
        lens_out[s] = length;
    }
}

// ---------------------------------------------------------------------------
// Compact.  A token's rows of one layer are split into 16-byte columns; a
// thread walks one column through the slot's list, reading ahead of what it
// writes: every later source lies past every destination written so far (keep
// ascends, so keep[i] >= i), so no column needs another's progress.  The warps
// of a CTA share 32 columns, and take eight tokens of the list each in turn, all
// of which are read before any is written.
//
// Bound by HBM where there are many columns: 8 slots x 8 layers, heads of 256
// bytes first, some 3400 of 8192 tokens kept, 282 us (1.78 GB, 6.3 TB/s); 32
// slots x 32 layers, every other of 8192 tokens, 4.94 ms (34 GB, 7.0 TB/s).  By
// each turn's chain of instructions where there are few: a slot of 4 layers of
// 8 heads, 4096 tokens, 67 us, with one warp a CTA 195.
// ---------------------------------------------------------------------------

// Whether slot s's list may be carried out, as tb_kv_compact's status; the
// whole CTA calls it.
__device__ int compact_verdict(const KvView &c, int s, int64_t first, const int32_t *list, int n, int most)
{
    __shared__ int verdict, skip;
    const int P = c.page_tokens;
    const int32_t *row = c.table + (int64_t)s * c.width;
    if (threadIdx.x == 0) {
        verdict = 0;
        skip = n;
    }
    __syncthreads();
    const int held = min(max(c.held[s], 0), c.width);
    const int64_t room = (int64_t)held * P;
    if (n > most || first < 0 || first + n > room)
        verdict = 2;
    else
#pragma unroll 4
        for (int i = threadIdx.x; i < n; i += blockDim.x) {
            const int k = list[i];
            if (k < 0 || first + k >= room || (i > 0 && list[i - 1] >= k) ||
                !is_page(c, row[(first + k) / P]) || !is_page(c, row[(first + i) / P]))
                verdict = 2;
            if (k != i)
                atomicMin(&skip, i);  // tokens before the first that moves stay where they are
        }
    __syncthreads();
    const bool bad = verdict != 0;
    __syncthreads();
    if (!bad) {
        // From the first page written, or the page of the new end, on: none shared.
        for (int64_t j = (first + skip) / P + threadIdx.x; j < held; j += blockDim.x)
            if (is_page(c, row[j]) && c.refs[row[j]] > 1)
                verdict = 1;
    }
    __syncthreads();
    return verdict;
}

__global__ void __launch_bounds__(kPlanThreads, 1)
    k_compact_check(const KvView c, const int32_t *start, const int32_t *keep, int32_t keep_stride,
                    const int32_t *count, int32_t *status)
{
    pdl_launch_dependents();
    pdl_wait_prerequisite();
    const int s = blockIdx.x, n = count[s];
    const int verdict =
        n < 0 ? 0 : compact_verdict(c, s, start[s], keep + (int64_t)s * keep_stride, n, keep_stride);
    if (threadIdx.x == 0) {
        status[s] = verdict;
        if (n >= 0 && !verdict)
            c.lens[s] = start[s] + n;
    }
}

constexpr int kSet = 8;         // tokens requested at a time
constexpr int kLookAhead = 4;   // blocks of 32 list entries looked up, or in use

// A warp's sets on their way to shared memory, where only their thread reads
// them, and its list entries.
template <int RING>
struct Moving {
    uint4 ring[RING][kSet][32];
    int64_t from[kLookAhead][32], to[kLookAhead][32];
};

// CHECK: no k_compact_check has run.
template <bool CHECK, int WARPS, int RING>
__global__ void __launch_bounds__(32 * WARPS)
    k_kv_compact(const KvView c, const int32_t *start, const int32_t *keep, int32_t keep_stride,
                 const int32_t *count, int32_t *status)
{
    extern __shared__ __align__(16) unsigned char raw[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto &[ring, from, to] = reinterpret_cast<Moving<RING> *>(raw)[warp];
    pdl_launch_dependents();
    pdl_wait_prerequisite();
    const int s = blockIdx.y, n = count[s], P = c.page_tokens;
    const int64_t first = start[s];
    const int32_t *list = keep + (int64_t)s * keep_stride, *row = c.table + (int64_t)s * c.width;
    if (CHECK) {
        const int verdict = n < 0 ? 0 : compact_verdict(c, s, first, list, n, keep_stride);
        if (blockIdx.x == 0 && threadIdx.x == 0) {
            status[s] = verdict;
            if (n >= 0 && !verdict)
                c.lens[s] = (int32_t)(first + n);
        }
        if (verdict)
            return;
    } else if (status[s]) {
        return;
    }
    if (n <= 0)
        return;
    const uint32_t cols = c.row_bytes / 16;
    const int64_t col = (int64_t)blockIdx.x * 32 + lane;
    const bool real = col < 2ll * c.layers * c.heads * cols;
    char *base = nullptr;
    if (real) {
        const int64_t half = col / ((int64_t)c.heads * cols), in = col % ((int64_t)c.heads * cols);
        base = pool_of(c, (int32_t)half) + in / cols * c.head_stride + in % cols * 16;
    }
    // A warp's block: its sets of four turns.
    auto index = [&](int block) { return kSet * (WARPS * (4 * block + lane / kSet) + warp) + lane % kSet; };
    // Looking up a block of 32 entries takes two dependent loads; both are
    // under way long before the block's tokens are requested.
    auto entry = [&](int block) {
        const int i = index(block);
        return i < n ? list[i] : 0;
    };
    auto pages = [&](int block, int k) {
        const int i = index(block);
        return i < n ? int2{row[(first + k) / P], row[(first + i) / P]} : int2{0, 0};
    };
    auto keep_block = [&](int block, int k, int2 page) {
        const int64_t f = first + k, t = first + index(block);
        const bool moves = index(block) < n && f != t;
        from[block % kLookAhead][lane] = moves ? page.x * c.page_stride + f % P * c.token_stride : -1;
        to[block % kLookAhead][lane] = moves ? page.y * c.page_stride + t % P * c.token_stride : -1;
    };
    auto places = [&](int64_t(&of)[kLookAhead][32], int set, int64_t(&x)[kSet]) {
        const int4 *p = reinterpret_cast<const int4 *>(&of[set / 4 % kLookAhead][set % 4 * kSet]);
#pragma unroll
        for (int u = 0; u < kSet / 2; ++u)
            reinterpret_cast<int4 *>(x)[u] = p[u];
    };
    auto request = [&](int set) {
        int64_t f[kSet];
        places(from, set, f);
#pragma unroll
        for (int u = 0; u < kSet; ++u)
            if (f[u] >= 0 && real)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                 smem_u32(&ring[set % RING][u][lane])),
                             "l"(base + f[u])
                             : "memory");
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int b = 0; b < 2; ++b) {
        const int k = entry(b);
        keep_block(b, k, pages(b, k));
    }
    int k2 = entry(2), k3 = entry(3);
    int2 p2 = pages(2, k2);
    __syncwarp();
    for (int k = 0; k < RING - 1; ++k)
        request(k);
    const int sets = (n + kSet * WARPS - 1) / (kSet * WARPS);
    for (int k = 0; k < sets; ++k) {
        if (k % 4 == 0) {  // a block of four sets begins; requests reach into the second after it
            const int block = k / 4;
            keep_block(block + 2, k2, p2);
            k2 = k3;
            p2 = pages(block + 3, k2);
            k3 = entry(block + 4);
            __syncwarp();
        }
        request(k + RING - 1);
        int64_t d[kSet];
        uint4 v[kSet];
        places(to, k, d);
        asm volatile("cp.async.wait_group %0;" ::"n"(RING - 1) : "memory");
#pragma unroll
        for (int u = 0; u < kSet; ++u)
            v[u] = ring[k % RING][u][lane];
        if (WARPS > 1)  // what the sets of this turn write has been read
            __syncthreads();
#pragma unroll
        for (int u = 0; u < kSet; ++u)
            if (d[u] >= 0 && real)
                *reinterpret_cast<uint4 *>(base + d[u]) = v[u];
        __syncwarp();
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
template <class... Args>
cudaError_t launch(void (*kernel)(Args...), dim3 grid, int threads, size_t smem, int cluster, bool pdl,
                   cudaStream_t stream, Args... args)
{
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_copy_pages(const KvView &c, const int32_t *src, const int32_t *dst,
                              const int32_t *tokens, int32_t n, bool pdl,
                              cudaStream_t stream)
{
    const int64_t jobs = 2ll * c.layers * n;
    const unsigned grid = (unsigned)(jobs < (1 << 30) ? jobs : 1 << 30);
    return launch(k_copy_pages, dim3(grid), kPageThreads, 0, 1, pdl, stream, c, src, dst, tokens, jobs);
}

namespace {

// Launches a kernel that hands out pages, with `words` words of shared memory a
// slot: its CTAs are one cluster, or one CTA.
template <class... Args>
cudaError_t launch_plan(void (*many)(Args...), void (*one)(Args...), const KvView &c, size_t words, bool pdl,
                        cudaStream_t stream, Args... args)
{
    const bool cluster = c.pages > kClusterPages;
    void (*kernel)(Args...) = cluster ? many : one;
    cudaError_t e = cudaSuccess;
    if (cluster)
        e = cudaFuncSetAttribute((const void *)kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess)
        return e;
    // Once a kernel and device, for the most slots there may be: a limit set to
    // each call's own size could fall between another thread's check and launch.
    if (resident_ctas((const void *)kernel, kPlanThreads, TB_KV_MAX_SLOTS * words * sizeof(int)) < 1)
        return cudaErrorInvalidConfiguration;
    const size_t smem = c.slots * words * sizeof(int);
    const int ctas = cluster ? kCluster : 1;
    return launch(kernel, dim3(ctas), kPlanThreads, smem, ctas, pdl, stream, args...);
}

}  // namespace

cudaError_t launch_kv_resize(const KvView &c, const int32_t *capacity, int32_t *status, bool pdl,
                             cudaStream_t stream)
{
    return launch_plan(k_kv_resize<true>, k_kv_resize<false>, c, 3, pdl, stream, c, capacity, status);
}

cudaError_t launch_kv_fork(const KvView &c, const int32_t *parents, int32_t *table_out,
                           int32_t *held_out, int32_t *lens_out, int32_t *status, bool pdl,
                           cudaStream_t stream)
{
    const cudaError_t e = launch_plan(k_fork_plan<true>, k_fork_plan<false>, c, 2, pdl, stream, c, parents,
                                      table_out, status);
    if (e != cudaSuccess)
        return e;
    const int per_row = (c.width + kPageThreads - 1) / kPageThreads, rows = c.slots * per_row;
    const int each = tail_lanes(c.slots, 2 * c.layers), groups = (2 * c.layers + each - 1) / each;
    return launch(k_fork_rest, dim3((unsigned)rows + (unsigned)(c.slots * groups)), kPageThreads, 0, 1, pdl,
                  stream, c, parents, table_out, held_out, lens_out, (const int32_t *)status, rows, per_row);
}

namespace {

template <int WARPS, int RING>
cudaError_t launch_compact(const KvView &c, const int32_t *start, const int32_t *keep, int32_t keep_stride,
                           const int32_t *count, int32_t *status, dim3 grid, bool pdl, cudaStream_t stream)
{
    // Every moving CTA checks its slot's list, or one a slot does in a launch
    // before, which costs 1.5 us but is done once.  All, and one: 128 CTAs and
    // lists of 8 tokens 5.3 and 6.8 us, of 64 6.7 and 7.8, of 256 11.0 and 11.9;
    // 256 CTAs, of 128 10.4 and 10.6, of 256 16.6 and 15.1; 512, of 64 10.9 and
    // 10.7, of 128 15.5 and 13.8; 1024, of 8 9.8 and 9.8, of 64 17.1 and 15.0.
    // (Eight warps take lists of 512 entries and more only.)
    const bool check = WARPS < 8 && keep_stride <= 256 && (int64_t)grid.x * grid.y * keep_stride <= 32768;
    void (*kernel)(KvView, const int32_t *, const int32_t *, int32_t, const int32_t *, int32_t *) =
        k_kv_compact<false, WARPS, RING>;
    if constexpr (WARPS < 8)
        if (check)
            kernel = k_kv_compact<true, WARPS, RING>;
    constexpr int bytes = WARPS * sizeof(Moving<RING>);
    if (resident_ctas((const void *)kernel, 32 * WARPS, bytes) < 1)  // once a kernel and device; allows the memory
        return cudaErrorInvalidConfiguration;
    if (!check) {
        const cudaError_t e = launch(k_compact_check, dim3(c.slots), kPlanThreads, 0, 1, pdl, stream, c, start,
                                     keep, keep_stride, count, status);
        if (e != cudaSuccess)
            return e;
    }
    return launch(kernel, grid, 32 * WARPS, bytes, 1, pdl, stream, c, start, keep, keep_stride, count,
                  status);
}

}  // namespace

cudaError_t launch_kv_compact(const KvView &c, const int32_t *start, const int32_t *keep,
                              int32_t keep_stride, const int32_t *count, int32_t *status,
                              bool pdl, cudaStream_t stream)
{
    const int64_t cols = 2ll * c.layers * c.heads * (c.row_bytes / 16);
    const dim3 grid((unsigned)((cols + 31) / 32), c.slots);
    const int64_t ctas = (int64_t)grid.x * grid.y;
    // More warps a CTA shorten a list's walk; fewer let more CTAs share an SM and
    // get to work sooner.  With 1, 4 and 8 warps: 128 CTAs, lists of 8 tokens 6.0,
    // 5.5 and 5.2 us, of 1024 55.9, 30.6 and 24.1; 256 CTAs, of 8 5.9, 5.7 and
    // 8.9, of 1024 66.9, 53.4 and 51.9; 1024, of 8 9.7, 11.0 and 18.3, of 128
    // 25.4, 23.2 and 33.1, of 512 101, 91 and 91, of 4096 707, 665 and 646; 8192,
    // of 8 28.4, 44.0 and 106, of 4096 5005, 4969 and 4946.
    if (keep_stride >= 512)
        return launch_compact<8, 4>(c, start, keep, keep_stride, count, status, grid, pdl, stream);
    if (keep_stride >= 128 || ctas <= 304)
        return launch_compact<4, 4>(c, start, keep, keep_stride, count, status, grid, pdl, stream);
    return launch_compact<1, 8>(c, start, keep, keep_stride, count, status, grid, pdl, stream);
}

}  // namespace tb
