// Attention for a tree of drafted tokens over the paged cache (sm_103a):
// softmax(scale q K^T + mask) V in one pass over the positions, matrix products
// on tcgen05 with scores, weights and output sums in tensor memory.

#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "tb_device.cuh"
#include "tb_kv.h"
#include "tb_umma.cuh"

namespace tb {
namespace {

using namespace dev;

// ---------------------------------------------------------------------------
// Work.  The query rows of a sequence that share a cache head are its (draft,
// head of the group) pairs: T * group rows that read the same keys and values.
// A unit is up to 256 of them; its work is the sequence's tiles of 128
// positions.  The tiles of all units, one after another, are dealt to the CTAs
// in equal runs, so a long sequence is split over many CTAs and short ones
// share one, whatever their lengths; a unit cut by a run's end leaves partial
// sums that k_tree_join puts together.
// ---------------------------------------------------------------------------
constexpr int kTile = 128;       // positions of a tile
constexpr int kRowTile = 128;    // rows of one matrix instruction
constexpr int kUnitRows = 256;   // rows of a unit: two row tiles
constexpr int kThreads = 384;    // warps 0-7: softmax; 8-10: loads; 11: matrix products
constexpr int kLoadWarps = 3;    // ... all of them where threads load
constexpr int kFixWarps = 2;     // ... else one asks for tiles, two look drafts over
constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 32;    // rows of a unit one CTA of k_tree_join takes

struct Seq {
    int slot, row0, T, n, end, tiles, units;  // units per cache head
};

__device__ __forceinline__ Seq seq_of(const TreePlan &p, int b)
{
    Seq s;
    s.row0 = min(max(p.q_start[b], 0), p.rows);
    s.T = max(min(p.q_start[b + 1], p.rows) - s.row0, 0);
    s.slot = p.seq_slots ? p.seq_slots[b] : b;
    const bool known = s.slot >= 0 && s.slot < p.c.slots;
    s.n = known ? min(max(p.c.lens[s.slot], 0), p.c.width * p.c.page_tokens) : 0;
    s.end = known ? s.n + s.T : 0;
    s.tiles = max((s.end + kTile - 1) / kTile, 1);
    s.units = (int)(((int64_t)s.T * p.group + kUnitRows - 1) / kUnitRows);
    return s;
}

__device__ __forceinline__ int64_t seq_work(const TreePlan &p, int b)
{
    const Seq s = seq_of(p, b);
    return (int64_t)s.units * s.tiles * p.c.heads;
}

// Start of CTA c's run of the `total` tiles on `ctas` CTAs.
__device__ __forceinline__ int64_t run_start(int64_t total, int ctas, int c)
{
    return total / ctas * c + total % ctas * c / ctas;
}

struct Place {
    int64_t total;  // tiles of all units
    int64_t at;     // the tile looked for
    int64_t off;    // ... counted from the first of its sequence
    int b;
    int ctas;       // CTAs that get a run
};

// Where run `c` of at most `grid` runs begins; the whole block calls it.
// words: 34 64-bit words of shared memory.
template <int THREADS>
__device__ Place find_run(const TreePlan &p, int grid, int c, int64_t *words)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto scan = [&](int64_t v, int64_t &sum) {  // sum before this thread; sum of all
        int64_t x = v;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d)
                x += y;
        }
        __syncthreads();
        if (lane == 31)
            words[warp] = x;
        __syncthreads();
        int64_t before = x - v;
        sum = 0;
        for (int w = 0; w < THREADS / 32; ++w) {
            const int64_t y = words[w];
            before += w < warp ? y : 0;
            sum += y;
        }
        return before;
    };
    Place r;
    int64_t mine = 0, one = 0;
    for (int b = threadIdx.x; b < p.seqs; b += THREADS)
        mine += one = seq_work(p, b);
    int64_t before = scan(mine, r.total);
    r.ctas = (int)(r.total < grid ? r.total : grid);
    r.b = 0;
    r.off = r.at = 0;
    if (c >= r.ctas)
        return r;
    r.at = run_start(r.total, r.ctas, c);
    int64_t base = 0, sum = r.total;
    for (int first = 0; first < p.seqs; first += THREADS) {
        const int b = first + (int)threadIdx.x;
        if (p.seqs > THREADS) {
            one = b < p.seqs ? seq_work(p, b) : 0;
            before = scan(one, sum);
        } else if (b >= p.seqs) {
            one = 0;
        }
        if (r.at >= base + before && r.at < base + before + one) {
            words[32] = b;
            words[33] = r.at - base - before;
        }
        base += sum;
    }
    __syncthreads();
    r.b = (int)words[32];
    r.off = words[33];
    return r;
}

// A run's part of one unit: tiles j0 .. j1 - 1 for rows r0 .. r0 + rows - 1.
struct Unit {
    Seq s;
    int head, r0, rows, j0, j1;
    __device__ bool two() const { return rows > kRowTile; }
    __device__ int tiles() const { return j1 - j0; }
    __device__ bool whole() const { return j0 == 0 && j1 == s.tiles; }
    __device__ bool tail(int j) const { return (j + 1) * kTile > s.n; }
};

struct Walk {
    const TreePlan &p;
    int64_t left;
    int b, unit, j;  // unit: of the sequence, head by head
    Seq s;
    __device__ Walk(const TreePlan &plan, const Place &at, int64_t tiles)
        : p(plan), left(tiles), b(at.b)
    {
        if (left > 0) {
            s = seq_of(p, b);
            unit = (int)(at.off / s.tiles);
            j = (int)(at.off % s.tiles);
        }
    }
    __device__ bool next(Unit &u)
    {
        if (left <= 0)
            return false;
        while (unit >= s.units * p.c.heads) {
            s = seq_of(p, ++b);  // there is one: tiles are left
            unit = j = 0;
        }
        u.s = s;
        u.head = unit / s.units;
        u.r0 = unit % s.units * kUnitRows;
        u.rows = (int)min((int64_t)s.T * p.group - u.r0, (int64_t)kUnitRows);
        u.j0 = j;
        u.j1 = (int)min((int64_t)s.tiles, j + left);
        left -= u.j1 - u.j0;
        j = 0;
        ++unit;
        return true;
    }
};

// ---------------------------------------------------------------------------
// Shared memory: query tiles, a ring of key and value tiles (128 positions
// each, in 128-byte swizzled rows of 64 elements), barriers.
//
// Two streams run side by side so that one's softmax hides the other's matrix
// products.  A unit of over 128 rows gives each stream a row tile and both the
// same key and value tiles; a smaller one gives them its only row tile and
// every second position tile, and their sums are put together at its end.
// ---------------------------------------------------------------------------
template <int DP>
struct Layout {
    static constexpr uint32_t kOperand = 128 * DP * 2;  // bytes of a tile of 128 x DP
    static constexpr int kStages = DP == 128 ? 5 : 8;
    static constexpr uint32_t kQ = 0, kRing = 2 * kOperand, kEnd = kRing + kStages * kOperand;
    static constexpr uint32_t kBars = kEnd;              // barriers
    static constexpr uint32_t kMisc = kBars + 320;
    static constexpr uint32_t kBytes = kMisc + 1536;
};

// Barriers, by number (8 bytes each).
enum {
    kFull = 0,        // [stage] a tile has landed
    kEmpty = 8,       // [stage] its readers are done
    kScores = 16,     // [stream] scores are in tensor memory
    kWeights = 18,    // [stream] weights are
    kSums = 20,       // [stream] the unit's output sums are
    kQuery = 22,      // query tiles are in shared memory, tensor memory is free
    kGive = 23,       // stream 1's half of the sums is in shared memory
    kTaken = 24,      // ... and has been read
    kLast = 25,       // after an expired wait: the products asked for are done
    kTail = 32,       // [stage] values to be looked over have landed
};

struct Misc {
    uint32_t tmem, abort;
    int bad[8];       // by unit: unit number + 1 where a drafted value is not finite
    int64_t words[34];
    float top[kRowTile], sum[kRowTile];  // of stream 1
};
static_assert(sizeof(Misc) <= 1536, "Misc");

struct Cta {
    uint32_t smem, bars;
    Misc *misc;
    uint32_t *status;
    uint64_t limit;
    __device__ uint32_t bar(int i) const { return bars + 8 * i; }
    // Waits for a phase; false once any wait of the CTA has run out.
    __device__ bool wait(int i, uint32_t parity) const
    {
        volatile uint32_t *abort = &misc->abort;
        if (limit ? mbar_try_wait(bar(i), parity) : mbar_test_wait(bar(i), parity))
            return true;
        const uint64_t t0 = limit ? global_ns() : 0;
        while (limit) {
            if (mbar_try_wait(bar(i), parity))
                return true;
            if (*abort)
                return false;
            if (global_ns() - t0 > limit)
                break;
        }
        *abort = 1;
        if (status)
            *reinterpret_cast<volatile uint32_t *>(status) = 1u;
        return false;
    }
};

// Place in the ring of the keys and values of the i-th tile of n, counted from
// the unit's first load: the order in which the products use them.
__device__ __forceinline__ int key_item(bool two, int i)
{
    return two ? 2 * i : i < 2 ? i : 2 * i - 1;
}
__device__ __forceinline__ int value_item(bool two, int i, int n)
{
    return two ? 2 * i + 1 : i + min(n, i + 2);
}

__device__ __forceinline__ uint32_t swizzled(uint32_t row, uint32_t chunk)  // 16-byte chunks
{
    return (chunk >> 3) * (128 * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

__device__ __forceinline__ uint4 lds16(uint32_t smem)
{
    uint4 r;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "r"(smem)
                 : "memory");
    return r;
}
__device__ __forceinline__ void sts16(uint32_t smem, const uint4 &v)
{
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(smem), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ void sts4(uint32_t smem, float v)
{
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(smem), "f"(v) : "memory");
}
__device__ __forceinline__ float lds4(uint32_t smem)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(smem) : "memory");
    return v;
}

// Zeroes the elements of a pair that are not finite; true if there was one.
template <bool BF16>
__device__ __forceinline__ bool clean(uint32_t &pair)
{
    constexpr uint32_t e = BF16 ? 0x7f80u : 0x7c00u;
    const bool lo = (pair & e) == e, hi = (pair >> 16 & e) == e;
    if (lo)
        pair &= 0xffff0000u;
    if (hi)
        pair &= 0x0000ffffu;
    return lo || hi;
}

// ---------------------------------------------------------------------------
// Loads.  A value that a row does not see must not reach it, not even times a
// weight of 0: values past the sequence's end read as zeros, and drafted values
// that are not finite are zeroed in shared memory and added at the unit's end
// to the rows that see them.
// ---------------------------------------------------------------------------

// Which tile (*i of the unit's n) of which pool is the unit's item-th load.
__device__ __forceinline__ bool is_value(bool two, int item, int n, int *i)
{
    if (two) {
        *i = item >> 1;
        return item & 1;
    }
    const int ahead = min(n, 2), rest = item - ahead, pairs = max(n - 2, 0);
    if (rest < 0) {
        *i = item;
        return false;
    }
    if (rest >= 2 * pairs) {  // V0 K2 V1 K3 ... and then the last values
        *i = rest - pairs;
        return true;
    }
    *i = rest & 1 ? (rest >> 1) + 2 : rest >> 1;
    return !(rest & 1);
}

// Pages of a multiple of 8 tokens: one lane per box of `box` positions (the
// largest power of two that divides a page, at most a tile), by tensor maps of
// (dim, token, head, page); positions without a page read as zeros.
struct Maps {
    CUtensorMap pool[2];
    int box;
    int token_dim, head_dim;  // places of the token and the head among dims 1..3
};

template <int DP>
__device__ void box_role(const TreePlan &p, const Maps &maps, const Cta &cta, Walk walk)
{
    using L = Layout<DP>;
    const KvView &c = p.c;
    const int lane = threadIdx.x & 31, boxes = kTile / maps.box;
    uint32_t k = 0, tail_use = 0, tail_parity = 0;  // by stage: its last load, uses of kTail
    Unit u;
    while (walk.next(u)) {
        const int n = u.tiles();
        for (int item = 0; item < 2 * n; ++item, ++k) {
            int i;
            const bool value = is_value(u.two(), item, n, &i);
            const int j = u.j0 + i, pos = j * kTile + lane * maps.box;
            int page = c.pages;  // past the pool: zeros
            if (lane < boxes && pos < u.s.end && pos / c.page_tokens < c.width) {
                page = __ldg(c.table + (int64_t)u.s.slot * c.width + pos / c.page_tokens);
                if (page < 0 || page > c.pages)
                    page = c.pages;
            }
            const uint32_t stage = k % L::kStages, tile = cta.smem + L::kRing + stage * L::kOperand;
            const bool tail = value && u.tail(j);
            bool ok = true;
            if (lane == 0) {
                ok = cta.wait(kEmpty + stage, (k / L::kStages & 1) ^ 1);
                if (ok) {
                    mbar_expect_tx(cta.bar((tail ? kTail : kFull) + stage), L::kOperand);
                    if (!tail)
                        mbar_arrive(cta.bar(kFull + stage));
                }
            }
            if (!__all_sync(0xffffffffu, ok)) {
                // Let the tiles asked for land (bounded).
                for (uint32_t x = k - min(k, (uint32_t)L::kStages); x < k; ++x) {
                    const uint32_t s = x % L::kStages;
                    if (tail_use >> s & 1)
                        mbar_wait_bounded(cta.bar(kTail + s), tail_parity >> s & 1 ^ 1);
                    else
                        mbar_wait_bounded(cta.bar(kFull + s), x / L::kStages & 1);
                }
                return;
            }
            tail_use = (tail_use & ~(1u << stage)) | (uint32_t)tail << stage;
            tail_parity ^= (uint32_t)tail << stage;
            if (lane < boxes) {
                const int token = pos % c.page_tokens;
                int at[4] = {0, page, page, page};
                at[maps.token_dim] = token;
                at[maps.head_dim] = u.head;
#pragma unroll
                for (int h = 0; h < DP / 64; ++h)
                    asm volatile(
                        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::"
                        "complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
                            tile + h * (128 * 128) + lane * maps.box * 128),
                        "l"(&maps.pool[value]), "r"(64 * h), "r"(at[1]), "r"(at[2]), "r"(at[3]),
                        "r"(cta.bar((tail ? kTail : kFull) + stage))
                        : "memory");
            }
            __syncwarp();
        }
    }
}

// Looks over the values of the tiles that hold drafts.
template <int DP, bool BF16>
__device__ void fix_role(const TreePlan &p, const Cta &cta, Walk walk)
{
    using L = Layout<DP>;
    constexpr int kChunks = DP / 8;
    const int lane = threadIdx.x & 31, tid = threadIdx.x - 9 * 32;
    uint32_t k = 0, parity = 0;
    Unit u;
    for (int units = 0; walk.next(u); ++units) {
        const int n = u.tiles();
        for (int i = max(u.s.n / kTile - u.j0, 0); i < n; ++i) {
            const uint32_t item = k + value_item(u.two(), i, n), stage = item % L::kStages;
            const uint32_t tile = cta.smem + L::kRing + stage * L::kOperand;
            if (!__all_sync(0xffffffffu, cta.wait(kTail + stage, parity >> stage & 1)))
                return;
            parity ^= 1u << stage;
            const int base = (u.j0 + i) * kTile;
            for (int x = max(u.s.n - base, 0) * kChunks + tid; x < kTile * kChunks; x += 32 * kFixWarps) {
                const uint32_t at = tile + swizzled(x / kChunks, x % kChunks);
                if (base + x / kChunks >= u.s.end) {
                    sts16(at, uint4{0, 0, 0, 0});
                } else {
                    uint4 v = lds16(at);
                    const bool a = clean<BF16>(v.x), b = clean<BF16>(v.y), d = clean<BF16>(v.z),
                               e = clean<BF16>(v.w);
                    if (a || b || d || e) {
                        sts16(at, v);
                        cta.misc->bad[units & 7] = units + 1;
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(cta.bar(kFull + stage));
        }
        k += 2 * n;
    }
}

// Any other page: each of three warps takes 16 rows of a tile at a time, its
// lanes 16 bytes each, by asynchronous copies, and looks over its own drafts.
constexpr int kInFlight = 2;  // tiles behind the one being requested

template <int DP, bool BF16>
__device__ void load_role(const TreePlan &p, const Cta &cta, Walk walk)
{
    using L = Layout<DP>;
    constexpr int kChunks = DP / 8;            // 16-byte chunks of a row
    constexpr int kLanesRows = 32 / kChunks;   // rows a warp covers in one step
    const KvView &c = p.c;
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - 8;
    const int chunk = lane % kChunks;
    uint32_t k = 0;     // loads asked for
    uint32_t done = 0;  // loads handed over
    struct Asked {
        int first_draft, end;  // of a value tile: positions from .. to are drafts; 0, 0: keys
        int unit, base;
    } asked[kInFlight + 1];
    Unit u;
    int units = 0;
    // The oldest load in flight has landed: look its drafts over, hand it on.
    auto hand_over = [&]() {
        const Asked &a = asked[0];
        const uint32_t tile = cta.smem + L::kRing + done % L::kStages * L::kOperand;
        if (a.end > a.base && a.first_draft < a.base + kTile && a.end > a.first_draft) {
            for (int block = warp; block < kTile / 16; block += kLoadWarps)
                for (int r = 0; r < 16; r += kLanesRows) {
                    const int row = block * 16 + r + lane / kChunks, pos = a.base + row;
                    if (pos >= a.first_draft && pos < a.end) {
                        uint4 v = lds16(tile + swizzled(row, chunk));
                        const bool x = clean<BF16>(v.x), y = clean<BF16>(v.y), z = clean<BF16>(v.z),
                                   w = clean<BF16>(v.w);
                        if (x || y || z || w) {
                            sts16(tile + swizzled(row, chunk), v);
                            cta.misc->bad[a.unit & 7] = a.unit + 1;
                        }
                    }
                }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(cta.bar(kFull + done % L::kStages));
        ++done;
#pragma unroll
        for (int i = 0; i < kInFlight; ++i)
            asked[i] = asked[i + 1];
    };
    for (; walk.next(u); ++units) {
        const int n = u.tiles(), items = 2 * n;
        for (int item = 0; item < items; ++item, ++k) {
            int i;
            const bool value = is_value(u.two(), item, n, &i);
            const int base = (u.j0 + i) * kTile;
            const uint32_t stage = k % L::kStages, tile = cta.smem + L::kRing + stage * L::kOperand;
            bool ok = lane != 0 || cta.wait(kEmpty + stage, (k / L::kStages & 1) ^ 1);
            if (!__all_sync(0xffffffffu, ok))
                goto out;
            const char *pool = c.pool[value] + u.head * c.head_stride;
            for (int block = warp; block < kTile / 16; block += kLoadWarps) {
                int64_t at = -1;
                const int pos = base + block * 16 + (lane & 15);
                if (pos < u.s.end && pos / c.page_tokens < c.width) {
                    const int page = c.table[(int64_t)u.s.slot * c.width + pos / c.page_tokens];
                    if (page >= 0 && page < c.pages)
                        at = page * c.page_stride + pos % c.page_tokens * c.token_stride;
                }
#pragma unroll
                for (int r = 0; r < 16; r += kLanesRows) {
                    const int row = r + lane / kChunks;
                    const int64_t from = __shfl_sync(0xffffffffu, at, row);
                    const bool real = from >= 0 && chunk * 16 < c.row_bytes;
                    const char *src = real ? pool + from + chunk * 16 : c.pool[0];
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                     tile + swizzled(block * 16 + row, chunk)),
                                 "l"(src), "r"(real ? 16 : 0)
                                 : "memory");
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            const Asked now{value ? u.s.n : 0, value ? u.s.end : 0, units, base};
            if (k - done == kInFlight) {
                asked[kInFlight] = now;
                asm volatile("cp.async.wait_group %0;" ::"n"(kInFlight) : "memory");
                hand_over();
            } else {
#pragma unroll
                for (int s = 0; s < kInFlight; ++s)
                    if ((uint32_t)s == k - done)
                        asked[s] = now;
            }
        }
    }
out:
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    while (done < k)
        hand_over();
}

// ---------------------------------------------------------------------------
// Matrix products: one thread.  Tensor memory columns: scores of the streams
// at 0 and 128 (their weights, 16 bits each, over the scores' first half),
// output sums at 256 and 384.
// ---------------------------------------------------------------------------
template <int DP, bool BF16>
__device__ void product_role(const TreePlan &p, const Cta &cta, Walk walk)
{
    using L = Layout<DP>;
    constexpr uint32_t kScoreDesc = umma_idesc(BF16, kTile, false);
    constexpr uint32_t kSumDesc = umma_idesc(BF16, DP, true);
    const uint32_t tmem = cta.misc->tmem, ring = cta.smem + L::kRing;
    uint32_t k = 0;               // loads before this unit
    uint32_t weights[2] = {0, 0}; // weight tiles taken per stream
    uint32_t units = 0;
    Unit u;

    auto scores = [&](int stream, bool two, uint32_t stage) {
        const uint32_t q = cta.smem + L::kQ + (two ? stream : 0) * L::kOperand;
        const uint32_t key = ring + stage * L::kOperand;
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk) {
            const uint32_t off = (kk >> 2) * (128 * 128) + (kk & 3) * 32;
            umma_ss(tmem + stream * 128, umma_desc(q + off, 0), umma_desc(key + off, 0), kScoreDesc,
                    kk > 0);
        }
    };
    auto sums = [&](int stream, uint32_t stage, bool add) {
        const uint32_t value = ring + stage * L::kOperand;
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
            umma_ts(tmem + 256 + stream * 128, tmem + stream * 128 + kk * 8,
                    umma_desc(value + kk * 16 * 128, 128 * 128), kSumDesc, add || kk > 0);
    };
    auto landed = [&](uint32_t item) { return cta.wait(kFull + item % L::kStages, item / L::kStages & 1); };
    auto release = [&](uint32_t item) { umma_commit(cta.bar(kEmpty + item % L::kStages)); };

    for (; walk.next(u); ++units) {
        const int n = u.tiles();
        const bool two = u.two();
        if (!cta.wait(kQuery, units & 1))
            return;
        tc_fence_after();
        for (int s = 0; s < 2; ++s) {  // the first scores of each stream
            const int i = two ? 0 : s;
            if (i >= n)
                break;
            const uint32_t item = k + key_item(two, i);
            if (!landed(item))
                return;
            tc_fence_after();
            scores(s, two, item % L::kStages);
            umma_commit(cta.bar(kScores + s));
            if (!two || s == 1)
                release(item);
        }
        const int steps = two ? n : (n + 1) / 2;
        for (int i = 0; i < steps; ++i)
            for (int s = 0; s < 2; ++s) {
                const int j = two ? i : 2 * i + s, after = two ? j + 1 : j + 2;
                if (j >= n)
                    break;
                const uint32_t value = k + value_item(two, j, n);
                if (!landed(value) || !cta.wait(kWeights + s, weights[s] & 1))
                    return;
                ++weights[s];
                tc_fence_after();
                sums(s, value % L::kStages, i > 0);
                if (!two || s == 1)
                    release(value);
                if (after < n) {
                    const uint32_t item = k + key_item(two, after);
                    if (!landed(item))
                        return;
                    tc_fence_after();
                    scores(s, two, item % L::kStages);
                    umma_commit(cta.bar(kScores + s));
                    if (!two || s == 1)
                        release(item);
                } else {
                    umma_commit(cta.bar(kSums + s));
                }
            }
        k += 2 * n;
    }
}

// ---------------------------------------------------------------------------
// Softmax: a thread is a row of its stream's row tile.
// ---------------------------------------------------------------------------
// Partial sums of a cut unit: [slot][row] maxima (of scores times scale *
// log2 e), sums and, unnormalised, outputs.  Run c writes the unit it begins
// inside of to slot 2 c and one that goes on after it to slot 2 c + 1.
__host__ __device__ constexpr uint64_t part_floats(int dp)
{
    return (uint64_t)kUnitRows * (dp + 2);
}

__device__ __forceinline__ float *part_of(const TreePlan &p, int dp, int slot)
{
    return static_cast<float *>(p.workspace) + slot * part_floats(dp);
}

// The bits of mask row `row` from draft `d` (possibly negative) on, for 32
// positions: committed ones are seen, drafts from T on are not.
__device__ __forceinline__ uint32_t seen_word(const TreePlan &p, const Seq &s, int64_t row, int d)
{
    if (d <= -32)
        return 0xffffffffu;
    const uint32_t *words = p.mask + row * p.mask_words;
    auto word = [&](int w) { return w < p.mask_words ? __ldg(words + w) : 0u; };
    uint32_t v;
    if (d < 0) {
        v = word(0);
        if (s.T < 32)
            v &= (1u << s.T) - 1;
        return v << -d | (0xffffffffu >> (32 + d));
    }
    if (d >= s.T)
        return 0;
    v = __funnelshift_r(word(d >> 5), word((d >> 5) + 1), d & 31);
    return s.T - d < 32 ? v & ((1u << (s.T - d)) - 1) : v;
}

template <int DP, bool BF16>
__device__ void softmax_role(const TreePlan &p, const Cta &cta, Walk walk, int run)
{
    using L = Layout<DP>;
    constexpr int kChunks = DP / 8;
    const int stream = threadIdx.x >> 7, tid = threadIdx.x & 127;
    const int lane = threadIdx.x & 31, warp = tid >> 5;
    const uint32_t lanes = cta.misc->tmem + ((uint32_t)(warp * 32) << 16);
    const uint32_t score_cols = lanes + stream * 128, sum_cols = lanes + 256 + stream * 128;
    const float scale = fabsf(p.scale), c = scale * 1.44269504088896340736f;
    const uint32_t flip = p.scale < 0.0f ? 0x80008000u : 0u;
    // The running maximum moves only when a row's grows by 8 powers of two:
    // weights stay below 2^8, exact in the 32-bit sums, and most tiles need no
    // pass over the output sums.
    const float slack = c > 0.0f ? 8.0f / c : INFINITY;
    uint32_t tiles_seen = 0, sums_seen[2] = {0, 0}, gives = 0;
    bool other_ran = false;
    Unit u;
    for (int units = 0; walk.next(u); ++units) {
        const bool two = u.two();
        // The query tiles are free once both streams' products have read them.
        if (other_ran && !__all_sync(0xffffffffu, cta.wait(kSums + 1 - stream, sums_seen[1]++ & 1)))
            return;
        other_ran = two || stream == 1 || u.tiles() > 1;
        // Query rows, swizzled; rows past the unit's read as zeros.
        const int q_rows = two ? kUnitRows : kRowTile;
        for (int i = threadIdx.x; i < q_rows * kChunks; i += 256) {
            const int row = i / kChunks, chunk = i % kChunks;
            uint4 v{0, 0, 0, 0};
            if (row < u.rows && chunk * 16 < p.c.row_bytes) {
                const int r = u.r0 + row;
                v = __ldg(reinterpret_cast<const uint4 *>(
                    p.q + (int64_t)(u.s.row0 + r / p.group) * p.q_row +
                    (int64_t)(u.head * p.group + r % p.group) * p.q_head + chunk * 16));
                v.x ^= flip, v.y ^= flip, v.z ^= flip, v.w ^= flip;
            }
            sts16(cta.smem + L::kQ + (row >> 7) * L::kOperand + swizzled(row & 127, chunk), v);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(cta.bar(kQuery));

        const int mine = (two ? stream * kRowTile : 0) + tid;  // row of the unit
        const bool active = mine - lane < u.rows;              // any row of the warp
        const int64_t q_row = u.s.row0 + min(u.r0 + mine, u.s.T * p.group - 1) / p.group;
        const int step = two ? 1 : 2, first = u.j0 + (two ? 0 : stream);
        float top = -INFINITY, sum = 0.0f;
        for (int j = first; j < u.j1; j += step) {
            if (!__all_sync(0xffffffffu, cta.wait(kScores + stream, tiles_seen++ & 1)))
                return;
            tc_fence_after();
            if (active) {
                uint32_t s[4][32];
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    tmem_load32(s[g], score_cols + 32 * g);
                tmem_wait_load();
                uint32_t seen[4] = {~0u, ~0u, ~0u, ~0u};
                const bool tail = u.tail(j);
                if (tail) {
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        seen[g] = u.s.end > 0 ? seen_word(p, u.s, q_row, j * kTile + 32 * g - u.s.n) : 0;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!(seen[g] >> i & 1))
                                s[g][i] = __float_as_uint(-INFINITY);
                    }
                }
                float m[4];
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    m[g] = __uint_as_float(s[g][0]);
#pragma unroll
                    for (int i = 1; i < 32; ++i)
                        m[g] = fmaxf(m[g], __uint_as_float(s[g][i]));
                }
                const float here = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
                const bool moves = here > (top == -INFINITY ? top : top + slack);
                float old = 1.0f;
                if (moves) {
                    old = top == -INFINITY ? 0.0f : exp2_fast((top - here) * c);
                    top = here;
                    sum *= old;
                }
                if (j != first && __any_sync(0xffffffffu, moves)) {
                    for (int g = 0; g < DP / 32; ++g) {
                        uint32_t o[32];
                        tmem_load32(o, sum_cols + 32 * g);
                        tmem_wait_load();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * old);
                        tmem_store32(sum_cols + 32 * g, o);
                    }
                }
                const float shift = top == -INFINITY ? 0.0f : top * c;
                float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int g = 0; g < 4; ++g)
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        float w = exp2_fast(fmaf(__uint_as_float(s[g][i]), c, -shift));
                        if (tail && !(seen[g] >> i & 1))
                            w = 0.0f;
                        part[i & 3] += w;
                        s[g][i] = __float_as_uint(w);
                    }
                sum += (part[0] + part[1]) + (part[2] + part[3]);
                // Weights in 16 bits for the second product, as its operand
                // type asks: a relative error of at most half an ulp each; the
                // sum above is of the unrounded ones.
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    uint32_t w[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        w[i] = pack16<BF16>(__uint_as_float(s[2 * g + i / 16][2 * i % 32]),
                                            __uint_as_float(s[2 * g + i / 16][2 * i % 32 + 1]));
                    tmem_store32(score_cols + 32 * g, w);
                }
                tmem_wait_store();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(cta.bar(kWeights + stream));
        }
        const bool any = first < u.j1;
        if (any) {
            if (!__all_sync(0xffffffffu, cta.wait(kSums + stream, sums_seen[0]++ & 1)))
                return;
            tc_fence_after();
        }

        // The unit's end.  With one row tile stream 1 hands its sums to stream
        // 0 through the free query tile, half the columns at a time, column by
        // column so that neighbours write neighbouring words.
        const uint32_t box = cta.smem + L::kQ + L::kOperand + tid * 4;
        constexpr int kHalf = DP / 2;
        const bool joins = !two && u.tiles() > 1;
        if (joins && stream == 1) {
            cta.misc->top[tid] = top;
            cta.misc->sum[tid] = sum;
            for (int h = 0; h < 2; ++h) {
                if (active)
                    for (int g = 0; g < kHalf / 32; ++g) {
                        uint32_t o[32];
                        tmem_load32(o, sum_cols + h * kHalf + 32 * g);
                        tmem_wait_load();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            sts4(box + (32 * g + i) * 512, __uint_as_float(o[i]));
                    }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(cta.bar(kGive));
                if (!__all_sync(0xffffffffu, cta.wait(kTaken, gives++ & 1)))
                    return;
            }
        }
        if (!two && stream == 1)
            continue;
        float a = 1.0f, b = 0.0f;  // factors of the two streams' sums
        if (joins) {
            if (!__all_sync(0xffffffffu, cta.wait(kGive, gives & 1)))
                return;
            const float other = cta.misc->top[tid], most = fmaxf(top, other);
            a = top == -INFINITY ? 0.0f : exp2_fast((top - most) * c);
            b = other == -INFINITY ? 0.0f : exp2_fast((other - most) * c);
            if (top == most)  // also where both are -inf or infinite
                a = 1.0f;
            if (other == most)
                b = 1.0f;
            top = most;
            sum = sum * a + cta.misc->sum[tid] * b;
        }
        const bool whole = u.whole();
        const bool bad = *(volatile int *)&cta.misc->bad[units & 7] == units + 1;
        const bool real = mine < u.rows;
        const int r = u.r0 + mine, q_head = u.head * p.group + r % p.group;
        char *out = p.out + q_row * p.o_row + (int64_t)q_head * p.o_head;
        float *part = part_of(p, DP, 2 * run + (u.j0 == 0 ? 1 : 0));
        const float inv = whole ? (sum == 0.0f ? 0.0f : 1.0f / sum) : 1.0f;
        if (real) {
            const float log2_top = top == -INFINITY ? top : top * c;
            if (!whole) {
                part[mine] = log2_top;
                part[kUnitRows + mine] = sum;
            } else if (p.lse) {
                p.lse[q_row * p.q_heads + q_head] =
                    top == -INFINITY && sum == 0.0f ? -INFINITY : top * scale + logf(sum);
            }
        }
        for (int g = 0; g < DP / 32; ++g) {
            if (joins && g == kHalf / 32) {  // the second half of stream 1's sums
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(cta.bar(kTaken));
                ++gives;
                if (!__all_sync(0xffffffffu, cta.wait(kGive, gives & 1)))
                    return;
            }
            if (active) {
                uint32_t o[32];
                tmem_load32(o, sum_cols + 32 * g);
                tmem_wait_load();
                float x[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    x[i] = __uint_as_float(o[i]) * a;
                    if (joins)
                        x[i] = fmaf(lds4(box + (g % (kHalf / 32) * 32 + i) * 512), b, x[i]);
                }
                if (bad && real) {
                    // Drafted values that are not finite, for the rows that see them.
                    const int from = max(u.j0 * kTile - u.s.n, 0);
                    const int to = min(u.j1 * kTile - u.s.n, u.s.T);
                    for (int d = from; d < to; ++d) {
                        const int pos = u.s.n + d;
                        if (!(seen_word(p, u.s, q_row, d) & 1u) || pos / p.c.page_tokens >= p.c.width)
                            continue;
                        const int page = p.c.table[(int64_t)u.s.slot * p.c.width + pos / p.c.page_tokens];
                        if (page < 0 || page >= p.c.pages)
                            continue;
                        const char *v = p.c.pool[1] + page * p.c.page_stride +
                                        pos % p.c.page_tokens * p.c.token_stride + u.head * p.c.head_stride;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (32 * g + i < p.head_dim) {
                                const uint32_t e = reinterpret_cast<const uint16_t *>(v)[32 * g + i];
                                const uint32_t big = BF16 ? 0x7f80u : 0x7c00u, frac = BF16 ? 0x7fu : 0x3ffu;
                                if ((e & big) == big)
                                    x[i] += e & frac ? NAN : e >> 15 ? -INFINITY : INFINITY;
                            }
                    }
                }
                if (real) {
                    if (whole) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (32 * g + 8 * q < p.head_dim) {
                                uint4 v;
                                v.x = pack16<BF16>(x[8 * q] * inv, x[8 * q + 1] * inv);
                                v.y = pack16<BF16>(x[8 * q + 2] * inv, x[8 * q + 3] * inv);
                                v.z = pack16<BF16>(x[8 * q + 4] * inv, x[8 * q + 5] * inv);
                                v.w = pack16<BF16>(x[8 * q + 6] * inv, x[8 * q + 7] * inv);
                                *reinterpret_cast<uint4 *>(out + (32 * g + 8 * q) * 2) = v;
                            }
                    } else {
                        float4 *to = reinterpret_cast<float4 *>(part + 2 * kUnitRows + mine * DP + 32 * g);
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            to[q] = make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
                    }
                }
            }
        }
        if (joins) {  // and every warp has read its part before the query tile is written again
            __syncwarp();
            if (lane == 0)
                mbar_arrive(cta.bar(kTaken));
            if (!__all_sync(0xffffffffu, cta.wait(kTaken, gives++ & 1)))
                return;
        }
    }
}

template <int DP, bool BF16, bool BOXES>
__global__ void __launch_bounds__(kThreads, 1)
    k_tree(const __grid_constant__ TreePlan p, const __grid_constant__ Maps maps)
{
    using L = Layout<DP>;
    extern __shared__ __align__(1024) unsigned char raw[];
    const uint32_t at = smem_u32(raw), pad = (1024 - (at & 1023)) & 1023;
    Cta cta;
    cta.smem = at + pad;
    cta.bars = cta.smem + L::kBars;
    cta.misc = reinterpret_cast<Misc *>(raw + pad + L::kMisc);
    cta.status = p.status;
    cta.limit = p.wait_ns;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < L::kStages; ++i) {
            mbar_init_count(cta.bar(kFull + i), BOXES ? kFixWarps : kLoadWarps);
            mbar_init_count(cta.bar(kTail + i), 1);
            mbar_init_count(cta.bar(kEmpty + i), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init_count(cta.bar(kScores + s), 1);
            mbar_init_count(cta.bar(kWeights + s), 4);
            mbar_init_count(cta.bar(kSums + s), 1);
        }
        mbar_init_count(cta.bar(kQuery), 8);
        mbar_init_count(cta.bar(kGive), 4);
        mbar_init_count(cta.bar(kTaken), 4);
        mbar_init_count(cta.bar(kLast), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        cta.misc->abort = 0;
        for (int i = 0; i < 8; ++i)
            cta.misc->bad[i] = 0;
    }
    if (warp == 8)
        tmem_alloc(smem_u32(&cta.misc->tmem));
    pdl_wait_prerequisite();
    pdl_launch_dependents();
    const Place place = find_run<kThreads>(p, gridDim.x, blockIdx.x, cta.misc->words);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if ((int)blockIdx.x < place.ctas) {
        const Walk walk(p, place, run_start(place.total, place.ctas, blockIdx.x + 1) - place.at);
        // The block was launched with 384 * 168 registers: 128 * 72 stay with
        // the last four warps, 256 * 216 are all of the rest.
        if (warp < 8) {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
            softmax_role<DP, BF16>(p, cta, walk, blockIdx.x);
        } else {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
            if (warp == 8 + kLoadWarps) {
                if (lane == 0)
                    product_role<DP, BF16>(p, cta, walk);
            } else if (!BOXES) {
                load_role<DP, BF16>(p, cta, walk);
            } else if (warp == 8) {
                box_role<DP>(p, maps, cta, walk);
            } else {
                fix_role<DP, BF16>(p, cta, walk);
            }
        }
    }
    // After an expired wait products may still run: let them end (bounded).
    if (threadIdx.x == 8 * 32 + kLoadWarps * 32 && cta.misc->abort) {
        umma_commit(cta.bar(kLast));
        mbar_wait_bounded(cta.bar(kLast), 0);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_free(cta.misc->tmem);
    }
}

// ---------------------------------------------------------------------------
// Joins the parts of the units that run ends cut: CTA (x, y) looks at the end
// of run x and takes rows kJoinRows y onwards of the unit it falls into, if
// no earlier run ends in that unit.  A warp takes a row at a time.
// ---------------------------------------------------------------------------
template <int DP, bool BF16>
__global__ void __launch_bounds__(kJoinThreads) k_tree_join(const TreePlan p, int grid)
{
    __shared__ int64_t words[34];
    pdl_launch_dependents();
    // Lengths and row starts were final before the launch ahead began: only
    // the parts have to be waited for.
    const Place at = find_run<kJoinThreads>(p, grid, blockIdx.x + 1, words);
    if ((int)blockIdx.x + 1 >= at.ctas)
        return;
    Walk walk(p, at, 1);
    Unit u;
    walk.next(u);
    const int64_t unit_start = at.at - u.j0;
    const int row0 = blockIdx.y * kJoinRows;
    if (u.j0 == 0 || row0 >= u.rows || run_start(at.total, at.ctas, blockIdx.x) > unit_start)
        return;
    pdl_wait_prerequisite();
    const int64_t unit_end = unit_start + u.s.tiles;
    int last = blockIdx.x + 1;  // the unit's last run
    while (last + 1 < at.ctas && run_start(at.total, at.ctas, last + 1) < unit_end)
        ++last;
    const int lane = threadIdx.x & 31;
    constexpr int kPer = DP / 32;
    for (int row = row0 + (threadIdx.x >> 5); row < min(row0 + kJoinRows, u.rows);
         row += kJoinThreads / 32) {
        float top = -INFINITY, sum = 0.0f, x[kPer];
        for (int run = blockIdx.x; run <= last; ++run)
            top = fmaxf(top, part_of(p, DP, 2 * run + (run == (int)blockIdx.x))[row]);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            x[i] = 0.0f;
#pragma unroll 4
        for (int run = blockIdx.x; run <= last; ++run) {
            const float *part = part_of(p, DP, 2 * run + (run == (int)blockIdx.x));
            const float t = part[row], f = t == top ? 1.0f : t == -INFINITY ? 0.0f : exp2_fast(t - top);
            sum = fmaf(part[kUnitRows + row], f, sum);
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                x[i] = fmaf(part[2 * kUnitRows + row * DP + lane * kPer + i], f, x[i]);
        }
        const int r = u.r0 + row, q_head = u.head * p.group + r % p.group;
        const int64_t q_row = u.s.row0 + r / p.group;
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        uint32_t *out = reinterpret_cast<uint32_t *>(p.out + q_row * p.o_row + (int64_t)q_head * p.o_head);
        if (lane * kPer < p.head_dim)
#pragma unroll
            for (int i = 0; i < kPer / 2; ++i)
                out[lane * kPer / 2 + i] = pack16<BF16>(x[2 * i] * inv, x[2 * i + 1] * inv);
        if (p.lse && lane == 0)
            p.lse[q_row * p.q_heads + q_head] =
                top == -INFINITY && sum == 0.0f ? -INFINITY : top * 0.69314718055994530942f + logf(sum);
    }
}

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

// Tensor maps of the two pools; false where the pages' shape does not allow
// them (the kernel then loads by threads).
bool make_maps(const TreePlan &p, Maps *m)
{
    using Encode = decltype(&cuTensorMapEncodeTiled);
    static const Encode encode = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                             &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return reinterpret_cast<Encode>(fn);
    }();
    const KvView &c = p.c;
    if (!encode || c.page_tokens % 8)
        return false;
    m->box = 8;
    while (m->box < kTile && c.page_tokens % (2 * m->box) == 0)
        m->box *= 2;
    // Dimensions in the order of their strides.
    struct Dim {
        int64_t stride;
        uint32_t extent, box;
        int what;  // 0 token, 1 head, 2 page
    } dim[3] = {{c.token_stride, (uint32_t)c.page_tokens, (uint32_t)m->box, 0},
                {c.head_stride, (uint32_t)c.heads, 1, 1},
                {c.page_stride, (uint32_t)c.pages, 1, 2}};
    for (Dim &d : dim)
        if (d.extent == 1)  // its stride says nothing
            d.stride = c.row_bytes;
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2 - i; ++j)
            if (dim[j].stride > dim[j + 1].stride) {
                const Dim d = dim[j];
                dim[j] = dim[j + 1];
                dim[j + 1] = d;
            }
    cuuint64_t extent[4] = {(cuuint64_t)p.head_dim}, stride[3];
    cuuint32_t box[4] = {64}, step[4] = {1, 1, 1, 1};
    for (int i = 0; i < 3; ++i) {
        extent[i + 1] = dim[i].extent;
        stride[i] = (cuuint64_t)dim[i].stride;
        box[i + 1] = dim[i].box;
        if (dim[i].what == 0)
            m->token_dim = i + 1;
        if (dim[i].what == 1)
            m->head_dim = i + 1;
    }
    for (int x = 0; x < 2; ++x)
        if (encode(&m->pool[x],
                   p.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                   c.pool[x], extent, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return false;
    return true;
}

template <int DP, bool BF16, bool BOXES>
cudaError_t launch_loads(const TreePlan &p, const Maps &maps, int num_sms, bool pdl, cudaStream_t stream)
{
    constexpr size_t smem = Layout<DP>::kBytes + 1024;
    if (resident_ctas((const void *)k_tree<DP, BF16, BOXES>, kThreads, smem) < 1)
        return cudaErrorInvalidConfiguration;
    return launch(k_tree<DP, BF16, BOXES>, dim3(num_sms), kThreads, smem, pdl, stream, p, maps);
}

template <int DP, bool BF16>
cudaError_t launch_dim(const TreePlan &p, int num_sms, bool pdl, cudaStream_t stream)
{
    alignas(64) Maps maps;
    const cudaError_t e = make_maps(p, &maps)
                              ? launch_loads<DP, BF16, true>(p, maps, num_sms, pdl, stream)
                              : launch_loads<DP, BF16, false>(p, maps, num_sms, pdl, stream);
    if (e != cudaSuccess || num_sms < 2)
        return e;
    return launch(k_tree_join<DP, BF16>, dim3(num_sms - 1, kUnitRows / kJoinRows), kJoinThreads, 0, pdl,
                  stream, p, num_sms);
}

}  // namespace

uint64_t tree_workspace_bytes(int num_sms, int head_dim)
{
    return 2 * (uint64_t)num_sms * part_floats(head_dim <= 64 ? 64 : 128) * sizeof(float);
}

cudaError_t launch_tree(const TreePlan &p, int num_sms, bool pdl, cudaStream_t stream)
{
    if (p.head_dim <= 64)
        return p.bf16 ? launch_dim<64, true>(p, num_sms, pdl, stream)
                      : launch_dim<64, false>(p, num_sms, pdl, stream);
    return p.bf16 ? launch_dim<128, true>(p, num_sms, pdl, stream)
                  : launch_dim<128, false>(p, num_sms, pdl, stream);
}

}  // namespace tb
