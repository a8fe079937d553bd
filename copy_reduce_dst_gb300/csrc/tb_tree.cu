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
// A unit is up to 128 of them per stream; its work is the sequence's tiles of
// 128 positions, and kUnitCost tiles' worth of beginning and ending it.  The work
// of all units, one after another, is dealt to the CTAs in equal runs, so a long
// sequence is split over many CTAs and short ones share one, whatever their
// lengths; a unit cut by a run's end leaves partial sums that k_tree_join puts
// together.
//
// A stream is four warps that do the softmax of one 128-row tile.  The kernel
// comes with one stream, two CTAs on an SM: one's softmax, first loads and last
// stores hide the other's, which is what short sequences need; and with two
// streams, one CTA on an SM: both row tiles use the same keys and values, which
// halves what has to come from L2 when there are more than 128 rows.
//
// The mathematics: with m the running maximum of a row's scores s_j (scaled) and
// l = sum exp(s_j - m), o = sum exp(s_j - m) v_j over the positions so far, a new
// maximum m' multiplies l and o by exp(m - m'); parts of one row (m, l, o) are
// joined the same way, and out = o / l, lse = m + ln l.  Powers are of two,
// scale * log2 e being part of the exponent's factor.
//
// What bounds it: up to about 128 rows a cache head, the keys and values from
// HBM (8 sequences of 32768 positions, 32 rows: 174 us, 6.2 TB/s; 32 sequences
// of up to 4096, 128 rows: 63 us, 4.3 TB/s; 40 us of that at the copy rate, 6 for
// the join, the rest start and uneven ends of the runs); above, each stream's chain of scores,
// maximum, weights and sums (131072 positions, 512 rows in two streams: 238 us,
// 1155 TFLOP/s, tensor pipe 50% busy); for small calls the two launches and one
// tile's chain (500 positions, 32 rows: 11 us).
// ---------------------------------------------------------------------------
constexpr int kTile = 128;       // positions of a tile
constexpr int kRowTile = 128;    // rows of one matrix instruction
constexpr int kLoadWarps = 3;    // load by threads, or ...
constexpr int kFixWarps = 2;     // ... one asks for tiles and two look drafts over
constexpr int kJoinThreads = 256;
// What a unit costs besides its tiles, in tiles.  With 0, 1, 2, 3 and 4: 32 chats
// 73, 69, 68, 69 and 69 us, 96 short ones 66, 53, 52, 53 and 54.
constexpr int kUnitCost = 2;

struct Seq {
    int slot, row0, T, n, end, tiles, units;  // units per cache head
};

__device__ __forceinline__ Seq seq_of(const TreePlan &p, int b, int unit_rows)
{
    Seq s;
    s.row0 = min(max(p.q_start[b], 0), p.rows);
    s.T = max(min(p.q_start[b + 1], p.rows) - s.row0, 0);
    s.slot = p.seq_slots ? p.seq_slots[b] : b;
    const bool known = s.slot >= 0 && s.slot < p.c.slots;
    s.n = known ? min(max(p.c.lens[s.slot], 0), p.c.width * p.c.page_tokens) : 0;
    s.end = known ? s.n + s.T : 0;
    s.tiles = max((s.end + kTile - 1) / kTile, 1);
    s.units = (s.T * p.group + unit_rows - 1) / unit_rows;  // rows * q_heads fits
    return s;
}

// Work is counted in 32 bits; the host refuses calls that might have more.
__device__ __forceinline__ int work_of(const TreePlan &p, const Seq &s)
{
    return s.units * p.c.heads * (s.tiles + kUnitCost);
}

struct Place {
    int total;  // work of all units
    int at;     // where the run begins
    int off;    // ... counted from the beginning of its sequence
    int b;
    int ctas;   // CTAs that get a run
    int each;   // work of every run; `more` of the runs have one on top
    int more;
    Seq s;
    // Start of run c.
    __device__ int start(int c) const { return each * c + (int)((uint32_t)(more * c) / (uint32_t)ctas); }
};

// Shared memory of find_run.
struct Found {
    int sum[32], b, off, falls;
    Seq s;
};

// Where run `c` of at most `grid` runs begins; the whole block calls it.
template <int THREADS>
__device__ Place find_run(const TreePlan &p, int unit_rows, int grid, int c, Found &found)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto scan = [&](int v, int &sum) {  // sum before this thread; sum of all
        int x = v;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d)
                x += y;
        }
        __syncthreads();
        if (lane == 31)
            found.sum[warp] = x;
        __syncthreads();
        const int w = lane < THREADS / 32 ? found.sum[lane] : 0;
        sum = __reduce_add_sync(0xffffffffu, w);
        return x - v + __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
    };
    Place r{};
    Seq s{};
    int mine = 0, one = 0;
    for (int b = threadIdx.x; b < p.seqs; b += THREADS) {
        s = seq_of(p, b, unit_rows);
        mine += one = work_of(p, s);
    }
    int before = scan(mine, r.total);
    r.ctas = min(r.total, grid);
    if (c >= r.ctas)
        return r;
    r.each = r.total / r.ctas;
    r.more = r.total - r.each * r.ctas;
    r.at = r.start(c);
    int base = 0, sum = r.total;
    for (int first = 0; first < p.seqs; first += THREADS) {
        const int b = first + (int)threadIdx.x;
        if (p.seqs > THREADS) {
            one = 0;
            if (b < p.seqs) {
                s = seq_of(p, b, unit_rows);
                one = work_of(p, s);
            }
            before = scan(one, sum);
        }
        if (r.at >= base + before && r.at - base - before < one) {
            found.b = b;
            found.off = r.at - base - before;
            found.s = s;
        }
        base += sum;
    }
    __syncthreads();
    r.b = found.b;
    r.off = found.off;
    r.s = found.s;
    return r;
}

// A run's part of one unit: tiles j0 .. j1 - 1 for rows r0 .. r0 + rows - 1.  A
// unit's own cost comes before its first tile; a run that ends within that has
// no part of the unit.
struct Unit {
    Seq s;
    int number;  // within the run
    int head, r0, rows, j0, j1;
    __device__ int tiles() const { return j1 - j0; }
    __device__ bool whole() const { return j0 == 0 && j1 == s.tiles; }
    __device__ bool tail(int j) const { return (j + 1) * kTile > s.n; }
};

struct Walk {
    const TreePlan &p;
    int left, unit_rows, number, b, unit, at;  // unit: of the sequence, head by head; at: within its work
    Seq s;
    __device__ Walk(const TreePlan &plan, int rows, const Place &place, int work)
        : p(plan), left(work), unit_rows(rows), number(0), b(place.b), s(place.s)
    {
        unit = place.off / (s.tiles + kUnitCost);
        at = place.off - unit * (s.tiles + kUnitCost);
    }
    __device__ bool next(Unit &u)
    {
        while (left > 0) {
            if (unit >= s.units * p.c.heads) {
                s = seq_of(p, ++b, unit_rows);  // there is one: work is left
                unit = 0;
                continue;
            }
            const int end = min(s.tiles + kUnitCost, at + left);
            u.j0 = max(at - kUnitCost, 0);
            u.j1 = end - kUnitCost;
            left -= end - at;
            at = 0;
            const int mine = unit++;
            if (u.j0 >= u.j1)
                continue;
            u.s = s;
            u.number = number++;
            u.head = mine / s.units;
            u.r0 = (mine - u.head * s.units) * unit_rows;
            u.rows = min(s.T * p.group - u.r0, unit_rows);
            return true;
        }
        return false;
    }
};

// ---------------------------------------------------------------------------
// Shared memory: a query tile per stream, a ring of key and value tiles, all in
// 128-byte swizzled rows of 64 elements, and barriers.  A stage of the ring
// holds 128 positions, or 64 where two CTAs of 128 dimensions share an SM.
// Tensor memory: scores of stream s from column 128 s on, their weights (16
// bits each) over the first half of them, the output sums after all scores.
// ---------------------------------------------------------------------------
template <int DP_, bool BF16_, int STREAMS_>
struct Shape {
    static constexpr int DP = DP_, STREAMS = STREAMS_;
    static constexpr bool BF16 = BF16_;
    static constexpr int kPos = STREAMS == 1 && DP == 128 ? 64 : 128;  // positions of a stage
    static constexpr int kParts = kTile / kPos;                        // stages of a tile
    static constexpr uint32_t kHalf = kPos * 128;                      // next 64 dimensions of a stage
    static constexpr uint32_t kStage = kPos * DP * 2, kQuery = kRowTile * DP * 2;
    static constexpr int kStages = STREAMS == 2 ? (DP == 128 ? 5 : 8) : DP == 128 ? 4 : 5;
    static constexpr uint32_t kRing = STREAMS * kQuery;
    static constexpr uint32_t kBars = kRing + kStages * kStage;
    static constexpr uint32_t kMisc = kBars + 320, kBytes = kMisc + 512;
    static constexpr int kUnitRows = STREAMS * kRowTile;
    static constexpr int kSoftmaxWarps = 4 * STREAMS;  // then three of loads, one of products
    static constexpr int kThreads = 32 * (kSoftmaxWarps + 4);
    static constexpr int kCols = 256 * STREAMS;
    __device__ static constexpr uint32_t score_col(int stream) { return 128 * stream; }
    __device__ static constexpr uint32_t sum_col(int stream) { return 128 * (STREAMS + stream); }
};

// Barriers, by number (8 bytes each).
enum {
    kFull = 0,        // [stage] has landed
    kEmpty = 8,       // [stage] its readers are done (a softmax warp says so)
    kTail = 16,       // [stage] values to be looked over have landed
    kQuery = 24,      // [stream] the query tile is in shared memory
    kScores = 26,     // [stream] scores are in tensor memory
    kWeights = 28,    // [stream] weights are; the unit's sums may be written
    kSums = 30,       // [stream] the unit's sums are in tensor memory
    kLast = 32,       // after an expired wait: the products asked for are done
};

struct Misc {
    uint32_t tmem, abort;
    int bad[8];       // by unit: its number + 1 where a drafted value is not finite
    Found found;
};
static_assert(sizeof(Misc) <= 512, "Misc");

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
        const uint64_t begun = limit ? global_ns() : 0;
        while (limit) {
            if (mbar_try_wait(bar(i), parity))
                return true;
            if (*abort)
                return false;
            if (global_ns() - begun > limit)
                break;
        }
        *abort = 1;
        if (status)
            *reinterpret_cast<volatile uint32_t *>(status) = 1u;
        return false;
    }
    // The same, asking without pause, as the thread that issues the products does:
    // being woken takes longer (304 units of 4096 positions, dim 64: 66 us, 70
    // woken; with the softmax warps polling as well 131072 positions take 258 us
    // for 243).
    __device__ bool poll(int i, uint32_t parity) const
    {
        volatile uint32_t *abort = &misc->abort;
        if (mbar_test_wait(bar(i), parity))
            return true;
        const uint64_t begun = limit ? global_ns() : 0;
        if (limit)
            do {
#pragma unroll 1
                for (int k = 0; k < 256; ++k)
                    if (mbar_test_wait(bar(i), parity))
                        return true;
                if (*abort)
                    return false;
            } while (global_ns() - begun <= limit);
        *abort = 1;
        if (status)
            *reinterpret_cast<volatile uint32_t *>(status) = 1u;
        return false;
    }
    // wait() for a whole warp; all lanes ask, which measured faster than one
    // asking for all (the large tree 258 us against 309).
    __device__ bool wait_warp(int i, uint32_t parity) const
    {
        return __all_sync(0xffffffffu, wait(i, parity));
    }
};

// Place of a 16-byte chunk of a row; half: bytes from one 64 elements to the next.
__device__ __forceinline__ uint32_t swizzled(uint32_t half, uint32_t row, uint32_t chunk)
{
    return (chunk >> 3) * half + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
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

// The order in which the products use them: the keys of a tile, its values, the
// keys of the next.

// Pages of a multiple of 8 tokens (a box has to begin at a multiple of 1024 bytes
// of a swizzled tile, eight rows; by threads the same pages take two to three
// times as long: 131072 positions, 128 rows in pages of 16 300 us, by boxes 110;
// 32 chats in pages of 32 168 and 66): one lane per box of `box` positions (the
// largest power of two that divides a page, at most a tile), by tensor maps of
// (dim, token, head, page); positions without a page read as zeros.
struct Maps {
    CUtensorMap pool[2];
    int box;
    int token_dim, head_dim;  // places of the token and the head among dims 1..3
};

template <class S>
__device__ void box_role(const TreePlan &p, const Maps &maps, const Cta &cta, Walk walk)
{
    const KvView &c = p.c;
    const int lane = threadIdx.x & 31, boxes = S::kPos / maps.box;
    uint32_t stage = 0, empty = 1;               // the next stage and the parity it waits for
    uint32_t k = 0, tail_use = 0, tail_parity = 0;  // loads; by stage: its last one, uses of kTail
    // Waits (bounded) until the last loads of the stages have landed.  However
    // the role ends: where another one's wait has run out, nobody else waits for
    // them, and a CTA must not leave while they write its shared memory.
    auto landed = [&]() {
        for (uint32_t y = k - min(k, (uint32_t)S::kStages); y < k; ++y) {
            const uint32_t s = y % S::kStages;
            if (tail_use >> s & 1)
                mbar_wait_bounded(cta.bar(kTail + s), (tail_parity >> s & 1) ^ 1);
            else
                mbar_wait_bounded(cta.bar(kFull + s), y / S::kStages & 1);
        }
    };
    Unit u;
    while (walk.next(u)) {
        // The table is read 32 boxes at a time, a lane each, one group ahead:
        // its latency would otherwise come before every load.
        const int32_t *row = c.table + (int64_t)u.s.slot * c.width;
        auto look_up = [&](int group, int &page, int &token) {
            const int pos = (32 * group + lane) * maps.box, at = pos / c.page_tokens;
            token = pos - at * c.page_tokens;
            page = pos < u.s.end && at < c.width ? row[at] : -1;
        };
        int first = u.j0 * (kTile / maps.box);  // the stage's first box
        int group = first / 32, page, token, next_page, next_token;
        look_up(group, page, token);
        look_up(group + 1, next_page, next_token);
        for (int j = u.j0; j < u.j1; ++j) {
            if (first / 32 != group) {
                group = first / 32;
                page = next_page;
                token = next_token;
                look_up(group + 1, next_page, next_token);
            }
            // A tile's boxes lie in one group: 32 is a multiple of their number.
#pragma unroll 1
            for (int x = 0; x < 2 * S::kParts; ++x) {
                const bool value = x >= S::kParts;
                const int part = value ? x - S::kParts : x;
                const int from = (first + part * boxes + lane) & 31;
                int at_page = __shfl_sync(0xffffffffu, page, from);
                const int at_token = __shfl_sync(0xffffffffu, token, from);
                if (at_page < 0 || at_page >= c.pages)
                    at_page = c.pages;  // past the pool: zeros
                const uint32_t to = cta.smem + S::kRing + stage * S::kStage;
                const bool tail = value && u.tail(j);
                const uint32_t full = cta.bar((tail ? kTail : kFull) + stage);
                bool ok = true;
                if (lane == 0) {
                    ok = cta.wait(kEmpty + stage, empty);
                    if (ok) {
                        mbar_expect_tx(full, S::kStage);
                        if (!tail)  // in the second fixing warp's place
                            mbar_arrive(full);
                    }
                }
                if (!__all_sync(0xffffffffu, ok)) {
                    landed();
                    return;
                }
                if (lane < boxes) {
                    const int a = maps.token_dim == 1 ? at_token : maps.head_dim == 1 ? u.head : at_page;
                    const int b = maps.token_dim == 2 ? at_token : maps.head_dim == 2 ? u.head : at_page;
                    const int d = maps.token_dim == 3 ? at_token : maps.head_dim == 3 ? u.head : at_page;
#pragma unroll
                    for (int h = 0; h < S::DP / 64; ++h)
                        asm volatile(
                            "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::"
                            "complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
                                to + h * S::kHalf + lane * maps.box * 128),
                            "l"(&maps.pool[value]), "r"(64 * h), "r"(a), "r"(b), "r"(d), "r"(full)
                            : "memory");
                }
                __syncwarp();
                tail_use = (tail_use & ~(1u << stage)) | (uint32_t)tail << stage;
                tail_parity ^= (uint32_t)tail << stage;
                ++k;
                if (++stage == S::kStages) {
                    stage = 0;
                    empty ^= 1;
                }
            }
            first += kTile / maps.box;
        }
    }
    landed();
}

// Looks over the values of the tiles that hold drafts.
template <class S>
__device__ void fix_role(const TreePlan &p, const Cta &cta, Walk walk)
{
    constexpr int kChunks = S::DP / 8;
    const int lane = threadIdx.x & 31, tid = threadIdx.x - 32 * (S::kSoftmaxWarps + 1);
    uint32_t k = 0, parity = 0;
    Unit u;
    while (walk.next(u)) {
        for (int j = max(u.s.n / kTile, u.j0); j < u.j1; ++j)
            for (int part = 0; part < S::kParts; ++part) {
                const uint32_t item = k + (2 * (j - u.j0) + 1) * S::kParts + part;
                const uint32_t stage = item % S::kStages, at = cta.smem + S::kRing + stage * S::kStage;
                if (!cta.wait_warp(kTail + stage, parity >> stage & 1))
                    return;
                parity ^= 1u << stage;
                const int base = j * kTile + part * S::kPos;
                for (int x = max(u.s.n - base, 0) * kChunks + tid; x < S::kPos * kChunks;
                     x += 32 * kFixWarps) {
                    const uint32_t to = at + swizzled(S::kHalf, x / kChunks, x % kChunks);
                    if (base + x / kChunks >= u.s.end) {
                        sts16(to, uint4{0, 0, 0, 0});
                    } else {
                        uint4 v = lds16(to);
                        const bool a = clean<S::BF16>(v.x), b = clean<S::BF16>(v.y),
                                   d = clean<S::BF16>(v.z), e = clean<S::BF16>(v.w);
                        if (a || b || d || e) {
                            sts16(to, v);
                            cta.misc->bad[u.number & 7] = u.number + 1;
                        }
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                mbar_arrive_if(cta.bar(kFull + stage), lane == 0);
            }
        k += 2 * S::kParts * u.tiles();
    }
}

// Any other page: each of three warps takes 16 rows of a stage at a time, its
// lanes 16 bytes each, by asynchronous copies, and looks over its own drafts.
// (131072 tokens x 128 rows: 160 us in pages of 20 and 181 of one, 122 by
// tensor maps in pages of 8; those, loaded this way, took 283 before stages were
// handed on while the next one's place is waited for.)
constexpr int kInFlight = 2;  // stages behind the one being requested; with 3: 212 us

template <class S>
__device__ void load_role(const TreePlan &p, const Cta &cta, Walk walk)
{
    constexpr int kChunks = S::DP / 8;         // 16-byte chunks of a row
    constexpr int kLanesRows = 32 / kChunks;   // rows a warp covers in one step
    const KvView &c = p.c;
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - S::kSoftmaxWarps;
    const int chunk = lane % kChunks;
    uint32_t k = 0;     // stages asked for
    uint32_t done = 0;  // stages handed over
    // A stage has 4 or 8 blocks: the warp that takes most of them changes.
    auto first_block = [&](uint32_t x) { return (int)((warp + x) % kLoadWarps); };
    struct Asked {
        int base, drafts, end, unit;  // positions drafts .. end - 1 of a value stage are drafts
    } asked[kInFlight + 1];
    Unit u;
    // The oldest stage in flight has landed: look its drafts over, hand it on.
    auto hand_over = [&]() {
        const Asked &a = asked[0];
        const uint32_t at = cta.smem + S::kRing + done % S::kStages * S::kStage;
        if (a.drafts < a.end && a.drafts < a.base + S::kPos && a.end > a.base) {
            for (int block = first_block(done); block < S::kPos / 16; block += kLoadWarps)
                for (int r = 0; r < 16; r += kLanesRows) {
                    const int row = block * 16 + r + lane / kChunks, pos = a.base + row;
                    if (pos >= a.drafts && pos < a.end) {
                        const uint32_t to = at + swizzled(S::kHalf, row, chunk);
                        uint4 v = lds16(to);
                        const bool x = clean<S::BF16>(v.x), y = clean<S::BF16>(v.y),
                                   z = clean<S::BF16>(v.z), w = clean<S::BF16>(v.w);
                        if (x || y || z || w) {
                            sts16(to, v);
                            cta.misc->bad[a.unit & 7] = a.unit + 1;
                        }
                    }
                }
        }
        fence_proxy_async_smem();
        __syncwarp();
        mbar_arrive_if(cta.bar(kFull + done % S::kStages), lane == 0);
        ++done;
#pragma unroll
        for (int i = 0; i < kInFlight; ++i)
            asked[i] = asked[i + 1];
    };
    // The same of `flying` stages that may still be on their way.
    auto hand_over_oldest = [&](uint32_t flying) {
        if (flying == 1)
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        else if (flying == 2)
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        else
            asm volatile("cp.async.wait_group 2;" ::: "memory");
        hand_over();
    };
    bool ok = true;
    while (ok && walk.next(u)) {
        for (int x = 2 * S::kParts * u.j0; x < 2 * S::kParts * u.j1; ++x, ++k) {
            const int base = x / (2 * S::kParts) * kTile + x % S::kParts * S::kPos;
            const bool value = x / S::kParts & 1;
            const uint32_t stage = k % S::kStages, to = cta.smem + S::kRing + stage * S::kStage;
            // While the stage's last readers are at work, what has landed is handed on.
            const uint32_t parity = (k / S::kStages & 1) ^ 1;
            while (k != done && !__all_sync(0xffffffffu, mbar_test_wait(cta.bar(kEmpty + stage), parity)))
                hand_over_oldest(k - done);
            ok = lane != 0 || cta.wait(kEmpty + stage, parity);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok)
                break;
            const char *pool = c.pool[value] + u.head * c.head_stride;
            for (int block = first_block(k); block < S::kPos / 16; block += kLoadWarps) {
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
                                     to + swizzled(S::kHalf, block * 16 + row, chunk)),
                                 "l"(src), "r"(real ? 16 : 0)
                                 : "memory");
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            const Asked now{base, value ? u.s.n : 0, value ? u.s.end : 0, u.number};
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
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    while (done < k)
        hand_over();
}

// ---------------------------------------------------------------------------
// Matrix products: one thread.  The next scores are written where the weights
// are that the sums issued before them read, with no wait between the two.  What
// this relies on: the tensor core runs the products that one thread issues one
// after another.  The PTX manual promises that order for products of one
// accumulator and shape; these have two.  No weight has been seen overwritten
// (results repeat bit for bit); a wait would cost the products' and the commit's
// latency once a tile.
// ---------------------------------------------------------------------------
template <class S>
__device__ void product_role(const TreePlan &p, const Cta &cta, Walk walk)
{
    constexpr uint32_t kScoreDesc = umma_idesc(S::BF16, S::kPos, false);
    constexpr uint32_t kSumDesc = umma_idesc(S::BF16, S::DP, true);
    const uint32_t tmem = cta.misc->tmem, ring = cta.smem + S::kRing;
    uint32_t stage = 0, landed = 0;      // the next stage and the parity of its phase
    uint32_t weights[2] = {0, 0};        // weight tiles taken per stream
    uint32_t queries[2] = {0, 0};        // query tiles
    Unit u;

    auto scores = [&](int stream, int part, uint32_t at) {
        const uint32_t q = umma_desc_low(cta.smem + stream * S::kQuery, 0);
        const uint32_t key = umma_desc_low(ring + at * S::kStage, 0);
        const uint32_t d = tmem + S::score_col(stream) + part * S::kPos;
#pragma unroll
        for (int kk = 0; kk < S::DP / 16; ++kk)
            umma_ss(d, umma_desc(q, (kk >> 2) * (kRowTile * 128) + (kk & 3) * 32),
                    umma_desc(key, (kk >> 2) * S::kHalf + (kk & 3) * 32), kScoreDesc, kk > 0);
    };
    auto sums = [&](int stream, int part, uint32_t at, bool add) {
        const uint32_t value = umma_desc_low(ring + at * S::kStage, S::kHalf);
        const uint32_t from = tmem + S::score_col(stream) + part * (S::kPos / 2);
        const uint32_t d = tmem + S::sum_col(stream);
#pragma unroll
        for (int kk = 0; kk < S::kPos / 16; ++kk)
            umma_ts(d, from + kk * 8, umma_desc(value, kk * 16 * 128), kSumDesc, kk > 0 || add);
    };
    // Waits for the next stage to land and takes it.
    auto take = [&](uint32_t &at) {
        at = stage;
        if (!cta.poll(kFull + at, landed))
            return false;
        if (++stage == S::kStages) {
            stage = 0;
            landed ^= 1;
        }
        return true;
    };

    while (walk.next(u)) {
        const int streams = u.rows > kRowTile ? 2 : 1;
        for (int j = u.j0; j <= u.j1; ++j) {
            // Sums of tile j - 1 and scores of tile j, stream by stream.
            uint32_t values[S::kParts], keys[S::kParts];
#pragma unroll 1
            for (int s = 0; s < streams; ++s) {
                if (j > u.j0) {
                    // The values have mostly landed by now: asking before the weights
                    // are there costs nothing.  (The same for the next keys holds
                    // up the sums: 32 chats 73 us for 66.)
                    if (s == 0)
#pragma unroll
                        for (int part = 0; part < S::kParts; ++part)
                            if (!take(values[part]))
                                return;
                    if (!cta.poll(kWeights + s, weights[s]++ & 1))
                        return;
                    tc_fence_after();
#pragma unroll
                    for (int part = 0; part < S::kParts; ++part) {
                        sums(s, part, values[part], j > u.j0 + 1 || part > 0);
                        if (S::STREAMS == 1)
                            umma_commit(cta.bar(kEmpty + values[part]));
                    }
                } else if (!cta.poll(kQuery + s, queries[s]++ & 1)) {
                    return;
                }
                if (j == u.j1) {
                    umma_commit(cta.bar(kSums + s));
                    continue;
                }
#pragma unroll
                for (int part = 0; part < S::kParts; ++part) {
                    if (s == 0 && !take(keys[part]))
                        return;
                    tc_fence_after();
                    scores(s, part, keys[part]);
                    if (S::STREAMS == 1)
                        umma_commit(cta.bar(kEmpty + keys[part]));
                }
                umma_commit(cta.bar(kScores + s));
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Softmax: a thread is a row of its stream's row tile.
// ---------------------------------------------------------------------------
// Weights of f16 are 2^7 times exp(s - m).  The running maximum may lag by 2^8, so
// they stay at or below 2^15, inside the type; what a long context's many small
// ones add up to is kept: 16 bits hold weights down to 2^-21 of the largest in
// full and others to within 2^-32 of it (2^-14 and 2^-25 without: 131072
// positions, 17 below one in the exponent, moved the output by 2e-3 of their value).  Sums
// and outputs grow alike, which leaves the quotient; the logarithm takes the
// sums back.
template <bool BF16>
constexpr float kLift = BF16 ? 0.0f : 7.0f;
template <bool BF16>
constexpr float kUnlift = BF16 ? 1.0f : 0.0078125f;

// Partial sums of a cut unit: [slot][row] maxima (of scores times scale *
// log2 e), sums and, unnormalised, outputs.  Run c writes the unit it begins
// inside of to slot 2 c and one that goes on after it to slot 2 c + 1.
__host__ __device__ constexpr uint64_t part_floats(int unit_rows, int dp)
{
    return (uint64_t)unit_rows * (dp + 2);
}

template <class S>
__device__ __forceinline__ float *part_of(const TreePlan &p, int slot)
{
    return static_cast<float *>(p.workspace) + slot * part_floats(S::kUnitRows, S::DP);
}

// Where run c begins inside a unit and no earlier run does: what is to be
// joined.  Entry c of an array after the parts; rows = 0: nothing.
struct Cut {
    int row0, head, r0, rows, parts, unused[3];
};

template <class S>
__device__ __forceinline__ Cut *cuts_of(const TreePlan &p, int ctas)
{
    return reinterpret_cast<Cut *>(part_of<S>(p, 2 * ctas));
}

template <class S>
__device__ void note_cut(const TreePlan &p, const Place &place, Walk walk)
{
    Cut cut{};
    Unit u;
    if ((int)blockIdx.x < place.ctas && walk.next(u) && u.j0 > 0) {
        const int begin = place.at - u.j0, end = begin + u.s.tiles;  // of its tiles
        if (place.start((int)blockIdx.x - 1) <= begin) {
            int last = (int)min((int64_t)end * place.ctas / place.total, (int64_t)place.ctas - 1);
            while (place.start(last) >= end)
                --last;
            while (last + 1 < place.ctas && place.start(last + 1) < end)
                ++last;
            cut = Cut{u.s.row0, u.head, u.r0, u.rows, last - (int)blockIdx.x + 2, {}};
        }
    }
    cuts_of<S>(p, gridDim.x)[blockIdx.x] = cut;
}

// A row of the mask.  The first 64 drafts' bits are read when the unit begins;
// by the time they are needed they are there.
struct MaskRow {
    const uint32_t *words;
    int count, T;
    uint32_t first, second;
    __device__ MaskRow(const TreePlan &p, const Seq &s, int64_t row)
        : words(p.mask + row * p.mask_words), count(p.mask_words), T(s.end > 0 ? s.T : 0)
    {
        first = count > 0 ? words[0] : 0;
        second = count > 1 ? words[1] : 0;
    }
    __device__ uint32_t word(int w) const
    {
        return w == 0 ? first : w == 1 ? second : w < count ? words[w] : 0;
    }
    // Bits for 32 positions from draft d (negative: committed positions, seen)
    // on; drafts from T on are not seen.
    __device__ uint32_t seen(int d) const
    {
        if (d <= -32)
            return 0xffffffffu;
        if (d >= T)
            return 0;
        const int w = d >> 5;  // -1 for the word before the first: all seen
        uint32_t v = __funnelshift_r(w < 0 ? 0xffffffffu : word(w), word(w + 1), d & 31);
        return T - d < 32 ? v & ((1u << (T - d)) - 1) : v;
    }
};

// The sums of a row of the unit, from its columns of tensor memory to the output
// or, if the unit goes on in another run, to the workspace.  Whole warps call it.
template <class S>
__device__ __forceinline__ void write_unit(const TreePlan &p, const Cta &cta, const Unit &u, int run,
                                           int mine, uint32_t sum_cols, float top, float sum, float c)
{
    if (mine - (int)(threadIdx.x & 31) >= u.rows)
        return;
    const bool whole = u.whole(), real = mine < u.rows;
    const bool bad = *(volatile int *)&cta.misc->bad[u.number & 7] == u.number + 1;
    const int r = min(u.r0 + mine, u.s.T * p.group - 1), draft = r / p.group;
    const int64_t q_row = u.s.row0 + draft;
    const int q_head = u.head * p.group + r - draft * p.group;
    char *out = p.out + q_row * p.o_row + (int64_t)q_head * p.o_head;
    float *part = part_of<S>(p, 2 * run + (u.j0 == 0 ? 1 : 0));
    const float inv = !whole ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
    if (real) {
        if (!whole) {
            part[mine] = top == -INFINITY ? top : top * c;
            part[S::kUnitRows + mine] = sum;
        } else if (p.lse) {
            p.lse[q_row * p.q_heads + q_head] =
                top == -INFINITY && sum == 0.0f ? -INFINITY : top * fabsf(p.scale) + logf(sum * kUnlift<S::BF16>);
        }
    }
#pragma unroll 1
    for (int g = 0; g < S::DP / 32; ++g) {
        uint32_t o[32];
        __syncwarp();  // rows part ways below; tensor memory is read by whole warps
        tmem_load32(o, sum_cols + 32 * g);
        tmem_wait_load(o);
        if (!real)
            continue;
        if (bad) {
            // Drafted values that are not finite, for the rows that see them.
            const MaskRow mask(p, u.s, q_row);
            const int from = max(u.j0 * kTile - u.s.n, 0), to = min(u.j1 * kTile - u.s.n, u.s.T);
            for (int d = from; d < to; ++d) {
                const int pos = u.s.n + d;
                if (!(mask.seen(d) & 1u) || pos / p.c.page_tokens >= p.c.width)
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
                        const uint32_t big = S::BF16 ? 0x7f80u : 0x7c00u, frac = S::BF16 ? 0x7fu : 0x3ffu;
                        if ((e & big) == big)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) +
                                                   (e & frac ? NAN : e >> 15 ? -INFINITY : INFINITY));
                    }
            }
        }
        if (whole) {
#pragma unroll
            for (int w = 0; w < 4; ++w)
                if (32 * g + 8 * w < p.head_dim) {
                    uint32_t v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        v[i] = pack16<S::BF16>(__uint_as_float(o[8 * w + 2 * i]) * inv,
                                               __uint_as_float(o[8 * w + 2 * i + 1]) * inv);
                    *reinterpret_cast<uint4 *>(out + (32 * g + 8 * w) * 2) = uint4{v[0], v[1], v[2], v[3]};
                }
        } else {
            uint4 *to = reinterpret_cast<uint4 *>(part + 2 * S::kUnitRows + mine * S::DP + 32 * g);
#pragma unroll
            for (int w = 0; w < 8; ++w)
                to[w] = uint4{o[4 * w], o[4 * w + 1], o[4 * w + 2], o[4 * w + 3]};
        }
    }
}

template <class S>
__device__ void softmax_role(const TreePlan &p, const Cta &cta, Walk walk, int run)
{
    constexpr int kChunks = S::DP / 8;
    const int stream = threadIdx.x >> 7, tid = threadIdx.x & 127;
    const int lane = threadIdx.x & 31, warp = tid >> 5;
    const uint32_t lanes = cta.misc->tmem + ((uint32_t)(warp * 32) << 16);
    const uint32_t score_cols = lanes + S::score_col(stream), sum_cols = lanes + S::sum_col(stream);
    const uint32_t query = cta.smem + stream * S::kQuery;
    // A scale of 0 makes all weights equal: any c that leaves scores * c at 0
    // does, and unlike 0 it leaves a hidden -inf alone.
    const float scale = fabsf(p.scale), c = scale > 0.0f ? scale * 1.44269504088896340736f : 1e-38f;
    const uint32_t flip = p.scale < 0.0f ? 0x80008000u : 0u;
    // The running maximum moves only when a row's grows by 8 powers of two:
    // weights stay below 2^8, exact in the 32-bit sums, and most tiles need no
    // pass over the output sums.
    const float slack = 8.0f / c;
    uint32_t tiles_seen = 0, sums_seen = 0;

    Unit before, u;
    bool begun = false;
    float top = 0.0f, sum = 0.0f;
    // Two CTAs on an SM have short rings: the issuing thread commits to the
    // barrier of each stage.  With two streams the ring is longer, and the first
    // thread of the unit's last stream hands the stages back when it hears of
    // the products' end, which spares the issuing thread 100 cycles a commit.
    uint32_t stage = 0;
    auto hand_back = [&](const Unit &of) {
        if (S::STREAMS == 1)
            return;
        mbar_arrive_if(cta.bar(kEmpty + stage),
                       stream * kRowTile + kRowTile >= of.rows && (threadIdx.x & 127) == 0);
        stage = stage + 1 == S::kStages ? 0 : stage + 1;
    };
    for (;;) {
        bool more;  // a further unit has rows for this stream
        uint32_t others = 0;  // stages that units without rows for this stream use before that
        while ((more = walk.next(u)) && u.rows <= stream * kRowTile)
            others += 2 * u.tiles();
        // The query rows of the stream's tile are on their way while the last
        // unit's last product runs, and its first scores while the last sums
        // are read: those are not written again before this stream's next
        // weights.  Rows past the unit's read as zeros.
        uint4 q[kChunks];
        if (more) {
            const int step = 128 / kChunks, d_step = step / p.group, h_step = step - d_step * p.group;
            const int row = stream * kRowTile + tid / kChunks;
            int draft = (u.r0 + row) / p.group, h = u.r0 + row - draft * p.group;
            const char *from = p.q + (int64_t)u.head * p.group * p.q_head + tid % kChunks * 16;
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                q[i] = uint4{0, 0, 0, 0};
                if (row + i * step < u.rows && tid % kChunks * 16 < p.c.row_bytes)
                    q[i] = *reinterpret_cast<const uint4 *>(
                        from + (int64_t)(u.s.row0 + draft) * p.q_row + (int64_t)h * p.q_head);
                draft += d_step;
                h += h_step;
                if (h >= p.group) {
                    h -= p.group;
                    ++draft;
                }
            }
        }
        if (begun) {
            if (!cta.wait_warp(kSums + stream, sums_seen++ & 1))
                return;
            tc_fence_after();
            hand_back(before);  // the last values
        }
        stage = (stage + others) % S::kStages;
        if (more) {
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                q[i].x ^= flip, q[i].y ^= flip, q[i].z ^= flip, q[i].w ^= flip;
                sts16(query + swizzled(kRowTile * 128, i * (128 / kChunks) + tid / kChunks, tid % kChunks),
                      q[i]);
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            mbar_arrive_if(cta.bar(kQuery + stream), lane == 0);
        }
        if (begun)
            write_unit<S>(p, cta, before, run, stream * kRowTile + tid, sum_cols, top, sum, c);
        if (!more)
            return;

        const int mine = stream * kRowTile + tid;         // row of the unit
        const bool active = mine - lane < u.rows;         // any row of the warp
        const MaskRow mask(p, u.s, u.s.row0 + min(u.r0 + mine, u.s.T * p.group - 1) / p.group);
        top = -INFINITY;
        sum = 0.0f;
        for (int j = u.j0; j < u.j1; ++j) {
            if (!cta.wait_warp(kScores + stream, tiles_seen++ & 1))
                return;
            tc_fence_after();
            if (j > u.j0)
                hand_back(u);  // the values of the tile before
            hand_back(u);      // this tile's keys
            if (active) {
                // Scores are read twice, 32 columns at a time: for the maximum,
                // and for the weights, which take the place of scores already
                // read.  (A read takes 20 cycles; holding all 128 in registers
                // or unrolling this leaves too few of them for two CTAs, and
                // code too long for the instruction cache.)
                uint32_t s[32];
                if (u.tail(j))  // what is hidden becomes -inf in its place
#pragma unroll 1
                    for (int g = 0; g < 4; ++g) {
                        const uint32_t seen = mask.seen(j * kTile + 32 * g - u.s.n);
                        if (__all_sync(0xffffffffu, seen == 0xffffffffu))
                            continue;
                        tmem_load32(s, score_cols + 32 * g);
                        tmem_wait_load(s);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            s[i] = seen >> i & 1 ? s[i] : 0xff800000u;
                        tmem_store32(score_cols + 32 * g, s);
                        tmem_wait_store();
                    }
                float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                for (int g = 0; g < 4; ++g) {
                    tmem_load32(s, score_cols + 32 * g);
                    tmem_wait_load(s);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        m[i & 3] = fmaxf(m[i & 3], __uint_as_float(s[i]));
                }
                const float here = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
                const bool moves = here > (top == -INFINITY ? top : top + slack);
                float old = 1.0f;
                if (moves) {
                    old = top == -INFINITY ? 0.0f : exp2_fast((top - here) * c);
                    top = here;
                    sum *= old;
                }
                const bool any = __any_sync(0xffffffffu, moves);  // brings the lanes together too
                if (j != u.j0 && any) {
#pragma unroll 1
                    for (int g = 0; g < S::DP / 16; ++g) {
                        uint32_t o[16];
                        tmem_load16(o, sum_cols + 16 * g);
                        tmem_wait_load(o);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * old);
                        tmem_store16(sum_cols + 16 * g, o);
                    }
                }
                const float shift = top == -INFINITY ? 0.0f : fmaf(top, c, -kLift<S::BF16>);
                float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                // Weights in 16 bits for the second product, as its operand
                // type asks: a relative error of at most half an ulp each, for
                // f16 down to 2^-21 of the largest; the sum is of the unrounded
                // ones.
#pragma unroll 1
                for (int g = 0; g < 4; ++g) {
                    uint32_t w[16];
                    tmem_load32(s, score_cols + 32 * g);
                    tmem_wait_load(s);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float a = exp2_fast(fmaf(__uint_as_float(s[2 * i]), c, -shift));
                        const float b = exp2_fast(fmaf(__uint_as_float(s[2 * i + 1]), c, -shift));
                        part[2 * i & 3] += a;
                        part[(2 * i + 1) & 3] += b;
                        w[i] = pack16<S::BF16>(a, b);
                    }
                    tmem_store16(score_cols + 16 * g, w);
                }
                sum += (part[0] + part[1]) + (part[2] + part[3]);
                tmem_wait_store();
            }
            tc_fence_before();
            __syncwarp();
            mbar_arrive_if(cta.bar(kWeights + stream), lane == 0);
        }
        before = u;
        begun = true;
    }
}

template <class S, bool BOXES>
__global__ void __launch_bounds__(S::kThreads, 3 - S::STREAMS)
    k_tree(const __grid_constant__ TreePlan p, const __grid_constant__ Maps maps)
{
    extern __shared__ __align__(1024) unsigned char raw[];
    const uint32_t at = smem_u32(raw), pad = (1024 - (at & 1023)) & 1023;
    Cta cta;
    cta.smem = at + pad;
    cta.bars = cta.smem + S::kBars;
    cta.misc = reinterpret_cast<Misc *>(raw + pad + S::kMisc);
    cta.status = p.status;
    cta.limit = p.wait_ns;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init_count(cta.bar(kFull + i), BOXES ? kFixWarps : kLoadWarps);
            mbar_init_count(cta.bar(kEmpty + i), 1);
            mbar_init_count(cta.bar(kTail + i), 1);
        }
        for (int s = 0; s < S::STREAMS; ++s) {
            mbar_init_count(cta.bar(kQuery + s), 4);
            mbar_init_count(cta.bar(kScores + s), 1);
            mbar_init_count(cta.bar(kWeights + s), 4);
            mbar_init_count(cta.bar(kSums + s), 1);
        }
        mbar_init_count(cta.bar(kLast), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        cta.misc->abort = 0;
        for (int i = 0; i < 8; ++i)
            cta.misc->bad[i] = 0;
    }
    if (warp == S::kSoftmaxWarps)
        tmem_alloc<S::kCols>(smem_u32(&cta.misc->tmem));
    pdl_wait_prerequisite();
    pdl_launch_dependents();
    // Ascending sequences have no more rows than there are, which is what keeps
    // the work in 32 bits; others are not dealt out at all.  A warp of its own
    // looks: in the loop of find_run it made the kernel's code 4% slower.
    if (warp == S::kSoftmaxWarps + 1) {
        int falls = 0;
#pragma unroll 4
        for (int b = lane; b < p.seqs; b += 32)
            falls |= p.q_start[b] > p.q_start[b + 1];
        falls = __any_sync(0xffffffffu, falls);
        if (lane == 0)
            cta.misc->found.falls = falls;
    }
    Place place = find_run<S::kThreads>(p, S::kUnitRows, gridDim.x, blockIdx.x, cta.misc->found);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (cta.misc->found.falls)
        place.ctas = 0;
    const bool runs = (int)blockIdx.x < place.ctas;
    const Walk walk(p, S::kUnitRows, place, runs ? place.start(blockIdx.x + 1) - place.at : 0);
    if (threadIdx.x == 32 * (S::kSoftmaxWarps + 2))
        note_cut<S>(p, place, walk);
    __syncwarp();  // the register instructions below are for whole warps
    if (runs) {
        // Registers a thread: launched with 168 (two streams) or 128; what the
        // last four warps give up is what the softmax warps take.
        //   128 * 72 + 256 * 216 = 384 * 168,   128 * 72 + 128 * 184 = 256 * 128
        if (warp < S::kSoftmaxWarps) {
            if (S::STREAMS == 2)
                asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
            else
                asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
            softmax_role<S>(p, cta, walk, blockIdx.x);
        } else {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
            if (warp == S::kSoftmaxWarps + 3) {
                if (lane == 0)
                    product_role<S>(p, cta, walk);
            } else if (!BOXES) {
                load_role<S>(p, cta, walk);
            } else if (warp == S::kSoftmaxWarps) {
                box_role<S>(p, maps, cta, walk);
            } else {
                fix_role<S>(p, cta, walk);
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    // After an expired wait products may still run: let them end (bounded).  Every
    // role has ended by now, so that none sets the word later.
    if (cta.misc->abort) {
        if (threadIdx.x == 32 * (S::kSoftmaxWarps + 3)) {
            umma_commit(cta.bar(kLast));
            mbar_wait_bounded(cta.bar(kLast), 0);
        }
        __syncwarp();
        tc_fence_before();
        __syncthreads();
    }
    if (warp == S::kSoftmaxWarps) {
        tc_fence_after();
        tmem_free<S::kCols>(cta.misc->tmem);
    }
}

// ---------------------------------------------------------------------------
// Joins the parts of the units that run ends cut, o and l by the powers of two of
// their maxima's distance to the largest: CTA (x, y) takes the y-th rows of the
// unit whose first cut is run x + 1's start.  DP / 4 lanes read a row, 16 bytes
// each, ROWS rows and SIDE parts of them at a time, all of whose loads are under
// way before the first is used.  Bound by those loads' latency, from L2: of the 63
// us of 32 chats it takes 6 (up to 40 MB of parts).
// ---------------------------------------------------------------------------
template <class S, int ROWS>
constexpr int kJoinRows = kJoinThreads / (S::DP / 4) * ROWS;  // rows of a CTA

template <class S, int ROWS, int SIDE>
__global__ void __launch_bounds__(kJoinThreads) k_tree_join(const TreePlan p, int ctas)
{
    pdl_launch_dependents();
    pdl_wait_prerequisite();
    const Cut u = cuts_of<S>(p, ctas)[blockIdx.x + 1];
    if ((int)blockIdx.y * kJoinRows<S, ROWS> >= u.rows)
        return;
    constexpr int kLanes = S::DP / 4;
    const int lane = threadIdx.x % kLanes, parts = u.parts;
    const int row0 = blockIdx.y * kJoinRows<S, ROWS> + threadIdx.x / kLanes * ROWS;
    const float *first = part_of<S>(p, 2 * blockIdx.x + 1);  // the unit begins in this run
    const int64_t pitch = 2 * part_floats(S::kUnitRows, S::DP);
    float top[ROWS], sum[ROWS];
    float4 x[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        top[r] = -INFINITY;
        sum[r] = 0.0f;
        x[r] = float4{0.0f, 0.0f, 0.0f, 0.0f};
    }
#pragma unroll 1
    for (int i0 = 0; i0 < parts; i0 += SIDE) {
        float t[ROWS][SIDE], l[ROWS][SIDE];
        float4 v[ROWS][SIDE];
#pragma unroll
        for (int i = 0; i < SIDE; ++i) {
            // Later parts lie in the slots of units begun before their run.
            const float *from = first + (i0 + i) * pitch -
                                (i0 + i > 0 ? part_floats(S::kUnitRows, S::DP) : 0);
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                const int row = row0 + r;
                const bool is = i0 + i < parts && row < u.rows;
                t[r][i] = is ? from[row] : -INFINITY;
                l[r][i] = is ? from[S::kUnitRows + row] : 0.0f;
                v[r][i] = is ? *reinterpret_cast<const float4 *>(from + 2 * S::kUnitRows + row * S::DP + lane * 4)
                             : float4{0.0f, 0.0f, 0.0f, 0.0f};
            }
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            float most = top[r];
#pragma unroll
            for (int i = 0; i < SIDE; ++i)
                most = fmaxf(most, t[r][i]);
            const float old = top[r] == most ? 1.0f : exp2_fast(top[r] - most);
            top[r] = most;
            sum[r] *= old;
            x[r].x *= old, x[r].y *= old, x[r].z *= old, x[r].w *= old;
#pragma unroll
            for (int i = 0; i < SIDE; ++i)
                if (i0 + i < parts) {
                    const float f = t[r][i] == most ? 1.0f : exp2_fast(t[r][i] - most);
                    sum[r] = fmaf(l[r][i], f, sum[r]);
                    x[r].x = fmaf(v[r][i].x, f, x[r].x);
                    x[r].y = fmaf(v[r][i].y, f, x[r].y);
                    x[r].z = fmaf(v[r][i].z, f, x[r].z);
                    x[r].w = fmaf(v[r][i].w, f, x[r].w);
                }
        }
    }
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
        if (row0 + k >= u.rows)
            break;
        const int r = u.r0 + row0 + k, draft = r / p.group, q_head = u.head * p.group + r - draft * p.group;
        const int64_t q_row = u.row0 + draft;
        const float inv = sum[k] == 0.0f ? 0.0f : 1.0f / sum[k];
        if (lane * 4 < p.head_dim)
            *reinterpret_cast<uint2 *>(p.out + q_row * p.o_row + (int64_t)q_head * p.o_head + lane * 8) =
                uint2{pack16<S::BF16>(x[k].x * inv, x[k].y * inv), pack16<S::BF16>(x[k].z * inv, x[k].w * inv)};
        if (p.lse && lane == 0)
            p.lse[q_row * p.q_heads + q_head] = top[k] == -INFINITY && sum[k] == 0.0f
                                                    ? -INFINITY
                                                    : top[k] * 0.69314718055994530942f + logf(sum[k] * kUnlift<S::BF16>);
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

// Tensor maps of the two pools, boxes of at most `positions`; false where the pages' shape does not allow
// them (the kernel then loads by threads).
bool make_maps(const TreePlan &p, int positions, Maps *m)
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
    while (m->box < positions && c.page_tokens % (2 * m->box) == 0)
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

template <class S, bool BOXES>
cudaError_t launch_loads(const TreePlan &p, const Maps &maps, int ctas, bool pdl, cudaStream_t stream)
{
    constexpr size_t smem = S::kBytes + 1024;
    // (The occupancy query counts one CTA of any kernel that allocates tensor
    // memory; two of 256 columns each do share an SM, as timed.)
    if (resident_ctas((const void *)k_tree<S, BOXES>, S::kThreads, smem) < 1)
        return cudaErrorInvalidConfiguration;
    return launch(k_tree<S, BOXES>, dim3(ctas), S::kThreads, smem, pdl, stream, p, maps);
}

template <class S, int ROWS, int SIDE>
cudaError_t launch_join(const TreePlan &p, int rows, int ctas, bool pdl, cudaStream_t stream)
{
    constexpr int each = kJoinRows<S, ROWS>;
    return launch(k_tree_join<S, ROWS, SIDE>, dim3(ctas - 1, (rows + each - 1) / each), kJoinThreads, 0, pdl,
                  stream, p, ctas);
}

template <class S>
cudaError_t launch_shape(const TreePlan &p, int num_sms, bool pdl, cudaStream_t stream)
{
    alignas(64) Maps maps;
    const int ctas = num_sms * (3 - S::STREAMS);
    const cudaError_t e = make_maps(p, S::kPos, &maps)
                              ? launch_loads<S, true>(p, maps, ctas, pdl, stream)
                              : launch_loads<S, false>(p, maps, ctas, pdl, stream);
    if (e != cudaSuccess || ctas < 2)
        return e;
    const int rows = p.rows < S::kUnitRows / p.group ? p.rows * p.group : S::kUnitRows;
    // Rows and parts at a time.  Few units have many parts and few rows in all:
    // 1 and 8 (131072 positions, 128 rows 106 us; 1 and 16 107, 2 and 8 108; one
    // chat 11.4, 12.0, 11.7).  Many units have two or three: 2 and 2, more rows in
    // flight (32 chats 62.9 us; 1 and 8 66.3, 2 and 4 63.7, 4 and 4 69.0; 16
    // sequences of 8192, 256 rows 142, 149, 143, 152).
    const bool many = (int64_t)p.seqs * p.c.heads * 16 <= ctas;  // parts a unit
    return many ? launch_join<S, 1, 8>(p, rows, ctas, pdl, stream) : launch_join<S, 2, 2>(p, rows, ctas, pdl, stream);
}

template <int DP, bool BF16>
cudaError_t launch_dim(const TreePlan &p, int num_sms, bool pdl, cudaStream_t stream)
{
    // By the mean rows of a sequence and cache head.  8 sequences of 8192, one
    // stream and two: 64 rows 62 and 73 us, 128 71 and 76, 136 107 and 80, 192
    // 110 and 83, 256 115 and 91, 384 159 and 143, 1024 338 and 272; 64 sequences
    // of up to 1000, 8 to 512 rows 113 and 104.
    if ((int64_t)p.rows * p.group > (int64_t)kRowTile * p.seqs)
        return launch_shape<Shape<DP, BF16, 2>>(p, num_sms, pdl, stream);
    return launch_shape<Shape<DP, BF16, 1>>(p, num_sms, pdl, stream);
}

}  // namespace

uint64_t tree_workspace_bytes(int num_sms, int head_dim)
{
    // Two slots a run, and a cut; two streams have half the runs and twice the rows.
    return 4 * (uint64_t)num_sms * part_floats(kRowTile, head_dim <= 64 ? 64 : 128) * sizeof(float) +
           2 * num_sms * sizeof(Cut);
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
