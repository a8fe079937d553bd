"""Tree attention against its definition in 64 bits.

Bounds, from the number formats (u = 2^-8 for bf16, 2^-11 for f16, the unit
roundoff): the weights are rounded once to the cache's type before they meet
the values (u * sum p|v|), the result once more (u * |out|); a logit's 32-bit
sum is off by at most (dim + 8) 2^-24 sum|q||k| scale, which enters a weight as
a relative error; weights below 2^-25 of the largest may be lost in f16."""
import numpy as np
import pytest

import cache_model

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from copy_reduce_dst_gb300 import _build  # noqa: E402

_build.build()
from copy_reduce_dst_gb300 import tb  # noqa: E402

TYPES = {"bf16": (torch.bfloat16, 2.0**-8), "f16": (torch.float16, 2.0**-11)}


@pytest.fixture(scope="module")
def ctx():
    with tb.Context(0) as c:
        yield c


class Case:
    """Random pools, rows and trees for sequences of lens[b] committed and drafts[b] drafted tokens."""

    def __init__(self, ctx, lens, drafts, q_heads=4, heads=2, dim=64, P=16, dtype="bf16", layout="NHD",
                 layers=1, layer=0, seed=0, words=None, width=None, slots=None, spread=1.0, check_rows=None):
        g = torch.Generator().manual_seed(seed)
        self.ctx, self.lens, self.drafts, self.layout, self.dtype = ctx, lens, drafts, layout, dtype
        self.layer, self.P, self.slot_of, self.check_rows = layer, P, slots, check_rows
        seqs, t = len(lens), TYPES[dtype][0]
        need = [-(-(n + d) // P) for n, d in zip(lens, drafts)]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g).to(torch.int32)
        n_slots = seqs if slots is None else max(slots) + 1
        table = torch.full((n_slots, width or max(need + [1])), -1, dtype=torch.int32)
        self.all_lens = torch.zeros(n_slots, dtype=torch.int32)
        held, at = torch.zeros(n_slots, dtype=torch.int32), 0
        for b in range(seqs):
            s = b if slots is None else slots[b]
            table[s, :need[b]] = order[at:at + need[b]]
            held[s], self.all_lens[s] = need[b], lens[b]
            at += need[b]
        shape = (layers, pages, P, heads, dim)
        self.pools = [torch.randn(shape, generator=g).mul_(spread).to(t) for _ in "kv"]
        rows = sum(drafts)
        self.q = torch.randn(rows, q_heads, dim, generator=g).to(t)
        self.q_start = np.concatenate([[0], np.cumsum(drafts)]).astype(np.int32)
        self.words = words if words is not None else -(-max(drafts + [1]) // 32)
        mask = np.zeros((rows, self.words), np.int64)
        rng = np.random.default_rng(seed)
        for b, d in enumerate(drafts):
            parents = [-1] + [int(rng.integers(-1, i)) for i in range(1, d)]
            for i, row in enumerate(tb.tree_mask(parents[:d])):
                row = row[:self.words]
                mask[self.q_start[b] + i, :len(row)] = row
        self.mask = mask.astype(np.int32)
        self.rows = None if check_rows is None else sorted(rng.choice(rows, check_rows, replace=False).tolist())
        self.table, self.held = table, held
        self.scale = dim ** -0.5

    def run(self, lse=True, stream=None):
        pools = [p.cuda() if self.layout == "NHD" else p.transpose(2, 3).contiguous().cuda() for p in self.pools]
        c = tb.kv_cache(*pools, self.table.cuda(), self.held.cuda(), self.all_lens.cuda(),
                        torch.ones(pools[0].shape[1], dtype=torch.int32, device="cuda"), layout=self.layout)
        q = self.q.cuda()
        out = torch.full_like(q, float("nan"))
        got = torch.full(q.shape[:2], float("nan"), device="cuda") if lse else None
        work = torch.empty(self.ctx.tree_attention_workspace(c, q.shape[1]), dtype=torch.uint8, device="cuda")
        work.fill_(255)
        slots = None if self.slot_of is None else torch.tensor(self.slot_of, dtype=torch.int32, device="cuda")
        self.args = (c, self.layer, q, torch.from_numpy(self.q_start).cuda(), torch.from_numpy(self.mask).cuda(), out,
                     work)
        self.kw = dict(scale=self.scale, lse=got, seq_slots=slots)
        torch.cuda.synchronize()
        self.ctx.tree_attention(*self.args, **self.kw, stream=stream)
        torch.cuda.synchronize()
        return out, got

    def want(self):
        k, v = (p[self.layer].float().numpy() for p in self.pools)
        return cache_model.tree_attention(self.q.float().numpy(), k, v, self.table.numpy(), self.all_lens.numpy(),
                                          self.q_start, self.mask.astype(np.int64) & 0xFFFFFFFF, self.scale,
                                          self.slot_of, self.rows)

    def check(self, **kw):
        out, lse = self.run(**kw)
        self.compare(out, lse)
        return out, lse

    def compare(self, out, lse):
        want, want_lse, reach, logit = self.want()
        u, dim = TYPES[self.dtype][1], self.q.shape[2]
        slack = (dim + 8) * 2.0**-24 * logit + 2.0**-20
        longest = max(n + d for n, d in zip(self.lens, self.drafts))
        biggest = float(self.pools[1].float().nan_to_num(0, 0, 0).abs().max())
        lost = longest * 2.0**-25 * biggest if self.dtype == "f16" else 0.0
        bound = u * np.abs(want) * 1.01 + (u * 1.01 + 2 * slack)[..., None] * reach * (1 + u) + lost + 1e-7
        off = np.abs(out.float().cpu().numpy().astype(np.float64) - want)
        if self.rows is not None:  # the model did these
            off, bound = off[self.rows], bound[self.rows]
            want_lse, slack = want_lse[self.rows], slack[self.rows]
            lse = None if lse is None else lse[self.rows]
        assert np.all(off <= bound), float((off / bound).max())
        if lse is not None:
            got = lse.cpu().numpy().astype(np.float64)
            np.testing.assert_array_equal(np.isneginf(got), np.isneginf(want_lse))
            real = ~np.isneginf(want_lse)
            assert np.all(np.abs(got - want_lse)[real] <= (slack + 2.0**-20 * (1 + np.abs(want_lse)))[real])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("dim", [8, 64, 80, 128])
@pytest.mark.parametrize("P", [1, 5, 16, 24, 64])
def test_types_layouts_dims_pages(ctx, dtype, layout, dim, P):
    Case(ctx, [150, 37], [9, 3], dim=dim, P=P, dtype=dtype, layout=layout, seed=dim + P).check()


@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 111, 112, 113, 120, 127, 128, 129, 255, 256, 257, 384, 1000])
@pytest.mark.parametrize("t", [1, 8, 33])
def test_lengths_about_tiles(ctx, n, t):
    Case(ctx, [n], [t], seed=n + t).check()


@pytest.mark.parametrize("q_heads,heads", [(1, 1), (6, 6), (7, 1), (10, 2), (64, 4), (40, 8), (129, 1), (300, 2)])
@pytest.mark.parametrize("t", [1, 5, 16])
def test_groups(ctx, q_heads, heads, t):
    Case(ctx, [70, 200], [t, t], q_heads=q_heads, heads=heads, dim=128, seed=q_heads).check()


@pytest.mark.parametrize("t", [31, 32, 64, 65, 130, 300])
def test_large_trees(ctx, t):
    """More rows than a tile, mask words past the first, drafts over several tiles."""
    Case(ctx, [90, 3], [t, 7], q_heads=6, heads=2, seed=t).check()


@pytest.mark.parametrize("drafts", [[48, 48, 48], [48, 3, 40, 16, 17], [33, 1, 1, 32]])
@pytest.mark.parametrize("P", [16, 5])
def test_units_of_one_and_two_row_tiles(ctx, drafts, P):
    """Sequences of 8 to 384 rows per cache head, several tiles long, one after another in a run."""
    lens = [900 + 130 * b for b in range(len(drafts))]
    Case(ctx, lens, drafts, q_heads=8, heads=1, P=P, seed=sum(drafts)).check()
    Case(ctx, lens * 12, drafts * 12, q_heads=16, heads=2, dim=128, P=P, seed=P, check_rows=40).check()


def test_ragged_batch_with_empty_sequences(ctx):
    lens = [0, 5, 0, 700, 128, 1, 33, 64]
    drafts = [0, 4, 3, 12, 0, 1, 0, 9]
    Case(ctx, lens, drafts, seed=1).check()


def test_many_short_sequences(ctx):
    g = np.random.default_rng(2)
    lens, drafts = g.integers(0, 90, 400).tolist(), g.integers(0, 4, 400).tolist()
    Case(ctx, lens, drafts, q_heads=2, heads=1, seed=2).check()


def test_one_long_sequence_split_over_the_gpu(ctx):
    Case(ctx, [40001], [3], q_heads=2, heads=1, P=64, seed=3).check()
    Case(ctx, [20000, 17, 9000], [2, 5, 1], q_heads=4, heads=2, dtype="f16", seed=4).check()


def test_slots_layers_and_wide_tables(ctx):
    Case(ctx, [50, 20, 90], [4, 2, 6], slots=[4, 0, 2], layers=3, layer=2, width=40, seed=5).check()


def test_keys_and_values_side_by_side(ctx):
    """Pools that are views of one tensor, pages outermost, a gap after each token's heads."""
    c = Case(ctx, [70, 130], [5, 9], q_heads=6, heads=3, layers=2, layer=1, seed=20)
    want, want_lse = c.run()
    cache, layer, q, q_start, mask, out, work = c.args
    k = c.pools[0]
    whole = torch.full((k.shape[1], 2, k.shape[0], k.shape[2], k.shape[3] + 1, k.shape[4]), float("nan"),
                       dtype=k.dtype, device="cuda")
    views = []
    for i in range(2):
        view = whole[:, i, :, :, :-1].permute(1, 0, 2, 3, 4)
        view.copy_(c.pools[i])
        views.append(view)
    apart = tb.kv_cache(*views, *cache.tensors[2:])
    again, lse = torch.full_like(out, 7.0), torch.empty_like(want_lse)
    c.ctx.tree_attention(apart, layer, q, q_start, mask, again, work, scale=c.scale, lse=lse)
    torch.cuda.synchronize()
    assert torch.equal(again, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("P", [16, 5])
def test_missing_pages_read_as_zeros(ctx, P):
    c = Case(ctx, [90, 40], [3, 2], P=P, seed=21)
    zero = int(c.table[0, 1])  # a page that the table no longer names: the zeros of what is expected
    c.table[0, 1], c.table[0, 3], c.table[1, 0] = -1, 2**30, c.pools[0].shape[1]
    assert zero not in c.table
    out, lse = c.run()
    for pool in c.pools:
        pool[:, zero] = 0.0
    c.table[0, 1] = c.table[0, 3] = c.table[1, 0] = zero
    c.compare(out, lse)


def test_unknown_slots_see_nothing(ctx):
    c = Case(ctx, [20, 30, 10], [2, 3, 1], slots=[0, 1, 2], seed=22)
    c.run()
    cache, layer, q, q_start, mask, out, work = c.args
    slots = torch.tensor([0, 7, -1], dtype=torch.int32, device="cuda")
    lse = torch.zeros(6, 4, device="cuda")
    c.ctx.tree_attention(cache, layer, q, q_start, mask, out, work, scale=c.scale, lse=lse, seq_slots=slots)
    torch.cuda.synchronize()
    assert torch.all(out[2:] == 0) and torch.all(torch.isneginf(lse[2:])) and torch.isfinite(lse[:2]).all()


def test_one_slot_read_by_several_sequences(ctx):
    """Two trees after the same committed tokens: the drafts' places are shared, so the same drafts."""
    c = Case(ctx, [50], [4], seed=23)
    once, _ = c.run()
    cache, layer, q, q_start, mask, out, work = c.args
    twice = torch.empty(8, *q.shape[1:], dtype=q.dtype, device="cuda")
    c.ctx.tree_attention(cache, layer, q.repeat(2, 1, 1), torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda"),
                         mask.repeat(2, 1), twice, work, scale=c.scale,
                         seq_slots=torch.zeros(2, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert np.all(np.abs(twice.float().cpu().numpy() - once.repeat(2, 1, 1).float().cpu().numpy()) <= 2.0**-7)


def test_rows_that_see_nothing(ctx):
    c = Case(ctx, [0, 40, 0], [3, 2, 5], seed=6)
    c.mask[1] = 0          # a row without committed tokens that sees no draft either
    c.mask[5:7] = 0
    c.mask[3] = 0          # committed tokens only
    out, lse = c.check()
    assert torch.all(out[[1, 5, 6]] == 0) and torch.all(torch.isneginf(lse[[1, 5, 6]]))


def test_masks_beyond_trees_and_short_masks(ctx):
    c = Case(ctx, [30], [40], seed=7)
    c.mask[:] = np.random.default_rng(7).integers(-2**31, 2**31, c.mask.shape)  # bits past the drafts too
    c.check()
    Case(ctx, [30], [40], seed=8, words=1).check()  # drafts from 32 on are hidden
    Case(ctx, [30], [4], seed=8, words=0).check()
    Case(ctx, [3], [4], seed=8, words=5).check()


@pytest.mark.parametrize("P", [16, 5])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_bad_numbers_in_hidden_places(ctx, bad, P):
    """NaN and infinities past the sequence, in free pages, and in drafts that a row does not see."""
    c = Case(ctx, [100, 7], [6, 6], P=P, seed=9)
    k, v = c.pools
    used = torch.zeros(k.shape[1], P, dtype=torch.bool)
    for b in range(2):
        for j in range(c.lens[b] + c.drafts[b]):
            used[c.table[b, j // P], j % P] = True
    for pool in (k, v):
        pool[:, ~used] = bad
    # Draft 2 of sequence 0 is bad and seen by no row but its own; draft 4 of sequence 1 by none.
    c.mask[:12] &= ~(1 << 2)
    c.mask[2] |= 1 << 2
    c.mask[6:12] &= ~(1 << 4)
    for b, d in ((0, 2), (1, 4)):
        j = c.lens[b] + d
        k[:, c.table[b, j // P], j % P] = bad
        v[:, c.table[b, j // P], j % P, :, ::3] = bad
    out, lse = c.run()
    want, want_lse, _, _ = c.want()
    rows = [i for i in range(12) if i != 2]
    assert np.all(np.isfinite(want[rows]))
    assert np.all(np.abs(out.float().cpu().numpy()[rows] - want[rows]) <= 2.0**-6)
    assert np.all(np.abs(lse.cpu().numpy()[rows] - want_lse[rows]) <= 1e-4)


def test_bad_values_in_seen_drafts_reach_the_rows_that_see_them(ctx):
    c = Case(ctx, [40], [5], seed=10)
    v = c.pools[1]
    j = 40 + 3
    v[:, c.table[0, j // 16], j % 16, :, 7] = float("inf")
    v[:, c.table[0, j // 16], j % 16, :, 9] = float("nan")
    c.mask[:5] &= ~(1 << 3)
    c.mask[3:5] |= 1 << 3
    out, _ = c.run()
    assert torch.isfinite(out[:3]).all()
    assert torch.isposinf(out[3:, :, 7]).all() and torch.isnan(out[3:, :, 9]).all()
    rest = [d for d in range(64) if d not in (7, 9)]
    assert torch.isfinite(out[3:][:, :, rest]).all()
    v[:, c.table[0, j // 16], j % 16, :, [7, 9]] = 0.0  # the other elements as with any finite value there
    want = c.want()[0]
    assert np.all(np.abs(out.float().cpu().numpy()[:, :, rest] - want[:, :, rest]) <= 2.0**-6)


def test_large_logits(ctx):
    """Scores in the hundreds: weights from one to nothing, maxima that grow tile by tile."""
    c = Case(ctx, [700], [4], dim=128, spread=4.0, seed=11)
    grows = torch.ones(c.pools[0].shape[1])
    grows[c.table[0].long()] = torch.linspace(0.2, 6.0, c.table.shape[1])
    c.pools[0] *= grows.view(1, -1, 1, 1, 1).to(c.pools[0].dtype)
    c.check()
    c.scale = -0.5
    c.check()
    c.scale = 0.0
    c.check()


def test_strided_rows(ctx):
    """q and out as slices of a projection's output."""
    c = Case(ctx, [60, 9], [3, 5], q_heads=4, heads=2, seed=12)
    want, _ = c.run()
    cache, layer, q, q_start, mask, out, work = c.args
    wide = torch.randn(8, 4 + 2 + 2, 64, device="cuda").to(q.dtype)
    wide[:, :4] = q
    to = torch.zeros(4, 8, 128, device="cuda", dtype=q.dtype)
    c.ctx.tree_attention(cache, layer, wide[:, :4], q_start, mask, to.transpose(0, 1)[:, :, 64:], work, **c.kw)
    torch.cuda.synchronize()
    assert torch.equal(to.transpose(0, 1)[:, :, 64:], want)
    assert int((to[:, :, :64] != 0).sum()) == 0


def test_same_bits_twice_on_a_side_stream_and_without_lse(ctx):
    c = Case(ctx, [5000, 30, 800], [8, 8, 3], q_heads=8, heads=2, dim=128, seed=13)
    a, la = c.run()
    b, lb = c.run(stream=torch.cuda.Stream())
    d, _ = c.run(lse=False)
    assert torch.equal(a, b) and torch.equal(la, lb) and torch.equal(a, d)


def test_graph_replay_follows_the_lengths(ctx):
    c = Case(ctx, [300, 40], [4, 4], width=40, seed=14)
    c.run()
    cache, layer, q, q_start, mask, out, work = c.args
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        c.ctx.tree_attention(*c.args, **c.kw, stream=stream)
    lens = torch.tensor([137, 12], dtype=torch.int32)
    cache.tensors[4].copy_(lens)
    graph.replay()
    torch.cuda.synchronize()
    c.all_lens = lens
    want = c.want()[0]
    assert np.all(np.abs(out.float().cpu().numpy() - want) <= 2.0**-6)


def test_offsets_past_32_bits(ctx):
    """A pool of over 4 GiB whose last pages hold the sequence."""
    pages, P = 70000, 16
    k, v = (torch.zeros(1, pages, P, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    assert k.numel() * 2 > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(0)
    k[:, -2:] = torch.randn(1, 2, P, 16, 128, generator=g, device="cuda").to(k.dtype)
    v[:, -2:] = torch.randn(1, 2, P, 16, 128, generator=g, device="cuda").to(k.dtype)
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    one = torch.ones(pages, dtype=torch.int32, device="cuda")
    c = tb.kv_cache(k, v, table, one[:1] * 2, one[:1] * 29, one)
    q = torch.randn(2, 16, 128, generator=g, device="cuda").to(k.dtype)
    out = torch.empty_like(q)
    mask = torch.tensor(tb.tree_mask([-1, 0]), dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    work = torch.empty(ctx.tree_attention_workspace(c, 16), dtype=torch.uint8, device="cuda")
    ctx.tree_attention(c, 0, q, start, mask, out, work)
    torch.cuda.synchronize()
    want = cache_model.tree_attention(
        q.float().cpu().numpy(), k[0, -2:].float().cpu().numpy(), v[0, -2:].float().cpu().numpy(),
        np.array([[1, 0]]), np.array([29]), np.array([0, 2]), mask.cpu().numpy().astype(np.int64), 128 ** -0.5)[0]
    assert np.all(np.abs(out.float().cpu().numpy() - want) <= 2.0**-6)


def test_refusals(ctx):
    c = Case(ctx, [20], [3], seed=15)
    c.run()
    cache, layer, q, q_start, mask, out, work = c.args

    def refused(code, *args, **kw):
        with pytest.raises(tb.TBError) as e:
            ctx.tree_attention(*args, **kw)
        assert e.value.code == code

    refused(tb.TB_EINVAL, cache, 1, q, q_start, mask, out, work)
    refused(tb.TB_EINVAL, cache, -1, q, q_start, mask, out, work)
    refused(tb.TB_EINVAL, cache, 0, q[:, :3], q_start, mask, out[:, :3], work)
    refused(tb.TB_EINVAL, cache, 0, q, q_start, mask, out, work[:8])
    refused(tb.TB_EINVAL, cache, 0, q, q_start, mask, out, work[1:])
    refused(tb.TB_EINVAL, cache, 0, q, q_start, mask, out, work, scale=float("nan"))
    refused(tb.TB_EINVAL, cache, 0, q, torch.zeros(3, dtype=torch.int32, device="cuda"), mask, out, work)
    refused(tb.TB_ENOTSUP, cache, 0, q, torch.zeros(5000, dtype=torch.int32, device="cuda"), mask, out, work,
            seq_slots=torch.zeros(4999, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        ctx.tree_attention(cache, 0, q.float(), q_start, mask, out, work)
    with pytest.raises(ValueError):
        ctx.tree_attention(cache, 0, q, q_start, mask, out[:2], work)
    with pytest.raises(ValueError):
        ctx.tree_attention(cache, 0, q, q_start, mask[:2], out, work)
    with pytest.raises(TypeError):
        ctx.tree_attention(cache, 0, q, q_start.long(), mask, out, work)
    wide = torch.zeros(1, 4, 16, 2, 136, dtype=torch.bfloat16, device="cuda")
    big = tb.kv_cache(wide, wide, *cache.tensors[2:5], torch.zeros(4, dtype=torch.int32, device="cuda"))
    q2 = torch.zeros(3, 4, 136, dtype=torch.bfloat16, device="cuda")
    refused(tb.TB_ENOTSUP, big, 0, q2, q_start, mask, q2.clone(), work)
    f = wide[..., :64].float()
    single = tb.kv_cache(f, f, *cache.tensors[2:5], torch.zeros(4, dtype=torch.int32, device="cuda"))
    refused(tb.TB_ENOTSUP, single, 0, q.float(), q_start, mask, out.float(), work)
    # nothing to do is no error
    ctx.tree_attention(cache, 0, q[:0], q_start[:1], mask[:0], out[:0], work)
    torch.cuda.synchronize()


def test_expired_wait_is_reported_by_the_next_call(ctx):
    """A limit of 0 lets the kernel's first wait run out: it stops, and the next call says so."""
    with tb.Context(0, tb.options(kernel_wait_ns=0)) as hasty:
        c = Case(hasty, [3000], [4], seed=16)
        c.run()
        with pytest.raises(tb.TBError) as e:
            hasty.tree_attention(*c.args, **c.kw)
        assert e.value.code == tb.TB_ETIMEOUT
    Case(ctx, [3000], [4], seed=16).check()


@pytest.mark.parametrize("lens,drafts,q_heads,dim", [([3000], [4], 4, 64), ([90], [7], 8, 128), ([700, 20, 5000], [40, 3, 60], 16, 128)])
def test_calls_after_stopped_ones_are_right(ctx, lens, drafts, q_heads, dim):
    """What a stopped call had asked for must have landed before it ends: the calls
    behind it on the stream use the same shared memory.  Runs that fit the ring
    (their loads are all asked for without a wait) and runs that do not."""
    case = dict(q_heads=q_heads, heads=2, dim=dim, seed=24)
    right = Case(ctx, lens, drafts, **case)
    want, want_lse = (x.clone() for x in right.check())
    with tb.Context(0, tb.options(kernel_wait_ns=0)) as hasty:
        stopped = Case(hasty, lens, drafts, **case)
        stopped.run()
        for _ in range(30):
            right.args[5].fill_(7.0)
            right.kw["lse"].fill_(7.0)
            try:
                hasty.tree_attention(*stopped.args, **stopped.kw)
            except tb.TBError as e:
                assert e.code == tb.TB_ETIMEOUT
            ctx.tree_attention(*right.args, **right.kw)
            got, lse = right.args[5].clone(), right.kw["lse"].clone()
            torch.cuda.synchronize()
            assert torch.equal(got, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("seqs", [3, 700])
def test_query_rows_that_do_not_ascend_are_left_alone(ctx, seqs):
    """Sequences that name rows again could make more work than the call's counts
    hold: nothing is computed then."""
    c = Case(ctx, [40] * seqs, [2] * seqs, seed=25)
    c.run()
    cache, layer, q, q_start, mask, out, work = c.args
    for at, value in ((1, 2 * seqs), (seqs, 0), (seqs - 1, -5)):
        bad = q_start.clone()
        bad[at] = value
        out.fill_(7.0)
        c.kw["lse"].fill_(7.0)
        ctx.tree_attention(cache, layer, q, bad, mask, out, work, **c.kw)
        torch.cuda.synchronize()
        assert bool((out == 7.0).all()) and bool((c.kw["lse"] == 7.0).all())
    ctx.tree_attention(*c.args, **c.kw)
    torch.cuda.synchronize()
    c.rows = None if seqs < 10 else list(range(0, 2 * seqs, 97))
    c.compare(out, c.kw["lse"])


@pytest.mark.parametrize("below", [9.0, 14.0, 16.5, 17.0, 17.5, 18.0, 20.0])
@pytest.mark.parametrize("lens", [[2000] * 320, [131072, 17, 900]])
def test_many_small_weights_of_f16_add_up(ctx, below, lens):
    """One position leads all others by `below` in the exponent: their weights are far
    below f16's 2^-14, their sum is not.  16-bit weights 2^7 times exp(s - m) are off by
    2^-11 of each or, below 2^-21, by 2^-32 each; the whole result by those and its
    own rounding."""
    c = Case(ctx, lens, [1] * len(lens), q_heads=1, heads=1, dim=64, P=64, dtype="f16", seed=26,
             check_rows=3)
    g = torch.Generator().manual_seed(27)
    k, v = c.pools
    k.zero_()
    v.copy_(torch.rand(v.shape, generator=g) + 0.5)
    c.q.fill_(1.0)
    c.scale, c.rows = 0.125, [0, 1, len(lens) - 1]
    leaders = [(b, n // 3) for b, n in enumerate(lens)]
    for b, j in leaders:
        k[0, c.table[b, j // c.P], j % c.P] = below / 8.0  # 64 products of one: exact
        v[0, c.table[b, j // c.P], j % c.P] = 0.0
    out, lse = c.run()
    want, want_lse, reach, logit = (x[c.rows] for x in c.want())
    u, slack = 2.0**-11, (64 + 8) * 2.0**-24 * logit + 2.0**-20
    tail = u * reach + np.array([lens[i] for i in c.rows])[:, None, None] * 2.0**-32 * float(v.max())
    bound = u * want * 1.01 + (tail + 2 * slack[..., None] * reach) * (1 + u) + 2.0**-25
    off = np.abs(out.float().cpu().numpy().astype(np.float64)[c.rows] - want)
    assert np.all(off <= bound), float((off / bound).max())
    assert np.all(np.abs(lse.cpu().numpy()[c.rows] - want_lse) <= slack + 2.0**-20 * (1 + np.abs(want_lse)))


def test_infinite_values_under_small_f16_weights(ctx):
    c = Case(ctx, [300], [2], q_heads=1, heads=1, dim=64, dtype="f16", seed=28)
    k, v = c.pools
    k.zero_()
    c.q.fill_(1.0)
    c.scale = 0.125
    k[0, c.table[0, 1], 3] = 2.25  # 18 above the others
    v[0, c.table[0, 0], 5, :, 7] = float("inf")
    out, _ = c.run()
    assert torch.isposinf(out[:, :, 7]).all() and torch.isfinite(out[:, :, 8:]).all()
