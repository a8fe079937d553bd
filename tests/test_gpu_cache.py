"""The page operations of the paged cache against a plain model: every bit of
the pools, the table, the counts and the lengths has to be the model's."""
import threading

import numpy as np
import pytest

from cache_model import CacheModel

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from copy_reduce_dst_gb300 import _build  # noqa: E402

_build.build()
from copy_reduce_dst_gb300 import tb  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "byte": torch.uint8}


@pytest.fixture(scope="module")
def ctx():
    with tb.Context(0) as c:
        yield c


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Cache:
    """A cache on the GPU and its model, filled with random bits."""

    def __init__(self, layers=2, pages=24, P=4, heads=2, dim=16, slots=5, width=6, layout="NHD",
                 dtype="bf16", seed=0):
        g = np.random.default_rng(seed)
        self.layout, t = layout, TYPES[dtype]
        size = torch.empty(0, dtype=t).element_size()
        shape = (layers, pages, P, heads, dim * size)
        bits = [g.integers(0, 256, shape, dtype=np.uint8) for _ in "kv"]
        self.pools = []
        if layout == "mixed":  # keys and values side by side, pages outermost, gaps after a token
            self.whole = torch.zeros(pages, layers, P, heads, 2, dim * size + 16, dtype=torch.uint8,
                                     device="cuda")
            for i in range(2):
                view = self.whole[:, :, :, :, i, :dim * size].permute(1, 0, 2, 3, 4)
                view.copy_(dev(bits[i]))
                self.pools.append(view.view(t))
        else:
            for b in bits:
                b = dev(b) if layout == "NHD" else dev(b.transpose(0, 1, 3, 2, 4))
                self.pools.append(b.view(t))
        self.table = dev(np.full((slots, width), -1, np.int32))
        self.held, self.lens = (dev(np.zeros(slots, np.int32)) for _ in "hl")
        self.refs = dev(np.zeros(pages, np.int32))
        self.status = dev(np.full(1, -7, np.int32))
        self.model = CacheModel(*bits, *(x.cpu().numpy() for x in (self.table, self.held, self.lens,
                                                                   self.refs)))
        self.describe()

    def describe(self):
        self.c = tb.kv_cache(*self.pools, self.table, self.held, self.lens, self.refs,
                             layout="HND" if self.layout == "HND" else "NHD")

    def set_lens(self, lens):
        self.model.lens[:] = lens
        self.lens.copy_(dev(np.asarray(lens, np.int32)))

    def resize(self, ctx, capacity, stream=None):
        ctx.kv_resize(self.c, dev(np.asarray(capacity, np.int32)), self.status, stream)
        return self.model.resize(capacity)

    def fork(self, ctx, parents):
        out = [torch.full_like(x, 77) for x in (self.table, self.held, self.lens)]
        ctx.kv_fork(self.c, dev(np.asarray(parents, np.int32)), *out, self.status)
        self.table, self.held, self.lens = out
        self.describe()
        return self.model.fork(parents)

    def compact(self, ctx, start, keep, count):
        status = dev(np.full(len(start), -7, np.int32))
        ctx.kv_compact(self.c, *(dev(np.asarray(x, np.int32)) for x in (start, keep, count)), status)
        want = self.model.compact(start, np.asarray(keep), count)
        assert status.cpu().numpy().tolist() == want.tolist()

    def check(self, status=None):
        torch.cuda.synchronize()
        if status is not None:
            assert int(self.status) == status
        m = self.model
        for name in ("table", "held", "lens", "refs"):
            np.testing.assert_array_equal(getattr(self, name).cpu().numpy(), getattr(m, name), name)
        for got, want in zip(self.pools, (m.k, m.v)):
            got = got.view(torch.uint8).contiguous().cpu().numpy()
            if self.layout == "HND":
                got = got.transpose(0, 1, 3, 2, 4)
            np.testing.assert_array_equal(got, want)
        if self.layout == "mixed":  # the gaps
            assert int(self.whole[..., -16:].max()) == 0
        np.testing.assert_array_equal(m.refs, np.bincount(m.table[m.table >= 0],
                                                          minlength=m.refs.size))


LAYOUTS = ["NHD", "HND", "mixed"]


# ---------------------------------------------------------------------------
# Copy
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f16", 8), ("f32", 20), ("byte", 48)])
@pytest.mark.parametrize("P,heads", [(1, 1), (16, 3), (5, 8), (64, 1)])
def test_copy_pages(ctx, layout, dtype, dim, P, heads):
    x = Cache(layers=3, pages=40, P=P, heads=heads, dim=dim, layout=layout, dtype=dtype, seed=P)
    g = np.random.default_rng(P * 7 + heads)
    order = g.permutation(40).astype(np.int32)
    src, dst = order[:20], order[20:]
    src[3], dst[5], src[6], dst[7] = -1, -1, 40, 2**31 - 1  # skipped
    ctx.kv_copy_pages(x.c, dev(src), dev(dst))
    x.model.copy_pages(src, dst)
    x.check()
    tokens = g.integers(-1, P + 2, 20).astype(np.int32)  # nothing, a part, all, clamped
    ctx.kv_copy_pages(x.c, dev(dst), dev(src), 19, tokens=dev(tokens))
    x.model.copy_pages(dst[:19], src[:19], tokens)
    x.check()


def test_copy_many_layers_and_one_entry(ctx):
    x = Cache(layers=70, pages=3, P=16, heads=2, dim=64)
    ctx.kv_copy_pages(x.c, dev(np.array([2], np.int32)), dev(np.array([0], np.int32)))
    x.model.copy_pages([2], [0])
    x.check()
    ctx.kv_copy_pages(x.c, dev(np.zeros(0, np.int32)), dev(np.zeros(0, np.int32)))
    x.check()


def test_copy_past_32_bit_offsets(ctx):
    # 5 GiB of one-layer pages; the last page lies past 2^32 bytes
    pages, bytes_ = 80, 64 << 20
    pool = torch.zeros(2, 1, pages, 64, 8, bytes_ // 512, dtype=torch.uint8, device="cuda")
    pool[:, 0, 1] = 3
    pool[0, 0, 1, 5] = 9
    c = tb.kv_cache(pool[0], pool[1])
    ctx.kv_copy_pages(c, dev(np.array([1], np.int32)), dev(np.array([pages - 1], np.int32)))
    torch.cuda.synchronize()
    assert torch.equal(pool[:, 0, 1], pool[:, 0, pages - 1])
    assert int(pool[:, 0, 2:pages - 1].max()) == 0


# ---------------------------------------------------------------------------
# Resize
# ---------------------------------------------------------------------------
def test_resize_takes_the_lowest_free_pages_and_gives_back(ctx):
    x = Cache(slots=4, width=6, pages=16, P=4)
    assert x.resize(ctx, [5, 0, 9, 4]) == 0  # 2, 0, 3, 1 pages
    x.check(0)
    assert x.table[2, :4].tolist() == [2, 3, 4, -1]
    x.set_lens([5, 0, 8, 1])
    assert x.resize(ctx, [-1, 8, 4, 0]) == 0  # slot 2 gives two back, slot 3 its only one
    x.check(0)
    assert x.table[1, :2].tolist() == [6, 7]  # not yet the pages given back by the same call
    assert x.resize(ctx, [24, 8, 4, 12]) == 0
    x.check(0)


def test_resize_refuses_as_a_whole(ctx):
    x = Cache(slots=3, width=4, pages=7, P=4)
    assert x.resize(ctx, [16, 4, 0]) == 0
    x.check(0)
    assert x.resize(ctx, [0, 16, 4]) == 2  # 4 more pages, 2 free: 2 missing; nothing given back
    x.check(2)
    assert x.resize(ctx, [-1, 17, 0]) == -1  # 5 pages in a row of 4
    x.check(-1)
    assert x.resize(ctx, [2**31 - 1, -1, -1]) == -1
    x.check(-1)


def test_resize_does_not_cut_inside_a_shared_page(ctx):
    x = Cache(slots=3, width=4, pages=12, P=4)
    x.resize(ctx, [9, 0, 0])
    x.set_lens([9, 0, 0])
    assert x.fork(ctx, [0, 0, -1]) == 0
    x.check(0)
    assert x.resize(ctx, [6, -1, -1]) == -1  # page 1 is shared and would be written again
    x.check(-1)
    assert x.resize(ctx, [4, -1, -1]) == 0
    x.check(0)


@pytest.mark.parametrize("slots,width,pages,P", [(1, 1, 1, 1), (70, 40, 2500, 8), (1500, 3, 6000, 16),
                                                 (8192, 2, 20000, 1), (3, 3000, 70001, 5)])
def test_resize_random(ctx, slots, width, pages, P):
    x = Cache(layers=1, heads=1, dim=8, slots=slots, width=width, pages=pages, P=P)
    g = np.random.default_rng(slots + pages)
    for _ in range(4):
        capacity = g.integers(-1, width * P + 1, slots)
        capacity[g.random(slots) < 0.3] = 0
        want = x.resize(ctx, capacity.tolist())
        x.check(want)
        x.set_lens(np.minimum(x.model.held * P, g.integers(0, width * P + 1, slots)))


# ---------------------------------------------------------------------------
# Fork
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("P,lens", [(4, [9, 8, 1, 0, 4]), (1, [3, 1, 0, 6, 2]), (5, [5, 29, 30, 4, 6])])
def test_fork(ctx, layout, P, lens):
    x = Cache(slots=5, width=6, pages=60, P=P, layout=layout)
    x.resize(ctx, [min(n + 6, 6 * P) for n in lens])  # spare pages beyond the tokens
    x.set_lens(lens)
    for parents in ([0, 0, 0, 3, 4], [1, 0, 1, -1, 2], [4, 4, 4, 4, 4], [0, 1, 2, 3, 4], [-1, -1, 3, 3, -5],
                    [-1] * 5):
        assert x.fork(ctx, parents) == 0
        x.check(0)
    assert int(x.refs.max()) == 0


def test_fork_refuses_as_a_whole(ctx):
    x = Cache(slots=4, width=3, pages=5, P=4)
    x.resize(ctx, [6, 5, 0, 0])
    x.set_lens([6, 5, 0, 0])
    assert x.fork(ctx, [0, 1, 0, 1]) == 1  # one page free, two part-filled pages to copy
    x.check(1)
    assert x.fork(ctx, [0, 1, 4, -1]) == -1
    x.check(-1)
    assert x.fork(ctx, [-1, 1, 1, -1]) == 0
    x.check(0)


@pytest.mark.parametrize("slots,width,P,pages", [(300, 20, 3, 8000), (8192, 1, 2, 20000), (12, 700, 16, 9000)])
def test_fork_random(ctx, slots, width, P, pages):
    x = Cache(layers=2, heads=1, dim=8, slots=slots, width=width, pages=pages, P=P)
    g = np.random.default_rng(slots)
    x.resize(ctx, np.full(slots, width * P).tolist())
    x.set_lens(g.integers(0, width * P + 1, slots))
    for _ in range(3):
        parents = g.integers(-1, slots, slots).tolist()
        x.check(x.fork(ctx, parents))


# ---------------------------------------------------------------------------
# Compact
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("P,dtype,dim", [(4, "bf16", 64), (1, "f32", 4), (16, "byte", 16)])
def test_compact(ctx, layout, P, dtype, dim):
    width = 64 // P
    x = Cache(slots=5, width=width, pages=5 * width, P=P, layout=layout, dtype=dtype, dim=dim, heads=3)
    x.resize(ctx, [64] * 5)
    x.set_lens([64] * 5)
    g = np.random.default_rng(P)
    keep = np.sort([g.permutation(40)[:30] for _ in range(5)], axis=1)
    keep[3] = np.arange(30)  # nothing moves
    keep[4] = np.arange(30) + 10  # each token onto the place that the token ten before it left
    x.compact(ctx, [20, 0, 33 - 9, 5, 0], keep, [30, 17, 0, 30, 30])
    x.check()
    x.compact(ctx, [1, 2, 3, 4, 5], keep[:, :1], [1, -1, 0, 1, 1])
    x.check()


def test_compact_long_list(ctx):
    x = Cache(layers=1, slots=2, width=150, pages=300, P=8, heads=1, dim=8)
    x.resize(ctx, [1200, 1200])
    x.set_lens([1200, 1100])
    g = np.random.default_rng(3)
    keep = np.stack([np.sort(g.permutation(1150)[:1001]), np.concatenate([np.arange(500), np.arange(501) + 600])])
    x.compact(ctx, [50, 0], keep, [1001, 1001])
    x.check()


def test_compact_short_lists_of_many_slots(ctx):
    slots, P = 150, 5
    x = Cache(layers=8, slots=slots, width=5, pages=5 * slots, P=P, heads=2, dim=64)
    x.resize(ctx, [25] * slots)
    x.set_lens([11] * slots)
    g = np.random.default_rng(4)
    keep = np.sort([g.permutation(14)[:4] for _ in range(slots)], axis=1)
    keep[7] = [0, 3, 3, 4]  # does not ascend
    keep[8] = [0, 2, 4, 14]  # past the slot's pages
    x.compact(ctx, [11] * slots, keep, g.integers(-1, 5, slots).tolist())
    x.check()


def test_compact_refusals(ctx):
    x = Cache(slots=6, width=4, pages=40, P=4)
    x.resize(ctx, [16] * 5 + [0])
    x.set_lens([9, 16, 16, 16, 16, 0])
    assert x.fork(ctx, [0, 1, 2, 3, 4, 0]) == 0
    # slot 0 shares its first two pages: a move inside them, a cut inside them, a move after them
    for start, keep, count in ((0, [0, 2], 2), (5, [0, 1], 0), (8, [0, 1], 1)):
        x.compact(ctx, [start, 0, 0, 0, 0, 0], [keep, [1, 0], [0, 16], [0, 0], [-1, 2], [0, 1]],
                  [count, 2, 2, 2, 2, 1])
        x.check()
    x.compact(ctx, [0, 15, -1, 13, 0, 0], [[0, 1]] * 6, [3, 2, 1, 2, -1, 0])
    x.check()


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("seed", range(6))
def test_random_steps(ctx, seed):
    """Resizes, forks and compactions in a random order."""
    g = np.random.default_rng(100 + seed)
    slots, P = int(g.integers(2, 12)), int(g.choice([1, 3, 4, 16]))
    width = int(g.integers(2, 20))
    x = Cache(slots=slots, width=width, pages=slots * width, P=P, layout=LAYOUTS[seed % 3], seed=seed)
    for _ in range(25):
        what = g.integers(0, 4)
        if what == 0:
            x.check(x.resize(ctx, g.integers(-1, width * P + 1, slots).tolist()))
        elif what == 1:  # tokens appended inside the pages held
            x.set_lens([int(g.integers(n, h * P + 1)) for n, h in zip(x.model.lens, x.model.held)])
        elif what == 2:
            x.check(x.fork(ctx, g.integers(-1, slots, slots).tolist()))
        else:
            start = [int(g.integers(0, n + 1)) for n in x.model.lens]
            most = max(int(n) - s for n, s in zip(x.model.lens, start))
            keep = np.sort(np.stack([g.permutation(most + 1) for _ in range(slots)])[:, :most // 2 + 1], axis=1)
            count = g.integers(-1, keep.shape[1] + 1, slots).tolist()
            x.compact(ctx, start, keep, count)
            x.check()


def test_side_stream_and_graph(ctx):
    """Calls on a stream of their own, and replayed from a graph."""
    x = Cache(slots=3, width=4, pages=20, P=4)
    stream = torch.cuda.Stream()
    capacity, status = dev(np.array([5, 9, 0], np.int32)), x.status
    out = [torch.empty_like(t) for t in (x.table, x.held, x.lens)]
    parents = dev(np.array([0, 1, 1], np.int32))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        ctx.kv_resize(x.c, capacity, status, stream)
        ctx.kv_fork(x.c, parents, *out, status, stream)
    graph.replay()
    torch.cuda.synchronize()
    assert x.model.resize([5, 9, 0]) == 0 and x.model.fork([0, 1, 1]) == 0
    x.table, x.held, x.lens = out
    x.check(0)


# ---------------------------------------------------------------------------
# Refusals
# ---------------------------------------------------------------------------
def refused(code, call, *args, **kw):
    with pytest.raises(tb.TBError) as e:
        call(*args, **kw)
    assert e.value.code == code


def test_refusals(ctx):
    x = Cache()
    one, many = x.status, dev(np.zeros(5, np.int32))
    s = x.c.struct

    def with_(**kw):
        old = {n: getattr(s, n) for n in kw}
        for n, v in kw.items():
            setattr(s, n, v)
        return lambda: [setattr(s, n, v) for n, v in old.items()]

    for bad in (dict(k=None), dict(layers=0), dict(page_tokens=0), dict(dtype=9), dict(k=s.k + 8),
                dict(page_stride=s.page_stride + 8), dict(token_stride=16), dict(head_stride=0),
                dict(pages=2**31 - 1, page_stride=2**60)):
        undo = with_(**bad)
        refused(tb.TB_EINVAL, ctx.kv_copy_pages, x.c, many, many)
        undo()
    undo = with_(layers=70000)
    refused(tb.TB_ENOTSUP, ctx.kv_copy_pages, x.c, many, many)
    undo()
    refused(tb.TB_EINVAL, ctx.kv_copy_pages, x.c, many, many, -1)
    for bad in (dict(table=None), dict(refs=None), dict(held=None), dict(lens=None), dict(table_width=0)):
        undo = with_(**bad)
        refused(tb.TB_EINVAL, lambda: ctx._ok(tb.lib.tb_kv_resize(
            ctx.handle, x.c.ref, many.data_ptr(), one.data_ptr(), None), ""))
        undo()
    undo = with_(table_width=2**30)
    refused(tb.TB_ENOTSUP, lambda: ctx._ok(tb.lib.tb_kv_resize(
        ctx.handle, x.c.ref, many.data_ptr(), one.data_ptr(), None), ""))
    undo()
    undo = with_(slots=tb.TB_KV_MAX_SLOTS + 1)
    refused(tb.TB_ENOTSUP, lambda: ctx._ok(tb.lib.tb_kv_resize(
        ctx.handle, x.c.ref, many.data_ptr(), one.data_ptr(), None), ""))
    undo()
    refused(tb.TB_EINVAL, ctx.kv_fork, x.c, many, x.table, torch.empty_like(x.held), torch.empty_like(x.lens), one)
    refused(tb.TB_EINVAL, ctx.kv_compact, x.c, x.lens, many[:, None].contiguous(), many, torch.empty_like(many))
    refused(tb.TB_EINVAL, ctx.kv_compact, x.c, many, many[:, None].contiguous(), x.lens, torch.empty_like(many))
    refused(tb.TB_EINVAL, ctx.kv_fork, x.c, many, torch.empty_like(x.table), x.held, torch.empty_like(x.lens), one)
    with pytest.raises(ValueError):
        ctx.kv_resize(x.c, dev(np.zeros(4, np.int32)), one)
    with pytest.raises(TypeError):
        ctx.kv_resize(x.c, dev(np.zeros(5, np.int64)), one)
    with pytest.raises(ValueError):
        ctx.kv_copy_pages(x.c, many, many, 6)
    with pytest.raises(TypeError):
        ctx.kv_copy_pages(x.c, many.cpu(), many)
    with pytest.raises(ValueError):
        tb.kv_cache(x.pools[0], x.pools[1][:, :1])
    with pytest.raises(ValueError):
        tb.kv_cache(x.pools[0], None)
    x.check()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("shift", ["same", "token", "head", "page", "layer", "part of a row", "backwards"])
def test_compact_refuses_pools_that_share_memory(ctx, layout, shift):
    """One pool for both would have its tokens moved twice, the second time from
    places already written."""
    x = Cache(slots=2, width=4, pages=10, P=4, heads=3, dim=32, layers=2, layout=layout)
    s, many = x.c.struct, dev(np.zeros(2, np.int32))
    s.v = s.k + {"same": 0, "token": s.token_stride, "head": s.head_stride, "page": 7 * s.page_stride,
                 "layer": s.layer_stride, "part of a row": 2 * s.head_stride + 16,
                 "backwards": -3 * s.page_stride - 2 * s.token_stride - 48}[shift]
    refused(tb.TB_EINVAL, ctx.kv_compact, x.c, many, many[:, None].contiguous(), many, torch.empty_like(many))


def test_compact_of_the_two_halves_of_a_pools_rows(ctx):
    """One pool with rows of 48 elements described as keys of 16 and values of 16,
    with a gap between them: nothing is shared."""
    x = Cache(slots=2, width=4, pages=10, P=4, heads=3, dim=16, layers=2)
    whole = torch.zeros(2, 10, 4, 3, 48, dtype=torch.bfloat16, device="cuda")
    for pool, at in zip(x.pools, (32, 0)):
        whole[..., at:at + 16] = pool
    x.pools = [whole[..., 32:], whole[..., :16]]
    x.describe()
    x.resize(ctx, [16, 16])
    x.set_lens([16, 11])
    x.compact(ctx, [3, 0], [[0, 2, 5, 6], [1, 2, 3, 9]], [4, 4])
    x.check()
    assert int((whole[..., 16:32] != 0).sum()) == 0


def test_arrays_that_overlap_are_refused(ctx):
    """What a call writes must not be what it reads, or another thing that it writes."""
    x = Cache(slots=3, width=4, pages=12, P=4)
    x.resize(ctx, [9, 5, 0])
    x.set_lens([9, 4, 0])
    x.check(0)
    ints = dev(np.zeros(64, np.int32))
    three, one, table = (lambda i: ints[i:i + 3]), x.status, ints[32:44].view(3, 4)
    s = x.c.struct
    # resize: capacity and status against what changes, status against capacity
    for capacity in (x.held, x.refs[2:5], x.table[1, :3]):
        refused(tb.TB_EINVAL, ctx.kv_resize, x.c, capacity, one)
    for status in (x.held[2:], x.lens[:1], x.refs[11:], x.table[2, 3:]):
        refused(tb.TB_EINVAL, ctx.kv_resize, x.c, three(0), status)
    refused(tb.TB_EINVAL, ctx.kv_resize, x.c, three(0), ints[2:3])
    # fork: each output against each input and the other outputs
    good = dict(parents=three(0), table_out=table, held_out=three(4), lens_out=three(8), status=ints[12:13])
    for name, value in (("table_out", x.refs.view(3, 4)), ("table_out", ints[6:18].view(3, 4)), ("held_out", x.lens),
                        ("held_out", three(1)), ("held_out", x.table[0, 1:]), ("lens_out", x.held),
                        ("lens_out", three(5)), ("lens_out", x.refs[:3]), ("status", ints[2:3]), ("status", x.lens[2:]),
                        ("status", ints[10:11]), ("status", ints[40:41]), ("parents", x.refs[9:])):
        refused(tb.TB_EINVAL, ctx.kv_fork, x.c, **{**good, name: value})
    # compact: status against everything, keep against lens
    keep = ints[32:38].view(3, 2)
    good = dict(start=three(0), keep=keep, count=three(4), status=three(8))
    for name, value in (("status", three(1)), ("status", three(5)), ("status", ints[37:40]), ("status", x.lens),
                        ("status", x.held), ("status", x.refs[4:7]), ("keep", x.lens.view(3, 1)), ("start", x.lens)):
        refused(tb.TB_EINVAL, ctx.kv_compact, x.c, **{**good, name: value})
    x.check(0)
    # neighbours are fine, and so are the lengths as capacities
    ctx.kv_resize(x.c, x.lens, ints[3:4])
    assert x.model.resize([9, 4, 0]) == 0
    x.check()
    ints[:3] = torch.tensor([0, 1, -1])
    out = (ints[3:15].view(3, 4), ints[15:18], ints[18:21])
    ctx.kv_fork(x.c, ints[:3], *out, ints[21:22])
    x.table, x.held, x.lens = out
    x.describe()
    assert x.model.fork([0, 1, -1]) == 0
    x.check()
    assert int(ints[21]) == 0


def test_calls_run_on_the_current_stream(ctx):
    """Without stream= a call runs behind what the current stream still has to do,
    and is captured where that stream is."""
    x = Cache(slots=3, width=6, pages=20, P=4)
    busy, stream = torch.randn(8192, 8192, device="cuda").bfloat16(), torch.cuda.Stream()
    late = dev(np.array([9, 5, 22], np.int32))
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        for _ in range(40):
            busy @ busy
        ctx.kv_resize(x.c, late + 1, x.status)  # made behind the products, dropped at once
        reuse = torch.full((3,), 1, dtype=torch.int32, device="cuda")
        for _ in range(10):
            busy @ busy
        x.lens.copy_(late)
        out = [torch.full_like(t, 77) for t in (x.table, x.held, x.lens)]
        ctx.kv_fork(x.c, reuse - 1, *out, x.status)
    torch.cuda.synchronize()
    assert x.model.resize([10, 6, 23]) == 0
    x.model.lens[:] = [9, 5, 22]
    assert x.model.fork([0, 0, 0]) == 0
    x.table, x.held, x.lens = out
    x.describe()
    x.check(0)
    start, count, status = x.lens.clone(), dev(np.array([1, 1, 0], np.int32)), torch.zeros_like(x.lens)
    keep, src, dst = torch.zeros(3, 1, dtype=torch.int32, device="cuda"), dev(np.array([0], np.int32)), dev(np.array([19], np.int32))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ctx.kv_resize(x.c, start + 4, x.status)
        ctx.kv_compact(x.c, start, keep, count, status)
        ctx.kv_copy_pages(x.c, src, dst)
    graph.replay()
    assert x.model.resize([13, 13, 13]) == 0
    x.model.compact([9, 9, 9], np.zeros((3, 1), np.int32), [1, 1, 0])
    x.model.copy_pages([0], [19])
    x.check(0)
    assert status.tolist() == [0, 0, 0]


def test_threads_with_caches_of_different_sizes(ctx):
    """Two threads, a context and a stream each: the shared memory that one's calls
    need must not be taken from the other's."""
    failed = []

    def work(slots, calls):
        try:
            stream = torch.cuda.Stream()
            with tb.Context(0) as own:
                x = Cache(layers=1, heads=1, dim=8, slots=slots, width=1, pages=16, P=1)
                capacity, parents = dev(np.zeros(slots, np.int32)), dev(np.full(slots, -1, np.int32))
                out = [torch.empty_like(t) for t in (x.table, x.held, x.lens)]
                torch.cuda.synchronize()
                for _ in range(calls):
                    own.kv_resize(x.c, capacity, x.status, stream)
                    own.kv_fork(x.c, parents, *out, x.status, stream)
                stream.synchronize()
        except Exception as e:  # told to the test below
            failed.append(e)

    threads = [threading.Thread(target=work, args=(slots, 4000)) for slots in (8192, 4000, 5200, 7000)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


def test_statuses_of_cuts_in_shared_pages(ctx):
    """A cut inside a shared page: the whole resize is refused with -1, a compaction
    that moves nothing with 1, the other slots' growth and moves apart.  Then what
    the header says to do about it."""
    x = Cache(slots=3, width=5, pages=20, P=4)
    x.resize(ctx, [9, 0, 4])
    x.set_lens([9, 0, 4])
    assert x.fork(ctx, [0, 0, 2]) == 0
    assert x.resize(ctx, [6, -1, 12]) == -1
    x.check(-1)
    x.compact(ctx, [6, 0, 1], [[0], [0], [2]], [0, -1, 1])
    x.check()
    assert x.lens.tolist() == [9, 9, 2]
    page = int(x.table[0, 1])  # two of its tokens are to stay
    assert x.resize(ctx, [4, -1, 12]) == 0
    assert x.resize(ctx, [6, -1, -1]) == 0
    own = int(x.table[0, 1])
    assert own != page
    ctx.kv_copy_pages(x.c, dev(np.array([page], np.int32)), x.table[0, 1:2], tokens=dev(np.array([2], np.int32)))
    x.model.copy_pages([page], [own], [2])
    x.set_lens([6, 9, 2])
    x.check(0)


@pytest.mark.parametrize("slots,layers,n", [(2, 1, 300), (2, 1, 257), (3, 8, 511), (40, 8, 140), (150, 8, 100),
                                            (150, 8, 31), (2, 1, 512)])
def test_compact_lists_of_every_length(ctx, slots, layers, n):
    """Every form of the moving kernel: one, four and eight warps, with the lists
    looked through by each of its CTAs or by a launch before."""
    P, span = 8, n + n // 3 + 9
    width = -(-(span + 20) // P)
    x = Cache(layers=layers, slots=slots, width=width, pages=slots * width, P=P, heads=2, dim=64, seed=n)
    x.resize(ctx, [width * P] * slots)
    x.set_lens([span + 20] * slots)
    g = np.random.default_rng(n)
    keep = np.sort([g.permutation(span)[:n] for _ in range(slots)], axis=1)
    keep[1, n // 2] = keep[1, n // 2 - 1]  # does not ascend
    count = g.integers(n // 2, n + 1, slots)
    count[1] = n
    x.compact(ctx, g.integers(0, 21, slots).tolist(), keep, count.tolist())
    x.check()


def test_resize_of_a_pool_of_millions_of_pages(ctx):
    """More pages than the hand-out keeps in registers (4096 a warp, 512 warps): the
    free ones beyond are looked for again."""
    pages, slots, width = 3000001, 600, 40
    g = np.random.default_rng(29)
    refs = np.ones(pages, np.int32)
    refs[g.choice(pages, 20000, replace=False)] = 0
    share = pages // 512
    refs[200 * share + 4096:201 * share] = 0  # a run past the 4096th page of a warp's share
    free = np.flatnonzero(refs == 0)
    table, held, lens = dev(np.full((slots, width), -1, np.int32)), dev(np.zeros(slots, np.int32)), dev(np.zeros(slots, np.int32))
    counts, status = dev(refs), dev(np.full(1, -7, np.int32))
    c = tb.kv_cache(None, None, table, held, lens, counts, page_tokens=4)
    need = g.integers(20, width + 1, slots)
    ctx.kv_resize(c, dev((4 * need).astype(np.int32)), status)
    torch.cuda.synchronize()
    total = int(need.sum())
    assert int(status) == 0 and 10000 < total < free.size
    want = np.full((slots, width), -1, np.int32)
    want[np.arange(width) < need[:, None]] = free[:total]
    np.testing.assert_array_equal(table.cpu().numpy(), want)
    np.testing.assert_array_equal(held.cpu().numpy(), need)
    refs[free[:total]] = 1
    np.testing.assert_array_equal(counts.cpu().numpy(), refs)
    # Nearly all of the rest, then all given back.
    rest = free.size - total
    grow = need.copy()
    for s in range(slots):
        more = min(width - int(need[s]), rest - 1)
        grow[s], rest = grow[s] + more, rest - more
    ctx.kv_resize(c, dev((4 * grow).astype(np.int32)), status)
    torch.cuda.synchronize()
    left = int((counts == 0).sum())
    assert int(status) == 0 and left == free.size - int(grow.sum())
    order = np.concatenate([np.arange(need[s], grow[s]) + s * width for s in range(slots)])
    np.testing.assert_array_equal(table.cpu().numpy().ravel()[order], free[total:total + order.size])
    ctx.kv_resize(c, dev(np.zeros(slots, np.int32)), status)
    torch.cuda.synchronize()
    assert int(status) == 0 and int((counts == 0).sum()) == free.size and bool((table == -1).all())
    want = np.ones(pages, np.int32)
    want[free] = 0
    np.testing.assert_array_equal(counts.cpu().numpy(), want)
