"""Cases of the paged-cache operators: pages copied, held and freed, forked and
compacted, and attention for a tree of drafted tokens over the pages.

``listed()`` names the cases, ``draw(rng)`` makes more of the same ranges,
``prepare(case, seed)`` what a serving program has in hand before the call and
``run(state)`` one pass: with ``own`` set through libtb's entry points, else in
plain torch operations.  ``exact(case, seed)`` is the attention's definition in
64 bits; the page operators only move bits and whole numbers.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
DEV = "cuda"


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _copy(name, pairs, layers, pages, page_tokens=16, kv_heads=8, head_dim=128, dtype="bf16",
          layout="NHD", partial=False):
    return dict(name=name, op="copy", pairs=pairs, layers=layers, pages=pages,
                page_tokens=page_tokens, kv_heads=kv_heads, head_dim=head_dim, dtype=dtype,
                layout=layout, partial=partial)


def _resize(name, slots, width, moving, page_tokens=16):
    return dict(name=name, op="resize", slots=slots, width=width, moving=moving,
                page_tokens=page_tokens)


def _fork(name, groups, beams, tokens, layers, page_tokens=16, kv_heads=8, head_dim=128,
          dtype="bf16", layout="NHD"):
    return dict(name=name, op="fork", groups=groups, beams=beams, tokens=tokens, layers=layers,
                page_tokens=page_tokens, kv_heads=kv_heads, head_dim=head_dim, dtype=dtype,
                layout=layout)


def _compact(name, slots, layers, start, span, keep, page_tokens=16, kv_heads=8, head_dim=128,
             dtype="bf16", layout="NHD"):
    return dict(name=name, op="compact", slots=slots, layers=layers, start=start, span=span,
                keep=keep, page_tokens=page_tokens, kv_heads=kv_heads, head_dim=head_dim,
                dtype=dtype, layout=layout)


def _tree(name, seqs, tokens, drafts, q_heads, kv_heads=8, head_dim=128, page_tokens=16,
          dtype="bf16", layout="NHD", ragged=False):
    return dict(name=name, op="tree", seqs=seqs, tokens=tokens, drafts=drafts, q_heads=q_heads,
                kv_heads=kv_heads, head_dim=head_dim, page_tokens=page_tokens, dtype=dtype,
                layout=layout, ragged=ragged)


def listed():
    return [
        # A short prompt's pages copied on write in a small two-layer cache.
        _copy("copy 8 pages", 8, layers=2, pages=512),
        # A cache's pages moved beside one another before a transfer, all layers at once.
        _copy("copy 1000 pages x 16 layers", 1000, layers=16, pages=2048),
        # A small server's step: some requests end, others are admitted.
        _resize("resize 16 slots", 16, width=64, moving=0.5),
        # A large server's step: 512 slots of up to 4096 pages, a tenth of them changing.
        _resize("resize 512 slots", 512, width=4096, moving=0.1),
        # One beam search of four beams after a short prompt.
        _fork("fork 4 beams", 1, 4, tokens=500, layers=4),
        # 32 beam searches of eight beams after long prompts.
        _fork("fork 32 x 8 beams", 32, 8, tokens=4007, layers=8),
        # The accepted path of a small draft tree moved behind the committed tokens.
        _compact("accept a draft", 4, layers=2, start=300, span=16, keep=4),
        # Half of the tokens of long sequences dropped from a heads-first cache.
        _compact("keep half of 8192 tokens", 8, layers=8, start=0, span=8192, keep=4096,
                 dtype="f16", layout="HND"),
        # One chat, a tree of eight drafted tokens, a short cache: latency.
        _tree("tree of 8, one chat", 1, 500, 8, q_heads=32),
        # A batch of chats of mixed lengths, trees of 32.
        _tree("tree of 32, 32 chats", 32, 4096, 32, q_heads=32, page_tokens=32, layout="HND",
              ragged=True),
        # One long document with a large tree: 8 query heads share a cache head.
        _tree("tree of 64, 131072 tokens", 1, 131072, 64, q_heads=64, page_tokens=64, dtype="f16"),
        # Many short chats of a small model, one query head per cache head, odd pages.
        _tree("trees of up to 12, 96 chats", 96, 700, 12, q_heads=12, kv_heads=12, head_dim=64,
              page_tokens=24, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["copy", "resize", "fork", "compact", "tree", "tree", "tree"])
    page = rng.choice([1, 5, 8, 16, 16, 24, 32, 64, 128])
    kind = dict(kv_heads=rng.choice([1, 2, 4, 5, 8]), head_dim=rng.choice([64, 80, 96, 128]),
                dtype=rng.choice(["bf16", "f16"]), layout=rng.choice(["NHD", "HND"]))
    if op == "copy":
        pairs, layers = _log_int(rng, 1, 700), _log_int(rng, 1, 16)
        page = rng.choice([8, 16, 24, 32])
        case = _copy("", pairs, layers, 2 * pairs + _log_int(rng, 1, 500), page, partial=rng.random() < 0.3,
                     **kind)
    elif op == "resize":
        case = _resize("", _log_int(rng, 1, 512), _log_int(rng, 1, 4096), round(rng.uniform(0.02, 0.9), 2), page)
    elif op == "fork":
        case = _fork("", _log_int(rng, 1, 24), rng.randint(2, 8), _log_int(rng, 1, 3000), _log_int(rng, 1, 8), page,
                     **kind)
    elif op == "compact":
        span = _log_int(rng, 2, 4000)
        case = _compact("", _log_int(rng, 1, 12), _log_int(rng, 1, 8), _log_int(rng, 1, 2000), span,
                        rng.randint(1, span), page, **kind)
    else:
        heads = kind.pop("kv_heads")
        seqs = _log_int(rng, 1, 64)
        drafts = _log_int(rng, 1, 64)
        group = rng.choice([1, 2, 3, 4, 7, 8])
        most = 100_000_000 // (seqs * heads * group * drafts)  # scores of the plain form
        tokens = _log_int(rng, 1, max(1, min(50_000, most, 200_000 // seqs)))
        case = _tree("", seqs, tokens, drafts, heads * group, heads, page_tokens=page, ragged=rng.random() < 0.6,
                     **kind)
    del case["name"]
    return case


def _ceil(a, b):
    return -(-a // b)


def _lengths(c):
    """Committed and drafted tokens of each sequence of a tree case: the same for every seed."""
    rng = random.Random(c["seqs"] * 1000003 + c["tokens"])
    if not c["ragged"]:
        return [c["tokens"]] * c["seqs"], [c["drafts"]] * c["seqs"]
    lens = [max(1, int(c["tokens"] * rng.uniform(0.05, 1.0))) for _ in range(c["seqs"])]
    return lens, [rng.randint(1, c["drafts"]) for _ in range(c["seqs"])]


def _capacities(c):
    """Two capacities in tokens for each slot of a resize case; the moving slots swap full and freed."""
    rng = random.Random(c["slots"] * 1000003 + c["width"])
    a, b = [], []
    for _ in range(c["slots"]):
        tokens = max(1, int(c["width"] * c["page_tokens"] * rng.uniform(0.2, 0.9)))
        if rng.random() < c["moving"]:
            one, two = rng.choice([(tokens, 0), (0, tokens), (tokens, tokens // 2)])
        else:  # a slot that goes on: a page more now and then
            one, two = tokens, min(tokens + rng.randint(0, 1) * c["page_tokens"], c["width"] * c["page_tokens"])
        a.append(one)
        b.append(two)
    return a, b


def work(case):
    c = case
    row = c.get("kv_heads", 0) * c.get("head_dim", 0) * 2 * 2  # bytes of a token's keys and values in a layer
    if c["op"] == "copy":
        share = 0.5 if c["partial"] else 1.0
        return {"bytes": 2 * c["pairs"] * c["page_tokens"] * share * row * c["layers"] + 12 * c["pairs"], "flops": 0}
    if c["op"] == "resize":
        a, b = _capacities(c)
        p = c["page_tokens"]
        moved = sum(abs(_ceil(x, p) - _ceil(y, p)) for x, y in zip(a, b))
        # Each page that changes hands: its table entry written or read, its count read and written, twice a pass.
        return {"bytes": 2 * (12 * moved + 16 * c["slots"]), "flops": 0}
    if c["op"] == "fork":
        slots = c["groups"] * c["beams"]
        pages = _ceil(c["tokens"] + 1, c["page_tokens"])
        tail = c["tokens"] % c["page_tokens"]
        copies = slots * (1 - 1 / c["beams"]) ** c["beams"]  # beams that are no row's first child, on average
        # Rows read and written, a count for each entry read and written, tails copied.
        return {"bytes": slots * (16 * pages + 24) + 2 * copies * tail * row * c["layers"], "flops": 0}
    if c["op"] == "compact":
        return {"bytes": c["slots"] * c["keep"] * (2 * row * c["layers"] + 4), "flops": 0}
    lens, drafts = _lengths(c)
    rows = sum(drafts)
    cache = sum(n + t for n, t in zip(lens, drafts)) * row
    scores = sum(t * (n + t) for n, t in zip(lens, drafts)) * c["q_heads"]
    return {"bytes": cache + rows * c["q_heads"] * (c["head_dim"] * 4 + 4), "flops": 4 * scores * c["head_dim"]}


# ---------------------------------------------------------------------------
# What a program has in hand
# ---------------------------------------------------------------------------
def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _pools(c, pages, layers, gen):
    p, h, d = c["page_tokens"], c["kv_heads"], c["head_dim"]
    shape = (layers, pages, p, h, d) if c["layout"] == "NHD" else (layers, pages, h, p, d)
    return [torch.randn(shape, generator=gen, device=DEV, dtype=DTYPES[c["dtype"]]) for _ in "kv"]


def _tokens_first(pool, c):
    """The pool as [layers, pages, tokens, heads, dim], whatever its layout."""
    return pool if c["layout"] == "NHD" else pool.permute(0, 1, 3, 2, 4)


def _rows(held, width, pages, gen):
    """A page table whose slots hold `held` pages each, scattered over the pool."""
    held = torch.tensor(held, device=DEV)
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    at = torch.arange(width, device=DEV)
    index = (held.cumsum(0) - held)[:, None] + at
    return torch.where(at < held[:, None], order[index.clamp(max=pages - 1)], -1)


def _counts(table, pages):
    """How many table entries name each page."""
    named = torch.where(table >= 0, table, pages).flatten().long()
    return torch.zeros(pages + 1, dtype=torch.int32, device=DEV).scatter_add_(
        0, named, torch.ones_like(named, dtype=torch.int32))[:pages].contiguous()


def _trees(c, drafts, gen_cpu):
    """Packed ancestor masks of random trees, [rows, words]: bit j of row i for draft j."""
    n, t = c["seqs"], max(drafts)
    words = _ceil(t, 32)
    parent = torch.stack([torch.zeros(n, dtype=torch.long)] + [
        torch.randint(-1, i, (n,), generator=gen_cpu) for i in range(1, t)], 1)
    parent[:, 0] = -1
    seen = torch.zeros(n, t + 1, words * 32, dtype=torch.bool)  # row t stands for "no parent"
    every = torch.arange(n)
    for i in range(t):
        seen[:, i] = seen[every, parent[:, i] % (t + 1)]
        seen[:, i, i] = True
    bits = (seen[:, :t].view(n, t, words, 32).long() << torch.arange(32)).sum(-1)
    bits = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32)
    return torch.cat([bits[b, :drafts[b]] for b in range(n)]).to(DEV)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": c, "op": c["op"]}
    p = c["page_tokens"]
    if c["op"] == "copy":
        s["k"], s["v"] = _pools(c, c["pages"], c["layers"], gen)
        order = torch.randperm(c["pages"], generator=gen, device=DEV).to(torch.int32)
        s["src"], s["dst"] = order[:c["pairs"]].contiguous(), order[c["pairs"]:2 * c["pairs"]].contiguous()
        s["tokens"] = torch.randint(0, p + 1, (c["pairs"],), generator=gen, device=DEV,
                                    dtype=torch.int32) if c["partial"] else None
    elif c["op"] == "resize":
        a, b = _capacities(c)
        held = [_ceil(x, p) for x in b]
        pages = sum(max(_ceil(x, p), _ceil(y, p)) for x, y in zip(a, b)) + c["slots"]
        s["table"] = _rows(held, c["width"], pages, gen)
        s["held"], s["lens"], s["refs"] = _ints(held), _ints(b), _counts(s["table"], pages)
        s["capacity"], s["short"] = (_ints(a), _ints(b)), _ints([0])
    elif c["op"] == "fork":
        slots = c["groups"] * c["beams"]
        shared = c["tokens"] // p  # pages of the prompt that a group's beams share
        width = shared + 2
        pages = c["groups"] * shared + 4 * slots
        order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
        group = torch.arange(slots, device=DEV) // c["beams"]
        prompt = group[:, None] * shared + torch.arange(shared, device=DEV)
        private = c["groups"] * shared + 2 * torch.arange(slots, device=DEV)[:, None] + torch.arange(2, device=DEV)
        s["table"] = order[torch.cat([prompt, private], 1)].contiguous()
        s["held"], s["lens"] = _ints([width] * slots), _ints([c["tokens"]] * slots)
        s["refs"] = _counts(s["table"], pages)
        pick = torch.randint(0, c["beams"], (slots,), generator=gen, device=DEV)
        s["parents"] = (group * c["beams"] + pick).to(torch.int32)
        s["next"] = {n: torch.empty_like(s[n]) for n in ("table", "held", "lens")}
        s["k"], s["v"] = _pools(c, pages, c["layers"], gen)
        s["short"] = _ints([0])
    elif c["op"] == "compact":
        held = _ceil(c["start"] + c["span"], p)
        pages = held * c["slots"] + 16
        s["k"], s["v"] = _pools(c, pages, c["layers"], gen)
        s["table"] = _rows([held] * c["slots"], held, pages, gen)
        s["held"], s["lens"] = _ints([held] * c["slots"]), _ints([c["start"] + c["span"]] * c["slots"])
        s["refs"] = _counts(s["table"], pages)
        chosen = torch.rand(c["slots"], c["span"], generator=gen, device=DEV).argsort(1)[:, :c["keep"]]
        s["keep"] = chosen.sort(1).values.to(torch.int32)
        s["start"] = _ints([c["start"]] * c["slots"])
        s["count"] = torch.randint((c["keep"] + 1) // 2, c["keep"] + 1, (c["slots"],), generator=gen,
                                   device=DEV, dtype=torch.int32)
        s["status"] = _ints([0] * c["slots"])
    else:
        lens, drafts = _lengths(c)
        held = [_ceil(n + t, p) for n, t in zip(lens, drafts)]
        pages = sum(held) + 8
        s["k"], s["v"] = _pools(c, pages, 1, gen)
        s["table"] = _rows(held, max(held), pages, gen)
        s["held"], s["lens"], s["refs"] = _ints(held), _ints(lens), _counts(s["table"], pages)
        rows = sum(drafts)
        s["q"] = torch.randn(rows, c["q_heads"], c["head_dim"], generator=gen, device=DEV, dtype=DTYPES[c["dtype"]])
        s["q_start"] = _ints([sum(drafts[:b]) for b in range(c["seqs"] + 1)])
        s["mask"] = _trees(c, drafts, torch.Generator().manual_seed(seed))
        s["scale"] = c["head_dim"] ** -0.5
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(rows, c["q_heads"], device=DEV)
        s["most"] = (max(n + t for n, t in zip(lens, drafts)), max(drafts))  # a program knows its longest sequence and tree
    if own:
        _handles(s)
    return s


def _handles(s):
    """The context, the cache's description and the workspace that a program keeps."""
    from copy_reduce_dst_gb300 import tb
    c = s["case"]
    s["ctx"] = tb.Context(0)
    pools = {n: s.get(n) for n in ("k", "v")}
    s["cache"] = tb.kv_cache(**pools, table=s.get("table"), held=s.get("held"), lens=s.get("lens"),
                             refs=s.get("refs"), layout=c.get("layout", "NHD"), page_tokens=c["page_tokens"])
    if c["op"] == "fork":  # the table that the next step forks
        n = s["next"]
        s["next_cache"] = tb.kv_cache(**pools, table=n["table"], held=n["held"], lens=n["lens"], refs=s["refs"],
                                      layout=c["layout"], page_tokens=c["page_tokens"])
    if c["op"] == "tree":
        need = s["ctx"].tree_attention_workspace(s["cache"], c["q_heads"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV)


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    s = state
    return (_run_own if own else _run_plain)[s["op"]](s)


def _bits(pool):
    """A pool's bits as whole numbers: what is only moved has to arrive as it was."""
    return pool.view(torch.int32)


def _stream():
    return torch.cuda.current_stream()


def _own_copy(s):
    s["ctx"].kv_copy_pages(s["cache"], s["src"], s["dst"], s["case"]["pairs"], tokens=s["tokens"], stream=_stream())
    return {"k": _bits(s["k"]), "v": _bits(s["v"])}


def _plain_copy(s):
    c = s["case"]
    src, dst = s["src"].long(), s["dst"].long()
    for name in ("k", "v"):
        pool = _tokens_first(s[name], c)
        moved = pool[:, src]
        if s["tokens"] is not None:
            taken = torch.arange(c["page_tokens"], device=DEV) < s["tokens"][:, None]
            moved = torch.where(taken[None, :, :, None, None], moved, pool[:, dst])
        pool[:, dst] = moved
    return {"k": _bits(s["k"]), "v": _bits(s["v"])}


def _own_resize(s):
    for capacity in s["capacity"]:
        s["ctx"].kv_resize(s["cache"], capacity, s["short"], stream=_stream())
    return {n: s[n] for n in ("table", "held", "lens", "refs", "short")}


def _plain_resize(s):
    table, held, refs = s["table"], s["held"], s["refs"]
    at = torch.arange(table.shape[1], device=DEV)
    idle = torch.arange(table.numel(), device=DEV).view_as(table) % refs.numel()  # where an unchanged entry adds 0
    for capacity in s["capacity"]:
        need = torch.where(capacity < 0, held, (capacity + s["case"]["page_tokens"] - 1) // s["case"]["page_tokens"])
        grow = (need - held).clamp(min=0)
        short = (grow.sum() - (refs == 0).sum()).clamp(min=0)
        s["short"].copy_(short)
        need, grow = torch.where(short > 0, held, need), torch.where(short > 0, 0, grow)
        free = torch.argsort((refs > 0).to(torch.int8), stable=True)  # the lowest free pages first
        new = (at >= held[:, None]) & (at < need[:, None])
        gone = (at >= need[:, None]) & (at < held[:, None])
        rank = (grow.cumsum(0) - grow)[:, None] + at - held[:, None]
        refs.scatter_add_(0, torch.where(gone, table, idle).flatten(), -gone.flatten().to(torch.int32))
        taken = torch.where(new, free[rank.clamp(0, free.numel() - 1)], idle)
        refs.scatter_add_(0, taken.flatten(), new.flatten().to(torch.int32))
        table.copy_(torch.where(new, taken.to(torch.int32), torch.where(gone, -1, table)))
        held.copy_(need)
        s["lens"].copy_(torch.where((capacity < 0) | (short > 0), s["lens"], torch.minimum(s["lens"], capacity)))
    return {n: s[n] for n in ("table", "held", "lens", "refs", "short")}


def _forked(s):
    s["table"], s["held"], s["lens"], s["next"] = (*s["next"].values(), {n: s[n] for n in ("table", "held", "lens")})
    names = ("table", "held", "lens", "refs", "short")
    return {**{n: s[n] for n in names}, "k": _bits(s["k"]), "v": _bits(s["v"])}


def _own_fork(s):
    n = s["next"]
    s["ctx"].kv_fork(s["cache"], s["parents"], n["table"], n["held"], n["lens"], s["short"], stream=_stream())
    s["cache"], s["next_cache"] = s["next_cache"], s["cache"]
    return _forked(s)


def _plain_fork(s):
    c, n = s["case"], s["next"]
    p, table, held, lens, refs = c["page_tokens"], s["table"], s["held"], s["lens"], s["refs"]
    slots, width = table.shape
    at, every = torch.arange(width, device=DEV), torch.arange(slots, device=DEV)
    lives, parent = s["parents"] >= 0, s["parents"].clamp(min=0).long()
    children = torch.zeros(slots, dtype=torch.int32, device=DEV).scatter_add_(0, parent, lives.to(torch.int32))
    # The slot itself, else the first child, goes on with a row's last page and its spare ones.
    claim = torch.where(lives, torch.where(parent == every, -1, every), slots)
    first = torch.full((slots,), slots, device=DEV).scatter_reduce_(0, parent, claim, "amin")
    heir = lives & (claim == first[parent])
    full, tail = (lens // p)[parent], (lens % p)[parent]
    fresh = lives & ~heir & (tail > 0)
    short = (fresh.sum() - (refs == 0).sum()).clamp(min=0)
    s["short"].copy_(short)
    free = torch.argsort((refs > 0).to(torch.int8), stable=True)
    count = fresh.cumsum(0)
    rank = torch.where(fresh, count - 1, count[-1] + (~fresh).cumsum(0) - 1)
    page = free[rank]  # a page of its own for each slot; those that need none leave it as it is
    # Pages before the last part-filled one gain a holder for each child but one; the others pass to the heir.
    change = torch.where(at < (lens // p)[:, None], (children - 1)[:, None], torch.where(children == 0, -1, 0)[:, None])
    change = torch.where((at < held[:, None]) & (short == 0), change, 0)
    used = torch.where(at < held[:, None], table, 0).long()
    refs.scatter_add_(0, used.flatten(), change.flatten().to(torch.int32))
    refs.scatter_add_(0, page, (fresh & (short == 0)).to(torch.int32))
    keep = torch.where(heir, held[parent], full + (tail > 0))
    row = torch.where(at < keep[:, None], table[parent], -1)
    source = row.gather(1, full.clamp(max=width - 1).long()[:, None])[:, 0].clamp(min=0).long()
    row = torch.where(fresh[:, None] & (at == full[:, None]), page[:, None].to(torch.int32), row)
    row = torch.where(lives[:, None], row, -1)
    n["table"].copy_(torch.where(short > 0, table, row))
    n["held"].copy_(torch.where(short > 0, held, torch.where(lives, keep, 0)))
    n["lens"].copy_(torch.where(short > 0, lens, torch.where(lives, lens[parent], 0)))
    taken = (torch.arange(p, device=DEV) < tail[:, None]) & (fresh & (short == 0))[:, None]
    for name in ("k", "v"):
        pool = _tokens_first(s[name], c)
        pool[:, page] = torch.where(taken[None, :, :, None, None], pool[:, source], pool[:, page])
    return _forked(s)


def _own_compact(s):
    s["ctx"].kv_compact(s["cache"], s["start"], s["keep"], s["count"], s["status"], stream=_stream())
    return {"k": _bits(s["k"]), "v": _bits(s["v"]), "lens": s["lens"], "status": s["status"]}


def _plain_compact(s):
    c, p = s["case"], s["case"]["page_tokens"]
    index = torch.arange(s["keep"].shape[1], device=DEV)
    to = (s["start"][:, None] + index).long()
    at = (s["start"][:, None] + s["keep"]).long()
    kept = (index < s["count"][:, None])[None, :, :, None, None]
    from_page, to_page = s["table"].gather(1, at // p).long(), s["table"].gather(1, to // p).long()
    for name in ("k", "v"):
        pool = _tokens_first(s[name], c)
        pool[:, to_page, to % p] = torch.where(kept, pool[:, from_page, at % p], pool[:, to_page, to % p])
    s["lens"].copy_(s["start"] + s["count"])
    return {"k": _bits(s["k"]), "v": _bits(s["v"]), "lens": s["lens"], "status": s["status"]}


def _own_tree(s):
    s["ctx"].tree_attention(s["cache"], 0, s["q"], s["q_start"], s["mask"], s["out"], s["workspace"],
                            scale=s["scale"], lse=s["lse"], stream=_stream())
    return {"out": s["out"], "lse": s["lse"]}


def _plain_tree(s):
    c = s["case"]
    longest, t = s["most"]
    heads, group, d = c["kv_heads"], c["q_heads"] // c["kv_heads"], c["head_dim"]
    lens, q_start = s["lens"].long(), s["q_start"].long()
    drafts = q_start[1:] - q_start[:-1]
    # Keys and values of every position, [seqs, heads, positions, dim].
    where = torch.arange(longest, device=DEV)
    page = s["table"][:, where // c["page_tokens"]].clamp(min=0).long()
    key, value = (_tokens_first(s[n], c)[0][page, where % c["page_tokens"]].transpose(1, 2).float() for n in ("k", "v"))
    rows = q_start[:-1, None] + torch.arange(t, device=DEV)
    real = torch.arange(t, device=DEV) < drafts[:, None]
    rows = torch.where(real, rows, 0)
    query = s["q"].float()[rows].view(-1, t, heads, group, d).permute(0, 2, 3, 1, 4)
    scores = (query.reshape(-1, heads, group * t, d) @ key.transpose(2, 3)).view(-1, heads, group, t, longest)
    # A committed position is seen by every row, a drafted one where the row's bit says so.
    bits = ((s["mask"][..., None] >> torch.arange(32, device=DEV)) & 1).flatten(1).bool()[rows]
    draft = where - lens[:, None]
    seen = bits.gather(2, draft.clamp(0, t - 1)[:, None].expand(-1, t, -1)) & (draft < drafts[:, None])[:, None]
    seen = (seen | (draft < 0)[:, None])[:, None, None]
    scores = torch.where(seen, scores * s["scale"], -math.inf)
    top = scores.amax(-1, keepdim=True)
    weight = torch.exp(scores - torch.where(top > -math.inf, top, 0.0))
    total = weight.sum(-1, keepdim=True)
    value = torch.where((draft < drafts[:, None])[:, None, :, None], value, 0.0)
    mixed = (weight.view(-1, heads, group * t, longest) @ value).view(-1, heads, group, t, d)
    mixed = mixed / torch.where(total > 0, total, 1.0)
    seq = torch.bucketize(torch.arange(s["q"].shape[0], device=DEV), q_start[1:], right=True)
    at = torch.arange(s["q"].shape[0], device=DEV) - q_start[seq]
    mixed = mixed.permute(0, 3, 1, 2, 4)[seq, at]
    lse = (top + total.log())[..., 0].permute(0, 3, 1, 2)[seq, at]
    s["out"].copy_(mixed.reshape(s["out"].shape))
    s["lse"].copy_(lse.reshape(s["lse"].shape))
    return {"out": s["out"], "lse": s["lse"]}


_run_own = {"copy": _own_copy, "resize": _own_resize, "fork": _own_fork, "compact": _own_compact, "tree": _own_tree}
_run_plain = {"copy": _plain_copy, "resize": _plain_resize, "fork": _plain_fork, "compact": _plain_compact,
              "tree": _plain_tree}


def exact(case, seed):
    """The tree attention in 64 bits, one sequence and cache head at a time."""
    if case["op"] != "tree":
        return None
    s = prepare(case, seed)
    lens, drafts = _lengths(case)
    p, group = case["page_tokens"], case["q_heads"] // case["kv_heads"]
    out, lse = s["out"].double(), s["lse"].double()
    first = 0
    for b, (n, t) in enumerate(zip(lens, drafts)):
        pages = s["table"][b, :_ceil(n + t, p)].long()
        mask = s["mask"][first:first + t]
        tree = torch.stack([(mask[:, j // 32] >> (j % 32)) & 1 for j in range(t)], 1).bool()
        hidden = torch.cat([torch.zeros(t, n, dtype=torch.bool, device=DEV), ~tree], 1)
        for h in range(case["kv_heads"]):
            pool = [s[x][0][pages, :, h] if case["layout"] == "NHD" else s[x][0][pages, h] for x in ("k", "v")]
            key, value = (x.reshape(-1, case["head_dim"])[:n + t].double() for x in pool)
            heads = slice(h * group, (h + 1) * group)
            query = s["q"][first:first + t, heads].double()
            logits = torch.einsum("tgd,nd->tgn", query, key) * s["scale"]
            logits = logits.masked_fill(hidden[:, None], -math.inf)
            lse[first:first + t, heads] = torch.logsumexp(logits, -1)
            out[first:first + t, heads] = torch.einsum("tgn,nd->tgd", torch.softmax(logits, -1), value)
        first += t
    return {"out": out, "lse": lse}
