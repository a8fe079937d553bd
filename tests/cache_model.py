"""A plain model of the paged cache for the tests: loops over slots, pages and
tokens with whole numbers and copies only, and the tree attention in 64 bits.
It shares nothing with the library."""
import numpy as np

NONE = -1


class CacheModel:
    """k, v: [layers, pages, tokens, heads, dim] arrays; the rest as tb_kv_cache."""

    def __init__(self, k, v, table, held, lens, refs):
        self.k, self.v = k.copy(), v.copy()
        self.table, self.held, self.lens, self.refs = (x.copy() for x in (table, held, lens, refs))
        self.P = k.shape[2]

    def copy_pages(self, src, dst, tokens=None):
        for i, (s, d) in enumerate(zip(src, dst)):
            if not (0 <= s < self.refs.size and 0 <= d < self.refs.size):
                continue
            t = self.P if tokens is None else min(max(int(tokens[i]), 0), self.P)
            for pool in (self.k, self.v):
                pool[:, d, :t] = pool[:, s, :t]

    def _take(self, free):
        page = free.pop(0)
        self.refs[page] = 1
        return page

    def resize(self, capacity):
        width = self.table.shape[1]
        grow, need = [], []
        for s, cap in enumerate(capacity):
            n = int(self.held[s]) if cap < 0 else -(-int(cap) // self.P)
            if n > width:
                return -1
            if 0 <= cap < self.lens[s] and cap % self.P and self.refs[self.table[s, n - 1]] > 1:
                return -1
            need.append(n)
            grow.append(max(n - int(self.held[s]), 0))
        free = [p for p in range(self.refs.size) if self.refs[p] == 0]
        if sum(grow) > len(free):
            return sum(grow) - len(free)
        for s in range(len(need)):
            for j in range(int(self.held[s]), need[s]):
                self.table[s, j] = self._take(free)
        for s in range(len(need)):
            for j in range(need[s], int(self.held[s])):
                self.refs[self.table[s, j]] -= 1
                self.table[s, j] = NONE
            self.held[s] = need[s]
            if capacity[s] >= 0:
                self.lens[s] = min(self.lens[s], capacity[s])
        return 0

    def fork(self, parents):
        slots = len(parents)
        if any(p >= slots for p in parents):
            return -1
        children = [[s for s in range(slots) if parents[s] == p] for p in range(slots)]
        heir = [p if p in c else (c[0] if c else None) for p, c in enumerate(children)]
        needy = [s for s in range(slots) if parents[s] >= 0 and heir[parents[s]] != s
                 and self.lens[parents[s]] % self.P]
        free = [p for p in range(self.refs.size) if self.refs[p] == 0]
        if len(needy) > len(free):
            return len(needy) - len(free)
        fresh = {s: self._take(free) for s in needy}
        table = np.full_like(self.table, NONE)
        held, lens = np.zeros_like(self.held), np.zeros_like(self.lens)
        for s, p in enumerate(parents):
            if p < 0:
                continue
            n = int(self.lens[p])
            row = [int(x) for x in self.table[p, :self.held[p]]]
            if heir[p] != s:
                row = row[:-(-n // self.P)]
                if s in fresh:
                    for pool in (self.k, self.v):
                        pool[:, fresh[s], :n % self.P] = pool[:, row[-1], :n % self.P]
                    row[-1] = fresh[s]
            table[s, :len(row)] = row
            held[s], lens[s] = len(row), n
        self.table, self.held, self.lens = table, held, lens
        self.refs[:] = np.bincount(table[table >= 0], minlength=self.refs.size)
        return 0

    def compact(self, start, keep, count):
        status = np.zeros(len(start), np.int32)
        for s in range(len(start)):
            n, first = int(count[s]), int(start[s])
            if n < 0:
                continue
            room = int(self.held[s]) * self.P
            if n > keep.shape[1] or first < 0 or first + n > room:
                status[s] = 2
                continue
            ks = [int(x) for x in keep[s, :n]]
            if any(k < 0 or first + k >= room for k in ks) or any(a >= b for a, b in zip(ks, ks[1:])):
                status[s] = 2
                continue
            moved = [i for i, k in enumerate(ks) if k != i]
            since = (first + (moved[0] if moved else n)) // self.P
            if any(self.refs[p] > 1 for p in self.table[s, since:self.held[s]]):
                status[s] = 1
                continue
            for i, k in enumerate(ks):
                a, b = first + k, first + i
                pa, pb = self.table[s, a // self.P], self.table[s, b // self.P]
                for pool in (self.k, self.v):
                    pool[:, pb, b % self.P] = pool[:, pa, a % self.P]
            self.lens[s] = first + n
        return status


def tree_attention(q, k, v, table, lens, q_start, mask, scale, slots=None, only=None):
    """(out, lse, reach, logit): the attention of one layer's pools [pages,
    tokens, heads, dim] in 64 bits; reach = sum of p |v| per output element and
    logit = the largest scale * sum |q||k| of a row, for error bounds.  only:
    the rows wanted (default: all)."""
    rows, q_heads, dim = q.shape
    P, heads = k.shape[1], k.shape[2]
    group = q_heads // heads
    out, reach = np.zeros(q.shape), np.zeros(q.shape)
    lse, logit = np.full((rows, q_heads), -np.inf), np.zeros((rows, q_heads))
    for b in range(len(q_start) - 1):
        slot = b if slots is None else slots[b]
        r0, t = q_start[b], q_start[b + 1] - q_start[b]
        n = int(lens[slot])
        at = np.arange(n + t)
        page = table[slot, at // P]
        for i in range(t):
            if only is not None and r0 + i not in only:
                continue
            seen = [j for j in range(t) if j // 32 < mask.shape[1]
                    and int(mask[r0 + i, j // 32]) >> (j % 32) & 1]
            cols = np.concatenate([np.arange(n), n + np.array(seen, int)]).astype(int)
            if cols.size == 0:
                continue
            for h in range(q_heads):
                ks = k[page[cols], at[cols] % P, h // group].astype(np.float64)
                vs = v[page[cols], at[cols] % P, h // group].astype(np.float64)
                x = q[r0 + i, h].astype(np.float64)
                s = scale * (ks @ x)
                m = s.max()
                p = np.exp(s - m)
                total = p.sum()
                out[r0 + i, h] = p @ vs / total
                reach[r0 + i, h] = p @ np.abs(vs) / total
                lse[r0 + i, h] = m + np.log(total)
                logit[r0 + i, h] = abs(scale) * (np.abs(ks) @ np.abs(x)).max()
    return out, lse, reach, logit
