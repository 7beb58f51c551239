"""Plain implementations, in 64 bits and loops, of the paged-cache operators,
and the random steps that the tests run them on."""
import math

import numpy as np
import torch

E4M3 = torch.float8_e4m3fn
BF16 = torch.bfloat16


def random_tree(rng, n):
    """Ancestor words (uint64) of a random tree of n nodes, each under one of the four before it."""
    words = np.zeros(n, np.uint64)
    for i in range(n):
        above = words[int(rng.integers(max(0, i - 4), i))] if i else np.uint64(0)
        words[i] = above | np.uint64(1) << np.uint64(i)
    return words


def page_table(rng, held, width, pool):
    ids, table, at = rng.permutation(pool).astype(np.int32), np.full((len(held), width), -1, np.int32), 0
    for b, n in enumerate(held):
        table[b, :n] = ids[at:at + n]
        at += n
    return table


def new_cache(shape, e4m3, layout, gen, device):
    """A cache seen as [..., pages, heads, rows, dim] whose memory runs in `layout`: "hnd" (as seen), "nhd"
    (rows before heads) or "kv" (keys and values of a page side by side); and the scales of 8 bits."""
    *lead, pages, heads, rows, dim = shape

    def fill(s):
        x = torch.randn(s, generator=gen, dtype=torch.float32)
        return (x * 60).clamp(-448, 448).to(E4M3).to(device) if e4m3 else x.to(BF16).to(device)

    if layout == "hnd":
        k, v = fill(shape), fill(shape)
    elif layout == "nhd":
        k, v = (fill([*lead, pages, rows, heads, dim]).transpose(-2, -3) for _ in range(2))
    else:
        both = fill([*lead, pages, 2, heads, rows, dim])
        k, v = both.select(len(lead) + 1, 0), both.select(len(lead) + 1, 1)
    scale = (lambda: (torch.rand(heads, generator=gen) * 0.02 + 0.01).to(device)) if e4m3 else (lambda: None)
    return k, v, scale(), scale()


class Step:
    """Sequences with contexts `lengths` and `sizes` new tokens each, tensors on `device`."""

    def __init__(self, lengths, sizes, heads, kv_heads, dim, page, e4m3=False, layout="hnd", seed=0, spare=3, device="cuda",
                 masks=None, width_more=0):
        rng, gen = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
        self.lengths_h, self.sizes_h = np.asarray(lengths), np.asarray(sizes)
        held = -(-(self.lengths_h + self.sizes_h) // page)
        self.pool = int(held.sum()) + spare
        self.table_h = page_table(rng, held, max(1, int(held.max())) + width_more, self.pool)
        self.starts_h = np.concatenate([[0], np.cumsum(self.sizes_h)])
        self.tokens = int(self.starts_h[-1])
        self.words = np.concatenate([random_tree(rng, int(n)) for n in self.sizes_h]) if masks is None else masks
        self.heads, self.kv, self.dim, self.page, self.device = heads, kv_heads, dim, page, device
        self.k, self.v, self.ks, self.vs = new_cache((self.pool, kv_heads, page, dim), e4m3, layout, gen, device)
        self.q = torch.randn((self.tokens, heads, dim), generator=gen).to(BF16).to(device)
        to = lambda a, t: torch.from_numpy(np.ascontiguousarray(a)).to(t).to(device)  # noqa: E731
        self.table, self.lengths, self.starts = (to(a, torch.int32) for a in (self.table_h, self.lengths_h, self.starts_h))
        self.mask = to(self.words.view(np.int64), torch.int64)
        self.max_tree = max(1, int(self.sizes_h.max()))

    def slots(self, b, upto):
        """Page ids and rows of positions 0 .. upto - 1 of row b."""
        pos = np.arange(upto)
        return (torch.from_numpy(self.table_h[b, pos // self.page].astype(np.int64)).to(self.device),
                torch.from_numpy(pos % self.page).to(self.device))

    def sees(self, b, chain=False):
        """bool [sizes[b], lengths[b] + sizes[b]]"""
        n, at = int(self.sizes_h[b]), int(self.starts_h[b])
        s = np.ones((n, int(self.lengths_h[b]) + n), bool)
        for i in range(n):
            for j in range(n):
                s[i, int(self.lengths_h[b]) + j] = j <= i if chain else bool(int(self.words[at + i]) >> j & 1)
        return torch.from_numpy(s).to(self.device)

    def attention(self, scale=None, chain=False):
        """float64 result and, per element, sum_j p_j |v_j|. Only seen keys and values are read."""
        out = torch.zeros((self.tokens, self.heads, self.dim), dtype=torch.float64, device=self.device)
        mag = torch.zeros_like(out)
        group = self.heads // self.kv
        scale = 1 / math.sqrt(self.dim) if scale is None else scale
        for b in range(len(self.lengths_h)):
            n, lo = int(self.sizes_h[b]), int(self.starts_h[b])
            if n == 0:
                continue
            ids, rows = self.slots(b, int(self.lengths_h[b]) + n)
            sees = self.sees(b, chain)
            any_sees = sees.any(0)
            for h in range(self.kv):
                k = self.k.float()[ids, h, rows].double() if self.k.dtype == E4M3 else self.k[ids, h, rows].double()
                v = self.v.float()[ids, h, rows].double() if self.v.dtype == E4M3 else self.v[ids, h, rows].double()
                if self.ks is not None:
                    k, v = k * self.ks[h].double(), v * self.vs[h].double()
                for g in range(h * group, (h + 1) * group):
                    for i in range(n):
                        w = sees[i] & any_sees
                        if not w.any():
                            continue
                        s = k[w] @ self.q[lo + i, g].double() * scale
                        p = torch.exp(s - s.max())
                        p = p / p.sum()
                        out[lo + i, g] = p @ v[w]
                        mag[lo + i, g] = p @ v[w].abs()
        return out, mag


def attention_bound(ref, mag):
    """The result is rounded once to bf16 (2^-8 relative), and a weight e^(s - m) may be (2^-8 relative each, against
    a sum of unrounded ones); float32 scores, exponentials and sums add less than 2^-12 of the weighted magnitudes."""
    return 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -12) * mag + 1e-30


def greedy(words, draft, target):
    """Accepted nodes of one tree, by walking down."""
    n = len(words)
    path = [0] if n else []
    while path:
        step = None
        for c in range(path[-1] + 1, n):
            above = [a for a in range(c) if int(words[c]) >> a & 1]
            if above and above[-1] == path[-1] and draft[c] == target[path[-1]]:
                step = c
                break
        if step is None:
            break
        path.append(step)
    return path


class Table:
    """A page table and its pool on the host: free, fork and reserve as the header describes them."""

    def __init__(self, table, lengths, refs, page):
        self.table, self.lengths, self.refs, self.page = table.copy(), lengths.copy(), refs.copy(), page

    def free(self, rows):
        for b in rows:
            for c, id_ in enumerate(self.table[b]):
                if id_ >= 0:
                    self.refs[id_] -= 1
                    self.table[b, c] = -1
            self.lengths[b] = 0

    def _lowest(self, n):
        free = np.flatnonzero(self.refs == 0)
        return None if len(free) < n else list(free[:n])

    def fork(self, src, dst):
        """The pages to copy, [(from, to, rows)], or None."""
        part = [self.lengths[s] % self.page > 0 for s in src]
        new = self._lowest(sum(part))
        if new is None:
            return None
        copies = []
        for s, d, p in zip(src, dst, part):
            full = self.lengths[s] // self.page
            self.table[d, :full] = self.table[s, :full]
            np.add.at(self.refs, self.table[s, :full], 1)
            if p:
                id_ = new.pop(0)
                self.table[d, full] = id_
                self.refs[id_] = 1
                copies.append((int(self.table[s, full]), int(id_), int(self.lengths[s] % self.page)))
            self.lengths[d] = self.lengths[s]
        return copies

    def reserve(self, rows, want):
        more = [max(0, -(-w // self.page) - int((self.table[b] >= 0).sum())) for b, w in zip(rows, want)]
        new = self._lowest(sum(more))
        if new is None:
            return False
        for b, m in zip(rows, more):
            have = int((self.table[b] >= 0).sum())
            for i in range(m):
                self.table[b, have + i] = new[0]
                self.refs[new.pop(0)] = 1
        return True
