"""Plain implementations, in 64 bits or exact, of the sampled verify step and of the adapters."""
from fractions import Fraction

import numpy as np
import torch


def parents(words):
    """Parent of each node by its ancestor word, -1 where it has none."""
    out = []
    for i, w in enumerate(words):
        above = int(w) & ((1 << i) - 1)
        out.append(above.bit_length() - 1)
    return out


def sampled(p, q, draft, words, u, exact=True):
    """(path, token) of one tree: p, q [nodes, vocab] numpy float32 (q None), by the header's rules, in fractions or
    (exact=False) float64."""
    n = len(words)
    if n == 0:
        return [], -1
    num = (lambda x: Fraction(float(x))) if exact else float
    total = (lambda r: sum(r, Fraction(0))) if exact else (lambda r: float(np.sum(r)))

    def row(x):
        x = np.minimum(np.nan_to_num(np.maximum(np.nan_to_num(x, nan=0.0, posinf=1.0, neginf=0.0), 0.0)), 1.0)
        return [Fraction(float(v)) for v in x] if exact else x.astype(np.float64)

    def less(pr, qr, c):
        return [max(a - c * b, Fraction(0)) for a, b in zip(pr, qr)] if exact else np.maximum(pr - c * qr, 0.0)

    above = parents(words)
    path, vocab = [0], p.shape[1]
    while True:
        node = path[-1]
        pr = row(p[node])
        qr = row(q[node]) if q is not None else None
        c, s, step, asked, gone = num(0), num(1), None, 0, []
        for i in range(node + 1, n):
            x = int(draft[i])
            if above[i] != node or not 0 <= x < vocab:
                continue
            if q is not None:
                if asked:
                    s = total(less(pr, qr, c))
                left, chance = max(pr[x] - c * qr[x], num(0)), qr[x]
            else:
                if asked:
                    s = total([0 if j in gone else v for j, v in enumerate(pr)])
                left, chance = num(0) if x in gone else pr[x], num(1)
            if num(u[i]) * chance * s < left:
                step = i
                break
            c, asked = c + s, asked + 1
            gone.append(x)
        if step is None:
            break
        path.append(step)
    if q is not None and asked:
        w = less(pr, qr, c)
    else:
        w = list(pr)
        for x in gone:
            w[x] = num(0)
    if total(w) == 0:
        w = pr
    if total(w) == 0:
        return path, -1
    goal = min(max(num(u[0]), num(0)), num(np.float32(1 - 2.0 ** -24))) * total(w)
    if not exact:
        return path, int(np.argmax(np.cumsum(w) > goal))
    run = Fraction(0)
    for j, v in enumerate(w):
        run += v
        if run > goal:
            return path, j


def tree(rng, n, width=64):
    """Ancestor words (uint64) of a random tree, no node with more than `width` children."""
    words, kids = np.zeros(n, np.uint64), [0] * n
    for i in range(1, n):
        free = [j for j in range(i) if kids[j] < width]
        at = int(rng.choice(free[-6:]))
        kids[at] += 1
        words[i] = words[at]
        words[i] |= np.uint64(1) << np.uint64(i)
    if n:
        words |= np.uint64(1)
    return words


def adapted(y, x, a, b, which, scale):
    """float64 result and its error bound, from tensors and the adapter of every token (list).

    The result is rounded once to bf16 (2^-8). t = x A^T goes on in two bf16 parts, 2^-16 of it. A float32 sum of n terms
    is off by at most n 2^-23 of the terms' magnitudes (2^-23: the tensor cores cut where others round): inner / 16 sums
    of products and 64 parts in the first product, rank / 8 steps in the second, and the addition to y."""
    y, x, a, b = (v.double().cpu() for v in (y, x, a, b))
    out, bound = y.clone(), 0 * y
    inner, rank = x.shape[1], a.shape[1]
    for t, e in enumerate(which):
        if e < 0:
            continue
        s = 1.0 if scale is None else float(scale[e])
        low = a[e] @ x[t]
        mag = a[e].abs() @ x[t].abs()
        out[t] = y[t] + s * (b[e] @ low)
        wide = abs(s) * (b[e].abs() @ mag)
        bound[t] = 2.0 ** -8 * out[t].abs() + 2.0 ** -15 * abs(s) * (b[e].abs() @ low.abs()) \
            + 2.0 ** -23 * (inner / 16 + rank / 8 + 72) * wide + 2.0 ** -23 * y[t].abs() + 1e-36
    return out, bound


def stored(gen, *shape, std=1.0):
    return (torch.randn(shape, generator=gen) * std).to(torch.bfloat16)
