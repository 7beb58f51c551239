"""One verify step over a paged key/value cache: the attention of drafted
token trees, and what keeps the cache around it.

  attention  tree_attention: every drafted token attends to its sequence's
             cached context and to its own ancestors in the draft tree
  append     kv_append: new keys and values into the pages (bf16 or e4m3)
  commit     tree_accept, kv_compact: the greedy walk down the tree and the
             accepted rows moved to the end of the context, in every layer
  pages      kv_free, kv_fork, kv_reserve: rows of the page table dropped,
             branched off a sequence (the part-filled last page copied), and
             given room for the next tokens

`run` computes them in plain torch operations, or with `own` through the
package's entry points. Shapes: caches [pages, kv heads, page, dim] (with a
leading layer axis for commit and pages), q [tokens, heads, dim]; sequence b
owns tokens starts[b] .. starts[b+1], whose keys and values sit at positions
lengths[b], lengths[b] + 1, ... of its context.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _attention(name, batch, tree, heads, kv_heads, dim, context, page, e4m3=False, ragged=False):
    return {"name": name, "op": "attention", "batch": batch, "tree": tree, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "context": context, "page": page, "e4m3": e4m3, "ragged": ragged}


def _append(name, batch, tokens, kv_heads, dim, context, page, e4m3=False):
    return {"name": name, "op": "append", "batch": batch, "tokens": tokens, "kv_heads": kv_heads, "dim": dim,
            "context": context, "page": page, "e4m3": e4m3}


def _commit(name, batch, tree, layers, kv_heads, dim, context, page):
    return {"name": name, "op": "commit", "batch": batch, "tree": tree, "layers": layers, "kv_heads": kv_heads,
            "dim": dim, "context": context, "page": page}


def _pages(name, forks, layers, kv_heads, dim, context, page, pool):
    return {"name": name, "op": "pages", "forks": forks, "layers": layers, "kv_heads": kv_heads, "dim": dim,
            "context": context, "page": page, "pool": pool}


def listed():
    return [
        # one user's ordinary decode step early in a conversation: latency is all there is
        _attention("attn_decode_1x1_ctx257", 1, 1, 40, 8, 128, 257, 16),
        # one user's verify step: a 16-node draft tree over a document
        _attention("attn_verify_1x16_ctx8191", 1, 16, 40, 8, 128, 8191, 64),
        # a small server's verify step: users with drafts of 1 to 8 tokens and contexts of all ages
        _attention("attn_verify_12x8_ragged", 12, 8, 32, 8, 128, 4097, 32, ragged=True),
        # a full server's decode step over an 8-bit cache
        _attention("attn_decode_48x1_e4m3", 48, 1, 40, 8, 128, 16384, 64, e4m3=True, ragged=True),
        # one user, five drafted tokens, a very long context, wide heads
        _attention("attn_verify_1x5_ctx131071_d256", 1, 5, 24, 4, 256, 131071, 128),
        # wide trees (64 nodes) for many users: the arithmetic weighs as much as the cache
        _attention("attn_tree_16x64", 16, 64, 40, 8, 128, 4095, 64, ragged=True),
        # the verify step's own keys and values, one layer
        _append("append_12x8", 12, 8, 8, 128, 1500, 32),
        # eight prompts of 4,096 tokens into an 8-bit cache, one layer
        _append("append_8x4096_e4m3", 8, 4096, 8, 128, 77, 64, e4m3=True),
        # the end of one user's verify step, all layers
        _commit("commit_1x16_l32", 1, 16, 32, 8, 128, 2047, 16),
        # the same for a full server with wide trees
        _commit("commit_32x32_l48", 32, 32, 48, 8, 128, 200, 64),
        # four samples continued from one prompt
        _pages("pages_4_l32", 4, 32, 8, 128, 333, 16, 256),
        # beams re-branched on a full server
        _pages("pages_48_l32", 48, 32, 8, 128, 1000, 64, 512),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _unnamed(kind, *sizes):
    return {k: v for k, v in kind("", *sizes).items() if k != "name"}


def draw(rng):
    op = rng.choice(["attention"] * 5 + ["append", "append", "commit", "commit", "pages", "pages"])
    kv_heads, dim, page = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128, 128, 256]), rng.choice([16, 32, 64, 128])
    e4m3 = rng.random() < 0.3
    if op == "attention":
        group = rng.choice([1, 2, 3, 4, 5, 6, 8, 12])
        batch, tree, context = _log_int(rng, 1, 48), _log_int(rng, 1, 64), _log_int(rng, 1, 131071)
        # within the largest listed cases: 400 MB of bf16 cache, 30 GFLOP
        context = min(context, 400_000_000 // (batch * kv_heads * dim * 4))
        context = max(1, min(context, 30_000_000_000 // (4 * batch * tree * kv_heads * group * dim)))
        return _unnamed(_attention, batch, tree, kv_heads * group, kv_heads, dim, context, page, e4m3, rng.random() < 0.6)
    if op == "append":
        batch, tokens = _log_int(rng, 1, 48), _log_int(rng, 1, 4096)
        tokens = max(1, min(tokens, 24000 // batch))
        return _unnamed(_append, batch, tokens, kv_heads, dim, _log_int(rng, 1, 4000), page, e4m3)
    layers = _log_int(rng, 1, 40)
    if op == "commit":
        batch = _log_int(rng, 1, 32)
        context = _log_int(rng, 1, 2000)
        context = max(1, min(context, 200_000 // (batch * layers)))
        return _unnamed(_commit, batch, _log_int(rng, 1, 64), layers, kv_heads, dim, context, page)
    pool = max(64, min(_log_int(rng, 128, 4096), 1_000_000_000 // (layers * kv_heads * page * dim * 2)))
    forks = max(1, min(_log_int(rng, 1, 48), pool // 6))
    return _unnamed(_pages, forks, layers, kv_heads, dim, max(1, min(_log_int(rng, 1, 2000), page * (pool // 4))), page, pool)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _trees(rng, sizes):
    """Ancestor words (a node's own bit included) and parents of random draft trees, node 0 the root."""
    mask, parent = np.zeros(int(sizes.sum()), np.uint64), np.zeros(int(sizes.sum()), np.int64)
    at = 0
    for n in sizes:
        for i in range(int(n)):
            p = int(rng.integers(max(0, i - 4), i)) if i else -1
            parent[at + i] = p
            mask[at + i] = (mask[at + p] if i else np.uint64(0)) | (np.uint64(1) << np.uint64(i))
        at += int(n)
    return mask.view(np.int64), parent


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _cache(gen, shape, e4m3):
    """A cache's stored values and, for 8 bits, the float32 scale of each kv head."""
    if not e4m3:
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16), None
    codes = torch.empty(shape, device="cuda", dtype=torch.float8_e4m3fn)
    codes.copy_(torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16).mul_(80).clamp_(-E4M3_MAX, E4M3_MAX))
    return codes, torch.rand(shape[-3], generator=gen, device="cuda") * 0.01 + 0.01


def _sizes(case):
    """Per sequence: context length and number of new tokens (they go by the case, not by the seed)."""
    rng, n, top = np.random.default_rng(case["batch"]), case["batch"], case["context"]
    most = case["tokens"] if case["op"] == "append" else case["tree"]
    if case["op"] == "attention" and not case["ragged"]:
        return np.full(n, top, np.int64), np.full(n, most, np.int64)
    lengths = np.maximum(1, np.exp(rng.uniform(np.log(top / 8 + 1), np.log(top + 1), n)).astype(np.int64) - 1)
    new = rng.integers(1 if case["op"] == "attention" else (most + 1) // 2, most + 1, n)
    lengths[0], new[0] = top, most
    if case["op"] == "attention" and n >= 4 and most > 1:
        new[n // 2] = 0  # a sequence that sits this step out
    return lengths, new


def _table(rng, held, width, pool):
    """Page ids of each sequence (held[b] of them, the rest -1), scattered over the pool."""
    ids, table, at = rng.permutation(pool).astype(np.int32), np.full((len(held), width), -1, np.int32), 0
    for b, n in enumerate(held):
        table[b, :n] = ids[at:at + n]
        at += n
    return table


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    kv, dim, page = case["kv_heads"], case["dim"], case["page"]
    s = {"op": case["op"], "page": page}
    if case["op"] == "attention":
        lengths, sizes = _sizes(case)
        held = -(-(lengths + sizes) // page)
        table = _table(rng, held, int(held.max()), int(held.sum()) + 3)
        starts = np.concatenate([[0], np.cumsum(sizes)])
        mask, _ = _trees(rng, sizes)
        s["k_cache"], s["k_scale"] = _cache(gen, (int(held.sum()) + 3, kv, page, dim), case["e4m3"])
        s["v_cache"], s["v_scale"] = _cache(gen, (int(held.sum()) + 3, kv, page, dim), case["e4m3"])
        s |= {"q": randn(int(starts[-1]), case["heads"], dim), "table": _cuda(table), "mask": _cuda(mask),
              "lengths": _cuda(lengths.astype(np.int32)), "starts": _cuda(starts.astype(np.int32)), "tree": case["tree"]}
    elif case["op"] == "append":
        lengths, sizes = _sizes(case)
        held = -(-(lengths + sizes) // page)
        table = _table(rng, held, int(held.max()), int(held.sum()) + 3)
        s["k_cache"], s["k_scale"] = _cache(gen, (int(held.sum()) + 3, kv, page, dim), case["e4m3"])
        s["v_cache"], s["v_scale"] = _cache(gen, (int(held.sum()) + 3, kv, page, dim), case["e4m3"])
        rows = randn(int(sizes.sum()), 2 * kv, dim)  # the tail of a fused query/key/value product
        s |= {"k": rows[:, :kv], "v": rows[:, kv:], "table": _cuda(table), "lengths": _cuda(lengths.astype(np.int32)),
              "starts": _cuda(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32))}
    elif case["op"] == "commit":
        n, tree = case["batch"], case["tree"]
        lengths, sizes = _sizes(case)
        held = -(-(lengths + sizes) // page)
        table = _table(rng, held, int(held.max()), int(held.sum()) + 3)
        starts = np.concatenate([[0], np.cumsum(sizes)])
        mask, parent = _trees(rng, sizes)
        draft, target = rng.integers(0, 248320, len(mask)), rng.integers(0, 248320, len(mask))
        for b in range(n):  # the model agrees with some child of most nodes
            for i in range(1, int(sizes[b])):
                if rng.random() < 0.6:
                    target[starts[b] + parent[starts[b] + i]] = draft[starts[b] + i]
        shape = (case["layers"], int(held.sum()) + 3, kv, page, dim)
        s |= {"k_cache": randn(*shape), "v_cache": randn(*shape), "table": _cuda(table), "mask": _cuda(mask),
              "draft": _cuda(draft), "target": _cuda(target), "lengths": _cuda(lengths.astype(np.int32)),
              "starts": _cuda(starts.astype(np.int32)), "tree": tree}
    else:
        # rows: sources (a few shared prompts), then one row per branch, each now holding an older branch
        forks, pool = case["forks"], case["pool"]
        prompts = max(1, forks // 8)
        sized = np.random.default_rng(forks)  # lengths go by the case, not by the seed
        lengths = np.concatenate([sized.integers(max(1, case["context"] // 2), case["context"] + 1, prompts),
                                  sized.integers(1, page + 1, forks)])
        room = (pool // 2 - forks) // prompts  # pages a prompt may hold, so that every branch finds room
        lengths[:prompts] = np.minimum(lengths[:prompts], page * max(1, room))
        held = -(-lengths // page)
        width = int(held.max()) + 2
        table = _table(rng, held, width, pool)
        refs = np.zeros(pool, np.int32)
        np.add.at(refs, table[table >= 0], 1)
        dst = (prompts + rng.permutation(forks)).astype(np.int32)
        src = rng.integers(0, prompts, forks).astype(np.int32)
        shape = (case["layers"], pool, kv, page, dim)
        s |= {"k_cache": randn(*shape), "v_cache": randn(*shape), "table": _cuda(table), "refs": _cuda(refs),
              "lengths": _cuda(lengths.astype(np.int32)), "src": _cuda(src), "dst": _cuda(dst),
              "want": _cuda((lengths[src] + rng.integers(1, 17, forks)).astype(np.int32))}
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _own(s)
    return {"attention": _plain_attention, "append": _plain_append, "commit": _plain_commit, "pages": _plain_pages}[s["op"]](s)


def _own(s):
    import gemm_w4a16_group_gb300 as w4
    if s["op"] == "attention":
        return w4.tree_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["starts"], s["mask"],
                                 s["tree"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    if s["op"] == "append":
        w4.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["starts"],
                     k_scale=s["k_scale"], v_scale=s["v_scale"])
        return s["k_cache"], s["v_cache"]
    if s["op"] == "commit":
        path, count, token = w4.tree_accept(s["target"], s["draft"], s["mask"], s["starts"], s["tree"])
        lengths = w4.kv_compact(s["k_cache"], s["v_cache"], s["table"], s["lengths"], path, count)
        return path, count, token, lengths, s["k_cache"], s["v_cache"]
    w4.kv_free(s["table"], s["lengths"], s["refs"], s["dst"])
    forked = w4.kv_fork(s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["refs"], s["src"], s["dst"])
    grown = w4.kv_reserve(s["table"], s["refs"], s["dst"], s["want"], s["page"])
    return forked, grown, s["table"], s["lengths"], s["refs"], s["k_cache"], s["v_cache"]


def _owners(starts, tokens):
    """Sequence and index within it of every token."""
    at = torch.arange(tokens, device=starts.device)
    seq = torch.searchsorted(starts[1:].contiguous(), at.to(starts.dtype), right=True)
    return seq, at - starts[seq]


def _by_position(cache, scale, table):
    """A paged cache as float32 [sequences, kv heads, positions, dim]."""
    x = cache.view(torch.uint8)[table.clamp(min=0).long()].view(cache.dtype) if scale is not None else cache[table.clamp(min=0).long()]
    x = x.transpose(1, 2).flatten(2, 3).float()
    return x if scale is None else x * scale[None, :, None, None]


def _plain_attention(s):
    q, table, lengths, starts, mask, page, tree = (s[k] for k in ("q", "table", "lengths", "starts", "mask", "page", "tree"))
    tokens, heads, dim = q.shape
    k, v = _by_position(s["k_cache"], s["k_scale"], table), _by_position(s["v_cache"], s["v_scale"], table)
    n, kv, top, _ = k.shape
    seq, node = _owners(starts, tokens)
    padded = torch.zeros((n, tree, heads, dim), device=q.device)
    padded[seq, node] = q.float()
    words = torch.zeros((n, tree), device=q.device, dtype=torch.int64)
    words[seq, node] = mask
    sizes = starts[1:] - starts[:-1]
    ahead = torch.arange(top, device=q.device)[None] - lengths[:, None]  # index among the new tokens
    new = (ahead >= 0) & (ahead < sizes[:, None])
    on = ((words[:, :, None] >> ahead.clamp(0, 63)[:, None, :]) & 1).bool()
    sees = (ahead < 0)[:, None, :] | (new[:, None, :] & on)  # [n, tree, positions]
    v = torch.where((ahead < sizes[:, None])[:, None, :, None], v, 0.0)
    group = heads // kv
    a = padded.view(n, tree, kv, group, dim).permute(0, 2, 1, 3, 4).reshape(n, kv, tree * group, dim)
    x = (a @ k.transpose(-1, -2)).view(n, kv, tree, group, top) * (1.0 / math.sqrt(dim))
    x = x.masked_fill(~sees[:, None, :, None, :], -math.inf)
    high = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(high == -math.inf, 0.0, high))
    total = x.sum(-1, keepdim=True)
    y = (x.view(n, kv, tree * group, top) @ v).view(n, kv, tree, group, dim) / torch.where(total == 0, 1.0, total)
    return y.permute(0, 2, 1, 3, 4).reshape(n, tree, heads, dim)[seq, node].to(q.dtype)


def _plain_append(s):
    seq, i = _owners(s["starts"], s["k"].shape[0])
    at = s["lengths"][seq] + i
    pages, rows = s["table"][seq, at // s["page"]].long(), at % s["page"]
    if s["k_scale"] is None:
        s["k_cache"][pages, :, rows] = s["k"]
        s["v_cache"][pages, :, rows] = s["v"]
    else:
        code = lambda x, scale: (x.float() / scale[None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)  # noqa: E731
        s["k_cache"].view(torch.uint8)[pages, :, rows] = code(s["k"], s["k_scale"]).view(torch.uint8)
        s["v_cache"].view(torch.uint8)[pages, :, rows] = code(s["v"], s["v_scale"]).view(torch.uint8)
    return s["k_cache"], s["v_cache"]


def _plain_commit(s):
    target, draft, starts, mask, tree, page = (s[k] for k in ("target", "draft", "starts", "mask", "tree", "page"))
    n = starts.numel() - 1
    seq, node = _owners(starts, mask.numel())
    pad = lambda x: torch.zeros((n, tree), device=x.device, dtype=x.dtype).index_put_((seq, node), x)  # noqa: E731
    words, drafts, targets = pad(mask), pad(draft), pad(target)
    sizes = starts[1:] - starts[:-1]
    idx = torch.arange(tree, device=mask.device)
    there = idx[None] < sizes[:, None]
    above = ((words[:, :, None] >> idx) & 1).bool() & (idx[None, :] < idx[:, None])  # [n, node, proper ancestor]
    parent = torch.where(above, idx, -1).amax(-1)
    fits = there & (parent >= 0) & (drafts == targets.gather(1, parent.clamp(min=0)))
    twin = fits[:, :, None] & fits[:, None, :] & (parent[:, :, None] == parent[:, None, :]) & (idx[None, :] < idx[:, None])
    fits = fits & ~twin.any(-1)  # of equal siblings the first
    root = idx == 0
    taken = there & (root | ((above | torch.eye(tree, dtype=torch.bool, device=mask.device)) & ~(fits | root)[:, None, :]).any(-1).logical_not() & above[:, :, 0])
    count = taken.sum(-1, dtype=torch.int32)
    order = torch.where(taken, idx, tree).sort(-1).values
    path = torch.where(order < tree, order, -1).to(torch.int32)
    last = torch.where(taken, idx, 0).amax(-1, keepdim=True)
    token = torch.where(count > 0, targets.gather(1, last)[:, 0], -1)
    rows = torch.arange(n, device=mask.device)[:, None]
    move = path >= 0
    # past the accepted rows the root's row, which stays where it is, once more
    at, to = s["lengths"][:, None] + path.clamp(min=0), s["lengths"][:, None] + torch.where(move, idx, 0)
    pa, ra, pt, rt = s["table"][rows, at // page].long(), at % page, s["table"][rows, to // page].long(), to % page
    s["k_cache"][:, pt, :, rt] = s["k_cache"][:, pa, :, ra]
    s["v_cache"][:, pt, :, rt] = s["v_cache"][:, pa, :, ra]
    return path, count, token, s["lengths"] + count, s["k_cache"], s["v_cache"]


def _plain_pages(s):
    table, lengths, refs, src, dst, page = (s[k] for k in ("table", "lengths", "refs", "src", "dst", "page"))
    src, dst, pool, width = src.long(), dst.long(), refs.numel(), table.shape[1]
    cols = torch.arange(width, device=table.device)
    # free
    old = table[dst]
    refs.index_add_(0, old.clamp(min=0).flatten().long(), -(old >= 0).flatten().to(torch.int32))
    table[dst], lengths[dst] = -1, 0
    # fork: whole pages are shared, the part-filled one is copied into the lowest free page
    size = lengths[src]
    full, rest = size // page, size % page
    part, old = rest > 0, table[src]
    shared = cols[None] < full[:, None]
    free = (refs == 0).cumsum(0)
    rank = part.cumsum(0)
    forked = (rank[-1:] <= free[-1:]).to(torch.int32)
    new = torch.searchsorted(free, rank).clamp(max=pool - 1)
    refs.index_add_(0, old.clamp(min=0).flatten().long(), (shared & (old >= 0)).flatten().to(torch.int32) * forked)
    refs.index_add_(0, new, part.to(torch.int32) * forked)
    mine = torch.where(shared, old, torch.where(part[:, None] & (cols[None] == full[:, None]), new[:, None].to(torch.int32), -1))
    table[dst] = torch.where(forked > 0, mine, table[dst])
    lengths[dst] = torch.where(forked > 0, size, lengths[dst])
    go = part & (forked > 0)
    last = old.gather(1, full[:, None].long().clamp(max=width - 1))[:, 0]
    from_page = torch.where(go, last, old[:, 0]).long()
    to_page = torch.where(go, new, from_page)  # a branch without a copy writes its first page back as it is
    here = (torch.arange(page, device=table.device)[None] < rest[:, None]) & go[:, None]
    here = here[None, :, None, :, None]
    s["k_cache"][:, to_page] = torch.where(here, s["k_cache"][:, from_page], s["k_cache"][:, to_page])
    s["v_cache"][:, to_page] = torch.where(here, s["v_cache"][:, from_page], s["v_cache"][:, to_page])
    # reserve: the lowest free pages, row after row
    have = (table[dst] >= 0).sum(-1)
    more = ((s["want"] + page - 1) // page - have).clamp(min=0)
    ends = more.cumsum(0)
    free = (refs == 0).cumsum(0)
    grown = (ends[-1:] <= free[-1:]).to(torch.int32)
    k = cols[None] - have[:, None]
    gets = (k >= 0) & (k < more[:, None]) & (grown > 0)
    got = torch.searchsorted(free, (ends - more)[:, None] + k.clamp(min=0) + 1).clamp(max=pool - 1)
    table[dst] = torch.where(gets, got.to(torch.int32), table[dst])
    refs.index_add_(0, got.flatten(), gets.flatten().to(torch.int32))
    return forked, grown, table, lengths, refs, s["k_cache"], s["v_cache"]


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its results in 64 bits
# ---------------------------------------------------------------------------
def work(case):
    kv, dim, elt = case["kv_heads"], case["dim"], 1 if case.get("e4m3") else 2
    if case["op"] == "attention":
        lengths, sizes = _sizes(case)
        live = sizes > 0
        keys, pairs = int(((lengths + sizes) * live).sum()), int(((lengths + sizes / 2) * sizes).sum())
        tokens = int(sizes.sum())
        return {"bytes": keys * kv * dim * 2 * elt + tokens * (case["heads"] * dim * 4 + 8), "flops": 4 * pairs * case["heads"] * dim}
    if case["op"] == "append":
        return {"bytes": int(_sizes(case)[1].sum()) * kv * dim * 2 * (2 + elt), "flops": 0}
    if case["op"] == "commit":  # about two accepted rows of a sequence change place
        return {"bytes": case["batch"] * (case["tree"] * 32 + 2 * case["layers"] * kv * dim * 2 * 2 * 2), "flops": 0}
    half = (case["page"] + 1) // 2
    return {"bytes": case["pool"] * 4 + case["forks"] * (case["context"] // case["page"] + 1) * 12 + case["forks"] * case["layers"] * kv * half * dim * 2 * 2 * 2,
            "flops": 0}


def exact(case, seed):
    """Attention from its definition, and the 8-bit rows of an append before their rounding; the rest moves values and counts."""
    if case["op"] == "append" and case["e4m3"]:
        s = prepare(case, seed)
        out = []
        for new, cache, scale in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
            want = cache.double()
            starts, lengths, table = s["starts"].tolist(), s["lengths"].tolist(), s["table"].long()
            for b in range(len(lengths)):
                pos = torch.arange(lengths[b], lengths[b] + starts[b + 1] - starts[b], device="cuda")
                rows = new[starts[b]:starts[b + 1]].double() / scale.double()[:, None]
                want[table[b, pos // s["page"]], :, pos % s["page"]] = rows.clamp(-E4M3_MAX, E4M3_MAX)
            out.append(want)
        return tuple(out)
    if case["op"] != "attention":
        return None
    s = prepare(case, seed)
    q, page = s["q"].double(), s["page"]
    starts, lengths = s["starts"].tolist(), s["lengths"].tolist()
    out = torch.zeros_like(q)
    group = q.shape[1] // case["kv_heads"]
    for b in range(len(lengths)):
        lo, hi = starts[b], starts[b + 1]
        if lo == hi:
            continue
        n = lengths[b] + hi - lo
        pos = torch.arange(n, device="cuda")
        ids = s["table"][b, :-(-n // page)].long()
        sees = torch.ones((hi - lo, n), dtype=torch.bool, device="cuda")
        words = s["mask"][lo:hi].cpu().numpy().view(np.uint64)
        bits = [[bool(int(w) >> j & 1) for j in range(hi - lo)] for w in words]
        sees[:, lengths[b]:] = torch.tensor(bits, device="cuda")
        for h in range(case["kv_heads"]):
            k, v = (c[ids, h].double().reshape(-1, case["dim"])[pos] * (1 if f is None else f[h].double())
                    for c, f in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])))
            for g in range(h * group, (h + 1) * group):
                x = (q[lo:hi, g] @ k.T / case["dim"] ** 0.5).masked_fill(~sees, -math.inf)
                out[lo:hi, g] = torch.nan_to_num(torch.softmax(x, -1)) @ v
    return out
