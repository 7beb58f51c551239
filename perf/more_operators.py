"""The sampled verify step of users with adapters of their own: what joins the
greedy one of operators.py.

  probabilities  probabilities: the head's bf16 logits to float32
                 probabilities, at each row's temperature and above each
                 row's floor
  sample         tree_sample: the walk down each row's draft tree by the
                 target's and the drafter's probabilities and given random
                 numbers, and the token drawn at its end
  lora           lora_add: every row's own low-rank adapter beside a shared
                 projection

`run` computes them in plain torch operations, or with `own` through the
package's entry points. Sequence b owns tokens starts[b] .. starts[b+1].
"""
import math

import numpy as np
import torch

own = False


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _probabilities(name, tokens, vocab, mixed=False, top=0):
    return {"name": name, "op": "probabilities", "tokens": tokens, "vocab": vocab, "mixed": mixed, "top": top}


def _sample(name, batch, tree, width, vocab, drawn=True):
    return {"name": name, "op": "sample", "batch": batch, "tree": tree, "width": width, "vocab": vocab, "drawn": drawn}


def _lora(name, batch, tokens, adapters, rank, inner, outer, ragged=False):
    return {"name": name, "op": "lora", "batch": batch, "tokens": tokens, "adapters": adapters, "rank": rank, "inner": inner,
            "outer": outer, "ragged": ragged}


def listed():
    return [
        # one user's next token: one row of the output head
        _probabilities("probs_1x248320", 1, 248320),
        # a server's verify step: 256 nodes of 32 users, each with a temperature of their own, some greedy
        _probabilities("probs_256x248320_mixed", 256, 248320, mixed=True),
        # a smaller vocabulary of odd width, kept to the 50 largest logits
        _probabilities("probs_24x32001_top50", 24, 32001, mixed=True, top=50),
        # one user, five drafted tokens in a row
        _sample("sample_1x6_chain", 1, 6, 1, 248320),
        # a server's users with drawn trees of up to 8 nodes
        _sample("sample_32x8_trees", 32, 8, 3, 248320),
        # trees of a drafter that picks the likeliest tokens (nothing drawn, so no probabilities of its own)
        _sample("sample_12x16_picked", 12, 16, 4, 32001, drawn=False),
        # ordinary decoding, nothing drafted: one draw for each of 64 users
        _sample("sample_64x1", 64, 1, 1, 128000, drawn=False),
        # one user's token through an attention projection
        _lora("lora_1x1_r16_5120x5120", 1, 1, 8, 16, 5120, 5120),
        # a server's decode step through gate and up: 48 users on 12 adapters
        _lora("lora_48x1_r64_5120x34816", 48, 1, 12, 64, 5120, 34816),
        # a server's verify step through the down projection: 16 users with 1 to 8 tokens, some without an adapter
        _lora("lora_16x8_r32_17408x5120", 16, 8, 6, 32, 17408, 5120, ragged=True),
        # one user's prompt through gate and up
        _lora("lora_1x4096_r16_5120x34816", 1, 4096, 2, 16, 5120, 34816),
        # six users' prompts through the fused query, key and value projection
        _lora("lora_6x2000_r64_5120x7168", 6, 2000, 5, 64, 5120, 7168, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _unnamed(kind, *sizes):
    return {k: v for k, v in kind("", *sizes).items() if k != "name"}


def draw(rng):
    op = rng.choice(["probabilities", "sample", "sample", "lora", "lora", "lora"])
    vocab = _log_int(rng, 1000, 248320)
    if op == "probabilities":
        return _unnamed(_probabilities, _log_int(rng, 1, 256), vocab, rng.random() < 0.7, rng.choice([0, 0, 1, 20, 400]))
    if op == "sample":
        batch, tree = _log_int(rng, 1, 64), _log_int(rng, 1, 24)
        tree = max(1, min(tree, 60_000_000 // (batch * vocab)))
        return _unnamed(_sample, batch, tree, rng.randint(1, 4), vocab, rng.random() < 0.6)
    rank = rng.choice([8, 16, 16, 24, 32, 64, 128])
    inner, outer = 8 * _log_int(rng, 32, 17408 // 8), _log_int(rng, 250, 34816)
    if rng.random() < 0.6:
        batch, tokens = _log_int(rng, 1, 64), _log_int(rng, 1, 16)
    else:
        batch, tokens = _log_int(rng, 1, 8), _log_int(rng, 64, 4096)
        tokens = max(1, min(tokens, 100_000_000 // (batch * max(inner, outer))))
    return _unnamed(_lora, batch, tokens, _log_int(rng, 1, 16), rank, inner, outer, rng.random() < 0.6)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _sizes(case):
    """New tokens of each sequence (they go by the case, not by the seed); the first has the most."""
    n, most = case["batch"], case["tokens"] if case["op"] == "lora" else case["tree"]
    if case["op"] == "lora" and not case["ragged"]:
        return np.full(n, most, np.int64)
    sizes = np.random.default_rng(n).integers((most + 7) // 8, most + 1, n)
    sizes[0] = most
    return sizes


def _adapters(case):
    """The adapter of each sequence, -1 where it has none (by the case, not by the seed)."""
    n = case["batch"]
    which = np.random.default_rng(n + 1).permutation(np.arange(n) % case["adapters"])
    if case["ragged"] and n >= 4:
        which[n // 3] = which[n // 2] = -1
    return which


def _logits(gen, tokens, vocab):
    """A head's logits: a broad bulk, and a few dozen tokens that stand out."""
    x = torch.randn((tokens, vocab), generator=gen, device="cuda").mul_(2.0)
    few = torch.randint(0, vocab, (tokens, 40), generator=gen, device="cuda")
    # (amax: a token may be chosen twice, and the inputs go by the seed alone)
    return x.scatter_reduce_(1, few, 9.0 + 3.0 * torch.randn((tokens, 40), generator=gen, device="cuda"), "amax")


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    if case["op"] == "probabilities":
        logits = _logits(gen, case["tokens"], case["vocab"]).to(torch.bfloat16)
        s = {"op": "probabilities", "logits": logits, "temperature": None, "floor": None}
        if case["mixed"]:
            t = 0.5 + torch.rand(case["tokens"], generator=gen, device="cuda")
            t[::5] = 0.0  # greedy users
            s["temperature"] = t
        if case["top"]:
            s["floor"] = torch.topk(logits, case["top"]).values[:, -1].float()
        return s
    sizes = _sizes(case)
    starts = np.concatenate([[0], np.cumsum(sizes)])
    tokens = int(starts[-1])
    if case["op"] == "sample":
        # random trees, node 0 the root; no node has more than `width` children
        words, parent = np.zeros(tokens, np.uint64), np.zeros(tokens, np.int64)
        for b, n in enumerate(sizes):
            kids, at = np.zeros(int(n), np.int64), int(starts[b])
            for i in range(int(n)):
                free = [j for j in range(max(0, i - 4), i) if kids[j] < case["width"]]
                p = int(rng.choice(free)) if i else -1
                if i:
                    kids[p] += 1
                parent[at + i] = at + max(p, 0)
                words[at + i] = (words[at + p] if i else np.uint64(0)) | (np.uint64(1) << np.uint64(i))
        ahead = _logits(gen, tokens, case["vocab"])
        p = torch.softmax(ahead / 0.9, -1)
        ahead += 0.7 * torch.randn(ahead.shape, generator=gen, device="cuda")  # what a drafter takes them for
        above = _cuda(parent)
        if case["drawn"]:
            q = torch.softmax(ahead / 0.9, -1)
            draft = torch.multinomial(q, case["width"], replacement=True, generator=gen)
        else:
            q, draft = None, torch.topk(ahead, case["width"]).indices
        order = np.zeros(tokens, np.int64)  # of a node among its parent's children
        seen = {}
        for i in range(tokens):
            if words[i] & (words[i] - np.uint64(1)):
                order[i] = seen.get(parent[i], 0)
                seen[parent[i]] = order[i] + 1
        return {"op": "sample", "p": p, "q": q, "draft": draft[above, _cuda(order)].contiguous(), "mask": _cuda(words.view(np.int64)),
                "starts": _cuda(starts.astype(np.int32)), "tree": case["tree"], "width": case["width"],
                "u": torch.rand(tokens, generator=gen, device="cuda")}
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    rank, inner, outer, store = case["rank"], case["inner"], case["outer"], case["adapters"]
    return {"op": "lora", "x": randn(tokens, inner).to(torch.bfloat16), "y": randn(tokens, outer).to(torch.bfloat16),
            "a": randn(store, rank, inner).div_(math.sqrt(inner)).to(torch.bfloat16),
            "b": randn(store, outer, rank).mul_(0.5 / math.sqrt(rank)).to(torch.bfloat16),
            "scale": 0.5 + torch.rand(store, generator=gen, device="cuda"),
            "adapter": _cuda(_adapters(case).astype(np.int32)), "starts": _cuda(starts.astype(np.int32))}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _own(s)
    return {"probabilities": _plain_probabilities, "sample": _plain_sample, "lora": _plain_lora}[s["op"]](s)


def _own(s):
    import gemm_w4a16_group_gb300 as w4
    if s["op"] == "probabilities":
        return w4.probabilities(s["logits"], s["temperature"], s["floor"])
    if s["op"] == "sample":
        return w4.tree_sample(s["p"], s["q"], s["draft"], s["mask"], s["starts"], s["u"], s["tree"])
    return w4.lora_add(s["y"], s["x"], s["a"], s["b"], s["adapter"], s["starts"], s["scale"])


def _owners(starts, tokens):
    """Sequence and index within it of every token."""
    at = torch.arange(tokens, device=starts.device)
    seq = torch.searchsorted(starts[1:].contiguous(), at.to(starts.dtype), right=True)
    return seq, at - starts[seq]


def _plain_probabilities(s):
    x = s["logits"].float()
    kept = x if s["floor"] is None else x.masked_fill(x < s["floor"][:, None], -math.inf)
    top = kept.amax(-1, keepdim=True)
    x = kept - torch.where(top == -math.inf, 0.0, top)
    if s["temperature"] is not None:
        x = x / torch.where(s["temperature"] > 0, s["temperature"], 1.0)[:, None]
    x = torch.exp(x)
    total = x.sum(-1, keepdim=True)
    x = x / torch.where(total == 0, 1.0, total)
    if s["temperature"] is None:
        return x
    first = torch.zeros_like(x).scatter_(1, kept.argmax(-1, keepdim=True), 1.0)
    return torch.where((s["temperature"] > 0)[:, None], x, first)


def _plain_sample(s):
    p, q, starts, tree = s["p"], s["q"], s["starts"], s["tree"]
    tokens, vocab = p.shape
    n = starts.numel() - 1
    seq, node = _owners(starts, tokens)
    pad = lambda x: torch.zeros((n, tree), device=x.device, dtype=x.dtype).index_put_((seq, node), x)  # noqa: E731
    words, draft, u = pad(s["mask"]), pad(s["draft"]), pad(s["u"]).double()
    sizes = starts[1:] - starts[:-1]
    idx = torch.arange(tree, device=p.device)
    there = idx[None] < sizes[:, None]
    above = ((words[:, :, None] >> idx) & 1).bool() & (idx[None, :] < idx[:, None])  # [n, node, proper ancestor]
    parent = torch.where(above, idx, -1).amax(-1)
    kid = there & (parent >= 0)
    older = kid[:, :, None] & kid[:, None, :] & (parent[:, :, None] == parent[:, None, :]) & (idx[None, :] < idx[:, None])
    order = older.sum(-1)
    under = (starts[:-1, None] + parent.clamp(min=0)).long().clamp(max=tokens - 1)  # the parent's place in p and q
    px = p[under, draft].double()
    step = torch.full((tokens,), -1, device=p.device)  # the child that each node goes on to
    push = lambda to, x, how: to.scatter_reduce(0, under.flatten(), x.flatten(), how)  # noqa: E731
    if q is None:
        twin = (older & (draft[:, :, None] == draft[:, None, :])).any(-1)
        gone = torch.where(older & ~twin[:, None, :], px[:, None, :], 0.0).sum(-1)
        left = torch.where(order == 0, 1.0, p.double().sum(-1)[under] - gone)
        fits = kid & (u * left < torch.where(twin, 0.0, px))
        first = push(torch.full((tokens,), tree, device=p.device), torch.where(fits, idx, tree), "amin")
        step = torch.where(first < tree, first, -1)
    else:
        qx = q[under, draft].double()
        c, total = torch.zeros(tokens, device=p.device, dtype=torch.float64), torch.ones(tokens, device=p.device, dtype=torch.float64)
        for k in range(s["width"]):  # a round needs the sums of what the round before left
            asked = kid & (order == k)
            fits = asked & (step[under] < 0) & (u * qx * total[under] < (px - c[under] * qx).clamp(min=0))
            step = push(step, torch.where(fits, idx, -1), "amax")
            refused = (push(torch.zeros_like(step), asked.long(), "amax") > 0) & (step < 0)
            c = torch.where(refused, c + total, c)
            if k + 1 < s["width"]:
                total = torch.where(refused, (p.double() - c[:, None] * q.double()).clamp_(min=0).sum(-1), total)
    good = (idx == 0) | (kid & (step[under] == idx))
    chain = above | torch.eye(tree, dtype=torch.bool, device=p.device)
    taken = there & (~chain | good[:, None, :]).all(-1) & ((idx == 0) | above[:, :, 0])
    count = taken.sum(-1, dtype=torch.int32)
    nodes = torch.where(taken, idx, tree).sort(-1).values
    path = torch.where(nodes < tree, nodes, -1).to(torch.int32)
    last = torch.where(taken, idx, 0).amax(-1)
    at = (starts[:-1] + last).long().clamp(max=tokens - 1)
    whole = p[at].double()
    if q is None:
        rest = whole.scatter_reduce(1, draft, torch.where(kid & (parent == last[:, None]), 0.0, math.inf).double(), "amin")
    else:
        rest = (whole - c[at][:, None] * q[at].double()).clamp_(min=0)
    rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, whole)
    upto = rest.cumsum(-1)
    token = (upto <= u[:, :1] * upto[:, -1:]).sum(-1)
    return path, count, torch.where((count > 0) & (upto[:, -1] > 0), token, -1)


def _plain_lora(s):
    y, x, a, b = s["y"], s["x"], s["a"], s["b"]
    store, rank, _ = a.shape
    which = s["adapter"][_owners(s["starts"], x.shape[0])[0]]
    t = (x.float() @ a.float().flatten(0, 1).T).view(-1, store, rank) * s["scale"][None, :, None]
    t = torch.where((which[:, None] == torch.arange(store, device=x.device))[:, :, None], t, 0.0)
    z = y.float() + t.flatten(1) @ b.float().transpose(1, 2).flatten(0, 1)
    return torch.where(which[:, None] >= 0, z, y.float()).to(y.dtype)


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its results in 64 bits
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "probabilities":
        return {"bytes": case["tokens"] * case["vocab"] * 6, "flops": case["tokens"] * case["vocab"] * 5}
    tokens = int(_sizes(case).sum())
    if case["op"] == "sample":  # one row where each walk ends, of both distributions where something can be refused
        both = 2 if case["drawn"] and case["tree"] > 1 else 1
        return {"bytes": case["batch"] * (case["vocab"] * 4 * both + case["tree"] * 4 + 12) + tokens * 20,
                "flops": case["batch"] * case["vocab"] * 2 * both}
    sizes, which, per = _sizes(case), _adapters(case), case["rank"] * (case["inner"] + case["outer"])
    mine = int(sizes[which >= 0].sum())
    used = len(set(which[which >= 0].tolist()))
    return {"bytes": mine * case["inner"] * 2 + tokens * case["outer"] * 4 + used * per * 2, "flops": 2 * mine * per}


def exact(case, seed):
    """Probabilities and adapted products from their definitions; a walk's outputs are whole numbers."""
    if case["op"] == "sample":
        return None
    s = prepare(case, seed)
    if case["op"] == "lora":
        out, starts = s["y"].double(), s["starts"].tolist()
        for b, e in enumerate(s["adapter"].tolist()):
            if e >= 0:
                rows = slice(starts[b], starts[b + 1])
                out[rows] += ((s["x"][rows].double() @ s["a"][e].double().T) * s["scale"][e].double()) @ s["b"][e].double().T
        return out
    out = torch.zeros(s["logits"].shape, device="cuda", dtype=torch.float64)
    for i in range(case["tokens"]):
        row = s["logits"][i].double()
        t = 1.0 if s["temperature"] is None else float(s["temperature"][i])
        kept = torch.ones_like(row, dtype=torch.bool) if s["floor"] is None else row >= s["floor"][i].double()
        if t > 0:
            out[i, kept] = torch.softmax(row[kept] / t, 0)
        else:
            out[i, int(torch.nonzero(row == row[kept].max())[0])] = 1.0
    return out
