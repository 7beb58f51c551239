"""Speculative decoding with draft trees on INT4 weights and a paged cache.

    python examples/verify_step.py [--steps 12] [--e4m3]

A small decoder with random weights (INT4, group 128) answers two prompts. A
drafter guesses a tree of tokens; one verify step then runs the whole tree
through the model: kv_reserve, and per layer gemm, kv_append, tree_attention,
gemm, gateup_silu, gemm; gemm_argmax picks a token for every node, tree_accept
walks down the tree and kv_compact keeps the accepted rows in every layer. One
prompt is branched with kv_fork and the original dropped with kv_free. The same
model, one token at a time, has to say the same (with an 8-bit cache nearly: the
two ways' keys round differently where two codes are equally near).
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gemm_w4a16_group_gb300 as w4  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, FFN, VOCAB, LAYERS, GROUP = 512, 8, 2, 64, 1024, 4096, 3, 128


def random_weight(rows, cols, gen):
    codes = torch.randint(1, 16, (rows, cols // 8, 8), generator=gen)  # q - 8 in -7 .. 7
    q = (codes << torch.arange(0, 32, 4)).sum(-1).to(torch.int32)  # the top nibble wraps into the sign
    s = (torch.rand((rows, cols // GROUP), generator=gen) * 0.01 + 0.005).to(torch.bfloat16)
    return q.cuda(), s.cuda()


class Model:
    def __init__(self, seed=0):
        gen = torch.Generator().manual_seed(seed)
        pack = lambda n, k: w4.repack(*random_weight(n, k, gen), None, n, k, GROUP, True)  # noqa: E731
        self.embed = torch.randn((VOCAB, HIDDEN), generator=gen).to(torch.bfloat16).cuda()
        self.layers = []
        for _ in range(LAYERS):
            gate, up = random_weight(FFN, HIDDEN, gen), random_weight(FFN, HIDDEN, gen)
            self.layers.append((pack((HEADS + 2 * KV_HEADS) * DIM, HIDDEN), pack(HIDDEN, HEADS * DIM),
                                w4.repack_gateup(*gate, None, *up, None, FFN, HIDDEN, GROUP, True), pack(HIDDEN, FFN)))
        self.head = pack(VOCAB, HIDDEN)

    @staticmethod
    def norm(x):
        return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def picks(self, tokens, cache, lengths, starts, mask, max_tree):
        """The model's pick after each of `tokens`, whose keys and values join the cache."""
        x = self.embed[tokens]
        for i, (qkv, proj, gate_up, down) in enumerate(self.layers):
            y = w4.gemm(self.norm(x), qkv, (HEADS + 2 * KV_HEADS) * DIM, HIDDEN, GROUP, True)
            y = y.view(-1, HEADS + 2 * KV_HEADS, DIM)
            w4.kv_append(y[:, HEADS:HEADS + KV_HEADS], y[:, HEADS + KV_HEADS:], cache.k[i], cache.v[i], cache.table,
                         lengths, starts, **cache.scales)
            o = w4.tree_attention(y[:, :HEADS], cache.k[i], cache.v[i], cache.table, lengths, starts, mask, max_tree,
                                  **cache.scales)
            x = x + w4.gemm(o.view(-1, HEADS * DIM), proj, HIDDEN, HEADS * DIM, GROUP, True)
            h = w4.gateup_silu(self.norm(x), gate_up, FFN, HIDDEN, GROUP, True)
            x = x + w4.gemm(h, down, HIDDEN, FFN, GROUP, True)
        return w4.gemm_argmax(self.norm(x), self.head, VOCAB, HIDDEN, GROUP, True)[0]


class Cache:
    def __init__(self, rows, pages=64, page_rows=16, width=16, e4m3=False):
        dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
        shape = (LAYERS, pages, KV_HEADS, page_rows, DIM)
        self.k, self.v = (torch.empty(shape, dtype=dtype, device="cuda") for _ in range(2))
        one = torch.full((KV_HEADS,), 0.05, device="cuda")
        self.scales = {"k_scale": one, "v_scale": one} if e4m3 else {}
        i32 = {"dtype": torch.int32, "device": "cuda"}
        self.table = torch.full((rows, width), -1, **i32)
        self.lengths, self.refs, self.page_rows = torch.zeros(rows, **i32), torch.zeros(pages, **i32), page_rows

    def reserve(self, rows, want):
        """Room for want[i] tokens in table row rows[i] (int32 tensors)."""
        if int(w4.kv_reserve(self.table, self.refs, rows, want, self.page_rows)) != 1:
            raise RuntimeError("the cache is full")


def ints(*a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def prefill(model, cache, row, prompt):
    """The prompt's keys and values, up to 64 tokens at a time; the pick after its last token."""
    rows = cache.table.shape[0]
    cache.reserve(ints(row), ints(len(prompt) + 64))
    for at in range(0, len(prompt), w4.MAX_TREE):
        part = prompt[at:at + w4.MAX_TREE]
        starts = ints(*[0] * (row + 1), *[len(part)] * (rows - row))
        pick = model.picks(part, cache, cache.lengths, starts, None, len(part))[-1]
        cache.lengths[row] += len(part)
    return pick


def drafts(last, truth, gen):
    """A drafter: 7 guesses under the last token, three levels deep, some of them right (`truth`: what a good drafter
    would know). Tokens and ancestor words, node 0 the last token itself."""
    parent = [-1, 0, 0, 1, 1, 2, 3, 4]
    words = [1]
    for i in range(1, 8):
        words.append(words[parent[i]] | 1 << i)
    guess = torch.randint(0, VOCAB, (8,), generator=gen).tolist()
    guess[0] = int(last)
    on = 0
    for depth, token in enumerate(truth[:3]):
        kids = [i for i in range(1, 8) if parent[i] == on]
        if not kids or float(torch.rand(1, generator=gen)) < 0.25:
            break
        on = kids[int(torch.randint(0, len(kids), (1,), generator=gen))]
        guess[on] = token
    return guess, words


def stepwise(model, prompts, steps, e4m3=False):
    """Greedy decoding, one token of every row at a time."""
    cache = Cache(len(prompts), e4m3=e4m3)
    last = torch.stack([prefill(model, cache, b, p) for b, p in enumerate(prompts)])
    said = [last]
    starts = ints(*range(len(prompts) + 1))
    every = ints(*range(len(prompts)))
    for _ in range(steps - 1):
        cache.reserve(every, cache.lengths + 1)
        last = model.picks(last, cache, cache.lengths, starts, None, 1)
        cache.lengths += 1
        said.append(last)
    return torch.stack(said, 1).tolist()


def speculative(model, prompts, steps, truth, e4m3=False, seed=1):
    """The same with drafted trees; returns the tokens and the number of verify steps."""
    gen = torch.Generator().manual_seed(seed)
    n = len(prompts)
    cache = Cache(n + 1, e4m3=e4m3)  # one row to branch into
    said = [[int(prefill(model, cache, b, p))] for b, p in enumerate(prompts)]
    # branch the first prompt, and go on in the branch: the original is dropped
    if int(w4.kv_fork(cache.k, cache.v, cache.table, cache.lengths, cache.refs, ints(0), ints(n))) != 1:
        raise RuntimeError("the cache is full")
    w4.kv_free(cache.table, cache.lengths, cache.refs, ints(0))
    rows = [n, *range(1, n)]  # the table row of each prompt
    verifies = 0
    while min(len(s) for s in said) < steps:
        tokens, words, starts = [], [], [0]
        for r in range(n + 1):  # tokens in the order of the table's rows
            if r in rows:
                b = rows.index(r)
                g, w = drafts(said[b][-1], truth[b][len(said[b]):], gen)
                tokens += g
                words += w
            starts.append(len(tokens))
        starts = ints(*starts)
        tokens = torch.tensor(tokens, device="cuda")
        mask = torch.tensor(words, device="cuda")
        cache.reserve(ints(*rows), cache.lengths[torch.tensor(rows, device="cuda")] + 8)
        target = model.picks(tokens, cache, cache.lengths, starts, mask, 8)
        path, count, token = w4.tree_accept(target, tokens, mask, starts, 8)
        cache.lengths = w4.kv_compact(cache.k, cache.v, cache.table, cache.lengths, path, count)
        for b, r in enumerate(rows):
            accepted = [int(tokens[int(starts[r]) + i]) for i in path[r, 1:int(count[r])].tolist()]
            said[b] += accepted + [int(token[r])]
        verifies += 1
    if w4.kernel_status() != 0:
        raise RuntimeError(f"kernel status {w4.kernel_status()}")
    return [s[:steps] for s in said], verifies


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=24)
    ap.add_argument("--e4m3", action="store_true", help="an 8-bit cache")
    a = ap.parse_args()
    gen = torch.Generator().manual_seed(5)
    prompts = [torch.randint(0, VOCAB, (n,), generator=gen).cuda() for n in (37, 90)]
    model = Model()
    want = stepwise(model, prompts, a.steps, a.e4m3)
    said, verifies = speculative(model, prompts, a.steps, want, a.e4m3)
    print(f"{a.steps} tokens of {len(prompts)} prompts in {verifies} verify steps")
    for b, s in enumerate(said):
        print(f"prompt {b}: {s}  {'as' if s == want[b] else 'NOT as'} one token at a time")
    return 0 if said == want or a.e4m3 else 1


if __name__ == "__main__":
    sys.exit(main())
