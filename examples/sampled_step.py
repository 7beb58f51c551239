"""Speculative decoding of a model that samples, with an adapter for each user.

    python examples/sampled_step.py [--steps 24] [--temperature 0.8]

The model of verify_step.py answers three prompts: two users have a low-rank
adapter of their own beside every layer's first product (lora_add), the third has
none. A drafter that knows the last token alone draws a tree; one verify step runs
the tree through the model, probabilities turns both heads' logits into p and q at
the users' temperatures, tree_sample walks down the tree and draws the token at
its end, and kv_compact keeps the accepted rows. What comes out is distributed as
if every token had been sampled from the model by itself; at temperature 0 the
walk is tree_accept's.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

from verify_step import (DIM, GROUP, HEADS, HIDDEN, KV_HEADS, LAYERS, VOCAB, Cache, Model, ints, w4)  # noqa: E402

RANK, STORE = 16, 2
PARENT = (-1, 0, 0, 1, 1, 2, 2)  # a node's parent in a drafted tree, two children each
WORDS = [1]
for _i in range(1, len(PARENT)):
    WORDS.append(WORDS[PARENT[_i]] | 1 << _i)


class Adapted(Model):
    def __init__(self, seed=0):
        super().__init__(seed)
        gen = torch.Generator().manual_seed(seed + 1)
        bf16 = lambda *shape: torch.randn(shape, generator=gen).to(torch.bfloat16).cuda()  # noqa: E731
        self.a = bf16(LAYERS, STORE, RANK, HIDDEN) * HIDDEN ** -0.5
        self.b = bf16(LAYERS, STORE, (HEADS + 2 * KV_HEADS) * DIM, RANK)
        self.scale = torch.full((STORE,), 0.5, device="cuda")

    def head_of(self, x):
        return w4.gemm(x, self.head, VOCAB, HIDDEN, GROUP, True)

    def logits(self, tokens, cache, starts, mask, max_tree, adapter):
        def beside(i, h, y):
            w4.lora_add(y, h, self.a[i], self.b[i], adapter, starts, self.scale, out=y)
        return self.head_of(self.hidden(tokens, cache, cache.lengths, starts, mask, max_tree, beside))

    def drafter(self, tokens):
        """Logits by the last token alone."""
        return self.head_of(self.norm(self.embed[tokens]))


class Users:
    """Prompts in the cache, one table row each, with what the next step starts from."""

    def __init__(self, model, prompts, adapter, temperature, seed):
        self.model, self.n = model, len(prompts)
        self.adapter, self.temperature = ints(*adapter), temperature
        self.gen = torch.Generator("cuda").manual_seed(seed)
        self.cache = Cache(self.n)
        self.every = ints(*range(self.n))
        self.last = torch.empty(self.n, dtype=torch.int64, device="cuda")
        for r, prompt in enumerate(prompts):
            self.cache.reserve(ints(r), ints(len(prompt) + 64))
            for at in range(0, len(prompt), w4.MAX_TREE):
                part = prompt[at:at + w4.MAX_TREE]
                starts = ints(*[0] * (r + 1), *[len(part)] * (self.n - r))
                x = model.logits(part, self.cache, starts, None, len(part), self.adapter)[-1:]
                self.cache.lengths[r] += len(part)
            p = w4.probabilities(x, self.temperatures(1))
            self.last[r:r + 1] = w4.tree_sample(p, None, self.last[:1], None, ints(0, 1), self.numbers(1), 1)[2]

    def numbers(self, n):
        return torch.rand(n, generator=self.gen, device="cuda")

    def temperatures(self, n):
        return torch.full((n,), self.temperature, device="cuda")

    def step(self):
        """One token of every user."""
        n, starts = self.n, ints(*range(self.n + 1))
        self.cache.reserve(self.every, self.cache.lengths + 1)
        p = w4.probabilities(self.model.logits(self.last, self.cache, starts, None, 1, self.adapter), self.temperatures(n))
        self.cache.lengths += 1
        self.last = w4.tree_sample(p, None, self.last, None, starts, self.numbers(n), 1)[2]
        return [[int(t)] for t in self.last]

    def verify(self):
        """A drafted tree of every user: the accepted tokens and the one drawn behind them."""
        n, size = self.n, len(PARENT)
        tokens = torch.empty((n, size), dtype=torch.int64, device="cuda")
        tokens[:, 0] = self.last
        q = torch.empty((n, size, VOCAB), device="cuda")
        for i in range(size):  # children are drawn from q at their parent, each on its own
            if i:
                tokens[:, i] = torch.multinomial(q[:, PARENT[i]], 1, generator=self.gen)[:, 0]
            q[:, i] = w4.probabilities(self.model.drafter(tokens[:, i]), self.temperatures(n))
        tokens, q = tokens.view(-1), q.view(-1, VOCAB)
        mask = torch.tensor(WORDS, device="cuda").repeat(n)
        starts = ints(*range(0, n * size + 1, size))
        self.cache.reserve(self.every, self.cache.lengths + size)
        p = w4.probabilities(self.model.logits(tokens, self.cache, starts, mask, size, self.adapter), self.temperatures(n * size))
        path, count, self.last = w4.tree_sample(p, q, tokens, mask, starts, self.numbers(n * size), size)
        c = self.cache
        c.lengths = w4.kv_compact(c.k, c.v, c.table, c.lengths, path, count)
        accepted = [tokens.view(n, size)[r, path[r, 1:int(count[r])].long()].tolist() for r in range(n)]
        return [a + [int(t)] for a, t in zip(accepted, self.last)]


def decode(model, prompts, adapter, temperature, steps, trees, seed=1):
    """`steps` tokens of every prompt, and the number of steps it took."""
    users = Users(model, prompts, adapter, temperature, seed)
    said, calls = [[int(t)] for t in users.last], 0
    while min(len(s) for s in said) < steps:
        for s, new in zip(said, users.verify() if trees else users.step()):
            s += new
        calls += 1
    status = w4.kernel_status()
    if status != 0:
        raise RuntimeError(f"kernel status {status}")
    return [s[:steps] for s in said], calls


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=24)
    ap.add_argument("--temperature", type=float, default=0.8)
    a = ap.parse_args()
    gen = torch.Generator().manual_seed(5)
    prompts = [torch.randint(0, VOCAB, (n,), generator=gen).cuda() for n in (37, 90, 12)]
    model = Adapted()
    for name, trees in (("one token at a time", False), ("drafted trees", True)):
        said, calls = decode(model, prompts, [0, 1, -1], a.temperature, a.steps, trees)
        print(f"{name}: {a.steps} tokens of {len(prompts)} users in {calls} steps")
        for b, s in enumerate(said):
            print(f"  user {b}: {s}")
    return 0


if __name__ == "__main__":
    sys.exit(main())
