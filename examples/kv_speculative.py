"""Speculative serving in miniature, on one GPU: the operators of a step over
the paged cache as an engine would run them, with nothing about lengths on the
host.

Every step gives each sequence a tree of drafted tokens.  `kv_extend` gives it
the pages for them (and takes back what the last step's rejected tokens had),
`kv_tree` makes the masks and positions, once for all layers.  A layer rotates
and writes the drafted tokens' keys and values (`kv_rotary_write`) and attends
(`kv_tree_attention`).  Of each tree one branch is accepted, here at random, and
`kv_keep` moves it to the front in all layers; the next step drops the others.

The random tensors stand for a model's projections; what is shown is the calls,
their order and their buffers.  Run: python examples/kv_speculative.py
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import lossless_kv_cache_gb300 as sz  # noqa: E402

KV_HEADS, HEADS, HEAD_DIM, LAYERS = 2, 8, 128, 3
PAGE_TOKENS = 16


class Engine:
    """`batch` sequences, their pages, a cache a layer, and the buffers of a step of at
    most `drafted` tokens a sequence."""

    def __init__(self, batch, drafted, max_len, dtype=torch.float8_e4m3fn, x=torch.bfloat16, device="cuda"):
        pool = batch * -(-max_len // PAGE_TOKENS)
        ints = lambda *s: torch.zeros(*s, dtype=torch.int32, device=device)  # noqa: E731
        self.batch, self.rows = batch, batch * drafted
        self.pages = sz.KVPages.empty(pool, PAGE_TOKENS, batch, max_len, device)
        self.step = sz.KVStep(batch, self.rows, drafted, max_len, device)
        self.caches = [sz.KVCache.empty(pool, PAGE_TOKENS, KV_HEADS, HEAD_DIM, dtype, device) for _ in range(LAYERS)]
        self.layers = sz.KVLayers(self.caches)
        self.kv = self.step.batch_of(self.pages)
        self.tree = sz.KVTree(self.kv)
        self.bufs = sz.KVAttentionBuffers(self.caches[0], self.kv, HEADS)
        # a context stretched fourfold: 2,048 positions to 8,192
        self.rotary = sz.KVRotary(sz.rotary_frequencies(HEAD_DIM, 500000.0, factor=4.0, original_len=2048), device=device)
        # what a step is given, and what it says of itself
        self.new, self.drop, self.kept = ints(batch), ints(batch), ints(batch)
        self.parents, self.path = ints(self.rows), ints(self.rows)
        self.q = torch.zeros(LAYERS, self.rows, HEADS, HEAD_DIM, dtype=x, device=device)
        self.k, self.v = (torch.zeros(LAYERS, self.rows, KV_HEADS, HEAD_DIM, dtype=x, device=device) for _ in range(2))
        self.out = torch.zeros_like(self.q)
        self.status, self.worst = ints(4), ints(1)

    def note(self, status):
        """Keeps a call's status, in stream order: the next call clears the word."""
        torch.maximum(self.worst, status[:1], out=self.worst)

    def forward(self):
        """One step of the target over the drafted trees; asynchronous."""
        sz.kv_extend(self.pages, self.new, self.step, drop=self.drop)
        self.note(self.step.status)
        sz.kv_tree(self.kv, self.parents, self.tree)
        self.note(self.tree.status)
        for i, cache in enumerate(self.caches):
            sz.kv_rotary_write(cache, self.kv, self.rotary, self.q[i], self.q[i], self.k[i], self.v[i], self.status,
                               positions=self.tree.position)
            self.note(self.status)
            sz.kv_tree_attention(cache, self.kv, self.tree, self.q[i], self.out[i], self.bufs, 1.0 / math.sqrt(HEAD_DIM))
            self.note(self.bufs.status)

    def accept(self):
        """The accepted branches to the front; what the next step drops."""
        sz.kv_keep(self.layers, self.kv, self.path, self.kept, self.status)
        self.note(self.status)
        torch.sub(self.new, self.kept, out=self.drop)


def draft(engine, g, sizes):
    """Random trees of these sizes, a random branch of each, and random projections, on the
    CPU: (parents, branches of numbers within the tree)."""
    parents, branches = [], []
    for t in sizes:
        tree = [int(torch.randint(max(-1, i - 4), i, (), generator=g)) for i in range(t)]
        branch = []
        node = int(torch.randint(0, t, (), generator=g)) if t else -1
        while node >= 0:
            branch.insert(0, node)
            node = tree[node]
        parents += tree
        branches.append(branch)
    rows = len(parents)
    for t in (engine.q, engine.k, engine.v):
        t[:, :rows] = torch.randn(t[:, :rows].shape, generator=g).to(t.dtype)
    return parents, branches


def give(engine, sizes, parents, branches):
    """A step's inputs to the device."""
    ints = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    path = []
    for t, branch in zip(sizes, branches):
        path += branch + [-1] * (t - len(branch))
    engine.new.copy_(ints(sizes))
    engine.kept.copy_(ints([len(b) for b in branches]))
    engine.parents[: len(parents)] = ints(parents)
    engine.path[: len(path)] = ints(path)


def run(steps=6, batch=4, drafted=12, dtype=torch.float8_e4m3fn, x=torch.bfloat16, seed=0, device="cuda", step=None):
    """Returns (engine, what was accepted: for each sequence and layer its q, k, v and attention).
    step: what runs a step instead of forward and accept (a captured graph's replay)."""
    g = torch.Generator().manual_seed(seed)
    engine = Engine(batch, drafted, max_len=steps * drafted + drafted, dtype=dtype, x=x, device=device)
    replay = step(engine) if step else None
    history = [[] for _ in range(batch)]
    for n in range(steps):
        sizes = [int(torch.randint(1, drafted + 1, (), generator=g)) if (n + b) % 5 else 0 for b in range(batch)]
        parents, branches = draft(engine, g, sizes)
        q, k, v = (t.cpu().clone() for t in (engine.q, engine.k, engine.v))
        give(engine, sizes, parents, branches)
        if replay:
            replay()
        else:
            engine.forward()
            engine.accept()
        out, first = engine.out.cpu(), 0
        for b, branch in enumerate(branches):
            history[b] += [[t[:, first + i] for t in (q, k, v, out)] for i in branch]
            first += sizes[b]
    # the last step's rejected tokens go too
    engine.new.zero_()
    sz.kv_extend(engine.pages, engine.new, engine.step, drop=engine.drop)
    engine.note(engine.step.status)
    return engine, [[torch.stack(t, 1) for t in zip(*h)] for h in history]


if __name__ == "__main__":
    engine, history = run()
    assert int(engine.worst) == sz.OK
    print("accepted tokens:", engine.pages.kv_len.tolist(), "pages:", engine.pages.held.tolist(),
          "free pages: %d of %d" % (int(engine.pages.count), engine.pages.free.numel()))
