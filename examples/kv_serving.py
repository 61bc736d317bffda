"""Disaggregated serving in miniature, on one GPU: the paged-cache operators
and the lossless codec as a serving engine would run them together.

A prefill side takes a prompt in chunks.  Each chunk's keys and values are
quantised into the E5M2 pages of its cache (`kv_write`) and its queries attend
over all pages so far (`kv_attention`).  The finished cache is compressed
losslessly page by page list (`encode_paged_into`), and a decode side, whose
pool hands out other pages, restores it (`decode_paged_into`).  There the
sequence goes on token by token (`kv_write`, `kv_attention`), and at the end
the cache is read back (`kv_read`).

The random tensors stand for a model's projections; what is shown is the
calls, their order and their buffers.  Run: python examples/kv_serving.py
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import lossless_kv_cache_gb300 as sz  # noqa: E402

KV_HEADS, HEADS, HEAD_DIM = 8, 32, 128
PAGE_TOKENS = 16  # 16,384 elements of 8 heads of 128: the codec's pages hold whole tiles


class Side:
    """A cache of one layer and the pages that one sequence has in it."""

    def __init__(self, pages, order, device):
        self.cache = sz.KVCache.empty(pages, PAGE_TOKENS, KV_HEADS, HEAD_DIM, torch.float8_e5m2, device)
        self.pages = torch.tensor(order, dtype=torch.int32, device=device)
        self.cu_tokens = torch.zeros(2, dtype=torch.int32, device=device)
        self.kv_len = torch.zeros(1, dtype=torch.int32, device=device)
        self.status = torch.zeros(4, dtype=torch.int32, device=device)
        self.worst = torch.zeros(1, dtype=torch.int32, device=device)
        self.buffers = {}

    def note(self, status):
        """Keeps a call's status, in stream order: the next call clears the word."""
        torch.maximum(self.worst, status[:1], out=self.worst)

    def step(self, q, k, v):
        """The next tokens of the sequence: into the cache, then over it.  Returns
        their attention; asynchronous."""
        new = q.shape[0]
        self.cu_tokens[1] = new
        self.kv_len += new
        batch = sz.KVBatch(self.cu_tokens, self.kv_len, self.pages[None], new, new, self.pages.numel() * PAGE_TOKENS)
        if new not in self.buffers:
            self.buffers[new] = sz.KVAttentionBuffers(self.cache, batch, HEADS)
        out = torch.empty_like(q)
        sz.kv_write(self.cache, batch, k, v, self.status)
        self.note(self.status)
        sz.kv_attention(self.cache, batch, q, out, self.buffers[new], 1.0 / math.sqrt(HEAD_DIM))
        self.note(self.buffers[new].status)
        return out

    def read(self, tokens):
        """K and V of the last `tokens` tokens, BF16."""
        self.cu_tokens[1] = tokens
        batch = sz.KVBatch(self.cu_tokens, self.kv_len, self.pages[None], tokens, tokens,
                           self.pages.numel() * PAGE_TOKENS)
        k, v = (torch.empty(tokens, KV_HEADS, HEAD_DIM, dtype=torch.bfloat16, device=self.pages.device)
                for _ in range(2))
        sz.kv_read(self.cache, batch, k, v, self.status)
        self.note(self.status)
        return k, v


def send(sender, receiver, used):
    """Moves the first `used` pages of the sequence: K and V as compressed
    containers, the scales (1 byte in 128) as they are.  Returns (bytes of the
    pages, bytes that would cross the link)."""
    page_elems = PAGE_TOKENS * KV_HEADS * HEAD_DIM
    n = used * page_elems
    raw = link = 0
    for name in "kv":
        pool, to = (getattr(s.cache, name).view(torch.uint8).view(-1) for s in (sender, receiver))
        sample = torch.cat([getattr(sender.cache, name)[p].view(torch.uint8).reshape(-1)
                            for p in sender.pages[: min(used, 8)].tolist()])
        codebook, _ = sz.calibrate(sample, sz.FP8_E5M2)
        bufs = sz.EncodeBuffers(n, sz.FP8_E5M2)
        sz.encode_paged_into(pool, sender.pages[:used], page_elems, codebook, bufs)
        size, status = int(bufs.size[0]), int(bufs.status[0])
        assert status == sz.OK
        container = bufs.out[:size].clone()  # what the link carries
        sz.decode_paged_into(container, size, to, receiver.pages[:used], page_elems, sz.FP8_E5M2, receiver.status)
        receiver.note(receiver.status)
        scale_from, scale_to = (getattr(s.cache, name + "_scale") for s in (sender, receiver))
        scale_to[receiver.pages[:used].long()] = scale_from[sender.pages[:used].long()]
        raw += n
        link += size
    receiver.kv_len.copy_(sender.kv_len)
    return raw, link


def run(prompt=1000, chunk=384, steps=8, seed=0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)

    def project(tokens):
        q, k, v = (torch.randn(tokens, h, HEAD_DIM, generator=g, device=device) for h in (HEADS, KV_HEADS, KV_HEADS))
        return q.bfloat16(), k.bfloat16(), (0.5 * v).bfloat16()

    pages = -(-(prompt + steps) // PAGE_TOKENS)
    pool = pages + 13
    prefill = Side(pool, torch.randperm(pool)[:pages].tolist(), device)
    decode = Side(pool, torch.randperm(pool)[:pages].tolist(), device)
    outs = []
    for first in range(0, prompt, chunk):
        outs.append(prefill.step(*project(min(chunk, prompt - first))))
    raw, link = send(prefill, decode, -(-prompt // PAGE_TOKENS))
    for _ in range(steps):
        qkv = project(1)
        outs.append(decode.step(*qkv))
        # the sending side could have gone on itself, with the same result
        assert torch.equal(outs[-1], prefill.step(*qkv))
    k, v = decode.read(prompt + steps)
    k2, v2 = prefill.read(prompt + steps)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    assert int(prefill.worst) == sz.OK and int(decode.worst) == sz.OK  # of every call
    return torch.cat(outs), raw, link


if __name__ == "__main__":
    out, raw, link = run()
    print("%d tokens attended, E5M2 pages %d bytes, on the link %d bytes (%.3fx)"
          % (out.shape[0], raw, link, raw / link))
