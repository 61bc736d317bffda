"""Caches of some thousands of keys, made on the GPU, and the reference of
attention over them in 64 bits: whole sequences at a time, in doubles.  NaN in
V reaches the rows that see it (infinities are not planted here)."""
import math

import torch

import lossless_kv_cache_gb300 as sz
from tests.kv_reference import FP8, Step, round_fp8


class LongStep(Step):
    """A Step of the first layout whose values are made and held on the GPU."""

    def __init__(self, dtype, lens, page=16, kv_heads=8, dim=128, seed=0, x=torch.bfloat16, spread=0.3):
        self.gen = torch.Generator().manual_seed(seed)
        on_gpu = torch.Generator(device="cuda").manual_seed(seed)
        self.dtype, self.lens, self.page, self.kv_heads, self.dim = dtype, lens, page, kv_heads, dim
        self.x = dtype if dtype in (torch.bfloat16, torch.float16) else x
        self.fp8 = dtype in FP8
        counts = [-(-n // page) for _, n in lens]
        self.pages = sum(counts) + 2
        order = torch.randperm(self.pages, generator=self.gen).to(torch.int32)
        self.table = torch.full((len(lens), max(counts + [1])), -7, dtype=torch.int32)
        at = 0
        for b, c in enumerate(counts):
            self.table[b, :c] = order[at: at + c]
            at += c
        self.cu = [0]
        for t, _ in lens:
            self.cu.append(self.cu[-1] + t)
        self.tokens = self.cu[-1]
        self.host, pools, scales = {}, [], []
        for name in "kv":
            chan = torch.exp(spread * torch.randn(kv_heads, dim, generator=on_gpu, dtype=torch.float64, device="cuda"))
            val = torch.randn(self.pages, page, kv_heads, dim, generator=on_gpu, dtype=torch.float64, device="cuda")
            val = (val * chan).to(self.x).double()
            scale = None
            if self.fp8:
                m, e = torch.frexp(val.abs().amax(-1))
                top = 16 if dtype == torch.float8_e5m2 else 9
                k = torch.where(m <= 0.875, e - top, e - top + 1)
                q = round_fp8(torch.ldexp(val, -k[..., None]), dtype)
                scale = (k + 127).to(torch.uint8).transpose(1, 2).contiguous()
                val = torch.ldexp(q, k[..., None])
                pools.append(q.float().to(dtype))
            else:
                pools.append(val.to(dtype))
            scales.append(scale)
            self.host[name] = val
        self.cache = sz.KVCache(*pools, *scales)
        self.max_new, self.max_kv = max(t for t, _ in lens), max(n for _, n in lens)
        self.batch = sz.KVBatch(torch.tensor(self.cu, dtype=torch.int32).cuda(),
                                torch.tensor([n for _, n in lens], dtype=torch.int32).cuda(), self.table.cuda(),
                                self.tokens, self.max_new, self.max_kv)
        self.status = torch.full((4,), -1, dtype=torch.int32, device="cuda")

    def held(self, b, name):
        n = self.lens[b][1]
        pages = self.table[b, : -(-n // self.page)].long().cuda()
        return self.host[name][pages].reshape(-1, self.kv_heads, self.dim)[:n]


def attention64(step, q, scale, causal=True, window=0):
    """What kv_reference.attention returns, for packed q on the CPU."""
    tokens, heads, dim = q.shape
    kv_heads = step.kv_heads
    group = heads // kv_heads
    out = torch.zeros(tokens, heads, dim, dtype=torch.float64)
    mag = torch.zeros(tokens, heads, dim, dtype=torch.float64)
    lse = torch.full((tokens, heads), -math.inf, dtype=torch.float64)
    size = torch.zeros(tokens, heads, dtype=torch.float64)
    for b, (t, n) in enumerate(step.lens):
        if t == 0 or n == 0:
            continue
        k, v = (step.held(b, name).cuda().transpose(0, 1) for name in "kv")  # (kv_heads, n, dim)
        nan = torch.isnan(v)
        v = torch.where(nan, torch.zeros_like(v), v)
        x = q[step.cu[b]: step.cu[b] + t].cuda().double()
        x = x.view(t, kv_heads, group, dim).transpose(0, 1).reshape(kv_heads, t * group, dim)
        j = torch.arange(n, device="cuda")
        p = (n - t + torch.arange(t, device="cuda")).repeat_interleave(group)[:, None]
        seen = (p >= 0) & (j >= 0)
        if causal:
            seen = seen & (j <= p)
        if window:
            seen = seen & (j > p - window)
        s = torch.where(seen, x @ k.transpose(1, 2) * scale, torch.full((), -math.inf, device="cuda", dtype=x.dtype))
        norm = torch.logsumexp(s, -1)
        w = torch.exp(s - torch.where(torch.isfinite(norm), norm, torch.zeros_like(norm))[..., None])
        most = torch.where(seen, x.abs() @ k.abs().transpose(1, 2) * abs(scale), torch.zeros_like(s)).amax(-1)
        o, m = w @ v, w @ v.abs()
        if bool(nan.any()):
            o = torch.where(seen.double() @ nan.double() > 0, torch.full_like(o, math.nan), o)
        rows = slice(step.cu[b], step.cu[b] + t)

        def packed(y, last):
            return y.view(kv_heads, t, group, *last).transpose(0, 1).reshape(t, heads, *last).cpu()

        out[rows], mag[rows] = packed(o, (dim,)), packed(m, (dim,))
        lse[rows], size[rows] = packed(norm, ()), packed(most, ())
    return out, lse, mag, size


def vary_scales(step, name, low, high):
    """Multiplies every (token, head) of an FP8 pool by a power of two of its own."""
    shape = (step.pages, step.page, step.kv_heads)
    e = torch.randint(low, high + 1, shape, generator=step.gen)
    scale = getattr(step.cache, name + "_scale")
    scale.copy_(scale.cpu().int() + e.transpose(1, 2))
    step.host[name] = torch.ldexp(step.host[name], e[..., None].to(step.host[name].device))
