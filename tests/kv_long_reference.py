"""The reference of attention in 64 bits for caches of some thousands of keys:
whole sequences at a time, on the GPU, in doubles.  NaN in V reaches the rows
that see it (infinities are not planted here)."""
import math

import torch


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
    scale.copy_((scale.cpu().int() + e.transpose(1, 2)).to(torch.uint8))
    step.host[name] = torch.ldexp(step.host[name], e[..., None])
