"""Plain 64-bit reference of the paged-cache operators, on the CPU, one
sequence and one row at a time, and the step descriptions the tests share."""
import math

import torch

import lossless_kv_cache_gb300 as sz

FP8 = {torch.float8_e5m2: (57344.0, 2, -14), torch.float8_e4m3fn: (448.0, 3, -6)}
RAW = {torch.bfloat16: torch.int16, torch.float16: torch.int16, torch.float8_e5m2: torch.uint8,
       torch.float8_e4m3fn: torch.uint8}


def round_fp8(x, dtype):
    """Doubles rounded half to even onto an FP8 grid (no overflow expected)."""
    _, bits, lowest = FP8[dtype]
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), torch.clamp(e - 1, min=lowest) - bits)
    return torch.round(x / step) * step


def quantise(x, dtype):
    """(values in units of the scale, scale exponent k) of rows of doubles; inf
    and NaN elements take no part in k and come out as they are."""
    largest = FP8[dtype][0]
    finite = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    most = finite.abs().amax(-1)
    k = torch.zeros(most.shape, dtype=torch.int32)
    for i in torch.nonzero(most > 0).tolist():
        e = -126
        while most[tuple(i)].item() > math.ldexp(largest, e):
            e += 1
        k[tuple(i)] = e
    q = round_fp8(torch.ldexp(finite, -k[..., None]), dtype)
    special = x
    if dtype == torch.float8_e4m3fn:  # no infinity
        special = torch.where(torch.isinf(x), torch.full_like(x, math.nan), x)
    return torch.where(torch.isfinite(x), q, special), k


class Step:
    """A cache and a step on the GPU, with its description on the CPU.

    lens: (new, held) of each sequence.  layout: "nhd", "hnd" (pages of
    [head][token][dim]) or "kv" (K and V side by side in one pool)."""

    def __init__(self, dtype, lens, page=16, kv_heads=2, dim=128, seed=0, layout="nhd", extra_pages=2, spare_rows=0,
                 fill="random", spread=1.0, x=torch.bfloat16):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.lens, self.page, self.kv_heads, self.dim = dtype, lens, page, kv_heads, dim
        self.x = dtype if dtype in (torch.bfloat16, torch.float16) else x
        counts = [-(-max(n, 0) // page) for _, n in lens]
        self.pages = sum(counts) + extra_pages
        order = torch.randperm(self.pages, generator=g).tolist()
        width = max(counts + [1])
        self.table = torch.full((len(lens), width), -7, dtype=torch.int32)  # unused entries are never looked at
        for b, c in enumerate(counts):
            self.table[b, :c] = torch.tensor(order[sum(counts[:b]): sum(counts[:b]) + c], dtype=torch.int32)
        self.tokens = sum(t for t, _ in lens) + spare_rows
        cu = [0]
        for t, _ in lens:
            cu.append(cu[-1] + t)
        self.cu = cu
        self.fp8 = dtype in FP8
        shape = (self.pages, page, kv_heads, dim)
        self.host = {}   # values in doubles
        pools, scales = [], []
        for name in "kv":
            chan = torch.exp(spread * torch.randn(kv_heads, dim, generator=g, dtype=torch.float64))
            val = torch.randn(shape, generator=g, dtype=torch.float64) * chan
            val = val.to(self.x).double()
            if fill == "zeros":
                val = torch.zeros_like(val)
            if self.fp8:
                # quick here: exponents from frexp, the same rule
                most = val.abs().amax(-1)
                m, e = torch.frexp(most)
                top = 16 if dtype == torch.float8_e5m2 else 9
                k = torch.where(most > 0, torch.where(m <= 0.875, e - top, e - top + 1), torch.zeros_like(e))
                q = round_fp8(torch.ldexp(val, -k[..., None]), dtype)
                pools.append(q.to(torch.float32).to(dtype))
                scales.append((k + 127).to(torch.uint8).transpose(1, 2).contiguous().cuda())
                self.host[name] = torch.ldexp(q, k[..., None])
            else:
                pools.append(val.to(dtype))
                scales.append(None)
                self.host[name] = val
        raw = RAW[dtype]
        bits = [p.view(raw) for p in pools]
        if layout == "nhd":
            dev = [b.cuda().view(dtype) for b in bits]
        elif layout == "hnd":
            dev = [b.transpose(1, 2).contiguous().cuda().view(dtype).transpose(1, 2) for b in bits]
        else:
            both = torch.stack(bits, 1).cuda().view(dtype)
            dev = [both[:, 0], both[:, 1]]
        self.cache = sz.KVCache(dev[0], dev[1], scales[0], scales[1])
        self.max_new = max([t for t, _ in lens] + [0])
        self.max_kv = max([n for _, n in lens] + [1])
        self.batch = sz.KVBatch(torch.tensor(cu, dtype=torch.int32).cuda(),
                                torch.tensor([n for _, n in lens], dtype=torch.int32).cuda(), self.table.cuda(),
                                self.tokens, self.max_new, self.max_kv)
        self.status = torch.full((4,), -1, dtype=torch.int32, device="cuda")
        self.gen = g

    def place(self, b, pos):
        return int(self.table[b, pos // self.page]), pos % self.page

    def held(self, b, name):
        """Positions 0 .. held - 1 of sequence b in doubles (held, kv_heads, dim)."""
        n = self.lens[b][1]
        pages = self.table[b, : -(-n // self.page)].long()
        return self.host[name][pages].reshape(-1, self.kv_heads, self.dim)[:n]

    def new_rows(self, spread=1.0):
        """Packed random rows of K or V."""
        return (torch.randn(self.tokens, self.kv_heads, self.dim, generator=self.gen) * spread).to(self.x)

    def set_value(self, name, b, pos, head, d, value):
        """Plants a value (also NaN or an infinity) in the cache."""
        pg, off = self.place(b, pos)
        pool = self.cache.k if name == "k" else self.cache.v
        one = torch.tensor([value], dtype=torch.float32).to(self.dtype).view(RAW[self.dtype])
        pool.view(RAW[self.dtype])[pg, off, head, d] = one.cuda()[0]
        scale = 1.0
        if self.fp8:
            s = self.cache.k_scale if name == "k" else self.cache.v_scale
            scale = 2.0 ** (int(s[pg, head, off]) - 127)
        self.host[name][pg, off, head, d] = one.view(self.dtype).double().item() * scale


def attention(step, q, scale, causal=True, window=0):
    """(out, lse, weight of |v|, score error scale) in doubles for packed q (CPU)."""
    tokens, heads, dim = q.shape
    group = heads // step.kv_heads
    out = torch.zeros(tokens, heads, dim, dtype=torch.float64)
    mag = torch.zeros(tokens, heads, dim, dtype=torch.float64)
    lse = torch.full((tokens, heads), -math.inf, dtype=torch.float64)
    size = torch.zeros(tokens, heads, dtype=torch.float64)
    for b, (t, n) in enumerate(step.lens):
        if t == 0 or n == 0:
            continue
        k, v = step.held(b, "k"), step.held(b, "v")
        j = torch.arange(n)
        for h in range(step.kv_heads):
            for i in range(t):
                p = n - t + i
                if p < 0:
                    continue
                seen = j >= 0
                if causal:
                    seen = seen & (j <= p)
                if window:
                    seen = seen & (j > p - window)
                r = step.cu[b] + i
                x = q[r, h * group: (h + 1) * group].double()
                kk, vv = k[seen, h], v[seen, h]
                s = x @ kk.T * scale
                norm = torch.logsumexp(s, -1)
                w = torch.exp(s - norm[:, None])
                out[r, h * group: (h + 1) * group] = w @ vv
                mag[r, h * group: (h + 1) * group] = w @ vv.abs()
                lse[r, h * group: (h + 1) * group] = norm
                size[r, h * group: (h + 1) * group] = (x.abs() @ kk.abs().T * abs(scale)).amax(-1)
    return out, lse, mag, size


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def check_attention(step, out, lse, ref, weight_type):
    """Compares with the reference, element by element.

    Errors counted: a score is a sum of dim products in 32 bits, each addition
    off by at most 2^-23 of the sum of magnitudes (the tensor cores truncate),
    and is scaled and shifted in 32 bits; exp2 is off by 2^-22; a weight is
    rounded to weight_type; sums over keys are in 32 bits; the result is
    rounded to its type."""
    r_out, r_lse, mag, size = ref
    keys = max(n for _, n in step.lens)
    score = (step.dim + 4) * 2.0 ** -23 * size + 2.0 ** -22 * (1 + r_lse.abs().nan_to_num(0, 0, 0))
    sums = (keys / 8 + 16) * 2.0 ** -23
    rel = half_step(weight_type) + 2 * score[..., None] + 2 * sums
    tol = rel * mag + half_step(out.dtype) * (1 + rel) * r_out.abs() + 1e-30
    # the least weights, times the largest value, where FP16 rounds to its subnormal steps
    tol = tol + (keys * 2.0 ** -38 + torch.finfo(out.dtype).smallest_normal * torch.finfo(out.dtype).eps)
    got = out.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(r_out))
    fine = torch.isfinite(r_out)
    assert torch.equal(got[~fine].nan_to_num(7.0), r_out[~fine].nan_to_num(7.0))
    over = ((got - r_out).abs() / tol)[fine]
    assert over.numel() == 0 or over.max() <= 1, float(over.max())
    if lse is not None:
        got = lse.double().cpu()
        none = torch.isinf(r_lse)
        assert torch.equal(got[none], r_lse[none])
        ok = (got - r_lse).abs() <= score + sums + 2.0 ** -22 * (1 + r_lse.abs())
        assert bool(ok[~none].all())
