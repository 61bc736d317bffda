"""Measured cases of the paged-cache operators: writing a chunk of keys and
values into a paged cache (quantising them where the cache is FP8), reading
them back, and attention of a chunk of new tokens (one token each included)
over the cache.

`run` computes an operator either in its plain form (elementary torch
operations in 32 bits) or, with `own` set, through the package's entry points.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
#: cache types: (torch dtype, bytes, exponent of 2^e with largest finite = 0.875 * 2^e)
TYPES = {"bf16": (torch.bfloat16, 2, None), "fp16": (torch.float16, 2, None),
         "e5m2": (torch.float8_e5m2, 1, 16), "e4m3": (torch.float8_e4m3fn, 1, 9)}


def _case(name, op, type, x, batch, new, kv, ragged=False, page=16, kv_heads=8, heads=32, dim=128, causal=True,
          window=0):
    return {"name": name, "op": op, "type": type, "x": x, "batch": batch, "new": new, "kv": kv, "ragged": ragged,
            "page": page, "kv_heads": kv_heads, "heads": heads, "dim": dim, "causal": causal, "window": window}


def listed():
    return [
        # one decoding step of 64 sequences: each appends its token to an E5M2 cache (latency)
        _case("write_step_e5m2", "write", "e5m2", "bf16", 64, 1, 2048),
        # prompts of mixed length enter an E4M3 cache, FP16 model, pages that end inside a chunk
        _case("write_ragged_e4m3", "write", "e4m3", "fp16", 7, 2501, 4099, ragged=True, page=64),
        # the layer of 32,768 tokens (8 heads x 128) quantised to E5M2 as it is written
        _case("write_layer_e5m2", "write", "e5m2", "bf16", 1, 32768, 32768),
        # a few sequences read back for a host copy or another kernel
        _case("read_ragged_e4m3", "read", "e4m3", "fp16", 9, 1200, 1500, ragged=True, page=32, kv_heads=4, dim=64),
        # the E5M2 layer of 65,536 tokens read back as BF16
        _case("read_layer_e5m2", "read", "e5m2", "bf16", 1, 65536, 65536),
        # decoding a handful of short chats (latency)
        _case("step_short_bf16", "attention", "bf16", "bf16", 4, 1, 500),
        # one long document being decoded: few rows, a long axis
        _case("step_long_bf16", "attention", "bf16", "bf16", 1, 1, 65536),
        # a full serving batch decoding over a quantised cache
        _case("step_batch_e5m2", "attention", "e5m2", "bf16", 64, 1, 8192),
        # a ragged batch that verifies up to 3 drafted tokens, heads of 64, sliding window
        _case("step_ragged_fp16", "attention", "fp16", "fp16", 33, 3, 9001, ragged=True, page=32, heads=24, dim=64,
              window=4096),
        # chunks of several prompts in one call, quantised cache
        _case("chunk_ragged_e4m3", "attention", "e4m3", "bf16", 6, 777, 5000, ragged=True, page=64),
        # one prompt of 8,192 tokens, no history, FP16
        _case("prompt_fp16", "attention", "fp16", "fp16", 1, 8192, 8192, page=128),
        # a chunk of 2,048 new tokens over a cache of 32,768
        _case("chunk_long_bf16", "attention", "bf16", "bf16", 1, 2048, 32768),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["write", "read", "attention", "attention", "attention", "attention"])
    type = rng.choice(["bf16", "fp16", "e5m2", "e5m2", "e4m3"])
    x = type if type in ("bf16", "fp16") else rng.choice(["bf16", "bf16", "fp16"])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 8])
    group = rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 16])
    dim = rng.choice([64, 128, 128])
    page = rng.choice([1, 4, 8, 16, 16, 32, 64, 128, 256])
    if op != "attention":
        # up to half the tokens of the largest listed layer
        tokens = _log_int(rng, 1, 32768)
        batch = min(_log_int(rng, 1, 64), tokens)
        new = tokens // batch
        kv = new + _log_int(rng, 1, 4096)
    elif rng.random() < 0.5:  # decoding steps
        new = rng.choice([1, 1, 1, 2, 4])
        kv = _log_int(rng, new, 65536)
        batch = _log_int(rng, 1, max(1, min(64, 262144 // kv)))
    else:  # chunks: at most a quarter of the largest listed case's scores
        new = _log_int(rng, 2, 4096)
        kv = _log_int(rng, new, max(new, min(32768, 16777216 // new)))
        group = min(group, 8)
        batch = _log_int(rng, 1, max(1, min(8, 16777216 // (new * kv))))
    c = _case("", op, type, x, batch, new, kv, ragged=batch > 1 and rng.random() < 0.6, page=page,
              kv_heads=kv_heads, heads=kv_heads * group, dim=dim, causal=op != "attention" or rng.random() < 0.85,
              window=rng.choice([0, 0, 0, _log_int(rng, 1, kv)]) if op == "attention" else 0)
    del c["name"]
    return c


def _lengths(case):
    """(new tokens, tokens in the cache) of every sequence: all the case's largest, or spread below it; one
    sequence of a ragged batch has nothing new."""
    n, new, kv = case["batch"], case["new"], case["kv"]
    if not case["ragged"]:
        return [new] * n, [kv] * n
    r = random.Random(n * 1000003 + new * 1009 + kv)
    news, kvs = [], []
    for b in range(n):
        t = new if b == 0 else 0 if b == 2 else r.randint(1, new)
        news.append(t)
        kvs.append(kv if b == 0 else max(t, _log_int(r, max(1, kv // 64), kv)))
    return news, kvs


def _pair_count(case):
    """Allowed (query, key) pairs of one head, over all sequences."""
    news, kvs = _lengths(case)
    total = 0
    for t, n in zip(news, kvs):
        first = n - t
        if not case["causal"]:
            # the window bounds how far back a query sees; keys ahead are all seen
            w = case["window"]
            total += t * n if not w else sum(n - max(0, p - w + 1) for p in range(first, n))
        else:
            w = case["window"] or n + 1
            total += sum(min(p + 1, w) for p in range(first, n))
    return total


def _keys_needed(case):
    news, kvs = _lengths(case)
    w = case["window"]
    return sum(0 if not t else n if not w else min(n, t + w - 1) for t, n in zip(news, kvs))


def work(case):
    size = TYPES[case["type"]][1]
    row = case["kv_heads"] * case["dim"]
    scale = case["kv_heads"] if size == 1 else 0
    tokens = sum(_lengths(case)[0])
    if case["op"] != "attention":
        # K and V once in one form and once in the other
        return {"bytes": 2 * tokens * (2 * row + size * row + scale), "flops": 2 * tokens * row * 2 if size == 1 else 0}
    q = tokens * case["heads"] * case["dim"] * 2
    return {"bytes": 2 * q + 4 * tokens * case["heads"] + 2 * _keys_needed(case) * (size * row + scale),
            "flops": 4 * _pair_count(case) * case["heads"] * case["dim"]}


# ------------------------------------------------------------------ inputs

def _power(e):
    """2^e for integers -126 .. 127, exactly."""
    return ((e + 127).to(torch.int32) << 23).view(torch.float32)


def _quantise(x, type):
    """Rows of x (last axis) in an FP8 type and the exponents of their power-of-two scales: the smallest k with
    every finite |x| <= largest * 2^k."""
    dtype, _, top = TYPES[type]
    x = x.float()
    most = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(-1)
    m, e = torch.frexp(most)
    k = torch.where(m <= 0.875, e - top, e - top + 1)
    k = torch.where(most > 0, k, torch.zeros_like(k)).clamp(-126, 127)
    return (x * _power(-k)[..., None]).to(dtype), k


def _values(bits, scale, at, type):
    """Rows `at` (flat token slots) of a pool, as 32-bit values. scale: (pages, heads, page tokens)."""
    pages, page, heads, dim = bits.shape
    flat = bits.view(torch.uint8 if scale is not None else torch.int16).reshape(pages * page, heads, dim)
    x = flat[at].view(TYPES[type][0]).float()
    if scale is None:
        return x
    return x * _power(scale[at // page, :, at % page].to(torch.int32) - 127)[..., None]


def _place(state, b, pos):
    """The pool's token slots of positions `pos` of sequences `b`."""
    page = state["page"]
    return state["table"][b, pos // page].long() * page + pos % page


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    randn = lambda *s: torch.randn(s, generator=g, device=DEVICE)  # noqa: E731
    news, kvs = _lengths(case)
    page, heads, dim, type = case["page"], case["kv_heads"], case["dim"], case["type"]
    dtype, size, _ = TYPES[type]
    x = TYPES[case["x"]][0]
    counts = [-(-n // page) for n in kvs]
    pages = sum(counts) + 3
    width = max(max(counts), 1)
    order = torch.randperm(pages, generator=g, device=DEVICE).to(torch.int32)
    first = torch.tensor([sum(counts[:b]) for b in range(len(counts))], device=DEVICE)
    held = torch.tensor(counts, device=DEVICE)
    column = torch.arange(width, device=DEVICE)
    # entries past a sequence's pages are never used
    table = torch.where(column < held[:, None], order[(first[:, None] + column).clamp(max=pages - 1)].int(), -1).int()
    s = {"op": case["op"], "type": type, "page": page, "causal": case["causal"], "window": case["window"],
         "x": x, "table": table, "max_new": max(news), "max_kv": max(max(kvs), 1), "tokens": sum(news),
         "cu": torch.tensor([sum(news[:b]) for b in range(len(news) + 1)], dtype=torch.int32, device=DEVICE),
         "kv_len": torch.tensor(kvs, dtype=torch.int32, device=DEVICE), "scale": 1.0 / math.sqrt(dim)}
    channel = torch.exp(randn(2, heads, dim)) * torch.tensor([0.5, 0.25], device=DEVICE)[:, None, None]
    for i, name in enumerate("kv"):
        if case["op"] == "write":
            s[name] = torch.zeros(pages, page, heads, dim, dtype=torch.uint8 if size == 1 else torch.int16,
                                  device=DEVICE).view(dtype)
            s[name + "_scale"] = torch.zeros(pages, heads, page, dtype=torch.uint8, device=DEVICE) if size == 1 else None
            # K and V as slices of one projection's output would be strided; here each is its own tensor
            s[name + "_new"] = (randn(s["tokens"], heads, dim) * channel[i]).to(x)
        else:
            values = (randn(pages, page, heads, dim) * channel[i])
            if size == 1:
                s[name], k = _quantise(values.to(x), type)
                s[name + "_scale"] = (k + 127).to(torch.uint8).transpose(1, 2).contiguous()
            else:
                s[name], s[name + "_scale"] = values.to(dtype), None
            del values
    if case["op"] == "attention":
        s["q"] = randn(s["tokens"], case["heads"], dim).to(x)
    if own:
        import lossless_kv_cache_gb300 as sz

        s["cache"] = sz.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        s["batch"] = sz.KVBatch(s["cu"], s["kv_len"], s["table"], s["tokens"], s["max_new"], s["max_kv"])
        s["status"] = torch.zeros(4, dtype=torch.int32, device=DEVICE)
        if case["op"] == "read":
            s["k_out"] = torch.empty(s["tokens"], heads, dim, dtype=x, device=DEVICE)
            s["v_out"] = torch.empty_like(s["k_out"])
        if case["op"] == "attention":
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(s["tokens"], case["heads"], dtype=torch.float32, device=DEVICE)
            s["bufs"] = sz.KVAttentionBuffers(s["cache"], s["batch"], case["heads"])
    return s


# --------------------------------------------------------------------- run

def _pools(s):
    """The written pools: FP8 elements as the values they stand for, and their scales' exponents."""
    got = {"k": s["k"], "v": s["v"]}
    if s["k_scale"] is not None:
        got.update(k_scale=s["k_scale"], v_scale=s["v_scale"])
    return got


def _rows(s):
    """Sequence and cache position of every packed row: a sequence's rows are its last positions."""
    t = torch.arange(s["tokens"], device=DEVICE, dtype=torch.int32)
    b = torch.searchsorted(s["cu"], t, right=True) - 1
    return b, s["kv_len"][b].long() - (s["cu"][b + 1] - t).long()


def _plain_write(s):
    b, pos = _rows(s)
    at = _place(s, b, pos)
    for name in "kv":
        pool, new = s[name], s[name + "_new"]
        pages, page, heads, dim = pool.shape
        if s[name + "_scale"] is None:
            pool.view(pages * page, heads, dim)[at] = new
        else:
            bits, k = _quantise(new, s["type"])
            pool.view(torch.uint8).view(pages * page, heads, dim)[at] = bits.view(torch.uint8)
            s[name + "_scale"][at // page, :, at % page] = (k + 127).to(torch.uint8)
    return _pools(s)


def _plain_read(s):
    b, pos = _rows(s)
    at = _place(s, b, pos)
    return {n: _values(s[n], s[n + "_scale"], at, s["type"]).to(s["x"]) for n in "kv"}


def _plain_attention(s):
    q = s["q"]
    tokens, heads, dim = q.shape
    kv_heads = s["k"].shape[2]
    group, batch = heads // kv_heads, s["kv_len"].numel()
    # keys and values, padded to the longest sequence; places past a sequence's end hold nothing
    pos = torch.arange(s["max_kv"], device=DEVICE)
    n = s["kv_len"].long()
    held = pos < n[:, None]
    at = torch.where(held, _place(s, torch.arange(batch, device=DEVICE)[:, None], pos), 0)
    zero = torch.zeros((), device=DEVICE)
    k, v = (torch.where(held[..., None, None], _values(s[x], s[x + "_scale"], at, s["type"]), zero) for x in "kv")
    # queries, padded to the longest chunk: (batch, kv head, new * group, dim)
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    i = torch.arange(s["max_new"], device=DEVICE)
    there = i < new[:, None]
    row = (s["cu"][:-1, None] + i).long().clamp(max=tokens - 1)
    query = q[row].float().view(batch, s["max_new"], kv_heads, group, dim).transpose(1, 2)
    scores = torch.matmul(query.reshape(batch, kv_heads, s["max_new"] * group, dim), k.permute(0, 2, 3, 1))
    scores = scores.view(batch, kv_heads, s["max_new"], group, s["max_kv"]).mul_(s["scale"])
    # a query at position p sees keys p - window + 1 .. p (without causal: up to the end)
    p = (n - new)[:, None] + i
    seen = held[:, None, :] & there[..., None]
    if s["causal"]:
        seen = seen & (pos <= p[..., None])
    if s["window"]:
        seen = seen & (pos > p[..., None] - s["window"])
    scores.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    most = scores.amax(-1, keepdim=True)
    low = torch.where(torch.isfinite(most), most, zero)
    weight = scores.sub_(low).exp_()
    total = weight.sum(-1, keepdim=True)
    out = torch.matmul(weight.view(batch, kv_heads, s["max_new"] * group, s["max_kv"]), v.transpose(1, 2))
    out = out.view(batch, kv_heads, s["max_new"], group, dim) / torch.where(total > 0, total, zero + 1)
    lse = (low + total.log()).squeeze(-1)  # a row that sees nothing: 0, and log(0)
    packed = torch.nonzero(there.reshape(-1)).squeeze(-1)
    out = out.transpose(1, 2).reshape(batch * s["max_new"], heads, dim)[packed]
    lse = lse.transpose(1, 2).reshape(batch * s["max_new"], heads)[packed]
    return {"out": out.to(s["x"]), "lse": lse}


def run(s):
    if not own:
        return {"write": _plain_write, "read": _plain_read, "attention": _plain_attention}[s["op"]](s)
    import lossless_kv_cache_gb300 as sz

    if s["op"] == "write":
        sz.kv_write(s["cache"], s["batch"], s["k_new"], s["v_new"], s["status"])
        return _pools(s)
    if s["op"] == "read":
        sz.kv_read(s["cache"], s["batch"], s["k_out"], s["v_out"], s["status"])
        return {"k": s["k_out"], "v": s["v_out"]}
    sz.kv_attention(s["cache"], s["batch"], s["q"], s["out"], s["bufs"], s["scale"], causal=s["causal"],
                    window=s["window"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------- 64-bit values

def _power64(e):
    """2^e in doubles, exactly (pow and exp2 are not always exact on the GPU)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _rounded(x, type):
    """Doubles rounded to an FP8 type (half to even) on its grid of steps."""
    bits, lowest = (2, -14) if type == "e5m2" else (3, -6)
    e = torch.frexp(x.abs())[1] - 1  # |x| in [2^e, 2^(e+1))
    step = _power64(torch.clamp(e, min=lowest) - bits)
    return torch.round(x / step) * step


def _exact_rows(case, s):
    """Pool page and offset of every packed row, found one sequence at a time."""
    cu, n, table = s["cu"].tolist(), s["kv_len"].tolist(), s["table"].cpu()
    pages, offsets = [], []
    for b in range(len(n)):
        pos = torch.arange(n[b] - (cu[b + 1] - cu[b]), n[b])
        pages.append(table[b, torch.div(pos, case["page"], rounding_mode="floor")].long())
        offsets.append(pos % case["page"])
    return torch.cat(pages).to(DEVICE), torch.cat(offsets).to(DEVICE)


def _exact_pool(s, name, type):
    """A whole pool's values in doubles (pages, page tokens, heads, dim)."""
    x = s[name].to(torch.float32).double()
    if s[name + "_scale"] is None:
        return x
    return x * _power64(s[name + "_scale"].int() - 127).transpose(1, 2)[..., None]


def exact(case, seed):
    s = prepare(case, seed)
    type = case["type"]
    if case["op"] == "write":
        page, offset = _exact_rows(case, s)
        got = {}
        for name in "kv":
            x = s[name + "_new"].double()
            pool = torch.zeros(s[name].shape, dtype=torch.float64, device=DEVICE)
            if TYPES[type][1] == 1:
                largest = 57344.0 if type == "e5m2" else 448.0
                most = x.abs().amax(-1, keepdim=True)
                # smallest k with most <= largest * 2^k, found by counting from a guess that is at most one off
                k = torch.floor(torch.log2(most.clamp(min=1e-300) / largest) - 1e-6)
                k = torch.where(most <= largest * _power64(k), k, k + 1)
                k = torch.where(most > 0, k, torch.zeros_like(k)).clamp(-126, 127)
                x = _rounded(x / _power64(k), type)
            pool[page, offset] = x
            got[name] = pool
        if TYPES[type][1] == 1:
            got.update(k_scale=None, v_scale=None)
        return got
    pools = [_exact_pool(s, name, type) for name in "kv"]
    if case["op"] == "read":
        page, offset = _exact_rows(case, s)
        return {"k": pools[0][page, offset], "v": pools[1][page, offset]}
    cu, lens = s["cu"].tolist(), s["kv_len"].tolist()
    group = case["heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEVICE)
    for b, n in enumerate(lens):
        t = cu[b + 1] - cu[b]
        if not t or not n:
            continue
        pages = s["table"][b, : -(-n // case["page"])].long()
        for h in range(case["kv_heads"]):
            k, v = (x[pages, :, h].reshape(-1, case["dim"])[:n] for x in pools)
            j = torch.arange(n, device=DEVICE)
            for lo in range(0, t, 1024):
                hi = min(t, lo + 1024)
                q = s["q"][cu[b] + lo: cu[b] + hi, h * group: (h + 1) * group].double()
                p = torch.arange(n - t + lo, n - t + hi, device=DEVICE)[:, None]
                hidden = torch.zeros(hi - lo, n, dtype=torch.bool, device=DEVICE)
                if case["causal"]:
                    hidden |= j > p
                if case["window"]:
                    hidden |= j <= p - case["window"]
                z = torch.einsum("tgd,nd->tgn", q, k) / math.sqrt(case["dim"])
                z = z.masked_fill(hidden[:, None], -math.inf)
                norm = torch.logsumexp(z, -1)
                z = torch.exp(z - torch.where(torch.isfinite(norm), norm, torch.zeros_like(norm))[..., None])
                out[cu[b] + lo: cu[b] + hi, h * group: (h + 1) * group] = torch.einsum("tgn,nd->tgd", z, v)
                lse[cu[b] + lo: cu[b] + hi, h * group: (h + 1) * group] = norm
    return {"out": out, "lse": lse}
