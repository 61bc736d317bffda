"""Measured cases of the paged-cache operators of a speculative serving step:
page tables, slots and positions built on the GPU from the lengths that a step
asks for; rotary positions of queries and keys with the write into the cache;
attention of a tree of drafted tokens over the cache; and the accepted branch
moved to the front of the drafted tokens in every layer.

`run` computes an operator either in its plain form (elementary torch
operations, in 32 bits; angles in 64) or, with `own` set, through the package's
entry points.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
#: cache types: (torch dtype, bytes, exponent of 2^e with largest finite = 0.875 * 2^e)
TYPES = {"bf16": (torch.bfloat16, 2, None), "fp16": (torch.float16, 2, None),
         "e5m2": (torch.float8_e5m2, 1, 16), "e4m3": (torch.float8_e4m3fn, 1, 9)}


def _extend(name, batch, new, kv, page, drop=0.0):
    """drop: share of the sequences that give up tokens (rejected drafts; a quarter of them all, being finished)."""
    return {"name": name, "op": "extend", "batch": batch, "new": new, "kv": kv, "page": page, "drop": drop}


def _rotary(name, type, x, batch, new, kv, ragged=False, page=16, kv_heads=8, heads=32, dim=128, rot=128,
            interleaved=False, base=10000.0, factor=1.0, ahead=0):
    """rot: rotated elements of a head.  factor: how far past its original 8,192 positions the context is stretched.
    ahead: positions are given, that far past the places in the cache."""
    return {"name": name, "op": "rotary", "type": type, "x": x, "batch": batch, "new": new, "kv": kv, "ragged": ragged,
            "page": page, "kv_heads": kv_heads, "heads": heads, "dim": dim, "rot": rot, "interleaved": interleaved,
            "base": base, "factor": factor, "ahead": ahead}


def _tree(name, type, x, batch, new, kv, ragged=False, page=16, kv_heads=8, heads=32, dim=128, window=0):
    """new: drafted tokens of a sequence; kv: its tokens before them."""
    return {"name": name, "op": "tree", "type": type, "x": x, "batch": batch, "new": new, "kv": kv, "ragged": ragged,
            "page": page, "kv_heads": kv_heads, "heads": heads, "dim": dim, "window": window}


def _keep(name, type, layers, batch, new, kv, ragged=False, page=16, kv_heads=8, dim=128):
    return {"name": name, "op": "keep", "type": type, "x": "fp16" if type == "fp16" else "bf16", "layers": layers,
            "batch": batch, "new": new, "kv": kv, "ragged": ragged, "page": page, "kv_heads": kv_heads, "dim": dim}


def listed():
    return [
        # one decoding step of 64 sequences: a token each, a page for every sixteenth of them (latency)
        _extend("extend_step", 64, 1, 2048, 16),
        # a serving step of 256 sequences: prompts enter beside drafts, some drafts are given up, some sequences end
        _extend("extend_mixed", 256, 333, 5000, 16, drop=0.5),
        # queries and keys of one decoding step of 64 sequences into an E5M2 cache (latency)
        _rotary("rotary_step_e5m2", "e5m2", "bf16", 64, 1, 2048),
        # prompts of mixed length, FP16 model that rotates half of each head in pairs of neighbours, context stretched
        # eightfold, E4M3 cache, pages that end inside a chunk
        _rotary("rotary_ragged_e4m3", "e4m3", "fp16", 7, 2501, 4099, ragged=True, page=64, rot=64, interleaved=True,
                base=500000.0, factor=8.0, ahead=60000),
        # the layer of 32,768 tokens (8 heads x 128, 32 query heads) as it enters an E5M2 cache
        _rotary("rotary_layer_e5m2", "e5m2", "bf16", 1, 32768, 32768),
        # two short chats that verify a tree of seven drafted tokens (latency)
        _tree("tree_few_bf16", "bf16", "bf16", 2, 7, 600),
        # a serving batch that verifies sixteen drafted tokens each over a quantised cache
        _tree("tree_batch_e5m2", "e5m2", "bf16", 32, 16, 4096),
        # ragged trees over ragged contexts, heads of 64, a sliding window
        _tree("tree_ragged_fp16", "fp16", "fp16", 17, 25, 9001, ragged=True, page=32, heads=24, dim=64, window=4096),
        # trees of 64 tokens over long contexts: as much arithmetic as memory traffic
        _tree("tree_wide_bf16", "bf16", "bf16", 8, 64, 16384),
        # one long document, quantised
        _tree("tree_long_e4m3", "e4m3", "bf16", 1, 32, 65536, page=64),
        # the accepted branches of a batch in all 32 layers of a quantised cache
        _keep("keep_layers_e5m2", "e5m2", 32, 64, 16, 200),
        # of a few ragged trees, FP16, pages of 32, heads of 64 (latency)
        _keep("keep_few_fp16", "fp16", 2, 5, 25, 300, ragged=True, page=32, dim=64),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["extend", "rotary", "rotary", "tree", "tree", "tree", "keep"])
    type = rng.choice(["bf16", "fp16", "e5m2", "e5m2", "e4m3"])
    x = type if type in ("bf16", "fp16") else rng.choice(["bf16", "bf16", "fp16"])
    page = rng.choice([1, 4, 8, 16, 16, 32, 64, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 8])
    group = rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 16])
    dim = rng.choice([64, 128, 128])
    ragged = rng.random() < 0.6
    if op == "extend":
        batch = _log_int(rng, 1, 2000)
        c = _extend("", batch, _log_int(rng, 1, max(1, 65536 // batch)), _log_int(rng, 1, max(1, 1500000 // batch)),
                    page, rng.choice([0.0, 0.2, 0.5, 0.9]))
    elif op == "rotary":
        # up to half the tokens of the largest listed layer
        tokens = _log_int(rng, 1, 16384)
        batch = min(_log_int(rng, 1, 64), tokens)
        new = tokens // batch
        c = _rotary("", type, x, batch, new, new + _log_int(rng, 1, 4096), batch > 1 and ragged, page, kv_heads,
                    kv_heads * min(group, 8), dim, rng.choice([dim, dim, dim // 2, dim // 4]), rng.random() < 0.4,
                    rng.choice([10000.0, 500000.0, 1000000.0]), rng.choice([1.0, 1.0, 4.0, 32.0]),
                    rng.choice([0, 0, _log_int(rng, 1, 1000000)]))
    elif op == "tree":
        # at most half the scores and keys of the largest listed case
        new = _log_int(rng, 1, 200)
        kv = _log_int(rng, 1, min(65536, 4000000 // new))
        heads = kv_heads * (min(group, 8) if new > 16 else group)
        most = min(65536 // kv, 134217728 // (new * kv * heads))
        c = _tree("", type, x, _log_int(rng, 1, max(1, min(64, most))), new, kv, ragged, page, kv_heads, heads, dim,
                  rng.choice([0, 0, 0, _log_int(rng, 1, kv)]))
    else:
        new = _log_int(rng, 1, 64)
        c = _keep("", type, rng.choice([1, 2, 5, 16, 32]), _log_int(rng, 1, 48), new, _log_int(rng, 1, 200), ragged,
                  min(page, 64), kv_heads, dim)
    del c["name"]
    return c


def _lengths(case):
    """(new tokens, tokens before them) of every sequence: all the case's largest, or spread below it; one sequence
    of a ragged batch has nothing new."""
    n, new, kv = case["batch"], case["new"], case["kv"]
    if case["op"] == "rotary":
        kv -= new
    if not case["ragged"]:
        return [new] * n, [kv] * n
    r = random.Random(n * 1000003 + new * 1009 + kv)
    news = [new if b == 0 else 0 if b == 2 else r.randint(1, new) for b in range(n)]
    return news, [kv if b == 0 else _log_int(r, max(1, kv // 64), max(1, kv)) for b in range(n)]


def _extend_lengths(case):
    """(new, held tokens, dropped, pages held) of every sequence: mostly a token each, and prompts of up to the
    case's size beside them; the sequences that give up tokens are spread over the batch."""
    r = random.Random(case["batch"] * 1000003 + case["new"] * 1009 + case["kv"])
    rows = []
    for b in range(case["batch"]):
        kv = case["kv"] if b == 0 else _log_int(r, max(1, case["kv"] // 32), case["kv"])
        new = case["new"] if b == 0 or case["drop"] == 0 else r.choice([0, 1, 1, 1, r.randint(1, case["new"])])
        drop, spare = 0, 0
        if b and r.random() < case["drop"]:
            done = r.random() < 0.25
            drop, new = (kv, 0) if done else (r.randint(0, min(kv, 64)), new)
            spare = r.choice([0, 0, 1, 3])
        rows.append((new, kv, drop, -(-kv // case["page"]) + spare))
    return [list(c) for c in zip(*rows)]


def _kept(case):
    """Accepted tokens of every sequence."""
    r = random.Random(case["batch"] * 7919 + case["new"])
    return [0 if not t else r.randint(1, max(1, t // 3)) if b % 5 else t for b, t in enumerate(_lengths(case)[0])]


def work(case):
    if case["op"] == "extend":
        new, kv, drop, held = _extend_lengths(case)
        need = [-(-(n - d + t) // case["page"]) for t, n, d in zip(new, kv, drop)]
        moved = sum(abs(a - b) for a, b in zip(need, held))
        # new, drop, lengths and held pages in, and the three arrays out; pages between list and tables; rows
        return {"bytes": 4 * 7 * case["batch"] + 8 * moved + 12 * sum(new), "flops": 0}
    size = TYPES[case["type"]][1]
    row = case["kv_heads"] * case["dim"]
    scale = case["kv_heads"] if size == 1 else 0
    news, kvs = _lengths(case)
    tokens = sum(news)
    if case["op"] == "rotary":
        q = case["heads"] * case["dim"]
        cache = 2 * (size * row + scale)
        rotated = case["rot"] * (case["heads"] + case["kv_heads"])
        return {"bytes": tokens * (4 * q + 4 * row + cache + (4 if case["ahead"] else 0)),
                "flops": tokens * (3 * rotated + (2 * row * 2 if size == 1 else 0))}
    if case["op"] == "keep":
        return {"bytes": 2 * 2 * case["layers"] * sum(_kept(case)) * (size * row + scale) + 4 * tokens, "flops": 0}
    w = case["window"]
    q = tokens * case["heads"] * case["dim"] * 2
    # the keys before a tree that its first row sees, and the tree's own; every row's keys before the tree
    held = [0 if not t else t + (min(n, w - 1) if w else n) for t, n in zip(news, kvs)]
    pairs = sum(t * ((min(n, w) if w else n) + 1) for t, n in zip(news, kvs))
    return {"bytes": 2 * q + 4 * tokens * (case["heads"] + 2) + 2 * sum(held) * (size * row + scale),
            "flops": 4 * pairs * case["heads"] * case["dim"]}


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


def _frequencies(case):
    """(radians a position turns each pair of elements by, factor on the rotated values), in doubles.  A stretched
    context leaves pairs that turn often over its original length as they are, slows those that hardly turn by the
    factor, and goes over from one to the other in between."""
    half, original, low, high = case["rot"] // 2, 8192, 1.0, 32.0
    f = torch.tensor([case["base"] ** (-j / half) for j in range(half)], dtype=torch.float64)
    if case["factor"] != 1.0:
        keep = ((original * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        f = f * (keep + (1 - keep) / case["factor"])
    return f, 1.0 if case["factor"] == 1.0 else 0.1 * math.log(case["factor"]) + 1.0


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def _starts(counts):
    return [sum(counts[:b]) for b in range(len(counts) + 1)]


def _prepare_extend(case, g):
    new, kv, drop, held = _extend_lengths(case)
    page = case["page"]
    need = [-(-(n - d + t) // page) for t, n, d in zip(new, kv, drop)]
    more = sum(max(0, a - b) for a, b in zip(need, held))
    pages, width = sum(held) + more + 7, max(max(need), max(held))
    order = torch.randperm(pages, generator=g, device=DEVICE).int()
    first = torch.cumsum(_ints(held), 0) - _ints(held)
    column = torch.arange(width, device=DEVICE)
    has = column < _ints(held)[:, None]
    table = torch.where(has, order[(first[:, None] + column).clamp(max=pages - 1)], -1).int()
    free = torch.cat([order[sum(held):], torch.full((sum(held),), -1, dtype=torch.int32, device=DEVICE)])
    tokens = sum(new)
    s = {"op": "extend", "page": page, "new": _ints(new), "kv_len": _ints(kv), "drop": _ints(drop) if any(drop) else None,
         "held": _ints(held), "table": table, "free": free, "count": _ints([pages - sum(held)]), "tokens": tokens}
    if own:
        import lossless_kv_cache_gb300 as sz

        s["pages"] = sz.KVPages(s["free"], s["count"], s["table"], s["held"], s["kv_len"], page)
        s["after"] = s["pages"].ahead()
        most = max(n - d + t for t, n, d in zip(new, kv, drop))
        s["step"] = sz.KVStep(case["batch"], tokens, max(new), max(most, 1))
    return s


def _prepare_keep(case, g, s, news, kvs, pages):
    heads, dim, page, layers = case["kv_heads"], case["dim"], case["page"], case["layers"]
    dtype, size, _ = TYPES[case["type"]]
    for name in "kv":
        if size == 1:
            bits = torch.randint(0, 256, (layers, pages, page, heads, dim), generator=g, device=DEVICE, dtype=torch.uint8)
            # no infinities and NaN, which compare as nothing
            bits &= 0xFB if case["type"] == "e5m2" else 0xFE
            s[name] = bits.view(dtype)
            s[name + "_scale"] = torch.randint(100, 140, (layers, pages, heads, page), generator=g, device=DEVICE,
                                               dtype=torch.uint8)
        else:
            s[name] = torch.randn((layers, pages, page, heads, dim), generator=g, device=DEVICE).to(dtype)
            s[name + "_scale"] = None
    # a branch: ascending tokens of the tree
    kept = _ints(_kept(case))
    u = torch.rand((len(news), max(news)), generator=g, device=DEVICE)
    i = torch.arange(max(news), device=DEVICE)
    rank = torch.where(i < _ints(news)[:, None], u, 2.0).argsort(-1).argsort(-1)
    chosen = torch.where(rank < kept[:, None], i, max(news)).sort(-1).values
    path = torch.where(i < kept[:, None], chosen, -1).int()
    s["path"] = path[i < _ints(news)[:, None]].contiguous()
    s["kept"] = kept
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    if case["op"] == "extend":
        return _prepare_extend(case, g)
    randn = lambda *s: torch.randn(s, generator=g, device=DEVICE)  # noqa: E731
    news, kvs = _lengths(case)
    page, heads, dim, type = case["page"], case["kv_heads"], case["dim"], case["type"]
    dtype, size, _ = TYPES[type]
    x = TYPES[case["x"]][0]
    counts = [-(-(n + t) // page) for t, n in zip(news, kvs)]
    pages = sum(counts) + 3
    width = max(max(counts), 1)
    order = torch.randperm(pages, generator=g, device=DEVICE).to(torch.int32)
    first = torch.tensor(_starts(counts)[:-1], device=DEVICE)
    column = torch.arange(width, device=DEVICE)
    # entries past a sequence's pages are never used
    table = torch.where(column < torch.tensor(counts, device=DEVICE)[:, None],
                        order[(first[:, None] + column).clamp(max=pages - 1)].int(), -1).int()
    lens = [n + t for t, n in zip(news, kvs)]
    s = {"op": case["op"], "type": type, "page": page, "x": x, "table": table, "max_new": max(news),
         "max_kv": max(max(lens), 1), "tokens": sum(news), "cu": _ints(_starts(news)), "kv_len": _ints(lens)}
    if case["op"] == "keep":
        _prepare_keep(case, g, s, news, kvs, pages)
    else:
        channel = torch.exp(randn(2, heads, dim)) * torch.tensor([0.5, 0.25], device=DEVICE)[:, None, None]
        for i, name in enumerate("kv"):
            if case["op"] == "rotary":
                s[name] = torch.zeros(pages, page, heads, dim, dtype=torch.uint8 if size == 1 else torch.int16,
                                      device=DEVICE).view(dtype)
                s[name + "_scale"] = torch.full((pages, heads, page), 127, dtype=torch.uint8,
                                                device=DEVICE) if size == 1 else None
                s[name + "_new"] = (randn(s["tokens"], heads, dim) * channel[i]).to(x)
                continue
            values = randn(pages, page, heads, dim) * channel[i]
            if size == 1:
                s[name], k = _quantise(values.to(x), type)
                s[name + "_scale"] = (k + 127).to(torch.uint8).transpose(1, 2).contiguous()
            else:
                s[name], s[name + "_scale"] = values.to(dtype), None
            del values
        s["q"] = randn(s["tokens"], case["heads"], dim).to(x)
    if case["op"] == "rotary":
        frequencies, s["magnitude"] = _frequencies(case)
        s["frequencies"], s["interleaved"] = frequencies.to(DEVICE), case["interleaved"]
        b, pos = _rows(s)
        s["position"] = (pos + case["ahead"]).int() if case["ahead"] else None
    if case["op"] == "tree":
        # random trees with a bias to the tokens before: parent of token i among -1 .. i - 1
        b, pos = _rows(s)
        i = pos - (s["kv_len"] - (s["cu"][1:] - s["cu"][:-1]))[b]
        u = torch.rand(s["tokens"], generator=g, device=DEVICE)
        s["parents"] = torch.minimum(((1 - u * u) * (i + 1)).floor().int() - 1, i.int() - 1).contiguous()
        s["window"], s["scale"] = case["window"], 1.0 / math.sqrt(dim)
    if own:
        import lossless_kv_cache_gb300 as sz

        if case["op"] == "keep":
            per_layer = [[t[i] if t is not None else None for t in (s["k"], s["v"], s["k_scale"], s["v_scale"])]
                         for i in range(case["layers"])]
            s["layers"] = sz.KVLayers([sz.KVCache(*t) for t in per_layer])
        else:
            s["cache"] = sz.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
            s["out"] = torch.empty_like(s["q"])
        s["batch"] = sz.KVBatch(s["cu"], s["kv_len"], s["table"], s["tokens"], s["max_new"], s["max_kv"])
        s["status"] = torch.zeros(4, dtype=torch.int32, device=DEVICE)
        if case["op"] == "rotary":
            s["rotary"] = sz.KVRotary(frequencies, interleaved=case["interleaved"], magnitude=s["magnitude"])
        if case["op"] == "tree":
            s["lse"] = torch.empty(s["tokens"], case["heads"], dtype=torch.float32, device=DEVICE)
            s["tree"] = sz.KVTree(s["batch"], window=case["window"])
            s["bufs"] = sz.KVAttentionBuffers(s["cache"], s["batch"], case["heads"])
    return s


# --------------------------------------------------------------------- run

def _rows(s):
    """Sequence and cache position of every packed row: a sequence's rows are its last positions."""
    t = torch.arange(s["tokens"], device=DEVICE, dtype=torch.int32)
    b = torch.searchsorted(s["cu"], t, right=True) - 1
    return b, s["kv_len"][b].long() - (s["cu"][b + 1] - t).long()


def _place(s, b, pos):
    """The pool's token slots of positions `pos` of sequences `b`."""
    return s["table"][b, pos // s["page"]].long() * s["page"] + pos % s["page"]


def _plain_extend(s):
    page, table = s["page"], s["table"]
    new, n, held = s["new"].long(), s["kv_len"].long(), s["held"].long()
    n = n + new - (s["drop"].long() if s["drop"] is not None else 0)
    need = (n + page - 1) // page
    more, less = (need - held).clamp(min=0), (held - need).clamp(min=0)
    column = torch.arange(table.shape[1], device=DEVICE)
    # pages given up go on top of the list, those of the last sequence first and a sequence's last page first
    top = s["count"].long() + less.sum()
    given = (column >= need[:, None]) & (column < held[:, None])
    at = top - less.cumsum(0)[:, None] + held[:, None] - 1 - column
    s["free"][at[given]] = table[given]
    # and pages are taken from the top, by the first sequence first
    taken = (column >= held[:, None]) & (column < need[:, None])
    at = top - 1 - (more.cumsum(0) - more)[:, None] - (column - held[:, None])
    table[taken] = s["free"][at[taken]]
    cu = torch.nn.functional.pad(new.cumsum(0), (1, 0))
    row = torch.arange(s["tokens"], device=DEVICE)
    b = torch.searchsorted(cu, row, right=True) - 1
    pos = n[b] - (cu[b + 1] - row)
    return {"cu": cu.int(), "kv_len": n.int(), "held": need.int(), "count": (top - more.sum()).int(), "table": table,
            "free": s["free"], "position": pos.int(), "slot": table[b, pos // page].long() * page + pos % page}


def _pools(s):
    """The written pools: FP8 elements, and their scales as the powers of two that they stand for."""
    got = {"k": s["k"], "v": s["v"]}
    if s["k_scale"] is not None:
        got.update({n + "_scale": s[n + "_scale"].view(torch.float8_e8m0fnu) for n in "kv"})
    return got


def _rotated(s, x, cos, sin):
    """x (tokens, heads, dim) with its first elements rotated, in 32 bits: pairs of neighbours, or of the two halves."""
    half = cos.shape[-1]
    x = x.float()
    turned, rest = x[..., : 2 * half], x[..., 2 * half:]
    if s["interleaved"]:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = turned[..., :half], turned[..., half:]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, rest], -1)


def _plain_rotary(s):
    b, pos = _rows(s)
    at, page = _place(s, b, pos), s["page"]
    angle = (pos if s["position"] is None else s["position"]).double()[:, None] * s["frequencies"]
    cos, sin = ((f(angle) * s["magnitude"]).float()[:, None] for f in (torch.cos, torch.sin))
    rows = {"k": _rotated(s, s["k_new"], cos, sin), "v": s["v_new"].float()}
    for name, x in rows.items():
        pool = s[name]
        pages, _, heads, dim = pool.shape
        if s[name + "_scale"] is None:
            pool.view(pages * page, heads, dim)[at] = x.to(pool.dtype)
        else:
            bits, k = _quantise(x, s["type"])
            pool.view(torch.uint8).view(pages * page, heads, dim)[at] = bits.view(torch.uint8)
            s[name + "_scale"][at // page, :, at % page] = (k + 127).to(torch.uint8)
    return {"q": _rotated(s, s["q"], cos, sin).to(s["x"]), **_pools(s)}


def _plain_tree(s):
    q = s["q"]
    tokens, heads, dim = q.shape
    kv_heads, most_new, most_kv = s["k"].shape[2], s["max_new"], s["max_kv"]
    group, batch = heads // kv_heads, s["kv_len"].numel()
    n, new = s["kv_len"].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    # (batch, token, ancestor or the token itself), the tree's tokens padded to the largest tree
    i = torch.arange(most_new, device=DEVICE)
    there = i < new[:, None]
    row = (s["cu"][:-1, None] + i).long().clamp(max=tokens - 1)
    parent = torch.where(there, s["parents"][row].long(), -1)
    reach = ((parent[..., None] == i) | (i[:, None] == i)).float()
    for _ in range(max(1, (most_new - 1).bit_length())):  # chains of twice the length at a time
        reach = (torch.matmul(reach, reach) > 0).float()
    depth = reach.sum(-1).long() - 1
    reach = reach > 0
    position = (n - new)[:, None] + depth
    if s["window"]:
        reach = reach & (depth[..., None] - depth[:, None] < s["window"])
    # keys and values, padded to the longest sequence; places past a sequence's end hold nothing
    pos = torch.arange(most_kv, device=DEVICE)
    held = pos < n[:, None]
    at = torch.where(held, _place(s, torch.arange(batch, device=DEVICE)[:, None], pos), 0)
    zero = torch.zeros((), device=DEVICE)
    k, v = (torch.where(held[..., None, None], _values(s[x], s[x + "_scale"], at, s["type"]), zero) for x in "kv")
    query = q[row].float().view(batch, most_new, kv_heads, group, dim).transpose(1, 2)
    scores = torch.matmul(query.reshape(batch, kv_heads, most_new * group, dim), k.permute(0, 2, 3, 1))
    scores = scores.view(batch, kv_heads, most_new, group, most_kv).mul_(s["scale"])
    # a token sees what was there before the tree (within its window), its ancestors and itself
    j = (pos - (n - new)[:, None]).clamp(0, most_new - 1)
    before = pos < (n - new)[:, None]
    seen = torch.where(before[:, None], True, reach.gather(2, j[:, None].expand(-1, most_new, -1)))
    seen = seen & held[:, None] & there[..., None]
    if s["window"]:
        seen = seen & (~before[:, None] | (pos > position[..., None] - s["window"]))
    scores.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True)
    low = torch.where(torch.isfinite(top), top, zero)
    weight = scores.sub_(low).exp_()
    total = weight.sum(-1, keepdim=True)
    out = torch.matmul(weight.view(batch, kv_heads, most_new * group, most_kv), v.transpose(1, 2))
    out = out.view(batch, kv_heads, most_new, group, dim) / torch.where(total > 0, total, zero + 1)
    lse = (low + total.log()).squeeze(-1)
    packed = torch.nonzero(there.reshape(-1)).squeeze(-1)
    out = out.transpose(1, 2).reshape(batch * most_new, heads, dim)[packed]
    lse = lse.transpose(1, 2).reshape(batch * most_new, heads)[packed]
    return {"out": out.to(s["x"]), "lse": lse, "position": position.reshape(-1)[packed].int()}


def _plain_keep(s):
    b, pos = _rows(s)
    i = torch.arange(s["tokens"], device=DEVICE) - s["cu"][b]
    moved = i < s["kept"][b]
    b, pos, i = b[moved], pos[moved], i[moved]
    to, source = _place(s, b, pos), _place(s, b, pos - i + s["path"][moved])
    page = s["page"]
    for name in "kv":
        pool = s[name].view(torch.uint8 if s[name + "_scale"] is not None else torch.int16)
        layers, pages, _, heads, dim = pool.shape
        flat = pool.view(layers, pages * page, heads, dim)
        flat[:, to] = flat[:, source]
        if s[name + "_scale"] is not None:
            scale = s[name + "_scale"]
            scale[:, to // page, :, to % page] = scale[:, source // page, :, source % page]
    return _kept_pools(s)


def _kept_pools(s):
    got = {"k": s["k"], "v": s["v"]}
    if s["k_scale"] is not None:
        got.update(k_scale=s["k_scale"], v_scale=s["v_scale"])
    return got


def run(s):
    if not own:
        return {"extend": _plain_extend, "rotary": _plain_rotary, "tree": _plain_tree, "keep": _plain_keep}[s["op"]](s)
    import lossless_kv_cache_gb300 as sz

    if s["op"] == "extend":
        after, step = s["after"], s["step"]
        sz.kv_extend(s["pages"], s["new"], step, drop=s["drop"], after=after)
        return {"cu": step.cu_tokens, "kv_len": after.kv_len, "held": after.held, "count": after.count,
                "table": s["table"], "free": s["free"], "position": step.position, "slot": step.slot}
    if s["op"] == "rotary":
        sz.kv_rotary_write(s["cache"], s["batch"], s["rotary"], s["q"], s["out"], s["k_new"], s["v_new"], s["status"],
                           positions=s["position"])
        return {"q": s["out"], **_pools(s)}
    if s["op"] == "tree":
        sz.kv_tree(s["batch"], s["parents"], s["tree"])
        sz.kv_tree_attention(s["cache"], s["batch"], s["tree"], s["q"], s["out"], s["bufs"], s["scale"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"], "position": s["tree"].position}
    sz.kv_keep(s["layers"], s["batch"], s["path"], s["kept"], s["status"])
    return _kept_pools(s)


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
    """Pool page and offset of every packed row, found one sequence at a time, and its position."""
    cu, n, table = s["cu"].tolist(), s["kv_len"].tolist(), s["table"].cpu()
    pages, offsets, places = [], [], []
    for b in range(len(n)):
        pos = torch.arange(n[b] - (cu[b + 1] - cu[b]), n[b])
        pages.append(table[b, torch.div(pos, case["page"], rounding_mode="floor")].long())
        offsets.append(pos % case["page"])
        places.append(pos)
    return tuple(torch.cat(p).to(DEVICE) for p in (pages, offsets, places))


def _exact_rotary(case, s):
    page, offset, place = _exact_rows(case, s)
    half = case["rot"] // 2
    f, magnitude = _frequencies(case)
    turn = (place.double() + case["ahead"])[:, None] * f.to(DEVICE)
    spin = torch.polar(torch.full_like(turn, magnitude), turn)[:, None]

    def rotated(x):
        x = x.double()
        part = x[..., : case["rot"]]
        part = part.unflatten(-1, (half, 2)) if case["interleaved"] else part.unflatten(-1, (2, half)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(part.contiguous()) * spin)
        z = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
        return torch.cat([z, x[..., case["rot"]:]], -1)

    got = {"q": rotated(s["q"])}
    fp8 = TYPES[case["type"]][1] == 1
    for name, x in (("k", rotated(s["k_new"])), ("v", s["v_new"].double())):
        pool = torch.zeros(s[name].shape, dtype=torch.float64, device=DEVICE)
        if fp8:
            largest = 57344.0 if case["type"] == "e5m2" else 448.0
            most = x.abs().amax(-1, keepdim=True)
            # smallest k with most <= largest * 2^k, found by counting from a guess that is at most one off
            k = torch.floor(torch.log2(most.clamp(min=1e-300) / largest) - 1e-6)
            k = torch.where(most <= largest * _power64(k), k, k + 1)
            k = torch.where(most > 0, k, torch.zeros_like(k)).clamp(-126, 127)
            x = _rounded(x / _power64(k), case["type"])
        pool[page, offset] = x
        got[name] = pool
    if fp8:
        got.update(k_scale=None, v_scale=None)
    return got


def _exact_pool(s, name):
    """A whole pool's values in doubles (pages, page tokens, heads, dim)."""
    x = s[name].to(torch.float32).double()
    if s[name + "_scale"] is None:
        return x
    return x * _power64(s[name + "_scale"].int() - 127).transpose(1, 2)[..., None]


def _exact_tree(case, s):
    pools = [_exact_pool(s, name) for name in "kv"]
    cu, lens, parents = s["cu"].tolist(), s["kv_len"].tolist(), s["parents"].tolist()
    group = case["heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEVICE)
    for b, n in enumerate(lens):
        t = cu[b + 1] - cu[b]
        if not t:
            continue
        first = n - t
        # what each token does not see, walking up its branch
        hidden = torch.ones(t, n, dtype=torch.bool)
        for i in range(t):
            branch = [i]
            while parents[cu[b] + branch[-1]] >= 0:
                branch.append(parents[cu[b] + branch[-1]])
            position = first + len(branch) - 1
            hidden[i, max(0, position - case["window"] + 1) if case["window"] else 0: first] = False
            for up, j in enumerate(branch):
                hidden[i, first + j] = bool(case["window"]) and up >= case["window"]
        hidden = hidden.to(DEVICE)
        pages = s["table"][b, : -(-n // case["page"])].long()
        for h in range(case["kv_heads"]):
            k, v = (x[pages, :, h].reshape(-1, case["dim"])[:n] for x in pools)
            q = s["q"][cu[b]: cu[b] + t, h * group: (h + 1) * group].double()
            z = torch.einsum("tgd,nd->tgn", q, k) / math.sqrt(case["dim"])
            z = z.masked_fill(hidden[:, None], -math.inf)
            norm = torch.logsumexp(z, -1)
            out[cu[b]: cu[b] + t, h * group: (h + 1) * group] = torch.einsum("tgn,nd->tgd", torch.exp(z - norm[..., None]), v)
            lse[cu[b]: cu[b] + t, h * group: (h + 1) * group] = norm
    return {"out": out, "lse": lse, "position": None}


def _exact_keep(case, s):
    cu, lens, table = s["cu"].tolist(), s["kv_len"].tolist(), s["table"].tolist()
    path, kept = s["path"].tolist(), s["kept"].tolist()
    page = case["page"]
    got = {name: s[name].float().double() for name in "kv"}
    if s["k_scale"] is not None:
        got.update(k_scale=None, v_scale=None)
    to, source = [], []
    for b, n in enumerate(lens):
        first = n - (cu[b + 1] - cu[b])
        for i in range(kept[b]):
            to.append((table[b][(first + i) // page], (first + i) % page))
            j = first + path[cu[b] + i]
            source.append((table[b][j // page], j % page))
    to, source = torch.tensor(to, device=DEVICE).T, torch.tensor(source, device=DEVICE).T
    for name in "kv":
        got[name][:, to[0], to[1]] = got[name][:, source[0], source[1]]
    return got


def exact(case, seed):
    if case["op"] == "extend":
        return None
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "tree": _exact_tree, "keep": _exact_keep}[case["op"]](case, s)
