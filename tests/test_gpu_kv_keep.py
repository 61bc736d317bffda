"""GPU: accepted branches moved to the front of the drafted tokens, bit by bit."""
import random

import pytest
import torch

import lossless_kv_cache_gb300 as sz
from tests.kv_reference import RAW, Step

pytestmark = pytest.mark.gpu

BF16, FP16, E5M2, E4M3 = torch.bfloat16, torch.float16, torch.float8_e5m2, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib(splitzip_lib):
    assert torch.cuda.is_available()
    return splitzip_lib


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def bits(cache):
    """(K, V[, scales as (page, token, head)]) of a cache on the CPU."""
    raw = torch.uint8 if cache.k_scale is not None else torch.int16
    got = [t.view(raw).cpu().clone() for t in (cache.k, cache.v)]
    if cache.k_scale is not None:
        got += [t.cpu().transpose(1, 2).clone() for t in (cache.k_scale, cache.v_scale)]
    return got


def layers_of(step, count, layout="nhd"):
    """`count` caches of the step's geometry, of random bits."""
    caches = [step.cache]
    while len(caches) < count:
        c = sz.KVCache.empty(step.pages, step.page, step.kv_heads, step.dim, step.dtype)
        if layout == "hnd":
            pools = [t.view(RAW[step.dtype]).transpose(1, 2).contiguous().view(step.dtype).transpose(1, 2)
                     for t in (c.k, c.v)]
            c = sz.KVCache(*pools, c.k_scale, c.v_scale)
        caches.append(c)
    for n, c in enumerate(caches):
        g = torch.Generator(device="cuda").manual_seed(n)
        for t in (c.k, c.v, c.k_scale, c.v_scale):
            if t is not None:
                raw = t.view(torch.uint8 if t.element_size() == 1 else torch.int16)
                raw.copy_(torch.randint(0, 255, raw.shape, generator=g, device="cuda").to(raw.dtype) * (1 if n % 2 else 3))
    return caches


def branch_of(step, seed):
    """(path, kept) of random ascending branches."""
    r = random.Random(seed)
    path, kept = [], []
    for t, n in step.lens:
        k = r.choice([0, t, r.randint(0, t)]) if n >= t else 0
        chosen = sorted(r.sample(range(t), k))
        path += chosen + [r.choice([-1, 5, 1 << 30]) for _ in range(t - k)]  # what is past the count is not looked at
        kept.append(k)
    return path, kept


def moved(step, before, path, kept):
    want = [x.clone() for x in before]
    for b, (t, n) in enumerate(step.lens):
        for i in range(kept[b]):
            to, source = step.place(b, n - t + i), step.place(b, n - t + path[step.cu[b] + i])
            for x, y in zip(want, before):
                x[to] = y[source]
    return want


def check(step, layers=1, layout="nhd", seed=0, path=None, kept=None):
    caches = layers_of(step, layers, layout)
    before = [bits(c) for c in caches]
    if path is None:
        path, kept = branch_of(step, seed)
    status = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    sz.kv_keep(sz.KVLayers(caches), step.batch, ints(path + [7] * (step.tokens - len(path))), ints(kept), status)
    torch.cuda.synchronize()
    assert int(status[0]) == sz.OK
    for c, old in zip(caches, before):
        for got, want in zip(bits(c), moved(step, old, path, kept)):
            assert torch.equal(got, want)


LENS = [(7, 60), (1, 1), (0, 9), (40, 99), (16, 16), (100, 217), (2, 2)]


@pytest.mark.parametrize("dtype", [BF16, FP16, E5M2, E4M3])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [1, 16, 64])
def test_types_and_pages(dtype, dim, page):
    for seed in range(3):
        check(Step(dtype, LENS, dim=dim, page=page), seed=seed)


@pytest.mark.parametrize("kv_heads", [1, 2, 3, 4, 5, 8, 16])
def test_heads(kv_heads):
    check(Step(E5M2, LENS, kv_heads=kv_heads))
    check(Step(FP16, LENS, kv_heads=kv_heads, dim=64))


@pytest.mark.parametrize("layers", [2, 64, 65, 130])
def test_layers(layers):
    check(Step(E4M3, [(7, 20), (12, 30)], dim=64), layers)
    check(Step(BF16, [(7, 20), (12, 30)], dim=64, layout="hnd"), layers, "hnd")


def test_long_moves_by_one():
    """Every source is the next token's destination."""
    t = 90
    check(Step(BF16, [(t, t + 5)]), path=list(range(1, t)) + [0], kept=[t - 1])
    check(Step(E5M2, [(t, t)], page=4), path=list(range(9, t)) + [0] * 9, kept=[t - 9])


def test_many_sequences_and_rows_behind_the_last():
    check(Step(E5M2, [(1 + i % 5, 9 + i % 40) for i in range(700)], kv_heads=1, dim=64))
    check(Step(E5M2, LENS, spare_rows=9))


def test_what_is_out_of_range_is_left_as_it_was():
    lens = [(6, 30), (5, 20), (4, 3)]
    good = [1, 3, 5, 0, 0, 0, 0, 2, 4, 0, 0, 0, 0, 0, 0]
    for path, kept in (([3, 1, 5] + good[3:], [3, 3, 0]), ([1, 1, 5] + good[3:], [3, 3, 0]),
                       ([-1, 1, 5] + good[3:], [3, 3, 0]), ([1, 3, 6] + good[3:], [3, 3, 0]), (good, [7, 3, 0]),
                       (good, [-1, 3, 0]), (good, [1 << 30, 3, 0]), ([0, 1, 2, 3, 4, 1 << 30] + good[6:], [6, 3, 0])):
        step = Step(E5M2, lens)
        before = bits(step.cache)
        status = torch.zeros(4, dtype=torch.int32, device="cuda")
        sz.kv_keep(sz.KVLayers([step.cache]), step.batch, ints(path), ints(kept), status)
        assert int(status[0]) == sz.ERR_INVALID_ARG
        want = moved(step, before, path, [0, 3, 0])  # the other sequence's are moved
        assert all(torch.equal(a, b) for a, b in zip(bits(step.cache), want))
    # tokens without a place
    step = Step(E5M2, lens)
    before = bits(step.cache)
    sz.kv_keep(sz.KVLayers([step.cache]), step.batch, ints(good), ints([0, 0, 1]), status)
    assert int(status[0]) == sz.ERR_INVALID_ARG
    assert all(torch.equal(a, b) for a, b in zip(bits(step.cache), before))
    # a page out of range: skipped
    step = Step(BF16, [(20, 40)])
    before = bits(step.cache)
    step.batch.page_table[0, 2] = step.pages
    path = list(range(2, 20)) + [0, 0]
    sz.kv_keep(sz.KVLayers([step.cache]), step.batch, ints(path), ints([18]), status)
    assert int(status[0]) == sz.ERR_INVALID_ARG
    want = [x.clone() for x in before]
    for i in range(18):
        if (20 + i) // 16 != 2 and (20 + path[i]) // 16 != 2:
            for x, y in zip(want, before):
                x[step.place(0, 20 + i)] = y[step.place(0, 20 + path[i])]
    assert all(torch.equal(a, b) for a, b in zip(bits(step.cache), want))
    # entries
    step = Step(BF16, lens)
    before = bits(step.cache)
    step.batch.kv_len[0] = 1 << 29
    sz.kv_keep(sz.KVLayers([step.cache]), step.batch, ints(good), ints([3, 0, 0]), status)
    assert int(status[0]) == sz.ERR_INVALID_ARG
    assert all(torch.equal(a, b) for a, b in zip(bits(step.cache), before))


def test_helpers_refuse_what_does_not_go_together():
    step = Step(BF16, [(3, 9), (2, 8)])
    layers = sz.KVLayers([step.cache])
    path, kept = ints([0] * 5), ints([0, 0])
    for p, k in ((ints([0] * 4), kept), (path, ints([0])), (path.long(), kept), (path, kept.cpu()),
                 (ints([0] * 10)[::2], kept)):
        with pytest.raises(ValueError):
            sz.kv_keep(layers, step.batch, p, k, step.status)
    other = Step(BF16, [(3, 9), (2, 8)], page=4)
    with pytest.raises(sz.SplitZipError):
        sz.kv_keep(sz.KVLayers([step.cache, other.cache]), step.batch, path, kept, step.status)


@pytest.mark.parametrize("dtype", [E5M2, E4M3])
def test_scales_given_twice_are_refused(dtype):
    """They would be moved twice, at once; nothing is launched."""
    step = Step(dtype, [(5, 30), (2, 8)])
    other = layers_of(step, 2)[1]
    a = step.cache
    path, kept = ints([1, 3, 4, 0, 0, 1, 0]), ints([3, 1])
    for caches in ([sz.KVCache(a.k, a.v, a.k_scale, a.k_scale)],
                   [a, sz.KVCache(other.k, other.v, a.k_scale, other.v_scale)],
                   [a, sz.KVCache(other.k, other.v, other.k_scale, a.v_scale)],
                   [a, sz.KVCache(other.k, other.v, a.v_scale, other.v_scale)]):
        before = [bits(c) for c in caches]
        step.status.fill_(-1)
        with pytest.raises(sz.SplitZipError):
            sz.kv_keep(sz.KVLayers(caches), step.batch, path, kept, step.status)
        torch.cuda.synchronize()
        assert int(step.status[0]) == -1
        assert all(torch.equal(x, y) for c, old in zip(caches, before) for x, y in zip(bits(c), old))
    check(Step(dtype, LENS), 2)


@pytest.mark.parametrize("kept", [0, 1, 4])
def test_tokens_without_a_place_are_reported_whatever_is_kept(kept):
    step = Step(E5M2, [(4, 3), (3, 20), (0, 0)])
    before = bits(step.cache)
    path = [0, 1, 2, 3, 1, 2, 0]
    sz.kv_keep(sz.KVLayers([step.cache]), step.batch, ints(path), ints([kept, 2, 0]), step.status)
    assert int(step.status[0]) == sz.ERR_INVALID_ARG
    assert all(torch.equal(a, b) for a, b in zip(bits(step.cache), moved(step, before, path, [0, 2, 0])))
