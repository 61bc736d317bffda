"""GPU: tree attention over caches long enough that every ring of the kernels
goes round, and over FP8 pages whose scales differ little and much.  Trees are
chains here, whose rows see what causal attention shows them, so that the long
reference serves; tests/test_gpu_kv_tree.py has other shapes."""
import math

import pytest
import torch

import lossless_kv_cache_gb300 as sz
from tests.kv_long_reference import LongStep, attention64, vary_scales
from tests.kv_reference import RAW, check_attention, half_step
from tests.test_gpu_kv_weights import most_weight, shift_scales

pytestmark = pytest.mark.gpu

BF16, FP16, E5M2, E4M3 = torch.bfloat16, torch.float16, torch.float8_e5m2, torch.float8_e4m3fn
TYPES = [(BF16, BF16), (FP16, FP16), (E5M2, BF16), (E5M2, FP16), (E4M3, BF16), (E4M3, FP16)]


@pytest.fixture(scope="module", autouse=True)
def _lib(splitzip_lib):
    assert torch.cuda.is_available()
    return splitzip_lib


def run(step, q, scale, window=0):
    """(out, lse) of chains, twice, bit for bit the same."""
    parents = torch.cat([torch.arange(-1, t - 1) for t, _ in step.lens]).int().cuda()
    tree = sz.KVTree(step.batch, window)
    sz.kv_tree(step.batch, parents, tree)
    bufs = sz.KVAttentionBuffers(step.cache, step.batch, q.shape[1])
    first = None
    for _ in range(2):
        out = torch.full_like(q, 77.0)
        lse = torch.full(q.shape[:2], 77.0, device="cuda")
        sz.kv_tree_attention(step.cache, step.batch, tree, q, out, bufs, scale, lse=lse)
        torch.cuda.synchronize()
        assert int(tree.status[0]) == sz.OK and int(bufs.status[0]) == sz.OK
        if first is not None:
            assert torch.equal(out.view(torch.int16), first[0].view(torch.int16))
            assert torch.equal(lse.view(torch.int32), first[1].view(torch.int32))
        first = (out, lse)
    return first


def check(step, group=4, scale=None, window=0):
    scale = 0.3 / math.sqrt(step.dim) if scale is None else scale  # flat enough that every key counts
    q = torch.randn(step.tokens, step.kv_heads * group, step.dim, generator=step.gen).to(step.x)
    out, lse = run(step, q.cuda(), scale, window)
    check_attention(step, out, lse, attention64(step, q, scale, True, window), FP16 if step.dtype == FP16 else BF16)


# 8 kv heads and 4 query heads each, 128 rows a tile and 128 keys a unit, over 152 blocks: pieces of
# up to 40 units, several pieces of up to 12 a block, many of 1 to 4; more sequences than a warp deals
LONG = [(32, 9000), (20, 3000), (9, 1500)]
SEVERAL = [(17 + b % 12, 1500 - 7 * b) for b in range(24)]
MANY = [(9 + b % 3, 100 + 2 * b) for b in range(150)]


def plant_nan(step):
    """NaN in V at positions that only some rows see, and at one that all do."""
    for b, (t, n) in enumerate(step.lens):
        step.set_value("v", b, n - t, b % 8, 5, math.nan)
        step.set_value("v", b, n - 1, b % 8, 9, math.nan)
        if b % 3 == 0:
            step.set_value("v", b, n // 3, (b + 1) % 8, 11, math.nan)


@pytest.mark.parametrize("lens", [LONG, SEVERAL, MANY], ids=["long", "several", "many"])
@pytest.mark.parametrize("dtype,x", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
def test_long_shares(dtype, x, dim, lens):
    step = LongStep(dtype, lens, dim=dim, x=x)
    check(step)
    check(step, window=500)
    plant_nan(step)
    check(step)


@pytest.mark.parametrize("page", [1, 8, 16, 64, 512])
@pytest.mark.parametrize("dtype", [BF16, E5M2])
def test_pages(dtype, page):
    check(LongStep(dtype, [(32, 2500), (10, 777), (21, 130)], page=page))


@pytest.mark.parametrize("group,t", [(1, 17), (1, 128), (3, 7), (3, 42), (5, 25), (7, 18), (16, 8), (64, 2)])
@pytest.mark.parametrize("dtype", [FP16, E4M3])
def test_rows_of_a_tile(dtype, group, t):
    """Up to 128 rows, groups that do not divide them."""
    check(LongStep(dtype, [(t, 4500), (max(1, t // 2), 4100), (1, 60)], kv_heads=2), group=group)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_more_rows_than_a_tile(dtype):
    check(LongStep(dtype, [(33, 3000), (64, 2000), (5, 1000)], kv_heads=4))
    check(LongStep(dtype, [(200, 3000), (1, 2000)], kv_heads=2), group=2)


@pytest.mark.parametrize("lens", [LONG, SEVERAL], ids=["long", "several"])
@pytest.mark.parametrize("dtype,x", [(E5M2, BF16), (E4M3, FP16), (E4M3, BF16)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("k_low,k_high,v_low,v_high", [(-3, 3, -3, 3), (-30, 0, -2, 2), (-1, 1, -25, 5)])
def test_a_scale_for_each_key(dtype, x, dim, lens, k_low, k_high, v_low, v_high):
    """Scales near enough to be brought to one a unit, and keys that keep their own."""
    step = LongStep(dtype, lens, dim=dim, x=x)
    vary_scales(step, "k", k_low, k_high)
    vary_scales(step, "v", v_low, v_high)
    check(step)
    plant_nan(step)
    check(step)


def own_size(step, q, out, ref, scale):
    """Errors held to the result's own size.  As for kv_reference.check_attention, but for weights
    that FP16 holds in its subnormal steps, 2^-24.  The largest is at least 2^7 (the reference lags
    the maximum by 2^8 at most) of the largest scale of a unit whose keys are within 2^6 of it, and V's
    elements are up to 2^15.8 and, of the largest key's row, 2^14.8 and more: each is off by 2^-25 /
    2^(7 + 14.8 - 6 - 15.8) <= 2^-24 of the largest product of a weight and a value."""
    r_out, _, mag, size = ref
    keys = max(n for _, n in step.lens)
    score = (step.dim + 4) * 2.0 ** -23 * size + 2.0 ** -21
    rel = half_step(FP16) + 2 * score[..., None] + 2 * (keys / 8 + 16) * 2.0 ** -23
    tol = rel * mag + half_step(BF16) * (1 + rel) * r_out.abs()
    tol = tol + keys * 2.0 ** -24 * most_weight(step, q, scale)[..., None]
    worst = float(((out.double().cpu() - r_out).abs() / tol).max())
    assert worst <= 1, worst


@pytest.mark.parametrize("dtype", [E5M2, E4M3])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("small", [0, -10, -40, -75])
@pytest.mark.parametrize("zeros", [False, True])
def test_small_values_and_rows_of_zeros(dtype, dim, small, zeros):
    """However small the values of V are; a row of zeros is written with the scale 2^0."""
    lens = [(9, 900), (12, 300)]
    step = LongStep(dtype, lens, dim=dim, kv_heads=2)
    step.host = {name: x.cpu() for name, x in step.host.items()}
    step.held = lambda b, name: step.host[name][step.table[b, : -(-lens[b][1] // step.page)].long()].reshape(
        -1, step.kv_heads, dim)[: lens[b][1]]
    shift_scales(step, "v", small)
    u = torch.randn(dim, generator=step.gen, dtype=torch.float64)
    q = (u + 0.3 * torch.randn(step.tokens, 8, dim, generator=step.gen)).to(BF16)
    scale = 1 / math.sqrt(dim)
    aligned = (2.0 * torch.sign(u) * 10 / (scale * u.abs().sum() * 2.0)).float().to(dtype)  # a score of about 10
    if zeros:
        for b, (t, n) in enumerate(lens):
            for pos in (0, 5, n // 2, n - t - 1, n - t):
                pg, off = step.place(b, pos)
                step.cache.k.view(RAW[dtype])[pg, off] = aligned.view(RAW[dtype]).cuda()
                step.cache.k_scale[pg, :, off] = 127
                step.host["k"][pg, off] = aligned.double()
                step.cache.v.view(RAW[dtype])[pg, off] = 0
                step.cache.v_scale[pg, :, off] = 127
                step.host["v"][pg, off] = 0.0
    out, _ = run(step, q.cuda(), scale)
    own_size(step, q, out, attention64(step, q, scale), scale)


@pytest.mark.parametrize("dtype", [E5M2, E4M3])
def test_values_that_grow_along_the_sequence(dtype):
    """From unit to unit, and far past the first's: the reference follows."""
    for rise in (3, -3, 9, -9):
        step = LongStep(dtype, [(12, 1500), (5, 700)], kv_heads=2)
        for b, (t, n) in enumerate(step.lens):
            for pos in range(n):
                pg, off = step.place(b, pos)
                e = max(-40, min(40, rise * (pos // 128)))
                step.cache.v_scale[pg, :, off] = (step.cache.v_scale[pg, :, off].int() + e).to(torch.uint8)
                step.host["v"][pg, off] = torch.ldexp(step.host["v"][pg, off], torch.tensor(e, device="cuda"))
        check(step)


@pytest.mark.parametrize("dtype,x", [(BF16, BF16), (FP16, FP16), (E5M2, BF16), (E5M2, FP16)])
def test_infinite_scores(dtype, x):
    """+infinity: the rows that see it are NaN; -infinity: a weight of 0."""
    for value in (math.inf, -math.inf):
        step = LongStep(dtype, [(12, 600), (30, 300)], kv_heads=2, x=x)
        q = torch.randn(step.tokens, 8, 128, generator=step.gen).to(step.x)
        q[:, :, 7] = q[:, :, 7].abs() + 1
        at = [n - 2 for _, n in step.lens]
        for b, pos in enumerate(at):
            for h in range(2):
                step.set_value("k", b, pos, h, 7, value)
        out, lse = run(step, q.cuda(), 0.05)
        seen = torch.zeros(step.tokens, dtype=torch.bool)
        for b, (t, n) in enumerate(step.lens):
            seen[step.cu[b + 1] - 2: step.cu[b + 1]] = value > 0
        assert bool(torch.isnan(out.cpu()[seen]).all()) and bool(torch.isnan(lse.cpu()[seen]).all())
        ref, ref_lse, mag, _ = attention64(step, q, 0.05)
        step.host["k"][~torch.isfinite(step.host["k"])] = 0.0
        size = attention64(step, q, 0.05)[3]
        keep = ~seen
        check_attention(step, out.cpu()[keep], lse.cpu()[keep],
                        (ref.nan_to_num(0.0)[keep], ref_lse[keep], mag.nan_to_num(0.0)[keep], size[keep]),
                        FP16 if x == FP16 and dtype == FP16 else BF16)


@pytest.mark.parametrize("dtype", [E5M2, E4M3, BF16])
def test_looks_at_its_own_values(dtype):
    """Units that look at V before their product, for NaN or for rows of zeros, the one tile of it in
    turns: the same bits however the groups' steps fall."""
    for seed in range(3):
        step = LongStep(dtype, [(8 + b % 4, 100 + 3 * b) for b in range(150)], seed=seed)
        plant_nan(step)
        q = torch.randn(step.tokens, 32, 128, generator=step.gen).to(step.x).cuda()
        first = run(step, q, 0.03)
        for _ in range(25):
            out, lse = run(step, q, 0.03)
            assert torch.equal(out.view(torch.int16), first[0].view(torch.int16)) and torch.equal(lse, first[1])
        if dtype != BF16:
            vary_scales(step, "v", -12, 0)
            first = run(step, q, 0.03)
            for _ in range(25):
                out, lse = run(step, q, 0.03)
                assert torch.equal(out.view(torch.int16), first[0].view(torch.int16)) and torch.equal(lse, first[1])


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [4, 16])
@pytest.mark.parametrize("lens,kv_heads,group", [([(5, 9000)], 1, 4), ([(8, 3000)] * 12, 2, 4), ([(32, 2500), (3, 7000)], 3, 1),
                                                 ([(2, 600), (1, 300)] * 16, 1, 16)])
def test_few_rows_do_with_the_workspace_that_they_ask_for(dtype, dim, page, lens, kv_heads, group):
    """17 to 32 rows of a sequence; nothing behind it is touched."""
    step = LongStep(dtype, lens, page=page, kv_heads=kv_heads, dim=dim)
    q = torch.randn(step.tokens, kv_heads * group, dim, generator=step.gen).to(step.x)
    parents = torch.cat([torch.arange(-1, t - 1) for t, _ in lens]).int().cuda()
    tree = sz.KVTree(step.batch)
    sz.kv_tree(step.batch, parents, tree)
    bufs = sz.KVAttentionBuffers(step.cache, step.batch, kv_heads * group)
    bufs.ws = torch.full((bufs.ws_bytes + (1 << 22),), 0xA5, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q).cuda(), torch.empty(q.shape[:2], device="cuda")
    scale = 0.3 / math.sqrt(dim)
    for _ in range(2):
        sz.kv_tree_attention(step.cache, step.batch, tree, q.cuda(), out, bufs, scale, lse=lse)
        assert int(bufs.status[0]) == sz.OK
        assert bool((bufs.ws[bufs.ws_bytes:] == 0xA5).all())
        check_attention(step, out, lse, attention64(step, q, scale), BF16)
