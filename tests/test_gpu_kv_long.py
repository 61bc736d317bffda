"""GPU: attention over caches long enough that every ring of the kernels goes
round: pieces of many units of keys, several pieces a block, all of them
against the formula in 64 bits within the documented roundings."""
import math

import pytest
import torch

import lossless_kv_cache_gb300 as sz
from tests.kv_long_reference import LongStep, attention64, vary_scales
from tests.kv_reference import check_attention

pytestmark = pytest.mark.gpu

BF16, FP16, E5M2, E4M3 = torch.bfloat16, torch.float16, torch.float8_e5m2, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib(splitzip_lib):
    assert torch.cuda.is_available()
    return splitzip_lib


def weight_type(step, group):
    """What the exponentials are rounded to for the product with V."""
    if step.x == FP16 or (step.fp8 and step.max_new * group <= 32):
        return FP16
    return BF16


def check(step, group=4, scale=None, causal=True, window=0):
    scale = 0.3 / math.sqrt(step.dim) if scale is None else scale  # flat enough that every key counts
    q = torch.randn(step.tokens, step.kv_heads * group, step.dim, generator=step.gen).to(step.x)
    dev = q.cuda()
    bufs = sz.KVAttentionBuffers(step.cache, step.batch, step.kv_heads * group)
    ref = attention64(step, q, scale, causal, window)
    first = None
    for _ in range(2):
        out = torch.full_like(dev, 77.0)
        lse = torch.full(q.shape[:2], 77.0, device="cuda")
        sz.kv_attention(step.cache, step.batch, dev, out, bufs, scale, causal=causal, window=window, lse=lse)
        torch.cuda.synchronize()
        assert int(bufs.status[0]) == sz.OK
        check_attention(step, out, lse, ref, weight_type(step, group))
        if first is not None:  # bit for bit the same each time (as integers, for NaN)
            assert torch.equal(out.view(torch.int16), first[0].view(torch.int16))
            assert torch.equal(lse.view(torch.int32), first[1].view(torch.int32))
        first = (out, lse)


# Chunks of 8 kv heads and 4 query heads each, 256 rows a tile and 128 keys a unit, over 152
# blocks: pieces of up to 40 units; three or four pieces of up to 12; eight and more of 1 to 4.
LONG = [(512, 9000), (200, 3000), (64, 1500)]
SEVERAL = [(70, 1500 - 7 * b) for b in range(24)]
MANY = [(33, 100 + 2 * b) for b in range(150)]


@pytest.mark.parametrize("lens", [LONG, SEVERAL, MANY], ids=["long", "several", "many"])
@pytest.mark.parametrize("dtype", [E5M2, E4M3])
@pytest.mark.parametrize("dim", [64, 128])
def test_chunks_with_a_scale_for_each_key(dtype, dim, lens):
    """FP16 queries over FP8 pages, whose scores take K's scales after the product: each key's
    has to be its own for as long as a unit waits for its softmax."""
    step = LongStep(dtype, lens, dim=dim, x=FP16)
    vary_scales(step, "k", -3, 3)
    check(step)
    # NaN at positions that only some rows see hold the softmax up, while the loaders go on
    for b, (t, n) in enumerate(lens):
        step.set_value("v", b, n - t, b % 8, 5, math.nan)
        step.set_value("v", b, n - 1, b % 8, 9, math.nan)
    check(step)
    check(step, window=500)


TYPES = [(BF16, BF16), (FP16, FP16), (E5M2, BF16), (E5M2, FP16), (E4M3, BF16), (E4M3, FP16)]


def plant_nan(step, every):
    """NaN in V where some of a sequence's rows see it, and before all of its rows for some."""
    for b, (t, n) in enumerate(step.lens):
        if b % every == 0 and t > 0:
            step.set_value("v", b, max(0, n - t + b % 3), b % step.kv_heads, 5, math.nan)
            step.set_value("v", b, n - 1, (b + 1) % step.kv_heads, 9, math.nan)
            if b % (2 * every) == 0:
                step.set_value("v", b, n // 3, (b + 2) % step.kv_heads, 11, math.nan)


@pytest.mark.parametrize("lens", [LONG, SEVERAL, MANY], ids=["long", "several", "many"])
@pytest.mark.parametrize("page", [16, 4])
@pytest.mark.parametrize("dtype,x", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
def test_chunks(dtype, x, dim, page, lens):
    """Every instance of the chunk kernel: 16-bit pages of eight tokens and more are read by tensor
    maps, smaller ones row by row."""
    step = LongStep(dtype, lens, dim=dim, x=x, page=page)
    if step.fp8:
        vary_scales(step, "k", -2, 2)
        vary_scales(step, "v", -2, 2)
    check(step)
    plant_nan(step, 1 if page == 16 else 7)
    check(step, window=900)


@pytest.mark.parametrize("dtype,x", TYPES)
@pytest.mark.parametrize("page", [8, 256])
def test_chunks_without_causality_and_other_pages(dtype, x, page):
    step = LongStep(dtype, [(300, 4001), (129, 2600), (40, 3333)], x=x, page=page)
    check(step, causal=False)
    check(step, causal=False, window=1000)
    check(step, group=3)


# Shares of the step kernel, 64 keys a unit, over up to 608 blocks: about 11 units of one item or
# two; 12 of several items; 12 of one item that 76 blocks share.
STEP_LONG = [(1, 3500 + 11 * b) for b in range(16)]
STEP_MANY = [(1, 190 + 4 * b) for b in range(130)]
STEP_ONE = [(1, 60007)]


@pytest.mark.parametrize("lens", [STEP_LONG, STEP_MANY, STEP_ONE], ids=["long", "many", "one"])
@pytest.mark.parametrize("page", [16, 4])
@pytest.mark.parametrize("dtype,x", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
def test_steps(dtype, x, dim, page, lens):
    """Every instance of the step kernel, by 4, 16 and 32 rows a sequence."""
    for new in (1, 4, 8):
        step = LongStep(dtype, [(new, n) for _, n in lens], dim=dim, x=x, page=page)
        if step.fp8:
            vary_scales(step, "k", -2, 2)
            vary_scales(step, "v", -2, 2)
        check(step)
        if new > 1:
            plant_nan(step, 1 if page == 16 else 7)
            check(step, window=1500)


@pytest.mark.parametrize("dtype,x", [(BF16, BF16), (E4M3, FP16)])
@pytest.mark.parametrize("most", [1, 9, 700])
def test_batches_of_thousands(dtype, x, most):
    """More sequences than one round of the chunk kernel's plan (1,024) or of the step kernel's
    scan (128) takes, with none, one or many tiles of rows in turn."""
    lens = [(min(most, (0, 1, 3, 1, 9, 1, 0, 40)[b % 8]), 1 + b * 7 % 90) for b in range(2600)]
    for b in (3, 1023, 1024, 2050, 2599):
        lens[b] = (most, 1400 + b % 5)
    step = LongStep(dtype, [(t, max(n, t)) for t, n in lens], kv_heads=2, dim=64, x=x)
    check(step, group=3)
