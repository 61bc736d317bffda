"""GPU: attention over caches long enough that every ring of the kernels goes
round: pieces of many units of keys, several pieces a block, all of them
against the formula in 64 bits within the documented roundings."""
import math

import pytest
import torch

import lossless_kv_cache_gb300 as sz
from tests.kv_long_reference import attention64, vary_scales
from tests.kv_reference import Step, check_attention

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
    step = Step(dtype, lens, kv_heads=8, dim=dim, x=FP16, spread=0.3)
    vary_scales(step, "k", -3, 3)
    check(step)
    # NaN at positions that only some rows see hold the softmax up, while the loaders go on
    for b, (t, n) in enumerate(lens):
        step.set_value("v", b, n - t, b % 8, 5, math.nan)
        step.set_value("v", b, n - 1, b % 8, 9, math.nan)
    check(step)
    check(step, window=500)
