"""GPU: the paged-cache operators and the codec together, as the example runs
them: chunks into an E5M2 cache, a lossless transfer to other pages, decoding
there, bit for bit as without the transfer."""
import pytest
import torch

import lossless_kv_cache_gb300 as sz
from examples import kv_serving

pytestmark = pytest.mark.gpu


def test_serving_example(splitzip_lib):
    out, raw, link = kv_serving.run(prompt=300, chunk=128, steps=3)
    assert out.shape == (303, kv_serving.HEADS, kv_serving.HEAD_DIM)
    assert bool(torch.isfinite(out).all())
    # 7 bits an element; 3 bytes for each zero of the last page's unwritten slots (an
    # exponent of their own) and for each element under 2^-15 of its row's largest (one in
    # 10,000 of normal values, counted as one in 1,000); headers and indices
    empty = -300 % kv_serving.PAGE_TOKENS * kv_serving.KV_HEADS * kv_serving.HEAD_DIM * 2
    assert link <= raw * 7 // 8 + 3 * (empty + raw // 1000) + 1024


def test_chunks_and_steps_agree_within_roundings(splitzip_lib):
    """The same tokens in one chunk or one by one: the same cache, and attention
    that differs by its roundings (each result is off by 2^-8 of the weights'
    rounding and 2^-8 of its own, of values below the largest |v|)."""
    g = torch.Generator(device="cuda").manual_seed(3)
    n = 40
    q, k, v = (torch.randn(n, h, 128, generator=g, device="cuda").bfloat16() for h in (32, 8, 8))
    order = list(range(5, 9))
    one, many = (kv_serving.Side(12, order, "cuda") for _ in range(2))
    a = one.step(q, k, v)
    b = torch.cat([many.step(q[i: i + 1], k[i: i + 1], v[i: i + 1]) for i in range(n)])
    for x, y in ((one.cache.k, many.cache.k), (one.cache.v, many.cache.v)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert torch.equal(one.cache.k_scale, many.cache.k_scale)
    assert float((a.float() - b.float()).abs().max()) <= 4 * 2.0 ** -8 * float(v.float().abs().max())


def test_an_early_failure_is_not_lost(splitzip_lib):
    """Each call clears its status word; the example keeps the worst of all calls."""
    g = torch.Generator(device="cuda").manual_seed(4)
    qkv = [torch.randn(20, h, 128, generator=g, device="cuda").bfloat16() for h in (32, 8, 8)]
    side = kv_serving.Side(4, [3, 1], "cuda")
    side.pages[1] = 9  # past the pool
    side.step(*qkv)
    side.pages[1] = 1
    side.step(*(x[:1] for x in qkv))
    assert int(side.status[0]) == sz.OK
    assert int(side.worst) == sz.ERR_INVALID_ARG
