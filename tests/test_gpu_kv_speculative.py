"""GPU: the operators of a speculative step together, as the example runs them:
what trees of drafted tokens leave in the caches, and what they attended, is
what the accepted tokens alone give."""
import math

import pytest
import torch

import lossless_kv_cache_gb300 as sz
from examples import kv_speculative as example

pytestmark = pytest.mark.gpu

BF16, FP16, E5M2, E4M3 = torch.bfloat16, torch.float16, torch.float8_e5m2, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib(splitzip_lib):
    assert torch.cuda.is_available()
    return splitzip_lib


def bits(t):
    return t.contiguous().view(torch.int16)


def check(engine, history):
    assert int(engine.worst) == sz.OK
    lens = [h[0].shape[1] if h else 0 for h in history]
    assert engine.pages.kv_len.tolist() == lens
    assert engine.pages.held.tolist() == [-(-n // example.PAGE_TOKENS) for n in lens]
    assert int(engine.pages.count) == engine.pages.free.numel() - sum(engine.pages.held.tolist())
    rows, x = sum(lens), engine.q.dtype
    cu = torch.tensor([sum(lens[:b]) for b in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    # the accepted tokens of all sequences in one step into caches of their own
    pages = sz.KVPages.empty(engine.pages.free.numel(), example.PAGE_TOKENS, len(lens), max(lens))
    step = sz.KVStep(len(lens), rows, max(lens), max(lens))
    sz.kv_extend(pages, torch.tensor(lens, dtype=torch.int32, device="cuda"), step)
    assert torch.equal(step.cu_tokens, cu)
    batch = step.batch_of(pages)
    old = sz.KVBatch(cu, engine.pages.kv_len, engine.pages.table, rows, max(lens), max(lens))
    bufs = sz.KVAttentionBuffers(engine.caches[0], batch, example.HEADS)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    for i, cache in enumerate(engine.caches):
        q, k, v, out = (torch.cat([h[n][i] for h in history if h]).cuda() for n in range(4))
        alone = sz.KVCache.empty(pages.free.numel(), example.PAGE_TOKENS, example.KV_HEADS, example.HEAD_DIM,
                                 cache.k.dtype)
        sz.kv_rotary_write(alone, batch, engine.rotary, q, q, k, v, status)
        assert int(status[0]) == sz.OK
        got = []
        for c, b in ((cache, old), (alone, batch)):
            pair = torch.empty(2, rows, example.KV_HEADS, example.HEAD_DIM, dtype=x, device="cuda")
            sz.kv_read(c, b, pair[0], pair[1], status)
            assert int(status[0]) == sz.OK
            got.append(pair)
        assert torch.equal(bits(got[0]), bits(got[1]))
        causal = torch.empty_like(q)
        sz.kv_attention(alone, batch, q, causal, bufs, 1.0 / math.sqrt(example.HEAD_DIM))
        assert int(bufs.status[0]) == sz.OK
        # each of the two rounds its weights (half a step of at most BF16, of sums of at most the largest
        # value) and its result; the scores' own errors, in 32 bits, are far below
        most = got[0][1].float().abs().max()
        tol = 2 * torch.finfo(BF16).eps / 2 * (most + causal.float().abs()) * (1 + 2.0 ** -6)
        assert bool(((out.float() - causal.float()).abs() <= tol).all())


@pytest.mark.parametrize("dtype,x", [(BF16, BF16), (FP16, FP16), (E5M2, BF16), (E4M3, FP16)])
@pytest.mark.parametrize("drafted", [3, 12, 40])
def test_accepted_tokens_are_what_is_left(dtype, x, drafted):
    check(*example.run(steps=7, batch=5, drafted=drafted, dtype=dtype, x=x, seed=drafted))


@pytest.mark.parametrize("drafted", [4, 20])
def test_a_captured_step(drafted):
    """One graph of a whole step, replayed over other lengths, trees and branches."""
    def capture(engine):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            engine.forward()
            engine.accept()
        engine.drop.zero_()
        return graph.replay

    check(*example.run(steps=9, batch=4, drafted=drafted, dtype=E5M2, step=capture))
