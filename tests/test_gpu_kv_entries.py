"""GPU: steps whose integer arrays are wrong.  Every call reports them, also
where no packed row belongs to the sequence, and nothing is written but to new
positions of sequences whose own entries are in range."""
import math

import pytest
import torch

import lossless_kv_cache_gb300 as sz
from tests.kv_reference import RAW, Step

pytestmark = pytest.mark.gpu

BF16, E5M2 = torch.bfloat16, torch.float8_e5m2


@pytest.fixture(scope="module", autouse=True)
def _lib(splitzip_lib):
    assert torch.cuda.is_available()
    return splitzip_lib


def write(step):
    x = step.new_rows().cuda()
    sz.kv_write(step.cache, step.batch, x, x, step.status)
    return int(step.status[0])


def read(step):
    x = step.new_rows().cuda()
    sz.kv_read(step.cache, step.batch, x, x.clone(), step.status)
    return int(step.status[0])


def attend(step):
    q = torch.randn(step.tokens, 8, step.dim, generator=step.gen).to(step.x).cuda()
    bufs = sz.KVAttentionBuffers(step.cache, step.batch, 8)
    sz.kv_attention(step.cache, step.batch, q, torch.empty_like(q), bufs, 0.1)
    return int(bufs.status[0])


CALLS = pytest.mark.parametrize("call", [write, read, attend])


@CALLS
@pytest.mark.parametrize("lens", [[(3, 40), (0, 20), (2, 9)], [(40, 40), (0, 20), (2, 9)], [(0, 40), (0, 20)]])
@pytest.mark.parametrize("bad", [-1, 41, 1 << 29, -(1 << 31)])
def test_a_bad_length_without_new_tokens_is_reported(call, lens, bad):
    for dtype in (BF16, E5M2):
        step = Step(dtype, lens)
        assert call(step) == sz.OK
        step.batch.kv_len[1] = bad
        assert call(step) == sz.ERR_INVALID_ARG
        step.batch.kv_len[1] = 20
        assert call(step) == sz.OK


@CALLS
def test_a_bad_length_far_into_a_large_batch_is_reported(call):
    lens = [(1 if b % 7 == 0 else 0, 5 + b % 11) for b in range(3000)]
    step = Step(BF16, lens, kv_heads=1, dim=64)
    assert call(step) == sz.OK
    for b in (1, 1025, 2999):
        step.batch.kv_len[b] = 16
        assert call(step) == sz.ERR_INVALID_ARG
        step.batch.kv_len[b] = lens[b][1]
    assert call(step) == sz.OK


@CALLS
@pytest.mark.parametrize("cu", [[0, 5, 8, 3, 9], [0, 5, 3, 8, 9], [0, 9, 9, 9, 8], [0, 3, 6, 10, 9], [4, 2, 9, 9, 9]])
def test_offsets_that_descend_are_reported(call, cu):
    step = Step(BF16, [(3, 40), (2, 30), (2, 20), (2, 10)])
    step.batch.desc.max_tokens = 9
    assert call(step) == sz.OK
    step.batch.cu_tokens.copy_(torch.tensor(cu, dtype=torch.int32))
    assert call(step) == sz.ERR_INVALID_ARG


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("cu", [[0, 5, 8, 3, 9], [0, 5, 3, 8, 9], [0, 9, 9, 9, 8], [4, 2, 9, 9, 9], [0, 6, 7, 2, 9]])
def test_offsets_that_descend_write_to_new_positions_only(dtype, cu):
    """Rows between descending offsets are in no sequence or in several: they go to a
    place that one of these has for them, or nowhere."""
    lens = [(3, 40), (2, 30), (2, 20), (2, 10)]
    step = Step(dtype, lens)
    step.batch.desc.max_tokens = 9
    step.batch.cu_tokens.copy_(torch.tensor(cu, dtype=torch.int32))
    before = {n: getattr(step.cache, n).view(RAW[dtype]).cpu().clone() for n in "kv"}
    scales = {n: getattr(step.cache, n + "_scale").cpu().clone() for n in "kv"} if step.fp8 else {}
    allowed = torch.zeros(step.pages, step.page, dtype=torch.bool)
    for b, (_, n) in enumerate(lens):
        for pos in range(max(0, n - max(0, cu[b + 1] - cu[b])), n):
            allowed[step.place(b, pos)] = True
    assert write(step) == sz.ERR_INVALID_ARG
    for n in "kv":
        changed = (getattr(step.cache, n).view(RAW[dtype]).cpu() != before[n]).flatten(2).any(-1)
        assert not bool((changed & ~allowed).any())
        if step.fp8:
            changed = (getattr(step.cache, n + "_scale").cpu() != scales[n]).any(1)
            assert not bool((changed & ~allowed).any())


def test_tensors_off_the_device_are_refused():
    step = Step(BF16, [(3, 40), (1, 20)])
    x = step.new_rows()
    for status in (torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.int64, device="cuda"),
                   torch.zeros(0, dtype=torch.int32, device="cuda")):
        for call in (sz.kv_write, sz.kv_read):
            with pytest.raises(ValueError):
                call(step.cache, step.batch, x.cuda(), x.cuda(), status)
    for call in (sz.kv_write, sz.kv_read):
        with pytest.raises(ValueError):
            call(step.cache, step.batch, x, x.cuda(), step.status)
        with pytest.raises(ValueError):
            call(step.cache, step.batch, x.cuda(), x, step.status)
    q = torch.randn(step.tokens, 8, step.dim).to(BF16)
    bufs = sz.KVAttentionBuffers(step.cache, step.batch, 8)
    for args, lse in (((q, q.cuda()), None), ((q.cuda(), q), None), ((q.cuda(), q.cuda()), torch.zeros(step.tokens, 8))):
        with pytest.raises(ValueError):
            sz.kv_attention(step.cache, step.batch, *args, bufs, 0.1, lse=lse)
    assert write(step) == sz.OK and attend(step) == sz.OK


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("dtype", [BF16, E5M2])
def test_a_step_that_holds_nothing_needs_no_page_table(dtype, new):
    step = Step(dtype, [(new, 0), (0, 0), (new, 0)])
    step.batch = sz.KVBatch(step.batch.cu_tokens, step.batch.kv_len, torch.empty(3, 0, dtype=torch.int32, device="cuda"),
                            step.tokens, new, 0)
    assert write(step) == sz.OK
    k, v = (torch.full((step.tokens, 2, 128), 7.0, dtype=BF16, device="cuda") for _ in range(2))
    sz.kv_read(step.cache, step.batch, k, v, step.status)
    assert int(step.status[0]) == sz.OK and not bool(k.any()) and not bool(v.any())
    q = torch.randn(step.tokens, 8, 128, generator=step.gen).to(BF16).cuda()
    out, lse = torch.full_like(q, 7.0), torch.zeros(step.tokens, 8, device="cuda")
    bufs = sz.KVAttentionBuffers(step.cache, step.batch, 8)
    sz.kv_attention(step.cache, step.batch, q, out, bufs, 0.1, lse=lse)
    assert int(bufs.status[0]) == sz.OK and not bool(out.any()) and bool((lse == -math.inf).all())
    step.batch.kv_len[1] = 1  # past max_kv_len
    assert write(step) == read(step) == attend(step) == sz.ERR_INVALID_ARG
