"""GPU: attention of new tokens over a paged cache against the formula in 64
bits, element by element, within the roundings that the operator documents."""
import math

import pytest
import torch

import lossless_kv_cache_gb300 as sz
from tests.kv_reference import Step, attention, check_attention

pytestmark = pytest.mark.gpu

BF16, FP16, E5M2, E4M3 = torch.bfloat16, torch.float16, torch.float8_e5m2, torch.float8_e4m3fn
TYPES = [(BF16, BF16), (FP16, FP16), (E5M2, BF16), (E5M2, FP16), (E4M3, BF16), (E4M3, FP16)]


@pytest.fixture(scope="module", autouse=True)
def _lib(splitzip_lib):
    assert torch.cuda.is_available()
    return splitzip_lib


def run(step, q, scale, causal=True, window=0, out=None, bufs=None, lse=True):
    q = q if q.is_cuda else q.cuda()
    heads = q.shape[1]
    bufs = bufs or sz.KVAttentionBuffers(step.cache, step.batch, heads)
    out = torch.full(q.shape, 77.0, dtype=q.dtype, device="cuda") if out is None else out
    lse = torch.full(q.shape[:2], 77.0, device="cuda") if lse else None
    sz.kv_attention(step.cache, step.batch, q, out, bufs, scale, causal=causal, window=window, lse=lse)
    torch.cuda.synchronize()
    return out, lse, int(bufs.status[0])


def weight_type(step):
    return FP16 if step.dtype == FP16 else BF16


def check(step, group=4, scale=None, causal=True, window=0, q_spread=1.0):
    scale = 1 / math.sqrt(step.dim) if scale is None else scale
    q = (torch.randn(step.tokens, step.kv_heads * group, step.dim, generator=step.gen) * q_spread).to(step.x)
    out, lse, status = run(step, q, scale, causal, window)
    assert status == sz.OK
    check_attention(step, out, lse, attention(step, q, scale, causal, window), weight_type(step))


STEP_LENS = [(1, 1), (1, 63), (1, 64), (1, 65), (0, 40), (1, 300), (1, 16)]
CHUNK_LENS = [(40, 40), (1, 130), (0, 9), (33, 257), (7, 8), (130, 141)]


@pytest.mark.parametrize("dtype,x", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
def test_step_types(dtype, x, dim):
    check(Step(dtype, STEP_LENS, dim=dim, x=x))


@pytest.mark.parametrize("dtype,x", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
def test_chunk_types(dtype, x, dim):
    check(Step(dtype, CHUNK_LENS, dim=dim, x=x))


@pytest.mark.parametrize("kv_heads,group", [(1, 1), (8, 1), (1, 16), (3, 3), (2, 5), (1, 7), (2, 8), (1, 33), (1, 64)])
def test_heads(kv_heads, group):
    check(Step(BF16, [(1, 90), (3, 77), (1, 5)], kv_heads=kv_heads, dim=64), group=group)
    check(Step(E5M2, [(1, 90), (20, 77), (11, 150)], kv_heads=kv_heads, dim=64), group=group)


@pytest.mark.parametrize("page", [1, 2, 4, 8, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_pages(page, dtype):
    check(Step(dtype, [(1, 333), (2, 70), (1, 129)], page=page))
    check(Step(dtype, [(65, 333), (9, 70), (129, 129)], page=page))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 2, 17, 64, 100, 5000])
def test_masks(causal, window):
    for dtype in (BF16, E5M2):
        check(Step(dtype, [(1, 333), (4, 70), (3, 3)], kv_heads=1, dim=64), causal=causal, window=window)
        check(Step(dtype, [(70, 333), (100, 100), (3, 200)], kv_heads=1, dim=64), causal=causal, window=window)


@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_see_nothing(causal):
    """Sequences that hold nothing, and rows of negative position."""
    for lens in ([(1, 0), (3, 2), (2, 2), (4, 0)], [(50, 0), (60, 31), (70, 70)]):
        step = Step(BF16, lens, spare_rows=3)
        q = torch.randn(step.tokens, 8, 128, generator=step.gen).to(BF16)
        out, lse, status = run(step, q, 0.1, causal)
        assert status == sz.OK
        used = step.cu[-1]
        # rows past the last sequence are left alone
        assert bool((out[used:] == 77.0).all()) and bool((lse[used:] == 77.0).all())
        ref = attention(step, q, 0.1, causal)
        check_attention(step, out[:used], lse[:used], tuple(x[:used] for x in ref), BF16)
        first = step.cu[1]
        t, n = lens[1]
        assert bool((out[first: first + t - n] == 0).all())
        assert bool((lse[first: first + t - n] == -math.inf).all())


@pytest.mark.parametrize("dtype", [BF16, FP16, E5M2, E4M3])
@pytest.mark.parametrize("lens", [[(1, 50), (2, 35)], [(40, 50), (20, 150)]])
def test_nothing_unseen_has_a_part(dtype, lens):
    """Token slots past a sequence's end, and pages of nobody, hold NaN."""
    step = Step(dtype, lens)
    q = torch.randn(step.tokens, 8, 128, generator=step.gen).to(step.x)
    used = torch.zeros(step.pages, step.page, dtype=torch.bool)
    for b, (_, n) in enumerate(lens):
        for pos in range(n):
            used[step.place(b, pos)] = True
    nan = {BF16: 0x7FC0, FP16: 0x7E00, E5M2: 0x7F, E4M3: 0x7F}[dtype]
    raw = torch.uint8 if step.fp8 else torch.int16
    for pool in (step.cache.k, step.cache.v):
        pool.view(raw)[~used.cuda()] = nan
    if step.fp8:
        for s in (step.cache.k_scale, step.cache.v_scale):
            s.transpose(1, 2)[~used.cuda()] = 254
    out, lse, status = run(step, q, 0.09)
    assert status == sz.OK
    check_attention(step, out, lse, attention(step, q, 0.09), weight_type(step))


@pytest.mark.parametrize("dtype", [BF16, FP16, E5M2, E4M3])
@pytest.mark.parametrize("window", [0, 6, 30])
@pytest.mark.parametrize("lens", [[(3, 40)], [(70, 200)], [(130, 130)]])
def test_special_values_reach_only_the_rows_that_see_them(dtype, window, lens):
    """A NaN in K, and NaN and infinities in V, at positions that only some rows see."""
    t, n = lens[0]
    step = Step(dtype, lens, kv_heads=1)
    step.set_value("v", 0, n - 2, 0, 3, math.nan)
    step.set_value("v", 0, n - 1, 0, 100, math.nan)
    if dtype != E4M3:
        step.set_value("v", 0, n - 2, 0, 70, math.inf)
        step.set_value("v", 0, n - t, 0, 5, -math.inf)
        step.set_value("v", 0, n - t + 1, 0, 5, math.inf)
    step.set_value("k", 0, n - 1, 0, 9, math.nan)
    q = torch.randn(step.tokens, 4, 128, generator=step.gen).to(step.x)
    out, lse, status = run(step, q, 0.05, True, window)
    assert status == sz.OK
    # 64 bits: weights of what a row does not see are left out, not multiplied by 0
    ref_out, ref_lse, mag, size = attention(step, q, 0.05, True, window)
    last = torch.zeros(step.tokens, dtype=torch.bool)
    last[t - 1] = True  # the row that sees the NaN key: all NaN
    assert bool(torch.isnan(out[last.cuda()]).all()) and bool(torch.isnan(lse[last.cuda()]).all())
    rest = ~last
    sub = Step.__new__(Step)
    sub.__dict__.update(step.__dict__)
    mag = mag.nan_to_num(0, 0, 0)
    check_attention(sub, out.cpu()[rest], lse.cpu()[rest], (ref_out[rest], ref_lse[rest], mag[rest], size[rest]),
                    weight_type(step))


def test_scores_that_dwarf_and_scores_alike():
    """Logits of some hundreds (one key takes all), equal logits, negative and zero scale."""
    for lens in ([(1, 200), (2, 77)], [(50, 200), (65, 77)]):
        for scale in (2.0, -0.3, 0.0):
            check(Step(BF16, lens, spread=0.3), scale=scale)
        check(Step(FP16, lens, spread=0.3), q_spread=4.0, scale=1.0)
        step = Step(E5M2, lens, fill="zeros")
        q = torch.randn(step.tokens, 8, 128, generator=step.gen).to(BF16)
        out, lse, status = run(step, q, 1.0)
        assert status == sz.OK and bool((out == 0).all())
        check_attention(step, out, lse, attention(step, q, 1.0), BF16)


@pytest.mark.parametrize("layout", ["hnd", "kv"])
@pytest.mark.parametrize("dtype", [BF16, E5M2])
def test_layouts(layout, dtype):
    check(Step(dtype, [(1, 90), (2, 33)], layout=layout))
    check(Step(dtype, [(77, 190), (31, 33)], layout=layout))


@pytest.mark.parametrize("lens", [[(1, 190), (2, 33)], [(77, 190), (31, 33)]])
def test_strided_queries_and_output_in_place(lens):
    step = Step(BF16, lens)
    qkv = torch.randn(step.tokens, 8 + 2 + 2, 128, generator=step.gen).to(BF16)
    q = qkv[:, :8]
    ref = attention(step, q, 0.1)
    dev = qkv.cuda()
    other = dev[:, 8:].clone()
    out, lse, status = run(step, dev[:, :8], 0.1, out=dev[:, :8])
    assert status == sz.OK
    check_attention(step, out, lse, ref, BF16)
    assert torch.equal(dev[:, 8:], other)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_long_axis_is_split_and_joined(dtype):
    check(Step(dtype, [(1, 20011)], kv_heads=1, dim=64), group=2)
    check(Step(dtype, [(1, 9000), (1, 3), (1, 1500), (1, 64)], kv_heads=2, dim=64), group=3)
    check(Step(dtype, [(65, 9001)], kv_heads=1, dim=64), group=1)


def test_many_sequences():
    lens = [(1 if b % 5 else b % 3, (b * 37) % 150 + 2) for b in range(400)]
    check(Step(BF16, lens, kv_heads=1, dim=64), group=2)


def test_results_repeat_and_workspace_needs_no_clearing():
    step = Step(E5M2, [(1, 3000), (2, 900), (30, 700)])
    q = torch.randn(step.tokens, 8, 128, generator=step.gen).to(BF16).cuda()
    bufs = sz.KVAttentionBuffers(step.cache, step.batch, 8)
    want = None
    for fill in (0, 255, 0x7F, 1):
        bufs.ws.fill_(fill)
        out, lse, status = run(step, q, 0.1, bufs=bufs)
        assert status == sz.OK
        if want is not None:
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        want = (out, lse)
        again, lse, _ = run(step, q, 0.1, bufs=bufs)
        assert torch.equal(again, out)


def test_without_lse_own_stream_and_graph():
    for lens in ([(1, 900), (2, 90)], [(77, 900), (20, 90)]):
        step = Step(BF16, lens)
        q = torch.randn(step.tokens, 8, 128, generator=step.gen).to(BF16).cuda()
        out, _, _ = run(step, q, 0.1)
        bufs = sz.KVAttentionBuffers(step.cache, step.batch, 8)
        got = torch.empty_like(q)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        sz.kv_attention(step.cache, step.batch, q, got, bufs, 0.1, stream=side)
        side.synchronize()
        assert torch.equal(out, got)
        graph = torch.cuda.CUDAGraph()
        got.zero_()
        with torch.cuda.graph(graph):
            sz.kv_attention(step.cache, step.batch, q, got, bufs, 0.1)
        for _ in range(3):
            got.zero_()
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, got)
        # the same captured call, a shorter step
        step.batch.kv_len.sub_(3)
        step.lens = [(t, n - 3) for t, n in step.lens]
        graph.replay()
        torch.cuda.synchronize()
        check_attention(step, got, None, attention(step, q.cpu(), 0.1), BF16)


@pytest.mark.parametrize("new", [1, 40])
def test_bad_entries_are_reported_and_others_stand(new):
    for what in ("page", "page-negative", "len", "cu", "new"):
        step = Step(BF16, [(new, 90), (new, 70), (new, 50)])
        q = torch.randn(step.tokens, 8, 128, generator=step.gen).to(BF16)
        ref = attention(step, q, 0.1)
        if what == "page":
            step.batch.page_table[1, 2] = step.pages
        elif what == "page-negative":
            step.batch.page_table[1, 0] = -1
        elif what == "len":
            step.batch.kv_len[1] = -1
        elif what == "cu":
            step.batch.cu_tokens[0] = -1  # sequence 0 is out
        else:
            step.batch.kv_len[1] = 91  # past max_kv_len
        out, lse, status = run(step, q, 0.1)
        assert status == sz.ERR_INVALID_ARG, what
        rows = slice(2 * new, 3 * new)
        sub = Step.__new__(Step)
        sub.__dict__.update(step.__dict__)
        check_attention(sub, out[rows], lse[rows], tuple(x[rows] for x in ref), BF16)
        # the next call's status is its own
        step.batch.page_table.copy_(step.table)
        step.batch.kv_len.copy_(torch.tensor([n for _, n in step.lens], dtype=torch.int32))
        step.batch.cu_tokens.copy_(torch.tensor(step.cu, dtype=torch.int32))
        out, lse, status = run(step, q, 0.1)
        assert status == sz.OK
        check_attention(step, out, lse, ref, BF16)


def test_offsets_past_32_bits():
    """Pages at the far end of pools of more than 2^32 bytes."""
    small = Step(E5M2, [(2, 200), (40, 60)], kv_heads=8)
    n = small.pages
    pages = (5 << 30) // (small.page * 8 * 128)
    pools, scales = [], []
    for name in "kv":
        pool = torch.empty(pages, small.page, 8, 128, dtype=torch.uint8, device="cuda")
        pool[pages - n:] = getattr(small.cache, name).view(torch.uint8)
        scale = torch.empty(pages, 8, small.page, dtype=torch.uint8, device="cuda")
        scale[pages - n:] = getattr(small.cache, name + "_scale")
        pools.append(pool.view(E5M2))
        scales.append(scale)
    q = torch.randn(small.tokens, 32, 128, generator=small.gen).to(BF16)
    small.cache = sz.KVCache(*pools, *scales)
    small.batch.page_table.add_(pages - n)
    out, lse, status = run(small, q, 0.1)
    assert status == sz.OK
    check_attention(small, out, lse, attention(small, q, 0.1), BF16)


@pytest.mark.parametrize("dtype", [E5M2, E4M3])
@pytest.mark.parametrize("lens", [[(1, 300), (2, 35)], [(40, 300), (20, 150)]])
def test_largest_fp16_values_in_fp8_pages(dtype, lens):
    """65,504 is 65,536 after its rounding to FP8, which FP16 does not hold;
    the sums over V, of both signs, do fit the result."""
    step = Step(dtype, lens, x=FP16)
    top, k = (32768.0, 1) if dtype == E5M2 else (256.0, 8)
    sign = torch.randint(0, 2, step.host["v"].shape, generator=step.gen).double() * 2 - 1
    step.cache.v.copy_((sign * top).float().to(dtype))
    step.cache.v_scale.fill_(127 + k)
    step.host["v"] = torch.ldexp(sign * top, torch.tensor(k))
    q = (torch.randn(step.tokens, 8, 128, generator=step.gen) * 0.1).to(FP16)
    out, lse, status = run(step, q, 0.05, causal=False)
    assert status == sz.OK
    ref = attention(step, q, 0.05, causal=False)
    assert bool((ref[0].abs() < 65504).all())
    check_attention(step, out, lse, ref, FP16)
