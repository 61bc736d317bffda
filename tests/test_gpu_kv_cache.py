"""GPU: writing rows into a paged cache and reading them back.  The stored FP8
values and scales must be the reference's exactly (one rounding, to nearest
even, of an exact quotient), 16-bit caches hold the bits, and everything else
in the pools stays as it was."""
import math

import pytest
import torch

import lossless_kv_cache_gb300 as sz
from tests.kv_reference import FP8, RAW, Step, quantise

pytestmark = pytest.mark.gpu

BF16, FP16, E5M2, E4M3 = torch.bfloat16, torch.float16, torch.float8_e5m2, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib(splitzip_lib):
    assert torch.cuda.is_available()
    return splitzip_lib


def written(step, rows, name):
    """What the pool (values) and scale should be after writing `rows`."""
    pool = getattr(step.cache, name).view(RAW[step.dtype]).cpu().clone().view(step.dtype).double()
    scale = None
    if step.fp8:
        scale = getattr(step.cache, name + "_scale").cpu().clone()
        q, k = quantise(rows.double(), step.dtype)
    else:
        q = rows.double()
    for b, (t, n) in enumerate(step.lens):
        for i in range(t):
            pos = n - t + i
            if pos < 0:
                continue
            pg, off = step.place(b, pos)
            pool[pg, off] = q[step.cu[b] + i]
            if step.fp8:
                scale[pg, :, off] = (k[step.cu[b] + i] + 127).to(torch.uint8)
    return pool, scale


def same(got, want):
    return torch.equal(got.nan_to_num(12345.0, 1e300, -1e300), want.nan_to_num(12345.0, 1e300, -1e300))


def check_written(step, k, v):
    want = {"k": written(step, k, "k"), "v": written(step, v, "v")}
    sz.kv_write(step.cache, step.batch, k.cuda(), v.cuda(), step.status)
    torch.cuda.synchronize()
    assert int(step.status[0]) == sz.OK
    for name in "kv":
        got = getattr(step.cache, name).view(RAW[step.dtype]).cpu().view(step.dtype).double()
        assert same(got, want[name][0]), name
        if step.fp8:
            assert torch.equal(getattr(step.cache, name + "_scale").cpu(), want[name][1]), name


LENS = [(3, 40), (0, 9), (1, 1), (17, 17), (5, 64), (33, 100)]


@pytest.mark.parametrize("dtype,x", [(E5M2, BF16), (E5M2, FP16), (E4M3, BF16), (E4M3, FP16), (BF16, BF16), (FP16, FP16)])
@pytest.mark.parametrize("page,heads,dim", [(16, 2, 128), (1, 3, 64), (64, 8, 128), (8, 1, 64), (4, 5, 128)])
def test_write(dtype, x, page, heads, dim):
    step = Step(dtype, LENS, page=page, kv_heads=heads, dim=dim, x=x, spare_rows=2)
    check_written(step, step.new_rows(1.0), step.new_rows(30.0))


@pytest.mark.parametrize("layout", ["hnd", "kv"])
@pytest.mark.parametrize("dtype", [E5M2, E4M3, BF16])
def test_write_layouts(dtype, layout):
    step = Step(dtype, LENS, layout=layout)
    check_written(step, step.new_rows(), step.new_rows())


@pytest.mark.parametrize("dtype", [E5M2, E4M3])
@pytest.mark.parametrize("x", [BF16, FP16])
def test_write_special_rows(dtype, x):
    """Zeros, the type's extremes, powers of two on both sides of a scale's border, halfway cases, NaN, infinities."""
    big, tiny = torch.finfo(x).max, torch.finfo(x).smallest_normal * torch.finfo(x).eps
    rows = [[0.0], [-0.0, 0.0], [big], [-big, tiny], [tiny], [1.75], [1.75, 1.0], [1.7578125], [-1.875, 0.3],
            [math.inf], [math.nan, 2.0], [-math.inf, 3.0, 0.01], [math.nan], [math.inf, -math.inf, math.nan, 1e-3],
            [448.0], [449.0], [464.0], [57344.0 if x == BF16 else 57300.0], [1.0, 1.125, 1.0625, 1.03125, 1.1875, 0.09375]]
    k = torch.zeros(len(rows), 2, 64, dtype=torch.float64)
    for i, r in enumerate(rows):
        k[i, 0, 5: 5 + len(r)] = torch.tensor(r, dtype=torch.float64)
        k[i, 1, : len(r)] = -torch.tensor(r, dtype=torch.float64)
        k[i, 1, 60:] = 2.0 ** -7
    k = k.to(x)
    step = Step(dtype, [(len(rows), 30)], dim=64, x=x)
    check_written(step, k, k.flip(0))


def test_write_every_bf16_value():
    """Every BF16 bit pattern as an element, next to an element that sets the scale."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF16)
    for dtype in (E5M2, E4M3):
        step = Step(dtype, [(1024, 1024)], kv_heads=1, dim=64, fill="zeros")
        check_written(step, bits.view(1024, 1, 64), bits.flip(0).view(1024, 1, 64))


def test_write_strided_rows_and_rows_without_a_place():
    lens = [(6, 4), (2, 20), (4, 0), (3, 3)]  # the first two rows of sequence 0 and all of sequence 2 have no place
    step = Step(E5M2, lens, kv_heads=2, dim=128)
    qkv = torch.randn(step.tokens, 4 + 2 + 2, 128, generator=step.gen).to(BF16)
    k, v = qkv[:, 4:6], qkv[:, 6:8]
    want = {"k": written(step, k, "k"), "v": written(step, v, "v")}
    dev = qkv.cuda()
    sz.kv_write(step.cache, step.batch, dev[:, 4:6], dev[:, 6:8], step.status)
    torch.cuda.synchronize()
    assert int(step.status[0]) == sz.OK
    for name in "kv":
        got = getattr(step.cache, name).view(torch.uint8).cpu().view(E5M2).double()
        assert same(got, want[name][0])
        assert torch.equal(getattr(step.cache, name + "_scale").cpu(), want[name][1])


@pytest.mark.parametrize("dtype,x", [(E5M2, BF16), (E5M2, FP16), (E4M3, BF16), (E4M3, FP16), (BF16, BF16), (FP16, FP16)])
@pytest.mark.parametrize("page,heads,dim", [(16, 2, 128), (1, 3, 64), (128, 4, 64)])
def test_read(dtype, x, page, heads, dim):
    lens = LENS + [(4, 2)]
    step = Step(dtype, lens, page=page, kv_heads=heads, dim=dim, x=x, spare_rows=1)
    fill = torch.full((step.tokens, heads, dim), 99.0, dtype=x)
    k, v = fill.cuda(), fill.cuda()
    sz.kv_read(step.cache, step.batch, k, v, step.status)
    torch.cuda.synchronize()
    assert int(step.status[0]) == sz.OK
    for name, got in (("k", k), ("v", v)):
        want = fill.clone()
        for b, (t, n) in enumerate(lens):
            values = step.held(b, name)
            for i in range(t):
                pos = n - t + i
                want[step.cu[b] + i] = values[pos].to(x) if pos >= 0 else 0
        assert torch.equal(got.cpu(), want)


def test_read_special_values():
    for dtype in (E5M2, E4M3):
        step = Step(dtype, [(5, 5)], kv_heads=1, dim=64)
        step.set_value("v", 0, 2, 0, 7, math.nan)
        if dtype == E5M2:
            step.set_value("v", 0, 3, 0, 9, -math.inf)
        k = torch.empty(5, 1, 64, dtype=BF16, device="cuda")
        v = torch.empty_like(k)
        sz.kv_read(step.cache, step.batch, k, v, step.status)
        assert same(v.cpu().double(), step.held(0, "v"))


def test_write_then_read_returns_what_the_type_holds():
    step = Step(E5M2, [(50, 50), (3, 77)], page=32)
    k, v = step.new_rows(), step.new_rows(100.0)
    sz.kv_write(step.cache, step.batch, k.cuda(), v.cuda(), step.status)
    ko, vo = torch.empty_like(k).cuda(), torch.empty_like(v).cuda()
    sz.kv_read(step.cache, step.batch, ko, vo, step.status)
    for x, y in ((k, ko.cpu()), (v, vo.cpu())):
        # half a step of 2 mantissa bits, or of the row's smallest step (2^-16 * 2^k, 2^k <= 2 max / 57344)
        x, y = x.double(), y.double()
        tol = torch.maximum(x.abs() * 2.0 ** -3, x.abs().amax(-1, keepdim=True) * 2 / 57344 * 2.0 ** -17)
        assert bool(((x - y).abs() <= tol).all())


def test_bad_entries_are_reported_and_touch_nothing():
    for what in ("page", "page-negative", "len", "cu", "new"):
        step = Step(E5M2, [(3, 40), (2, 20)], extra_pages=1)
        before = {n: getattr(step.cache, n).view(torch.uint8).cpu().clone() for n in "kv"}
        if what == "page":
            step.batch.page_table[0, 2] = step.pages
        elif what == "page-negative":
            step.batch.page_table[0, 2] = -1
        elif what == "len":
            step.batch.kv_len[0] = 41  # past max_kv_len
        elif what == "cu":
            step.batch.cu_tokens[0] = -2
        else:
            step.batch.cu_tokens[1] = 5  # sequence 0: 5 new, past max_tokens; sequence 1: none
        k = step.new_rows().cuda()
        sz.kv_write(step.cache, step.batch, k, k, step.status)
        torch.cuda.synchronize()
        assert int(step.status[0]) == sz.ERR_INVALID_ARG, what
        for n in "kv":
            now = getattr(step.cache, n).view(torch.uint8).cpu()
            changed = (now != before[n]).flatten(2).any(-1)
            allowed = torch.zeros_like(changed)
            for b in (0, 1):
                for i in range(step.lens[b][0]):
                    allowed[step.place(b, step.lens[b][1] - step.lens[b][0] + i)] = True
            assert not bool((changed & ~allowed).any()), what
        sz.kv_read(step.cache, step.batch, torch.empty_like(k), torch.empty_like(k), step.status)
        assert int(step.status[0]) == sz.ERR_INVALID_ARG, what


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes, pages on both sides of that."""
    heads, dim, page = 8, 128, 16
    pages = (5 << 30) // (page * heads * dim)
    pool = torch.empty(pages, page, heads, dim, dtype=torch.uint8, device="cuda")
    scale = torch.full((2, pages, heads, page), 127, dtype=torch.uint8, device="cuda")
    cache = sz.KVCache(pool.view(E5M2), pool.view(E5M2), scale[0], scale[1])  # K and V alias: only K is looked at
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32, device="cuda")
    batch = sz.KVBatch(torch.tensor([0, 40], dtype=torch.int32, device="cuda"),
                       torch.tensor([40], dtype=torch.int32, device="cuda"), table, 40, 40, 40)
    x = torch.randn(40, heads, dim).to(BF16).cuda()
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    sz.kv_write(cache, batch, x, x, status)
    out = torch.empty_like(x)
    sz.kv_read(cache, batch, out, torch.empty_like(x), status)
    assert int(status[0]) == sz.OK
    q, k = quantise(x.cpu().double(), E5M2)
    assert torch.equal(out.cpu().double(), torch.ldexp(q, k[..., None]))
    assert torch.equal(pool[pages - 1, 5].cpu().view(E5M2).double(), q[5])


def test_own_stream_and_graph():
    step = Step(E4M3, [(7, 30), (2, 9)])
    k, v = step.new_rows().cuda(), step.new_rows().cuda()
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sz.kv_write(step.cache, step.batch, k, v, step.status)
        sz.kv_read(step.cache, step.batch, ko, vo, step.status)
    side.synchronize()
    want = ko.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sz.kv_write(step.cache, step.batch, k, v, step.status)
        sz.kv_read(step.cache, step.batch, ko, vo, step.status)
    k.mul_(2.0)  # the scale takes a power of two
    graph.replay()
    torch.cuda.synchronize()
    assert int(step.status[0]) == sz.OK
    assert torch.equal(ko, want * 2.0)


def test_nothing_new():
    step = Step(E5M2, [(0, 5), (0, 0)])
    empty = torch.empty(0, 2, 128, dtype=BF16, device="cuda")
    sz.kv_write(step.cache, step.batch, empty, empty, step.status)
    assert int(step.status[0]) == sz.OK
