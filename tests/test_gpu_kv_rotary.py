"""GPU: rotary positions with the write into the cache, against the formula in
64 bits, element by element.

Errors counted.  The angle: 24 bits of the fraction of a turn exactly and 24
more to first order (under 2^-40 rad off), a rounding of 2^-25 with them; the
sine and cosine are off by two units of their last place at most (2^-22): at
most 2^-21 together.  Their product with the magnitude, two products and a sum add four
roundings of 2^-24.  So an element of a pair (a, b) is off by at most
2^-20 * magnitude * (|a| + |b|) before it is rounded to its type."""
import math

import pytest
import torch

import lossless_kv_cache_gb300 as sz
from tests.kv_reference import FP8, RAW, Step, half_step, quantise

pytestmark = pytest.mark.gpu

BF16, FP16, E5M2, E4M3 = torch.bfloat16, torch.float16, torch.float8_e5m2, torch.float8_e4m3fn
TYPES = [(BF16, BF16), (FP16, FP16), (E5M2, BF16), (E5M2, FP16), (E4M3, BF16), (E4M3, FP16)]
LENS = [(40, 40), (1, 130), (0, 9), (33, 257), (7, 8), (5, 5)]


@pytest.fixture(scope="module", autouse=True)
def _lib(splitzip_lib):
    assert torch.cuda.is_available()
    return splitzip_lib


def rotated(x, position, frequencies, interleaved, magnitude):
    """(x turned, size of the 32-bit error) in doubles; x (tokens, heads, dim) on the CPU."""
    x = x.double()
    half = frequencies.numel()
    angle = (position.double()[:, None] * frequencies).remainder(2 * math.pi)[:, None]
    # far positions: the product in doubles, the turn in doubles and the frequency in turns are off by a rounding each
    slack = (position.double().abs()[:, None] * frequencies)[:, None] * 2.0 ** -51
    cos, sin = torch.cos(angle) * magnitude, torch.sin(angle) * magnitude
    turned = x[..., : 2 * half]
    a, b = (turned[..., 0::2], turned[..., 1::2]) if interleaved else (turned[..., :half], turned[..., half:])
    p, q = a * cos - b * sin, a * sin + b * cos
    off = (a.abs() + b.abs()) * abs(magnitude) * (2.0 ** -20 + slack)
    y = torch.stack([p, q], -1).flatten(-2) if interleaved else torch.cat([p, q], -1)
    e = torch.stack([off, off], -1).flatten(-2) if interleaved else torch.cat([off, off], -1)
    rest = x[..., 2 * half:]
    return torch.cat([y, rest], -1), torch.cat([e, torch.zeros_like(rest)], -1)


def near(got, want, off, dtype):
    """`got` is `want`, off by `off` and a rounding to `dtype`."""
    got = got.double().cpu()
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2
    tol = off + half_step(dtype) * (want.abs() + off) + tiny
    fine = want.abs() + tol < torch.finfo(dtype).max  # others may round to infinity
    assert bool(((got - want).abs() <= tol)[fine].all()), float(((got - want).abs() / tol)[fine].max())


def places(step):
    return torch.cat([torch.arange(n - t, n) for t, n in step.lens] + [torch.zeros(0, dtype=torch.int64)])


def run(step, heads, frequencies, interleaved=False, magnitude=1.0, given=None, q=None, k=None, v=None, q_out=None):
    rows = step.tokens
    q = torch.randn(rows, heads, step.dim, generator=step.gen).to(step.x) if q is None else q
    k = step.new_rows() if k is None else k
    v = step.new_rows() if v is None else v
    rotary = sz.KVRotary(frequencies, interleaved=interleaved, magnitude=magnitude)
    dev = [t if t.is_cuda else t.cuda() for t in (q, k, v)]
    q_out = torch.full_like(dev[0], 77.0) if q_out is None else q_out
    sz.kv_rotary_write(step.cache, step.batch, rotary, dev[0], q_out, dev[1], dev[2], step.status,
                       positions=None if given is None else given.int().cuda())
    torch.cuda.synchronize()
    return q, k, v, q_out


def check_cache(step, name, want, off, position_of):
    """The new rows in the pages: off by `off` and one rounding; everything else as it was."""
    pool = step.cache.k if name == "k" else step.cache.v
    got = pool.view(RAW[step.dtype]).cpu().view(step.dtype)
    scale = (step.cache.k_scale if name == "k" else step.cache.v_scale)
    scale = scale.cpu() if step.fp8 else None
    row = 0
    host = step.host[name].clone()
    written = torch.zeros(host.shape[:2], dtype=torch.bool)
    for b, (t, n) in enumerate(step.lens):
        for i in range(t):
            pos = n - t + i
            r = step.cu[b] + i
            row += 1
            if pos < 0:
                continue
            page, slot = step.place(b, pos)
            written[page, slot] = True
            x = got[page, slot].float().double()
            w, e = want[r], off[r]
            if not step.fp8:
                near(x, w, e, step.dtype)
                continue
            largest, bits, lowest = FP8[step.dtype]
            for h in range(step.kv_heads):
                exp = int(scale[page, h, slot]) - 127
                _, k = quantise(w[h], step.dtype)
                if exp != int(k):  # the row's largest may be either side of the limit
                    _, lo = quantise(w[h] * (1 - 2.0 ** -18), step.dtype)
                    _, hi = quantise(w[h] * (1 + 2.0 ** -18), step.dtype)
                    assert exp in (int(lo), int(hi))
                unit = math.ldexp(1.0, exp)
                at = torch.where(x[h] == 0, torch.tensor(lowest), torch.clamp(torch.frexp(x[h])[1] - 1, min=lowest))
                half = torch.ldexp(torch.ones_like(x[h]), at - bits - 1) * unit
                assert bool(((x[h] * unit - w[h]).abs() <= half * (1 + 2.0 ** -18) + e[h]).all())
    # what no row belongs to is untouched
    untouched = ~written
    if step.fp8:
        unit = torch.ldexp(torch.ones(scale.shape, dtype=torch.float64), scale.int() - 127).transpose(1, 2)[..., None]
        values = got.float().double() * unit
    else:
        values = got.double()
    assert torch.equal(values[untouched], host[untouched])


def check(dtype, x, lens=LENS, dim=128, rot=None, interleaved=False, group=4, kv_heads=2, page=16, layout="nhd",
          magnitude=1.0, given=None, base=10000.0, spare=0, seed=0):
    step = Step(dtype, lens, page=page, kv_heads=kv_heads, dim=dim, x=x, layout=layout, spare_rows=spare, seed=seed)
    f = sz.rotary_frequencies(rot or dim, base)
    position = places(step) if given is None else given(step)
    position = torch.cat([position, torch.full((spare,), 5)])
    q, k, v, q_out = run(step, kv_heads * group, f, interleaved, magnitude, None if given is None else position)
    assert int(step.status[0]) == sz.OK
    rows = step.tokens - spare
    want, off = rotated(q, position, f, interleaved, magnitude)
    near(q_out[:rows], want[:rows], off[:rows], step.x)
    assert bool((q_out[rows:] == 77).all())
    want, off = rotated(k, position, f, interleaved, magnitude)
    check_cache(step, "k", want, off, position)
    check_cache(step, "v", v.double(), torch.zeros_like(off), position)


@pytest.mark.parametrize("dtype,x", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim", [64, 128])
def test_types_and_layouts(dtype, x, interleaved, dim):
    check(dtype, x, dim=dim, interleaved=interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(64, 16), (64, 32), (64, 48), (128, 16), (128, 32), (128, 64), (128, 96), (128, 112)])
def test_part_of_the_head(interleaved, dim, rot):
    check(E4M3, BF16, dim=dim, rot=rot, interleaved=interleaved)
    check(FP16, FP16, dim=dim, rot=rot, interleaved=interleaved)


@pytest.mark.parametrize("kv_heads,group", [(1, 1), (1, 7), (3, 5), (5, 1), (8, 4), (9, 2), (16, 16)])
@pytest.mark.parametrize("dim", [64, 128])
def test_head_counts(kv_heads, group, dim):
    check(E5M2, BF16, lens=[(5, 30), (1, 3)], kv_heads=kv_heads, group=group, dim=dim)


@pytest.mark.parametrize("page,layout", [(1, "nhd"), (4, "hnd"), (64, "kv"), (256, "hnd")])
def test_pages(page, layout):
    check(E4M3, FP16, page=page, layout=layout)
    check(BF16, BF16, page=page, layout=layout)


@pytest.mark.parametrize("magnitude", [1.2079441541679836, -0.5, 0.0, 300.0])
def test_magnitudes(magnitude):
    check(BF16, BF16, magnitude=magnitude)
    check(E5M2, FP16, magnitude=magnitude, lens=[(9, 9), (1, 40)])


def test_given_positions():
    """Far ones, negative ones, the same twice."""
    most = (1 << 30) - 1

    def given(step):
        p = torch.arange(step.tokens) * 97777 % 1000003
        p[:9] = torch.tensor([0, 1, -1, most, -most, most, 1 << 20, (1 << 31) - 1, -(1 << 31)])
        return p

    for base in (10000.0, 1000000.0):
        check(BF16, BF16, given=given, base=base)
        check(FP16, FP16, given=given, base=base, interleaved=True)
        check(E4M3, FP16, given=given, base=base, rot=64)


@pytest.mark.parametrize("tokens", [1, 2, 63, 300, 4863, 4865, 9000])
def test_few_and_many_tokens(tokens):
    """Either side of how a token's heads are dealt to warps."""
    check(E5M2, BF16, lens=[(tokens, tokens + 3)], kv_heads=2, group=3, dim=64, seed=tokens)


def test_rows_without_a_sequence_or_a_place():
    check(E5M2, BF16, spare=5)
    check(FP16, FP16, spare=3)
    # more new tokens than the sequence holds: the first have no place, and their queries are turned all the same
    step = Step(BF16, [(6, 4), (2, 20)])
    f = sz.rotary_frequencies(128)
    q, k, v, q_out = run(step, 4, f)
    assert int(step.status[0]) == sz.OK
    want, off = rotated(q, places(step), f, False, 1.0)
    near(q_out, want, off, BF16)
    want, off = rotated(k, places(step), f, False, 1.0)
    check_cache(step, "k", want, off, None)


def test_in_place_and_slices_of_a_projection():
    step = Step(E4M3, LENS, kv_heads=2)
    f = sz.rotary_frequencies(128)
    fused = torch.randn(step.tokens, 8 + 2 + 2, 128, generator=step.gen).to(BF16)
    dev = fused.cuda()
    run(step, 8, f, q=dev[:, :8], k=dev[:, 8:10], v=dev[:, 10:], q_out=dev[:, :8])
    assert int(step.status[0]) == sz.OK
    want, off = rotated(fused[:, :8], places(step), f, False, 1.0)
    near(dev[:, :8], want, off, BF16)
    assert torch.equal(dev[:, 8:].cpu(), fused[:, 8:])
    want, off = rotated(fused[:, 8:10], places(step), f, False, 1.0)
    check_cache(step, "k", want, off, None)


def test_without_queries():
    step = Step(E5M2, LENS)
    f = sz.rotary_frequencies(64)
    k, v = step.new_rows(), step.new_rows()
    sz.kv_rotary_write(step.cache, step.batch, sz.KVRotary(f), None, None, k.cuda(), v.cuda(), step.status)
    assert int(step.status[0]) == sz.OK
    want, off = rotated(k, places(step), f, False, 1.0)
    check_cache(step, "k", want, off, None)


@pytest.mark.parametrize("dtype", [BF16, E5M2, E4M3])
def test_no_turn_is_a_plain_write(dtype):
    """Frequencies of zero: the bits that kv_write stores, infinities and NaN included."""
    steps = [Step(dtype, LENS, seed=4) for _ in range(2)]
    k, v = steps[0].new_rows(), steps[0].new_rows()
    for t in (k, v):
        t[0, 0, 3], t[1, 1, 70], t[2, 0, 64], t[3, 0] = math.inf, -math.inf, math.nan, 0.0
        t[4, 1, 5] = 1e-38
    run(steps[0], 2, torch.zeros(32, dtype=torch.float64), k=k, v=v)
    # the rotation of an infinity by nothing makes a NaN of its partner (0 times infinity)
    special = torch.zeros(steps[0].tokens, 2, dtype=torch.bool)
    special[0, 0] = special[2, 0] = True
    sz.kv_write(steps[1].cache, steps[1].batch, k.cuda(), v.cuda(), steps[1].status)
    torch.cuda.synchronize()
    raw = RAW[dtype]
    assert torch.equal(steps[0].cache.v.view(raw), steps[1].cache.v.view(raw))
    a, b = (s.cache.k.view(raw).cpu() for s in steps)
    for bq, (t, n) in enumerate(LENS):
        for i in range(t):
            page, slot = steps[0].place(bq, n - t + i)
            for h in range(2):
                if not special[steps[0].cu[bq] + i, h]:
                    assert torch.equal(a[page, slot, h], b[page, slot, h])
    if steps[0].fp8:
        assert torch.equal(steps[0].cache.v_scale, steps[1].cache.v_scale)
        assert torch.equal(steps[0].cache.k_scale, steps[1].cache.k_scale)


@pytest.mark.parametrize("dtype", [BF16, E5M2, E4M3])
def test_infinities_and_nan_of_a_key(dtype):
    """They reach their pair; the other elements keep their scale."""
    step = Step(dtype, [(4, 4)], kv_heads=1)
    f = sz.rotary_frequencies(128)
    k = step.new_rows()
    k[1, 0, 5], k[2, 0, 70] = math.inf, math.nan
    clean = k.clone()
    clean[1, 0, 5] = clean[1, 0, 69] = clean[2, 0, 70] = clean[2, 0, 6] = 0.0
    run(step, 2, f, k=k)
    got = step.cache.k.view(RAW[dtype]).cpu().view(dtype).float()
    want, off = rotated(clean, places(step), f, False, 1.0)
    for pos, pair in ((1, (5, 69)), (2, (6, 70))):
        page, slot = step.place(0, pos)
        row = got[page, slot, 0]
        assert not torch.isfinite(row[list(pair)]).any()
        others = [i for i in range(128) if i not in pair]
        unit = 2.0 ** (int(step.cache.k_scale[page, 0, slot]) - 127) if step.fp8 else 1.0
        err = (row[others].double() * unit - want[pos, 0, others]).abs()
        size = want[pos, 0].abs().max()
        assert bool((err <= half_step(dtype) * want[pos, 0, others].abs() + 2.0 ** -9 * size + off[pos, 0, others]).all())
        if dtype == E4M3:
            assert torch.isnan(row[list(pair)]).all()


def test_bad_pages_and_entries_are_reported():
    f = sz.rotary_frequencies(128)
    step = Step(E5M2, [(3, 40), (2, 20)])
    before = step.cache.k.view(torch.uint8).clone()
    step.batch.page_table[0, 2] = step.pages  # the page of positions 32 .. 47
    q, k, v, q_out = run(step, 4, f)
    assert int(step.status[0]) == sz.ERR_INVALID_ARG
    want, off = rotated(q, places(step), f, False, 1.0)
    near(q_out, want, off, BF16)  # the queries are turned
    page, slot = step.place(0, 39)
    assert torch.equal(step.cache.k.view(torch.uint8)[page, slot], before[page, slot])
    page, slot = step.place(1, 19)
    assert not torch.equal(step.cache.k.view(torch.uint8)[page, slot], before[page, slot])
    step = Step(E5M2, [(3, 40), (2, 20)])
    step.batch.kv_len[1] = 1 << 29
    run(step, 4, f)
    assert int(step.status[0]) == sz.ERR_INVALID_ARG


def test_helpers_refuse_what_does_not_go_together():
    step = Step(BF16, [(3, 40)])
    r = sz.KVRotary(sz.rotary_frequencies(128))
    q, k = torch.zeros(3, 4, 128, dtype=BF16, device="cuda"), torch.zeros(3, 2, 128, dtype=BF16, device="cuda")
    for args, error in (((q, None, k, k), ValueError), ((None, q, k, k), ValueError), ((q, q[:, :2], k, k), ValueError),
                        ((q.half(), q, k, k), TypeError), ((q, q, k, k.half()), TypeError), ((q, q, q, k), ValueError),
                        ((q[0], q[0], k, k), ValueError), ((q.cpu(), q, k, k), ValueError)):
        with pytest.raises(error):
            sz.kv_rotary_write(step.cache, step.batch, r, *args, step.status)
    for p in (torch.zeros(3, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"),
              torch.zeros(6, dtype=torch.int32, device="cuda")[::2], torch.zeros(3, dtype=torch.int32)):
        with pytest.raises(ValueError):
            sz.kv_rotary_write(step.cache, step.batch, r, q, q, k, k, step.status, positions=p)
    with pytest.raises(sz.SplitZipError):  # more elements than the head has
        half = Step(BF16, [(3, 40)], dim=64)
        sz.kv_rotary_write(half.cache, half.batch, r, None, None, k[..., :64], k[..., :64], half.status)
