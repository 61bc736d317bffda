"""GPU: what the roundings of the weights are taken against in attention over
FP8 pages.  Errors are held to the result's own size, however small the values
of V are, and not to an absolute one."""
import math

import pytest
import torch

import lossless_kv_cache_gb300 as sz
from tests.kv_long_reference import attention64
from tests.kv_reference import RAW, Step, check_attention, half_step

pytestmark = pytest.mark.gpu

BF16, FP16, E5M2, E4M3 = torch.bfloat16, torch.float16, torch.float8_e5m2, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib(splitzip_lib):
    assert torch.cuda.is_available()
    return splitzip_lib


def shift_scales(step, name, e):
    scale = getattr(step.cache, name + "_scale")
    scale.copy_((scale.int() + e).to(torch.uint8))
    step.host[name] = torch.ldexp(step.host[name], torch.tensor(e))


def most_weight(step, q, scale):
    """For each (row, head) the largest weight times its key's largest |v|, in doubles (causal)."""
    tokens, heads, _ = q.shape
    group = heads // step.kv_heads
    most = torch.zeros(tokens, heads, dtype=torch.float64)
    for b, (t, n) in enumerate(step.lens):
        k, v = step.held(b, "k"), step.held(b, "v")
        for i in range(t):
            p = n - t + i
            for h in range(heads):
                s = k[: p + 1, h // group] @ q[step.cu[b] + i, h].double() * scale
                most[step.cu[b] + i, h] = (torch.softmax(s, 0) * v[: p + 1, h // group].abs().amax(-1)).amax()
    return most


@pytest.mark.parametrize("dtype", [E5M2, E4M3])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("small", [0, -10, -40])
@pytest.mark.parametrize("lens", [[(1, 900), (2, 300)], [(4, 700)]])
def test_rows_of_zeros_in_v_leave_the_others_their_weights(dtype, dim, small, lens):
    """A row of zeros is written with the scale 2^0, ordinary ones with 2^-14 and less (E5M2).
    Where its key has the largest score, the weights of the others are all of the result."""
    step = Step(dtype, lens, dim=dim, spread=0.3)
    shift_scales(step, "v", small)
    u = torch.randn(dim, generator=step.gen, dtype=torch.float64)
    q = (u + 0.3 * torch.randn(step.tokens, 8, dim, generator=step.gen)).to(BF16)
    scale = 1 / math.sqrt(dim)
    aligned = (2.0 * torch.sign(u) * 10 / (scale * u.abs().sum() * 2.0)).float().to(dtype)  # a score of about 10
    for b, (t, n) in enumerate(lens):
        for pos in (0, 5, n // 2, n - t - 1, n - t):
            pg, off = step.place(b, pos)
            step.cache.k.view(RAW[dtype])[pg, off] = aligned.view(RAW[dtype]).cuda()
            step.cache.k_scale[pg, :, off] = 127
            step.host["k"][pg, off] = aligned.double()
            step.cache.v.view(RAW[dtype])[pg, off] = 0
            step.cache.v_scale[pg, :, off] = 127
            step.host["v"][pg, off] = 0.0
    out = torch.empty(q.shape, dtype=BF16, device="cuda")
    bufs = sz.KVAttentionBuffers(step.cache, step.batch, 8)
    sz.kv_attention(step.cache, step.batch, q.cuda(), out, bufs, scale)
    assert int(bufs.status[0]) == sz.OK
    ref, _, mag, size = attention64(step, q, scale)
    # As for kv_reference.check_attention, but for the weights that FP16 holds in its subnormal
    # steps: each is off by 2^-39 of the largest weight by scale, V's elements are up to M of
    # their scale (the type's largest value), and the largest of a row is over M / 2 of it.
    keys = max(n for _, n in lens)
    score = (dim + 4) * 2.0 ** -23 * size + 2.0 ** -21
    rel = half_step(FP16) + 2 * score[..., None] + 2 * (keys / 8 + 16) * 2.0 ** -23
    tol = rel * mag + half_step(BF16) * (1 + rel) * ref.abs()
    tol = tol + keys * 2.0 ** -38 * most_weight(step, q, scale)[..., None]
    worst = float(((out.double().cpu() - ref).abs() / tol).max())
    assert worst <= 1


@pytest.mark.parametrize("dtype,x", [(BF16, BF16), (FP16, FP16), (E5M2, BF16), (E5M2, FP16)])
@pytest.mark.parametrize("lens", [[(3, 300), (2, 2)], [(70, 600), (40, 40)]])
def test_infinite_scores(dtype, x, lens):
    """+infinity: the rows that see it are NaN; -infinity: a weight of 0, and a row that sees
    nothing else sees nothing."""
    dim, heads, scale = 128, 8, 0.05
    for value in (math.inf, -math.inf):
        step = Step(dtype, lens, x=x, spread=0.3)
        q = torch.randn(step.tokens, heads, dim, generator=step.gen).to(step.x)
        q[:, :, 7] = q[:, :, 7].abs() + 1
        at = [n - 2 for _, n in lens]
        for b, pos in enumerate(at):
            for h in range(2):
                step.set_value("k", b, pos, h, 7, value)
        step.set_value("k", 1, 0, 0, 7, value)
        out, lse = torch.empty_like(q).cuda(), torch.empty(q.shape[:2], device="cuda")
        bufs = sz.KVAttentionBuffers(step.cache, step.batch, heads)
        sz.kv_attention(step.cache, step.batch, q.cuda(), out, bufs, scale, lse=lse)
        assert int(bufs.status[0]) == sz.OK
        seen = torch.zeros(step.tokens, heads, dtype=torch.bool)
        for b, (t, n) in enumerate(lens):
            for i in range(t):
                seen[step.cu[b] + i] = n - t + i >= at[b]
                if b == 1 and n == t:  # from position 0 on, the first kv head
                    seen[step.cu[b] + i, : heads // 2] = True
        if value > 0:
            assert bool(torch.isnan(out.cpu()[seen]).all()) and bool(torch.isnan(lse.cpu()[seen]).all())
        else:
            first = step.cu[1]  # sees position 0 alone
            assert bool((out[first, : heads // 2] == 0).all()) and bool((lse[first, : heads // 2] == -math.inf).all())
            seen[:] = False
        ref, ref_lse, mag, _ = attention64(step, q, scale)
        step.host["k"][~torch.isfinite(step.host["k"])] = 0.0
        size = attention64(step, q, scale)[3]
        ref, mag = ref.nan_to_num(0.0), mag.nan_to_num(0.0)
        keep = ~seen
        weight = FP16 if x == FP16 or (step.fp8 and step.max_new * heads // 2 <= 32) else BF16
        check_attention(step, out.cpu()[keep], lse.cpu()[keep], (ref[keep], ref_lse[keep], mag[keep], size[keep]), weight)
