"""GPU: tree attention over FP8 pages whose scales say little of the values'
size, whole units of rows of zeros, or differ far from unit to unit."""
import math

import pytest
import torch

import lossless_kv_cache_gb300 as sz
from tests.kv_long_reference import LongStep, attention64
from tests.kv_reference import RAW, Step, check_attention, quantise
from tests.test_gpu_kv_tree import attention, parents_of, seen_by_tree
from tests.test_gpu_kv_tree import run as run_tree
from tests.test_gpu_kv_tree_long import own_size, run
from tests.test_gpu_kv_weights import shift_scales

pytestmark = pytest.mark.gpu

BF16, E5M2, E4M3 = torch.bfloat16, torch.float8_e5m2, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib(splitzip_lib):
    assert torch.cuda.is_available()
    return splitzip_lib


def aligned_step(dtype, dim, lens, heads=32):
    """(step, q, scale, a row of K whose score is about 10 for every q)."""
    step = LongStep(dtype, lens, dim=dim, kv_heads=8)
    step.host = {name: x.cpu() for name, x in step.host.items()}
    step.held = lambda b, name: step.host[name][step.table[b, : -(-lens[b][1] // step.page)].long()].reshape(
        -1, step.kv_heads, dim)[: lens[b][1]]
    u = torch.randn(dim, generator=step.gen, dtype=torch.float64)
    q = (u + 0.3 * torch.randn(step.tokens, heads, dim, generator=step.gen)).to(BF16)
    scale = 1 / math.sqrt(dim)
    return step, q, scale, torch.sign(u) * 10 / (scale * u.abs().sum())


def set_rows(step, name, b, positions, row):
    """Rows of all heads as kv_write leaves them: a row of zeros has the scale 2^0."""
    pool, scales = (step.cache.k, step.cache.k_scale) if name == "k" else (step.cache.v, step.cache.v_scale)
    elements, k = quantise(row[None], step.dtype)
    k, bits = int(k[0]), elements[0].float().to(step.dtype)
    at = torch.tensor([step.place(b, pos) for pos in positions])
    pages, slots = at[:, 0], at[:, 1]
    step.host[name][pages, slots] = torch.ldexp(bits.double(), torch.tensor(k))
    pool.view(RAW[step.dtype])[pages.cuda(), slots.cuda()] = bits.view(RAW[step.dtype]).cuda()
    scales.transpose(1, 2)[pages.cuda(), slots.cuda()] = 127 + k


def whole_units(n):
    """Positions of units of 128 keys: the first, one that both groups come to later, the last."""
    return {"first": range(128), "middle": range(384, 512), "last": range((n - 1) // 128 * 128, n),
            "first and middle": [*range(128), *range(256, 512)], "all but one": [*range(256), *range(384, n)]}


@pytest.mark.parametrize("dtype,dim", [(E5M2, 128), (E4M3, 128), (E4M3, 64)])
@pytest.mark.parametrize("small", [0, -8, -12, -40])
@pytest.mark.parametrize("where", list(whole_units(1)))
def test_units_of_nothing_but_zeros(dtype, dim, small, where):
    """They are written with the scale 2^0, larger than the others', and add nothing: the weights
    of the others, whose scores are lower, are all of the result."""
    n = 7 * 128 + 1
    step, q, scale, row = aligned_step(dtype, dim, [(5, n)] * 20)  # a block has 13 units or 14, a whole sequence's
    shift_scales(step, "v", small)
    positions = whole_units(n)[where]
    for b in range(20):
        set_rows(step, "k", b, positions, row)
        set_rows(step, "v", b, positions, torch.zeros(dim, dtype=torch.float64))
    out, _ = run(step, q.cuda(), scale)
    own_size(step, q, out, attention64(step, q, scale), scale)


@pytest.mark.parametrize("dtype", [E5M2, E4M3])
@pytest.mark.parametrize("at", [5, 300, 500])
def test_a_value_that_dwarfs_the_ones_after_it(dtype, at):
    """The sum of weights is of every key, down to values 2^100 smaller than another's."""
    step, q, scale, row = aligned_step(dtype, 128, [(5, 897)] * 20)
    shift_scales(step, "v", -30)
    large = torch.ldexp(torch.sign(torch.randn(128, generator=step.gen, dtype=torch.float64)), torch.tensor(70))
    for b in range(20):
        set_rows(step, "k", b, [at], row)
        set_rows(step, "v", b, [at], large)
    out, _ = run(step, q.cuda(), scale)
    own_size(step, q, out, attention64(step, q, scale), scale)


@pytest.mark.parametrize("dtype,dim", [(E5M2, 128), (E4M3, 64)])
@pytest.mark.parametrize("seed", range(3))
def test_units_of_any_scale(dtype, dim, seed):
    step, q, scale, _ = aligned_step(dtype, dim, [(5, 897)] * 20)
    jumps = torch.tensor([-55, -31, 0, 31, 40])
    for b in range(20):
        e = jumps[torch.randint(len(jumps), (8,), generator=torch.Generator().manual_seed(31 * seed + b))]
        at = torch.tensor([step.place(b, pos) for pos in range(897)])
        by = e[torch.arange(897) // 128]
        step.host["v"][at[:, 0], at[:, 1]] = torch.ldexp(step.host["v"][at[:, 0], at[:, 1]], by[:, None, None])
        scales = step.cache.v_scale.transpose(1, 2)
        at = at.cuda()
        scales[at[:, 0], at[:, 1]] = (scales[at[:, 0], at[:, 1]].int() + by.cuda()[:, None].int()).to(torch.uint8)
    out, _ = run(step, q.cuda(), scale)
    own_size(step, q, out, attention64(step, q, scale), scale)


@pytest.mark.parametrize("dtype", [E5M2, E4M3])
@pytest.mark.parametrize("t,before", [(2, 70), (7, 200), (30, 70), (70, 60)], ids=["8", "28", "120", "280"])
def test_scales_of_slots_that_a_row_does_not_see(dtype, t, before):
    """Whatever was left in them, 0 and 255 too, with the number of rows that each kernel takes."""
    for k_scale, v_scale in ((255, 255), (127, 255), (255, 127), (0, 0), (255, 0), (254, 254)):
        step = Step(dtype, [(t, t + before), (1, 5)])
        parents = parents_of(step, "roots")  # of t tokens, each sees itself alone
        hidden = [0, t - 1]
        for i in hidden:
            pg, off = step.place(0, before + i)
            step.cache.k_scale[pg, :, off] = k_scale
            step.cache.v_scale[pg, :, off] = v_scale
        q = torch.randn(step.tokens, 8, step.dim, generator=step.gen).to(step.x)
        out, lse, status, _ = run_tree(step, parents, q, 0.1)
        assert status == sz.OK
        ref = attention(step, q, 0.1, seen_by_tree(step, parents, 0))
        keep = torch.tensor([r for r in range(step.tokens) if r not in hidden], dtype=torch.long)
        if len(keep) > 0:
            check_attention(step, out.cpu()[keep], lse.cpu()[keep], [x[keep] for x in ref], BF16)
