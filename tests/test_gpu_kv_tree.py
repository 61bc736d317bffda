"""GPU: attention of trees of drafted tokens over a paged cache against the
formula in 64 bits, element by element, within the roundings that
splitzip_kv_attention documents; masks and positions value by value."""
import math
import random

import pytest
import torch

import lossless_kv_cache_gb300 as sz
from tests.kv_reference import Step, check_attention
from tests.kv_reference import attention as causal_attention

pytestmark = pytest.mark.gpu

BF16, FP16, E5M2, E4M3 = torch.bfloat16, torch.float16, torch.float8_e5m2, torch.float8_e4m3fn
TYPES = [(BF16, BF16), (FP16, FP16), (E5M2, BF16), (E5M2, FP16), (E4M3, BF16), (E4M3, FP16)]


@pytest.fixture(scope="module", autouse=True)
def _lib(splitzip_lib):
    assert torch.cuda.is_available()
    return splitzip_lib


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def grow(t, shape, r):
    """Parents of a tree of t tokens."""
    if shape == "chain":
        return list(range(-1, t - 1))
    if shape == "roots":
        return [-1] * t
    return [r.randint(max(-1, i - 9), i - 1) for i in range(t)]


def parents_of(step, shape="random", seed=1):
    r = random.Random(seed)
    return [p for t, _ in step.lens for p in grow(t, shape, r)]


def branches(step, parents):
    """For every packed row its branch, from itself up."""
    rows = []
    for b, (t, _) in enumerate(step.lens):
        for i in range(t):
            branch = [i]
            while parents[step.cu[b] + branch[-1]] >= 0:
                branch.append(parents[step.cu[b] + branch[-1]])
            rows.append(branch)
    return rows


def attention(step, q, scale, seen):
    """As kv_reference.attention, with the positions seen(b, i) of every row."""
    tokens, heads, dim = q.shape
    group = heads // step.kv_heads
    out, mag = (torch.zeros(tokens, heads, dim, dtype=torch.float64) for _ in range(2))
    lse = torch.full((tokens, heads), -math.inf, dtype=torch.float64)
    size = torch.zeros(tokens, heads, dtype=torch.float64)
    for b, (t, n) in enumerate(step.lens):
        if t == 0 or n == 0:
            continue
        k, v = step.held(b, "k"), step.held(b, "v")
        for i in range(t):
            sees = seen(b, i)
            if not sees.any():
                continue
            r = step.cu[b] + i
            for h in range(step.kv_heads):
                hs = slice(h * group, (h + 1) * group)
                x, kk, vv = q[r, hs].double(), k[sees, h], v[sees, h]
                s = x @ kk.T * scale
                norm = torch.logsumexp(s, -1)
                w = torch.exp(s - norm[:, None])
                out[r, hs], mag[r, hs], lse[r, hs] = w @ vv, w @ vv.abs(), norm
                size[r, hs] = (x.abs() @ kk.abs().T * abs(scale)).amax(-1)
    return out, lse, mag, size


def seen_by_tree(step, parents, window):
    rows = branches(step, parents)

    def seen(b, i):
        t, n = step.lens[b]
        first = n - t
        sees = torch.zeros(n, dtype=torch.bool)
        if first + i < 0:
            return sees
        branch = rows[step.cu[b] + i]
        position = first + len(branch) - 1
        sees[max(0, position - window + 1) if window else 0: max(first, 0)] = True
        for j in branch[: window or None]:
            if first + j >= 0:
                sees[first + j] = True
        return sees

    return seen


def run(step, parents, q, scale, window=0, tree=None, out=None, bufs=None):
    q = q if q.is_cuda else q.cuda()
    if tree is None:
        tree = sz.KVTree(step.batch, window)
        tree.mask.fill_(-1)
        tree.status.fill_(-1)
        given = parents + [0] * (step.tokens - len(parents))
        sz.kv_tree(step.batch, ints(given), tree)
        assert int(tree.status[0]) == sz.OK
    bufs = bufs or sz.KVAttentionBuffers(step.cache, step.batch, q.shape[1])
    out = torch.full(q.shape, 77.0, dtype=q.dtype, device="cuda") if out is None else out
    lse = torch.full(q.shape[:2], 77.0, device="cuda")
    sz.kv_tree_attention(step.cache, step.batch, tree, q, out, bufs, scale, lse=lse)
    torch.cuda.synchronize()
    return out, lse, int(bufs.status[0]), tree


def weight_type(step):
    return FP16 if step.dtype == FP16 else BF16


def check(step, group=4, scale=None, window=0, shape="random", q_spread=1.0, spare=0):
    scale = 1 / math.sqrt(step.dim) if scale is None else scale
    q = (torch.randn(step.tokens, step.kv_heads * group, step.dim, generator=step.gen) * q_spread).to(step.x)
    parents = parents_of(step, shape)
    out, lse, status, tree = run(step, parents, q, scale, window)
    assert status == sz.OK
    rows = step.tokens - spare
    ref = [x[:rows] for x in attention(step, q[:rows], scale, seen_by_tree(step, parents, window))]
    check_attention(step, out[:rows], lse[:rows], ref, weight_type(step))
    assert bool((out[rows:] == 77).all()) and bool((lse[rows:] == 77).all())
    position = [n - t + len(br) - 1 for (t, n), rows_of in zip(step.lens, split(step, branches(step, parents)))
                for br in rows_of]
    assert tree.position.tolist()[:rows] == position


def split(step, rows):
    return [rows[step.cu[b]: step.cu[b + 1]] for b in range(len(step.lens))]


# trees of few rows by any group, then of many; what is before them ends on and beside units of keys
FEW = [(1, 1), (2, 65), (0, 40), (2, 300), (1, 64), (2, 2), (2, 17), (2, 66)]
MANY = [(40, 40), (1, 130), (0, 9), (33, 257), (7, 8), (70, 198), (64, 192), (33, 161), (17, 128)]


@pytest.mark.parametrize("dtype,x", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens", [FEW, MANY])
def test_types(dtype, x, dim, lens):
    check(Step(dtype, lens, dim=dim, x=x))


@pytest.mark.parametrize("shape", ["chain", "roots", "random"])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_shapes(dtype, shape):
    check(Step(dtype, FEW), shape=shape)
    check(Step(dtype, [(8, 20), (4, 90)]), group=2, shape=shape)   # tiles of sixteen rows
    check(Step(dtype, MANY), shape=shape)


@pytest.mark.parametrize("t", [1, 2, 3, 7, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300, 1024])
def test_sizes_of_trees(t):
    """Words of the mask, units of keys and tiles of rows begin and end inside trees."""
    for before in (0, 1, 50, 127, 128):
        if t < 300 or before in (0, 50):
            check(Step(BF16, [(t, t + before), (0, 3), (1, 1)], kv_heads=1), group=1)
    if t <= 129:
        check(Step(E5M2, [(t, t + 40)], kv_heads=1), group=5)


@pytest.mark.parametrize("group,kv_heads", [(1, 1), (1, 8), (3, 3), (5, 1), (7, 2), (8, 4), (16, 1), (64, 1)])
def test_heads(group, kv_heads):
    check(Step(FP16, [(3, 90), (5, 37)], kv_heads=kv_heads), group=group)
    check(Step(E4M3, [(20, 90), (9, 300)], kv_heads=kv_heads, dim=64), group=group)


@pytest.mark.parametrize("page,layout", [(1, "nhd"), (4, "hnd"), (8, "kv"), (64, "hnd"), (256, "nhd")])
@pytest.mark.parametrize("dtype", [BF16, E5M2])
def test_pages(dtype, page, layout):
    check(Step(dtype, FEW, page=page, layout=layout))
    check(Step(dtype, MANY, page=page, layout=layout))


@pytest.mark.parametrize("window", [1, 2, 3, 15, 64, 100, 1000, (1 << 32) - 1])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_windows(dtype, window):
    check(Step(dtype, FEW), window=window)
    check(Step(dtype, MANY), window=window)
    check(Step(dtype, MANY), window=window, shape="chain")
    check(Step(dtype, [(2, 700), (2, 30)]), window=window, shape="roots")


def test_rows_without_a_place_and_behind_the_last_sequence():
    for dtype in (BF16, E5M2):
        check(Step(dtype, [(5, 3), (2, 60), (2, 0)]), group=2)
        check(Step(dtype, [(50, 30), (2, 60), (9, 0)], spare_rows=7), spare=7)
        check(Step(dtype, [(1, 9)], spare_rows=3), spare=3)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30, 3.0])
def test_scales(scale):
    check(Step(BF16, FEW), scale=scale)
    check(Step(BF16, MANY), scale=scale)


def words_of(step, tree, fill):
    """A mask of the caller's own: fill(row, word)."""
    mask = torch.tensor([[fill(r, w) for w in range(tree.words)] for r in range(step.tokens)], dtype=torch.int64)
    tree.mask.copy_(torch.where(mask >= 1 << 31, mask - (1 << 32), mask).int())
    return mask


@pytest.mark.parametrize("lens", [[(2, 2), (2, 40), (1, 1)], [(40, 40), (33, 300), (65, 90)]])
@pytest.mark.parametrize("dtype", [FP16, E4M3])
def test_masks_of_the_callers_own(dtype, lens):
    """Any bits, bits past the last token, none at all: rows that see nothing."""
    step = Step(dtype, lens)
    tree = sz.KVTree(step.batch, 30)
    r = random.Random(4)
    mask = words_of(step, tree, lambda row, w: 0 if row % 3 == 0 else r.getrandbits(32))
    tree.position.copy_(torch.tensor([r.choice([-50, 0, 31, 39, 299, 1 << 30]) for _ in range(step.tokens)]).int())
    position = tree.position.tolist()

    def seen(b, i):
        t, n = step.lens[b]
        first, row = n - t, step.cu[b] + i
        sees = torch.zeros(n, dtype=torch.bool)
        p = min(max(position[row], first), first + i)
        sees[max(0, p - 30 + 1): first] = True
        for j in range(t):
            sees[first + j] = bool(int(mask[row, j // 32]) >> (j % 32) & 1)
        return sees

    q = torch.randn(step.tokens, 8, step.dim, generator=step.gen).to(step.x)
    out, lse, status, _ = run(step, None, q, 0.1, tree=tree)
    assert status == sz.OK
    ref = attention(step, q, 0.1, seen)
    assert any(torch.isinf(ref[1]).any(-1).tolist())  # rows of nothing are among them
    check_attention(step, out, lse, ref, weight_type(step))


@pytest.mark.parametrize("dtype,x", TYPES)
@pytest.mark.parametrize("t,before,window", [(2, 60, 0), (2, 200, 5), (40, 100, 0), (60, 70, 9)])
def test_what_a_row_does_not_see_has_no_part_in_it(dtype, x, t, before, window):
    """NaN and infinities of K and V in other branches, and behind the window."""
    step = Step(dtype, [(t, t + before), (1, 5)], x=x)
    parents = parents_of(step, "random", seed=6)
    seen = seen_by_tree(step, parents, window)
    r = random.Random(2)
    spots = [before + 1, before + t // 2, before + t - 1]
    for n, pos in enumerate(spots):
        value = [math.nan, math.inf, -math.inf][n] if dtype != E4M3 else math.nan
        step.set_value("v", 0, pos, n % 2, r.randrange(step.dim), value)
        step.set_value("k", 0, pos, 1 - n % 2, r.randrange(step.dim), math.nan)
    if window:
        step.set_value("v", 0, 3, 0, 7, math.nan)
        step.set_value("k", 0, 2, 1, 7, math.nan)
    q = torch.randn(step.tokens, 8, step.dim, generator=step.gen).to(step.x)
    out, lse, status, _ = run(step, parents, q, 0.1, window)
    assert status == sz.OK
    ref = attention(step, q, 0.1, seen)
    r_out, r_lse = ref[0], ref[1]
    # a row that sees a NaN of K is NaN throughout
    gone = torch.isnan(r_lse)
    assert torch.isnan(out.cpu()[gone]).all() and torch.isnan(lse.cpu()[gone]).all()
    assert gone.any() and not gone.all()
    keep = ~gone
    blank = torch.zeros((), dtype=torch.float64)
    r_out = torch.where(keep[..., None], r_out, blank)
    fine = (torch.where(keep[..., None].cuda(), out, torch.zeros_like(out)), torch.where(keep.cuda(), lse, torch.zeros_like(lse)))
    ref = (r_out, torch.where(keep, r_lse, blank), torch.where(keep[..., None], ref[2], blank).nan_to_num(0, 0, 0),
           torch.where(keep, ref[3], blank).nan_to_num(0, 0, 0))
    check_attention(step, fine[0], fine[1], ref, weight_type(step))


def test_a_chain_is_causal_attention():
    """The same bits as kv_attention gives."""
    for lens in ([(2, 200), (1, 9), (2, 65)], [(40, 300), (17, 17), (9, 128)]):
        for dtype in (BF16, E5M2):
            step = Step(dtype, lens)
            q = torch.randn(step.tokens, 8, step.dim, generator=step.gen).to(step.x).cuda()
            out, lse, status, _ = run(step, parents_of(step, "chain"), q, 0.09)
            assert status == sz.OK
            bufs = sz.KVAttentionBuffers(step.cache, step.batch, 8)
            want, want_lse = torch.empty_like(out), torch.empty_like(lse)
            sz.kv_attention(step.cache, step.batch, q, want, bufs, 0.09, lse=want_lse)
            assert bool(((out - want).abs() <= 2.0 ** -6 * want.abs() + 2.0 ** -9).all())
            assert bool(((lse - want_lse).abs() <= 2.0 ** -12 * (1 + want_lse.abs())).all())


def test_long_contexts_and_many_sequences():
    step = Step(BF16, [(3, 9000), (0, 5), (3, 70), (2, 4097)], kv_heads=1)
    check(step, group=3)
    step = Step(E4M3, [(40, 6000), (1, 5), (25, 3001)], kv_heads=1, page=64)
    check(step, group=2)
    step = Step(E5M2, [(1 + i % 3, 3 + 5 * i % 77) for i in range(300)], kv_heads=1, dim=64)
    check(step, group=2)
    step = Step(BF16, [(1 + i % 23, 30 + 5 * i % 77) for i in range(150)], kv_heads=1, dim=64)
    check(step, group=4)


def test_bad_parents_and_entries_are_reported():
    lens = [(3, 9), (40, 50), (2, 8), (4, 7)]
    for seq, at, value in ((0, 0, 0), (0, 2, 2), (1, 39, 39), (1, 5, -2), (2, 1, 1 << 30), (3, 0, -(1 << 31))):
        for extra in (0, 300):  # a block for all sequences, and several
            step = Step(BF16, lens + [(0, 1)] * extra)
            parents = parents_of(step)
            parents[step.cu[seq] + at] = value
            tree = sz.KVTree(step.batch)
            tree.mask.fill_(-1)
            sz.kv_tree(step.batch, ints(parents), tree)
            assert int(tree.status[0]) == sz.ERR_INVALID_ARG
            rows = slice(step.cu[seq], step.cu[seq + 1])
            assert not tree.mask[rows].any()
            t, n = lens[seq]
            assert tree.position[rows].tolist() == list(range(n - t, n))
            other = 1 if seq != 1 else 3
            assert tree.mask[step.cu[other]: step.cu[other + 1]].any(-1).all()
    step = Step(BF16, lens)
    step.batch.kv_len[1] = -4
    tree = sz.KVTree(step.batch)
    tree.mask.fill_(-1)
    sz.kv_tree(step.batch, ints(parents_of(step)), tree)
    assert int(tree.status[0]) == sz.ERR_INVALID_ARG
    assert bool((tree.mask[step.cu[1]: step.cu[2]] == -1).all())
    q = torch.zeros(step.tokens, 8, 128, dtype=BF16, device="cuda")
    bufs = sz.KVAttentionBuffers(step.cache, step.batch, 8)
    sz.kv_tree_attention(step.cache, step.batch, tree, q, torch.empty_like(q), bufs, 0.1)
    assert int(bufs.status[0]) == sz.ERR_INVALID_ARG


@pytest.mark.parametrize("lens", [[(2, 100), (2, 50)], [(40, 100), (33, 70)]])
def test_bad_pages_are_reported(lens):
    step = Step(E5M2, lens)
    for entry in (-1, step.pages, 1 << 30):
        step.batch.page_table[0, 1] = entry
        q = torch.randn(step.tokens, 8, step.dim, generator=step.gen).to(step.x)
        parents = parents_of(step)
        out, lse, status, _ = run(step, parents, q, 0.1)
        assert status == sz.ERR_INVALID_ARG
        rows = slice(step.cu[1], step.cu[2])
        ref = attention(step, q, 0.1, seen_by_tree(step, parents, 0))
        check_attention(step, out[rows], lse[rows], [x[rows] for x in ref], weight_type(step))


def test_a_captured_step_with_other_trees():
    """Masks, lengths and trees change between replays within the step's maxima."""
    for lens in ([(2, 60), (2, 90)], [(30, 60), (20, 90)]):
        step = Step(E5M2, lens, extra_pages=9)
        q = torch.randn(step.tokens, 8, step.dim, generator=step.gen).to(step.x)
        parents = ints(parents_of(step))
        tree = sz.KVTree(step.batch)
        bufs = sz.KVAttentionBuffers(step.cache, step.batch, 8)
        dev, out = q.cuda(), torch.zeros(q.shape, dtype=q.dtype, device="cuda")
        lse = torch.zeros(q.shape[:2], device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            sz.kv_tree(step.batch, parents, tree)
            sz.kv_tree_attention(step.cache, step.batch, tree, dev, out, bufs, 0.1, lse=lse)
        for seed, lens_now in ((1, lens), (2, [(lens[0][0] - 1, 44), (lens[1][0], 77)]), (3, [(1, 33), (0, 5)])):
            step.lens = lens_now
            step.cu = [0, lens_now[0][0], lens_now[0][0] + lens_now[1][0]]
            now = parents_of(step, "random", seed)
            parents[: len(now)] = ints(now)
            step.batch.cu_tokens.copy_(ints(step.cu))
            step.batch.kv_len.copy_(ints([n for _, n in lens_now]))
            out.fill_(77)
            graph.replay()
            torch.cuda.synchronize()
            assert int(bufs.status[0]) == sz.OK and int(tree.status[0]) == sz.OK
            rows = step.cu[-1]
            ref = [x[:rows] for x in attention(step, q[:rows], 0.1, seen_by_tree(step, now, 0))]
            check_attention(step, out[:rows], lse[:rows], ref, weight_type(step))
            assert bool((out[rows:] == 77).all())


def test_helpers_refuse_what_does_not_go_together():
    step = Step(BF16, [(3, 9), (2, 8)])
    tree = sz.KVTree(step.batch)
    other = Step(BF16, [(4, 9)])
    q = torch.zeros(step.tokens, 8, 128, dtype=BF16, device="cuda")
    bufs = sz.KVAttentionBuffers(step.cache, step.batch, 8)
    with pytest.raises(ValueError):
        sz.kv_tree(other.batch, ints([0] * 4), tree)
    with pytest.raises(ValueError):
        sz.kv_tree_attention(step.cache, step.batch, sz.KVTree(other.batch), q, q.clone(), bufs, 0.1)
    for p in (ints([0] * 4), ints([0] * 10)[::2], torch.zeros(5, dtype=torch.int64, device="cuda"),
              torch.zeros(5, dtype=torch.int32)):
        with pytest.raises(ValueError):
            sz.kv_tree(step.batch, p, tree)
    with pytest.raises(TypeError):
        sz.kv_tree_attention(step.cache, step.batch, tree, q, q.half(), bufs, 0.1)
    with pytest.raises(sz.SplitZipError):
        sz.KVTree(Step(BF16, [(1025, 1025)]).batch)


@pytest.mark.parametrize("batch,most", [(1, 1), (32, 33), (32, 64), (33, 64), (5, 65), (300, 20), (3, 1024), (40, 200)])
@pytest.mark.parametrize("window", [0, 1, 40, 700])
def test_masks_and_positions(batch, most, window):
    """Of steps that one block takes and of others, ancestors any number of words back, whatever the mask held."""
    r = random.Random(batch * most + window)
    sizes = [r.randrange(most + 1) for _ in range(batch - 1)] + [most]
    lens = [r.randrange(3 * t + 5) for t in sizes]  # some of fewer tokens than the tree
    parents, bits, positions = [], [], []
    words = min(32, -(-most // 32) + 1)
    for b, (t, n) in enumerate(zip(sizes, lens)):
        up = [[lambda i: i - 1, lambda i: r.randrange(-1, i), lambda i: -1 if i % 3 else r.randrange(-1, i),
               lambda i: max(-1, i - 1 - r.randrange(40))][b % 4](i) for i in range(t)]
        lines = []
        for i, p in enumerate(up):
            lines.append((lines[p] if p >= 0 else []) + [i])
            bits.append([sum(1 << (j % 32) for j in (lines[i][-window:] if window else lines[i]) if j // 32 == w)
                         for w in range(words)])
            positions.append(n - t + len(lines[i]) - 1)
        parents += up
    cu = [sum(sizes[:b]) for b in range(batch + 1)]
    step = sz.KVBatch(ints(cu), ints(lens), torch.zeros(batch, max(lens) + 1, dtype=torch.int32, device="cuda"),
                      cu[-1], most, max(max(lens), 1))
    tree = sz.KVTree(step, window)
    tree.mask = torch.full((cu[-1], words), -1, dtype=torch.int32, device="cuda")  # wider than it has to be
    tree.desc.d_mask, tree.desc.words = tree.mask.data_ptr(), words
    tree.status.fill_(-1)
    sz.kv_tree(step, ints(parents), tree)
    assert int(tree.status[0]) == sz.OK
    assert (tree.mask.long() & 0xFFFFFFFF).tolist() == bits
    assert tree.position.tolist() == positions
    if most > 1:
        parents[cu[-1] - 1] = most - 1  # a parent of its own
        sz.kv_tree(step, ints(parents), tree)
        assert int(tree.status[0]) == sz.ERR_INVALID_ARG
        last = cu[-1] - most
        assert (tree.mask.long() & 0xFFFFFFFF).tolist() == bits[:last] + [[0] * words] * most


# up to 128 rows of a sequence: trees longer than their sequence, none, of no place, beside keys' units
TILE = [(12, 12), (10, 3), (0, 9), (16, 1), (9, 0), (32, 300), (11, 140), (1, 128), (20, 129), (17, 256)]


@pytest.mark.parametrize("dtype,x", TYPES)
@pytest.mark.parametrize("dim,page,layout", [(128, 16, "hnd"), (64, 8, "nhd"), (128, 128, "kv"), (64, 1024, "hnd")])
def test_one_tile_of_rows(dtype, x, dim, page, layout):
    for window in (0, 1, 9, 130, (1 << 32) - 1):
        check(Step(dtype, TILE, dim=dim, x=x, page=page, layout=layout, spare_rows=5), window=window, spare=5)


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("lens", [FEW, TILE, MANY], ids=["few", "tile", "many"])
def test_two_streams_at_once(dtype, lens):
    """Two layers' calls with buffers of their own, one tree for both."""
    steps = [Step(dtype, lens, seed=seed) for seed in (1, 2)]
    parents = parents_of(steps[0], "random")
    qs = [torch.randn(s.tokens, 8, s.dim, generator=s.gen).to(s.x).cuda() for s in steps]
    bufs = [sz.KVAttentionBuffers(s.cache, s.batch, 8) for s in steps]
    want = [run(s, parents, q, 0.1, bufs=b) for s, q, b in zip(steps, qs, bufs)]
    streams = [torch.cuda.Stream() for _ in steps]
    outs = [torch.zeros_like(q) for q in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, q, out, b, w, stream in zip(steps, qs, outs, bufs, want, streams):
            with torch.cuda.stream(stream):
                out.zero_()
                sz.kv_tree_attention(s.cache, s.batch, want[0][3], q, out, b, 0.1)
        torch.cuda.synchronize()
        for out, b, w in zip(outs, bufs, want):
            assert int(b.status[0]) == sz.OK and torch.equal(out.view(torch.int16), w[0].view(torch.int16))


@pytest.mark.parametrize("dtype", [FP16, E4M3])
@pytest.mark.parametrize("lens", [FEW, TILE, MANY, [(9, 3000), (30, 2000)]], ids=["few", "tile", "many", "shares"])
def test_results_in_the_queries_place(dtype, lens):
    step = Step(dtype, lens)
    parents = parents_of(step, "random")
    q = torch.randn(step.tokens, 8, step.dim, generator=step.gen).to(step.x).cuda()
    want, want_lse, _, tree = run(step, parents, q, 0.1)
    out, lse, status, _ = run(step, parents, q, 0.1, tree=tree, out=q)
    assert status == sz.OK and out is q and torch.equal(lse, want_lse)
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("lens", [[(2, 200), (1, 9), (2, 65)], [(6, 500), (7, 300)], [(40, 300), (17, 17), (9, 128)],
                                  [(80, 300), (3, 129)]], ids=["8", "28", "160", "320"])
@pytest.mark.parametrize("dtype,x", TYPES)
@pytest.mark.parametrize("window", [0, 50])
def test_a_chain_sees_what_causal_attention_shows(dtype, x, lens, window):
    """Both within their roundings of the causal formula, whichever kernels take them."""
    step = Step(dtype, lens, x=x)
    q = torch.randn(step.tokens, 8, step.dim, generator=step.gen).to(step.x)
    ref = causal_attention(step, q, 0.09, True, window)
    out, lse, status, _ = run(step, parents_of(step, "chain"), q, 0.09, window)
    assert status == sz.OK
    check_attention(step, out, lse, ref, weight_type(step))
    bufs = sz.KVAttentionBuffers(step.cache, step.batch, 8)
    sz.kv_attention(step.cache, step.batch, q.cuda(), out, bufs, 0.09, window=window, lse=lse)
    assert int(bufs.status[0]) == sz.OK
    check_attention(step, out, lse, ref, weight_type(step))


@pytest.mark.parametrize("lens", [FEW, [(7, 300), (1, 40), (5, 130)], TILE], ids=["few", "28", "tile"])
@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("max_tokens", [0, 7, 30, 100])
def test_maxima_far_above_the_steps_own(dtype, lens, max_tokens):
    """What a captured step has: kernels are chosen by maxima that its sequences do not come near."""
    step = Step(dtype, lens)
    table = torch.full((len(lens), 2048), -7, dtype=torch.int32, device="cuda")
    table[:, : step.table.shape[1]] = step.batch.page_table
    most = max(step.max_new, min(max_tokens, step.tokens))
    step.batch = sz.KVBatch(step.batch.cu_tokens, step.batch.kv_len, table, step.tokens, most, 32768)
    for window in (0, 60):
        check(step, window=window)
