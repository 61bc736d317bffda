"""GPU: page tables, lengths, slots and positions of a step against lists on the
CPU, value by value."""
import random

import pytest
import torch

import lossless_kv_cache_gb300 as sz

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(splitzip_lib):
    assert torch.cuda.is_available()
    return splitzip_lib


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Lists:
    """The same bookkeeping with Python lists."""

    def __init__(self, pool, page, batch, width, seed):
        self.r = random.Random(seed)
        self.page, self.width, self.pool = page, width, pool
        self.free = list(range(pool))
        self.r.shuffle(self.free)
        self.tables = [[] for _ in range(batch)]
        self.lens = [0] * batch

    def fill(self, lens, spare=None):
        """Sequences of these lengths, with pages to spare."""
        for b, n in enumerate(lens):
            self.lens[b] = n
            for _ in range(-(-n // self.page) + (spare[b] if spare else 0)):
                self.tables[b].append(self.free.pop())

    def on_gpu(self):
        table = torch.full((len(self.lens), self.width), -9, dtype=torch.int32)
        for b, t in enumerate(self.tables):
            table[b, : len(t)] = torch.tensor(t, dtype=torch.int32)
        free = self.free + [-5] * (self.pool - len(self.free))
        return sz.KVPages(ints(free), ints([len(self.free)]), table.cuda(), ints([len(t) for t in self.tables]),
                          ints(self.lens), self.page)

    def extend(self, new, drop):
        """(cu, position, slot) of the step; the lists as they are after it."""
        need = []
        for b, n in enumerate(self.lens):
            self.lens[b] = n - drop[b] + new[b]
            need.append(-(-self.lens[b] // self.page))
        for b in reversed(range(len(new))):
            while len(self.tables[b]) > need[b]:
                self.free.append(self.tables[b].pop())
        for b in range(len(new)):
            while len(self.tables[b]) < need[b]:
                self.tables[b].append(self.free.pop())
        cu, position, slot = [0], [], []
        for b, t in enumerate(new):
            cu.append(cu[-1] + t)
            for p in range(self.lens[b] - t, self.lens[b]):
                position.append(p)
                slot.append(self.tables[b][p // self.page] * self.page + p % self.page)
        return cu, position, slot


def check(lists, pages, step, expected, tables_before):
    cu, position, slot = expected
    torch.cuda.synchronize()
    assert int(step.status[0]) == sz.OK
    assert step.cu_tokens.tolist() == cu
    assert pages.kv_len.tolist() == lists.lens
    assert pages.held.tolist() == [len(t) for t in lists.tables]
    assert pages.count.tolist() == [len(lists.free)]
    assert pages.free.tolist()[: len(lists.free)] == lists.free
    table = pages.table.tolist()
    for b, t in enumerate(lists.tables):
        assert table[b][: len(t)] == t
        assert table[b][len(t):] == tables_before[b][len(t):]  # entries past its pages are left as they were
    assert step.position.tolist()[: cu[-1]] == position
    assert step.slot.tolist()[: cu[-1]] == slot
    assert bool((step.position[cu[-1]:] == -77).all()) and bool((step.slot[cu[-1]:] == -77).all())


def step_for(batch, tokens, max_tokens, max_kv_len):
    s = sz.KVStep(batch, tokens, max_tokens, max_kv_len)
    s.position.fill_(-77)
    s.slot.fill_(-77)
    s.status.fill_(-1)
    return s


def scenario(batch, page, most_len, most_new, seed, drops=True):
    r = random.Random(seed)
    lens = [r.choice([0, 1, page, r.randint(0, most_len)]) for _ in range(batch)]
    spare = [r.choice([0, 0, 0, 1, 2, 5]) for _ in range(batch)]
    new = [r.choice([0, 1, 1, r.randint(0, most_new)]) for _ in range(batch)]
    drop = [r.choice([0, 0, n, r.randint(0, n)]) if drops else 0 for n in lens]
    need = [-(-(n + most_new) // page) + 5 for n in lens]
    lists = Lists(sum(need) + 3, page, batch, max(need), seed)
    lists.fill(lens, spare)
    return lists, new, drop


@pytest.mark.parametrize("batch,page,most_len,most_new", [
    (1, 16, 100, 40), (3, 1, 20, 9), (33, 16, 300, 50), (64, 4, 50, 1), (1000, 16, 60, 5), (1024, 8, 30, 3),
    (1025, 16, 40, 4), (3000, 2, 20, 2), (40, 256, 5000, 700), (7, 65536, 200000, 3000), (2, 16, 5, 20000)])
@pytest.mark.parametrize("in_place", [True, False])
def test_against_lists(batch, page, most_len, most_new, in_place):
    lists, new, drop = scenario(batch, page, most_len, most_new, batch * 7 + page)
    pages = lists.on_gpu()
    before = pages.table.tolist()
    step = step_for(batch, sum(new) + 5, max(new + [1]), max(most_len + most_new, 1))
    after = None if in_place else pages.ahead()
    held = [t.clone() for t in (pages.held, pages.kv_len, pages.count)]
    expected = lists.extend(new, drop)
    sz.kv_extend(pages, ints(new), step, drop=ints(drop), after=after)
    check(lists, after or pages, step, expected, before)
    if not in_place:  # what they were read from is as it was
        assert all(torch.equal(a, b) for a, b in zip(held, (pages.held, pages.kv_len, pages.count)))
        # and the same call again gives the same
        sz.kv_extend(pages, ints(new), step, drop=ints(drop), after=after)
        check(lists, after, step, expected, before)


@pytest.mark.parametrize("rows", [2047, 2048, 2049, 4100])
def test_either_side_of_the_rows_that_the_planning_block_takes(rows):
    """The choice goes by the rows that there is room for; both give the same."""
    for spare in (0, 5000):
        lists = Lists(1000, 16, 5, 700, 3)
        lists.fill([100, 0, 33, 16, 7])
        pages = lists.on_gpu()
        before = pages.table.tolist()
        new = [rows - 1200, 0, 1, 1198, 1]
        step = step_for(5, rows + spare, max(new), 12000)
        expected = lists.extend(new, [0] * 5)
        sz.kv_extend(pages, ints(new), step)
        check(lists, pages, step, expected, before)


def test_a_run_of_steps_in_place():
    lists = Lists(400, 4, 20, 60, 5)
    pages = lists.on_gpu()
    r = random.Random(9)
    step = step_for(20, 20 * 12, 12, 240)
    for _ in range(60):
        drop = [r.choice([0, 0, n, r.randint(0, n)]) for n in lists.lens]
        new = [r.randint(0, 12) if n - d < 60 else 0 for n, d in zip(lists.lens, drop)]
        before = pages.table.tolist()
        expected = lists.extend(new, drop)
        step.position.fill_(-77)
        step.slot.fill_(-77)
        sz.kv_extend(pages, ints(new), step, drop=ints(drop))
        check(lists, pages, step, expected, before)
    sz.kv_extend(pages, ints([0] * 20), step, drop=pages.kv_len.clone())
    assert sorted(pages.free.tolist()) == list(range(400)) and pages.count.tolist() == [400]


def test_a_step_taken_back_leaves_the_list_as_it_was():
    lists, new, _ = scenario(50, 4, 90, 30, 11, drops=False)
    lists.tables = [t[: -(-n // 4)] for t, n in zip(lists.tables, lists.lens)]  # no pages to spare
    pages = lists.on_gpu()
    free, count = pages.free.tolist(), int(pages.count)
    step = step_for(50, sum(new), max(new), 200)
    sz.kv_extend(pages, ints(new), step)
    assert int(pages.count) < count
    sz.kv_extend(pages, ints([0] * 50), step, drop=ints(new))
    assert int(pages.count) == count and pages.free.tolist()[:count] == free[:count]
    assert pages.kv_len.tolist() == lists.lens


def unchanged(pages, step, status, drop=None, new=None, after=None):
    snap = [t.clone() for t in (pages.free, pages.count, pages.table, pages.held, pages.kv_len)]
    step.position.fill_(-77)
    step.slot.fill_(-77)
    step.cu_tokens.fill_(5)
    sz.kv_extend(pages, new, step, drop=drop, after=after)
    torch.cuda.synchronize()
    assert int(step.status[0]) == status
    assert all(torch.equal(a, b) for a, b in zip(snap, (pages.free, pages.count, pages.table, pages.held, pages.kv_len)))
    assert not step.cu_tokens.any()
    assert bool((step.position == -77).all()) and bool((step.slot == -77).all())
    if after is not None:
        assert all(torch.equal(a, b) for a, b in ((pages.count, after.count), (pages.held, after.held),
                                                  (pages.kv_len, after.kv_len)))


@pytest.mark.parametrize("batch,tokens", [(6, 500), (1500, 9000)])
def test_too_few_pages_change_nothing(batch, tokens):
    lists = Lists(batch * 2 + 4, 16, batch, 20, 2)
    lists.fill([16] * batch)
    pages = lists.on_gpu()
    step = step_for(batch, tokens, 100, 300)
    new = [1] * batch
    new[2] = 16 * 5 + 1  # six pages; batch + 4 are free
    unchanged(pages, step, sz.ERR_CAPACITY, new=ints(new))
    unchanged(pages, step, sz.ERR_CAPACITY, new=ints(new), after=pages.ahead())
    new[2] = 16 * 4 + 1  # five: exactly those that there are
    sz.kv_extend(pages, ints(new), step)
    assert int(step.status[0]) == sz.OK and int(pages.count) == 0
    # a page given up in the same step counts
    lists = Lists(8, 16, 3, 8, 2)
    lists.fill([64, 16, 16])
    pages, step = lists.on_gpu(), step_for(3, 100, 64, 128)
    unchanged(pages, step, sz.ERR_CAPACITY, new=ints([0, 0, 33]))
    expected = lists.extend([0, 0, 33], [17, 0, 0])
    before = pages.table.tolist()
    step.position.fill_(-77)
    step.slot.fill_(-77)
    sz.kv_extend(pages, ints([0, 0, 33]), step, drop=ints([17, 0, 0]))
    check(lists, pages, step, expected, before)


def test_entries_out_of_range_change_nothing():
    def fresh(count=None, held=None, lens=None):
        lists = Lists(40, 16, 3, 6, 2)
        lists.fill([40, 5, 16])
        pages = lists.on_gpu()
        for t, v in ((pages.count, count), (pages.held, held), (pages.kv_len, lens)):
            if v is not None:
                t.copy_(ints(v))
        return pages

    big = (1 << 31) - 1
    step = step_for(3, 50, 40, 90)
    zero = ints([0, 0, 0])
    for new in ([-1, 0, 0], [0, 41, 0], [0, 0, big], [0, -big, 0], [30, 21, 0], [0, 40, 40]):
        unchanged(fresh(), step, sz.ERR_INVALID_ARG, new=ints(new))
    for drop in ([41, 0, 0], [0, -1, 0], [0, 0, big], [0, -big - 1, 0]):
        unchanged(fresh(), step, sz.ERR_INVALID_ARG, new=zero, drop=ints(drop))
    unchanged(fresh(), step_for(3, 50, 40, 39), sz.ERR_INVALID_ARG, new=zero)          # longer than the step allows
    unchanged(fresh(), step_for(3, 100, 100, 1000), sz.ERR_INVALID_ARG, new=ints([60, 0, 0]))  # than the table holds
    for count in ([-1], [41], [big], [-big - 1]):
        unchanged(fresh(count=count), step, sz.ERR_INVALID_ARG, new=zero)
    for held in ([2, 1, 1], [3, 0, 1], [7, 1, 1], [-1, 1, 1], [3, 1, big]):
        unchanged(fresh(held=held), step, sz.ERR_INVALID_ARG, new=zero)
    for lens in ([-1, 5, 16], [big, 5, 16], [49, 5, 16]):
        unchanged(fresh(lens=lens), step, sz.ERR_INVALID_ARG, new=zero)
    # pages that would not fit the list: more given up than the pool has
    pages = fresh(count=[39])
    unchanged(pages, step, sz.ERR_INVALID_ARG, new=zero, drop=ints([40, 0, 0]))


def test_sequences_of_nothing():
    lists = Lists(4, 16, 40, 2, 2)
    pages = lists.on_gpu()
    before = pages.table.tolist()
    step = step_for(40, 0, 0, 16)
    expected = lists.extend([0] * 40, [0] * 40)
    sz.kv_extend(pages, ints([0] * 40), step)
    check(lists, pages, step, expected, before)


def test_another_stream_and_a_captured_step():
    lists = Lists(300, 16, 9, 30, 4)
    pages = lists.on_gpu()
    step = step_for(9, 60, 40, 400)
    new, drop = ints([0] * 9), ints([0] * 9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        sz.kv_extend(pages, new, step, drop=drop)
    r = random.Random(3)
    for _ in range(20):
        n = [r.randint(0, 6) for _ in range(9)]
        d = [r.randint(0, min(x, 3)) for x in lists.lens]
        before = pages.table.tolist()
        new.copy_(ints(n))
        drop.copy_(ints(d))
        step.position.fill_(-77)
        step.slot.fill_(-77)
        expected = lists.extend(n, d)
        graph.replay()
        check(lists, pages, step, expected, before)


def test_helpers_refuse_what_does_not_go_together():
    pages = sz.KVPages.empty(10, 16, 3, 100)
    step = sz.KVStep(3, 10, 5, 100)
    other = sz.KVPages.empty(10, 16, 3, 100)
    good = ints([1, 0, 0])
    with pytest.raises(ValueError):
        sz.kv_extend(pages, good, step, after=other)         # another list
    with pytest.raises(ValueError):
        sz.kv_extend(pages, good, sz.KVStep(4, 10, 5, 100))
    for new in (ints([1, 0]), good.long(), good.cpu(), ints([1, 0, 0, 0, 0, 0])[::2]):
        with pytest.raises(ValueError):
            sz.kv_extend(pages, new, step)
    with pytest.raises(ValueError):
        sz.KVPages(pages.free, pages.count, pages.table[:, ::2], pages.held, pages.kv_len, 16)
    with pytest.raises(ValueError):
        sz.KVPages(pages.free, pages.count, pages.table[:1].expand(3, -1), pages.held, pages.kv_len, 16)
    sz.kv_extend(pages, good, step)
    assert int(step.status[0]) == sz.OK and pages.kv_len.tolist() == [1, 0, 0]


def test_a_step_is_of_its_pages():
    """With pages of another size the table's entries past a sequence's pages would be taken for its own."""
    pages = sz.KVPages.empty(8, 32, 2, 120)
    pages.table = torch.zeros(2, 8, dtype=torch.int32, device="cuda")
    pages = sz.KVPages(pages.free, pages.count, pages.table, pages.held, pages.kv_len, 32)
    step = sz.KVStep(2, 4, 2, 120)
    batch = step.batch_of(pages)
    sz.kv_extend(pages, ints([2, 1]), step)
    rows = torch.zeros(4, 2, 128, dtype=torch.bfloat16, device="cuda")
    status = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    for many, size in ((8, 16), (16, 16), (8, 64), (7, 32)):
        cache = sz.KVCache.empty(many, size, 2, 128, torch.bfloat16)
        rotary = sz.KVRotary(sz.rotary_frequencies(128))
        for call in (lambda: sz.kv_write(cache, batch, rows, rows, status),
                     lambda: sz.kv_rotary_write(cache, batch, rotary, None, None, rows, rows, status),
                     lambda: sz.kv_tree_attention(cache, batch, sz.KVTree(batch), rows, rows.clone(), None, 0.1),
                     lambda: sz.kv_keep(sz.KVLayers([cache]), batch, ints([0] * 4), ints([0, 0]), status)):
            with pytest.raises(ValueError):
                call()
    assert int(status[0]) == -1
    for many in (8, 9):
        sz.kv_write(sz.KVCache.empty(many, 32, 2, 128, torch.bfloat16), batch, rows, rows, status)
        assert int(status[0]) == sz.OK


@pytest.mark.parametrize("room", [4095, 4096, 4097, 4100])
@pytest.mark.parametrize("short", [0, 1, 3000])
@pytest.mark.parametrize("batch", [5, 300])
def test_either_side_of_the_room_that_the_planning_block_maps(room, short, batch):
    """Up to 4,096 rows that there is room for are mapped by the block that plans, however many there are."""
    lists = Lists(5000, 16, batch, 700, 3)
    lists.fill([100, 0, 33, 16, 7] * (batch // 5))
    pages = lists.on_gpu()
    before = pages.table.tolist()
    new = [room - short - batch + 2] + [0] + [1] * (batch - 2)
    step = step_for(batch, room, max(new), 12000)
    expected = lists.extend(new, [0] * batch)
    sz.kv_extend(pages, ints(new), step)
    check(lists, pages, step, expected, before)
