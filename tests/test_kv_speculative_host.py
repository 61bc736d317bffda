"""The operators of a speculative step, what needs no GPU: refusals of bad
arguments before any GPU work, frequencies and their fixed-point form."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

import lossless_kv_cache_gb300 as sz
from tests.test_kv_host import (A, BATCH, CACHE, INVALID_BATCH, INVALID_CACHE, ROWS, UNSUPPORTED_BATCH,
                                UNSUPPORTED_CACHE, desc)

PAGES = dict(d_free=A, d_free_count=A, d_held=A, d_kv_len=A, d_page_table=A, table_stride=8, table_pages=7,
             pool_pages=100, page_tokens=16, batch=3)
STEP = dict(d_free_count=A, d_held=A, d_kv_len=A, d_cu_tokens=A, d_position=A, d_slot=A, tokens=10, max_tokens=5,
            max_kv_len=64)
ROTARY = dict(d_turns=A, d_position=A, rotary_dim=128, interleaved=0, magnitude=1.0)
TREE = dict(d_mask=A, d_position=A, words=1, window=0)


def extend(pages=None, step=None, new=A, drop=None, ws=A, ws_bytes=1 << 30, status=A):
    return sz.splitzip_kv_extend(desc(sz.KVPagesDesc, PAGES, pages or {}), new, drop,
                                 desc(sz.KVStepDesc, STEP, step or {}), ws, ws_bytes, status, 0)


def rotate(cache=None, batch=None, rotary=None, q=None, q_out=None, q_heads=8, k=None, v=None, dtype=sz.BF16, status=A):
    wide = dict(ROWS, token_stride=8 * 128)
    q, q_out = (None if r == "none" else desc(sz.KVRowsDesc, wide, r or {}) for r in (q, q_out))
    return sz.splitzip_kv_rotary_write(desc(sz.KVCacheDesc, CACHE, cache or {}), desc(sz.KVBatchDesc, BATCH, batch or {}),
                                       desc(sz.KVRotaryDesc, ROTARY, rotary or {}), q, q_out, q_heads,
                                       desc(sz.KVRowsDesc, ROWS, k or {}), desc(sz.KVRowsDesc, ROWS, v or {}), dtype,
                                       status, 0)


def tree(batch=None, parent=A, tree=None, status=A):
    return sz.splitzip_kv_tree(desc(sz.KVBatchDesc, BATCH, batch or {}), parent, desc(sz.KVTreeDesc, TREE, tree or {}),
                               status, 0)


def attend(cache=None, batch=None, tree=None, q=None, out=None, lse=A, dtype=sz.BF16, q_heads=8, scale=0.1, ws=A,
           ws_bytes=1 << 40, status=A):
    rows = dict(ROWS, token_stride=8 * 128)
    return sz.splitzip_kv_tree_attention(desc(sz.KVCacheDesc, CACHE, cache or {}),
                                         desc(sz.KVBatchDesc, BATCH, batch or {}), desc(sz.KVTreeDesc, TREE, tree or {}),
                                         desc(sz.KVRowsDesc, rows, q or {}), desc(sz.KVRowsDesc, rows, out or {}), lse,
                                         dtype, q_heads, scale, ws, ws_bytes, status, 0)


def keep(cache=None, batch=None, count=2, other=None, path=A, kept=A, status=A):
    array = (sz.KVCacheDesc * max(count, 1))(*[
        desc(sz.KVCacheDesc, CACHE, {"d_k": A + 8192 * i, "d_v": A + 8192 * i + 4096, **(cache or {}),
                                     **(other or {} if i else {})}) for i in range(max(count, 1))])
    return sz.splitzip_kv_keep(array, count, desc(sz.KVBatchDesc, BATCH, batch or {}), path, kept, status, 0)


@pytest.mark.parametrize("call", [rotate, attend, keep])
def test_bad_caches_and_steps_are_refused(splitzip_lib, call):
    for kw in INVALID_CACHE:
        assert call(cache=kw) == sz.ERR_INVALID_ARG, kw
    for kw in UNSUPPORTED_CACHE:
        assert call(cache=kw) == sz.ERR_UNSUPPORTED, kw
    for kw in INVALID_BATCH:
        assert call(batch=kw) == sz.ERR_INVALID_ARG, kw
    for kw in UNSUPPORTED_BATCH:
        assert call(batch=kw) == sz.ERR_UNSUPPORTED, kw


@pytest.mark.parametrize("call", [extend, rotate, tree, attend, keep])
def test_bad_status_words_are_refused(splitzip_lib, call):
    assert call(status=None) == sz.ERR_INVALID_ARG
    assert call(status=A + 2) == sz.ERR_INVALID_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU error path")
@pytest.mark.parametrize("call", [extend, rotate, tree, attend, keep])
def test_valid_calls_without_gpu_report_a_cuda_error(splitzip_lib, call):
    assert call() in (sz.ERR_CUDA, sz.ERR_UNSUPPORTED)


def test_extend_arguments_are_checked(splitzip_lib):
    for name in ("d_free", "d_free_count", "d_held", "d_kv_len", "d_page_table"):
        assert extend(pages={name: None}) == sz.ERR_INVALID_ARG, name
        assert extend(pages={name: A + 2}) == sz.ERR_INVALID_ARG, name
    for name in ("d_free_count", "d_held", "d_kv_len", "d_cu_tokens"):
        assert extend(step={name: None}) == sz.ERR_INVALID_ARG, name
        assert extend(step={name: A + 2}) == sz.ERR_INVALID_ARG, name
    for kw in (dict(page_tokens=0), dict(page_tokens=24), dict(page_tokens=1 << 17), dict(batch=0), dict(pool_pages=0),
               dict(table_pages=9)):
        assert extend(pages=kw) == sz.ERR_INVALID_ARG, kw
    for kw in (dict(batch=70000), dict(pool_pages=1 << 31), dict(table_pages=1 << 31, table_stride=1 << 31),
               dict(table_stride=1 << 33)):
        assert extend(pages=kw) == sz.ERR_UNSUPPORTED, kw
    for kw in (dict(d_position=A + 2), dict(d_slot=A + 4), dict(max_tokens=11)):
        assert extend(step=kw) == sz.ERR_INVALID_ARG, kw
    for kw in (dict(tokens=1 << 30), dict(max_kv_len=1 << 30)):
        assert extend(step=kw) == sz.ERR_UNSUPPORTED, kw
    for kw in (dict(new=None), dict(new=A + 2), dict(drop=A + 2), dict(ws=None), dict(ws=A + 8)):
        assert extend(**kw) == sz.ERR_INVALID_ARG, kw
    need = ctypes.c_uint64(0)
    assert sz.splitzip_kv_extend_workspace_size(3, need) == sz.OK and need.value > 0
    assert extend(ws_bytes=need.value - 1) == sz.ERR_CAPACITY
    assert sz.splitzip_kv_extend_workspace_size(0, need) == sz.ERR_INVALID_ARG
    assert sz.splitzip_kv_extend_workspace_size(65537, need) == sz.ERR_UNSUPPORTED


def test_rotary_arguments_are_checked(splitzip_lib):
    for kw in (dict(rotary_dim=0), dict(rotary_dim=24), dict(rotary_dim=144), dict(d_turns=None), dict(d_turns=A + 4),
               dict(d_position=A + 2), dict(magnitude=math.inf), dict(magnitude=math.nan)):
        assert rotate(rotary=kw) == sz.ERR_INVALID_ARG, kw
    for name in ("q", "q_out", "k", "v"):
        for kw in (dict(d=None), dict(d=A + 8), dict(token_stride=1028), dict(head_stride=132), dict(head_stride=64),
                   dict(token_stride=64)):
            assert rotate(**{name: kw}) == sz.ERR_INVALID_ARG, (name, kw)
        if name[0] == "q":
            assert rotate(**{name: "none"}) == sz.ERR_INVALID_ARG, name
    assert rotate(q_heads=0) == sz.ERR_INVALID_ARG
    assert rotate(q_heads=70000) == sz.ERR_UNSUPPORTED
    assert rotate(dtype=sz.FP8_E5M2) == sz.ERR_INVALID_ARG
    assert rotate(cache=dict(type=sz.KV_BF16), dtype=sz.FP16) == sz.ERR_INVALID_ARG


def test_tree_arguments_are_checked(splitzip_lib):
    for call in (tree, attend):
        for kw in (dict(d_mask=None), dict(d_mask=A + 2), dict(d_position=None), dict(d_position=A + 2), dict(words=0),
                   dict(words=33)):
            assert call(tree=kw) == sz.ERR_INVALID_ARG, kw
        assert call(batch=dict(tokens=2000, max_tokens=1025), tree=dict(words=32)) == sz.ERR_UNSUPPORTED
        assert call(batch=dict(tokens=2000, max_tokens=1000), tree=dict(words=31)) == sz.ERR_INVALID_ARG
    assert tree(parent=None) == sz.ERR_INVALID_ARG
    assert tree(parent=A + 2) == sz.ERR_INVALID_ARG
    for kw in INVALID_BATCH:
        if "d_page_table" not in kw and "table_stride" not in kw and kw != dict(max_kv_len=65):
            assert tree(batch=kw) == sz.ERR_INVALID_ARG, kw
    for kw in (dict(q_heads=0), dict(q_heads=7), dict(scale=math.nan), dict(scale=math.inf), dict(lse=A + 2),
               dict(ws=None), dict(ws=A + 8), dict(dtype=3)):
        assert attend(**kw) == sz.ERR_INVALID_ARG, kw
    assert attend(q_heads=2 * 65) == sz.ERR_UNSUPPORTED
    need = ctypes.c_uint64(0)
    assert sz.splitzip_kv_attention_workspace_size(desc(sz.KVCacheDesc, CACHE, {}), desc(sz.KVBatchDesc, BATCH, {}), 8,
                                                   need) == sz.OK
    assert attend(ws_bytes=need.value - 1) == sz.ERR_CAPACITY


def test_keep_arguments_are_checked(splitzip_lib):
    assert keep(count=0) == sz.ERR_INVALID_ARG
    assert keep(count=257) == sz.ERR_UNSUPPORTED
    for kw in (dict(path=None), dict(path=A + 2), dict(kept=None), dict(kept=A + 2)):
        assert keep(**kw) == sz.ERR_INVALID_ARG, kw
    for kw in (dict(pool_pages=8), dict(page_tokens=8), dict(kv_heads=1), dict(head_dim=64), dict(type=sz.KV_FP8_E4M3),
               dict(page_stride=16 * 3 * 128), dict(token_stride=3 * 128), dict(head_stride=256)):
        assert keep(other=kw) == sz.ERR_INVALID_ARG, kw
    # a pool given twice would be moved twice
    for kw in (dict(d_k=A), dict(d_v=A + 4096), dict(d_k=A + 4096), dict(d_v=A)):
        assert keep(other=kw) == sz.ERR_INVALID_ARG, kw
    assert keep(count=1, cache=dict(d_v=A)) == sz.ERR_INVALID_ARG


def test_frequencies():
    f = sz.rotary_frequencies(64, 10000.0)
    assert f.shape == (32,) and f[0] == 1.0
    assert torch.allclose(f, torch.tensor([10000.0 ** (-2 * j / 64) for j in range(32)], dtype=torch.float64), rtol=1e-15)
    assert torch.allclose(sz.rotary_frequencies(64, 10000.0, factor=4.0), f / 4, rtol=1e-15)
    g = sz.rotary_frequencies(64, 10000.0, factor=4.0, original_len=8192, turns=(1.0, 32.0))
    made = 8192 * f / (2 * math.pi)
    assert bool((g[made >= 32] == f[made >= 32]).all())
    assert torch.allclose(g[made <= 1], f[made <= 1] / 4, rtol=1e-15)
    between = (made > 1) & (made < 32)
    part = (made[between] - 1) / 31
    assert between.any() and torch.allclose(g[between], f[between] * (part + (1 - part) / 4), rtol=1e-12)


def test_turns_are_the_frequencies_modulo_a_turn():
    """Off by half of 2^-64 of a turn, and by the rounding of the quotient in doubles."""
    f = torch.tensor([1.0, 0.1, 1e-9, 0.0, 6.5, 100.0, -2.5, 3.141592653589793], dtype=torch.float64)
    r = sz.KVRotary(f, device="cpu")
    assert r.rotary_dim == 16
    two_pi = Fraction("6.28318530717958647692528676655900576839433879875021")
    for x, t in zip(f.tolist(), r.turns.tolist()):
        exact = Fraction(x) / two_pi
        off = (Fraction(t % (1 << 64), 1 << 64) - exact) % 1
        off = min(off, 1 - off)
        assert off <= abs(exact) * Fraction(1, 1 << 51) + Fraction(1, 1 << 65), x


def test_bad_frequencies_are_refused():
    for f in (torch.ones(0), torch.ones(7), torch.ones(4, 2), torch.tensor([math.nan] * 8), torch.tensor([math.inf] * 8)):
        with pytest.raises(ValueError):
            sz.KVRotary(f, device="cpu")


def test_helpers_refuse_tensors_off_the_device(splitzip_lib):
    ints = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        sz.KVPages(ints(4), ints(1), ints(2, 3), ints(2), ints(2), 16)
    with pytest.raises(ValueError):
        sz._int32(ints(4), (4,), "kept", 0)
    with pytest.raises(ValueError):
        sz.KVLayers([])
    with pytest.raises(ValueError):
        sz.KVTree(None, window=-1)
    with pytest.raises(ValueError):
        sz.KVTree(None, window=1 << 32)


def size_of(heads=32, **kw):
    need = ctypes.c_uint64(0)
    cache = desc(sz.KVCacheDesc, CACHE, dict(kv_heads=kw.pop("kv_heads", 8), token_stride=8 * 128,
                                             page_stride=16 * 8 * 128))
    batch = desc(sz.KVBatchDesc, BATCH, dict(table_stride=1 << 20, **kw))
    assert sz.splitzip_kv_attention_workspace_size(cache, batch, heads, need) == sz.OK
    return need.value


def test_workspace_of_steps_of_few_rows_is_the_step_kernels(splitzip_lib):
    """Two parts of 16 rows for each of 608 blocks and their counters, up to 32 rows of a sequence."""
    step = 2560 + 608 * 2 * 16 * (128 + 2) * 4
    for t in (1, 4, 5, 8):
        assert size_of(batch=64, tokens=64 * t, max_tokens=t, max_kv_len=2000) == step, t
    assert size_of(batch=64, tokens=64 * 9, max_tokens=9, max_kv_len=2000) > step


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU error path")
def test_trees_do_with_that_workspace(splitzip_lib):
    """Whatever the sizes: the call is not refused for want of it, and is with a byte less."""
    for kv_heads, group in ((1, 1), (1, 17), (2, 4), (8, 4), (3, 16)):
        for t in (1, 3, 5, 8, 17, 32, 33, 100):
            for n in (1, 2, 7, 64, 400):
                for kv in (1, 65, 500, 1171, 8193, 100000):
                    step = dict(batch=n, max_tokens=t, max_kv_len=kv)
                    for tokens in {t, t * n}:
                        heads = kv_heads * group
                        need = size_of(heads, kv_heads=kv_heads, tokens=tokens, **step)
                        rows = dict(token_stride=heads * 128)
                        kw = dict(batch=dict(table_stride=1 << 20, tokens=tokens, **step), q_heads=heads, q=rows, out=rows,
                                  tree=dict(words=-(-t // 32)),
                                  cache=dict(kv_heads=kv_heads, token_stride=8 * 128, page_stride=16 * 8 * 128))
                        assert attend(ws_bytes=need, **kw) in (sz.ERR_CUDA, sz.ERR_UNSUPPORTED)
                        assert attend(ws_bytes=need - 1, **kw) == sz.ERR_CAPACITY
