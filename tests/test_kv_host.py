"""Paged-cache operators, what needs no GPU: refusals of bad arguments before
any GPU work, and workspace sizes."""
import ctypes
import math
import types

import pytest
import torch

import lossless_kv_cache_gb300 as sz

A = 1 << 20  # a 16-byte aligned address that no refused call looks at

CACHE = dict(d_k=A, d_v=A, d_k_scale=A, d_v_scale=A, pool_pages=9, page_stride=16 * 2 * 128, token_stride=2 * 128,
             head_stride=128, page_tokens=16, kv_heads=2, head_dim=128, type=sz.KV_FP8_E5M2)
BATCH = dict(d_cu_tokens=A, d_kv_len=A, d_page_table=A, table_stride=4, batch=3, tokens=10, max_tokens=5, max_kv_len=64)
ROWS = dict(d=A, token_stride=256, head_stride=128)


def desc(cls, base, kw):
    d = dict(base, **kw)
    c = cls()
    for name, value in d.items():
        setattr(c, name, value)
    return c


def rw(fn, cache=None, batch=None, k=None, v=None, dtype=sz.BF16, status=A):
    return fn(desc(sz.KVCacheDesc, CACHE, cache or {}), desc(sz.KVBatchDesc, BATCH, batch or {}),
              desc(sz.KVRowsDesc, ROWS, k or {}), desc(sz.KVRowsDesc, ROWS, v or {}), dtype, status, 0)


def attend(cache=None, batch=None, q=None, out=None, lse=A, dtype=sz.BF16, q_heads=8, scale=0.1, causal=1, window=0,
           ws=A, ws_bytes=1 << 40, status=A):
    rows = dict(ROWS, token_stride=8 * 128)
    return sz.splitzip_kv_attention(desc(sz.KVCacheDesc, CACHE, cache or {}), desc(sz.KVBatchDesc, BATCH, batch or {}),
                                    desc(sz.KVRowsDesc, rows, q or {}), desc(sz.KVRowsDesc, rows, out or {}), lse,
                                    dtype, q_heads, scale, causal, window, ws, ws_bytes, status, 0)


write = lambda **kw: rw(sz.splitzip_kv_write, **kw)  # noqa: E731
read = lambda **kw: rw(sz.splitzip_kv_read, **kw)  # noqa: E731

INVALID_CACHE = [dict(d_k=None), dict(d_v=None), dict(d_k=A + 8), dict(d_v=A + 4), dict(d_k_scale=None),
                 dict(d_v_scale=None), dict(pool_pages=0), dict(page_tokens=0), dict(page_tokens=24),
                 dict(page_tokens=1 << 17), dict(kv_heads=0), dict(kv_heads=2000), dict(type=4), dict(type=-1),
                 dict(page_stride=4096 + 8), dict(token_stride=264), dict(head_stride=120)]
UNSUPPORTED_CACHE = [dict(head_dim=96), dict(head_dim=256), dict(head_dim=0), dict(pool_pages=1 << 33),
                     dict(page_stride=1 << 48)]
INVALID_BATCH = [dict(d_cu_tokens=None), dict(d_kv_len=None), dict(d_page_table=None), dict(d_kv_len=A + 2),
                 dict(batch=0), dict(max_tokens=11), dict(table_stride=3), dict(max_kv_len=65)]
UNSUPPORTED_BATCH = [dict(batch=70000), dict(tokens=1 << 30), dict(max_kv_len=1 << 30, table_stride=1 << 30)]


@pytest.mark.parametrize("call", [write, read, attend])
def test_bad_caches_and_steps_are_refused(splitzip_lib, call):
    for kw in INVALID_CACHE:
        assert call(cache=kw) == sz.ERR_INVALID_ARG, kw
    for kw in UNSUPPORTED_CACHE:
        assert call(cache=kw) == sz.ERR_UNSUPPORTED, kw
    for kw in INVALID_BATCH:
        assert call(batch=kw) == sz.ERR_INVALID_ARG, kw
    for kw in UNSUPPORTED_BATCH:
        assert call(batch=kw) == sz.ERR_UNSUPPORTED, kw
    assert call(status=None) == sz.ERR_INVALID_ARG
    assert call(status=A + 2) == sz.ERR_INVALID_ARG


@pytest.mark.parametrize("call", [write, read, attend])
def test_types_that_do_not_go_together_are_refused(splitzip_lib, call):
    bf16, fp16 = dict(type=sz.KV_BF16), dict(type=sz.KV_FP16)
    assert call(dtype=sz.FP8_E5M2) == sz.ERR_INVALID_ARG
    assert call(dtype=3) == sz.ERR_INVALID_ARG
    assert call(cache=bf16, dtype=sz.FP16) == sz.ERR_INVALID_ARG
    assert call(cache=fp16, dtype=sz.BF16) == sz.ERR_INVALID_ARG


@pytest.mark.parametrize("call,names", [(write, "kv"), (read, "kv"), (attend, ("q", "out"))])
def test_bad_rows_are_refused(splitzip_lib, call, names):
    for name in names:
        for kw in (dict(d=None), dict(d=A + 8), dict(token_stride=1028), dict(head_stride=132), dict(head_stride=64),
                   dict(token_stride=64)):
            assert call(**{name: kw}) == sz.ERR_INVALID_ARG, (name, kw)


def test_attention_arguments_are_checked(splitzip_lib):
    assert attend(q_heads=0) == sz.ERR_INVALID_ARG
    assert attend(q_heads=7) == sz.ERR_INVALID_ARG           # no multiple of 2 kv heads
    assert attend(q_heads=2 * 65) == sz.ERR_UNSUPPORTED
    for scale in (math.nan, math.inf, -math.inf):
        assert attend(scale=scale) == sz.ERR_INVALID_ARG
    assert attend(lse=A + 2) == sz.ERR_INVALID_ARG
    assert attend(ws=None) == sz.ERR_INVALID_ARG
    assert attend(ws=A + 8) == sz.ERR_INVALID_ARG
    need = ctypes.c_uint64(0)
    assert sz.splitzip_kv_attention_workspace_size(desc(sz.KVCacheDesc, CACHE, {}), desc(sz.KVBatchDesc, BATCH, {}), 8,
                                                   need) == sz.OK
    assert need.value > 0
    assert attend(ws_bytes=need.value - 1) == sz.ERR_CAPACITY


def test_workspace_size_needs_no_pointers_and_covers_smaller_steps(splitzip_lib):
    """The size asked for the largest step is enough for any smaller one (a captured graph, a last batch)."""
    none = dict(d_k=None, d_v=None, d_k_scale=None, d_v_scale=None)
    cache = desc(sz.KVCacheDesc, CACHE, none)

    def size(**kw):
        out = ctypes.c_uint64(0)
        b = desc(sz.KVBatchDesc, BATCH, dict(d_cu_tokens=None, d_kv_len=None, d_page_table=None, table_stride=1 << 20,
                                             **kw))
        assert sz.splitzip_kv_attention_workspace_size(cache, b, 8, out) == sz.OK
        return out.value

    for big in (dict(batch=64, tokens=64, max_tokens=1), dict(batch=8, tokens=9000, max_tokens=5000),
                dict(batch=1, tokens=2048, max_tokens=2048), dict(batch=300, tokens=1000, max_tokens=40)):
        most = size(max_kv_len=100000, **big)
        for t in (1, 2, 3, 7, 16, 17, 33, 100, 511, 5000):
            for n in (1, 2, 50, 300):
                for kv in (0, 1, 64, 1000, 100000):
                    small = dict(batch=min(n, big["batch"]), max_tokens=min(t, big["max_tokens"]),
                                 tokens=max(min(t * n, big["tokens"]), min(t, big["max_tokens"])))
                    assert size(max_kv_len=kv, **small) <= most


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU error path")
def test_valid_calls_without_gpu_report_a_cuda_error(splitzip_lib):
    for call in (write, read, attend):
        assert call() in (sz.ERR_CUDA, sz.ERR_UNSUPPORTED)


def test_helpers_refuse_wrong_tensors(splitzip_lib):
    cpu = torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sz.KVCache(cpu, cpu)                                  # not on a GPU
    with pytest.raises(TypeError):
        sz.KVCache(cpu.float(), cpu.float())                  # no cache type
    with pytest.raises(ValueError):
        sz.KVCache(cpu[0], cpu[0])                            # no pages
    i32 = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        sz.KVBatch(i32, i32[:2], i32[None, :2], 1, 1, 1)      # not on a GPU


def test_workspace_covers_steps_of_fewer_new_tokens_with_rows_to_spare(splitzip_lib):
    """The same packed rows, but fewer new tokens of a sequence at most: such a step takes the
    kernel for few rows, whatever the kernel of the larger one."""
    cache = desc(sz.KVCacheDesc, CACHE, dict(kv_heads=1, token_stride=128, page_stride=16 * 128))

    def size(heads, **kw):
        out = ctypes.c_uint64(0)
        b = desc(sz.KVBatchDesc, BATCH, dict(table_stride=1 << 20, **kw))
        assert sz.splitzip_kv_attention_workspace_size(cache, b, heads, out) == sz.OK
        return out.value

    for heads in (1, 4, 8, 33):
        for tokens in (2, 33, 121, 500, 4000):
            for batch in (1, 7, 64):
                for kv in (0, 1, 490, 20000, 1 << 20):
                    sizes = dict(tokens=tokens, batch=batch, max_kv_len=kv)
                    most = size(heads, max_tokens=tokens, **sizes)
                    for t in (0, 1, 2, 3, 8, 9, 32, 33):
                        assert size(heads, max_tokens=min(t, tokens), **sizes) <= most, (heads, sizes, t)


def test_helpers_take_no_status_word_or_rows_off_the_device(splitzip_lib):
    """A CPU tensor's address, or another device's, is never handed to a kernel."""
    good = dict(status=torch.zeros(4, dtype=torch.int32), rows=torch.zeros(5, 2, 128, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        sz._kv_status(good["status"], 0)
    with pytest.raises(ValueError):
        sz._kv_rows(good["rows"], 5, 2, 128, 0, "k")
    with pytest.raises(ValueError):
        sz._device_tensor(torch.zeros(5, 8), torch.float32, (5, 8), "lse", 0)


class OnDevice:
    """What the helpers look at of a tensor, on a device that is not there."""
    is_cuda = True

    def __init__(self, t, index):
        self.t, self.index, self.device = t, index, "cuda:%d" % index

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_helpers_refuse_tensors_of_several_devices(splitzip_lib, monkeypatch):
    def on(index, *shape, dtype=torch.int32):
        return OnDevice(torch.zeros(*shape, dtype=dtype), index)

    def cache(k, v, *scales, dtype=torch.float8_e5m2):
        return sz.KVCache(on(k, 4, 16, 2, 128, dtype=dtype), on(v, 4, 16, 2, 128, dtype=dtype),
                          *(on(i, 4, 2, 16, dtype=torch.uint8) for i in scales))

    def batch(cu, n, table):
        return sz.KVBatch(on(cu, 4), on(n, 3), on(table, 3, 2), 5, 5, 32)

    assert cache(1, 1, 1, 1).device == 1 and batch(1, 1, 1).device == 1
    for devices in ((0, 1, 0, 0), (0, 0, 1, 0), (0, 0, 0, 1)):
        with pytest.raises(ValueError):
            cache(*devices)
    for devices in ((1, 0, 0), (0, 1, 0), (0, 0, 1)):
        with pytest.raises(ValueError):
            batch(*devices)
    for c, b in ((0, 1), (1, 0)):
        with pytest.raises(ValueError):
            batch(b, b, b).check(cache(c, c, c, c))
    batch(1, 1, 1).check(cache(1, 1, 1, 1))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 70 + d)
    stream = types.SimpleNamespace(device=torch.device("cuda:0"), cuda_stream=9)
    assert sz._kv_stream(None, 0) == 70 and sz._kv_stream(stream, 0) == 9
    stream.device = torch.device("cuda:1")
    for s, device in ((None, 1), (stream, 0), (stream, 1)):  # not the current device, not the tensors'
        with pytest.raises(ValueError):
            sz._kv_stream(s, device)
    assert sz._kv_status(on(1, 4), 1) > 0
    for bad in (on(0, 4), on(1, 4, dtype=torch.int64), on(1, 0)):
        with pytest.raises(ValueError):
            sz._kv_status(bad, 1)


@pytest.mark.parametrize("window", [-1, -5000, 1 << 32, (1 << 32) + 5])
def test_windows_that_are_no_unsigned_32_bit_number_are_refused(splitzip_lib, window):
    with pytest.raises(ValueError, match="window"):
        sz.kv_attention(None, None, None, None, None, 0.1, window=window)


@pytest.mark.parametrize("call", [write, read, attend])
def test_pools_past_the_address_space_are_refused(splitzip_lib, call):
    """Pages by stride is looked at without wrapping past 64 bits."""
    for pages, stride in ((1 << 24, 1 << 40), (1 << 30, 1 << 34), ((1 << 31) - 1, 1 << 40), (3 << 24, 1 << 40)):
        assert call(cache=dict(pool_pages=pages, page_stride=stride)) == sz.ERR_UNSUPPORTED, (pages, stride)


def test_rows_past_31_bits_are_refused(splitzip_lib):
    """Rows of a sequence (new tokens by query heads of a group) are counted in 31 bits."""
    q = dict(token_stride=128 * 128)
    for tokens in (1 << 25, (1 << 25) + 1, 1 << 26, (1 << 30) - 1):
        assert attend(batch=dict(tokens=tokens, max_tokens=tokens), q=q, out=q, q_heads=2 * 64) == sz.ERR_UNSUPPORTED
        out = ctypes.c_uint64(0)
        b = desc(sz.KVBatchDesc, BATCH, dict(tokens=tokens, max_tokens=tokens))
        assert sz.splitzip_kv_attention_workspace_size(desc(sz.KVCacheDesc, CACHE, {}), b, 2 * 64, out) == sz.ERR_UNSUPPORTED
        b = desc(sz.KVBatchDesc, BATCH, dict(tokens=tokens, max_tokens=(1 << 25) - 8))
        assert sz.splitzip_kv_attention_workspace_size(desc(sz.KVCacheDesc, CACHE, {}), b, 2 * 64, out) == sz.OK


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU error path")
@pytest.mark.parametrize("call", [write, read, attend])
def test_a_step_that_holds_nothing_needs_no_page_table(splitzip_lib, call):
    assert call(batch=dict(max_kv_len=0, table_stride=0, d_page_table=None)) in (sz.ERR_CUDA, sz.ERR_UNSUPPORTED)
    assert call(batch=dict(max_kv_len=1, table_stride=1, d_page_table=None)) == sz.ERR_INVALID_ARG
    assert call(batch=dict(max_kv_len=0, table_stride=0, d_page_table=A + 2)) == sz.ERR_INVALID_ARG
