"""SplitZip lossless KV-cache codec for GB300 (sm_103a).

Thin ctypes binding of the C ABI in include/splitzip.h: the ``splitzip_*``
functions below take the same arguments as the C entry points (device
pointers as Python ints, a CUDA stream handle as an int) and return the same
status codes.  Every step of the codec runs in the CUDA kernels of
``libsplitzip.so``; this module only marshals arguments.  The torch helpers at
the end (``calibrate``, ``encode``, ``decode``) allocate device memory with
torch and call the same entry points.  ``kv_write``, ``kv_read`` and
``kv_attention`` are the operators over the paged cache that the codec moves;
``kv_extend``, ``kv_rotary_write``, ``kv_tree``, ``kv_tree_attention`` and
``kv_keep`` are the rest of a (speculative) serving step over it.

Method: "SplitZip: Ultra Fast Lossless KV Compression for Disaggregated LLM
Serving", section "Method: SplitZip".
"""
import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsplitzip.so")

BF16 = 0
FP8_E5M2 = 1
FP16 = 2
OK, ERR_INVALID_ARG, ERR_CAPACITY, ERR_CORRUPT, ERR_CUDA, ERR_TIMEOUT, ERR_UNSUPPORTED = range(7)
DEFAULT_CHUNK_ELEMS = 65536
HEADER_BYTES = 64
KV_BF16, KV_FP8_E5M2, KV_FP16, KV_FP8_E4M3 = BF16, FP8_E5M2, FP16, 3  # splitzip_kv_type_t
NOALLOC_SCRATCH_BYTES = 32 << 20  # SPLITZIP_NOALLOC_SCRATCH_BYTES


class SplitZipError(RuntimeError):
    def __init__(self, status, where=""):
        self.status = status
        super().__init__("%s: %s (status %d)" % (where, splitzip_status_string(status), status))


class Codebook(ctypes.Structure):
    """splitzip_codebook_t: code i stands for exponent exps[i]."""
    _fields_ = [("dtype", ctypes.c_uint8), ("exps", ctypes.c_uint8 * 16)]

    def values(self):
        return list(self.exps)

    @classmethod
    def make(cls, dtype, exps):
        cb = cls()
        cb.dtype = dtype
        for i, e in enumerate(exps):
            cb.exps[i] = int(e)
        return cb


class Header(ctypes.Structure):
    """splitzip_header_t."""
    _fields_ = [
        ("n_elems", ctypes.c_uint64),
        ("total_escapes", ctypes.c_uint64),
        ("size", ctypes.c_uint64),
        ("index_off", ctypes.c_uint64),
        ("counts_off", ctypes.c_uint64),
        ("nibble_off", ctypes.c_uint64),
        ("signmant_off", ctypes.c_uint64),
        ("escrec_off", ctypes.c_uint64),
        ("chunk_elems", ctypes.c_uint32),
        ("n_chunks", ctypes.c_uint32),
        ("dtype", ctypes.c_uint8),
        ("codebook", ctypes.c_uint8 * 16),
    ]


class EncodeItem(ctypes.Structure):
    """splitzip_encode_item_t."""
    _fields_ = [("d_in", ctypes.c_void_p), ("n", ctypes.c_uint64), ("d_out", ctypes.c_void_p),
                ("out_capacity", ctypes.c_uint64), ("d_out_size", ctypes.c_void_p)]


class DecodeItem(ctypes.Structure):
    """splitzip_decode_item_t."""
    _fields_ = [("d_in", ctypes.c_void_p), ("in_bytes", ctypes.c_uint64), ("d_out", ctypes.c_void_p),
                ("n", ctypes.c_uint64)]


class KVCacheDesc(ctypes.Structure):
    """splitzip_kv_cache_t."""
    _fields_ = [("d_k", ctypes.c_void_p), ("d_v", ctypes.c_void_p), ("d_k_scale", ctypes.c_void_p),
                ("d_v_scale", ctypes.c_void_p), ("pool_pages", ctypes.c_uint64), ("page_stride", ctypes.c_uint64),
                ("token_stride", ctypes.c_uint64), ("head_stride", ctypes.c_uint64), ("page_tokens", ctypes.c_uint32),
                ("kv_heads", ctypes.c_uint32), ("head_dim", ctypes.c_uint32), ("type", ctypes.c_int32)]


class KVBatchDesc(ctypes.Structure):
    """splitzip_kv_batch_t."""
    _fields_ = [("d_cu_tokens", ctypes.c_void_p), ("d_kv_len", ctypes.c_void_p), ("d_page_table", ctypes.c_void_p),
                ("table_stride", ctypes.c_uint64), ("batch", ctypes.c_uint32), ("tokens", ctypes.c_uint32),
                ("max_tokens", ctypes.c_uint32), ("max_kv_len", ctypes.c_uint32)]


class KVRowsDesc(ctypes.Structure):
    """splitzip_kv_rows_t."""
    _fields_ = [("d", ctypes.c_void_p), ("token_stride", ctypes.c_uint64), ("head_stride", ctypes.c_uint64)]


class KVPagesDesc(ctypes.Structure):
    """splitzip_kv_pages_t."""
    _fields_ = [("d_free", ctypes.c_void_p), ("d_free_count", ctypes.c_void_p), ("d_held", ctypes.c_void_p),
                ("d_kv_len", ctypes.c_void_p), ("d_page_table", ctypes.c_void_p), ("table_stride", ctypes.c_uint64),
                ("table_pages", ctypes.c_uint32), ("pool_pages", ctypes.c_uint32), ("page_tokens", ctypes.c_uint32),
                ("batch", ctypes.c_uint32)]


class KVStepDesc(ctypes.Structure):
    """splitzip_kv_step_t."""
    _fields_ = [("d_free_count", ctypes.c_void_p), ("d_held", ctypes.c_void_p), ("d_kv_len", ctypes.c_void_p),
                ("d_cu_tokens", ctypes.c_void_p), ("d_position", ctypes.c_void_p), ("d_slot", ctypes.c_void_p),
                ("tokens", ctypes.c_uint32), ("max_tokens", ctypes.c_uint32), ("max_kv_len", ctypes.c_uint32)]


class KVRotaryDesc(ctypes.Structure):
    """splitzip_kv_rotary_t."""
    _fields_ = [("d_turns", ctypes.c_void_p), ("d_position", ctypes.c_void_p), ("rotary_dim", ctypes.c_uint32),
                ("interleaved", ctypes.c_int32), ("magnitude", ctypes.c_float)]


class KVTreeDesc(ctypes.Structure):
    """splitzip_kv_tree_t."""
    _fields_ = [("d_mask", ctypes.c_void_p), ("d_position", ctypes.c_void_p), ("words", ctypes.c_uint32),
                ("window", ctypes.c_uint32)]


MAX_BATCH = 256                 # SPLITZIP_MAX_BATCH
MAX_BATCH_ITEM_ELEMS = 1 << 26  # SPLITZIP_MAX_BATCH_ITEM_ELEMS
MAX_TREE_TOKENS = 1024          # SPLITZIP_MAX_TREE_TOKENS
MAX_LAYERS = 256                # SPLITZIP_MAX_LAYERS


class _Address(ctypes.c_void_p):
    """A pointer argument: an integer address, None (NULL), or an object with
    data_ptr() (a torch tensor).  Anything else -- notably a str or bytes, which
    plain c_void_p would turn into the address of its host buffer -- is a
    TypeError, so a wrong value never reaches a kernel as an address."""

    @classmethod
    def from_param(cls, obj):
        if obj is None or isinstance(obj, bool):
            if obj is None:
                return None
            raise TypeError("pointer argument: expected an address, got bool")
        if isinstance(obj, int):
            return ctypes.c_void_p(obj)
        if isinstance(obj, ctypes.c_void_p):
            return obj
        if hasattr(obj, "data_ptr"):
            return ctypes.c_void_p(obj.data_ptr())
        raise TypeError("pointer argument: expected an integer address, None or a tensor, got %s"
                        % type(obj).__name__)


_u64, _u32, _int, _vp = ctypes.c_uint64, ctypes.c_uint32, ctypes.c_int, _Address
_P_u64 = ctypes.POINTER(ctypes.c_uint64)
_P_cache, _P_batch, _P_rows = (ctypes.POINTER(t) for t in (KVCacheDesc, KVBatchDesc, KVRowsDesc))
_P_pages, _P_step, _P_rotary, _P_tree = (ctypes.POINTER(t) for t in (KVPagesDesc, KVStepDesc, KVRotaryDesc, KVTreeDesc))

# name -> (restype, argtypes); mirrors include/splitzip.h
SIGNATURES = {
    "splitzip_status_string": (ctypes.c_char_p, [_int]),
    "splitzip_exponent_histogram": (_int, [_vp, _u64, _int, _vp, _vp]),
    "splitzip_calibrate": (_int, [_vp, _int, _int, ctypes.POINTER(Codebook)]),
    "splitzip_compressed_size": (_int, [_u64, _int, _u32, _u64, _P_u64]),
    "splitzip_max_compressed_size": (_int, [_u64, _int, _u32, _P_u64]),
    "splitzip_encode_workspace_size": (_int, [_u64, _int, _u32, _P_u64]),
    "splitzip_encode": (_int, [_vp, _u64, _int, ctypes.POINTER(Codebook), _u32, _vp, _u64, _vp, _u64, _vp,
                               _vp, _vp]),
    "splitzip_encode_noalloc": (_int, [_vp, _u64, _int, ctypes.POINTER(Codebook), _u32, _vp, _u64, _vp, _vp,
                                       _vp]),
    "splitzip_decode": (_int, [_vp, _u64, _vp, _u64, _int, _vp, _vp]),
    "splitzip_parse_header": (_int, [_vp, _u64, ctypes.POINTER(Header)]),
    "splitzip_calibrate_device": (_int, [_vp, _u64, _int, _vp, _vp, _vp]),
    "splitzip_ablation_max_size": (_int, [_u64, _int, _u32, _int, _P_u64]),
    "splitzip_ablation_encode": (_int, [_vp, _u64, _int, ctypes.POINTER(Codebook), _u32, _int, _vp, _u64, _vp, _vp,
                                        _vp]),
    "splitzip_ablation_decode": (_int, [_vp, _u64, _vp, _u64, _int, _int, _vp, _vp]),
    "splitzip_encode_paged": (_int, [_vp, _u64, _vp, _u64, _u64, _int, ctypes.POINTER(Codebook), _u32, _vp, _u64, _vp,
                                     _u64, _vp, _vp, _vp]),
    "splitzip_decode_paged": (_int, [_vp, _u64, _vp, _u64, _vp, _u64, _u64, _int, _vp, _vp]),
    "splitzip_encode_device_codebook": (_int, [_vp, _u64, _int, _vp, _u32, _vp, _u64, _vp, _u64, _vp, _vp, _vp]),
    "splitzip_transfer_scratch_size": (_int, [_u64, _int, _u32, _u64, _int, _P_u64, _P_u64]),
    "splitzip_transfer": (_int, [_vp, _vp, _u64, _int, ctypes.POINTER(Codebook), _u32, _u64, _int, _vp, _u64, _vp,
                                 _u64, _P_u64, ctypes.POINTER(ctypes.c_float), _vp]),
    "splitzip_selftest_bounded_wait": (_int, [_u64, _vp, _vp, _vp]),
    "splitzip_merge": (_int, [ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(ctypes.c_uint64), _u32, _vp, _u64,
                              _P_u64]),
    "splitzip_encode_batch_workspace_size": (_int, [ctypes.POINTER(ctypes.c_uint64), _u32, _int, _u32, _P_u64]),
    "splitzip_encode_batch": (_int, [ctypes.POINTER(EncodeItem), _u32, _int, ctypes.POINTER(Codebook), _u32, _vp,
                                     _u64, _vp, _vp]),
    "splitzip_decode_batch": (_int, [ctypes.POINTER(DecodeItem), _u32, _int, _vp, _vp]),
    "splitzip_kv_write": (_int, [_P_cache, _P_batch, _P_rows, _P_rows, _int, _vp, _vp]),
    "splitzip_kv_read": (_int, [_P_cache, _P_batch, _P_rows, _P_rows, _int, _vp, _vp]),
    "splitzip_kv_attention_workspace_size": (_int, [_P_cache, _P_batch, _u32, _P_u64]),
    "splitzip_kv_attention": (_int, [_P_cache, _P_batch, _P_rows, _P_rows, _vp, _int, _u32, ctypes.c_float, _int, _u32,
                                     _vp, _u64, _vp, _vp]),
    "splitzip_kv_extend_workspace_size": (_int, [_u32, _P_u64]),
    "splitzip_kv_extend": (_int, [_P_pages, _vp, _vp, _P_step, _vp, _u64, _vp, _vp]),
    "splitzip_kv_rotary_write": (_int, [_P_cache, _P_batch, _P_rotary, _P_rows, _P_rows, _u32, _P_rows, _P_rows, _int,
                                        _vp, _vp]),
    "splitzip_kv_tree": (_int, [_P_batch, _vp, _P_tree, _vp, _vp]),
    "splitzip_kv_tree_attention": (_int, [_P_cache, _P_batch, _P_tree, _P_rows, _P_rows, _vp, _int, _u32, ctypes.c_float,
                                          _vp, _u64, _vp, _vp]),
    "splitzip_kv_keep": (_int, [_P_cache, _u32, _P_batch, _vp, _vp, _vp, _vp]),
}

_lib = None


def lib():
    """The loaded libsplitzip.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libsplitzip.so is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


# ---------------------------------------------------------------- C entry points

def splitzip_status_string(status):
    return lib().splitzip_status_string(status).decode()


def splitzip_exponent_histogram(d_x, n, dtype, d_hist256, stream):
    return lib().splitzip_exponent_histogram(d_x, n, dtype, d_hist256, stream)


def splitzip_calibrate(hist256, hist_is_device, dtype, out_cb):
    return lib().splitzip_calibrate(hist256, hist_is_device, dtype, ctypes.byref(out_cb))


def splitzip_compressed_size(n, dtype, chunk_elems, total_escapes, out_bytes):
    return lib().splitzip_compressed_size(n, dtype, chunk_elems, total_escapes, ctypes.byref(out_bytes))


def splitzip_max_compressed_size(n, dtype, chunk_elems, out_bytes):
    return lib().splitzip_max_compressed_size(n, dtype, chunk_elems, ctypes.byref(out_bytes))


def splitzip_encode_workspace_size(n, dtype, chunk_elems, out_bytes):
    return lib().splitzip_encode_workspace_size(n, dtype, chunk_elems, ctypes.byref(out_bytes))


def splitzip_encode(d_in, n, dtype, cb, chunk_elems, d_out, out_capacity, d_ws, ws_bytes, d_out_size,
                    d_status, stream):
    return lib().splitzip_encode(d_in, n, dtype, ctypes.byref(cb), chunk_elems, d_out, out_capacity, d_ws,
                                 ws_bytes, d_out_size, d_status, stream)


def splitzip_encode_noalloc(d_in, n, dtype, cb, chunk_elems, d_out, out_capacity, d_out_size, d_status, stream):
    return lib().splitzip_encode_noalloc(d_in, n, dtype, ctypes.byref(cb), chunk_elems, d_out, out_capacity,
                                         d_out_size, d_status, stream)


def splitzip_decode(d_in, in_bytes, d_out, n, dtype, d_status, stream):
    return lib().splitzip_decode(d_in, in_bytes, d_out, n, dtype, d_status, stream)


def splitzip_parse_header(h_blob, nbytes, out):
    return lib().splitzip_parse_header(h_blob, nbytes, ctypes.byref(out))


def splitzip_encode_paged(d_pool, pool_pages, d_pages, n_pages, page_elems, dtype, cb, chunk_elems, d_out,
                          out_capacity, d_ws, ws_bytes, d_out_size, d_status, stream):
    return lib().splitzip_encode_paged(d_pool, pool_pages, d_pages, n_pages, page_elems, dtype, ctypes.byref(cb),
                                       chunk_elems, d_out, out_capacity, d_ws, ws_bytes, d_out_size, d_status, stream)


def splitzip_decode_paged(d_in, in_bytes, d_pool, pool_pages, d_pages, n_pages, page_elems, dtype, d_status, stream):
    return lib().splitzip_decode_paged(d_in, in_bytes, d_pool, pool_pages, d_pages, n_pages, page_elems, dtype,
                                       d_status, stream)


def splitzip_ablation_max_size(n, dtype, chunk_elems, variant, out_bytes):
    return lib().splitzip_ablation_max_size(n, dtype, chunk_elems, variant, ctypes.byref(out_bytes))


def splitzip_ablation_encode(d_in, n, dtype, cb, chunk_elems, variant, d_out, out_capacity, d_out_size, d_status,
                             stream):
    return lib().splitzip_ablation_encode(d_in, n, dtype, ctypes.byref(cb), chunk_elems, variant, d_out,
                                          out_capacity, d_out_size, d_status, stream)


def splitzip_ablation_decode(d_in, in_bytes, d_out, n, dtype, variant, d_status, stream):
    return lib().splitzip_ablation_decode(d_in, in_bytes, d_out, n, dtype, variant, d_status, stream)


def splitzip_calibrate_device(d_x, n, dtype, d_hist256, d_cb, stream):
    return lib().splitzip_calibrate_device(d_x, n, dtype, d_hist256, d_cb, stream)


def splitzip_encode_device_codebook(d_in, n, dtype, d_cb, chunk_elems, d_out, out_capacity, d_ws, ws_bytes,
                                    d_out_size, d_status, stream):
    return lib().splitzip_encode_device_codebook(d_in, n, dtype, d_cb, chunk_elems, d_out, out_capacity, d_ws,
                                                 ws_bytes, d_out_size, d_status, stream)


def splitzip_transfer_scratch_size(n, dtype, chunk_elems, piece_elems, compress, out_device_bytes, out_host_bytes):
    return lib().splitzip_transfer_scratch_size(n, dtype, chunk_elems, piece_elems, compress,
                                                ctypes.byref(out_device_bytes), ctypes.byref(out_host_bytes))


def splitzip_transfer(d_src, d_dst, n, dtype, cb, chunk_elems, piece_elems, compress, d_scratch, d_scratch_bytes,
                      h_stage, h_stage_bytes, out_link_bytes, out_ms, stream):
    """out_link_bytes: ctypes.c_uint64 or None; out_ms: ctypes.c_float or None."""
    return lib().splitzip_transfer(d_src, d_dst, n, dtype, None if cb is None else ctypes.byref(cb), chunk_elems,
                                   piece_elems, compress, d_scratch, d_scratch_bytes, h_stage, h_stage_bytes,
                                   None if out_link_bytes is None else ctypes.byref(out_link_bytes),
                                   None if out_ms is None else ctypes.byref(out_ms), stream)


def splitzip_selftest_bounded_wait(limit_cycles, d_status, d_cycles, stream):
    return lib().splitzip_selftest_bounded_wait(limit_cycles, d_status, d_cycles, stream)


def splitzip_merge(h_parts, part_bytes, count, h_out, out_capacity, out_bytes):
    """h_parts: ctypes array of c_void_p; part_bytes: ctypes array of c_uint64."""
    return lib().splitzip_merge(h_parts, part_bytes, count, h_out, out_capacity, ctypes.byref(out_bytes))


def splitzip_encode_batch_workspace_size(h_n, count, dtype, chunk_elems, out_bytes):
    """h_n: ctypes array of c_uint64."""
    return lib().splitzip_encode_batch_workspace_size(h_n, count, dtype, chunk_elems, ctypes.byref(out_bytes))


def splitzip_encode_batch(h_items, count, dtype, cb, chunk_elems, d_ws, ws_bytes, d_status, stream):
    """h_items: ctypes array of EncodeItem."""
    return lib().splitzip_encode_batch(h_items, count, dtype, ctypes.byref(cb), chunk_elems, d_ws, ws_bytes, d_status,
                                       stream)


def splitzip_decode_batch(h_items, count, dtype, d_status, stream):
    """h_items: ctypes array of DecodeItem."""
    return lib().splitzip_decode_batch(h_items, count, dtype, d_status, stream)


def splitzip_kv_write(cache, batch, k, v, dtype, d_status, stream):
    """cache, batch, k, v: KVCacheDesc, KVBatchDesc, KVRowsDesc, KVRowsDesc."""
    return lib().splitzip_kv_write(ctypes.byref(cache), ctypes.byref(batch), ctypes.byref(k), ctypes.byref(v), dtype,
                                   d_status, stream)


def splitzip_kv_read(cache, batch, k, v, dtype, d_status, stream):
    return lib().splitzip_kv_read(ctypes.byref(cache), ctypes.byref(batch), ctypes.byref(k), ctypes.byref(v), dtype,
                                  d_status, stream)


def splitzip_kv_attention_workspace_size(cache, batch, q_heads, out_bytes):
    return lib().splitzip_kv_attention_workspace_size(ctypes.byref(cache), ctypes.byref(batch), q_heads,
                                                      ctypes.byref(out_bytes))


def splitzip_kv_attention(cache, batch, q, out, d_lse, dtype, q_heads, scale, causal, window, d_ws, ws_bytes, d_status,
                          stream):
    return lib().splitzip_kv_attention(ctypes.byref(cache), ctypes.byref(batch), ctypes.byref(q), ctypes.byref(out),
                                       d_lse, dtype, q_heads, scale, causal, window, d_ws, ws_bytes, d_status, stream)


def splitzip_kv_extend_workspace_size(batch, out_bytes):
    return lib().splitzip_kv_extend_workspace_size(batch, ctypes.byref(out_bytes))


def splitzip_kv_extend(pages, d_new, d_drop, step, d_ws, ws_bytes, d_status, stream):
    """pages, step: KVPagesDesc, KVStepDesc."""
    return lib().splitzip_kv_extend(ctypes.byref(pages), d_new, d_drop, ctypes.byref(step), d_ws, ws_bytes, d_status,
                                    stream)


def splitzip_kv_rotary_write(cache, batch, rotary, q, q_out, q_heads, k, v, dtype, d_status, stream):
    """rotary: KVRotaryDesc; q, q_out: KVRowsDesc, or both None."""
    return lib().splitzip_kv_rotary_write(ctypes.byref(cache), ctypes.byref(batch), ctypes.byref(rotary),
                                          None if q is None else ctypes.byref(q),
                                          None if q_out is None else ctypes.byref(q_out), q_heads, ctypes.byref(k),
                                          ctypes.byref(v), dtype, d_status, stream)


def splitzip_kv_tree(batch, d_parent, tree, d_status, stream):
    """tree: KVTreeDesc."""
    return lib().splitzip_kv_tree(ctypes.byref(batch), d_parent, ctypes.byref(tree), d_status, stream)


def splitzip_kv_tree_attention(cache, batch, tree, q, out, d_lse, dtype, q_heads, scale, d_ws, ws_bytes, d_status,
                               stream):
    return lib().splitzip_kv_tree_attention(ctypes.byref(cache), ctypes.byref(batch), ctypes.byref(tree), ctypes.byref(q),
                                            ctypes.byref(out), d_lse, dtype, q_heads, scale, d_ws, ws_bytes, d_status,
                                            stream)


def splitzip_kv_keep(h_caches, count, batch, d_path, d_kept, d_status, stream):
    """h_caches: ctypes array of KVCacheDesc."""
    return lib().splitzip_kv_keep(h_caches, count, ctypes.byref(batch), d_path, d_kept, d_status, stream)


# ------------------------------------------------------------ size helpers

def _size_call(fn, *args):
    out = ctypes.c_uint64(0)
    st = fn(*args, out)
    if st != OK:
        raise SplitZipError(st, fn.__name__)
    return out.value


def max_compressed_size(n, dtype, chunk_elems=DEFAULT_CHUNK_ELEMS):
    return _size_call(splitzip_max_compressed_size, n, dtype, chunk_elems)


def compressed_size(n, dtype, chunk_elems, total_escapes):
    return _size_call(splitzip_compressed_size, n, dtype, chunk_elems, total_escapes)


def workspace_size(n, dtype, chunk_elems=DEFAULT_CHUNK_ELEMS):
    return _size_call(splitzip_encode_workspace_size, n, dtype, chunk_elems)


def merge(parts):
    """Join host containers (numpy uint8 arrays, tensor order) of consecutive
    whole-chunk pieces into the container of the whole tensor (numpy uint8)."""
    import numpy as np
    arrs = [np.ascontiguousarray(p, dtype=np.uint8) for p in parts]
    ptrs = (ctypes.c_void_p * len(arrs))(*[a.ctypes.data for a in arrs])
    sizes = (ctypes.c_uint64 * len(arrs))(*[a.size for a in arrs])
    total = ctypes.c_uint64(0)
    _check(splitzip_merge(ptrs, sizes, len(arrs), None, 0, total), "splitzip_merge")
    out = np.empty(max(total.value, 1), dtype=np.uint8)
    _check(splitzip_merge(ptrs, sizes, len(arrs), out.ctypes.data, out.size, total), "splitzip_merge")
    return out[: total.value]


def parse_header(blob_bytes):
    """Header of a container held in host memory (bytes / numpy / torch CPU)."""
    import numpy as np
    buf = np.ascontiguousarray(np.frombuffer(bytes(blob_bytes), dtype=np.uint8)) \
        if isinstance(blob_bytes, (bytes, bytearray)) else np.ascontiguousarray(blob_bytes).view(np.uint8)
    h = Header()
    st = splitzip_parse_header(buf.ctypes.data, buf.size, h)
    if st != OK:
        raise SplitZipError(st, "splitzip_parse_header")
    return h


# ------------------------------------------------------------ torch helpers

def _torch():
    import torch
    return torch


def _stream_handle(stream):
    if stream is not None:
        return stream.cuda_stream
    # the current stream of the current device, without the Stream object that
    # torch.cuda.current_stream() makes (3 us of a call)
    c = _torch()._C
    return c._cuda_getCurrentRawStream(c._cuda_getDevice())


def _bits_dtype(dtype):
    torch = _torch()
    return torch.uint8 if dtype == FP8_E5M2 else torch.int16


def _check(st, where):
    if st != OK:
        raise SplitZipError(st, where)


def calibrate(x, dtype, stream=None):
    """Exponent histogram of the device tensor ``x`` (raw bits) on the GPU,
    then the Top-16 codebook.  Synchronises."""
    torch = _torch()
    hist = torch.empty(256, dtype=torch.int64, device=x.device)
    _check(splitzip_exponent_histogram(x.data_ptr(), x.numel(), dtype, hist.data_ptr(), _stream_handle(stream)),
           "splitzip_exponent_histogram")
    torch.cuda.current_stream().synchronize() if stream is None else stream.synchronize()
    h = hist.cpu()
    cb = Codebook()
    _check(splitzip_calibrate(h.data_ptr(), 0, dtype, cb), "splitzip_calibrate")
    return cb, h


class EncodeBuffers:
    """Device buffers for one encode of n elements (capacity-sized)."""

    def __init__(self, n, dtype, chunk_elems=DEFAULT_CHUNK_ELEMS, device="cuda"):
        torch = _torch()
        self.n, self.dtype, self.chunk_elems = n, dtype, chunk_elems
        self.capacity = max_compressed_size(n, dtype, chunk_elems)
        self.ws_bytes = workspace_size(n, dtype, chunk_elems)
        self.out = torch.empty(self.capacity, dtype=torch.uint8, device=device)
        self.ws = torch.empty(max(self.ws_bytes, 16), dtype=torch.uint8, device=device)
        self.size = torch.zeros(2, dtype=torch.int64, device=device)   # [0] = container bytes
        self.status = torch.zeros(4, dtype=torch.int32, device=device)  # [0] = status


def encode_into(x, cb, bufs, stream=None):
    """Enqueue the encode of device tensor ``x`` into ``bufs`` (asynchronous)."""
    _check(splitzip_encode(x.data_ptr(), x.numel(), bufs.dtype, cb, bufs.chunk_elems, bufs.out.data_ptr(),
                           bufs.capacity, bufs.ws.data_ptr(), bufs.ws_bytes, bufs.size.data_ptr(),
                           bufs.status.data_ptr(), _stream_handle(stream)), "splitzip_encode")


def encode(x, cb, dtype, chunk_elems=DEFAULT_CHUNK_ELEMS, stream=None):
    """Encode device tensor ``x``; returns the container as a uint8 device
    tensor of its exact size.  Synchronises to read the size."""
    bufs = EncodeBuffers(x.numel(), dtype, chunk_elems, device=x.device)
    encode_into(x, cb, bufs, stream)
    size, status = int(bufs.size[0].item()), int(bufs.status[0].item())
    _check(status, "splitzip_encode (device)")
    return bufs.out[:size]


def decode_into(blob, in_bytes, out, n, dtype, status, stream=None):
    _check(splitzip_decode(blob.data_ptr(), in_bytes, out.data_ptr() if n else 0, n, dtype, status.data_ptr(),
                           _stream_handle(stream)), "splitzip_decode")


def decode(blob, n, dtype, stream=None):
    """Decode a device container into a new device tensor of raw bits."""
    torch = _torch()
    out = torch.empty(max(n, 1), dtype=_bits_dtype(dtype), device=blob.device)
    status = torch.zeros(4, dtype=torch.int32, device=blob.device)
    decode_into(blob, blob.numel(), out, n, dtype, status, stream)
    _check(int(status[0].item()), "splitzip_decode (device)")
    return out[:n]


def batch_workspace_size(ns, dtype, chunk_elems=DEFAULT_CHUNK_ELEMS):
    arr = (ctypes.c_uint64 * len(ns))(*ns)
    out = ctypes.c_uint64(0)
    _check(splitzip_encode_batch_workspace_size(arr, len(ns), dtype, chunk_elems, out),
           "splitzip_encode_batch_workspace_size")
    return out.value


def encode_batch(xs, cb, dtype, chunk_elems=DEFAULT_CHUNK_ELEMS, stream=None):
    """Encode each device tensor of ``xs`` into its own container with one
    batched call; returns the containers (uint8 device tensors of their exact
    sizes).  Synchronises to read the sizes."""
    torch = _torch()
    dev = xs[0].device
    caps = [max_compressed_size(x.numel(), dtype, chunk_elems) for x in xs]
    outs = [torch.empty(c, dtype=torch.uint8, device=dev) for c in caps]
    sizes = torch.zeros(len(xs), dtype=torch.int64, device=dev)
    status = torch.zeros(4, dtype=torch.int32, device=dev)
    ws_bytes = batch_workspace_size([x.numel() for x in xs], dtype, chunk_elems)
    ws = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=dev)
    items = (EncodeItem * len(xs))()
    for i, (x, o, c) in enumerate(zip(xs, outs, caps)):
        items[i] = EncodeItem(x.data_ptr() if x.numel() else 0, x.numel(), o.data_ptr(), c,
                              sizes.data_ptr() + 8 * i)
    _check(splitzip_encode_batch(items, len(xs), dtype, cb, chunk_elems, ws.data_ptr(), ws_bytes, status.data_ptr(),
                                 _stream_handle(stream)), "splitzip_encode_batch")
    _check(int(status[0].item()), "splitzip_encode_batch (device)")
    return [o[: int(n)] for o, n in zip(outs, sizes.cpu().tolist())]


def decode_batch_status(blobs, ns, dtype, stream=None):
    """Decode device containers ``blobs`` (element counts ``ns``) with one
    batched call; returns (device status, decoded tensors)."""
    torch = _torch()
    dev = blobs[0].device
    outs = [torch.empty(max(n, 1), dtype=_bits_dtype(dtype), device=dev) for n in ns]
    status = torch.full((4,), -1, dtype=torch.int32, device=dev)
    items = (DecodeItem * len(blobs))()
    for i, (b, o, n) in enumerate(zip(blobs, outs, ns)):
        items[i] = DecodeItem(b.data_ptr(), b.numel(), o.data_ptr() if n else 0, n)
    _check(splitzip_decode_batch(items, len(blobs), dtype, status.data_ptr(), _stream_handle(stream)),
           "splitzip_decode_batch")
    return int(status[0].item()), [o[:n] for o, n in zip(outs, ns)]


def transfer_scratch_size(n, dtype, piece_elems, compress=True, chunk_elems=DEFAULT_CHUNK_ELEMS):
    """(device bytes, pinned host bytes) that splitzip_transfer needs."""
    d, h = ctypes.c_uint64(0), ctypes.c_uint64(0)
    _check(splitzip_transfer_scratch_size(n, dtype, chunk_elems, piece_elems, int(compress), d, h),
           "splitzip_transfer_scratch_size")
    return d.value, h.value


class TransferBuffers:
    """Device scratch and pinned host staging for splitzip_transfer."""

    def __init__(self, n, dtype, piece_elems, compress=True, chunk_elems=DEFAULT_CHUNK_ELEMS, device="cuda"):
        torch = _torch()
        self.n, self.dtype, self.piece_elems = n, dtype, piece_elems
        self.compress, self.chunk_elems = bool(compress), chunk_elems
        d, h = transfer_scratch_size(n, dtype, piece_elems, compress, chunk_elems)
        self.device = torch.empty(max(d, 16), dtype=torch.uint8, device=device)
        self.host = torch.empty(max(h, 16), dtype=torch.uint8, pin_memory=True)


def transfer(src, dst, cb, bufs, stream=None):
    """Move device tensor src into dst across the GPU <-> host link (see
    splitzip_transfer); returns (GPU milliseconds, bytes over the link each way)."""
    link, ms = ctypes.c_uint64(0), ctypes.c_float(0.0)
    _check(splitzip_transfer(src.data_ptr(), dst.data_ptr(), bufs.n, bufs.dtype, cb if bufs.compress else None,
                             bufs.chunk_elems, bufs.piece_elems, int(bufs.compress), bufs.device.data_ptr(),
                             bufs.device.numel(), bufs.host.data_ptr(), bufs.host.numel(), link, ms,
                             _stream_handle(stream)), "splitzip_transfer")
    return ms.value, link.value


def calibrate_device(x, dtype, hist=None, cb=None, stream=None):
    """Online calibration on the device (no host synchronisation): returns
    (histogram, codebook) as device tensors (256 int64; 17 uint8 laid out as
    splitzip_codebook_t: dtype, then the 16 exponents)."""
    torch = _torch()
    hist = torch.empty(256, dtype=torch.int64, device=x.device) if hist is None else hist
    cb = torch.empty(32, dtype=torch.uint8, device=x.device) if cb is None else cb
    _check(splitzip_calibrate_device(x.data_ptr(), x.numel(), dtype, hist.data_ptr(), cb.data_ptr(),
                                     _stream_handle(stream)), "splitzip_calibrate_device")
    return hist, cb


def encode_into_device_codebook(x, d_cb, bufs, stream=None):
    """encode_into with the codebook in device memory (see calibrate_device)."""
    _check(splitzip_encode_device_codebook(x.data_ptr(), x.numel(), bufs.dtype, d_cb.data_ptr(), bufs.chunk_elems,
                                           bufs.out.data_ptr(), bufs.capacity, bufs.ws.data_ptr(), bufs.ws_bytes,
                                           bufs.size.data_ptr(), bufs.status.data_ptr(), _stream_handle(stream)),
           "splitzip_encode_device_codebook")


def encode_paged_into(pool, pages, page_elems, cb, bufs, stream=None):
    """Encode the pages `pages` (device int32 tensor) of `pool` (a device tensor
    of whole pages, raw bits) into `bufs` (sized for len(pages) * page_elems)."""
    _check(splitzip_encode_paged(pool.data_ptr(), pool.numel() // page_elems, pages.data_ptr(), pages.numel(),
                                 page_elems, bufs.dtype, cb, bufs.chunk_elems, bufs.out.data_ptr(), bufs.capacity,
                                 bufs.ws.data_ptr(), bufs.ws_bytes, bufs.size.data_ptr(), bufs.status.data_ptr(),
                                 _stream_handle(stream)), "splitzip_encode_paged")


def decode_paged_into(blob, in_bytes, pool, pages, page_elems, dtype, status, stream=None):
    """Decode a container into the pages `pages` of `pool`."""
    _check(splitzip_decode_paged(blob.data_ptr(), in_bytes, pool.data_ptr(), pool.numel() // page_elems,
                                 pages.data_ptr(), pages.numel(), page_elems, dtype, status.data_ptr(),
                                 _stream_handle(stream)), "splitzip_decode_paged")


# ablation formats (see splitzip_ablation_encode): 0 = Top-16, 1 = Top-8, 2 = Top-15 + sentinel
ABL_TOP16, ABL_TOP8, ABL_TOP15_SENTINEL = 0, 1, 2
ABL_CODES = {ABL_TOP16: 16, ABL_TOP8: 8, ABL_TOP15_SENTINEL: 15}


def ablation_codebook(cb16, variant):
    """The variant's codebook: the first k exponents of a Top-16 codebook, then zeros."""
    k = ABL_CODES[variant]
    vals = list(cb16.values())[:k]
    c = Codebook()
    c.dtype = cb16.dtype
    for i in range(16):
        c.exps[i] = vals[i] if i < k else 0
    return c


def ablation_max_size(n, dtype, variant, chunk_elems=DEFAULT_CHUNK_ELEMS):
    return _size_call(splitzip_ablation_max_size, n, dtype, chunk_elems, variant)


def ablation_encode(x, cb, dtype, variant, chunk_elems=DEFAULT_CHUNK_ELEMS, stream=None):
    """Encode device tensor x in an ablation format; returns the container
    (uint8 device tensor of its exact size).  Synchronises."""
    torch = _torch()
    cap = ablation_max_size(x.numel(), dtype, variant, chunk_elems)
    out = torch.empty(max(cap, 16), dtype=torch.uint8, device=x.device)
    size = torch.zeros(2, dtype=torch.int64, device=x.device)
    status = torch.zeros(4, dtype=torch.int32, device=x.device)
    _check(splitzip_ablation_encode(x.data_ptr(), x.numel(), dtype, cb, chunk_elems, variant, out.data_ptr(), cap,
                                    size.data_ptr(), status.data_ptr(), _stream_handle(stream)),
           "splitzip_ablation_encode")
    _check(int(status[0].item()), "splitzip_ablation_encode (device)")
    return out[: int(size[0].item())]


def ablation_decode_status(blob, n, dtype, variant, stream=None):
    torch = _torch()
    out = torch.empty(max(n, 1), dtype=_bits_dtype(dtype), device=blob.device)
    status = torch.full((4,), -1, dtype=torch.int32, device=blob.device)
    _check(splitzip_ablation_decode(blob.data_ptr(), blob.numel(), out.data_ptr() if n else 0, n, dtype, variant,
                                    status.data_ptr(), _stream_handle(stream)), "splitzip_ablation_decode")
    return int(status[0].item()), out[:n]


# paged-cache operators (see splitzip_kv_write, splitzip_kv_read, splitzip_kv_attention)

def _kv_type_of(t):
    torch = _torch()
    types = {torch.bfloat16: KV_BF16, torch.float16: KV_FP16, torch.float8_e5m2: KV_FP8_E5M2,
             torch.float8_e4m3fn: KV_FP8_E4M3}
    if t.dtype not in types:
        raise TypeError("cache element type: expected bfloat16, float16, float8_e5m2 or float8_e4m3fn, got %s" % t.dtype)
    return types[t.dtype]


def _device_tensor(t, dtype, shape, what, device=None):
    """device: the index of the device that t has to be on (None: any)."""
    if not t.is_cuda or t.dtype != dtype or t.shape != tuple(shape):
        raise ValueError("%s: expected a CUDA tensor of %s and shape %s, got %s %s on %s"
                         % (what, dtype, tuple(shape), t.dtype, tuple(t.shape), t.device))
    if device is not None and t.get_device() != device:
        raise ValueError("%s: expected a tensor on cuda:%d, got one on %s" % (what, device, t.device))
    return t


class KVCache:
    """One layer's paged cache: pools k and v of shape (pages, page_tokens,
    kv_heads, head_dim), any strides with a contiguous last axis (a
    permuted view of [page][head][token][dim] will do), bfloat16, float16,
    float8_e5m2 or float8_e4m3fn.  FP8 caches take k_scale and v_scale, uint8
    (pages, kv_heads, page_tokens).  The codec takes an E5M2 cache's pools as
    raw bits: k.view(torch.uint8)."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        torch = _torch()
        self.type = _kv_type_of(k)
        fp8 = self.type in (KV_FP8_E5M2, KV_FP8_E4M3)
        if k.dim() != 4:
            raise ValueError("k: expected (pages, page_tokens, kv_heads, head_dim), got %s" % (tuple(k.shape),))
        pages, page_tokens, heads, dim = k.shape
        _device_tensor(k, k.dtype, k.shape, "k")
        self.device = k.get_device()
        _device_tensor(v, k.dtype, k.shape, "v", self.device)
        if k.stride() != v.stride() or k.stride(3) != 1:
            raise ValueError("k and v: expected the same strides and a contiguous last axis, got %s and %s"
                             % (k.stride(), v.stride()))
        if fp8:
            for s, what in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                if s is None or not s.is_contiguous():
                    raise ValueError("%s: an FP8 cache needs a contiguous scale tensor" % what)
                _device_tensor(s, torch.uint8, (pages, heads, page_tokens), what, self.device)
        self.k, self.v = k, v
        self.page_tokens, self.kv_heads, self.head_dim = page_tokens, heads, dim
        self.k_scale, self.v_scale = (k_scale, v_scale) if fp8 else (None, None)
        self.desc = KVCacheDesc(k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if fp8 else None,
                                v_scale.data_ptr() if fp8 else None, pages, k.stride(0), k.stride(1), k.stride(2),
                                page_tokens, heads, dim, self.type)

    @classmethod
    def empty(cls, pages, page_tokens, kv_heads, head_dim, dtype, device="cuda"):
        """A cache of zeros; dtype: a torch dtype."""
        torch = _torch()
        fp8 = dtype in (torch.float8_e5m2, torch.float8_e4m3fn)
        raw = torch.uint8 if fp8 else torch.int16
        pools = [torch.zeros(pages, page_tokens, kv_heads, head_dim, dtype=raw, device=device).view(dtype)
                 for _ in range(2)]
        scales = [torch.full((pages, kv_heads, page_tokens), 127, dtype=torch.uint8, device=device)
                  for _ in range(2)] if fp8 else [None, None]
        return cls(*pools, *scales)


class KVBatch:
    """One step of a batch, the same for every layer (splitzip_kv_batch_t):
    int32 device tensors cu_tokens (batch + 1), kv_len (batch) and page_table
    (batch, at least the pages of max_kv_len tokens); the packed tensors' row
    count; the most new tokens and the most tokens of a sequence.  The device
    tensors may be updated in place between steps within those maxima, by which
    alone kernels and workspaces are chosen."""

    def __init__(self, cu_tokens, kv_len, page_table, tokens, max_tokens, max_kv_len):
        torch = _torch()
        batch = kv_len.numel()
        _device_tensor(cu_tokens, torch.int32, (batch + 1,), "cu_tokens")
        self.device = cu_tokens.get_device()
        _device_tensor(kv_len, torch.int32, (batch,), "kv_len", self.device)
        if page_table.dim() != 2 or page_table.stride(1) != 1:
            raise ValueError("page_table: expected (batch, pages) with a contiguous last axis")
        _device_tensor(page_table, torch.int32, (batch, page_table.shape[1]), "page_table", self.device)
        if not (cu_tokens.is_contiguous() and kv_len.is_contiguous()):
            raise ValueError("cu_tokens and kv_len: expected contiguous tensors")
        # a row's entries end where the table does, whatever the stride between rows
        self.table_pages = page_table.shape[1]
        self.cu_tokens, self.kv_len, self.page_table = cu_tokens, kv_len, page_table
        self.tokens, self.max_kv_len = tokens, max_kv_len
        self.pages = None  # the KVPages that the table is of, where known
        self.desc = KVBatchDesc(cu_tokens.data_ptr(), kv_len.data_ptr(), page_table.data_ptr(), page_table.stride(0),
                                batch, tokens, max_tokens, max_kv_len)

    def check(self, cache):
        """Raises where the step is on another device than the cache, where the page table is
        narrower than max_kv_len tokens need, and where it is of pages unlike the cache's."""
        if self.device != cache.device:
            raise ValueError("cache on cuda:%d and step on cuda:%d: expected one device" % (cache.device, self.device))
        if self.table_pages * cache.page_tokens < self.max_kv_len:
            raise SplitZipError(ERR_INVALID_ARG, "page_table of %d pages for %d tokens"
                                % (self.table_pages, self.max_kv_len))
        pages = self.pages
        if pages is not None and (pages.page_tokens != cache.page_tokens or pages.desc.pool_pages > cache.desc.pool_pages):
            raise ValueError("step over a pool of %d pages of %d tokens: expected a cache of as many and such, got %d of %d"
                             % (pages.desc.pool_pages, pages.page_tokens, cache.desc.pool_pages, cache.page_tokens))


_ROW_TYPES = {}


def _kv_stream(stream, device):
    """Handle of a stream of `device`, which has to be the current device."""
    c = _torch()._C
    current = c._cuda_getDevice()
    if current != device or (stream is not None and stream.device.index != device):
        raise ValueError("tensors on cuda:%d: expected it to be the current device (cuda:%d) and the stream's (%s)"
                         % (device, current, "cuda:%d" % current if stream is None else stream.device))
    return c._cuda_getCurrentRawStream(current) if stream is None else stream.cuda_stream


def _kv_rows(t, tokens, heads, dim, device, what):
    """(KVRowsDesc, dtype constant) of a packed (tokens, heads, head_dim) tensor."""
    if not _ROW_TYPES:
        torch = _torch()
        _ROW_TYPES.update({torch.bfloat16: BF16, torch.float16: FP16})
    dtype = _ROW_TYPES.get(t.dtype)
    if dtype is None:
        raise TypeError("%s: expected bfloat16 or float16, got %s" % (what, t.dtype))
    strides = t.stride()
    if t.get_device() != device or t.shape != (tokens, heads, dim) or strides[2] != 1:
        raise ValueError("%s: expected a tensor (%d, %d, %d) on cuda:%d with a contiguous last axis, got %s of strides "
                         "%s on %s" % (what, tokens, heads, dim, device, tuple(t.shape), strides, t.device))
    return KVRowsDesc(t.data_ptr(), strides[0], strides[1]), dtype


def _kv_status(t, device):
    """Address of a status word; the kernels write to it."""
    if t.get_device() != device or t.dtype != _torch().int32 or t.numel() < 1:
        raise ValueError("status: expected an int32 tensor on cuda:%d, got %s %s on %s"
                         % (device, t.dtype, tuple(t.shape), t.device))
    return t.data_ptr()


def _kv_rw(call, cache, batch, k, v, status, stream):
    d, heads, dim, device = cache.desc, cache.kv_heads, cache.head_dim, cache.device
    batch.check(cache)
    rk, dtype = _kv_rows(k, batch.tokens, heads, dim, device, "k")
    rv, dtype_v = _kv_rows(v, batch.tokens, heads, dim, device, "v")
    if dtype != dtype_v:
        raise TypeError("k and v: expected the same type")
    _check(call(d, batch.desc, rk, rv, dtype, _kv_status(status, device), _kv_stream(stream, device)), call.__name__)


def kv_write(cache, batch, k, v, status, stream=None):
    """Enqueue the write of the new tokens' keys and values, packed (tokens,
    kv_heads, head_dim) tensors, into `cache`'s pages (asynchronous; status:
    device int32, as for decode_into)."""
    _kv_rw(splitzip_kv_write, cache, batch, k, v, status, stream)


def kv_read(cache, batch, k, v, status, stream=None):
    """Enqueue the read of every sequence's last tokens from `cache`'s pages into
    the packed tensors k and v (asynchronous)."""
    _kv_rw(splitzip_kv_read, cache, batch, k, v, status, stream)


def kv_attention_workspace_size(cache, batch, q_heads):
    out = ctypes.c_uint64(0)
    _check(splitzip_kv_attention_workspace_size(cache.desc, batch.desc, q_heads, out),
           "splitzip_kv_attention_workspace_size")
    return out.value


class KVAttentionBuffers:
    """Device workspace and status word of kv_attention, for any step of at most
    `batch`'s sizes on caches of `cache`'s geometry."""

    def __init__(self, cache, batch, q_heads):
        torch = _torch()
        device = batch.kv_len.device
        self.q_heads, self.device = q_heads, batch.device
        self.ws_bytes = kv_attention_workspace_size(cache, batch, q_heads)
        self.ws = torch.empty(max(self.ws_bytes, 16), dtype=torch.uint8, device=device)
        self.status = torch.zeros(4, dtype=torch.int32, device=device)  # [0] = status


def kv_attention(cache, batch, q, out, bufs, scale, causal=True, window=0, lse=None, stream=None):
    """Enqueue the attention of the new tokens' queries over `cache`'s pages
    (asynchronous).  q, out: packed (tokens, q_heads, head_dim); lse: None or
    float32 (tokens, q_heads); bufs: KVAttentionBuffers; window: how many positions a
    row sees up to its own, 0: all."""
    if not 0 <= window < 1 << 32:
        raise ValueError("window: expected 0 (none) or a number of positions, got %d" % window)
    batch.check(cache)
    device = cache.device
    if bufs.device != device:
        raise ValueError("bufs: expected buffers on cuda:%d, got cuda:%d" % (device, bufs.device))
    rq, dtype = _kv_rows(q, batch.tokens, bufs.q_heads, cache.head_dim, device, "q")
    ro, dtype_o = _kv_rows(out, batch.tokens, bufs.q_heads, cache.head_dim, device, "out")
    if dtype != dtype_o:
        raise TypeError("q and out: expected the same type")
    if lse is not None:
        if not lse.is_contiguous():
            raise ValueError("lse: expected a contiguous tensor")
        _device_tensor(lse, _torch().float32, (batch.tokens, bufs.q_heads), "lse", device)
        lse = lse.data_ptr()
    _check(splitzip_kv_attention(cache.desc, batch.desc, rq, ro, lse, dtype, bufs.q_heads, scale, int(causal), window,
                                 bufs.ws.data_ptr(), bufs.ws_bytes, bufs.status.data_ptr(), _kv_stream(stream, device)),
           "splitzip_kv_attention")


# a step around the paged cache (see splitzip_kv_extend, splitzip_kv_rotary_write, splitzip_kv_tree,
# splitzip_kv_tree_attention, splitzip_kv_keep)

def _int32(t, shape, what, device):
    """A contiguous int32 tensor of `shape` on cuda:`device`."""
    _device_tensor(t, _torch().int32, shape, what, device)
    if not t.is_contiguous():
        raise ValueError("%s: expected a contiguous tensor" % what)
    return t


class KVPages:
    """The pages of one pool, the same for every layer's cache, and the
    sequences that hold them (splitzip_kv_pages_t): int32 device tensors free
    (one entry for each page of the pool), count (1), table (batch, pages), held
    (batch) and kv_len (batch)."""

    def __init__(self, free, count, table, held, kv_len, page_tokens):
        batch = kv_len.numel()
        if not free.is_cuda:
            raise ValueError("free: expected a CUDA tensor, got one on %s" % free.device)
        self.device = free.get_device()
        _int32(free, (free.numel(),), "free", self.device)
        _int32(count, (1,), "count", self.device)
        if table.dim() != 2 or table.stride(1) != 1:
            raise ValueError("table: expected (batch, pages) with a contiguous last axis")
        if batch > 1 and table.stride(0) < table.shape[1]:
            raise ValueError("table: expected rows that do not overlap")
        _device_tensor(table, _torch().int32, (batch, table.shape[1]), "table", self.device)
        _int32(held, (batch,), "held", self.device)
        _int32(kv_len, (batch,), "kv_len", self.device)
        self.free, self.count, self.table, self.held, self.kv_len = free, count, table, held, kv_len
        self.page_tokens = page_tokens
        self.desc = KVPagesDesc(free.data_ptr(), count.data_ptr(), held.data_ptr(), kv_len.data_ptr(), table.data_ptr(),
                                max(table.stride(0), table.shape[1]), table.shape[1], free.numel(), page_tokens, batch)

    @classmethod
    def empty(cls, pool_pages, page_tokens, batch, max_kv_len, device="cuda"):
        """All pages free, `batch` sequences of no tokens that may grow to max_kv_len."""
        torch = _torch()
        zeros = lambda *s: torch.zeros(*s, dtype=torch.int32, device=device)  # noqa: E731
        return cls(torch.arange(pool_pages - 1, -1, -1, dtype=torch.int32, device=device),
                   torch.full((1,), pool_pages, dtype=torch.int32, device=device),
                   zeros(batch, -(-max_kv_len // page_tokens)), zeros(batch), zeros(batch), page_tokens)

    def ahead(self):
        """The same list and tables with a count, held pages and lengths of their
        own: where kv_extend leaves the next step's while this one's are in use."""
        return KVPages(self.free, self.count.clone(), self.table, self.held.clone(), self.kv_len.clone(),
                       self.page_tokens)


class KVStep:
    """What kv_extend makes for a step of at most `tokens` new tokens, max_tokens
    of one sequence: device tensors cu_tokens (int32, batch + 1), position (int32,
    tokens) and slot (int64, tokens), the status word and the workspace."""

    def __init__(self, batch, tokens, max_tokens, max_kv_len, device="cuda"):
        torch = _torch()
        ints = lambda *s: torch.zeros(*s, dtype=torch.int32, device=device)  # noqa: E731
        self.batch, self.tokens, self.max_tokens, self.max_kv_len = batch, tokens, max_tokens, max_kv_len
        self.cu_tokens, self.position, self.status = ints(batch + 1), ints(tokens), ints(4)
        self.slot = torch.zeros(tokens, dtype=torch.int64, device=device)
        self.ws_bytes = _size_call(splitzip_kv_extend_workspace_size, batch)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=device)
        self.device = self.cu_tokens.get_device()

    def batch_of(self, pages):
        """The KVBatch of this step over `pages`, as kv_extend left them: for caches of pages
        of the same size, and of as many at least."""
        batch = KVBatch(self.cu_tokens, pages.kv_len, pages.table, self.tokens, self.max_tokens, self.max_kv_len)
        batch.pages = pages
        return batch


def kv_extend(pages, new, step, drop=None, after=None, stream=None):
    """Enqueue the page tables and lengths of a step (asynchronous): sequence b
    gives up drop[b] tokens, then takes new[b] more (int32 device tensors).  after:
    KVPages of the same list and tables that receive count, held pages and
    lengths (None: pages itself).  Nothing changes, and cu_tokens is all zeros,
    where step.status says so."""
    device, batch = pages.device, pages.kv_len.numel()
    after = pages if after is None else after
    if step.device != device or after.device != device:
        raise ValueError("pages, step and after: expected one device")
    if step.batch != batch or after.kv_len.numel() != batch or after.free is not pages.free or \
            after.table is not pages.table:
        raise ValueError("step and after: expected those of %d sequences and of the same list and tables" % batch)
    _int32(new, (batch,), "new", device)
    if drop is not None:
        _int32(drop, (batch,), "drop", device)
    to = after.desc
    _check(splitzip_kv_extend(pages.desc, new.data_ptr(), None if drop is None else drop.data_ptr(),
                              KVStepDesc(to.d_free_count, to.d_held, to.d_kv_len, step.cu_tokens.data_ptr(),
                                         step.position.data_ptr(), step.slot.data_ptr(), step.tokens, step.max_tokens,
                                         step.max_kv_len),
                              step.ws.data_ptr(), step.ws_bytes, step.status.data_ptr(), _kv_stream(stream, device)),
           "splitzip_kv_extend")


def rotary_frequencies(rotary_dim, base=10000.0, factor=1.0, original_len=0, turns=(1.0, 32.0)):
    """Radians a position of each pair (float64, rotary_dim / 2): base^(-2j /
    rotary_dim).  factor: how far the context is stretched.  Without original_len
    every pair is slowed by it; with it, pairs that make at most turns[0] turns
    over the original length are, those of turns[1] and more stay as they are, and
    those between are in proportion to their turns: the published interpolation
    "by parts" with (1, 32), and the one of models that state a low and a high
    factor of (1, 4).  Implementations that ramp over the number of the pair,
    between limits rounded to whole pairs, have other frequencies between the two:
    give those to KVRotary as they are."""
    torch = _torch()
    j = torch.arange(0, rotary_dim, 2, dtype=torch.float64)
    f = torch.tensor([float(base) ** (-x / rotary_dim) for x in j.tolist()], dtype=torch.float64)
    stay = torch.zeros_like(f)
    if original_len:
        made = original_len * f / 6.283185307179586
        stay = ((made - turns[0]) / (turns[1] - turns[0])).clamp(0, 1)
    return f * (stay + (1 - stay) / factor)


class KVRotary:
    """Rotary positions (splitzip_kv_rotary_t).  frequencies: radians a position of
    each pair, float64 on the CPU (rotary_frequencies, or any); interleaved: pairs
    of neighbouring elements, else of the two halves of the first 2 *
    len(frequencies) elements; magnitude: a factor on what is rotated."""

    def __init__(self, frequencies, interleaved=False, magnitude=1.0, device="cuda"):
        torch = _torch()
        f = frequencies.detach().to("cpu", torch.float64)
        if f.dim() != 1 or f.numel() == 0 or f.numel() % 8 or not bool(torch.isfinite(f).all()):
            raise ValueError("frequencies: expected finite ones, a multiple of 8 of them")
        # turns a position as a fraction of 2^64, without its whole turns
        turns = [(round(x / 6.283185307179586 * 2.0 ** 64) & (1 << 64) - 1) for x in f.tolist()]
        self.turns = torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns], dtype=torch.int64, device=device)
        self.rotary_dim, self.interleaved, self.magnitude = 2 * f.numel(), bool(interleaved), float(magnitude)
        self.device = self.turns.get_device()
        self.desc = KVRotaryDesc(self.turns.data_ptr(), None, self.rotary_dim, int(self.interleaved), self.magnitude)


def kv_rotary_write(cache, batch, rotary, q, q_out, k, v, status, positions=None, stream=None):
    """Enqueue the rotation of the new tokens' queries q into q_out (packed (tokens,
    q_heads, head_dim); q_out may be q, both may be None) and of their keys k, and
    the write of the rotated keys and of the values v into `cache`'s pages
    (asynchronous; status: device int32, as for kv_write).  positions: int32
    (tokens), None: the tokens' places in the cache."""
    d, heads, dim, device = cache.desc, cache.kv_heads, cache.head_dim, cache.device
    batch.check(cache)
    if rotary.device != device:
        raise ValueError("rotary: expected frequencies on cuda:%d, got cuda:%d" % (device, rotary.device))
    rk, dtype = _kv_rows(k, batch.tokens, heads, dim, device, "k")
    rv, dtype_v = _kv_rows(v, batch.tokens, heads, dim, device, "v")
    rq = ro = None
    q_heads, types = 0, {dtype, dtype_v}
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out: expected both or neither")
    if q is not None:
        q_heads = q.shape[1] if q.dim() == 3 else 0
        rq, dtype_q = _kv_rows(q, batch.tokens, q_heads, dim, device, "q")
        ro, dtype_o = _kv_rows(q_out, batch.tokens, q_heads, dim, device, "q_out")
        types |= {dtype_q, dtype_o}
    if len(types) > 1:
        raise TypeError("q, q_out, k and v: expected the same type")
    turn = rotary.desc
    if positions is not None:
        _int32(positions, (batch.tokens,), "positions", device)
        turn = KVRotaryDesc(turn.d_turns, positions.data_ptr(), turn.rotary_dim, turn.interleaved, turn.magnitude)
    _check(splitzip_kv_rotary_write(d, batch.desc, turn, rq, ro, q_heads, rk, rv, dtype, _kv_status(status, device),
                                    _kv_stream(stream, device)), "splitzip_kv_rotary_write")


class KVTree:
    """Masks and positions of a step's trees of drafted tokens (splitzip_kv_tree_t),
    the same for every layer: device tensors mask (int32 (tokens, words), 32 new
    tokens of the row's sequence a word) and position (int32, tokens), and kv_tree's
    status word.  window: how many positions a row sees up to its own, 0: all."""

    def __init__(self, batch, window=0):
        torch = _torch()
        if not 0 <= window < 1 << 32:
            raise ValueError("window: expected 0 (none) or a number of positions, got %d" % window)
        device = batch.kv_len.device
        self.tokens, self.max_tokens, self.device, self.window = batch.tokens, batch.desc.max_tokens, batch.device, window
        self.words = max(1, -(-self.max_tokens // 32))
        if self.max_tokens > MAX_TREE_TOKENS:
            raise SplitZipError(ERR_UNSUPPORTED, "trees of %d tokens" % self.max_tokens)
        self.mask = torch.zeros(self.tokens, self.words, dtype=torch.int32, device=device)
        self.position = torch.zeros(self.tokens, dtype=torch.int32, device=device)
        self.status = torch.zeros(4, dtype=torch.int32, device=device)  # [0] = status
        self.desc = KVTreeDesc(self.mask.data_ptr(), self.position.data_ptr(), self.words, window)

    def check(self, batch):
        """Raises where the tree is of another step."""
        if self.device != batch.device:
            raise ValueError("tree on cuda:%d and step on cuda:%d: expected one device" % (self.device, batch.device))
        if self.tokens != batch.tokens or self.max_tokens < batch.desc.max_tokens:
            raise ValueError("tree of %d rows, %d of a sequence: expected one of the step's %d and %d"
                             % (self.tokens, self.max_tokens, batch.tokens, batch.desc.max_tokens))


def kv_tree(batch, parents, tree, stream=None):
    """Enqueue masks and positions of a step's trees into `tree` (asynchronous).
    parents: int32 (tokens): a new token's parent among its sequence's new tokens,
    smaller than its own number, -1 for a successor of the last older token."""
    tree.check(batch)
    _int32(parents, (batch.tokens,), "parents", batch.device)
    _check(splitzip_kv_tree(batch.desc, parents.data_ptr(), tree.desc, tree.status.data_ptr(),
                            _kv_stream(stream, batch.device)), "splitzip_kv_tree")


def kv_tree_attention(cache, batch, tree, q, out, bufs, scale, lse=None, stream=None):
    """Enqueue the attention of trees of drafted tokens over `cache`'s pages: every
    row sees what was there before its tree, its ancestors and itself
    (asynchronous; arguments as kv_attention's)."""
    batch.check(cache)
    tree.check(batch)
    device = cache.device
    if bufs.device != device:
        raise ValueError("bufs: expected buffers on cuda:%d, got cuda:%d" % (device, bufs.device))
    rq, dtype = _kv_rows(q, batch.tokens, bufs.q_heads, cache.head_dim, device, "q")
    ro, dtype_o = _kv_rows(out, batch.tokens, bufs.q_heads, cache.head_dim, device, "out")
    if dtype != dtype_o:
        raise TypeError("q and out: expected the same type")
    if lse is not None:
        if not lse.is_contiguous():
            raise ValueError("lse: expected a contiguous tensor")
        _device_tensor(lse, _torch().float32, (batch.tokens, bufs.q_heads), "lse", device)
        lse = lse.data_ptr()
    _check(splitzip_kv_tree_attention(cache.desc, batch.desc, tree.desc, rq, ro, lse, dtype, bufs.q_heads, scale,
                                      bufs.ws.data_ptr(), bufs.ws_bytes, bufs.status.data_ptr(),
                                      _kv_stream(stream, device)), "splitzip_kv_tree_attention")


class KVLayers:
    """The caches of a model's layers, of one geometry, for kv_keep."""

    def __init__(self, caches):
        self.caches = list(caches)
        if not self.caches or any(c.device != self.caches[0].device for c in self.caches):
            raise ValueError("caches: expected some, on one device")
        self.descs = (KVCacheDesc * len(self.caches))(*[c.desc for c in self.caches])


def kv_keep(layers, batch, path, kept, status, stream=None):
    """Enqueue the move of the accepted new tokens to the front of them in every
    layer's pages (asynchronous): new token path[cu_tokens[b] + i] of sequence b to
    the place of new token i, for i < kept[b].  path: int32 (tokens), ascending in
    each sequence; kept: int32 (batch).  kv_extend drops the others."""
    cache = layers.caches[0]
    device = cache.device
    batch.check(cache)
    _int32(path, (batch.tokens,), "path", device)
    _int32(kept, (batch.desc.batch,), "kept", device)
    _check(splitzip_kv_keep(layers.descs, len(layers.caches), batch.desc, path.data_ptr(), kept.data_ptr(),
                            _kv_status(status, device), _kv_stream(stream, device)), "splitzip_kv_keep")
