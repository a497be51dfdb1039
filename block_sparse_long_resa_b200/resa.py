"""ctypes binding of libresa (include/resa.h).

Argument marshalling only: every step of the hot path runs in the CUDA
kernels of libresa.so.  Tensors are torch CUDA tensors (PyTorch provides the
device memory and the stream); the functions keep the C names and raise
ResaError on any status other than RESA_OK.  There is no fallback: if the
library is missing, importing it raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libresa.so")

RESA_OK = 0
STATUS_NAMES = {0: "RESA_OK", 1: "RESA_ERR_NULL", 2: "RESA_ERR_SHAPE", 3: "RESA_ERR_RANGE",
                4: "RESA_ERR_UNSUPPORTED", 5: "RESA_ERR_CUDA", 6: "RESA_ERR_DEVICE_CHECK"}
DEVERR_SEQ_LEN, DEVERR_PAGE, DEVERR_BLOCK, DEVERR_TOPK, DEVERR_CHUNK, DEVERR_TIMEOUT, DEVERR_ROW = (
    0x1, 0x2, 0x4, 0x8, 0x10, 0x20, 0x40)
DEVERR_NONFINITE = 0x80


class ResaError(RuntimeError):
    def __init__(self, status: int, where: str, code: int = 0):
        self.status = status
        self.code = code
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}"
                         + (f" (device error word 0x{code:x})" if code else ""))


class resa_config_t(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("sm_scale", ctypes.c_float)]


class resa_cache_t(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("desc", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("seq_len", ctypes.c_void_p),
                ("batch", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("rows", ctypes.c_void_p),
                ("table_rows", ctypes.c_int32)]
    # as make_cache sets them: index of the tensors' device, (kv heads, block, head) of the pages
    device, dims, tensors = None, None, ()


class resa_cache_q4_t(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_sf", ctypes.c_void_p),
                ("v_sf", ctypes.c_void_p), ("desc", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("seq_len", ctypes.c_void_p),
                ("batch", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("rows", ctypes.c_void_p),
                ("table_rows", ctypes.c_int32), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p)]
    device = dims = None  # of the tensors it was made of; None: of addresses


class resa_rope_t(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("inv_freq", ctypes.c_void_p), ("mscale", ctypes.c_float)]
    device = None


class resa_tokens_t(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("f", ctypes.c_int32),
                ("n_new", ctypes.c_void_p), ("positions", ctypes.c_void_p)]
    device = dims = None  # dims: (batch, q heads or None, kv heads, head)


_lib = None

_P = ctypes.c_void_p
_I = ctypes.c_int32
_SIGS = {
    "resa_workspace_size": ([_P, _I, _I, _I], ctypes.c_size_t),
    "resa_workspace_init": ([_P, ctypes.c_size_t, _P], ctypes.c_int),
    "resa_check_device_status": ([_P, ctypes.c_size_t, _P, _P], ctypes.c_int),
    "resa_build_descriptors": ([_P, _P, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "resa_append_token": ([_P, _P, _P, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "resa_select_blocks": ([_P, _P, _P, _P, _I, _P, _P, _P, _P, ctypes.c_size_t, _P],
                           ctypes.c_int),
    "resa_sparse_decode": ([_P, _P, _P, _P, _P, _I, _P, _P, _P, ctypes.c_size_t, _P],
                           ctypes.c_int),
    "resa_rectify_attention": ([_P, _P, _I, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
                               ctypes.c_int),
    "resa_decode_step": ([_P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
                         ctypes.c_int),
    "resa_sparse_decode_noalloc": ([_P, _P, _P, _P, _P, _I, _P, _P, _P, _P], ctypes.c_int),
    "resa_dense_decode": ([_P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "resa_append_rope": ([_P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "resa_append_rope_q4": ([_P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "resa_expand_q4": ([_P, _P, _P, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "resa_sparse_decode_q4": ([_P, _P, _P, _P, _P, _I, _P, _P, _P, ctypes.c_size_t, _P],
                              ctypes.c_int),
    "resa_attention_q4": ([_P, _P, _I, _P, _P, _P, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "resa_kernels_per_call": ([ctypes.c_char_p], ctypes.c_int32),
    "resa_decode_step_launches": ([_P, _I, _I, _I], ctypes.c_int32),
    "resa_status_string": ([ctypes.c_int], ctypes.c_char_p),
}


def lib() -> ctypes.CDLL:
    """Load libresa.so (built in-tree by block_sparse_long_resa_b200.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libresa.so is not built ({LIB_PATH}); run "
                               "`python -m block_sparse_long_resa_b200.build`")
        dll = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            fn = getattr(dll, name)
            fn.argtypes = args
            fn.restype = res
        _lib = dll
    return _lib


_addr = ctypes.addressof


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


@functools.lru_cache(maxsize=None)
def _cuda():
    """(handle of a device's current stream, current device): the Stream object that
    torch.cuda.current_stream() makes costs 3 us a call."""
    import torch
    torch.cuda.init()
    return torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _stream(stream) -> Optional[int]:
    if stream is None:
        handle, device = _cuda()
        return handle(device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _device(where: str, tensors) -> Optional[int]:
    """Device index (-1: host memory) of the tensors among these; None when there are only
    addresses, which are the caller's to vouch for."""
    dev = None
    for t in tensors:
        if t is None or isinstance(t, int):
            continue
        d = t.get_device()
        if dev is None:
            dev = d
        elif d != dev:
            raise ResaError(4, f"{where}: tensors on more than one device")
    return dev


def _home(where: str, stream, ws, cfg, cache):
    """(stream handle, device index) of a call whose workspace and cache have to be on the
    current device, the one that the launch goes to, and whose cache has to be of the
    configuration's shape."""
    dev = ws.get_device()
    if dev < 0:
        raise ResaError(4, f"{where}: the workspace is on {ws.device}")
    if cache.dims is not None:
        if cache.device != dev:
            raise ResaError(4, f"{where}: the cache is not on the workspace's device")
        if cache.dims != (cfg.num_kv_heads, cfg.block_size, cfg.head_dim):
            raise ResaError(2, f"{where}: (kv heads, block, head) are {cache.dims} in the cache, not "
                               f"{(cfg.num_kv_heads, cfg.block_size, cfg.head_dim)}")
    handle, device = _cuda()
    if dev != device():
        raise ResaError(4, f"{where}: the workspace is on {ws.device}, not the current device")
    return (handle(dev) if stream is None else _stream(stream)), dev


def _look_over(where: str, cfg, cache):
    """Check the memory of a cache of make_cache, which checks nothing, at the first call that
    asks.  (A struct of addresses is the caller's to vouch for.)"""
    if not cache.tensors:
        return
    k, v, desc, page_table, seq_len, rows = cache.tensors
    dims = tuple(k.shape[1:]) if k.dim() == 4 else (cfg.num_kv_heads, cfg.block_size, cfg.head_dim)
    n = k.shape[0] * dims[0] * dims[1] * dims[2]
    device = _device(where, cache.tensors)
    for name, t, dtype, size in (
            ("k", k, "bfloat16", n), ("v", v, "bfloat16", n), ("desc", desc, "bfloat16", 2 * n // dims[1]),
            ("page_table", page_table, "int32", 0), ("seq_len", seq_len, "int32", page_table.shape[0]),
            ("rows", rows, "int32", 0)):
        if t is None or isinstance(t, int):
            continue
        _expect(f"{where}: {name}", t, dtype)
        if t.numel() < size:
            raise ResaError(2, f"{where}: {name} has {t.numel()} elements of {size}")
    cache.device, cache.dims = device, dims


@functools.lru_cache(maxsize=None)
def _dtypes():
    import torch
    return torch.bfloat16, torch.float32, torch.int32


def _at(where: str, name: str, t, dtype, size: int, dev: int) -> Optional[int]:
    """_ptr of a tensor that has to hold `size` bytes of dtype, one element behind the other, on
    device ``dev``.  (It may be larger, and of any shape.)"""
    if t is None or isinstance(t, int):
        return t
    if (t.dtype is dtype and t.nbytes >= size and t.get_device() == dev and t.is_contiguous()):
        return t.data_ptr()
    if t.get_device() != dev:
        raise ResaError(4, f"{where}: {name} is on {t.device}, not on the workspace's device")
    if t.dtype is not dtype:
        raise ResaError(4, f"{where}: {name} is {t.dtype}, not {dtype}")
    if t.nbytes < size:
        raise ResaError(2, f"{where}: {name} has {t.nbytes} bytes of {size}")
    raise ResaError(4, f"{where}: {name} is not contiguous")


def _check(st: int, where: str):
    if st != RESA_OK:
        raise ResaError(st, where)


# ---------------------------------------------------------------------------
# Plain structs
# ---------------------------------------------------------------------------

def make_config(num_q_heads: int, num_kv_heads: int, head_dim: int, block_size: int = 16,
                sm_scale: float = 0.0) -> resa_config_t:
    return resa_config_t(num_q_heads, num_kv_heads, head_dim, block_size, sm_scale)


def _keep(struct, *tensors):
    """The struct holds addresses only: keep these tensors alive with it."""
    struct.tensors = tensors
    return struct


def _keep_at(where: str, struct, *tensors):
    """_keep, of tensors that have to be on one device."""
    struct.device = _device(where, tensors)
    return _keep(struct, *tensors)


def make_cache(k, v, desc, page_table, seq_len, rows=None) -> resa_cache_t:
    """Cache struct over torch tensors k/v [pages][Hkv][b][d] bf16, desc
    [pages][Hkv][2][d] bf16, page_table [B][max_pages] int32, seq_len [B] int32.

    With ``rows`` (int32 device tensor [n]) the call covers the n sequences in
    those rows of page_table / seq_len (the row map of resa_cache_t).  The struct
    keeps all of them alive."""
    nrows = int(page_table.shape[0])
    return _keep(resa_cache_t(_ptr(k), _ptr(v), _ptr(desc), _ptr(page_table), _ptr(seq_len),
                              nrows if rows is None else int(rows.numel()),
                              int(page_table.shape[1]), int(k.shape[0]), _ptr(rows),
                              0 if rows is None else nrows),
                 k, v, desc, page_table, seq_len, rows)


def _expect(name: str, t, dtype: str, shape=None):
    """Refuse a tensor whose memory is not what the C ABI takes it for."""
    if t is None:
        return
    if str(t.dtype) not in tuple("torch." + d for d in dtype.split("|")):
        raise ResaError(4, f"{name}: {t.dtype}, not {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ResaError(2, f"{name}: shape {tuple(t.shape)}, not {tuple(shape)}")
    if not t.is_contiguous():
        raise ResaError(4, f"{name} is not contiguous")


def make_cache_q4(k, k_sf, v, v_sf, desc, page_table, seq_len, rows=None, k_scale=None,
                  v_scale=None) -> resa_cache_q4_t:
    """4-bit cache struct over torch tensors k/v [pages][Hkv][b][d/2] uint8 codes, k_sf/v_sf
    [pages][Hkv][b][d/16] float8_e4m3fn group scales, desc / page_table / seq_len / rows as in
    make_cache, and the heads' scales k_scale/v_scale [Hkv] fp32 (None: 1).  The struct keeps
    all of them alive."""
    pages, hkv, b, half = k.shape
    for name, t, dtype, shape in (
            ("k", k, "uint8", None), ("v", v, "uint8", k.shape),
            ("k_sf", k_sf, "float8_e4m3fn|uint8", (pages, hkv, b, half // 8)),
            ("v_sf", v_sf, "float8_e4m3fn|uint8", (pages, hkv, b, half // 8)),
            ("desc", desc, "bfloat16", (pages, hkv, 2, 2 * half)),
            ("page_table", page_table, "int32", None),
            ("seq_len", seq_len, "int32", page_table.shape[:1]), ("rows", rows, "int32", None),
            ("k_scale", k_scale, "float32", (hkv,)), ("v_scale", v_scale, "float32", (hkv,))):
        _expect("make_cache_q4: " + name, t, dtype, shape)
    nrows = int(page_table.shape[0])
    c = _keep_at("make_cache_q4",
                 resa_cache_q4_t(_ptr(k), _ptr(v), _ptr(k_sf), _ptr(v_sf), _ptr(desc),
                                 _ptr(page_table), _ptr(seq_len),
                                 nrows if rows is None else int(rows.numel()),
                                 int(page_table.shape[1]), int(k.shape[0]), _ptr(rows),
                                 0 if rows is None else nrows, _ptr(k_scale), _ptr(v_scale)),
                 k, k_sf, v, v_sf, desc, page_table, seq_len, rows, k_scale, v_scale)
    c.dims = (hkv, b, 2 * half)
    return c


def make_rope(rot_dim: int, inv_freq, interleaved: bool = False,
              mscale: float = 1.0) -> resa_rope_t:
    """Rotary embedding of the first ``rot_dim`` channels; inv_freq: fp32 device tensor
    [rot_dim / 2] (None when rot_dim is 0)."""
    if rot_dim:
        _expect("make_rope: inv_freq", inv_freq, "float32", (rot_dim // 2,))
    return _keep_at("make_rope", resa_rope_t(rot_dim, 1 if interleaved else 0,
                                             _ptr(inv_freq) if rot_dim else None, mscale),
                    inv_freq if rot_dim else None)


def _token_stride(t, name: str) -> int:
    """Elements between consecutive tokens of a [batch][f][heads][d] tensor."""
    if t.dim() != 4:
        raise ResaError(2, f"make_tokens: {name} is not [batch][f][heads][d]")
    b, f, h, d = t.shape
    tok = t.stride(1) if f > 1 else (t.stride(0) if b > 1 else h * d)
    if (tok < h * d or (d > 1 and t.stride(3) != 1) or (h > 1 and t.stride(2) != d)
            or (b > 1 and f > 1 and t.stride(0) != f * tok)):
        raise ResaError(4, f"make_tokens: {name} is not evenly strided by tokens")
    return tok


def make_tokens(q, k, v, n_new=None, positions=None) -> resa_tokens_t:
    """Fresh tokens of a call: q [batch][f][Hq][d] (or None), k, v [batch][f][Hkv][d] bf16, e.g.
    views of one fused projection output; n_new [batch] and positions [batch][f] int32 or None."""
    b, f = k.shape[:2]
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t is not None and (str(t.dtype) != "torch.bfloat16" or tuple(t.shape[:2]) != (b, f)):
            raise ResaError(2, f"make_tokens: {name} is not [batch][f][heads][d] bf16 as k is")
    if v.shape != k.shape or (q is not None and q.shape[3:] != k.shape[3:]):
        raise ResaError(2, "make_tokens: v has not k's heads, or the heads differ in size")
    _expect("make_tokens: n_new", n_new, "int32", (b,))
    _expect("make_tokens: positions", positions, "int32", (b, f))
    x = _keep_at("make_tokens",
                 resa_tokens_t(_ptr(q), _ptr(k), _ptr(v),
                               0 if q is None else _token_stride(q, "q"), _token_stride(k, "k"),
                               _token_stride(v, "v"), int(k.shape[1]), _ptr(n_new),
                               _ptr(positions)), q, k, v, n_new, positions)
    x.dims = (b, None if q is None else q.shape[2], k.shape[2], k.shape[3])
    return x


# ---------------------------------------------------------------------------
# Entry points (same names as the C ABI)
# ---------------------------------------------------------------------------

def resa_workspace_size(cfg: resa_config_t, batch: int, max_pages: int, max_chunk: int = 0) -> int:
    n = lib().resa_workspace_size(ctypes.byref(cfg), batch, max_pages, max_chunk)
    if n == 0:
        raise ResaError(2, "resa_workspace_size")
    return int(n)


def resa_workspace_init(ws, stream=None):
    _check(lib().resa_workspace_init(_ptr(ws), ws.numel(), _stream(stream)), "resa_workspace_init")


def resa_check_device_status(ws, stream=None, raise_on_error: bool = True) -> int:
    code = ctypes.c_uint32(0)
    st = lib().resa_check_device_status(_ptr(ws), ws.numel(), _stream(stream), ctypes.byref(code))
    if st != RESA_OK and (raise_on_error or st != 6):
        raise ResaError(st, "resa_check_device_status", code.value)
    return int(code.value)


def resa_build_descriptors(cfg, cache, first_block, ws, stream=None):
    _check(lib().resa_build_descriptors(ctypes.byref(cfg), ctypes.byref(cache), _ptr(first_block),
                                        _ptr(ws), ws.numel(), _stream(stream)),
           "resa_build_descriptors")


def resa_append_token(cfg, cache, k_new, v_new, ws, stream=None):
    _check(lib().resa_append_token(ctypes.byref(cfg), ctypes.byref(cache), _ptr(k_new),
                                   _ptr(v_new), _ptr(ws), ws.numel(), _stream(stream)),
           "resa_append_token")


def resa_select_blocks(cfg, cache, q, topk, max_topk: int, block_idx, block_cnt, scores, ws,
                       stream=None):
    _check(lib().resa_select_blocks(ctypes.byref(cfg), ctypes.byref(cache), _ptr(q), _ptr(topk),
                                    max_topk, _ptr(block_idx), _ptr(block_cnt), _ptr(scores),
                                    _ptr(ws), ws.numel(), _stream(stream)),
           "resa_select_blocks")


def resa_sparse_decode(cfg, cache, q, block_idx, block_cnt, max_topk: int, out, lse, ws,
                       stream=None):
    _check(lib().resa_sparse_decode(ctypes.byref(cfg), ctypes.byref(cache), _ptr(q),
                                    _ptr(block_idx), _ptr(block_cnt), max_topk, _ptr(out),
                                    _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)),
           "resa_sparse_decode")


def resa_rectify_attention(cfg, cache, f: int, q_chunk, k_new, v_new, out, lse, ws, stream=None):
    _check(lib().resa_rectify_attention(ctypes.byref(cfg), ctypes.byref(cache), f, _ptr(q_chunk),
                                        _ptr(k_new), _ptr(v_new), _ptr(out), _ptr(lse), _ptr(ws),
                                        ws.numel(), _stream(stream)),
           "resa_rectify_attention")


def resa_decode_step(cfg, cache, q, k_new, v_new, topk, max_topk: int, out, lse, block_idx,
                     block_cnt, ws, stream=None):
    _check(lib().resa_decode_step(ctypes.byref(cfg), ctypes.byref(cache), _ptr(q), _ptr(k_new),
                                  _ptr(v_new), _ptr(topk), max_topk, _ptr(out), _ptr(lse),
                                  _ptr(block_idx), _ptr(block_cnt), _ptr(ws), ws.numel(),
                                  _stream(stream)),
           "resa_decode_step")


def resa_dense_decode(cfg, cache, q, k_new, v_new, out, lse, ws, stream=None):
    """Dense decode: append the decode token and attend to every position."""
    _check(lib().resa_dense_decode(ctypes.byref(cfg), ctypes.byref(cache), _ptr(q), _ptr(k_new),
                                   _ptr(v_new), _ptr(out), _ptr(lse), _ptr(ws), ws.numel(),
                                   _stream(stream)),
           "resa_dense_decode")


def resa_sparse_decode_noalloc(cfg, cache, q, block_idx, block_cnt, max_topk: int, out, lse,
                               dev_error, stream=None):
    """resa_sparse_decode without a workspace, for callers that cannot allocate
    device memory (scratch lives in a fixed device array inside the library).
    dev_error: a device uint32 word (e.g. an int32 tensor element) that
    receives the device error bits; required."""
    _check(lib().resa_sparse_decode_noalloc(ctypes.byref(cfg), ctypes.byref(cache), _ptr(q),
                                            _ptr(block_idx), _ptr(block_cnt), max_topk, _ptr(out),
                                            _ptr(lse), _ptr(dev_error), _stream(stream)),
           "resa_sparse_decode_noalloc")


def _append_args(where: str, stream, cfg, cache, rope, tokens, q_out, ws):
    """(stream handle, address of q_out) of a rotary append."""
    st, dev = _home(where, stream, ws, cfg, cache)
    hq, batch = cfg.num_q_heads, cache.batch
    if rope.device is not None and rope.device != dev:
        raise ResaError(4, f"{where}: inv_freq is not on the workspace's device")
    if tokens.dims is not None:
        if tokens.device != dev:
            raise ResaError(4, f"{where}: the tokens are not on the workspace's device")
        n, heads, kv_heads, d = tokens.dims
        if (n < batch or (heads is not None and heads != hq) or kv_heads != cfg.num_kv_heads
                or d != cfg.head_dim):
            raise ResaError(2, f"{where}: (batch, q heads, kv heads, head) are {tokens.dims} in the tokens, "
                               f"{(batch, hq, cfg.num_kv_heads, cfg.head_dim)} in the call")
    return st, _at(where, "q_out", q_out, _dtypes()[0], 2 * batch * tokens.f * hq * cfg.head_dim, dev)


def resa_append_rope(cfg, cache, rope, tokens, q_out, ws, stream=None):
    """Append fresh tokens to the bf16 cache, queries and keys rotated on the way."""
    if cache.dims is None:
        _look_over("resa_append_rope", cfg, cache)
    st, out = _append_args("resa_append_rope", stream, cfg, cache, rope, tokens, q_out, ws)
    st = lib().resa_append_rope(_addr(cfg), _addr(cache), _addr(rope), _addr(tokens), out,
                                ws.data_ptr(), ws.nbytes, st)
    if st != RESA_OK:
        raise ResaError(st, "resa_append_rope")


def resa_append_rope_q4(cfg, cache, rope, tokens, q_out, ws, stream=None):
    """resa_append_rope into a 4-bit cache (make_cache_q4)."""
    st, out = _append_args("resa_append_rope_q4", stream, cfg, cache, rope, tokens, q_out, ws)
    st = lib().resa_append_rope_q4(_addr(cfg), _addr(cache), _addr(rope), _addr(tokens), out,
                                   ws.data_ptr(), ws.nbytes, st)
    if st != RESA_OK:
        raise ResaError(st, "resa_append_rope_q4")


def resa_expand_q4(cfg, cache, k_out, v_out, ws, stream=None):
    """Write a 4-bit cache's valid positions into bf16 pages k_out / v_out."""
    where = "resa_expand_q4"
    st, dev = _home(where, stream, ws, cfg, cache)
    bf16, _, _ = _dtypes()
    n = 2 * cache.num_pages * cfg.num_kv_heads * cfg.block_size * cfg.head_dim
    st = lib().resa_expand_q4(_addr(cfg), _addr(cache), _at(where, "k_out", k_out, bf16, n, dev),
                              _at(where, "v_out", v_out, bf16, n, dev), ws.data_ptr(), ws.nbytes, st)
    if st != RESA_OK:
        raise ResaError(st, where)


def resa_sparse_decode_q4(cfg, cache, q, block_idx, block_cnt, max_topk: int, out, lse, ws,
                          stream=None):
    """resa_sparse_decode over a 4-bit cache."""
    where = "resa_sparse_decode_q4"
    st, dev = _home(where, stream, ws, cfg, cache)
    bf16, f32, i32 = _dtypes()
    batch = cache.batch
    rows, units = 4 * batch * cfg.num_q_heads, 4 * batch * cfg.num_kv_heads  # bytes of a word each
    n = rows * cfg.head_dim
    try:  # the checks of _at, in line: seven calls of it take 1 us
        fit = (q.dtype is bf16 and q.nbytes >= n // 2 and q.get_device() == dev and q.is_contiguous()
               and block_idx.dtype is i32 and block_idx.nbytes >= units * (max_topk + 1)
               and block_idx.get_device() == dev and block_idx.is_contiguous()
               and block_cnt.dtype is i32 and block_cnt.nbytes >= units
               and block_cnt.get_device() == dev and block_cnt.is_contiguous()
               and out.dtype is f32 and out.nbytes >= n and out.get_device() == dev
               and out.is_contiguous()
               and (lse is None or (lse.dtype is f32 and lse.nbytes >= rows
                                    and lse.get_device() == dev and lse.is_contiguous())))
    except AttributeError:  # an address among them
        fit = False
    if fit:
        st = lib().resa_sparse_decode_q4(
            _addr(cfg), _addr(cache), q.data_ptr(), block_idx.data_ptr(), block_cnt.data_ptr(), max_topk,
            out.data_ptr(), None if lse is None else lse.data_ptr(), ws.data_ptr(), ws.nbytes, st)
    else:
        st = lib().resa_sparse_decode_q4(
            _addr(cfg), _addr(cache), _at(where, "q", q, bf16, n // 2, dev),
            _at(where, "block_idx", block_idx, i32, units * (max_topk + 1), dev),
            _at(where, "block_cnt", block_cnt, i32, units, dev), max_topk,
            _at(where, "out", out, f32, n, dev), _at(where, "lse", lse, f32, rows, dev),
            ws.data_ptr(), ws.nbytes, st)
    if st != RESA_OK:
        raise ResaError(st, where)


def resa_attention_q4(cfg, cache, f: int, n_new, q, out, lse, ws, stream=None):
    """Causal attention of each sequence's last n_new (None: f) tokens over its 4-bit cache."""
    where = "resa_attention_q4"
    st, dev = _home(where, stream, ws, cfg, cache)
    bf16, f32, i32 = _dtypes()
    batch = cache.batch
    rows = 4 * batch * f * cfg.num_q_heads  # bytes of a word each
    n = rows * cfg.head_dim
    st = lib().resa_attention_q4(
        _addr(cfg), _addr(cache), f,
        n_new if n_new is None else _at(where, "n_new", n_new, i32, 4 * batch, dev),
        _at(where, "q", q, bf16, n // 2, dev), _at(where, "out", out, f32, n, dev),
        lse if lse is None else _at(where, "lse", lse, f32, rows, dev), ws.data_ptr(), ws.nbytes, st)
    if st != RESA_OK:
        raise ResaError(st, where)


def resa_kernels_per_call(entry_point: str) -> int:
    return int(lib().resa_kernels_per_call(entry_point.encode()))


def resa_decode_step_launches(cfg, batch: int, max_pages: int, num_pages: int) -> int:
    """1 when resa_decode_step runs as one fused launch for this cache shape, else 3."""
    return int(lib().resa_decode_step_launches(ctypes.byref(cfg), batch, max_pages, num_pages))


def resa_status_string(status: int) -> str:
    return lib().resa_status_string(status).decode()
