"""Refusals of the rotary appends and of the 4-bit cache's entry points, without a GPU: the C
checks answer before anything is launched, the constructors before anything is called."""
import ctypes

import pytest
import torch

from block_sparse_long_resa_b200 import build as B
from block_sparse_long_resa_b200 import resa as R
from block_sparse_long_resa_b200.cache import LayerCacheQ4

WS = 1 << 34   # "bytes" of the workspace: enough for any of these calls


@pytest.fixture(scope="module")
def lib():
    B.build()
    return R.lib()


def q4_cache(**kw):
    c = R.resa_cache_q4_t(0x100000, 0x200000, 0x300000, 0x400000, 0x500000, 0x600000, 0x700000, 2,
                          64, 128, None, 0, 0x800000, 0x900000)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def bf_cache(**kw):
    c = R.resa_cache_t(0x100000, 0x200000, 0x300000, 0x600000, 0x700000, 2, 64, 128)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def rope(**kw):
    r = R.resa_rope_t(64, 0, 0xa00000, 1.0)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def tokens(**kw):
    t = R.resa_tokens_t(0xb00000, 0xc00000, 0xd00000, 0, 0, 0, 4, None, None)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


CFG = R.make_config(8, 2, 64, 16)


def append(lib, four, cfg=CFG, cache=None, r=None, t=None, q_out=0xe00000, ws=0xf00000, n=WS):
    cache = cache or (q4_cache() if four else bf_cache())
    f = lib.resa_append_rope_q4 if four else lib.resa_append_rope
    ref = lambda x: ctypes.byref(x) if x is not None else None
    return f(ref(cfg), ref(cache), ref(r or rope()), ref(t or tokens()), q_out, ws, n, None)


@pytest.mark.parametrize("four", [False, True], ids=["bf16", "q4"])
def test_append_refusals(lib, four):
    f = lib.resa_append_rope_q4 if four else lib.resa_append_rope
    c = ctypes.byref(q4_cache() if four else bf_cache())
    ok = (ctypes.byref(rope()), ctypes.byref(tokens()))
    assert f(None, c, *ok, 0xe00000, 0xf00000, WS, None) == 1
    assert f(ctypes.byref(CFG), None, *ok, 0xe00000, 0xf00000, WS, None) == 1
    assert f(ctypes.byref(CFG), c, None, ok[1], 0xe00000, 0xf00000, WS, None) == 1
    assert f(ctypes.byref(CFG), c, ok[0], None, 0xe00000, 0xf00000, WS, None) == 1
    a = lambda **kw: append(lib, four, **kw)
    assert a(cfg=R.make_config(8, 3, 64, 16)) == 2
    assert a(cfg=R.make_config(8, 2, 96, 16)) == 4
    assert a(q_out=None) == 1                              # queries without a place for them
    assert a(t=tokens(q=None)) == 1                        # and the other way round
    assert a(t=tokens(k=None)) == 1 and a(t=tokens(v=None)) == 1
    assert a(t=tokens(f=0)) == 3 and a(t=tokens(f=-3)) == 3
    assert a(r=rope(rot_dim=80)) == 3 and a(r=rope(rot_dim=-16)) == 3
    assert a(r=rope(rot_dim=24)) == 4
    assert a(r=rope(inv_freq=None)) == 1
    assert a(r=rope(mscale=float("inf"))) == 3 and a(r=rope(mscale=float("nan"))) == 3
    assert a(t=tokens(k_stride=64)) == 2                   # below one token's heads
    assert a(t=tokens(q_stride=512 + 4)) == 4              # not a multiple of 8
    assert a(t=tokens(q_stride=1024), q_out=0xb00000) == 2  # in place needs a contiguous q
    assert a(t=tokens(k=0xc00008)) == 4 and a(q_out=0xe00004) == 4
    assert a(t=tokens(n_new=0x100002)) == 4
    assert a(ws=None) == 1 and a(n=1000) == 2
    big = dict(batch=65536)
    assert a(cache=q4_cache(**big) if four else bf_cache(**big), n=1 << 60) == 4
    if four:
        for name in ("k", "v", "k_sf", "v_sf", "desc", "page_table", "seq_len"):
            assert a(cache=q4_cache(**{name: None})) == 1, name
        assert a(cache=q4_cache(k_sf=0x300008)) == 4 and a(cache=q4_cache(k_scale=0x800002)) == 4


def test_expand_refusals(lib):
    def e(cache=None, k=0x1000000, v=0x1100000, ws=0xf00000, n=WS):
        return lib.resa_expand_q4(ctypes.byref(CFG), ctypes.byref(cache or q4_cache()), k, v, ws, n, None)
    assert e(k=None) == 1 and e(v=None) == 1
    assert e(k=0x1000008) == 4
    assert e(cache=q4_cache(num_pages=0)) == 2
    assert e(cache=q4_cache(v_sf=None)) == 1
    assert e(cache=q4_cache(batch=65536), n=1 << 60) == 4
    assert e(n=8) == 2


def test_sparse_decode_q4_refusals(lib):
    def s(cfg=CFG, cache=None, q=0x1000000, idx=0x1100000, cnt=0x1200000, top=8, out=0x1300000,
          lse=None, ws=0xf00000, n=WS):
        return lib.resa_sparse_decode_q4(ctypes.byref(cfg), ctypes.byref(cache or q4_cache()), q, idx,
                                         cnt, top, out, lse, ws, n, None)
    assert s(q=None) == 1 and s(idx=None) == 1 and s(cnt=None) == 1 and s(out=None) == 1
    assert s(top=-1) == 3 and s(top=0x7fffffff) == 3 and s(top=1 << 30) == 3
    assert s(q=0x1000008) == 4 and s(idx=0x1100002) == 4 and s(lse=0x1300001) == 4
    assert s(cfg=R.make_config(34, 2, 64, 16)) == 4        # 17 heads a group
    assert s(ws=None) == 1 and s(n=16) == 2
    assert s(cache=q4_cache(rows=0x10, table_rows=0)) == 2


def test_attention_q4_refusals(lib):
    def t(f=1, n_new=None, q=0x1000000, out=0x1300000, n=WS, cache=None):
        return lib.resa_attention_q4(ctypes.byref(CFG), ctypes.byref(cache or q4_cache()), f, n_new, q,
                                     out, None, 0xf00000, n, None)
    assert t(q=None) == 1 and t(out=None) == 1
    assert t(f=0) == 3 and t(f=-1) == 3
    assert t(f=4097) == 4 and t(f=1 << 30) == 4 and t(f=0x7fffffff) == 4   # 4 heads a group
    assert t(n_new=0x1400002) == 4
    small = R.resa_workspace_size(CFG, 2, 64, 0)
    assert t(f=5, n=small) == 2                            # 20 rows: a workspace for chunks
    many = q4_cache(batch=1 << 20, max_pages=1 << 20)
    assert t(cache=many, n=1 << 62) == 3                   # entries of work past 32 bits


def test_kernels_per_call(lib):
    for name in ("resa_append_rope", "resa_append_rope_q4", "resa_expand_q4", "resa_sparse_decode_q4",
                 "resa_attention_q4"):
        assert R.resa_kernels_per_call(name) == 1


def test_constructors_refuse_other_memory():
    table = torch.zeros(2, 3, dtype=torch.int32)
    c = LayerCacheQ4.empty(6, 2, 16, 64, table)
    assert c.struct().num_pages == 6 and c.batch == 2 and c.max_pages == 3
    args = [c.k, c.k_sf, c.v, c.v_sf, c.desc, table, c.seq_len]

    def refuses(i, x, status, **kw):
        a = list(args)
        if i is not None:
            a[i] = x
        with pytest.raises(R.ResaError) as e:
            R.make_cache_q4(*a, **kw)
        assert e.value.status == status
    refuses(0, c.k.int(), 4)
    refuses(1, c.k_sf[:, :1], 2)
    refuses(2, c.v.transpose(1, 2).contiguous().transpose(1, 2), 4)
    refuses(4, c.desc.float(), 4)
    refuses(5, table.long(), 4)
    refuses(6, c.seq_len[:1], 2)
    refuses(None, None, 4, k_scale=torch.ones(2, dtype=torch.float64))
    refuses(None, None, 2, v_scale=torch.ones(3))
    k = torch.zeros(2, 5, 2, 64, dtype=torch.bfloat16)
    R.make_tokens(None, k, k)
    wide = torch.zeros(2, 5, 6 * 64, dtype=torch.bfloat16)
    t = R.make_tokens(wide[..., :128].unflatten(2, (2, 64)), wide[..., 128:256].unflatten(2, (2, 64)),
                      wide[..., 256:].unflatten(2, (2, 64)))
    assert t.q_stride == t.k_stride == 384 and t.f == 5
    for bad in (dict(k=k[:, ::2]), dict(k=k.transpose(2, 3)), dict(k=k[:, :1].expand(2, 5, 2, 64)),
                dict(v=k[:, :4]), dict(q=k.float()), dict(n_new=torch.zeros(2)),
                dict(n_new=torch.zeros(3, dtype=torch.int32)),
                dict(positions=torch.zeros(2, 4, dtype=torch.int32))):
        with pytest.raises(R.ResaError):
            R.make_tokens(**{**dict(q=None, k=k, v=k), **bad})
    with pytest.raises(R.ResaError):
        R.make_rope(64, torch.zeros(64))
    with pytest.raises(R.ResaError):
        R.make_rope(64, torch.zeros(32, dtype=torch.float64))


def test_binding_refuses_a_workspace_that_is_not_on_a_gpu(lib):
    table = torch.zeros(2, 3, dtype=torch.int32)
    c = LayerCacheQ4.empty(6, 2, 16, 64, table)
    with pytest.raises(R.ResaError) as e:
        R.resa_expand_q4(CFG, c.struct(), c.desc, c.desc, torch.zeros(64, dtype=torch.uint8))
    assert e.value.status == 4
