"""What the structs of the rotary append and of the 4-bit cache hold of their tensors, without a GPU."""
import gc
import weakref

import pytest
import torch

from block_sparse_long_resa_b200 import resa as R
from block_sparse_long_resa_b200.cache import LayerCache, LayerCacheQ4


def test_structs_keep_their_lengths_and_tables():
    """A struct holds addresses: the lengths made for one call live as long as it does."""
    table = torch.zeros(2, 3, dtype=torch.int32)
    c4 = LayerCacheQ4.empty(6, 2, 16, 64, table)
    k = torch.zeros(6, 2, 16, 64, dtype=torch.bfloat16)
    c16 = LayerCache(k, k, c4.desc, table, c4.seq_len)
    for make in (c4.struct, c4.select_struct, c16.struct):
        lens, rows = torch.tensor([5, 7], dtype=torch.int32), torch.tensor([1], dtype=torch.int32)
        seen = [weakref.ref(lens), weakref.ref(rows)]
        s = make(seq_len=lens, rows=rows)
        del lens, rows
        gc.collect()
        assert all(x() is not None for x in seen)
        assert s.seq_len == seen[0]().data_ptr() and s.rows == seen[1]().data_ptr()
        del s
        gc.collect()
        assert all(x() is None for x in seen)
    # and every other tensor that a 4-bit struct is made of
    args = [t.clone() for t in (c4.k, c4.k_sf, c4.v, c4.v_sf, c4.desc, table, c4.seq_len)]
    seen = [weakref.ref(t) for t in args]
    s = R.make_cache_q4(*args)
    del args
    gc.collect()
    assert all(x() is not None for x in seen)


def test_tokens_of_unlike_heads_are_refused():
    """k and v of other head counts, or heads of other sizes, would be read past their ends."""
    x = lambda h, d: torch.zeros(2, 5, h, d, dtype=torch.bfloat16)
    R.make_tokens(x(8, 64), x(2, 64), x(2, 64))
    for q, k, v in ((None, x(2, 64), x(1, 64)), (None, x(2, 64), x(4, 64)), (None, x(2, 128), x(2, 64)),
                    (None, x(2, 64), x(2, 128)), (x(8, 128), x(2, 64), x(2, 64)),
                    (x(8, 64), x(2, 128), x(2, 128))):
        with pytest.raises(R.ResaError) as e:
            R.make_tokens(q, k, v)
        assert e.value.status == 2


class FakeWorkspace:
    """The workspace of a device that this machine need not have."""

    def __init__(self, index=0):
        self.index, self.device, self.nbytes = index, f"cuda:{index}", 1 << 34

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 0x10000000


class Elsewhere:
    """A tensor whose memory is on the given device."""

    def __init__(self, t, index):
        self.t, self.index = t, index

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.t, name)


CFG = R.make_config(8, 2, 64, 16)


def calls(index=0):
    """Each entry point's call with every tensor on device `index`: name -> (function of the
    replaced arguments, the arguments)."""
    put = lambda t: Elsewhere(t, index)
    table = put(torch.zeros(2, 3, dtype=torch.int32))
    e = LayerCacheQ4.empty(6, 2, 16, 64, torch.zeros(2, 3, dtype=torch.int32))
    c4 = [put(x) for x in (e.k, e.k_sf, e.v, e.v_sf, e.desc)] + [table, put(e.seq_len)]
    k16 = put(torch.zeros(6, 2, 16, 64, dtype=torch.bfloat16))
    f = 5
    x = lambda *s, dtype=torch.bfloat16: put(torch.zeros(*s, dtype=dtype))
    i32, f32 = torch.int32, torch.float32
    inv, tok = x(32, dtype=f32), (x(2, f, 8, 64), x(2, f, 2, 64), x(2, f, 2, 64))

    def append(four, c=None, inv=inv, q=tok[0], k=tok[1], v=tok[2], n=None, q_out=x(2, f, 8, 64),
               ws=FakeWorkspace(index), cfg=CFG, stream=None):
        cache = R.make_cache_q4(*(c or c4)) if four else \
            R.make_cache(*(c or (k16, k16, c4[4], table, c4[6])))
        (R.resa_append_rope_q4 if four else R.resa_append_rope)(
            cfg, cache, R.make_rope(64, inv), R.make_tokens(q, k, v, n_new=n), q_out, ws, stream)

    def expand(c=None, k_out=k16, v_out=k16, ws=FakeWorkspace(index), cfg=CFG, stream=None):
        R.resa_expand_q4(cfg, R.make_cache_q4(*(c or c4)), k_out, v_out, ws, stream)

    def sparse(c=None, q=x(2, 8, 64), idx=x(2, 2, 4, dtype=i32), cnt=x(2, 2, dtype=i32), top=3,
               out=x(2, 8, 64, dtype=f32), lse=x(2, 8, dtype=f32), ws=FakeWorkspace(index), cfg=CFG,
               stream=None):
        R.resa_sparse_decode_q4(cfg, R.make_cache_q4(*(c or c4)), q, idx, cnt, top, out, lse, ws, stream)

    def attention(c=None, n=x(2, dtype=i32), q=x(2, f, 8, 64), out=x(2, f, 8, 64, dtype=f32),
                  lse=x(2, f, 8, dtype=f32), ws=FakeWorkspace(index), cfg=CFG, stream=None):
        R.resa_attention_q4(cfg, R.make_cache_q4(*(c or c4)), f, n, q, out, lse, ws, stream)

    return c4, {"append": lambda **kw: append(False, **kw), "append4": lambda **kw: append(True, **kw),
                "expand": expand, "sparse": sparse, "attention": attention}


class Launches:
    """Stands for the library: counts the calls that reach it."""

    def __init__(self):
        self.n = 0

    def __getattr__(self, name):
        def call(*args):
            self.n += 1
            return 0
        return call


@pytest.fixture
def launches(monkeypatch):
    """No library and no GPU: device 0 is the current one."""
    x = Launches()
    monkeypatch.setattr(R, "lib", lambda: x)
    monkeypatch.setattr(R, "_cuda", lambda: ((lambda i: 0x77), (lambda: 0)))
    return x


def refused(f, launches, status, **kw):
    n = launches.n
    with pytest.raises(R.ResaError) as e:
        f(**kw)
    assert e.value.status == status and launches.n == n, kw


def test_memory_of_the_host_or_of_another_device_is_refused(launches):
    c4, run = calls(0)
    for f in run.values():
        f()
        f(stream=0)
    assert launches.n == 10
    far = lambda t: [Elsewhere(t, -1), Elsewhere(t, 1)]
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)
    i32, f32 = torch.int32, torch.float32
    for name in ("append", "append4"):
        for kw in ([dict(inv=t) for t in far(z(32, dtype=f32))] + [dict(q_out=t) for t in far(z(2, 5, 8, 64))]
                   + [dict(n=t) for t in far(z(2, dtype=i32))] + [dict(k=t) for t in far(z(2, 5, 2, 64))]):
            refused(run[name], launches, 4, **kw)
    for name in ("append4", "expand", "sparse", "attention"):
        for i, t in enumerate(c4):
            for there in far(t.t):
                refused(run[name], launches, 4, c=c4[:i] + [there] + c4[i + 1:])
        all_there = [[Elsewhere(t.t, d) for t in c4] for d in (-1, 1)]
        for c in all_there:
            refused(run[name], launches, 4, c=c)
    for t in far(z(6, 2, 16, 64)):
        refused(run["expand"], launches, 4, k_out=t)
        refused(run["expand"], launches, 4, v_out=t)
        refused(run["append"], launches, 4, c=(t, t, c4[4], c4[5], c4[6]))
        refused(run["append"], launches, 4, c=(Elsewhere(t.t, 0), t, c4[4], c4[5], c4[6]))
    for kw in (dict(q=z(2, 8, 64)), dict(idx=z(2, 2, 4, dtype=i32)), dict(cnt=z(2, 2, dtype=i32)),
               dict(out=z(2, 8, 64, dtype=f32)), dict(lse=z(2, 8, dtype=f32))):
        refused(run["sparse"], launches, 4, **kw)
    for kw in (dict(q=z(2, 5, 8, 64)), dict(n=z(2, dtype=i32)), dict(out=z(2, 5, 8, 64, dtype=f32)),
               dict(lse=z(2, 5, 8, dtype=f32))):
        refused(run["attention"], launches, 4, **kw)


def test_calls_away_from_the_current_device_are_refused(launches):
    """Everything on device 1 while device 0 is current, with a stream given or not."""
    _, run = calls(1)
    for f in run.values():
        refused(f, launches, 4)
        refused(f, launches, 4, stream=0x1234)


def test_tensors_of_other_sizes_and_types_are_refused(launches):
    c4, run = calls(0)
    put = lambda t: Elsewhere(t, 0)
    z = lambda *s, dtype=torch.bfloat16: put(torch.zeros(*s, dtype=dtype))
    i32, f32 = torch.int32, torch.float32
    # a configuration that is not the cache's
    for cfg in (R.make_config(8, 4, 64, 16), R.make_config(8, 2, 128, 16), R.make_config(8, 2, 64, 32),
                R.make_config(8, 1, 64, 16)):
        for f in run.values():
            refused(f, launches, 2, cfg=cfg)
    for name in ("append", "append4"):
        f = run[name]
        # tokens of fewer sequences, of other heads
        refused(f, launches, 2, q=z(1, 5, 8, 64), k=z(1, 5, 2, 64), v=z(1, 5, 2, 64))
        refused(f, launches, 2, q=z(2, 5, 4, 64))
        refused(f, launches, 2, q=z(2, 5, 0, 64))
        refused(f, launches, 2, k=z(2, 5, 1, 64), v=z(2, 5, 1, 64))
        refused(f, launches, 2, q=z(2, 5, 8, 32), k=z(2, 5, 2, 32), v=z(2, 5, 2, 32))
        # a place for the queries that is too small, of other numbers, or with gaps
        refused(f, launches, 2, q_out=z(2, 4, 8, 64))
        refused(f, launches, 4, q_out=z(2, 5, 8, 64, dtype=f32))
        refused(f, launches, 4, q_out=put(torch.zeros(2, 5, 8, 128, dtype=torch.bfloat16)[..., :64]))
        f(q=None, q_out=None)
        f(q=z(3, 5, 8, 64), k=z(3, 5, 2, 64), v=z(3, 5, 2, 64))    # of more sequences than the call's
        f(q_out=z(2 * 5 * 8 * 64 + 64))
    k16, table, lens = z(6, 2, 16, 64), c4[5], c4[6]
    for c in ((k16, z(5, 2, 16, 64), c4[4], table, lens), (k16, k16, z(6, 2, 1, 64), table, lens),
              (k16, k16, c4[4], table, z(1, dtype=i32))):
        refused(run["append"], launches, 2, c=c)
    for c in ((z(6, 2, 16, 64, dtype=f32), k16, c4[4], table, lens),
              (k16, k16, c4[4], table, z(2, dtype=torch.int64)),
              (k16, k16, c4[4], z(2, 3, dtype=torch.int64), lens),
              (k16, k16, c4[4], put(torch.zeros(2, 6, dtype=i32)[:, :3]), lens)):
        refused(run["append"], launches, 4, c=c)
    for name in ("k_out", "v_out"):
        refused(run["expand"], launches, 2, **{name: z(5, 2, 16, 64)})
        refused(run["expand"], launches, 4, **{name: z(6, 2, 16, 64, dtype=torch.float16)})
    for status, kw in ((2, dict(q=z(1, 8, 64))), (4, dict(q=z(2, 8, 64, dtype=f32))),
                       (4, dict(q=put(torch.zeros(2, 64, 8, dtype=torch.bfloat16).transpose(1, 2)))),
                       (2, dict(top=4)), (2, dict(idx=z(2, 2, 3, dtype=i32))),
                       (4, dict(idx=z(2, 2, 4, dtype=torch.int64))), (2, dict(cnt=z(2, dtype=i32))),
                       (4, dict(cnt=z(2, 2, dtype=f32))), (4, dict(out=z(2, 8, 64))),
                       (2, dict(out=z(2, 8, 32, dtype=f32))), (2, dict(lse=z(8, dtype=f32))),
                       (4, dict(lse=z(2, 8)))):
        refused(run["sparse"], launches, status, **kw)
    run["sparse"](lse=None)
    for status, kw in ((2, dict(q=z(2, 4, 8, 64))), (4, dict(q=z(2, 5, 8, 64, dtype=f32))),
                       (2, dict(n=z(1, dtype=i32))), (4, dict(n=z(2, dtype=torch.int64))),
                       (4, dict(out=z(2, 5, 8, 64))), (2, dict(out=z(2, 8, 64, dtype=f32))),
                       (2, dict(lse=z(2, 8, dtype=f32))), (4, dict(lse=z(2, 5, 8)))):
        refused(run["attention"], launches, status, **kw)
    run["attention"](lse=None, n=None)
    # buffers may be larger than the call
    run["attention"](q=z(4, 5, 8, 64), out=z(4, 5, 8, 64, dtype=f32), lse=z(4, 5, 8, dtype=f32))
