"""The rotary append and the 4-bit cache's entry points against the numpy oracle in 64 bits."""
import numpy as np
import pytest
import torch

from block_sparse_long_resa_b200 import resa as R
from block_sparse_long_resa_b200.cache import workspace as R_workspace
from oracle import q4
from q4_problem import Problem, attention_tolerance, f64

pytestmark = pytest.mark.gpu

LAYOUTS = [(28, 4, 128, 16), (32, 2, 64, 32), (8, 8, 128, 64), (16, 1, 64, 16), (14, 2, 128, 32),
           (4, 2, 64, 64)]


def ids(x):
    return "-".join(map(str, x)) if isinstance(x, (tuple, list)) else str(x)


# ------------------------------------------------------------------------------------- appends

class Tokens:
    """Fresh tokens of a call, fused into one projection output or apart, rows of padding NaN."""

    def __init__(self, p, f, fresh, fused, key_size=1.0, shift=None):
        batch = len(fresh)
        q = p.rng.standard_normal((batch, f, p.hq, p.d))
        k = p.rng.standard_normal((batch, f, p.hkv, p.d)) * key_size
        v = p.rng.standard_normal((batch, f, p.hkv, p.d))
        self.q, self.k, self.v = q4.bf16(q), q4.bf16(k), q4.bf16(v)
        for i, n in enumerate(fresh):
            self.q[i, n:] = self.k[i, n:] = self.v[i, n:] = np.nan
        up = lambda x: torch.from_numpy(x).to(p.dev).bfloat16()
        if fused:
            x = torch.cat([up(self.q).flatten(2), up(self.k).flatten(2), up(self.v).flatten(2)], 2)
            nq, nk = p.hq * p.d, p.hkv * p.d
            self.tq = x[..., :nq].unflatten(2, (p.hq, p.d))
            self.tk = x[..., nq:nq + nk].unflatten(2, (p.hkv, p.d))
            self.tv = x[..., nq + nk:].unflatten(2, (p.hkv, p.d))
        else:
            self.tq, self.tk, self.tv = up(self.q), up(self.k), up(self.v)
        self.n = torch.tensor(fresh, dtype=torch.int32, device=p.dev)
        self.pos = None
        if shift is not None:
            self.pos = p.rng.integers(0, shift, (batch, f)).astype(np.int32)
            self.tpos = torch.from_numpy(self.pos).to(p.dev)

    def struct(self, with_n=True, with_q=True):
        return R.make_tokens(self.tq if with_q else None, self.tk, self.tv,
                             n_new=self.n if with_n else None,
                             positions=None if self.pos is None else self.tpos)


APPENDS = [  # lens (after the append), fresh, f, rot, interleaved, fused, shift
    ([1, 16, 17, 64, 65], [1, 1, 1, 1, 1], 1, 1.0, False, True, None),
    ([40, 3, 100, 0, 129], [40, 3, 33, 0, 2], 40, 0.5, True, False, None),
    ([300, 5, 77], [300, 0, 50], 301, 1.0, True, True, 1 << 20),
    ([70, 33], [64, 1], 64, 0.0, False, False, None),
    ([130, 200], [100, 100], 100, 48, False, True, 5),
]


@pytest.mark.parametrize("four", [False, True], ids=["bf16", "q4"])
@pytest.mark.parametrize("layout", LAYOUTS, ids=ids)
@pytest.mark.parametrize("case", range(len(APPENDS)))
def test_append(cuda_device, case, layout, four):
    lens, fresh, f, rot, inter, fused, shift = APPENDS[case]
    hq, hkv, d, b = layout
    rot = rot if isinstance(rot, int) else int(d * rot)
    p = Problem(100 + case, lens, hq, hkv, d, b, cuda_device)
    t = Tokens(p, f, fresh, fused, shift=shift)
    inv = (1e4 ** (-np.arange(0, rot, 2) / max(rot, 1))).astype(np.float32)
    rope = R.make_rope(rot, torch.from_numpy(inv).to(cuda_device), interleaved=inter, mscale=1.25)
    up = lambda x: torch.from_numpy(x).to(cuda_device).bfloat16()
    k, v = up(p.k16), up(p.v16)
    q_out = torch.full((len(lens), f, hq, d), 9.0, dtype=torch.bfloat16, device=cuda_device)
    if four:
        R.resa_append_rope_q4(p.cfg, p.cache4(), rope, t.struct(), q_out, p.ws)
    else:
        cache = R.make_cache(k, v, p.desc, p.t_table, p.t_len)
        R.resa_append_rope(p.cfg, cache, rope, t.struct(), q_out, p.ws)
    assert p.status() == 0

    kc, ks, vc, vs = p.kc.copy(), p.ks.copy(), p.vc.copy(), p.vs.copy()
    k16, v16, desc = p.k16.copy(), p.v16.copy(), np.full(p.desc.shape, 7.0)
    want_q = np.full(q_out.shape, 9.0)
    tol_q = np.zeros(q_out.shape)
    for i, (L, n) in enumerate(zip(lens, fresh)):
        if n == 0:
            continue
        at = np.arange(L - n, L)
        pos = at if t.pos is None else t.pos[i, :n]
        want_q[i, :n] = q4.rotate(t.q[i, :n], pos, inv, rot, inter, 1.25)
        # half a bf16 step, and 2^-20 of the pair's size for the angle, sine and products in 32 bits
        tol_q[i, :n] = np.abs(want_q[i, :n]) * 2.0 ** -8 + 2.0 ** -20 * 1.25 * 2 * np.abs(t.q[i, :n]).max()
        kn = q4.bf16(q4.rotate(t.k[i, :n], pos, inv, rot, inter, 1.25))
        vn = t.v[i, :n]
        page, slot = p.table[i, at // b], at % b
        if four:
            kc[page, :, slot], ks[page, :, slot] = q4.quantise(kn, p.gk[:, None])
            vc[page, :, slot], vs[page, :, slot] = q4.quantise(vn, p.gv[:, None])
        else:
            k16[page, :, slot], v16[page, :, slot] = kn, vn
        for blk in range((L - n) // b, (L - 1) // b + 1):
            pg, m = p.table[i, blk], min(b, L - blk * b)
            x = q4.bf16(q4.values(kc[pg, :, :m], ks[pg, :, :m]) * p.gk[:, None, None].astype(float)) \
                if four else k16[pg, :, :m]
            desc[pg, :, 0], desc[pg, :, 1] = x.min(1), x.max(1)
    got = f64(q_out)
    assert (np.abs(got - want_q) <= tol_q).all()
    np.testing.assert_array_equal(f64(p.desc), desc)
    if four:
        for name, c, s, tc, ts in (("k", kc, ks, p.k4, p.k_sf), ("v", vc, vs, p.v4, p.v_sf)):
            np.testing.assert_array_equal(ts.view(torch.uint8).cpu().numpy(), s, err_msg=name)
            np.testing.assert_array_equal(tc.cpu().numpy(), q4.pack(c), err_msg=name)
    else:
        np.testing.assert_array_equal(f64(k), k16)
        np.testing.assert_array_equal(f64(v), v16)


def test_append_without_queries_and_in_place(cuda_device):
    """q NULL leaves the keys' path alone; q_out may be q itself."""
    p = Problem(7, [50, 20], 8, 2, 64, 16, cuda_device)
    inv = torch.tensor(1e4 ** (-np.arange(0, 64, 2) / 64), dtype=torch.float32, device=cuda_device)
    t = Tokens(p, 20, [20, 20], False)
    rope = R.make_rope(64, inv)
    k1, v1 = (torch.from_numpy(x).to(cuda_device).bfloat16() for x in (p.k16, p.v16))
    k2, v2 = k1.clone(), v1.clone()
    d2 = p.desc.clone()
    apart = torch.empty_like(t.tq)
    R.resa_append_rope(p.cfg, R.make_cache(k1, v1, p.desc, p.t_table, p.t_len), rope,
                       t.struct(with_n=False), apart, p.ws)
    R.resa_append_rope(p.cfg, R.make_cache(k2, v2, d2, p.t_table, p.t_len), rope,
                       t.struct(with_n=False, with_q=False), None, p.ws)
    assert torch.equal(k1, k2) and torch.equal(v1, v2) and torch.equal(p.desc, d2)
    R.resa_append_rope(p.cfg, R.make_cache(k2, v2, d2, p.t_table, p.t_len), rope,
                       t.struct(with_n=False), t.tq, p.ws)
    assert torch.equal(t.tq, apart)
    assert p.status() == 0


def test_append_one_token_equals_append_token(cuda_device):
    """Without a rotation, one token a sequence is resa_append_token."""
    p = Problem(8, [1, 16, 33, 200], 28, 4, 128, 16, cuda_device)
    t = Tokens(p, 1, [1] * 4, False)
    k1, v1 = (torch.from_numpy(x).to(cuda_device).bfloat16() for x in (p.k16, p.v16))
    k2, v2 = k1.clone(), v1.clone()
    c1 = R.make_cache(k1, v1, p.desc, p.t_table, p.t_len)
    R.resa_build_descriptors(p.cfg, c1, None, p.ws)
    d2 = p.desc.clone()
    c2 = R.make_cache(k2, v2, d2, p.t_table, p.t_len)
    R.resa_append_rope(p.cfg, c1, R.make_rope(0, None), t.struct(with_q=False), None, p.ws)
    # the descriptors of the keys before the token, then the token folded in
    first = torch.zeros(4, dtype=torch.int32, device=cuda_device)
    lens = torch.clamp(p.t_len - 1, min=1)
    short = R.make_cache(k2, v2, d2, p.t_table, lens)
    R.resa_build_descriptors(p.cfg, short, first, p.ws)
    R.resa_append_token(p.cfg, c2, t.tk, t.tv, p.ws)
    assert torch.equal(k1, k2) and torch.equal(v1, v2) and torch.equal(p.desc, d2)
    assert p.status() == 0


def test_append_extreme_values(cuda_device):
    """Zeros, the smallest and largest scales, halfway points, infinity and NaN in 4 bits."""
    p = Problem(9, [64], 2, 1, 64, 16, cuda_device, head_scales=False)
    x = np.zeros((1, 64, 1, 64))
    x[0, 1, 0, :] = 1.0
    x[0, 2, 0, :16] = [0, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5]
    x[0, 3] = 2.0 ** -9 * x[0, 2]
    x[0, 4] = 448 * x[0, 2]
    x[0, 5, 0, ::3] = 3e38
    x[0, 6, 0, 5] = 1e-38
    x[0, 7, 0, :16] = 2.0 ** -10 * np.arange(16)
    x[0, 8:] = np.exp(p.rng.standard_normal((56, 1, 64)) * 6) * p.rng.choice([-1, 1], (56, 1, 64))
    x = q4.bf16(x)
    k = torch.from_numpy(x).to(cuda_device).bfloat16()
    tok = R.make_tokens(None, k, k)
    R.resa_append_rope_q4(p.cfg, p.cache4(), R.make_rope(0, None), tok, None, p.ws)
    assert p.status() == 0
    code, s = q4.quantise(x[0], np.ones((1, 1), np.float32))
    at = np.arange(64)
    page, slot = p.table[0, at // 16], at % 16
    for c, sf in ((p.k4, p.k_sf), (p.v4, p.v_sf)):
        np.testing.assert_array_equal(sf.view(torch.uint8).cpu().numpy()[page, :, slot], s)
        np.testing.assert_array_equal(c.cpu().numpy()[page, :, slot], q4.pack(code))
    # infinity is stored as the largest value, NaN as 0, and the error word says so
    k[0, 0, 0, :4] = torch.tensor([float("inf"), float("-inf"), float("nan"), 1.0])
    R.resa_append_rope_q4(p.cfg, p.cache4(), R.make_rope(0, None), tok, None, p.ws)
    assert p.status() == R.DEVERR_NONFINITE
    assert p.k_sf.view(torch.uint8)[page[0], 0, 0, 0].item() == 126
    assert p.k4[page[0], 0, 0, 0].item() == 0xf7 and p.k4[page[0], 0, 0, 1].item() == 0x00


# ----------------------------------------------------------------------------------- expansion

@pytest.mark.parametrize("layout", LAYOUTS, ids=ids)
def test_expand(cuda_device, layout):
    hq, hkv, d, b = layout
    p = Problem(20, [1, 0, b - 1, b, b + 1, 517], hq, hkv, d, b, cuda_device)
    k = torch.full((p.num_pages, hkv, b, d), 5.0, dtype=torch.bfloat16, device=cuda_device)
    v = torch.full_like(k, 6.0)
    R.resa_expand_q4(p.cfg, p.cache4(), k, v, p.ws)
    assert p.status() == 0
    live = p.live[:, None, :, None]
    with np.errstate(invalid="ignore"):
        sk, sv = np.minimum(p.ks, 126), np.minimum(p.vs, 126)
        wk = np.where(live, q4.bf16(q4.values(p.kc, sk) * p.gk[:, None, None].astype(float)), 5.0)
        wv = np.where(live, q4.bf16(q4.values(p.vc, sv) * p.gv[:, None, None].astype(float)), 6.0)
    np.testing.assert_array_equal(f64(k), wk)
    np.testing.assert_array_equal(f64(v), wv)


# ------------------------------------------------------------------------------- sparse decode

def sparse(p, idx, cnt, max_topk, q, rows=None):
    n = q.shape[0]
    out = torch.full((n, p.hq, p.d), 3.0, device=p.dev)
    lse = torch.full((n, p.hq), 3.0, device=p.dev)
    R.resa_sparse_decode_q4(p.cfg, p.cache4(rows=rows), q, idx, cnt, max_topk, out, lse, p.ws)
    return f64(out), f64(lse)


def check_rows(p, out, lse, q, i, h, blocks, limit):
    """Rows out [n, d], lse [n] of queries q [n, d] (float64) over blocks of (sequence i, head h)."""
    k, v, pos = p.keys_values(i, h, blocks)
    lim = np.searchsorted(pos, limit) if blocks is None else np.full(len(q), len(pos))
    o, z, a, mag, vsum = q4.attention(q, k, v, lim, p.d ** -0.5)
    to, tz = attention_tolerance(mag[:, None], len(pos), a, vsum)
    assert (np.abs(out - o) <= to).all(), (i, h, np.abs(out - o).max(), to.min())
    fin = np.isfinite(z)
    assert (np.abs(lse[fin] - z[fin]) <= tz[:, 0][fin] + 2.0 ** -22 * np.abs(z[fin])).all(), (i, h)
    assert (lse[~fin] == -np.inf).all()


@pytest.mark.parametrize("layout", LAYOUTS, ids=ids)
def test_sparse_decode(cuda_device, layout):
    hq, hkv, d, b = layout
    lens = [1, b, 3 * b + 1, 2000, 700, 5003]
    p = Problem(30, lens, hq, hkv, d, b, cuda_device)
    q = q4.bf16(p.rng.standard_normal((len(lens), hq, d)))
    max_topk = max(-(-L // b) for L in lens)
    idx = np.full((len(lens), hkv, max_topk + 1), 1 << 30, dtype=np.int32)
    cnt = np.zeros((len(lens), hkv), dtype=np.int32)
    lists = {}
    for i, L in enumerate(lens):
        for h in range(hkv):
            nb = -(-L // b)
            m = 0 if (i, h) == (3, 0) else int(p.rng.integers(1, nb + 1))
            lists[i, h] = p.rng.permutation(nb)[:m]       # any order, the last block or not
            idx[i, h, :m], cnt[i, h] = lists[i, h], m
    t = lambda x: torch.from_numpy(x).to(cuda_device)
    out, lse = sparse(p, t(idx), t(cnt), max_topk, t(q).bfloat16())
    assert p.status() == 0
    g = p.g
    for (i, h), blocks in lists.items():
        r = slice(h * g, (h + 1) * g)
        check_rows(p, out[i, r], lse[i, r], q[i, r], i, h, blocks, None)
    # the same lists through a row map, in another order
    rows = np.array([4, 2, 5], dtype=np.int32)
    o2, l2 = sparse(p, t(idx[rows]), t(cnt[rows]), max_topk, t(q[rows]).bfloat16(), rows=t(rows))
    for j, i in enumerate(rows):
        for h in range(hkv):
            r = slice(h * g, (h + 1) * g)
            check_rows(p, o2[j, r], l2[j, r], q[i, r], i, h, lists[i, h], None)


def test_sparse_decode_large_logits(cuda_device):
    """Logits of hundreds: one key takes nearly all the weight, the running maximum grows often."""
    p = Problem(31, [3000], 28, 4, 128, 16, cuda_device, key_size=8.0)
    q = q4.bf16(p.rng.standard_normal((1, 28, 128)) * 20)
    nb = -(-3000 // 16)
    idx = np.tile(np.arange(nb, dtype=np.int32), (1, 4, 1))
    cnt = np.full((1, 4), nb, dtype=np.int32)
    t = lambda x: torch.from_numpy(x).to(cuda_device)
    out, lse = sparse(p, t(idx), t(cnt), nb - 1, t(q).bfloat16())
    for h in range(4):
        check_rows(p, out[0, 7 * h:7 * h + 7], lse[0, 7 * h:7 * h + 7], q[0, 7 * h:7 * h + 7], 0, h,
                   np.arange(nb), None)


# ------------------------------------------------------------------------------ dense and chunk

def chunk(p, f, fresh, q, rows=None):
    n = q.shape[0]
    out = torch.full((n, f, p.hq, p.d), 3.0, device=p.dev)
    lse = torch.full((n, f, p.hq), 3.0, device=p.dev)
    R.resa_attention_q4(p.cfg, p.cache4(rows=rows), f, fresh, q, out, lse, p.ws)
    return f64(out), f64(lse)


CHUNKS = [  # lens, f, fresh
    ([1, 17, 64, 65, 1000, 4099], 1, None),
    ([3, 200, 129], 2, None),
    ([40, 700, 64, 0], 33, [33, 0, 7, 0]),
    ([1500], 64, None),
    ([128, 130, 391], 128, [128, 1, 77]),
    ([700, 333], 333, [301, 333]),
]


@pytest.mark.parametrize("layout", LAYOUTS, ids=ids)
@pytest.mark.parametrize("case", range(len(CHUNKS)))
def test_attention(cuda_device, case, layout):
    lens, f, fresh = CHUNKS[case]
    hq, hkv, d, b = layout
    p = Problem(40 + case, lens, hq, hkv, d, b, cuda_device, max_chunk=f)
    q = q4.bf16(p.rng.standard_normal((len(lens), f, hq, d)))
    n_new = fresh if fresh is not None else [f] * len(lens)
    for i, n in enumerate(n_new):
        q[i, n:] = np.nan
    t_n = None if fresh is None else torch.tensor(fresh, dtype=torch.int32, device=cuda_device)
    tq = torch.from_numpy(q).to(cuda_device).bfloat16()
    out, lse = chunk(p, f, t_n, tq)
    assert p.status() == 0
    g = p.g
    for i, n in enumerate(n_new):
        assert (out[i, n:] == 3.0).all() and (lse[i, n:] == 3.0).all()   # rows of padding
        limit = np.repeat(np.arange(lens[i] - n, lens[i]) + 1, g)
        for h in range(hkv if n else 0):
            r = slice(h * g, (h + 1) * g)
            check_rows(p, out[i, :n, r].reshape(-1, d), lse[i, :n, r].reshape(-1),
                       q[i, :n, r].reshape(-1, d), i, h, None, limit)
    # a second call gives the same bits: nothing depends on the order of arrival
    o2, l2 = chunk(p, f, t_n, tq)
    assert np.array_equal(out, o2) and np.array_equal(lse, l2)


def test_attention_row_map(cuda_device):
    p = Problem(60, [100, 900, 50, 333], 28, 4, 128, 16, cuda_device, max_chunk=20)
    q = q4.bf16(p.rng.standard_normal((2, 20, 28, 128)))
    rows = torch.tensor([3, 1], dtype=torch.int32, device=cuda_device)
    out, lse = chunk(p, 20, None, torch.from_numpy(q).to(cuda_device).bfloat16(), rows=rows)
    assert p.status() == 0
    for j, i in enumerate((3, 1)):
        limit = np.repeat(np.arange(p.lens[i] - 20, p.lens[i]) + 1, 7)
        for h in range(4):
            r = slice(7 * h, 7 * h + 7)
            check_rows(p, out[j, :, r].reshape(-1, 128), lse[j, :, r].reshape(-1),
                       q[j, :, r].reshape(-1, 128), i, h, None, limit)


# ----------------------------------------------------------------------------- errors and misuse

def test_device_errors_skip_the_item(cuda_device):
    dev = cuda_device
    p = Problem(70, [100, 100, 100], 8, 2, 64, 16, dev, max_chunk=40)
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    tok = Tokens(p, 4, [4, 4, 4], False)
    rope = R.make_rope(0, None)
    q_out = torch.full((3, 4, 8, 64), 9.0, dtype=torch.bfloat16, device=dev)

    def append(n, lens=None, rows=None):
        q_out.fill_(9.0)
        tok.n = t(n)
        R.resa_append_rope_q4(p.cfg, p.cache4(rows=rows, seq_len=lens), rope, tok.struct(), q_out, p.ws)
        return p.status()

    assert append([4, 5, -1]) == R.DEVERR_CHUNK
    assert (q_out[1:] == 9.0).all() and not (q_out[0] == 9.0).any()
    assert append([4, 4, 4], lens=t([3, 100, 100])) == R.DEVERR_CHUNK
    assert append([4, 4, 0], lens=t([100, 1 << 30, -5])) == R.DEVERR_SEQ_LEN
    assert append([4, 4, 4], rows=t([0, 7, 2])) == R.DEVERR_ROW | R.DEVERR_SEQ_LEN
    p.t_table[1, 6] = p.num_pages
    before = p.k4.clone()
    assert append([0, 4, 0]) == R.DEVERR_PAGE
    assert torch.equal(before, p.k4)
    k16 = torch.zeros(p.num_pages, 2, 16, 64, dtype=torch.bfloat16, device=dev)
    R.resa_expand_q4(p.cfg, p.cache4(), k16, k16.clone(), p.ws)
    assert p.status() == R.DEVERR_PAGE
    # attention: the bad page's keys are left out
    for f in (1, 40):
        q = torch.randn(3, f, 8, 64, device=dev).bfloat16()
        out, lse = chunk(p, f, None, q)
        assert p.status() == R.DEVERR_PAGE
        assert np.isfinite(out).all() and (out != 3.0).all()
        out, lse = chunk(p, f, t([f, 0, f + 1]), q)
        assert p.status() == R.DEVERR_CHUNK
        assert (out[1:] == 3.0).all() and (lse[1:] == 3.0).all() and (out[0] != 3.0).all()
    # block lists: ids outside the sequence are skipped, a list of nothing else gives zeros
    q = torch.randn(3, 8, 64, device=dev).bfloat16()
    idx = t([[[0, -1, 6]] * 2, [[0, 7, 1 << 30]] * 2, [[-5, 99, 7]] * 2])
    cnt = torch.full((3, 2), 3, dtype=torch.int32, device=dev)
    out, lse = sparse(p, idx, cnt, 2, q)
    assert p.status() == R.DEVERR_BLOCK
    p.refresh()
    assert (out[2] == 0).all() and (lse[2] == -np.inf).all()
    qf = f64(q)
    for h in range(2):
        r = slice(4 * h, 4 * h + 4)
        check_rows(p, out[0, r], lse[0, r], qf[0, r], 0, h, np.array([0, 6]), None)
        check_rows(p, out[1, r], lse[1, r], qf[1, r], 1, h, np.array([0]), None)
    # a sequence of no length: zeros, as resa_sparse_decode gives
    bad = p.cache4(seq_len=t([0, 100, 100]))
    o = torch.full((3, 8, 64), 3.0, device=dev)
    R.resa_sparse_decode_q4(p.cfg, bad, q, idx, cnt, 2, o, None, p.ws)
    assert p.status() & R.DEVERR_SEQ_LEN
    assert (o[0] == 0).all()


# ------------------------------------------------------------------------------ used together

@pytest.mark.parametrize("layout", [(28, 4, 128, 16), (8, 2, 64, 32)], ids=ids)
def test_cycle_on_the_four_bit_cache(cuda_device, layout):
    """A prompt, decode steps with selected blocks, a rectification and the hand-over to bf16:
    append, resa_select_blocks on the 4-bit cache's descriptors, sparse decode, chunk attention,
    expansion, and the bf16 entry points on the expanded pages."""
    hq, hkv, d, b = layout
    dev = cuda_device
    f, steps, prompt = 8, 8, [300, 70]
    batch = len(prompt)
    p = Problem(80, [n + steps for n in prompt], hq, hkv, d, b, dev, max_chunk=max(prompt))
    inv = torch.tensor(1e4 ** (-np.arange(0, d, 2) / d), dtype=torch.float32, device=dev)
    rope = R.make_rope(d, inv)
    lens = torch.tensor(prompt, dtype=torch.int32, device=dev)
    n_new = lens.clone()
    c4 = p.cache4(seq_len=lens)
    t = Tokens(p, max(prompt), prompt, True)
    q_rot = torch.zeros(batch, max(prompt), hq, d, dtype=torch.bfloat16, device=dev)
    out = torch.zeros(batch, max(prompt), hq, d, device=dev)
    R.resa_append_rope_q4(p.cfg, c4, rope, t.struct(), q_rot, p.ws)
    R.resa_attention_q4(p.cfg, c4, max(prompt), n_new, q_rot, out, None, p.ws)

    def bf16_pages():
        k = torch.zeros(p.num_pages, hkv, b, d, dtype=torch.bfloat16, device=dev)
        v = torch.zeros_like(k)
        R.resa_expand_q4(p.cfg, c4, k, v, p.ws)
        return k, v

    topk = torch.tensor([5, 2], dtype=torch.int32, device=dev)
    idx = torch.zeros(batch, hkv, 6, dtype=torch.int32, device=dev)
    cnt = torch.zeros(batch, hkv, dtype=torch.int32, device=dev)
    late = []
    for s in range(steps):
        lens += 1
        one = Tokens(p, 1, [1] * batch, True)
        late.append(one)
        q1 = torch.empty(batch, 1, hq, d, dtype=torch.bfloat16, device=dev)
        o1 = torch.empty(batch, hq, d, device=dev)
        R.resa_append_rope_q4(p.cfg, c4, rope, one.struct(with_n=False), q1, p.ws)
        sel = R.make_cache(p.k4, p.v4, p.desc, p.t_table, lens)
        R.resa_select_blocks(p.cfg, sel, q1, topk, 5, idx, cnt, None, p.ws)
        R.resa_sparse_decode_q4(p.cfg, c4, q1, idx, cnt, 5, o1, None, p.ws)
        if s in (0, steps - 1):
            k, v = bf16_pages()
            c16 = R.make_cache(k, v, p.desc.clone(), p.t_table, lens)
            before = c16.desc
            fresh_desc = torch.zeros_like(p.desc)
            c16d = R.make_cache(k, v, fresh_desc, p.t_table, lens)
            R.resa_build_descriptors(p.cfg, c16d, None, p.ws)
            used = np.unique(np.concatenate([p.table[i, :-(-int(n) // b)] for i, n in enumerate(lens.tolist())]))
            assert torch.equal(fresh_desc[used.tolist()], p.desc[used.tolist()])
            o16 = torch.empty(batch, hq, d, device=dev)
            R.resa_sparse_decode(p.cfg, c16, q1, idx, cnt, 5, o16, None, p.ws)
            # the bf16 pages round each value by 2^-8 of itself: logits move by 2^-8 of
            # sum |q k| <= |q| |k| (below 2 * d here), outputs by 2^-8 of the largest value too
            x = (2.0 ** -8) * (q1.float().norm(dim=-1).max() * k.float().norm(dim=-1).max() * d ** -0.5 * 2 + 1)
            assert (o1 - o16).abs().max() <= x * v.float().abs().max()
    # rectification: the last f tokens again, against every position
    kf = torch.cat([x.tk for x in late], 1).contiguous()
    vf = torch.cat([x.tv for x in late], 1).contiguous()
    qf = torch.cat([x.tq for x in late], 1).contiguous()
    k4, sf = p.k4.clone(), p.k_sf.view(torch.uint8).clone()
    qr = torch.empty_like(qf)
    R.resa_append_rope_q4(p.cfg, c4, rope, R.make_tokens(qf, kf, vf), qr, p.ws)
    assert torch.equal(k4, p.k4) and torch.equal(sf, p.k_sf.view(torch.uint8))
    o = torch.empty(batch, f, hq, d, device=dev)
    R.resa_attention_q4(p.cfg, c4, f, None, qr, o, None, p.ws)
    assert p.status() == 0
    # the last row of the chunk is a dense decode step: both within the bound of the exact result
    kb, vb = bf16_pages()
    mag = float(qr.float().norm(dim=-1).max() * kb.float().norm(dim=-1).max()) * d ** -0.5
    tol, _ = attention_tolerance(mag, max(p.lens), float(vb.abs().max()))
    o1 = torch.empty(batch, hq, d, device=dev)
    R.resa_attention_q4(p.cfg, c4, 1, None, qr[:, -1].contiguous(), o1, None, p.ws)
    assert (o[:, -1] - o1).abs().max() <= 2 * tol
    assert p.status() == 0


def test_graph_capture_and_replay(cuda_device):
    """Captured on a side stream, replayed with other inputs in the same buffers; two graphs share
    one workspace on one stream."""
    dev = cuda_device
    p = Problem(90, [500, 130], 28, 4, 128, 16, dev, max_chunk=16)
    q = torch.randn(2, 16, 28, 128, device=dev).bfloat16()
    q1 = torch.randn(2, 28, 128, device=dev).bfloat16()
    idx = torch.tensor([[[0, 3, 31]] * 4, [[1, 2, 8]] * 4], dtype=torch.int32, device=dev)
    cnt = torch.full((2, 4), 3, dtype=torch.int32, device=dev)
    out, out1 = torch.zeros(2, 16, 28, 128, device=dev), torch.zeros(2, 28, 128, device=dev)
    tok = Tokens(p, 16, [16, 16], False)
    q_out = torch.zeros_like(tok.tq)
    rope = R.make_rope(0, None)
    c4 = p.cache4()
    st = torch.cuda.Stream()

    def first():
        R.resa_append_rope_q4(p.cfg, c4, rope, tok.struct(with_n=False), q_out, p.ws)
        R.resa_attention_q4(p.cfg, c4, 16, None, q, out, None, p.ws)

    def second():
        R.resa_sparse_decode_q4(p.cfg, c4, q1, idx, cnt, 2, out1, None, p.ws)

    with torch.cuda.stream(st):
        first()
        second()
    st.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1, stream=st):
        first()
    with torch.cuda.graph(g2, stream=st):
        second()
    for seed in range(3):
        torch.manual_seed(seed)
        for x in (q, q1, tok.tq, tok.tk, tok.tv):
            x.copy_(torch.randn(x.shape, device=dev))
        g1.replay()
        g2.replay()
        g1.replay()
        torch.cuda.synchronize()
        got, got1, gq = out.clone(), out1.clone(), q_out.clone()
        out.zero_(), out1.zero_(), q_out.zero_()
        first()
        second()
        assert torch.equal(got, out) and torch.equal(got1, out1) and torch.equal(gq, q_out)
    assert p.status() == 0


# ------------------------------------------------------------- further shapes, splits and streams

@pytest.mark.parametrize("inter", [False, True], ids=["half", "adjacent"])
@pytest.mark.parametrize("rot", [16, 48, 112])
@pytest.mark.parametrize("d", [64, 128])
def test_append_partial_rotations(cuda_device, d, rot, inter):
    """Rotations of a part of the head, positions of any sign."""
    if rot > d:
        rot = 32
    p = Problem(11, [37, 50], 4, 2, d, 16, cuda_device)
    t = Tokens(p, 37, [37, 20], False)
    pos = np.stack([np.arange(37) * 1001 - 17000, np.arange(37) - 18]).astype(np.int32)
    inv = (1e4 ** (-np.arange(0, rot, 2) / rot)).astype(np.float32)
    t_pos, t_inv = torch.from_numpy(pos).to(cuda_device), torch.from_numpy(inv).to(cuda_device)
    tok = R.make_tokens(t.tq, t.tk, t.tv, n_new=t.n, positions=t_pos)
    k, v = (torch.from_numpy(x).to(cuda_device).bfloat16() for x in (p.k16, p.v16))
    q_out = torch.zeros_like(t.tq)
    R.resa_append_rope(p.cfg, R.make_cache(k, v, p.desc, p.t_table, p.t_len),
                       R.make_rope(rot, t_inv, interleaved=inter), tok, q_out, p.ws)
    assert p.status() == 0
    for i, (L, n) in enumerate(((37, 37), (50, 20))):
        at = np.arange(L - n, L)
        page, slot = p.table[i, at // 16], at % 16
        want = q4.bf16(q4.rotate(t.k[i, :n], pos[i, :n], inv, rot, inter))
        np.testing.assert_array_equal(f64(k)[page, :, slot], want)
        q = q4.rotate(t.q[i, :n], pos[i, :n], inv, rot, inter)
        tol = np.abs(q) * 2.0 ** -8 + 2.0 ** -20 * 2 * np.abs(t.q[i, :n]).max()
        assert (np.abs(f64(q_out)[i, :n] - q) <= tol).all()


def test_expand_to_pages_aligned_to_16_bytes(cuda_device):
    p = Problem(21, [100, 3], 4, 2, 64, 16, cuda_device)
    n = p.num_pages * 2 * 16 * 64
    want_k, want_v = (torch.zeros(n, dtype=torch.bfloat16, device=cuda_device) for _ in range(2))
    raw = torch.zeros(2, n + 64, dtype=torch.bfloat16, device=cuda_device)
    k, v = raw[0, 8:8 + n], raw[1, 8:8 + n]
    assert k.data_ptr() % 32 == 16
    R.resa_expand_q4(p.cfg, p.cache4(), want_k, want_v, p.ws)
    R.resa_expand_q4(p.cfg, p.cache4(), k, v, p.ws)
    assert torch.equal(k, want_k) and torch.equal(v, want_v) and p.status() == 0
    assert (raw[:, :8] == 0).all() and (raw[:, 8 + n:] == 0).all()


SPLITS = [  # layout, lens, width of the table in keys: whole units, even shares, the line of blocks
    ((28, 4, 128, 16), [5, 700, 1900], 2048),
    ((28, 4, 128, 16), [5, 700, 1900], 40000),
    ((32, 2, 64, 32), [1, 64, 3000, 9], 40000),
    ((16, 8, 128, 16), [1 + 7 * i for i in range(40)], 40000),       # more units than SMs
    ((8, 8, 64, 64), [3000] + [2 + i for i in range(17)], 40000),    # one long unit among short ones
    ((14, 2, 128, 16), [20000, 1, 19999], 20100),
    ((16, 8, 64, 32), [1 + 9 * i for i in range(60)], 9600),         # more units than threads
    ((32, 2, 64, 16), [900 - 6 * i for i in range(140)], 9600),
]


@pytest.mark.parametrize("case", range(len(SPLITS)))
def test_attention_splits(cuda_device, case):
    """The same rows whichever way the units are shared out among the CTAs."""
    (hq, hkv, d, b), lens, width = SPLITS[case]
    extra = max(0, width // b - (-(-max(lens) // b)))
    p = Problem(61 + case, lens, hq, hkv, d, b, cuda_device, extra_pages=extra)
    q = q4.bf16(p.rng.standard_normal((len(lens), hq, d)))
    tq = torch.from_numpy(q).to(cuda_device).bfloat16()
    out, lse = chunk(p, 1, None, tq.unsqueeze(1).contiguous())
    assert p.status() == 0
    for i in sorted({0, 1, len(lens) // 2, len(lens) - 1}):
        for h in range(hkv):
            r = slice(h * p.g, (h + 1) * p.g)
            check_rows(p, out[i, 0, r], lse[i, 0, r], q[i, r], i, h, None, np.full(p.g, lens[i]))
    o2, l2 = chunk(p, 1, None, tq.unsqueeze(1).contiguous())
    assert np.array_equal(out, o2) and np.array_equal(lse, l2)


CLUSTERS = [  # layout, lens, width of the table in keys, rows a sequence: units of 8, 4 and 2 CTAs
    ((28, 4, 128, 16), [1, 383, 385, 6001], 6016, 1),
    ((28, 4, 128, 16), [4000, 2, 17, 400, 1600, 3999, 769], 4000, 1),
    ((28, 4, 128, 16), [1 + 150 * i for i in range(13)], 2000, 1),
    ((32, 2, 64, 32), [3, 1500, 4095], 4096, 1),
    ((32, 2, 64, 32), [2 + 180 * i for i in range(11)], 2048, 1),
    ((32, 2, 128, 16), [1000 - 31 * i for i in range(30)], 1008, 1),
    ((8, 8, 64, 64), [5000], 5120, 7),
    ((14, 2, 128, 16), [2, 2500, 771], 2512, 2),
]


@pytest.mark.parametrize("case", range(len(CLUSTERS)))
def test_attention_clusters(cuda_device, case):
    """Units that a thread-block cluster shares, some of its CTAs without a key."""
    (hq, hkv, d, b), lens, width, f = CLUSTERS[case]
    p = Problem(161 + case, lens, hq, hkv, d, b, cuda_device, extra_pages=width // b - (-(-max(lens) // b)))
    q = q4.bf16(p.rng.standard_normal((len(lens), f, hq, d)))
    tq = torch.from_numpy(q).to(cuda_device).bfloat16()
    out, lse = chunk(p, f, None, tq)
    assert p.status() == 0
    limit = np.repeat(np.arange(f), p.g)
    for i in sorted({0, 1 % len(lens), len(lens) // 2, len(lens) - 1}):
        for h in range(hkv):
            rows = lambda x: x[i, :, h * p.g:(h + 1) * p.g].reshape((-1,) + x.shape[3:])
            check_rows(p, rows(out), rows(lse), rows(q), i, h, None, lens[i] - f + 1 + limit)
    o2, l2 = chunk(p, f, None, tq)
    assert np.array_equal(out, o2) and np.array_equal(lse, l2)


@pytest.mark.parametrize("layout,lens,f", [((28, 4, 128, 16), [3000, 130, 900], 40),
                                           ((16, 8, 64, 32), [70 + 40 * i for i in range(24)], 20)],
                         ids=["few", "many"])
def test_chunk_large_logits_and_splits(cuda_device, layout, lens, f):
    """The running maximum grows in the middle of a sequence; units shared among CTAs or many a CTA."""
    hq, hkv, d, b = layout
    p = Problem(72, lens, hq, hkv, d, b, cuda_device, max_chunk=f, key_size=4.0, extra_pages=60)
    q = q4.bf16(p.rng.standard_normal((len(lens), f, hq, d)) * 6)
    out, lse = chunk(p, f, None, torch.from_numpy(q).to(cuda_device).bfloat16())
    assert p.status() == 0
    for i in sorted({0, 1, len(lens) - 1}):
        limit = np.repeat(np.arange(lens[i] - f, lens[i]) + 1, p.g)
        for h in range(0, hkv, 3):
            r = slice(h * p.g, (h + 1) * p.g)
            check_rows(p, out[i, :, r].reshape(-1, d), lse[i, :, r].reshape(-1),
                       q[i, :, r].reshape(-1, d), i, h, None, limit)


def test_queries_of_every_size(cuda_device):
    """Rows of zeros, of bf16's smallest and of large values, in one call each way."""
    p = Problem(73, [600], 8, 1, 128, 16, cuda_device, max_chunk=16)
    size = np.array([0.0, 1e-38, 1e-30, 1e-10, 1.0, 30.0, 100.0, 1e-3])
    for f in (1, 16):
        q = q4.bf16(p.rng.standard_normal((1, f, 8, 128)) * size[:, None])
        out, lse = chunk(p, f, None, torch.from_numpy(q).to(cuda_device).bfloat16())
        assert p.status() == 0
        limit = np.repeat(np.arange(600 - f, 600) + 1, 8)
        check_rows(p, out[0].reshape(-1, 128), lse[0].reshape(-1), q[0].reshape(-1, 128), 0, 0, None, limit)


def test_non_finite_values_stay_in_their_rows(cuda_device):
    """A NaN query row gives NaN, a NaN group scale the rows that see it; the others are untouched."""
    p = Problem(74, [200, 300], 8, 2, 64, 16, cuda_device, max_chunk=10)
    for f in (1, 10):
        q = torch.randn(2, f, 8, 64, device=cuda_device).bfloat16()
        good, _ = chunk(p, f, None, q)
        bad = q.clone()
        bad[0, 0, 1, 3] = float("nan")
        out, lse = chunk(p, f, None, bad)
        assert np.isnan(out[0, 0, 1]).all() and np.isnan(lse[0, 0, 1])
        out[0, 0, 1] = good[0, 0, 1]
        assert np.array_equal(out, good)
    sf = p.k_sf.view(torch.uint8)
    page = int(p.table[1, 5])
    keep = sf[page, 0, 3, 0].item()
    sf[page, 0, 3, 0] = 0x7f
    out, _ = chunk(p, 1, None, q[:, :1].contiguous())
    sf[page, 0, 3, 0] = keep
    ref, _ = chunk(p, 1, None, q[:, :1].contiguous())
    assert np.isnan(out[1, 0, :4]).all()
    out[1, 0, :4] = ref[1, 0, :4]
    assert np.array_equal(out, ref) and p.status() == 0


def test_two_streams_with_a_workspace_each(cuda_device):
    """Calls on two streams at once, each with its own workspace and outputs."""
    dev = cuda_device
    ps = [Problem(75 + i, [3000, 500], 28, 4, 128, 16, dev, max_chunk=12, extra_pages=2000) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in ps]
    data = []
    for p in ps:
        q = torch.randn(2, 12, 28, 128, device=dev).bfloat16()
        data.append((q, torch.zeros(2, 12, 28, 128, device=dev), torch.zeros(2, 28, 128, device=dev)))
    want = []
    for p, (q, out, o1) in zip(ps, data):
        R.resa_attention_q4(p.cfg, p.cache4(), 12, None, q, out, None, p.ws)
        R.resa_attention_q4(p.cfg, p.cache4(), 1, None, q[:, 0].contiguous(), o1, None, p.ws)
        want.append((out.clone(), o1.clone()))
    torch.cuda.synchronize()
    firsts = [q[:, 0].contiguous() for q, _, _ in data]
    torch.cuda.synchronize()
    for _ in range(10):
        for p, s, (q, out, o1), q1 in zip(ps, streams, data, firsts):
            R.resa_attention_q4(p.cfg, p.cache4(), 12, None, q, out, None, p.ws, stream=s)
            R.resa_attention_q4(p.cfg, p.cache4(), 1, None, q1, o1, None, p.ws, stream=s)
    torch.cuda.synchronize()
    for p, (_, out, o1), (a, b) in zip(ps, data, want):
        assert torch.equal(out, a) and torch.equal(o1, b) and p.status() == 0


def test_layer_cache_q4_from_nothing(cuda_device):
    """The holder: an empty cache, tokens appended in two calls, selection and attention on it."""
    from block_sparse_long_resa_b200.cache import LayerCacheQ4, workspace
    dev = cuda_device
    table = torch.arange(12, dtype=torch.int32, device=dev).view(2, 6).flip(1).contiguous()
    lc = LayerCacheQ4.empty(12, 2, 16, 64, table, k_scale=torch.full((2,), 0.5, device=dev))
    cfg = R.make_config(4, 2, 64, 16)
    ws = workspace(cfg, lc.batch, lc.max_pages, 0, dev)
    rng = np.random.default_rng(76)
    k = q4.bf16(rng.standard_normal((2, 50, 2, 64)))
    v = q4.bf16(rng.standard_normal((2, 50, 2, 64)))
    up = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(dev).bfloat16()
    for a, e in ((0, 41), (41, 50)):
        tk, tv = up(k[:, a:e]), up(v[:, a:e])
        lc.seq_len.fill_(e)
        R.resa_append_rope_q4(cfg, lc.struct(), R.make_rope(0, None), R.make_tokens(None, tk, tv), None, ws)
    q = up(rng.standard_normal((2, 4, 64)))
    topk = torch.full((2,), 9, dtype=torch.int32, device=dev)     # every block
    idx = torch.zeros(2, 2, 10, dtype=torch.int32, device=dev)
    cnt = torch.zeros(2, 2, dtype=torch.int32, device=dev)
    R.resa_select_blocks(cfg, lc.select_struct(), q, topk, 9, idx, cnt, None, ws)
    assert cnt.tolist() == [[4, 4]] * 2
    a, b = torch.zeros(2, 4, 64, device=dev), torch.zeros(2, 4, 64, device=dev)
    R.resa_sparse_decode_q4(cfg, lc.struct(), q, idx, cnt, 9, a, None, ws)
    R.resa_attention_q4(cfg, lc.struct(), 1, None, q, b, None, ws)
    assert torch.equal(a, b)                                       # the same blocks in the same order
    assert R.resa_check_device_status(ws, raise_on_error=False) == 0
    for i in range(2):
        for h in range(2):
            kc, ks = q4.quantise(k[i, :, h], np.full((50, 1), 0.5, np.float32))
            vc, vs = q4.quantise(v[i, :, h], np.ones((50, 1), np.float32))
            o, _, w, mag, vsum = q4.attention(f64(q)[i, 2 * h:2 * h + 2], q4.values(kc, ks) * 0.5,
                                              q4.values(vc, vs), [50, 50], 0.125)
            tol, _ = attention_tolerance(mag[:, None], 50, w, vsum)
            assert (np.abs(f64(a)[i, 2 * h:2 * h + 2] - o) <= tol).all()


def test_pages_past_four_gigabytes(cuda_device):
    """Byte offsets past 32 bits (and element offsets, in the bf16 pages): the last pages of large
    pools hold what the pages of small ones do."""
    dev = cuda_device
    hq, hkv, d, b, f = 16, 8, 128, 64, 130
    lens = torch.tensor([200, 130], dtype=torch.int32, device=dev)
    torch.manual_seed(77)
    q, k, v = (torch.randn(2, f, h, d, device=dev).bfloat16() for h in (hq, hkv, hkv))
    q1 = torch.randn(2, hq, d, device=dev).bfloat16()
    inv = torch.tensor(1e4 ** (-np.arange(0, d, 2) / d), dtype=torch.float32, device=dev)
    idx = torch.tensor([[[3, 0]] * hkv, [[1, 2]] * hkv], dtype=torch.int32, device=dev)
    cnt = torch.full((2, hkv), 2, dtype=torch.int32, device=dev)
    cfg, got = R.make_config(hq, hkv, d, b), []
    for pages in (8, 132000):                                    # 32 KB of codes a page: 4.3 GB
        p4 = [torch.zeros(pages, hkv, b, d // 2, dtype=torch.uint8, device=dev) for _ in range(2)]
        sf = [torch.zeros(pages, hkv, b, d // 16, dtype=torch.uint8, device=dev) for _ in range(2)]
        p16 = [torch.zeros(pages, hkv, b, d, dtype=torch.bfloat16, device=dev) for _ in range(4)]
        desc = [torch.zeros(pages, hkv, 2, d, dtype=torch.bfloat16, device=dev) for _ in range(2)]
        table = (pages - 1 - torch.arange(8, dtype=torch.int32, device=dev)).view(2, 4).contiguous()
        ws = R_workspace(cfg, 2, 4, f, dev)
        c4 = R.make_cache_q4(p4[0], sf[0], p4[1], sf[1], desc[0], table, lens)
        c16 = R.make_cache(p16[0], p16[1], desc[1], table, lens)
        rope, toks = R.make_rope(d, inv), R.make_tokens(q, k, v)
        qa, qb = torch.zeros_like(q), torch.zeros_like(q)
        R.resa_append_rope_q4(cfg, c4, rope, toks, qa, ws)
        R.resa_append_rope(cfg, c16, rope, toks, qb, ws)
        R.resa_expand_q4(cfg, c4, p16[2], p16[3], ws)
        o, o1, o2 = (torch.zeros(2, n, hq, d, device=dev) for n in (f, 1, 1))
        R.resa_attention_q4(cfg, c4, f, None, qa, o, None, ws)
        R.resa_attention_q4(cfg, c4, 1, None, q1, o1, None, ws)
        R.resa_sparse_decode_q4(cfg, c4, q1, idx, cnt, 1, o2, None, ws)
        assert R.resa_check_device_status(ws, raise_on_error=False) == 0
        got.append([x[pages - 8:].clone() for x in p4 + sf + p16 + desc] + [qa, qb, o, o1, o2])
        del p4, sf, p16, desc, c4, c16
    for x, y in zip(*got):
        assert torch.equal(x, y)
    assert all(x.abs().float().max() > 0 for x in got[0])


@pytest.mark.parametrize("width", [512, 2000, 40000], ids=["whole", "cluster", "grid"])
def test_captured_decode_with_a_bad_sequence(cuda_device, width):
    """Every way of sharing units out, captured and replayed: a sequence whose length is out of
    range is reported and skipped (dense) or zeroed (sparse), the others keep their results."""
    dev = cuda_device
    p = Problem(78, [500, 37, 400], 28, 4, 128, 16, dev, extra_pages=width // 16 - 32)
    q = torch.randn(3, 28, 128, device=dev).bfloat16()
    lens = p.t_len.clone()
    most = width // 16 - 1
    idx = torch.arange(most + 1, dtype=torch.int32, device=dev).expand(3, 4, most + 1).contiguous()
    cnt = torch.tensor([[32] * 4, [3] * 4, [25] * 4], dtype=torch.int32, device=dev)
    c4 = p.cache4(seq_len=lens)
    a, b = torch.zeros(3, 28, 128, device=dev), torch.zeros(3, 28, 128, device=dev)
    za, zb = torch.zeros(3, 28, device=dev), torch.zeros(3, 28, device=dev)

    def calls():
        R.resa_attention_q4(p.cfg, c4, 1, None, q, a, za, p.ws)
        R.resa_sparse_decode_q4(p.cfg, c4, q, idx, cnt, most, b, zb, p.ws)

    calls()
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(za, zb) and p.status() == 0
    want, wantz = a.clone(), za.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    lens[1] = -1
    for x in (a, b, za, zb):
        x.fill_(7.0)
    g.replay()
    assert p.status() & 0x1f != 0
    for got, z, at_bad, z_bad in ((a, za, 7.0, 7.0), (b, zb, 0.0, -np.inf)):
        for i in (0, 2):
            assert torch.equal(got[i], want[i]) and torch.equal(z[i], wantz[i])
        assert (got[1] == at_bad).all() and (z[1] == z_bad).all()
    R.resa_workspace_init(p.ws)
    lens[1] = 37
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want) and p.status() == 0
