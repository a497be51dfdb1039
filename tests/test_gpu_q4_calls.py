"""Calls of the 4-bit cache's entry points that a program may make around them: structs over
temporaries, memory of other kinds, long pieces of work, many units."""
import numpy as np
import pytest
import torch

from block_sparse_long_resa_b200 import resa as R
from block_sparse_long_resa_b200.cache import workspace
from oracle import q4
from q4_problem import Problem, f64
from test_gpu_q4 import check_rows, ids

pytestmark = pytest.mark.gpu


def test_struct_over_temporary_lengths(cuda_device):
    """Lengths made for one call, memory of their size taken and filled before it: the call reads
    the lengths, reports the sequence without a length and keeps the others' results."""
    dev = cuda_device
    p = Problem(301, [100, 100, 70], 8, 2, 64, 16, dev)
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    q = q4.bf16(p.rng.standard_normal((3, 8, 64)))
    tq = torch.from_numpy(q).to(dev).bfloat16()
    idx = t([[[0, 3, 6]] * 2, [[0, 1, 6]] * 2, [[2, 3, 4]] * 2])
    cnt = t([[3, 3]] * 3)
    out, lse = torch.full((3, 8, 64), 3.0, device=dev), torch.full((3, 8), 3.0, device=dev)
    c4 = p.cache4(seq_len=t([0, 100, 70]))
    over = [torch.full((3,), 1, dtype=torch.int32, device=dev) for _ in range(8)]
    R.resa_sparse_decode_q4(p.cfg, c4, tq, idx, cnt, 2, out, lse, p.ws)
    assert p.status() == R.DEVERR_SEQ_LEN
    assert (out[0] == 0).all() and (lse[0] == -np.inf).all()
    for i in (1, 2):
        for h in range(2):
            r = slice(4 * h, 4 * h + 4)
            check_rows(p, f64(out)[i, r], f64(lse)[i, r], q[i, r], i, h, idx[i, h].cpu().numpy(), None)
    assert all((x == 1).all() for x in over)


def test_sequence_of_two_to_the_31_keys(cuda_device):
    """The longest sequence that the header allows, over a few pages that repeat: a decode step, a
    chunk and an append at its end."""
    dev = cuda_device
    hq, d, b, few = 8, 64, 64, 64
    p = Problem(302, [few * b], hq, 1, d, b, dev, spare=0, extra_pages=0)
    pages = (2 ** 31 - 1) // b
    L = pages * b
    table = torch.from_numpy(p.table[0]).to(dev).repeat(-(-pages // few))[:pages].view(1, pages).contiguous()
    lens = torch.tensor([L], dtype=torch.int32, device=dev)
    ws = workspace(p.cfg, 1, pages, 3, dev)
    c4 = R.make_cache_q4(p.k4, p.k_sf, p.v4, p.v_sf, p.desc, table, lens, k_scale=p.t_gk, v_scale=p.t_gv)
    k, v, _ = p.keys_values(0, 0)
    times = np.full(few * b, pages // few, dtype=float)
    times[:pages % few * b] += 1                              # how often a key stands in the sequence
    # a row's sum grows by a tile of 128 keys at a time, 2^24 tiles over 148 CTAs, each addition off
    # by 2^-24 of it at most; the same of O.  (Weights, logits and merges: below a thousandth of it.)
    tol = 1.01 * (2 ** 24 / 148 + 1) * 2.0 ** -24
    for f in (1, 3):
        q = q4.bf16(p.rng.standard_normal((f, hq, d)))
        out = torch.full((f, hq, d), 3.0, device=dev)
        lse = torch.full((f, hq), 3.0, device=dev)
        R.resa_attention_q4(p.cfg, c4, f, None, torch.from_numpy(q).to(dev).bfloat16(), out, lse, ws)
        assert R.resa_check_device_status(ws, raise_on_error=False) == 0
        for r in range(f):
            n = times.copy()
            for pos in range(L - f + r + 1, L):
                n[pos % (few * b)] -= 1
            x = q[r] @ k.T * d ** -0.5
            w = np.exp(x - x.max(1, keepdims=True)) * n
            z = w.sum(1, keepdims=True)
            assert (np.abs(f64(out)[r] - w @ v / z) <= 2 * tol * (w @ np.abs(v) / z)).all()
            assert (np.abs(f64(lse)[r] - (x.max(1) + np.log(z[:, 0]))) <= tol + 2.0 ** -20).all()
    # three tokens at its end go where they go at the end of the pages' first run
    t = torch.randn(1, 3, 1, d, device=dev).bfloat16()
    blk = (pages - 1) % few
    short = torch.tensor([(blk + 1) * b], dtype=torch.int32, device=dev)
    got = []
    for at in (p.cache4(seq_len=short), c4):
        for x in (p.k4, p.v4, p.desc):
            x.zero_()
        R.resa_append_rope_q4(p.cfg, at, R.make_rope(0, None), R.make_tokens(None, t, t), None, ws if at is c4 else p.ws)
        got.append([x.clone() for x in (p.k4, p.v4, p.k_sf.view(torch.uint8), p.v_sf.view(torch.uint8), p.desc)])
    assert R.resa_check_device_status(ws, raise_on_error=False) == 0 and p.status() == 0
    assert all(torch.equal(x, y) for x, y in zip(*got)) and got[0][0].any()


# --------------------------------------------------------------- long pieces of work, many units

class Codes:
    """A 4-bit cache of random codes and group scales over pages in random order, with logits spread
    so far that a few keys take a row's weight: one tile read from a wrong page shows."""

    def __init__(self, seed, lens, hq, hkv, d, b, dev, max_chunk=0, width=0):
        self.rng = rng = np.random.default_rng(seed)
        self.lens, self.hq, self.hkv, self.d, self.b, self.g, self.dev = lens, hq, hkv, d, b, hq // hkv, dev
        need = [-(-L // b) for L in lens]
        n, self.max_pages = sum(need), max(max(need), width // b)
        order, at = rng.permutation(n).astype(np.int32), 0
        self.table = np.full((len(lens), self.max_pages), n + 5, dtype=np.int32)
        for i, m in enumerate(need):
            self.table[i, :m] = order[at:at + m]
            at += m
        codes = lambda: rng.integers(0, 256, (n, hkv, b, d // 2), dtype=np.uint8)
        scales = lambda lo, hi: rng.integers(lo, hi, (n, hkv, b, d // 16), dtype=np.uint8)
        self.k, self.v, self.ks, self.vs = codes(), codes(), scales(0x28, 0x38), scales(0x20, 0x30)
        up = lambda x: torch.from_numpy(x).to(dev)
        self.cfg = R.make_config(hq, hkv, d, b)
        self.c4 = R.make_cache_q4(up(self.k), up(self.ks), up(self.v), up(self.vs),
                                  torch.zeros(n, hkv, 2, d, dtype=torch.bfloat16, device=dev), up(self.table),
                                  torch.tensor(lens, dtype=torch.int32, device=dev))
        self.ws = workspace(self.cfg, len(lens), self.max_pages, max_chunk, dev)

    def queries(self, *shape):
        return q4.bf16(self.rng.standard_normal((*shape, self.d)) * 3)

    def keys_values(self, i, h, blocks=None):
        L, b = self.lens[i], self.b
        blocks = np.arange(-(-L // b)) if blocks is None else np.asarray(blocks)
        pos = (blocks[:, None] * b + np.arange(b)).ravel()
        pos = pos[pos < L]
        page, slot = self.table[i, pos // b], pos % b
        k = q4.values(q4.unpack(self.k[page, h, slot]), self.ks[page, h, slot])
        return k, q4.values(q4.unpack(self.v[page, h, slot]), self.vs[page, h, slot]), pos

    def attention(self, f, q, fresh=None):
        n = len(self.lens)
        out = torch.full((n, f, self.hq, self.d), 3.0, device=self.dev)
        lse = torch.full((n, f, self.hq), 3.0, device=self.dev)
        t_n = None if fresh is None else torch.tensor(fresh, dtype=torch.int32, device=self.dev)
        R.resa_attention_q4(self.cfg, self.c4, f, t_n, torch.from_numpy(q).to(self.dev).bfloat16(), out, lse, self.ws)
        assert R.resa_check_device_status(self.ws, raise_on_error=False) == 0
        return f64(out), f64(lse)

    def check(self, out, lse, q, i, h, n):
        rows = lambda x: x[i, :n, h * self.g:(h + 1) * self.g].reshape((-1,) + x.shape[3:])
        limit = np.repeat(np.arange(self.lens[i] - n, self.lens[i]) + 1, self.g)
        check_rows(self, rows(out), rows(lse), rows(q), i, h, None, limit)


@pytest.mark.parametrize("layout", [(16, 8, 128, 16), (128, 8, 64, 16), (24, 8, 64, 64)], ids=ids)
def test_many_units_of_middling_length_whole(cuda_device, layout):
    """Units for most SMs, each a CTA's: up to 22 steps a warp with 12 warps, 32 with 8, so that the
    places of a piece's tiles are fetched anew on the way."""
    hq, hkv, d, b = layout
    lens = [8100 - 530 * i for i in range(15)] + [8191]
    p = Codes(310, lens, hq, hkv, d, b, cuda_device, width=8192)
    q = p.queries(16, 1, hq)
    out, lse = p.attention(1, q)
    for i in (0, 1, 7, 14, 15):
        for h in (0, 3, 7):
            p.check(out, lse, q, i, h, 1)


@pytest.mark.parametrize("layout", [(32, 8, 64, 16), (128, 8, 64, 32)], ids=ids)
def test_long_pieces_over_the_grid(cuda_device, layout):
    """About 7000 keys a CTA (18 steps a warp with 12 warps, 27 with 8): every position, all blocks
    listed in random order, and a chunk of 55 tiles a CTA."""
    hq, hkv, d, b = layout
    L = 130021
    p = Codes(320, [L], hq, hkv, d, b, cuda_device, max_chunk=9)
    q = p.queries(1, 9, hq)
    for f in (1, 9):
        qf = np.ascontiguousarray(q[:, :f])
        out, lse = p.attention(f, qf)
        for h in range(hkv):
            p.check(out, lse, qf, 0, h, f)
    nb = -(-L // b)
    lists = np.stack([p.rng.permutation(nb) for _ in range(hkv)]).astype(np.int32)[None]
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(cuda_device)
    out = torch.zeros(1, hq, d, device=cuda_device)
    lse = torch.zeros(1, hq, device=cuda_device)
    R.resa_sparse_decode_q4(p.cfg, p.c4, t(q[:, 0]).bfloat16(), t(lists), torch.full((1, hkv), nb, dtype=torch.int32, device=cuda_device),
                            nb - 1, out, lse, p.ws)
    assert R.resa_check_device_status(p.ws, raise_on_error=False) == 0
    for h in range(hkv):
        r = slice(h * p.g, (h + 1) * p.g)
        check_rows(p, f64(out)[0, r], f64(lse)[0, r], q[0, 0, r], 0, h, np.arange(nb), None)


@pytest.mark.parametrize("layout,lens,f", [
    ((32, 8, 128, 16), [1500 - 3 * i for i in range(16)], 6),          # pieces of 10 tiles, 16-token pages
    ((16, 8, 64, 16), [20 + 7 * i for i in range(50)], 20),            # 400 units, one row group each
    ((16, 8, 64, 32), [200 + 61 * i for i in range(30)], 200),         # 480 units of two row groups
    ((4, 2, 128, 16), [9000, 130, 4000, 131, 132, 2500], 130),         # unequal: units that begin inside a share
    ((14, 2, 64, 64), [300] * 60 + [9000], 40),
], ids=lambda x: str(x) if isinstance(x, int) else "-".join(map(str, x[:4])))
def test_chunks_of_long_pieces_and_many_units(cuda_device, layout, lens, f):
    """The chunk kernel where a piece's pages take several fetches, where there are more units than
    threads, and where shares begin and end inside units."""
    hq, hkv, d, b = layout
    p = Codes(330, lens, hq, hkv, d, b, cuda_device, max_chunk=f)
    fresh = [min(f, L) - (i % 3 if L > f else 0) for i, L in enumerate(lens)]
    fresh[1] = min(fresh[1], 3)
    q = p.queries(len(lens), f, hq)
    out, lse = p.attention(f, q, fresh)
    for i in sorted({0, 1, 2, len(lens) // 2, len(lens) - 2, len(lens) - 1}):
        assert (out[i, fresh[i]:] == 3.0).all() and (lse[i, fresh[i]:] == 3.0).all()
        for h in sorted({0, hkv // 2, hkv - 1}):
            p.check(out, lse, q, i, h, fresh[i])
    o2, l2 = p.attention(f, q, fresh)
    assert np.array_equal(out, o2) and np.array_equal(lse, l2)


@pytest.mark.parametrize("f", [1, 2])
def test_small_weights_beside_a_large_one(cuda_device, f):
    """Two keys, the first with nearly all the weight and values of zero: the output is the second's
    weight times its values, down to the steps that a weight is stored in.  f = 2 is the chunk kernel
    (24 rows a kv head)."""
    n, hq, d = 400, 12, 64
    p = Codes(340, [2] * n, hq, 1, d, 16, cuda_device, max_chunk=f)
    first = p.table[:, 0]
    p.k[first, 0, 0], p.k[first, 0, 1], p.v[first, 0, 0] = 0x77, 0x11, 0    # codes of 6, 0.5 and 0
    p.ks[first, 0, :2] = 0x38                                               # times 1
    for x, y in ((p.c4.tensors[0], p.k), (p.c4.tensors[1], p.ks), (p.c4.tensors[2], p.v)):
        x.copy_(torch.from_numpy(y))
    # logits of the first key from 14 to 24, a twelfth of that for the second
    q = q4.bf16(p.rng.uniform(14, 24, (n, f, hq, 1)) / (6 * d ** 0.5) + np.zeros(d))
    out, lse = p.attention(f, q)
    k, v = zip(*((a, b) for a, b, _ in (p.keys_values(i, 0) for i in range(n))))
    assert all((a[0] == 6).all() and (a[1] == 0.5).all() for a in k) and all((b[0] == 0).all() for b in v)
    v = np.stack(v)[:, 1][:, None]                                          # [n, 1, d]
    x = q[:, -1].sum(-1) * 6 * d ** -0.5
    y = x * 11 / 12
    want = (1 / (1 + np.exp(y)))[..., None] * v
    # 2^-36 of the row's largest weight, which is 1 here; relatively as attention_tolerance has it
    tol = np.abs(want) * (2 * 10 * 2.0 ** -22 * x[..., None] + 2.0 ** -20 + 2 * 65 * 2.0 ** -22)
    assert (np.abs(out[:, -1] - want) <= tol + 2.0 ** -36 * np.abs(v)).all()
    assert (np.abs(lse[:, -1] - (x + np.log1p(np.exp(-y)))) <= 10 * 2.0 ** -22 * x + 2.0 ** -20 + 65 * 2.0 ** -22).all()
