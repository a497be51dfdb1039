"""Calls of the 4-bit cache's entry points that a program may make around them: structs over
temporaries, memory of other kinds, long pieces of work, many units."""
import numpy as np
import pytest
import torch

from block_sparse_long_resa_b200 import resa as R
from block_sparse_long_resa_b200.cache import workspace
from oracle import q4
from q4_problem import Problem, f64
from test_gpu_q4 import check_rows

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
