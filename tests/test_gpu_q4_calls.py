"""Calls of the 4-bit cache's entry points that a program may make around them: structs over
temporaries, memory of other kinds, long pieces of work, many units."""
import numpy as np
import pytest
import torch

from block_sparse_long_resa_b200 import resa as R
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
