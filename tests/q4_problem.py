"""Problems of the 4-bit cache and of the rotary append for the tests: a pool of pages in random
order with spare pages, pages of one sequence never another's, slots past the end poisoned."""
import numpy as np
import torch

from block_sparse_long_resa_b200 import resa as R
from block_sparse_long_resa_b200.cache import workspace
from oracle import q4


def f64(t):
    return t.detach().cpu().double().numpy()


class Problem:
    """A 4-bit cache (and the bf16 pages it came from) of sequences of the given lengths."""

    def __init__(self, seed, lens, hq, hkv, d, b, dev, max_chunk=0, spare=3, extra_pages=2,
                 key_size=1.0, head_scales=True):
        rng = np.random.default_rng(seed)
        self.rng, self.dev = rng, dev
        self.hq, self.hkv, self.d, self.b, self.g = hq, hkv, d, b, hq // hkv
        self.lens = list(lens)
        batch = len(lens)
        need = [-(-max(L, 0) // b) for L in lens]
        self.max_pages = max(1, max(need)) + extra_pages
        self.num_pages = sum(need) + spare
        order = rng.permutation(self.num_pages)
        # entries past a sequence's last block are out of range: touching one is an error
        table = np.full((batch, self.max_pages), self.num_pages + 7, dtype=np.int32)
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = order[at:at + n]
            at += n
        self.table = table
        shape = (self.num_pages, hkv, b, d)
        ch = np.exp(0.5 * rng.standard_normal((hkv, 1, d))) * key_size
        self.k16 = q4.bf16(rng.standard_normal(shape) * ch)
        self.v16 = q4.bf16(rng.standard_normal(shape))
        self.gk = (np.float32(0.25) * (1 + rng.random(hkv, dtype=np.float32))) if head_scales else np.ones(hkv, np.float32)
        self.gv = (np.float32(0.25) * (1 + rng.random(hkv, dtype=np.float32))) if head_scales else np.ones(hkv, np.float32)
        self.kc, self.ks = q4.quantise(self.k16, self.gk[:, None, None])
        self.vc, self.vs = q4.quantise(self.v16, self.gv[:, None, None])
        live = np.zeros((self.num_pages, b), dtype=bool)
        for i, L in enumerate(lens):
            for j in range(need[i]):
                live[table[i, j], :max(0, min(b, L - j * b))] = True
        self.live = live
        dead = ~live[:, None, :, None].repeat(hkv, 1)
        # poison: scales of NaN (e4m3 0x7f) and full codes
        self.ks = np.where(dead, 0x7f, self.ks).astype(np.uint8)
        self.vs = np.where(dead, 0x7f, self.vs).astype(np.uint8)
        self.kc = np.where(dead, 15, self.kc).astype(np.uint8)
        self.vc = np.where(dead, 15, self.vc).astype(np.uint8)
        up = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(dev)
        self.k4, self.v4 = up(q4.pack(self.kc)), up(q4.pack(self.vc))
        self.k_sf = up(self.ks).view(torch.float8_e4m3fn)
        self.v_sf = up(self.vs).view(torch.float8_e4m3fn)
        self.t_table, self.t_len = up(table), up(np.asarray(lens, dtype=np.int32))
        self.t_gk, self.t_gv = up(self.gk), up(self.gv)
        self.desc = torch.full((self.num_pages, hkv, 2, d), 7.0, dtype=torch.bfloat16, device=dev)
        self.cfg = R.make_config(hq, hkv, d, b)
        self.ws = workspace(self.cfg, batch, self.max_pages, max_chunk, dev)

    def cache4(self, rows=None, seq_len=None):
        return R.make_cache_q4(self.k4, self.k_sf, self.v4, self.v_sf, self.desc, self.t_table,
                               self.t_len if seq_len is None else seq_len, rows=rows,
                               k_scale=self.t_gk, v_scale=self.t_gv)

    def keys_values(self, i, h, blocks=None):
        """What the cache holds of sequence i, head h (all positions, or those of the blocks):
        float64 k, v and the positions."""
        L, b = self.lens[i], self.b
        blocks = range(-(-L // b)) if blocks is None else blocks
        pos = np.concatenate([np.arange(x * b, min(L, (x + 1) * b)) for x in blocks]
                             or [np.zeros(0, int)]).astype(int)
        page, slot = self.table[i, pos // b], pos % b
        k = q4.values(self.kc[page, h, slot], self.ks[page, h, slot]) * float(self.gk[h])
        v = q4.values(self.vc[page, h, slot], self.vs[page, h, slot]) * float(self.gv[h])
        return k, v, pos

    def refresh(self):
        """Take the codes and scales as the calls left them."""
        self.kc, self.vc = (q4.unpack(x.cpu().numpy()) for x in (self.k4, self.v4))
        self.ks, self.vs = (x.view(torch.uint8).cpu().numpy() for x in (self.k_sf, self.v_sf))

    def status(self):
        return R.resa_check_device_status(self.ws, raise_on_error=False)


def attention_tolerance(mag, n, a, vsum=0.0):
    """Bounds on |out - exact|, with a = sum p |v| and vsum = sum |v|, and on |lse - exact|.

    Logits: the products are exact and at most d = 128 of them are added in fp32 in the matrix
    unit, which may drop bits below 2^-22 of the running magnitude at each of 8 steps, and the
    scaling rounds twice more: at most 10 * 2^-22 of sum |q k| = mag.  Weights: e^(2 delta) - 1,
    2^-21 for the exponential, 2^-21 for the two fp16 halves, whose absolute rounding is half of
    fp16's smallest step, 2^-25, where the row's largest weight is at least 2^11 (weights are
    scaled by 2^13 with 2 powers of slack in the maximum, or by 2^12 with 3, less one for the
    maximum's rounding up: 2^(12 - 1)): 2^-36 of |v| for every key.  Sums over n weights: one addition
    a 16-position step, split over at least 1 warp, 2^-22 each, and 64 more for the merges."""
    delta = 10 * 2.0 ** -22 * mag
    sums = (n / 16 + 64) * 2.0 ** -22
    return a * (2 * delta + 2.0 ** -20 + 2 * sums) + 2.0 ** -36 * vsum + 1e-30, delta + 2.0 ** -20 + sums
