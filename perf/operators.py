"""Cases of the rotary append and of the 4-bit paged KV cache: what is measured.

Operators (``op`` of a case):

* ``append``   rotate q and k of up to f fresh tokens a sequence and append k, v
               to the bf16 paged cache, with the block descriptors kept up to date;
* ``append4``  the same into the 4-bit cache, read back as bf16 pages
               (append, then expansion of the cache);
* ``expand4``  4-bit pages to bf16 pages;
* ``sparse4``  decode attention over listed blocks of the 4-bit cache;
* ``attn4``    causal attention of the last f tokens over every position of the
               4-bit cache (f = 1: dense decode).

4-bit format: 16 channels of one token and head form a group; with the head's
scale g and y = x / g, s = e4m3(max |y| / 6) and each channel is e2m1(y / s);
it stands for e2m1 * s * g.  Channel 2j is the low nibble of byte j.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
THETA = 1.0e6


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _case(op, name=None, **kw):
    c = dict(op=op, batch=1, f=1, hq=28, hkv=4, d=128, b=16, ctx=0, low=0, rot=128,
             interleaved=False, fused=False, ragged=False, shift=0, topk=0, empty=False)
    c.update(kw)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # one decode step of a 32-sequence batch: k and v of one token each into their pages
        _case("append", "append_step_b32", batch=32, low=100, ctx=2000, fused=True),
        # a prompt of 8192 tokens written at once, the projections' fused output read in place
        _case("append", "append_prompt_8k", f=8192, fused=True),
        # a decode step on the 4-bit cache: 32 short sequences, half-rotated heads of 64 channels
        _case("append4", "append4_step_b32", batch=32, low=33, ctx=250, hq=8, hkv=2, d=64, rot=32),
        # padded prompts of different lengths, one of them empty, blocks of 64 tokens, pairs interleaved
        _case("append4", "append4_prompts_ragged", batch=5, f=2777, low=0, ctx=111, hq=32, hkv=8,
              b=64, interleaved=True, ragged=True),
        # a short 4-bit cache handed over as bf16 pages
        _case("expand4", "expand4_2k", hq=4, hkv=2, d=64, ctx=2048),
        # four long sequences handed over for bf16 rectification
        _case("expand4", "expand4_4x65k", batch=4, low=65000, ctx=65536),
        # sparse decode of one 32K layer, a tenth of the blocks
        _case("sparse4", "sparse4_32k", ctx=32768, topk=205),
        # the same at 256K
        _case("sparse4", "sparse4_256k", ctx=262144, topk=1638),
        # continuous batch of unequal sequences, one slot without any block
        _case("sparse4", "sparse4_cbatch", batch=32, low=8192, ctx=131072, topk=1311, empty=True),
        # dense decode of one 256K layer
        _case("attn4", "attn4_dense_256k", ctx=262144),
        # dense decode of a batch with odd lengths, 16 heads a group, 64 channels, blocks of 32
        _case("attn4", "attn4_dense_b16", batch=16, low=17, ctx=9001, hq=32, hkv=2, d=64, b=32),
        # the chunk of a rectification: 32 tokens against 65536, four sequences
        _case("attn4", "attn4_chunk_4x65k", batch=4, f=32, low=65000, ctx=65536),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append4", "expand4", "sparse4", "sparse4", "attn4", "attn4", "attn4"])
    hq, hkv = rng.choice([(28, 4), (32, 8), (8, 8), (16, 1), (4, 2), (14, 2), (32, 2), (24, 8)])
    d = rng.choice([64, 128])
    kw = dict(hq=hq, hkv=hkv, d=d, b=rng.choice([16, 32, 64]), rot=rng.choice([d, d, d // 2, 48, 0]))
    if op in ("append", "append4"):
        kw["batch"] = _log(rng, 1, 64)
        kw["f"] = rng.choice([1, _log(rng, 1, max(1, 8192 // kw["batch"]))])
        kw["low"] = rng.randrange(0, 200)
        kw["ctx"] = kw["low"] + rng.randrange(0, 1500)
        kw["interleaved"] = rng.random() < 0.4
        kw["fused"] = rng.random() < 0.5
        kw["ragged"] = rng.random() < 0.5
        kw["shift"] = rng.choice([0, 0, rng.randrange(1, 1 << 20)])
    elif op == "expand4":
        kw["batch"] = _log(rng, 1, 32)
        kw["ctx"] = _log(rng, 1, 131072 // kw["batch"])
        kw["low"] = rng.randrange(1, kw["ctx"] + 1)
    elif op == "sparse4":
        kw["batch"] = _log(rng, 1, 32)
        kw["ctx"] = _log(rng, 1, min(262144, 1500000 // kw["batch"]))
        kw["low"] = rng.randrange(1, kw["ctx"] + 1)
        kw["topk"] = rng.choice([0, _log(rng, 1, max(1, kw["ctx"] // kw["b"] // 8 + 1))])
        kw["empty"] = rng.random() < 0.3
    else:
        kw["batch"] = _log(rng, 1, 24)
        kw["f"] = rng.choice([1, 1, 2, _log(rng, 2, 64), _log(rng, 32, 512)])
        kw["ctx"] = max(kw["f"], _log(rng, 1, max(1, 65536 // kw["batch"] // (1 + kw["f"] // 64))))
        kw["low"] = rng.randrange(kw["f"], kw["ctx"] + 1)
        kw["ragged"] = kw["f"] > 1 and rng.random() < 0.5
    return _case(op, **kw)


def _lengths(case):
    """(tokens in the cache before the call, fresh tokens) of each sequence: spread between
    ``low`` and ``ctx`` and, where ragged, between 0 and f."""
    n, before, fresh = case["batch"], [], []
    for i in range(n):
        t = ((i * 37 + 11) % n) / (n - 1) if n > 1 else 1.0
        before.append(case["low"] + int((case["ctx"] - case["low"]) * t))
        u = ((i * 29 + 5) % n) / (n - 1) if n > 1 else 0.7
        fresh.append(int(case["f"] * u) if case["ragged"] else case["f"])
    return before, fresh


def _total(case):
    before, fresh = _lengths(case)
    if case["op"] in ("append", "append4"):
        return [p + n for p, n in zip(before, fresh)]
    return [max(p, 1) for p in before]


def _counts(case):
    """Blocks in each sequence's list: the selected ones and the current one."""
    return [0 if case["empty"] and i == 0 else min(case["topk"], (L - 1) // case["b"]) + 1
            for i, L in enumerate(_total(case))]


def work(case):
    hq, hkv, d, b = case["hq"], case["hkv"], case["d"], case["b"]
    before, fresh = _lengths(case)
    total = _total(case)
    row4 = hkv * (d // 2 + d // 16) * 2          # a token's key and value, 4-bit
    row16 = hkv * d * 2 * 2                      # the same in bf16
    if case["op"] in ("append", "append4"):
        tokens = sum(fresh)
        blocks = sum((L - 1) // b - (L - n) // b + 1 for L, n in zip(total, fresh) if n)
        bytes_ = tokens * (hq * d * 2 * 2 + row16) + blocks * hkv * 2 * d * 2
        # the keys already in the first touched block, for its descriptor
        old = sum((L - n) % b for L, n in zip(total, fresh) if n)
        if case["op"] == "append":
            bytes_ += tokens * row16 + old * hkv * d * 2
        else:
            bytes_ += tokens * row4 + sum(total) * (row4 + row16)
        return {"bytes": bytes_, "flops": tokens * (hq + hkv) * case["rot"] * 3}
    if case["op"] == "expand4":
        return {"bytes": sum(total) * (row4 + row16), "flops": sum(total) * hkv * d * 4}
    if case["op"] == "sparse4":
        seen = sum(max(0, (c - 1) * b + (L - 1) % b + 1) if c else 0
                   for c, L in zip(_counts(case), total))
        io = case["batch"] * hq * (d * 6 + 4) + sum(_counts(case)) * hkv * 4
        return {"bytes": seen * row4 + io, "flops": 4 * hq * d * seen}
    pairs = sum(n * (L - n) + n * (n + 1) // 2 for L, n in zip(total, fresh))
    io = sum(fresh) * hq * (d * 6 + 4)
    return {"bytes": sum(L for L, n in zip(total, fresh) if n) * row4 + io,
            "flops": 4 * hq * d * pairs}


# ---------------------------------------------------------------------------
# The 4-bit format, plain
# ---------------------------------------------------------------------------

def _quantise(x, g):
    """x [..., Hkv, n, d] fp32 and the heads' scales g [Hkv]: codes uint8 [..., d / 2] and group
    scales e4m3 [..., d / 16]."""
    y = x * (1.0 / g)[:, None, None]
    y = y.unflatten(-1, (-1, 16))
    a = y.abs()
    six = torch.full((), 6.0, device=x.device)      # a tensor: a true division
    s = (a.amax(-1) / six).clamp_max(448.0).to(torch.float8_e4m3fn)
    t = s.float().unsqueeze(-1)
    code = torch.zeros(y.shape, dtype=torch.uint8, device=x.device)
    for bound, tie_up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False),
                          (3.5, True), (5.0, False)):
        code += (a >= bound * t) if tie_up else (a > bound * t)
    code = torch.where(t > 0, code, torch.zeros_like(code)) + 8 * (y < 0).to(torch.uint8)
    code = code.flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], s


def _values(codes, s):
    """What codes and scales stand for, without the head's scale, fp32."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    nib = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)
    return (lut[nib.int()].unflatten(-1, (-1, 16)) * s.float().unsqueeze(-1)).flatten(-2)


# ---------------------------------------------------------------------------
# State
# ---------------------------------------------------------------------------

def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    op, batch, f = case["op"], case["batch"], case["f"]
    hq, hkv, d, b, rot = case["hq"], case["hkv"], case["d"], case["b"], case["rot"]
    _, fresh = _lengths(case)
    total = _total(case)
    st = dict(case)
    pages = [max(1, -(-L // b)) for L in total]
    width, count = max(pages), sum(pages)
    # pages of a pool in random order
    order = torch.randperm(count, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros(batch, width, dtype=torch.int32, device=dev)
    first = 0
    for i, n in enumerate(pages):
        table[i, :n] = order[first:first + n]
        first += n
    st["table"] = table
    st["len"] = torch.tensor(total, dtype=torch.int32, device=dev)
    st["fresh"] = torch.tensor(fresh, dtype=torch.int32, device=dev) if case["ragged"] else None
    # keys have channels of unequal size, as a model's do
    kscale = torch.exp(0.5 * randn(hkv, 1, d))
    st["g"] = 0.25 * (1 + torch.rand(2, hkv, generator=gen, device=dev))
    if op == "append":
        st["k"] = (randn(count, hkv, b, d) * kscale).bfloat16()
        st["v"] = randn(count, hkv, b, d).bfloat16()
    else:
        st["k4"], st["ks"] = _quantise((randn(count, hkv, b, d) * kscale).bfloat16().float(), st["g"][0])
        st["v4"], st["vs"] = _quantise(randn(count, hkv, b, d).bfloat16().float(), st["g"][1])
    st["desc"] = torch.zeros(count, hkv, 2, d, dtype=torch.bfloat16, device=dev)
    if op in ("append4", "expand4"):
        st["k16"] = torch.zeros(count, hkv, b, d, dtype=torch.bfloat16, device=dev)
        st["v16"] = torch.zeros(count, hkv, b, d, dtype=torch.bfloat16, device=dev)
    if op in ("append", "append4"):
        q, kn, vn = randn(batch, f, hq, d), randn(batch, f, hkv, d) * kscale[:, 0], randn(batch, f, hkv, d)
        if case["fused"]:                        # views of one projection output
            x = torch.cat([q.flatten(2), kn.flatten(2), vn.flatten(2)], dim=2).bfloat16()
            st["q"] = x[..., :hq * d].unflatten(2, (hq, d))
            st["kn"] = x[..., hq * d:(hq + hkv) * d].unflatten(2, (hkv, d))
            st["vn"] = x[..., (hq + hkv) * d:].unflatten(2, (hkv, d))
        else:
            st["q"], st["kn"], st["vn"] = q.bfloat16(), kn.bfloat16(), vn.bfloat16()
        st["q_out"] = torch.zeros(batch, f, hq, d, dtype=torch.bfloat16, device=dev)
        st["inv_freq"] = THETA ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float32) / max(rot, 1))
        st["pos"] = None
        if case["shift"]:                        # positions that are not the cache's own
            p = st["len"][:, None] - (st["fresh"] if case["ragged"] else st["len"] * 0 + f)[:, None]
            st["pos"] = (p + torch.arange(f, device=dev) + case["shift"]).to(torch.int32).contiguous()
    elif op == "sparse4":
        st["q"] = randn(batch, hq, d).bfloat16()
        st["max_topk"] = case["topk"]
        n = case["topk"] + 1
        cnt = torch.tensor(_counts(case), dtype=torch.int32, device=dev)
        idx = torch.full((batch, hkv, n), -1, dtype=torch.int32, device=dev)
        for i in range(batch):
            m, c = (total[i] - 1) // b, _counts(case)[i]
            if c:
                pick = torch.rand(hkv, max(m, 1), generator=gen, device=dev)[:, :m].argsort(1)[:, :c - 1]
                idx[i, :, :c - 1] = pick.sort(1).values.int()
                idx[i, :, c - 1] = m
        st["idx"], st["cnt"] = idx, cnt[:, None].expand(batch, hkv).contiguous()
        st["out"] = torch.zeros(batch, hq, d, device=dev)
        st["lse"] = torch.zeros(batch, hq, device=dev)
    elif op == "attn4":
        st["q"] = randn(batch, f, hq, d).bfloat16()
        st["out"] = torch.zeros(batch, f, hq, d, device=dev)
        st["lse"] = torch.zeros(batch, f, hq, device=dev)
    if own:
        _handles(st, width, dev)
    return st


def _handles(st, width, dev):
    """The structs and the workspace that a program keeps beside its buffers."""
    from block_sparse_long_resa_b200 import resa as R
    from block_sparse_long_resa_b200.cache import workspace
    st["R"] = R
    st["cfg"] = R.make_config(st["hq"], st["hkv"], st["d"], st["b"])
    if st["op"] == "append":
        st["cache"] = R.make_cache(st["k"], st["v"], st["desc"], st["table"], st["len"])
    else:
        st["cache"] = R.make_cache_q4(st["k4"], st["ks"], st["v4"], st["vs"], st["desc"], st["table"],
                                      st["len"], k_scale=st["g"][0], v_scale=st["g"][1])
    if st["op"] in ("append", "append4"):
        st["rope"] = R.make_rope(st["rot"], st["inv_freq"], interleaved=st["interleaved"])
        st["tokens"] = R.make_tokens(st["q"], st["kn"], st["vn"], n_new=st["fresh"], positions=st["pos"])
    st["ws"] = workspace(st["cfg"], st["batch"], width, st["f"] if st["op"] == "attn4" else 0, dev)


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(st):
    op = st["op"]
    if own:
        R = st["R"]
        if op == "append":
            R.resa_append_rope(st["cfg"], st["cache"], st["rope"], st["tokens"], st["q_out"], st["ws"])
        elif op == "append4":
            R.resa_append_rope_q4(st["cfg"], st["cache"], st["rope"], st["tokens"], st["q_out"], st["ws"])
            R.resa_expand_q4(st["cfg"], st["cache"], st["k16"], st["v16"], st["ws"])
        elif op == "expand4":
            R.resa_expand_q4(st["cfg"], st["cache"], st["k16"], st["v16"], st["ws"])
        elif op == "sparse4":
            R.resa_sparse_decode_q4(st["cfg"], st["cache"], st["q"], st["idx"], st["cnt"], st["max_topk"],
                                    st["out"], st["lse"], st["ws"])
        else:
            R.resa_attention_q4(st["cfg"], st["cache"], st["f"], st["fresh"], st["q"], st["out"],
                                st["lse"], st["ws"])
    elif op == "append":
        _append(st, st["k"], st["v"])
    elif op == "append4":
        _expand(st)
        _append(st, st["k16"], st["v16"])
    elif op == "expand4":
        _expand(st)
    elif op == "sparse4":
        _sparse(st)
    else:
        _attention(st)
    if op == "append":
        return {"q": st["q_out"], "k": st["k"], "v": st["v"], "desc": st["desc"]}
    if op == "append4":
        return {"q": st["q_out"], "k": st["k16"], "v": st["v16"], "desc": st["desc"]}
    if op == "expand4":
        return {"k": st["k16"], "v": st["v16"]}
    return {"out": st["out"], "lse": st["lse"]}


def _rotate(x, pos, st):
    """x [batch, f, heads, d] bf16 rotated by its positions; angles and products in 64 bits."""
    rot = st["rot"]
    if rot == 0:
        return x
    ang = pos.double()[..., None] * st["inv_freq"].double()
    c, s = ang.cos()[:, :, None], ang.sin()[:, :, None]
    y = x[..., :rot].double()
    if st["interleaved"]:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:]
        y = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    return torch.cat([y.float().bfloat16(), x[..., rot:]], dim=-1)


def _append(st, kp, vp):
    """Writes the rotated q, the fresh keys and values (kp, vp: the bf16 pages) and the descriptors."""
    f, b = st["f"], st["b"]
    n = st["fresh"] if st["fresh"] is not None else torch.full_like(st["len"], f)
    r = torch.arange(f, device=n.device)
    slot = (st["len"] - n)[:, None] + r                          # position in the cache
    live = r < n[:, None]
    pos = st["pos"] if st["pos"] is not None else slot
    st["q_out"][live] = _rotate(st["q"], pos, st)[live]
    k = _rotate(st["kn"], pos, st)[live]
    v = st["vn"][live]
    page = st["table"].gather(1, (slot // b).clamp(0, st["table"].shape[1] - 1).long())[live]
    if st["op"] == "append4":                                    # stored in 4 bits, read back
        k = _stored(k, st["g"][0])
        v = _stored(v, st["g"][1])
    at = page.long() * b + (slot % b)[live]
    kp.transpose(1, 2)[at // b, at % b] = k
    vp.transpose(1, 2)[at // b, at % b] = v
    # descriptors of the touched blocks, over their positions below the length
    blk = ((st["len"] - n) // b)[:, None] + torch.arange(f // b + 2, device=n.device)
    touched = (blk <= ((st["len"] - 1) // b)[:, None]) & (n > 0)[:, None]
    which = st["table"].gather(1, blk.clamp(0, st["table"].shape[1] - 1).long())[touched].long()
    inside = blk[touched][:, None] * b + torch.arange(b, device=n.device) < \
        st["len"][:, None].expand_as(blk)[touched][:, None]
    keys = kp[which].float()
    hide = ~inside[:, None, :, None]
    lo = keys.masked_fill(hide, math.inf).amin(2)
    hi = keys.masked_fill(hide, -math.inf).amax(2)
    st["desc"][which] = torch.stack([lo, hi], dim=2).bfloat16()


def _stored(x, g):
    """What the 4-bit cache holds of tokens x [n, Hkv, d], as bf16."""
    codes, s = _quantise(x.float().unsqueeze(-2), g)
    return (_values(codes, s) * g[:, None, None]).squeeze(-2).bfloat16()


def _expand(st):
    b = st["b"]
    at = torch.arange(st["table"].shape[1], device=st["table"].device)
    live = at < ((st["len"] + b - 1) // b)[:, None]
    pages = st["table"][live].long()
    inside = (at[:, None] * b + torch.arange(b, device=at.device)) < st["len"][:, None, None]
    inside = inside[live][:, None, :, None]
    for to, codes, s, g in (("k16", "k4", "ks", 0), ("v16", "v4", "vs", 1)):
        x = (_values(st[codes][pages], st[s][pages]) * st["g"][g][:, None, None]).bfloat16()
        st[to][pages] = torch.where(inside, x, st[to][pages])


def _softmax_av(q, k, v, seen, scale):
    """q [..., rows, d], k, v [..., n, d], seen [..., rows, n]: output and log-sum-exp, fp32."""
    x = torch.matmul(q, k.transpose(-1, -2)) * scale
    x = x.masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m > -math.inf, m, torch.zeros_like(m)))
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(z > 0, z, torch.ones_like(z))
    return o, (m + z.log()).squeeze(-1)


def _sparse(st):
    batch, hq, hkv, d, b = st["batch"], st["hq"], st["hkv"], st["d"], st["b"]
    idx, n = st["idx"], st["max_topk"] + 1
    j = torch.arange(n, device=idx.device)
    listed_ = j < st["cnt"][..., None]
    blk = torch.where(listed_, idx, torch.zeros_like(idx)).long()
    page = st["table"].long()[:, None, :].expand(-1, hkv, -1).gather(2, blk)
    head = torch.arange(hkv, device=idx.device)[None, :, None]
    k = (_values(st["k4"][page, head], st["ks"][page, head]) * st["g"][0][:, None, None, None])
    v = (_values(st["v4"][page, head], st["vs"][page, head]) * st["g"][1][:, None, None, None])
    pos = blk[..., None] * b + torch.arange(b, device=idx.device)
    seen = ((pos < st["len"][:, None, None, None]) & listed_[..., None]).flatten(2)
    q = st["q"].float().unflatten(1, (hkv, hq // hkv))
    o, lse = _softmax_av(q, k.flatten(2, 3), v.flatten(2, 3), seen[:, :, None], d ** -0.5)
    st["out"].copy_(o.flatten(1, 2))
    st["lse"].copy_(lse.flatten(1, 2))


def _attention(st):
    f, hq, hkv, d, b = st["f"], st["hq"], st["hkv"], st["d"], st["b"]
    g = hq // hkv
    page = st["table"].long()
    k = (_values(st["k4"][page], st["ks"][page]) * st["g"][0][:, None, None]).transpose(1, 2).flatten(2, 3)
    v = (_values(st["v4"][page], st["vs"][page]) * st["g"][1][:, None, None]).transpose(1, 2).flatten(2, 3)
    n = st["fresh"] if st["fresh"] is not None else torch.full_like(st["len"], f)
    r = torch.arange(f, device=n.device)
    last = (st["len"] - n)[:, None] + r                                   # [batch, f]
    seen = torch.arange(k.shape[2], device=n.device) <= last[..., None]   # [batch, f, keys]
    q = st["q"].float().unflatten(2, (hkv, g)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    o, lse = _softmax_av(q, k, v, seen.repeat_interleave(g, dim=1)[:, None], d ** -0.5)
    live = r < n[:, None]
    o = o.unflatten(2, (f, g)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    lse = lse.unflatten(2, (f, g)).permute(0, 2, 1, 3).flatten(2, 3)
    st["out"][live] = o[live]
    st["lse"][live] = lse[live]


# ---------------------------------------------------------------------------
# From the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _round_steps(x, least, bits, most):
    """x rounded to `bits` bits after the leading one, half to even; steps below 2^least are equal."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** (least - 4)))).clamp_min(least)
    step = torch.exp2(e - bits)
    return (torch.round(x / step) * step).clamp(-most, most)


def _held(x, g):
    """What 4 bits hold of x [..., d] (64 bits) with the head's scale g [..., 1]."""
    y = (x / g).unflatten(-1, (-1, 16))
    s = _round_steps(y.abs().amax(-1, keepdim=True) / 6, -6, 3, 448.0)
    code = _round_steps(torch.where(s > 0, y / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(y)),
                        0, 1, 6.0)
    return (code * s).flatten(-2) * g


def _decode(codes, s):
    """The cache's codes and scales as 64-bit numbers, from their bits."""
    n = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).to(torch.float64)
    sign, mag = 1 - 2 * torch.floor(n / 8), n % 8
    e, m = torch.floor(mag / 2), mag % 2
    x = sign * torch.where(e > 0, (1 + m / 2) * torch.exp2(e - 1), m / 2)
    u = s.view(torch.uint8).to(torch.float64)
    e, m = torch.floor(u / 8), u % 8
    t = torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 7), m / 8 * 2.0 ** -6)
    return (x.unflatten(-1, (-1, 16)) * t.unsqueeze(-1)).flatten(-2)


def exact(case, seed):
    st = prepare(case, seed)
    op, b, d, hq, hkv = case["op"], case["b"], case["d"], case["hq"], case["hkv"]
    g = hq // hkv
    total = _total(case)
    _, fresh = _lengths(case)
    gk, gv = st["g"].double()
    table = st["table"].long()
    if op in ("append", "append4", "expand4"):
        if op == "append":
            k, v = st["k"].double(), st["v"].double()
        else:
            k, v = st["k16"].double(), st["v16"].double()
            for i, L in enumerate(total):
                t = torch.arange(L, device="cuda")
                for to, codes, s, gh in ((k, "k4", "ks", gk), (v, "v4", "vs", gv)):
                    at = table[i, :-(-L // b)]
                    x = (_decode(st[codes][at], st[s][at]) * gh[:, None, None]).transpose(1, 2).flatten(0, 1)
                    to.transpose(1, 2)[table[i, t // b], t % b] = x[:L]
        if op == "expand4":
            return {"k": k, "v": v}
        qo, desc = st["q_out"].double(), st["desc"].double()
        rot = case["rot"]
        for i, (L, n) in enumerate(zip(total, fresh)):
            if not n:
                continue
            t = torch.arange(L - n, L, device="cuda")
            ang = torch.outer((t + case["shift"]).double(), st["inv_freq"].double())
            turn = torch.polar(torch.ones_like(ang), ang)[:, None]

            def turned(x):
                x = x.double()
                p = x[..., :rot]
                p = torch.complex(p[..., 0::2], p[..., 1::2]) if case["interleaved"] else \
                    torch.complex(p[..., :rot // 2].contiguous(), p[..., rot // 2:].contiguous())
                p = torch.view_as_real(p * turn)
                p = p.flatten(-2) if case["interleaved"] else torch.cat([p[..., 0], p[..., 1]], -1)
                return torch.cat([p, x[..., rot:]], -1)

            qo[i, :n] = turned(st["q"][i, :n])
            kn, vn = turned(st["kn"][i, :n]), st["vn"][i, :n].double()
            if op == "append4":
                kn = _held(kn.float().bfloat16().double(), gk[:, None])
                vn = _held(vn, gv[:, None])
            k.transpose(1, 2)[table[i, t // b], t % b] = kn
            v.transpose(1, 2)[table[i, t // b], t % b] = vn
            for blk in range((L - n) // b, (L - 1) // b + 1):
                page, m = table[i, blk], min(b, L - blk * b)
                desc[page, :, 0] = k[page, :, :m].amin(1)
                desc[page, :, 1] = k[page, :, :m].amax(1)
        return {"q": qo, "k": k, "v": v, "desc": desc}
    out, lse = st["out"].double(), st["lse"].double()
    counts = _counts(case)
    for i, L in enumerate(total):
        for h in range(hkv):
            if op == "sparse4":
                at = st["idx"][i, h, :counts[i]].long()
            else:
                at = torch.arange(-(-L // b), device="cuda")
            heads = slice(h * g, (h + 1) * g)
            pos = (at[:, None] * b + torch.arange(b, device="cuda")).flatten()
            page = table[i, at]
            k = (_decode(st["k4"][page, h], st["ks"][page, h]) * gk[h]).flatten(0, 1)[pos < L]
            v = (_decode(st["v4"][page, h], st["vs"][page, h]) * gv[h]).flatten(0, 1)[pos < L]
            pos = pos[pos < L]
            if op == "sparse4":
                x = st["q"][i, heads].double() @ k.T / math.sqrt(d)
                if not k.shape[0]:
                    out[i, heads], lse[i, heads] = 0, -math.inf
                    continue
                out[i, heads], lse[i, heads] = torch.softmax(x, -1) @ v, torch.logsumexp(x, -1)
            elif fresh[i]:
                n = fresh[i]
                x = torch.einsum("rgd,nd->rgn", st["q"][i, :n, heads].double(), k) / math.sqrt(d)
                row = L - n + torch.arange(n, device="cuda")
                x = x.masked_fill(pos > row[:, None, None], -math.inf)
                out[i, :n, heads] = torch.einsum("rgn,nd->rgd", torch.softmax(x, -1), v)
                lse[i, :n, heads] = torch.logsumexp(x, -1)
    return {"out": out, "lse": lse}
