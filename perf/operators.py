"""Operators of the FP8 cache and of scored attention, for measurement.

Four operators over the paged pool (16-token blocks, head_dim 128):

* ``store``: appends K/V rows to an FP8 pool. A block of 16 tokens of one kv
  head holds e4m3 codes with one power-of-two scale (a byte e for 2^(e - 127),
  0 for an empty block); a row that needs a larger scale raises the block's,
  and the codes already there are rounded to it.
* ``decode``: single-token attention of a batch over such a pool.
* ``extend``: attention of a chunk of new tokens over such a pool.
* ``scored``: decode or extend attention over a pool of any kind, with scores
  capped by a tanh, biased by distance, and masked by a window and a prefix.

``run`` computes them in elementary torch operations, or, where ``own`` is set,
by the package's calls. Blocks are scattered over the pool in every case.
"""
import math
import random

import torch

own = False

D, BLOCK = 128, 16
SCALE = 1.0 / math.sqrt(D)
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one decode step of a handful of requests: the call's latency
        dict(name="store, 4 new tokens", op="store", mode="step", tokens=4, kv_heads=8, q="f16"),
        # one decode step of a full batch: one row in each of 256 blocks
        dict(name="store, 256 new tokens", op="store", mode="step", tokens=256, kv_heads=8, q="bf16"),
        # a prefill chunk at the usual threshold, beginning inside a block
        dict(name="store, chunk of 4096", op="store", mode="chunk", tokens=4096, kv_heads=8, q="f16"),
        # a few short requests: latency
        dict(name="decode, 4 short requests", op="decode", batch=4, lo=17, hi=100, q_heads=16, kv_heads=8, q="f16"),
        # a serving batch of mixed lengths with grouped queries
        dict(name="decode, 256 mixed, group of 4", op="decode", batch=256, lo=256, hi=2048, q_heads=32, kv_heads=8, q="f16"),
        # a full batch at 4K without grouping: the most bytes for each query
        dict(name="decode, 128 x 4096, group of 1", op="decode", batch=128, lo=4096, hi=4096, q_heads=32, kv_heads=32, q="f16"),
        # two documents of about 100K tokens: few rows, a long axis
        dict(name="decode, 2 long, group of 8", op="decode", batch=2, lo=90001, hi=131071, q_heads=64, kv_heads=8, q="bf16"),
        # a fresh 4096-token prompt
        dict(name="extend, prompt of 4096", op="extend", batch=1, lo=4096, hi=4096, c_lo=4096, c_hi=4096, q_heads=32, kv_heads=8, q="f16"),
        # ragged chunks, some of a single token, over cached prefixes
        dict(name="extend, 7 ragged chunks", op="extend", batch=7, lo=701, hi=4001, c_lo=1, c_hi=701, q_heads=32, kv_heads=8, q="bf16"),
        # a layer of capped scores and a sliding window over a 16-bit cache
        dict(name="scored decode, cap and window", op="scored", form="decode", batch=32, lo=512, hi=4096, q_heads=16, kv_heads=8, q="bf16", kind="bf16", cap=50.0, window=1024, alibi=False, prefix=False),
        # scores that fall with the distance, over the FP8 cache
        dict(name="scored decode, distance bias", op="scored", form="decode", batch=64, lo=256, hi=2048, q_heads=32, kv_heads=32, q="f16", kind="fp8", cap=0.0, window=0, alibi=True, prefix=False),
        # two prompts in chunks, capped, with a window and a prefix seen from both sides
        dict(name="scored extend, cap, window, prefix", op="scored", form="extend", batch=2, lo=3901, hi=4096, c_lo=2000, c_hi=2048, q_heads=32, kv_heads=8, q="f16", kind="fp8", cap=30.0, window=1024, alibi=False, prefix=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "decode", "extend", "scored"])
    q = rng.choice(["f16", "bf16"])
    if op == "store":
        mode = rng.choice(["step", "chunk"])
        return dict(op=op, mode=mode, tokens=_log(rng, 1, 256 if mode == "step" else 4096),
                    kv_heads=rng.choice([1, 2, 3, 4, 8]), q=q)
    kv_heads, group = rng.choice([(32, 1), (8, 2), (8, 4), (8, 8), (2, 16), (5, 3), (4, 6), (1, 8)])
    c = dict(op=op, q=q, q_heads=kv_heads * group, kv_heads=kv_heads)
    form = rng.choice(["decode", "extend"]) if op == "scored" else op
    if form == "decode":
        c["hi"] = _log(rng, 2, 100000)
        c["lo"] = max(1, _log(rng, 1, c["hi"]))
        tokens = 262144 * 32 // (kv_heads * group)
        c["batch"] = _log(rng, 1, max(1, min(256, tokens // c["hi"])))
    else:
        c["hi"] = _log(rng, 16, 4096)
        c["lo"] = _log(rng, 1, c["hi"])
        c["c_hi"] = _log(rng, 1, min(c["hi"], 65536 // max(32, kv_heads * group)))
        c["c_lo"] = _log(rng, 1, c["c_hi"])
        c["batch"] = _log(rng, 1, max(1, min(16, 2 ** 28 // (c["hi"] * c["c_hi"] * kv_heads * group))))
    if op == "scored":
        c.update(form=form, kind=rng.choice(["fp8", "fp8", "int8", q]),
                 cap=rng.choice([0.0, 20.0, 30.0, 50.0]), window=rng.choice([0, 0, _log(rng, 1, 2048)]),
                 alibi=rng.choice([False, True]), prefix=form == "extend" and rng.choice([False, True]))
        if not (c["cap"] or c["window"] or c["alibi"] or c["prefix"]):
            c["cap"] = 30.0
    return c


# ---- inputs ---------------------------------------------------------------------


def _shape(case):
    """Lengths (and chunk lengths) of the requests: the case gives them, so that
    outputs have the same shape for every seed."""
    rng = random.Random("%(batch)d %(lo)d %(hi)d" % case)
    lens = [rng.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    lens[rng.randrange(len(lens))] = case["hi"]
    chunks = None
    if "c_hi" in case:
        chunks = [min(rng.randint(case["c_lo"], case["c_hi"]), n) for n in lens]
    return lens, chunks


def _values(n, heads, dtype, gen, chan):
    """Rows [n, heads, D] with a few channels of larger size, as K and V have."""
    return (torch.randn(n, heads, D, device="cuda", generator=gen) * chan).to(dtype)


def _channels(heads, gen):
    return 1.0 + 7.0 * (torch.rand(heads, D, device="cuda", generator=gen) < 0.01)


def _block_exponent(amax):
    """The smallest e >= -126 with amax <= 448 * 2^e, as the byte e + 127; 0 where amax is 0."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.where(amax > 0, (e + 127).clamp(1, 254), torch.zeros_like(e))


def _pool_side(kind, nb, heads, gen):
    """K or V of a pool of nb blocks, in the pool's layout: codes, and scales."""
    row = {"fp8": D, "int8": D, "f16": 2 * D, "bf16": 2 * D}[kind]
    codes = torch.empty(nb, BLOCK, heads, row, dtype=torch.uint8, device="cuda")
    sz = None
    if kind == "fp8":
        sz = torch.empty(nb, heads, dtype=torch.uint8, device="cuda")
    elif kind == "int8":
        sz = torch.empty(nb, heads, BLOCK, 2, dtype=torch.float16, device="cuda")
    chan = _channels(heads, gen)
    step = max(1, (1 << 27) // (BLOCK * heads * D))
    for b in range(0, nb, step):
        n = min(step, nb - b)
        x = _values(n * BLOCK, heads, DT.get(kind, torch.float16), gen, chan).view(n, BLOCK, heads, D)
        if kind == "fp8":
            x = x.float()
            e = _block_exponent(x.abs().amax(dim=(1, 3)))
            s = torch.exp2(e.float() - 127.0)
            sz[b:b + n] = e.to(torch.uint8)
            codes[b:b + n] = (x / s[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        elif kind == "int8":
            x = x.float()
            lo, hi = x.amin(-1), x.amax(-1)
            s, z = ((hi - lo) / 255.0).half(), lo.half()
            c = ((x - z.float()[..., None]) / s.float()[..., None]).round().clamp(0, 255)
            codes[b:b + n] = c.to(torch.uint8)
            sz[b:b + n] = torch.stack([s, z], -1).transpose(1, 2)
        else:
            codes[b:b + n] = x.view(torch.uint8)
    return codes, sz if kind != "int8" else (None if sz is None else sz.view(torch.int32).squeeze(-1))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    h, dt = case["kv_heads"], DT[case["q"]]
    st = dict(case)
    if case["op"] == "store":
        return _prepare_store(case, st, gen, h, dt)
    kind = case.get("kind", "fp8")
    lens, chunks = _shape(case)
    width = [(n + BLOCK - 1) // BLOCK for n in lens]
    nb, mb = sum(width), max(width)
    perm = torch.randperm(nb, device="cuda", generator=gen, dtype=torch.int32)
    first = torch.tensor([0] + width, device="cuda").cumsum(0)[:-1, None]
    cols = torch.arange(mb, device="cuda")[None]
    used = cols < torch.tensor(width, device="cuda")[:, None]
    table = torch.where(used, perm[(first + cols).clamp(max=nb - 1)], -1).to(torch.int32)
    k, k_sz = _pool_side(kind, nb, h, gen)
    v, v_sz = _pool_side(kind, nb, h, gen)
    rows = sum(chunks) if chunks else len(lens)
    gain = 3.0 if case.get("cap") else 1.0
    st.update(kind=kind, k=k, v=v, k_sz=k_sz, v_sz=v_sz, table=table, nb=nb,
              lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), max_len=max(lens), rows=rows,
              qs=(torch.randn(rows, case["q_heads"], D, device="cuda", generator=gen) * gain).to(dt),
              out=torch.empty(rows, case["q_heads"], D, dtype=dt, device="cuda"))
    if chunks:
        st["max_chunk"] = max(chunks)
        st["indptr"] = torch.tensor([0] + chunks, device="cuda").cumsum(0).to(torch.int32)
    st["slopes"] = st["prefix_lens"] = None
    if case.get("alibi"):
        hq = case["q_heads"]
        st["slopes"] = torch.exp2(-8.0 * torch.arange(1, hq + 1, device="cuda", dtype=torch.float32) / hq)
    if case.get("prefix"):
        share = torch.rand(len(lens), device="cuda", generator=gen)
        st["prefix_lens"] = (share * st["lens"]).to(torch.int32)
    return st


def _prepare_store(case, st, gen, h, dt):
    """A pool that holds the tokens before the new ones: `step` adds one token
    to each of many requests, `chunk` a run of tokens to one."""
    n = case["tokens"]
    if case["mode"] == "step":
        nb = 4 * n
        blocks = torch.randperm(nb, device="cuda", generator=gen)[:n]
        offs = torch.randint(0, BLOCK, (n,), device="cuda", generator=gen)
        slots = blocks * BLOCK + offs
    else:
        start = (5 * n + 3) % BLOCK
        need = (start + n + BLOCK - 1) // BLOCK
        nb = 2 * need
        blocks = torch.randperm(nb, device="cuda", generator=gen)[:need]
        pos = torch.arange(start, start + n, device="cuda")
        slots = blocks[pos // BLOCK] * BLOCK + pos % BLOCK
    k, k_sz = _pool_side("fp8", nb, h, gen)
    v, v_sz = _pool_side("fp8", nb, h, gen)
    ck, cv = _channels(h, gen), _channels(h, gen)
    st.update(kind="fp8", nb=nb, k=k, v=v, k_sz=k_sz, v_sz=v_sz, slots=slots.to(torch.int64),
              k_new=_values(n, h, dt, gen, ck), v_new=_values(n, h, dt, gen, cv))
    return st


# ---- one pass -------------------------------------------------------------------


def run(st):
    if own:
        return _run_own(st)
    if st["op"] == "store":
        return _store_plain(st)
    return _attend_plain(st)


def _stored(st):
    """A pool's codes as e4m3 values, and its scales' exponents."""
    return [st["k"].view(torch.float8_e4m3fn), st["v"].view(torch.float8_e4m3fn), st["k_sz"], st["v_sz"]]


def _store_side(codes, exps, new, slots):
    nb, heads = exps.shape
    blk, off = slots // BLOCK, slots % BLOCK
    x = new.float()
    idx = blk[:, None].expand(-1, heads)
    amax = torch.zeros(nb, heads, device=x.device).scatter_reduce(0, idx, x.abs().amax(-1), "amax")
    fresh = torch.zeros(nb, dtype=torch.int32, device=x.device).scatter_reduce(
        0, blk, (off == 0).to(torch.int32), "amax") > 0
    old = torch.where(fresh[:, None], 0, exps.to(torch.int32))
    now = torch.maximum(old, _block_exponent(amax))
    # codes that stay, at the block's new scale
    ratio = torch.exp2((old - now).float())[blk][:, None, :, None]
    was = old[blk][:, None, :, None] > 0
    kept = codes[blk].view(torch.float8_e4m3fn).float()
    kept = torch.where(was, kept * ratio, torch.zeros_like(kept)).to(torch.float8_e4m3fn).view(torch.uint8)
    grown = ((old < now) & ~fresh[:, None])[blk][:, None, :, None]
    codes[blk] = torch.where(grown, kept, codes[blk])
    s = torch.exp2(now[blk].float() - 127.0)[..., None]
    codes[blk, off] = (x / s).to(torch.float8_e4m3fn).view(torch.uint8)
    exps[blk] = now[blk].to(torch.uint8)


def _store_plain(st):
    _store_side(st["k"], st["k_sz"], st["k_new"], st["slots"])
    _store_side(st["v"], st["v_sz"], st["v_new"], st["slots"])
    return _stored(st)


def _side_values(st, codes, sz, table):
    """[B, T, H, D] in 32 bits: the values that the blocks of the tables stand for."""
    b, w = table.shape
    c = codes[table.clamp(min=0).long()]
    if st["kind"] == "fp8":
        x = c.view(torch.float8_e4m3fn).float()
        x = x * torch.exp2(sz[table.clamp(min=0).long()].float() - 127.0)[:, :, None, :, None]
    elif st["kind"] == "int8":
        s = sz[table.clamp(min=0).long()].view(torch.float16).view(b, w, -1, BLOCK, 2).float().transpose(2, 3)
        x = c.float() * s[..., :1] + s[..., 1:]
    else:
        x = c.view(DT[st["kind"]]).float()
    return x.reshape(b, w * BLOCK, -1, D)


def _attend_plain(st):
    hq, h = st["q_heads"], st["kv_heads"]
    g, lens = hq // h, st["lens"].long()
    k = _side_values(st, st["k"], st["k_sz"], st["table"])
    v = _side_values(st, st["v"], st["v_sz"], st["table"])
    b, t = k.shape[:2]
    if "indptr" in st:
        first, last = st["indptr"][:-1].long(), st["indptr"][1:].long()
        c = st["max_chunk"]
        i = torch.arange(c, device=k.device)
        row = (first[:, None] + i).clamp(max=st["rows"] - 1)
        live = first[:, None] + i < last[:, None]
        pos = lens[:, None] - (last - first)[:, None] + i
    else:
        c = 1
        row = torch.arange(b, device=k.device)[:, None]
        live, pos = torch.ones_like(row, dtype=torch.bool), lens[:, None] - 1
    q = st["qs"].float()[row].view(b, c, h, g, D).permute(0, 2, 3, 1, 4).reshape(b, h, g * c, D)
    s = (q @ k.permute(0, 2, 3, 1)).view(b, h, g, c, t) * SCALE
    if st.get("cap"):
        s = st["cap"] * torch.tanh(s / st["cap"])
    at = torch.arange(t, device=k.device)
    gap = at - pos[..., None]  # [B, C, T]
    if st.get("slopes") is not None:
        s = s - st["slopes"].view(h, g, 1, 1) * gap.abs().float()[:, None, None]
    seen = gap <= 0
    if st.get("prefix_lens") is not None:
        seen = seen | (at < st["prefix_lens"].long()[:, None, None])
    if st.get("window"):
        seen = seen & (gap > -st["window"])
    seen = seen & (at < lens[:, None, None])
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    o = (p.view(b, h, g * c, t) @ v.transpose(1, 2)).view(b, h, g, c, D).permute(0, 3, 1, 2, 4)
    o = o.reshape(b, c, hq, D).to(st["qs"].dtype)
    return o[live] if "indptr" in st else o[:, 0]


def _run_own(st):
    import paged_quantized_kv_store_gb300 as kvq
    if "pool" not in st:  # what a server keeps from step to step
        st["pool"] = kvq.KVPool(st["k"], st["v"], st["k_sz"], st["v_sz"], st["nb"], st["kv_heads"], st["kind"])
        if st["op"] != "store":
            if "indptr" in st:
                n = kvq.paged_extend_attn_workspace_size(st["batch"], st["rows"], st["q_heads"], st["kv_heads"], st["max_len"])
            else:
                n = kvq.paged_decode_attn_workspace_size(st["batch"], st["q_heads"], st["kv_heads"], st["max_len"])
            st["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
            st["score"] = kvq.Score(st.get("cap") or 0.0, st.get("window") or 0, st["slopes"], st["prefix_lens"])
    pool = st["pool"]
    if st["op"] == "store":
        kvq.kv_store_quant(pool, st["k_new"], st["v_new"], st["slots"])
        return _stored(st)
    if st["op"] == "decode":
        kvq.paged_decode_attn(pool, st["qs"], st["out"], st["table"], st["lens"], st["max_len"], SCALE, workspace=st["ws"])
    elif st["op"] == "extend":
        kvq.paged_extend_attn(pool, st["qs"], st["out"], st["indptr"], st["lens"], st["table"], st["max_len"], SCALE, workspace=st["ws"])
    elif "indptr" in st:
        kvq.paged_extend_attn_scored(pool, st["score"], st["qs"], st["out"], st["indptr"], st["lens"], st["table"], st["max_len"], SCALE, workspace=st["ws"])
    else:
        kvq.paged_decode_attn_scored(pool, st["score"], st["qs"], st["out"], st["table"], st["lens"], st["max_len"], SCALE, workspace=st["ws"])
    return st["out"]


# ---- what one pass cannot do without ---------------------------------------------


def _pairs(case, lens, chunks):
    """(query, token) pairs that are attended, and tokens that some query attends.
    The prefix, whose lengths the seed gives, is counted as half of each request."""
    pairs = tokens = 0
    w = case.get("window") or 1 << 60
    for i, n in enumerate(lens):
        c = chunks[i] if chunks else 1
        p = n // 2 if case.get("prefix") else 0
        for_row = 0
        for pos in range(n - c, n):
            for_row += max(pos + 1, p) - max(0, pos + 1 - w)
        pairs += for_row
        tokens += n - max(0, n - c + 1 - w)
    return pairs, tokens


def work(case):
    h = case["kv_heads"]
    if case["op"] == "store":
        n = case["tokens"]
        blocks = n if case["mode"] == "step" else (n + BLOCK - 1) // BLOCK
        return {"bytes": 2 * n * h * (2 * D + D) + 2 * blocks * h * 2 + 8 * n, "flops": 2 * 3 * n * h * D}
    lens, chunks = _shape(case)
    pairs, tokens = _pairs(case, lens, chunks)
    per = {"fp8": D + 1.0 / BLOCK, "int8": D + 4, "f16": 2 * D, "bf16": 2 * D}[case.get("kind", "fp8")]
    rows = sum(chunks) if chunks else len(lens)
    return {"bytes": 2 * tokens * h * per + 4 * rows * case["q_heads"] * D + 4 * (tokens // BLOCK + 2 * len(lens)),
            "flops": 4 * pairs * case["q_heads"] * D}


# ---- the same in 64 bits ----------------------------------------------------------


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_store(st) if case["op"] == "store" else _exact_attention(st)


def _grid():
    """The 127 finite e4m3 magnitudes, in order."""
    return torch.tensor([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10)
                         for c in range(127)], dtype=torch.float64, device="cuda")


def _nearest(x):
    """x, at most 448 in size, rounded to the nearest e4m3 value, ties to the even code."""
    g, a = _grid(), x.abs().contiguous()
    hi = torch.searchsorted(g, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = g[hi] - a, a - g[lo]
    take = torch.where(up == down, hi % 2 == 0, up < down)
    return torch.sign(x) * torch.where(take, g[hi], g[lo])


def _exact_store(st):
    outs, scales = [], []
    for name in ("k", "v"):
        val = st[name].view(torch.float8_e4m3fn).double()
        exps = st[name + "_sz"].cpu().tolist()
        new = st[name + "_new"].double()
        big = new.abs().amax(-1).cpu().tolist()
        at = {}
        for i, slot in enumerate(st["slots"].cpu().tolist()):
            at.setdefault(slot // BLOCK, []).append((slot % BLOCK, i))
        shift = torch.zeros(len(exps), len(exps[0]), dtype=torch.float64)
        for blk, rows in at.items():
            begins = any(o == 0 for o, _ in rows)
            for h in range(len(exps[0])):
                a = max(big[i][h] for _, i in rows)
                e = 0
                if a > 0:
                    e = 1
                    while 448.0 * 2.0 ** (e - 127) < a:
                        e += 1
                before = 0 if begins else exps[blk][h]
                e = max(e, before)
                shift[blk, h] = 0.0 if begins or before == 0 else float(before - e)
                exps[blk][h] = e
        moved = _nearest(val * torch.exp2(shift.cuda())[:, None, :, None])
        val = torch.where((shift.cuda() != 0)[:, None, :, None], moved, val)
        unit = torch.exp2(torch.tensor(exps, dtype=torch.float64) - 127.0).cuda()
        slots = st["slots"]
        val.view(-1, *val.shape[2:])[slots] = _nearest(new / unit[slots // BLOCK][..., None])
        outs.append(val)
        scales.append(torch.tensor(exps, dtype=torch.uint8))
    return outs + scales


def _exact_values(st, name, ids):
    """[T, H, D] in 64 bits of the blocks `ids`."""
    c, sz = st[name][ids], st[name + "_sz"]
    if st["kind"] == "fp8":
        x = c.view(torch.float8_e4m3fn).double() * torch.pow(2.0, sz[ids].double() - 127.0)[:, None, :, None]
    elif st["kind"] == "int8":
        f = sz[ids].view(torch.float16).view(len(ids), -1, BLOCK, 2).permute(0, 2, 1, 3).double()
        x = c.double() * f[..., :1] + f[..., 1:]
    else:
        x = c.view(DT[st["kind"]]).double()
    return x.reshape(-1, st["kv_heads"], D)


def _exact_attention(st):
    hq, h = st["q_heads"], st["kv_heads"]
    g = hq // h
    out = torch.zeros(st["rows"], hq, D, dtype=torch.float64, device="cuda")
    ptr = st["indptr"].cpu().tolist() if "indptr" in st else list(range(len(st["lens"]) + 1))
    lens = st["lens"].cpu().tolist()
    for b, n in enumerate(lens):
        ids = st["table"][b, : (n + BLOCK - 1) // BLOCK].long()
        k, v = _exact_values(st, "k", ids)[:n], _exact_values(st, "v", ids)[:n]
        q = st["qs"][ptr[b]:ptr[b + 1]].double()
        pos = torch.arange(n - len(q), n, device="cuda")[:, None]
        at = torch.arange(n, device="cuda")[None]
        allowed = at <= pos
        if st.get("prefix_lens") is not None:
            allowed = allowed | (at < int(st["prefix_lens"][b]))
        if st.get("window"):
            allowed = allowed & (at + st["window"] > pos)
        for j in range(hq):
            s = q[:, j] @ k[:, j // g].T / math.sqrt(D)
            if st.get("cap"):
                s = torch.tanh(s / st["cap"]) * st["cap"]
            if st.get("slopes") is not None:
                s = s - float(st["slopes"][j]) * (pos - at).abs()
            s = torch.where(allowed, s, -math.inf)
            w = torch.exp(s - s.max(1, keepdim=True).values)
            out[ptr[b]:ptr[b + 1], j] = (w @ v[:, j // g]) / w.sum(1, keepdim=True)
    return out
