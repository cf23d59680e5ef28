"""FP8 and scored attention as programs may call them: random shapes and
scores, two calls at once, captured calls replayed on other lengths, padded
batches, large batches, long contexts. Against the 64-bit reference of
fp8_ref, with the bounds that it derives (scored INT8/INT4: the framework's
tolerance of quantized pools).
"""
import math

import numpy as np
import pytest
import torch

import paged_quantized_kv_store_gb300 as kvq
import test_gpu_fp8 as base

pytestmark = pytest.mark.gpu

from gpu_harness import i32, i64  # noqa: E402

SM = 1.0 / math.sqrt(128)
HEADS = [(8, 8), (32, 8), (16, 2), (7, 1), (15, 5), (64, 1), (40, 40), (24, 2)]


class Call:
    """An attention call with a canary behind its outputs and its workspace."""

    def __init__(self, pool, q, bt, lens, indptr=None, score=None, variant="auto", rows=None,
                 max_len=None):
        self.pool, self.q, self.score, self.variant = pool, q, score, variant
        self.rows = q.shape[0] if rows is None else rows
        self.bt, self.lens = i32(bt), i32(lens)
        self.indptr = None if indptr is None else i32(indptr)
        self.max_len = max(1, int(max(lens))) if max_len is None else max_len
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        if indptr is None:
            n = kvq.paged_decode_attn_workspace_size(len(lens), q.shape[1], pool.kv_heads,
                                                     self.max_len, 0)
        else:
            n = kvq.paged_extend_attn_workspace_size(len(lens), q.shape[0], q.shape[1],
                                                     pool.kv_heads, self.max_len)
        self.ws = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        self.n = n
        self.out = torch.full((q.shape[0] + 3,) + tuple(q.shape[1:]), 77.0, dtype=q.dtype,
                              device="cuda")

    def __call__(self):
        first = [self.pool] if self.score is None else [self.pool, self.score]
        out, ws = self.out[: self.q.shape[0]], self.ws[: self.n]
        if self.indptr is None:
            f = kvq.paged_decode_attn if self.score is None else kvq.paged_decode_attn_scored
            f(*first, self.q, out, self.bt, self.lens, self.max_len, SM, 0, ws, self.err)
        else:
            f = kvq.paged_extend_attn if self.score is None else kvq.paged_extend_attn_scored
            f(*first, self.q, out, self.indptr, self.lens, self.bt, self.max_len, SM, ws, self.err,
              None, self.variant)
        return out

    def check(self):
        assert int(self.err.item()) == 0
        assert (self.out[self.rows:] == 77.0).all(), "rows behind the last sequence"
        assert (self.ws[self.n:] == 0xA5).all(), "bytes behind the workspace"


def random_case(seed):
    r = np.random.RandomState(1000 + seed)
    kind = ["fp8", "fp8", "fp8", "int8", "int4", "f16", "bf16"][r.randint(7)]
    dtype = kind if kind in base.DT else ["f16", "bf16"][r.randint(2)]
    hq, hkv = HEADS[r.randint(len(HEADS))]
    form = ["decode", "extend"][r.randint(2)]
    batch = int(r.choice([1, 2, 5, 12]))
    top = int(r.choice([70, 400, 1500, 5000])) // (1 if batch < 3 else 3)
    lens = r.randint(0, top + 1, batch)
    lens[r.randint(batch)] = top
    combo = "".join(c for c in "cwap" if r.rand() < 0.4)
    window = int(r.choice([1, 20, 64, 300, 1111]))
    indptr = None
    if form == "extend":
        most = max(1, 4_000_000 // (hq * max(1, int(lens.sum()))))
        chunks = [r.randint(0, min(n, most) + 1) if r.rand() < 0.8 else min(n, 1) for n in lens]
        indptr = np.concatenate([[0], np.cumsum(chunks)])
        if indptr[-1] == 0:
            chunks[int(np.argmax(lens))] = 1
            indptr = np.concatenate([[0], np.cumsum(chunks)])
    return kind, dtype, hq, hkv, lens.tolist(), indptr, combo, window, float(r.choice([0.7, 4.0, 30.0]))


@pytest.mark.parametrize("seed", range(48))
def test_random_calls(gpu, seed):
    kind, dtype, hq, hkv, lens, indptr, combo, window, cap = random_case(seed)
    # (the plain attention over the other kinds may read rows behind the last token)
    scored = bool(set(combo) - ({"p"} if indptr is None else set()))
    pool, bt = base.make_pool(kind, lens, hkv, 500 + seed, dtype, poison=kind == "fp8" or scored)
    rows = len(lens) if indptr is None else int(indptr[-1])
    q = base.randn(600 + seed, rows, hq, 128, dtype=dtype, scale=2.0)
    score, kw = base.score_of(combo, hq, len(lens), lens, cap, window)
    if indptr is None:
        kw["prefix"] = None  # a decode's query is its request's last token
    if not combo:
        score = score if seed % 2 else None
    variants = ["auto", "mma_sync"] + ([] if kind == "bf16" or kind in ("int8", "int4") and not combo
                                       else ["tcgen05"])
    for variant in variants if indptr is not None else ["auto"]:
        call = Call(pool, q, bt, lens, indptr, score, variant)
        got = call().clone()
        call.check()
        base.compare(pool, got, q, bt, lens, indptr, **kw)
        assert torch.equal(call(), got)  # the same inputs give the same bits


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group", [2, 3, 4, 5, 7, 8])
@pytest.mark.parametrize("hkv", [1, 2, 5, 8, 12, 16])
def test_decode_groups(gpu, hkv, group, dtype):
    """2 to 8 q heads per kv head, any number of kv heads; V's scales far apart,
    blocks of zeros that hold NaN codes, windows of block ids that end inside
    a request, ids outside the pool."""
    for lens in ([0, 1, 15, 16, 17, 300, 513, 1100], [2500], [9001, 0, 40]):
        pool, bt = base.make_pool("fp8", lens, hkv, 60 + hkv, dtype, v_spread=dtype == "bf16")
        for name in ("k", "v"):
            at = int(bt[int(np.argmax(lens)), 3])
            getattr(pool, name + "_sz")[at, hkv - 1] = 0
            getattr(pool, name)[at, :, hkv - 1] = 0x7F
        q = base.randn(61, len(lens), group * hkv, 128, dtype=dtype)
        call = Call(pool, q, bt, lens)
        got = call().clone()
        call.check()
        base.compare(pool, got, q, bt, lens)
        assert torch.equal(call(), got)
        bad = bt.copy()
        bad[int(np.argmax(lens)), 2] = pool.num_blocks
        call.bt = i32(bad)
        assert torch.isfinite(call()).all()
        assert int(call.err.item()) == kvq.DEV_ERR_BITS["block_id"]


@pytest.mark.parametrize("group,dtype", [(4, "f16"), (8, "bf16")])
def test_decode_groups_long(gpu, group, dtype):
    """Shares long enough that their ends are handed out from a counter (over
    128 blocks for each of two CTAs an SM)."""
    lens = [110001, 109000, 120007, 112000, 111111, 128016]
    pool, bt = base.make_pool("fp8", lens, 1, 71, dtype)
    q = base.randn(72, len(lens), group, 128, dtype=dtype)
    call = Call(pool, q, bt, lens)
    for _ in range(2):
        call()
        call.check()
        base.compare(pool, call.out[: len(lens)], q, bt, lens)


@pytest.mark.parametrize("form", ["decode", "extend"])
def test_two_calls_at_once(gpu, form):
    """Two calls on two streams, each with its workspace, over one pool."""
    lens = [3000, 17, 900]
    pool, bt = base.make_pool("fp8", lens, 8, 21)
    calls = []
    for i, combo in enumerate(("", "cwap")):
        score, _ = base.score_of(combo, 32, 3, lens)
        if form == "decode":
            calls.append(Call(pool, base.randn(22 + i, 3, 32, 128), bt, lens, None, score))
        else:
            ptr = [0, 40 + i, 50 + i, 400]
            calls.append(Call(pool, base.randn(22 + i, 400, 32, 128), bt, lens, ptr, score, "tcgen05"))
    alone = [c().clone() for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip(calls, streams):
            c.out.fill_(77.0)
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                c()
        torch.cuda.synchronize()
        for c, a in zip(calls, alone):
            c.check()
            assert torch.equal(c.out[: a.shape[0]], a)


@pytest.mark.parametrize("variant", ["mma_sync", "tcgen05"])
@pytest.mark.parametrize("rows,top", [(33, 5000), (700, 900)])
def test_captured_extend_on_other_lengths(gpu, variant, rows, top):
    """An extend captured with its tables and lengths in device buffers, then
    replayed on shorter chunks and contexts; its rows behind the last chunk
    are left as they were. 33 rows over 5000 tokens: the context is cut."""
    lens, hq, hkv = [top, top // 2, 40], 16, 4
    pool, bt = base.make_pool("fp8", lens, hkv, 23, "bf16")
    score, kw = base.score_of("cw", hq, 3, lens, window=700)
    q = base.randn(24, rows, hq, 128, dtype="bf16")
    call = Call(pool, q, bt, lens, [0, rows - 9, rows - 2, rows], score, variant)
    plain = Call(pool, q, bt, lens, [0, rows - 9, rows - 2, rows], None, variant)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call(), plain()
    stream.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        call()
        plain()
    for now, ptr in ((lens, [0, rows - 9, rows - 2, rows]), ([top - 1, 17, 0], [0, 20, 25, 25]),
                     ([64, 65, 16], [0, 1, 2, 18]), ([0, 0, 0], [0, 0, 0, 0])):
        for c in (call, plain):
            c.lens.copy_(i32(now))
            c.indptr.copy_(i32(ptr))
            c.out.fill_(77.0)
            c.rows = ptr[-1]
        g.replay()
        torch.cuda.synchronize()
        for c, k in ((call, kw), (plain, {})):
            c.check()
            base.compare(pool, c.out[: ptr[-1]], q[: ptr[-1]], bt, now, ptr, **k)


def test_captured_decode_on_other_lengths(gpu):
    """A padded decode batch: requests of no tokens get rows of zeros, and
    lengths may be anything up to the captured maximum."""
    lens, hq, hkv = [5000, 300, 16, 1], 32, 8
    pool, bt = base.make_pool("fp8", lens, hkv, 25)
    q = base.randn(26, 4, hq, 128)
    score, kw = base.score_of("cwa", hq, 4, lens, window=700)
    call, plain = Call(pool, q, bt, lens, None, score), Call(pool, q, bt, lens)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call(), plain()
    stream.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        call()
        plain()
    for now in (lens, [1, 0, 0, 0], [0, 0, 0, 0], [4999, 0, 15, 1], [112, 113, 16, 0]):
        for c in (call, plain):
            c.lens.copy_(i32(now))
            c.out.fill_(77.0)
        g.replay()
        torch.cuda.synchronize()
        for c, k in ((call, kw), (plain, {})):
            c.check()
            base.compare(pool, c.out[:4], q, bt, now, **k)
            assert (c.out[:4][torch.tensor(now) == 0] == 0).all()


@pytest.mark.parametrize("form", ["decode", "extend"])
def test_large_batches(gpu, form):
    """More requests than the tcgen05 kernels take."""
    r = np.random.RandomState(4)
    lens = r.randint(0, 40, 5001).tolist()
    pool, bt = base.make_pool("fp8", lens, 2, 27)
    score, kw = base.score_of("cw", 4, len(lens), lens)
    if form == "decode":
        q = base.randn(28, len(lens), 4, 128)
        call = Call(pool, q, bt, lens, None, score)
        call()
        call.check()
        base.compare(pool, call.out[: len(lens)], q, bt, lens, **kw)
        return
    ptr = np.concatenate([[0], np.cumsum([min(n, i % 19) for i, n in enumerate(lens)])])
    q = base.randn(28, int(ptr[-1]), 4, 128)
    call = Call(pool, q, bt, lens, ptr, score)
    call()
    call.check()
    base.compare(pool, call.out[: int(ptr[-1])], q, bt, lens, ptr, **kw)
    call.variant = "tcgen05"
    with pytest.raises(kvq.KvqError):
        call()


@pytest.mark.parametrize("rows", [1, 5, 70])
@pytest.mark.parametrize("score", [False, True])
def test_few_rows_over_a_long_context(gpu, rows, score):
    n = 70001
    pool, bt = base.make_pool("fp8", [n], 2, 29, "bf16")
    q = base.randn(30, rows, 8, 128, dtype="bf16")
    s, kw = base.score_of("ca" if score else "", 8, 1, [n])
    for variant in ("mma_sync", "tcgen05"):
        call = Call(pool, q, bt, [n], [0, rows], s if score else None, variant)
        call()
        call.check()
        base.compare(pool, call.out[:rows], q, bt, [n], [0, rows], **kw)


@pytest.mark.parametrize("variant", ["mma_sync", "tcgen05"])
def test_prefix_lengths_out_of_range(gpu, variant):
    """Prefixes below 0 and beyond the request count as none and as all of it."""
    lens, ptr = [150, 90, 300], [0, 100, 130, 260]
    pool, bt = base.make_pool("fp8", lens, 2, 31)
    q = base.randn(32, 260, 8, 128)
    for p in ([-5, 1 << 30, -(1 << 31)], [(1 << 31) - 1, 0, 299]):
        call = Call(pool, q, bt, lens, ptr, kvq.Score(prefix_lens=i32(p)), variant)
        call()
        call.check()
        base.compare(pool, call.out[:260], q, bt, lens, ptr,
                     prefix=np.clip(np.array(p, np.int64), 0, lens))


def test_lengths_out_of_range(gpu):
    """A length beyond max_kv_len, a chunk beyond its length, an indptr beyond
    the rows: flagged, nothing of them written, the other requests served."""
    lens = [150, 90, 300]
    pool, bt = base.make_pool("fp8", lens, 2, 33)
    q = base.randn(34, 60, 8, 128)
    for now, ptr, top in (([150, 90, 305], [0, 20, 40, 60], 300), ([150, 90, 3], [0, 20, 40, 60], 300),
                          ([150, 90, 300], [0, 20, 40, 61], 300)):
        for variant in ("mma_sync", "tcgen05"):
            call = Call(pool, q, bt, now, ptr, kvq.Score(20.0), variant, max_len=top)
            call()
            assert int(call.err.item()) == kvq.DEV_ERR_BITS["length"]
            assert (call.ws[call.n:] == 0xA5).all() and (call.out[60:] == 77.0).all()
            base.compare(pool, call.out[:40], q[:40], bt[:2], now[:2], ptr[:3], cap=20.0)


def test_empty_calls(gpu):
    pool, _ = base.make_pool("fp8", [40], 2, 35)
    q = base.randn(36, 0, 8, 128)
    e = torch.empty(0, 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
    for score in (None, kvq.Score(5.0, 3)):
        f = [pool] if score is None else [pool, score]
        d = kvq.paged_decode_attn if score is None else kvq.paged_decode_attn_scored
        x = kvq.paged_extend_attn if score is None else kvq.paged_extend_attn_scored
        d(*f, q, q, e, i32([]), 40, SM, 0, ws)
        x(*f, q, q, i32([0]), i32([]), e, 40, SM, ws)
        x(*f, q, q, i32([0, 0]), i32([40]), i32([[0]]), 40, SM, ws)
    kvq.kv_store_quant(pool, torch.empty(0, 2, 128, dtype=torch.float16, device="cuda"),
                       torch.empty(0, 2, 128, dtype=torch.float16, device="cuda"), i64([]))
    torch.cuda.synchronize()
