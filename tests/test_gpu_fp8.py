"""FP8 pools and scored attention on the GPU against 64-bit references.

Store: codes and scale bytes bit-exact. Attention: within the bounds that
fp8_ref.assert_within derives (scored INT8/INT4: the framework's tolerance of
quantized pools, 2e-3 or 1e-2).
"""
import math

import numpy as np
import pytest
import torch

import fp8_ref
import paged_quantized_kv_store_gb300 as kvq

pytestmark = pytest.mark.gpu

from gpu_harness import assert_close, i32, i64  # noqa: E402

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
SM = 1.0 / math.sqrt(128)


def randn(seed, *shape, dtype="f16", scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(DT[dtype]).cuda()


# ---- store ----------------------------------------------------------------------


def check_store(pool, ref, k, v, slots, dev_err=None):
    """Stores on both sides and compares every byte of the pool."""
    kvq.kv_store_quant(pool, k, v, i64(slots), dev_err)
    for name, rows in (("k", k), ("v", v)):
        fp8_ref.store_side(ref[name], ref[name + "_sz"], rows.double().cpu().numpy(), list(slots))
        assert np.array_equal(getattr(pool, name + "_sz").cpu().numpy(), ref[name + "_sz"]), name
        assert np.array_equal(getattr(pool, name).cpu().numpy(), ref[name]), name


def host_copy(pool):
    return {n: getattr(pool, n).cpu().numpy().copy() for n in ("k", "v", "k_sz", "v_sz")}


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads", [1, 3, 8])
@pytest.mark.parametrize("n,start", [(1, 0), (1, 5), (15, 1), (16, 0), (17, 15), (33, 7), (300, 9)])
def test_store_chunk(gpu, dtype, heads, n, start):
    """A run of tokens into scattered blocks, after an earlier store of smaller values."""
    nb = (start + n + 15) // 16 + 3
    perm = np.random.RandomState(n).permutation(nb)
    slots = np.array([perm[p // 16] * 16 + p % 16 for p in range(start + n)])
    pool = kvq.KVPool.allocate(nb, heads, "fp8")
    ref = host_copy(pool)
    if start:
        check_store(pool, ref, randn(1, start, heads, 128, dtype=dtype, scale=0.1),
                    randn(2, start, heads, 128, dtype=dtype, scale=3.0), slots[:start])
    check_store(pool, ref, randn(3, n, heads, 128, dtype=dtype),
                randn(4, n, heads, 128, dtype=dtype), slots[start:])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_store_token_by_token_grows_the_scale(gpu, dtype):
    """Sixteen decode steps of many requests, sizes that rise and fall by powers of ten."""
    pool = kvq.KVPool.allocate(40, 2, "fp8")
    ref = host_copy(pool)
    for step in range(20):
        blocks = np.random.RandomState(step // 16).permutation(40)[:33]
        size = 10.0 ** ((step * 7) % 5 - 3)
        check_store(pool, ref, randn(step, 33, 2, 128, dtype=dtype, scale=size),
                    randn(99 + step, 33, 2, 128, dtype=dtype, scale=1 / size),
                    blocks * 16 + step % 16)


def test_store_special_values_and_skipped_tokens(gpu):
    pool = kvq.KVPool.allocate(9, 2, "fp8")
    pool.k.fill_(0x7F)  # rows nobody wrote hold NaN codes
    pool.v.fill_(0xFF)
    ref = host_copy(pool)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = randn(5, 12, 2, 128), randn(6, 12, 2, 128)
    k[0] = 0.0
    k[1, 0, 3], k[1, 0, 4], k[1, 1, 5] = float("inf"), -float("inf"), float("nan")
    k[2], v[2, :, :64] = 6e-8, 65504.0
    v[3] = float("inf")
    v[4] = -0.0
    # (a skipped token ends a run: two runs of one block in a call would race)
    slots = [0, 16, 32, 48, 64, -1, 80, 200 * 16, 133, -5, 96 + 3, 112]
    check_store(pool, ref, k, v, slots, err)
    assert gpu.kvq_check_error(err) == kvq.DEV_ERR_BITS["slot"]


def test_store_bf16_whole_range(gpu):
    pool = kvq.KVPool.allocate(4, 1, "fp8")
    ref = host_copy(pool)
    e = torch.arange(-133, 128, dtype=torch.float64)
    vals = torch.ldexp(torch.ones(261, dtype=torch.float64), e.int())
    rows = torch.zeros(48, 1, 128, dtype=torch.float64)
    for i in range(48):
        rows[i, 0] = vals[(i * 5) % 133:][:128] * (1.0 if i % 2 else -1.4921875)
    rows = rows.to(torch.bfloat16).cuda()
    check_store(pool, ref, rows, rows.flip(0), list(range(48)))


def test_store_rewrites_a_middle_row_and_starts_blocks_anew(gpu):
    pool = kvq.KVPool.allocate(3, 4, "fp8")
    ref = host_copy(pool)
    for i, (size, slots) in enumerate([(1.0, range(16)), (30.0, [7]), (0.01, [3]), (0.01, [0]),
                                       (0.5, [20]), (0.5, [17, 19]), (2.0, [47, 46, 45])]):
        slots = list(slots)
        if slots == [47, 46, 45]:  # falling slots: three runs, which race in one block
            continue
        check_store(pool, ref, randn(20 + i, len(slots), 4, 128, scale=size),
                    randn(40 + i, len(slots), 4, 128, scale=size), slots)


# ---- attention ------------------------------------------------------------------


def make_pool(kind, lens, heads, seed, dtype="f16", v_spread=False, poison=True):
    """A pool of scattered blocks filled through the store, and its tables.
    poison: rows behind each request's last token, and blocks of no request,
    hold NaN. v_spread: the size of V changes by up to 2^36 between blocks."""
    lens = np.asarray(lens)
    nblk = (lens + 15) // 16
    total = int(nblk.sum()) + 3
    perm = np.random.RandomState(seed).permutation(total)
    mb = max(1, int(nblk.max()))
    bt = np.full((len(lens), mb), -1, dtype=np.int64)
    at = 0
    slots = []
    for b, n in enumerate(nblk):
        bt[b, :n] = perm[at:at + n]
        at += n
        p = np.arange(lens[b])
        slots.append(bt[b, p // 16] * 16 + p % 16)
    slots = np.concatenate(slots)
    pool = kvq.KVPool.allocate(total, heads, kind)
    if poison:
        fill = {"fp8": 0x7F, "f16": 0xFF, "bf16": 0xFF}.get(kind, 0x33)
        pool.k.fill_(fill)
        pool.v.fill_(fill)
        if kind in ("int8", "int4"):
            pool.k_sz.fill_(-1)  # NaN scales and zeros
            pool.v_sz.fill_(-1)
    in_dt = kind if kind in DT else dtype
    n = len(slots)
    k = randn(seed + 1, n, heads, 128, dtype=in_dt)
    v = randn(seed + 2, n, heads, 128, dtype="bf16" if v_spread else in_dt)
    if v_spread:
        e = np.random.RandomState(seed).randint(-18, 19, (total,))
        v = (v.double() * torch.from_numpy(2.0 ** e[slots // 16])[:, None, None].cuda()).bfloat16()
        k = k.bfloat16()
    if n:
        kvq.kv_store_quant(pool, k, v, i64(slots))
    return pool, bt


def run_decode(pool, q, bt, lens, score=None, num_splits=0, err=None, stream=None):
    out = torch.full_like(q, float("nan"))
    msl = max(1, int(max(lens)))
    ws = torch.empty(kvq.paged_decode_attn_workspace_size(len(lens), q.shape[1], pool.kv_heads,
                                                          msl, num_splits),
                     dtype=torch.uint8, device="cuda")
    a = (q, out, i32(bt), i32(lens), msl, SM, num_splits, ws, err, stream)
    if score is None:
        kvq.paged_decode_attn(pool, *a)
    else:
        kvq.paged_decode_attn_scored(pool, score, *a)
    return out


def run_extend(pool, q, bt, lens, indptr, score=None, variant="auto", err=None):
    out = torch.full_like(q, float("nan"))
    ws = torch.empty(kvq.paged_extend_attn_workspace_size(len(lens), q.shape[0], q.shape[1],
                                                          pool.kv_heads, max(lens)),
                     dtype=torch.uint8, device="cuda")
    a = (q, out, i32(indptr), i32(lens), i32(bt), int(max(lens)), SM, ws, err, None, variant)
    if score is None:
        kvq.paged_extend_attn(pool, *a)
    else:
        kvq.paged_extend_attn_scored(pool, score, *a)
    return out


def compare(pool, got, q, bt, lens, indptr=None, cap=0.0, window=0, slopes=None, prefix=None):
    ref, amp, big = fp8_ref.attend(pool, q, bt, lens, SM, indptr, cap, window, slopes, prefix)
    if pool.kv_dtype in ("int8", "int4"):
        assert_close(got.double().cpu().numpy(), ref)
        return
    vmax = 0.0 if pool.kv_dtype == "bf16" else float(amp.max(initial=0.0))
    fp8_ref.assert_within(got, ref, amp, big, max(lens), vmax)


LENS = [0, 1, 15, 16, 17, 31, 33, 250, 513]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv", [(8, 8), (16, 8), (32, 8), (12, 4), (15, 5), (16, 1), (16, 2),
                                    (32, 2), (32, 32), (24, 3)])
def test_decode_fp8(gpu, dtype, hq, hkv):
    pool, bt = make_pool("fp8", LENS, hkv, 100 + hq, dtype)
    q = randn(7, len(LENS), hq, 128, dtype=dtype)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for splits in (0, 1, 3):
        out = run_decode(pool, q, bt, LENS, num_splits=splits, err=err)
        assert gpu.kvq_check_error(err) == 0
        compare(pool, out, q, bt, LENS)


@pytest.mark.parametrize("hq,hkv", [(8, 8), (32, 8)])
def test_decode_fp8_lone_and_long(gpu, hq, hkv):
    """One request alone, and a long one beside short ones."""
    for lens in ([641], [0, 1043, 0], [9001, 3, 700]):
        pool, bt = make_pool("fp8", lens, hkv, 11, "bf16")
        q = randn(8, len(lens), hq, 128, dtype="bf16")
        compare(pool, run_decode(pool, q, bt, lens), q, bt, lens)


@pytest.mark.parametrize("form", ["decode", "extend"])
@pytest.mark.parametrize("hkv", [2, 8])
def test_fp8_v_scales_far_apart(gpu, form, hkv):
    """V blocks whose scales lie up to 2^36 apart, bf16 queries of any size."""
    lens = [700, 90, 16]
    pool, bt = make_pool("fp8", lens, hkv, 12, "bf16", v_spread=True)
    if form == "decode":
        q = randn(9, 3, 4 * hkv, 128, dtype="bf16")
        q[1] *= 2.0 ** -40
        compare(pool, run_decode(pool, q, bt, lens), q, bt, lens)
    else:
        indptr = [0, 300, 390, 391]
        q = randn(9, 391, 4 * hkv, 128, dtype="bf16")
        for variant in ("mma_sync", "tcgen05"):
            compare(pool, run_extend(pool, q, bt, lens, indptr, variant=variant), q, bt, lens, indptr)


def test_fp8_blocks_of_zeros(gpu):
    """A scale of 0 makes its block's codes zeros, whatever they are."""
    lens = [100, 40]
    pool, bt = make_pool("fp8", lens, 2, 13)
    for name in ("k", "v"):
        getattr(pool, name + "_sz")[bt[0, 2]] = 0
        getattr(pool, name + "_sz")[bt[1, 0], 1] = 0
        getattr(pool, name)[bt[0, 2]] = 0x7F
        getattr(pool, name)[bt[1, 0], :, 1] = 0xFF
    q = randn(10, 2, 8, 128)
    compare(pool, run_decode(pool, q, bt, lens), q, bt, lens)
    indptr = [0, 90, 130]
    q = randn(10, 130, 8, 128)
    for variant in ("mma_sync", "tcgen05"):
        compare(pool, run_extend(pool, q, bt, lens, indptr, variant=variant), q, bt, lens, indptr)


def score_of(combo, hq, batch, lens, cap=4.0, window=37):
    """(Score, the reference's arguments). cap near the scores' own size."""
    cap = cap if "c" in combo else 0.0
    window = window if "w" in combo else 0
    slopes = prefix = None
    if "a" in combo:
        slopes = torch.exp2(-8.0 * torch.arange(1, hq + 1, dtype=torch.float32) / hq).cuda()
    if "p" in combo:
        prefix = np.array([(n * (2 * i + 1)) // (2 * batch) for i, n in enumerate(lens)], np.int32)
    s = kvq.Score(cap, window, slopes, None if prefix is None else i32(prefix))
    return s, dict(cap=cap, window=window, slopes=slopes, prefix=prefix)


@pytest.mark.parametrize("kind,dtype", [("fp8", "f16"), ("fp8", "bf16"), ("f16", "f16"),
                                        ("bf16", "bf16"), ("int8", "f16"), ("int8", "bf16"),
                                        ("int4", "f16"), ("int4", "bf16")])
@pytest.mark.parametrize("combo", ["c", "w", "a", "cwa"])
def test_decode_scored(gpu, kind, dtype, combo):
    for hq, hkv in ((8, 8), (32, 8), (12, 4), (24, 2)):
        pool, bt = make_pool(kind, LENS, hkv, 200 + hq, dtype)
        q = randn(17, len(LENS), hq, 128, dtype=dtype, scale=2.0)
        s, kw = score_of(combo, hq, len(LENS), LENS)
        compare(pool, run_decode(pool, q, bt, LENS, s), q, bt, LENS, **kw)


@pytest.mark.parametrize("window", [1, 15, 16, 17, 512, 100000])
def test_decode_windows(gpu, window):
    pool, bt = make_pool("fp8", LENS + [2000], 4, 31)
    q = randn(18, len(LENS) + 1, 16, 128)
    out = run_decode(pool, q, bt, LENS + [2000], kvq.Score(window=window))
    compare(pool, out, q, bt, LENS + [2000], window=window)


@pytest.mark.parametrize("cap", [1e-6, 0.5, 50.0, 1e6])
def test_decode_caps(gpu, cap):
    pool, bt = make_pool("fp8", LENS, 4, 32)
    q = randn(19, len(LENS), 16, 128, scale=8.0)
    compare(pool, run_decode(pool, q, bt, LENS, kvq.Score(cap)), q, bt, LENS, cap=cap)


def test_scores_of_nothing_are_the_plain_attention(gpu):
    pool, bt = make_pool("int8", LENS, 8, 33, poison=False)
    q = randn(20, len(LENS), 32, 128)
    assert torch.equal(run_decode(pool, q, bt, LENS, kvq.Score()), run_decode(pool, q, bt, LENS))


CHUNKS = [[1], [40, 0, 1, 130, 17, 16], [600, 3]]
CTX = [[777], [40, 50, 1, 400, 18, 300], [600, 900]]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("variant", ["mma_sync", "tcgen05"])
@pytest.mark.parametrize("hq,hkv", [(8, 8), (32, 8), (15, 5), (16, 1)])
def test_extend_fp8(gpu, dtype, variant, hq, hkv):
    for c, lens in zip(CHUNKS, CTX):
        pool, bt = make_pool("fp8", lens, hkv, 300 + hq, dtype)
        indptr = np.concatenate([[0], np.cumsum(c)])
        q = randn(27, int(indptr[-1]), hq, 128, dtype=dtype)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = run_extend(pool, q, bt, lens, indptr, variant=variant, err=err)
        assert gpu.kvq_check_error(err) == 0
        compare(pool, out, q, bt, lens, indptr)


@pytest.mark.parametrize("kind,dtype", [("fp8", "f16"), ("fp8", "bf16"), ("f16", "f16"),
                                        ("bf16", "bf16"), ("int8", "f16"), ("int8", "bf16"),
                                        ("int4", "f16"), ("int4", "bf16")])
@pytest.mark.parametrize("combo", ["c", "w", "a", "p", "wp", "cwap"])
def test_extend_scored(gpu, kind, dtype, combo):
    for c, lens in zip(CHUNKS, CTX):
        pool, bt = make_pool(kind, lens, 4, 400, dtype)
        indptr = np.concatenate([[0], np.cumsum(c)])
        q = randn(28, int(indptr[-1]), 12, 128, dtype=dtype, scale=2.0)
        s, kw = score_of(combo, 12, len(lens), lens)
        for variant in ("mma_sync",) if kind == "bf16" else ("mma_sync", "tcgen05"):
            out = run_extend(pool, q, bt, lens, indptr, s, variant)
            compare(pool, out, q, bt, lens, indptr, **kw)


@pytest.mark.parametrize("variant", ["mma_sync", "tcgen05"])
@pytest.mark.parametrize("cap", [1e-6, 0.5, 8.0, 50.0, 1e6])
def test_extend_caps(gpu, variant, cap):
    """Scores far below the cap, near it and beyond it in one tile."""
    lens, indptr = [150, 70], [0, 140, 200]
    pool, bt = make_pool("fp8", lens, 2, 41)
    q = randn(29, 200, 8, 128, scale=8.0)
    q[::3] *= 0.05
    out = run_extend(pool, q, bt, lens, indptr, kvq.Score(cap), variant)
    compare(pool, out, q, bt, lens, indptr, cap=cap)


@pytest.mark.parametrize("variant", ["mma_sync", "tcgen05"])
@pytest.mark.parametrize("window", [1, 16, 63, 64, 65, 300, 5000])
def test_extend_windows(gpu, variant, window):
    """Windows shorter than a tile, at its size and longer than the context."""
    lens, indptr = [900, 70], [0, 700, 770]
    pool, bt = make_pool("fp8", lens, 2, 42, "bf16")
    q = randn(30, 770, 4, 128, dtype="bf16")
    out = run_extend(pool, q, bt, lens, indptr, kvq.Score(window=window), variant)
    compare(pool, out, q, bt, lens, indptr, window=window)


@pytest.mark.parametrize("variant", ["mma_sync", "tcgen05"])
@pytest.mark.parametrize("scale", [0.0, -0.09])
def test_extend_other_softmax_scales(gpu, monkeypatch, variant, scale):
    monkeypatch.setitem(globals(), "SM", scale)
    lens, indptr = [200, 70], [0, 140, 200]
    pool, bt = make_pool("fp8", lens, 2, 43)
    q = randn(31, 200, 8, 128)
    for s, kw in ((None, {}), score_of("cwap", 8, 2, lens)):
        out = run_extend(pool, q, bt, lens, indptr, s, variant)
        compare(pool, out, q, bt, lens, indptr, **kw)


# ---- together, and as programs call them ---------------------------------------------


def test_bad_blocks_are_skipped_and_flagged(gpu):
    lens = [64, 100]
    pool, bt = make_pool("fp8", lens, 2, 14)
    bad = bt.copy()
    bad[0, 1], bad[1, 6] = pool.num_blocks, -7
    q = randn(11, 2, 8, 128)
    for score in (None, kvq.Score(30.0, 90)):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = run_decode(pool, q, bad, lens, score, err=err)
        assert gpu.kvq_check_error(err) == kvq.DEV_ERR_BITS["block_id"]
        assert torch.isfinite(out).all()


def test_prompt_then_steps(gpu):
    """A prompt stored and attended in two chunks, then decode steps: every
    output against the reference on what the pool holds at that moment."""
    heads, hq, n0 = 4, 16, 301
    pool = kvq.KVPool.allocate(64, heads, "fp8")
    perm = np.random.RandomState(3).permutation(64)
    bt = perm[None, :32]
    slots = np.array([perm[p // 16] * 16 + p % 16 for p in range(400)])
    k, v = randn(50, 400, heads, 128), randn(51, 400, heads, 128)
    k[100:] *= 5.0  # later tokens outgrow their blocks' scales
    q = randn(52, 400, hq, 128)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for a, b in ((0, 171), (171, n0)):
        kvq.kv_store_quant(pool, k[a:b], v[a:b], i64(slots[a:b]), err)
        out = run_extend(pool, q[a:b].contiguous(), bt, [b], [0, b - a], err=err)
        compare(pool, out, q[a:b], bt, [b], [0, b - a])
    step = kvq.DecodeStep(pool, 1, hq, 32, 512, torch.float16, fused=True)
    r2t = i32(np.pad(slots, (0, 112))[None])
    for n in range(n0, n0 + 21):
        out = step(r2t, i32([0]), i32([n + 1]), q[n:n + 1], k[n:n + 1], v[n:n + 1],
                   i64(slots[n:n + 1]), SM)
        compare(pool, out, q[n:n + 1], bt, [n + 1])
    assert gpu.kvq_check_error(step.dev_err) == 0 and gpu.kvq_check_error(err) == 0
    # a fork: the blocks copied, the copy attended
    dst = kvq.KVPool.allocate(64, heads, "fp8")
    ids = np.arange(21, dtype=np.int32)
    kvq.kvq_copy_blocks(pool, dst, i32(bt[0, :21]), i32(ids))
    a = run_decode(pool, q[:1].contiguous(), bt, [n0 + 21])
    assert torch.equal(a, run_decode(dst, q[:1].contiguous(), ids[None], [n0 + 21]))


@pytest.mark.parametrize("heads", [1, 3, 8])
def test_copy_and_swap(gpu, heads):
    pool, bt = make_pool("fp8", [200], heads, 15)
    host = kvq.KVPool.allocate(20, heads, "fp8", pinned=True)
    back = kvq.KVPool.allocate(20, heads, "fp8")
    ids = i32(bt[0])
    to = i32(np.arange(len(bt[0]))[::-1].copy())
    kvq.kvq_copy_blocks(pool, host, ids, to)
    kvq.kvq_copy_blocks(host, back, to, to)
    for n in ("k", "v", "k_sz", "v_sz"):
        assert torch.equal(getattr(back, n)[to.long()], getattr(pool, n)[ids.long()]), n


def test_graph_and_other_stream(gpu):
    """A step captured once and replayed on new inputs, on a stream of its own."""
    lens = [257, 64, 1000]
    pool, bt = make_pool("fp8", lens, 4, 16)
    s, kw = score_of("cwa", 16, 3, lens)
    q, k = randn(60, 3, 16, 128), randn(61, 3, 4, 128)
    slots = i64([bt[b, (n - 1) // 16] * 16 + (n - 1) % 16 for b, n in enumerate(lens)])
    out, out2 = torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty(kvq.paged_decode_attn_workspace_size(3, 16, 4, 1000), dtype=torch.uint8,
                     device="cuda")
    t, sl = i32(bt), i32(lens)

    def step():
        kvq.kv_store_quant(pool, k, k, slots)
        kvq.paged_decode_attn(pool, q, out, t, sl, 1000, SM, 0, ws)
        kvq.paged_decode_attn_scored(pool, s, q, out2, t, sl, 1000, SM, 0, ws)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        step()
    for seed in (70, 71):
        q.copy_(randn(seed, 3, 16, 128))
        k.copy_(randn(seed + 5, 3, 4, 128, scale=float(seed - 69)))
        g.replay()
        torch.cuda.synchronize()
        compare(pool, out, q, bt, lens)
        compare(pool, out2, q, bt, lens, **kw)


def test_offsets_past_32_bits(gpu):
    """A pool of over 2^32 bytes for K: the blocks used lie at its end."""
    heads, nb = 8, (1 << 32) // (16 * 8 * 128) + 64
    pool = kvq.KVPool.allocate(nb, heads, "fp8")
    n = 500
    bt = (nb - 1 - np.arange(32))[None]
    slots = np.array([bt[0, p // 16] * 16 + p % 16 for p in range(n)])
    k, v = randn(80, n, heads, 128), randn(81, n, heads, 128)
    kvq.kv_store_quant(pool, k, v, i64(slots))
    small = kvq.KVPool.allocate(32, heads, "fp8")
    ids = np.arange(32)[None]
    kvq.kv_store_quant(small, k, v, i64(np.arange(n)))
    q = randn(82, 1, 32, 128)
    a, b = run_decode(pool, q, bt, [n]), run_decode(small, q, ids, [n])
    assert torch.equal(a, b)
    q = randn(83, n, 32, 128)
    for variant in ("mma_sync", "tcgen05"):
        a = run_extend(pool, q, bt, [n], [0, n], variant=variant)
        assert torch.equal(a, run_extend(small, q, ids, [n], [0, n], variant=variant))
    compare(small, a, q, ids, [n], [0, n])
