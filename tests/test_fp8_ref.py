"""The FP8 reference against torch's own e4m3 and closed forms (no GPU), and
the argument checks of the FP8 and scored entry points."""
import ctypes

import numpy as np
import pytest
import torch

import fp8_ref
import paged_quantized_kv_store_gb300 as kvq
from paged_quantized_kv_store_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return kvq.load()


def test_codes_and_rounding_match_the_type():
    every = torch.arange(256, dtype=torch.uint8)
    v = every.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, fp8_ref.E4M3, equal_nan=True)
    x = np.concatenate([np.linspace(-448, 448, 200001), np.ldexp(np.linspace(-8, 8, 4001), -9)])
    mid = (fp8_ref.E4M3[:126] + fp8_ref.E4M3[1:127]) / 2
    x = np.concatenate([x, mid, -mid])
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(fp8_ref.encode(x.astype(np.float32).astype(np.float64)), want)


@pytest.mark.parametrize("q", [-30, -9, 0, 3, 15])
@pytest.mark.parametrize("m", [1.0, 1.5, 1.75, 1.7500001, 1.99])
def test_scale_is_the_smallest_that_holds(q, m):
    a = m * 2.0 ** q
    e = fp8_ref.scale_for(a)
    assert a <= 448 * 2.0 ** (e - 127) and (e == 1 or a > 448 * 2.0 ** (e - 128))


def test_growth_moves_normal_codes_exactly():
    codes = np.zeros((1, 16, 1, 128), np.uint8)
    scales = np.zeros((1, 1), np.uint8)
    row = np.linspace(-1, 1, 128)[None, None]
    fp8_ref.store_side(codes, scales, row, [0])
    before = fp8_ref.E4M3[codes[0, 0, 0]] * fp8_ref.unit(scales[0, 0])
    fp8_ref.store_side(codes, scales, row * 16, [1])
    after = fp8_ref.E4M3[codes[0, 0, 0]] * fp8_ref.unit(scales[0, 0])
    normal = np.abs(before) >= 2.0 ** -6 * fp8_ref.unit(scales[0, 0])
    assert normal.sum() > 100 and np.array_equal(before[normal], after[normal])


def _pool(**kw):
    d = dict(k=16, v=32, k_sz=48, v_sz=64, num_blocks=4, block_size=16, kv_heads=2,
             head_dim=128, kv_dtype=kvq.KVQ_FP8)
    d.update(kw)
    return kvq._Pool(*(d[f] for f, _ in kvq._Pool._fields_))


def test_fp8_pool_refusals(lib):
    f, p = lib.kv_store_quant, 256
    assert f(ctypes.byref(_pool()), None, None, 0, None, 0, None, None) == 0
    assert f(ctypes.byref(_pool(k_sz=None)), p, p, 0, p, 1, None, None) == 1
    assert f(ctypes.byref(_pool(v_sz=65)), p, p, 0, p, 1, None, None) == 1
    assert f(ctypes.byref(_pool(kv_heads=40000)), p, p, 0, p, 1, None, None) == 2
    assert f(ctypes.byref(_pool()), p, p, kvq.KVQ_FP8, p, 1, None, None) == 2
    assert f(ctypes.byref(_pool(kv_dtype=3)), p, p, 0, p, 1, None, None) == 2
    # the cascade has no FP8 form
    assert lib.paged_decode_attn_shared_prefix(
        ctypes.byref(_pool()), p, 0, p, p, 4, p, 2, 4, 64, 0.1, p, p, p, 1, 2, 2, 0, p, 1 << 30,
        None, None) == 2
    # copies are between pools of one kind
    assert lib.kvq_copy_blocks(ctypes.byref(_pool()), ctypes.byref(_pool(kv_dtype=kvq.KVQ_INT8)),
                               p, p, 3, None, None) == 1
    assert kvq.KVPool.allocate(3, 5, "fp8", device="cpu").nbytes() == 2 * (3 * 16 * 5 * 128 + 15)


@pytest.mark.parametrize("form", ["decode", "extend"])
def test_score_refusals(lib, form):
    p = 256

    def call(score, pool=None, q_dtype=0, hq=4, batch=2):
        sp = None if score is None else ctypes.byref(kvq._Score(*score))
        pool = ctypes.byref(pool or _pool())
        if form == "decode":
            return lib.paged_decode_attn_scored(pool, sp, p, q_dtype, p, p, 4, p, batch, hq, 64,
                                                0.1, 0, None, 0, None, None)
        return lib.paged_extend_attn_scored(pool, sp, p, q_dtype, p, p, p, p, 4, batch, 8, hq, 64,
                                            0.1, 0, None, 0, None, None)

    assert call(None) == 1
    assert call((-1.0, 0, None, None)) == 1
    assert call((float("nan"), 0, None, None)) == 1
    assert call((float("inf"), 0, None, None)) == 1
    assert call((1e-9, 0, None, None)) == 2 and call((1e9, 0, None, None)) == 2
    assert call((0.0, -1, None, None)) == 1
    assert call((0.0, 0, 258, None)) == 1 and call((0.0, 0, None, 257)) == 1
    assert call((30.0, 8, None, None), hq=3) == 1
    assert call((30.0, 8, None, None), q_dtype=kvq.KVQ_INT8) == 2
    assert call((30.0, 8, None, None), pool=_pool(kv_dtype=kvq.KVQ_BF16)) == 2
    assert call((30.0, 8, None, None), batch=-1) == 1


def test_score_struct_checks_its_tensors():
    s = kvq.Score(30.0, 8, torch.zeros(4), torch.zeros(2, dtype=torch.int32))
    c = s.c_struct(4, 2)
    assert c.softcap == 30.0 and c.window == 8 and c.alibi_slopes and c.prefix_lens
    for bad in (kvq.Score(alibi_slopes=torch.zeros(5)),
                kvq.Score(alibi_slopes=torch.zeros(4, dtype=torch.float64)),
                kvq.Score(alibi_slopes=torch.zeros(8)[::2]),
                kvq.Score(prefix_lens=torch.zeros(2, dtype=torch.int64)),
                kvq.Score(prefix_lens=torch.zeros(3, dtype=torch.int32))):
        with pytest.raises(ValueError):
            bad.c_struct(4, 2)
