"""Plain 64-bit references of the FP8 pool and of scored attention (tests only).

The store works token by token from the definition in kvq.h, on numpy arrays
of codes and scale bytes; the attention on the values that a pool stands for.
"""
from __future__ import annotations

import numpy as np
import torch

D, BLOCK = 128, 16

# value of every e4m3 code (0x7F and 0xFF are NaN)
E4M3 = np.array([(-1.0 if c & 0x80 else 1.0) *
                 (np.nan if (c & 0x7F) == 0x7F else
                  (c & 7) * 2.0 ** -9 if (c & 0x78) == 0 else
                  (8 + (c & 7)) * 2.0 ** (((c >> 3) & 15) - 10)) for c in range(256)])
_MAG = E4M3[:127]


def encode(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 codes, ties to the even code, 448 beyond it, NaN for NaN."""
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=1e300, neginf=-1e300)), 448.0)
    hi = np.searchsorted(_MAG, a).clip(max=126)
    lo = np.maximum(hi - 1, 0)
    up, down = _MAG[hi] - a, a - _MAG[lo]
    c = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    c = np.where(np.signbit(x), c | 0x80, c)
    return np.where(np.isnan(x), (c & 0x80) | 0x7F, c).astype(np.uint8)


def scale_for(amax: float) -> int:
    if amax == 0:
        return 0
    e = 1
    while 448.0 * 2.0 ** (e - 127) < amax:
        e += 1
    return e


def unit(e):
    e = np.asarray(e, dtype=np.int64)
    return np.where(e == 0, 0.0, np.ldexp(1.0, e - 127))


def store_side(codes, scales, rows, slots):
    """codes [nb, 16, H, 128], scales [nb, H] updated in place; rows float64 [N, H, 128]."""
    nb, heads = scales.shape
    runs = []
    for i, s in enumerate(slots):
        if not 0 <= s < nb * BLOCK:
            continue
        if runs and runs[-1][-1] == i - 1 and slots[i - 1] // BLOCK == s // BLOCK and slots[i - 1] < s:
            runs[-1].append(i)
        else:
            runs.append([i])
    for run in runs:
        blk = slots[run[0]] // BLOCK
        offs = [slots[i] % BLOCK for i in run]
        for h in range(heads):
            x = rows[run, h]
            fin = np.abs(x[np.isfinite(x)])
            old = 0 if 0 in offs else int(scales[blk, h])
            now = max(old, scale_for(fin.max() if fin.size else 0.0))
            if 0 not in offs and now > old:
                keep = [o for o in range(BLOCK) if o not in offs]
                c = encode(E4M3[codes[blk, keep, h]] * 2.0 ** (old - now))
                codes[blk, keep, h] = 0 if old == 0 else c
            scales[blk, h] = now
            with np.errstate(invalid="ignore"):
                y = x / (unit(now) if now else 1.0)
            codes[blk, offs, h] = encode(y)


def pool_values(pool, name):
    """[nb, 16, H, 128] float64 on the host: what the pool's K or V stands for."""
    c = getattr(pool, name).cpu().numpy()
    sz = getattr(pool, name + "_sz")
    if pool.kv_dtype == "fp8":
        e = sz.cpu().numpy()
        u = unit(e)[:, None, :, None]
        return np.where(u == 0, 0.0, E4M3[c] * u)
    if pool.kv_dtype in ("f16", "bf16"):
        dt = torch.float16 if pool.kv_dtype == "f16" else torch.bfloat16
        return getattr(pool, name).view(dt).double().cpu().numpy()
    f = sz.cpu().contiguous().view(torch.float16).double().numpy()
    f = f.reshape(pool.num_blocks, pool.kv_heads, BLOCK, 2).transpose(0, 2, 1, 3)
    if pool.kv_dtype == "int4":
        c = np.stack([c & 15, c >> 4], -1).reshape(*c.shape[:-1], D)
    return c * f[..., :1] + f[..., 1:]


def attend(pool, q, tables, lens, sm_scale, indptr=None, cap=0.0, window=0, slopes=None,
           prefix=None):
    """(outputs, amplitudes, largest score size) in 64 bits. q: device tensor
    [rows, Hq, 128]; tables, lens, indptr, prefix: numpy. The amplitude of an
    output is the weighted mean of its tokens' largest |v|: what a relative
    error in the weights is multiplied with."""
    k, v = pool_values(pool, "k"), pool_values(pool, "v")
    x = q.double().cpu().numpy()
    rows, hq, _ = x.shape
    g = hq // pool.kv_heads
    out = np.zeros_like(x)
    amp = np.zeros((rows, hq, 1))
    big = 0.0
    ptr = np.arange(len(lens) + 1) if indptr is None else indptr
    sl = None if slopes is None else slopes.double().cpu().numpy()
    for b, n in enumerate(lens):
        r = np.arange(ptr[b], ptr[b + 1])
        if n == 0 or r.size == 0:
            continue
        ids = tables[b, : (n + BLOCK - 1) // BLOCK]
        kb = k[ids].reshape(-1, pool.kv_heads, D)[:n]
        vb = v[ids].reshape(-1, pool.kv_heads, D)[:n]
        pos = np.arange(n - r.size, n)[:, None]
        at = np.arange(n)[None]
        seen = at <= pos
        if prefix is not None:
            seen = seen | (at < prefix[b])
        if window:
            seen = seen & (at > pos - window)
        for h in range(hq):
            s = x[r, h] @ kb[:, h // g].T * sm_scale
            big = max(big, float((np.abs(x[r, h]) @ np.abs(kb[:, h // g]).T * abs(sm_scale)).max()))
            if cap:
                s = cap * np.tanh(s / cap)
            if sl is not None:
                s = s - sl[h] * np.abs(pos - at)
            s = np.where(seen, s, -np.inf)
            w = np.exp(s - s.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            out[r, h] = w @ vb[:, h // g]
            amp[r, h] = w @ np.abs(vb[:, h // g]).max(1, keepdims=True)
    return out, amp, big


def assert_within(got, ref, amp, big, tokens, vmax):
    """|got - ref| within what the arithmetic allows:
      eps/2 of the output's type, relative to the value (one rounding);
      amp * 2^-11 (each weight rounded to fp16 once);
      amp * 2 * 2^-20 * big (scores summed in fp32: |ds| <= 2^-20 sum |q k| sm_scale,
        and the exponentials' 2^-22, enter numerator and denominator);
      tokens * 2^-23 * vmax (weights below fp16's normal range)."""
    eps = torch.finfo(got.dtype).eps / 2
    g = got.double().cpu().numpy()
    assert np.isfinite(g).all()
    tol = eps * np.abs(ref) + amp * (2.0 ** -11 + 2.0 ** -19 * (big + 1)) + tokens * 2.0 ** -23 * vmax
    err = np.abs(g - ref)
    bad = err > tol
    if bad.any():
        i = np.unravel_index(np.argmax(err - tol), err.shape)
        raise AssertionError(f"{bad.sum()} of {bad.size} outputs off; worst at {i}: got {g[i]}, "
                             f"ref {ref[i]}, allowed {tol[i]}")
