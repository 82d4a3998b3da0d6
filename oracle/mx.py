"""CPU oracle for MXFP4 experts and for the biased router -- TEST
INFRASTRUCTURE (see oracle/fp8.py: nothing of the HIP path calls it).

MXFP4 (OCP Microscaling formats): E2M1 elements (sign, 2 exponent bits with
bias 1, 1 mantissa bit; magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6), one E8M0 scale
2^(b - 127) per 32 consecutive elements of a row, b = 255 NaN.  A block's
exponent is the smallest integer in [-127, 127] with max|block| <= 6 * 2^s (0
for an all-zero block); codes are nearest, ties to even.  A block that holds
an infinity or NaN has scale 255 and zero codes.  float64 on exact values.
"""
from __future__ import annotations

import numpy as np

from . import moe_oracle as orc
from .fp8 import bf16_round, swiglu_hidden

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = 32
F32_MAX = float(np.finfo(np.float32).max)


def e2m1_encode(v) -> np.ndarray:
    """Code of the nearest E2M1 value of each |v| <= 6, ties to the even code,
    the sign bit following the input's."""
    a = np.abs(np.asarray(v, dtype=np.float64))
    # the borders between neighbours; on a border the even code (side "left"
    # where the lower code is even)
    mid = (E2M1[1:] + E2M1[:-1]) / 2
    code = np.searchsorted(mid, a, side="left")
    code = np.where((code < 7) & (a == mid[np.minimum(code, 6)]) & (code % 2 == 1), code + 1, code)
    return (code + 8 * np.signbit(v)).astype(np.uint8)


def e2m1_decode(codes) -> np.ndarray:
    c = np.asarray(codes)
    return np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]


def block_exponent(amax: float) -> int:
    """By search: the smallest s in [-127, 127] with amax <= 6 * 2^s."""
    if amax == 0:
        return 0
    s = int(np.clip(np.ceil(np.log2(amax / 6.0)) + 2, -127, 127))
    while s > -127 and amax <= np.ldexp(6.0, s - 1):
        s -= 1
    return s


def block_exponents(amax) -> np.ndarray:
    """block_exponent of every element: amax = m * 2^e with m in [0.5, 1), and
    6 * 2^s = 0.75 * 2^(s + 3)."""
    m, e = np.frexp(np.asarray(amax, dtype=np.float64))
    s = np.where(m <= 0.75, e - 3, e - 2).astype(np.int64)
    return np.where(m == 0, 0, np.clip(s, -127, 127))


def quantize_rows(x):
    """[.., C] -> (codes uint8 [.., C], E8M0 bytes uint8 [.., C / 32])."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(x.shape[:-1] + (-1, BLOCK))
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    s = block_exponents(np.abs(b).max(-1))
    codes = e2m1_encode(np.ldexp(b, -s[..., None]))
    return codes.reshape(x.shape), np.where(bad, 255, s + 127).astype(np.uint8)


def dequantize_rows(codes, e8m0) -> np.ndarray:
    v = e2m1_decode(codes).reshape(e8m0.shape + (BLOCK,))
    sc = np.where(e8m0 == 255, np.nan, np.ldexp(1.0, e8m0.astype(np.int64) - 127))
    return (v * sc[..., None]).reshape(codes.shape)


def fake_quant_rows(x) -> np.ndarray:
    return dequantize_rows(*quantize_rows(x))


def pack(codes) -> np.ndarray:
    """Two codes a byte, element 2i in the low half."""
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(q) -> np.ndarray:
    return np.stack((q & 15, q >> 4), -1).reshape(q.shape[:-1] + (-1,))


def route_biased(cfg, logits, bias=None, routed_scale=1.0):
    """Token by token.  Returns (ids [T, k], w float64 [T, k], gap [T]); gap
    is the smallest difference between two selection values (or group scores)
    that decided something, over their size: below a few 2^-53 the order is
    the rounding's."""
    T, E = logits.shape
    b = np.zeros(E) if bias is None else bias.astype(np.float64)
    ids = np.full((T, cfg.k), -1, dtype=np.int32)
    w = np.zeros((T, cfg.k))
    gap = np.full(T, np.inf)
    per = E // cfg.n_group
    for t in range(T):
        l = logits[t].astype(np.float64)
        live = [e for e in range(E) if l[e] > -F32_MAX and b[e] > -np.inf]
        l = np.minimum(l, F32_MAX)
        s = np.zeros(E)
        if live:
            if cfg.score == "sigmoid":
                with np.errstate(over="ignore"):
                    s[live] = 1.0 / (1.0 + np.exp(-l[live]))
            else:
                z = np.exp(l[live] - l[live].max())
                s[live] = z / z.sum()
        c = s + b
        pool = live
        if cfg.n_group > 1:
            gs = []
            for g in range(cfg.n_group):
                m = sorted((c[e] for e in live if e // per == g), reverse=True)
                gs.append(sum(m[:cfg.group_score_topn]) if m else -np.inf)
            order = sorted(range(cfg.n_group), key=lambda g: (-gs[g], g))
            keep = set(order[:cfg.topk_group])
            if cfg.topk_group < cfg.n_group:
                hi, lo = gs[order[cfg.topk_group - 1]], gs[order[cfg.topk_group]]
                if np.isfinite(hi) and np.isfinite(lo) and hi != lo:
                    gap[t] = min(gap[t], (hi - lo) / max(abs(hi), abs(lo)))
            pool = [e for e in live if e // per in keep]
        order = sorted(pool, key=lambda e: (-c[e], e))
        win = order[:cfg.k]
        for i in range(min(len(order) - 1, cfg.k)):
            hi, lo = c[order[i]], c[order[i + 1]]
            if np.isfinite(hi) and np.isfinite(lo) and hi != lo:
                gap[t] = min(gap[t], (hi - lo) / max(abs(hi), abs(lo)))
        ids[t, :len(win)] = win
        sw = s[win]
        if cfg.renormalize:
            sw = sw / sw.sum() if sw.sum() > 0 else np.zeros(len(win))
        w[t, :len(win)] = sw * float(np.float32(routed_scale))
    return ids, w, gap


def expert(x_rows, w13_e, w2_e, acts_fp4: bool) -> np.ndarray:
    """One expert's outputs on dequantized weights: h is rounded to bf16 (and
    through MXFP4, as the rows of x, with FP4 activations)."""
    if acts_fp4:
        x_rows = fake_quant_rows(x_rows)
    h = bf16_round(swiglu_hidden(x_rows, w13_e))
    if acts_fp4:
        h = fake_quant_rows(h)
    return h @ w2_e.T


def layer_forward(cfg, ids, w, x64, w13, w2, sw13=None, sw2=None, acts_fp4=False):
    """out [T, H] of routed ids / weights (id -1: nothing) on dequantized
    weights, before the output's own rounding; dropped slots of the
    fixed-capacity layout add nothing."""
    out = np.zeros((cfg.T, cfg.H))
    cap = cfg.T * cfg.k
    if cfg.capacity_factor_permille > 0:
        cap = orc.capacity(cfg.T * cfg.k, cfg.E, cfg.capacity_factor_permille)
    for e in range(cfg.E):
        t, j = (i[:cap] for i in np.nonzero(ids == e))   # in increasing t * k + j
        if t.size:
            out[t] += w[t, j][:, None] * expert(x64[t], w13[e], w2[e], acts_fp4)
    if sw13 is not None:
        out += expert(x64, sw13, sw2, acts_fp4)
    return out
