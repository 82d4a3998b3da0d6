"""Helpers of the MXFP4 and biased-routing tests: seeded operands on the host
and the device, the oracle's outputs and how far the kernels' may be from
them."""
from __future__ import annotations

import numpy as np
import torch

from oracle import mx as omx
from oracle.fp8 import bf16_round
from tests import gpu_util as gu

BF16_HALF = 2.0 ** -8    # half a bf16 step, relative to the value


def bf16_rows(rng, rows, cols, std=1.0):
    """Rows of bf16 values (float64)."""
    return bf16_round(rng.standard_normal((rows, cols)) * std)


def to_bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(gu.dev()).bfloat16()


def u8(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(gu.dev())


class Experts:
    """n experts of H x I in MXFP4: the packed codes and scales, and the
    values they stand for."""

    def __init__(self, rng, n, H, I, std=0.05):
        self.q13, self.s13, self.w13 = self._mats(rng, n, 2 * I, H, std)
        self.q2, self.s2, self.w2 = self._mats(rng, n, H, I, std)

    @staticmethod
    def _mats(rng, n, R, C, std):
        # rows of different size, so that a scale read from another row shows
        w = rng.standard_normal((n, R, C)) * std * np.exp2(rng.integers(-2, 3, (n, R, 1)))
        c, s = omx.quantize_rows(w)
        return omx.pack(c), s, omx.dequantize_rows(c, s)

    def device(self):
        return tuple(u8(a) for a in (self.q13, self.s13, self.q2, self.s2))


def expert_tol(x_rows, w13, w2, acts_fp4):
    """(y, tol) of one expert's rows: the oracle's outputs before their own
    rounding, and a bound on the kernel's distance from them.

    The kernel's fp32 sums of K terms in another order are taken to be within
    2^-20 sqrt(K) of the root-sum-square of the terms (16 times the usual size
    of that error), silu's exp and division within 2^-20 of h.  Where that
    band around an element of h holds two bf16 values (or two codes, or its
    block two scales), the kernel may hold the other one: the slack of y is
    the sum of those steps times |W2|."""
    I = w13.shape[0] // 2
    K = x_rows.shape[1]
    x = omx.fake_quant_rows(x_rows) if acts_fp4 else x_rows
    wg, wu = w13[:I], w13[I:]
    g, u = x @ wg.T, x @ wu.T
    g2, u2 = np.sqrt(x ** 2 @ (wg ** 2).T), np.sqrt(x ** 2 @ (wu ** 2).T)
    with np.errstate(over="ignore"):
        sig = 1.0 / (1.0 + np.exp(-g))
    h = g * sig * u
    dh = 2.0 ** -20 * (np.sqrt(K) * (np.abs(sig * (1 + g * (1 - sig)) * u) * g2 +
                                     np.abs(g * sig) * u2) + np.abs(h))
    held = bf16_round(h)
    lo, hi = bf16_round(h - dh), bf16_round(h + dh)
    step = np.abs(hi - lo)
    if acts_fp4:
        # per block: the scales its band allows, and the codes each gives
        def blocks(a):
            return a.reshape(a.shape[0], -1, 32)
        a_lo = np.maximum(np.abs(blocks(h)) - blocks(dh), 0).max(-1)
        a_hi = (np.abs(blocks(h)) + blocks(dh)).max(-1)
        exps = [omx.block_exponents(bf16_round(a)) for a in (a_lo, a_hi)]
        vals = []
        for s in exps:
            sc = np.ldexp(1.0, s)[..., None]
            for v in (lo, hi):
                vals.append((omx.e2m1_decode(omx.e2m1_encode(np.clip(blocks(v) / sc, -6, 6))) *
                             sc).reshape(h.shape))
        held = omx.fake_quant_rows(held)
        step = np.abs(np.array(vals) - held).max(0)
    y = held @ w2.T
    acc = 2.0 ** -20 * np.sqrt(I) * np.sqrt(held ** 2 @ (w2 ** 2).T)
    return y, step @ np.abs(w2).T + acc


def check_close(got, ref, tol, what=""):
    """|got - ref| <= tol + half a bf16 step of ref (and of what tol adds)."""
    lim = tol + BF16_HALF * (np.abs(ref) + tol)
    bad = ~(np.abs(got - ref) <= lim)
    assert not bad.any(), (
        f"{what}: {bad.sum()} of {bad.size} elements off, worst "
        f"{np.abs(got - ref)[bad].max()} at {np.argwhere(bad)[0]}, allowed {lim[bad].min()}")
    # the slack must stay small beside the outputs, or the check means nothing
    assert np.median(tol) <= 0.02 * np.abs(ref).max(), (np.median(tol), np.abs(ref).max())


def quantize(moe, t):
    """The library's MXFP4 codes and scales of a device tensor."""
    q = torch.empty(t.shape[:-1] + (t.shape[-1] // 2,), dtype=torch.uint8, device=t.device)
    s = torch.empty(t.shape[:-1] + (t.shape[-1] // 32,), dtype=torch.uint8, device=t.device)
    moe.moe_quantize_mxfp4(t, q, s)
    return q, s
