"""The MXFP4 and biased-routing oracle against facts that do not come from
it: the format's tables, brute force over all codes and all subsets, and the
router without a bias."""
import itertools

import numpy as np
import pytest

import moe_inputs as mi
from oracle import moe_oracle as orc
from oracle import mx as omx


def test_e2m1_values_and_rounding():
    """All 16 codes; ties fall to the even code; the middle values."""
    assert omx.e2m1_decode(np.arange(8)).tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6]
    assert omx.e2m1_decode(np.arange(8, 16)).tolist() == [0, -.5, -1, -1.5, -2, -3, -4, -6]
    v = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.2500001, 4.9999, 6.0, -0.0, -0.3, -5.0]
    c = [0, 2, 2, 4, 4, 6, 6, 1, 6, 7, 8, 9, 14]
    assert omx.e2m1_encode(v).tolist() == c


@pytest.mark.parametrize("amax,s", [(0.0, 0), (6.0, 0), (6.0000001, 1), (3.0, -1), (12.0, 1),
                                    (1.0, -2), (2.0 ** -149, -127), (3.4e38, 126),
                                    (6 * 2.0 ** -127, -127), (6.1 * 2.0 ** -127, -126)])
def test_block_exponent(amax, s):
    assert omx.block_exponent(amax) == s
    assert omx.block_exponents(np.array([amax, 1.0])).tolist() == [s, -2]


def test_block_exponents_agree_with_the_search():
    rng = np.random.default_rng(4)
    a = np.concatenate([rng.random(500) * np.exp2(rng.integers(-150, 128, 500)),
                        np.ldexp(6.0, np.arange(-140, 120)), np.ldexp(1.0, np.arange(-149, 128))])
    assert omx.block_exponents(a).tolist() == [omx.block_exponent(v) for v in a]


def test_quantize_is_nearest_and_round_trips():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((16, 96)) * np.exp2(rng.integers(-20, 20, (16, 1)))
    x[3, 32:64] = 0
    c, s = omx.quantize_rows(x)
    back = omx.dequantize_rows(c, s)
    grid = omx.e2m1_decode(np.arange(16))
    for r in range(16):
        for b in range(3):
            sc = 2.0 ** (int(s[r, b]) - 127)
            blk = x[r, 32 * b:32 * b + 32]
            assert np.abs(blk).max() <= 6 * sc
            if np.abs(blk).max() > 0:
                assert np.abs(blk).max() > 3 * sc      # the next smaller scale is too small
            best = np.abs(blk[:, None] - grid * sc).min(1)
            assert (np.abs(back[r, 32 * b:32 * b + 32] - blk) == best).all()
    assert (omx.dequantize_rows(*omx.quantize_rows(back)) == back).all()
    assert (omx.unpack(omx.pack(c)) == c).all()
    x[0, 5], x[1, 40] = np.inf, np.nan
    c, s = omx.quantize_rows(x)
    assert s[0, 0] == 255 and s[1, 1] == 255 and (c[0, :32] == 0).all()
    assert np.isnan(omx.dequantize_rows(c, s)[0, :32]).all()


def test_route_without_bias_is_the_plain_router():
    """No bias: sigmoid scores order experts as their logits do, and the full
    softmax does too (the plain router's renormalised weights differ only in
    the denominator, which renormalisation removes)."""
    for kw in (dict(score="sigmoid"), dict(score="softmax"),
               dict(score="sigmoid", n_group=4, topk_group=2, group_score_topn=2)):
        cfg = mi.MoEShape("r", T=50, H=128, E=32, k=4, I=128, seed=5, **kw)
        lg = mi.logits(cfg)
        ids, w, _ = omx.route_biased(cfg, lg)
        ref_ids, ref_w, _ = orc.route(cfg, lg)
        assert (ids == ref_ids).all()
        np.testing.assert_allclose(w, ref_w, rtol=1e-12)


def test_route_biased_against_all_subsets():
    """The winners are the k-subset with the largest selection values among
    the subsets the kept groups allow; weights follow the scores alone."""
    rng = np.random.default_rng(2)
    cfg = mi.MoEShape("r", T=40, H=128, E=8, k=3, I=128, score="sigmoid", n_group=4,
                      topk_group=2, group_score_topn=1, seed=3)
    lg = rng.standard_normal((40, 8)).astype(np.float32)
    b = (rng.standard_normal(8) * 0.5).astype(np.float32)
    ids, w, _ = omx.route_biased(cfg, lg, b, 2.5)
    s = 1 / (1 + np.exp(-lg.astype(np.float64)))
    c = s + b.astype(np.float64)
    for t in range(40):
        gs = [max(c[t, 2 * g], c[t, 2 * g + 1]) for g in range(4)]
        keep = max(itertools.combinations(range(4), 2), key=lambda p: sum(gs[g] for g in p))
        best = max(itertools.combinations([e for e in range(8) if e // 2 in keep], 3),
                   key=lambda p: sum(c[t, list(p)]))
        assert sorted(ids[t]) == sorted(best)
        assert (np.diff(c[t, ids[t]]) < 0).all()
        np.testing.assert_allclose(w[t], 2.5 * s[t, ids[t]] / s[t, ids[t]].sum(), rtol=1e-12)


def test_route_biased_masks():
    cfg = mi.MoEShape("r", T=4, H=128, E=4, k=3, I=128, score="softmax", renormalize=0)
    lg = np.zeros((4, 4), np.float32)
    lg[0] = -np.inf
    lg[1] = [-np.inf, np.nan, 1, np.finfo(np.float32).min]
    lg[2] = [np.inf, 0, np.inf, 0]
    ids, w, _ = omx.route_biased(cfg, lg, np.array([0, 0, 0, -np.inf], np.float32), 1.0)
    assert ids.tolist() == [[-1] * 3, [2, -1, -1], [0, 2, 1], [0, 1, 2]]
    assert w[0].tolist() == [0, 0, 0] and w[1].tolist() == [1, 0, 0]
    assert w[2].tolist() == [0.5, 0.5, 0]
    np.testing.assert_allclose(w[3], 1 / 3)
