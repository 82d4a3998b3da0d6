"""moe_route_biased on the GPU against the float64 oracle: ids equal, weights
within the rounding of one fp32 value."""
import numpy as np
import pytest
import torch

import moe_inputs as mi
from oracle import mx as omx
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_segments_amd as m
    return m


def _run(moe, cfg, lg, bias, scale):
    ids = torch.full((cfg.T, cfg.k), 99, dtype=torch.int32, device=gu.dev())
    w = torch.full((cfg.T, cfg.k), 99.0, device=gu.dev())
    b = None if bias is None else torch.from_numpy(bias).to(gu.dev())
    moe.moe_route_biased(cfg, torch.from_numpy(lg).to(gu.dev()), b, scale, ids, w)
    torch.cuda.synchronize()
    return ids.cpu().numpy(), w.cpu().numpy().astype(np.float64)


def _check(moe, cfg, lg, bias, scale=1.0, ties=False):
    ids, w = _run(moe, cfg, lg, bias, scale)
    ref_ids, ref_w, gap = omx.route_biased(cfg, lg, bias, scale)
    # an order that hangs on less than the rounding of a few 64-bit steps is
    # not decided by the formulas; no input here is that close
    assert ties or gap.min() > 2.0 ** -48
    assert (ids == ref_ids).all(), np.argwhere(ids != ref_ids)[:5]
    # one rounding to fp32 (2^-24; 2^-149 below the normal range) of a value
    # good to a few 2^-53
    np.testing.assert_allclose(w, ref_w, rtol=2.0 ** -24 * (1 + 1e-6), atol=2.0 ** -149)


CASES = {}
for score in ("softmax", "sigmoid"):
    for E, k, ng, tg, tn in [(1, 1, 1, 1, 1), (2, 2, 1, 1, 1), (7, 3, 1, 1, 1), (64, 2, 1, 1, 1),
                             (65, 8, 1, 1, 1), (128, 8, 1, 1, 1), (200, 32, 1, 1, 1),
                             (256, 8, 8, 4, 2), (512, 6, 16, 3, 1), (1000, 10, 1, 1, 1),
                             (1024, 32, 64, 8, 3), (24, 6, 4, 2, 6), (60, 5, 6, 2, 2),
                             (160, 6, 8, 3, 1), (33, 11, 11, 6, 3), (72, 8, 8, 4, 2),
                             (96, 4, 2, 1, 2), (16, 4, 16, 4, 1), (320, 8, 5, 3, 2)]:
        CASES[f"{score}-E{E}k{k}g{ng}"] = mi.MoEShape(
            "r", T=37, H=128, E=E, k=k, I=128, score=score, n_group=ng, topk_group=tg,
            group_score_topn=tn, renormalize=(E + ng) % 2)


@pytest.mark.parametrize("name", CASES)
def test_random(moe, name):
    cfg = CASES[name]
    rng = np.random.default_rng(cfg.E * 100 + cfg.k)
    lg = rng.standard_normal((cfg.T, cfg.E)).astype(np.float32)
    bias = (rng.standard_normal(cfg.E) * 0.1).astype(np.float32)
    _check(moe, cfg, lg, bias, 2.5)
    _check(moe, cfg, lg, None)


@pytest.mark.parametrize("name", ["softmax-E7k3g1", "sigmoid-E256k8g8", "sigmoid-E33k11g11",
                                  "softmax-E1024k32g64", "softmax-E72k8g8", "sigmoid-E200k32g1"])
def test_masked_experts_and_rows(moe, name):
    cfg = CASES[name]
    rng = np.random.default_rng(5)
    lg = rng.standard_normal((cfg.T, cfg.E)).astype(np.float32)
    for p, v in ((0.3, -np.inf), (0.1, np.nan), (0.1, np.finfo(np.float32).min)):
        lg[rng.random(lg.shape) < p] = v
    lg[3], lg[4], lg[5] = -np.inf, np.nan, np.finfo(np.float32).min
    lg[6, 1:] = -np.inf
    lg[6, 0] = 0
    bias = (rng.standard_normal(cfg.E) * 0.1).astype(np.float32)
    bias[-1], bias[cfg.E // 2] = -np.inf, np.nan
    _check(moe, cfg, lg, bias, 1.5)


@pytest.mark.parametrize("name", ["softmax-E64k2g1", "sigmoid-E128k8g1", "sigmoid-E256k8g8",
                                  "softmax-E320k8g5", "sigmoid-E60k5g6"])
def test_ties_go_to_the_lower_id(moe, name):
    """Logits and biases on a coarse grid: equal selection values and, summed
    from equal members, equal group scores."""
    cfg = CASES[name].replace(T=200)
    rng = np.random.default_rng(6)
    lg = (rng.integers(-2, 3, (cfg.T, cfg.E)) * 0.5).astype(np.float32)
    lg[lg == 0] = np.where(rng.random((lg == 0).sum()) < 0.5, -0.0, 0.0)
    lg[:20] = 0
    _check(moe, cfg, lg, None)
    if cfg.score == "sigmoid":     # (a softmax's sum may round either way)
        bias = (rng.integers(0, 3, cfg.E) * 0.25).astype(np.float32)
        _check(moe, cfg, lg, bias, 1.0, ties=True)


def test_saturated_and_extreme_logits(moe):
    """Scores at 1 and at 0, +inf, and a bias that outweighs every score."""
    cfg = mi.MoEShape("r", T=6, H=128, E=16, k=4, I=128, score="sigmoid")
    lg = np.zeros((6, 16), np.float32)
    lg[0] = np.linspace(30, 36, 16)          # 64-bit scores still differ
    lg[1] = np.linspace(100, 200, 16)        # all 1: ids in order
    lg[2] = -np.linspace(800, 900, 16)       # all 0: weights 0
    lg[3, 5], lg[3, 9] = np.inf, 3e38
    lg[4] = -np.linspace(80, 110, 16)
    lg[5] = np.linspace(-1e-38, 1e-38, 16)
    _check(moe, cfg, lg, None, ties=True)
    bias = np.linspace(0, 100, 16).astype(np.float32)
    _check(moe, cfg, lg, bias, ties=True)
    bias[3], bias[7] = np.inf, 3e38
    _check(moe, cfg, lg, bias, ties=True)
    _check(moe, cfg.replace(score="softmax"), lg, None, ties=True)
    _check(moe, cfg.replace(score="softmax", renormalize=0), lg, None, ties=True)


@pytest.mark.parametrize("name", ["softmax-E7k3g1", "sigmoid-E128k8g1", "softmax-E128k8g1",
                                  "sigmoid-E256k8g8", "softmax-E256k8g8", "softmax-E512k6g16",
                                  "sigmoid-E200k32g1", "softmax-E16k4g16"])
@pytest.mark.parametrize("step", [1, 16, 256])
def test_near_ties(moe, name, step):
    """Logits a few fp32 steps apart, among the picked and at the cut, in some
    tokens of a wave and not in others: no fp32 score tells them apart, the
    64-bit ones do."""
    cfg = CASES[name].replace(T=64)
    rng = np.random.default_rng(step)
    lg = rng.standard_normal((cfg.T, cfg.E)).astype(np.float32)
    lg[rng.random(lg.shape) < 0.05] = -np.inf
    for t in range(0, cfg.T, 3):
        v = np.float32(rng.uniform(0.5, 2.5))
        at = rng.choice(cfg.E, max(2, cfg.E // 3), replace=False)
        near = (v.view(np.int32) + step * rng.permutation(at.size)).astype(np.int32)
        lg[t, at] = near.view(np.float32)
    _check(moe, cfg, lg, None)
    # a large bias of one value: the sums tell them apart less, the order stays
    _check(moe, cfg, lg, np.full(cfg.E, 0.75, np.float32), 2.5)


def test_biases_of_both_signs_cancel_in_group_scores(moe):
    """Group scores near zero from large members: what a sum in fp32 loses is
    no order."""
    for score in ("softmax", "sigmoid"):
        cfg = mi.MoEShape("r", T=100, H=128, E=64, k=4, I=128, score=score, n_group=8,
                          topk_group=3, group_score_topn=8)
        rng = np.random.default_rng(12)
        lg = rng.standard_normal((cfg.T, 64)).astype(np.float32)
        half = rng.uniform(50, 100, 32).astype(np.float32)
        bias = np.empty(64, np.float32)
        bias[0::2], bias[1::2] = half, -half
        _check(moe, cfg, lg, bias)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 1000, 4097])
def test_batch_sizes(moe, T):
    cfg = CASES["sigmoid-E256k8g8"].replace(T=T)
    rng = np.random.default_rng(T)
    _check(moe, cfg, rng.standard_normal((T, 256)).astype(np.float32),
           (rng.standard_normal(256) * 0.1).astype(np.float32))


@pytest.mark.parametrize("T", [1025, 4098])
@pytest.mark.parametrize("name", ["softmax-E7k3g1", "softmax-E64k2g1", "softmax-E128k8g1",
                                  "sigmoid-E65k8g1", "sigmoid-E256k8g8", "softmax-E24k6g4",
                                  "sigmoid-E60k5g6", "sigmoid-E320k8g5", "softmax-E512k6g16",
                                  "softmax-E33k11g11", "sigmoid-E200k32g1", "softmax-E16k4g16"])
def test_larger_batches(moe, name, T):
    """Several tokens a wave, masked experts and whole masked rows among them."""
    cfg = CASES[name].replace(T=T)
    rng = np.random.default_rng(T + cfg.E)
    lg = rng.standard_normal((T, cfg.E)).astype(np.float32)
    lg[rng.random((T, cfg.E)) < 0.2] = -np.inf
    lg[::7] = np.finfo(np.float32).min
    bias = (rng.standard_normal(cfg.E) * 0.1).astype(np.float32)
    _check(moe, cfg, lg, bias, 2.5)


def test_offset_views(moe):
    """Rows that start off a 16-byte boundary (4-byte alignment suffices)."""
    cfg = CASES["softmax-E65k8g1"]
    rng = np.random.default_rng(8)
    lg = rng.standard_normal((cfg.T, cfg.E)).astype(np.float32)
    for E in (65, 64, 256):
        c = cfg.replace(E=E)
        buf = torch.empty(cfg.T * E + 1, device=gu.dev())
        buf[1:] = torch.from_numpy(rng.standard_normal(cfg.T * E).astype(np.float32)).to(gu.dev())
        v = buf[1:].view(cfg.T, E)
        ids, w = gu.empty((cfg.T, 8), torch.int32), gu.empty((cfg.T, 8), torch.float32)
        moe.moe_route_biased(c, v, None, 1.0, ids, w)
        ref, _, _ = omx.route_biased(c, v.cpu().numpy(), None)
        assert (ids.cpu().numpy() == ref).all()
    del lg
