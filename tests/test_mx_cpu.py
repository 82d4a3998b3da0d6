"""The biased router's and the MXFP4 calls' refusals, without a GPU: every
call here fails its checks (or has nothing to do), so nothing is launched."""
import ctypes

import pytest
import torch

import mixture_experts_layer_segments_amd as moe
import moe_inputs as mi

FAKE = 1 << 20     # 256-byte aligned non-null address, never dereferenced
DEC = mi.WORKLOADS["decode_bf16"]
DSK = mi.WORKLOADS["deepseek_v3_bf16"]


def _route(cfg, logits=FAKE, bias=FAKE, scale=1.0, ids=FAKE, w=FAKE):
    return moe.lib.moe_route_biased(ctypes.byref(moe.make_config(cfg)), logits, bias, scale, ids,
                                    w, None)


@pytest.mark.parametrize("scale", [0.0, -1.0, float("inf"), float("nan")])
def test_route_scale_must_be_finite_and_positive(scale):
    assert _route(DSK, scale=scale) == -1


def test_route_refusals():
    assert _route(DSK, logits=None) == -1
    assert _route(DSK, ids=None) == -1
    assert _route(DSK, w=FAKE + 2) == -1
    assert _route(DSK, bias=FAKE + 1) == -1
    assert _route(DSK.replace(k=40)) == -2
    assert _route(DSK.replace(topk_group=0)) == -1
    assert _route(DSK.replace(score="softmax", topk_group=9)) == -1
    assert _route(DSK.replace(T=0), logits=None, bias=None, ids=None, w=None) == 0


def test_groups_with_softmax_scores_only_where_a_bias_routes():
    """The plain router refuses them; sizes and the calls that do not route
    take the configuration."""
    cfg = DSK.replace(score="softmax")
    c = moe.make_config(cfg)
    assert moe.lib.moe_route_topk(ctypes.byref(c), FAKE, FAKE, FAKE, None) == -2
    assert moe.moe_workspace_size(cfg) == moe.moe_workspace_size(DSK) > 0
    assert moe.moe_num_segments(cfg) == 256
    assert _route(cfg.replace(T=0)) == 0
    assert _route(cfg, logits=None) == -1


@pytest.mark.parametrize("call,wide_at", [("moe_quantize_mxfp4", 0), ("moe_dequantize_mxfp4", 2)])
def test_row_conversion_refusals(call, wide_at):
    f = getattr(moe.lib, call)

    def go(dtype, rows, cols, wide=FAKE, q=FAKE, s=FAKE):
        a = [q, s]
        a.insert(wide_at, wide)
        return f(dtype, rows, cols, *a, None)
    assert go(2, 4, 32) == -1
    assert go(1, 4, 48) == -1
    assert go(1, 4, 0) == -1
    assert go(1, -1, 32) == -1
    assert go(1, 4, 32, wide=None) == -1
    assert go(1, 4, 32, wide=FAKE + 8) == -1
    assert go(1, 4, 32, q=FAKE + 4) == -1
    assert go(1, 4, 32, s=FAKE + 1) == -1
    assert go(1, 1 << 40, 64) == -2
    assert go(1, (1 << 29) + 1, 32) == -2
    assert go(0, 0, 32, None, None, None) == 0


def _ffn(cfg, a4=False, ws=None, wsb=None, **kw):
    c = moe.make_config(cfg)
    a = dict(x=FAKE, xs=FAKE, so=FAKE, se=FAKE, q13=FAKE, s13=FAKE, q2=FAKE, s2=FAKE, rs=None,
             y=FAKE)
    a.update(kw)
    x = [a["x"], a["xs"]] if a4 else [a["x"]]
    f = moe.lib.moe_grouped_ffn_w4a4 if a4 else moe.lib.moe_grouped_ffn_mxfp4w
    return f(ctypes.byref(c), *x, a["so"], a["se"], a["q13"], a["s13"], a["q2"], a["s2"], a["rs"],
             a["y"], FAKE if ws is None else ws, moe.moe_workspace_size(cfg) if wsb is None else wsb,
             None)


@pytest.mark.parametrize("a4", [False, True])
def test_grouped_ffn_refusals(a4):
    assert _ffn(DEC.replace(dtype="f32"), a4) == -2
    assert _ffn(DEC.replace(I=192), a4) == -2
    assert _ffn(DEC.replace(H=8192 + 64), a4) == -2
    for name in ("x", "so", "se", "q13", "s13", "q2", "s2", "y"):
        assert _ffn(DEC, a4, **{name: None}) == -1, name
    assert _ffn(DEC, a4, s13=FAKE + 2) == -1
    assert _ffn(DEC, a4, q2=FAKE + 8) == -1
    assert _ffn(DEC, a4, wsb=16) == -3
    assert _ffn(DEC.replace(T=0), a4, x=None, y=None) == 0
    if a4:
        assert _ffn(DEC, a4, xs=None) == -1
        assert _ffn(DEC, a4, xs=FAKE + 2) == -1


@pytest.mark.parametrize("call", ["moe_layer_forward_mxfp4w", "moe_layer_forward_w4a4"])
def test_layer_refusals(call):
    def go(cfg, scale=1.0, logits=FAKE, x=FAKE, shared=None, wsb=None, s13=FAKE, bias=None):
        c = moe.make_config(cfg)
        return getattr(moe.lib, call)(
            ctypes.byref(c), logits, bias, scale, x, FAKE, s13, FAKE, FAKE, *[shared] * 4, FAKE,
            FAKE, FAKE, FAKE, FAKE, FAKE, moe.moe_workspace_size(cfg) if wsb is None else wsb, None)
    assert go(DEC, scale=0.0) == -1
    assert go(DEC, logits=None) == -1
    assert go(DEC, x=FAKE + 4) == -1
    assert go(DEC, s13=None) == -1
    assert go(DEC, bias=FAKE + 2) == -1
    assert go(DEC, wsb=100) == -3
    assert go(DSK) == -1                      # the shared expert's weights are missing
    assert go(DEC.replace(I=64)) == -2
    assert go(DEC.replace(dtype="f32")) == -2
    assert go(DEC.replace(T=0), logits=None) == 0


def test_binding_checks_types_and_sizes():
    """Wrong types and short tensors never reach the library."""
    cfg = mi.MoEShape("b", T=4, H=128, E=8, k=2, I=128)
    lg = torch.zeros(4, 8)
    ids, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(ValueError, match="logits must be"):
        moe.moe_route_biased(cfg, lg.bfloat16(), None, 1.0, ids, w, 0)
    with pytest.raises(ValueError, match="bias must hold 8"):
        moe.moe_route_biased(cfg, lg, torch.zeros(7), 1.0, ids, w, 0)
    with pytest.raises(ValueError, match="topk_ids must be"):
        moe.moe_route_biased(cfg, lg, None, 1.0, ids.long(), w, 0)
    with pytest.raises(ValueError, match="on the GPU"):
        moe.moe_route_biased(cfg, lg, None, 1.0, ids, w, 0)
    src = torch.zeros(4, 64)
    q, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="not torch.float16"):
        moe.moe_quantize_mxfp4(src.half(), q, s, 0)
    with pytest.raises(ValueError, match="q must hold 128"):
        moe.moe_quantize_mxfp4(src, q[:3], s, 0)
    with pytest.raises(ValueError, match="scale must hold 8"):
        moe.moe_dequantize_mxfp4(q, s[:2], src, 0)
