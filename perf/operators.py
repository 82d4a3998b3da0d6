"""Cases of the biased router and of the microscaled 4-bit (MXFP4) operators:
their inputs, one pass through each, and the work a pass cannot do without.

``own`` False runs the plain form (elementary torch operations), True the
library's calls.  Kinds of case:

``route``   moe_route_biased: softmax or sigmoid scores, a selection bias per
            expert, expert groups, top-k, renormalised and scaled weights.
``rows``    moe_quantize_mxfp4 and moe_dequantize_mxfp4: rows through E2M1
            codes with one power-of-two scale per 32 elements and back.
``w4``      moe_grouped_ffn_mxfp4w: the grouped SwiGLU experts on MXFP4
            weights and bf16 activations.
``w4a4``    moe_quantize_mxfp4 of the permuted rows and
            moe_grouped_ffn_w4a4: MXFP4 activations too.
"""
import functools
import math

import numpy as np
import torch

own = False

FLT_MAX = float(torch.finfo(torch.float32).max)
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ the cases
def _route(name, T, E, k, score, n_group=1, topk_group=1, topn=1, renorm=True, scale=1.0,
           masked=False):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "score": score,
            "n_group": n_group, "topk_group": topk_group, "topn": topn, "renorm": renorm,
            "scale": scale, "masked": masked}


def _rows(name, rows, cols):
    return {"name": name, "op": "rows", "rows": rows, "cols": cols}


def _ffn(name, op, T, H, E, k, I, zipf):
    return {"name": name, "op": op, "T": T, "H": H, "E": E, "k": k, "I": I, "zipf": zipf}


def listed():
    return [
        # one token of a decode step through the group-limited router of the
        # DeepSeek-V3-shaped layer: launch latency
        _route("route_token", 1, 256, 8, "sigmoid", 8, 4, 2, True, 2.5),
        # its prefill batch, padded: whole rows and some experts masked
        _route("route_prefill_groups", 4096, 256, 8, "sigmoid", 8, 4, 2, True, 2.5, masked=True),
        # the ragged layer's batch: softmax scores over an odd batch, flat top-k
        _route("route_softmax", 16383, 128, 8, "softmax", renorm=False),
        # activations of a 64-token decode batch
        _rows("rows_decode", 64, 8192),
        # activations of a long prefill, or a shard of expert weights
        _rows("rows_prefill", 65537, 4096),
        # one token through 8 of 256 experts: eight weight streams of one row
        _ffn("w4_token", "w4", 1, 7168, 256, 8, 2048, 0.0),
        # the 64-token decode layer: every active expert's weights once
        _ffn("w4_decode", "w4", 64, 8192, 64, 2, 2048, 0.0),
        # prefill with a mild skew: segments of 60 to 260 rows
        _ffn("w4_prefill", "w4", 4000, 8192, 64, 2, 2048, 0.12),
        # ragged segments, empty ones to thousands of rows, odd batch
        _ffn("w4_ragged", "w4", 5003, 4096, 128, 8, 1536, 1.5),
        # FP4 activations: a decode batch, the DeepSeek-V3-shaped prefill, and
        # the ragged layer at its full batch
        _ffn("w4a4_decode", "w4a4", 64, 8192, 64, 2, 2048, 0.0),
        _ffn("w4a4_prefill", "w4a4", 4096, 7168, 256, 8, 2048, 1.0),
        _ffn("w4a4_ragged", "w4a4", 16384, 4096, 128, 8, 1536, 1.5),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "rows", "w4", "w4", "w4a4", "w4a4"])
    if op == "route":
        E = _log_int(rng, 2, 512)
        T = _log_int(rng, 1, 16384)
        k = rng.randint(1, min(E, 16))
        score = rng.choice(["softmax", "sigmoid"])
        n_group, topk_group, topn = 1, 1, 1
        if rng.random() < 0.5:
            n_group = rng.choice([2, 4, 8, 16])
            per = max(2, E // n_group)
            E = n_group * per
            k = min(k, E)
            topk_group = rng.randint(min(n_group, -(-k // per)), n_group)
            topn = rng.randint(1, 2)
        case = _route("", T, E, k, score, n_group, topk_group, topn, rng.random() < 0.7,
                      rng.choice([1.0, 2.5]), rng.random() < 0.3)
    elif op == "rows":
        cols = 32 * _log_int(rng, 1, 512)
        case = _rows("", _log_int(rng, 1, max(1, 65537 * 4096 // cols)), cols)
    else:
        H, I = 128 * _log_int(rng, 2, 64), 128 * _log_int(rng, 1, 32)
        E = _log_int(rng, 1, 256)
        k = rng.randint(1, min(E, 8))
        # at most the largest listed case's weights and row products
        while E > k and E * H * I > 256 * 7168 * 2048:
            E -= 1
        most = max(1, int(131072 * 4096 * 1536 / (k * H * I)))
        case = _ffn("", op, _log_int(rng, 1, min(16384, most)), H, E, k, I,
                    rng.choice([0.0, 0.12, 1.0, 1.5]))
    del case["name"]
    return case


# ------------------------------------------------------------------ the inputs
@functools.lru_cache(maxsize=64)
def _counts(T, E, k, zipf):
    """Rows per expert (busiest first where zipf > 0): every token picks its k
    experts by Gumbel noise over the popularity log((i + 1)^-zipf)."""
    rng = np.random.default_rng([T, E, k, int(zipf * 1000)])
    z = rng.gumbel(size=(T, E)) - zipf * np.log(np.arange(1, E + 1))
    ids = np.argpartition(-z, k - 1, axis=1)[:, :k]
    return tuple(int(n) for n in np.bincount(ids.ravel(), minlength=E))


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _pow2(s):
    """2^s in 64 bits, exactly."""
    return ((s.long() + 1023) << 52).view(torch.float64)


def _quantize(x):
    """Codes (values of E2M1, signed) and exponents of rows in 32-blocks: the
    smallest power of two with max|block| <= 6 * 2^s, ties to even."""
    b = x.float().reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1)
    m, e = torch.frexp(amax)
    s = torch.where(m <= 0.75, e - 3, e - 2)
    s = torch.where(amax == 0, torch.zeros_like(s), s).clamp(-127, 127)
    v = (b.double() * _pow2(-s).unsqueeze(-1)).float()
    a = v.abs()
    r = torch.where(a < 2, torch.round(a * 2) * 0.5,
                    torch.where(a < 4, torch.round(a), torch.round(a * 0.5) * 2))
    return torch.copysign(r, v), s


def _values(v, s):
    """The rows that codes and exponents stand for, in 32 bits."""
    return (v.double() * _pow2(s).unsqueeze(-1)).float().flatten(-2)


def _pack(v):
    """E2M1 values -> codes, two a byte, the even element in the low half."""
    a = v.abs()
    c = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a * 0.5 + 4)).to(torch.uint8)
    c = c + (torch.signbit(v).to(torch.uint8) << 3)
    c = c.reshape(*c.shape[:-2], -1)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _mx_weights(g, n, rows, cols):
    """n matrices of N(0, 0.02) weights in MXFP4."""
    q = torch.empty(n, rows, cols // 2, dtype=torch.uint8, device="cuda")
    sc = torch.empty(n, rows, cols // 32, dtype=torch.uint8, device="cuda")
    for i in range(n):
        w = torch.randn(rows, cols, generator=g, device="cuda") * 0.02
        v, s = _quantize(w)
        q[i] = _pack(v)
        sc[i] = (s + 127).to(torch.uint8)
    return q, sc


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": case}
    if case["op"] == "route":
        T, E = case["T"], case["E"]
        rank = torch.randperm(E, generator=g, device="cuda")
        lg = torch.randn(T, E, generator=g, device="cuda") - torch.log1p(rank.float()) * 0.5
        if case["masked"]:
            lg[torch.rand(T, E, generator=g, device="cuda") < 0.05] = float("-inf")
            lg[torch.rand(T, generator=g, device="cuda") < 0.05] = -FLT_MAX
        st["logits"] = lg
        st["bias"] = torch.randn(E, generator=g, device="cuda") * 0.05
        st["ids"] = torch.empty(T, case["k"], dtype=torch.int32, device="cuda")
        st["w"] = torch.empty(T, case["k"], dtype=torch.float32, device="cuda")
    elif case["op"] == "rows":
        R, C = case["rows"], case["cols"]
        # channels of different size, as activations have
        amp = torch.exp(torch.randn(C, generator=g, device="cuda"))
        st["x"] = torch.empty(R, C, dtype=torch.bfloat16, device="cuda")
        for r in range(0, R, 8192):
            n = min(8192, R - r)
            st["x"][r:r + n] = torch.randn(n, C, generator=g, device="cuda") * amp
        st["q"] = torch.empty(R, C // 2, dtype=torch.uint8, device="cuda")
        st["s"] = torch.empty(R, C // 32, dtype=torch.uint8, device="cuda")
        st["y"] = torch.empty(R, C, dtype=torch.bfloat16, device="cuda")
    else:
        T, H, E, k, I = (case[n] for n in ("T", "H", "E", "k", "I"))
        R = T * k
        order = torch.randperm(E, generator=g, device="cuda").tolist()
        cnt = _counts(T, E, k, case["zipf"])
        st["lens"] = [cnt[o] for o in order]
        st["seg_offsets"] = torch.tensor([0] + list(np.cumsum(st["lens"])), dtype=torch.int32,
                                         device="cuda")
        st["seg_expert"] = torch.arange(E, dtype=torch.int32, device="cuda")
        st["x"] = torch.randn(R, H, generator=g, device="cuda").bfloat16()
        st["row_scale"] = torch.rand(R, generator=g, device="cuda") * 0.9 + 0.05
        st["w13"], st["w13_s"] = _mx_weights(g, E, 2 * I, H)
        st["w2"], st["w2_s"] = _mx_weights(g, E, H, I)
        st["y"] = torch.empty(R, H, dtype=torch.bfloat16, device="cuda")
        if case["op"] == "w4a4":
            st["xq"] = torch.empty(R, H // 2, dtype=torch.uint8, device="cuda")
            st["xs"] = torch.empty(R, H // 32, dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    c = st["case"]
    if own:
        return _run_own(st, c)
    if c["op"] == "route":
        return _plain_route(st["logits"], st["bias"], c)
    if c["op"] == "rows":
        return _plain_rows(st["x"])
    return _plain_ffn(st, c)


def _config(st, c):
    """The layer description, made once and kept beside the buffers."""
    import mixture_experts_layer_segments_amd as moe
    if "cfg" not in st:
        cfg = moe.MoEConfig(T=c["T"], E=c["E"], k=c["k"], H=c.get("H", 128), I=c.get("I", 128),
                            score=(moe.MOE_SCORE_SIGMOID if c.get("score") == "sigmoid"
                                   else moe.MOE_SCORE_SOFTMAX),
                            n_group=c.get("n_group", 1), topk_group=c.get("topk_group", 1),
                            group_score_topn=c.get("topn", 1),
                            renormalize=int(c.get("renorm", True)), split_ways=1,
                            act_dtype=moe.MOE_DT_BF16)
        if c["op"] != "route":
            st["ws"] = torch.empty(moe.moe_workspace_size(cfg), dtype=torch.uint8, device="cuda")
        st["cfg"] = cfg
    return moe, st["cfg"]


def _run_own(st, c):
    if c["op"] == "route":
        moe, cfg = _config(st, c)
        moe.moe_route_biased(cfg, st["logits"], st["bias"], c["scale"], st["ids"], st["w"])
        return st["ids"], st["w"]
    if c["op"] == "rows":
        import mixture_experts_layer_segments_amd as moe
        moe.moe_quantize_mxfp4(st["x"], st["q"], st["s"])
        moe.moe_dequantize_mxfp4(st["q"], st["s"], st["y"])
        return st["y"]
    moe, cfg = _config(st, c)
    if c["op"] == "w4":
        moe.moe_grouped_ffn_mxfp4w(cfg, st["x"], st["seg_offsets"], st["seg_expert"], st["w13"],
                                   st["w13_s"], st["w2"], st["w2_s"], st["row_scale"], st["y"],
                                   st["ws"])
    else:
        moe.moe_quantize_mxfp4(st["x"], st["xq"], st["xs"])
        moe.moe_grouped_ffn_w4a4(cfg, st["xq"], st["xs"], st["seg_offsets"], st["seg_expert"],
                                 st["w13"], st["w13_s"], st["w2"], st["w2_s"], st["row_scale"],
                                 st["y"], st["ws"])
    return st["y"]


def _plain_route(logits, bias, c):
    """Scores in 64 bits (they are compared with each other)."""
    l = logits.double()
    off = ~(l > -FLT_MAX) | ~(bias.double() > -math.inf)   # masked experts (NaN among them)
    l = l.clamp(max=FLT_MAX)
    if c["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        top = torch.where(off, torch.full_like(l, -math.inf), l).amax(-1, keepdim=True)
        e = torch.where(off, torch.zeros_like(l), torch.exp(l - top))
        s = e / e.sum(-1, keepdim=True)
    s = torch.where(off, torch.zeros_like(s), s)
    pick = torch.where(off, torch.full_like(s, -math.inf), s + bias.double())
    T, E = pick.shape
    if c["n_group"] > 1:
        per = E // c["n_group"]
        best = pick.view(T, -1, per).sort(stable=True, dim=-1, descending=True)[0][..., :c["topn"]]
        gs = torch.where(best > -math.inf, best, torch.zeros_like(best)).sum(-1)
        gs = torch.where(best[..., 0] > -math.inf, gs, torch.full_like(gs, -math.inf))
        keep = gs.sort(stable=True, dim=-1, descending=True)[1][:, :c["topk_group"]]
        kept = torch.zeros_like(gs, dtype=torch.bool).scatter_(1, keep, True)
        pick = torch.where(kept.repeat_interleave(per, 1), pick, torch.full_like(pick, -math.inf))
    v, ids = pick.sort(stable=True, dim=-1, descending=True)
    v, ids = v[:, :c["k"]], ids[:, :c["k"]]
    w = torch.where(v > -math.inf, s.gather(1, ids), torch.zeros_like(v))
    if c["renorm"]:
        t = w.sum(-1, keepdim=True)
        w = torch.where(t > 0, w / t, torch.zeros_like(w))
    ids = torch.where(v > -math.inf, ids, torch.full_like(ids, -1))
    return ids.int(), (w * c["scale"]).float()


def _plain_rows(x):
    y = torch.empty_like(x)
    for r in range(0, x.shape[0], 16384):
        v, s = _quantize(x[r:r + 16384])
        y[r:r + 16384] = _values(v, s)
    return y


def _weight(q, s, lut):
    """One matrix of MXFP4 weights in fp32."""
    v = torch.stack((lut[(q & 15).int()], lut[(q >> 4).int()]), -1).reshape(q.shape[0], -1, 32)
    return _values(v, s.long() - 127)


def _plain_ffn(st, c):
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    I = c["I"]

    def act(rows):
        """FP4 activations: bf16 rows as their codes stand for."""
        if c["op"] == "w4":
            return rows.float()
        return _values(*_quantize(rows))

    r0 = 0
    for e, n in enumerate(st["lens"]):
        if n == 0:
            continue
        gu = act(st["x"][r0:r0 + n]) @ _weight(st["w13"][e], st["w13_s"][e], lut).t()
        g, u = gu[:, :I], gu[:, I:]
        # h is held in bf16 by definition (it is what FP4 activations quantize)
        h = (g / (1.0 + torch.exp(-g)) * u).bfloat16()
        y = act(h) @ _weight(st["w2"][e], st["w2_s"][e], lut).t()
        st["y"][r0:r0 + n] = y * st["row_scale"][r0:r0 + n, None]
        r0 += n
    return st["y"]


# ------------------------------------------------------------------ the work
def work(case):
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * (4 * E + 8 * k) + 4 * E, "flops": T * E * 8}
    if case["op"] == "rows":
        n = case["rows"] * case["cols"]
        # bf16 in, codes and scales out; the codes and scales in, bf16 out
        return {"bytes": 4 * n + 2 * (n // 2 + n // 32), "flops": 4 * n}
    T, H, E, k, I = (case[n] for n in ("T", "H", "E", "k", "I"))
    active = sum(n > 0 for n in _counts(T, E, k, case["zipf"]))
    rows = T * k
    b = active * 3 * H * I * 17 // 32 + rows * (2 * H + 2 * H + 4) + 8 * E
    return {"bytes": b, "flops": 6 * H * I * rows}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(st["logits"].cpu().numpy(), st["bias"].cpu().numpy(), case)
    if case["op"] == "rows":
        y = torch.empty(st["x"].shape, dtype=torch.float64, device="cuda")
        for r in range(0, y.shape[0], 8192):
            y[r:r + 8192] = _exact_fp4(st["x"][r:r + 8192])
        return y
    return _exact_ffn(st, case)


def _exact_route(logits, bias, c):
    T, E, k = c["T"], c["E"], c["k"]
    l, b = logits.astype(np.float64), bias.astype(np.float64)
    live = (l > -FLT_MAX) & (b > -np.inf)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if c["score"] == "sigmoid":
            s = np.where(live, np.reciprocal(1.0 + np.exp(-l)), 0.0)
        else:
            z = np.where(live, l, -np.inf)
            z = np.exp(z - z.max(1, keepdims=True))
            s = np.where(live, z / z.sum(1, keepdims=True), 0.0)
    pick = np.where(live, s + b, -np.inf)
    if c["n_group"] > 1:
        grp = -np.sort(-pick.reshape(T, c["n_group"], -1), axis=2)
        score = grp[:, :, 0].copy()
        for j in range(1, c["topn"]):
            more = grp[:, :, j]
            score = np.where(more > -np.inf, score + np.where(more > -np.inf, more, 0.0), score)
        rank = np.argsort(np.argsort(-score, axis=1, kind="stable"), axis=1, kind="stable")
        pick = np.where(np.repeat(rank < c["topk_group"], E // c["n_group"], axis=1), pick,
                        -np.inf)
    ids = np.argsort(-pick, axis=1, kind="stable")[:, :k]
    ok = np.take_along_axis(pick, ids, 1) > -np.inf
    w = np.where(ok, np.take_along_axis(s, ids, 1), 0.0)
    if c["renorm"]:
        t = w.sum(1, keepdims=True)
        w = np.divide(w, t, out=np.zeros_like(w), where=t > 0)
    return (torch.from_numpy(np.where(ok, ids, -1).astype(np.int32)),
            torch.from_numpy(w * c["scale"]))


def _exact_fp4(x):
    """What MXFP4 makes of rows, in 64 bits: each block's grid of steps from
    its largest element, each element on the nearest step, ties to even."""
    b = x.double().reshape(x.shape[0], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(amax / 6.0))
    e = torch.where(amax > 6.0 * torch.exp2(e), e + 1, e)
    e = torch.where(amax <= 6.0 * torch.exp2(e - 1), e - 1, e)
    e = torch.where(amax == 0, torch.zeros_like(e), e).clamp(-127, 127)
    v = b / torch.exp2(e)
    step = 0.5 + 0.5 * (v.abs() >= 2) + 1.0 * (v.abs() >= 4)
    return (torch.round(v / step) * step * torch.exp2(e)).reshape(x.shape)


def _exact_weight(q, s):
    c = torch.stack((q % 16, torch.div(q, 16, rounding_mode="floor")), -1).flatten(-2).double()
    m = c % 8
    ex = torch.floor(m / 2)
    mag = torch.where(ex == 0, m * 0.5, (2.0 + m % 2) * torch.exp2(ex - 2.0))
    val = torch.where(c >= 8, -mag, mag)
    return val * torch.exp2(s.double() - 127.0).repeat_interleave(32, -1)


def _exact_ffn(st, c):
    I = c["I"]
    out = torch.zeros(st["y"].shape, dtype=torch.float64, device="cuda")
    fp4 = c["op"] == "w4a4"
    r0 = 0
    for e, n in enumerate(st["lens"]):
        if n == 0:
            continue
        w13 = _exact_weight(st["w13"][e], st["w13_s"][e])
        w2 = _exact_weight(st["w2"][e], st["w2_s"][e])
        for a in range(r0, r0 + n, 4096):
            z = min(a + 4096, r0 + n)
            x = st["x"][a:z]
            x = _exact_fp4(x) if fp4 else x.double()
            g = torch.matmul(x, w13[:I].t())
            u = torch.matmul(x, w13[I:].t())
            h = (g * torch.sigmoid(g) * u).bfloat16()
            h = _exact_fp4(h) if fp4 else h.double()
            out[a:z] = torch.matmul(h, w2.t()) * st["row_scale"][a:z, None].double()
        r0 += n
    return out
