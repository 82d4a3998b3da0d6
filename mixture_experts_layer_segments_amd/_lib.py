"""ctypes binding of libmoe.so (argument marshalling only)."""
from __future__ import annotations

import ctypes
import os

# torch first: its HIP runtime must be the one libmoe.so binds to.  Loading
# libmoe.so first would pull in a second copy of libamdhip64 (same soname,
# different file) that does not share torch's device state.
import torch  # noqa: F401

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = 0, -1, -2, -3, -4
MOE_DT_F32, MOE_DT_BF16 = 0, 1
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_SPLIT_PARITY, MOE_SPLIT_BOUNDED = 0, 1

EXPORTED_SYMBOLS = (
    "moe_status_string", "moe_num_segments", "moe_workspace_size", "moe_route_topk",
    "moe_permute", "moe_grouped_ffn", "moe_unpermute_combine", "moe_layer_forward",
    "moe_quantize_fp8", "moe_grouped_ffn_fp8w", "moe_layer_forward_fp8w",
    "moe_layer_plan_offsets", "moe_num_rows", "moe_quantize_act_fp8", "moe_grouped_ffn_w8a8",
    "moe_layer_forward_w8a8", "moe_layer_forward_static", "moe_route_biased",
    "moe_quantize_mxfp4", "moe_dequantize_mxfp4", "moe_grouped_ffn_mxfp4w",
    "moe_grouped_ffn_w4a4", "moe_layer_forward_mxfp4w", "moe_layer_forward_w4a4",
)
MOE_STATIC_WORKSPACE_BYTES = 64 * 1024 * 1024   # include/moe.h


class MoEConfig(ctypes.Structure):
    """Mirror of ``moe_config`` in include/moe.h."""
    _fields_ = [(n, ctypes.c_int32) for n in (
        "T", "H", "E", "k", "I", "score", "n_group", "topk_group", "group_score_topn",
        "renormalize", "n_hot_split", "split_ways", "shared_I", "act_dtype", "split_mode",
        "split_c_permille", "capacity_factor_permille")]


class MoEError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {moe_status_string(status)} ({status})")
        self.status = status


if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build the HIP library first "
        "(python -c 'import __graft_entry__ as g; g.build()')")

lib = ctypes.CDLL(LIB_PATH)

_p = ctypes.c_void_p
_cfgp = ctypes.POINTER(MoEConfig)
lib.moe_status_string.restype = ctypes.c_char_p
lib.moe_status_string.argtypes = [ctypes.c_int]
lib.moe_num_segments.restype = ctypes.c_int32
lib.moe_num_segments.argtypes = [_cfgp]
lib.moe_workspace_size.restype = ctypes.c_size_t
lib.moe_workspace_size.argtypes = [_cfgp]
lib.moe_num_rows.restype = ctypes.c_int32
lib.moe_num_rows.argtypes = [_cfgp]
lib.moe_layer_plan_offsets.restype = ctypes.c_int
lib.moe_layer_plan_offsets.argtypes = [_cfgp, ctypes.POINTER(ctypes.c_size_t)]
lib.moe_route_topk.restype = ctypes.c_int
lib.moe_route_topk.argtypes = [_cfgp, _p, _p, _p, _p]
lib.moe_permute.restype = ctypes.c_int
lib.moe_permute.argtypes = [_cfgp] + [_p] * 10 + [ctypes.c_size_t, _p]
lib.moe_grouped_ffn.restype = ctypes.c_int
lib.moe_grouped_ffn.argtypes = [_cfgp] + [_p] * 8 + [ctypes.c_size_t, _p]
lib.moe_unpermute_combine.restype = ctypes.c_int
lib.moe_unpermute_combine.argtypes = [_cfgp] + [_p] * 6
lib.moe_layer_forward.restype = ctypes.c_int
lib.moe_layer_forward.argtypes = [_cfgp] + [_p] * 12 + [ctypes.c_size_t, _p]
lib.moe_quantize_fp8.restype = ctypes.c_int
lib.moe_quantize_fp8.argtypes = [ctypes.c_int32] * 3 + [_p] * 4
lib.moe_grouped_ffn_fp8w.restype = ctypes.c_int
lib.moe_grouped_ffn_fp8w.argtypes = [_cfgp] + [_p] * 10 + [ctypes.c_size_t, _p]
lib.moe_layer_forward_fp8w.restype = ctypes.c_int
lib.moe_layer_forward_fp8w.argtypes = [_cfgp] + [_p] * 16 + [ctypes.c_size_t, _p]
lib.moe_quantize_act_fp8.restype = ctypes.c_int
lib.moe_quantize_act_fp8.argtypes = [ctypes.c_int32] * 2 + [_p] * 4
lib.moe_grouped_ffn_w8a8.restype = ctypes.c_int
lib.moe_grouped_ffn_w8a8.argtypes = [_cfgp] + [_p] * 11 + [ctypes.c_size_t, _p]
lib.moe_layer_forward_w8a8.restype = ctypes.c_int
lib.moe_layer_forward_w8a8.argtypes = [_cfgp] + [_p] * 16 + [ctypes.c_size_t, _p]
lib.moe_layer_forward_static.restype = ctypes.c_int
lib.moe_layer_forward_static.argtypes = [_cfgp] + [_p] * 12

lib.moe_route_biased.restype = ctypes.c_int
lib.moe_route_biased.argtypes = [_cfgp, _p, _p, ctypes.c_float, _p, _p, _p]
for _f in (lib.moe_quantize_mxfp4, lib.moe_dequantize_mxfp4):
    _f.restype = ctypes.c_int
    _f.argtypes = [ctypes.c_int32, ctypes.c_int64, ctypes.c_int32] + [_p] * 4
lib.moe_grouped_ffn_mxfp4w.restype = ctypes.c_int
lib.moe_grouped_ffn_mxfp4w.argtypes = [_cfgp] + [_p] * 10 + [ctypes.c_size_t, _p]
lib.moe_grouped_ffn_w4a4.restype = ctypes.c_int
lib.moe_grouped_ffn_w4a4.argtypes = [_cfgp] + [_p] * 11 + [ctypes.c_size_t, _p]
for _f in (lib.moe_layer_forward_mxfp4w, lib.moe_layer_forward_w4a4):
    _f.restype = ctypes.c_int
    _f.argtypes = [_cfgp, _p, _p, ctypes.c_float] + [_p] * 15 + [ctypes.c_size_t, _p]


def make_config(shape) -> MoEConfig:
    """MoEConfig from any object with the layer's fields (T, H, E, k, I,
    dtype 'f32'|'bf16', score 'softmax'|'sigmoid', n_group, topk_group,
    group_score_topn, renormalize, n_hot_split, split_ways, split_mode
    'parity'|'bounded', split_c_permille, shared_I, capacity_factor_permille)."""
    g = lambda n, d: getattr(shape, n, d)  # noqa: E731
    return MoEConfig(
        T=shape.T, H=shape.H, E=shape.E, k=shape.k, I=shape.I,
        score=MOE_SCORE_SIGMOID if g("score", "softmax") == "sigmoid" else MOE_SCORE_SOFTMAX,
        n_group=g("n_group", 1), topk_group=g("topk_group", 1),
        group_score_topn=g("group_score_topn", 2), renormalize=int(g("renormalize", 1)),
        n_hot_split=g("n_hot_split", 0), split_ways=g("split_ways", 1),
        shared_I=g("shared_I", 0),
        act_dtype=MOE_DT_F32 if g("dtype", "bf16") == "f32" else MOE_DT_BF16,
        split_mode=MOE_SPLIT_BOUNDED if g("split_mode", "parity") == "bounded" else MOE_SPLIT_PARITY,
        split_c_permille=g("split_c_permille", 0),
        capacity_factor_permille=g("capacity_factor_permille", 0))


def moe_status_string(status: int) -> str:
    return lib.moe_status_string(status).decode()


def _cfg(cfg) -> MoEConfig:
    return cfg if isinstance(cfg, MoEConfig) else make_config(cfg)


def moe_num_segments(cfg) -> int:
    return int(lib.moe_num_segments(ctypes.byref(_cfg(cfg))))


def moe_num_rows(cfg) -> int:
    return int(lib.moe_num_rows(ctypes.byref(_cfg(cfg))))


def moe_workspace_size(cfg) -> int:
    return int(lib.moe_workspace_size(ctypes.byref(_cfg(cfg))))


def moe_layer_plan_offsets(cfg) -> dict:
    """Byte offsets of seg_offsets, seg_expert, assign_to_row and
    row_to_token inside the layer call's workspace."""
    off = (ctypes.c_size_t * 4)()
    _check(lib.moe_layer_plan_offsets(ctypes.byref(_cfg(cfg)), off), "moe_layer_plan_offsets")
    return dict(zip(("seg_offsets", "seg_expert", "assign_to_row", "row_to_token"), off))


def _ptr(t):
    """Device address of a tensor (or an int address / None)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensors passed to libmoe must be contiguous")
    if t.device.type != "cuda":
        raise ValueError("tensors passed to libmoe must be on the GPU")
    return t.data_ptr()


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


# (a Stream object is 2.5 us of a small call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is None:
            return torch.cuda.current_stream().cuda_stream
        return _raw_stream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoEError(status, where)


def moe_route_topk(cfg, logits, topk_ids, topk_w, stream=None):
    _check(lib.moe_route_topk(ctypes.byref(_cfg(cfg)), _ptr(logits), _ptr(topk_ids),
                              _ptr(topk_w), _stream(stream)), "moe_route_topk")


def moe_permute(cfg, x, topk_ids, x_perm, seg_offsets, seg_expert, assign_to_row,
                row_to_token, counts, balancedness, workspace, stream=None):
    _check(lib.moe_permute(ctypes.byref(_cfg(cfg)), _ptr(x), _ptr(topk_ids), _ptr(x_perm),
                           _ptr(seg_offsets), _ptr(seg_expert), _ptr(assign_to_row),
                           _ptr(row_to_token), _ptr(counts), _ptr(balancedness),
                           _ptr(workspace), _nbytes(workspace), _stream(stream)), "moe_permute")


def moe_grouped_ffn(cfg, x_perm, seg_offsets, seg_expert, w13, w2, row_scale, y_perm,
                    workspace, stream=None):
    _check(lib.moe_grouped_ffn(ctypes.byref(_cfg(cfg)), _ptr(x_perm), _ptr(seg_offsets),
                               _ptr(seg_expert), _ptr(w13), _ptr(w2), _ptr(row_scale),
                               _ptr(y_perm), _ptr(workspace), _nbytes(workspace),
                               _stream(stream)), "moe_grouped_ffn")


def moe_unpermute_combine(cfg, y_perm, assign_to_row, topk_w, shared_y, out, stream=None):
    _check(lib.moe_unpermute_combine(ctypes.byref(_cfg(cfg)), _ptr(y_perm), _ptr(assign_to_row),
                                     _ptr(topk_w), _ptr(shared_y), _ptr(out), _stream(stream)),
           "moe_unpermute_combine")


def moe_layer_forward(cfg, logits, x, w13, w2, shared_w13, shared_w2, out, topk_ids, topk_w,
                      counts, balancedness, workspace, stream=None):
    _check(lib.moe_layer_forward(ctypes.byref(_cfg(cfg)), _ptr(logits), _ptr(x), _ptr(w13),
                                 _ptr(w2), _ptr(shared_w13), _ptr(shared_w2), _ptr(out),
                                 _ptr(topk_ids), _ptr(topk_w), _ptr(counts), _ptr(balancedness),
                                 _ptr(workspace), _nbytes(workspace), _stream(stream)),
           "moe_layer_forward")


def moe_layer_forward_static(cfg, logits, x, w13, w2, shared_w13, shared_w2, out, topk_ids,
                             topk_w, counts, balancedness, stream=None):
    """moe_layer_forward on the library's own per-GPU workspace (allocates
    nothing; overlapping calls on one GPU race)."""
    _check(lib.moe_layer_forward_static(ctypes.byref(_cfg(cfg)), _ptr(logits), _ptr(x), _ptr(w13),
                                        _ptr(w2), _ptr(shared_w13), _ptr(shared_w2), _ptr(out),
                                        _ptr(topk_ids), _ptr(topk_w), _ptr(counts),
                                        _ptr(balancedness), _stream(stream)),
           "moe_layer_forward_static")


def moe_quantize_fp8(src, q, scale, stream=None):
    """src [n, rows, cols] (or [rows, cols]) bf16 -> q uint8 same shape, scale
    fp32 [n, rows/128, cols/128]."""
    shape = tuple(src.shape)
    n, rows, cols = (1,) + shape if len(shape) == 2 else shape
    _check(lib.moe_quantize_fp8(n, rows, cols, _ptr(src), _ptr(q), _ptr(scale), _stream(stream)),
           "moe_quantize_fp8")


def moe_grouped_ffn_fp8w(cfg, x_perm, seg_offsets, seg_expert, w13_q, w13_scale, w2_q, w2_scale,
                         row_scale, y_perm, workspace, stream=None):
    _check(lib.moe_grouped_ffn_fp8w(ctypes.byref(_cfg(cfg)), _ptr(x_perm), _ptr(seg_offsets),
                                    _ptr(seg_expert), _ptr(w13_q), _ptr(w13_scale), _ptr(w2_q),
                                    _ptr(w2_scale), _ptr(row_scale), _ptr(y_perm),
                                    _ptr(workspace), _nbytes(workspace), _stream(stream)),
           "moe_grouped_ffn_fp8w")


def moe_layer_forward_fp8w(cfg, logits, x, w13_q, w13_scale, w2_q, w2_scale, shared_w13_q,
                           shared_w13_scale, shared_w2_q, shared_w2_scale, out, topk_ids, topk_w,
                           counts, balancedness, workspace, stream=None):
    _check(lib.moe_layer_forward_fp8w(
        ctypes.byref(_cfg(cfg)), _ptr(logits), _ptr(x), _ptr(w13_q), _ptr(w13_scale), _ptr(w2_q),
        _ptr(w2_scale), _ptr(shared_w13_q), _ptr(shared_w13_scale), _ptr(shared_w2_q),
        _ptr(shared_w2_scale), _ptr(out), _ptr(topk_ids), _ptr(topk_w), _ptr(counts),
        _ptr(balancedness), _ptr(workspace), _nbytes(workspace), _stream(stream)),
        "moe_layer_forward_fp8w")


def moe_quantize_act_fp8(src, q, scale, stream=None):
    """src [rows, cols] bf16 -> q uint8 [rows, cols], scale fp32 [rows, cols/128]."""
    rows, cols = tuple(src.shape)
    _check(lib.moe_quantize_act_fp8(rows, cols, _ptr(src), _ptr(q), _ptr(scale), _stream(stream)),
           "moe_quantize_act_fp8")


def moe_grouped_ffn_w8a8(cfg, x_perm_q, x_perm_scale, seg_offsets, seg_expert, w13_q, w13_scale,
                         w2_q, w2_scale, row_scale, y_perm, workspace, stream=None):
    _check(lib.moe_grouped_ffn_w8a8(ctypes.byref(_cfg(cfg)), _ptr(x_perm_q), _ptr(x_perm_scale),
                                    _ptr(seg_offsets), _ptr(seg_expert), _ptr(w13_q),
                                    _ptr(w13_scale), _ptr(w2_q), _ptr(w2_scale), _ptr(row_scale),
                                    _ptr(y_perm), _ptr(workspace), _nbytes(workspace),
                                    _stream(stream)),
           "moe_grouped_ffn_w8a8")


def moe_layer_forward_w8a8(cfg, logits, x, w13_q, w13_scale, w2_q, w2_scale, shared_w13_q,
                           shared_w13_scale, shared_w2_q, shared_w2_scale, out, topk_ids, topk_w,
                           counts, balancedness, workspace, stream=None):
    _check(lib.moe_layer_forward_w8a8(
        ctypes.byref(_cfg(cfg)), _ptr(logits), _ptr(x), _ptr(w13_q), _ptr(w13_scale), _ptr(w2_q),
        _ptr(w2_scale), _ptr(shared_w13_q), _ptr(shared_w13_scale), _ptr(shared_w2_q),
        _ptr(shared_w2_scale), _ptr(out), _ptr(topk_ids), _ptr(topk_w), _ptr(counts),
        _ptr(balancedness), _ptr(workspace), _nbytes(workspace), _stream(stream)),
        "moe_layer_forward_w8a8")


def _args(*specs):
    """Addresses of (name, tensor, dtype, numel): each of that type, at least
    that many elements, contiguous and on the current device (addresses and
    None pass as they are)."""
    addresses, placed, last = [], (), None
    for name, t, dtype, numel in specs:
        if t is None or type(t) is int:
            addresses.append(t)
            continue
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
        if t.numel() < numel:
            raise ValueError(f"{name} must hold {numel} elements, not {t.numel()}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        device = t.get_device()   # -1: not a GPU's
        if device != last:        # (one check for a run of one device's)
            last = device
            placed += ((name, device),)
        addresses.append(t.data_ptr())
    for name, device in placed:
        if device < 0:
            raise ValueError(f"{name} must be on the GPU")
        if device != torch.cuda.current_device():
            raise ValueError(f"{name} is on cuda:{device}, the current device is "
                             f"cuda:{torch.cuda.current_device()}")
    return addresses


def _workspace(t):
    """Address and bytes of a workspace of any type."""
    return (*_args(("workspace", t, t.dtype, 0)), _nbytes(t))


def moe_route_biased(cfg, logits, bias, routed_scale, topk_ids, topk_w, stream=None):
    """Top-k routing on scores + bias (bias fp32 [E] or None), the weights
    from the scores, times routed_scale; empty slots get id -1, weight 0."""
    c = _cfg(cfg)
    logits, bias, topk_ids, topk_w = _args(
        ("logits", logits, torch.float32, c.T * c.E), ("bias", bias, torch.float32, c.E),
        ("topk_ids", topk_ids, torch.int32, c.T * c.k),
        ("topk_w", topk_w, torch.float32, c.T * c.k))
    _check(lib.moe_route_biased(ctypes.byref(c), logits, bias, routed_scale, topk_ids, topk_w,
                                _stream(stream)), "moe_route_biased")


def _mx_rows(wide, q, scale):
    """dtype, rows and cols of a conversion between wide [.., cols] and MXFP4,
    and the addresses of the three."""
    if wide.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"MXFP4 rows convert from and to float32 and bfloat16, not {wide.dtype}")
    cols, n = wide.shape[-1], wide.numel()
    dtype = MOE_DT_F32 if wide.dtype == torch.float32 else MOE_DT_BF16
    return (dtype, n // cols if cols else 0, cols), _args(
        ("rows", wide, wide.dtype, 0), ("q", q, torch.uint8, n // 2),
        ("scale", scale, torch.uint8, n // 32))


def moe_quantize_mxfp4(src, q, scale, stream=None):
    """src [.., cols] bf16 or fp32 -> q uint8 [.., cols/2] (two E2M1 codes a
    byte), scale uint8 [.., cols/32] (E8M0)."""
    shape, (src, q, scale) = _mx_rows(src, q, scale)
    _check(lib.moe_quantize_mxfp4(*shape, src, q, scale, _stream(stream)), "moe_quantize_mxfp4")


def moe_dequantize_mxfp4(q, scale, dst, stream=None):
    """The values of MXFP4 rows, to dst [.., cols] bf16 or fp32."""
    shape, (dst, q, scale) = _mx_rows(dst, q, scale)
    _check(lib.moe_dequantize_mxfp4(*shape, q, scale, dst, _stream(stream)),
           "moe_dequantize_mxfp4")


def _mx_weights(c, I, n, w13_q, w13_scale, w2_q, w2_scale, name=""):
    """The specs of n experts of intermediate size I in MXFP4."""
    return ((name + "w13_q", w13_q, torch.uint8, n * I * c.H),
            (name + "w13_scale", w13_scale, torch.uint8, n * I * c.H // 16),
            (name + "w2_q", w2_q, torch.uint8, n * I * c.H // 2),
            (name + "w2_scale", w2_scale, torch.uint8, n * I * c.H // 32))


def _mx_ffn(c, x, seg_offsets, seg_expert, weights, row_scale, y_perm):
    """The addresses of a grouped FFN's tensors (x: the specs of its rows)."""
    S, R = moe_num_segments(c), moe_num_rows(c)
    return _args(*x(R), ("seg_offsets", seg_offsets, torch.int32, S + 1),
                 ("seg_expert", seg_expert, torch.int32, S),
                 *_mx_weights(c, c.I, c.E, *weights),
                 ("row_scale", row_scale, torch.float32, R),
                 ("y_perm", y_perm, torch.bfloat16, R * c.H))


def moe_grouped_ffn_mxfp4w(cfg, x_perm, seg_offsets, seg_expert, w13_q, w13_scale, w2_q, w2_scale,
                           row_scale, y_perm, workspace, stream=None):
    """moe_grouped_ffn on MXFP4 weights: w13_q uint8 [E, 2I, H/2] + w13_scale
    uint8 [E, 2I, H/32], w2_q [E, H, I/2] + w2_scale [E, H, I/32]."""
    c = _cfg(cfg)
    a = _mx_ffn(c, lambda R: (("x_perm", x_perm, torch.bfloat16, R * c.H),), seg_offsets,
                seg_expert, (w13_q, w13_scale, w2_q, w2_scale), row_scale, y_perm)
    _check(lib.moe_grouped_ffn_mxfp4w(ctypes.byref(c), *a, *_workspace(workspace),
                                      _stream(stream)), "moe_grouped_ffn_mxfp4w")


def moe_grouped_ffn_w4a4(cfg, x_perm_q, x_perm_scale, seg_offsets, seg_expert, w13_q, w13_scale,
                         w2_q, w2_scale, row_scale, y_perm, workspace, stream=None):
    """moe_grouped_ffn_mxfp4w on MXFP4 rows: x_perm_q uint8 [R, H/2] +
    x_perm_scale uint8 [R, H/32]."""
    c = _cfg(cfg)
    a = _mx_ffn(c, lambda R: (("x_perm_q", x_perm_q, torch.uint8, R * c.H // 2),
                              ("x_perm_scale", x_perm_scale, torch.uint8, R * c.H // 32)),
                seg_offsets, seg_expert, (w13_q, w13_scale, w2_q, w2_scale), row_scale, y_perm)
    _check(lib.moe_grouped_ffn_w4a4(ctypes.byref(c), *a, *_workspace(workspace),
                                    _stream(stream)), "moe_grouped_ffn_w4a4")


def _mx_layer(fn, where, cfg, logits, route_bias, routed_scale, x, w, sw, out, topk_ids, topk_w,
              counts, balancedness, workspace, stream):
    c = _cfg(cfg)
    logits, route_bias, *rest = _args(
        ("logits", logits, torch.float32, c.T * c.E),
        ("route_bias", route_bias, torch.float32, c.E),
        ("x", x, torch.bfloat16, c.T * c.H), *_mx_weights(c, c.I, c.E, *w),
        *_mx_weights(c, c.shared_I, 1, *sw, name="shared_"),
        ("out", out, torch.bfloat16, c.T * c.H),
        ("topk_ids", topk_ids, torch.int32, c.T * c.k),
        ("topk_w", topk_w, torch.float32, c.T * c.k), ("counts", counts, torch.int32, c.E),
        ("balancedness", balancedness, torch.float32, 1))
    _check(fn(ctypes.byref(c), logits, route_bias, routed_scale, *rest, *_workspace(workspace),
              _stream(stream)), where)


def moe_layer_forward_mxfp4w(cfg, logits, route_bias, routed_scale, x, w13_q, w13_scale, w2_q,
                             w2_scale, shared_w13_q, shared_w13_scale, shared_w2_q,
                             shared_w2_scale, out, topk_ids, topk_w, counts, balancedness,
                             workspace, stream=None):
    """The layer on MXFP4 weights, routed by moe_route_biased."""
    _mx_layer(lib.moe_layer_forward_mxfp4w, "moe_layer_forward_mxfp4w", cfg, logits, route_bias,
              routed_scale, x, (w13_q, w13_scale, w2_q, w2_scale),
              (shared_w13_q, shared_w13_scale, shared_w2_q, shared_w2_scale), out, topk_ids,
              topk_w, counts, balancedness, workspace, stream)


def moe_layer_forward_w4a4(cfg, logits, route_bias, routed_scale, x, w13_q, w13_scale, w2_q,
                           w2_scale, shared_w13_q, shared_w13_scale, shared_w2_q,
                           shared_w2_scale, out, topk_ids, topk_w, counts, balancedness,
                           workspace, stream=None):
    """The layer on MXFP4 weights and activations, routed by moe_route_biased."""
    _mx_layer(lib.moe_layer_forward_w4a4, "moe_layer_forward_w4a4", cfg, logits, route_bias,
              routed_scale, x, (w13_q, w13_scale, w2_q, w2_scale),
              (shared_w13_q, shared_w13_scale, shared_w2_q, shared_w2_scale), out, topk_ids,
              topk_w, counts, balancedness, workspace, stream)
