"""Tensor-level calls of a decode step around the balanced exchange: the
router's expert choice, the experts' products with 4-bit weights, and the
whole expert layer for a few tokens.

As in ``api``: dtypes, devices and sizes are checked here, outputs are
allocated when none are given, and the C entry point enqueues on the current
stream of the tensors' device (or on ``stream``). What is allocated here is
taken from that stream's pool, so it may be used there at once.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _binding as B
from .api import _BF16_LIKE, _need, _opt

_LOGIT_CODES = {torch.float32: B.MEP_SCALE_F32, torch.bfloat16: B.MEP_SCALE_BF16,
                torch.float16: B.MEP_SCALE_F16}
_SCORING = {"softmax": B.MEP_SCORE_SOFTMAX, "sigmoid": B.MEP_SCORE_SIGMOID}
_KINDS = {"int4": B.MEP_WEIGHT_INT4, "fp4": B.MEP_WEIGHT_FP4}
_MASKS = (torch.uint8, torch.bool)


def _device(t, name, *others):
    """Device of t, which every other tensor given must share."""
    if t is None:
        raise ValueError(f"{name} is required")
    d = t.device
    for o in others:
        if o is not None and o.device != d:
            raise ValueError(f"tensors are on different devices: {name} on {d}, one on {o.device}")
    return d


def _shape(t, name, *dims):
    if tuple(t.shape) != dims:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {dims}")


_NO_CONTEXT = contextlib.nullcontext()


def _alloc(stream):
    """Allocations inside belong to the stream that the call runs on."""
    return _NO_CONTEXT if stream is None else torch.cuda.stream(stream)


# Handle of a device's current stream. torch.cuda.current_stream() makes a
# Stream object first, 3-4 us of a call that takes 6 on the GPU.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _run(name, device, stream, fn, *args):
    if device.type != "cuda":
        raise ValueError(f"{name}: tensors must be on a GPU, not on {device}")
    if stream is not None and stream.device != device:
        raise ValueError(f"{name}: the stream is on {stream.device}, the tensors on {device}")
    handle = _raw_stream(device.index) if stream is None else stream.cuda_stream
    if device.index == torch.cuda.current_device():
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, handle)
    B.check(name, rc)


def route(logits, K, bias=None, scoring="softmax", n_group=1, topk_group=1, renormalize=True,
          scale=1.0, topk_ids=None, scores=None, stream=None):
    """mep_route. logits [T,E] float32 / bfloat16 / float16, bias [E] float32.
    Returns (topk_ids [T,K] int32, scores [T,K] float32)."""
    dev = _device(logits, "logits", bias, topk_ids, scores)
    T, E = logits.shape
    if logits.dtype not in _LOGIT_CODES:
        raise ValueError(f"logits has dtype {logits.dtype}")
    if scoring not in _SCORING:
        raise ValueError(f"scoring is {scoring!r}, expected one of {sorted(_SCORING)}")
    lp = _need(logits, "logits", logits.dtype)
    if topk_ids is None or scores is None:
        with _alloc(stream):
            if topk_ids is None:
                topk_ids = torch.empty(T, K, dtype=torch.int32, device=dev)
            if scores is None:
                scores = torch.empty(T, K, dtype=torch.float32, device=dev)
    _run("mep_route", dev, stream, B.mep_route, T, E, K, lp, _LOGIT_CODES[logits.dtype],
         _opt(bias, "bias", torch.float32, E), _SCORING[scoring], n_group, topk_group,
         int(bool(renormalize)), float(scale), _need(topk_ids, "topk_ids", torch.int32, T * K),
         _need(scores, "scores", torch.float32, T * K))
    return topk_ids, scores


def route_grad(logits, topk_ids, dscores, scoring="softmax", renormalize=True, scale=1.0,
               dlogits=None, stream=None):
    """mep_route_grad: the gradient of route's scores with respect to the
    logits. Returns dlogits [T,E] of the logits' dtype."""
    dev = _device(logits, "logits", topk_ids, dscores, dlogits)
    T, E = logits.shape
    _, K = topk_ids.shape
    if logits.dtype not in _LOGIT_CODES:
        raise ValueError(f"logits has dtype {logits.dtype}")
    if scoring not in _SCORING:
        raise ValueError(f"scoring is {scoring!r}, expected one of {sorted(_SCORING)}")
    lp = _need(logits, "logits", logits.dtype)
    if dlogits is None:
        with _alloc(stream):
            dlogits = torch.empty_like(logits)
    _run("mep_route_grad", dev, stream, B.mep_route_grad, T, E, K, lp,
         _LOGIT_CODES[logits.dtype], _need(topk_ids, "topk_ids", torch.int32, T * K),
         _need(dscores, "dscores", torch.float32, T * K), _SCORING[scoring],
         int(bool(renormalize)), float(scale),
         _need(dlogits, "dlogits", logits.dtype, T * E))
    return dlogits


class Q4Weights:
    """E matrices [N,K] in the packed 4-bit layout (q4_pack makes them)."""

    def __init__(self, E, N, K, kind, group, codes, scales, zeros):
        self.E, self.N, self.K, self.kind, self.group = E, N, K, kind, group
        self.codes, self.scales, self.zeros = codes, scales, zeros
        self.device = codes.device
        self._view = B.Weights(_KINDS[kind], E, N, K, group, _LOGIT_CODES[scales.dtype],
                               codes.data_ptr(), scales.data_ptr(),
                               None if zeros is None else zeros.data_ptr())


def q4_pack(codes, scales, zeros=None, group=128, kind="int4", stream=None):
    """mep_pack_weights: codes [E,N,K] (or [N,K]) uint8, scales [E,N,G]
    bfloat16 / float16 and zeros [E,N,G] uint8 (int4 only, optional) into a
    Q4Weights. Done once, when the weights are loaded."""
    dev = _device(codes, "codes", scales, zeros)
    if kind not in _KINDS:
        raise ValueError(f"kind is {kind!r}, expected one of {sorted(_KINDS)}")
    if codes.dim() not in (2, 3):
        raise ValueError("codes must be [E, N, K] or [N, K]")
    E, N, K = codes.shape if codes.dim() == 3 else (1, *codes.shape)
    nc, ns = B.mep_packed_code_bytes(E, N, K), B.mep_packed_scale_count(E, N, K, group)
    if nc == 0 or ns == 0:
        raise ValueError(f"unsupported weights E={E} N={N} K={K} group={group}")
    G = -(-K // group)
    cp = _need(codes, "codes", torch.uint8, E * N * K)
    sp = _need(scales, "scales", (torch.bfloat16, torch.float16), E * N * G)
    zp = _opt(zeros, "zeros", torch.uint8, E * N * G)
    with _alloc(stream):
        pc = torch.empty(nc, dtype=torch.uint8, device=dev)
        ps = torch.empty(ns, dtype=scales.dtype, device=dev)
        pz = None if zeros is None else torch.empty(ns, dtype=torch.uint8, device=dev)
    _run("mep_pack_weights", dev, stream, B.mep_pack_weights, E, N, K, _KINDS[kind], group, cp,
         sp, zp, pc.data_ptr(), ps.data_ptr(), None if pz is None else pz.data_ptr())
    return Q4Weights(E, N, K, kind, group, pc, ps, pz)


def q4_quantize(w, group=128, kind="int4", scale_dtype=torch.bfloat16, stream=None):
    """mep_quant_weights: bf16 w [E,N,K] (or [N,K]) to (codes uint8 of its
    shape, scales [..., N, G]), as q4_pack takes them."""
    dev = _device(w, "w")
    if kind not in _KINDS:
        raise ValueError(f"kind is {kind!r}, expected one of {sorted(_KINDS)}")
    if scale_dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"scale_dtype is {scale_dtype}")
    if w.dim() not in (2, 3):
        raise ValueError("w must be [E, N, K] or [N, K]")
    E, N, K = w.shape if w.dim() == 3 else (1, *w.shape)
    if group not in (32, 64, 128):
        raise ValueError(f"group is {group}, expected 32, 64 or 128")
    wp = _need(w, "w", _BF16_LIKE)
    with _alloc(stream):
        codes = torch.empty(w.shape, dtype=torch.uint8, device=dev)
        scales = torch.empty(*w.shape[:-1], -(-K // group), dtype=scale_dtype, device=dev)
    _run("mep_quant_weights", dev, stream, B.mep_quant_weights, E, N, K, _KINDS[kind], group,
         _LOGIT_CODES[scale_dtype], wp, codes.data_ptr(), scales.data_ptr())
    return codes, scales


def expert_matvec_q4(x, w, ids=None, first=0, mask=None, out=None, out_dtype=torch.bfloat16,
                     stream=None):
    """mep_expert_matvec: out[t,r] = W[ids[t,r] - first] x[t] (x [T,K]) or
    x[t,r] (x [T,R,K]); without ids, out[t] = W x[t] (one matrix). `out`
    bfloat16 or float32; rows of skipped routes are left untouched (zero in
    an output allocated here). Returns out [T,R,N], or [T,N]."""
    if not isinstance(w, Q4Weights):
        raise ValueError("w must be a Q4Weights")
    dev = _device(x, "x", w, ids, mask, out)
    if ids is None:
        if x.dim() != 2:
            raise ValueError("x must be [T, K] without ids")
        T, R = x.shape[0], 0
        shape = (T, w.N)
    else:
        T, R = ids.shape
        if x.dim() == 3 and tuple(x.shape[:2]) != (T, R) or x.dim() == 2 and x.shape[0] != T:
            raise ValueError(f"x has shape {tuple(x.shape)}, ids {tuple(ids.shape)}")
        shape = (T, R, w.N)
    if x.dim() not in (2, 3) or x.shape[-1] != w.K:
        raise ValueError(f"x has shape {tuple(x.shape)}, the weights take {w.K} inputs")
    xp = _need(x, "x", _BF16_LIKE)
    if out is None:
        make = torch.empty if ids is None else torch.zeros
        with _alloc(stream):
            out = make(shape, dtype=out_dtype, device=dev)
    _shape(out, "out", *shape)
    op = _need(out, "out", _BF16_LIKE + (torch.float32,))
    f32 = out.dtype == torch.float32
    _run("mep_expert_matvec", dev, stream, B.mep_expert_matvec, T, R, first, xp,
         int(x.dim() == 3), _opt(ids, "ids", torch.int32),
         _opt(mask, "mask", _MASKS, T * R), ctypes.byref(w._view), None if f32 else op,
         op if f32 else None)
    return out


def moe_layer_workspace(T, K, I, device=None):
    """Workspace of moe_layer for these sizes (device uint8 tensor)."""
    n = B.mep_moe_layer_workspace_size(T, K, I)
    if n == 0:
        raise ValueError(f"unsupported layer sizes T={T} K={K} I={I}")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def _layer_weights(w, name):
    """(view, E, N, K) of a Q4Weights or a bf16 tensor [E,N,K]."""
    if isinstance(w, Q4Weights):
        return w._view, w.E, w.N, w.K
    if w is None or w.dim() != 3:
        raise ValueError(f"{name} must be a Q4Weights or a bf16 tensor [E, N, K]")
    E, N, K = w.shape
    p = _need(w, name, _BF16_LIKE)
    return B.Weights(B.MEP_WEIGHT_BF16, E, N, K, 0, 0, p, None, None), E, N, K


def moe_layer(x, ids, scores, w13, w2, first=0, mask=None, workspace=None, out_bf16=True,
              out_f32=False, stream=None):
    """mep_moe_layer. x [T,H] bf16, ids [T,K] int32, scores [T,K] float32,
    mask [T,K] (0: the route is skipped); w13 [E,2I,H] (gate rows, then up
    rows) and w2 [E,H,I], both bf16 tensors or both Q4Weights. Ids outside
    [first, first + E) are skipped. out_bf16 / out_f32: True to allocate, a
    tensor to write into, or False/None. Returns (out_bf16, out_f32)."""
    outs = [o for o in (out_bf16, out_f32) if isinstance(o, torch.Tensor)]
    dev = _device(x, "x", ids, scores, mask, w13, w2, workspace, *outs)
    T, H = x.shape
    _, K = ids.shape
    v13, _, N13, K13 = _layer_weights(w13, "w13")
    v2, _, _, I = _layer_weights(w2, "w2")
    if K13 != H or N13 != 2 * I:
        raise ValueError(f"w13 is [E, {N13}, {K13}], expected [E, {2 * I}, {H}]")
    xp = _need(x, "x", _BF16_LIKE)
    if workspace is None or out_bf16 is True or out_f32 is True:
        with _alloc(stream):
            if workspace is None:
                workspace = moe_layer_workspace(T, K, I, dev)
            if out_bf16 is True:
                out_bf16 = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
            if out_f32 is True:
                out_f32 = torch.empty(T, H, dtype=torch.float32, device=dev)
    out_bf16 = None if out_bf16 is False else out_bf16
    out_f32 = None if out_f32 is False else out_f32
    _run("mep_moe_layer", dev, stream, B.mep_moe_layer, T, K, H, I, first, xp,
         _need(ids, "ids", torch.int32, T * K), _need(scores, "scores", torch.float32, T * K),
         _opt(mask, "mask", _MASKS, T * K), ctypes.byref(v13), ctypes.byref(v2),
         _need(workspace, "workspace", torch.uint8), workspace.numel(),
         _opt(out_bf16, "out_bf16", _BF16_LIKE, T * H),
         _opt(out_f32, "out_f32", torch.float32, T * H))
    return out_bf16, out_f32
