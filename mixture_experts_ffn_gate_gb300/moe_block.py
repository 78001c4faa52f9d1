"""ctypes binding of the block's operators in libmoeffn.so (C ABI in
include/moe_block.h): norm, gate, the experts for a routing that is passed in,
their gradients, and the orthogonalised update.

As in ``moe_ffn``: argument marshalling only, C names, torch tensors for
device buffers, the stream defaults to torch's current stream, and no CPU
fallback.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple

import torch

from . import moe_ffn as _m
from .moe_ffn import MOE_ERR_UNSUPPORTED_SHAPE, MoeFfnError, _empty_on, mx_scale_bytes

MOE_BF16 = 0
MOE_F32 = 1
MOE_SCORE_SOFTMAX = 0
MOE_SCORE_SIGMOID = 1

_TYPES = {torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}
_SCORES = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}


class moe_gate_opts(ctypes.Structure):
    """Mirror of ``struct moe_gate_opts``."""
    _fields_ = [("score", ctypes.c_int32), ("groups", ctypes.c_int32), ("topk_groups", ctypes.c_int32),
                ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float), ("reserved", ctypes.c_int32 * 3)]


def declare(L):
    """The argument types of moe_block.h's functions (``moe_ffn.lib`` calls it once)."""
    vp, i64, i32, f32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    opts, gate = ctypes.POINTER(_m.moe_ffn_opts), ctypes.POINTER(moe_gate_opts)
    for name, args in (
            ("moe_rms_norm_forward", [vp, i32, vp, i32, vp, f32, i64, i64, vp, vp, vp, vp, vp]),
            ("moe_rms_norm_backward", [vp, i32, vp, vp, i32, vp, f32, i64, i64, vp, vp, vp, sz, vp]),
            ("moe_gate_forward", [vp, vp, i64, i64, i64, gate, vp, vp, vp, vp]),
            ("moe_gate_backward", [vp, vp, vp, i64, i64, i64, gate, vp, vp]),
            ("moe_ffn_forward_routed", [vp] * 8 + [i64] * 5 + [vp, vp, sz, opts, vp]),
            ("moe_ffn_backward_routed", [vp] * 6 + [i64] * 5 + [vp] * 5 + [sz, i32, opts, vp]),
            ("moe_ffn_forward_routed_train", [vp] * 5 + [i64] * 5 + [vp, vp, sz, opts, vp]),
            ("moe_orthogonalize", [vp, i32, i64, i64, i64, i32, f32, f32, f32, f32, f32, vp, vp, sz, vp])):
        f = getattr(L, name)
        f.argtypes, f.restype = args, i32
    for name, n in (("moe_rms_norm_backward_workspace_bytes", 2), ("moe_ffn_routed_workspace_bytes", 5),
                    ("moe_ffn_routed_backward_workspace_bytes", 5),
                    ("moe_orthogonalize_workspace_bytes", 3)):
        f = getattr(L, name)
        f.argtypes, f.restype = [i64] * n, sz


# A call of one token takes a few microseconds on the GPU, so the wrappers keep
# their own part short: one test per tensor, the raw stream, no lock.
def _lib():
    return _m._lib or _m.lib()


def _is(t, shape, dtype, name):
    """t is a contiguous CUDA tensor of this shape and type."""
    if t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous():
        return
    if t.dtype is not dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor")
    raise ValueError(f"{name} must be {list(shape)}, got {tuple(t.shape)}")


def _type(t, name):
    code = _TYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    return code


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream, device):
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else _m._stream(stream)


def _check(status, what):
    if status:
        raise MoeFfnError(status, what)


def _workspace(n, device, stream, what):
    if n == 0:
        raise MoeFfnError(MOE_ERR_UNSUPPORTED_SHAPE, what)
    return (torch.empty if stream is None else _empty_on(stream))((n,), dtype=torch.uint8, device=device)


def _size(t, name="workspace"):
    """The bytes of a workspace or state of the caller's."""
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    return t.numel() * t.element_size()


# ------------------------------------------------------------------ norm
class NormOutput(NamedTuple):
    y: torch.Tensor | None        # BF16 [T, H]
    h: torch.Tensor | None        # the new residual stream [T, H], its type; None without a residual
    codes: torch.Tensor | None    # MXFP8: E4M3 codes uint8 [T, H]
    scales: torch.Tensor | None   # and E8M0 scales uint8 [T, mx_scale_bytes(H)]


def moe_rms_norm_forward(x, weight, residual=None, eps: float = 1e-6, bf16: bool = True, mxfp8: bool = False, y=None,
                         h=None, codes=None, scales=None, stream=None) -> NormOutput:
    """h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight, per row:
    x bf16 or f32 [T,H], residual (nullable) bf16 or f32 [T,H], weight f32
    [H].  y in BF16 (``bf16``) and / or MXFP8 (``mxfp8``).  ``h`` may be
    ``residual`` itself."""
    T, H = x.shape
    _is(x, (T, H), x.dtype, "x")
    _is(weight, (H,), torch.float32, "weight")
    dev, empty = x.device, torch.empty if stream is None else _empty_on(stream)
    xt, rt = _type(x, "x"), 0
    if residual is not None:
        rt = _type(residual, "residual")
        _is(residual, (T, H), residual.dtype, "residual")
        if h is None:
            h = empty((T, H), dtype=residual.dtype, device=dev)
        else:
            _is(h, (T, H), residual.dtype, "h")
    elif h is not None:
        raise ValueError("h needs a residual")
    if y is not None:
        _is(y, (T, H), torch.bfloat16, "y")
    elif bf16:
        y = empty((T, H), dtype=torch.bfloat16, device=dev)
    if codes is not None or scales is not None or mxfp8:
        Sh = mx_scale_bytes(H)
        if codes is None:
            codes = empty((T, H), dtype=torch.uint8, device=dev)
        if scales is None:
            scales = empty((T, Sh), dtype=torch.uint8, device=dev)
        _is(codes, (T, H), torch.uint8, "codes")
        _is(scales, (T, Sh), torch.uint8, "scales")
    p = _ptr
    _check(_lib().moe_rms_norm_forward(p(x), xt, p(residual), rt, p(weight), eps, T, H, p(h), p(y), p(codes),
                                      p(scales), _stream(stream, dev)), "moe_rms_norm_forward")
    return NormOutput(y, h, codes, scales)


def moe_rms_norm_backward_workspace_bytes(T, H) -> int:
    return int(_m.lib().moe_rms_norm_backward_workspace_bytes(T, H))


def new_rms_norm_backward_workspace(T, H, device="cuda", stream=None):
    return _workspace(moe_rms_norm_backward_workspace_bytes(T, H), device, stream, "workspace size")


def moe_rms_norm_backward(h, weight, dy, dres=None, eps: float = 1e-6, dh=None, dweight=None, workspace=None,
                          stream=None):
    """(dh, dweight f32 [H]) of the norm of h bf16 or f32 [T,H] for dy bf16
    or f32 [T,H] = dL/dy; dres (nullable, h's type) is the gradient that
    reaches h besides, and ``dh`` (h's type) may be ``dres`` itself."""
    T, H = h.shape
    ht, gt = _type(h, "h"), _type(dy, "dy")
    _is(h, (T, H), h.dtype, "h")
    _is(dy, (T, H), dy.dtype, "dy")
    _is(weight, (H,), torch.float32, "weight")
    if dres is not None:
        _is(dres, (T, H), h.dtype, "dres")
    empty = torch.empty if stream is None else _empty_on(stream)
    if dh is None:
        dh = empty((T, H), dtype=h.dtype, device=h.device)
    else:
        _is(dh, (T, H), h.dtype, "dh")
    if dweight is None:
        dweight = empty((H,), dtype=torch.float32, device=h.device)
    else:
        _is(dweight, (H,), torch.float32, "dweight")
    if workspace is None:
        workspace = new_rms_norm_backward_workspace(T, H, device=h.device, stream=stream)
    p = _ptr
    _check(_lib().moe_rms_norm_backward(p(h), ht, p(weight), p(dy), gt, p(dres), eps, T, H, p(dh), p(dweight),
                                        p(workspace), _size(workspace), _stream(stream, h.device)),
           "moe_rms_norm_backward")
    return dh, dweight


# ------------------------------------------------------------------ gate
class GateOutput(NamedTuple):
    topk_idx: torch.Tensor          # int32 [T, k]
    topk_w: torch.Tensor            # f32 [T, k]
    counts: torch.Tensor | None     # int32 [E]


@functools.lru_cache(maxsize=64)
def _gate_opts(score, renormalize, scale, groups=1, topk_groups=1):
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, got {score!r}")
    if scale == 0.0:
        raise ValueError("scale must not be 0")  # 0 means 1 in the C struct
    return ctypes.byref(moe_gate_opts(_SCORES[score], groups, topk_groups, int(renormalize), scale))


def moe_gate_forward(logits, k: int, bias=None, score: str = "softmax", groups: int = 1, topk_groups: int = 1,
                     renormalize: bool = True, scale: float = 1.0, topk_idx=None, topk_w=None, counts=None,
                     stream=None) -> GateOutput:
    """The k experts of each token and their weights, from logits f32 [T,E]
    and the balance bias f32 [E] (nullable).  ``counts``: an int32 [E] tensor
    for the experts' loads, or True for a new one."""
    T, E = logits.shape
    _is(logits, (T, E), torch.float32, "logits")
    if bias is not None:
        _is(bias, (E,), torch.float32, "bias")
    dev, empty = logits.device, torch.empty if stream is None else _empty_on(stream)
    if topk_idx is None:
        topk_idx = empty((T, k), dtype=torch.int32, device=dev)
    else:
        _is(topk_idx, (T, k), torch.int32, "topk_idx")
    if topk_w is None:
        topk_w = empty((T, k), dtype=torch.float32, device=dev)
    else:
        _is(topk_w, (T, k), torch.float32, "topk_w")
    if counts is True:
        counts = empty((E,), dtype=torch.int32, device=dev)
    elif counts is not None:
        _is(counts, (E,), torch.int32, "counts")
    o = _gate_opts(score, renormalize, scale, groups, topk_groups)
    p = _ptr
    _check(_lib().moe_gate_forward(p(logits), p(bias), T, E, k, o, p(topk_idx), p(topk_w), p(counts),
                                   _stream(stream, dev)), "moe_gate_forward")
    return GateOutput(topk_idx, topk_w, counts)


def moe_gate_backward(logits, topk_idx, dtopk_w, score: str = "softmax", renormalize: bool = True, scale: float = 1.0,
                      dlogits=None, stream=None):
    """dlogits f32 [T,E] for dtopk_w f32 [T,k] = dL/dtopk_w of the choice
    topk_idx int32 [T,k] that moe_gate_forward made from ``logits`` with the
    same score, renormalize and scale."""
    T, E = logits.shape
    k = topk_idx.shape[1]
    _is(logits, (T, E), torch.float32, "logits")
    _is(topk_idx, (T, k), torch.int32, "topk_idx")
    _is(dtopk_w, (T, k), torch.float32, "dtopk_w")
    if dlogits is None:
        empty = torch.empty if stream is None else _empty_on(stream)
        dlogits = empty((T, E), dtype=torch.float32, device=logits.device)
    else:
        _is(dlogits, (T, E), torch.float32, "dlogits")
    o = _gate_opts(score, renormalize, scale)
    p = _ptr
    _check(_lib().moe_gate_backward(p(logits), p(topk_idx), p(dtopk_w), T, E, k, o, p(dlogits),
                                    _stream(stream, logits.device)), "moe_gate_backward")
    return dlogits


# ------------------------------------------------------------------ experts
def moe_ffn_routed_workspace_bytes(T, H, I, E, k) -> int:
    return int(_m.lib().moe_ffn_routed_workspace_bytes(T, H, I, E, k))


def moe_ffn_routed_backward_workspace_bytes(T, H, I, E, k) -> int:
    return int(_m.lib().moe_ffn_routed_backward_workspace_bytes(T, H, I, E, k))


# Their workspaces and the training pair's state: moe_ffn's, which are as
# large as these calls need.
new_routed_workspace = _m.new_workspace
new_routed_backward_workspace = _m.new_backward_workspace


def _routing(topk_idx, topk_w, T):
    k = topk_idx.shape[1]
    _is(topk_idx, (T, k), torch.int32, "topk_idx")
    _is(topk_w, (T, k), torch.float32, "topk_w")
    return k


def _experts(x, w_gate_up, w_down, dtype=torch.bfloat16):
    T, H = x.shape
    E, _, I = w_down.shape
    _is(w_gate_up, (E, 2 * I, H), dtype, "w_gate_up")
    _is(w_down, (E, H, I), dtype, "w_down")
    return T, H, I, E


def _new(t, shape, name, device, stream):
    if t is None:
        return (torch.empty if stream is None else _empty_on(stream))(shape, dtype=torch.float32, device=device)
    _is(t, shape, torch.float32, name)
    return t


def moe_ffn_forward_routed(x, topk_idx, topk_w, w_gate_up, w_down, x_scale=None, w_gate_up_scale=None,
                           w_down_scale=None, out=None, workspace=None, opts: _m.moe_ffn_opts | None = None,
                           stream=None):
    """out f32 [T,H] = sum_j topk_w[t,j] * expert topk_idx[t,j] of x[t].  x
    bf16 [T,H], or E4M3 codes uint8 with x_scale; weights bf16, or E4M3 codes
    uint8 with both scales (the layouts of moe_ffn_forward_mxfp8)."""
    T, H, I, E = _experts(x, w_gate_up, w_down, torch.bfloat16 if w_gate_up_scale is None else torch.uint8)
    k = _routing(topk_idx, topk_w, T)
    if x_scale is None:
        _is(x, (T, H), torch.bfloat16, "x")
    else:
        _is(x, (T, H), torch.uint8, "x")
        _is(x_scale, (T, mx_scale_bytes(H)), torch.uint8, "x_scale")
    if (w_gate_up_scale is None) != (w_down_scale is None):
        raise ValueError("w_gate_up_scale and w_down_scale go together")
    if w_down_scale is not None:
        _is(w_gate_up_scale, (E, 2 * I, mx_scale_bytes(H)), torch.uint8, "w_gate_up_scale")
        _is(w_down_scale, (E, H, mx_scale_bytes(I)), torch.uint8, "w_down_scale")
    out = _new(out, (T, H), "out", x.device, stream)
    if workspace is None:
        workspace = new_routed_workspace(T, H, I, E, k, device=x.device, stream=stream)
    p = _ptr
    _check(_lib().moe_ffn_forward_routed(
        p(x), p(x_scale), p(topk_idx), p(topk_w), p(w_gate_up), p(w_gate_up_scale), p(w_down), p(w_down_scale), T, H,
        I, E, k, p(out), p(workspace), _size(workspace), None if opts is None else ctypes.byref(opts),
        _stream(stream, x.device)), "moe_ffn_forward_routed")
    return out


def moe_ffn_forward_routed_train(x, topk_idx, topk_w, w_gate_up, w_down, state, out=None,
                                 opts: _m.moe_ffn_opts | None = None, stream=None):
    """The same for bf16 x and weights, keeping in ``state``
    (moe_ffn.new_train_state) what moe_ffn_backward_routed needs."""
    T, H, I, E = _experts(x, w_gate_up, w_down)
    k = _routing(topk_idx, topk_w, T)
    _is(x, (T, H), torch.bfloat16, "x")
    out = _new(out, (T, H), "out", x.device, stream)
    p = _ptr
    _check(_lib().moe_ffn_forward_routed_train(
        p(x), p(topk_idx), p(topk_w), p(w_gate_up), p(w_down), T, H, I, E, k, p(out), p(state), _size(state, "state"),
        None if opts is None else ctypes.byref(opts), _stream(stream, x.device)), "moe_ffn_forward_routed_train")
    return out


def moe_ffn_backward_routed(x, topk_idx, topk_w, w_gate_up, w_down, dout, dx=None, dtopk_w=None, dw_gate_up=None,
                            dw_down=None, workspace=None, state=None, opts: _m.moe_ffn_opts | None = None,
                            stream=None):
    """(dx f32 [T,H], dtopk_w f32 [T,k], dw_gate_up f32 [E,2I,H], dw_down f32
    [E,H,I]) for dout f32 [T,H].  ``state``: the state that
    moe_ffn_forward_routed_train left for the same arguments, instead of a
    workspace (moe_ffn.new_backward_workspace)."""
    T, H, I, E = _experts(x, w_gate_up, w_down)
    k = _routing(topk_idx, topk_w, T)
    _is(x, (T, H), torch.bfloat16, "x")
    _is(dout, (T, H), torch.float32, "dout")
    dev = x.device
    dx = _new(dx, (T, H), "dx", dev, stream)
    dtopk_w = _new(dtopk_w, (T, k), "dtopk_w", dev, stream)
    dw_gate_up = _new(dw_gate_up, (E, 2 * I, H), "dw_gate_up", dev, stream)
    dw_down = _new(dw_down, (E, H, I), "dw_down", dev, stream)
    if state is not None and workspace is not None:
        raise ValueError("pass a workspace or a state, not both")
    ws = state if state is not None else workspace
    if ws is None:
        ws = _m.new_backward_workspace(T, H, I, E, k, device=dev, stream=stream)
    p = _ptr
    _check(_lib().moe_ffn_backward_routed(
        p(x), p(topk_idx), p(topk_w), p(w_gate_up), p(w_down), p(dout), T, H, I, E, k, p(dx), p(dtopk_w),
        p(dw_gate_up), p(dw_down), p(ws), _size(ws, "workspace" if state is None else "state"), int(state is not None),
        None if opts is None else ctypes.byref(opts), _stream(stream, x.device)), "moe_ffn_backward_routed")
    return dx, dtopk_w, dw_gate_up, dw_down


# ------------------------------------------------------------------ orthogonalised updates
def moe_orthogonalize_workspace_bytes(B, M, N) -> int:
    return int(_m.lib().moe_orthogonalize_workspace_bytes(B, M, N))


def new_orthogonalize_workspace(B, M, N, device="cuda", stream=None):
    return _workspace(moe_orthogonalize_workspace_bytes(B, M, N), device, stream, "workspace size")


def moe_orthogonalize(g, steps: int = 5, coefficients=(3.4445, -4.7750, 2.0315), eps: float = 1e-7,
                      out_scale: float = 1.0, out=None, workspace=None, stream=None):
    """bf16 [B,M,N]: each matrix of g (bf16 or f32 [B,M,N]) divided by its
    Frobenius norm plus eps and put through ``steps`` of X = a X + (b A +
    c A A) X, A = X X^T; times out_scale.  Coefficients that could take a
    singular value beyond 1.9 before the last step are refused."""
    B, M, N = g.shape
    gt = _type(g, "g")
    _is(g, (B, M, N), g.dtype, "g")
    if out is None:
        empty = torch.empty if stream is None else _empty_on(stream)
        out = empty((B, M, N), dtype=torch.bfloat16, device=g.device)
    else:
        _is(out, (B, M, N), torch.bfloat16, "out")
    if workspace is None:
        workspace = new_orthogonalize_workspace(B, M, N, device=g.device, stream=stream) if B else g.new_empty(0)
    a, b, c = coefficients
    p = _ptr
    _check(_lib().moe_orthogonalize(p(g), gt, B, M, N, steps, a, b, c, eps, out_scale, p(out), p(workspace),
                                    _size(workspace), _stream(stream, g.device)), "moe_orthogonalize")
    return out
