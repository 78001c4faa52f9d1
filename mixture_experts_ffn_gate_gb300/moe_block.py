"""ctypes binding of the block's operators in libmoeffn.so (C ABI in
include/moe_block.h): norm, gate, the experts for a routing that is passed in,
their gradients, the load-balance loss, the gradients' norm, and the
orthogonalised and AdamW updates.

As in ``moe_ffn``: argument marshalling only, C names, torch tensors for
device buffers, the stream defaults to torch's current stream, and no CPU
fallback.
"""
from __future__ import annotations

import array
import bisect
import ctypes
import functools
import math
import operator
from typing import NamedTuple

import torch

from . import _build
from . import moe_ffn as _m
from .moe_ffn import MOE_ERR_UNSUPPORTED_SHAPE, MoeFfnError, _empty_on, mx_scale_bytes

MOE_BF16 = 0
MOE_F32 = 1
MOE_SCORE_SOFTMAX = 0
MOE_SCORE_SIGMOID = 1

_TYPES = {torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}
_ROUNDINGS = {"auto": 0, "nearest": 1, "random": 2}   # MOE_ADAMW_ROUND_*
_SCORES = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}


class moe_gate_opts(ctypes.Structure):
    """Mirror of ``struct moe_gate_opts``."""
    _fields_ = [("score", ctypes.c_int32), ("groups", ctypes.c_int32), ("topk_groups", ctypes.c_int32),
                ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float), ("reserved", ctypes.c_int32 * 3)]


class moe_balance_opts(ctypes.Structure):
    """Mirror of ``struct moe_balance_opts``."""
    _fields_ = [("score", ctypes.c_int32), ("coef", ctypes.c_float), ("z_coef", ctypes.c_float),
                ("reserved", ctypes.c_int32 * 5)]


class moe_tensor(ctypes.Structure):
    """Mirror of ``struct moe_tensor``."""
    _fields_ = [("data", ctypes.c_void_p), ("n", ctypes.c_int64), ("type", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class moe_adamw_tensor(ctypes.Structure):
    """Mirror of ``struct moe_adamw_tensor``."""
    _fields_ = ([(f, ctypes.c_void_p) for f in ("w", "master", "grad", "m", "v", "m_scale", "v_scale")]
                + [("n", ctypes.c_int64)] + [(f, ctypes.c_int32) for f in ("w_type", "grad_type", "state_bits")]
                + [("lr_factor", ctypes.c_float), ("weight_decay", ctypes.c_float), ("reserved", ctypes.c_int32)])


class moe_adamw_opts(ctypes.Structure):
    """Mirror of ``struct moe_adamw_opts``."""
    _fields_ = ([(f, ctypes.c_double) for f in ("lr", "beta1", "beta2", "eps")]
                + [("step", ctypes.c_int64), ("state_rounding", ctypes.c_int32), ("reserved", ctypes.c_int32 * 5)])


def declare(L):
    """The argument types of moe_block.h's functions (``moe_ffn.lib`` calls it once)."""
    vp, i64, i32, f32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    opts, gate, balance = (ctypes.POINTER(c) for c in (_m.moe_ffn_opts, moe_gate_opts, moe_balance_opts))
    for name, args in (
            ("moe_rms_norm_forward", [vp, i32, vp, i32, vp, f32, i64, i64, vp, vp, vp, vp, vp]),
            ("moe_rms_norm_backward", [vp, i32, vp, vp, i32, vp, f32, i64, i64, vp, vp, vp, sz, vp]),
            ("moe_gate_forward", [vp, vp, i64, i64, i64, gate, vp, vp, vp, vp]),
            ("moe_gate_backward", [vp, vp, vp, i64, i64, i64, gate, vp, vp]),
            ("moe_ffn_forward_routed", [vp] * 8 + [i64] * 5 + [vp, vp, sz, opts, vp]),
            ("moe_ffn_backward_routed", [vp] * 6 + [i64] * 5 + [vp] * 5 + [sz, i32, opts, vp]),
            ("moe_ffn_forward_routed_train", [vp] * 5 + [i64] * 5 + [vp, vp, sz, opts, vp]),
            ("moe_orthogonalize", [vp, i32, i64, i64, i64, i32, f32, f32, f32, f32, f32, vp, vp, sz, vp]),
            ("moe_balance_loss_forward", [vp] * 3 + [i64] * 4 + [balance, vp, vp, vp, vp, sz, vp]),
            ("moe_balance_loss_backward", [vp] * 3 + [i64] * 4 + [balance, vp, vp, vp, vp]),
            ("moe_grad_norm", [ctypes.POINTER(moe_tensor), i64, f32, vp, vp, sz, vp]),
            ("moe_adamw_step", [ctypes.POINTER(moe_adamw_tensor), i64, ctypes.POINTER(moe_adamw_opts), vp, vp, vp, vp,
                                sz, vp])):
        f = getattr(L, name)
        f.argtypes, f.restype = args, i32
    for name, n in (("moe_rms_norm_backward_workspace_bytes", 2), ("moe_ffn_routed_workspace_bytes", 5),
                    ("moe_ffn_routed_backward_workspace_bytes", 5),
                    ("moe_orthogonalize_workspace_bytes", 3), ("moe_balance_loss_workspace_bytes", 3),
                    ("moe_grad_norm_workspace_bytes", 1)):
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


def _here(device, *others):
    """The tensors are on one device, and it is the current one, where the library runs."""
    for t in others:
        if t is not None and t.device != device:
            raise ValueError(f"tensors on {t.device} and on {device}")
    if device.index != torch._C._cuda_getDevice():
        raise ValueError(f"tensors on {device}, but the current device is cuda:{torch.cuda.current_device()}")


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


# The structs of a few settings are kept by the settings' values: a tensor among
# them is read at every call, since a cache would take it by its identity.
def _gate_opts(score, renormalize, scale, groups=1, topk_groups=1):
    return _kept_gate_opts(score, bool(renormalize), float(scale), operator.index(groups), operator.index(topk_groups))


@functools.lru_cache(maxsize=64)
def _kept_gate_opts(score, renormalize, scale, groups, topk_groups):
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


# ------------------------------------------------------------------ load-balance loss
class BalanceOutput(NamedTuple):
    loss: torch.Tensor      # f32 [3]: coef * balance + z_coef * z, balance, z
    counts: torch.Tensor    # int32 [S, E]: tokens of a sequence that chose an expert
    prob: torch.Tensor      # f32 [S, E]: the sequence's mean probabilities


def moe_balance_loss_workspace_bytes(T, S, E) -> int:
    return int(_m.lib().moe_balance_loss_workspace_bytes(T, S, E))


def new_balance_workspace(T, E, S=1, device="cuda", stream=None):
    """For T tokens, E experts and S sequences."""
    return _workspace(moe_balance_loss_workspace_bytes(T, S, E), device, stream, "workspace size")


def _balance_opts(score, coef, z_coef):
    return _kept_balance_opts(score, float(coef), float(z_coef))


@functools.lru_cache(maxsize=64)
def _kept_balance_opts(score, coef, z_coef):
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, got {score!r}")
    return ctypes.byref(moe_balance_opts(_SCORES[score], coef, z_coef))


def _sequences(seq_offsets):
    if seq_offsets.dim() != 1 or seq_offsets.shape[0] < 2:
        raise ValueError(f"seq_offsets must be [sequences + 1], got {tuple(seq_offsets.shape)}")
    _is(seq_offsets, seq_offsets.shape, torch.int32, "seq_offsets")
    return seq_offsets.shape[0] - 1


def moe_balance_loss_forward(logits, topk_idx, score: str = "softmax", coef: float = 1e-2, z_coef: float = 0.0,
                             seq_offsets=None, loss=None, counts=None, prob=None, workspace=None,
                             stream=None) -> BalanceOutput:
    """The load-balance loss of logits f32 [T,E] for the gate's choice
    topk_idx int32 [T,k], with each expert's count and mean probability:
    balance = sum_i n_i / N * E * sum_e counts / (k n_i) * prob over the
    sequences of seq_offsets (int32 [S+1], nullable: all tokens are one),
    z = the mean of logsumexp(logits)^2."""
    T, E = logits.shape
    k = topk_idx.shape[1]
    _is(logits, (T, E), torch.float32, "logits")
    _is(topk_idx, (T, k), torch.int32, "topk_idx")
    S = 1 if seq_offsets is None else _sequences(seq_offsets)
    dev, empty = logits.device, torch.empty if stream is None else _empty_on(stream)
    _here(dev, topk_idx, seq_offsets, loss, counts, prob, workspace)
    if loss is None:
        loss = empty((3,), dtype=torch.float32, device=dev)
    else:
        _is(loss, (3,), torch.float32, "loss")
    if counts is None:
        counts = empty((S, E), dtype=torch.int32, device=dev)
    else:
        _is(counts, (S, E), torch.int32, "counts")
    if prob is None:
        prob = empty((S, E), dtype=torch.float32, device=dev)
    else:
        _is(prob, (S, E), torch.float32, "prob")
    if workspace is None:
        workspace = new_balance_workspace(T, E, S, device=dev, stream=stream)
    status = _lib().moe_balance_loss_forward(
        logits.data_ptr(), topk_idx.data_ptr(), _ptr(seq_offsets), T, S, E, k, _balance_opts(score, coef, z_coef),
        loss.data_ptr(), counts.data_ptr(), prob.data_ptr(), workspace.data_ptr(), _size(workspace),
        _stream(stream, dev))
    _check(status, "moe_balance_loss_forward")
    return BalanceOutput(loss, counts, prob)


def moe_balance_loss_backward(logits, counts, k: int, score: str = "softmax", coef: float = 1e-2, z_coef: float = 0.0,
                              seq_offsets=None, dloss=None, dlogits_in=None, dlogits=None, stream=None):
    """dlogits f32 [T,E] = dloss * d loss[0] / d logits + dlogits_in, for
    the counts int32 [S,E] of moe_balance_loss_forward and the same score,
    coefficients and sequences.  dloss f32 [1] (nullable: 1); dlogits_in f32
    [T,E] (nullable), which ``dlogits`` may be itself."""
    T, E = logits.shape
    _is(logits, (T, E), torch.float32, "logits")
    S = 1 if seq_offsets is None else _sequences(seq_offsets)
    dev = logits.device
    _here(dev, counts, seq_offsets, dloss, dlogits_in, dlogits)
    _is(counts, (S, E), torch.int32, "counts")
    if dloss is not None:
        _is(dloss, (1,), torch.float32, "dloss")
    if dlogits_in is not None:
        _is(dlogits_in, (T, E), torch.float32, "dlogits_in")
    if dlogits is None:
        empty = torch.empty if stream is None else _empty_on(stream)
        dlogits = empty((T, E), dtype=torch.float32, device=dev)
    else:
        _is(dlogits, (T, E), torch.float32, "dlogits")
    status = _lib().moe_balance_loss_backward(
        logits.data_ptr(), counts.data_ptr(), _ptr(seq_offsets), T, S, E, k, _balance_opts(score, coef, z_coef),
        _ptr(dloss), _ptr(dlogits_in), dlogits.data_ptr(), _stream(stream, dev))
    _check(status, "moe_balance_loss_backward")
    return dlogits


# ------------------------------------------------------------------ clipping and AdamW
STATE_BLOCK = 256   # elements that share a scale of an 8-bit state


def _one_device(devices, what):
    """The one device of a list's tensors, None of an empty one."""
    if len(devices) > 1:
        raise ValueError(f"{what} are on several devices: {sorted(map(str, devices))}")
    return next(iter(devices), None)


def _addresses(tensors):
    return list(map(torch.Tensor.data_ptr, tensors))


def _same_memory(tensors, addresses):
    """Whether the tensors of a list have the addresses packed in bytes."""
    return _pack(_addresses(tensors)) == addresses


def _pack(addresses):
    return array.array("Q", addresses).tobytes()


_tensors = _build.load_tensors()
if _tensors is not None:
    _same_memory = _tensors.same_memory


def _span(t):
    return t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()


class GradList:
    """The gradients of a step, bf16 or f32, as moe_grad_norm takes them: made
    once for tensors that keep their memory (others are refused then)."""

    def __init__(self, grads):
        self.grads = list(grads)
        for i, g in enumerate(self.grads):
            if not (g.is_cuda and g.is_contiguous()):
                _is(g, g.shape, g.dtype, f"grads[{i}]")
        self.device = _one_device({g.device for g in self.grads}, "grads")
        addresses = _addresses(self.grads)
        self.addresses = _pack(addresses)
        self.array = (moe_tensor * len(self.grads))(
            *(moe_tensor(a, g.numel(), _type(g, "a gradient")) for a, g in zip(addresses, self.grads)))

    def check(self):
        if not _same_memory(self.grads, self.addresses):
            raise ValueError("a gradient's memory is no longer the one that it was given with")


def moe_grad_norm_workspace_bytes(count) -> int:
    return int(_m.lib().moe_grad_norm_workspace_bytes(count))


def new_grad_norm_workspace(count, device="cuda", stream=None):
    """For ``count`` gradients."""
    return _workspace(moe_grad_norm_workspace_bytes(count), device, stream, "workspace size")


def moe_grad_norm(grads, max_norm: float = math.inf, out=None, workspace=None, stream=None):
    """f32 [2]: the norm of all gradients together, and the factor that clips
    it to max_norm (1 where it is not above; NaN where the norm is no finite
    number).  ``grads``: a list of tensors, a GradList or an AdamWPlan."""
    if isinstance(grads, AdamWPlan):
        grads = grads.grad_list()
    if isinstance(grads, GradList):
        grads.check()
    else:
        grads = GradList(grads)
    n, dev = len(grads.grads), grads.device
    if dev is None:
        dev = torch.device("cuda", torch.cuda.current_device()) if out is None else out.device
    _here(dev, out, workspace)
    if out is None:
        out = (torch.empty if stream is None else _empty_on(stream))((2,), dtype=torch.float32, device=dev)
    else:
        _is(out, (2,), torch.float32, "out")
    if workspace is None:
        workspace = new_grad_norm_workspace(n, device=dev, stream=stream)
    _check(_lib().moe_grad_norm(grads.array, n, max_norm, out.data_ptr(), workspace.data_ptr(), _size(workspace),
                                _stream(stream, dev)), "moe_grad_norm")
    return out


class AdamWState(NamedTuple):
    """The moments of a weight: f32 tensors of its shape; or E4M3 tensors
    (torch.float8_e4m3fn) with f32 scales [ceil(elements / STATE_BLOCK)], of
    which v's stand for sqrt(v)."""
    m: torch.Tensor
    v: torch.Tensor
    m_scale: torch.Tensor | None = None
    v_scale: torch.Tensor | None = None


def new_adamw_state(weight, bits: int = 32) -> AdamWState:
    """The state of a weight before its first step, in 32 or in 8 bits."""
    if bits not in (8, 32):
        raise ValueError(f"bits must be 8 or 32, got {bits}")
    shape, dev = tuple(weight.shape), weight.device
    if bits == 32:
        return AdamWState(*(torch.zeros(shape, dtype=torch.float32, device=dev) for _ in range(2)))
    blocks = -(-weight.numel() // STATE_BLOCK)
    return AdamWState(*(torch.zeros(shape, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn) for _ in range(2)),
                      *(torch.zeros(blocks, dtype=torch.float32, device=dev) for _ in range(2)))


class AdamWPlan:
    """The tensors of an AdamW step, checked once: weights (bf16 or f32,
    updated in place), their states, FP32 masters (nullable, per weight) of
    which the weights are the rounding, and each weight's weight_decay and
    lr_factor (one number or a list).  Gradients (bf16 or f32, the weights'
    shapes) are given here or by set_grads; a captured step reads the ones
    that it was captured with.  The tensors keep their memory for as long as
    the plan is used: a step of which a weight, master, moment, scale or
    gradient has other memory (``w.data = ...``) is refused, and takes a new
    plan or set_grads."""

    def __init__(self, weights, states, masters=None, weight_decay=0.0, lr_factor=1.0, grads=None):
        self.weights, self.states = list(weights), [AdamWState(*s) for s in states]
        n = len(self.weights)
        self.masters = [None] * n if masters is None else list(masters)
        decay, factor = ([x] * n if isinstance(x, (int, float)) else list(x) for x in (weight_decay, lr_factor))
        for name, x in (("states", self.states), ("masters", self.masters), ("weight_decay", decay),
                        ("lr_factor", factor)):
            if len(x) != n:
                raise ValueError(f"{name}: {len(x)} for {n} weights")
        rows, devices, spans = [], set(), []
        self._written = []  # all that a step writes, with the addresses that its descriptors have

        def written(t, shape, dtype, name):  # its address, after the checks
            if not (t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous()):
                _is(t, shape, dtype, f"{name}[{len(rows)}]")
            at = t.data_ptr()
            devices.add(t.device)
            spans.append((at, at + t.numel() * t.element_size()))
            self._written.append(t)
            return at

        for w, s, master, d, f in zip(self.weights, self.states, self.masters, decay, factor):
            shape, elements, bits8 = w.shape, w.numel(), s.m_scale is not None or s.v_scale is not None
            if bits8 and (s.m_scale is None or s.v_scale is None):
                raise ValueError(f"states[{len(rows)}]: m_scale and v_scale go together")
            kind, blocks = torch.float8_e4m3fn if bits8 else torch.float32, (-(-elements // STATE_BLOCK),)
            rows.append(moe_adamw_tensor(
                written(w, shape, w.dtype, "weights"),
                None if master is None else written(master, shape, torch.float32, "masters"), None,
                written(s.m, shape, kind, "m of weights"), written(s.v, shape, kind, "v of weights"),
                written(s.m_scale, blocks, torch.float32, "m_scale of weights") if bits8 else None,
                written(s.v_scale, blocks, torch.float32, "v_scale of weights") if bits8 else None,
                elements, _type(w, f"weights[{len(rows)}]"), 0, 8 if bits8 else 32, f, d))
        self.array = (moe_adamw_tensor * n)(*rows)
        self.device = _one_device(devices, "weights and states")
        self._written_at = [s[0] for s in spans]
        self._spans = sorted(s for s in spans if s[0] < s[1])
        if any(b[0] < a[1] for a, b in zip(self._spans, self._spans[1:])):
            raise ValueError("weights, masters and states must not overlap: each is updated once")
        self.grads = self._grad_list = None
        if grads is not None:
            self.set_grads(grads)

    def set_grads(self, grads):
        """The gradients of the steps from here on, which the plan keeps; None
        lets go of them."""
        if grads is None:
            self.grads = self._grad_list = None
            return
        grads = list(grads)
        addresses = []
        if len(grads) != len(self.weights):
            raise ValueError(f"grads: {len(grads)} for {len(self.weights)} weights")
        for i, (g, w) in enumerate(zip(grads, self.weights)):
            if not (g.dtype in _TYPES and g.shape == w.shape and g.is_cuda and g.is_contiguous()):
                _is(g, w.shape, g.dtype, f"grads[{i}]")
                _type(g, f"grads[{i}]")
            if g.device != self.device:
                raise ValueError(f"grads[{i}] is on {g.device}, not on {self.device}")
            start, end = _span(g)
            at = bisect.bisect_left(self._spans, (end,))  # the spans from here on start behind it
            if start < end and at and self._spans[at - 1][1] > start:
                raise ValueError(f"grads[{i}] overlaps with a weight, master or state")
            addresses.append(start)
        for d, g, start in zip(self.array, grads, addresses):
            d.grad, d.grad_type = start, _TYPES[g.dtype]
        self.grads, self._grad_list = grads, None
        self._tensors, self._addresses = self._written + grads, _pack(self._written_at + addresses)

    def grad_list(self) -> GradList:
        if self.grads is None:
            raise ValueError("the plan has no gradients yet")
        if self._grad_list is None:
            self._grad_list = GradList(self.grads)
        return self._grad_list


def moe_adamw_step(plan: AdamWPlan, step, lr=1e-3, betas=(0.9, 0.999), eps: float = 1e-8, grad_scale=None,
                   workspace=None, stream=None, rounding: str = "auto") -> None:
    """One AdamW step of the plan's weights, in place.  ``step``: its number,
    from 1; or an int32 CUDA tensor [1] with the steps taken so far, to which
    the call adds one (a plan without weights does too).  ``lr``: a number or an f32 CUDA tensor [1].
    ``grad_scale`` f32 [1] (nullable; moe_grad_norm's [1:]): the gradients'
    factor; where it is NaN or infinite nothing changes.  With tensors for
    step and lr a captured step's replays go on counting.  ``rounding`` of
    8-bit states: "nearest", which follows the gradients with betas up to 0.95;
    "random", which does with any; "auto", the one or the other by the betas."""
    if rounding not in _ROUNDINGS:
        raise ValueError(f"rounding must be one of {sorted(_ROUNDINGS)}, got {rounding!r}")
    if plan.grads is None and plan.weights:
        raise ValueError("the plan has no gradients yet")
    if plan.weights and not _same_memory(plan._tensors, plan._addresses):
        raise ValueError("a tensor's memory is no longer the one that the plan was made for: "
                         "weights, masters, states and gradients keep theirs")
    counter = lr_at = None
    if isinstance(step, torch.Tensor):
        _is(step, (1,), torch.int32, "step")
        counter, step = step, 0
    if isinstance(lr, torch.Tensor):
        _is(lr, (1,), torch.float32, "lr")
        lr_at, lr = lr, 0.0
    if grad_scale is not None:
        _is(grad_scale, (1,), torch.float32, "grad_scale")
    dev = plan.device
    if dev is None:  # no weights: the device that counts, where there is one
        dev = next((t.device for t in (counter, lr_at, grad_scale) if t is not None), None)
    if dev is not None:
        _here(dev, counter, lr_at, grad_scale, workspace)
    if counter is not None and workspace is None:
        workspace = _workspace(256, dev, stream, "workspace size")
    o = moe_adamw_opts(lr, betas[0], betas[1], eps, step, _ROUNDINGS[rounding])
    p = _ptr
    _check(_lib().moe_adamw_step(plan.array, len(plan.weights), ctypes.byref(o), p(grad_scale), p(lr_at), p(counter),
                                 p(workspace), 0 if workspace is None else _size(workspace),
                                 None if dev is None else _stream(stream, dev)), "moe_adamw_step")
