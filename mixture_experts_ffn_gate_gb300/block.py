"""A Mixture-of-Experts block on the library's operators, as they are used
together: norm with the residual's addition, gate, experts, their gradients
and the experts' orthogonalised update.

    python -m mixture_experts_ffn_gate_gb300.block

runs a serving step (one token and a batch, BF16 and 8-bit tokens) and a few
training steps of a small block on synthetic data, and prints the loss.
"""
from __future__ import annotations

import collections
import dataclasses
import math

import torch

from . import moe_block as mb
from . import moe_ffn as m


@dataclasses.dataclass
class GateSettings:
    """How the gate chooses (moe_gate_forward)."""
    k: int
    score: str = "sigmoid"
    groups: int = 1
    topk_groups: int = 1
    renormalize: bool = True
    scale: float = 1.0

    def backward_args(self):
        return dict(score=self.score, renormalize=self.renormalize, scale=self.scale)


class MoeBlock:
    """The weights of one block and its steps.

    norm_weight f32 [H]; w_router f32 [E,H]; balance_bias f32 [E] or None;
    w_gate_up bf16 [E,2I,H]; w_down bf16 [E,H,I].  The router projection is a
    plain matrix product of the caller's framework (torch) in FP32.
    """

    def __init__(self, norm_weight, w_router, balance_bias, w_gate_up, w_down, gate: GateSettings, eps: float = 1e-6):
        self.norm_weight, self.w_router, self.balance_bias = norm_weight, w_router, balance_bias
        self.w_gate_up, self.w_down, self.gate, self.eps = w_gate_up, w_down, gate, eps
        self.E, self.H, self.I = w_down.shape
        self._serving: collections.OrderedDict = collections.OrderedDict()

    # Serving workspaces that are kept: the fused decode kernel is quicker on
    # one that it has used before.
    KEPT = 8

    def _serving_workspace(self, T, device):
        """The workspace of the serving steps of T tokens on the current
        stream; of those least recently used only KEPT stay.  A step that is
        being captured has its own, which lives as long as its graph."""
        if torch.cuda.is_current_stream_capturing():
            return mb.new_routed_workspace(*self._shape(T), device=device)
        key = (T, torch.cuda.current_stream(device).cuda_stream)
        ws = self._serving.pop(key, None)
        if ws is None:
            ws = mb.new_routed_workspace(*self._shape(T), device=device)
        self._serving[key] = ws
        if len(self._serving) > self.KEPT:
            self._serving.popitem(last=False)
        return ws

    def _shape(self, T):
        return T, self.H, self.I, self.E, self.gate.k

    def choose(self, y):
        """The gate on normed tokens y bf16 [T,H]: (logits, GateOutput)."""
        logits = torch.matmul(y.float(), self.w_router.t())
        g = self.gate
        return logits, mb.moe_gate_forward(logits, g.k, bias=self.balance_bias, score=g.score, groups=g.groups,
                                           topk_groups=g.topk_groups, renormalize=g.renormalize, scale=g.scale,
                                           counts=True)

    def serve(self, x, residual, mxfp8_tokens: bool = False):
        """One forward step: x f32 or bf16 [T,H] joins the residual stream;
        returns (experts' output f32 [T,H], new stream, experts' loads).  With
        mxfp8_tokens the experts read the normed tokens in 8 bits."""
        T = x.shape[0]
        n = mb.moe_rms_norm_forward(x, self.norm_weight, residual=residual, eps=self.eps, mxfp8=mxfp8_tokens)
        _, choice = self.choose(n.y)
        ws = self._serving_workspace(T, x.device)
        tokens = dict(x=n.codes, x_scale=n.scales) if mxfp8_tokens else dict(x=n.y)
        out = mb.moe_ffn_forward_routed(topk_idx=choice.topk_idx, topk_w=choice.topk_w, w_gate_up=self.w_gate_up,
                                        w_down=self.w_down, workspace=ws, **tokens)
        return out, n.h, choice.counts

    def train_forward(self, x, residual):
        """The forward pass of a training step: (out, new stream, saved).
        `saved` holds this call's own state (g and u of every assignment), so
        any number of forward calls may come before their backward calls."""
        T = x.shape[0]
        n = mb.moe_rms_norm_forward(x, self.norm_weight, residual=residual, eps=self.eps)
        logits, choice = self.choose(n.y)
        state = m.new_train_state(*self._shape(T), device=x.device)
        out = mb.moe_ffn_forward_routed_train(n.y, choice.topk_idx, choice.topk_w, self.w_gate_up, self.w_down, state)
        return out, n.h, (n.y, n.h, logits, choice, state)

    def train_backward(self, saved, dout, dstream):
        """Its gradients for dout f32 [T,H] and dstream (the gradient that
        reaches the new stream besides): a dict; "x" is that of both x and the
        residual.  The norm's are taken at the new stream, h as it is kept."""
        y, h, logits, choice, state = saved
        dy, dw, dw_gate_up, dw_down = mb.moe_ffn_backward_routed(y, choice.topk_idx, choice.topk_w, self.w_gate_up,
                                                                 self.w_down, dout, state=state)
        dlogits = mb.moe_gate_backward(logits, choice.topk_idx, dw, **self.gate.backward_args())
        dy = torch.addmm(dy, dlogits, self.w_router)
        dx, dnorm = mb.moe_rms_norm_backward(h, self.norm_weight, dy, dres=dstream, eps=self.eps)
        return dict(x=dx, norm_weight=dnorm, w_router=torch.matmul(dlogits.t(), y.float()), w_gate_up=dw_gate_up,
                    w_down=dw_down, loads=choice.counts)

    def update(self, grads, lr: float, experts_lr: float, balance_rate: float = 0.0):
        """One step: the experts' matrices by their orthogonalised gradients,
        the others by the gradients, and the balance bias against the loads."""
        for name in ("w_gate_up", "w_down"):
            g, w = grads[name], getattr(self, name)
            _, M, N = g.shape
            step = mb.moe_orthogonalize(g, out_scale=-experts_lr * math.sqrt(max(1.0, M / N)))
            w.add_(step)
        self.norm_weight.add_(grads["norm_weight"], alpha=-lr)
        self.w_router.add_(grads["w_router"], alpha=-lr)
        if self.balance_bias is not None and balance_rate:
            loads = grads["loads"].float()
            self.balance_bias.add_(torch.sign(loads.mean() - loads), alpha=balance_rate)


def synthetic_block(H=256, I=128, E=16, gate=None, seed=0, device="cuda"):
    """A block with random weights."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def randn(*shape, std):
        return torch.randn(*shape, generator=g, device=device) * std

    return MoeBlock(torch.ones(H, device=device), randn(E, H, std=H ** -0.5), torch.zeros(E, device=device),
                    randn(E, 2 * I, H, std=H ** -0.5).bfloat16(), randn(E, H, I, std=I ** -0.5).bfloat16(),
                    gate or GateSettings(k=4, groups=4, topk_groups=2))


def train(block: MoeBlock, tokens=64, steps=8, seed=1, lr=1e-2, experts_lr=2e-2):
    """Fits the block's output to a fixed target; returns the losses."""
    g = torch.Generator(device=block.norm_weight.device)
    g.manual_seed(seed)
    x, stream, target = (torch.randn(tokens, block.H, generator=g, device=g.device) for _ in range(3))
    stream = stream.bfloat16()
    losses = []
    for _ in range(steps):
        out, h, saved = block.train_forward(x, stream)
        diff = out - target
        losses.append(0.5 * diff.square().mean().item())
        grads = block.train_backward(saved, diff / diff.numel(), torch.zeros_like(h))
        block.update(grads, lr, experts_lr, balance_rate=1e-3)
    return losses


def main():
    block = synthetic_block()
    for T in (1, 64):
        x = torch.randn(T, block.H, device="cuda")
        stream = torch.randn(T, block.H, device="cuda").bfloat16()
        out, _, loads = block.serve(x, stream)
        out8, _, _ = block.serve(x, stream, mxfp8_tokens=True)
        diff = ((out8 - out).norm() / out.norm()).item()
        print(f"serving {T:2d} tokens: {int((loads > 0).sum())} of {block.E} experts, "
              f"8-bit tokens differ by {diff:.3f}")
    losses = train(block)
    print("training: " + " ".join(f"{v:.4f}" for v in losses))
    if m.moe_ffn_device_faults():
        raise SystemExit("a kernel's bounded wait gave up")


if __name__ == "__main__":
    main()
