"""The binding's and the C entries' own part of the block's operators, on the
host: where a call on a stream allocates, with a stand-in for the library."""
import contextlib

import pytest
import torch

from mixture_experts_ffn_gate_gb300 import moe_block as mb
from mixture_experts_ffn_gate_gb300 import moe_ffn as m

pytestmark = pytest.mark.cpu


# ------------------------------------------------------------------ streams
class Library:
    """Every entry succeeds, every workspace has 64 KB."""

    def __getattr__(self, name):
        return lambda *a: 1 << 16 if name.endswith("_bytes") else 0


class Watch:
    """Which stream torch allocates and zeroes on, and which tensors are
    kept for the current one."""

    def __init__(self, monkeypatch):
        self.stream, self.made, self.zeroed, self.kept = "current", [], [], []
        empty, like, zero = torch.empty, torch.empty_like, torch.Tensor.zero_

        @contextlib.contextmanager
        def on(stream):
            before, self.stream = self.stream, stream
            yield
            self.stream = before

        def made(t):
            self.made.append((self.stream, t))
            return t

        def zeroed(t):
            self.zeroed.append(self.stream)
            return zero(t)

        class Current:
            cuda_stream = 7

        patch = monkeypatch.setattr
        patch(m, "_lib", Library())
        patch(m, "_dev", lambda *a: None)
        patch(mb, "_is", lambda *a: None)
        patch(torch, "empty", lambda *a, **kw: made(empty(*a, **kw)))
        patch(torch, "empty_like", lambda *a, **kw: made(like(*a, **kw)))
        patch(torch.Tensor, "zero_", zeroed)
        patch(torch.Tensor, "record_stream", lambda t, s: self.kept.append((s, t)))
        patch(torch.cuda, "stream", on)
        patch(torch.cuda, "current_stream", lambda device=None: Current)
        patch(torch.cuda, "ExternalStream", lambda handle, device=None: handle)


def calls():
    T, H, I, E, k = 4, 64, 64, 8, 2
    x, y = torch.zeros(T, H).bfloat16(), torch.zeros(T, H)
    gu, d = torch.zeros(E, 2 * I, H).bfloat16(), torch.zeros(E, H, I).bfloat16()
    gq, dq, gs, ds = gu.byte(), d.byte(), torch.zeros(E, 2 * I, 16).byte(), torch.zeros(E, H, 16).byte()
    w, l, ti, tw = torch.ones(H), torch.zeros(T, E), torch.zeros(T, k).int(), torch.zeros(T, k)
    state = torch.zeros(1 << 16).byte()
    return {
        "norm": lambda **s: mb.moe_rms_norm_forward(x, w, residual=x, mxfp8=True, **s),
        "norm_backward": lambda **s: mb.moe_rms_norm_backward(x, w, y, **s),
        "gate": lambda **s: mb.moe_gate_forward(l, k, counts=True, **s),
        "gate_backward": lambda **s: mb.moe_gate_backward(l, ti, tw, **s),
        "routed": lambda **s: mb.moe_ffn_forward_routed(x, ti, tw, gu, d, **s),
        "routed_train": lambda **s: mb.moe_ffn_forward_routed_train(x, ti, tw, gu, d, state, **s),
        "routed_backward": lambda **s: mb.moe_ffn_backward_routed(x, ti, tw, gu, d, y, **s),
        "orthogonalize": lambda **s: mb.moe_orthogonalize(d, **s),
        "forward": lambda **s: m.moe_ffn_forward(x, l, gu, d, k, **s),
        "forward_ex": lambda **s: m.moe_ffn_forward_ex(x, l, gu, d, k, **s),
        "router": lambda **s: m.moe_ffn_forward_router(x, torch.zeros(E, H).bfloat16(), None, gu, d, k, **s),
        "mxfp8": lambda **s: m.moe_ffn_forward_mxfp8(x, l, gq, gs, dq, ds, k, **s),
        "backward": lambda **s: m.moe_ffn_backward(x, l, gu, d, y, k, **s),
        "train": lambda **s: m.moe_ffn_forward_train(x, l, gu, d, k, state, **s),
        "train_backward": lambda **s: m.moe_ffn_backward_train(x, l, gu, d, y, k, state, **s),
    }


def tensors(r):
    return [t for v in (r if isinstance(r, tuple) else (r,)) if v is not None for t in [v]]


@pytest.mark.parametrize("name", sorted(calls()))
def test_a_call_on_a_stream_allocates_there(monkeypatch, name):
    """What a call makes for itself is in the order of the stream that the
    call runs on; its outputs also wait for the current stream's readers."""
    call = calls()[name]
    watch = Watch(monkeypatch)
    out = tensors(call(stream=5))
    assert watch.made and all(s == 5 for s, _ in watch.made)
    assert all(s == 5 for s in watch.zeroed)
    for t in out:
        assert any(t is kept and s.cuda_stream == 7 for s, kept in watch.kept)


@pytest.mark.parametrize("make", ["new_workspace", "new_router_workspace", "new_backward_workspace",
                                  "new_train_state"])
def test_a_workspace_for_a_stream_is_made_there(monkeypatch, make):
    watch = Watch(monkeypatch)
    getattr(m, make)(4, 64, 64, 8, 2, device="cpu", stream=5)
    assert [s for s, _ in watch.made] == [5] and watch.zeroed == [5] and watch.stream == "current"


@pytest.mark.parametrize("stream", [None, 7])
def test_the_current_stream_is_the_default(monkeypatch, stream):
    """7 is the current stream's handle."""
    monkeypatch.setattr(mb, "_stream", lambda s, device: 7)
    call = calls()["orthogonalize"]
    watch = Watch(monkeypatch)
    call(stream=stream)
    assert watch.made and all(s == "current" for s, _ in watch.made) and not watch.kept
