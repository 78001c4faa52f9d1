"""The binding's and the C entries' own part of the block's operators, on the
host: where a call on a stream allocates, with a stand-in for the library;
the coefficients that the orthogonalisation takes."""
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
        patch(mb, "_size", lambda t, name=None: t.numel() * t.element_size())
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


# ------------------------------------------------------------------ the orthogonalisation's coefficients
USUAL = (3.4445, -4.7750, 2.0315)


def largest(coefficients, steps, slack=1.0, points=2001):
    """The largest singular value that a product reads, and the largest
    eigenvalue of b A + c A A, by trying many singular values of [0, 1];
    `slack`: how much each step may raise the largest one besides."""
    a, b, c = coefficients
    grid, end, top, poly = torch.linspace(0, 1, points, dtype=torch.float64), 1.0, 0.0, 0.0
    for _ in range(steps):
        s = grid * end
        t = s * s
        top, poly = max(top, end), max(poly, (b * t + c * t * t).abs().max().item())
        end = slack * (s * (a + b * t + c * t * t)).abs().max().item()
    return top, poly


@pytest.fixture(scope="module")
def L():
    from mixture_experts_ffn_gate_gb300 import _build
    _build.build()
    return m.lib()


def accepted(L, coefficients, steps):
    """B = 0: nothing is enqueued, and every check of the numbers runs."""
    status = L.moe_orthogonalize(None, 1, 0, 64, 96, steps, *coefficients, 1e-7, 1.0, None, None, 0, None)
    assert status in (m.MOE_OK, m.MOE_ERR_INVALID_ARG)
    return status == m.MOE_OK


@pytest.mark.parametrize("coefficients,steps,want", [
    (USUAL, 1, True), (USUAL, 5, True), (USUAL, 32, True), ((1.5, -0.5, 0.0), 32, True), ((2.0, -1.5, 0.5), 32, True),
    ((1.875, -1.25, 0.375), 32, True), ((4.0, -8.0, 4.2), 5, True), ((0.0, 0.0, 0.0), 32, True),
    ((16.0, 0.0, 0.0), 1, True), ((16.0, 0.0, 0.0), 2, False),       # the last step's X may be any size
    ((3.0, -0.5, 0.0), 1, True), ((3.0, -0.5, 0.0), 2, False),       # 1, then 2.5: A is 6.25
    ((2.0, 0.0, 0.0), 2, False), ((1.8, 0.0, 0.0), 2, True), ((1.8, 0.0, 0.0), 3, False),
    ((-1.8, 0.0, 0.0), 2, True), ((-2.5, 0.0, 0.0), 2, False), ((1.2, 0.0, 0.0), 3, True), ((1.2, 0.0, 0.0), 6, False),
    ((0.0, 16.0, 16.0), 1, False), ((0.0, 14.0, 14.0), 1, True), ((0.0, 16.0, -16.0), 1, True),
    ((0.0, -12.0, 16.0), 2, False), ((3.4445, -4.7750, 5.0), 5, False), ((float("nan"), 0.0, 0.0), 1, False)])
def test_coefficients_that_leave_the_range_are_refused(L, coefficients, steps, want):
    assert accepted(L, coefficients, steps) is want


def test_accepted_coefficients_stay_in_range(L):
    """No accepted set takes any singular value out of FP16's range, and every
    refused one would with the roundings' part in a hundred per step."""
    g = torch.Generator().manual_seed(0)
    sets = torch.rand(1000, 3, generator=g, dtype=torch.float64) * torch.tensor([8.0, 12.0, 8.0]) - \
        torch.tensor([4.0, 9.0, 1.0])
    seen = {True: 0, False: 0}
    for coefficients in sets.float().double().tolist():
        for steps in (1, 2, 5):
            ok = accepted(L, coefficients, steps)
            seen[ok] += 1
            if ok:
                top, poly = largest(coefficients, steps)
                assert top < 2.0 and poly < 32.0, (coefficients, steps)
            else:  # the grid misses an extremum by 1e-5 of it
                top, poly = largest(coefficients, steps, 1.01 * (1 + 1e-4))
                assert top > 1.9 or poly > 30.0 * (1 - 1e-4), (coefficients, steps)
    assert min(seen.values()) > 100


# ------------------------------------------------------------------ workspace sizes
SHAPE = (2048, 6144, 2048, 256, 8)


@pytest.mark.parametrize("make,plain,routed", [
    ("new_workspace", "moe_ffn_workspace_bytes", "moe_ffn_routed_workspace_bytes"),
    ("new_backward_workspace", "moe_ffn_backward_workspace_bytes", "moe_ffn_routed_backward_workspace_bytes"),
    ("new_train_state", "moe_ffn_train_state_bytes", "moe_ffn_routed_backward_workspace_bytes")])
def test_a_workspace_for_the_layer_alone_is_no_larger(L, make, plain, routed):
    meta = getattr(m, make)(*SHAPE, device="meta", routed=False)
    assert meta.numel() == getattr(L, plain)(*SHAPE)
    assert getattr(m, make)(*SHAPE, device="meta").numel() == getattr(L, routed)(*SHAPE) > meta.numel()


@pytest.mark.parametrize("name", ["forward_ex", "mxfp8"])
def test_the_layers_own_workspace_is_the_layers(monkeypatch, name):
    """Without one of the caller's, a call with logits makes no room for a given routing."""
    call = calls()[name]
    watch = Watch(monkeypatch)
    monkeypatch.setattr(m, "_lib", type("Sizes", (Library,), {"moe_ffn_routed_workspace_bytes":
                                                              lambda self, *a: 1 << 20})())
    call(stream=5)
    assert [t.numel() for _, t in watch.made if t.dtype is torch.uint8] == [1 << 16]


# ------------------------------------------------------------------ the caller's buffers
@pytest.mark.parametrize("name,buffer", [("norm_backward", "workspace"), ("routed", "workspace"),
                                         ("routed_backward", "workspace"), ("routed_backward", "state"),
                                         ("routed_train", None), ("orthogonalize", "workspace")])
def test_a_workspace_in_host_memory_is_refused(monkeypatch, name, buffer):
    """Its address is the kernels' to write to."""
    call = calls()[name]
    monkeypatch.setattr(m, "_lib", Library())
    monkeypatch.setattr(mb, "_is", lambda *a: None)
    monkeypatch.setattr(mb, "_stream", lambda s, device: 0)
    with pytest.raises(ValueError, match="CUDA"):
        call(**({buffer: torch.zeros(1 << 20, dtype=torch.uint8)} if buffer else {}))
