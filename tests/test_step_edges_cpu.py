"""Edges of the training step's operators on the host: plans whose tensors moved,
calls without tensors, arguments that are tensors."""
import ctypes

import pytest
import torch

from mixture_experts_ffn_gate_gb300 import moe_block as mb

pytestmark = pytest.mark.cpu


@pytest.fixture()
def on_host(monkeypatch):
    """The plan's checks but for the device, on host tensors."""
    def check(t, shape, dtype, name):
        if t.dtype is not dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
            raise ValueError(name)
    monkeypatch.setattr(mb, "_is", check)


class Library:
    """In the library's place: notes the calls that reach it, with every argument."""

    def __init__(self, monkeypatch):
        self.calls = []
        monkeypatch.setattr(mb, "_lib", lambda: self)
        monkeypatch.setattr(mb, "_here", lambda *a: None)
        monkeypatch.setattr(mb, "_stream", lambda *a: None)

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("what", ["w", "master", "grad", "m", "v", "m_scale", "v_scale"])
def test_a_step_refuses_every_tensor_whose_memory_has_changed(monkeypatch, on_host, bits, what):
    """The plan's descriptors have the old memory, which is free by then."""
    if bits == 32 and "scale" in what:
        return
    library = Library(monkeypatch)
    w, master, g = torch.zeros(300).bfloat16(), torch.zeros(300), torch.zeros(300)
    s = mb.new_adamw_state(w, bits)
    plan = mb.AdamWPlan([torch.zeros(8).bfloat16(), w], [mb.new_adamw_state(torch.zeros(8)), s], masters=[None, master],
                        grads=[torch.zeros(8), g])
    t = dict(w=w, master=master, grad=g, **s._asdict())[what]
    mb.moe_adamw_step(plan, 1)
    kept = t.data
    t.data = t.detach().clone()
    with pytest.raises(ValueError, match="no longer"):
        mb.moe_adamw_step(plan, 2)
    assert len(library.calls) == 1
    t.data = kept
    mb.moe_adamw_step(plan, 2)
    assert [name for name, _ in library.calls] == ["moe_adamw_step"] * 2


def test_settings_that_are_tensors_are_read_at_every_call():
    """A coefficient that is annealed in place: the struct that the library
    gets has its value, not the first call's."""
    x = torch.tensor(0.5)
    for value in (0.5, 0.25, 2.0):
        x.fill_(value)
        for coef, z_coef in ((x, 0.0), (0.0, x)):
            o = mb._balance_opts("sigmoid", coef, z_coef)._obj
            assert (o.coef, o.z_coef) == (float(coef), float(z_coef))
        assert mb._gate_opts("softmax", True, x)._obj.scale == value
    groups = torch.tensor(2)
    for value in (2, 4):
        groups.fill_(value)
        assert mb._gate_opts("softmax", True, 1.0, groups, 1)._obj.groups == value
    for groups, topk_groups in ((2.5, 1), (2, 1.0), ("2", 1)):
        with pytest.raises(TypeError):
            mb._gate_opts("softmax", True, 1.0, groups, topk_groups)


def test_the_rounding_of_8_bit_states(monkeypatch, on_host):
    """By the betas unless it is given; others are refused, by the library too."""
    from mixture_experts_ffn_gate_gb300 import _build, moe_ffn
    _build.build()
    for bad in (-1, 3):
        o = mb.moe_adamw_opts(1e-3, 0.9, 0.99, 1e-8, 1, bad)
        assert moe_ffn.lib().moe_adamw_step(None, 0, ctypes.byref(o), None, None, None, None, 0, None) == 1
    library = Library(monkeypatch)
    w = torch.zeros(300)
    plan = mb.AdamWPlan([w], [mb.new_adamw_state(w, 8)], grads=[torch.zeros(300)])
    for rounding, code in (("auto", 0), ("nearest", 1), ("random", 2)):
        mb.moe_adamw_step(plan, 1, rounding=rounding)
        assert library.calls[-1][1][2]._obj.state_rounding == code
    with pytest.raises(ValueError, match="rounding"):
        mb.moe_adamw_step(plan, 1, rounding="up")


def test_addresses_are_compared_natively_as_in_python():
    """The built module and the plain comparison, which is what there is without it."""
    from mixture_experts_ffn_gate_gb300 import _build
    _build.build_tensors()
    native = _build.load_tensors().same_memory
    ts = [torch.zeros(n) for n in (3, 0, 5)] + [torch.zeros(8)[2:], torch.nn.Parameter(torch.zeros(4))]
    plain = lambda tensors, addresses: mb._pack(mb._addresses(tensors)) == addresses
    at = mb._pack(mb._addresses(ts))
    for same in (native, plain, mb._same_memory):
        assert same(ts, at) and same([], b"") and not same(ts, at[:8] + at[:8] + at[16:])
        kept, ts[2].data = ts[2].data, torch.zeros(5)
        assert not same(ts, at)
        ts[2].data = kept
        assert same(ts, at)
    for bad in ((tuple(ts), at), (ts, list(at)), (ts, at[:-8]), ([1], at[:8])):
        with pytest.raises((TypeError, ValueError)):
            native(*bad)


@pytest.mark.parametrize("bits", [8, None])
def test_a_block_whose_weight_is_another_tensor_is_refused(monkeypatch, on_host, bits):
    """Its step would go on with the tensor that the block no longer reads."""
    from mixture_experts_ffn_gate_gb300 import block as b
    library = Library(monkeypatch)
    block = b.MoeBlock(torch.ones(8), torch.zeros(4, 8), None, torch.zeros(4, 6, 8).bfloat16(),
                       torch.zeros(4, 8, 3).bfloat16(), b.GateSettings(k=2))
    monkeypatch.setattr(block, "update_experts", lambda *a: None)
    monkeypatch.setattr(mb, "new_grad_norm_workspace", lambda *a, **k: torch.zeros(256, dtype=torch.uint8))
    monkeypatch.setattr(mb, "_size", lambda t: t.numel())
    opt = b.BlockAdamW(block, bits=bits)
    names = ("norm_weight", "w_router", "w_gate_up", "w_down")
    grads = {n: torch.zeros(getattr(block, n).shape) for n in names}
    opt.step(grads)
    assert [name for name, _ in library.calls] == ["moe_grad_norm", "moe_adamw_step"]
    for n in names if bits else names[:2]:
        kept = getattr(block, n)
        setattr(block, n, kept.clone())
        with pytest.raises(ValueError, match="no longer"):
            opt.step(grads)
        setattr(block, n, kept)
    assert len(library.calls) == 2
    opt.step(grads)


def test_an_empty_plan_checks_its_arguments_and_counts(monkeypatch):
    """As the library does: bad numbers are refused, a counter reaches it."""
    from mixture_experts_ffn_gate_gb300 import _build
    _build.build()
    plan = mb.AdamWPlan([], [], grads=[])
    assert mb.moe_adamw_step(plan, 1) is None
    for bad in (dict(step=0), dict(lr=float("nan")), dict(betas=(0.9, 1.0)), dict(eps=-1.0)):
        with pytest.raises(mb.MoeFfnError):
            mb.moe_adamw_step(plan, **{**dict(step=1), **bad})
    with pytest.raises(ValueError):
        mb.moe_adamw_step(plan, torch.zeros(1))
    library = Library(monkeypatch)
    monkeypatch.setattr(mb, "_is", lambda *a: None)
    monkeypatch.setattr(mb, "_size", lambda t: t.numel())
    monkeypatch.setattr(mb, "_workspace", lambda n, *a: torch.zeros(n, dtype=torch.uint8))
    counter = torch.zeros(1, dtype=torch.int32)
    mb.moe_adamw_step(plan, counter)
    (name, args), = library.calls
    assert name == "moe_adamw_step" and args[1] == 0 and args[5] == counter.data_ptr() and args[7] == 256
