"""The block's operators on the host: the 64-bit definitions that the GPU
tests use are pinned (derivatives against differences, selection against a
stable sort, closed forms), and the C entries and the binding refuse bad
arguments before any CUDA call."""
import ctypes

import numpy as np
import pytest
import torch

from tests import block_ref as ref

pytestmark = pytest.mark.cpu

FAKE = 0x10000  # 16- and 256-byte aligned, never dereferenced: every case fails validation first
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    from mixture_experts_ffn_gate_gb300 import _build, moe_ffn
    _build.build()
    return moe_ffn.lib()


def opts(**f):
    from mixture_experts_ffn_gate_gb300 import moe_block as mb
    o = mb.moe_gate_opts()
    for n, v in f.items():
        setattr(o, n, v)
    return o


# ------------------------------------------------------------------ the definitions
def difference(f, x, direction, step=1e-6):
    return (f(x + step * direction) - f(x - step * direction)) / (2 * step)


def test_norm_gradient_is_the_derivative():
    r = np.random.default_rng(0)
    h, w, dy, dres = r.normal(size=(3, 24)), r.normal(size=24), r.normal(size=(3, 24)), r.normal(size=(3, 24))
    f = lambda h, w: (ref.norm(h, None, w, 1e-3)[1] * dy).sum() + (h * dres).sum()  # noqa: E731
    dh, dw, _, _ = ref.norm_grad(h, w, dy, dres, 1e-3)
    d, e = r.normal(size=h.shape), r.normal(size=w.shape)
    assert np.isclose((dh * d).sum(), difference(lambda v: f(v, w), h, d), rtol=1e-7)
    assert np.isclose((dw * e).sum(), difference(lambda v: f(h, v), w, e), rtol=1e-7)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_gate_gradient_is_the_derivative(kind, renormalize):
    r = np.random.default_rng(1)
    logits, dw = r.normal(size=(4, 9)), r.normal(size=(4, 3))
    idx, _ = ref.gate(logits, 3, None, kind, 1, 1, renormalize, 1.7)

    def f(l):
        p = np.take_along_axis(ref.scores(l, kind), idx, 1)
        return (1.7 * (p / p.sum(axis=1, keepdims=True) if renormalize else p) * dw).sum()
    d = r.normal(size=logits.shape)
    g = ref.gate_grad(logits, idx, dw, kind, renormalize, 1.7)
    assert np.isclose((g * d).sum(), difference(f, logits, d), rtol=1e-6)


def test_experts_gradient_is_the_derivative():
    r = np.random.default_rng(2)
    T, H, I, E, k = 3, 6, 4, 5, 2
    a = dict(x=r.normal(size=(T, H)), w=r.normal(size=(T, k)), wgu=r.normal(size=(E, 2 * I, H)),
             wd=r.normal(size=(E, H, I)))
    idx, dout = np.array([[0, 3], [3, 3], [4, -1]]), r.normal(size=(T, H))
    got = dict(zip(("x", "w", "wgu", "wd"), ref.experts_grad(a["x"], idx, a["w"], a["wgu"], a["wd"], dout)))
    for name, v in a.items():
        d = r.normal(size=v.shape)
        f = lambda v: (ref.experts(**{**a, name: v}, idx=idx) * dout).sum()  # noqa: E731
        assert np.isclose((got[name] * d).sum(), difference(f, v, d), rtol=1e-6), name
    assert got["w"][1, 1] == got["w"][2, 1] == 0


def test_gate_choice_is_a_stable_sort():
    r = np.random.default_rng(3)
    logits = r.integers(-2, 3, size=(20, 12)).astype(np.float64)
    idx, w = ref.gate(logits, 5, None, "softmax", 1, 1, True, 1.0)
    assert np.array_equal(idx, np.argsort(-logits, axis=1, kind="stable")[:, :5])
    assert np.allclose(w.sum(axis=1), 1)
    # groups of three, two kept: the groups of the largest maxima
    idx, _ = ref.gate(logits, 4, None, "sigmoid", 4, 2, False, 1.0)
    for t in range(20):
        best = np.argsort(-logits[t].reshape(4, 3).max(axis=1), kind="stable")[:2]
        assert set(idx[t] // 3) <= set(best)


def test_mx_values_are_the_formats():
    v = ref.e4m3_values()
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, t, equal_nan=True)


def test_orthogonalize_maps_singular_values():
    """Every singular value goes through the polynomial; the singular vectors stay."""
    r = np.random.default_rng(4)
    a, b, c = 3.4445, -4.7750, 2.0315
    g = r.normal(size=(7, 4))
    u, s, vt = np.linalg.svd(g, full_matrices=False)
    s = s / np.linalg.norm(s)
    for _ in range(5):
        s = s * (a + b * s ** 2 + c * s ** 4)
    assert np.allclose(ref.orthogonalize(g, 5, (a, b, c), 0.0), (u * s) @ vt, atol=1e-12)


# ------------------------------------------------------------------ refusals of the C entries
@pytest.mark.parametrize("case,want", [
    (dict(T=-1), 1), (dict(H=0), 1), (dict(H=16385), 2), (dict(eps=-1.0), 1), (dict(eps=NAN), 1), (dict(eps=INF), 1),
    (dict(T=1 << 40), 2), (dict(x=None), 1), (dict(w=None), 1), (dict(y=None), 1), (dict(x=FAKE + 8), 1),
    (dict(y=FAKE + 2), 1), (dict(h=FAKE), 1), (dict(h=FAKE, r=FAKE, rt=2), 1), (dict(xt=2), 1), (dict(xt=-1), 1),
    (dict(q=FAKE), 1), (dict(s=FAKE), 1), (dict(q=FAKE, s=FAKE, H=40), 2), (dict(q=FAKE, s=FAKE + 1), 1),
    (dict(T=0, x=None), 0),
])
def test_norm_forward_refusals(L, case, want):
    a = dict(x=FAKE, xt=1, r=None, rt=0, w=FAKE, eps=1e-6, T=4, H=64, h=None, y=FAKE, q=None, s=None)
    a.update(case)
    assert L.moe_rms_norm_forward(a["x"], a["xt"], a["r"], a["rt"], a["w"], a["eps"], a["T"], a["H"], a["h"], a["y"],
                                  a["q"], a["s"], None) == want


@pytest.mark.parametrize("case,want", [
    (dict(T=-1), 1), (dict(H=0), 1), (dict(H=20000), 2), (dict(eps=-1.0), 1), (dict(ht=3), 1), (dict(gt=7), 1),
    (dict(h=None), 1), (dict(w=None), 1), (dict(dy=None), 1), (dict(dh=None), 1), (dict(dw=None), 1),
    (dict(dres=FAKE + 4), 1), (dict(ws=None), 1), (dict(ws=FAKE + 16), 1), (dict(n=16), 5), (dict(T=0, dw=None), 1),
])
def test_norm_backward_refusals(L, case, want):
    a = dict(h=FAKE, ht=0, w=FAKE, dy=FAKE, gt=1, dres=None, eps=1e-6, T=4, H=64, dh=FAKE, dw=FAKE, ws=FAKE, n=1 << 40)
    a.update(case)
    assert L.moe_rms_norm_backward(a["h"], a["ht"], a["w"], a["dy"], a["gt"], a["dres"], a["eps"], a["T"], a["H"],
                                   a["dh"], a["dw"], a["ws"], a["n"], None) == want


@pytest.mark.parametrize("case,o,want", [
    (dict(T=-1), {}, 1), (dict(E=0), {}, 1), (dict(k=0), {}, 1), (dict(k=17), {}, 1), (dict(E=1025), {}, 2),
    (dict(E=64, k=33), {}, 2), (dict(l=None), {}, 1), (dict(idx=None), {}, 1), (dict(w=None), {}, 1),
    (dict(b=FAKE + 4), {}, 1), (dict(c=FAKE + 8), {}, 1), ({}, dict(score=2), 1), ({}, dict(score=-1), 1),
    ({}, dict(scale=NAN), 1), ({}, dict(groups=-1), 1), ({}, dict(groups=3, topk_groups=1), 1),
    ({}, dict(groups=4, topk_groups=0), 1), ({}, dict(groups=4, topk_groups=5), 1),
    (dict(k=8), dict(groups=4, topk_groups=1), 1), (dict(E=1024), dict(groups=64, topk_groups=64), 2),
    ({}, dict(reserved=(0, 0, 1)), 1), (dict(T=0, l=None), {}, 0), (dict(T=1 << 40), {}, 2),
])
def test_gate_forward_refusals(L, case, o, want):
    a = dict(l=FAKE, b=None, T=4, E=16, k=2, idx=FAKE, w=FAKE, c=None)
    a.update(case)
    o = opts(**{n: (ctypes.c_int32 * 3)(*v) if n == "reserved" else v for n, v in o.items()})
    assert L.moe_gate_forward(a["l"], a["b"], a["T"], a["E"], a["k"], ctypes.byref(o), a["idx"], a["w"], a["c"],
                              None) == want


@pytest.mark.parametrize("case,want", [
    (dict(T=-1), 1), (dict(k=17), 1), (dict(E=2000), 2), (dict(l=None), 1), (dict(idx=None), 1), (dict(dw=None), 1),
    (dict(d=None), 1), (dict(d=FAKE + 4), 1), (dict(T=0, l=None), 0),
])
def test_gate_backward_refusals(L, case, want):
    a = dict(l=FAKE, idx=FAKE, dw=FAKE, T=4, E=16, k=2, d=FAKE)
    a.update(case)
    assert L.moe_gate_backward(a["l"], a["idx"], a["dw"], a["T"], a["E"], a["k"], None, a["d"], None) == want


@pytest.mark.parametrize("case,want", [
    (dict(T=-1), 1), (dict(k=9), 1), (dict(H=200), 2), (dict(E=1025), 2), (dict(x=None), 1), (dict(idx=None), 1),
    (dict(w=None), 1), (dict(gu=None), 1), (dict(d=None), 1), (dict(out=None), 1), (dict(idx=FAKE + 4), 1),
    (dict(gus=FAKE), 1), (dict(ds=FAKE), 1), (dict(xs=FAKE + 1), 1), (dict(ws=None), 1), (dict(ws=FAKE + 16), 1),
    (dict(n=1024), 5), (dict(T=0, x=None), 0),
])
def test_routed_forward_refusals(L, case, want):
    a = dict(x=FAKE, xs=None, idx=FAKE, w=FAKE, gu=FAKE, gus=None, d=FAKE, ds=None, T=4, H=256, I=128, E=8, k=2,
             out=FAKE, ws=FAKE, n=1 << 40)
    a.update(case)
    assert L.moe_ffn_forward_routed(a["x"], a["xs"], a["idx"], a["w"], a["gu"], a["gus"], a["d"], a["ds"], a["T"],
                                    a["H"], a["I"], a["E"], a["k"], a["out"], a["ws"], a["n"], None, None) == want


@pytest.mark.parametrize("case,want", [
    (dict(T=-1), 1), (dict(k=9), 1), (dict(H=200), 2), (dict(x=None), 1), (dict(idx=None), 1), (dict(w=None), 1),
    (dict(gu=None), 1), (dict(d=None), 1), (dict(dout=None), 1), (dict(dx=None), 1), (dict(dw=None), 1),
    (dict(dgu=None), 1), (dict(dd=FAKE + 8), 1), (dict(ws=None), 1), (dict(ws=FAKE + 16), 1), (dict(n=1024), 5),
    (dict(T=0, dgu=None), 1),
])
def test_routed_backward_refusals(L, case, want):
    a = dict(x=FAKE, idx=FAKE, w=FAKE, gu=FAKE, d=FAKE, dout=FAKE, T=4, H=256, I=128, E=8, k=2, dx=FAKE, dw=FAKE,
             dgu=FAKE, dd=FAKE, ws=FAKE, n=1 << 40)
    a.update(case)
    assert L.moe_ffn_backward_routed(a["x"], a["idx"], a["w"], a["gu"], a["d"], a["dout"], a["T"], a["H"], a["I"],
                                     a["E"], a["k"], a["dx"], a["dw"], a["dgu"], a["dd"], a["ws"], a["n"], 0, None,
                                     None) == want


def test_routed_training_refusals(L):
    from mixture_experts_ffn_gate_gb300 import moe_ffn as m
    args = [FAKE] * 5 + [4, 256, 128, 8, 2, FAKE, FAKE]
    assert L.moe_ffn_forward_routed_train(*args, 1024, None, None) == m.MOE_ERR_WORKSPACE_TOO_SMALL
    o = m.moe_ffn_opts()
    o.path = m.MOE_PATH_DECODE
    assert L.moe_ffn_forward_routed_train(*args, 1 << 40, ctypes.byref(o), None) == m.MOE_ERR_UNSUPPORTED_SHAPE
    for i in (0, 1, 2, 3, 4, 10, 11):
        bad = list(args)
        bad[i] = None
        assert L.moe_ffn_forward_routed_train(*bad, 1 << 40, None, None) == m.MOE_ERR_INVALID_ARG, i


@pytest.mark.parametrize("case,want", [
    (dict(B=-1), 1), (dict(M=0), 1), (dict(N=0), 1), (dict(M=32769), 2), (dict(B=70000), 2), (dict(steps=0), 1),
    (dict(steps=33), 2), (dict(t=2), 1), (dict(a=17.0), 1), (dict(a=NAN), 1), (dict(b=-15.5), 1), (dict(c=INF), 1),
    (dict(eps=-1.0), 1), (dict(eps=NAN), 1), (dict(scale=INF), 1), (dict(g=None), 1), (dict(out=None), 1),
    (dict(out=FAKE + 2), 1), (dict(ws=None), 1), (dict(ws=FAKE + 16), 1), (dict(n=1024), 5), (dict(B=0, g=None), 0),
])
def test_orthogonalize_refusals(L, case, want):
    a = dict(g=FAKE, t=1, B=2, M=64, N=96, steps=5, a=3.4445, b=-4.775, c=2.0315, eps=1e-7, scale=1.0, out=FAKE,
             ws=FAKE, n=1 << 40)
    a.update(case)
    assert L.moe_orthogonalize(a["g"], a["t"], a["B"], a["M"], a["N"], a["steps"], a["a"], a["b"], a["c"], a["eps"],
                               a["scale"], a["out"], a["ws"], a["n"], None) == want


def test_workspace_sizes(L):
    assert L.moe_rms_norm_backward_workspace_bytes(4, 64) >= 4 * 64 * 4
    assert L.moe_rms_norm_backward_workspace_bytes(-1, 64) == 0
    assert L.moe_ffn_routed_workspace_bytes(4, 256, 128, 8, 2) >= L.moe_ffn_workspace_bytes(4, 256, 128, 8, 2) + 2048
    assert L.moe_ffn_routed_workspace_bytes(4, 256, 128, 8, 9) == 0
    assert L.moe_orthogonalize_workspace_bytes(2, 64, 96) >= 2 * (64 * 96 * 5 + 64 * 64 * 4)
    assert L.moe_orthogonalize_workspace_bytes(2, 64, 96) == L.moe_orthogonalize_workspace_bytes(2, 96, 64)
    assert L.moe_orthogonalize_workspace_bytes(1, 40000, 8) == 0


# ------------------------------------------------------------------ refusals of the binding
def test_binding_refuses_host_tensors_and_shapes(L):
    from mixture_experts_ffn_gate_gb300 import moe_block as mb
    x, w = torch.zeros(2, 64), torch.ones(64)
    with pytest.raises(ValueError, match="CUDA"):
        mb.moe_rms_norm_forward(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        mb.moe_rms_norm_backward(x, w, x)
    with pytest.raises(ValueError, match="CUDA"):
        mb.moe_gate_forward(x, 2)
    with pytest.raises(ValueError, match="CUDA"):
        mb.moe_gate_backward(x, torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2))
    with pytest.raises(ValueError, match="CUDA"):
        mb.moe_ffn_forward_routed(x.bfloat16(), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2),
                                  torch.zeros(4, 128, 64).bfloat16(), torch.zeros(4, 64, 64).bfloat16())
    with pytest.raises(ValueError, match="CUDA"):
        mb.moe_orthogonalize(torch.zeros(1, 4, 4))
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        mb.moe_orthogonalize(torch.zeros(1, 4, 4, dtype=torch.float16))
    with pytest.raises(ValueError, match="score"):
        mb._gate_opts("tanh", True, 1.0)
    with pytest.raises(ValueError, match="scale"):
        mb._gate_opts("softmax", True, 0.0)


def test_gate_opts_layout():
    from mixture_experts_ffn_gate_gb300 import moe_block as mb
    assert ctypes.sizeof(mb.moe_gate_opts) == 32
    assert mb.moe_gate_opts.scale.offset == 16
