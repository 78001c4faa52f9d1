"""The training step's later operators on the host: their 64-bit definitions
are pinned (derivatives against differences, closed forms), and the C entries
and the binding refuse bad arguments before any CUDA call."""
import ctypes
import math

import numpy as np
import pytest
import torch

from tests import step_ref as ref

pytestmark = pytest.mark.cpu

FAKE = 0x10000  # 16- and 256-byte aligned, never dereferenced: every case fails validation first
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    from mixture_experts_ffn_gate_gb300 import _build, moe_ffn
    _build.build()
    return moe_ffn.lib()


@pytest.fixture(scope="module")
def mb():
    from mixture_experts_ffn_gate_gb300 import moe_block
    return moe_block


# ------------------------------------------------------------------ the definitions
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("z_coef", [0.0, 0.3])
@pytest.mark.parametrize("offsets", [None, [2, 5, 5, 9]])
def test_balance_gradient_is_the_derivative(kind, z_coef, offsets):
    r = np.random.default_rng(0)
    logits, idx = r.normal(size=(11, 6)), np.array([r.permutation(6)[:3] for _ in range(11)])
    _, counts, _ = ref.balance(logits, idx, kind, 0.7, z_coef, offsets)
    got, _ = ref.balance_grad(logits, counts, 3, kind, 0.7, z_coef, offsets, dloss=1.3)
    for _ in range(3):
        d, h = r.normal(size=logits.shape), 1e-6
        lo, hi = (1.3 * ref.balance(logits + s * h * d, idx, kind, 0.7, z_coef, offsets)[0][0] for s in (-1, 1))
        assert np.isclose((got * d).sum(), (hi - lo) / (2 * h), rtol=1e-6)


def test_an_even_choice_of_even_experts_has_balance_one():
    idx = np.arange(24).reshape(8, 3) % 6
    loss, counts, prob = ref.balance(np.zeros((8, 6)), idx, "softmax", 1.0, 1.0)
    assert np.allclose(loss, [1 + math.log(6) ** 2, 1, math.log(6) ** 2])
    assert (counts == 4).all() and np.allclose(prob, 1 / 6)
    loss, _, _ = ref.balance(np.where(np.arange(6) == 0, 50.0, 0.0) + np.zeros((8, 6)), np.zeros((8, 1), int),
                             "softmax", 1.0, 0.0)
    assert np.isclose(loss[1], 6)  # all of it on one of six


def test_counts_leave_out_repeated_and_invalid_slots():
    idx = np.array([[0, 0, 3], [-1, 2, 9], [1, 2, 1]])
    _, counts, _ = ref.balance(np.zeros((3, 4)), idx, "softmax", 1.0, 0.0)
    assert counts.tolist() == [[1, 1, 2, 1]]


def test_adamw_is_the_textbook_one():
    """The first step moves by lr in the gradient's direction; a run of steps
    equals torch's in FP64."""
    r = np.random.default_rng(1)
    w0, grads = r.normal(size=20), r.normal(size=(5, 20))
    w, m, v = w0.copy(), np.zeros(20), np.zeros(20)
    for t, g in enumerate(grads, 1):
        w, m, v, *_ = ref.adamw(w, g, m, v, t, 0.1, 0.9, 0.95, 1e-8, 0.2)
        if t == 1:
            assert np.allclose(w, w0 * (1 - 0.1 * 0.2) - 0.1 * np.sign(g), atol=1e-6)
    p = torch.nn.Parameter(torch.from_numpy(w0.copy()))
    o = torch.optim.AdamW([p], lr=0.1, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.2)
    for g in grads:
        p.grad = torch.from_numpy(g.copy())
        o.step()
    assert np.allclose(p.detach().numpy(), w, rtol=1e-12)


def test_codes_are_torchs():
    r = np.random.default_rng(2)
    x = (r.normal(size=700) * 10.0 ** r.uniform(-6, 0, size=700))
    q, scale, _ = ref.to_codes(x)
    t = torch.from_numpy(x / np.repeat(scale, 256)[:700]).clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    # torch goes by FP32 first
    assert (t != q).sum() <= 1 and len(scale) == 3
    ties = np.array([448.0] + [17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10] + [0.0] * 251)
    assert ref.to_codes(ties)[0][:5].tolist() == [448.0, 16.0, 20.0, 0.0, 2.0 ** -8]


def test_slots_of_blocks_and_sequences_are_distinct():
    """A block of rows that meets a sequence adds to the slot block + sequence:
    distinct for every pair, below the number of blocks and sequences together,
    and a sequence's are those from its first row's block to its last one's."""
    r = np.random.default_rng(3)
    for _ in range(200):
        T, S, chunk = int(r.integers(1, 300)), int(r.integers(1, 80)), int(r.integers(1, 40))
        off = np.concatenate(([0], np.sort(r.integers(0, T + 1, S))))
        blocks, pairs = -(-T // chunk), set()
        for b in range(blocks):
            for i in range(S):
                if max(off[i], b * chunk) < min(off[i + 1], (b + 1) * chunk):
                    pairs.add((b, i))
        slots = [b + i for b, i in pairs]
        assert len(set(slots)) == len(slots) and all(s < blocks + S for s in slots)
        for i in range(S):
            mine = sorted(b for b, j in pairs if j == i)
            want = list(range(off[i] // chunk, (off[i + 1] - 1) // chunk + 1)) if off[i] < off[i + 1] else []
            assert mine == want


# ------------------------------------------------------------------ refusals of the C entries
def balance_opts(mb, **f):
    o = mb.moe_balance_opts(0, 1e-2, 0.0)
    for n, v in f.items():
        setattr(o, n, v)
    return o


@pytest.mark.parametrize("case,want", [
    (dict(T=-1), 1), (dict(S=0), 1), (dict(E=0), 1), (dict(k=0), 1), (dict(k=9), 1), (dict(E=1025), 2),
    (dict(E=64, k=33), 2), (dict(T=1 << 30), 2), (dict(T=1 << 29), 2), (dict(S=(1 << 20) + 1), 2), (dict(S=2, off=None), 1),
    (dict(T=1 << 40), 2),
    (dict(o=None), 1), (dict(score=2), 1), (dict(score=-1), 1), (dict(coef=NAN), 1), (dict(z_coef=INF), 1),
    (dict(reserved=1), 1), (dict(logits=None), 1), (dict(idx=None), 1), (dict(loss=None), 1), (dict(counts=None), 1),
    (dict(prob=None), 1), (dict(logits=FAKE + 4), 1), (dict(idx=FAKE + 8), 1), (dict(off=FAKE + 4), 1),
    (dict(loss=FAKE + 4), 1), (dict(counts=FAKE + 4), 1), (dict(prob=FAKE + 4), 1), (dict(ws=None), 1),
    (dict(ws=FAKE + 16), 1), (dict(n=100), 5), (dict(T=0, loss=None), 1),
])
def test_balance_forward_refusals(L, mb, case, want):
    a = dict(logits=FAKE, idx=FAKE, off=FAKE, T=64, S=3, E=8, k=4, loss=FAKE, counts=FAKE, prob=FAKE, ws=FAKE,
             n=1 << 40, o=balance_opts(mb))
    for name, v in case.items():
        if name == "reserved":
            a["o"].reserved[2] = v
        elif name in ("score", "coef", "z_coef"):
            setattr(a["o"], name, v)
        else:
            a[name] = v
    o = None if a["o"] is None else ctypes.byref(a["o"])
    assert L.moe_balance_loss_forward(a["logits"], a["idx"], a["off"], a["T"], a["S"], a["E"], a["k"], o, a["loss"],
                                      a["counts"], a["prob"], a["ws"], a["n"], None) == want


@pytest.mark.parametrize("case,want", [
    (dict(T=-1), 1), (dict(S=0), 1), (dict(k=9), 1), (dict(E=1025), 2), (dict(S=2, off=None), 1), (dict(o=None), 1),
    (dict(logits=None), 1), (dict(counts=None), 1), (dict(out=None), 1), (dict(logits=FAKE + 4), 1),
    (dict(counts=FAKE + 4), 1), (dict(base=FAKE + 8), 1), (dict(out=FAKE + 8), 1), (dict(dloss=FAKE + 2), 1),
    (dict(T=0, logits=None), 0),
])
def test_balance_backward_refusals(L, mb, case, want):
    a = dict(logits=FAKE, counts=FAKE, off=FAKE, T=64, S=3, E=8, k=4, dloss=FAKE, base=FAKE, out=FAKE,
             o=balance_opts(mb))
    a.update(case)
    o = None if a["o"] is None else ctypes.byref(a["o"])
    assert L.moe_balance_loss_backward(a["logits"], a["counts"], a["off"], a["T"], a["S"], a["E"], a["k"], o,
                                       a["dloss"], a["base"], a["out"], None) == want


def test_workspace_sizes(L, mb):
    assert mb.moe_balance_loss_workspace_bytes(64, 1, 1025) == 0 == mb.moe_balance_loss_workspace_bytes(-1, 1, 8)
    assert mb.moe_balance_loss_workspace_bytes(0, 1, 8) > 0
    assert mb.moe_balance_loss_workspace_bytes(1 << 20, 4, 256) < 1 << 23
    assert mb.moe_grad_norm_workspace_bytes(-1) == 0 == mb.moe_grad_norm_workspace_bytes(65537)
    assert mb.moe_grad_norm_workspace_bytes(0) > 0


@pytest.mark.parametrize("case,want", [
    (dict(count=-1), 1), (dict(count=65537), 2), (dict(list=None), 1), (dict(max_norm=0.0), 1),
    (dict(max_norm=-1.0), 1), (dict(max_norm=NAN), 1), (dict(out=None), 1), (dict(out=FAKE + 2), 1), (dict(ws=None), 1),
    (dict(ws=FAKE + 16), 1), (dict(bytes=16), 5), (dict(type=2), 1), (dict(reserved=1), 1), (dict(data=None), 1),
    (dict(data=FAKE + 4), 1), (dict(n=-1), 1), (dict(n=1 << 43), 2), (dict(n=1 << 42), 2),
])
def test_grad_norm_refusals(L, mb, case, want):
    a = dict(count=2, max_norm=1.0, out=FAKE, ws=FAKE, bytes=1 << 40)
    g = (mb.moe_tensor * 2)(mb.moe_tensor(FAKE, 8, 1, 0), mb.moe_tensor(FAKE, 8, 0, 0))
    a["list"] = g
    for name, v in case.items():
        if name in a:
            a[name] = v
        else:
            setattr(g[1], name, v)
    assert L.moe_grad_norm(a["list"], a["count"], a["max_norm"], a["out"], a["ws"], a["bytes"], None) == want


@pytest.mark.parametrize("case,want", [
    (dict(count=-1), 1), (dict(count=65537), 2), (dict(list=None), 1), (dict(o=None), 1), (dict(lr=-1.0), 1),
    (dict(lr=NAN), 1), (dict(lr=INF), 1), (dict(lr=1e300), 1), (dict(beta1=1.0), 1), (dict(beta1=-0.1), 1),
    (dict(beta2=1.0), 1), (dict(beta2=NAN), 1), (dict(eps=-1.0), 1), (dict(eps=INF), 1), (dict(step=0), 1),
    (dict(opts_reserved=1), 1), (dict(scale=FAKE + 2), 1), (dict(lr_at=FAKE + 2), 1), (dict(counter=FAKE + 2), 1),
    (dict(counter=FAKE, ws=None), 1), (dict(counter=FAKE, ws=FAKE + 16), 1), (dict(counter=FAKE, bytes=64), 5),
    (dict(w=None), 1), (dict(w=FAKE + 8), 1), (dict(master=FAKE + 4), 1), (dict(grad=None), 1), (dict(grad=FAKE + 2), 1),
    (dict(m=None), 1), (dict(v=FAKE + 4), 1), (dict(state_bits=16), 1), (dict(state_bits=8), 1),
    (dict(state_bits=8, m_scale=FAKE, v_scale=FAKE + 2), 1), (dict(n=-1), 1), (dict(n=1 << 43), 2), (dict(w_type=2), 1),
    (dict(grad_type=-1), 1), (dict(lr_factor=NAN), 1), (dict(weight_decay=INF), 1), (dict(reserved=1), 1),
])
def test_adamw_refusals(L, mb, case, want):
    a = dict(count=2, o=mb.moe_adamw_opts(1e-3, 0.9, 0.99, 1e-8, 1), scale=None, lr_at=None, counter=None, ws=FAKE,
             bytes=256)
    t = (mb.moe_adamw_tensor * 2)()
    for d in t:
        d.w = d.grad = d.m = d.v = FAKE
        d.n, d.state_bits, d.lr_factor, d.w_type, d.grad_type = 8, 32, 1.0, 0, 1
    a["list"] = t
    for name, v in case.items():
        if name in a:
            a[name] = v
        elif name == "opts_reserved":
            a["o"].reserved[0] = v
        else:
            setattr(a["o"] if name in ("lr", "beta1", "beta2", "eps", "step") else t[1], name, v)
    o = None if a["o"] is None else ctypes.byref(a["o"])
    assert L.moe_adamw_step(a["list"], a["count"], o, a["scale"], a["lr_at"], a["counter"], a["ws"], a["bytes"],
                            None) == want


def test_the_structs_have_the_headers_sizes(mb):
    assert [ctypes.sizeof(c) for c in (mb.moe_balance_opts, mb.moe_tensor, mb.moe_adamw_tensor, mb.moe_adamw_opts)] == \
        [32, 24, 88, 64]


# ------------------------------------------------------------------ the binding
def test_the_binding_refuses_host_tensors_and_shapes(mb):
    l, idx = torch.zeros(4, 8), torch.zeros(4, 2).int()
    for call in (lambda: mb.moe_balance_loss_forward(l, idx), lambda: mb.moe_balance_loss_backward(l, idx, 2),
                 lambda: mb.GradList([l]), lambda: mb.moe_grad_norm([l]),
                 lambda: mb.AdamWPlan([l], [mb.new_adamw_state(l)])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError, match="bits"):
        mb.new_adamw_state(l, bits=16)
    with pytest.raises(ValueError, match="score"):
        mb._balance_opts("tanh", 1.0, 0.0)
    with pytest.raises(ValueError, match="states"):
        mb.AdamWPlan([l, l], [mb.new_adamw_state(l)])


@pytest.fixture()
def on_host(monkeypatch, mb):
    """The plan's other checks, on host tensors."""
    def check(t, shape, dtype, name):
        if t.dtype is not dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
            raise ValueError(name)
    monkeypatch.setattr(mb, "_is", check)
    return mb


def test_a_plan_refuses_what_does_not_fit(on_host):
    mb, w = on_host, torch.zeros(300)
    s8 = mb.new_adamw_state(w, 8)
    assert s8.m.dtype is torch.float8_e4m3fn and s8.m_scale.shape == (2,) and s8.m_scale.data_ptr()
    plan = mb.AdamWPlan([w], [s8], weight_decay=0.1)
    assert plan.array[0].state_bits == 8 and plan.array[0].n == 300 and plan.array[0].lr_factor == 1.0
    with pytest.raises(ValueError, match="no gradients"):
        mb.moe_adamw_step(plan, 1)
    with pytest.raises(ValueError, match="no gradients"):
        mb.moe_grad_norm(plan)
    for grads in ([], [torch.zeros(299)], [torch.zeros(300).half()]):
        with pytest.raises(ValueError):
            plan.set_grads(grads)
    bad = [
        ([w], [mb.AdamWState(s8.m, s8.v)], {}),                                  # codes without scales
        ([w], [mb.AdamWState(s8.m, s8.v, s8.m_scale)], {}),
        ([w], [mb.AdamWState(s8.m, s8.v, s8.m_scale[:1], s8.v_scale)], {}),
        ([w], [mb.new_adamw_state(w[:299])], {}),
        ([w.half()], [mb.new_adamw_state(w)], {}),
        ([w], [mb.new_adamw_state(w)], dict(masters=[w.bfloat16()])),
        ([w], [mb.new_adamw_state(w)], dict(masters=[w])),                       # the weight itself
        ([w, w], [mb.new_adamw_state(w), mb.new_adamw_state(w)], {}),            # twice
        ([w, torch.zeros(300)], [s8, s8], {}),                                   # a state twice
        ([w], [mb.new_adamw_state(w)], dict(weight_decay=[0.1, 0.1])),
    ]
    both = torch.zeros(400)
    bad.append(([both[:300], both[100:]], [mb.new_adamw_state(w), mb.new_adamw_state(w)], {}))  # overlapping views
    for weights, states, more in bad:
        with pytest.raises(ValueError):
            mb.AdamWPlan(weights, states, **more)


def test_an_empty_plan_does_nothing(mb):
    plan = mb.AdamWPlan([], [], grads=[])
    assert mb.moe_adamw_step(plan, 1) is None


# ------------------------------------------------------------------ streams
def test_calls_on_a_stream_allocate_there(monkeypatch, on_host):
    """What a call makes for itself is allocated on the stream that the call
    runs on, and its outputs also wait for the current stream's readers."""
    from mixture_experts_ffn_gate_gb300 import moe_ffn as m
    from tests.test_block_edges_cpu import Watch
    mb = on_host
    l, idx, w = torch.zeros(4, 8), torch.zeros(4, 2).int(), torch.zeros(64)
    counts, off = torch.zeros(3, 8).int(), torch.zeros(4).int()
    plan = mb.AdamWPlan([w], [mb.new_adamw_state(w)], grads=[w.clone()])
    calls = [lambda **s: mb.moe_balance_loss_forward(l, idx, seq_offsets=off, **s),
             lambda **s: [mb.moe_balance_loss_backward(l, counts, 2, seq_offsets=off, **s)],
             lambda **s: [mb.moe_grad_norm(plan, **s)],
             lambda **s: [mb.moe_adamw_step(plan, torch.zeros(1).int(), **s)]]
    for call in calls:
        with monkeypatch.context() as patch:
            watch = Watch(patch)
            patch.setattr(mb, "_here", lambda *a: None)
            out = [t for t in call(stream=5) if t is not None]
            assert watch.made and all(s == 5 for s, _ in watch.made)
            for t in out:
                assert any(t is kept and s.cuda_stream == 7 for s, kept in watch.kept)
            assert m._lib is not None


def test_tensors_of_other_devices_are_refused(monkeypatch, mb):
    class On:
        def __init__(self, index):
            self.device = torch.device("cuda", index)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    mb._here(On(0).device, On(0), None)
    with pytest.raises(ValueError, match="current device"):
        mb._here(On(1).device, On(1))
    with pytest.raises(ValueError, match="on cuda:1 and on cuda:0"):
        mb._here(On(0).device, On(1))


def test_a_plan_lets_go_of_its_gradients(on_host):
    mb, w = on_host, torch.zeros(16)
    plan = mb.AdamWPlan([w], [mb.new_adamw_state(w)], grads=[w.clone()])
    plan.set_grads(None)
    assert plan.grads is None
    with pytest.raises(ValueError, match="no gradients"):
        mb.moe_adamw_step(plan, 1)


def test_a_plan_refuses_gradients_that_it_would_write_to_and_moved_weights(on_host):
    mb = on_host
    both = torch.zeros(1024)
    w, s = both[256:512], mb.new_adamw_state(both[256:512])
    plan = mb.AdamWPlan([w], [s])
    plan.set_grads([both[512:768]])
    plan.set_grads([both[:256]])
    for g in (w, both[500:756], both[1:257], s.m, s.v):
        with pytest.raises(ValueError, match="overlaps"):
            plan.set_grads([g])
    free = torch.zeros(256)
    plan = mb.AdamWPlan([free], [mb.new_adamw_state(free)], grads=[torch.zeros(256)])
    for t in (free, plan.grads[0]):
        kept = t.data
        t.data = torch.zeros(256)
        with pytest.raises(ValueError, match="no longer"):
            mb.moe_adamw_step(plan, 1)
        t.data = kept
    listed = mb.GradList([free])
    free.data = torch.zeros(256)
    with pytest.raises(ValueError, match="no longer"):
        mb.moe_grad_norm(listed)
