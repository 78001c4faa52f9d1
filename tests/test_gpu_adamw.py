"""The gradients' norm and the AdamW step against their 64-bit definitions."""
import math

import numpy as np
import pytest
import torch

from mixture_experts_ffn_gate_gb300 import moe_block as mb
from tests import step_ref as ref
from tests.block_ref import U

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HOW = dict(lr=1e-2, betas=(0.9, 0.95), eps=1e-8)


def f64(t):
    return t.detach().cpu().double().numpy().reshape(-1)


def make(n, w="f32", g="f32", master=False, bits=32, seed=0, used=True):
    """(weight, state, master, gradient) of n elements; ``used``: a state with a past."""
    r = torch.Generator().manual_seed(seed * 7919 + n)
    full = torch.randn(n, generator=r)
    grad = (torch.randn(n, generator=r) * 10 ** torch.empty(n).uniform_(-3, 0, generator=r)).to(TYPES[g]).cuda()
    state = mb.new_adamw_state(full.cuda(), bits)
    if used and n:
        m, v = 0.1 * torch.randn(n, generator=r), torch.randn(n, generator=r).square() * 0.01
        if bits == 32:
            state.m.copy_(m), state.v.copy_(v)
        else:
            for t, s, x in ((state.m, state.m_scale, m), (state.v, state.v_scale, v.sqrt())):
                q, scale, _ = ref.to_codes(x.double().numpy())
                t.copy_(torch.from_numpy(q).float().cuda().to(torch.float8_e4m3fn))
                s.copy_(torch.from_numpy(scale).float())
    return full.to(TYPES[w]).cuda(), state, full.cuda() if master else None, grad


def moments(state):
    if state.m_scale is None:
        return f64(state.m), f64(state.v)
    return (ref.from_codes(f64(state.m.float()), f64(state.m_scale)),
            ref.from_codes(f64(state.v.float()), f64(state.v_scale)) ** 2)


def before(w, state, master, grad):
    return f64(w if master is None else master), f64(grad), *moments(state)


def check(old, w, state, master, step, factor=1.0, lr=1e-2, betas=(0.9, 0.95), eps=1e-8, decay=0.0):
    w0, g, m0, v0 = old
    w1, m1, v1, ew, em, ev = ref.adamw(w0, g * factor, m0, v0, step, lr, *betas, eps, decay)
    if factor != 1.0:  # one product more in every term of g
        em, ev, ew = em + U * np.abs(g), ev + 2 * U * v1, 1.5 * ew
    if state.m_scale is not None:  # code times scale, and its square
        em, ev, ew = em + U * np.abs(m0), ev + 3 * U * v0, 1.5 * ew
    if master is not None:
        assert (np.abs(f64(master) - w1) <= ew).all()
        assert torch.equal(w, master.to(w.dtype))
    else:
        half = 2.0 ** -8 * np.abs(w1) if w.dtype is torch.bfloat16 else 0.0  # one rounding
        assert (np.abs(f64(w) - w1) <= ew * 1.01 + half * 1.01).all()
    if state.m_scale is None:
        assert (np.abs(f64(state.m) - m1) <= em).all() and (np.abs(f64(state.v) - v1) <= ev).all()
        return
    for codes, scale, x, err in ((state.m, state.m_scale, m1, em), (state.v, state.v_scale, np.sqrt(v1), None)):
        # sqrt(v): half of v's relative error, and its own rounding
        err = err if err is not None else (4 + 3) * U * x
        q, s, gap = ref.to_codes(x)
        assert (np.abs(f64(scale) - s) <= 4 * U * s + np.repeat(1, len(s)) * err.max()).all()
        got = f64(codes.float())
        if codes is state.v:
            q = np.where((x > 0) & (q == 0), 2.0 ** -9, q)
        # the exact code, unless the value is as near to a tie as FP32 can tell
        with np.errstate(invalid="ignore", divide="ignore"):
            near = err / np.abs(x) + np.repeat([err[b * 256: b * 256 + 256].max() for b in range(len(s))], 256)[: len(x)] \
                / np.repeat(np.maximum(s, 1e-300) * 448, 256)[: len(x)] + 8 * U
        off = got != q
        assert (gap[off] <= near[off]).all()
        assert off.mean() <= 0.01 or off.sum() <= 1
        assert (np.abs(got[off] - q[off]) <= np.maximum(np.abs(q[off]) / 7, 2.0 ** -9)).all()  # the next code


SIZES = [1, 2, 3, 4, 5, 7, 8, 9, 31, 255, 256, 257, 511, 1000, 2049, 4095, 4096, 4097, 12345, 70001]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("w,master", [("f32", False), ("bf16", False), ("bf16", True), ("f32", True)])
@pytest.mark.parametrize("g", ["f32", "bf16"])
def test_every_type_and_size(bits, w, master, g):
    tensors = [make(n, w, g, master, bits) for n in SIZES]
    old = [before(*t) for t in tensors]
    plan = mb.AdamWPlan([t[0] for t in tensors], [t[1] for t in tensors], masters=[t[2] for t in tensors],
                        weight_decay=0.1, grads=[t[3] for t in tensors])
    mb.moe_adamw_step(plan, 7, **HOW)
    for o, t in zip(old, tensors):
        check(o, *t[:3], 7, decay=0.1)


@pytest.mark.parametrize("bits", [32, 8])
def test_the_first_steps_from_zero(bits):
    w, s, master, g = make(3000, "bf16", "f32", True, bits, used=False)
    plan = mb.AdamWPlan([w], [s], masters=[master], grads=[g])
    for step in range(1, 6):
        old = before(w, s, master, g)
        mb.moe_adamw_step(plan, step, **HOW)
        check(old, w, s, master, step)
        g.mul_(-0.7)


def test_many_tensors_of_every_kind():
    """More than one launch takes, empty ones among them, each with its own rates."""
    r = np.random.default_rng(0)
    tensors, decay, factor = [], [], []
    for i in range(700):
        n = 0 if i % 97 == 5 else int(r.integers(1, 900))
        w = ("f32", "bf16")[i % 2]
        tensors.append(make(n, w, ("f32", "bf16")[i // 2 % 2], i % 3 == 0, (32, 8)[i // 4 % 2], i))
        decay.append(0.1 * (i % 4)), factor.append(0.5 + i % 3)
    old = [before(*t) for t in tensors]
    plan = mb.AdamWPlan([t[0] for t in tensors], [t[1] for t in tensors], masters=[t[2] for t in tensors],
                        weight_decay=decay, lr_factor=factor, grads=[t[3] for t in tensors])
    mb.moe_adamw_step(plan, 3, **HOW)
    for o, t, d, f in zip(old, tensors, decay, factor):
        if t[0].numel():
            check(o, *t[:3], 3, decay=d, lr=1e-2 * f)


@pytest.mark.parametrize("bits", [32, 8])
def test_nothing_beside_a_tensor_is_written(bits):
    """Views into larger buffers: 16-byte aligned starts, odd ends."""
    n, at = 1003, 256
    kinds = dict(w=torch.float32, master=torch.float32, m=torch.float32 if bits == 32 else torch.uint8,
                 v=torch.float32 if bits == 32 else torch.uint8, m_scale=torch.float32, v_scale=torch.float32)
    buffers = {x: torch.full((2048,), 3, dtype=t, device="cuda") for x, t in kinds.items()}
    view = {x: b[at: at + (4 if "scale" in x else n)] for x, b in buffers.items()}
    if bits == 8:
        view["m"], view["v"] = (view[x].view(torch.float8_e4m3fn) for x in "mv")
    state = mb.AdamWState(view["m"], view["v"], *((view["m_scale"], view["v_scale"]) if bits == 8 else ()))
    plan = mb.AdamWPlan([view["w"]], [state], masters=[view["master"]], grads=[torch.ones(n, device="cuda")])
    mb.moe_adamw_step(plan, 1, **HOW)
    for x, b in buffers.items():
        end = at + (4 if "scale" in x else n)
        assert (b[:at] == 3).all() and (b[end:] == 3).all(), x
        if bits == 8 or "scale" not in x:
            assert (b[at:end] != 3).any(), x


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_gradients_decay_the_moments(bits):
    """With 8 bits through the scale alone: the codes stay."""
    w, s, _, g = make(1024, bits=bits)
    g.zero_()
    codes, m0, v0 = s.m.clone(), *moments(s)
    plan = mb.AdamWPlan([w], [s], grads=[g])
    for step in range(1, 21):
        mb.moe_adamw_step(plan, step, lr=0.0, betas=(0.9, 0.95))
    m, v = moments(s)
    # twenty roundings of the scale, and of sqrt(v)'s
    assert (np.abs(m - m0 * 0.9 ** 20) <= 100 * U * np.abs(m0)).all()
    assert (np.abs(v - v0 * 0.95 ** 20) <= 200 * U * v0).all()
    if bits == 8:
        assert torch.equal(s.m.view(torch.uint8), codes.view(torch.uint8))


def test_small_second_moments_keep_a_code():
    """Next to a large one: sqrt(v) is never rounded to zero, m may be."""
    g = torch.full((512,), 1e-7, device="cuda")
    g[3] = 100.0
    w = torch.zeros(512, device="cuda")
    s = mb.new_adamw_state(w, 8)
    mb.moe_adamw_step(mb.AdamWPlan([w], [s], grads=[g]), 1, **HOW)
    v = s.v.float()[:256]
    assert (v > 0).all() and v[3] == 448 and (v == 2.0 ** -9).sum() == 255
    assert (s.v.float()[256:] == 448).all() and torch.isfinite(w).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_zeros_and_extremes(bits):
    """Gradients of zeros, of the smallest and of large numbers."""
    for value in (0.0, 1e-45, 1e-38, 1e-25, 1e15):
        w = torch.ones(600, device="cuda")
        s = mb.new_adamw_state(w, bits)
        g = torch.full((600,), value, device="cuda")
        plan = mb.AdamWPlan([w], [s], grads=[g])
        for step in (1, 2):
            mb.moe_adamw_step(plan, step, **HOW)
        assert all(torch.isfinite(t.float()).all() for t in (w, s.m, s.v)), value
        if value >= 1e15:  # the full step each time; eps does not count
            assert torch.allclose(w, torch.full_like(w, 0.98), rtol=1e-5)
        if value <= 1e-25:
            assert torch.allclose(w, torch.ones_like(w), rtol=1e-5)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_nan_stays_with_its_element_an_infinity_with_its_block(bits):
    w, s, _, g = make(1000, bits=bits)
    g[7], g[300] = NAN, INF
    plan = mb.AdamWPlan([w], [s], grads=[g])
    mb.moe_adamw_step(plan, 2, **HOW)
    bad = torch.isnan(w)
    assert bad[7] and bad[300] and bad.sum() == 2
    m, v = moments(s)
    others = np.ones(1000, bool)
    others[7] = False
    others[256:512 if bits == 8 else 301] = False
    if bits == 32:
        others[256:300] = True
    assert np.isnan(m[7]) and np.isnan(v[7]) and np.isfinite(m[others]).all() and np.isfinite(v[others]).all()
    assert not np.isfinite(m[300])


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("factor", [1.0, 0.25, NAN, INF, -INF])
@pytest.mark.parametrize("on_device", [False, True])
def test_the_factor_and_a_step_that_is_left_out(bits, factor, on_device):
    w, s, master, g = make(5000, "bf16", "f32", True, bits)
    old = before(w, s, master, g)
    kept = [t.clone() for t in (w, master)] + [t.clone().view(torch.uint8) for t in s if t is not None]
    plan = mb.AdamWPlan([w], [s], masters=[master], grads=[g])
    scale = torch.tensor([factor], device="cuda")
    step, how = (torch.tensor([3], dtype=torch.int32, device="cuda"), dict(HOW, lr=torch.tensor([1e-2], device="cuda"))) \
        if on_device else (4, HOW)
    mb.moe_adamw_step(plan, step, grad_scale=scale, **how)
    if math.isfinite(factor):
        check(old, w, s, master, 4, factor, lr=float(np.float32(1e-2)) if on_device else 1e-2)
    else:
        for a, b in zip([w, master] + [t.view(torch.uint8) for t in s if t is not None], kept):
            assert torch.equal(a, b)
    if on_device:
        assert step.item() == (4 if math.isfinite(factor) else 3)


def test_host_and_device_numbers_give_the_same_bits():
    runs = []
    for on_device in (False, True):
        w, s, master, g = make(3000, "bf16", "bf16", True, 8)
        plan = mb.AdamWPlan([w], [s], masters=[master], weight_decay=0.1, grads=[g])
        step, lr = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([0.25], device="cuda")
        for i in range(1, 4):
            mb.moe_adamw_step(plan, step if on_device else i, lr=lr if on_device else 0.25)
        runs.append([master, *(t.view(torch.uint8) for t in s)])
    assert all(torch.equal(a, b) for a, b in zip(*runs))


# ------------------------------------------------------------------ norm
@pytest.mark.parametrize("sizes", [[1], [3], [0, 5, 0], [4096], [16383, 16384, 16385], [1] * 17, [100] * 600,
                                   [1 << 21, 7, 12345, 999999], list(range(40))])
@pytest.mark.parametrize("kind", ["f32", "bf16", "both"])
def test_norm(sizes, kind):
    r = torch.Generator().manual_seed(len(sizes))
    grads = [torch.randn(n, generator=r).to(TYPES[kind if kind != "both" else ("f32", "bf16")[i % 2]]).cuda()
             for i, n in enumerate(sizes)]
    want, _ = ref.norm([f64(g) for g in grads], 1.0)
    # a thread's four sums take the squares of its share one after another;
    # the root halves the relative error, and is rounded
    share = max(1, sum(sizes) / (152 * 256 * 4))
    for limit in (0.5 * want if want else 1.0, 2.0 * want if want else 2.0, INF):
        got = f64(mb.moe_grad_norm(grads, max_norm=limit))
        assert abs(got[0] - want) <= (16 + share) * U * want
        factor = float(np.float32(limit)) / want if want > limit else 1.0
        assert abs(got[1] - factor) <= (18 + share) * U * factor


def test_norm_of_nothing():
    for grads in ([], [torch.empty(0, device="cuda")]):
        assert f64(mb.moe_grad_norm(grads, max_norm=1.0)).tolist() == [0.0, 1.0]
    assert f64(mb.moe_grad_norm([torch.zeros(100, device="cuda")], max_norm=1.0)).tolist() == [0.0, 1.0]


@pytest.mark.parametrize("value", [1e-18, 1e-10, 1e18, 1e20, 1e30, 1e36])
def test_norm_over_the_range(value):
    g = [torch.full((n,), value, device="cuda") for n in (3, 5000, 100)]
    want = float(np.float32(value)) * math.sqrt(5103)
    got = f64(mb.moe_grad_norm(g, max_norm=value))
    assert abs(got[0] - want) <= 40 * U * want
    assert abs(got[1] - 1 / math.sqrt(5103)) <= 40 * U


@pytest.mark.parametrize("value", [NAN, INF, -INF, 3e38])
def test_a_norm_that_is_no_number_leaves_the_step_out(value):
    w, s, _, g = make(2000)
    g[5] = g[6] = g[7] = g[1999] = value
    kept = w.clone()
    plan = mb.AdamWPlan([w], [s], grads=[g])
    clip = mb.moe_grad_norm(plan, max_norm=1.0)
    assert torch.isnan(clip[1]) and not torch.isfinite(clip[0])
    mb.moe_adamw_step(plan, 1, grad_scale=clip[1:], **HOW)
    assert torch.equal(w, kept)


def test_norm_repeats_in_old_workspaces():
    g = [torch.randn(n, device="cuda") for n in (100000, 3, 77777)]
    want, ws = mb.moe_grad_norm(g), mb.new_grad_norm_workspace(3)
    for fill in (0, 255, 99):
        ws.fill_(fill)
        assert torch.equal(mb.moe_grad_norm(mb.GradList(g), workspace=ws), want)


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("bits", [32, 8])
def test_a_captured_update_counts_on(bits):
    """Norm, factor and step in one graph, against the same calls one by one."""
    def fresh():
        ts = [make(n, w, "f32", w == "bf16", b, n) for n, w, b in ((500, "f32", 32), (9001, "bf16", bits), (257, "f32", bits))]
        plan = mb.AdamWPlan([t[0] for t in ts], [t[1] for t in ts], masters=[t[2] for t in ts], weight_decay=0.1,
                            grads=[t[3] for t in ts])
        return plan, torch.tensor([4], dtype=torch.int32, device="cuda"), torch.tensor([1e-2], device="cuda")

    def once(plan, step, lr):
        clip = mb.moe_grad_norm(plan, max_norm=1.0)
        mb.moe_adamw_step(plan, step, lr=lr, grad_scale=clip[1:])
        return clip
    a, b = fresh(), fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = once(*a)
    for i in range(3):
        graph.replay()
        clip = once(*b)
        assert torch.equal(captured.view(torch.int32), clip.view(torch.int32))
        for x, y in zip(a[0].weights + [s.m.view(torch.uint8) for s in a[0].states],
                        b[0].weights + [s.m.view(torch.uint8) for s in b[0].states]):
            assert torch.equal(x, y)
        for plan, _, lr in (a, b):
            lr.mul_(0.5)
            for k, g in enumerate(plan.grads):
                g.mul_(-0.9 + 0.1 * k)
        if i == 1:
            for plan, _, _ in (a, b):
                plan.grads[0][0] = NAN  # the next one is left out
    assert a[1].item() == b[1].item() == 6


def test_streams():
    tensors = [make(40000, "bf16", "f32", True, 8, i) for i in range(4)]
    old = [before(*t) for t in tensors]
    plans = [mb.AdamWPlan([w], [s], masters=[m], grads=[g]) for w, s, m, g in tensors]
    side = [torch.cuda.Stream() for _ in plans]
    torch.cuda.synchronize()
    steps = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in plans]
    torch.cuda.synchronize()
    for plan, s, step in zip(plans, side, steps):
        clip = mb.moe_grad_norm(plan, stream=s)
        mb.moe_adamw_step(plan, step, grad_scale=clip[1:], stream=s, **HOW)
    torch.cuda.synchronize()
    for o, t in zip(old, tensors):
        check(o, *t[:3], 1)


def test_new_gradients_take_the_old_ones_place():
    w, s, master, g = make(1000)
    plan = mb.AdamWPlan([w], [s], grads=[g])
    first = mb.moe_grad_norm(plan)
    plan.set_grads([(2 * g).bfloat16()])
    assert abs((mb.moe_grad_norm(plan)[0] / first[0]).item() - 2) < 1e-2
    old = before(w, s, master, plan.grads[0])
    mb.moe_adamw_step(plan, 1, **HOW)
    check(old, w, s, master, 1)


def test_refusals_on_the_device():
    w = torch.zeros(64, device="cuda")
    s = mb.new_adamw_state(w)
    plan = mb.AdamWPlan([w], [s], grads=[torch.zeros(64, device="cuda")])
    for bad in (dict(step=torch.zeros(1, device="cuda")), dict(step=torch.zeros(1).int()),
                dict(lr=torch.zeros(2, device="cuda")), dict(grad_scale=torch.zeros(1, device="cuda").double()),
                dict(grad_scale=torch.zeros((), device="cuda"))):
        with pytest.raises(ValueError):
            mb.moe_adamw_step(plan, **{**dict(step=1), **bad})
    for bad in (dict(step=0), dict(lr=-1.0), dict(betas=(1.0, 0.9)), dict(eps=-1.0), dict(lr=NAN)):
        with pytest.raises(mb.MoeFfnError):
            mb.moe_adamw_step(plan, **{**dict(step=1), **bad})
    with pytest.raises(mb.MoeFfnError):
        mb.moe_grad_norm(plan, max_norm=0.0)
    big = torch.zeros(100, device="cuda")
    with pytest.raises(mb.MoeFfnError):  # an address that is no multiple of 16
        mb.moe_grad_norm([big[1:]])
    with pytest.raises(mb.MoeFfnError):
        mb.moe_adamw_step(mb.AdamWPlan([big[1:]], [mb.new_adamw_state(big[1:])], grads=[torch.zeros_like(big[1:])]), 1)
    with pytest.raises(ValueError):
        mb.AdamWPlan([big[::2]], [mb.new_adamw_state(big[::2])])


def test_more_than_32_bits_of_elements():
    """The last elements of a tensor of 2^31 + 1000, 8-bit states, and its norm."""
    n = (1 << 31) + 1000
    w = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    s = mb.new_adamw_state(w, 8)
    g[-1], g[-257], g[5] = 3.0, -4.0, 12.0
    plan = mb.AdamWPlan([w], [s], grads=[g])
    assert f64(mb.moe_grad_norm(plan, max_norm=INF))[0] == 13.0
    mb.moe_adamw_step(plan, 1, lr=0.5, betas=(0.5, 0.5))
    assert w[-1] == -0.5 and w[-257] == 0.5 and w[5] == -0.5
    assert int((w != 0).sum()) == 3 and int((s.m.view(torch.uint8) != 0).sum()) == 3
    assert s.m_scale[-1].item() * 448 == pytest.approx(1.5, rel=1e-6)


@pytest.mark.parametrize("g", ["f32", "bf16"])
@pytest.mark.parametrize("factor", [None, 0.37])
def test_codes_are_those_of_the_formula_in_fp32(g, factor):
    """Operation by operation in torch, each rounded once; the quotient by the
    scale is the rounded one (torch's division)."""
    n = 1 << 22
    w, s, _, grad = make(n, "f32", g, False, 8)
    top = 1.0 / 448.0

    def quantised(x, up):
        blocks = x.view(-1, 256)
        scale = (blocks.abs().amax(1) * torch.tensor(top, device="cuda")).clamp_min(2.0 ** -126)
        q = blocks / scale[:, None]
        if up:
            q = torch.where(blocks > 0, q.clamp_min(2.0 ** -9), q)
        return q.clamp(-448, 448).to(torch.float8_e4m3fn).view(-1).view(torch.uint8), scale
    gf = grad.float() if factor is None else grad.float() * torch.tensor(factor, device="cuda")
    m = s.m.float() * s.m_scale.repeat_interleave(256)
    v = (s.v.float() * s.v_scale.repeat_interleave(256)).square()
    b1, a1, b2, a2 = (torch.tensor(x, dtype=torch.float32, device="cuda") for x in (0.9, 1 - 0.9, 0.95, 1 - 0.95))
    want = [*quantised(b1 * m + a1 * gf, False), *quantised((b2 * v + (a2 * gf) * gf).sqrt(), True)]
    plan = mb.AdamWPlan([w], [s], grads=[grad])
    mb.moe_adamw_step(plan, 9, grad_scale=None if factor is None else torch.tensor([factor], device="cuda"), **HOW)
    got = [s.m.view(torch.uint8), s.m_scale, s.v.view(torch.uint8), s.v_scale]
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_small_decay_is_not_rounded_away(bits):
    """lr * weight_decay of 2e-6 over 50 steps with gradients of zero: what is
    lost is w's own rounding, at random (half a unit a step at most, its sum's
    spread sqrt(50) of it), and not the factor's."""
    n = 1 << 16
    w = (1 + torch.rand(n, generator=torch.Generator().manual_seed(1))).cuda()
    w0 = w.double()
    plan = mb.AdamWPlan([w], [mb.new_adamw_state(w, bits)], weight_decay=0.1, grads=[torch.zeros(n, device="cuda")])
    for step in range(1, 51):
        mb.moe_adamw_step(plan, step, lr=2e-5)
    lost = ((w.double() / w0 - (1 - 2e-6) ** 50) / 1e-4)
    # the mean over 2^16 elements; a step rounds off at most 2^-24 of w, 3% of the decay, both ways
    assert abs(lost.mean().item()) <= 3e-3
