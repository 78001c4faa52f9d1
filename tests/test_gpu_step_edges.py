"""Edges of the training step's operators on the device, against 64 bits."""
import numpy as np
import pytest
import torch

from mixture_experts_ffn_gate_gb300 import block as b
from mixture_experts_ffn_gate_gb300 import moe_block as mb
from tests import step_ref as ref
from tests.block_ref import U

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ the loss
@pytest.mark.parametrize("low,high", [(-3, 3), (8, 12), (10, 25), (-5, 40), (-30, -10)])
@pytest.mark.parametrize("T,E", [(20, 16), (300, 64), (70, 257), (33, 1000)])
@pytest.mark.parametrize("z_coef", [0.0, 1e-9])
def test_sigmoid_gradient_of_saturated_logits(low, high, T, E, z_coef):
    """1 - q is a factor of the gradient however small it is.  The bound: s and
    1 - q are off by a row's relative error each, and so are a (a rounded
    product) and the mean of a under s."""
    r = np.random.default_rng(E + low + 100)
    logits = r.uniform(low, high, size=(T, E)).astype(np.float32)
    counts = r.integers(0, T, size=(1, E)).astype(np.int32)
    got = mb.moe_balance_loss_backward(torch.from_numpy(logits).cuda(), torch.from_numpy(counts).cuda(), 4,
                                       score="sigmoid", coef=1.0, z_coef=z_coef).cpu().double().numpy()
    l = logits.astype(np.float64)
    q, rest = 1 / (1 + np.exp(-l)), 1 / (1 + np.exp(l))
    s, a = q / q.sum(1, keepdims=True), E * counts / (4.0 * T * T)
    mean = (a * s).sum(1, keepdims=True)
    want = s * rest * (a - mean)
    rel = np.array([ref.row_error(row, E) for row in logits])[:, None]
    bound = 2 * rel * s * rest * (a + mean) + 4 * U * np.abs(want)
    if z_coef:
        e = np.exp(l - l.max(1, keepdims=True))
        lse = l.max(1) + np.log(e.sum(1))
        z = 2 * z_coef / T * lse[:, None] * e / e.sum(1, keepdims=True)
        # the softmax's and the logarithm's error, and the sum's rounding
        bound += 2 * rel * np.abs(z) + 2 * z_coef / T * rel * e / e.sum(1, keepdims=True) + 4 * U * np.abs(z + want)
        want = want + z
    assert (np.abs(got - want) <= bound).all()


@pytest.mark.parametrize("value,q", [(30.0, 1.0), (1e30, 1.0), (float("inf"), 1.0), (0.0, 0.5), (-0.0, 0.5), (-200.0, 0.0),
                                     (float("-inf"), 0.0)])
def test_sigmoid_gradient_next_to_extreme_logits(value, q):
    """Their own gradient is zero where q (1 - q) is, and they count in the others' sum as q."""
    logits = torch.tensor([[value, 0.5, -1.0, value]])
    counts = torch.tensor([[3, 1, 0, 0]], dtype=torch.int32)
    got = mb.moe_balance_loss_backward(logits.cuda(), counts.cuda(), 2, score="sigmoid", coef=1.0).cpu().double()[0]
    x = torch.sigmoid(torch.tensor([0.5, -1.0], dtype=torch.float64))
    p = torch.tensor([q, x[0], x[1], q], dtype=torch.float64)
    rest = torch.tensor([1 / (1 + np.exp(value)) if value < 700 else 0.0, 1 - x[0], 1 - x[1], 0.0], dtype=torch.float64)
    rest[3] = rest[0]
    a = 4 * counts[0].double() / 2.0
    s = p / p.sum()
    want = s * rest * (a - (a * s).sum())
    assert (got - want).abs().max().item() <= 200 * U * a.sum().item()
    assert ((got - want).abs() <= 200 * U * s * rest * (a + (a * s).sum()) + 1e-37).all()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [24, 200])
def test_probabilities_of_far_logits(kind, E):
    """Their error does not grow with the logits.  2^y is off by two units in the
    last place (4 U), c's product and 1 + x by U, a reciprocal by 2 U: 8 U, and
    |l| / 20 U for ln 2's rounding; the sum over the row 13 additions, its
    reciprocal 2 U, the product and the mean of one row 2 U: 33 U.  The largest
    softmax logit is 0, so the differences are exact."""
    r = np.random.default_rng(E)
    T = 300
    logits = r.uniform(-85, 0 if kind == "softmax" else 85, size=(T, E)).astype(np.float32)
    logits[:, 0] = 0.0
    idx = np.zeros((T, 1), np.int32)
    got = mb.moe_balance_loss_forward(torch.from_numpy(logits).cuda(), torch.from_numpy(idx).cuda(), score=kind,
                                      seq_offsets=torch.arange(T + 1, dtype=torch.int32, device="cuda"))
    l = logits.astype(np.float64)
    q = np.exp(l) if kind == "softmax" else 1 / (1 + np.exp(-l))
    s = q / q.sum(1, keepdims=True)
    bound = (34 + np.abs(l) / 20) * U * s
    assert (np.abs(got.prob.cpu().double().numpy() - s) <= bound).all()
    # the gradient: s again, a's products 6 U, the mean under s 50 U of its own
    counts = r.integers(0, T, size=(1, E)).astype(np.int32)
    d = mb.moe_balance_loss_backward(torch.from_numpy(logits).cuda(), torch.from_numpy(counts).cuda(), 1, score=kind,
                                     coef=float(T)).cpu().double().numpy()
    a = E * counts / float(T)
    mean = (a * s).sum(1, keepdims=True)
    rest = 1.0 if kind == "softmax" else 1 / (1 + np.exp(l))
    want = s * rest * (a - mean)
    assert (np.abs(d - want) <= (96 + np.abs(l) / 10) * U * s * rest * (a + mean) + 2.0 ** -126).all()


@pytest.mark.parametrize("T", [20, 400])
def test_rows_of_sigmoids_below_the_normal_numbers(T):
    """Each counts as zero, so a row of nothing else has no probability and no
    gradient of the balance, but the z of its finite logits."""
    r = np.random.default_rng(T)
    logits = r.normal(size=(T, 40)).astype(np.float32)
    logits[3], logits[5], logits[7] = -88.0, -88.0, -float("inf")
    logits[5, 11] = 0.0
    idx = np.argsort(-logits, axis=1, kind="stable")[:, :4].astype(np.int32)
    how = dict(score="sigmoid", coef=0.5, z_coef=0.25)
    got = mb.moe_balance_loss_forward(torch.from_numpy(logits).cuda(), torch.from_numpy(idx).cuda(), **how)
    l = logits.astype(np.float64)
    q = np.where(l < -87.5, 0.0, 1 / (1 + np.exp(-l.clip(-500))))
    total = q.sum(1, keepdims=True)
    s = np.divide(q, total, out=np.zeros_like(q), where=total > 0)
    prob = s.mean(0)
    rel = (ref.row_error(logits[0], 40) + (T / 8 + 100) * U)
    assert (np.abs(got.prob.cpu().double().numpy()[0] - prob) <= rel * prob).all()
    top = l.max(1, keepdims=True, initial=-1e300)
    e = np.where(np.isfinite(l), np.exp(l - top), 0.0)
    lse = np.where(np.isfinite(top[:, 0]) & (e.sum(1) > 0), top[:, 0] + np.log(np.maximum(e.sum(1), 1e-300)), 0.0)
    assert lse[7] == 0 and abs(lse[3] + 88 - np.log(40)) < 1e-9
    z = (lse ** 2).mean()
    # a logarithm's error, twice over in the square, of lse up to 88
    assert abs(got.loss[2].item() - z) <= (2 * 88 * (rel + 4 * U * 88) + rel * 88 * 88) * 2 / T + rel * z
    counts = np.bincount(idx.ravel(), minlength=40)[None]
    assert np.array_equal(got.counts.cpu().numpy(), counts)
    d = mb.moe_balance_loss_backward(torch.from_numpy(logits).cuda(), got.counts, 4, **how).cpu().double().numpy()
    want = 2 * 0.25 / T * lse[:, None] * np.divide(e, e.sum(1, keepdims=True), out=np.zeros_like(e),
                                                   where=e.sum(1, keepdims=True) > 0)
    assert (d[7] == 0).all()
    assert (np.abs(d[3] - want[3]) <= 2 * (ref.row_error(logits[3], 40) + 4 * U) * np.abs(want[3])).all()
    assert np.isfinite(d).all() and (np.abs(d[5, 12:] - want[5, 12:]) <= 1e-30).all()


def loss_in_64_bits(logits, idx, offsets, kind, coef, z_coef):
    """(loss [3], prob [S,E]) of ascending offsets from 0 to T, on the device."""
    T, E = logits.shape
    S, k = len(offsets) - 1, idx.shape[1]
    l = logits.double()
    q = torch.softmax(l, 1) if kind == "softmax" else torch.sigmoid(l)
    s = q / q.sum(1, keepdim=True)
    n = (offsets[1:] - offsets[:-1]).long()
    seq = torch.repeat_interleave(torch.arange(S, device=l.device), n)
    prob = torch.zeros(S, E, dtype=torch.float64, device=l.device).index_add_(0, seq, s) / n.clamp_min(1)[:, None]
    chosen = torch.zeros(S, E, dtype=torch.float64, device=l.device)
    chosen.index_put_((seq[:, None].expand_as(idx), idx.long()), torch.ones_like(idx, dtype=torch.float64), accumulate=True)
    bal = E * (chosen * prob).sum() / (k * T)
    z = torch.logsumexp(l, 1).square().sum() / T
    return torch.stack((coef * bal + z_coef * z, bal, z)), prob


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,S,even", [(6000, 256, 4096, False), (9000, 1000, 3000, False), (1 << 18, 96, 1 << 18, True),
                                        (1 << 20, 32, 1 << 20, True), (50000, 8, 100000, False), (40000, 40, 305, False)])
def test_losses_of_many_sequences(kind, T, E, S, even):
    """Within a bound that does not grow with them: a row's error; for a
    sequence's probabilities its rows (below 2000, of which a lane adds up one in
    16 at most), a block's warps and the slots; the experts of a tile and one
    rounding in a block's part; at most 30 parts in each of a lane's four sums, and
    twelve sums of those.  ``even``:
    every sequence is the same row, so that no rounding cancels another."""
    g = torch.Generator(device="cuda").manual_seed(S)
    if even:
        logits = torch.randn(1, E, generator=g, device="cuda").expand(T, E).contiguous()
        off = torch.arange(T + 1, dtype=torch.int32, device="cuda")
        idx = torch.arange(3, dtype=torch.int32, device="cuda").expand(T, 3).contiguous()
    else:
        logits = torch.randn(T, E, generator=g, device="cuda")
        cuts = torch.randint(0, T + 1, (S - 1,), generator=g, device="cuda").sort().values
        off = torch.cat((cuts.new_zeros(1), cuts, cuts.new_full((1,), T))).int()
        idx = torch.topk(logits, 3, dim=1).indices.int()
        assert (off[1:] - off[:-1]).max() < 2000
    r = mb.moe_balance_loss_forward(logits, idx, score=kind, coef=0.5, z_coef=0.25, seq_offsets=off)
    want, prob = loss_in_64_bits(logits, idx, off, kind, 0.5, 0.25)
    row = logits[: 1 if even else T].double()
    rel = (48 + E / 32 + 2 * (2 * row.abs().max().item() + row.abs().max().item())) * U
    assert ((r.prob.double() - prob).abs() <= (rel + 300 * U) * prob).all()
    got = r.loss.double()
    assert abs(got[1] - want[1]) <= (rel + 400 * U) * want[1]
    # a logarithm is off by its sum's relative error and its own rounding
    lse = torch.logsumexp(row, 1)
    z = (2 * lse.abs() * (rel + 4 * U * lse.abs())).max().item() + 400 * U * lse.square().max().item()
    assert abs(got[2] - want[2]) <= z
    assert abs(got[0] - want[0]) <= 0.5 * (rel + 400 * U) * want[1] + 0.25 * z + 4 * U * want[0]


# ------------------------------------------------------------------ 8-bit states
def moment(codes, scale):
    return codes.float().double() * scale.double().repeat_interleave(256)[: codes.numel()].view(codes.shape)


def follow(betas, phases, rounding=None, blocks=40):
    """sqrt(v) and m of 8-bit states over those of 32-bit ones after each of
    the phases (steps, factors of the gradients), every second element apart."""
    n = blocks * 256
    w8, w32 = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    s8, s32, g = mb.new_adamw_state(w8, 8), mb.new_adamw_state(w32, 32), torch.empty(n, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(3)
    plans = [mb.AdamWPlan([w], [s], grads=[g]) for w, s in ((w8, s8), (w32, s32))]
    t, out = 0, []
    how = {} if rounding is None else dict(rounding=rounding)
    for steps, even, odd in phases:
        factor = torch.tensor([even, odd], device="cuda").repeat(n // 2)
        for _ in range(steps):
            t += 1
            g.copy_(torch.randn(n, generator=gen, device="cuda") * factor)
            for plan in plans:
                mb.moe_adamw_step(plan, t, lr=1e-3, betas=betas, **how)
        r = (moment(s8.v, s8.v_scale) / s32.v.double().sqrt()).cpu().numpy()
        d = (moment(s8.m, s8.m_scale) - s32.m.double()).cpu().numpy()
        out.append([(r[i::2], d[i::2] / np.sqrt(np.mean(s32.m.cpu().numpy()[i::2] ** 2.0))) for i in (0, 1)])
    return out


@pytest.mark.parametrize("betas,steps", [((0.9, 0.95), 300), ((0.9, 0.99), 1500), ((0.9, 0.999), 6000),
                                         ((0.99, 0.999), 6000)])
def test_8_bit_second_moments_follow_their_gradients(betas, steps):
    """As 32-bit ones do: steady gradients, then half of the elements' fall
    fourfold, then the others' rise fourfold (six time constants of v each, after
    which 1/400 of the old v is left: a tenth of the new one's, 5% of its root).
    A code moves by its spacing (9% of the value on average) with a chance of
    what sqrt(v) changes over it, (1 - beta2) / 2 times about 1 for Gaussian
    gradients, and is drawn back by 1 - beta2 of its distance: a variance of
    0.09 / 4 of the square, 15% rms, 17% with the last step's rounding and the
    old v.  Rounded to nearest, up to a beta2 of 0.95, it is off by half a
    spacing more where gradients fell: 15% at the median, 25% rms."""
    nearest = betas[1] <= 0.95
    for phase, both in enumerate(follow(betas, [(steps, 1.0, 1.0), (steps, 0.25, 1.0), (steps, 0.25, 4.0)])):
        for r, _ in both:
            assert abs(np.median(r) - 1) <= (0.2 if nearest else 0.07), (phase, np.median(r))
            assert np.sqrt(np.mean((r - 1) ** 2)) <= (0.35 if nearest else 0.25), phase


def test_8_bit_first_moments_follow_at_betas_close_to_one():
    """Unbiased: m's error over m's size averages to nothing (10240 elements of
    30% rms: 0.3%), and is a fraction of it."""
    for both in follow((0.99, 0.999), [(1500, 1.0, 1.0), (1500, 0.1, 1.0)]):
        for _, d in both:
            assert abs(d.mean()) <= 0.03 and np.sqrt(np.mean(d ** 2)) <= 0.6


def test_gradients_of_zero_beside_others_let_the_second_moment_decay():
    """sqrt(v) of elements without gradients, in blocks whose scale stays: after
    three time constants its mean is exp(-1.5) of what it was (10240 elements of
    40% rms at most: 0.4%; the sum of their roundings is unbiased)."""
    n = 80 * 256
    w, g = torch.zeros(n, device="cuda"), torch.ones(n, device="cuda")
    s = mb.new_adamw_state(w, 8)
    plan = mb.AdamWPlan([w], [s], grads=[g])
    mb.moe_adamw_step(plan, 1, betas=(0.9, 0.0))   # v = 1
    before = moment(s.v, s.v_scale)[::2].mean().item()
    g[::2] = 0.0
    for t in range(2, 302):
        mb.moe_adamw_step(plan, t, betas=(0.9, 0.99))
    r = moment(s.v, s.v_scale)[::2].mean().item() / before
    assert abs(r / 0.99 ** 150 - 1) <= 0.03


def codes_in_fp32(w, s, g, b1, b2):
    """The quotients that a step's codes are the rounding of, operation by
    operation in FP32, for m and sqrt(v)."""
    b1, a1, b2, a2, top = (torch.tensor(x, dtype=torch.float32, device="cuda") for x in (b1, 1 - b1, b2, 1 - b2, 1 / 448))
    m = s.m.float() * s.m_scale.repeat_interleave(256)
    v = (s.v.float() * s.v_scale.repeat_interleave(256)).square()
    out = []
    for x in (b1 * m + a1 * g, (b2 * v + (a2 * g) * g).sqrt()):
        scale = (x.view(-1, 256).abs().amax(1) * top).clamp_min(2.0 ** -126)
        out.append(((x.view(-1, 256) / scale[:, None]).clamp(-448, 448).view(-1), scale))
    return out


def neighbours(q):
    """The E4M3 numbers below and above |q|, equal where |q| is one."""
    a = q.double().abs()
    gap = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6))) - 3)
    lo = torch.floor(a / gap) * gap
    return lo, torch.where(a == lo, lo, lo + gap)


@pytest.mark.parametrize("b1,b2,rounding", [(0.9, 0.999, "auto"), (0.96, 0.9, "auto"), (0.9, 0.95, "random")])
def test_random_rounding_is_to_a_neighbour_and_unbiased(b1, b2, rounding):
    n = 1 << 21
    gen = torch.Generator(device="cuda").manual_seed(1)
    w, g = torch.zeros(n, device="cuda"), torch.randn(n, generator=gen, device="cuda")
    g *= torch.exp2(torch.randint(-12, 1, (n,), generator=gen, device="cuda").float())
    s = mb.new_adamw_state(w, 8)
    plan = mb.AdamWPlan([w], [s], grads=[g])
    mb.moe_adamw_step(plan, 1, betas=(0.5, 0.5), rounding="nearest")
    g.copy_(torch.randn(n, generator=gen, device="cuda") * 0.3)
    state = [t.clone() for t in s]
    want = codes_in_fp32(w, s, g, b1, b2)
    mb.moe_adamw_step(plan, 7, betas=(b1, b2), rounding=rounding)
    ups = []
    for (q, scale), got, got_scale in zip(want, (s.m, s.v), (s.m_scale, s.v_scale)):
        assert torch.equal(scale, got_scale)
        code = got.float().double()
        lo, hi = neighbours(q)
        if got is s.v:
            lo, hi = (torch.where(q > 0, x.clamp_min(2.0 ** -9), x) for x in (lo, hi))
        assert ((code.abs() == lo) | (code.abs() == hi)).all()
        assert (torch.sign(code) == torch.sign(q.double()))[code != 0].all()
        inside = hi > lo
        f = ((q.double().abs() - lo) / (hi - lo))[inside]
        up = (code.abs() == hi)[inside]
        ups.append((inside, up.double() - f, (code.abs() == hi).double()))
        # a coin of chance f, 2^20 values to it: six standard deviations in all and in tenths
        for part in [torch.ones_like(up)] + [(f >= k / 10) & (f < (k + 1) / 10) for k in range(10)]:
            count = int(part.sum())
            assert count > 1000
            spread = (f[part] * (1 - f[part])).sum().sqrt().item()
            assert abs((up.double() - f)[part].sum().item()) <= 6 * spread + count * 2.0 ** -20
    # m's and sqrt(v)'s coins are two: their product's mean is nothing
    a, b = (torch.zeros(n, dtype=torch.float64, device="cuda").masked_scatter_(i, d) for i, d, _ in ups)
    assert abs((a * b).sum().item()) <= 6 * (a * b).square().sum().sqrt().item()
    # the same step again: the same bits; another step, another tensor in the list: others
    first = [t.clone() for t in s]

    def again(step, front=0):
        for t, x in zip(s, state):
            t.copy_(x)
        empty = [torch.zeros(0, device="cuda") for _ in range(front)]
        p = mb.AdamWPlan(empty + [w], [mb.new_adamw_state(t, 8) for t in empty] + [s], grads=[t.clone() for t in empty] + [g])
        mb.moe_adamw_step(p, step, betas=(b1, b2), rounding=rounding)
        return [torch.equal(t.view(torch.uint8), x.view(torch.uint8)) for t, x in zip(s, first)]
    assert all(again(7)) and all(again(torch.tensor([6], dtype=torch.int32, device="cuda")))
    for other in (again(8), again(7, front=1)):
        assert other == [False, False, True, True]


@pytest.mark.parametrize("n", [1, 7, 255, 257, 4097, 70001])
def test_random_rounding_of_odd_sizes_extremes_and_nan(n):
    w, g = torch.ones(n, device="cuda"), torch.randn(n, generator=torch.Generator().manual_seed(n)).cuda()
    g[::3] = 0.0
    s = mb.new_adamw_state(w, 8)
    plan = mb.AdamWPlan([w], [s], grads=[g])
    for t in range(1, 4):
        mb.moe_adamw_step(plan, t)
    assert all(torch.isfinite(t.float()).all() for t in (w, *s))
    assert (s.m.float()[::3] == 0).all() and (s.v.float()[::3] == 0).all() and (w[::3] == 1).all()
    # what is not zero has a code; the largest element's is the largest
    assert (s.v.float()[g != 0] > 0).all()
    if n > 1:
        assert s.v.float()[:256].max() == 448
    g[n // 2] = float("nan")
    mb.moe_adamw_step(plan, 4)
    for t in (w, s.m.float(), s.v.float()):
        assert torch.isnan(t[n // 2]) and int(torch.isnan(t).sum()) == 1


def test_nearest_rounding_of_any_betas():
    n = 1 << 16
    w, g = torch.zeros(n, device="cuda"), torch.randn(n, device="cuda")
    s = mb.new_adamw_state(w, 8)
    plan = mb.AdamWPlan([w], [s], grads=[g])
    mb.moe_adamw_step(plan, 1, betas=(0.5, 0.5))
    g.normal_()
    want = codes_in_fp32(w, s, g, 0.9, 0.999)
    mb.moe_adamw_step(plan, 2, betas=(0.9, 0.999), rounding="nearest")
    for (q, _), got in zip(want, (s.m, s.v)):
        code = q.to(torch.float8_e4m3fn).float()
        if got is s.v:
            code = torch.where(q > 0, code.clamp_min(2.0 ** -9), code)
        assert torch.equal(got.float(), code)


def test_a_captured_step_draws_anew():
    """With the step's number on the device: replays equal the steps one by one."""
    runs = []
    for captured in (True, False):
        gen = torch.Generator(device="cuda").manual_seed(0)
        w, g = torch.zeros(5000, device="cuda"), torch.randn(5000, generator=gen, device="cuda")
        s, step = mb.new_adamw_state(w, 8), torch.zeros(1, dtype=torch.int32, device="cuda")
        plan = mb.AdamWPlan([w], [s], grads=[g])
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                mb.moe_adamw_step(plan, step)
        for _ in range(5):
            graph.replay() if captured else mb.moe_adamw_step(plan, step)
            g.mul_(0.9)
        runs.append([w, *(t.view(torch.uint8) for t in s)])
    assert all(torch.equal(a, b) for a, b in zip(*runs))


# ------------------------------------------------------------------ the block's step
NAMES = ("norm_weight", "w_router", "w_gate_up", "w_down")


def block_step(bits):
    block = b.synthetic_block(balance=b.BalanceSettings())
    opt = b.BlockAdamW(block, lr=1e-2, bits=bits)
    g = torch.Generator().manual_seed(1)
    x, stream, dout = (torch.randn(20, 256, generator=g).cuda() for _ in range(3))
    _, h, saved = block.train_forward(x, stream.bfloat16())
    return block, opt, block.train_backward(saved, dout, torch.zeros_like(h))


def all_of(block, opt):
    states = [t for s in opt.plan.states for t in s if t is not None]
    masters = [t for t in opt.plan.masters if t is not None]
    return [t.clone().view(torch.uint8) for t in
            [getattr(block, n) for n in NAMES] + [block.balance_bias, opt.step_count] + masters + states]


@pytest.mark.parametrize("bits", [8, 32, None])
@pytest.mark.parametrize("where", NAMES)
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_step_that_is_left_out_changes_nothing_of_the_block(bits, where, value):
    """The experts with orthogonalised updates and the balance bias among the
    rest; a step after it takes all of them along."""
    block, opt, grads = block_step(bits)
    block.balance_bias.normal_()
    block.balance_bias[3] = -0.0
    block.w_down.view(-1)[:2] = torch.tensor([0.0, -0.0])
    before = all_of(block, opt)
    good = grads[where].clone()
    grads[where].view(-1)[7] = value
    clip = opt.step(grads, balance_rate=1e-3)
    assert not torch.isfinite(clip[1])
    assert all(torch.equal(x, y) for x, y in zip(all_of(block, opt), before))
    grads[where].copy_(good)
    opt.step(grads, balance_rate=1e-3)
    after = all_of(block, opt)
    assert not any(torch.equal(x, y) for x, y in zip(after[:6], before[:6]))
    assert all(torch.isfinite(getattr(block, n)).all() for n in NAMES)


def test_a_captured_step_is_left_out_on_the_device():
    runs = []
    _, opt, grads = block_step(None)
    opt.step(grads)
    for captured in (True, False):
        block, opt, grads = block_step(None)
        step = lambda: opt.step(grads, balance_rate=1e-3)
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        for i in range(4):
            kept = grads["w_down"].view(-1)[5].clone()
            if i % 2:
                grads["w_down"].view(-1)[5] = float("nan")
            graph.replay() if captured else step()
            grads["w_down"].view(-1)[5] = kept
        assert opt.step_count.item() == 2
        runs.append(all_of(block, opt))
    assert all(torch.equal(x, y) for x, y in zip(*runs))


def test_a_plan_without_weights_counts():
    """Unless the step is left out: the counter of plans of which one is empty."""
    w, step = torch.zeros(64, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    none = mb.AdamWPlan([], [], grads=[])
    some = mb.AdamWPlan([w], [mb.new_adamw_state(w)], grads=[torch.ones(64, device="cuda")])
    for t, plan in enumerate((none, some, none, none), 1):
        mb.moe_adamw_step(plan, step)
        assert step.item() == t
    mb.moe_adamw_step(none, step, grad_scale=torch.tensor([float("nan")], device="cuda"))
    assert step.item() == 4
    mb.moe_adamw_step(none, 5, lr=torch.ones(1, device="cuda"))
    assert step.item() == 4


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-38, 1e-39, 1e-44, 1e-46, 1e-60, 0.0])
@pytest.mark.parametrize("on_device", [False, True])
def test_an_eps_below_the_normal_numbers_is_above_zero(bits, eps, on_device):
    """Where v is 0 it is the denominator, and m / eps is 0 with m; with eps 0
    that is 0 / 0.  Elsewhere it does not count: a first step is lr times the
    gradient's sign, off by the step's 16 roundings and those of w; and 1 / b
    and 1 / sqrt(b) of the betas' complements, in FP64."""
    n = 1000
    w, g = torch.ones(n, device="cuda"), torch.randn(n, generator=torch.Generator().manual_seed(2)).cuda()
    g[::2] = 0.0
    s = mb.new_adamw_state(w, bits)
    step = torch.zeros(1, dtype=torch.int32, device="cuda") if on_device else 1
    mb.moe_adamw_step(mb.AdamWPlan([w], [s], grads=[g]), step, lr=0.125, eps=eps)
    if eps:
        assert (w[::2] == 1).all()
    else:
        assert torch.isnan(w[::2]).all()
    want = 1 - 0.125 * torch.sign(g[1::2])
    assert (w[1::2] - want).abs().max().item() <= (0.125 * 24 + 3 * 1.125) * U
