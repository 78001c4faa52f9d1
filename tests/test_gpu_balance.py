"""The load-balance loss and its gradient against their 64-bit definitions."""
import math

import numpy as np
import pytest
import torch

from mixture_experts_ffn_gate_gb300 import moe_block as mb
from tests import step_ref as ref
from tests.block_ref import U

pytestmark = pytest.mark.gpu
INF = float("inf")


def inputs(T, E, k, seed=0, spread=1.0):
    r = np.random.default_rng(seed)
    logits = (r.normal(size=(T, E)) * spread + 0.7 * r.normal(size=E)).astype(np.float32)
    idx = np.argsort(-logits, axis=1, kind="stable")[:, :k].astype(np.int32)
    return logits, idx


def offsets_of(T, S, seed=0, first=0, behind=0):
    if not S:
        return None
    r = np.random.default_rng(seed)
    return np.concatenate(([first], np.sort(r.integers(first, T - behind + 1, size=S - 1)), [T - behind])).astype(np.int32)


def cuda(a):
    return None if a is None else torch.from_numpy(a).cuda()


def check_forward(r, logits, idx, kind, coef, z_coef, offsets):
    want, counts, prob = ref.balance(logits, idx, kind, coef, z_coef, offsets)
    T, E = logits.shape
    assert np.array_equal(r.counts.cpu().numpy(), counts)
    # a probability's error, and at most T / 8 + 100 additions in a row of
    # what a warp, a block and the second kernel add up
    rel = max((ref.row_error(row, E) for row in logits), default=0) + (T / 8 + 100) * U
    got = r.prob.cpu().double().numpy()
    assert (np.abs(got - prob) <= rel * prob).all()
    loss = r.loss.cpu().double().numpy()
    bal = rel + (E + len(counts) * E / 32 / 32 + 64) * U
    assert abs(loss[1] - want[1]) <= bal * abs(want[1])
    # z: a row's lse is off by the sum's relative error and a few roundings of its own size
    lse = max((abs(v) for v in ref.probabilities(logits, kind)[1]), default=0)
    z = (2 * lse * (rel + 4 * U * lse) + rel * lse * lse) if z_coef else 0.0
    assert abs(loss[2] - want[2]) <= z
    assert abs(loss[0] - want[0]) <= abs(coef) * bal * abs(want[1]) + abs(z_coef) * z + 4 * U * (
        abs(coef * want[1]) + abs(z_coef * want[2]))
    return counts


def run(T, E, k, kind, coef=0.3, z_coef=0.0, offsets=None, seed=0, spread=1.0, base=False):
    logits, idx = inputs(T, E, k, seed, spread)
    how = dict(score=kind, coef=coef, z_coef=z_coef, seq_offsets=cuda(offsets))
    r = mb.moe_balance_loss_forward(cuda(logits), cuda(idx), **how)
    counts = check_forward(r, logits, idx, kind, coef, z_coef, offsets)
    b = np.random.default_rng(1).normal(size=(T, E)).astype(np.float32) if base else None
    got = mb.moe_balance_loss_backward(cuda(logits), r.counts, k, dloss=torch.full((1,), 1.7, device="cuda"),
                                       dlogits_in=cuda(b), **how)
    up = float(np.float32(1.7))
    want, bound = ref.balance_grad(logits, counts, k, kind, coef, z_coef, offsets, up, b)
    assert (np.abs(got.cpu().double().numpy() - want) <= bound).all()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("z_coef", [0.0, 0.05])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (7, 3, 3), (64, 16, 4), (65, 16, 4), (100, 5, 2), (33, 32, 32),
                                   (200, 60, 6), (129, 64, 8), (77, 127, 8), (300, 128, 8)])
def test_small(kind, z_coef, T, E, k):
    run(T, E, k, kind, z_coef=z_coef, seed=T + E, base=T % 2 == 0)


@pytest.mark.parametrize("T,E,k", [(90, 160, 8), (90, 253, 8), (90, 256, 8), (70, 257, 1), (70, 384, 8), (66, 509, 10),
                                   (66, 512, 10), (70, 513, 4), (70, 768, 8), (70, 769, 8), (65, 1000, 16),
                                   (65, 1021, 32), (65, 1024, 8)])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_every_row_width(kind, T, E, k):
    run(T, E, k, kind, z_coef=0.01, seed=E, base=True)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,S,first,behind", [(40, 16, 1, 0, 0), (64, 16, 5, 3, 7), (64, 16, 64, 0, 0),
                                                (64, 16, 65, 0, 0), (3, 8, 200, 0, 0), (1500, 32, 3, 100, 300),
                                                (2000, 64, 37, 0, 0), (1700, 128, 900, 1, 1), (900, 8, 1500, 0, 5),
                                                (500, 20, 2, 500, 0), (400, 256, 4, 0, 400)])
def test_sequences(kind, T, E, S, first, behind):
    """Empty ones, single rows, more of them than rows, rows before and behind, ends inside and at a block's end."""
    run(T, E, 4, kind, z_coef=0.02, offsets=offsets_of(T, S, T, first, behind), seed=S, base=True)


@pytest.mark.parametrize("T,E,S", [(512, 16, 0), (513, 16, 0), (256, 128, 0), (257, 128, 3), (128, 256, 3), (128, 256, 4),
                                   (129, 256, 0), (32, 1000, 0), (33, 1000, 2), (48, 500, 3), (49, 500, 0), (511, 7, 3)])
def test_where_one_block_becomes_several(T, E, S):
    for kind in ("softmax", "sigmoid"):
        run(T, E, min(E, 8), kind, z_coef=0.02, offsets=offsets_of(T, S, E, 1, 2), seed=T, base=True)


def test_more_sequences_than_the_grid_is_deep():
    run(3000, 8, 2, "sigmoid", z_coef=0.1, offsets=offsets_of(3000, 40000, 3, 5, 11), base=True)


def test_thousands_of_rows():
    run(20000, 12, 3, "softmax", z_coef=0.01, offsets=offsets_of(20000, 6, 1, 17, 29), spread=3.0)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [20, 300])
def test_slots_that_repeat_or_name_no_expert(kind, T):
    logits, idx = inputs(T, 12, 5)
    r = np.random.default_rng(3)
    idx = np.where(r.random(idx.shape) < 0.3, r.integers(-3, 16, size=idx.shape), idx).astype(np.int32)
    idx[0] = 7
    idx[1] = -1
    got = mb.moe_balance_loss_forward(cuda(logits), cuda(idx), score=kind, coef=0.3, z_coef=0.1)
    check_forward(got, logits, idx, kind, 0.3, 0.1, None)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [30, 200])
def test_masked_experts_and_rows_without_any(kind, T):
    """Logits of -inf and of the lowest number; a row of nothing else."""
    logits, idx = inputs(T, 40, 4)
    logits[:, 5:9] = -INF
    logits[3] = -INF
    logits[4] = np.finfo(np.float32).min
    logits[5, 1:] = np.finfo(np.float32).min
    how = dict(score=kind, coef=0.3, z_coef=0.1 if kind == "softmax" else 0.0)
    if kind == "softmax":
        logits[4, 0] = 0.0  # a lowest maximum would square to infinity in z
    r = mb.moe_balance_loss_forward(cuda(logits), cuda(idx), **how)
    ok = np.where(np.isfinite(logits) & (logits > -1e30), logits, -INF).astype(np.float32)
    counts = check_forward(r, ok, idx, kind, how["coef"], how["z_coef"], None)
    got = mb.moe_balance_loss_backward(cuda(logits), r.counts, 4, **how).cpu().double().numpy()
    want, bound = ref.balance_grad(ok, counts, 4, kind, how["coef"], how["z_coef"])
    assert np.isfinite(got).all() and (np.abs(got - want) <= bound).all()
    assert (got[3] == 0).all() and (got[:, 5:9] == 0).all()


@pytest.mark.parametrize("value", [np.finfo(np.float32).min, -1e30, 0.0, 1e30, np.finfo(np.float32).max])
@pytest.mark.parametrize("T", [5, 100])
def test_rows_of_one_number_are_even(value, T):
    """Also where its exponential, or its product with a constant, is beyond FP32."""
    logits = np.full((T, 20), value, np.float32)
    idx = np.arange(T * 4, dtype=np.int32).reshape(T, 4) % 20
    r = mb.moe_balance_loss_forward(cuda(logits), cuda(idx), coef=0.5)
    assert np.allclose(r.prob.cpu().numpy(), 0.05, rtol=1e-6)
    assert abs(r.loss[1].item() - 1) <= 1e-5 and abs(r.loss[0].item() - 0.5) <= 1e-5
    skewed = torch.arange(20, device="cuda", dtype=torch.int32)[None]
    d = mb.moe_balance_loss_backward(cuda(logits), skewed, 4, coef=0.5)
    want, bound = ref.balance_grad(logits, skewed.cpu().numpy(), 4, "softmax", 0.5, 0.0)
    assert (np.abs(d.cpu().double().numpy() - want) <= 48 * U * np.abs(want) + 48 * U * 0.5 * 20 / (4 * T * T)).all()


@pytest.mark.parametrize("T", [40, 400])
def test_rows_of_no_sequence_are_not_read(T):
    """NaN and infinities before the first sequence and behind the last."""
    logits, idx = inputs(T, 24, 3)
    off = np.array([5, 20, T - 6], np.int32)
    dirty, dirty_idx = logits.copy(), idx.copy()
    dirty[:5], dirty[T - 6:, ::2], dirty[T - 6:, 1::2] = math.nan, INF, -INF
    dirty_idx[:5] = 10 ** 9
    base = np.random.default_rng(0).normal(size=logits.shape).astype(np.float32)
    for kind in ("softmax", "sigmoid"):
        how = dict(score=kind, z_coef=0.1, seq_offsets=cuda(off))
        a = mb.moe_balance_loss_forward(cuda(logits), cuda(idx), **how)
        b = mb.moe_balance_loss_forward(cuda(dirty), cuda(dirty_idx), **how)
        for x, y in zip(a, b):
            assert torch.equal(x, y)
        for base_in in (None, cuda(base)):
            g = mb.moe_balance_loss_backward(cuda(dirty), a.counts, 3, dlogits_in=base_in, **how)
            h = mb.moe_balance_loss_backward(cuda(logits), a.counts, 3, dlogits_in=base_in, **how)
            assert torch.equal(g, h)
            want = torch.zeros(T, 24, device="cuda") if base_in is None else base_in
            assert torch.equal(g[:5], want[:5]) and torch.equal(g[T - 6:], want[T - 6:])


@pytest.mark.parametrize("T", [30, 300])
def test_a_nan_stays_in_its_sequence_and_row(T):
    logits, idx = inputs(T, 16, 4)
    logits[12, 3] = math.nan
    off = cuda(np.array([0, 10, 20, T], np.int32))
    r = mb.moe_balance_loss_forward(cuda(logits), cuda(idx), seq_offsets=off)
    assert torch.isnan(r.loss[:2]).all() and torch.isnan(r.prob[1]).all()
    assert torch.isfinite(r.prob[[0, 2]]).all()
    d = mb.moe_balance_loss_backward(cuda(logits), r.counts, 4, seq_offsets=off)
    assert torch.isnan(d[12]).all() and torch.isfinite(torch.cat((d[:12], d[13:]))).all()


@pytest.mark.parametrize("S", [1, 100])
def test_no_rows(S):
    off = None if S == 1 else torch.zeros(S + 1, dtype=torch.int32, device="cuda")
    l, idx = torch.empty(0, 8, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda")
    out = dict(loss=torch.full((3,), 9.0, device="cuda"), counts=torch.full((S, 8), 9, dtype=torch.int32, device="cuda"),
               prob=torch.full((S, 8), 9.0, device="cuda"))
    r = mb.moe_balance_loss_forward(l, idx, z_coef=1.0, seq_offsets=off, **out)
    assert all((t == 0).all() for t in r)
    assert mb.moe_balance_loss_backward(l, r.counts, 2, seq_offsets=off).shape == (0, 8)


@pytest.mark.parametrize("T,E,S", [(50, 16, 3), (3000, 48, 9), (700, 256, 1)])
def test_repeats_in_place_and_old_workspaces(T, E, S):
    """The same bits again, in a workspace full of other data, and with the gradient in the place of the one that comes in."""
    logits, idx = inputs(T, E, 4)
    off = cuda(offsets_of(T, S, 2, 1, 3))
    how = dict(score="sigmoid", z_coef=0.1, seq_offsets=off)
    ws = mb.new_balance_workspace(T, E, S)
    want = mb.moe_balance_loss_forward(cuda(logits), cuda(idx), **how)
    for fill in (0, 255, 77):
        ws.fill_(fill)
        for a, b in zip(want, mb.moe_balance_loss_forward(cuda(logits), cuda(idx), workspace=ws, **how)):
            assert torch.equal(a, b)
    base = torch.randn(T, E, device="cuda")
    a = mb.moe_balance_loss_backward(cuda(logits), want.counts, 4, dlogits_in=base, **how)
    b = mb.moe_balance_loss_backward(cuda(logits), want.counts, 4, dlogits_in=base, dlogits=base, **how)
    assert b is base and torch.equal(a, b)


def test_offsets_out_of_order_stay_in_bounds():
    """Meaningless, but neither a hang nor an access out of bounds (tensors with guards around them)."""
    T, E = 300, 16
    logits, idx = inputs(T, E, 2)
    for off in ([0, 200, 100, 300], [-5, 10, 1 << 30, 20], [300, 0, 0, 0], [7, 7, 7, 7]):
        off = torch.tensor(off, dtype=torch.int32, device="cuda")
        guard = torch.full((3 * T, E), 5.0, device="cuda")
        counts = torch.full((9, E), 3, dtype=torch.int32, device="cuda")
        r = mb.moe_balance_loss_forward(cuda(logits), cuda(idx), seq_offsets=off, counts=counts[3:6])
        mb.moe_balance_loss_backward(cuda(logits), r.counts, 2, seq_offsets=off, dlogits=guard[T: 2 * T])
        torch.cuda.synchronize()
        assert (guard[:T] == 5).all() and (guard[2 * T:] == 5).all()
        assert (counts[:3] == 3).all() and (counts[6:] == 3).all()


def test_streams_and_graphs():
    T, E, k = 900, 64, 4
    logits, idx = inputs(T, E, k)
    off = offsets_of(T, 5)
    l, i, o = cuda(logits), cuda(idx), cuda(off)
    how = dict(score="sigmoid", z_coef=0.1, seq_offsets=o)
    want = mb.moe_balance_loss_forward(l, i, **how)
    grad = mb.moe_balance_loss_backward(l, want.counts, k, **how)
    side = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for s in side * 4:
        r = mb.moe_balance_loss_forward(l, i, stream=s, **how)
        got.append((r, mb.moe_balance_loss_backward(l, r.counts, k, stream=s, **how)))
    torch.cuda.synchronize()
    for r, g in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want)) and torch.equal(g, grad)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = mb.moe_balance_loss_forward(l, i, **how)
        g = mb.moe_balance_loss_backward(l, r.counts, k, **how)
    for seed in (5, 6):
        logits, idx = inputs(T, E, k, seed)
        off = offsets_of(T, 5, seed, 2, 9)
        l.copy_(cuda(logits)), i.copy_(cuda(idx)), o.copy_(cuda(off))
        graph.replay()
        eager = mb.moe_balance_loss_forward(l, i, **how)
        assert all(torch.equal(a, b) for a, b in zip(r, eager))
        assert torch.equal(g, mb.moe_balance_loss_backward(l, eager.counts, k, **how))
        check_forward(r, logits, idx, "sigmoid", 1e-2, 0.1, off)


def test_the_gradient_joins_the_gates():
    """Gate, its gradient, the loss's gradient added in place: torch's autograd of the same in FP64."""
    T, E, k = 50, 32, 4
    logits, _ = inputs(T, E, k)
    l, dw = cuda(logits), torch.randn(T, k, device="cuda")
    choice = mb.moe_gate_forward(l, k, score="sigmoid", renormalize=True)
    loss = mb.moe_balance_loss_forward(l, choice.topk_idx, score="sigmoid", coef=0.5, z_coef=0.2)
    d = mb.moe_gate_backward(l, choice.topk_idx, dw, score="sigmoid", renormalize=True)
    mb.moe_balance_loss_backward(l, loss.counts, k, score="sigmoid", coef=0.5, z_coef=0.2, dlogits_in=d, dlogits=d)
    x = l.double().requires_grad_(True)
    s = torch.sigmoid(x)
    w = s.gather(1, choice.topk_idx.long())
    w = w / w.sum(1, keepdim=True)
    f = torch.bincount(choice.topk_idx.flatten().long(), minlength=E).double() / (T * k)
    total = ((w * dw.double()).sum() + 0.5 * E * (f * (s / s.sum(1, keepdim=True)).mean(0)).sum()
             + 0.2 * torch.logsumexp(x, 1).square().mean())
    total.backward()
    # each of the two is within 1e-5 of the size of its largest terms
    assert (d.double() - x.grad).abs().max().item() <= 2e-5 * dw.abs().max().item()


def test_refusals_on_the_device():
    l, idx = torch.zeros(8, 4, device="cuda"), torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    for bad in (dict(logits=l.half()), dict(logits=l.t()), dict(topk_idx=idx.long()), dict(topk_idx=idx[:7]),
                dict(seq_offsets=torch.zeros(3, device="cuda")), dict(seq_offsets=torch.zeros(1, device="cuda").int()),
                dict(seq_offsets=torch.zeros(3).int()), dict(loss=torch.zeros(2, device="cuda")),
                dict(counts=torch.zeros(2, 4, device="cuda").int()), dict(prob=torch.zeros(1, 5, device="cuda"))):
        with pytest.raises(ValueError):
            mb.moe_balance_loss_forward(**{**dict(logits=l, topk_idx=idx), **bad})
    c = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    for bad in (dict(counts=c.float()), dict(counts=c.repeat(2, 1)), dict(dloss=torch.zeros((), device="cuda")),
                dict(dlogits_in=l[:7]), dict(dlogits=l.double())):
        with pytest.raises(ValueError):
            mb.moe_balance_loss_backward(**{**dict(logits=l, counts=c, k=2), **bad})
    with pytest.raises(mb.MoeFfnError):
        mb.moe_balance_loss_backward(l, c, 5)
    with pytest.raises(mb.MoeFfnError):
        mb.moe_balance_loss_forward(l, idx, coef=math.nan)


def test_more_than_32_bits_of_logits():
    """2^31 logits and some: the last rows' part in the counts, the loss and the gradient."""
    E = 1024
    T = (1 << 31) // E + 500
    l = torch.zeros(T, E, device="cuda")
    l[-1, 5] = 20.0
    idx = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    idx[-3:] = 1000
    off = torch.tensor([0, T - 2, T], dtype=torch.int32, device="cuda")
    r = mb.moe_balance_loss_forward(l, idx, coef=1.0, seq_offsets=off)
    assert r.counts[0, 0] == T - 3 and r.counts[0, 1000] == 1 and r.counts[1, 1000] == 2
    p = torch.softmax(l[-1].double(), 0)
    want = (p + 1 / E) / 2
    assert ((r.prob[1].double() - want).abs() <= 200 * U * want).all()
    d = mb.moe_balance_loss_backward(l, r.counts, 1, coef=1.0, seq_offsets=off)
    a = torch.zeros(E, dtype=torch.float64, device="cuda")
    a[1000] = E / T
    want = p * (a - (a * p).sum())
    assert ((d[-1].double() - want).abs() <= 200 * U * (p * (a + (a * p).sum()))).all()
    assert torch.isfinite(d[:: 1 << 16]).all()
