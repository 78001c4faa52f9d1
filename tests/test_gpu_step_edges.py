"""Edges of the training step's operators on the device, against 64 bits."""
import numpy as np
import pytest
import torch

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
