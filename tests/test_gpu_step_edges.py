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
