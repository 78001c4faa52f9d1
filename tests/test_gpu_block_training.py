"""The block's training step with the load-balance loss and AdamW: its
gradients against torch's in FP64, its update against the 64-bit definitions,
and a whole step in a CUDA graph."""
import numpy as np
import pytest
import torch

from mixture_experts_ffn_gate_gb300 import block as b
from mixture_experts_ffn_gate_gb300 import moe_block as mb
from tests import step_ref as ref
from tests.test_gpu_block_example import plain

pytestmark = pytest.mark.gpu

NAMES = ("norm_weight", "w_router", "w_gate_up", "w_down")


def tokens(T, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(T, 256, generator=g).cuda(), torch.randn(T, 256, generator=g).bfloat16().cuda(),
            torch.randn(T, 256, generator=g).cuda(), torch.randn(T, 256, generator=g).bfloat16().cuda()]


@pytest.mark.parametrize("offsets", [None, [0, 7, 7, 30]])
def test_gradients_with_the_balance_loss(offsets):
    block, T = b.synthetic_block(balance=b.BalanceSettings(coef=3.0, z_coef=0.5)), 40
    x, stream, dout, dstream = tokens(T)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    out, h, saved = block.train_forward(x, stream, seq_offsets=off)
    grads = block.train_backward(saved, dout, dstream, dbalance=torch.full((1,), 2.0, device="cuda"))
    idx = saved.choice.topk_idx.long()
    leaf = {n: getattr(block, n).double().requires_grad_(True) for n in NAMES}
    other = b.MoeBlock(leaf["norm_weight"], leaf["w_router"], None, leaf["w_gate_up"], leaf["w_down"], block.gate)
    xs = x.double().requires_grad_(True)
    want = plain(other, xs, stream.double(), idx)
    hs = xs + stream.double()
    y = hs / torch.sqrt(hs.square().mean(1, keepdim=True) + block.eps) * leaf["norm_weight"]
    logits = y @ leaf["w_router"].t()
    s = torch.sigmoid(logits)
    s = s / s.sum(1, keepdim=True)
    ends = [0, T] if offsets is None else offsets
    N, loss = ends[-1] - ends[0], 0.0
    for lo, hi in zip(ends, ends[1:]):
        if hi > lo:
            c = torch.bincount(idx[lo:hi].flatten(), minlength=16).double()
            loss = loss + (hi - lo) / N * 16 * (c / (4 * (hi - lo)) * s[lo:hi].mean(0)).sum()
    z = torch.logsumexp(logits[ends[0]: ends[-1]], 1).square().sum() / N
    loss = 3.0 * loss + 0.5 * z
    assert abs(saved.balance.loss[0].item() - loss.item()) <= 2e-2 * loss.item()  # tokens rounded to BF16
    ((want * dout.double()).sum() + (hs * dstream.double()).sum() + 2.0 * loss).backward()
    for name, r in [("x", xs.grad)] + [(n, v.grad) for n, v in leaf.items()]:
        # BF16 tokens, stream and gradient of the stream
        assert ((grads[name].double() - r).norm() / r.norm()).item() <= 2e-2, name


def test_without_settings_the_step_is_the_one_it_was():
    x, stream, dout, dstream = tokens(33)
    runs = []
    for balance in (None, b.BalanceSettings(coef=0.0, z_coef=0.0)):
        block = b.synthetic_block(balance=balance)
        out, h, saved = block.train_forward(x, stream)
        assert (saved.balance is None) == (balance is None)
        runs.append((out, h, block.train_backward(saved, dout, dstream)))
    (a, p, g), (c, q, d) = runs
    assert torch.equal(a, c) and torch.equal(p, q)
    for name in g:  # coefficients of zero add zeros
        assert torch.equal(g[name], d[name]), name


@pytest.mark.parametrize("bits", [8, 32, None])
def test_an_adamw_step_of_the_block(bits):
    block = b.synthetic_block(balance=b.BalanceSettings())
    opt = b.BlockAdamW(block, lr=1e-2, max_norm=0.5, bits=bits)
    x, stream, dout, dstream = tokens(40)
    _, _, saved = block.train_forward(x, stream)
    grads = block.train_backward(saved, dout / 100, dstream / 100)
    before = {n: getattr(block, n).detach().cpu().double().numpy().reshape(-1) for n in NAMES}
    clip = opt.step(grads)
    g = {n: grads[n].cpu().double().numpy().reshape(-1) for n in NAMES}
    norm, factor = ref.norm(g.values(), 0.5)
    assert np.allclose(clip.cpu().numpy(), [norm, factor], rtol=1e-5) and factor < 1
    assert opt.step_count.item() == 1
    for n in opt.names:
        zeros = np.zeros_like(g[n])
        decay = 0.0 if n == "norm_weight" else 0.1
        want, *_, err, _, _ = ref.adamw(before[n], g[n] * factor, zeros, zeros, 1, float(np.float32(1e-2)), 0.9, 0.95,
                                        1e-8, decay)
        # the factor's own error (1e-5 above) leaves sign(g) as it is but next to eps
        err = 2 * err + 1e-2 * 1e-5
        got = getattr(block, n)
        half = 2.0 ** -8 * np.abs(want) if got.dtype is torch.bfloat16 else 0.0
        assert (np.abs(got.cpu().double().numpy().reshape(-1) - want) <= err + 1.01 * half).all(), n
    if bits is None:
        assert any((getattr(block, n).cpu().double().numpy().reshape(-1) != before[n]).any() for n in ("w_down",))


def test_training_runs():
    for bits in (8, None):
        block = b.synthetic_block(balance=b.BalanceSettings(z_coef=1e-3))
        losses = b.train(block, steps=4, optimizer=b.BlockAdamW(block, bits=bits))
        assert len(losses) == 4 and np.isfinite(losses).all()


def test_a_step_whose_gradients_are_no_numbers_is_left_out():
    block = b.synthetic_block()
    opt = b.BlockAdamW(block)
    x, stream, dout, dstream = tokens(20)
    _, _, saved = block.train_forward(x, stream)
    grads = block.train_backward(saved, dout, dstream)
    before = {n: getattr(block, n).clone() for n in NAMES}
    good = grads["w_down"].clone()
    grads["w_down"][3, 5, 7] = float("nan")
    opt.step(grads)
    assert opt.step_count.item() == 0 and all(torch.equal(getattr(block, n), v) for n, v in before.items())
    grads["w_down"] = good
    opt.step(grads)
    assert opt.step_count.item() == 1 and all(not torch.equal(getattr(block, n), v) for n, v in before.items())


def test_a_captured_training_step():
    """Forward, loss, backward, clipping and update in one graph: its replays
    give the bits of the same steps one by one."""
    def fresh():
        block = b.synthetic_block(balance=b.BalanceSettings(z_coef=1e-3))
        return block, b.BlockAdamW(block, lr=1e-2)

    def step(block, opt, x, stream, target):
        out, h, saved = block.train_forward(x, stream)
        grads = block.train_backward(saved, (out - target) / out.numel(), torch.zeros_like(h))
        return out, saved.balance.loss, opt.step(grads)
    x, stream, target, _ = tokens(48)
    warm = fresh()
    step(*warm, x, stream, target)
    one, two = fresh(), fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*one, x, stream, target)
    for i in range(4):
        graph.replay()
        want = step(*two, x, stream, target)
        for a, c in zip(got, want):
            assert torch.equal(a, c), i
        for n in NAMES:
            assert torch.equal(getattr(one[0], n), getattr(two[0], n)), n
        x.mul_(0.9)
    assert one[1].step_count.item() == 4


def test_the_plan_of_a_block_keeps_its_masters_in_step():
    block = b.synthetic_block()
    opt = b.BlockAdamW(block, bits=8)
    b.train(block, steps=3, optimizer=opt)
    for w, master in zip(opt.plan.weights, opt.plan.masters):
        if master is not None:
            assert torch.equal(w, master.to(w.dtype))
    assert isinstance(opt.plan, mb.AdamWPlan)
