"""The block example: its steps agree with torch on the same weights, and
training lowers the loss."""
import pytest
import torch

from mixture_experts_ffn_gate_gb300 import block as b
from mixture_experts_ffn_gate_gb300 import moe_ffn as m

pytestmark = pytest.mark.gpu


def plain(block, x, stream, idx):
    """The block in torch FP64 (autograd) for the choice idx."""
    h = x + stream
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + block.eps) * block.norm_weight.double()
    s = torch.sigmoid(y @ block.w_router.double().t()).gather(1, idx)
    w = s / s.sum(1, keepdim=True) * block.gate.scale
    out = torch.zeros_like(y)
    for e in range(block.E):
        gu = y @ block.w_gate_up[e].double().t()
        a = torch.nn.functional.silu(gu[:, : block.I]) * gu[:, block.I:]
        out = out + (w * (idx == e)).sum(1, keepdim=True) * (a @ block.w_down[e].double().t())
    return out


@pytest.mark.parametrize("T", [1, 4, 33])
def test_serving_step(T):
    block = b.synthetic_block()
    g = torch.Generator().manual_seed(T)
    x, stream = torch.randn(T, 256, generator=g).cuda(), torch.randn(T, 256, generator=g).bfloat16().cuda()
    out, h, loads = block.serve(x, stream)
    _, choice = block.choose(b.mb.moe_rms_norm_forward(x, block.norm_weight, residual=stream).y)
    want = plain(block, x.double(), stream.double(), choice.topk_idx.long())
    # the normed tokens are rounded to BF16 on their way: 2^-8 at most each, 1.7e-3 in the mean square
    assert ((out.double() - want).norm() / want.norm()).item() <= 1e-2
    assert torch.equal(h, (x + stream.float()).bfloat16()) and loads.sum().item() == T * 4
    out8, _, _ = block.serve(x, stream, mxfp8_tokens=True)
    assert ((out8 - out).norm() / out.norm()).item() <= 0.1  # three mantissa bits: 2^-4 at most


def test_training_step_gradients():
    block, T = b.synthetic_block(), 40
    g = torch.Generator().manual_seed(0)
    x, dout = torch.randn(T, 256, generator=g).cuda(), torch.randn(T, 256, generator=g).cuda()
    stream, dstream = (torch.randn(T, 256, generator=g).bfloat16().cuda() for _ in range(2))
    out, h, saved = block.train_forward(x, stream)
    grads = block.train_backward(saved, dout, dstream)
    idx = saved[3].topk_idx.long()
    leaf = {n: getattr(block, n).double().requires_grad_(True) for n in ("norm_weight", "w_router", "w_gate_up",
                                                                       "w_down")}
    other = b.MoeBlock(leaf["norm_weight"], leaf["w_router"], None, leaf["w_gate_up"], leaf["w_down"], block.gate)
    xs = x.double().requires_grad_(True)
    want = plain(other, xs, stream.double(), idx)
    ((want * dout.double()).sum() + ((xs + stream.double()) * dstream.double()).sum()).backward()
    for name, r in [("x", xs.grad)] + [(n, v.grad) for n, v in leaf.items()]:
        # BF16 tokens, stream and gradient of the stream
        assert ((grads[name].double() - r).norm() / r.norm()).item() <= 2e-2, name


def test_training_lowers_the_loss():
    m.moe_ffn_device_faults(clear=True)
    losses = b.train(b.synthetic_block(), steps=10)
    assert losses[-1] < 0.9 * losses[0] and all(y < x * 1.02 for x, y in zip(losses, losses[1:]))
    assert m.moe_ffn_device_faults() == 0
