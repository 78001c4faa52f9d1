"""The block example's steps beside one another: several forward passes
before their backward passes, several streams, many numbers of tokens."""
import pytest
import torch

from mixture_experts_ffn_gate_gb300 import block as b

pytestmark = pytest.mark.gpu


def tokens(T, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(T, 256, generator=g).cuda(), torch.randn(T, 256, generator=g).bfloat16().cuda(),
            torch.randn(T, 256, generator=g).cuda(), torch.randn(T, 256, generator=g).bfloat16().cuda()]


@pytest.mark.parametrize("T", [1, 33])
def test_forwards_before_their_backwards(T):
    """Micro-batches of equal size: each backward pass has its own forward pass's intermediates."""
    block = b.synthetic_block()
    batches = [tokens(T, s) for s in range(3)]
    want = []
    for x, stream, dout, dstream in batches:
        _, _, saved = block.train_forward(x, stream)
        want.append(block.train_backward(saved, dout, dstream))
    saved = [block.train_forward(x, stream)[2] for x, stream, _, _ in batches]
    got = [block.train_backward(s, dout, dstream) for s, (_, _, dout, dstream) in zip(saved, batches)]
    for a, c in zip(got, want):
        for name in c:
            assert torch.equal(a[name], c[name]), name


def test_serving_on_two_streams():
    block = b.synthetic_block()
    batches = [tokens(4, s)[:2] for s in range(2)]
    want = [block.serve(x, stream)[0].clone() for x, stream in batches]
    sides = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for side, (x, stream) in zip(sides, batches):
            with torch.cuda.stream(side):
                got.append(block.serve(x, stream)[0])
        torch.cuda.synchronize()
        for a, c in zip(got, want):
            assert torch.equal(a, c)
    spaces = [ws.data_ptr() for ws in block._serving.values()]
    assert len(spaces) == 3 and len(set(spaces)) == 3  # one for each stream that served


def test_serving_keeps_a_bounded_number_of_workspaces():
    block = b.synthetic_block()
    for T in [*range(1, 20), 1, 2]:
        block.serve(*tokens(T, T)[:2])
    assert len(block._serving) == block.KEPT


@pytest.mark.parametrize("T", [2, 20])
def test_a_captured_serving_step_outlives_the_kept_workspaces(T):
    block = b.synthetic_block()
    x, stream = tokens(T, 1)[:2]
    want = block.serve(x, stream)[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block.serve(x, stream)[0]
    for other in range(30, 50):
        block.serve(*tokens(other, other)[:2])
    waste = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (1 << 16, 1 << 20, 1 << 22) * 8]
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
    del waste
