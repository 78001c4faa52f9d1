"""The block's operators in the kernels' instances that small shapes do not
reach: every tile width of the orthogonalisation, the three-term products at
the accuracy that they are there for, thousands of tokens, gates of hundreds
of experts with a bias."""
import numpy as np
import pytest
import torch

from mixture_experts_ffn_gate_gb300 import moe_block as mb
from mixture_experts_ffn_gate_gb300 import moe_ffn as m
from tests.test_gpu_block import USUAL, check_gate, dev, layer, logits_of, ortho_tol, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_faults():
    m.moe_ffn_device_faults(clear=True)
    yield
    assert m.moe_ffn_device_faults(clear=True) == 0, "a kernel's bounded wait gave up"


def rel(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


# ------------------------------------------------------------------ experts
# Three BF16 terms hold an FP32 operand to 2^-24.  The tensor cores round each
# addition toward zero, by at most 2^-23 of a running sum that grows to its
# value: half of that over a chain of 16 (a segment of 256 products, the rows
# of an expert in steps of 16) is 1e-6, and two products follow one another.
# Two terms would leave 2.6e-6, one chain for all products of a long expert
# 2.7e-6 (315 rows).
TERMS = 2e-6


def exact(x, idx, w, wgu, wd, dout):
    """In 64 bits on the GPU, expert by expert: out, dx, dw, dwgu, dwd, and of
    every slot the product of the lengths of act and q."""
    T, k = idx.shape
    E, H, I = wd.shape
    x, dout, w = x.double(), dout.double(), w.double()
    out, dx = torch.zeros_like(x), torch.zeros_like(x)
    dw, size = torch.zeros_like(w), torch.zeros_like(w)
    dwgu, dwd = wgu.new_zeros((E, 2 * I, H), dtype=torch.float64), wgu.new_zeros((E, H, I), dtype=torch.float64)
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        g, u = (x[t] @ wgu[e].double().T).split(I, dim=1)
        s = torch.sigmoid(g)
        a, wt, q = g * s * u, w[t, j][:, None], dout[t] @ wd[e].double()
        out.index_add_(0, t, wt * (a @ wd[e].double().T))
        dw[t, j], size[t, j] = (a * q).sum(1), a.norm(dim=1) * q.norm(dim=1)
        da = wt * q
        dgu = torch.cat((da * u * s * (1 + g * (1 - s)), da * g * s), dim=1)
        dx.index_add_(0, t, dgu @ wgu[e].double())
        dwgu[e], dwd[e] = dgu.T @ x[t], (wt * dout[t]).T @ a
    return out, dx, dw, dwgu, dwd, size


@pytest.mark.parametrize("T,H,I,E,k", [(24, 4096, 192, 6, 3), (64, 1024, 512, 16, 4), (512, 512, 256, 16, 4),
                                       (700, 256, 192, 2, 1), (2048, 256, 128, 64, 8), (5000, 128, 64, 40, 3)])
def test_routed_products_have_their_three_terms(T, H, I, E, k):
    """Outputs and every gradient, recomputed and from the training state."""
    x, wgu, wd = layer(T, H, I, E, seed=90)
    g = torch.Generator().manual_seed(T)
    idx = torch.rand(T, E, generator=g).topk(k).indices.int().cuda()
    w, dout = randn(T, k, seed=91), randn(T, H, seed=92)
    out, dx, dw, dwgu, dwd, size = exact(x, idx, w, wgu, wd, dout)
    o = m.moe_ffn_opts()
    o.path = m.MOE_PATH_GROUPED
    args = x, idx, w, wgu, wd
    got = mb.moe_ffn_forward_routed(*args, opts=o)
    assert rel(got, out) <= TERMS
    state = m.new_train_state(T, H, I, E, k)
    assert torch.equal(mb.moe_ffn_forward_routed_train(*args, state), got)
    grads = mb.moe_ffn_backward_routed(*args, dout)
    for name, a, b in zip(("dx", "dwgu", "dwd"), (grads[0], grads[2], grads[3]), (dx, dwgu, dwd)):
        assert rel(a, b) <= TERMS, name
    # a weight's gradient is a product of vectors that may cancel: beside their lengths
    assert (grads[1].double() - dw).norm() <= TERMS * size.norm()
    for a, b in zip(mb.moe_ffn_backward_routed(*args, dout, state=state), grads):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ the orthogonalisation's tile widths
def instance(B, M, N):
    """The widths of the symmetric products' and of apply's tiles (launch_orthogonalize's rule)."""
    m_, n = min(M, N), max(M, N)
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    rows, cols = -(-m_ // 256), -(-m_ // 128)

    def fit(tiles):
        return tiles <= pairs if B == 1 else 12 * B * tiles <= 13 * pairs
    if not fit(sum(cols - 2 * r for r in range(rows))):
        return 256, 256
    return 128, 128 if fit(rows * -(-n // 128)) else 256


WIDTHS = [(1, 1536, 2048), (1, 2048, 1536), (6, 768, 2048), (1, 1537, 1999), (2, 2051, 770), (16, 777, 1100), (16, 1101, 777),
          (9, 1024, 1024), (20, 513, 900), (1, 1000, 1000), (1, 999, 1203), (3, 600, 400)]


def test_the_shapes_below_reach_every_instance():
    assert {instance(*s) for s in WIDTHS} == {(128, 128), (128, 256), (256, 256)}


@pytest.mark.parametrize("B,M,N", WIDTHS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_orthogonalize_of_every_tile_width(B, M, N, dtype):
    g = randn(B, M, N, seed=M + N, dtype=dtype)
    out, (a, b, c) = mb.moe_orthogonalize(g), USUAL
    for i in range(B):
        x = g[i].double() / (g[i].double().norm() + 1e-7)
        x = x.T if M > N else x
        for _ in range(5):
            s = x @ x.T
            x = a * x + (b * s + c * s @ s) @ x
        assert rel(out[i], x.T if M > N else x) <= ortho_tol(M, N), i


# ------------------------------------------------------------------ gates of hundreds of experts with a bias
@pytest.mark.parametrize("T,E,k,groups,kept", [(20, 384, 8, 1, 1), (20, 384, 8, 8, 4), (12, 512, 9, 1, 1), (12, 512, 8, 8, 3),
                                               (300, 260, 6, 1, 1), (6, 1000, 5, 10, 4), (4, 1024, 32, 32, 2),
                                               (5, 1023, 17, 1, 1), (7, 640, 10, 20, 5)])
@pytest.mark.parametrize("kind,renormalize", [("sigmoid", True), ("sigmoid", False), ("softmax", True),
                                              ("softmax", False)])
def test_gate_with_a_bias_over_many_experts(T, E, k, groups, kept, kind, renormalize):
    bias = np.random.default_rng(E).normal(size=E).astype(np.float32) * 0.5
    logits = logits_of(T, E, 14, bias, kind, groups)
    check_gate(logits, k, bias, kind, groups, kept, renormalize, 1.5)


@pytest.mark.parametrize("T,E,k", [(3, 5, 2), (17, 60, 10), (40, 128, 8), (9, 256, 8)])
def test_gate_with_a_bias_and_plain_softmax_weights(T, E, k):
    bias = np.random.default_rng(E).normal(size=E).astype(np.float32) * 0.3
    check_gate(logits_of(T, E, 15, bias, "softmax"), k, bias, "softmax", 1, 1, False, 2.5)
