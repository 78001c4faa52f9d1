"""The block's operators where they are easily wrong: slots without an
expert beside experts that are not numbers, calls on other streams.  Values against the same calls
without the disturbance, bit for bit, and against the 64-bit definitions."""
import numpy as np
import pytest
import torch

from mixture_experts_ffn_gate_gb300 import moe_block as mb
from mixture_experts_ffn_gate_gb300 import moe_ffn as m
from tests import block_ref as ref
from tests.test_gpu_block import dev, f64, layer, randn

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.fixture(autouse=True)
def _no_faults():
    m.moe_ffn_device_faults(clear=True)
    yield
    assert m.moe_ffn_device_faults(clear=True) == 0, "a kernel's bounded wait gave up"


# ------------------------------------------------------------------ dropped slots
UNUSED = 4  # the experts that no slot uses are the lowest


def masked_routing(T, E, k, seed=0):
    """A routing over the experts from UNUSED on, a third of its slots dropped
    (the first token's all): (idx, w, which are dropped)."""
    r = np.random.default_rng(seed)
    idx = np.stack([UNUSED + r.permutation(E - UNUSED)[:k] for _ in range(T)]).astype(np.int64)
    w = r.normal(size=(T, k)).astype(np.float32)
    for t in range(T):
        for j in range(1, k):
            if r.random() < 0.4:
                idx[t, j] = [-1, E, idx[t, 0], -7][r.integers(4)]
    idx[0] = -1
    if T > 1:
        idx[1] = [UNUSED] + [UNUSED] * (k - 1)
    dropped = np.array([[not 0 <= idx[t, j] < E or idx[t, j] in idx[t, :j] for j in range(k)] for t in range(T)])
    return idx, w, dropped


def options(path):
    o = m.moe_ffn_opts()
    o.path = path
    return o


@pytest.mark.parametrize("T,path", [(1, m.MOE_PATH_AUTO), (2, m.MOE_PATH_AUTO), (4, m.MOE_PATH_AUTO),
                                    (9, m.MOE_PATH_DECODE), (2, m.MOE_PATH_GROUPED), (30, m.MOE_PATH_GROUPED),
                                    (90, m.MOE_PATH_AUTO)])
@pytest.mark.parametrize("k", [3, 9])
def test_dropped_slots_add_nothing(T, path, k):
    """Neither through their weights nor through an expert that stands in for them."""
    H, I, E = 256, 128, 16
    x, wgu, wd = layer(T, H, I, E, seed=40)
    idx, w, dropped = masked_routing(T, E, k, seed=T + k)
    clean = np.where(dropped, np.float32(0), w)
    args = dev(idx, torch.int32), dev(clean)
    want = mb.moe_ffn_forward_routed(x, *args, wgu, wd, opts=options(path))
    exact = ref.experts(f64(x), idx, clean.astype(np.float64), f64(wgu), f64(wd))
    assert ref.rel(f64(want), exact) <= 1e-5  # the two sides' own check: test_gpu_block.py has the tolerance
    gu_bad, d_bad = wgu.clone(), wd.clone()
    gu_bad[0], d_bad[1], d_bad[2], gu_bad[3] = NAN, INF, -INF, INF
    w_bad = np.where(dropped, np.float32([NAN, INF, -INF])[np.arange(T * k).reshape(T, k) % 3], w)
    got = mb.moe_ffn_forward_routed(x, args[0], dev(w_bad), gu_bad, d_bad, opts=options(path))
    assert torch.equal(got, want) and not got[0].any()


@pytest.mark.parametrize("T", [1, 3, 7, 30])
def test_dropped_slots_add_nothing_with_mxfp8_weights(T):
    from mixture_experts_ffn_gate_gb300 import synth
    from tests import gpu_util as gu
    wl = gu.custom(T, 256, 128, 16, 3, name="dropped_mx")
    gq, gs, dq, ds = (t.cuda() for t in synth.make_weights_mxfp8(wl))
    x, _ = (t.cuda() for t in synth.make_tokens(wl, T))
    idx, w, dropped = masked_routing(T, 16, 3, seed=T)
    idx = dev(idx, torch.int32)
    want = mb.moe_ffn_forward_routed(x, idx, dev(np.where(dropped, np.float32(0), w)), gq, dq, w_gate_up_scale=gs,
                                     w_down_scale=ds)
    gq_bad = gq.clone()
    gq_bad[:UNUSED] = 0x7f  # the code of NaN
    got = mb.moe_ffn_forward_routed(x, idx, dev(np.where(dropped, np.float32(NAN), w)), gq_bad, dq,
                                    w_gate_up_scale=gs, w_down_scale=ds)
    assert torch.equal(got, want) and torch.isfinite(got).all()


@pytest.mark.parametrize("T,k", [(1, 3), (5, 9), (40, 3), (300, 2)])
def test_dropped_slots_have_no_gradient(T, k):
    H, I, E = 192, 128, 16
    x, wgu, wd = layer(T, H, I, E, seed=50)
    idx, w, dropped = masked_routing(T, E, k, seed=T + k)
    dout, clean = randn(T, H, seed=60), np.where(dropped, np.float32(0), w)
    ti = dev(idx, torch.int32)
    want = mb.moe_ffn_backward_routed(x, ti, dev(clean), wgu, wd, dout)
    exact = ref.experts_grad(f64(x), idx, clean.astype(np.float64), f64(wgu), f64(wd), f64(dout))
    for g, r in zip((want[0], want[2], want[3]), (exact[0], exact[2], exact[3])):
        assert ref.rel(f64(g), r) <= 1e-5
    # experts and a token that no slot reaches, and the weights of dropped slots
    gu_bad, d_bad, x_bad, dout_bad = wgu.clone(), wd.clone(), x.clone(), dout.clone()
    gu_bad[0], d_bad[1], gu_bad[2], x_bad[0], dout_bad[0] = NAN, INF, -INF, INF, INF
    args = x_bad, ti, dev(np.where(dropped, np.float32(NAN), w)), gu_bad, d_bad
    state = m.new_train_state(T, H, I, E, k)
    out = mb.moe_ffn_forward_routed_train(*args, state)
    assert torch.isfinite(out).all() and not out[0].any()
    for got in (mb.moe_ffn_backward_routed(*args, dout_bad), mb.moe_ffn_backward_routed(*args, dout_bad, state=state)):
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert not got[0][0].any() and not f64(got[1])[dropped].any()
        assert not got[2][:UNUSED].any() and not got[3][:UNUSED].any()


def test_a_weight_of_minus_zero_is_a_weight():
    """Its slot is in use: the weight has a gradient and the output no change."""
    x, wgu, wd = layer(6, 256, 128, 8, seed=70)
    idx = dev(np.random.default_rng(1).permuted(np.tile(np.arange(8), (6, 1)), axis=1)[:, :3], torch.int32)
    w, dout = randn(6, 3, seed=71), randn(6, 256, seed=72)
    w[:, 1] = 0.0
    minus = w.clone()
    minus[:, 1] = -0.0
    for o in (None, options(m.MOE_PATH_DECODE)):
        a, b = (mb.moe_ffn_forward_routed(x, idx, v, wgu, wd, opts=o) for v in (w, minus))
        assert torch.equal(a, b)
    a, b = (mb.moe_ffn_backward_routed(x, idx, v, wgu, wd, dout) for v in (w, minus))
    assert all(torch.equal(p, q) for p, q in zip(a, b)) and b[1][:, 1].all()


# ------------------------------------------------------------------ streams
def stream_calls(T=12):
    """The calls that make a workspace of their own."""
    H, I, E, k = 512, 256, 16, 4
    x, wgu, wd = layer(T, H, I, E, seed=80)
    r = np.random.default_rng(2)
    idx = dev(np.stack([r.permutation(E)[:k] for _ in range(T)]), torch.int32)
    w, dout, logits, nw = randn(T, k, seed=81), randn(T, H, seed=82), randn(T, E, seed=83), randn(H, seed=84)
    wr, batch = randn(E, H, seed=85, dtype=torch.bfloat16), randn(3, 300, 400, seed=86)
    return {
        "norm_backward": lambda **s: mb.moe_rms_norm_backward(x, nw, dout, **s),
        "routed": lambda **s: (mb.moe_ffn_forward_routed(x, idx, w, wgu, wd, **s),),
        "routed_decode": lambda **s: (mb.moe_ffn_forward_routed(x[:2], idx[:2], w[:2], wgu, wd, **s),),
        "routed_backward": lambda **s: mb.moe_ffn_backward_routed(x, idx, w, wgu, wd, dout, **s),
        "orthogonalize": lambda **s: (mb.moe_orthogonalize(batch, **s),),
        "forward_ex": lambda **s: (m.moe_ffn_forward_ex(x, logits, wgu, wd, k, **s),),
        "router": lambda **s: (m.moe_ffn_forward_router(x[:2], wr, None, wgu, wd, k, **s),),
    }


@pytest.mark.parametrize("name", ["norm_backward", "routed", "routed_decode", "routed_backward", "orthogonalize",
                                  "forward_ex", "router"])
@pytest.mark.parametrize("by_handle", [False, True])
def test_calls_on_another_stream_keep_their_workspace(name, by_handle):
    """The call waits on its stream while the current one takes and fills all
    the memory that torch has given back."""
    call = stream_calls()[name]
    want = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about 10 ms
    got = call(stream=side.cuda_stream if by_handle else side)
    waste = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (1 << 12, 1 << 16, 1 << 20, 1 << 22) * 8]
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    del waste


# ------------------------------------------------------------------ the orthogonalisation's range
@pytest.mark.parametrize("M,N", [(1, 200), (60, 40), (300, 500), (2, 1000)])
@pytest.mark.parametrize("coefficients,steps", [((1.8, 0.0, 0.0), 2), ((-1.8, 0.0, 0.0), 2), ((3.0, -0.5, 0.0), 1),
                                                ((3.4445, -4.7750, 2.0315), 10), ((16.0, 0.0, 0.0), 1),
                                                ((0.0, 14.0, 14.0), 1)])
def test_matrices_of_one_row_stay_finite(M, N, coefficients, steps):
    """All of the weight in one row (a singular value of 1 in one entry of A),
    with coefficients near the limits."""
    g = torch.zeros(2, M, N)
    g[0, M // 2] = randn(N, seed=M).cpu()
    g[1] = torch.outer(randn(M, seed=N).cpu(), randn(N, seed=N + 1).cpu())
    out = f64(mb.moe_orthogonalize(g.cuda(), steps=steps, coefficients=coefficients))
    assert np.isfinite(out).all()
    if abs(coefficients[0]) ** steps > 500:
        return  # the tolerance is of five steps of slope 3.4 at zero, which raise the roundings 485 times
    for b in range(2):
        want = ref.orthogonalize(f64(g[b]), steps, coefficients, 1e-7)
        # FP16 roundings of X, A and b A + c A A, as in test_gpu_block.py, and BF16's of each element
        assert ref.rel(out[b], want) <= 2.7e-3 + 2.0 ** -8


# ------------------------------------------------------------------ the gate
@pytest.mark.parametrize("E,groups,kept", [(24, 1, 1), (64, 8, 3), (384, 1, 1), (512, 4, 2), (1000, 1, 1)])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_gate_rows_without_softmax_scores(E, groups, kept, renormalize, bad):
    """All of the row's scores are NaN, which tie above every number: the
    bias has no say, the lowest experts are chosen."""
    k, r = 6, np.random.default_rng(E)
    logits, bias = r.normal(size=(5, E)).astype(np.float32), r.normal(size=E).astype(np.float32)
    clean = mb.moe_gate_forward(dev(logits), k, bias=dev(bias), groups=groups, topk_groups=kept,
                                renormalize=renormalize)
    logits[1, E - 3] = logits[3, 0] = bad
    out = mb.moe_gate_forward(dev(logits), k, bias=dev(bias), groups=groups, topk_groups=kept,
                              renormalize=renormalize)
    for t in range(5):
        if t in (1, 3):
            assert out.topk_idx[t].tolist() == list(range(k)) and torch.isnan(out.topk_w[t]).all()
        else:
            assert torch.equal(out.topk_idx[t], clean.topk_idx[t]) and torch.equal(out.topk_w[t], clean.topk_w[t])


@pytest.mark.parametrize("E", [32, 24, 20])
def test_gate_chooses_by_the_scores_that_it_returns(E):
    """With a bias of zero the choice is the order of the returned sigmoid
    scores, bit for bit: logits so close that neighbours' scores are equal or
    one unit apart."""
    r = np.random.default_rng(E)
    base = np.concatenate([r.uniform(-20, 20, 3000), r.uniform(-88.7, -86, 500), r.uniform(-104, -88.7, 200),
                           r.uniform(-2, 2, 1000)]).astype(np.float32)
    step = np.spacing(np.abs(base)) * r.integers(1, 5, size=base.shape)
    logits = (base[:, None] + step[:, None] * r.permuted(np.tile(np.arange(E), (len(base), 1)), axis=1))
    logits = dev(logits.astype(np.float32))
    out = mb.moe_gate_forward(logits, E, bias=torch.zeros(E).cuda(), score="sigmoid", renormalize=False)
    w, idx = out.topk_w.cpu().numpy(), out.topk_idx.cpu().numpy()
    assert np.all((w[:, :-1] > w[:, 1:]) | ((w[:, :-1] == w[:, 1:]) & (idx[:, :-1] < idx[:, 1:])))
    assert np.array_equal(np.sort(idx, axis=1), np.tile(np.arange(E), (len(base), 1)))
    s = 1 / (1 + np.exp(-f64(logits)))
    # expf and two roundings
    assert np.all(np.abs(w - np.take_along_axis(s, idx, 1)) <= s.max(axis=1, keepdims=True) * 2.0 ** -20 + 1e-38)


# ------------------------------------------------------------------ the orthogonalisation's norm
@pytest.mark.parametrize("M,N", [(70, 90), (71, 33), (256, 256), (300, 520), (520, 300), (301, 77)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_orthogonalize_does_not_see_the_scale(M, N, dtype):
    """A power of two on the whole matrix changes no bit, also where the
    squares leave FP32's range at either end."""
    g = randn(2, M, N, seed=M, dtype=dtype)
    want = mb.moe_orthogonalize(g, eps=0.0)
    assert torch.isfinite(want).all() and want.any()
    for p in (-80, -70, -20, 20, 60, 64, 100):
        assert torch.equal(mb.moe_orthogonalize(g * 2.0 ** p, eps=0.0), want), p
    mixed = torch.stack([g[0] * 2.0 ** 90, g[1]])
    assert torch.equal(mb.moe_orthogonalize(mixed, eps=0.0), want)
    # a norm that no FP32 number holds is no silent zero
    beyond = torch.stack([torch.full((M, N), 3e38, dtype=dtype, device="cuda"), g[1]])
    out = mb.moe_orthogonalize(beyond, eps=0.0)
    assert torch.isnan(out[0]).all() and torch.equal(out[1], want[1])
