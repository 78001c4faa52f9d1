"""The block's operators on the GPU against their 64-bit definitions
(tests/block_ref.py).  Tolerances come from the arithmetic, beside each
check: U is half a unit in the last place of FP32."""
import numpy as np
import pytest
import torch

from mixture_experts_ffn_gate_gb300 import moe_block as mb
from mixture_experts_ffn_gate_gb300 import moe_ffn as m
from tests import block_ref as ref
from tests.block_ref import U

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
BF16_HALF = 2.0 ** -8  # a value's largest relative rounding to BF16


@pytest.fixture(autouse=True)
def _no_faults():
    m.moe_ffn_device_faults(clear=True)
    yield
    assert m.moe_ffn_device_faults(clear=True) == 0, "a kernel's bounded wait gave up"


def dev(a, dtype=F32):
    return torch.as_tensor(np.asarray(a)).to(dtype).cuda()


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def randn(*shape, seed=0, std=1.0, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


# ------------------------------------------------------------------ norm
NORM_SHAPES = [(1, 1), (1, 64), (3, 7), (5, 96), (2, 1000), (1, 2048), (17, 2056), (700, 333), (4, 7168), (2, 16384),
               (3, 16383), (1300, 32)]


@pytest.mark.parametrize("T,H", NORM_SHAPES)
@pytest.mark.parametrize("xt,rt", [(BF16, None), (F32, None), (F32, BF16), (BF16, BF16), (BF16, F32), (F32, F32)])
def test_norm_forward(T, H, xt, rt):
    x, w = randn(T, H, seed=1, dtype=xt), 1 + randn(H, seed=2, std=0.2)
    res = None if rt is None else randn(T, H, seed=3, std=3.0, dtype=rt)
    mx = H % 32 == 0
    out = mb.moe_rms_norm_forward(x, w, residual=res, eps=1e-5, mxfp8=mx)
    h, y = ref.norm(f64(x), f64(res), f64(w), 1e-5)
    # sums over H: 16 terms in turn and at most 10 levels; the root halves it
    fp = 40 * U
    assert np.all(np.abs(f64(out.y) - y) <= np.abs(y) * (BF16_HALF + fp) + 1e-30)
    if res is None:
        assert out.h is None
    else:
        exact = (x.float() + res.float()).to(rt)  # one FP32 addition, rounded once more
        assert torch.equal(out.h, exact)
    if not mx:
        assert out.codes is None
        return
    codes, scales = out.codes.cpu().numpy(), out.scales.cpu().numpy()
    assert scales.shape == (T, m.mx_scale_bytes(H)) and not scales[:, H // 32:].any()
    top = np.abs(y).reshape(T, H // 32, 32).max(axis=2)
    e = scales[:, : H // 32].astype(np.int64) - 127 + 8  # floor(log2 top), or its neighbour at a power of two
    assert np.all(2.0 ** e <= top * (1 + fp)) and np.all(top * (1 - fp) < 2.0 ** (e + 1))
    step = np.repeat(2.0 ** (e - 8), 32, axis=1)
    v = np.clip(y / step, -448, 448)
    # a normal code is within 2^-4 of its value, a subnormal one within 2^-10
    tol = np.maximum(np.abs(v) * 2.0 ** -4, 2.0 ** -10) + np.abs(v) * fp * 2
    assert np.all(np.abs(ref.mx_values(codes, scales) / step - v) <= tol)


@pytest.mark.parametrize("T,H", [(9, 12), (3, 1004), (4, 4100), (2, 16380), (2000, 100)])
@pytest.mark.parametrize("xt,rt", [(BF16, None), (F32, BF16), (BF16, F32)])
def test_norm_forward_of_other_widths(T, H, xt, rt):
    """Rows of a multiple of four elements, not of eight; in place as well."""
    test_norm_forward(T, H, xt, rt)
    if rt is not None:
        x, w, res = randn(T, H, seed=1, dtype=xt), randn(H, seed=2), randn(T, H, seed=3, dtype=rt)
        want = mb.moe_rms_norm_forward(x, w, residual=res)
        got = mb.moe_rms_norm_forward(x, w, residual=res, h=res)
        assert torch.equal(got.y, want.y) and torch.equal(res, want.h)


def test_norm_in_place_and_outputs_of_the_caller():
    x, res, w = randn(9, 256, seed=1), randn(9, 256, seed=2, dtype=BF16), randn(256, seed=3)
    want = mb.moe_rms_norm_forward(x, w, residual=res, mxfp8=True)
    stream = res.clone()
    y = torch.empty_like(want.y)
    got = mb.moe_rms_norm_forward(x, w, residual=stream, h=stream, y=y, bf16=False)
    assert got.y is y and got.h is stream and got.codes is None
    assert torch.equal(stream, want.h) and torch.equal(y, want.y)
    only = mb.moe_rms_norm_forward(x, w, residual=res, bf16=False, mxfp8=True)
    assert only.y is None and torch.equal(only.codes, want.codes) and torch.equal(only.scales, want.scales)


def test_norm_special_values():
    x = torch.zeros(5, 64)
    x[1, 3] = float("inf")
    x[2, 40] = float("nan")
    x[3] = 1e-20     # squares below FP32's range: the eps remains
    x[4] = 3e19      # squares above it
    out = mb.moe_rms_norm_forward(x.cuda(), torch.ones(64).cuda(), eps=1e-6, mxfp8=True)
    y, s = f64(out.y), out.scales.cpu().numpy()
    assert not y[0].any() and np.all(s[0, :2] == 127) and not out.codes[0].any()
    assert np.isnan(y[1, 3]) and np.all(y[1, :3] == 0) and s[1, 0] == 255 and s[1, 1] == 127
    assert np.isnan(y[2]).all() and np.all(s[2, :2] == 255)
    assert np.allclose(y[3], 1e-17, rtol=BF16_HALF) and np.all(np.abs(ref.mx_values(
        out.codes.cpu().numpy(), s)[3] - 1e-17) <= 1e-17 / 16)
    assert not y[4].any()  # 3e19 / inf
    none = mb.moe_rms_norm_forward(torch.empty(0, 64).cuda(), torch.ones(64).cuda())
    assert none.y.shape == (0, 64)


@pytest.mark.parametrize("T,H", [(1, 1), (1, 64), (3, 7), (5, 96), (17, 2056), (700, 333), (4, 7168), (2, 16384),
                                 (3, 16383), (3000, 40)])
@pytest.mark.parametrize("ht,gt,with_res", [(BF16, F32, True), (F32, BF16, False), (F32, F32, True),
                                            (BF16, BF16, False)])
def test_norm_backward(T, H, ht, gt, with_res):
    h, dy = randn(T, H, seed=1, std=2.0, dtype=ht), randn(T, H, seed=2, dtype=gt)
    w = 1 + randn(H, seed=3, std=0.2)
    dres = randn(T, H, seed=4, dtype=ht) if with_res else None
    dh, dw = mb.moe_rms_norm_backward(h, w, dy, dres=dres, eps=1e-5)
    want, want_w, bound, bound_w = ref.norm_grad(f64(h), f64(w), f64(dy), f64(dres), 1e-5)
    half = BF16_HALF if ht is BF16 else U
    assert dh.dtype == ht
    assert np.all(np.abs(f64(dh) - want) <= bound + np.abs(want) * half + 1e-37)
    assert np.all(np.abs(f64(dw) - want_w) <= bound_w + np.abs(want_w) * 64 * U + 1e-37)
    # in place, the same bits again
    if with_res:
        into = dres.clone()
        dh2, dw2 = mb.moe_rms_norm_backward(h, w, dy, dres=into, eps=1e-5, dh=into)
        assert torch.equal(dh2, dh) and torch.equal(dw2, dw)


@pytest.mark.parametrize("T,H", [(9, 12), (6, 1004), (4, 4100), (2, 16380), (5000, 100), (9000, 36), (2500, 37)])
@pytest.mark.parametrize("ht,gt,with_res", [(BF16, F32, True), (F32, BF16, False), (F32, F32, True)])
def test_norm_backward_of_other_widths(T, H, ht, gt, with_res):
    """Rows of a multiple of four elements, not of eight; many short rows."""
    test_norm_backward(T, H, ht, gt, with_res)


def test_norm_backward_of_no_rows():
    dw = torch.full((64,), 7.0).cuda()
    mb.moe_rms_norm_backward(torch.empty(0, 64).cuda(), torch.ones(64).cuda(), torch.empty(0, 64).cuda(), dweight=dw)
    assert not dw.any()


# ------------------------------------------------------------------ gate
def check_gate(logits, k, bias=None, kind="softmax", groups=1, topk_groups=1, renormalize=True, scale=1.0):
    out = mb.moe_gate_forward(dev(logits), k, bias=None if bias is None else dev(bias), score=kind, groups=groups,
                              topk_groups=topk_groups, renormalize=renormalize, scale=scale, counts=True)
    idx, w = ref.gate(logits, k, bias, kind, groups, topk_groups, renormalize, scale)
    got = out.topk_idx.cpu().numpy()
    assert np.array_equal(got, idx)
    assert np.array_equal(out.counts.cpu().numpy(), np.bincount(idx.ravel(), minlength=logits.shape[1]))
    # exp's argument (a rounding of the difference), exp, the sum over E (32
    # lanes and 5 levels) or over k, and two divisions
    fin = np.where(np.isfinite(logits), logits, 0)
    spread = (fin.max(axis=1) - fin.min(axis=1) + np.abs(fin).max(axis=1))[:, None]
    tol = (logits.shape[1] / 32 + k + 16 + 2 * spread) * U
    assert np.all(np.abs(f64(out.topk_w) - w) <= np.abs(w) * tol + 1e-38)
    return got


def logits_of(T, E, seed, bias=None, kind="softmax", groups=1):
    """Random logits whose choice does not hang on an FP32 rounding: tokens
    with two values closer than that are replaced."""
    r = np.random.default_rng(seed)
    out = r.normal(size=(T, E)).astype(np.float32) * 2
    if bias is not None:
        for _ in range(200):
            bad = ref.gate_gap(out, bias, kind, groups) < 8 * U * 4
            if not bad.any():
                return out
            out[bad] = r.normal(size=(int(bad.sum()), E)).astype(np.float32) * 2
        raise AssertionError("no separated logits found")
    return out


SHAPES = [(1, 1, 1), (1, 8, 8), (3, 5, 2), (16, 33, 4), (17, 60, 10), (40, 128, 8), (9, 160, 6), (300, 256, 8),
          (5, 384, 12), (7, 500, 9), (4, 1024, 32), (2, 1023, 17)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("kind,renormalize,scale", [("softmax", True, 1.0), ("softmax", False, 2.5),
                                                    ("sigmoid", True, 2.5), ("sigmoid", False, 1.0)])
def test_gate_forward(T, E, k, kind, renormalize, scale):
    check_gate(logits_of(T, E, T + E), k, None, kind, 1, 1, renormalize, scale)


@pytest.mark.parametrize("T,E,k", [(3, 5, 2), (17, 60, 10), (40, 128, 8), (70, 64, 6), (9, 24, 3)])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_gate_with_a_bias(T, E, k, kind):
    bias = np.random.default_rng(5).normal(size=E).astype(np.float32) * 0.3
    check_gate(logits_of(T, E, 7, bias, kind), k, bias, kind, 1, 1, True, 1.5)


@pytest.mark.parametrize("T,E,k,groups,kept", [
    (20, 32, 4, 4, 2), (20, 256, 8, 8, 4), (20, 60, 6, 4, 1), (20, 60, 6, 6, 3), (5, 160, 6, 8, 3), (30, 64, 2, 32, 2),
    (9, 8, 3, 8, 5), (4, 1024, 32, 32, 2), (6, 96, 4, 2, 2), (3, 384, 8, 3, 1), (7, 1000, 5, 10, 4)])
@pytest.mark.parametrize("biased", [False, True])
def test_gate_with_groups(T, E, k, groups, kept, biased):
    bias = np.random.default_rng(6).normal(size=E).astype(np.float32) * 0.5 if biased and E <= 256 else None
    check_gate(logits_of(T, E, 8, bias, "sigmoid", groups), k, bias, "sigmoid", groups, kept, True, 1.0)


def test_gate_ties_and_signed_zeros():
    r = np.random.default_rng(9)
    logits = r.choice(np.array([-1.0, -0.0, 0.0, 1.0], np.float32), size=(50, 96))
    check_gate(logits, 7)
    check_gate(logits, 32, kind="sigmoid", renormalize=False)
    check_gate(logits, 5, groups=8, topk_groups=3)
    check_gate(np.zeros((3, 40), np.float32), 32)
    # a bias over equal scores decides, and equal sums of groups go to the lower
    bias = np.repeat(np.array([0.25, 0.5, 0.5, 0.25], np.float32), 4)
    got = check_gate(np.zeros((2, 16), np.float32), 3, bias, "sigmoid", 4, 1, True, 1.0)
    assert (got == [4, 5, 6]).all()


def test_gate_choices_from_one_lane():
    """All k largest in a run of neighbours: they sit in one lane, whose list is used up."""
    for E, k in ((1024, 32), (512, 16), (384, 12), (1024, 20)):
        logits = np.linspace(-3, -1, E).astype(np.float32)[None].repeat(4, 0)
        for t in range(4):
            at = [0, 32, E - 32, 333][t]
            logits[t, at:at + 32] += np.linspace(9, 5, 32).astype(np.float32)
        check_gate(logits, k)


@pytest.mark.parametrize("E", [20, 33, 100, 200, 384, 500, 1000])
def test_gate_equal_logits_in_every_lane(E):
    """Few distinct values: lists of equal keys that are used up, in every number of experts per lane."""
    r = np.random.default_rng(E)
    k = min(E, 32)
    logits = r.choice(np.array([-2.0, 0.5, 1.5], np.float32), size=(40, E), p=[0.6, 0.3, 0.1])
    logits[0] = 0.5
    logits[1, : E // 2] = 1.5
    check_gate(logits, k)
    check_gate(logits, k - 1, kind="sigmoid", renormalize=False)


def test_gate_saturated_sigmoid_scores_with_a_bias():
    """exp(-l) up to infinity; the scores are 0 or 1 to 1e-6, the bias keeps the choices 1/128 apart."""
    r = np.random.default_rng(12)
    logits = r.choice(np.array([-np.inf, -200, -89, -88, -87.5, -87, -20, 20, 90, np.inf], np.float32), size=(70, 60))
    bias = (r.permutation(60) / 128).astype(np.float32)
    check_gate(logits, 12, bias, "sigmoid")


def test_gate_reads_what_the_kernel_before_it_writes():
    """Logits and bias that come straight from a kernel that lets the next one start early."""
    H, I, E, k = 1024, 512, 16, 4
    r = np.random.default_rng(21)
    wgu, wd = (dev(r.normal(size=s) * 0.2, BF16) for s in ((E, 2 * I, H), (E, H, I)))
    idx, w = dev(np.arange(k)[None], torch.int32), dev(np.full((1, k), 0.25))
    x, logits = torch.empty(1, H, dtype=BF16, device="cuda"), dev(r.normal(size=(1, H)))
    ws, out = m.new_workspace(1, H, I, E, k), torch.empty(1, H, device="cuda")

    def experts():
        out.zero_()
        mb.moe_ffn_forward_routed(x, idx, w, wgu, wd, out=out, workspace=ws)

    def run(between):
        experts()
        between()
        a = mb.moe_gate_forward(out, 16, score="sigmoid")
        experts()
        between()
        return (*a[:2], *mb.moe_gate_forward(logits, 16, bias=out[0], score="sigmoid", counts=True))

    x.zero_()
    run(torch.cuda.synchronize)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(lambda: None)
    for _ in range(20):
        x.copy_(dev(r.normal(size=(1, H)), BF16))
        want = run(torch.cuda.synchronize)
        graph.replay()
        torch.cuda.synchronize()
        for g, t in zip(got, want):
            assert torch.equal(g, t)


def test_gate_masked_and_special_logits():
    logits = logits_of(6, 64, 10)
    logits[0] = -np.inf                     # nothing left: weights of zero, the lowest experts
    logits[1, 5:] = -np.inf                 # five left, eight asked for
    logits[2] = -200.0                      # every sigmoid score rounds to zero
    logits[3] = np.finfo(np.float32).min    # a mask's lowest value
    logits[4, ::2] = np.finfo(np.float32).min
    for kind in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            out = mb.moe_gate_forward(dev(logits), 8, score=kind, renormalize=renormalize)
            idx, w = ref.gate(logits, 8, None, kind, 1, 1, renormalize, 1.0)
            got = f64(out.topk_w)
            assert np.array_equal(out.topk_idx.cpu().numpy(), idx)
            assert np.isfinite(got).all()
            rows = [0, 1, 3, 4, 5] if kind == "sigmoid" else range(6)  # a sum below FP32's range counts as zero
            assert np.all(np.abs(got[rows] - w[rows]) <= np.abs(w[rows]) * 1e-4 + 1e-37)
    nan = logits_of(2, 40, 11)
    nan[0, 7] = np.nan
    out = mb.moe_gate_forward(dev(nan), 4)
    assert out.topk_idx[0, 0] == 7 and (out.topk_idx >= 0).all() and (out.topk_idx < 40).all()
    assert torch.isfinite(out.topk_w[1]).all()


def test_gate_of_no_tokens():
    counts = torch.full((12,), 3, dtype=torch.int32).cuda()
    out = mb.moe_gate_forward(torch.empty(0, 12).cuda(), 2, counts=counts)
    assert out.topk_idx.shape == (0, 2) and not counts.any()


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("kind,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True),
                                              ("sigmoid", False)])
def test_gate_backward(T, E, k, kind, renormalize):
    r = np.random.default_rng(T * E)
    logits, dw = logits_of(T, E, 12), r.normal(size=(T, k)).astype(np.float32)
    idx, _ = ref.gate(logits, k, None, kind, 1, 1, renormalize, 1.0)
    got = f64(mb.moe_gate_backward(dev(logits), dev(idx, torch.int32), dev(dw), score=kind, renormalize=renormalize,
                                   scale=2.0))
    want = ref.gate_grad(logits, idx, dw, kind, renormalize, 2.0)
    assert np.all(np.abs(got - want) <= ref.gate_grad_bound(logits, dw, kind, renormalize, 2.0))
    if kind == "sigmoid" or renormalize:
        rest = np.ones((T, E), bool)
        np.put_along_axis(rest, idx, False, 1)
        assert not got[rest].any()
    if renormalize and k == 1:
        assert not got.any()  # the one weight is the scale


def test_gate_backward_of_unused_slots():
    logits, dw = logits_of(4, 50, 13), np.random.default_rng(1).normal(size=(4, 5)).astype(np.float32)
    idx = np.array([[3, -1, 7, 3, 50], [-5, -5, -5, -5, -5], [0, 1, 2, 3, 4], [49, 1 << 30, 49, 8, -1]])
    for kind in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            got = f64(mb.moe_gate_backward(dev(logits), dev(idx, torch.int32), dev(dw), score=kind,
                                           renormalize=renormalize))
            want = ref.gate_grad(logits, idx, dw, kind, renormalize, 1.0)
            assert np.all(np.abs(got - want) <= ref.gate_grad_bound(logits, dw, kind, renormalize, 1.0))


# ------------------------------------------------------------------ experts
# The grouped path holds FP32 intermediates as pairs of BF16 values: a pair is
# within (2^-8 / sqrt 6)^2 = 2.6e-6 of its value in the root mean square, two
# of them and the product of their low parts 7.9e-6; sums of 256 terms on the
# tensor cores round toward zero 16 times, 1e-6.
PAIRS = 1e-5


def layer(T, H, I, E, seed=0):
    x = randn(T, H, seed=seed + 1, dtype=BF16)
    wgu, wd = randn(E, 2 * I, H, seed=seed + 2, std=H ** -0.5, dtype=BF16), randn(E, H, I, seed=seed + 3, std=I ** -0.5,
                                                                              dtype=BF16)
    return x, wgu, wd


def routing(T, E, k, seed=0, drop=False):
    r = np.random.default_rng(seed)
    idx = np.stack([r.permutation(E)[:k] for _ in range(T)]).astype(np.int64)
    w = r.normal(size=(T, k)).astype(np.float32)  # weights are used as they are, negative ones too
    if drop:
        idx[r.random((T, k)) < 0.2] = -1
        idx[0] = -1
        idx[-1, -1] = idx[-1, 0]
        idx[-1, 0] = E if k > 1 else idx[-1, 0]
    return idx, w


ROUTED = [(1, 256, 128, 8, 2), (2, 512, 256, 32, 4), (3, 320, 192, 5, 3), (4, 1024, 256, 64, 8), (5, 256, 128, 8, 8),
          (40, 384, 192, 12, 3), (33, 128, 64, 3, 1), (150, 640, 320, 4, 2), (1, 64, 64, 64, 32), (20, 64, 64, 40, 32)]


@pytest.mark.parametrize("T,H,I,E,k", ROUTED)
@pytest.mark.parametrize("drop", [False, True])
def test_routed_forward(T, H, I, E, k, drop):
    x, wgu, wd = layer(T, H, I, E)
    idx, w = routing(T, E, k, drop=drop)
    out = mb.moe_ffn_forward_routed(x, dev(idx, torch.int32), dev(w), wgu, wd)
    want = ref.experts(f64(x), idx, w.astype(np.float64), f64(wgu), f64(wd))
    assert ref.rel(f64(out), want) <= PAIRS
    if drop:
        assert not out[0].any()


@pytest.mark.parametrize("T", [1, 2, 3, 4, 9])
def test_routed_decode_has_the_routers_bits(T):
    """Given the router's own choice, the decode path gives the layer's output bit for bit."""
    x, wgu, wd = layer(T, 512, 256, 32)
    logits = randn(T, 32, seed=5)
    idx, w = torch.empty(T, 4, dtype=torch.int32).cuda(), torch.empty(T, 4).cuda()
    o = m.moe_ffn_opts()
    o.path = m.MOE_PATH_DECODE
    want = m.moe_ffn_forward_ex(x, logits, wgu, wd, 4, topk_idx=idx, topk_w=w, opts=o)
    ws = mb.new_routed_workspace(T, 512, 256, 32, 4)
    for _ in range(3):  # the barrier's exchange, then the tagged one
        got = mb.moe_ffn_forward_routed(x, idx, w, wgu, wd, workspace=ws, opts=o)
        assert torch.equal(got, want)


@pytest.mark.parametrize("T", [1, 4, 7, 30])
def test_routed_mxfp8_weights_have_the_layers_bits(T):
    from mixture_experts_ffn_gate_gb300 import synth
    from tests import gpu_util as gu
    wl = gu.custom(T, 256, 128, 8, 2, name="routed_mx")
    gq, gs, dq, ds = (t.cuda() for t in synth.make_weights_mxfp8(wl))
    x, logits = (t.cuda() for t in synth.make_tokens(wl, T))
    idx, w = torch.empty(T, 2, dtype=torch.int32).cuda(), torch.empty(T, 2).cuda()
    want = m.moe_ffn_forward_mxfp8(x, logits, gq, gs, dq, ds, 2, topk_idx=idx, topk_w=w)
    got = mb.moe_ffn_forward_routed(x, idx, w, gq, dq, w_gate_up_scale=gs, w_down_scale=ds)
    assert torch.equal(got, want)


@pytest.mark.parametrize("T", [1, 4, 30])
def test_routed_mxfp8_tokens_are_their_values(T):
    _, wgu, wd = layer(T, 512, 128, 16)
    n = mb.moe_rms_norm_forward(randn(T, 512, seed=9), torch.ones(512).cuda(), mxfp8=True)
    wide = dev(ref.mx_values(n.codes.cpu().numpy(), n.scales.cpu().numpy()), BF16)
    idx, w = routing(T, 16, 4)
    idx, w = dev(idx, torch.int32), dev(w)
    want = mb.moe_ffn_forward_routed(wide, idx, w, wgu, wd)
    assert torch.equal(mb.moe_ffn_forward_routed(n.codes, idx, w, wgu, wd, x_scale=n.scales), want)


@pytest.mark.parametrize("T,H,I,E,k", [(1, 256, 128, 8, 2), (3, 320, 192, 5, 3), (40, 384, 192, 12, 3),
                                       (33, 128, 64, 3, 1), (90, 256, 128, 4, 2), (12, 64, 64, 40, 32),
                                       (150, 192, 64, 2, 2), (300, 64, 128, 3, 1)])
@pytest.mark.parametrize("drop", [False, True])
def test_routed_backward(T, H, I, E, k, drop):
    x, wgu, wd = layer(T, H, I, E, seed=20)
    idx, w = routing(T, E, k, seed=3, drop=drop)
    dout = randn(T, H, seed=30)
    args = (x, dev(idx, torch.int32), dev(w), wgu, wd)
    got = mb.moe_ffn_backward_routed(*args, dout)
    want = ref.experts_grad(f64(x), idx, w.astype(np.float64), f64(wgu), f64(wd), f64(dout))
    for name, g, r in zip(("dx", "dwgu", "dwd"), (got[0], got[2], got[3]), (want[0], want[2], want[3])):
        assert ref.rel(f64(g), r) <= PAIRS, name
    # one weight's gradient is one product of I terms: its error is that of the
    # pairs beside the product of the vectors' lengths, not beside their sum
    a_q = np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            e = idx[t, j]
            if 0 <= e < E:
                gu = f64(wgu[e]) @ f64(x[t])
                act = gu[:I] / (1 + np.exp(-gu[:I])) * gu[I:]
                a_q[t, j] = np.linalg.norm(act) * np.linalg.norm(f64(wd[e]).T @ f64(dout[t]))
    assert np.all(np.abs(f64(got[1]) - want[1]) <= PAIRS * a_q + 1e-30)
    dropped = np.array([[not 0 <= idx[t, j] < E or idx[t, j] in idx[t, :j] for j in range(k)] for t in range(T)])
    assert not f64(got[1])[dropped].any()
    untouched = [e for e in range(E) if e not in idx[~dropped]]
    assert not got[2][untouched].any() and not got[3][untouched].any()
    # the training pair: the same output as the forward call's grouped path, the same gradients
    state = m.new_train_state(T, H, I, E, k)
    o = m.moe_ffn_opts()
    o.path = m.MOE_PATH_GROUPED
    assert torch.equal(mb.moe_ffn_forward_routed_train(*args, state), mb.moe_ffn_forward_routed(*args, opts=o))
    for _ in range(2):
        for a, b in zip(mb.moe_ffn_backward_routed(*args, dout, state=state), got):
            assert torch.equal(a, b)


def test_routed_sums_over_long_rows():
    """K = 4096 in segments: one chain of tensor-core additions would be 1.1e-5 off."""
    x, wgu, wd = layer(24, 4096, 192, 6)
    idx, w = routing(24, 6, 3)
    out = mb.moe_ffn_forward_routed(x, dev(idx, torch.int32), dev(w), wgu, wd)
    xs, g, d = x.double(), wgu.double(), wd.double()
    want = torch.zeros(24, 4096, dtype=torch.float64, device="cuda")
    for e in range(6):
        gu = xs @ g[e].T
        y = (torch.nn.functional.silu(gu[:, :192]) * gu[:, 192:]) @ d[e].T
        want += (dev(w, torch.float64) * dev(idx == e, torch.float64)).sum(1, keepdim=True) * y
    assert ((out.double() - want).norm() / want.norm()).item() <= 5e-6  # one pair, and the segments


def test_routed_grid_widths_and_no_tokens():
    x, wgu, wd = layer(40, 256, 128, 8)
    idx, w = routing(40, 8, 2)
    idx, w = dev(idx, torch.int32), dev(w)
    want = mb.moe_ffn_forward_routed(x, idx, w, wgu, wd)
    for ctas in (1, 5, 151):
        o = m.moe_ffn_opts()
        o.gemm_ctas = ctas
        assert torch.equal(mb.moe_ffn_forward_routed(x, idx, w, wgu, wd, opts=o), want)
    none = mb.moe_ffn_forward_routed(x[:0], idx[:0], w[:0], wgu, wd)
    assert none.shape == (0, 256)
    grads = mb.moe_ffn_backward_routed(x[:0], idx[:0], w[:0], wgu, wd, torch.empty(0, 256).cuda())
    assert not grads[2].any() and not grads[3].any()


# ------------------------------------------------------------------ orthogonalised updates
# FP16 roundings of X, A and b A + c A A, 2^-12 / sqrt 3 each, in five steps
# whose polynomial's slope raises them: 2e-3 in 64-bit simulations with those
# roundings (64 x 64 Gaussian matrices are the worst), 2.7e-3 taken; and the
# output's rounding to BF16, 1.7e-3 in the root mean square of many elements,
# 2^-8 for a few.
def ortho_tol(M, N):
    return 2.7e-3 + (1.7e-3 if M * N >= 1000 else BF16_HALF)


USUAL = (3.4445, -4.7750, 2.0315)


@pytest.mark.parametrize("B,M,N", [(1, 1, 1), (2, 1, 40), (3, 5, 3), (1, 64, 64), (2, 65, 129), (3, 129, 65), (1, 256, 256),
                                   (2, 257, 300), (1, 300, 1000), (5, 31, 257), (1, 513, 512), (2, 768, 192),
                                   (20, 48, 80), (1, 1100, 700), (70, 260, 300), (90, 200, 256), (200, 40, 300),
                                   (300, 264, 8), (160, 130, 257), (1, 256, 257)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_orthogonalize(B, M, N, dtype):
    g = randn(B, M, N, seed=M + N, std=1e-3, dtype=dtype)
    out = f64(mb.moe_orthogonalize(g))
    for b in range(B):
        assert ref.rel(out[b], ref.orthogonalize(f64(g[b]), 5, USUAL, 1e-7)) <= ortho_tol(*g.shape[1:])


@pytest.mark.parametrize("M,N", [(300, 500), (500, 300)])
def test_orthogonalize_low_rank(M, N):
    """Few large singular values and many small ones, which the steps raise by hundreds."""
    g = torch.stack([randn(M, 4, seed=1) @ randn(4, N, seed=2) + randn(M, N, seed=3, std=0.01),
                     torch.outer(randn(M, seed=4), randn(N, seed=5)),
                     randn(M, 32, seed=6) @ randn(32, N, seed=7) + randn(M, N, seed=8, std=0.05)])
    out = f64(mb.moe_orthogonalize(g))
    for b in range(3):
        assert ref.rel(out[b], ref.orthogonalize(f64(g[b]), 5, USUAL, 1e-7)) <= ortho_tol(*g.shape[1:])


def test_orthogonalize_steps_coefficients_scale():
    g = randn(2, 100, 140, seed=1, std=5.0)
    for steps, co, scale in ((1, USUAL, 1.0), (2, (1.5, -0.5, 0.0), 0.25), (7, (2.0, -1.5, 0.5), -3.0),
                             (12, (1.875, -1.25, 0.375), 1.0)):
        out = f64(mb.moe_orthogonalize(g, steps=steps, coefficients=co, out_scale=scale))
        for b in range(2):
            assert ref.rel(out[b], scale * ref.orthogonalize(f64(g[b]), steps, co, 1e-7)) <= ortho_tol(100, 140)


def test_orthogonalize_special_matrices():
    g = randn(6, 70, 90, seed=2)
    g[1] = 0
    g[2, 3, 4] = float("nan")
    g[3, 69, 89] = float("inf")
    g[4] = 0
    g[4, 10, 20] = -2.0
    out = f64(mb.moe_orthogonalize(g))
    for b in (0, 4, 5):
        assert ref.rel(out[b], ref.orthogonalize(f64(g[b]), 5, USUAL, 1e-7)) <= ortho_tol(*g.shape[1:])
    assert not out[1].any()
    assert np.isnan(out[2]).all() and not np.isfinite(out[3]).any()
    assert mb.moe_orthogonalize(g[:0]).shape == (0, 70, 90)


@pytest.mark.parametrize("B,M,N", [(3, 300, 520), (2, 700, 300), (100, 30, 400), (5, 200, 100)])
def test_orthogonalize_repeats_streams_graphs(B, M, N):
    """The tiled products (one launch whose blocks wait on one another) and the small matrices."""
    g, ws = randn(B, M, N, seed=1), mb.new_orthogonalize_workspace(B, M, N)
    want = mb.moe_orthogonalize(g, workspace=ws)
    for _ in range(5):
        assert torch.equal(mb.moe_orthogonalize(g, workspace=ws), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = mb.moe_orthogonalize(g, workspace=ws)
    side.synchronize()
    assert torch.equal(again, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = mb.moe_orthogonalize(g, workspace=ws)
    g.copy_(randn(B, M, N, seed=2))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    fresh = mb.moe_orthogonalize(g)
    assert torch.equal(captured, fresh) and not torch.equal(fresh, want)


# ------------------------------------------------------------------ streams, graphs, repeats
def all_operators(s):
    """One call of each operator on the tensors of `s`, outputs allocated here."""
    n = mb.moe_rms_norm_forward(s["x32"], s["w"], residual=s["res"], mxfp8=True)
    g = mb.moe_gate_forward(s["logits"], 4, bias=s["bias"], score="sigmoid", groups=4, topk_groups=2, counts=True)
    out = mb.moe_ffn_forward_routed(n.y, g.topk_idx, g.topk_w, s["wgu"], s["wd"], workspace=s["ws"])
    dx, dw, dwgu, dwd = mb.moe_ffn_backward_routed(n.y, g.topk_idx, g.topk_w, s["wgu"], s["wd"], out, workspace=s["bws"])
    dl = mb.moe_gate_backward(s["logits"], g.topk_idx, dw, score="sigmoid")
    dh, dweight = mb.moe_rms_norm_backward(n.h, s["w"], dx, workspace=s["nws"])
    up = mb.moe_orthogonalize(dwd, workspace=s["ows"])
    return [*n, *g, out, dx, dw, dwgu, dwd, dl, dh, dweight, up]


def operands(T, seed=0):
    H, I, E = 256, 128, 16
    x, wgu, wd = layer(T, H, I, E, seed=seed)
    return dict(x32=randn(T, H, seed=seed + 7), w=1 + randn(H, seed=seed + 8, std=0.1), res=x, wgu=wgu, wd=wd,
                logits=randn(T, E, seed=seed + 9), bias=randn(E, seed=seed + 10, std=0.1),
                ws=mb.new_routed_workspace(T, H, I, E, 4), bws=m.new_backward_workspace(T, H, I, E, 4),
                nws=mb.new_rms_norm_backward_workspace(T, H), ows=mb.new_orthogonalize_workspace(E, H, I))


@pytest.mark.parametrize("T", [1, 3, 50])
def test_repeats_streams_and_graphs_give_the_same_bits(T):
    s = operands(T)
    want = all_operators(s)
    for _ in range(3):
        for a, b in zip(all_operators(s), want):
            assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = all_operators(s)
    side.synchronize()
    for a, b in zip(on_side, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = all_operators(s)
    other = operands(T, seed=100)
    fresh = all_operators(other)
    for name in ("x32", "w", "res", "wgu", "wd", "logits", "bias"):
        s[name].copy_(other[name])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(captured, fresh):
        assert torch.equal(a, b)


def test_large_offsets():
    """Rows whose elements lie past 2^31."""
    T, H = 140000, 16384
    x = torch.zeros((T, H), dtype=BF16, device="cuda")
    x[-1] = randn(H, seed=1, dtype=BF16)
    n = mb.moe_rms_norm_forward(x, torch.ones(H).cuda())
    one = mb.moe_rms_norm_forward(x[-1:], torch.ones(H).cuda())
    assert torch.equal(n.y[-1:], one.y)
    logits = torch.zeros((2200000, 1024), dtype=F32, device="cuda")
    logits[-1] = randn(1024, seed=2)
    g = mb.moe_gate_forward(logits, 2, counts=True)
    o = mb.moe_gate_forward(logits[-1:], 2)
    assert torch.equal(g.topk_idx[-1:], o.topk_idx) and torch.equal(g.topk_w[-1:], o.topk_w)
    assert g.counts.sum().item() == 2 * 2200000
