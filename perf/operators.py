"""The operators around the experts of a Mixture-of-Experts block, as measured cases.

A block's step is: the residual addition with its root-mean-square norm, the
gate (scores, top-k, weights), the experts' products for that routing, and in
training their gradients and the orthogonalised update of the experts'
weights.  Each case is one call of one of them:

  norm        h = x + residual, y = h / rms(h) * weight, in BF16 and in MXFP8
  norm_grad   the gradients of h and weight
  gate        top-k experts of T tokens, their weights, the experts' loads
  gate_grad   the logits' gradient for the chosen weights' gradient
  experts     the SwiGLU experts' weighted sum for a routing that is passed in
  experts_grad  its gradients: tokens, routing weights, both weight tensors
  ortho       Newton-Schulz orthogonalisation of a batch of updates

``run`` computes them in plain torch operations in 32 bits, or with the
library (``own``).
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS_NORM = 1e-6
EPS_ORTHO = 1e-7
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5


def listed():
    return [
        # one token of a serving step: the experts' FP32 output joins the BF16 residual stream
        dict(name="norm_decode", op="norm", T=1, H=2048, x="f32", residual="bf16", mxfp8=False),
        # a prefill's tokens, the normed rows in BF16 for the gate and in 8 bits to be stored or sent
        dict(name="norm_prefill_mxfp8", op="norm", T=16384, H=7168, x="f32", residual="bf16", mxfp8=True),
        # a training step's tokens (an odd number of them), FP32 gradient from the experts
        dict(name="norm_grad_train", op="norm_grad", T=8191, H=6144, h="bf16", dy="f32", residual="bf16"),
        # one token of a serving step
        dict(name="gate_decode", op="gate", T=1, E=128, k=8, score="softmax", bias=False, groups=1,
             topk_groups=1, renormalize=True, scale=1.0),
        # a prefill's tokens: sigmoid scores, a balance bias, the experts of 4 of 8 groups
        dict(name="gate_prefill_grouped", op="gate", T=16384, E=256, k=8, score="sigmoid", bias=True, groups=8,
             topk_groups=4, renormalize=True, scale=2.5),
        # a training step's tokens over many experts, weights not renormalised: every logit has a gradient
        dict(name="gate_grad_train", op="gate_grad", T=8191, E=384, k=8, score="softmax", renormalize=False,
             scale=1.0),
        # one token through the 2048-hidden serving layer
        dict(name="experts_decode", op="experts", T=1, H=2048, I=768, E=128, k=8),
        # a batch of 64 sequences through the 4096-hidden serving layer
        dict(name="experts_batch", op="experts", T=64, H=4096, I=1536, E=128, k=8),
        # a training step of the 2048-hidden layer
        dict(name="experts_grad_train", op="experts_grad", T=512, H=2048, I=768, E=128, k=8),
        # the tiny layer's eight gate/up gradients
        dict(name="ortho_tiny", op="ortho", B=8, M=256, N=256, g="f32"),
        # sixteen experts' gate/up gradients of the 2048-hidden layer
        dict(name="ortho_gate_up", op="ortho", B=16, M=1536, N=2048, g="f32"),
        # four experts' down-projection momenta of the 6144-hidden layer, tall ones, kept in BF16
        dict(name="ortho_down_tall", op="ortho", B=4, M=6144, N=2048, g="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "gate", "gate", "gate_grad", "experts", "experts_grad", "ortho",
                     "ortho"])
    if op == "norm":
        mxfp8 = rng.random() < 0.5
        H = 32 * _log(rng, 2, 256) if mxfp8 else _log(rng, 64, 8192)
        return dict(op=op, T=_log(rng, 1, 12000), H=H, x=rng.choice(["bf16", "f32"]),
                    residual=rng.choice(["none", "bf16", "f32"]), mxfp8=mxfp8)
    if op == "norm_grad":
        return dict(op=op, T=_log(rng, 1, 8000), H=_log(rng, 64, 8192), h=rng.choice(["bf16", "f32"]),
                    dy=rng.choice(["bf16", "f32"]), residual=rng.choice(["none", "bf16"]))
    E = rng.choice([8, 60, 64, 128, 160, 256, 384, 512])
    k = min(E, rng.choice([1, 2, 4, 6, 8, 8, 10]))
    if op == "gate":
        groups = rng.choice([g for g in (1, 2, 4, 8) if E % g == 0 and E // g >= k])
        score = rng.choice(["softmax", "sigmoid"])
        return dict(op=op, T=_log(rng, 1, 16000), E=E, k=k, score=score, bias=score == "sigmoid" and rng.random() < 0.7,
                    groups=groups, topk_groups=rng.randint(1, groups), renormalize=rng.random() < 0.6,
                    scale=rng.choice([1.0, 2.5]))
    if op == "gate_grad":
        return dict(op=op, T=_log(rng, 1, 16000), E=E, k=k, score=rng.choice(["softmax", "sigmoid"]),
                    renormalize=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]))
    if op == "ortho":
        m, n = _log(rng, 65, 2048), _log(rng, 65, 2048)
        b = max(1, min(16, int(2 ** 33 / (m * n * min(m, n)))))
        return dict(op=op, B=rng.randint(1, b), M=m, N=n, g=rng.choice(["f32", "bf16"]))
    E = rng.choice([8, 32, 64, 128])
    H, I = 64 * rng.randint(4, 32), 64 * rng.randint(2, 16)
    return dict(op=op, T=_log(rng, 1, 64 if op == "experts" else 400), H=H, I=I, E=E, k=min(E, rng.choice([1, 2, 4, 8])))


def work(c):
    op = c["op"]
    size = {"bf16": 2, "f32": 4, "none": 0}
    if op == "norm":
        row = size[c["x"]] + 2 * size[c["residual"]] + 2 + (33 / 32 if c["mxfp8"] else 0)
        return {"bytes": c["T"] * c["H"] * row + 4 * c["H"], "flops": 5 * c["T"] * c["H"]}
    if op == "norm_grad":
        row = 2 * size[c["h"]] + size[c["dy"]] + size[c["residual"]]
        return {"bytes": c["T"] * c["H"] * row + 8 * c["H"], "flops": 10 * c["T"] * c["H"]}
    if op == "gate":
        return {"bytes": 4 * c["T"] * c["E"] + 8 * c["T"] * c["k"] + 8 * c["E"], "flops": 4 * c["T"] * c["E"]}
    if op == "gate_grad":
        dense = c["score"] == "softmax" and not c["renormalize"]
        read = c["E"] if dense else c["k"]
        return {"bytes": 4 * c["T"] * (c["E"] + read) + 8 * c["T"] * c["k"], "flops": 4 * c["T"] * read}
    if op == "ortho":
        m, n = sorted((c["M"], c["N"]))
        # two of the three products of a step are symmetric: half of each is computed
        return {"bytes": c["B"] * m * n * (size[c["g"]] + 2), "flops": c["B"] * STEPS * (3 * m * m * n + m * m * m)}
    T, H, I, E, k = (c[x] for x in ("T", "H", "I", "E", "k"))
    touched = E * (1 - (1 - k / E) ** T)
    if op == "experts":
        return {"bytes": touched * 6 * H * I + T * H * 6 + 8 * T * k, "flops": 6 * H * I * T * k}
    return {"bytes": touched * 6 * H * I + E * 12 * H * I + T * H * 10 + 12 * T * k, "flops": 16 * H * I * T * k}


def prepare(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = c["op"]

    def randn(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, generator=gen, device=DEV) * std).to(dtype)

    s = dict(c)
    if op == "norm":
        T, H = c["T"], c["H"]
        s["x"] = randn(T, H, dtype=TYPES[c["x"]], std=0.5)
        s["residual"] = None if c["residual"] == "none" else randn(T, H, dtype=TYPES[c["residual"]], std=2.0)
        s["weight"] = 1.0 + randn(H, std=0.1)
    elif op == "norm_grad":
        T, H = c["T"], c["H"]
        s["h"] = randn(T, H, dtype=TYPES[c["h"]], std=2.0)
        s["weight"] = 1.0 + randn(H, std=0.1)
        s["dy"] = randn(T, H, dtype=TYPES[c["dy"]])
        s["dres"] = None if c["residual"] == "none" else randn(T, H, dtype=TYPES[c["h"]])
    elif op in ("gate", "gate_grad"):
        T, E = c["T"], c["E"]
        s["logits"] = randn(T, E) + randn(E, std=0.7)
        s["bias"] = randn(E, std=0.05) if c.get("bias") else None
        if op == "gate_grad":
            s["idx"] = torch.topk(s["logits"], c["k"], dim=1).indices.to(torch.int32)
            s["dw"] = randn(T, c["k"])
    elif op == "ortho":
        B, M, N = c["B"], c["M"], c["N"]
        r = max(1, min(M, N) // 8)
        # a gradient: a part of low rank from the step's tokens, and noise
        g = torch.matmul(randn(B, M, r), randn(B, r, N)) / math.sqrt(r) + randn(B, M, N, std=0.2)
        s["g"] = (1e-3 * g).to(TYPES[c["g"]])
    else:
        T, H, I, E, k = (c[x] for x in ("T", "H", "I", "E", "k"))
        s["x"] = randn(T, H, dtype=torch.bfloat16)
        s["wgu"] = torch.empty((E, 2 * I, H), dtype=torch.bfloat16, device=DEV)
        s["wd"] = torch.empty((E, H, I), dtype=torch.bfloat16, device=DEV)
        for e in range(E):
            s["wgu"][e] = randn(2 * I, H, dtype=torch.bfloat16, std=H ** -0.5)
            s["wd"][e] = randn(H, I, dtype=torch.bfloat16, std=I ** -0.5)
        top = torch.topk(randn(T, E), k, dim=1)
        s["idx"], s["w"] = top.indices.to(torch.int32), torch.softmax(top.values, dim=1)
        if op == "experts_grad":
            s["dout"] = randn(T, H)
        if own:  # the workspace that a user's program keeps
            from mixture_experts_ffn_gate_gb300 import moe_block as mb, moe_ffn as m
            new = m.new_workspace if op == "experts" else m.new_backward_workspace
            s["workspace"] = new(T, H, I, E, k)
            s["mb"] = mb
    if own and op == "ortho":
        from mixture_experts_ffn_gate_gb300 import moe_block as mb
        s["workspace"] = mb.new_orthogonalize_workspace(c["B"], c["M"], c["N"])
    if own and op == "norm_grad":
        from mixture_experts_ffn_gate_gb300 import moe_block as mb
        s["workspace"] = mb.new_rms_norm_backward_workspace(c["T"], c["H"])
    return s


def run(s):
    return _library(s) if own else _PLAIN[s["op"]](s)


# ------------------------------------------------------------------ the library
def _library(s):
    from mixture_experts_ffn_gate_gb300 import moe_block as mb
    op = s["op"]
    if op == "norm":
        r = mb.moe_rms_norm_forward(s["x"], s["weight"], residual=s["residual"], eps=EPS_NORM, mxfp8=s["mxfp8"])
        return dict(y=r.y, h=r.h, q=None if r.codes is None else _mx_values(r.codes, r.scales))
    if op == "norm_grad":
        dh, dweight = mb.moe_rms_norm_backward(s["h"], s["weight"], s["dy"], dres=s["dres"], eps=EPS_NORM,
                                               workspace=s["workspace"])
        return dict(dh=dh, dweight=dweight)
    if op == "gate":
        r = mb.moe_gate_forward(s["logits"], s["k"], bias=s["bias"], score=s["score"], groups=s["groups"],
                                topk_groups=s["topk_groups"], renormalize=s["renormalize"], scale=s["scale"],
                                counts=True)
        return dict(idx=r.topk_idx, w=r.topk_w, counts=r.counts)
    if op == "gate_grad":
        return mb.moe_gate_backward(s["logits"], s["idx"], s["dw"], score=s["score"], renormalize=s["renormalize"],
                                    scale=s["scale"])
    if op == "ortho":
        return mb.moe_orthogonalize(s["g"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS_ORTHO,
                                    workspace=s["workspace"])
    if op == "experts":
        return mb.moe_ffn_forward_routed(s["x"], s["idx"], s["w"], s["wgu"], s["wd"], workspace=s["workspace"])
    dx, dw, dwgu, dwd = mb.moe_ffn_backward_routed(s["x"], s["idx"], s["w"], s["wgu"], s["wd"], s["dout"],
                                                   workspace=s["workspace"])
    return dict(dx=dx, dw=dw, dwgu=dwgu, dwd=dwd)


def _mx_values(codes, scales):
    """The values that MXFP8 codes and scales stand for, which are BF16 numbers."""
    T, H = codes.shape
    f = torch.ldexp(torch.ones((), device=codes.device), scales[:, : H // 32].to(torch.int32) - 127)
    return (codes.view(torch.float8_e4m3fn).view(T, H // 32, 32).float() * f[..., None]).to(torch.bfloat16).view(T, H)


# ------------------------------------------------------------------ the plain forms
def _plain_norm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS_NORM) * s["weight"]
    out = dict(y=y.to(torch.bfloat16), h=None if s["residual"] is None else h.to(s["residual"].dtype), q=None)
    if s["mxfp8"]:
        T, H = y.shape
        b = y.view(T, H // 32, 32)
        amax = b.abs().amax(-1, keepdim=True)
        e = torch.where(amax > 0, torch.frexp(amax).exponent - 9, torch.zeros_like(amax, dtype=torch.int32))
        e = e.clamp(-126, 127)
        q = torch.ldexp(b, -e).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        out["q"] = torch.ldexp(q.float(), e).to(torch.bfloat16).view(T, H)
    return out


def _plain_norm_grad(s):
    h, dy, w = s["h"].float(), s["dy"].float(), s["weight"]
    r = torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS_NORM)
    n = h * r
    g = dy * w
    dh = r * (g - n * (g * n).mean(dim=1, keepdim=True))
    if s["dres"] is not None:
        dh = dh + s["dres"].float()
    return dict(dh=dh.to(s["h"].dtype), dweight=(dy * n).sum(dim=0))


def _scores(s, logits):
    if s["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(dim=1, keepdim=True))
    return e / e.sum(dim=1, keepdim=True)


def _plain_gate(s):
    logits, k, groups = s["logits"], s["k"], s["groups"]
    T, E = logits.shape
    scores = _scores(s, logits)
    # scores order the experts as the logits do; a bias moves the choice alone
    choice = logits if s["bias"] is None else scores + s["bias"]
    if groups > 1:
        v = choice.view(T, groups, E // groups)
        if s["bias"] is None:
            rank = v.amax(-1)
        else:
            rank = v.sort(dim=-1, descending=True).values[..., : 2].sum(-1)
        kept = rank.sort(dim=1, descending=True, stable=True).indices[:, : s["topk_groups"]]
        keep = torch.zeros((T, groups), dtype=torch.bool, device=logits.device).scatter_(1, kept, True)
        choice = torch.where(keep[..., None], v, torch.full_like(v, -math.inf)).view(T, E)
    idx = choice.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = scores.gather(1, idx)
    if s["renormalize"]:
        w = w / w.sum(dim=1, keepdim=True)
    counts = torch.zeros(E, dtype=torch.int32, device=logits.device)
    counts.scatter_add_(0, idx.reshape(-1), torch.ones(T * k, dtype=torch.int32, device=logits.device))
    return dict(idx=idx.to(torch.int32), w=w * s["scale"], counts=counts)


def _plain_gate_grad(s):
    logits, idx, dw = s["logits"], s["idx"].long(), s["dw"] * s["scale"]
    scores = _scores(s, logits)
    p = scores.gather(1, idx)
    if s["renormalize"]:
        total = p.sum(dim=1, keepdim=True)
        n = p / total
        dp = (dw - (dw * n).sum(dim=1, keepdim=True)) / total
    else:
        dp = dw
    if s["score"] == "sigmoid":
        return torch.zeros_like(logits).scatter_(1, idx, dp * p * (1.0 - p))
    ds = torch.zeros_like(logits).scatter_(1, idx, dp)
    return scores * (ds - (dp * p).sum(dim=1, keepdim=True))


def _plain_ortho(s):
    a, b, c = COEFFICIENTS
    x = s["g"].float()
    x = x / (x.square().sum(dim=(1, 2), keepdim=True).sqrt() + EPS_ORTHO)
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    for _ in range(STEPS):
        gram = torch.matmul(x, x.transpose(1, 2))
        x = a * x + torch.matmul(b * gram + c * torch.matmul(gram, gram), x)
    return (x.transpose(1, 2) if tall else x).to(torch.bfloat16).contiguous()


def _plain_experts(s):
    """A few tokens: the chosen experts' weights gathered for each.  More: every expert on every token,
    weighted by the routing (zero where it did not choose)."""
    x, I, E = s["x"].float(), s["I"], s["E"]
    if s["idx"].numel() < E:
        gu = torch.matmul(s["wgu"][s["idx"].long()].float(), x[:, None, :, None])[..., 0]
        g, u = gu[..., :I], gu[..., I:]
        act = g / (1.0 + torch.exp(-g)) * u * s["w"][..., None]
        return torch.matmul(s["wd"][s["idx"].long()].float(), act[..., None])[..., 0].sum(dim=1)
    coef = torch.zeros((x.shape[0], E), device=x.device).scatter_add_(1, s["idx"].long(), s["w"])
    gu = torch.matmul(x, s["wgu"].float().transpose(1, 2))
    g, u = gu[..., :I], gu[..., I:]
    act = g / (1.0 + torch.exp(-g)) * u * coef.t()[..., None]
    return torch.matmul(act, s["wd"].float().transpose(1, 2)).sum(dim=0)


def _plain_experts_grad(s):
    x, dout, I, E = s["x"].float(), s["dout"], s["I"], s["E"]
    coef = torch.zeros((x.shape[0], E), device=x.device).scatter_add_(1, s["idx"].long(), s["w"]).t()[..., None]
    wgu, wd = s["wgu"].float(), s["wd"].float()
    gu = torch.matmul(x, wgu.transpose(1, 2))
    g, u = gu[..., :I], gu[..., I:]
    sig = 1.0 / (1.0 + torch.exp(-g))
    act = g * sig * u
    q = torch.matmul(dout, wd)
    dw = (act * q).sum(-1).t().gather(1, s["idx"].long())
    da = coef * q
    dgu = torch.cat((da * u * sig * (1.0 + g * (1.0 - sig)), da * g * sig), dim=-1)
    dx = torch.matmul(dgu, wgu).sum(dim=0)
    dwgu = torch.matmul(dgu.transpose(1, 2), x)
    dwd = torch.matmul(dout.t(), coef * act)
    return dict(dx=dx, dw=dw, dwgu=dwgu, dwd=dwd)


_PLAIN = dict(norm=_plain_norm, norm_grad=_plain_norm_grad, gate=_plain_gate, gate_grad=_plain_gate_grad,
              ortho=_plain_ortho, experts=_plain_experts, experts_grad=_plain_experts_grad)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(c, seed):
    s = prepare(c, seed)
    return {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "gate": _exact_gate, "gate_grad": _exact_gate_grad,
            "ortho": _exact_ortho, "experts": _exact_experts, "experts_grad": _exact_experts}[c["op"]](s)


def _exact_norm(s):
    h = s["x"].double()
    if s["residual"] is not None:
        h += s["residual"].double()
    rms = (h.pow(2).sum(1) / h.shape[1] + EPS_NORM).sqrt()
    y = h / rms[:, None] * s["weight"].double()
    q = None
    if s["mxfp8"]:
        blocks = y.reshape(-1, 32)
        top = blocks.abs().max(dim=1, keepdim=True).values.clamp_min(1e-300)
        step = torch.exp2(torch.floor(torch.log2(top)) - 8)
        v = (blocks / step).clamp(-448, 448)
        # 3 mantissa bits above 2^-6, steps of 2^-9 below
        ulp = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
        q = (torch.round(v / ulp) * ulp * step).reshape(y.shape)
    return dict(y=y, h=None if s["residual"] is None else h, q=q)


def _exact_norm_grad(s):
    h, dy, w = (s[x].double() for x in ("h", "dy", "weight"))
    H = h.shape[1]
    ms = h.pow(2).sum(1, keepdim=True) / H + EPS_NORM
    # y = h w ms^-1/2;  d ms / d h = 2 h / H
    dms = -0.5 * (dy * w * h).sum(1, keepdim=True) * ms.pow(-1.5)
    dh = dy * w * ms.pow(-0.5) + dms * 2.0 * h / H
    if s["dres"] is not None:
        dh = dh + s["dres"].double()
    return dict(dh=dh, dweight=(dy * h * ms.pow(-0.5)).sum(0))


def _exact_scores(s):
    l = s["logits"].double()
    return torch.sigmoid(l) if s["score"] == "sigmoid" else torch.softmax(l, dim=1)


def _exact_gate(s):
    p = _exact_scores(s)
    T, E = p.shape
    order = s["logits"].double() if s["bias"] is None else p + s["bias"].double()
    if s["groups"] > 1:
        size = E // s["groups"]
        members = order.unflatten(1, (s["groups"], size))
        best = members.topk(1 if s["bias"] is None else min(2, size), dim=2).values.sum(2)
        limit = best.topk(s["topk_groups"], dim=1).values[:, -1:]
        order = members.masked_fill((best < limit)[..., None], -math.inf).flatten(1)
    chosen = order.topk(s["k"], dim=1).indices
    w = torch.gather(p, 1, chosen)
    if s["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    return dict(idx=None, w=s["scale"] * w, counts=None)


def _exact_gate_grad(s):
    logits = s["logits"].double().requires_grad_(True)
    p = torch.sigmoid(logits) if s["score"] == "sigmoid" else torch.softmax(logits, dim=1)
    w = p.gather(1, s["idx"].long())
    if s["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    with torch.enable_grad():
        (s["scale"] * w * s["dw"].double()).sum().backward()
    return logits.grad


def _exact_ortho(s):
    a, b, c = COEFFICIENTS
    out = []
    for g in s["g"]:
        x = g.double()
        x = x / (torch.linalg.matrix_norm(x) + EPS_ORTHO)
        for _ in range(STEPS):
            if x.shape[0] <= x.shape[1]:
                m = x @ x.T
                x = a * x + b * (m @ x) + c * (m @ (m @ x))
            else:
                m = x.T @ x
                x = a * x + b * (x @ m) + c * ((x @ m) @ m)
        out.append(x)
    return torch.stack(out)


def _exact_experts(s):
    x, idx, w, I, E = s["x"].double(), s["idx"].long(), s["w"].double(), s["I"], s["E"]
    grad = s["op"] == "experts_grad"
    out, dx, dw = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(w)
    dwgu = torch.zeros(s["wgu"].shape, dtype=torch.float64, device=x.device) if grad else None
    dwd = torch.zeros(s["wd"].shape, dtype=torch.float64, device=x.device) if grad else None
    for e in range(E):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        if not len(t):
            continue
        gate, up, down = s["wgu"][e, :I].double(), s["wgu"][e, I:].double(), s["wd"][e].double()
        xe, we = x[t], w[t, j][:, None]
        g, u = xe @ gate.T, xe @ up.T
        sig = torch.sigmoid(g)
        act = g * sig * u
        if not grad:
            out.index_add_(0, t, we * (act @ down.T))
            continue
        d = s["dout"].double()[t]
        back = d @ down
        dw[t, j] = (act * back).sum(1)
        dg = we * back * u * (sig + g * sig * (1 - sig))
        du = we * back * g * sig
        dx.index_add_(0, t, dg @ gate + du @ up)
        dwgu[e, :I], dwgu[e, I:] = dg.T @ xe, du.T @ xe
        dwd[e] = (we * d).T @ act
    return dict(dx=dx, dw=dw, dwgu=dwgu, dwd=dwd) if grad else out
