"""What a Mixture-of-Experts block's training step does after its gradients, as measured cases.

The gate's logits have a load-balance loss of their own; the step's gradients
are clipped by their common norm; AdamW updates many tensors at once.  Each
case is one call of one of them (``update``: the last two in a row):

  balance       the loss, the experts' counts and mean probabilities per sequence
  balance_grad  the logits' gradient, added to the one that the gate's weights gave
  grad_norm     the norm of many gradients and the factor that clips it
  adamw         one AdamW step of many tensors, its states in 32 or in 8 bits
  update        grad_norm, and the adamw step that takes its factor

``run`` computes them in plain torch operations in 32 bits, or with the
library (``own``).
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
COEF, Z_COEF = 1e-2, 1e-3
LR, BETAS, EPS, DECAY = 1e-3, (0.9, 0.95), 1e-8, 0.1
MAX_NORM = 1.0
BLOCK = 256      # elements that share a scale of an 8-bit state
TOP = 448.0      # the largest E4M3 value
LOWEST = 2.0 ** -9


def listed():
    return [
        # the block example's training step
        dict(name="balance_tiny", op="balance", T=64, E=16, k=4, score="sigmoid", z=False, S=0, pad=0),
        # a training step's tokens as one batch, with the loss that keeps the logits small
        dict(name="balance_step", op="balance", T=8191, E=128, k=8, score="softmax", z=True, S=0, pad=0),
        # many packed sequences of different lengths, rows behind the last one that belong to none
        dict(name="balance_packed", op="balance", T=131072, E=256, k=8, score="sigmoid", z=False, S=37, pad=1000),
        # one step's tokens over many experts
        dict(name="balance_grad_step", op="balance_grad", T=8191, E=384, k=8, score="softmax", z=True, S=0, pad=0,
             base=True),
        # the packed sequences again
        dict(name="balance_grad_packed", op="balance_grad", T=131072, E=256, k=8, score="sigmoid", z=False, S=37,
             pad=1000, base=True),
        # the gradients of the block example
        dict(name="grad_norm_tiny", op="grad_norm", layers=1, H=256, I=128, E=16, grad="f32"),
        # those of four layers with eight experts of the 2048-hidden size
        dict(name="grad_norm_layers", op="grad_norm", layers=4, H=2048, I=768, E=8, grad="f32"),
        # the block example's norm and router: what the orthogonalised update leaves
        dict(name="adamw_tiny", op="adamw", layers=1, H=256, I=0, E=16, w="bf16", master=False, grad="f32", bits=32),
        # BF16 experts with FP32 masters and states
        dict(name="adamw_master", op="adamw", layers=4, H=2048, I=768, E=8, w="bf16", master=True, grad="f32", bits=32),
        # the same with 8-bit states, gradients kept in BF16
        dict(name="adamw_8bit", op="adamw", layers=4, H=2048, I=768, E=8, w="bf16", master=True, grad="bf16", bits=8),
        # many layers of a small model, nothing a multiple of anything, FP32 weights and 8-bit states
        dict(name="adamw_many_odd", op="adamw", layers=48, H=501, I=87, E=3, w="f32", master=False, grad="f32", bits=8),
        # a whole step: norm, clipping and update of a small model
        dict(name="update_small", op="update", layers=12, H=512, I=250, E=4, w="bf16", master=True, grad="f32", bits=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["balance", "balance", "balance_grad", "balance_grad", "grad_norm", "adamw", "adamw", "adamw",
                     "update"])
    if op.startswith("balance"):
        E = rng.choice([3, 8, 16, 60, 64, 128, 160, 256, 384, 513, 1000])
        T = _log(rng, 1, min(131072, 131072 * 256 // E))
        S = rng.choice([0, 0, 1, _log(rng, 1, 200)])
        c = dict(op=op, T=T, E=E, k=min(E, rng.choice([1, 2, 4, 6, 8, 8, 10])), score=rng.choice(["softmax", "sigmoid"]),
                 z=rng.random() < 0.5, S=S, pad=rng.randint(0, T // 8) if S else 0)
        if op == "balance_grad":
            c["base"] = rng.random() < 0.6
        return c
    H, E, layers = _log(rng, 16, 2048), rng.randint(1, 16), _log(rng, 1, 48)
    most = 120_000_000 // (layers * E * 3 * H)
    I = _log(rng, 8, 768) if most >= 768 else max(1, min(768, most))
    c = dict(op=op, layers=layers, H=H, I=I, E=E, grad=rng.choice(["f32", "f32", "bf16"]))
    if op != "grad_norm":
        c["w"] = rng.choice(["bf16", "bf16", "f32"])
        c["master"] = c["w"] == "bf16" and rng.random() < 0.7
        c["bits"] = rng.choice([8, 32])
    return c


# ------------------------------------------------------------------ sizes
def _tensors(c):
    """(elements, whether an expert tensor) of each of the layers' tensors: norm and router weights, which are FP32
    with FP32 gradients and states, and the experts' two, in the case's types."""
    H, I, E = c["H"], c["I"], c["E"]
    layer = [(H, False), (E * H, False)] + ([(E * 2 * I * H, True), (E * H * I, True)] if I else [])
    return layer * c["layers"]


def _places(c, expert):
    """Where the tensors of one kind lie in their flat buffer, each at a multiple of BLOCK elements: (places, size)."""
    places, at = [], 0
    for n, e in _tensors(c):
        if e == expert:
            places.append((at, n))
            at += -(-n // BLOCK) * BLOCK
    return places, at


def work(c):
    size = {"bf16": 2, "f32": 4}
    if c["op"].startswith("balance"):
        T, E, k, S = c["T"], c["E"], c["k"], max(1, c["S"])
        if c["op"] == "balance":
            return {"bytes": 4 * T * E + 4 * T * k + 8 * S * E + 12, "flops": 6 * T * E}
        return {"bytes": 4 * T * E * (3 if c["base"] else 2) + 4 * S * E, "flops": 8 * T * E}
    bytes_, flops = 0, 0
    for n, expert in _tensors(c):
        g = size[c["grad"]] if expert else 4
        if c["op"] != "adamw":
            bytes_ += n * g
            flops += 2 * n
        if c["op"] != "grad_norm":
            if not expert:
                bytes_ += n * (g + 8 + 16)
            else:
                state = 16 if c["bits"] == 32 else 4 + 16 / BLOCK
                bytes_ += n * (g + state + (8 + size[c["w"]] if c["master"] else 2 * size[c["w"]]))
            flops += 15 * n
    return {"bytes": bytes_, "flops": flops}


# ------------------------------------------------------------------ inputs
def prepare(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def randn(*shape, dtype=torch.float32, std=1.0):
        return torch.randn(*shape, generator=gen, device=DEV).mul_(std).to(dtype)

    s = dict(c)
    if c["op"].startswith("balance"):
        T, E, k, S = c["T"], c["E"], c["k"], c["S"]
        # some experts are liked more than others: what the loss is for
        s["logits"] = randn(T, E) + randn(E, std=0.7)
        s["idx"] = torch.topk(s["logits"], k, dim=1).indices.to(torch.int32)
        s["offsets"] = None
        if S:  # packed sequences of any lengths, none included
            end = T - c["pad"]
            cuts = torch.randint(0, end + 1, (S - 1,), generator=gen, device=DEV).sort().values
            ends = torch.tensor([0, end], device=DEV)
            s["offsets"] = torch.cat((ends[:1], cuts, ends[1:])).to(torch.int32)
        if c["op"] == "balance_grad":
            s["dloss"] = torch.ones(1, device=DEV)
            s["base"] = randn(T, E, std=1e-4) if c["base"] else None
            s["counts"] = _counts(s, _sequence(s), max(1, S))
    else:
        kinds = {}
        for name, expert in (("plain", False), ("expert", True)):
            places, size = _places(c, expert)
            if not places:
                continue
            kinds[name] = b = dict(places=places)
            b["grad"] = randn(size, dtype=TYPES[c["grad"]] if expert else torch.float32, std=1e-3)
            if c["op"] == "grad_norm":
                continue
            w = randn(size, std=0.02)
            b["w"] = w.to(TYPES[c["w"]]) if expert else w
            b["master"] = w if expert and c["master"] else None
            b["bits"] = c["bits"] if expert else 32
            # states of a program that has run for a while
            b["m"], b["v"] = randn(size, std=3e-4), randn(size, std=1e-3).square_()
            b["m_scale"] = b["v_scale"] = None
            if b["bits"] == 8:
                b["m"], b["m_scale"] = _to_8bit(b["m"], False)
                b["v"], b["v_scale"] = _to_8bit(b["v"].sqrt_(), True)
        s["kinds"], s["step"] = kinds, 10
    if own:  # the workspaces and plans that a user's program keeps
        from mixture_experts_ffn_gate_gb300 import moe_block as mb
        if c["op"] == "balance":
            s["workspace"] = mb.new_balance_workspace(c["T"], c["E"], max(1, c["S"]))
        elif "kinds" in s:
            pieces = [(b, at, n) for b in s["kinds"].values() for at, n in b["places"]]
            grads = [b["grad"][at: at + n] for b, at, n in pieces]
            if c["op"] == "grad_norm":
                s["grads"] = mb.GradList(grads)
            else:
                s["plan"] = mb.AdamWPlan(
                    [b["w"][at: at + n] for b, at, n in pieces],
                    [mb.AdamWState(b["m"][at: at + n], b["v"][at: at + n],
                                   *(None if b["bits"] == 32 else b[x][at // BLOCK: (at + n + BLOCK - 1) // BLOCK]
                                     for x in ("m_scale", "v_scale"))) for b, at, n in pieces],
                    masters=[None if b["master"] is None else b["master"][at: at + n] for b, at, n in pieces],
                    weight_decay=[DECAY if b is s["kinds"].get("expert") else 0.0 for b, _, _ in pieces], grads=grads)
            if c["op"] != "adamw":
                s["workspace"] = mb.new_grad_norm_workspace(len(pieces))
    return s


def run(s):
    return _library(s) if own else _PLAIN[s["op"]](s)


# ------------------------------------------------------------------ the library
def _library(s):
    from mixture_experts_ffn_gate_gb300 import moe_block as mb
    op = s["op"]
    if op.startswith("balance"):
        how = dict(score=s["score"], coef=COEF, z_coef=Z_COEF if s["z"] else 0.0, seq_offsets=s["offsets"])
        if op == "balance":
            r = mb.moe_balance_loss_forward(s["logits"], s["idx"], workspace=s["workspace"], **how)
            return dict(loss=r.loss, counts=r.counts, prob=r.prob)
        return mb.moe_balance_loss_backward(s["logits"], s["counts"], s["k"], dloss=s["dloss"], dlogits_in=s["base"],
                                            **how)
    if op == "grad_norm":
        return mb.moe_grad_norm(s["grads"], max_norm=MAX_NORM, workspace=s["workspace"])
    clip = None
    if op == "update":
        clip = mb.moe_grad_norm(s["plan"], max_norm=MAX_NORM, workspace=s["workspace"])
    s["step"] += 1
    mb.moe_adamw_step(s["plan"], s["step"], lr=LR, betas=BETAS, eps=EPS, grad_scale=None if clip is None else clip[1:])
    return _answer(s, clip)


def _answer(s, clip):
    out = {name: {x: b[x] for x in ("w", "master", "m", "v", "m_scale", "v_scale")} for name, b in s["kinds"].items()}
    out["clip"] = clip
    return out


# ------------------------------------------------------------------ the plain forms
def _sequence(s):
    """The sequence of every row, S (or 1) for a row of none."""
    T = s["T"]
    if s["offsets"] is None:
        return torch.zeros(T, dtype=torch.long, device=DEV)
    return torch.searchsorted(s["offsets"][1:].long(), torch.arange(T, device=DEV), right=True)


def _counts(s, seq, S):
    """How many rows of each sequence chose each expert."""
    counts = torch.zeros((S + 1, s["E"]), dtype=torch.int32, device=DEV)
    counts.index_put_((seq[:, None].expand(s["idx"].shape), s["idx"].long()), torch.ones_like(s["idx"]),
                      accumulate=True)
    return counts[:S]


def _rows(s):
    """How many rows each sequence has, 32-bit floats."""
    if s["offsets"] is None:
        return torch.full((1,), float(s["T"]), device=DEV)
    return (s["offsets"][1:] - s["offsets"][:-1]).float()


def _probabilities(s):
    l = s["logits"]
    if s["score"] == "sigmoid":
        q = 1.0 / (1.0 + torch.exp(-l))
    else:
        q = torch.exp(l - l.amax(dim=1, keepdim=True))
    total = q.sum(dim=1, keepdim=True)
    return q, total, q / total


def _logsumexp(l):
    top = l.amax(dim=1, keepdim=True)
    e = torch.exp(l - top)
    total = e.sum(dim=1, keepdim=True)
    return top + torch.log(total), e / total


def _plain_balance(s):
    E, k, n, seq = s["E"], s["k"], _rows(s), _sequence(s)
    S = n.numel()
    _, _, p = _probabilities(s)
    sums = torch.zeros((S + 1, E), dtype=torch.float64, device=DEV).index_add_(0, seq, p.double())[:S].float()
    counts = _counts(s, seq, S)
    rows = n.sum().clamp_min(1.0)
    prob = sums / n.clamp_min(1.0)[:, None]
    f = counts / (k * n.clamp_min(1.0))[:, None]
    balance = (n / rows * E * (f * prob).sum(dim=1)).sum()
    z = torch.zeros((), device=DEV)
    if s["z"]:
        lse, _ = _logsumexp(s["logits"])
        z = ((lse[:, 0].square() * (seq < S)).double().sum() / rows).float()
    return dict(loss=torch.stack((COEF * balance + (Z_COEF if s["z"] else 0.0) * z, balance, z)), counts=counts,
                prob=prob)


def _plain_balance_grad(s):
    E, k, n, seq = s["E"], s["k"], _rows(s), _sequence(s)
    S = n.numel()
    rows = n.sum().clamp_min(1.0)
    q, total, p = _probabilities(s)
    share = torch.nn.functional.pad(s["counts"] / (k * n.clamp_min(1.0))[:, None], (0, 0, 0, 1))
    a = (s["dloss"] * COEF * E / rows * share)[seq]
    d = a - (a * p).sum(dim=1, keepdim=True)
    d = d * q * (1.0 - q) / total if s["score"] == "sigmoid" else d * p
    if s["z"]:
        lse, e = _logsumexp(s["logits"])
        d = d + s["dloss"] * 2.0 * Z_COEF / rows * lse * e
    d = d * (seq < S)[:, None]
    return d if s["base"] is None else d + s["base"]


def _pieces(s):
    return [(b, at, n) for b in s["kinds"].values() for at, n in b["places"]]


def _plain_grad_norm(s):
    squares = torch.stack([b["grad"][at: at + n].float().square().sum() for b, at, n in _pieces(s)])
    norm = squares.sum().sqrt()
    return torch.stack((norm, torch.where(norm > MAX_NORM, MAX_NORM / norm, torch.ones_like(norm))))


def _to_8bit(x, up):
    """E4M3 codes of x [n] and the scale of each BLOCK elements; ``up``: what is not zero stays so."""
    n = x.numel()
    b = torch.nn.functional.pad(x, (0, -n % BLOCK)).view(-1, BLOCK)
    scale = (b.abs().amax(dim=1) / TOP).clamp_min(2.0 ** -126)
    q = (b / scale[:, None]).clamp(-TOP, TOP)
    if up:
        q = torch.where(b > 0, q.clamp_min(LOWEST), q)
    return q.to(torch.float8_e4m3fn).view(-1)[:n], scale


def _from_8bit(codes, scale):
    return codes.float() * scale.repeat_interleave(BLOCK)[: codes.numel()]


def _plain_adamw(s, clip=None):
    s["step"] += 1
    bc1, bc2 = 1.0 - BETAS[0] ** s["step"], 1.0 - BETAS[1] ** s["step"]
    for b, at, n in _pieces(s):
        here, scales = slice(at, at + n), slice(at // BLOCK, (at + n + BLOCK - 1) // BLOCK)
        g = b["grad"][here].float()
        if clip is not None:
            g = g * clip[1]
        m, v = b["m"][here], b["v"][here]
        if b["bits"] == 8:
            m, v = _from_8bit(m, b["m_scale"][scales]), _from_8bit(v, b["v_scale"][scales]).square()
        m = BETAS[0] * m + (1.0 - BETAS[0]) * g
        v = BETAS[1] * v + (1.0 - BETAS[1]) * g * g
        w = b["w" if b["master"] is None else "master"][here].float()
        decay = DECAY if b is s["kinds"].get("expert") else 0.0
        w = w * (1.0 - LR * decay) - LR * (m / bc1) / ((v / bc2).sqrt() + EPS)
        b["w"][here] = w.to(b["w"].dtype)
        if b["master"] is not None:
            b["master"][here] = w
        if b["bits"] == 8:
            b["m"][here], b["m_scale"][scales] = _to_8bit(m, False)
            b["v"][here], b["v_scale"][scales] = _to_8bit(v.sqrt(), True)
        else:
            b["m"][here], b["v"][here] = m, v
    return _answer(s, clip)


def _plain_update(s):
    return _plain_adamw(s, _plain_grad_norm(s))


_PLAIN = dict(balance=_plain_balance, balance_grad=_plain_balance_grad, grad_norm=_plain_grad_norm, adamw=_plain_adamw,
              update=_plain_update)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(c, seed):
    s = prepare(c, seed)
    if c["op"].startswith("balance"):
        return _exact_balance(s)
    if c["op"] == "grad_norm":
        return _exact_clip(s)
    return _exact_adamw(s, _exact_clip(s) if c["op"] == "update" else None)


def _exact_balance(s):
    """The loss sequence by sequence; its gradient by automatic differentiation."""
    grad = s["op"] == "balance_grad"
    l = s["logits"].double().requires_grad_(grad)
    p = torch.softmax(l, 1) if s["score"] == "softmax" else torch.nn.functional.normalize(torch.sigmoid(l), p=1, dim=1)
    bounds = [0, s["T"]] if s["offsets"] is None else s["offsets"].tolist()
    total = bounds[-1] - bounds[0]
    balance, z = l.new_zeros(()), l.new_zeros(())
    prob = l.new_zeros((len(bounds) - 1, s["E"]))
    for i, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        if lo == hi:
            continue
        chosen = torch.bincount(s["idx"][lo:hi].flatten().long(), minlength=s["E"]).double() / (s["k"] * (hi - lo))
        mean = p[lo:hi].mean(0)
        prob[i] = mean.detach()
        balance = balance + (hi - lo) / total * s["E"] * torch.dot(chosen, mean)
    if s["z"]:
        z = torch.logsumexp(l[bounds[0]: bounds[-1]], 1).pow(2).sum() / max(total, 1)
    loss = COEF * balance + Z_COEF * z
    if not grad:
        return dict(loss=torch.stack((loss, balance, z)), counts=None, prob=prob)
    d = torch.zeros_like(l)
    if loss.requires_grad:
        d = torch.autograd.grad(loss, l, s["dloss"].double()[0])[0]
    return d if s["base"] is None else d + s["base"].double()


def _exact_clip(s):
    total = sum(float(b["grad"][at: at + n].double().pow(2).sum()) for b, at, n in _pieces(s))
    norm = math.sqrt(total)
    return torch.tensor([norm, min(1.0, MAX_NORM / norm)], dtype=torch.float64)


def _exact_adamw(s, clip):
    """Before what is kept in fewer bits is rounded; the codes' place holds the values over their scale."""
    t = s["step"] + 1
    out = {}
    for name, b in s["kinds"].items():
        out[name] = r = {x: None if b[x] is None else b[x].double() for x in ("w", "master", "m", "v", "m_scale",
                                                                             "v_scale")}
        for at, n in b["places"]:
            here, blocks = slice(at, at + n), slice(at // BLOCK, -(-(at + n) // BLOCK))
            g = b["grad"][here].double() * (1.0 if clip is None else float(clip[1]))
            m, v = r["m"][here], r["v"][here]
            if b["bits"] == 8:
                which = torch.arange(n, device=DEV) // BLOCK
                m, v = m * r["m_scale"][blocks][which], (v * r["v_scale"][blocks][which]).pow(2)
            m, v = torch.lerp(g, m, BETAS[0]), torch.lerp(g * g, v, BETAS[1])
            w = r["w" if b["master"] is None else "master"][here]
            step = (m / (1 - BETAS[0] ** t)) / (torch.sqrt(v / (1 - BETAS[1] ** t)) + EPS)
            w = w - LR * (step + (DECAY if name == "expert" else 0.0) * w)
            r["w"][here] = w
            if b["master"] is not None:
                r["master"][here] = w
            if b["bits"] == 8:
                for x, y in (("m", m), ("v", torch.sqrt(v))):
                    top = torch.zeros(int(which[-1]) + 1, dtype=torch.float64, device=DEV)
                    top = top.scatter_reduce(0, which, y.abs(), "amax").div(TOP).clamp_min(2.0 ** -126)
                    r[x][here], r[x + "_scale"][blocks] = y / top[which], top
            else:
                r["m"][here], r["v"][here] = m, v
    out["clip"] = clip
    return out
