"""Cases of the operators that stand around the expert layer in a training
step: layer norm, softmax cross entropy over a vocabulary, and the global
gradient norm with clipping.

``run`` computes a case in plain torch operations (``own`` false) or through
the library (``own`` true); ``exact`` is the same in 64 bits.  Hidden sizes
are those of the layer's workloads (2048 and 4096) or generic ones.
"""
import math
import random

import torch

own = False

EPS = 1e-5
IGNORE = -100
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token in front of the layer while generating: launch latency
        dict(name="norm_one_token", op="norm", T=1, H=4096, dtype="bf16", wtype="bf16", pad=0, train=False),
        # one training step's worth of tokens, forward and backward
        dict(name="norm_train", op="norm", T=16384, H=4096, dtype="bf16", wtype="bf16", pad=0, train=True),
        # fp32 activations and rows that are a slice of a wider buffer
        dict(name="norm_f32_strided", op="norm", T=5003, H=1536, dtype="f32", wtype="f32", pad=520, train=True),
        # an odd width: no row but the first starts at an aligned address
        dict(name="norm_odd_width", op="norm", T=4097, H=2049, dtype="bf16", wtype="f32", pad=0, train=True),
        # scoring a few tokens: the time to read the output weights once
        dict(name="xent_few_tokens", op="xent", T=7, H=2048, V=32000, masked=0.0, train=False),
        # scoring of a long batch: loss only
        dict(name="xent_eval", op="xent", T=16384, H=2048, V=65536, masked=0.1, train=False),
        # a small ragged step: odd token count and vocabulary, half of it masked (prompts)
        dict(name="xent_ragged", op="xent", T=1001, H=1032, V=10007, masked=0.5, train=True),
        # a step of a mid-size model with an odd vocabulary
        dict(name="xent_train_mid", op="xent", T=4096, H=2048, V=50001, masked=0.05, train=True),
        # a step of a large one
        dict(name="xent_train", op="xent", T=8192, H=4096, V=131072, masked=0.0, train=True),
        # gradients of a small model: latency
        dict(name="clip_small", op="clip", tensors=24, numel=200_003, dtype="f32", layer=False, clip=True),
        # the norm alone (logging), many tensors of odd sizes
        dict(name="norm_of_many", op="clip", tensors=300, numel=120_000_000, dtype="bf16", layer=False, clip=False),
        # the weight gradients of one expert layer of the 30B shape, its router and norms
        dict(name="clip_layer", op="clip", tensors=6, numel=604_000_000, dtype="bf16", layer=True, clip=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "xent", "clip"])
    if op == "norm":
        dtype = rng.choice(["bf16", "f32"])
        H = _log(rng, 64, 16384)
        if rng.random() < 0.7:
            H = max(8, H // 8 * 8)
        most = 16384 * 4096 // H if dtype == "bf16" else 8192 * 4096 // H
        return dict(op=op, T=_log(rng, 1, min(65536, most)), H=H, dtype=dtype, wtype=rng.choice([dtype, "f32"]),
                    pad=rng.choice([0, 0, 8, 24, 7]), train=rng.random() < 0.75)
    if op == "xent":
        H = 8 * _log(rng, 16, 512)
        V = _log(rng, 1000, 131072)
        most = min(16384, 4096 * 50001 * 2048 * 2 // (V * H))
        return dict(op=op, T=_log(rng, 1, most), H=H, V=V, masked=rng.choice([0.0, 0.1, 0.5]),
                    train=rng.random() < 0.7)
    clip = rng.random() < 0.75
    return dict(op=op, tensors=_log(rng, 1, 60 if clip else 400), numel=_log(rng, 50_000, 400_000_000),
                dtype=rng.choice(["bf16", "f32", "mixed"]), layer=False, clip=clip)


def _gen(seed, extra=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + extra)
    return g


def _randn(g, shape, dtype, scale=1.0):
    """N(0, scale^2), drawn in pieces so that no fp32 copy of a large tensor is needed."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    step = 1 << 27
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device="cuda").mul_(scale)
    return out


def _strided(t, pad):
    """The same rows as a view of a buffer that is `pad` columns wider."""
    if not pad:
        return t
    wide = torch.zeros((t.shape[0], t.shape[1] + pad), dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def _sizes(case):
    """(elements, type) of each gradient tensor of a clip case."""
    if case["layer"]:
        E, H, I = 128, 2048, 768
        return [(E * H * 2 * I, "bf16"), (E * I * H, "bf16"), (E * H, "f32"), (H, "f32"), (H, "f32"), (31_991, "bf16")]
    rng = random.Random(case["tensors"] * 7919 + case["numel"])
    w = [math.exp(rng.uniform(0, 5)) for _ in range(case["tensors"])]
    total = sum(w)
    kinds = {"bf16": ["bf16"], "f32": ["f32"], "mixed": ["bf16", "f32"]}[case["dtype"]]
    return [(max(1, int(case["numel"] * x / total)), rng.choice(kinds)) for x in w]


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    if case["op"] == "norm":
        T, H, dt, wt = case["T"], case["H"], DTYPES[case["dtype"]], DTYPES[case["wtype"]]
        # residual-stream rows: channels of different size and a mean that is not zero
        scale = torch.exp(0.5 * torch.randn(H, generator=g, device="cuda"))
        shift = 0.3 * torch.randn(H, generator=g, device="cuda")
        x = (torch.randn((T, H), generator=g, device="cuda") * scale + shift).to(dt)
        s["x"] = _strided(x, case["pad"])
        s["gamma"] = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(wt)
        s["beta"] = (0.1 * torch.randn(H, generator=g, device="cuda")).to(wt)
        if case["train"]:
            s["dy"] = _strided(_randn(g, (T, H), dt), case["pad"])
        if own:
            from mixture_experts_layer_18_gb300.training import LayerNorm
            s["norm"] = LayerNorm(T, H, dtype=dt, weight_dtype=wt, eps=EPS, backward=case["train"])
            s["io"] = s["norm"].empty_io()
    elif case["op"] == "xent":
        T, H, V = case["T"], case["H"], case["V"]
        W = _randn(g, (V, H), torch.bfloat16, 2.0 / math.sqrt(H))
        targets = torch.randint(0, V, (T,), generator=g, device="cuda")
        # hidden states after a norm; some tokens are well predicted, most are not
        sure = torch.rand((T, 1), generator=g, device="cuda") ** 2 * 3
        x = torch.randn((T, H), generator=g, device="cuda") + 1.25 * sure * W[targets].float()
        s["X"], s["W"] = x.to(torch.bfloat16), W
        if case["masked"]:
            targets[torch.rand(T, generator=g, device="cuda") < case["masked"]] = IGNORE
        s["targets"] = targets
        s["dloss"] = torch.ones(1, device="cuda")
        if own:
            from mixture_experts_layer_18_gb300.training import CrossEntropy
            s["xent"] = CrossEntropy(T, H, V, ignore_index=IGNORE, backward=case["train"])
            s["io"] = s["xent"].empty_io() if case["train"] else None
    else:
        s["grads"] = [_randn(g, (n,), DTYPES[kind], 10.0 ** (-(i % 3))) for i, (n, kind) in enumerate(_sizes(case))]
        s["max_norm"] = 1.0
        if own:
            from mixture_experts_layer_18_gb300.training import GradClip
            s["out"] = [torch.empty_like(t) for t in s["grads"]] if case["clip"] else None
            s["clip"] = GradClip(s["grads"], out=s["out"])
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _norm_own, "xent": _xent_own, "clip": _clip_own}[op](state)
    return {"norm": _norm_plain, "xent": _xent_plain, "clip": _clip_plain}[op](state)


def _norm_own(s):
    n, io = s["norm"], s["io"]
    n.forward(s["x"], s["gamma"], s["beta"], io["y"])
    if not s["case"]["train"]:
        return dict(y=io["y"])
    n.backward(s["dy"], s["x"], s["gamma"], io["dx"], io["dgamma"], io["dbeta"])
    return dict(y=io["y"], dx=io["dx"], dgamma=io["dgamma"], dbeta=io["dbeta"])


def _xent_own(s):
    c = s["xent"]
    c.forward(s["X"], s["W"], s["targets"])
    out = dict(loss=c.loss, mean=c.mean)
    if s["case"]["train"]:
        c.backward(s["X"], s["W"], s["targets"], s["dloss"], s["io"]["dX"], s["io"]["dW"], reduction="mean")
        out.update(dX=s["io"]["dX"], dW=s["io"]["dW"])
    return out


def _clip_own(s):
    c = s["clip"]
    if not s["case"]["clip"]:
        c.measure()
        return dict(norm=c.norm)
    c.clip(s["max_norm"])
    return dict(norm=c.norm, out=s["out"])


def _norm_plain(s):
    x, gamma, beta = s["x"].float(), s["gamma"].float(), s["beta"].float()
    mean = x.mean(1, keepdim=True)
    c = x - mean
    rstd = 1.0 / torch.sqrt((c * c).mean(1, keepdim=True) + EPS)
    xh = c * rstd
    out = dict(y=(xh * gamma + beta).to(s["x"].dtype))
    if s["case"]["train"]:
        dy = s["dy"].float()
        g = dy * gamma
        dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        out.update(dx=dx.to(s["x"].dtype), dgamma=(dy * xh).sum(0).to(s["gamma"].dtype),
                   dbeta=dy.sum(0).to(s["gamma"].dtype))
    return out


def _xent_plain(s):
    X, W, t = s["X"].float(), s["W"].float(), s["targets"]
    kept = t != IGNORE
    safe = torch.where(kept, t, torch.zeros_like(t))
    z = X @ W.T
    top = z.max(1, keepdim=True).values
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    loss = torch.log(total) + top - z.gather(1, safe[:, None])
    loss = torch.where(kept, loss[:, 0], torch.zeros_like(loss[:, 0]))
    count = kept.sum().clamp(min=1)
    out = dict(loss=loss, mean=loss.sum() / count)
    if s["case"]["train"]:
        del z
        scale = torch.where(kept, s["dloss"] / count, torch.zeros_like(loss))[:, None]
        dz = e.div_(total).mul_(scale)
        dz.scatter_add_(1, safe[:, None], -scale)
        out.update(dX=(dz @ W).to(s["X"].dtype), dW=(dz.T @ X).to(s["W"].dtype))
    return out


def _clip_plain(s):
    norm = torch.stack([(t.float() * t.float()).sum() for t in s["grads"]]).sum().sqrt()
    if not s["case"]["clip"]:
        return dict(norm=norm)
    c = torch.where(norm > s["max_norm"], s["max_norm"] / norm, torch.ones_like(norm))
    return dict(norm=norm, out=[(t.float() * c).to(t.dtype) for t in s["grads"]])


def work(case):
    if case["op"] == "norm":
        es, ws = (2 if case[k] == "bf16" else 4 for k in ("dtype", "wtype"))
        T, H = case["T"], case["H"]
        n = 4 if case["train"] else 2            # x, y; dy, dx
        w = 4 if case["train"] else 2            # gamma, beta; dgamma, dbeta
        return {"bytes": n * T * H * es + w * H * ws, "flops": (20 if case["train"] else 8) * T * H}
    if case["op"] == "xent":
        T, H, V = case["T"], case["H"], case["V"]
        n = 2 if case["train"] else 1            # X, W; dX, dW
        # the logits; in training also dX and dW (forming the logits twice is no part of it)
        return {"bytes": 2 * n * (T * H + V * H) + 12 * T, "flops": (6 if case["train"] else 2) * T * H * V}
    b = sum(n * (2 if kind == "bf16" else 4) for n, kind in _sizes(case))
    return {"bytes": (2 if case["clip"] else 1) * b, "flops": 2 * sum(n for n, _ in _sizes(case))}


# ------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _norm_exact(s)
    if case["op"] == "xent":
        if work(case)["flops"] > 8e12:
            return None
        return _xent_exact(s)
    return _clip_exact(s)


def _norm_exact(s):
    train = s["case"]["train"]
    T, H = s["x"].shape
    gamma, beta = s["gamma"].double(), s["beta"].double()
    y = torch.empty((T, H), dtype=torch.float64, device="cuda")
    dx = torch.empty_like(y) if train else None
    dgamma, dbeta = torch.zeros_like(gamma), torch.zeros_like(gamma)
    rows = max(1, (1 << 24) // H)
    for i in range(0, T, rows):
        x = s["x"][i:i + rows].double()
        mean = x.sum(1) / H
        var = torch.einsum("th,th->t", x - mean[:, None], x - mean[:, None]) / H
        inv = (var + EPS).pow(-0.5)
        xh = torch.einsum("th,t->th", x - mean[:, None], inv)
        y[i:i + rows] = xh * gamma + beta
        if train:
            dy = s["dy"][i:i + rows].double()
            # the row's Jacobian (I - 1 1^T / H - xh xh^T / H) / sigma applied to gamma * dy
            a = dy @ gamma / H
            b = torch.einsum("th,th,h->t", dy, xh, gamma) / H
            dx[i:i + rows] = (gamma * dy - a[:, None] - b[:, None] * xh) * inv[:, None]
            dgamma += torch.einsum("th,th->h", dy, xh)
            dbeta += torch.einsum("th->h", dy)
    return dict(y=y, dx=dx, dgamma=dgamma, dbeta=dbeta) if train else dict(y=y)


def _xent_exact(s):
    train = s["case"]["train"]
    T, V = s["X"].shape[0], s["W"].shape[0]
    W = s["W"].double()
    loss = torch.zeros(T, dtype=torch.float64, device="cuda")
    count = int((s["targets"] >= 0).sum())
    dX = torch.zeros((T, W.shape[1]), dtype=torch.float64, device="cuda") if train else None
    dW = torch.zeros_like(W) if train else None
    rows = max(1, (1 << 28) // V)
    for i in range(0, T, rows):
        t = s["targets"][i:i + rows]
        x = s["X"][i:i + rows].double()
        at = torch.nonzero(t >= 0)[:, 0]
        if not len(at):
            continue
        z = x[at] @ W.mT
        logp = torch.log_softmax(z, dim=1)
        pick = logp[torch.arange(len(at), device="cuda"), t[at]]
        loss[i + at] = -pick
        if train:
            d = logp.exp()
            d[torch.arange(len(at), device="cuda"), t[at]] -= 1
            d *= float(s["dloss"][0]) / count
            dX[i + at] = d @ W
            dW += d.mT @ x[at]
    out = dict(loss=loss, mean=loss.sum() / max(1, count))
    if train:
        out.update(dX=dX, dW=dW)
    return out


def _clip_exact(s):
    total, step = 0.0, 1 << 26
    for t in s["grads"]:
        for i in range(0, t.numel(), step):
            d = t[i:i + step].double()
            total += float(torch.dot(d, d))
    norm = math.sqrt(total)
    if not s["case"]["clip"]:
        return dict(norm=norm)
    c = min(1.0, s["max_norm"] / norm) if norm else 1.0
    return dict(norm=norm, out=[t.double() * c for t in s["grads"]])
