"""Cases of more operators of a training step around the expert layer: routing
by scores (softmax or sigmoid, a bias for balance, groups of experts), the
root-mean-square norm with the residual's addition and an MXFP8 output, and
the layer's activations kept in 8 bits for its backward pass.

``run`` computes a case in plain torch operations (``own`` false) or through
the library (``own`` true); ``exact`` is the same in 64 bits.  Hidden sizes,
experts and top-k are those of the layer's workloads or generic ones.
"""
import math

import torch

own = False

EPS = 1e-6
ALIGN = 128          # an expert's rows start at multiples of this
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token while generating: launch latency of the router and the permutation
        dict(name="route_one_token", op="route", T=1, E=256, k=8, score="sigmoid", bias=True, groups=8, top_groups=4,
             group_top=2, renorm=True, dtype="f32", pad=0, train=False),
        # a step's tokens: sigmoid scores, balance bias, half of the groups, with backward and the bias' update
        dict(name="route_train", op="route", T=16384, E=256, k=8, score="sigmoid", bias=True, groups=8, top_groups=4,
             group_top=2, renorm=True, dtype="f32", pad=0, train=True),
        # an odd number of experts and tokens, bf16 logits in a wider buffer, gates not renormalised (dense gradient)
        dict(name="route_ragged", op="route", T=1001, E=60, k=6, score="softmax", bias=False, groups=1, top_groups=1,
             group_top=1, renorm=False, dtype="bf16", pad=4, train=True),
        # a long batch over the layer's 128 experts with a bias, no groups
        dict(name="route_long", op="route", T=65536, E=128, k=8, score="softmax", bias=True, groups=1, top_groups=1,
             group_top=1, renorm=True, dtype="f32", pad=0, train=False),
        # one token in front of the layer: latency
        dict(name="rms_one_token", op="rms", T=1, H=4096, dtype="bf16", wtype="bf16", pad=0, residual=True, y=True,
             mx=True, train=False),
        # a step's tokens: the sum, its norm in bf16 for the layer and in 8 bits for the backward, and back
        dict(name="rms_train", op="rms", T=16384, H=4096, dtype="bf16", wtype="f32", pad=0, residual=True, y=True,
             mx=True, train=True),
        # fp32 rows of an odd width in a wider buffer
        dict(name="rms_odd_width", op="rms", T=5003, H=1999, dtype="f32", wtype="f32", pad=2, residual=True, y=True,
             mx=False, train=True),
        # the 8-bit output alone, no residual
        dict(name="rms_encode", op="rms", T=4097, H=2048, dtype="bf16", wtype="bf16", pad=0, residual=False, y=False,
             mx=True, train=False),
        # the layer's smallest workload, fp32: latency
        dict(name="ckpt_tiny", op="ckpt", T=256, H=128, E=8, k=2, I=64, dtype="f32"),
        # odd token count, few experts
        dict(name="ckpt_ragged", op="ckpt", T=1001, H=576, E=24, k=3, I=320, dtype="bf16"),
        # a step of the 30B layer
        dict(name="ckpt_30b", op="ckpt", T=16384, H=2048, E=128, k=8, I=768, dtype="bf16"),
        # a step of the 235B layer
        dict(name="ckpt_235b", op="ckpt", T=16384, H=4096, E=128, k=8, I=1536, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "rms", "ckpt"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        size = _log(rng, max(2, 8 // groups), 512 // groups)
        top_groups = rng.randint(1, groups)
        E = groups * size
        k = _log(rng, 1, min(16, top_groups * size))
        return dict(op=op, T=_log(rng, 1, min(65536, 16384 * 256 // E)), E=E, k=k, score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.7, groups=groups, top_groups=top_groups, group_top=rng.randint(1, 2),
                    renorm=rng.random() < 0.7, dtype=rng.choice(["f32", "f32", "bf16"]), pad=rng.choice([0, 0, 4, 3]),
                    train=rng.random() < 0.7)
    if op == "rms":
        dtype, mx = rng.choice(["bf16", "f32"]), rng.random() < 0.6
        H = _log(rng, 64, 16384)
        H = max(32, H // 32 * 32) if mx else H if rng.random() < 0.4 else max(8, H // 8 * 8)
        most = 16384 * 4096 // H if dtype == "bf16" else 8192 * 4096 // H
        return dict(op=op, T=_log(rng, 1, min(65536, most)), H=H, dtype=dtype, wtype=rng.choice([dtype, "f32"]),
                    pad=0 if mx else rng.choice([0, 0, 8, 7]), residual=rng.random() < 0.7, y=not mx or rng.random() < 0.7,
                    mx=mx, train=rng.random() < 0.7)
    H, I = 64 * _log(rng, 1, 64), 64 * _log(rng, 1, 24)
    E = _log(rng, 2, 256)
    k = _log(rng, 1, min(8, E))
    most = 16384 * 8 * 2048 // (k * max(H, 2 * I))
    return dict(op=op, T=_log(rng, 1, min(16384, most)), H=H, E=E, k=k, I=I, dtype=rng.choice(["bf16", "bf16", "f32"]))


def _gen(seed, extra=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + extra)
    return g


def _strided(t, pad):
    """The same rows as a view of a buffer that is `pad` columns wider."""
    if not pad:
        return t
    wide = torch.zeros((t.shape[0], t.shape[1] + pad), dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def _permutation(idx, E):
    """counts, padded_offsets, row_of_assign and assign_of_row of idx [T, k]:
    an expert's rows in the order of the assignments, from a multiple of ALIGN."""
    n, dev = idx.numel(), idx.device
    flat = idx.reshape(-1).long()
    counts = torch.zeros(E, dtype=torch.long, device=dev).scatter_add_(0, flat, torch.ones_like(flat))
    padded = (counts + ALIGN - 1) // ALIGN * ALIGN
    zero = torch.zeros(1, dtype=torch.long, device=dev)
    start, first = torch.cat([zero, padded.cumsum(0)]), torch.cat([zero, counts.cumsum(0)])
    order = torch.sort(flat, stable=True).indices
    e = flat[order]
    row = start[e] + torch.arange(n, device=dev) - first[e]
    row_of = torch.empty(n, dtype=torch.int32, device=dev)
    row_of[order] = row.int()
    assign_of = torch.full((n + ALIGN * E,), -1, dtype=torch.int32, device=dev)
    assign_of[row] = order.int()
    return counts.int(), start.int(), row_of, assign_of


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    if case["op"] == "route":
        T, E, k, dt = case["T"], case["E"], case["k"], DTYPES[case["dtype"]]
        # hidden states against router rows: some experts are liked by most tokens
        logits = torch.randn((T, E), generator=g, device="cuda") + 0.4 * torch.randn(E, generator=g, device="cuda")
        s["logits"] = _strided(logits.to(dt), case["pad"])
        # a bias after some hundred updates of 1e-3
        s["bias"] = 1e-3 * torch.randint(-60, 61, (E,), generator=g, device="cuda").float() if case["bias"] else None
        s["scale"], s["rate"] = 2.5 if case["renorm"] else 1.0, 1e-3
        if case["train"]:
            s["dgate"] = torch.randn((T, k), generator=g, device="cuda")
        if own:
            from mixture_experts_layer_18_gb300.training import Router
            s["router"] = Router(T, E, k, score=case["score"], groups=case["groups"], top_groups=case["top_groups"],
                                 group_top=case["group_top"], renormalise=case["renorm"], scale=s["scale"], dtype=dt)
            s["dlogits"] = torch.empty((T, E), dtype=dt, device="cuda")
            s["new_bias"] = torch.empty_like(s["bias"]) if case["bias"] else None
    elif case["op"] == "rms":
        T, H, dt, wt = case["T"], case["H"], DTYPES[case["dtype"]], DTYPES[case["wtype"]]
        # residual-stream rows (channels of different size) and a block's output
        scale = torch.exp(0.5 * torch.randn(H, generator=g, device="cuda"))
        s["x"] = _strided((torch.randn((T, H), generator=g, device="cuda") * scale).to(dt), case["pad"])
        if case["residual"]:
            s["residual"] = _strided((0.5 * torch.randn((T, H), generator=g, device="cuda")).to(dt), case["pad"])
        s["gamma"] = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(wt)
        if case["train"]:
            s["dy"] = _strided(torch.randn((T, H), generator=g, device="cuda").to(dt), case["pad"])
            s["dh"] = _strided(torch.randn((T, H), generator=g, device="cuda").to(dt), case["pad"])
        if own:
            from mixture_experts_layer_18_gb300.training import MXRows, RMSNorm
            s["norm"] = RMSNorm(T, H, dtype=dt, weight_dtype=wt, eps=EPS, backward=case["train"])
            io = s["norm"].empty_io()
            s["io"] = {n: _strided(v, case["pad"]) if v.ndim == 2 else v for n, v in io.items()}
            if case["mx"]:
                s["mx"], s["y8"] = MXRows(T, H), torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    else:
        T, H, E, I, k, dt = case["T"], case["H"], case["E"], case["I"], case["k"], DTYPES[case["dtype"]]
        s["X"] = torch.randn((T, H), generator=g, device="cuda").to(dt)
        # tokens in another order for each seed: an expert has as many rows every time
        logits = torch.randn((T, E), generator=_gen(T * 7919 + E), device="cuda")
        logits = logits[torch.randperm(T, generator=g, device="cuda")]
        top = torch.sort(logits, dim=1, descending=True, stable=True)
        idx = top.indices[:, :k]
        e = torch.exp(top.values[:, :k] - top.values[:, :1])
        s["gate"] = e / e.sum(1, keepdim=True)
        _, start, s["row_of"], s["assign_of"] = _permutation(idx, E)
        s["rows"] = int(start[-1])
        # the gate/up projections of unit rows, some channels larger; rows that pad an expert's are zero
        h = torch.empty((s["rows"], 2 * I), dtype=dt, device="cuda")
        wide = torch.exp(0.4 * torch.randn(2 * I, generator=g, device="cuda"))
        for i in range(0, s["rows"], 16384):
            n = min(16384, s["rows"] - i)
            h[i:i + n] = torch.randn((n, 2 * I), generator=g, device="cuda") * wide
        h[s["assign_of"][:s["rows"]] < 0] = 0
        s["h13"] = h
        if own:
            from mixture_experts_layer_18_gb300.layer import MoELayer
            L = MoELayer(T, H, E, I, k, mode="bf16" if dt == torch.bfloat16 else "f32", backward=False)
            L.route(logits)
            L.h13[:s["rows"]] = h
            s["layer"], s["ckpt"] = L, L.checkpoint()
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        return {"route": _route_own, "rms": _rms_own, "ckpt": _ckpt_own}[op](state)
    return {"route": _route_plain, "rms": _rms_plain, "ckpt": _ckpt_plain}[op](state)


# ------------------------------------------------------------ the library
def _route_own(s):
    r = s["router"]
    r.forward(s["logits"], s["bias"])
    out = dict(idx=r.topk_idx, gate=r.gate, counts=r.counts, padded=r.padded_offsets, row_of=r.row_of_assign,
               assign_of=r.assign_of_row)
    if s["case"]["train"]:
        r.backward(s["logits"], s["dgate"], s["dlogits"])
        out["dlogits"] = s["dlogits"]
        if s["bias"] is not None:
            r.update_bias(s["bias"], s["rate"], out=s["new_bias"])
            out["bias"] = s["new_bias"]
    return out


def _rms_own(s):
    c, n, io, out = s["case"], s["norm"], s["io"], {}
    n.forward(s["x"], s["gamma"], io["y"] if c["y"] else None, residual=s.get("residual"),
              h=io["h"] if c["residual"] else None, encoded=s.get("mx"))
    if c["y"]:
        out["y"] = io["y"]
    if c["residual"]:
        out["h"] = io["h"]
    if c["mx"]:
        s["mx"].decode(s["y8"])
        out["y8"] = s["y8"]
    if c["train"]:
        n.backward(s["dy"], io["h"] if c["residual"] else s["x"], s["gamma"], io["dx"], io["dgamma"], dh=s["dh"])
        out.update(dx=io["dx"], dgamma=io["dgamma"])
    return out


def _ckpt_own(s):
    L, n = s["layer"], s["rows"]
    L.save(s["ckpt"], s["X"])
    L.restore(s["ckpt"])
    return dict(x_perm=L.x_perm[:n], h13=L.h13[:n], act=L.act[:n])


# -------------------------------------------------------------- plain form
def _route_plain(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    # the choice in 64 bits: values next to one another decide it
    z = s["logits"].double()
    if c["score"] == "sigmoid":
        u = 1.0 / (1.0 + torch.exp(-z))
    else:
        u = torch.exp(z - z.max(1, keepdim=True).values)
        u = u / u.sum(1, keepdim=True)
    if s["bias"] is not None:
        u = u + s["bias"].double()
    if c["groups"] > 1:
        by = u.view(T, c["groups"], -1)
        value = torch.sort(by, dim=2, descending=True).values[:, :, :c["group_top"]].sum(2)
        best = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        stays = torch.zeros_like(value).scatter_(1, best, 1.0) > 0
        u = torch.where(stays[:, :, None], by, torch.full_like(by, -math.inf)).view(T, E)
    idx = torch.sort(u, dim=1, descending=True, stable=True).indices[:, :k]
    z = s["logits"].float()
    if c["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-z))
    else:
        p = torch.exp(z - z.max(1, keepdim=True).values)
        p = p / p.sum(1, keepdim=True)
    sel = p.gather(1, idx)
    gate = sel / sel.sum(1, keepdim=True) * s["scale"] if c["renorm"] else sel * s["scale"]
    counts, padded, row_of, assign_of = _permutation(idx, E)
    out = dict(idx=idx.int(), gate=gate, counts=counts, padded=padded, row_of=row_of, assign_of=assign_of)
    if c["train"]:
        inner = (gate * s["dgate"]).sum(1, keepdim=True)
        if c["score"] == "sigmoid":
            d = gate * (1.0 - sel) * (s["dgate"] - inner / s["scale"] if c["renorm"] else s["dgate"])
            dlogits = torch.zeros_like(p).scatter_(1, idx, d)
        elif c["renorm"]:
            dlogits = torch.zeros_like(p).scatter_(1, idx, gate * (s["dgate"] - inner / s["scale"]))
        else:
            dlogits = (-p * inner).scatter_add_(1, idx, gate * s["dgate"])
        out["dlogits"] = dlogits.to(s["logits"].dtype)
        if s["bias"] is not None:
            out["bias"] = s["bias"] + s["rate"] * torch.sign(T * k - counts.long() * E).float()
    return out


def _mx(v):
    """The values that the MXFP8 codes of v stand for: blocks of 32 columns, a
    scale of floor(log2(largest)) - 8, elements with 4 significant bits."""
    b = v.view(v.shape[0], -1, 32)
    top = b.abs().amax(2, keepdim=True)
    e = torch.clamp((top.view(torch.int32) >> 23) - 8, min=0)      # of the scale, plus 127
    scale = torch.where(e > 0, e << 23, torch.full_like(e, 1 << 22)).view(torch.float32)
    q = torch.clamp(b / scale, -448.0, 448.0).to(torch.float8_e4m3fn).float()
    return (q * scale).view(v.shape)


def _rms_plain(s):
    c, dt, out = s["case"], s["x"].dtype, {}
    x, gamma = s["x"].float(), s["gamma"].float()
    h = x + s["residual"].float() if c["residual"] else x
    rstd = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
    y = h * rstd * gamma
    if c["y"]:
        out["y"] = y.to(dt)
    if c["mx"]:
        out["y8"] = _mx(y).to(torch.bfloat16)
    if c["residual"]:
        out["h"] = h.to(dt)
    if c["train"]:
        if c["residual"]:
            h = out["h"].float()               # what the backward finds
        dy = s["dy"].float()
        xh, gy = h * rstd, dy * gamma
        dx = rstd * (gy - xh * (gy * xh).mean(1, keepdim=True)) + s["dh"].float()
        out.update(dx=dx.to(dt), dgamma=(dy * xh).sum(0).to(s["gamma"].dtype))
    return out


def _ckpt_plain(s):
    c, n, dt = s["case"], s["rows"], s["X"].dtype
    a = s["assign_of"][:n].long()
    real, a = (a >= 0)[:, None], a.clamp(min=0)
    x = _mx(s["X"].float()).to(dt)
    codes = _mx(s["h13"][s["row_of"].long()].float())          # in the order of the assignments
    x_perm = torch.where(real, x[a // c["k"]], torch.zeros((), dtype=dt, device="cuda"))
    h = torch.where(real, codes[a], torch.zeros((), device="cuda"))
    u, v = h[:, :c["I"]], h[:, c["I"]:]
    act = u / (1.0 + torch.exp(-u)) * v
    if dt == torch.bfloat16:
        act = act * s["gate"].view(-1)[a][:, None]
    return dict(x_perm=x_perm, h13=h.to(dt), act=act.to(dt))


def work(case):
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        es = 2 if case["dtype"] == "bf16" else 4
        b = T * E * es + 3 * T * k * 4 + (T * k + ALIGN * E) * 4 + 3 * E * 4
        if case["train"]:
            b += T * k * 4 + T * E * es
        return {"bytes": b, "flops": (12 if case["train"] else 8) * T * E}
    if case["op"] == "rms":
        T, H = case["T"], case["H"]
        es, ws = (2 if case[n] == "bf16" else 4 for n in ("dtype", "wtype"))
        n = 1 + 2 * case["residual"] + case["y"] + 3 * case["train"]      # x; residual, h; y; dy, dh, dx
        return {"bytes": T * H * (n * es + 2 * case["mx"]) + H * ws * (1 + case["train"]),
                "flops": (6 + 4 * case["mx"] + 10 * case["train"]) * T * H}
    T, H, I, k = case["T"], case["H"], case["I"], case["k"]
    es = 2 if case["dtype"] == "bf16" else 4
    # X and h13 in, x_perm, h13 and act out; the codes are held between the two
    return {"bytes": T * H * es + T * k * (H + 5 * I) * es + 2 * (T * H + T * k * 2 * I) * 33 // 32,
            "flops": 4 * (T * H + T * k * 2 * I) + 8 * T * k * I}


# ------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _route_exact, "rms": _rms_exact, "ckpt": _ckpt_exact}[case["op"]](s)


def _route_exact(s):
    c = s["case"]
    E, G = c["E"], c["groups"]
    z = s["logits"].double()
    logp = torch.nn.functional.logsigmoid(z) if c["score"] == "sigmoid" else torch.log_softmax(z, 1)
    b = torch.zeros(E, dtype=torch.float64, device="cuda") if s["bias"] is None else s["bias"].double()
    value = logp.exp() + b
    if G > 1:
        top = value.unflatten(1, (G, E // G)).topk(c["group_top"], dim=2).values.sum(2)
        floor = top.topk(c["top_groups"], dim=1).values[:, -1:]
        value = value.masked_fill((top < floor).repeat_interleave(E // G, 1), -math.inf)
    order = torch.argsort(value, dim=1, descending=True, stable=True)[:, :c["k"]]
    lp = logp.gather(1, order)
    gate = s["scale"] * (torch.softmax(lp, 1) if c["renorm"] else lp.exp())
    out = dict(idx=None, gate=gate, counts=None, padded=None, row_of=None, assign_of=None)
    if c["train"]:
        dw = s["dgate"].double()
        # d(log gate_j) reaches log s_j and, renormalised, every other chosen one
        dlog = gate * dw
        if c["renorm"]:
            dlog = dlog - gate / s["scale"] * torch.einsum("tk,tk->t", gate, dw)[:, None]
        full = torch.zeros_like(z).scatter_(1, order, dlog)
        out["dlogits"] = full * torch.sigmoid(-z) if c["score"] == "sigmoid" else \
            full - logp.exp() * full.sum(1, keepdim=True)
        if s["bias"] is not None:
            load = torch.bincount(order.reshape(-1), minlength=E).double()
            out["bias"] = b + s["rate"] * torch.sign(load.mean() - load)
    return out


def _below(v):
    """The largest power of two not above v."""
    return (v.view(torch.int64) >> 52 << 52).view(torch.float64)


def _mx_exact(v):
    """As _mx, from the formats' definition in 64 bits."""
    b = v.unflatten(1, (-1, 32))
    top = b.abs().max(2, keepdim=True).values
    scale = _below(top.clamp(min=2.0 ** -119)) / 256
    q = (b / scale).abs()
    step = _below(q.clamp(min=2.0 ** -6)) / 8
    q = torch.minimum(torch.round(q / step) * step, torch.full_like(q, 448.0))
    return (torch.sign(b) * q * scale).flatten(1)


def _rms_exact(s):
    c, out = s["case"], {}
    T, H = s["x"].shape
    gamma = s["gamma"].double()
    names = [n for n, on in (("y", c["y"]), ("y8", c["mx"]), ("h", c["residual"]), ("dx", c["train"])) if on]
    out = {n: torch.empty((T, H), dtype=torch.float64, device="cuda") for n in names}
    if c["train"]:
        out["dgamma"] = torch.zeros_like(gamma)
    rows = max(1, (1 << 24) // H)
    for i in range(0, T, rows):
        at = slice(i, i + rows)
        h = s["x"][at].double()
        if c["residual"]:
            h = h + s["residual"][at].double()
            out["h"][at] = h
        inv = (torch.einsum("th,th->t", h, h) / H + EPS).pow(-0.5)
        y = torch.einsum("th,t,h->th", h, inv, gamma)
        if c["y"]:
            out["y"][at] = y
        if c["mx"]:
            out["y8"][at] = _mx_exact(y)
        if c["train"]:
            dy = s["dy"][at].double()
            xh = h.to(s["x"].dtype).double() * inv[:, None]      # of the sum as it is stored
            # the row's Jacobian (I - xh xh^T / H) / rms applied to gamma * dy
            b = torch.einsum("th,th,h->t", dy, xh, gamma) / H
            out["dx"][at] = (gamma * dy - b[:, None] * xh) * inv[:, None] + s["dh"][at].double()
            out["dgamma"] += torch.einsum("th,th->h", dy, xh)
    return out


def _ckpt_exact(s):
    c, n = s["case"], s["rows"]
    X = _mx_exact(s["X"].double())
    x_perm = torch.zeros((n, c["H"]), dtype=torch.float64, device="cuda")
    h13 = torch.zeros((n, 2 * c["I"]), dtype=torch.float64, device="cuda")
    act = torch.zeros((n, c["I"]), dtype=torch.float64, device="cuda")
    rows = s["row_of"].long().view(-1, c["k"])
    for j in range(c["k"]):
        at = rows[:, j]
        x_perm[at] = X
        h = _mx_exact(s["h13"][at].double())
        h13[at] = h
        u, v = h.chunk(2, 1)
        a = u * torch.sigmoid(u) * v
        act[at] = a * s["gate"][:, j:j + 1].double() if s["X"].dtype == torch.bfloat16 else a
    return dict(x_perm=x_perm, h13=h13, act=act)
