"""Routing by scores on the GPU against its float64 definition.

The choice and the permutation are exact.  Gates and gradients: U = 2^-24 is the
unit roundoff of fp32.  Renormalised gates come from x = log s, whose error is
below U (2 |x| + 4); the difference to the largest, its exponential, the sum of up
to 32, the quotient and the scale add 2 |x| + 20 units, so a gate is within
U (4 max |x| + 24) of its value.  A softmax gate that is not renormalised divides
by a sum of exponentials that are off by (4 + 2 |x|) U, weighted with themselves
(at most log E on average), added up in at most 32 + 5 steps, and its own
exponential is off by (2 + |x|) U: U (80 + 2 |x|) with |x| the distance to the
largest logit.  Gradients carry the gates' error, twice where a sum of their
products enters, and a dozen roundings of their own."""
import numpy as np
import pytest

from oracle import moe_oracle as M
from oracle import training_oracle as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _device(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def _gate_tol(l, idx, gate, score, renorm):
    """Relative tolerance of the gates [T, k]."""
    ls = np.take_along_axis(l, idx, 1)
    fin = np.isfinite(ls)
    if renorm:
        x = np.where(fin, -np.logaddexp(0, -np.where(fin, ls, 0)) if score == "sigmoid" else ls, 0)
        return U * (4 * np.abs(x).max(1, keepdims=True) + 24) + 0 * gate
    if score == "sigmoid":
        return np.full_like(gate, 8 * U)
    top = l.max(1, keepdims=True)
    return U * (80 + 2 * np.where(fin, np.where(np.isfinite(top), top, 0) - np.where(fin, ls, 0), 0))


def _check(l, bias, k, router, dgate=None, dlogits=None, **how):
    """The router's arrays against the definition for float32 logits l (numpy)."""
    E = l.shape[1]
    idx, gate = O.route_by_scores(l, bias, k, **how)
    got = router.topk_idx.cpu().numpy()
    assert np.array_equal(got, idx), np.argwhere((got != idx).any(1))[:4].ravel()
    r = O._readable(l)
    score, renorm, scale = how.get("score", "softmax"), how.get("renormalise", True), how.get("scale", 1.0)
    tol = _gate_tol(r, idx, gate, score, renorm)
    # (below the smallest normal number a gate may be flushed)
    assert (np.abs(router.gate.double().cpu().numpy() - gate) <= tol * gate + scale * 2e-38).all()
    m = M.permute(idx, E)
    for name in ("counts", "offsets", "padded_offsets", "row_of_assign"):
        assert np.array_equal(getattr(router, name).cpu().numpy(), m[name]), name
    a = router.assign_of_row.cpu().numpy()
    n = int(m["padded_offsets"][-1])
    assert np.array_equal(a[:n], m["assign_of_row"][:n]) and (a[n:] == -1).all()
    if dlogits is None:
        return
    dg = np.asarray(dgate, np.float64)
    want = O.route_by_scores_backward(l, idx, gate, dg, score, renorm, scale)
    out = dlogits.double().cpu().numpy()
    stored = 2.0 ** -8 if str(dlogits.dtype) == "torch.bfloat16" else U
    size = (np.abs(gate * dg)).sum(1, keepdims=True)            # of the sum of products
    t = np.zeros_like(want)
    own = np.abs(gate * dg) + (gate * size / scale if renorm else 0)
    np.put_along_axis(t, idx, own, 1)
    if score == "softmax" and not renorm:
        t = t + O.scores(l, score) * size
    k_u = 2 * tol.max(1, keepdims=True) + 100 * U
    assert (np.abs(out - want) <= stored * np.abs(want) + (1 + stored) * k_u * t + 2e-38).all(), np.abs(out - want).max()


def _run(l, bias, k, dtype=None, pad=0, seed=0, **how):
    import torch
    from mixture_experts_layer_18_gb300.training import Router
    T, E = l.shape
    dt = torch.float32 if dtype is None else getattr(torch, dtype)
    wide = torch.full((T, E + pad), 77.0, dtype=dt, device="cuda")
    x = wide[:, :E]
    x.copy_(_device(l.astype(np.float32)))
    l = x.float().cpu().numpy()                                  # as stored
    r = Router(T, E, k, dtype=dt, **how)
    for a in (r.topk_idx, r.gate, r.counts, r.offsets, r.padded_offsets, r.row_of_assign, r.assign_of_row):
        a.fill_(-7)
    dg = np.random.default_rng(seed + 1).standard_normal((T, k)).astype(np.float32)
    dl = torch.full((T, E), 5.0, dtype=dt, device="cuda")
    b = None if bias is None else _device(np.asarray(bias, np.float32))
    r.forward(x, b)
    r.backward(x, _device(dg), dl)
    torch.cuda.synchronize()
    return l, r, dg, dl


# every lane width, one expert, odd counts, groups that lie across lanes; a few and
# many tokens (one warp each, blocks of 32 warps, several tokens per warp)
CASES = [
    (1, 1, 1, {}), (1, 256, 8, dict(score="sigmoid", groups=8, top_groups=4, group_top=2)),
    (5, 7, 7, dict(score="sigmoid")), (33, 32, 32, dict(renormalise=False)), (64, 33, 3, {}),
    (257, 60, 6, dict(renormalise=False)), (1000, 64, 4, dict(groups=4, top_groups=3, group_top=1)),
    (700, 96, 5, dict(score="sigmoid", groups=6, top_groups=2, group_top=2, scale=2.5)),
    (2049, 128, 8, dict(renormalise=False, scale=0.5)), (513, 160, 6, dict(groups=8, top_groups=3, group_top=2)),
    (5000, 256, 8, dict(score="sigmoid", groups=8, top_groups=4, group_top=2, scale=2.5)),
    (611, 257, 9, dict(score="sigmoid", renormalise=False)), (300, 512, 16, dict(groups=32, top_groups=5, group_top=1)),
    (97, 1000, 31, dict(score="sigmoid", groups=10, top_groups=7, group_top=2)), (40, 1024, 32, dict(score="sigmoid")),
    (700, 24, 2, dict(groups=12, top_groups=1, group_top=2, renormalise=False)),
    # many tokens per block: eight lanes per token, in whole and part rows, and what it leaves to the others
    (5003, 60, 6, {}), (4901, 128, 8, dict(renormalise=False)), (5003, 32, 8, dict(score="sigmoid", renormalise=False)),
    (4999, 256, 8, dict(groups=4, top_groups=2, group_top=2)), (5001, 248, 7, dict(score="sigmoid")), (5000, 20, 1, {}),
    (4903, 128, 5, dict(score="sigmoid", groups=8, top_groups=3, group_top=2)), (5000, 96, 9, {}),
    (4905, 64, 3, dict(score="sigmoid", groups=2, top_groups=1, group_top=1)), (4870, 30, 4, {}),
    (5003, 160, 6, dict(score="sigmoid", groups=8, top_groups=3, group_top=2, scale=2.5)), (5000, 250, 8, {}),
    (4903, 35, 5, dict(groups=5, top_groups=3, group_top=1, renormalise=False)),
    (5005, 14, 2, dict(groups=7, top_groups=2, group_top=2)), (4999, 99, 7, dict(score="sigmoid", groups=3, top_groups=2, group_top=2)),
    (5001, 513, 3, {}), (4997, 320, 8, dict(groups=16, top_groups=5, group_top=2)),
]


def _many(l, many):
    """The same rows as often as blocks of many tokens need."""
    return np.tile(l, (-(-5000 // len(l)), 1)) if many else l


@pytest.mark.parametrize("T,E,k,how", CASES)
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("dtype,pad", [("float32", 0), ("bfloat16", 3), ("float32", 5)])
def test_router_matches_definition(T, E, k, how, biased, dtype, pad):
    rng = np.random.default_rng(T + E)
    l = rng.standard_normal((T, E)) * 1.5
    bias = (1e-3 * rng.integers(-80, 81, E)).astype(np.float32) if biased else None
    l, r, dg, dl = _run(l, bias, k, dtype, pad, **how)
    _check(l, bias, k, r, dg, dl, **how)
    assert r.device_status() == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("many", [False, True])
def test_close_values_are_chosen_in_64_bits(score, groups, many):
    """Values apart by less than fp32 can tell: the bias makes up for the score's
    difference up to its own last bits."""
    rng = np.random.default_rng(11)
    T, E = 400, 64
    l = (rng.integers(-3, 4, (T, E)) + rng.integers(0, 9, (T, E)) * 2.0 ** -22).astype(np.float32)
    level = O.scores(l[:1], score)[0]
    bias = (0.5 - level).astype(np.float32)                      # token 0: all values within 2^-24 of 1/2
    l[1::2] = l[0]
    l[1::2] += rng.integers(0, 3, (T // 2, E)).astype(np.float32) * np.float32(2.0 ** -22)
    how = dict(score=score, groups=groups, top_groups=max(1, groups // 2), group_top=2 if groups > 1 else 1)
    l, r, dg, dl = _run(_many(l, many), bias, 6, **how)
    _check(l, bias, 6, r, dg, dl, **how)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [None, 0.0, 0.25])
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("many", [False, True])
def test_ties_go_to_the_lower_index(score, bias, groups, many):
    """Equal logits (a router of zeros, logits of few values) with equal biases."""
    rng = np.random.default_rng(5)
    l = rng.integers(0, 2, (300, 40)).astype(np.float32)
    l[:50] = 0.0
    l[50:60] = -0.0
    l[60:70, ::2] = -0.0
    b = None if bias is None else np.full(40, bias, np.float32)
    how = dict(score=score, groups=groups, top_groups=max(1, groups // 2), group_top=2 if groups > 1 else 1)
    l, r, dg, dl = _run(_many(l, many), b, 7, **how)
    _check(l, b, 7, r, dg, dl, **how)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("E", [32, 100, 256])
@pytest.mark.parametrize("bias", [None, 0.25])
def test_a_few_equal_logits(dtype, E, bias):
    """Two to five equal values among others, at the front, inside and at the end of
    the chosen, in any places."""
    rng = np.random.default_rng(E)
    l = np.stack([rng.permutation(E) for _ in range(5000)]).astype(np.float32) / 64 - 1
    order = np.argsort(-l, 1)
    for t in range(5000):
        i, n = rng.integers(0, 8), rng.integers(2, 6)
        l[t, order[t, i:i + n]] = l[t, order[t, i]]
    b = None if bias is None else np.full(E, bias, np.float32)
    how = dict(score="sigmoid")
    l, r, dg, dl = _run(l, b, 6, dtype, **how)
    _check(l, b, 6, r, dg, dl, **how)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E", [32, 40])
@pytest.mark.parametrize("many", [False, True])
def test_masked_experts(score, renorm, many, E):
    """-inf and the type's lowest value in masked places, tokens with fewer
    experts than top_k, with none, and groups left empty; large logits."""
    rng = np.random.default_rng(6)
    l = rng.standard_normal((200, E)).astype(np.float32)
    l[:60][rng.random((60, E)) < 0.5] = -np.inf
    l[60:90, 8:] = -np.inf
    l[90:100, 2:] = -np.inf
    l[100:130][rng.random((30, E)) < 0.5] = np.finfo(np.float32).min
    l[130:150] *= 200
    how = dict(score=score, renormalise=renorm)
    for bias, more in ((None, {}), (rng.standard_normal(E).astype(np.float32), {}),
                       (None, dict(groups=4, top_groups=2, group_top=1))):
        # (scores of the lowest value are 0 in 64 bits, like those of logits below -745)
        x, r, dg, dl = _run(_many(l, many), bias, 4, **how, **more)
        _check(x, bias, 4, r, dg, dl, **how, **more)
        assert r.device_status() == 0


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E,how", [(128, {}), (256, dict(score="sigmoid")), (128, dict(renormalise=False, groups=2, top_groups=1, group_top=2)),
                                   (256, dict(score="sigmoid", groups=8, top_groups=4, group_top=2)),
                                   (160, dict(score="softmax", groups=8, top_groups=1, group_top=1))])
def test_the_best_lie_next_to_each_other(E, how, biased, dtype):
    """The chosen, and sometimes those that are as good or nearly so, are neighbours."""
    rng = np.random.default_rng(E + biased)
    T, k, n = 5000, 8, 16
    l = rng.standard_normal((T, E)).astype(np.float32)
    at = rng.integers(0, E // n, T)[:, None] * n + np.arange(n)
    order = np.argsort(rng.random((T, n)), 1)
    best = (5 + 0.25 * order).astype(np.float32)
    near = rng.integers(0, 4, T)                                 # apart; one, two steps, or nothing between 8 and 9
    eighth = np.float32(5 + 0.25 * (n - k))
    ninth = {1: np.nextafter(eighth, np.float32(0)), 2: np.nextafter(np.nextafter(eighth, np.float32(0)), np.float32(0)), 3: eighth}
    for c, v in ninth.items():
        rows = np.where(near == c)[0]
        best[rows, np.argmax(order[rows] == n - k - 1, 1)] = v
    np.put_along_axis(l, at, best, 1)
    bias = np.repeat(rng.integers(-60, 61, E // n) * 1e-3, n) if biased else None
    l, r, dg, dl = _run(l, bias, k, dtype, **how)
    _check(l, None if bias is None else bias.astype(np.float32), k, r, dg, dl, **how)


def test_bad_logits_are_reported():
    """A token of masked experts only, NaN, +inf, a bias that is not finite: read
    as masked (as 0), reported, and the other tokens are as without them."""
    from mixture_experts_layer_18_gb300 import MOE_ERR_BAD_INPUT
    rng = np.random.default_rng(7)
    base = rng.standard_normal((50, 32)).astype(np.float32)
    b = (0.1 * rng.standard_normal(32)).astype(np.float32)
    for bad in ("row", "nan", "inf", "bias"):
        for score, many in (("softmax", False), ("sigmoid", False), ("softmax", True), ("sigmoid", True)):
            l, bias = _many(base.copy(), many), b.copy()
            if bad == "row":
                l[7] = -np.inf
            elif bad == "bias":
                bias[3], bias[9] = np.nan, np.inf
            else:
                l[7, 5] = np.nan if bad == "nan" else np.inf
            l, r, dg, dl = _run(l, bias, 4, score=score)
            _check(l, bias, 4, r, dg, dl, score=score)
            assert r.device_status() == MOE_ERR_BAD_INPUT
            if bad == "row":
                assert r.topk_idx[7].tolist() == [0, 1, 2, 3] and not r.gate[7].any() and not dl[7].any()


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("many", [False, True])
def test_bad_logits_that_are_chosen(renorm, many):
    """NaN and +inf among fewer finite logits than top_k: chosen as masked ones, gate and
    gradient 0, and the gradient of the others is that of -inf in their place."""
    from mixture_experts_layer_18_gb300 import MOE_ERR_BAD_INPUT
    rng = np.random.default_rng(17)
    l = np.full((20, 16), -np.inf, np.float32)
    l[:, :2] = rng.standard_normal((20, 2))
    l[::2, 2], l[::3, 3] = np.nan, np.inf
    l = _many(l, many)
    for score in ("softmax", "sigmoid"):
        x, r, dg, dl = _run(l, None, 4, score=score, renormalise=renorm)
        _check(x, None, 4, r, dg, dl, score=score, renormalise=renorm)
        assert r.device_status() == MOE_ERR_BAD_INPUT


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("T", [3, 900, 5000])
@pytest.mark.parametrize("off,pad", [(1, 0), (2, 2), (3, 5), (4, 8), (8, 0)])
def test_rows_at_any_address(dtype, T, off, pad):
    """Logits whose rows start anywhere, gradients of an odd place too."""
    import torch
    from mixture_experts_layer_18_gb300.training import Router
    rng = np.random.default_rng(off)
    dt, E, k = getattr(torch, dtype), 128, 8
    buf = torch.full((T, off + E + pad), 99.0, dtype=dt, device="cuda")
    x = buf[:, off:off + E]
    x.copy_(_device(rng.standard_normal((T, E)).astype(np.float32)))
    b = (1e-3 * rng.integers(-50, 50, E)).astype(np.float32)
    dg = rng.standard_normal((T, k)).astype(np.float32)
    flat = torch.full((T * E + 16,), 7.0, dtype=dt, device="cuda")
    dl = flat[off:off + T * E].view(T, E)
    r = Router(T, E, k, score="sigmoid", dtype=dt)
    r.forward(x, _device(b))
    r.backward(x, _device(dg), dl)
    torch.cuda.synchronize()
    _check(x.float().cpu().numpy(), b, k, r, dg, dl, score="sigmoid")
    assert (flat[:off] == 7.0).all() and (flat[off + T * E:] == 7.0).all()


def test_no_tokens():
    import torch
    from mixture_experts_layer_18_gb300.training import Router
    r = Router(0, 16, 2)
    for a in (r.counts, r.offsets, r.padded_offsets, r.assign_of_row):
        a.fill_(9)
    x = torch.zeros((0, 16), device="cuda")
    r.forward(x)
    r.backward(x, torch.zeros((0, 2), device="cuda"), torch.zeros((0, 16), device="cuda"))
    torch.cuda.synchronize()
    assert not r.counts.any() and not r.offsets.any() and not r.padded_offsets.any() and (r.assign_of_row == -1).all()


@pytest.mark.parametrize("T,E,k", [(70001, 16, 4), (200_003, 300, 9), (10_300_000, 8, 2)])
def test_many_tokens_are_placed_in_order(T, E, k):
    """More assignments per block than one round of the permutation takes; more tokens
    per block than 16 bits count."""
    import torch
    from mixture_experts_layer_18_gb300.training import Router
    g = torch.Generator(device="cuda").manual_seed(8)
    x = torch.randn((T, E), generator=g, device="cuda")
    x[:, 3] += 3
    r = Router(T, E, k)
    r.forward(x)
    idx = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(r.topk_idx.long(), idx)
    flat = idx.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E)
    start = torch.nn.functional.pad(((counts + 127) // 128 * 128).cumsum(0), (1, 0))
    first = torch.nn.functional.pad(counts.cumsum(0), (1, 0))
    e = flat[order]
    row = start[e] + torch.arange(T * k, device="cuda") - first[e]
    want = torch.empty_like(row)
    want[order] = row
    assert torch.equal(r.row_of_assign.long(), want) and torch.equal(r.counts.long(), counts)
    back = torch.full((T * k + 128 * E,), -1, device="cuda")
    back[want] = torch.arange(T * k, device="cuda")
    assert torch.equal(r.assign_of_row.long(), back)
    assert torch.equal(r.padded_offsets.long(), start) and torch.equal(r.offsets.long(), first)


def test_logits_past_32_bits():
    """More than 2^32 bytes and 2^31 elements of logits and gradients: the last rows are their own."""
    import torch
    from mixture_experts_layer_18_gb300.training import Router
    T, E, k = 2_200_001, 1000, 4
    x = torch.zeros((T, E), device="cuda")
    x[:, 5] = 1.0
    rng = np.random.default_rng(9)
    tail = rng.standard_normal((40, E)).astype(np.float32)
    x[-40:] = _device(tail)
    r = Router(T, E, k, renormalise=False)
    r.forward(x)
    dg = torch.ones((T, k), device="cuda")
    dl = torch.empty_like(x)
    r.backward(x, dg, dl)
    torch.cuda.synchronize()
    idx, gate = O.route_by_scores(tail, None, k, renormalise=False)
    assert np.array_equal(r.topk_idx[-40:].cpu().numpy(), idx)
    assert (r.topk_idx[:-40] == torch.tensor([5, 0, 1, 2], device="cuda")).all()
    assert np.abs(r.gate[-40:].double().cpu().numpy() - gate).max() <= 200 * U
    want = O.route_by_scores_backward(tail, idx, gate, np.ones((40, k)), "softmax", False, 1.0)
    assert np.abs(dl[-40:].double().cpu().numpy() - want).max() <= 400 * U
    assert int(r.counts.sum()) == T * k


def test_the_softmax_router_is_the_layers():
    """Without the extras: the layer's own router, array by array."""
    import torch
    from mixture_experts_layer_18_gb300.layer import MoELayer
    from mixture_experts_layer_18_gb300.training import Router
    g = torch.Generator(device="cuda").manual_seed(3)
    l = torch.randn((1003, 48), generator=g, device="cuda")
    L, r = MoELayer(1003, 64, 48, 64, 5, backward=False), Router(1003, 48, 5)
    L.route(l)
    r.forward(l)
    torch.cuda.synchronize()
    for name in ("topk_idx", "counts", "offsets", "padded_offsets", "row_of_assign", "assign_of_row"):
        assert torch.equal(getattr(L, name), getattr(r, name)), name
    assert (L.gate - r.gate).abs().max() <= 60 * U


def test_balance_bias():
    import torch
    from mixture_experts_layer_18_gb300.training import Router
    rng = np.random.default_rng(9)
    l = rng.standard_normal((640, 20)).astype(np.float32)
    b = (1e-3 * rng.integers(-9, 9, 20)).astype(np.float32)
    r = Router(640, 20, 2, score="sigmoid")
    t, out = _device(b), torch.empty(20, device="cuda")
    r.forward(_device(l), t)
    r.update_bias(t, 1e-3, out=out)
    want = O.balance_bias(r.counts.cpu().numpy(), np.float64(np.float32(1e-3)), b)
    assert np.array_equal(t.cpu().numpy(), b)
    assert (np.abs(out.double().cpu().numpy() - want) <= U * np.abs(want)).all()
    r.counts.fill_(64)                                            # an even load: unchanged
    r.update_bias(t, 1e-3)
    assert np.array_equal(t.cpu().numpy(), b)
    r.counts.copy_(torch.arange(20, dtype=torch.int32) * 100_000_000)     # sums past 32 bits
    r.update_bias(t, 1e-3)
    assert (t[:10].cpu().numpy() > b[:10]).all() and (t[10:].cpu().numpy() < b[10:]).all()


def test_captured_router_and_a_second_stream():
    """Replays follow the inputs; on a stream of its own the call waits for none."""
    import torch
    from mixture_experts_layer_18_gb300.training import Router
    rng = np.random.default_rng(10)
    how = dict(score="sigmoid", groups=4, top_groups=2, group_top=2)
    l = [rng.standard_normal((777, 64)).astype(np.float32) for _ in range(3)]
    b = (0.01 * rng.standard_normal(64)).astype(np.float32)
    r = Router(777, 64, 6, **how)
    x, t, dg, dl = _device(l[0]), _device(b), _device(rng.standard_normal((777, 6)).astype(np.float32)), \
        torch.empty((777, 64), device="cuda")
    r.forward(x, t)
    r.backward(x, dg, dl)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.forward(x, t)
        r.backward(x, dg, dl)
    for v in l[1:]:
        x.copy_(_device(v))
        graph.replay()
        torch.cuda.synchronize()
        _check(v, b, 6, r, dg.cpu().numpy(), dl, **how)
    s = torch.cuda.Stream()
    x.copy_(_device(l[0]))
    s.wait_stream(torch.cuda.current_stream())
    r.forward(x, t, stream=s)
    r.backward(x, dg, dl, stream=s)
    s.synchronize()
    _check(l[0], b, 6, r, dg.cpu().numpy(), dl, **how)


def test_bad_index_in_the_backward():
    from mixture_experts_layer_18_gb300 import MOE_ERR_BAD_INDEX
    l, r, dg, dl = _run(np.random.default_rng(1).standard_normal((9, 12)).astype(np.float32), None, 2)
    keep = dl.clone()
    r.topk_idx[4, 1] = 12
    r.topk_idx[5, 0] = -3
    r.backward(_device(l), _device(dg), dl)
    assert r.device_status() == MOE_ERR_BAD_INDEX
    rows = [i for i in range(9) if i not in (4, 5)]
    assert (dl[rows] == keep[rows]).all()
