"""The score router (sigmoid or softmax scores, selection bias, expert groups), its gradient and the step of
its bias against plain 64-bit NumPy versions.

Tolerances, from the arithmetic (u = 2^-24):
  ids, counts   equal
  weights       an exponential of a rounded argument (2 + |x| ulp), a sum of at most 512 (softmax) or 32
                (renormalised) terms added in a tree, a quotient:  (64 + 2 max|l|) u relative
  gradient      the same for each factor, over differences of at most sum |w dw| + |dw|:
                (256 + 8 max|l|) u (|dw| + max |dw|) scale; bf16: half a step more
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def pkg():
    import serving_topk_permute_gb300 as p
    p.lib()
    torch.cuda.set_device(0)
    return p


def scores(l, score):
    l = l.astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        top = l.max(1, keepdims=True)
        e = np.exp(l - np.where(np.isfinite(top), top, 0.0))
        return e / np.maximum(e.sum(1, keepdims=True), 1e-300)


def route(l, bias, mask, cfg):
    """Ids, weights, counts and the number of valid tokens of fp64 logits."""
    T, E = l.shape
    G, k = cfg.num_groups, cfg.top_k
    s = scores(l, cfg.score)
    b = np.zeros(E) if bias is None else bias.astype(np.float64)
    c = s + b
    may = (l != -np.inf) & (b != -np.inf)
    key = l if np.all(b == b[0]) else c  # equal biases: the logits' order, which is the scores'
    ids = np.full((T, k), -1, np.int64)
    w = np.zeros((T, k))
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        value = np.full(G, -np.inf)
        for g in range(G):
            at = np.arange(g * (E // G), (g + 1) * (E // G))
            best = np.sort(c[t, at[may[t, at]]])[::-1]
            if len(best):
                value[g] = best[:2].sum() if cfg.group_score == "top2" else best[0]
                if cfg.group_score == "max" and np.all(b == b[0]):
                    value[g] = l[t, at[may[t, at]]].max()
        kept = np.lexsort((np.arange(G), -value))[:cfg.top_groups]
        allowed = may[t] & np.isin(np.arange(E) // (E // G), kept)
        order = [e for e in np.lexsort((np.arange(E), -key[t])) if allowed[e]][:k]
        ids[t, :len(order)] = order
        if order:
            x = s[t, order]
            if cfg.renormalize:
                lo = l[t, order]
                if cfg.score == "softmax" or lo.max() < -30:
                    x = np.exp(lo - lo.max())
                x = x / x.sum()
            w[t, :len(order)] = cfg.scale * x
    counts = np.bincount(ids[ids >= 0], minlength=E)
    return ids, w, counts, int((ids[:, 0] >= 0).sum())


def logits_of(rng, T, E, dtype, scale=1.0, stride=None):
    l = torch.from_numpy(rng.standard_normal((T, E)) * scale).float()
    l = l.bfloat16() if dtype == "bf16" else l
    if stride:
        wide = torch.zeros((T, stride), dtype=l.dtype, device="cuda")
        wide[:, 1:1 + E] = l.cuda()
        return wide[:, 1:1 + E]
    return l.cuda()


def check(pkg, logits, bias, mask, cfg):
    r = pkg.ScoreRouter(cfg)
    o = r.forward(logits, None if bias is None else torch.from_numpy(bias).float().cuda(),
                  None if mask is None else torch.from_numpy(mask).cuda())
    l = logits.float().cpu().numpy().astype(np.float64)
    ids, w, counts, n = route(l, None if bias is None else bias.astype(np.float32), mask, cfg)
    assert np.array_equal(o.topk_ids.cpu().numpy(), ids)
    assert np.array_equal(o.counts.cpu().numpy(), counts)
    assert o.num_valid.item() == n
    big = np.abs(np.where(np.isfinite(l), l, 0)).max(initial=0)
    got = o.topk_weights.cpu().numpy().astype(np.float64)
    assert (np.abs(got - w) <= (64 + 2 * big) * U * np.abs(w) + abs(cfg.scale) * 2.0 ** -120).all()
    return r, o, ids, w


SHAPES = [  # T, E, k, groups, top groups
    (1, 256, 8, 8, 4), (64, 256, 8, 8, 4), (513, 256, 8, 8, 4), (2100, 256, 8, 1, 1), (130, 160, 6, 8, 3),
    (67, 60, 4, 6, 2), (33, 384, 8, 8, 4), (700, 512, 10, 16, 5), (50, 64, 8, 32, 8), (40, 8, 8, 1, 1), (7, 1, 1, 1, 1),
    (30, 32, 32, 4, 4), (29, 96, 32, 3, 1), (25, 510, 7, 17, 6), (20, 62, 2, 31, 2), (300, 128, 1, 2, 1),
]


@pytest.mark.parametrize("T,E,k,G,tg", SHAPES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_forward(pkg, T, E, k, G, tg, score, dtype):
    for i, (group, biased, renorm, masked, stride) in enumerate([
            ("top2", True, True, False, None), ("max", False, False, True, None), ("top2", False, True, True, E + 3),
            ("max", True, False, False, E + 3)]):
        rng = np.random.default_rng(T * 31 + E * 7 + i)
        cfg = pkg.ScoreRouterConfig(E, k, score, G, tg, group, renorm, 2.5 if renorm else 1.0)
        bias = (0.1 if score == "sigmoid" else 0.3 / E) * rng.standard_normal(E).astype(np.float32) if biased else None
        mask = rng.random(T) < 0.8 if masked else None
        check(pkg, logits_of(rng, T, E, dtype, 1.5, stride), bias, mask, cfg)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("levels", [1, 3])
def test_ties_and_near_ties(pkg, dtype, levels):
    """Few different logits, so that experts and groups tie; biases of a few levels, which tie too; and values
    whose fp32 scores agree although the exact ones do not."""
    rng = np.random.default_rng(5)
    T, E = 600, 64
    l = rng.integers(0, 3, (T, E)) * 0.5
    bias = (rng.integers(0, levels, E) * 0.25).astype(np.float32)
    for group in ("max", "top2"):
        cfg = pkg.ScoreRouterConfig(E, 6, "sigmoid", 8, 3, group)
        logits = torch.from_numpy(l).float()
        check(pkg, (logits.bfloat16() if dtype == "bf16" else logits).cuda(), bias, None, cfg)
    if dtype == "fp32":
        near = np.float32(9.0) + rng.integers(0, 40, (T, E)).astype(np.float32) * np.float32(2.0 ** -20)
        for b in (None, rng.permutation(E).astype(np.float32) * np.float32(2.0 ** -30)):
            check(pkg, torch.from_numpy(near).cuda(), b, None, pkg.ScoreRouterConfig(E, 6, "sigmoid", 8, 3, "max"))
            check_groups(pkg, near, b, pkg.ScoreRouterConfig(E, 6, "sigmoid", 8, 3, "top2"))


def check_groups(pkg, l, bias, cfg):
    """Sums of two of these scores agree to the last bits of 64: s(9 + x) is a line but for s'' x^2 / 2 <=
    1.3e-4 (40 2^-20)^2 / 2 < 2^-43, so the sums for logits 9 + a d, 9 + b d and 9 + c d, 9 + e d with a + b = c + e
    do. Values nearer than 2^-40 may be taken in either order, so any such set of groups will do; what is
    picked from it has to be right."""
    from itertools import combinations
    T, E = l.shape
    ids = pkg.ScoreRouter(cfg).forward(torch.from_numpy(l).cuda(), None if bias is None else
                                       torch.from_numpy(bias).cuda()).topk_ids.cpu().numpy()
    l = l.astype(np.float64)
    c = scores(l, "sigmoid") + (0.0 if bias is None else bias.astype(np.float64))
    key = l if bias is None else c
    size = E // cfg.num_groups
    value = np.sort(c.reshape(T, cfg.num_groups, size), axis=2)[:, :, -2:].sum(2)
    for t in range(T):
        order = np.lexsort((np.arange(E), -key[t]))
        ok = False
        for kept in combinations(range(cfg.num_groups), cfg.top_groups):
            left = [g for g in range(cfg.num_groups) if g not in kept]
            if value[t, list(kept)].min() > value[t, left].max() - 2.0 ** -40:
                ok = ok or np.array_equal(order[np.isin(order // size, kept)][:cfg.top_k], ids[t])
        assert ok, t


def test_bias_alone_decides_where_scores_are_equal(pkg):
    E = 256
    bias = np.random.default_rng(1).permutation(E).astype(np.float32) * 2.0 ** -12
    for score in ("sigmoid", "softmax"):
        check(pkg, torch.zeros((40, E), device="cuda"), bias, None, pkg.ScoreRouterConfig(E, 8, score, 8, 4))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("scale", [12.0, 60.0])
def test_far_logits(pkg, score, scale):
    """Scores that saturate or vanish: the order without a bias is the logits', weights stay shares."""
    rng = np.random.default_rng(3)
    l = torch.from_numpy(rng.standard_normal((200, 64)) * scale).float().cuda()
    check(pkg, l, None, None, pkg.ScoreRouterConfig(64, 4, score, 1, 1, "max"))
    check(pkg, l - 500.0, None, None, pkg.ScoreRouterConfig(64, 4, score, 4, 2, "max"))


def test_experts_that_may_not_be_taken(pkg):
    rng = np.random.default_rng(9)
    T, E = 90, 32
    l = rng.standard_normal((T, E))
    l[rng.random((T, E)) < 0.6] = -np.inf
    l[3] = -np.inf                 # a row that leaves nothing
    l[4, 8:] = -np.inf             # one group alone
    l[5, :] = -np.inf
    l[5, 17] = 0.5                 # one expert alone
    l[6] = np.finfo(np.float32).min
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    closed = bias.copy()
    closed[::3] = -np.inf
    for b in (None, bias, closed, np.full(E, -np.inf, np.float32)):
        for score in ("sigmoid", "softmax"):
            for group in ("max", "top2"):
                check(pkg, torch.from_numpy(l).float().cuda(), b, None,
                      pkg.ScoreRouterConfig(E, 6, score, 4, 2, group))


def test_not_finite(pkg):
    """NaN sorts first and makes weights NaN, a sigmoid of +inf is 1; other rows do not notice; masked rows
    may hold anything."""
    E, k = 64, 4
    rng = np.random.default_rng(2)
    l = torch.from_numpy(rng.standard_normal((6, E))).float().cuda()
    clean = l.clone()
    l[1, 40] = float("nan")
    l[2, 7] = float("inf")
    l[4] = float("nan")
    bias = torch.from_numpy(0.1 * rng.standard_normal(E)).float().cuda()
    mask = torch.tensor([1, 1, 1, 1, 0, 1], dtype=torch.bool, device="cuda")
    for b in (None, bias):
        for G, tg in ((1, 1), (4, 2)):
            for score in ("sigmoid", "softmax"):
                r = pkg.ScoreRouter(pkg.ScoreRouterConfig(E, k, score, G, tg))
                o, ref = r.forward(l, b, mask), r.forward(clean, b, mask)
                ids = o.topk_ids.cpu().numpy()
                for t in (0, 3, 4, 5):
                    assert torch.equal(o.topk_ids[t], ref.topk_ids[t])
                    assert torch.equal(o.topk_weights[t], ref.topk_weights[t])
                assert (ids[4] == -1).all() and (o.topk_weights[4] == 0).all()
                for t in (1, 2):
                    assert len(set(ids[t])) == k and ids[t].min() >= 0 and ids[t].max() < E
                assert o.num_valid.item() == 5 and o.counts.sum().item() == 5 * k
                assert torch.isnan(o.topk_weights[1]).all()
                if score == "sigmoid":
                    assert ids[1, 0] == 40 and 7 in ids[2] and torch.isfinite(o.topk_weights[2]).all()
                else:
                    assert torch.isnan(o.topk_weights[2]).any()


def test_no_tokens_and_optional_outputs(pkg):
    r = pkg.ScoreRouter(pkg.ScoreRouterConfig(64, 4, num_groups=8, top_groups=4))
    o = r.alloc(0)
    o.counts.fill_(7)
    o.num_valid.fill_(7)
    r.forward(torch.empty((0, 64), device="cuda"), out=o)
    assert (o.counts == 0).all() and o.num_valid.item() == 0
    for T in (9, 900):
        l = torch.randn((T, 64), device="cuda")
        full = r.forward(l)
        part = r.alloc(T)
        part.counts = None
        assert torch.equal(r.forward(l, out=part).topk_ids, full.topk_ids) and part.num_valid.item() == T
        part.num_valid = None
        part.topk_ids.zero_()
        assert torch.equal(r.forward(l, out=part).topk_ids, full.topk_ids)
    assert r.backward(torch.empty((0, 64), device="cuda"), o.topk_ids, torch.empty((0, 4), device="cuda")).shape == (0, 64)


def gradient(l, ids, dw, cfg):
    s = scores(l, cfg.score)
    d = np.zeros_like(s)
    for t in range(len(l)):
        slots = [j for j in range(cfg.top_k) if 0 <= ids[t, j] < cfg.num_experts]
        if not slots:
            continue
        e, g = ids[t, slots], cfg.scale * dw[t, slots]
        x = s[t, e]
        if cfg.renormalize:
            S = x.sum()
            g = (g - (g * x).sum() / S) / S
        if cfg.score == "sigmoid":
            d[t, e] = g * x * (1 - x)
        else:
            full = np.zeros(cfg.num_experts)
            full[e] = g
            d[t] = s[t] * (full - (s[t] * full).sum())
    return d


@pytest.mark.parametrize("T,E,k,G,tg", [s for s in SHAPES if s[0] < 2000])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient(pkg, T, E, k, G, tg, score, dtype, renorm):
    rng = np.random.default_rng(T + E)
    cfg = pkg.ScoreRouterConfig(E, k, score, G, tg, "top2", renorm, 2.5)
    for stride in (None, E + 3):
        logits = logits_of(rng, T, E, dtype, 1.5, stride)
        mask = torch.from_numpy(rng.random(T) < 0.8).cuda()
        r = pkg.ScoreRouter(cfg)
        ids = r.forward(logits, token_mask=mask).topk_ids
        if T > 20:
            ids[11, 0] = -1      # slots without an expert take no gradient, ids out of range neither
            ids[12, -1] = E + 5
            logits[13] = float("nan")
            ids[13] = -1
        dw = rng.standard_normal((T, k))
        out = None
        if stride:
            wide = torch.full((T, stride), 7.0, dtype=logits.dtype, device="cuda")
            out = wide[:, 2:2 + E]
        d = r.backward(logits, ids, torch.from_numpy(dw).float().cuda(), out=out)
        l = np.nan_to_num(logits.float().cpu().numpy().astype(np.float64))
        dw = dw.astype(np.float32).astype(np.float64)
        want = gradient(l, ids.cpu().numpy(), dw, cfg)
        got = d.float().cpu().numpy().astype(np.float64)
        tol = (256 + 8 * np.abs(l).max()) * U * cfg.scale * np.abs(dw).max(1, keepdims=True)
        if dtype == "bf16":
            tol = tol + np.abs(want) * 2.0 ** -8
        assert (np.abs(got - want) <= tol).all()
        if stride:
            assert (wide[:, :2] == 7).all() and (wide[:, 2 + E:] == 7).all()


@pytest.mark.parametrize("score,renorm", [("sigmoid", True), ("sigmoid", False), ("softmax", True), ("softmax", False)])
def test_gradient_against_differences(pkg, score, renorm):
    """Central differences of the weights that the forward pass returns (steps small enough that no choice
    changes, large enough for fp32: the quotient's error is some u / h + h^2)."""
    rng = np.random.default_rng(4)
    T, E, k, h = 16, 32, 4, 2.0 ** -6
    r = pkg.ScoreRouter(pkg.ScoreRouterConfig(E, k, score, 4, 2, "max", renorm, 1.5))
    l = torch.from_numpy(rng.permuted(np.tile(np.linspace(-3, 3, E), (T, 1)), axis=1)).float().cuda()
    dw = torch.from_numpy(rng.standard_normal((T, k))).float().cuda()
    o = r.forward(l)
    d = r.backward(l, o.topk_ids, dw)
    for e in range(E):
        step = torch.zeros((T, E), device="cuda")
        step[:, e] = h
        up, down = r.forward(l + step), r.forward(l - step)
        assert torch.equal(up.topk_ids, o.topk_ids) and torch.equal(down.topk_ids, o.topk_ids)
        diff = ((up.topk_weights.double() - down.topk_weights.double()) * dw.double()).sum(1) / (2 * h)
        assert (diff - d[:, e].double()).abs().max().item() <= 4 * (h * h + 64 * U / h)


def test_bias_step(pkg):
    for E in (1, 60, 512):
        r = pkg.ScoreRouter(pkg.ScoreRouterConfig(E, 1))
        counts = torch.randint(0, 50, (E,), dtype=torch.int32, device="cuda")
        counts[0] = 2 ** 31 - 1 if E > 1 else 3
        if E > 1:
            counts[1] = 2 ** 31 - 1
        bias = torch.randn(E, device="cuda")
        want = bias + 1e-3 * torch.sign(counts.double().mean() - counts.double()).float()
        assert torch.equal(r.update_bias(bias, counts, 1e-3), want)


def test_bias_evens_out_the_loads(pkg):
    """The operators together as in training without a balance loss: loads even out, step by step."""
    g = torch.Generator(device="cuda").manual_seed(0)
    E, T = 64, 4096
    r = pkg.ScoreRouter(pkg.ScoreRouterConfig(E, 4, num_groups=8, top_groups=4))
    l = torch.randn((T, E), generator=g, device="cuda") + torch.linspace(-1, 1, E, device="cuda")
    bias, out = torch.zeros(E, device="cuda"), r.alloc(T)
    first = r.forward(l, bias, out=out).counts.max().item()
    for _ in range(300):
        r.forward(l, bias, out=out)
        r.update_bias(bias, out.counts, 2e-3)
    assert r.forward(l, bias, out=out).counts.max().item() < first


def test_deterministic_and_captured(pkg):
    g = torch.Generator(device="cuda").manual_seed(3)
    T, E = 3001, 256
    r = pkg.ScoreRouter(pkg.ScoreRouterConfig(E, 8, num_groups=8, top_groups=4))
    l, bias = torch.randn((T, E), generator=g, device="cuda"), 0.1 * torch.randn(E, generator=g, device="cuda")
    dw, out, d = torch.randn((T, 8), generator=g, device="cuda"), r.alloc(T), torch.empty_like(l)
    eager = r.forward(l, bias)
    grad = r.backward(l, eager.topk_ids, dw)
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        r.forward(l, bias, out=out)
        with torch.cuda.graph(graph, stream=s):
            r.forward(l, bias, out=out)
            r.backward(l, out.topk_ids, dw, out=d)
    torch.cuda.synchronize()
    for _ in range(2):
        out.workspace.fill_(0xFF)
        d.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.topk_ids, eager.topk_ids) and torch.equal(out.topk_weights, eager.topk_weights)
        assert torch.equal(out.counts, eager.counts) and torch.equal(d, grad)


def test_rows_past_two_to_the_31_elements(pkg):
    """Offsets of rows and of gradients beyond 2^31 elements: a row stride of 2^23 + 8."""
    E, T, ld = 64, 300, 2 ** 23 + 8
    buf = torch.zeros(T * ld, dtype=torch.bfloat16, device="cuda")
    wide = buf.view(T, ld)[:, :E]
    l = torch.randn((T, E), device="cuda").bfloat16()
    wide.copy_(l)
    r = pkg.ScoreRouter(pkg.ScoreRouterConfig(E, 4, num_groups=4, top_groups=2))
    a, b = r.forward(wide), r.forward(l)
    assert torch.equal(a.topk_ids, b.topk_ids) and torch.equal(a.topk_weights, b.topk_weights)
    dw = torch.randn((T, 4), device="cuda")
    want = r.backward(l, b.topk_ids, dw)
    r.backward(l, b.topk_ids, dw, out=wide)
    assert torch.equal(wide, want)
