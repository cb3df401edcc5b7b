"""The operators around the experts (residual add with RMSNorm and quantised outputs, router with
balance loss and its gradient, microscaled linear product) against plain 64-bit NumPy versions.

Tolerances, from the arithmetic (u = 2^-24, half(v) = half a bf16 step at v):
  sum      fp32 add, one bf16 rounding:                    half + 2u|z|
  norm     64 terms a thread at most, 13 joins, a root:    half + 64u|y|
  codes    the format's nearest code of a value 64u off:   half a code step, widened by 2^-10
  quantise codes and scales of bf16 rows:                  equal, byte for byte
  router   ids, counts: equal; p: exp of a rounded difference d and a sum of E terms:
           (64 + |d|) u relative; its mean: plus one u per addend of the fixed-order sum
  linear   fp4 products are exact, fp32 sums:              half + 2^-20 sum|x w|
           MXFP8: the layer's own bound                    half + 2e-2 rms + 1e-3
"""
import numpy as np
import pytest
import torch

from oracle import formats as OF

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)


@pytest.fixture(scope="module")
def pkg():
    import serving_topk_permute_gb300 as p
    p.lib()
    return p


def bf16_dev(v, stride=None, offset=0):
    """v (float) rounded to bf16 on the device, rows `stride` elements apart, `offset` elements in."""
    t = torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).cuda().bfloat16()
    if stride is None and offset == 0:
        return t
    R, K = t.shape
    stride = stride or K
    buf = torch.zeros(R * stride + offset + K, dtype=torch.bfloat16, device="cuda")
    out = buf[offset:].as_strided((R, K), (stride, 1))
    out.copy_(t)
    return out


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def half_step(v):
    """Half a bf16 step at |v|."""
    m = np.maximum(np.abs(v), 2.0 ** -126)
    return np.ldexp(1.0, (np.floor(np.log2(m)) - 8).astype(np.int64))


def assert_within(got, want, tol, what):
    d = np.abs(got - want)
    bad = ~(d <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, worst {np.nanmax(d - tol):.3e} over at " \
                          f"{np.argwhere(bad)[0]}"


def rows_of(rng, T, H, big=True):
    x = rng.standard_normal((T, H))
    if big and H > 3:
        x[:, :: max(H // 3, 1)] *= 40.0
    return x


# ----------------------------------------------------------------------------- quantisation

FMTS = ("mxfp8", "nvfp4", "mxfp4")


def oracle_quantize(x, fmt):
    """Codes, row-major scales and row scales (or None) of fp32-representable rows."""
    if fmt == "mxfp8":
        return (*OF.mxfp8_quantize(x), None)
    if fmt == "mxfp4":
        return (*OF.mxfp4_quantize(x), None)
    gs = OF.nvfp4_global_scale(np.abs(x).max(axis=1))
    return (*OF.nvfp4_quantize(x, gs), gs)


def dequantize(codes, sf, gs, fmt):
    if fmt == "mxfp8":
        return OF.mxfp8_dequantize(codes, sf)
    if fmt == "mxfp4":
        return OF.mxfp4_dequantize(codes, sf)
    return OF.nvfp4_dequantize(codes, sf, gs)


def atoms_to_rows(atoms, rows, K, fmt):
    """Row-major scales out of the atom layout, and the bytes past K (which have to be zero)."""
    S = {"mxfp8": 1, "mxfp4": 2, "nvfp4": 4}[fmt]
    g = 16 if fmt == "nvfp4" else 32
    row_bytes = K if fmt == "mxfp8" else K // 2
    nks = -(-row_bytes // 128)
    a = atoms.reshape(-1, nks, S, 32, 4, 4)                    # [tile][stage][s][i][j][b]
    a = a.transpose(0, 4, 3, 1, 2, 5).reshape(-1, nks * S * 4)  # row 32 j + i of a tile, blocks in order
    return a[:rows, : K // g], a[:rows, K // g:]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,K,stride,offset", [
    (1, 32, None, 0), (3, 64, None, 0), (5, 96, 100, 1), (130, 2080, None, 0), (257, 416, 424, 8), (2, 16384, None, 0),
    (33, 8224, 8230, 3),
])
def test_quantize_equals_the_oracle(pkg, fmt, rows, K, stride, offset):
    rng = np.random.default_rng(rows * 1000 + K)
    x = bf16_dev(rows_of(rng, rows, K) * 2.0 ** rng.integers(-20, 20, (rows, 1)), stride, offset)
    if rows > 2:
        x[1].zero_()
        x[2, :32] = 0
    want, wsf, wgs = oracle_quantize(f64(x), fmt)
    q = pkg.quantize(x, fmt, "rows")
    np.testing.assert_array_equal(q.codes.cpu().numpy(), want)
    np.testing.assert_array_equal(q.sf.cpu().numpy()[: wsf.size].reshape(wsf.shape), wsf)
    qa = pkg.quantize(x, fmt, "atoms")
    np.testing.assert_array_equal(qa.codes.cpu().numpy(), want)
    got, past = atoms_to_rows(qa.sf.cpu().numpy(), rows, K, fmt)
    np.testing.assert_array_equal(got, wsf)
    assert not past.any()
    if fmt == "nvfp4":
        np.testing.assert_array_equal(q.row_scale.cpu().numpy(), wgs)
        np.testing.assert_array_equal(qa.row_scale.cpu().numpy(), wgs)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_quantize_marks_what_is_not_finite(pkg, fmt, bad):
    x = torch.randn(4, 128, device="cuda").bfloat16()
    clean = pkg.quantize(x, fmt, "rows")
    y = x.clone()
    y[1, 40] = bad
    q = pkg.quantize(y, fmt, "rows")
    sf, ref = q.sf.view(4, -1).cpu().numpy(), clean.sf.view(4, -1).cpu().numpy()
    if fmt == "nvfp4":
        assert np.isnan(q.row_scale[1].item())
        assert torch.equal(q.row_scale[[0, 2, 3]], clean.row_scale[[0, 2, 3]])
    else:
        assert sf[1, 1] == 255
        keep = np.ones_like(sf, dtype=bool)
        keep[1, 1] = False
        np.testing.assert_array_equal(sf[keep], ref[keep])
    assert torch.equal(q.codes[[0, 2, 3]], clean.codes[[0, 2, 3]])


# ----------------------------------------------------------------------------- norm

def norm64(x, r, gamma):
    z = x + (0.0 if r is None else r)
    return z, z / np.sqrt((z * z).mean(axis=1, keepdims=True) + EPS) * gamma


@pytest.mark.parametrize("T,H", [(1, 1), (1, 7), (3, 8), (5, 130), (2, 2050), (130, 1000), (7, 4096), (3, 7168),
                                 (2, 8200), (2, 16384), (2, 16383), (2, 16382)])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("stride", [0, 5, 8])
def test_norm_bf16(pkg, T, H, residual, stride):
    rng = np.random.default_rng(T * 7 + H)
    x = bf16_dev(rows_of(rng, T, H), H + stride)
    r = bf16_dev(3 * rows_of(rng, T, H), H + stride) if residual else None
    gamma = 1.0 + 0.2 * rng.standard_normal(H)
    g = torch.from_numpy(gamma.astype(np.float32)).cuda()
    out = torch.full((T, H + stride), 7.0, dtype=torch.bfloat16, device="cuda")
    total = torch.full((T, H + stride), 7.0, dtype=torch.bfloat16, device="cuda")
    got = pkg.add_rmsnorm(x, g, EPS, residual=r, sum_out=total[:, :H], out=out[:, :H])
    z, y = norm64(f64(x), None if r is None else f64(r), f64(g))
    assert_within(f64(got), y, half_step(y) * 1.01 + 64 * U * np.abs(y), "out")
    assert_within(f64(total[:, :H]), z, half_step(z) * 1.01 + 2 * U * np.abs(z), "sum")
    assert (out[:, H:] == 7).all() and (total[:, H:] == 7).all()


def test_norm_in_place_and_defaults(pkg):
    x = torch.randn(33, 512, device="cuda").bfloat16()
    r = torch.randn(33, 512, device="cuda").bfloat16()
    g = torch.rand(512, device="cuda") + 0.5
    total = torch.empty_like(x)
    want = pkg.add_rmsnorm(x, g, EPS, residual=r, sum_out=total)
    x2, r2 = x.clone(), r.clone()
    got = pkg.add_rmsnorm(x2, g, EPS, residual=r2, sum_out=r2, out=x2)
    assert torch.equal(got, want) and torch.equal(r2, total) and got.data_ptr() == x2.data_ptr()
    # zero rows: the norm of zero is zero, with eps alone under the root
    assert (pkg.add_rmsnorm(torch.zeros_like(x), g, EPS) == 0).all()
    assert pkg.add_rmsnorm(x[:0], g, EPS).shape == (0, 512)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,H,stride,layout", [(1, 32, 0, "rows"), (5, 96, 3, "rows"), (130, 2080, 0, "atoms"),
                                               (3, 7168, 8, "rows"), (2, 16384, 0, "atoms")])
def test_norm_quantised(pkg, fmt, T, H, stride, layout):
    rng = np.random.default_rng(T + H)
    x, r = bf16_dev(rows_of(rng, T, H), H + stride), bf16_dev(3 * rows_of(rng, T, H), H + stride)
    g = torch.from_numpy((1.0 + 0.2 * rng.standard_normal(H)).astype(np.float32)).cuda()
    q = pkg.Quantized.alloc(fmt, T, H, layout)
    out, total = torch.empty((T, H), dtype=torch.bfloat16, device="cuda"), torch.empty_like(x)
    pkg.add_rmsnorm(x, g, EPS, residual=r, sum_out=total, out=out, quantized=q)
    z, y = norm64(f64(x), f64(r), f64(g))
    assert_within(f64(out), y, half_step(y) * 1.01 + 64 * U * np.abs(y), "out")
    assert_within(f64(total), z, half_step(z) * 1.01 + 2 * U * np.abs(z), "sum")
    codes, sf = q.codes.cpu().numpy(), q.sf.cpu().numpy()
    B = 16 if fmt == "nvfp4" else 32
    sf = atoms_to_rows(sf, T, H, fmt)[0] if layout == "atoms" else sf.reshape(T, H // B)
    gs = q.row_scale.cpu().numpy() if fmt == "nvfp4" else None
    got = dequantize(codes, sf, gs, fmt)
    blocks = np.abs(y).reshape(T, H // B, B).max(axis=2)
    if fmt == "nvfp4":
        want_gs = np.abs(y).max(axis=1) / 2688.0
        assert_within(gs.astype(np.float64), want_gs, 70 * U * want_gs, "row scale")
        # block scales: nearest E4M3 of amax_b / (gs 6), whose quotient is a few u off
        ratio = blocks / (6.0 * want_gs[:, None])
        s = OF.E4M3_TABLE[sf]
        step = np.maximum(np.ldexp(1.0, (np.floor(np.log2(np.maximum(ratio, 2.0 ** -6))) - 3).astype(int)), 2.0 ** -9)
        assert_within(s, ratio, step / 2 * (1 + 2.0 ** -10), "block scale")
        scale = s * gs.astype(np.float64)[:, None]
    else:
        top = 448.0 if fmt == "mxfp8" else 6.0
        scale = np.ldexp(1.0, sf.astype(np.int64) - 127)
        lo, hi = blocks * (1 - 70 * U), blocks * (1 + 70 * U)
        assert (top * scale >= lo).all() and ((top * scale / 2 < hi) | (blocks == 0)).all()
    v = np.abs(y) / np.where(scale > 0, scale, 1.0).repeat(B, axis=1)
    if fmt == "mxfp8":
        step = np.maximum(np.ldexp(1.0, (np.floor(np.log2(np.maximum(v, 2.0 ** -6))) - 3).astype(int)), 2.0 ** -9)
    else:
        step = np.where(v < 2.0, 0.5, np.where(v < 4.0, 1.0, 2.0))
    limit = 448.0 if fmt == "mxfp8" else 6.0
    room = np.maximum(step / 2 * (1 + 2.0 ** -10), (v - limit))  # past the top code: saturated
    assert_within(got, y, room * scale.repeat(B, axis=1) + 64 * U * np.abs(y), "dequantised")


# ----------------------------------------------------------------------------- router

def router64(logits, mask, k, renorm, coef):
    """Plain 64-bit router. Masked or empty rows: ids -1, weights 0."""
    l = logits.astype(np.float64)
    T, E = l.shape
    ids, w, p = np.full((T, k), -1, np.int32), np.zeros((T, k)), np.zeros((T, E))
    counts, n = np.zeros(E, np.int64), 0
    for t in range(T):
        if (mask is not None and not mask[t]) or (l[t] == -np.inf).all():
            continue
        n += 1
        nan_first = np.where(np.isnan(l[t]), np.inf, l[t])
        order = sorted(range(E), key=lambda e: (not np.isnan(l[t][e]), -nan_first[e], e))[:k]
        with np.errstate(invalid="ignore"):
            e = np.exp(l[t] - (np.nan if np.isnan(l[t]).any() else l[t].max()))
            p[t] = e / e.sum()
        taken = [i for i in order if not l[t][i] == -np.inf]
        for j, i in enumerate(taken):
            ids[t, j] = i
            counts[i] += 1
        w[t, : len(taken)] = p[t, taken] / (p[t, taken].sum() if renorm else 1.0)
    mean = p.sum(axis=0) / max(n, 1)
    return ids, w, counts, n, mean, coef * E * (counts / (k * max(n, 1)) * mean).sum(), p


def check_router(pkg, logits_dev, mask, k, renorm=True, coef=0.02):
    E = logits_dev.shape[1]
    r = pkg.Router(pkg.RouterConfig(E, k, renorm, coef))
    m = None if mask is None else torch.from_numpy(mask).cuda()
    o = r.forward(logits_dev, token_mask=m, training=True)
    l = f64(logits_dev)
    ids, w, counts, n, mean, loss, p = router64(l, mask, k, renorm, coef)
    np.testing.assert_array_equal(o.topk_ids.cpu().numpy(), ids)
    np.testing.assert_array_equal(o.counts.cpu().numpy(), counts)
    assert o.num_valid.item() == n
    d = np.nanmax(np.where(np.isfinite(l), np.abs(l), 0)) * 2 if l.size else 0.0
    got = f64(o.topk_weights)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(w))
    fine = ~np.isnan(w)
    assert_within(got[fine], w[fine], 2 * (64 + d) * U * w[fine] + 1e-37, "weights")
    rel = (64 + d + len(l) / 4000 + 620) * U
    if np.isnan(mean).any():
        np.testing.assert_array_equal(np.isnan(f64(o.prob_mean)), np.isnan(mean))
        assert np.isnan(o.loss.item())
    else:
        assert_within(f64(o.prob_mean), mean, rel * mean + 1e-37, "prob_mean")
        assert_within(f64(o.loss), np.array([loss]), (rel + 16 * U) * abs(loss), "loss")
    # serving form: ids and weights alone, same bits
    s = r.alloc(len(l))
    s.counts = s.num_valid = None
    r.forward(logits_dev, token_mask=m, out=s)
    assert torch.equal(s.topk_ids, o.topk_ids)
    assert torch.equal(s.topk_weights.view(torch.int32), o.topk_weights.view(torch.int32))
    again = r.forward(logits_dev, token_mask=m, training=True)
    for name in ("topk_weights", "prob_mean", "loss"):
        assert torch.equal(getattr(again, name).view(torch.int32), getattr(o, name).view(torch.int32)), name
    return o


@pytest.mark.parametrize("T,E,k", [(0, 8, 2), (1, 1, 1), (1, 8, 8), (3, 5, 2), (64, 8, 2), (130, 60, 6), (77, 64, 8),
                                   (200, 96, 4), (33, 129, 32), (128, 256, 8), (1000, 256, 8), (65, 512, 10),
                                   (3000, 16, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("masked,renorm", [(False, True), (True, False)])
def test_router(pkg, T, E, k, dtype, masked, renorm):
    rng = np.random.default_rng(T + 31 * E + k)
    l = torch.from_numpy((2 * rng.standard_normal((T, E + 3))).astype(np.float32)).cuda().to(dtype)[:, :E]
    check_router(pkg, l, rng.random(T) < 0.7 if masked else None, k, renorm)


def test_router_ties_go_to_the_lowest_expert(pkg):
    l = torch.zeros(9, 100, device="cuda")
    l[1, ::2] = -0.0
    l[2] = torch.arange(100, device="cuda") // 10
    l[3, 64:] = 1.0
    o = check_router(pkg, l, None, 7)
    assert o.topk_ids[0].tolist() == list(range(7)) == o.topk_ids[1].tolist()
    assert o.topk_ids[2].tolist() == list(range(90, 97))
    assert o.topk_ids[3].tolist() == list(range(64, 71))


def test_router_empty_and_masked_rows(pkg):
    """Rows of -inf, rows with fewer finite experts than k, the lowest finite value, and NaN or
    infinity in masked rows, which must reach no output."""
    inf, low = float("inf"), torch.finfo(torch.float32).min
    rng = np.random.default_rng(3)
    l = torch.from_numpy(rng.standard_normal((12, 40)).astype(np.float32)).cuda()
    mask = np.ones(12, bool)
    l[0] = -inf
    l[1, 2:] = -inf
    l[2] = low
    l[3, 1:] = low
    l[4], l[5, 3], l[6] = float("nan"), inf, -inf
    mask[[4, 5, 6, 7]] = False
    l[8, :39] = -inf
    o = check_router(pkg, l, mask, 4)
    assert torch.isfinite(o.loss).all() and o.num_valid.item() == 7
    assert o.topk_ids[1].tolist()[2:] == [-1, -1] and o.topk_ids[8].tolist() == [39, -1, -1, -1]
    for everyone in (np.zeros(12, bool),):
        o = check_router(pkg, l, everyone, 4)
        assert o.loss.item() == 0.0 and o.num_valid.item() == 0 and (o.topk_ids == -1).all()


def test_router_not_a_number_in_a_valid_row(pkg):
    l = torch.zeros(3, 33, device="cuda")
    l[0, 7] = float("nan")
    l[0, 20] = -torch.tensor(float("nan"))
    l[1, 5] = float("inf")
    o = check_router(pkg, l, None, 3)
    assert o.topk_ids[0].tolist() == [7, 20, 0] and o.topk_ids[1].tolist() == [5, 0, 1]


def grad64(l, mask, ids, counts, n, k, renorm, coef, dw, dloss):
    T, E = l.shape
    d = np.zeros((T, E))
    for t in range(T):
        if (mask is not None and not mask[t]) or (l[t] == -np.inf).all():
            continue
        e = np.exp(l[t] - l[t].max())
        p = e / e.sum()
        g = dloss * coef * E * counts / (k * max(n, 1) ** 2) if dloss is not None else np.zeros(E)
        g = g.astype(np.float64).copy()
        at = [j for j in range(k) if ids[t, j] >= 0]
        if dw is not None:
            sel = ids[t, at]
            w = dw[t, at]
            if renorm:
                s = p[sel].sum()
                w = (w - (w * p[sel]).sum() / s) / s
            g[sel] += w
        d[t] = p * (g - (p * g).sum())
    return d


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 8), (3, 5, 2), (77, 64, 8), (40, 129, 32), (200, 256, 8),
                                   (31, 512, 10)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("masked,renorm,parts", [(False, True, "both"), (True, False, "both"), (True, True, "weights"),
                                                 (True, True, "loss")])
def test_router_gradient_formula(pkg, T, E, k, dtype, masked, renorm, parts):
    rng = np.random.default_rng(T + 17 * E + k)
    l = torch.from_numpy((2 * rng.standard_normal((T, E + 3))).astype(np.float32)).cuda().to(dtype)[:, :E]
    if T > 2 and E > 2:
        l[0] = -float("inf")
        l[1, 1:] = -float("inf")
    mask = rng.random(T) < 0.7 if masked else None
    r = pkg.Router(pkg.RouterConfig(E, k, renorm, 0.3))
    m = None if mask is None else torch.from_numpy(mask).cuda()
    o = r.forward(l, token_mask=m, training=True)
    dw = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda() if parts != "loss" else None
    dl = torch.full((1,), 1.7, device="cuda") if parts != "weights" else None
    got = r.backward(l, o.topk_ids, o.counts, o.num_valid, d_weights=dw, d_loss=dl, token_mask=m)
    assert got.dtype == dtype
    ids, counts, n = o.topk_ids.cpu().numpy(), o.counts.cpu().numpy(), o.num_valid.item()
    want = grad64(f64(l), mask, ids, counts, n, k, renorm, 0.3, None if dw is None else f64(dw),
                  None if dl is None else f64(dl)[0])
    # p (g - p.g): both parts carry a few tens of u relative to their own size, the sums too
    size = np.abs(want).max(axis=1, keepdims=True) if E > 1 else np.ones((T, 1))
    tol = 400 * U * np.maximum(size, 1e-6)
    if dtype is torch.bfloat16:
        tol = tol + half_step(want) * 1.01
    assert_within(f64(got), want, tol, "d_logits")


def test_router_gradient_against_differences(pkg):
    """Central differences of the 64-bit objective sum(dw w) + dl loss, counts held constant."""
    T, E, k, coef, dl = 6, 12, 3, 0.5, 0.8
    rng = np.random.default_rng(11)
    l = rng.standard_normal((T, E)).astype(np.float32).astype(np.float64)
    mask = np.array([1, 1, 0, 1, 1, 1], bool)
    for renorm in (True, False):
        r = pkg.Router(pkg.RouterConfig(E, k, renorm, coef))
        dev = torch.from_numpy(l.astype(np.float32)).cuda()
        m = torch.from_numpy(mask).cuda()
        o = r.forward(dev, token_mask=m, training=True)
        dw = rng.standard_normal((T, k)).astype(np.float32)
        got = f64(r.backward(dev, o.topk_ids, o.counts, o.num_valid, d_weights=torch.from_numpy(dw).cuda(),
                             d_loss=torch.full((1,), dl, device="cuda"), token_mask=m))
        ids, counts, n = o.topk_ids.cpu().numpy(), o.counts.cpu().numpy(), o.num_valid.item()

        def objective(x):
            p = np.exp(x) / np.exp(x).sum(axis=1, keepdims=True)
            total = 0.0
            for t in np.flatnonzero(mask):
                w = p[t, ids[t]]
                total += (dw[t].astype(np.float64) * (w / w.sum() if renorm else w)).sum()
            return total + np.float32(dl) * coef * E * (counts / (k * n) * p[mask].sum(axis=0) / n).sum()

        h = 1e-5
        for t in range(T):
            for e in range(E):
                up, down = l.copy(), l.copy()
                up[t, e] += h
                down[t, e] -= h
                diff = (objective(up) - objective(down)) / (2 * h)
                # h^2 of the differences, 1e-11 / h of their cancellation, the kernel's own rounding
                assert abs(got[t, e] - diff) <= 1e-6 + 400 * U, (t, e)


# ----------------------------------------------------------------------------- linear product

def linear_case(pkg, fmt, M, N, K, seed=0, x_stride=None):
    rng = np.random.default_rng(seed + M * 3 + N * 5 + K)
    x = bf16_dev(rows_of(rng, M, K) * np.exp(0.5 * rng.standard_normal((1, K))), x_stride)
    w = (rng.standard_normal((N, K)) / np.sqrt(K)).astype(np.float32)
    if fmt == "nvfp4":
        gs = OF.nvfp4_global_scale(np.abs(w).max()).reshape(1)
        codes, sf = OF.nvfp4_quantize(w, gs)
        wd = OF.nvfp4_dequantize(codes, sf, np.broadcast_to(gs, (N,)))
    else:
        gs = None
        codes, sf, _ = oracle_quantize(w.astype(np.float64), fmt)
        wd = dequantize(codes, sf, None, fmt)
    plan = pkg.LinearPlan(pkg.LinearConfig(N, K, max(M, 1), fmt))
    kw = plan.transform_weight(torch.from_numpy(codes).cuda(), torch.from_numpy(sf).cuda(),
                               None if gs is None else torch.from_numpy(gs.astype(np.float32)).cuda())
    return plan, kw, x, wd


def check_linear(got, x, wd, fmt, what=""):
    xd = dequantize(*oracle_quantize(f64(x), fmt), fmt)
    want = xd @ wd.T
    if fmt == "mxfp8":
        tol = half_step(want) * 1.01 + 2e-2 * np.sqrt(np.mean(want ** 2)) + 1e-3
    else:
        tol = half_step(want) * 1.01 + 2.0 ** -20 * (np.abs(xd) @ np.abs(wd).T)
    assert_within(f64(got), want, tol, f"{fmt} {what}")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 32), (1, 8, 64), (1, 264, 256), (2, 33, 96), (1, 4096, 2048), (3, 520, 7168), (4, 257, 288), (5, 100, 1056), (8, 1000, 512),
    (9, 256, 4096), (16, 2048, 768), (17, 640, 1056), (31, 96, 224), (32, 1536, 4096), (33, 264, 512), (63, 127, 320), (64, 520, 2080),
    (65, 129, 96), (100, 333, 2048), (127, 256, 544), (128, 2304, 1024), (129, 257, 256), (200, 4100, 288),
    (300, 520, 2080), (384, 1032, 16384), (513, 40, 64), (1200, 2600, 512),
])
def test_linear(pkg, fmt, M, N, K):
    plan, kw, x, wd = linear_case(pkg, fmt, M, N, K)
    ws = plan.alloc_workspace(M)
    ws.fill_(0xA5)  # what a workspace held before does not matter
    out = torch.full((M, N + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    plan.forward(x, kw, out=out[:, :N], workspace=ws)
    assert plan.last_status(ws) == 0
    check_linear(out[:, :N], x, wd, fmt, f"{M}x{N}x{K}")
    assert (out[:, N:] == 7).all()
    # contiguous output, the same inputs again, and the quantised form: same bits
    got = plan.forward(x, kw)
    assert torch.equal(got.view(torch.int16), out[:, :N].contiguous().view(torch.int16))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("K", [96, 2048, 7168, 16384])
@pytest.mark.parametrize("M", [2, 3, 6, 8, 9])
def test_linear_around_the_counts_that_are_quantised_inside(pkg, fmt, M, K):
    """From bf16 rows, and from the same rows quantised by quantize(): the same bits on both ways."""
    plan, kw, x, wd = linear_case(pkg, fmt, M, 392, K)
    got = plan.forward(x, kw)
    check_linear(got, x, wd, fmt, f"{M}x392x{K}")
    rows = plan.forward(pkg.quantize(x, fmt), kw)
    assert torch.equal(got.view(torch.int16), rows.view(torch.int16))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(1, 512, 1024), (7, 96, 96), (40, 300, 2080), (200, 1000, 512)])
def test_linear_from_quantised_rows(pkg, fmt, M, N, K):
    """Quantised input by quantize() or by the norm gives what the bf16 form gives on the same values."""
    plan, kw, x, wd = linear_case(pkg, fmt, M, N, K, x_stride=K + 5)
    want = plan.forward(x, kw)
    check_linear(want, x, wd, fmt)
    ws = plan.alloc_workspace(M)
    ws.fill_(0xA5)
    got = plan.forward(pkg.quantize(x, fmt), kw, workspace=ws)
    assert plan.last_status(ws) == 0
    check_linear(got, x, wd, fmt, "from quantised rows")
    q = pkg.Quantized.alloc(fmt, M, K)
    gamma = torch.rand(K, device="cuda") + 0.5
    pkg.add_rmsnorm(x, gamma, EPS, quantized=q)
    got = plan.forward(q, kw)
    sf = atoms_to_rows(q.sf.cpu().numpy(), M, K, fmt)[0]
    xd = dequantize(q.codes.cpu().numpy(), sf, None if fmt != "nvfp4" else q.row_scale.cpu().numpy(), fmt)
    ref = xd @ wd.T
    tol = half_step(ref) * 1.01 + (2e-2 * np.sqrt(np.mean(ref ** 2)) + 1e-3 if fmt == "mxfp8"
                                   else 2.0 ** -20 * (np.abs(xd) @ np.abs(wd).T))
    assert_within(f64(got), ref, tol, "from the norm")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 20, 140])
def test_linear_keeps_bad_rows_apart(pkg, fmt, M):
    """A row with a NaN or an infinity gives a row of NaN; the others keep their bits."""
    plan, kw, x, _ = linear_case(pkg, fmt, M, 300, 512)
    want = plan.forward(x, kw)
    y = x.clone()
    y[M - 1, 100] = float("nan")
    if M > 3:
        y[2, 511] = float("inf")
    got = plan.forward(y, kw)
    bad = [M - 1] + ([2] if M > 3 else [])
    good = [i for i in range(M) if i not in bad]
    assert torch.isnan(got[bad]).all()
    assert torch.equal(got[good].view(torch.int16), want[good].view(torch.int16))


@pytest.mark.parametrize("fmt", FMTS)
def test_linear_rows_do_not_depend_on_the_batch_around_them(pkg, fmt):
    """Zero rows give zeros."""
    plan, kw, x, _ = linear_case(pkg, fmt, 130, 264, 512)
    x[5].zero_()
    x[129].zero_()
    got = plan.forward(x, kw)
    assert (got[[5, 129]] == 0).all() and (got[4] != 0).any()
    assert plan.forward(x[:0], kw).shape == (0, 264)


# ----------------------------------------------------------------------------- streams, graphs, guards

def _everything(pkg, st, bufs):
    x, r, g, q, total, h, router, logits, ro, plan, kw, out, ws, dl = bufs
    pkg.add_rmsnorm(x, g, EPS, residual=r, sum_out=total, out=h, quantized=q, stream=st)
    router.forward(logits, out=ro, stream=st)
    router.backward(logits, ro.topk_ids, ro.counts, ro.num_valid, d_weights=ro.topk_weights, d_loss=ro.loss,
                    out=dl, stream=st)
    plan.forward(q, kw, out=out[0], workspace=ws, stream=st)
    plan.forward(h, kw, out=out[1], workspace=ws, stream=st)


def _buffers(pkg, fmt, T=96, H=512, N=520, E=64):
    plan, kw, x, _ = linear_case(pkg, fmt, T, N, H)
    r = torch.randn(T, H, device="cuda").bfloat16()
    router = pkg.Router(pkg.RouterConfig(E, 4, True, 0.1))
    return (x, r, torch.rand(H, device="cuda") + 0.5, pkg.Quantized.alloc(fmt, T, H), torch.empty_like(r),
            torch.empty_like(r), router, torch.randn(T, E, device="cuda"), router.alloc(T, training=True), plan, kw,
            [torch.empty((T, N), dtype=torch.bfloat16, device="cuda") for _ in range(2)], plan.alloc_workspace(T),
            torch.empty((T, E), device="cuda"))


def _results(bufs):
    q, total, h, ro, out, dl = bufs[3], bufs[4], bufs[5], bufs[8], bufs[11], bufs[13]
    return [t.clone() for t in (q.codes, total, h, ro.topk_ids, ro.topk_weights, ro.counts, ro.loss, *out, dl)]


@pytest.mark.parametrize("fmt", FMTS)
def test_other_stream_and_graph(pkg, fmt):
    bufs = _buffers(pkg, fmt)
    _everything(pkg, None, bufs)
    torch.cuda.synchronize()
    want = _results(bufs)
    side = torch.cuda.Stream()
    for t in (bufs[4], bufs[5], *bufs[11]):
        t.zero_()
    torch.cuda.synchronize()
    _everything(pkg, side, bufs)
    side.synchronize()
    for a, b in zip(_results(bufs), want):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        _everything(pkg, side, bufs)
    bufs[0].mul_(0.5)
    bufs[7].neg_()
    graph.replay()
    torch.cuda.synchronize()
    replayed = _results(bufs)
    _everything(pkg, None, bufs)
    torch.cuda.synchronize()
    for a, b in zip(replayed, _results(bufs)):
        assert torch.equal(a, b)
    assert not torch.equal(replayed[1], want[1])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [1, 13, 96, 300])
def test_nothing_outside_the_buffers_is_written(pkg, fmt, T):
    G, H, N, E = 4096, 480, 260, 60
    kept = []

    def guarded(nbytes):
        buf = torch.full((2 * G + nbytes,), 0xA5, dtype=torch.uint8, device="cuda")
        kept.append((buf, nbytes))
        return buf[G:G + nbytes]

    plan, kw, x, _ = linear_case(pkg, fmt, T, N, H)
    before = [t.clone() for t in (x, kw.codes, kw.sf)]
    q = pkg.Quantized(fmt, (T, H), guarded(T * H // pkg.block.VALUES_PER_BYTE[fmt]),
                      guarded(pkg.sf_size(fmt, "atoms", T, H)),
                      guarded(4 * T).view(torch.float32) if fmt == "nvfp4" else None, "atoms")
    bf = torch.bfloat16
    total, h, out = guarded(2 * T * H).view(bf).view(T, H), guarded(2 * T * H).view(bf).view(T, H), \
        guarded(2 * T * N).view(bf).view(T, N)
    pkg.add_rmsnorm(x, torch.ones(H, device="cuda"), EPS, residual=x, sum_out=total, out=h, quantized=q)
    plan.forward(h, kw, out=out, workspace=guarded(plan.workspace_size(T)))
    plan.forward(q, kw, out=out, workspace=guarded(plan.workspace_size(T)))
    router = pkg.Router(pkg.RouterConfig(E, 5, True, 0.1))
    i32, f32 = torch.int32, torch.float32
    o = pkg.RouterOutput(guarded(20 * T).view(i32).view(T, 5), guarded(20 * T).view(f32).view(T, 5),
                         guarded(4 * E).view(i32), guarded(4).view(i32), guarded(4 * E).view(f32), guarded(4).view(f32),
                         guarded(router.workspace_size(T)))
    logits = torch.randn(T, E, device="cuda")
    router.forward(logits, out=o)
    router.backward(logits, o.topk_ids, o.counts, o.num_valid, d_weights=o.topk_weights, d_loss=o.loss,
                    out=guarded(4 * T * E).view(f32).view(T, E))
    torch.cuda.synchronize()
    for buf, n in kept:
        assert (buf[:G] == 0xA5).all() and (buf[G + n:] == 0xA5).all(), n
    for a, b in zip(before, (x, kw.codes, kw.sf)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_linear_wait_limit_reports_and_the_context_survives(pkg):
    """With a limit of 1 ns the product's waits run out: the call returns, the status says so, and
    the default limit then gives the usual output."""
    plan, kw, x, _ = linear_case(pkg, "nvfp4", 300, 1024, 4096)
    ws = plan.alloc_workspace(300)
    want = plan.forward(x, kw, workspace=ws)
    assert plan.last_status(ws) == 0
    plan.set_wait_timeout(1)
    plan.forward(x, kw, workspace=ws)
    assert plan.last_status(ws) == 7
    assert plan.last_status(ws) == 0
    plan.set_wait_timeout(0)
    got = plan.forward(x, kw, workspace=ws)
    assert plan.last_status(ws) == 0
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("fmt,M,N,K", [("nvfp4", 1, 1024, 8192), ("mxfp8", 3, 520, 4096), ("mxfp4", 40, 2048, 7168),
                                       ("mxfp8", 700, 4104, 2048), ("nvfp4", 600, 8200, 1056)])
def test_linear_wait_limit_in_every_kernel(pkg, fmt, M, N, K):
    """The same for a product that quantises x itself, split ones and CTA pairs."""
    plan, kw, x, _ = linear_case(pkg, fmt, M, N, K)
    ws = plan.alloc_workspace(M)
    want = plan.forward(x, kw, workspace=ws).clone()
    assert plan.last_status(ws) == 0
    plan.set_wait_timeout(1)
    plan.forward(x, kw, workspace=ws)
    assert plan.last_status(ws) == 7
    plan.set_wait_timeout(0)
    got = plan.forward(x, kw, workspace=ws)
    assert plan.last_status(ws) == 0
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("fmt,M,N,K", [("nvfp4", 9, 1024, 8192), ("mxfp8", 130, 520, 4096), ("mxfp4", 700, 8200, 1056)])
def test_linear_wait_limit_from_quantised_rows(pkg, fmt, M, N, K):
    """The same from quantised rows, where the product's own kernel clears the status first: a
    workspace's old contents do not matter, and a wait that runs out is still reported."""
    plan, kw, x, _ = linear_case(pkg, fmt, M, N, K)
    rows = pkg.quantize(x, fmt)
    ws = plan.alloc_workspace(M)
    want = plan.forward(x, kw).clone()
    for fill, limit, status in ((0xA5, 0, 0), (0x5A, 1, 7), (0xFF, 0, 0)):
        ws.fill_(fill)
        plan.set_wait_timeout(limit)
        got = plan.forward(rows, kw, workspace=ws)
        assert plan.last_status(ws) == status
        if status == 0:
            assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(129, 9800, 96), (257, 12900, 64), (513, 4001, 4128), (1920, 1281, 544), (2049, 1031, 64),
                                   (384, 6400, 1056), (1216, 2048, 2080)])
def test_linear_past_and_at_one_wave_of_tiles(pkg, fmt, M, N, K):
    """More tiles of 128 x 128 than the GPU has SMs, just as many and just fewer; even and odd edges."""
    plan, kw, x, wd = linear_case(pkg, fmt, M, N, K)
    ws = plan.alloc_workspace(M)
    ws.fill_(0xA5)
    got = plan.forward(x, kw, workspace=ws)
    assert plan.last_status(ws) == 0
    check_linear(got, x, wd, fmt, f"{M}x{N}x{K}")
    rows = plan.forward(pkg.quantize(x, fmt), kw)
    assert torch.equal(got.view(torch.int16), rows.view(torch.int16))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(256, 7960, 96), (300, 8192, 288), (1025, 2100, 1056), (2000, 1031, 64)])
def test_linear_on_cta_pairs(pkg, fmt, M, N, K):
    """Sizes whose 256 x 256 tiles go to CTA pairs, with part-full last tiles on every side."""
    plan, kw, x, wd = linear_case(pkg, fmt, M, N, K)
    got = plan.forward(x, kw)
    check_linear(got, x, wd, fmt, f"{M}x{N}x{K}")
    got2 = plan.forward(pkg.quantize(x, fmt), kw)
    assert torch.equal(got.view(torch.int16), got2.view(torch.int16))
