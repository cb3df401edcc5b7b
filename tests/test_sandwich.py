"""The sandwich norm and its gradient against plain 64-bit NumPy versions.

Tolerances, from the arithmetic (u = 2^-24, half(v) = half a bf16 step at v, A = |alpha r| + |g u| elementwise, the
size of what z is the sum of). Sums over a row: 64 terms a thread at most, 13 joins, so 64u of the sum of magnitudes.
  sum      64u A + half
  out      the same through 1 / rms(z): 160u (|h| + |pre| A / rms(z)) + half
  stats    64u; of z: 64u + 128u mean(|z| A) / mean(z^2)
  codes    the format's nearest code of a value so far off
  gradient D = |ds| + (|e| + Z mean(|e| Z)) / rms(z), Z = A / rms(z), bounds dz's terms; each of a few sums over a row and
           products adds at most 128u of the magnitudes that go in:  dr 512u |alpha| D + half,
           df 1024u (|gt w| D + |fh| mean(|gt w fh| D)) / rms(f) + half
  columns  (1024 + rows) u of the sum of magnitudes
"""
import numpy as np
import pytest
import torch

from oracle import formats as OF
from test_block_ops import FMTS, assert_within, atoms_to_rows, bf16_dev, dequantize, f64, half_step, rows_of

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6
ALPHA = 0.9375


@pytest.fixture(scope="module")
def pkg():
    import serving_topk_permute_gb300 as p
    p.lib()
    torch.cuda.set_device(0)
    return p


def dev(v):
    return torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).cuda()


class Case:
    """Inputs on the device and in 64 bits, and the forward pass in 64 bits."""

    def __init__(self, T, H, gate, stride=0, offset=0, seed=0, alpha=ALPHA):
        rng = np.random.default_rng(T * 17 + H + seed)
        self.T, self.H, self.kind, self.alpha = T, H, gate, alpha
        self.f = bf16_dev(rows_of(rng, T, H), H + stride, offset)
        self.r = bf16_dev(3 * rows_of(rng, T, H), H + stride, offset)
        self.post, self.pre = dev(1.0 + 0.2 * rng.standard_normal(H)), dev(1.0 + 0.2 * rng.standard_normal(H))
        n = {"none": 0, "token": T, "channel": H}[gate]
        self.gate = dev(rng.uniform(-0.5, 1.0, n)) if n else None
        self.rng = rng
        f, r, post, pre = f64(self.f), f64(self.r), f64(self.post), f64(self.pre)
        self.g = 1.0 if self.gate is None else f64(self.gate)[:, None] if gate == "token" else f64(self.gate)
        self.rf = 1.0 / np.sqrt((f * f).mean(1, keepdims=True) + EPS)
        self.fh = f * self.rf
        self.u = post * self.fh
        self.z = alpha * r + self.g * self.u
        self.rz = 1.0 / np.sqrt((self.z ** 2).mean(1, keepdims=True) + EPS)
        self.h = pre * self.z * self.rz
        self.A = np.abs(alpha * r) + np.abs(self.g * self.u)
        self.h_off = 160 * U * (np.abs(self.h) + np.abs(pre) * self.A * self.rz)

    def kw(self):
        return dict(gate=self.gate, gate_kind=self.kind if self.gate is not None else None, alpha=self.alpha)

    def args(self):
        return self.f, self.r, self.post, self.pre

    def check_sum(self, got):
        assert_within(f64(got), self.z, 64 * U * self.A + half_step(self.z) * 1.01, "sum")

    def check_out(self, got):
        assert_within(f64(got), self.h, self.h_off + half_step(self.h) * 1.01, "out")

    def check_stats(self, got):
        s = got.cpu().numpy().astype(np.float64)
        assert_within(s[:, :1], self.rf, 64 * U * self.rf, "1 / rms(f)")
        far = (np.abs(self.z) * self.A).mean(1, keepdims=True) * self.rz ** 2
        assert_within(s[:, 1:], self.rz, (64 + 128 * far) * U * self.rz, "1 / rms(z)")


SHAPES = [(1, 1), (1, 7), (3, 8), (5, 130), (2, 2050), (130, 1000), (153, 40), (7, 4096), (200, 4104), (3, 7168),
          (160, 7168), (2, 8200), (2, 16384), (2, 16383), (153, 16382)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("gate", ["none", "token", "channel"])
@pytest.mark.parametrize("stride,offset", [(0, 0), (5, 1), (8, 8)])
def test_forward(pkg, T, H, gate, stride, offset):
    c = Case(T, H, gate, stride, offset)
    out = torch.full((T, H + stride), 7.0, dtype=torch.bfloat16, device="cuda")
    total = torch.full((T, H + stride), 7.0, dtype=torch.bfloat16, device="cuda")
    stats = torch.empty((T, 2), device="cuda")
    pkg.sandwich_norm(*c.args(), **c.kw(), eps=EPS, sum_out=total[:, :H], out=out[:, :H], stats=stats)
    c.check_out(out[:, :H])
    c.check_sum(total[:, :H])
    c.check_stats(stats)
    assert (out[:, H:] == 7).all() and (total[:, H:] == 7).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,H,stride,layout,gate", [
    (1, 32, 0, "rows", "none"), (5, 96, 3, "rows", "token"), (130, 2080, 0, "atoms", "channel"),
    (3, 7168, 8, "rows", "token"), (160, 7168, 0, "atoms", "channel"), (2, 16384, 0, "atoms", "none")])
def test_forward_quantised(pkg, fmt, T, H, stride, layout, gate):
    c = Case(T, H, gate, stride)
    q = pkg.Quantized.alloc(fmt, T, H, layout)
    out, total = torch.empty((T, H), dtype=torch.bfloat16, device="cuda"), torch.empty_like(c.f)
    assert pkg.sandwich_norm(*c.args(), **c.kw(), eps=EPS, sum_out=total, out=out, quantized=q) is out
    c.check_out(out)
    c.check_sum(total)
    codes, sf = q.codes.cpu().numpy(), q.sf.cpu().numpy()
    B = 16 if fmt == "nvfp4" else 32
    sf = atoms_to_rows(sf, T, H, fmt)[0] if layout == "atoms" else sf.reshape(T, H // B)
    gs = q.row_scale.cpu().numpy() if fmt == "nvfp4" else None
    got = dequantize(codes, sf, gs, fmt)
    blocks, off = (np.abs(v).reshape(T, H // B, B).max(axis=2) for v in (c.h, c.h_off))
    if fmt == "nvfp4":
        want_gs = np.abs(c.h).max(axis=1) / 2688.0
        assert_within(gs.astype(np.float64), want_gs, off.max(axis=1) / 2688.0 + 4 * U * want_gs, "row scale")
        scale = OF.E4M3_TABLE[sf] * gs.astype(np.float64)[:, None]
        # the nearest E4M3 to amax / (6 row scale): half a step of it, wider by what both are off
        ratio = blocks / (6.0 * want_gs[:, None])
        step = np.maximum(np.ldexp(1.0, (np.floor(np.log2(np.maximum(ratio, 2.0 ** -6))) - 3).astype(int)), 2.0 ** -9)
        room = step / 2 * (1 + 2.0 ** -8) + 2 * off.max(axis=1, keepdims=True) / (6.0 * want_gs[:, None])
        assert_within(OF.E4M3_TABLE[sf], ratio, room, "block scale")
    else:
        top = 448.0 if fmt == "mxfp8" else 6.0
        scale = np.ldexp(1.0, sf.astype(np.int64) - 127)
        assert (top * scale >= blocks - off).all() and ((top * scale / 2 < blocks + off) | (blocks == 0)).all()
    v = np.abs(c.h) / np.where(scale > 0, scale, 1.0).repeat(B, axis=1)
    if fmt == "mxfp8":
        step = np.maximum(np.ldexp(1.0, (np.floor(np.log2(np.maximum(v, 2.0 ** -6))) - 3).astype(int)), 2.0 ** -9)
    else:
        step = np.where(v < 2.0, 0.5, np.where(v < 4.0, 1.0, 2.0))
    room = np.maximum(step / 2 * (1 + 2.0 ** -10), v - (448.0 if fmt == "mxfp8" else 6.0))
    assert_within(got, c.h, room * scale.repeat(B, axis=1) + c.h_off, "dequantised")


def test_in_place_and_defaults(pkg):
    for H, stride in ((512, 0), (513, 0), (4100, 2), (7168, 0)):
        c = Case(33, H, "token", stride)
        total = torch.empty((33, H), dtype=torch.bfloat16, device="cuda")
        want = pkg.sandwich_norm(*c.args(), **c.kw(), sum_out=total)
        f2, r2 = c.f.clone(), c.r.clone()
        got = pkg.sandwich_norm(f2, r2, c.post, c.pre, **c.kw(), sum_out=r2, out=f2)
        assert torch.equal(got, want) and torch.equal(r2, total) and got.data_ptr() == f2.data_ptr()
    zero = torch.zeros((3, 64), dtype=torch.bfloat16, device="cuda")
    one = torch.ones(64, device="cuda")
    assert (pkg.sandwich_norm(zero, zero, one, one) == 0).all()
    assert pkg.sandwich_norm(zero[:0], zero[:0], one, one).shape == (0, 64)
    square = torch.zeros((64, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="gate_kind"):
        pkg.sandwich_norm(square, square, one, one, gate=one)
    pkg.sandwich_norm(square, square, one, one, gate=one, gate_kind="channel")


def test_rows_that_are_not_finite_stay_apart(pkg):
    c = Case(5, 1000, "channel")
    stats, clean = (torch.empty((5, 2), device="cuda") for _ in range(2))
    want = pkg.sandwich_norm(*c.args(), **c.kw(), stats=clean)
    c.f[1, 7] = float("nan")
    c.r[3, 900] = float("inf")
    got = pkg.sandwich_norm(*c.args(), **c.kw(), stats=stats)
    keep = [0, 2, 4]
    assert torch.equal(got[keep], want[keep]) and torch.equal(stats[keep], clean[keep])
    assert torch.isnan(got[1]).all() and not torch.isfinite(got[3, 900])


def gradient(c, ds, dh):
    """The gradients in 64 bits and what each may be off."""
    post, pre = f64(c.post), f64(c.pre)
    token = c.kind == "token"
    gt = c.g if token else 1.0
    w = post * c.g if c.kind == "channel" else post
    zh, Z, e = c.z * c.rz, c.A * c.rz, dh * pre
    mean = lambda v: v.mean(1, keepdims=True)  # noqa: E731
    dz = ds + c.rz * (e - zh * mean(e * zh))
    D = np.abs(ds) + c.rz * (np.abs(e) + Z * mean(np.abs(e) * Z))
    t = gt * w * dz
    df = c.rf * (t - c.fh * mean(t * c.fh))
    Df = c.rf * (np.abs(gt * w) * D + np.abs(c.fh) * mean(np.abs(gt * w * c.fh) * D))
    C, Cm = (gt * c.fh * dz).sum(0), (np.abs(gt * c.fh) * D).sum(0)
    many = (1024 + c.T) * U
    want = {"f": (df, 1024 * U * Df), "residual": (c.alpha * dz, 512 * U * abs(c.alpha) * D),
            "gamma_pre": ((dh * zh).sum(0), many * (np.abs(dh) * Z).sum(0)),
            "gamma_post": (C * (c.g if c.kind == "channel" else 1.0),
                           many * Cm * (np.abs(c.g) if c.kind == "channel" else 1.0))}
    if token:
        want["gate"] = ((w * c.fh * dz).sum(1), 1024 * U * (np.abs(w * c.fh) * D).sum(1))
    elif c.kind == "channel":
        want["gate"] = (C * post, many * Cm * np.abs(post))
    return want


def check_gradient(got, want, what=""):
    for name, (value, off) in want.items():
        g = getattr(got, name)
        if name in ("f", "residual"):
            off = off + half_step(value) * 1.01
        assert_within(g.double().cpu().numpy(), value, off, f"{what} d_{name}")


GRAD_SHAPES = SHAPES + [(700, 96), (1000, 2048), (340, 2050), (320, 5000)]


@pytest.mark.parametrize("T,H", GRAD_SHAPES)
@pytest.mark.parametrize("gate", ["none", "token", "channel"])
@pytest.mark.parametrize("stride,offset", [(0, 0), (5, 1), (8, 8)])
def test_gradient(pkg, T, H, gate, stride, offset):
    c = Case(T, H, gate, stride, offset)
    ds, dh = (bf16_dev(0.1 * rows_of(c.rng, T, H), H + stride, offset) for _ in range(2))
    stats = torch.empty((T, 2), device="cuda")
    pkg.sandwich_norm(*c.args(), **c.kw(), eps=EPS, stats=stats)
    wide = torch.full((2, T, H + stride), 7.0, dtype=torch.bfloat16, device="cuda")
    got = pkg.sandwich_norm_backward(*c.args(), stats, **c.kw(), d_sum=ds, d_out=dh, d_f=wide[0, :, :H],
                                     d_residual=wide[1, :, :H])
    check_gradient(got, gradient(c, f64(ds), f64(dh)))
    assert (wide[:, :, H:] == 7).all()


@pytest.mark.parametrize("H", [200, 201, 4096])
def test_gradient_of_one_output_in_place_and_without_gammas(pkg, H):
    c = Case(300, H, "channel")
    ds, dh = (bf16_dev(0.1 * rows_of(c.rng, 300, H)) for _ in range(2))
    zero = np.zeros((300, H))
    stats = torch.empty((300, 2), device="cuda")
    pkg.sandwich_norm(*c.args(), **c.kw(), eps=EPS, stats=stats)
    run = lambda **kw: pkg.sandwich_norm_backward(*c.args(), stats, **c.kw(), **kw)  # noqa: E731
    check_gradient(run(d_sum=ds), gradient(c, f64(ds), zero), "sum alone")
    check_gradient(run(d_out=dh), gradient(c, zero, f64(dh)), "out alone")
    both = run(d_sum=ds, d_out=dh)
    lean = run(d_sum=ds, d_out=dh, gammas=False)
    assert lean.gamma_post is None and lean.gamma_pre is None and lean.gate is None
    assert torch.equal(lean.f, both.f) and torch.equal(lean.residual, both.residual)
    s2, h2 = ds.clone(), dh.clone()
    inplace = run(d_sum=s2, d_out=h2, d_f=h2, d_residual=s2)
    for a, b in zip(inplace, both):
        assert torch.equal(a, b)


def test_gradient_without_rows(pkg):
    one, none = torch.ones(64, device="cuda"), torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    g = pkg.sandwich_norm_backward(none, none, one, one, torch.empty((0, 2), device="cuda"), gate=one, d_sum=none)
    assert g.f.shape == (0, 64) and (g.gamma_post == 0).all() and (g.gamma_pre == 0).all() and (g.gate == 0).all()


@pytest.mark.parametrize("gate", ["none", "token", "channel"])
def test_gradient_against_differences(pkg, gate):
    """Central differences of the formula, in 64 bits: what the gradient returns in fp32 is theirs to its own
    tolerance and h^2; d_f and d_residual also to half a bf16 step."""
    T, H, h = 4, 24, 1e-5
    c = Case(T, H, gate)
    ds, dh = (bf16_dev(rows_of(c.rng, T, H, big=False)) for _ in range(2))
    stats = torch.empty((T, 2), device="cuda")
    pkg.sandwich_norm(*c.args(), **c.kw(), eps=EPS, stats=stats)
    got = pkg.sandwich_norm_backward(*c.args(), stats, **c.kw(), d_sum=ds, d_out=dh)
    leaves = {"f": f64(c.f), "residual": f64(c.r), "gamma_post": f64(c.post), "gamma_pre": f64(c.pre)}
    if gate != "none":
        leaves["gate"] = f64(c.gate)

    def loss(v):
        g = 1.0 if gate == "none" else v["gate"][:, None] if gate == "token" else v["gate"]
        u = v["gamma_post"] * v["f"] / np.sqrt((v["f"] ** 2).mean(1, keepdims=True) + EPS)
        z = c.alpha * v["residual"] + g * u
        out = v["gamma_pre"] * z / np.sqrt((z ** 2).mean(1, keepdims=True) + EPS)
        return (z * f64(ds)).sum() + (out * f64(dh)).sum()

    formula = gradient(c, f64(ds), f64(dh))
    for name, value in leaves.items():
        diff = np.zeros_like(value)
        for i in np.ndindex(value.shape):
            up, down = dict(leaves), dict(leaves)
            up[name], down[name] = value.copy(), value.copy()
            up[name][i] += h
            down[name][i] -= h
            diff[i] = (loss(up) - loss(down)) / (2 * h)
        off = formula[name][1] + 1e-6 * (1 + np.abs(diff))
        if name in ("f", "residual"):
            off = off + half_step(diff) * 1.01
        assert_within(getattr(got, name).double().cpu().numpy(), diff, off, name)


def test_deterministic_and_captured(pkg):
    T, H = 777, 2050
    c = Case(T, H, "channel")
    ds, dh = (bf16_dev(0.1 * rows_of(c.rng, T, H)) for _ in range(2))
    stats, out = torch.empty((T, 2), device="cuda"), torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(pkg.sandwich_norm_workspace_size(T, H), dtype=torch.uint8, device="cuda")

    def step():
        pkg.sandwich_norm(*c.args(), **c.kw(), eps=EPS, out=out, stats=stats)
        return pkg.sandwich_norm_backward(*c.args(), stats, **c.kw(), d_sum=ds, d_out=dh, workspace=ws)

    eager = [t.clone() for t in (*step(), out, stats)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for _ in range(2):
        ws.fill_(0xFF)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, (*captured, out, stats)):
            assert torch.equal(a, b)


def test_rows_past_two_to_the_31_elements(pkg):
    T, H, ld = 300, 64, 2 ** 23 + 8
    c = Case(T, H, "token")
    buf = torch.zeros(T * ld, dtype=torch.bfloat16, device="cuda").view(T, ld)
    far = [buf[:, 128 * i:128 * i + H] for i in range(6)]
    far[0].copy_(c.f)
    far[1].copy_(c.r)
    stats, want_stats = torch.empty((T, 2), device="cuda"), torch.empty((T, 2), device="cuda")
    want = pkg.sandwich_norm(*c.args(), **c.kw(), stats=want_stats)
    pkg.sandwich_norm(far[0], far[1], c.post, c.pre, **c.kw(), out=far[2], stats=stats)
    assert torch.equal(far[2], want) and torch.equal(stats, want_stats)
    ds = bf16_dev(0.1 * rows_of(c.rng, T, H))
    far[3].copy_(ds)
    a = pkg.sandwich_norm_backward(*c.args(), stats, **c.kw(), d_sum=ds)
    b = pkg.sandwich_norm_backward(far[0], far[1], c.post, c.pre, stats, **c.kw(), d_sum=far[3], d_f=far[4],
                                   d_residual=far[5])
    for x, y in zip(a, b):
        assert torch.equal(x, y)
