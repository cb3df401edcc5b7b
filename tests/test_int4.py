"""The product with 4-bit integer weights against plain 64-bit NumPy versions.

Tolerances, from the arithmetic: codes, zero points and activations are multiplied exactly, sums and scales are fp32
(tensor cores keep some 2^-20 of the magnitudes that go in), the result is rounded once:
  half a bf16 step + 2^-20 sum |x w|
Above 16 tokens the weights are the bf16 values nearest to (q - z) s, which the 64-bit version computes too.

"""
import numpy as np
import pytest
import torch

from test_block_ops import assert_within, bf16_dev, f64, half_step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import serving_topk_permute_gb300 as p
    p.lib()
    torch.cuda.set_device(0)
    return p


def round_bf16(w):
    """The nearest bf16 values, ties to even, of float64 ones that fp32 holds exactly."""
    return torch.from_numpy(w.astype(np.float32)).bfloat16().double().numpy()


class Weight:
    def __init__(self, pkg, N, K, group, zeros, dtype, max_tokens=4096, seed=0):
        rng = np.random.default_rng(N * 3 + K + group + seed)
        groups = -(-K // group)
        q = rng.integers(0, 16, (N, K))
        z = rng.integers(0, 16, (N, groups)) if zeros else np.full((N, groups), 8)
        s = rng.standard_normal((N, groups)) * 0.02 + 0.03
        self.scales = torch.from_numpy(s).to(dtype).cuda()
        self.codes = torch.from_numpy((q[:, 0::2] | q[:, 1::2] << 4).astype(np.uint8)).cuda()
        self.zeros = torch.from_numpy(z.astype(np.uint8)).cuda() if zeros else None
        wide = lambda v: v.repeat(group, axis=1)[:, :K]  # noqa: E731
        self.exact = (q - wide(z)) * wide(self.scales.double().cpu().numpy())
        self.N, self.K = N, K
        self.plan = pkg.Int4LinearPlan(pkg.Int4LinearConfig(N, K, max_tokens, group, zeros, dtype))
        self.kernel = self.plan.transform_weight(self.codes, self.scales, self.zeros)

    def check(self, x, got, what=""):
        T = x.shape[0]
        xd = f64(x)
        w = self.exact if T <= 16 else round_bf16(self.exact)
        want, size = xd @ w.T, np.abs(xd) @ np.abs(w).T
        assert_within(f64(got), want, half_step(want) * 1.01 + 2.0 ** -20 * size, what)


def activations(rng, T, K, stride=None, offset=0):
    return bf16_dev(rng.standard_normal((T, K)) * np.exp(0.5 * rng.standard_normal((1, K))), stride, offset)


KINDS = [(32, True, torch.bfloat16), (64, False, torch.float16), (128, True, torch.float16), (128, False, torch.bfloat16),
         (64, True, torch.bfloat16), (32, False, torch.float16)]


@pytest.mark.parametrize("group,zeros,dtype", KINDS)
@pytest.mark.parametrize("T,N,K", [
    (1, 1, 32), (1, 16, 64), (1, 4096, 7168), (2, 17, 96), (3, 200, 1056), (8, 130, 4096), (9, 64, 160), (16, 333, 2080),
    (1, 100, 32768), (5, 48, 16416), (16, 7168, 512),
])
def test_few_tokens(pkg, T, N, K, group, zeros, dtype):
    rng = np.random.default_rng(T + N + K)
    w = Weight(pkg, N, K, group, zeros, dtype)
    x = activations(rng, T, K)
    w.check(x, w.plan.forward(x, w.kernel))


@pytest.mark.parametrize("group,zeros,dtype", KINDS)
@pytest.mark.parametrize("T,N,K", [
    (17, 1, 32), (17, 128, 64), (31, 129, 96), (32, 500, 2080), (33, 2999, 1056), (64, 256, 8192), (65, 100, 4096),
    (77, 2999, 2080), (128, 1000, 512), (129, 130, 160), (200, 4096, 1024), (257, 384, 2048), (600, 1000, 32), (1000, 257, 416),
])
def test_many_tokens(pkg, T, N, K, group, zeros, dtype):
    rng = np.random.default_rng(T + N + K)
    w = Weight(pkg, N, K, group, zeros, dtype)
    x = activations(rng, T, K)
    ws = w.plan.alloc_workspace(T)
    w.check(x, w.plan.forward(x, w.kernel, workspace=ws))
    assert w.plan.last_status(ws) == 0


def test_a_large_product(pkg):
    rng = np.random.default_rng(0)
    w = Weight(pkg, 3000, 2048, 128, False, torch.bfloat16)
    x = activations(rng, 2500, 2048)
    w.check(x, w.plan.forward(x, w.kernel))


@pytest.mark.parametrize("T", [1, 2, 8, 16, 40, 300])
@pytest.mark.parametrize("stride,offset", [(1, 0), (8, 8), (3, 5), (0, 1)])
def test_strides_and_alignment(pkg, T, stride, offset):
    N, K = 300, 352
    rng = np.random.default_rng(T)
    w = Weight(pkg, N, K, 64, True, torch.bfloat16)
    x = activations(rng, T, K, K + stride, offset)
    wide = torch.full((T, N + 7), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = w.plan.alloc_workspace(T)
    ws.fill_(0xA5)
    got = w.plan.forward(x, w.kernel, out=wide[:, 3:3 + N], workspace=ws)
    w.check(x, got)
    assert (wide[:, :3] == 7).all() and (wide[:, 3 + N:] == 7).all()


@pytest.mark.parametrize("T", [1, 12, 40, 300])
def test_rows_do_not_mix(pkg, T):
    """A token of NaN or infinity, and a feature whose scale is, stay in their row and column."""
    w = Weight(pkg, 260, 512, 64, False, torch.bfloat16)
    rng = np.random.default_rng(1)
    x = activations(rng, T, 512)
    clean = w.plan.forward(x, w.kernel)
    w.scales[100, 3] = float("nan")
    w.scales[200, 0] = float("inf")
    bad = w.plan.transform_weight(w.codes, w.scales)
    got = w.plan.forward(x, bad)
    keep = [n for n in range(260) if n not in (100, 200)]
    assert torch.equal(got[:, keep], clean[:, keep])
    assert torch.isnan(got[:, 100]).all() and not torch.isfinite(got[:, 200]).any()
    if T > 1:
        y = x.clone()
        y[T // 2, 7] = float("nan")
        y[T // 2, 300] = float("inf")
        got = w.plan.forward(y, w.kernel)
        rows = [t for t in range(T) if t != T // 2]
        assert torch.equal(got[rows], clean[rows]) and torch.isnan(got[T // 2]).all()


def test_rows_do_not_depend_on_the_batch_around_them(pkg):
    w = Weight(pkg, 520, 1056, 128, True, torch.bfloat16)
    rng = np.random.default_rng(2)
    x = activations(rng, 300, 1056)
    many = f64(w.plan.forward(x, w.kernel))
    for T in (1, 2, 8, 16, 17, 64, 128):
        part = f64(w.plan.forward(x[:T], w.kernel))
        # both are within their tolerance of what they stand for
        xd = f64(x[:T])
        off = 2.0 ** -8 * (np.abs(xd) @ np.abs(w.exact).T) * (2.0 ** -1 if T > 16 else 1.0)
        assert (np.abs(part - many[:T]) <= off + 2 * half_step(many[:T])).all()


def test_no_tokens(pkg):
    w = Weight(pkg, 64, 64, 32, False, torch.bfloat16)
    assert w.plan.forward(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), w.kernel).shape == (0, 64)


@pytest.mark.parametrize("T", [1, 9, 100, 700])
def test_deterministic_captured_and_on_another_stream(pkg, T):
    w = Weight(pkg, 1000, 2048, 128, False, torch.bfloat16)
    rng = np.random.default_rng(3)
    x = activations(rng, T, 2048)
    want = w.plan.forward(x, w.kernel)
    out, ws = torch.empty_like(want), w.plan.alloc_workspace(T)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        out.zero_()
        s.wait_stream(torch.cuda.current_stream())
        w.plan.forward(x, w.kernel, out=out, workspace=ws, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.plan.forward(x, w.kernel, out=out, workspace=ws)
        w.plan.forward(x, w.kernel, out=out, workspace=ws)
    for _ in range(2):
        out.zero_()
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_rows_past_two_to_the_31_elements(pkg):
    T, K, N, ld = 300, 64, 40, 2 ** 23 + 8
    w = Weight(pkg, N, K, 32, True, torch.bfloat16)
    rng = np.random.default_rng(4)
    x = activations(rng, T, K)
    buf = torch.zeros(T * ld, dtype=torch.bfloat16, device="cuda").view(T, ld)
    far = buf[:, :K]
    far.copy_(x)
    want = w.plan.forward(x, w.kernel)
    got = w.plan.forward(far, w.kernel, out=buf[:, 1024:1024 + N])
    assert torch.equal(got, want)
    got = w.plan.forward(far[:9], w.kernel, out=buf[:9, 2048:2048 + N])
    assert torch.equal(got, w.plan.forward(x[:9], w.kernel))
    assert torch.equal(w.plan.forward(far[290:], w.kernel), w.plan.forward(x[290:], w.kernel))


def test_waits_that_run_out(pkg):
    """With a limit of a nanosecond the product gives up, says so, and the next one is whole again."""
    for T, N, K in ((40, 1000, 8192), (700, 1000, 4096)):
        w = Weight(pkg, N, K, 128, False, torch.bfloat16)
        x = activations(np.random.default_rng(5), T, K)
        ws = w.plan.alloc_workspace(T)
        ws.fill_(0xA5)
        for limit in (0, 1, 0):
            w.plan.set_wait_timeout(limit)
            got = w.plan.forward(x, w.kernel, workspace=ws)
            assert w.plan.last_status(ws) == (7 if limit else 0)
            assert w.plan.last_status(ws) == 0
        w.check(x, got)
