"""Closer bounds for the operators around the experts, derived from their arithmetic (u = 2^-24), and what a
row's results may depend on.

  norm's codes  Squares: a chunk of 8 FMAs, 4 chunks, 10 joins, and z's own rounding counted twice: 24u,
                halved by the root; z and the product 2u more: y within 15u of its 64-bit value. A code is
                then the nearest one, or y lies within 15u of the edge between the two.
  products      E2M1 and E4M3 products are exact in fp32, and so are their scales: half a bf16 step and
                2^-20 of the terms' magnitudes for the order of the sums.
"""
import numpy as np
import pytest
import torch

from test_block_ops import (EPS, FMTS, U, assert_within, dequantize, f64, half_step, linear_case, oracle_quantize)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)
    import serving_topk_permute_gb300 as p
    p.lib()
    return p


def grid(fmt, device):
    """The format's magnitudes in ascending order."""
    if fmt == "mxfp4":
        v = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    else:
        v = [m * 2.0 ** -9 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:119]
    return torch.tensor(v, dtype=torch.float64, device=device)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("T,H", [(100, 7168), (2048, 7168), (3000, 2080), (700, 16384)])
def test_norm_codes_are_the_nearest_but_at_the_edges(pkg, fmt, T, H):
    g = torch.Generator(device="cuda").manual_seed(T + H)
    x = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    r = (3 * torch.randn((T, H), generator=g, device="cuda")).bfloat16()
    gamma = 1.0 + 0.1 * torch.randn(H, generator=g, device="cuda")
    q = pkg.Quantized.alloc(fmt, T, H, "rows")
    total = torch.empty_like(x)
    pkg.add_rmsnorm(x, gamma, EPS, residual=r, sum_out=total, quantized=q)
    codes, sf = q.codes.clone(), q.sf.clone()
    z = x.double() + r.double()
    y = z / torch.sqrt((z * z).mean(1, keepdim=True) + EPS) * gamma.double()
    room, top, m = 15 * U, 448.0 if fmt == "mxfp8" else 6.0, grid(fmt, "cuda")
    scale = torch.exp2(sf.view(T, H // 32).double() - 127)
    amax = y.abs().view(T, H // 32, 32).amax(2)
    # the smallest scale that holds the block, with room on either side
    assert (amax <= top * scale * (1 + room)).all() and (amax >= top * scale / 2 * (1 - room)).all()
    v = y.abs() / scale.repeat_interleave(32, 1)
    at = torch.bucketize(v, (m[1:] + m[:-1]) / 2)
    nearest = (m[at] - v).abs()
    if fmt == "mxfp8":
        got = codes.view(torch.float8_e4m3fn).double().abs()
    else:
        got = torch.stack((m[(codes & 7).long()], m[((codes >> 4) & 7).long()]), 2).view(T, H)
    assert ((got - v).abs() <= nearest + 2 * room * v).all()
    # few values are that near an edge: 2 * 15u |v| of a step, which is |v| / 16 at least
    assert int((got != m[at]).sum()) <= T * H * 2.0 ** -15
    for _ in range(20):  # the same bytes every time
        q.codes.zero_(), q.sf.zero_()
        pkg.add_rmsnorm(x, gamma, EPS, residual=r, sum_out=total, quantized=q)
        assert torch.equal(q.codes, codes) and torch.equal(q.sf, sf)


PRODUCTS = [(1, 264, 256), (5, 100, 1056), (9, 256, 4096), (16, 2048, 768), (64, 520, 2080), (128, 2304, 1024),
            (300, 520, 2080), (384, 1032, 16384), (1200, 2600, 512), (300, 8192, 96), (4, 257, 32)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_products_to_the_order_of_their_sums(pkg, fmt, M, N, K):
    """From bf16 rows and from the same rows quantised: the same bits, within the close bound."""
    plan, kw, x, wd = linear_case(pkg, fmt, M, N, K, seed=7)
    xd = dequantize(*oracle_quantize(f64(x), fmt), fmt)
    want, terms = xd @ wd.T, np.abs(xd) @ np.abs(wd).T
    got = plan.forward(x, kw)
    assert_within(f64(got), want, half_step(want) * 1.01 + 2.0 ** -20 * terms, f"{fmt} {M}x{N}x{K}")
    rows = plan.forward(pkg.quantize(x, fmt), kw)
    assert torch.equal(rows.view(torch.int16), got.view(torch.int16))


@pytest.mark.parametrize("fmt", FMTS)
def test_a_row_in_batches_of_other_sizes(pkg, fmt):
    """The batch decides how K is split and how a norm's sum is ordered. A row's codes from bf16 rows are the
    same in all of them; its products and norms agree to twice the bound of each."""
    K, N = 2080, 1032
    plan, kw, x, wd = linear_case(pkg, fmt, 1200, N, K)
    gamma = torch.rand(K, device="cuda") + 0.5
    full = pkg.quantize(x, fmt, "rows")
    base, norm = f64(plan.forward(x, kw)), f64(pkg.add_rmsnorm(x, gamma))
    xd = dequantize(*oracle_quantize(f64(x), fmt), fmt)
    bound = half_step(xd @ wd.T) * 1.01 + 2.0 ** -20 * (np.abs(xd) @ np.abs(wd).T)
    for n in (1, 2, 8, 9, 17, 65, 129, 152, 153, 600):
        q = pkg.quantize(x[:n], fmt, "rows")
        assert torch.equal(q.codes, full.codes[:n])
        assert torch.equal(q.sf.view(n, -1), full.sf.view(1200, -1)[:n])
        assert_within(f64(plan.forward(x[:n], kw)), base[:n], 2 * bound[:n], f"{n} rows")
        assert_within(f64(pkg.add_rmsnorm(x[:n], gamma)), norm[:n], 2 * half_step(norm[:n]) * 1.01
                      + 128 * U * np.abs(norm[:n]), f"norm of {n} rows")
