"""Bytes of the quantised forms that ordinary rows do not show: zeros of either sign, and blocks so far
below their row's magnitude that NVFP4 gives them the scale zero."""
import numpy as np
import pytest
import torch

from test_block_ops import EPS, FMTS, bf16_dev, f64, oracle_quantize

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)
    import serving_topk_permute_gb300 as p
    p.lib()
    return p


def rows_with_tiny_blocks(T, K):
    rng = np.random.default_rng(T + K)
    x = rng.standard_normal((T, K))
    x[:, 16:32] = -np.abs(x[:, 16:32]) * 1e-7   # all negative, scale zero next to 16 ordinary values
    x[:, 32:64] *= 1e-6                         # either sign, around the edge of the smallest scale
    x[:, 70] = -0.0
    if T > 1:
        x[1] = -0.0
        x[1, ::2] = 0.0
    if T > 2:
        x[2] = -0.0
        x[2, 5] = 3.0
    return x


def rows_of_codes(pkg, x, fmt):
    """Codes and row-major scales, and the row scales, by every way that quantises bf16 rows."""
    T, K = x.shape
    q = pkg.quantize(x, fmt, "rows")
    return q.codes.cpu().numpy(), q.sf.cpu().numpy().reshape(T, -1), \
        None if q.row_scale is None else q.row_scale.cpu().numpy()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,K,stride,offset", [(1, 128, None, 0), (7, 96, None, 0), (200, 2080, None, 0),
                                               (300, 8224, None, 0), (5, 416, 419, 1), (300, 2080, 2081, 3)])
def test_zeros_and_tiny_blocks_equal_the_oracle(pkg, fmt, T, K, stride, offset):
    x = bf16_dev(rows_with_tiny_blocks(T, K), stride, offset)
    want, wsf, wgs = oracle_quantize(f64(x), fmt)
    codes, sf, gs = rows_of_codes(pkg, x, fmt)
    np.testing.assert_array_equal(sf, wsf)
    np.testing.assert_array_equal(codes, want)
    if fmt == "nvfp4":
        np.testing.assert_array_equal(gs, wgs)
        assert (sf[0, 1] == 0) and not codes[0, 8:16].any()


@pytest.mark.parametrize("residual", [False, True])
def test_norm_gives_blocks_of_scale_zero_the_code_zero(pkg, residual):
    """The norm's NVFP4 form: where a block's scale is zero its codes are zero, whatever the values' signs."""
    T, H = 160, 2080
    x = bf16_dev(rows_with_tiny_blocks(T, H))
    r = torch.zeros_like(x) if residual else None
    q = pkg.Quantized.alloc("nvfp4", T, H, "rows")
    pkg.add_rmsnorm(x, torch.ones(H, device="cuda"), EPS, residual=r, quantized=q)
    sf, codes = q.sf.view(T, H // 16), q.codes.view(T, H // 16, 8)
    empty = sf == 0
    assert empty[:, 1].all() and int(empty.sum()) < empty.numel() // 2
    assert (codes[empty] == 0).all()


@pytest.mark.parametrize("wexp", [-70, 0, 70])
@pytest.mark.parametrize("M,N,K", [(1, 264, 544), (2, 520, 2080), (9, 264, 544), (60, 1032, 4096), (130, 264, 288),
                                   (600, 8200, 96)])
def test_products_of_very_small_and_large_rows(pkg, M, N, K, wexp):
    """NVFP4 rows and weights at magnitudes where the product of their two scales leaves the normal range of
    fp32 though the output does not. Tolerance as everywhere: half a bf16 step, and 2^-20 of the terms."""
    from test_block_ops import assert_within, half_step
    from oracle import formats as OF
    rng = np.random.default_rng(M + N + K)
    exps = np.linspace(-120, 100, M).round() if M > 2 else np.array([-108.0, 95.0])[:M]
    x = bf16_dev(rng.standard_normal((M, K)) * 2.0 ** exps[:, None])
    w = (rng.standard_normal((N, K)) * 2.0 ** wexp).astype(np.float32)
    gs = OF.nvfp4_global_scale(np.abs(w).max()).reshape(1)
    codes, sf = OF.nvfp4_quantize(w, gs)
    wd = OF.nvfp4_dequantize(codes, sf, np.broadcast_to(gs, (N,)))
    plan = pkg.LinearPlan(pkg.LinearConfig(N, K, M, "nvfp4"))
    kw = plan.transform_weight(torch.from_numpy(codes).cuda(), torch.from_numpy(sf).cuda(),
                               torch.from_numpy(gs.astype(np.float32)).cuda())
    xc, xsf, xgs = oracle_quantize(f64(x), "nvfp4")
    xd = OF.nvfp4_dequantize(xc, xsf, xgs)
    want, terms = xd @ wd.T, np.abs(xd) @ np.abs(wd).T
    seen = terms < 1e38  # larger outputs may overflow bf16
    for rows in (x, pkg.quantize(x, "nvfp4")):
        got = f64(plan.forward(rows, kw))
        assert_within(got[seen], want[seen], (half_step(want) * 1.01 + 2.0 ** -20 * terms)[seen], "out")
