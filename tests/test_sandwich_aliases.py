"""Rows written over rows that are read: refused at another stride (no GPU needed), right at the same one."""
import ctypes

import pytest
import torch

from test_sandwich_refusals import A, INVALID, S, params, pkg  # noqa: F401


@pytest.mark.parametrize("f,ldf,r,ldr,s,lds,o,ldo", [
    (A, 64, 2 * A, 72, 2 * A, 64, 3 * A, 64), (A, 72, 2 * A, 64, A, 64, 3 * A, 64), (A, 72, 2 * A, 64, None, 0, A, 64),
    (A, 64, 2 * A, 64, 3 * A, 64, 2 * A, 80),
])
def test_forward_at_another_stride(S, f, ldf, r, ldr, s, lds, o, ldo):  # noqa: F811
    p = params(S)
    assert S._lib().moe_sandwich_norm(3, 64, ctypes.byref(p), f, ldf, r, ldr, s, lds, o, ldo, None, None, None) == INVALID


@pytest.mark.parametrize("df,lddf,dr,lddr", [(3 * A, 72, 5 * A, 64), (4 * A, 72, 5 * A, 64), (5 * A, 64, 3 * A, 80),
                                             (5 * A, 64, 4 * A, 80)])
def test_backward_at_another_stride(S, df, lddf, dr, lddr):  # noqa: F811
    p = params(S)
    assert S._lib().moe_sandwich_norm_backward(3, 64, ctypes.byref(p), A, 64, 2 * A, 64, 6 * A, 3 * A, 64, 4 * A, 64, df, lddf,
                                               dr, lddr, None, None, None, None, 0, None) == INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(400, 2304), (200, 130), (5, 4096)])
def test_in_place(pkg, T, H):  # noqa: F811
    torch.cuda.set_device(0)
    g = torch.Generator(device="cuda").manual_seed(T + H)
    f, r, ds, do = (torch.randn((T, H), generator=g, device="cuda").bfloat16() for _ in range(4))
    post, pre = (1.0 + 0.1 * torch.randn(H, generator=g, device="cuda") for _ in range(2))
    z, h = torch.empty_like(f), torch.empty_like(f)
    stats = torch.empty((T, 2), device="cuda")
    pkg.sandwich_norm(f, r, post, pre, sum_out=z, out=h, stats=stats)
    f2, r2 = f.clone(), r.clone()
    pkg.sandwich_norm(f2, r2, post, pre, sum_out=r2, out=f2)
    assert torch.equal(r2, z) and torch.equal(f2, h)
    want = pkg.sandwich_norm_backward(f, r, post, pre, stats, d_sum=ds, d_out=do)
    a, b = ds.clone(), do.clone()
    got = pkg.sandwich_norm_backward(f, r, post, pre, stats, d_sum=a, d_out=b, d_f=b, d_residual=a)
    assert torch.equal(got.f, want.f) and torch.equal(got.residual, want.residual)
    assert torch.equal(got.gamma_post, want.gamma_post) and torch.equal(got.gamma_pre, want.gamma_pre)
