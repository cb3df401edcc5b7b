"""What the sandwich norm refuses, and its host-only calls: no GPU needed."""
import ctypes
import os

import pytest
import torch

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4
A = 1 << 20  # an address that is never read: every call below is refused before a launch


@pytest.fixture(scope="module")
def pkg():
    import serving_topk_permute_gb300 as p
    if not os.path.exists(p.library_path()):
        from serving_topk_permute_gb300 import build
        build.build()
    return p


@pytest.fixture(scope="module")
def S(pkg):
    from serving_topk_permute_gb300 import sandwich
    sandwich._lib()
    return sandwich


def params(S, **kw):
    base = dict(gamma_post=A, gamma_pre=A, gate=None, gate_kind=0, residual_scale=1.0, eps=1e-6)
    base.update(kw)
    return S.SandwichC(**base)


COMMON = [
    ({"T": -1}, {}, INVALID), ({"H": 0}, {}, INVALID), ({"H": 16385, "ld": 16385}, {}, INVALID),
    ({"f": None}, {}, INVALID), ({"r": None}, {}, INVALID), ({"f": A + 1}, {}, INVALID), ({"r": A + 1}, {}, INVALID),
    ({"ld": 63}, {}, INVALID), ({}, {"gamma_post": None}, INVALID), ({}, {"gamma_pre": None}, INVALID),
    ({}, {"gamma_pre": A + 2}, INVALID), ({}, {"gate_kind": 3}, UNSUPPORTED), ({}, {"gate_kind": 1}, INVALID),
    ({}, {"gate": A}, INVALID), ({}, {"gate": A + 2, "gate_kind": 2}, INVALID), ({}, {"eps": -1.0}, INVALID),
    ({}, {"eps": float("nan")}, INVALID), ({}, {"eps": float("inf")}, INVALID),
    ({}, {"residual_scale": float("inf")}, INVALID), ({"stats": A + 2}, {}, INVALID),
]


@pytest.mark.parametrize("kw,pkw,status", COMMON + [
    ({"out": None}, {}, INVALID), ({"out": A + 1}, {}, INVALID), ({"sum": A + 1}, {}, INVALID),
    ({"sum": 3 * A, "out": 3 * A}, {}, INVALID), ({"T": 0, "f": None}, {"gamma_post": None}, 0),
])
def test_forward_refusals(S, kw, pkw, status):
    a = dict(T=3, H=64, f=A, r=A, ld=64, sum=None, out=2 * A, stats=None)
    a.update(kw)
    p = params(S, **pkw)
    assert S._lib().moe_sandwich_norm(a["T"], a["H"], ctypes.byref(p), a["f"], a["ld"], a["r"], a["ld"], a["sum"],
                                      a["ld"], a["out"], a["ld"], None, a["stats"], None) == status


@pytest.mark.parametrize("q,H,status", [
    (dict(format=0), 64, UNSUPPORTED), (dict(format=1), 48, INVALID), (dict(format=2), 64, INVALID),
    (dict(format=1, row_scale=A), 64, INVALID), (dict(format=1, codes=A + 8), 64, INVALID),
])
def test_quantised_refusals(S, q, H, status):
    from serving_topk_permute_gb300.block import QuantC
    p, c = params(S), QuantC(**{**dict(sf_layout=0, codes=A, sf=A, row_scale=None), **q})
    assert S._lib().moe_sandwich_norm(3, H, ctypes.byref(p), A, H, A, H, None, 0, None, 0, ctypes.byref(c), None,
                                      None) == status


@pytest.mark.parametrize("kw,pkw,status", COMMON + [
    ({"stats": None}, {}, INVALID), ({"ds": None, "do": None}, {}, INVALID), ({"ds": A + 1}, {}, INVALID),
    ({"do": A + 1}, {}, INVALID), ({"df": None}, {}, INVALID), ({"dr": None}, {}, INVALID),
    ({"df": 3 * A, "dr": 3 * A}, {}, INVALID), ({"df": 3 * A + 1}, {}, INVALID), ({"dg": A}, {}, INVALID),
    ({"dg": A + 2}, {"gate": A, "gate_kind": 1}, INVALID), ({"dp": A + 2}, {}, INVALID), ({"ws": None}, {}, INVALID),
    ({"ws": A + 8}, {}, INVALID), ({"n": 64}, {}, WORKSPACE),
])
def test_backward_refusals(S, kw, pkw, status):
    a = dict(T=3, H=64, f=A, r=A, ld=64, stats=A, ds=A, do=A, df=3 * A, dr=4 * A, dg=None, dp=A, ws=A, n=1 << 24)
    a.update(kw)
    p = params(S, **pkw)
    assert S._lib().moe_sandwich_norm_backward(
        a["T"], a["H"], ctypes.byref(p), a["f"], a["ld"], a["r"], a["ld"], a["stats"], a["ds"], a["ld"], a["do"],
        a["ld"], a["df"], a["ld"], a["dr"], a["ld"], a["dg"], a["dp"], A, a["ws"], a["n"], None) == status


def test_null_parameters(S):
    assert S._lib().moe_sandwich_norm(3, 64, None, A, 64, A, 64, None, 0, A, 64, None, None, None) == INVALID


def test_workspace_sizes(pkg):
    size = pkg.sandwich_norm_workspace_size
    assert size(0, 64) >= 256 and size(1, 7) >= 2 * 4 * 7
    assert size(10 ** 6, 7168) == size(10 ** 5, 7168) >= 2 * 4 * 7168 * 152
    for bad in ((-1, 64), (3, 0), (3, 16385)):
        with pytest.raises(pkg.MoeError):
            size(*bad)


def test_binding_refusals(pkg):
    one, x = torch.ones(8), torch.zeros((3, 8), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.sandwich_norm(x, x, one, one)
    with pytest.raises(ValueError, match="2-D"):
        pkg.sandwich_norm(x[0], x, one, one)


def test_struct_matches_the_header(S):
    import re
    from conftest import ROOT
    text = open(os.path.join(ROOT, "include", "moe.h")).read()
    body = re.search(r"typedef struct moe_sandwich \{(.*?)\}", text, re.S).group(1)
    names = re.findall(r"^\s*(?:const float\*|int32_t|float)\s+(\w+);", body, re.M)
    assert names == [n for n, _ in S.SandwichC._fields_]
    for key, value in S.GATES.items():
        assert re.search(rf"#define MOE_GATE_{key.upper()}\s+{value}\b", text)
