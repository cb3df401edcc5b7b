"""What the product with 4-bit integer weights refuses, and its host-only calls: no GPU needed."""
import ctypes
import os
import re

import pytest
import torch

INVALID, UNSUPPORTED, CAPACITY, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def pkg():
    import serving_topk_permute_gb300 as p
    if not os.path.exists(p.library_path()):
        from serving_topk_permute_gb300 import build
        build.build()
    return p


@pytest.fixture(scope="module")
def I(pkg):
    from serving_topk_permute_gb300 import int4
    int4._lib()
    return int4


@pytest.mark.parametrize("kw,status", [
    ({}, 0), ({"out_features": 0}, INVALID), ({"out_features": 2 ** 20 + 1}, INVALID), ({"out_features": 1}, 0),
    ({"in_features": 0}, INVALID), ({"in_features": 48}, INVALID), ({"in_features": 32800}, INVALID),
    ({"in_features": 32768}, 0), ({"in_features": 32}, 0), ({"max_tokens": 0}, INVALID), ({"group_size": 16}, UNSUPPORTED),
    ({"group_size": 256}, UNSUPPORTED), ({"group_size": 0}, UNSUPPORTED), ({"zero_points": True}, 0),
    ({"scale_dtype": torch.float16}, 0),
])
def test_configurations(pkg, kw, status):
    base = dict(out_features=256, in_features=512, max_tokens=64)
    base.update(kw)
    assert pkg.int4_validate(pkg.Int4LinearConfig(**base)) == status


@pytest.mark.parametrize("field,value,status", [("zero_points", 2, INVALID), ("scale_type", 2, UNSUPPORTED),
                                                ("scale_type", -1, UNSUPPORTED)])
def test_raw_configurations(I, field, value, status):
    c = I.Int4ConfigC(256, 512, 64, 128, 0, 0)
    setattr(c, field, value)
    assert I._lib().moe_int4_config_validate(ctypes.byref(c)) == status
    h = ctypes.c_void_p()
    assert I._lib().moe_int4_plan(ctypes.byref(c), ctypes.byref(h)) == status and not h.value
    assert I._lib().moe_int4_config_validate(None) == INVALID


def test_null_plans(I):
    L, A = I._lib(), 1 << 20
    n = ctypes.c_size_t()
    w = I.Int4WeightC(A, A, None)
    assert L.moe_int4_set_wait_timeout(None, 0) == INVALID
    assert L.moe_int4_weight_size(None, ctypes.byref(n), ctypes.byref(n), ctypes.byref(n)) == INVALID
    assert L.moe_int4_transform_weight(None, ctypes.byref(w), ctypes.byref(w), None) == INVALID
    assert L.moe_int4_workspace_size(None, 1, ctypes.byref(n)) == INVALID
    assert L.moe_int4_forward(None, 1, A, 64, ctypes.byref(w), A, 64, A, 1 << 20, None) == INVALID
    assert L.moe_int4_last_status(None, A, None, ctypes.byref(ctypes.c_int32())) == INVALID
    assert L.moe_int4_plan_destroy(None) == 0


def test_scale_types(pkg):
    with pytest.raises(ValueError, match="scale_dtype"):
        pkg.int4_validate(pkg.Int4LinearConfig(64, 64, 1, scale_dtype=torch.float32))


def test_structs_match_the_header(I):
    from conftest import ROOT
    text = open(os.path.join(ROOT, "include", "moe.h")).read()
    body = re.search(r"typedef struct moe_int4_config \{(.*?)\}", text, re.S).group(1)
    assert re.findall(r"^\s*int32_t\s+(\w+);", body, re.M) == [n for n, _ in I.Int4ConfigC._fields_]
    body = re.search(r"typedef struct moe_int4_weight \{(.*?)\}", text, re.S).group(1)
    assert re.findall(r"^\s*void\*\s+(\w+);", body, re.M) == [n for n, _ in I.Int4WeightC._fields_]
    for dtype, value in I.SCALE_TYPES.items():
        name = {torch.bfloat16: "BF16", torch.float16: "F16"}[dtype]
        assert re.search(rf"#define MOE_SCALE_{name}\s+{value}\b", text)


A = 1 << 20


@pytest.mark.gpu
@pytest.mark.parametrize("kw,status", [
    ({"T": -1}, INVALID), ({"T": 65}, CAPACITY), ({"T": 0, "x": None}, 0), ({"x": None}, INVALID), ({"x": A + 1}, INVALID),
    ({"ldx": 511}, INVALID), ({"out": None}, INVALID), ({"out": A + 1}, INVALID), ({"out": A}, INVALID),
    ({"ldo": 255}, INVALID), ({"codes": None}, INVALID), ({"codes": A + 128}, INVALID), ({"scales": A + 128}, INVALID),
    ({"zeros": A}, INVALID), ({"ws": None}, INVALID), ({"ws": A + 128}, INVALID), ({"n": 64}, WORKSPACE),
])
def test_forward_refusals(pkg, I, kw, status):
    """Refused before a launch: no address is read."""
    a = dict(T=3, x=A, ldx=512, out=2 * A, ldo=256, codes=A, scales=A, zeros=None, ws=A, n=1 << 30)
    a.update(kw)
    plan = pkg.Int4LinearPlan(pkg.Int4LinearConfig(256, 512, 64))
    w = I.Int4WeightC(a["codes"], a["scales"], a["zeros"])
    assert I._lib().moe_int4_forward(plan._h, a["T"], a["x"], a["ldx"], ctypes.byref(w), a["out"], a["ldo"], a["ws"],
                                     a["n"], None) == status


@pytest.mark.gpu
def test_binding_refusals(pkg):
    plan = pkg.Int4LinearPlan(pkg.Int4LinearConfig(64, 128, 8, 64, True))
    other = pkg.Int4LinearPlan(pkg.Int4LinearConfig(64, 128, 8, 128, True))
    dev = dict(device="cuda")
    codes, zeros = torch.zeros((64, 64), dtype=torch.uint8, **dev), torch.zeros((64, 2), dtype=torch.uint8, **dev)
    scales = torch.ones((64, 2), dtype=torch.bfloat16, **dev)
    w = plan.transform_weight(codes, scales, zeros)
    x = torch.zeros((2, 128), dtype=torch.bfloat16, **dev)
    for bad in (dict(zeros=None), dict(scales=scales.half()), dict(scales=scales[:, :1]), dict(codes=codes[:, :32])):
        with pytest.raises(ValueError):
            plan.transform_weight(**{**dict(codes=codes, scales=scales, zeros=zeros), **bad})
    with pytest.raises(ValueError, match="laid out for"):
        other.forward(x, w)
    with pytest.raises(ValueError, match=r"\[T, 128\]"):
        plan.forward(x[:, :64], w)
    with pytest.raises(ValueError):
        plan.forward(x.half(), w)
    with pytest.raises(pkg.MoeError):
        plan.forward(torch.zeros((9, 128), dtype=torch.bfloat16, **dev), w)
    with pytest.raises(AttributeError):
        w.codes = codes
    w.codes.resize_(0)
    with pytest.raises(ValueError, match="resized"):
        plan.forward(x, w)
