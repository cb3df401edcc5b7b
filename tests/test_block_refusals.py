"""What the operators around the experts refuse, and the host-only calls: no GPU needed."""
import ctypes
import os

import pytest
import torch

INVALID, UNSUPPORTED, CAPACITY = 1, 2, 3


@pytest.fixture(scope="module")
def pkg():
    import serving_topk_permute_gb300 as p
    if not os.path.exists(p.library_path()):
        from serving_topk_permute_gb300 import build
        build.build()
    return p


@pytest.fixture(scope="module")
def C(pkg):
    from serving_topk_permute_gb300 import block
    block._lib()
    return block


A = 1 << 20  # an address that is never read: every call below is refused before a launch


def quant(C, **kw):
    base = dict(format=1, sf_layout=0, codes=A, sf=A, row_scale=None)
    base.update(kw)
    return C.QuantC(**base)


@pytest.mark.parametrize("args,status", [
    ((1, 0, 3, 64), 3 * 2), ((1, 1, 3, 64), 512), ((1, 1, 129, 160), 2 * 2 * 512), ((2, 0, 3, 64), 3 * 4),
    ((2, 1, 1, 288), 2 * 4 * 512), ((3, 1, 1, 256), 2 * 512), ((1, 1, 0, 64), 0),
])
def test_scale_sizes(C, args, status):
    n = ctypes.c_size_t()
    assert C._lib().moe_quant_sf_size(*args, ctypes.byref(n)) == 0
    assert n.value == status


@pytest.mark.parametrize("args,status", [
    ((0, 0, 3, 64), UNSUPPORTED), ((9, 0, 3, 64), UNSUPPORTED), ((1, 2, 3, 64), INVALID), ((1, 0, -1, 64), INVALID),
    ((1, 0, 3, 48), INVALID), ((1, 0, 3, 0), INVALID), ((1, 0, 3, 16416), INVALID),
])
def test_scale_size_refusals(C, args, status):
    n = ctypes.c_size_t()
    assert C._lib().moe_quant_sf_size(*args, ctypes.byref(n)) == status


@pytest.mark.parametrize("rows,K,x,stride,q,status", [
    (-1, 64, A, 64, {}, INVALID), (2, 33, A, 64, {}, INVALID), (2, 16416, A, 16416, {}, INVALID),
    (2, 64, None, 64, {}, INVALID), (2, 64, A + 1, 64, {}, INVALID), (2, 64, A, 63, {}, INVALID),
    (2, 64, A, 64, {"format": 0}, UNSUPPORTED), (2, 64, A, 64, {"codes": None}, INVALID),
    (2, 64, A, 64, {"codes": A + 8}, INVALID), (2, 64, A, 64, {"sf": None}, INVALID),
    (2, 64, A, 64, {"row_scale": A}, INVALID), (2, 64, A, 64, {"format": 2}, INVALID),
    (2, 64, A, 64, {"sf_layout": 3}, INVALID), (2, 64, A, 64, {"sf_layout": 1, "sf": A + 4}, INVALID),
    (0, 64, None, 0, {}, 0),
])
def test_quantize_refusals(C, rows, K, x, stride, q, status):
    assert C._lib().moe_quantize(rows, K, x, stride, ctypes.byref(quant(C, **q)), None) == status
    assert C._lib().moe_quantize(2, 64, A, 64, None, None) == INVALID


@pytest.mark.parametrize("kw,status", [
    ({"rows": -1}, INVALID), ({"H": 0}, INVALID), ({"H": 16385}, INVALID), ({"eps": -1.0}, INVALID),
    ({"eps": float("nan")}, INVALID), ({"eps": float("inf")}, INVALID), ({"x": None}, INVALID), ({"x": A + 1}, INVALID),
    ({"gamma": None}, INVALID), ({"gamma": A + 2}, INVALID), ({"out": None}, INVALID), ({"ldx": 63}, INVALID),
    ({"res": A, "ldr": 10}, INVALID), ({"sum": A, "lds": 10}, INVALID), ({"ldo": 10}, INVALID),
    ({"sum": 2 * A, "lds": 64}, INVALID),  # the sum and the output in one place
    ({"H": 40, "q": True}, INVALID), ({"rows": 0, "x": None, "gamma": None}, 0),
])
def test_norm_refusals(C, kw, status):
    a = dict(rows=2, H=64, x=A, ldx=64, res=None, ldr=0, gamma=A, eps=1e-6, sum=None, lds=0, out=2 * A, ldo=64, q=None)
    a.update(kw)
    q = ctypes.byref(quant(C)) if a["q"] else None
    assert C._lib().moe_add_rmsnorm(a["rows"], a["H"], a["x"], a["ldx"], a["res"], a["ldr"], a["gamma"], a["eps"],
                                    a["sum"], a["lds"], a["out"], a["ldo"], q, None) == status


@pytest.mark.parametrize("cfg,status", [
    ((0, 1, 1, 0, 0.0), INVALID), ((513, 1, 1, 0, 0.0), INVALID), ((8, 0, 1, 0, 0.0), INVALID),
    ((8, 9, 1, 0, 0.0), INVALID), ((64, 33, 1, 0, 0.0), INVALID), ((8, 2, 2, 0, 0.0), INVALID),
    ((8, 2, 1, 2, 0.0), UNSUPPORTED), ((8, 2, 1, 0, float("inf")), INVALID), ((8, 2, 1, 0, float("nan")), INVALID),
    ((8, 2, 0, 1, -1.0), 0), ((512, 32, 1, 0, 0.0), 0),
])
def test_router_config(C, cfg, status):
    n = ctypes.c_size_t()
    assert C._lib().moe_router_workspace_size(ctypes.byref(C.RouterConfigC(*cfg)), 5, ctypes.byref(n)) == status


@pytest.mark.parametrize("kw,status", [
    ({"T": -1}, INVALID), ({"logits": None}, INVALID), ({"logits": A + 2}, INVALID), ({"ld": 7}, INVALID),
    ({"ids": None}, INVALID), ({"w": None}, INVALID), ({"ids": A + 1}, INVALID), ({"counts": A + 2}, INVALID),
    ({"loss": A + 1}, INVALID), ({"ws": None}, INVALID), ({"ws": A + 16}, INVALID), ({"n": 8}, 4),
])
def test_router_forward_refusals(C, kw, status):
    a = dict(T=5, logits=A, ld=8, ids=A, w=A, counts=A, valid=A, mean=A, loss=A, ws=A, n=1 << 20)
    a.update(kw)
    cfg = C.RouterConfigC(8, 2, 1, 0, 0.1)
    assert C._lib().moe_router_forward(ctypes.byref(cfg), a["T"], a["logits"], a["ld"], None, a["ids"], a["w"],
                                       a["counts"], a["valid"], a["mean"], a["loss"], a["ws"], a["n"], None) == status


@pytest.mark.parametrize("kw,status", [
    ({"T": -1}, INVALID), ({"logits": None}, INVALID), ({"out": None}, INVALID), ({"ld": 7}, INVALID),
    ({"ldd": 7}, INVALID), ({"ids": None}, INVALID), ({"counts": None}, INVALID), ({"valid": None}, INVALID),
    ({"out": A + 2}, INVALID), ({"dw": A + 1}, INVALID), ({"T": 0}, 0),
])
def test_router_backward_refusals(C, kw, status):
    a = dict(T=5, logits=A, ld=8, ids=A, counts=A, valid=A, dw=A, dl=A, out=A, ldd=8)
    a.update(kw)
    cfg = C.RouterConfigC(8, 2, 1, 0, 0.1)
    assert C._lib().moe_router_backward(ctypes.byref(cfg), a["T"], a["logits"], a["ld"], None, a["ids"], a["counts"],
                                        a["valid"], a["dw"], a["dl"], a["out"], a["ldd"], None) == status


@pytest.mark.parametrize("kw,status", [
    ({}, 0), ({"fmt": "mxfp8"}, 0), ({"fmt": "mxfp4"}, 0), ({"fmt": "bf16"}, UNSUPPORTED), ({"out_features": 0}, INVALID),
    ({"out_features": (1 << 20) + 1}, INVALID), ({"in_features": 48}, INVALID), ({"in_features": 0}, INVALID),
    ({"in_features": 16416}, INVALID), ({"max_tokens": 0}, INVALID), ({"out_features": 7, "in_features": 96}, 0),
])
def test_linear_config(pkg, kw, status):
    base = dict(out_features=64, in_features=128, max_tokens=16, fmt="nvfp4")
    base.update(kw)
    assert pkg.linear_validate(pkg.LinearConfig(**base)) == status


def test_linear_calls_without_a_plan(C):
    L, n = C._lib(), ctypes.c_size_t()
    w = C.LinearWeightC(A, A, None)
    assert L.moe_linear_plan(None, None) == INVALID
    assert L.moe_linear_workspace_size(None, 1, ctypes.byref(n)) == INVALID
    assert L.moe_linear_weight_sf_size(None, ctypes.byref(n)) == INVALID
    assert L.moe_linear_transform_weight(None, ctypes.byref(w), ctypes.byref(w), None) == INVALID
    assert L.moe_linear_forward(None, 1, A, 64, ctypes.byref(w), A, 64, A, 1 << 20, None) == INVALID
    assert L.moe_linear_forward_quantized(None, 1, ctypes.byref(quant(C)), ctypes.byref(w), A, 64, A, 1 << 20,
                                          None) == INVALID
    assert L.moe_linear_set_wait_timeout(None, 0) == INVALID
    assert L.moe_linear_plan_destroy(None) == 0


def test_binding_refuses_what_is_not_a_device_tensor(pkg):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pkg.quantize(x, "mxfp8")
    with pytest.raises(ValueError):
        pkg.add_rmsnorm(x, torch.ones(64))
    with pytest.raises(ValueError):
        pkg.add_rmsnorm(x.float(), torch.ones(64))
    r = pkg.Router(pkg.RouterConfig(8, 2))
    with pytest.raises(ValueError):
        r.forward(torch.zeros(4, 8))
    with pytest.raises(ValueError):
        r.forward(torch.zeros(4, 8, dtype=torch.float64))
    with pytest.raises(pkg.MoeError):
        pkg.Router(pkg.RouterConfig(8, 9))
    with pytest.raises(ValueError):
        pkg.Quantized("mxfp8", (4, 64), torch.zeros(256, dtype=torch.uint8), torch.zeros(8, dtype=torch.uint8), None)


def test_binding_structs_match_the_header(pkg, C):
    from test_abi_cpu import _defines, _struct_fields
    assert [f for f, _ in C.QuantC._fields_] == _struct_fields("moe_quant")
    assert [f for f, _ in C.RouterConfigC._fields_] == _struct_fields("moe_router_config")
    assert [f for f, _ in C.LinearConfigC._fields_] == _struct_fields("moe_linear_config")
    assert [f for f, _ in C.LinearWeightC._fields_] == _struct_fields("moe_linear_weight")
    sf, lt = _defines("MOE_SF_"), _defines("MOE_LOGITS_")
    assert C.SF_LAYOUTS == {"rows": sf["MOE_SF_ROWS"], "atoms": sf["MOE_SF_ATOMS"]}
    assert C.LOGITS == {torch.float32: lt["MOE_LOGITS_F32"], torch.bfloat16: lt["MOE_LOGITS_BF16"]}
