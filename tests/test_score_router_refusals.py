"""What the score router refuses, and its host-only calls: no GPU needed."""
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
    from serving_topk_permute_gb300 import score_router
    score_router._lib()
    return score_router


def config(S, **kw):
    base = dict(num_experts=64, top_k=4, score=0, num_groups=8, top_groups=4, group_score=1, renormalize=1,
                logits_type=0, scale=1.0)
    base.update(kw)
    return S.ScoreRouterConfigC(**base)


@pytest.mark.parametrize("kw,status", [
    ({}, 0), ({"num_experts": 0}, INVALID), ({"num_experts": 520}, INVALID), ({"num_experts": 60}, INVALID),
    ({"top_k": 0}, INVALID), ({"top_k": 33}, INVALID), ({"top_k": 32}, 0), ({"top_k": 25, "top_groups": 3}, INVALID),
    ({"score": 2}, UNSUPPORTED), ({"score": -1}, UNSUPPORTED), ({"group_score": 2}, UNSUPPORTED),
    ({"num_groups": 0}, INVALID), ({"num_groups": 64, "top_groups": 4}, INVALID), ({"num_groups": 32}, 0),
    ({"top_groups": 0}, INVALID), ({"top_groups": 9}, INVALID), ({"renormalize": 2}, INVALID),
    ({"logits_type": 2}, UNSUPPORTED), ({"scale": float("inf")}, INVALID), ({"scale": float("nan")}, INVALID),
    ({"scale": 0.0}, 0),
])
def test_configurations(S, kw, status):
    n = ctypes.c_size_t()
    c = config(S, **kw)
    assert S._lib().moe_score_router_workspace_size(ctypes.byref(c), 10, ctypes.byref(n)) == status
    if status:  # every call checks it
        assert S._lib().moe_score_router_forward(ctypes.byref(c), 1, A, 64, None, None, A, A, None, None, None, 0,
                                                 None) == status
        assert S._lib().moe_score_router_backward(ctypes.byref(c), 1, A, 64, A, A, 2 * A, 64, None) == status


def test_workspace_sizes(pkg):
    r = pkg.ScoreRouter(pkg.ScoreRouterConfig(256, 8, num_groups=8, top_groups=4))
    assert r.workspace_size(0) > 0 and r.workspace_size(100) == r.workspace_size(0)
    assert r.workspace_size(10 ** 6) >= r.workspace_size(513) > 4 * 256
    with pytest.raises(pkg.MoeError):
        r.workspace_size(-1)


@pytest.mark.parametrize("kw,status", [
    ({"T": -1}, INVALID), ({"logits": None}, INVALID), ({"logits": A + 2}, INVALID), ({"ld": 63}, INVALID),
    ({"ids": None}, INVALID), ({"w": None}, INVALID), ({"ids": A + 2}, INVALID), ({"w": A + 1}, INVALID),
    ({"bias": A + 2}, INVALID), ({"counts": A + 2}, INVALID), ({"valid": A + 2}, INVALID), ({"ws": None}, INVALID),
    ({"ws": A + 128}, INVALID), ({"n": 100}, WORKSPACE),
])
def test_forward_refusals(S, kw, status):
    a = dict(T=600, logits=A, ld=64, bias=A, ids=A, w=A, counts=A, valid=A, ws=A, n=1 << 20)
    a.update(kw)
    c = config(S)
    assert S._lib().moe_score_router_forward(ctypes.byref(c), a["T"], a["logits"], a["ld"], a["bias"], None, a["ids"],
                                             a["w"], a["counts"], a["valid"], a["ws"], a["n"], None) == status


@pytest.mark.parametrize("kw,status", [
    ({"T": -1}, INVALID), ({"T": 0, "logits": None}, 0), ({"logits": None}, INVALID), ({"ids": None}, INVALID),
    ({"dw": None}, INVALID), ({"d": None}, INVALID), ({"d": A}, INVALID), ({"d": 2 * A + 2}, INVALID),
    ({"ld": 63}, INVALID), ({"ldd": 63}, INVALID), ({"dw": A + 2}, INVALID), ({"ids": A + 1}, INVALID),
])
def test_backward_refusals(S, kw, status):
    a = dict(T=600, logits=A, ld=64, ids=A, dw=A, d=2 * A, ldd=64)
    a.update(kw)
    for score, renorm in ((0, 1), (1, 0)):
        c = config(S, score=score, renormalize=renorm)
        assert S._lib().moe_score_router_backward(ctypes.byref(c), a["T"], a["logits"], a["ld"], a["ids"], a["dw"],
                                                  a["d"], a["ldd"], None) == status


@pytest.mark.parametrize("E,counts,rate,bias", [
    (0, A, 0.1, A), (513, A, 0.1, A), (8, None, 0.1, A), (8, A, 0.1, None), (8, A, float("nan"), A),
    (8, A + 2, 0.1, A), (8, A, 0.1, A + 1),
])
def test_bias_refusals(S, E, counts, rate, bias):
    assert S._lib().moe_score_router_update_bias(E, counts, rate, bias, None) == INVALID


def test_binding_refusals(pkg):
    with pytest.raises(ValueError, match="score must be"):
        pkg.ScoreRouter(pkg.ScoreRouterConfig(64, 4, score="tanh"))
    with pytest.raises(pkg.MoeError):
        pkg.ScoreRouter(pkg.ScoreRouterConfig(64, 4, num_groups=7))
    r = pkg.ScoreRouter(pkg.ScoreRouterConfig(64, 4))
    with pytest.raises(ValueError, match="CUDA"):
        r.forward(torch.zeros(3, 64))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        r.forward(torch.zeros((3, 64), dtype=torch.float16))
    with pytest.raises(ValueError, match="2-D"):
        r.forward(torch.zeros(64))
    with pytest.raises(AttributeError):
        r.cfg = None


def test_structs_match_the_header(S):
    import re
    from conftest import ROOT
    text = open(os.path.join(ROOT, "include", "moe.h")).read()
    body = re.search(r"typedef struct moe_score_router_config \{(.*?)\}", text, re.S).group(1)
    names = re.findall(r"^\s*(?:int32_t|float)\s+(\w+);", body, re.M)
    assert names == [n for n, _ in S.ScoreRouterConfigC._fields_]
    for name, table in (("SCORE", S.SCORES), ("GROUP", S.GROUP_SCORES)):
        for key, value in table.items():
            assert re.search(rf"#define MOE_{name}_{key.upper()}\s+{value}\b", text)
