"""Memory that the operators around the experts allocate on a given stream belongs to that stream: while
the call waits there, the caller's stream must not be handed the call's workspace or output."""
import pytest
import torch

pytestmark = pytest.mark.gpu

T, H, N = 200, 512, 384
FILL = 0x5A


@pytest.fixture(scope="module")
def pkg():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)
    import serving_topk_permute_gb300 as p
    p.lib()
    return p


def _inputs():
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((T, H), device="cuda", generator=g).bfloat16()
    w = torch.randn((N, H), device="cuda", generator=g).bfloat16()
    return x, w


def _calls(pkg):
    x, w = _inputs()
    wq = pkg.quantize(w, "nvfp4", "rows")
    plan = pkg.LinearPlan(pkg.LinearConfig(N, H, T, "nvfp4"))
    kw = plan.transform_weight(wq.codes, wq.sf.view(N, -1), torch.ones(1, device="cuda"))  # rows' scales left out
    router = pkg.Router(pkg.RouterConfig(64, 4, balance_coef=0.01))
    logits = x[:, :64].float().contiguous()
    gamma = torch.ones(H, device="cuda")
    ro = router.forward(logits, training=True)
    return {
        "linear": lambda s: plan.forward(x, kw, stream=s),
        "quantize": lambda s: pkg.quantize(x, "mxfp8", stream=s).codes,
        "norm": lambda s: pkg.add_rmsnorm(x, gamma, stream=s),
        "router": lambda s: router.forward(logits, training=True, stream=s).topk_weights,
        "gradient": lambda s: router.backward(logits, ro.topk_ids, d_weights=ro.topk_weights, stream=s),
    }


@pytest.mark.parametrize("name", ["linear", "quantize", "norm", "router", "gradient"])
def test_temporary_memory_belongs_to_the_stream(pkg, name):
    call = _calls(pkg)[name]
    want = call(None).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # some 10 ms, while the caller's stream goes on
    got = call(side)
    # blocks of every size that the call could have given back to the caller's stream
    taken = [torch.full((1 << b,), FILL, dtype=torch.uint8, device="cuda") for b in range(9, 21) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
    for t in taken:
        assert bool((t == FILL).all()), f"{name}: the call wrote memory that another stream had been given"


def test_tensors_of_a_handle_cannot_be_replaced(pkg):
    x, w = _inputs()
    q = pkg.quantize(x, "mxfp8")
    with pytest.raises(AttributeError):
        q.codes = q.codes.clone()
    wq = pkg.quantize(w, "mxfp8", "rows")
    plan = pkg.LinearPlan(pkg.LinearConfig(N, H, T, "mxfp8"))
    kw = plan.transform_weight(wq.codes, wq.sf.view(N, -1))
    with pytest.raises(AttributeError):
        kw.sf = kw.sf.clone()


@pytest.mark.parametrize("M", [40, 600])
def test_scales_of_rows_are_those_of_this_call(pkg, M):
    """Rows of very different magnitudes back to back through one workspace: each product takes the row
    scales that its own quantiser wrote, and the norm the gamma that the kernel before it wrote."""
    g = torch.Generator(device="cuda").manual_seed(5)
    xs = [(torch.randn((M, H), device="cuda", generator=g) * 4.0 ** i).bfloat16() for i in range(-3, 4)]
    wq = pkg.quantize(torch.randn((8200, H), device="cuda", generator=g).bfloat16(), "nvfp4", "rows")
    plan = pkg.LinearPlan(pkg.LinearConfig(8200, H, M, "nvfp4"))
    kw = plan.transform_weight(wq.codes, wq.sf.view(8200, -1), torch.ones(1, device="cuda"))
    ws = plan.alloc_workspace(M)
    want = []
    for x in xs:
        want.append(plan.forward(x, kw, workspace=ws))
        torch.cuda.synchronize()
    for _ in range(10):
        got = [plan.forward(x, kw, workspace=ws) for x in xs]
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    gammas = [torch.rand(H, device="cuda", generator=g) + 0.5 for _ in xs]
    want = [pkg.add_rmsnorm(x, gm) for x, gm in zip(xs, gammas)]
    gamma = torch.empty(H, device="cuda")
    for _ in range(10):
        got = []
        for x, gm in zip(xs, gammas):
            gamma.copy_(gm)
            got.append(pkg.add_rmsnorm(x, gamma))
        for a, b in zip(got, want):
            assert torch.equal(a, b)
