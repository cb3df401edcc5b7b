"""The operators around the experts where offsets pass 2^31 elements: the last rows of huge batches
equal the same rows computed alone, bit for bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)
    import serving_topk_permute_gb300 as p
    p.lib()
    return p


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def tail(T, H, n=5, seed=0):
    """A bf16 [T, H] of zeros whose last n rows hold numbers."""
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(seed)
    x[-n:] = torch.randn((n, H), generator=g, device="cuda").bfloat16()
    return x


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
def test_norm_and_quantiser(pkg, fmt):
    T, H = 300_001, 7168
    assert T * H > 2 ** 31
    x = tail(T, H)
    gamma = torch.rand(H, device="cuda") + 0.5
    q = pkg.Quantized.alloc(fmt, T, H, "rows")
    out = pkg.add_rmsnorm(x, gamma, residual=x, quantized=q, out=torch.empty_like(x))
    small = pkg.Quantized.alloc(fmt, 200, H, "rows")  # as many rows as take the same path
    want = pkg.add_rmsnorm(x[-200:], gamma, residual=x[-200:], quantized=small, out=torch.empty_like(x[-200:]))
    assert torch.equal(out[-200:], want) and (out[:-5] == 0).all()
    assert torch.equal(q.codes[-200:], small.codes)
    assert torch.equal(q.sf.view(T, -1)[-200:], small.sf.view(200, -1))
    del out, q
    q, small = pkg.quantize(x, fmt, "rows"), pkg.quantize(x[-200:], fmt, "rows")
    assert torch.equal(q.codes[-200:], small.codes)
    assert torch.equal(q.sf.view(T, -1)[-200:], small.sf.view(200, -1))


def test_router_and_gradient(pkg):
    T, E, k = 4_300_000, 512, 4
    assert T * E > 2 ** 31
    logits = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    logits[-600:] = torch.randn((600, E), generator=g, device="cuda").bfloat16()
    mask = torch.zeros(T, dtype=torch.bool, device="cuda")
    mask[-600:] = True
    r = pkg.Router(pkg.RouterConfig(E, k, True, 0.5))
    o = r.forward(logits, token_mask=mask, training=True)
    s = r.forward(logits[-600:], training=True)
    assert torch.equal(o.topk_ids[-600:], s.topk_ids) and torch.equal(o.topk_weights[-600:], s.topk_weights)
    assert torch.equal(o.counts, s.counts) and o.num_valid.item() == 600
    assert (o.topk_ids[:-600] == -1).all()
    dw = torch.zeros((T, k), device="cuda")
    dw[-600:] = torch.randn((600, k), generator=g, device="cuda")
    d = r.backward(logits, o.topk_ids, o.counts, o.num_valid, d_weights=dw, d_loss=o.loss, token_mask=mask)
    w = r.backward(logits[-600:], s.topk_ids, s.counts, s.num_valid, d_weights=dw[-600:].contiguous(), d_loss=o.loss)
    assert torch.equal(d[-600:], w) and (d[:-600] == 0).all()


def test_linear(pkg):
    T, N, K = 300_001, 7168, 64
    assert T * N > 2 ** 31
    plan = pkg.LinearPlan(pkg.LinearConfig(N, K, T, "mxfp8"))
    g = torch.Generator(device="cuda").manual_seed(2)
    codes = torch.randint(0, 120, (N, K), generator=g, device="cuda", dtype=torch.uint8)
    sf = torch.full((N, K // 32), 120, dtype=torch.uint8, device="cuda")
    w = plan.transform_weight(codes, sf)
    x = tail(T, K)
    out = plan.forward(x, w)
    # K here is one stage: every kernel adds its products in the same order
    assert torch.equal(out[-7:], plan.forward(x[-7:], w))
    assert (out[:-5] == 0).all()
