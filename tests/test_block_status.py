"""The status of a product whose waits run out: every CTA reports in a word of its own, so the status
depends neither on the order in which CTAs run nor on what the workspace held before."""
import pytest
import torch

pytestmark = pytest.mark.gpu

GIVEN_UP = 7
FILL = 0xA5
WORD = int.from_bytes(bytes([FILL] * 4), "little", signed=True)

# products that quantise x themselves, clusters that split K, unsplit tiles, CTA pairs, more tiles of
# 128 features than two for each SM
CASES = [("nvfp4", 1, 1024, 8192), ("mxfp8", 8, 520, 4096), ("nvfp4", 9, 1024, 8192), ("mxfp8", 130, 520, 4096),
         ("mxfp4", 40, 2048, 7168), ("nvfp4", 600, 8200, 1056), ("mxfp8", 4, 50000, 64)]


@pytest.fixture(scope="module")
def pkg():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)
    import serving_topk_permute_gb300 as p
    p.lib()
    return p


def product(pkg, fmt, M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    x = torch.randn((M, K), device="cuda", generator=g).bfloat16()
    w = pkg.quantize(torch.randn((N, K), device="cuda", generator=g).bfloat16(), fmt, "rows")
    plan = pkg.LinearPlan(pkg.LinearConfig(N, K, M, fmt))
    kw = plan.transform_weight(w.codes, w.sf.view(N, -1), torch.ones(1, device="cuda") if fmt == "nvfp4" else None)
    return plan, kw, x


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("fmt,M,N,K", CASES)
def test_each_cta_reports_in_its_own_word(pkg, fmt, M, N, K, quantised):
    plan, kw, x = product(pkg, fmt, M, N, K)
    if quantised:
        x = pkg.quantize(x, fmt)
    ws = plan.alloc_workspace(M)
    words = ws.view(torch.int32)
    ctas = None
    for limit in (0, 1, 0):
        ws.fill_(FILL)
        plan.set_wait_timeout(limit)
        plan.forward(x, kw, workspace=ws)
        torch.cuda.synchronize()
        n = words[0].item()
        assert 0 < n and (ctas is None or n == ctas)
        ctas = n
        said = words[1:1 + n].tolist()
        assert set(said) <= {0, GIVEN_UP} and (GIVEN_UP in said) == (limit == 1)
        assert words[1 + n].item() == WORD  # nothing past the last CTA's word
        assert plan.last_status(ws) == (GIVEN_UP if limit else 0)
        assert plan.last_status(ws) == 0


def test_one_cta_among_many_is_heard(pkg):
    """A report in any single word is the status."""
    plan, kw, x = product(pkg, "mxfp8", 4, 70000, 64)
    ws = plan.alloc_workspace(4)
    words = ws.view(torch.int32)
    plan.forward(x, kw, workspace=ws)
    torch.cuda.synchronize()
    n = words[0].item()
    assert n > 512
    for cta in (0, 1, 511, 512, n - 1):
        plan.forward(x, kw, workspace=ws)
        assert plan.last_status(ws) == 0
        plan.forward(x, kw, workspace=ws)
        words[1 + cta] = GIVEN_UP
        assert plan.last_status(ws) == GIVEN_UP
        assert plan.last_status(ws) == 0


def test_a_run_that_gave_up_is_reported_every_time(pkg):
    """Many times in a row, with the kernels back to back on the stream."""
    plan, kw, x = product(pkg, "nvfp4", 130, 1024, 8192)
    rows, ws = pkg.quantize(x, "nvfp4"), plan.alloc_workspace(130)
    other = plan.alloc_workspace(130)
    for i in range(100):
        plan.set_wait_timeout(0)
        plan.forward(rows, kw, workspace=other)
        plan.set_wait_timeout(1)
        plan.forward(rows, kw, workspace=ws)
        plan.set_wait_timeout(0)
        plan.forward(rows, kw, workspace=other)
        assert plan.last_status(ws) == GIVEN_UP and plan.last_status(other) == 0, i
