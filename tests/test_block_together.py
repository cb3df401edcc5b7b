"""The sandwich norm, the score router, the routed experts and the 4-bit projection as a model's block runs them:
each stage against its formula in 64 bits on the inputs it had, the gradients back through the block, and the whole
block captured, replayed and run on two streams at once."""

import numpy as np
import pytest
import torch

from oracle import formats as OF
from oracle import moe as OM

import serving_topk_permute_gb300 as lib

pytestmark = pytest.mark.gpu

E, K, GROUPS, TOP_GROUPS, H, I = 32, 4, 4, 2, 512, 384
EPS, SCALE = 1e-6, 2.5
HALF = 2.0 ** -8  # a bf16 rounding, relative


class Block:
    """residual1 = residual + norm(x W4^T); h; experts of h by score; residual2 = residual1 + gate norm(experts)."""

    def __init__(self, max_tokens, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.g = g
        normal = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.posts = [1.0 + 0.1 * normal(H) for _ in range(2)]
        self.pres = [1.0 + 0.1 * normal(H) for _ in range(2)]
        self.codes = torch.randint(0, 256, (H, H // 2), generator=g, device="cuda", dtype=torch.uint8)
        self.scales = (0.02 * (0.5 + torch.rand((H, H // 64), generator=g, device="cuda"))).bfloat16()
        self.zeros = torch.randint(4, 12, (H, H // 64), generator=g, device="cuda", dtype=torch.uint8)
        self.proj = lib.Int4LinearPlan(lib.Int4LinearConfig(H, H, max_tokens, 64, True))
        self.weight = self.proj.transform_weight(self.codes, self.scales, self.zeros)
        self.router = lib.ScoreRouter(lib.ScoreRouterConfig(E, K, num_groups=GROUPS, top_groups=TOP_GROUPS, scale=SCALE))
        self.gate = normal(E, H) * H ** -0.5
        self.bias = 0.1 * normal(E)
        self.experts = lib.Plan(lib.LayerConfig(E, H, I, K, max_tokens, "mxfp8"))

        def mxfp8(w):
            q = lib.quantize(w, "mxfp8", "rows")
            return q.codes, q.sf.view(w.shape[0], -1)

        w13, sf13 = mxfp8((normal(E * 2 * I, H) * H ** -0.5).bfloat16())
        w2, sf2 = mxfp8((normal(E * H, I) * I ** -0.5).bfloat16())
        self.checkpoint = {"w13": w13.view(E, 2 * I, H), "w13_sf": sf13.contiguous().view(E, 2 * I, H // 32),
                           "w2": w2.view(E, H, I), "w2_sf": sf2.contiguous().view(E, H, I // 32)}
        self.expert_weights = self.experts.transform_weights(self.checkpoint)

    def state(self, T):
        """Inputs, buffers and workspaces of one caller."""
        new = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
        s = {n: new(T, H) for n in ("x", "residual", "o", "z1", "h", "y", "z2", "h2")}
        s.update(gate=new(T, dtype=torch.float32), mask=torch.ones(T, dtype=torch.bool, device="cuda"),
                 stats1=new(T, 2, dtype=torch.float32), stats2=new(T, 2, dtype=torch.float32),
                 logits=new(T, E, dtype=torch.float32), routing=self.router.alloc(T),
                 ws4=self.proj.alloc_workspace(T), wse=self.experts.alloc_workspace(T))
        return s

    def fill(self, s, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        s["x"].normal_(generator=g)
        s["residual"].normal_(std=2.0, generator=g)
        s["gate"].uniform_(0.1, 1.0, generator=g)
        s["mask"][-1:] = False

    def forward(self, s):
        self.proj.forward(s["x"], self.weight, out=s["o"], workspace=s["ws4"])
        lib.sandwich_norm(s["o"], s["residual"], self.posts[0], self.pres[0], eps=EPS, sum_out=s["z1"], out=s["h"],
                          stats=s["stats1"])
        torch.mm(s["h"].float(), self.gate.t(), out=s["logits"])
        r = self.router.forward(s["logits"], self.bias, s["mask"], out=s["routing"])
        self.experts.forward(s["h"], r.topk_ids, r.topk_weights, self.expert_weights, workspace=s["wse"], out=s["y"])
        lib.sandwich_norm(s["y"], s["z1"], self.posts[1], self.pres[1], gate=s["gate"], eps=EPS, sum_out=s["z2"],
                          out=s["h2"], stats=s["stats2"])


def sandwich64(f, r, post, pre, gate):
    n = f * torch.rsqrt((f * f).mean(dim=1, keepdim=True) + EPS) * post
    z = r + (n if gate is None else gate[:, None] * n)
    return z, z * torch.rsqrt((z * z).mean(dim=1, keepdim=True) + EPS) * pre


def scores64(logits, ids, mask):
    p = torch.sigmoid(logits)
    pk = torch.where(ids >= 0, p.gather(1, ids.clamp(min=0)), 0.0)
    return torch.where(mask[:, None], SCALE * pk / pk.sum(dim=1, keepdim=True).clamp(min=1e-300), 0.0)


def within(got, want, slack):
    """bf16 results: half a step of the value, and of fp32 arithmetic what slack says"""
    got, want = got.double(), want.double()
    assert torch.isfinite(got).all()
    assert ((got - want).abs() <= HALF * want.abs() + slack).all(), ((got - want).abs() - HALF * want.abs()).max().item()


@pytest.fixture(scope="module")
def block():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)
    return Block(700)


@pytest.mark.parametrize("T", [1, 5, 16, 17, 150, 700])
def test_each_stage_of_the_block(block, T):
    s = block.state(T)
    block.fill(s, 10 + T)
    block.forward(s)
    torch.cuda.synchronize()
    assert block.proj.last_status(s["ws4"]) == 0
    f64 = lambda n: s[n].double()  # noqa: E731
    # the projection
    q = torch.stack((block.codes & 15, block.codes >> 4), dim=2).view(H, H).double()
    w = (q - block.zeros.double().repeat_interleave(64, 1)) * block.scales.double().repeat_interleave(64, 1)
    w = w if T <= 16 else w.bfloat16().double()
    want = f64("x") @ w.t()
    # H + 8 additions in fp32, each within 2^-24 of a partial sum that is below the sum of absolute products
    within(s["o"], want, (H + 8) * 2.0 ** -24 * (f64("x").abs() @ w.abs().t()))
    # the norms: a mean square of fewer than 32 additions in a row (a thread's, then a tree's) and ten more steps in
    # 32 bits, 2^-24 each: below 2^-18 of the values
    for f, r, z, h, n, gate in (("o", "residual", "z1", "h", 0, None), ("y", "z1", "z2", "h2", 1, s["gate"].double())):
        zw, hw = sandwich64(f64(f), f64(r), block.posts[n].double(), block.pres[n].double(), gate)
        within(s[z], zw, 2.0 ** -18 * (zw.abs() + f64(r).abs() + 1.0))
        within(s[h], hw, 2.0 ** -18 * (hw.abs() + 4.0))
    # the router: the experts are those of the best scores among the best groups, ids aside where they are too close
    ids = s["routing"].topk_ids.long()
    wr = scores64(f64("logits"), ids, s["mask"])
    assert ((s["routing"].topk_weights.double() - wr).abs() <= 2.0 ** -20 * SCALE).all()
    assert (ids[~s["mask"]] == -1).all() and (ids[s["mask"]] >= 0).all()
    assert torch.equal(torch.bincount(ids[ids >= 0], minlength=E).int(), s["routing"].counts)
    chosen = torch.sigmoid(f64("logits")) + block.bias.double()
    best = chosen.view(T, GROUPS, -1).topk(2, dim=2).values.sum(2).topk(TOP_GROUPS, dim=1).indices
    allowed = torch.zeros(T, GROUPS, dtype=torch.bool, device="cuda").scatter_(1, best, True).repeat_interleave(E // GROUPS, 1)
    top = torch.where(allowed, chosen, -10.0).topk(K, dim=1).values
    got = chosen.gather(1, ids.clamp(min=0))
    assert ((got - top).abs()[s["mask"]] <= 2.0 ** -20).all()
    # the experts, as the oracle has them
    ew = OM.ExpertWeights("mxfp8", **{k: v.cpu().numpy() for k, v in block.checkpoint.items()})
    bits = s["h"].view(torch.int16).cpu().numpy().view(np.uint16)
    want = OM.forward(OM.Layer(E, K, ew), bits, s["routing"].topk_ids.cpu().numpy(),
                      s["routing"].topk_weights.cpu().numpy(), return_parts=True)[1]["z"]
    y = s["y"].double().cpu().numpy()
    assert (np.abs(y - want) <= HALF * np.abs(want) + 2e-2 * np.sqrt(np.mean(want ** 2)) + 1e-3).all()
    assert (y[-1] == 0).all()  # the padded token


def test_quantised_rows_feed_the_projections_next_door(block):
    T = 77
    s = block.state(T)
    block.fill(s, 3)
    q = lib.Quantized.alloc("mxfp8", T, H, "atoms", "cuda")
    lib.sandwich_norm(s["x"], s["residual"], block.posts[0], block.pres[0], eps=EPS, sum_out=s["z1"], out=s["h"], quantized=q)
    g = torch.Generator(device="cuda").manual_seed(4)
    w = (torch.randn((H, H), generator=g, device="cuda") * H ** -0.5).bfloat16()
    wq = lib.quantize(w, "mxfp8", "rows")
    codes, sf = wq.codes, wq.sf.view(H, -1)
    plan = lib.LinearPlan(lib.LinearConfig(H, H, T, "mxfp8"))
    d = plan.forward(q, plan.transform_weight(codes, sf), workspace=plan.alloc_workspace(T))
    _, hw = sandwich64(s["x"].double(), s["residual"].double(), block.posts[0].double(), block.pres[0].double(), None)
    ref = hw.cpu().numpy() @ OF.mxfp8_dequantize(codes.cpu().numpy(), sf.cpu().numpy()).T
    # E4M3 roundings, within 2^-4 of each value, add up as their squares
    assert np.sqrt(np.mean((d.double().cpu().numpy() - ref) ** 2)) <= 2.0 ** -4 * np.sqrt(np.mean(ref ** 2))


def backward(block, s, c, d_z2, d_h2):
    """Back through the block, its experts taken as fixed rows c [E, H] that the weights mix."""
    T = s["x"].shape[0]
    b = {}
    two = lib.sandwich_norm_backward(s["y"], s["z1"], block.posts[1], block.pres[1], s["stats2"], gate=s["gate"],
                                     d_sum=d_z2, d_out=d_h2)
    ids = s["routing"].topk_ids.long()
    rows = c[ids.clamp(min=0)]  # [T, K, H]
    b["dw"] = torch.where(ids >= 0, (rows * two.f.float()[:, None, :]).sum(2), 0.0)
    b["dlogits"] = block.router.backward(s["logits"], s["routing"].topk_ids, b["dw"])
    b["dh"] = (b["dlogits"] @ block.gate).bfloat16()
    b["one"] = lib.sandwich_norm_backward(s["o"], s["residual"], block.posts[0], block.pres[0], s["stats1"],
                                          d_sum=two.residual, d_out=b["dh"])
    b["two"] = two
    assert T == ids.shape[0]
    return b


@pytest.mark.parametrize("T", [1, 33, 300])
def test_gradients_back_through_the_block(block, T):
    s = block.state(T)
    block.fill(s, 50 + T)
    block.forward(s)
    g = torch.Generator(device="cuda").manual_seed(T)
    c = torch.randn((E, H), generator=g, device="cuda")
    w = s["routing"].topk_weights
    s["y"].copy_((c[s["routing"].topk_ids.long().clamp(min=0)] * w[:, :, None]).sum(1))
    lib.sandwich_norm(s["y"], s["z1"], block.posts[1], block.pres[1], gate=s["gate"], eps=EPS, sum_out=s["z2"],
                      out=s["h2"], stats=s["stats2"])
    d_z2, d_h2 = (torch.randn((T, H), generator=g, device="cuda").bfloat16() for _ in range(2))
    b = backward(block, s, c, d_z2, d_h2)
    # each stage's gradient by autograd in 64 bits, at the values the stage had
    for n, f, r, gate, ds, do, got in ((1, "y", "z1", s["gate"], d_z2, d_h2, b["two"]),
                                       (0, "o", "residual", None, b["two"].residual, b["dh"], b["one"])):
        leaves = [t.double().requires_grad_() for t in (s[f], s[r], block.posts[n], block.pres[n])]
        gl = None if gate is None else gate.double().requires_grad_()
        z, h = sandwich64(*leaves, gl)
        ((z * ds.double()).sum() + (h * do.double()).sum()).backward()
        # a row's gradient: two reductions over H whose terms are below the row's largest gradient times its values
        for have, want in ((got.f, leaves[0].grad), (got.residual, leaves[1].grad)):
            within(have, want, 2.0 ** -16 * want.abs().amax(dim=1, keepdim=True) + 2.0 ** -18)
        for have, want in ((got.gamma_post, leaves[2].grad), (got.gamma_pre, leaves[3].grad)):
            assert ((have.double() - want).abs() <= 2.0 ** -16 * (want.abs().max() + T)).all()
        if gl is not None:
            assert ((got.gate.double() - gl.grad).abs() <= 2.0 ** -16 * (gl.grad.abs().max() + H)).all()
    logits = s["logits"].double().requires_grad_()
    (scores64(logits, s["routing"].topk_ids.long(), s["mask"]) * b["dw"].double()).sum().backward()
    assert ((b["dlogits"].double() - logits.grad).abs()
            <= 2.0 ** -18 * (logits.grad.abs() + b["dw"].double().abs().amax(dim=1, keepdim=True) * SCALE)).all()
    # and against differences: the loss along the logits' gradient, of the router alone (64 bits, central)
    if T > 1:
        d = b["dlogits"].double()
        step = 1e-5
        loss = lambda at: (scores64(at, s["routing"].topk_ids.long(), s["mask"]) * b["dw"].double()).sum()  # noqa: E731
        slope = (loss(s["logits"].double() + step * d) - loss(s["logits"].double() - step * d)) / (2 * step)
        assert abs(slope.item() - (d * d).sum().item()) <= 1e-4 * (d * d).sum().item()


@pytest.mark.parametrize("T", [3, 40, 520])
def test_captured_and_replayed_with_new_inputs(block, T):
    s, t = block.state(T), block.state(T)
    block.fill(s, 1)
    block.forward(s)  # warm-up
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.forward(s)
    for seed in (21, 22):
        block.fill(s, seed)
        block.fill(t, seed)
        graph.replay()
        block.forward(t)
        torch.cuda.synchronize()
        for n in ("o", "z1", "h", "z2", "h2", "y", "stats1", "stats2"):
            assert torch.equal(s[n], t[n]), n
        assert torch.equal(s["routing"].topk_ids, t["routing"].topk_ids)
        assert torch.equal(s["routing"].counts, t["routing"].counts)


def test_training_step_captured_while_an_eager_one_lives(block):
    T = 64
    s = block.state(T)
    block.fill(s, 5)
    block.forward(s)
    g = torch.Generator(device="cuda").manual_seed(6)
    c = torch.randn((E, H), generator=g, device="cuda")
    d_z2, d_h2 = (torch.randn((T, H), generator=g, device="cuda").bfloat16() for _ in range(2))
    eager = backward(block, s, c, d_z2, d_h2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = backward(block, s, c, d_z2, d_h2)
    graph.replay()
    torch.cuda.synchronize()
    for n in ("dw", "dlogits", "dh"):
        assert torch.equal(eager[n], held[n]), n
    for n in ("one", "two"):
        for a, b in zip(eager[n], held[n]):
            assert (a is None) == (b is None) and (a is None or torch.equal(a, b))


def test_two_streams_at_once(block):
    T = 200
    alone, a, b = block.state(T), block.state(T), block.state(T)
    for s in (alone, a, b):
        block.fill(s, 8)
    block.forward(alone)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for st, s in zip(streams, (a, b)):
            with torch.cuda.stream(st):
                block.forward(s)
    torch.cuda.synchronize()
    for s in (a, b):
        for n in ("o", "z1", "h", "y", "z2", "h2"):
            assert torch.equal(s[n], alone[n]), n
