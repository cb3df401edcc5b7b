"""Timing cases for operators beside the routed experts: the score router (sigmoid or softmax scores, a
selection bias, expert groups) and its gradient, the sandwich norm (a block's post-norm, gate, scaled
residual and the next block's pre-norm) and its gradient, and the product with 4-bit integer weights.

`own` selects between the operators' plain forms (elementary torch operations) and the library's kernels,
on the same inputs. Sizes follow this repository's workloads (hidden 2048, 4096 and 7168, 64 to 256 experts
with top 8) and odd sizes between them.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step's routing: sigmoid scores, balance bias, 4 of 8 groups; latency counts
        dict(name="route_decode", op="route", T=64, E=256, k=8, score="sigmoid", groups=8, top_groups=4,
             group_score="top2", bias=True, renorm=True, dtype="fp32", mask=False),
        # the same over a training or prefill batch with some padding tokens
        dict(name="route_prefill", op="route", T=16384, E=256, k=8, score="sigmoid", groups=8, top_groups=4,
             group_score="top2", bias=True, renorm=True, dtype="fp32", mask=True),
        # the gradient of a softmax router limited to 3 of 8 groups, experts no power of two, bf16 logits
        dict(name="route_grad_softmax", op="route_grad", T=777, E=160, k=6, score="softmax", groups=8, top_groups=3,
             group_score="max", bias=False, renorm=False, dtype="bf16", mask=False),
        # the gradient of the large batch above
        dict(name="route_grad", op="route_grad", T=16384, E=256, k=8, score="sigmoid", groups=8, top_groups=4,
             group_score="top2", bias=True, renorm=True, dtype="fp32", mask=True),
        # between two blocks of a decode step: 16 sequences, the next block's input as MXFP8 rows
        dict(name="norm_decode", op="norm", T=16, H=7168, gate="token", fmt="mxfp8", stats=False, strided=False),
        # the same over a training batch, row statistics kept for the backward pass
        dict(name="norm_train", op="norm", T=8192, H=7168, gate="channel", fmt="none", stats=True, strided=False),
        # the gradient for a small batch of odd rows sliced out of a wider buffer
        dict(name="norm_grad_ragged", op="norm_grad", T=500, H=2050, gate="token", strided=True),
        # the gradient of the training batch
        dict(name="norm_grad", op="norm_grad", T=8192, H=7168, gate="channel", strided=False),
        # one token through a 4-bit projection: weight streaming, latency counts
        dict(name="int4_token", op="int4", M=1, N=4096, K=7168, group=128, zeros=False, scale="bf16"),
        # a decode batch, small groups with zero points
        dict(name="int4_decode", op="int4", M=16, N=7168, K=4096, group=32, zeros=True, scale="bf16"),
        # ragged sizes between decoding and prefill, half-precision scales
        dict(name="int4_ragged", op="int4", M=77, N=2999, K=2080, group=64, zeros=True, scale="fp16"),
        # a prefill chunk through the gate/up projection of a dense block
        dict(name="int4_prefill", op="int4", M=2048, N=8192, K=4096, group=128, zeros=False, scale="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("route", "route_grad", "norm", "norm_grad", "int4", "int4"))
    if op in ("route", "route_grad"):
        E = rng.choice((8, 16, 60, 64, 96, 128, 160, 256, 384, 512))
        groups = rng.choice([g for g in (1, 2, 4, 6, 8, 16) if E % g == 0])
        top_groups = rng.randint(max(1, groups // 3), groups)
        k = rng.randint(1, min(10, top_groups * (E // groups)))
        return dict(op=op, T=_log_int(rng, 1, min(65536, 16384 * 256 // E)), E=E, k=k,
                    score=rng.choice(("sigmoid", "softmax")), groups=groups, top_groups=top_groups,
                    group_score=rng.choice(("max", "top2")), bias=rng.random() < 0.6, renorm=rng.random() < 0.7,
                    dtype=rng.choice(("fp32", "bf16")), mask=rng.random() < 0.4)
    if op == "norm":
        fmt = rng.choice(("none", "mxfp8"))
        H = _log_int(rng, 64, 8192)
        if fmt != "none":
            H = max(32, H // 32 * 32)
        return dict(op=op, T=_log_int(rng, 1, min(16384, 8192 * 7168 // H)), H=H,
                    gate=rng.choice(("none", "token", "channel")), fmt=fmt, stats=rng.random() < 0.5,
                    strided=rng.random() < 0.4)
    if op == "norm_grad":
        H = _log_int(rng, 64, 8192)
        return dict(op=op, T=_log_int(rng, 1, min(16384, 8192 * 7168 // H)), H=H,
                    gate=rng.choice(("none", "token", "channel")), strided=rng.random() < 0.4)
    N = _log_int(rng, 64, 8192)
    K = max(64, _log_int(rng, 256, 8192) // 32 * 32)
    M = _log_int(rng, 1, min(4096, 2048 * 8192 * 4096 // (N * K)))
    return dict(op="int4", M=M, N=N, K=K, group=rng.choice((32, 64, 128)), zeros=rng.random() < 0.5,
                scale=rng.choice(("bf16", "fp16")))


# ----------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 6151 + 29)


def _rows(g, T, H, strided, std=1.0):
    """bf16 rows with a few large channels, as deep layers have; strided: out of a wider buffer."""
    big = 1.0 + 15.0 * (torch.rand((1, H), generator=g, device=DEV) < 0.01).float()
    wide = torch.empty((T, H + 24 if strided else H), dtype=torch.bfloat16, device=DEV)
    wide[:, :H] = torch.randn((T, H), generator=g, device=DEV) * std * big
    return wide[:, :H]


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    s = {"case": c}
    if c["op"] in ("route", "route_grad"):
        T, E, k = c["T"], c["E"], c["k"]
        # a gate that prefers some experts, and the bias that balancing has given them by then
        pref = 0.5 * torch.randn(E, generator=g, device=DEV)
        logits = torch.randn((T, E), generator=g, device=DEV) + pref
        s["logits"] = logits.bfloat16() if c["dtype"] == "bf16" else logits
        spread = 0.2 if c["score"] == "sigmoid" else 0.5 / E
        s["bias"] = spread * (0.2 * torch.randn(E, generator=g, device=DEV) - pref) if c["bias"] else None
        s["mask"] = torch.rand(T, generator=g, device=DEV) < 0.9 if c["mask"] else None
        s["scale"] = 2.5 if c["renorm"] else 1.0
        if own:
            import serving_topk_permute_gb300 as pkg
            s["router"] = pkg.ScoreRouter(pkg.ScoreRouterConfig(
                E, k, score=c["score"], num_groups=c["groups"], top_groups=c["top_groups"],
                group_score=c["group_score"], renormalize=c["renorm"], scale=s["scale"]))
        if c["op"] == "route":
            if own:
                s["bufs"] = s["router"].alloc(T, device=DEV)
        else:
            # what a training step has in hand after the forward pass
            s["ids"] = _route_plain(s)["ids"]
            s["dw"] = torch.randn((T, k), generator=g, device=DEV)
            s["dlogits"] = torch.empty_like(s["logits"])
    elif c["op"] in ("norm", "norm_grad"):
        T, H = c["T"], c["H"]
        s["f"] = _rows(g, T, H, c["strided"])
        s["r"] = _rows(g, T, H, c["strided"], 3.0)
        s["post"] = 1.0 + 0.1 * torch.randn(H, generator=g, device=DEV)
        s["pre"] = 1.0 + 0.1 * torch.randn(H, generator=g, device=DEV)
        n = {"none": 0, "token": T, "channel": H}[c["gate"]]
        s["gate"] = 0.2 + torch.rand(n, generator=g, device=DEV) if n else None
        s["alpha"] = 0.9375
        if c["op"] == "norm":
            s["sum"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
            s["stats"] = torch.empty((T, 2), device=DEV) if c["stats"] else None
            if c["fmt"] == "none":
                s["out"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
            else:
                s["codes"] = torch.empty((T, H), dtype=torch.float8_e4m3fn, device=DEV)
                s["scales"] = torch.empty((T, H // 32), dtype=torch.float8_e8m0fnu, device=DEV)
                if own:
                    import serving_topk_permute_gb300 as pkg
                    s["q"] = pkg.Quantized("mxfp8", (T, H), s["codes"], s["scales"], None, "rows")
        else:
            s["stats"] = _norm_rows(s)["stats"]
            s["d_sum"] = _rows(g, T, H, c["strided"], 0.01)
            s["d_out"] = _rows(g, T, H, c["strided"], 0.01)
            s["d_f"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
            s["d_r"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
            if own:
                import serving_topk_permute_gb300 as pkg
                s["ws"] = torch.empty(pkg.sandwich_norm_workspace_size(T, H), dtype=torch.uint8, device=DEV)
    else:
        M, N, K, G = c["M"], c["N"], c["K"], c["group"]
        ch = torch.exp(0.5 * torch.randn((1, K), generator=g, device=DEV))
        s["x"] = (torch.randn((M, K), generator=g, device=DEV) * ch).bfloat16()
        s["codes"], s["scales"], s["zeros"] = _weight(g, N, K, G, c["zeros"], c["scale"])
        s["out"] = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
        if own:
            import serving_topk_permute_gb300 as pkg
            s["plan"] = pkg.Int4LinearPlan(pkg.Int4LinearConfig(N, K, M, group_size=G, zero_points=c["zeros"],
                                                                scale_dtype=s["scales"].dtype))
            s["w"] = s["plan"].transform_weight(s["codes"], s["scales"], s["zeros"])
            s["ws"] = s["plan"].alloc_workspace(M, device=DEV)
    return s


def _weight(g, N, K, G, zeros, scale):
    """A checkpoint's 4-bit weight: codes [N, K / 2] (element 2i in the low nibble), scales [N, groups] and
    zero points [N, groups] (one in a byte), rounded to nearest group by group."""
    groups = -(-K // G)
    w = torch.zeros((N, groups * G), device=DEV)
    w[:, :K] = torch.randn((N, K), generator=g, device=DEV) / math.sqrt(K)
    w = w.reshape(N, groups, G)
    if zeros:
        lo, hi = w.amin(2).clamp(max=0), w.amax(2).clamp(min=0)
        s = ((hi - lo) / 15).to(torch.bfloat16 if scale == "bf16" else torch.float16)
        z = (-lo / s.float()).round().clamp(0, 15)
    else:
        s = (w.abs().amax(2) / 7.5).to(torch.bfloat16 if scale == "bf16" else torch.float16)
        z = torch.full_like(s, 8.0, dtype=torch.float32)
    q = ((w / s.float()[:, :, None]).round() + z[:, :, None]).clamp(0, 15).to(torch.uint8)
    q = q.reshape(N, groups * G)[:, :K]
    return (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous(), s, z.to(torch.uint8) if zeros else None


def run(s):
    op = s["case"]["op"]
    if op == "route":
        return _route_own(s) if own else _route_plain(s)
    if op == "route_grad":
        return _route_grad_own(s) if own else _route_grad_plain(s)
    if op == "norm":
        return _norm_own(s) if own else _norm_plain(s)
    if op == "norm_grad":
        return _norm_grad_own(s) if own else _norm_grad_plain(s)
    return s["plan"].forward(s["x"], s["w"], out=s["out"], workspace=s["ws"]) if own else _int4_plain(s)


def work(case):
    c = case
    if c["op"] in ("route", "route_grad"):
        T, E, k = c["T"], c["E"], c["k"]
        row = E * (4 if c["dtype"] == "fp32" else 2)
        if c["op"] == "route":
            moved = T * row + 8 * T * k + 4 * E + (T if c["mask"] else 0) + (4 * E if c["bias"] else 0)
            return {"bytes": moved, "flops": 5 * T * E}
        dense = c["score"] == "softmax" and not c["renorm"]  # else only the picked logits have a gradient
        return {"bytes": T * row * (2 if dense else 1) + T * k * (8 if dense else 8 + row // E),
                "flops": T * (6 * E if dense else 8 * k)}
    if c["op"] == "norm":
        n = c["T"] * c["H"]
        moved = 6 * n + 8 * c["H"] + {"none": 0, "token": 4 * c["T"], "channel": 4 * c["H"]}[c["gate"]]
        moved += 2 * n if c["fmt"] == "none" else n + n // 32
        return {"bytes": moved + (8 * c["T"] if c["stats"] else 0), "flops": 12 * n}
    if c["op"] == "norm_grad":
        n = c["T"] * c["H"]
        moved = 12 * n + 8 * c["T"] + 16 * c["H"] + 2 * {"none": 0, "token": 4 * c["T"], "channel": 4 * c["H"]}[c["gate"]]
        return {"bytes": moved, "flops": 30 * n}
    M, N, K = c["M"], c["N"], c["K"]
    groups = -(-K // c["group"])
    moved = 2 * M * K + N * K // 2 + 2 * N * groups + (N * groups // 2 if c["zeros"] else 0) + 2 * M * N
    return {"bytes": moved, "flops": 2 * M * N * K}


# ----------------------------------------------------------------------------- the library's operators

def _route_own(s):
    b = s["router"].forward(s["logits"], bias=s["bias"], token_mask=s["mask"], out=s["bufs"])
    return {"ids": b.topk_ids, "weights": b.topk_weights, "counts": b.counts}


def _route_grad_own(s):
    return s["router"].backward(s["logits"], s["ids"], s["dw"], out=s["dlogits"])


def _norm_own(s):
    import serving_topk_permute_gb300 as pkg
    c = s["case"]
    pkg.sandwich_norm(s["f"], s["r"], s["post"], s["pre"], gate=s["gate"], alpha=s["alpha"], eps=EPS,
                      sum_out=s["sum"], out=s.get("out"), quantized=s.get("q"), stats=s["stats"])
    r = {"sum": s["sum"]}
    r.update({"out": s["out"]} if c["fmt"] == "none" else {"codes": s["codes"], "scales": s["scales"]})
    if c["stats"]:
        r["stats"] = s["stats"]
    return r


def _norm_grad_own(s):
    import serving_topk_permute_gb300 as pkg
    d = pkg.sandwich_norm_backward(s["f"], s["r"], s["post"], s["pre"], s["stats"], gate=s["gate"], alpha=s["alpha"],
                                   d_sum=s["d_sum"], d_out=s["d_out"], d_f=s["d_f"], d_residual=s["d_r"],
                                   workspace=s["ws"])
    r = {"d_f": d.f, "d_r": d.residual, "d_post": d.gamma_post, "d_pre": d.gamma_pre}
    if s["gate"] is not None:
        r["d_gate"] = d.gate
    return r


# ----------------------------------------------------------------------------- plain forms

def _scores(x, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    e = torch.exp(x - x.max(dim=1, keepdim=True).values)
    return e / e.sum(dim=1, keepdim=True)


def _route_plain(s):
    """Which experts: in 64 bits, where neighbours differ by less than 32 bits hold. The weights: in 32."""
    c = s["case"]
    x = s["logits"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    choice = _scores(x.double(), c["score"])
    if s["bias"] is not None:
        choice = choice + s["bias"].double()
    if c["top_groups"] < G:
        by_group = choice.reshape(T, G, E // G)
        best = torch.sort(by_group, dim=2, descending=True).values
        value = best[:, :, :2].sum(2) if c["group_score"] == "top2" else best[:, :, 0]
        kept = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        inside = torch.zeros((T, G), dtype=torch.bool, device=x.device).scatter(1, kept, True)
        choice = torch.where(inside[:, :, None], by_group, -math.inf).reshape(T, E)
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :k]
    w = _scores(x.float(), c["score"]).gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    w = w * s["scale"]
    if s["mask"] is not None:
        ids = torch.where(s["mask"][:, None], ids, -1)
        w = torch.where(s["mask"][:, None], w, 0.0)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=x.device)
    counts = counts.scatter_add(0, torch.where(ids < 0, E, ids).reshape(-1), torch.ones_like(ids).reshape(-1))[:E]
    return {"ids": ids.int(), "weights": w, "counts": counts.int()}


def _route_grad_plain(s):
    c = s["case"]
    p = _scores(s["logits"].float(), c["score"])
    ids = s["ids"].long()
    taken, at = ids >= 0, ids.clamp(min=0)
    pk = torch.where(taken, p.gather(1, at), 0.0)
    dw = torch.where(taken, s["dw"], 0.0) * s["scale"]
    if c["renorm"]:
        total = pk.sum(dim=1, keepdim=True).clamp(min=1e-38)
        dw = (dw - (dw * pk).sum(dim=1, keepdim=True) / total) / total
    dp = torch.zeros_like(p).scatter_add(1, at, torch.where(taken, dw, 0.0))
    if c["score"] == "sigmoid":
        d = dp * p * (1.0 - p)
    else:
        d = p * (dp - (p * dp).sum(dim=1, keepdim=True))
    return d.to(s["logits"].dtype)


def _gate(s):
    if s["gate"] is None:
        return 1.0
    return s["gate"][:, None] if s["case"]["gate"] == "token" else s["gate"]


def _norm_rows(s):
    f, r = s["f"].float(), s["r"].float()
    rf = torch.rsqrt((f * f).mean(dim=1, keepdim=True) + EPS)
    z = s["alpha"] * r + _gate(s) * (f * rf * s["post"])
    rz = torch.rsqrt((z * z).mean(dim=1, keepdim=True) + EPS)
    return {"z": z, "h": z * rz * s["pre"], "stats": torch.cat((rf, rz), 1)}


def _norm_plain(s):
    c = s["case"]
    n = _norm_rows(s)
    r = {"sum": n["z"].bfloat16()}
    if c["fmt"] == "none":
        r["out"] = n["h"].bfloat16()
    else:
        r["codes"], r["scales"] = _mxfp8(n["h"])
    if c["stats"]:
        r["stats"] = n["stats"]
    return r


def _mxfp8(y):
    """E4M3 codes and the power-of-two scale of each 32 elements: the smallest e with amax <= 448 * 2^e."""
    R, H = y.shape
    b = y.reshape(R, H // 32, 32)
    amax = b.abs().amax(2)
    frac, p = torch.frexp(amax)
    e = torch.where(amax > 0, (p - 9 + (frac > 0.875).int()).clamp(-126, 126), 0)
    v = b * ((127 - e) << 23).int().view(torch.float32)[:, :, None]
    return (v.clamp(-448.0, 448.0).reshape(R, H).to(torch.float8_e4m3fn),
            (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu))


def _norm_grad_plain(s):
    c = s["case"]
    f, r, g = s["f"].float(), s["r"].float(), _gate(s)
    rf, rz = s["stats"][:, :1], s["stats"][:, 1:]
    fn = f * rf
    u = fn * s["post"]
    zn = (s["alpha"] * r + g * u) * rz
    dh = s["d_out"].float()
    dzn = dh * s["pre"]
    dz = s["d_sum"].float() + rz * (dzn - zn * (dzn * zn).mean(dim=1, keepdim=True))
    du = dz * g
    dfn = du * s["post"]
    out = {"d_f": (rf * (dfn - fn * (dfn * fn).mean(dim=1, keepdim=True))).bfloat16(),
           "d_r": (s["alpha"] * dz).bfloat16(), "d_post": (du * fn).sum(0), "d_pre": (dh * zn).sum(0)}
    if c["gate"] != "none":
        out["d_gate"] = (dz * u).sum(1 if c["gate"] == "token" else 0)
    return out


def _int4_plain(s):
    c = s["case"]
    codes, G = s["codes"], c["group"]
    N, K = c["N"], c["K"]
    q = torch.stack((codes & 15, codes >> 4), dim=2).reshape(N, K).float()
    scale = s["scales"].float().repeat_interleave(G, dim=1)[:, :K]
    if s["zeros"] is None:
        w = (q - 8.0) * scale
    else:
        w = (q - s["zeros"].float().repeat_interleave(G, dim=1)[:, :K]) * scale
    return (s["x"].float() @ w.t()).bfloat16()


# ----------------------------------------------------------------------------- 64-bit values

def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "route":
        return _route_exact(s)
    if c["op"] == "route_grad":
        return _route_grad_exact(s)
    if c["op"] == "norm":
        z, h, stats = _norm_exact(s, s["f"].double(), s["r"].double(), s["post"].double(), s["pre"].double(),
                                  None if s["gate"] is None else s["gate"].double())
        r = {"sum": z}
        if c["fmt"] == "none":
            r["out"] = h
        else:
            r["codes"], r["scales"] = _mxfp8_exact(h)
        if c["stats"]:
            r["stats"] = stats
        return r
    if c["op"] == "norm_grad":
        leaves = {"d_f": s["f"], "d_r": s["r"], "d_post": s["post"], "d_pre": s["pre"]}
        if s["gate"] is not None:
            leaves["d_gate"] = s["gate"]
        leaves = {n: t.double().requires_grad_(True) for n, t in leaves.items()}
        z, h, _ = _norm_exact(s, leaves["d_f"], leaves["d_r"], leaves["d_post"], leaves["d_pre"], leaves.get("d_gate"))
        ((z * s["d_sum"].double()).sum() + (h * s["d_out"].double()).sum()).backward()
        return {n: t.grad for n, t in leaves.items()}
    N, K, G = c["N"], c["K"], c["group"]
    codes = s["codes"].long()
    w = torch.empty((N, K), dtype=torch.float64, device=DEV)
    w[:, 0::2], w[:, 1::2] = (codes % 16).double(), (codes // 16).double()
    for j in range(s["scales"].shape[1]):
        part = w[:, j * G:(j + 1) * G]
        part -= 8.0 if s["zeros"] is None else s["zeros"][:, j:j + 1].double()
        part *= s["scales"][:, j:j + 1].double()
    return torch.mm(s["x"].double(), w.t())


def _route_exact(s):
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    x = s["logits"].double()
    p = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, dim=1)
    choice = p if s["bias"] is None else p + s["bias"].double()
    grouped = choice.view(T, G, E // G)
    value = grouped.max(2).values
    if c["group_score"] == "top2" and E // G > 1:
        value = torch.topk(grouped, 2, dim=2).values.sum(2)
    kept = torch.argsort(value, dim=1, descending=True, stable=True)[:, :c["top_groups"]]
    group_of = torch.arange(E, device=DEV) // (E // G)
    allowed = (kept[:, :, None] == group_of).any(1)
    ids = torch.argsort(choice.masked_fill(~allowed, -math.inf), dim=1, descending=True, stable=True)[:, :k]
    w = torch.take_along_dim(p, ids, 1)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = w * s["scale"]
    if s["mask"] is not None:
        w = w * s["mask"][:, None]
    return {"ids": None, "weights": w, "counts": None}


def _route_grad_exact(s):
    """Through autograd of the weights, in 64 bits."""
    c = s["case"]
    x = s["logits"].double().requires_grad_(True)
    p = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, dim=1)
    rows = (s["ids"] >= 0).all(1)
    w = p[rows].gather(1, s["ids"][rows].long())
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    (w * s["scale"] * s["dw"][rows].double()).sum().backward()
    return x.grad


def _norm_exact(s, f, r, post, pre, gate):
    c = s["case"]
    rf = 1.0 / ((f ** 2).sum(1, keepdim=True) / c["H"] + EPS).sqrt()
    u = f * rf * post
    if gate is not None:
        u = u * (gate.unsqueeze(1) if c["gate"] == "token" else gate)
    z = r * s["alpha"] + u
    rz = 1.0 / ((z ** 2).sum(1, keepdim=True) / c["H"] + EPS).sqrt()
    return z, z * rz * pre, torch.cat((rf, rz), 1)


def _mxfp8_exact(y):
    R, H = y.shape
    b = y.reshape(R, H // 32, 32)
    amax = b.abs().amax(2)
    e = torch.ceil(torch.log2(torch.where(amax > 0, amax, 448.0) / 448.0))
    e = e + (amax > 448.0 * 2.0 ** e).int() - ((amax > 0) & (amax <= 448.0 * 2.0 ** (e - 1))).int()
    v = (b / (2.0 ** e)[:, :, None]).reshape(R, H)
    a = v.abs().clamp(max=448.0)
    step = 2.0 ** (torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.round(a / step) * step * torch.sign(v), 2.0 ** e
