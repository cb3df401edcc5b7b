"""Timing cases for the operators around the routed experts: the residual add with RMSNorm and an 8-bit
output, the router with its balance loss (forward and backward), and the microscaled linear product.

`own` selects between the operators' plain forms (elementary torch operations in 32 bits) and the
library's kernels, on the same inputs. Sizes follow this repository's workloads (hidden 2048, 4096 and
7168, 64 to 256 experts with top 8, intermediate 768 to 4096) and odd sizes between them.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
SF_BLOCK = {"mxfp8": 32, "mxfp4": 32, "nvfp4": 16}
EPS = 1e-6


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # a decode step's pre-expert norm: 16 sequences, latency counts
        dict(name="norm_decode", op="norm", T=16, H=7168, residual=True, fmt="mxfp8", strided=False),
        # the same norm over a whole prefill batch
        dict(name="norm_prefill", op="norm", T=8192, H=7168, residual=True, fmt="mxfp8", strided=False),
        # a norm without quantisation over rows sliced out of a wider buffer, hidden size no multiple of 8
        dict(name="norm_bf16_ragged", op="norm", T=2999, H=2050, residual=False, fmt="none", strided=True),
        # routing of one decode batch for serving: ids, weights and per-expert counts, no loss
        dict(name="router_decode", op="router", T=128, E=256, k=8, dtype="fp32", mask=False, loss=False, renorm=True),
        # a training micro-batch's router with the balance loss, some padding tokens
        dict(name="router_train", op="router", T=32768, E=256, k=8, dtype="fp32", mask=True, loss=True, renorm=True),
        # the gradient of that router, at a small batch with bf16 logits and at the large one
        dict(name="router_grad_small", op="router_grad", T=777, E=64, k=8, dtype="bf16", mask=False, renorm=True),
        dict(name="router_grad", op="router_grad", T=32768, E=256, k=8, dtype="fp32", mask=True, renorm=True),
        # one token through an NVFP4 projection: weight streaming, latency counts
        dict(name="linear_token", op="linear", M=1, N=4096, K=7168, fmt="nvfp4"),
        # a decode batch through an NVFP4 projection
        dict(name="linear_decode", op="linear", M=128, N=7168, K=4096, fmt="nvfp4"),
        # ragged sizes in MXFP4: rows, columns and K all off the tile grid
        dict(name="linear_ragged", op="linear", M=333, N=4100, K=2080, fmt="mxfp4"),
        # a shared expert's gate/up projection in MXFP8 over a prefill batch
        dict(name="linear_mxfp8", op="linear", M=4096, N=8192, K=4096, fmt="mxfp8"),
        # the largest: a square NVFP4 projection over a whole prefill batch
        dict(name="linear_prefill", op="linear", M=8192, N=7168, K=7168, fmt="nvfp4"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "router", "router_grad", "linear", "linear"))
    if op == "norm":
        fmt = rng.choice(("none", "mxfp8"))
        H = _log_int(rng, 64, 8192)
        if fmt != "none":
            H = max(32, H // 32 * 32)
        T = _log_int(rng, 1, min(16384, 8192 * 7168 // H))
        return dict(op=op, T=T, H=_not_excluded(H), residual=rng.random() < 0.7, fmt=fmt, strided=rng.random() < 0.4)
    if op in ("router", "router_grad"):
        E = rng.choice((8, 16, 60, 64, 96, 128, 160, 256, 384, 512))
        T = _log_int(rng, 1, min(65536, 32768 * 256 // E))
        k = rng.randint(1, min(10, E))
        c = dict(op=op, T=T, E=E, k=k, dtype=rng.choice(("fp32", "bf16")), mask=rng.random() < 0.5,
                 renorm=rng.random() < 0.7)
        if op == "router":
            c["loss"] = rng.random() < 0.6
        return c
    M = _log_int(rng, 1, 8192)
    N = _not_excluded(_log_int(rng, 64, 8192))
    K = _not_excluded(max(64, _log_int(rng, 256, 8192) // 32 * 32))
    return dict(op="linear", M=M, N=N, K=K, fmt=rng.choice(("nvfp4", "nvfp4", "mxfp4", "mxfp8")))


def _not_excluded(n):
    return n + 32 if n % 1024 == 0 and n // 1024 == 3 else n


# ----------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 13)


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    s = {"case": c}
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        wide = H + 24 if c["strided"] else H
        s["x"] = torch.randn((T, wide), generator=g, device=DEV).bfloat16()[:, :H]
        # a residual stream with a few large channels, as deep layers have
        big = 1.0 + 20.0 * (torch.rand((1, H), generator=g, device=DEV) < 0.01).float()
        s["r"] = (torch.randn((T, H), generator=g, device=DEV) * 3 * big).bfloat16() if c["residual"] else None
        s["gamma"] = 1.0 + 0.1 * torch.randn(H, generator=g, device=DEV)
        s["sum"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV) if c["residual"] else None
        if c["fmt"] == "none":
            s["out"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
        else:
            s["codes"] = torch.empty((T, H), dtype=torch.float8_e4m3fn, device=DEV)
            s["scales"] = torch.empty((T, H // 32), dtype=torch.float8_e8m0fnu, device=DEV)
            if own:
                import serving_topk_permute_gb300 as pkg
                s["q"] = pkg.Quantized("mxfp8", (T, H), s["codes"], s["scales"], None, "rows")
    elif c["op"] in ("router", "router_grad"):
        T, E, k = c["T"], c["E"], c["k"]
        bias = -1.1 * torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float32))
        logits = torch.randn((T, E), generator=g, device=DEV) + 0.5 * bias
        s["logits"] = logits.bfloat16() if c["dtype"] == "bf16" else logits
        s["mask"] = torch.rand(T, generator=g, device=DEV) < 0.9 if c["mask"] else None
        s["coef"] = 1e-2
        if own:
            import serving_topk_permute_gb300 as pkg
            s["router"] = pkg.Router(pkg.RouterConfig(E, k, renormalize=c["renorm"], balance_coef=s["coef"]))
            s["bufs"] = s["router"].alloc(T, training=c["op"] == "router_grad" or c["loss"], device=DEV)
        if c["op"] == "router_grad":
            # what a training step has in hand after the forward pass: ids, counts and upstream gradients
            f = _router_plain(s["logits"], s["mask"], k, c["renorm"], s["coef"])
            s["ids"], s["counts"], s["n"] = f["ids"], f["counts"], f["num_valid"]
            s["dw"] = torch.randn((T, k), generator=g, device=DEV)
            s["dloss"] = torch.rand(1, generator=g, device=DEV) + 0.5
            s["dlogits"] = torch.empty_like(s["logits"])
    else:
        M, N, K, fmt = c["M"], c["N"], c["K"], c["fmt"]
        # activations with a few large channels: what makes block scales differ
        ch = torch.exp(0.5 * torch.randn((1, K), generator=g, device=DEV))
        s["x"] = (torch.randn((M, K), generator=g, device=DEV) * ch).bfloat16()
        w = torch.randn((N, K), generator=g, device=DEV) / math.sqrt(K)
        values, scales, gs = _quantize_values(w, fmt, per_row=False)
        s["w_codes"], s["w_sf"] = _pack(values, fmt), scales
        s["w_gs"] = gs
        s["out"] = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
        if own:
            import serving_topk_permute_gb300 as pkg
            s["plan"] = pkg.LinearPlan(pkg.LinearConfig(N, K, M, fmt))
            s["w"] = s["plan"].transform_weight(s["w_codes"], s["w_sf"].view(torch.uint8), gs)
            s["ws"] = s["plan"].alloc_workspace(M, device=DEV)
    return s


def run(s):
    op = s["case"]["op"]
    if op == "norm":
        return _norm_own(s) if own else _norm_plain(s)
    if op == "router":
        return _router_own(s) if own else _router_run_plain(s)
    if op == "router_grad":
        return _router_grad_own(s) if own else _router_grad_plain(s)
    return s["plan"].forward(s["x"], s["w"], out=s["out"], workspace=s["ws"]) if own else _linear_plain(s)


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["T"] * c["H"]
        moved = 2 * n + (4 * n if c["residual"] else 0) + 4 * c["H"]
        moved += 2 * n if c["fmt"] == "none" else n + n // 32
        return {"bytes": moved, "flops": 8 * n}
    if c["op"] == "router":
        T, E, k = c["T"], c["E"], c["k"]
        moved = T * E * (4 if c["dtype"] == "fp32" else 2) + 8 * T * k + 4 * E + (T if c["mask"] else 0)
        return {"bytes": moved + (4 * E + 4 if c["loss"] else 0), "flops": 4 * T * E}
    if c["op"] == "router_grad":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": 2 * T * E * (4 if c["dtype"] == "fp32" else 2) + 8 * T * k + 4 * E + (T if c["mask"] else 0),
                "flops": 8 * T * E}
    M, N, K = c["M"], c["N"], c["K"]
    bits = 8 if c["fmt"] == "mxfp8" else 4
    return {"bytes": 2 * M * K + N * K * bits // 8 + N * K // SF_BLOCK[c["fmt"]] + 2 * M * N, "flops": 2 * M * N * K}


# ----------------------------------------------------------------------------- the library's operators

def _norm_own(s):
    import serving_topk_permute_gb300 as pkg
    if s["case"]["fmt"] == "none":
        pkg.add_rmsnorm(s["x"], s["gamma"], EPS, residual=s["r"], sum_out=s["sum"], out=s["out"])
        return {"out": s["out"], "sum": s["sum"]}
    pkg.add_rmsnorm(s["x"], s["gamma"], EPS, residual=s["r"], sum_out=s["sum"], quantized=s["q"])
    return {"codes": s["codes"], "scales": s["scales"], "sum": s["sum"]}


def _router_own(s):
    b = s["router"].forward(s["logits"], token_mask=s["mask"], out=s["bufs"])
    r = {"ids": b.topk_ids, "weights": b.topk_weights, "counts": b.counts}
    if s["case"]["loss"]:
        r["prob_mean"], r["loss"] = b.prob_mean, b.loss
    return r


def _router_grad_own(s):
    return s["router"].backward(s["logits"], s["ids"], s["counts"], s["n"], d_weights=s["dw"], d_loss=s["dloss"],
                                token_mask=s["mask"], out=s["dlogits"])


# ----------------------------------------------------------------------------- plain forms

def _norm_plain(s):
    c = s["case"]
    z = s["x"].float()
    if s["r"] is not None:
        z = z + s["r"].float()
    total = z.bfloat16() if s["r"] is not None else None
    y = z * torch.rsqrt((z * z).mean(dim=1, keepdim=True) + EPS) * s["gamma"]
    if c["fmt"] == "none":
        return {"out": y.bfloat16(), "sum": total}
    values, scales, _ = _quantize_values(y, "mxfp8", per_row=True)
    return {"codes": values.to(torch.float8_e4m3fn), "scales": scales, "sum": total}


def _router_plain(logits, mask, k, renorm, coef):
    """ids, weights, counts, mean probabilities and balance loss; -inf experts are never taken."""
    x = logits.float()
    T, E = x.shape
    order = torch.sort(x, dim=1, descending=True, stable=True)
    top, ids = order.values[:, :k], order.indices[:, :k]
    e = torch.exp(x - x.max(dim=1, keepdim=True).values)
    p = e / e.sum(dim=1, keepdim=True)
    w = p.gather(1, ids)
    if renorm:
        w = w / w.sum(dim=1, keepdim=True)
    ids = torch.where(top == -math.inf, -1, ids)
    if mask is not None:
        ids = torch.where(mask[:, None], ids, -1)
        w = torch.where(mask[:, None], w, 0.0)
        p = torch.where(mask[:, None], p, 0.0)
        n = mask.sum()
    else:
        n = torch.full((), T, device=x.device)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=x.device)
    counts = counts.scatter_add(0, torch.where(ids < 0, E, ids).reshape(-1), torch.ones_like(ids).reshape(-1))[:E]
    at_least_one = n.clamp(min=1).float()
    mean = p.sum(0) / at_least_one
    loss = coef * E * (counts.float() / (k * at_least_one) * mean).sum()
    return {"ids": ids.int(), "weights": w, "counts": counts.int(), "prob_mean": mean, "loss": loss.reshape(1),
            "num_valid": n.int().reshape(1), "p": p}


def _router_run_plain(s):
    c = s["case"]
    f = _router_plain(s["logits"], s["mask"], c["k"], c["renorm"], s["coef"])
    keep = ("ids", "weights", "counts") + (("prob_mean", "loss") if c["loss"] else ())
    return {name: f[name] for name in keep}


def _router_grad_plain(s):
    c = s["case"]
    x, ids = s["logits"].float(), s["ids"].long()
    T, E = x.shape
    e = torch.exp(x - x.max(dim=1, keepdim=True).values)
    p = e / e.sum(dim=1, keepdim=True)
    taken = ids >= 0
    at = ids.clamp(min=0)
    dw = torch.where(taken, s["dw"], 0.0)
    if c["renorm"]:
        pk = torch.where(taken, p.gather(1, at), 0.0)
        total = pk.sum(dim=1, keepdim=True).clamp(min=1e-38)
        dw = (dw - (dw * pk).sum(dim=1, keepdim=True) / total) / total
    n = s["n"].clamp(min=1).float()
    dp = (s["dloss"] * s["coef"] * E / (c["k"] * n * n)) * s["counts"].float().expand(T, E)
    dp = dp.scatter_add(1, at, torch.where(taken, dw, 0.0))
    d = p * (dp - (p * dp).sum(dim=1, keepdim=True))
    if s["mask"] is not None:
        d = torch.where(s["mask"][:, None], d, 0.0)
    return d.to(s["logits"].dtype)


def _linear_plain(s):
    c = s["case"]
    fmt, K = c["fmt"], c["K"]
    values, scales, gs = _quantize_values(s["x"].float(), fmt, per_row=True)
    x = _scaled(values, scales, fmt)
    w = _scaled(_unpack(s["w_codes"], fmt, K), s["w_sf"], fmt)
    y = x @ w.t()
    if fmt == "nvfp4":
        y = y * gs[:, None] * s["w_gs"]
    return y.bfloat16()


def _const(v, like):
    return torch.full((), v, dtype=like.dtype, device=like.device)


def _quantize_values(x, fmt, per_row):
    """Code values (fp32), block scales and, for NVFP4, the fp32 scale of each row or of the whole matrix."""
    R, K = x.shape
    B = SF_BLOCK[fmt]
    xb = x.reshape(R, K // B, B)
    amax = xb.abs().amax(dim=2)
    if fmt == "nvfp4":
        total = amax.amax(dim=1) if per_row else amax.max().reshape(1)
        gs = torch.where(total > 0, total / _const(2688.0, total), _const(1.0, total))
        g = gs[:, None] if per_row else gs
        sb = (amax / (g * 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
        eff = (sb.float() * g)[:, :, None]
        v = torch.where(eff > 0, xb / torch.where(eff > 0, eff, _const(1.0, eff)), _const(0.0, eff))
        return _round_e2m1(v).reshape(R, K), sb, gs
    top = 0.875 if fmt == "mxfp8" else 0.75
    frac, p = torch.frexp(amax)
    e = p - (9 if fmt == "mxfp8" else 3) + (frac > top).int()
    e = torch.where(amax > 0, e.clamp(-126, 126), 0)
    v = xb * _pow2(-e)[:, :, None]
    v = v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float() if fmt == "mxfp8" else _round_e2m1(v)
    return v.reshape(R, K), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu), None


def _pow2(e):
    return ((e + 127) << 23).int().view(torch.float32)


def _round_e2m1(v):
    """The nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with v's sign; ties to the even code."""
    return torch.tensor(E2M1, device=v.device)[_e2m1_magnitude(v)] * torch.sign(v)


def _e2m1_magnitude(v):
    a = v.abs()
    return ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))


def _pack(values, fmt):
    if fmt == "mxfp8":
        return values.to(torch.float8_e4m3fn).view(torch.uint8)
    code = (_e2m1_magnitude(values) + 8 * (values < 0)).to(torch.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _unpack(codes, fmt, K):
    if fmt == "mxfp8":
        return codes.view(torch.float8_e4m3fn).float()
    both = torch.stack((codes & 15, codes >> 4), dim=2).reshape(codes.shape[0], K).long()
    return torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)[both]


def _scaled(values, scales, fmt):
    R, K = values.shape
    sc = scales.float() if fmt == "nvfp4" else _pow2(scales.view(torch.uint8).int() - 127)
    return (values.reshape(R, K // SF_BLOCK[fmt], SF_BLOCK[fmt]) * sc[:, :, None]).reshape(R, K)


# ----------------------------------------------------------------------------- 64-bit values

def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "norm":
        z = s["x"].double() + (s["r"].double() if s["r"] is not None else 0.0)
        y = z / ((z ** 2).sum(1, keepdim=True) / c["H"] + EPS).sqrt() * s["gamma"].double()
        total = z if s["r"] is not None else None
        if c["fmt"] == "none":
            return {"out": y, "sum": total}
        v, e = _mx64(y, 448.0)
        return {"codes": _grid64(v, _e4m3_grid()), "scales": 2.0 ** e, "sum": total}
    if c["op"] == "router":
        p = torch.softmax(s["logits"].double(), dim=1)
        valid = s["mask"] if s["mask"] is not None else torch.ones(c["T"], dtype=torch.bool, device=DEV)
        ids = torch.argsort(s["logits"].double(), dim=1, descending=True, stable=True)[:, :c["k"]]
        w = torch.take_along_dim(p, ids, 1)
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True)
        out = {"ids": None, "weights": w * valid[:, None], "counts": None}
        if c["loss"]:
            n = max(int(valid.sum()), 1)
            counts = torch.bincount(ids[valid].reshape(-1), minlength=c["E"]).double()
            mean = p[valid].sum(0) / n
            out["prob_mean"] = mean
            out["loss"] = (s["coef"] * c["E"] * (counts * mean).sum() / (c["k"] * n)).reshape(1)
        return out
    if c["op"] == "router_grad":
        return _router_grad_exact(s)
    B = SF_BLOCK[c["fmt"]]
    M, N, K = c["M"], c["N"], c["K"]
    if c["fmt"] == "nvfp4":
        # the format's recipe decides scales and codes from fp32 quotients and products, each rounded to
        # nearest; what they stand for, and the sums, are 64-bit
        x = s["x"].float()
        gs = x.abs().amax(1) / torch.full((M,), 2688.0, device=DEV)
        gs = torch.where(gs > 0, gs, 1.0)
        blocks = x.reshape(M, K // B, B)
        sb = _grid64((blocks.abs().amax(2) / (gs * 6.0)[:, None]).double(), _e4m3_grid())
        eff = (sb.float() * gs[:, None])[:, :, None]
        q = _grid64(torch.where(eff > 0, blocks / eff.clamp(min=1e-38), 0.0).double(), _e2m1_grid())
        xd = (q * sb[:, :, None] * gs.double()[:, None, None]).reshape(M, K)
        w_scale = s["w_sf"].double() * s["w_gs"].double()
    else:
        v, e = _mx64(s["x"].double(), 448.0 if c["fmt"] == "mxfp8" else 6.0)
        q = _grid64(v, _e4m3_grid() if c["fmt"] == "mxfp8" else _e2m1_grid())
        xd = (q.reshape(M, K // B, B) * (2.0 ** e)[:, :, None]).reshape(M, K)
        w_scale = 2.0 ** (s["w_sf"].view(torch.uint8).double() - 127)
    codes = s["w_codes"]
    if c["fmt"] == "mxfp8":
        wv = codes.view(torch.float8_e4m3fn).double()
    else:
        wv = torch.empty((N, K), dtype=torch.float64, device=DEV)
        table = torch.cat((_e2m1_grid(), -_e2m1_grid()))
        wv[:, 0::2], wv[:, 1::2] = table[(codes % 16).long()], table[(codes // 16).long()]
    wd = (wv.reshape(N, K // B, B) * w_scale[:, :, None]).reshape(N, K)
    return torch.mm(xd, wd.t())


def _router_grad_exact(s):
    """Through autograd of the loss that the gradient belongs to, in 64 bits."""
    c = s["case"]
    x = s["logits"].double().requires_grad_(True)
    p = torch.softmax(x, dim=1)
    valid = s["mask"] if s["mask"] is not None else torch.ones(c["T"], dtype=torch.bool, device=DEV)
    n = max(int(valid.sum()), 1)
    w = p.gather(1, s["ids"].long().clamp(min=0))
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    share = s["counts"].double() / (c["k"] * n)
    loss = s["coef"] * c["E"] * (share * p[valid].sum(0) / n).sum()
    total = (w[valid] * s["dw"].double()[valid]).sum() + s["dloss"].double().sum() * loss
    total.backward()
    return x.grad


def _mx64(x, top):
    """Values scaled to their 32-element blocks' powers of two, and the exponents."""
    R, K = x.shape
    b = x.reshape(R, K // 32, 32)
    amax = b.abs().amax(2)
    e = torch.ceil(torch.log2(torch.where(amax > 0, amax, top) / top))
    e = e + (amax > top * 2.0 ** e).int() - ((amax > 0) & (amax <= top * 2.0 ** (e - 1))).int()
    return (b / (2.0 ** e)[:, :, None]).reshape(R, K), e


def _e2m1_grid():
    return torch.tensor(E2M1, dtype=torch.float64, device=DEV)


def _e4m3_grid():
    v = [m * 2.0 ** -9 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    return torch.tensor(v[:127], dtype=torch.float64, device=DEV)


def _grid64(x, grid):
    """The nearest grid value, ties to the even index, saturating; x's sign."""
    a = x.abs().clamp(max=float(grid[-1])).contiguous()
    hi = torch.searchsorted(grid, a).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    at = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return grid[at] * torch.sign(x)
