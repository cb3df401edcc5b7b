"""The feed-forward half of a transformer block, end to end on the library's kernels:

    residual' = residual + x                      add_rmsnorm (one pass: sum, bf16 rows and
    h         = RMSNorm(residual')                             MXFP8 rows of h)
    ids, w    = top-k softmax(h gate^T)           Router (with per-expert counts)
    y         = sum_j w_j expert_{ids_j}(h)       Plan.forward (the routed experts)
    d         = h W^T                             LinearPlan (from the MXFP8 rows of h)

and a few steps of gradient descent on the router's gate with the balance loss alone, which evens
out the experts' load (Router.backward gives the gradient of the logits).

    python examples/moe_block.py --tokens 512 --hidden 2048 --inter 768 --experts 64 --top-k 8
"""
from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import serving_topk_permute_gb300 as lib  # noqa: E402


def mxfp8(w: torch.Tensor):
    """Checkpoint codes and row-major scale bytes of bf16 rows."""
    q = lib.quantize(w, "mxfp8", "rows")
    return q.codes, q.sf.view(w.shape[0], -1)


@dataclass
class Output:
    y: torch.Tensor            # routed experts, bf16 [T, H]
    dense: torch.Tensor        # projection, bf16 [T, N]
    residual: torch.Tensor     # bf16 [T, H]
    hidden: torch.Tensor       # normalised rows, bf16 [T, H]
    routing: lib.RouterOutput


class MoeBlock:
    """Random weights; buffers for up to max_tokens tokens are allocated once."""

    def __init__(self, hidden=2048, inter=768, experts=64, top_k=8, dense=2048, max_tokens=512, coef=1e-2, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std=1.0):
            return torch.randn(shape, generator=g, device="cuda") * std

        H, I, E = hidden, inter, experts
        self.eps, self.gamma = 1e-6, 1.0 + 0.1 * normal(H)
        # a gate that prefers some experts, as an untrained one may
        self.gate = normal(E, H, std=H ** -0.5) + 0.02 * normal(E, 1)
        self.router = lib.Router(lib.RouterConfig(E, top_k, renormalize=True, balance_coef=coef))
        self.experts = lib.Plan(lib.LayerConfig(E, H, I, top_k, max_tokens, "mxfp8"))
        w13, w13_sf = mxfp8(normal(E * 2 * I, H, std=H ** -0.5).bfloat16())
        w2, w2_sf = mxfp8(normal(E * H, I, std=I ** -0.5).bfloat16())
        self.checkpoint = {"w13": w13.view(E, 2 * I, H), "w13_sf": w13_sf.contiguous().view(E, 2 * I, H // 32),
                           "w2": w2.view(E, H, I), "w2_sf": w2_sf.contiguous().view(E, H, I // 32)}
        self.expert_weights = self.experts.transform_weights(self.checkpoint)
        self.dense = lib.LinearPlan(lib.LinearConfig(dense, H, max_tokens, "mxfp8"))
        self.dense_checkpoint = mxfp8(normal(dense, H, std=H ** -0.5).bfloat16())
        self.dense_weight = self.dense.transform_weight(*self.dense_checkpoint)
        self.workspace = self.experts.alloc_workspace(max_tokens)
        self.dense_workspace = self.dense.alloc_workspace(max_tokens)

    def logits(self, h: torch.Tensor) -> torch.Tensor:
        return h.float() @ self.gate.t()

    def forward(self, x: torch.Tensor, residual: torch.Tensor) -> Output:
        T, H = x.shape
        h, total, q = torch.empty_like(x), torch.empty_like(x), lib.Quantized.alloc("mxfp8", T, H, "atoms", x.device)
        lib.add_rmsnorm(x, self.gamma, self.eps, residual=residual, sum_out=total, out=h, quantized=q)
        r = self.router.forward(self.logits(h))
        y = self.experts.forward(h, r.topk_ids, r.topk_weights, self.expert_weights, workspace=self.workspace)
        d = self.dense.forward(q, self.dense_weight, workspace=self.dense_workspace)
        return Output(y, d, total, h, r)

    def balance_step(self, h: torch.Tensor, lr: float):
        """One step down the balance loss; returns it (a device tensor) and the tokens per expert."""
        logits = self.logits(h)
        r = self.router.forward(logits, training=True)
        d_logits = self.router.backward(logits, r.topk_ids, r.counts, r.num_valid, d_loss=torch.ones(1, device="cuda"))
        self.gate -= lr * (d_logits.t() @ h.float())
        return r.loss, r.counts


def main(argv=None) -> dict:
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("tokens", 512), ("hidden", 2048), ("inter", 768), ("experts", 64), ("top-k", 8),
                        ("steps", 40)):
        p.add_argument("--" + name, type=int, default=value)
    p.add_argument("--lr", type=float, default=2.0)
    a = p.parse_args(argv)
    block = MoeBlock(a.hidden, a.inter, a.experts, a.top_k, a.hidden, a.tokens, coef=1.0)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((a.tokens, a.hidden), generator=g, device="cuda").bfloat16()
    residual = (2.0 * torch.randn((a.tokens, a.hidden), generator=g, device="cuda")
                + 0.3 * torch.ones(a.hidden, device="cuda")).bfloat16()
    out = block.forward(x, residual)
    history = [block.balance_step(out.hidden, a.lr) for _ in range(a.steps)]
    losses = [loss.item() for loss, _ in history]
    load = [c.max().item() * a.experts / (a.tokens * a.top_k) for _, c in history]
    print(f"block of {a.tokens} tokens: experts' output rms {out.y.float().square().mean().sqrt().item():.4f}, "
          f"projection rms {out.dense.float().square().mean().sqrt().item():.4f}")
    print(f"balance loss {losses[0]:.4f} -> {losses[-1]:.4f}; largest expert load {load[0]:.2f}x -> {load[-1]:.2f}x the mean")
    return {"output": out, "losses": losses, "load": load, "block": block, "x": x, "residual": residual}


if __name__ == "__main__":
    main()
