"""examples/moe_block.py: the operators together as a model's block uses them, against the oracle."""
import os
import sys

import numpy as np
import pytest
import torch

from conftest import ROOT
from oracle import formats as OF
from oracle import moe as OM

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def result():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import moe_block
    finally:
        sys.path.pop(0)
    return moe_block.main(["--tokens", "150", "--hidden", "512", "--inter", "384", "--experts", "16", "--top-k", "4",
                           "--steps", "25"])


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def test_block_outputs_match_the_oracle(result):
    out, block = result["output"], result["block"]
    z = f64(result["x"]) + f64(result["residual"])
    h = z / np.sqrt((z * z).mean(axis=1, keepdims=True) + block.eps) * f64(block.gamma)
    assert np.abs(f64(out.hidden) - h).max() <= 2.0 ** -8 * np.abs(h).max()
    ck = {k: v.cpu().numpy() for k, v in block.checkpoint.items()}
    ew = OM.ExpertWeights("mxfp8", **ck)
    ids, w = out.routing.topk_ids.cpu().numpy(), out.routing.topk_weights.cpu().numpy()
    bits = out.hidden.view(torch.int16).cpu().numpy().view(np.uint16)
    want = OM.forward(OM.Layer(16, 4, ew), bits, ids, w, return_parts=True)[1]["z"]
    half = 2.0 ** -8 * np.abs(want)
    assert (np.abs(f64(out.y) - want) <= half + 2e-2 * np.sqrt(np.mean(want ** 2)) + 1e-3).all()
    codes, sf = (t.cpu().numpy() for t in block.dense_checkpoint)
    wd = OF.mxfp8_dequantize(codes, sf)
    ref = h @ wd.T
    # the rows' own E4M3 rounding: each value within 2^-4 of itself, errors add up as their squares
    assert np.sqrt(np.mean((f64(out.dense) - ref) ** 2)) <= 2.0 ** -4 * np.sqrt(np.mean(ref ** 2))


def test_balance_loss_goes_down(result):
    losses, load = result["losses"], result["load"]
    assert losses[-1] < losses[0] and load[-1] < load[0]
    assert losses[-1] >= 0.99  # E sum f P is 1 for an even load (coefficient 1)
