"""The product with 4-bit weights where it has tiles for every SM: whole rounds of tiles, tiles that are left and cut,
ragged tokens and features, one block of K and many. Tolerances as in test_int4.py."""
import numpy as np
import pytest
import torch

from test_int4 import KINDS, Weight, activations, pkg  # noqa: F401

pytestmark = pytest.mark.gpu


# tiles of 256 x 256: 32 (cut in two), 51, 72, 80 (four left, cut in four), 96 (twenty left), 140, 152 (none left), 153
@pytest.mark.parametrize("group,zeros,dtype", KINDS[:3])
@pytest.mark.parametrize("T,N,K", [
    (512, 4096, 96), (513, 4100, 160), (2048, 2049, 1056), (1024, 5120, 544), (700, 8000, 64), (1100, 7000, 512),
    (2048, 4864, 256), (4096, 2300, 32), (1025, 7681, 1184), (544, 9728, 2080),
])
def test_tiles_for_every_sm(pkg, T, N, K, group, zeros, dtype):  # noqa: F811
    rng = np.random.default_rng(T + N + K)
    w = Weight(pkg, N, K, group, zeros, dtype)
    x = activations(rng, T, K)
    ws = w.plan.alloc_workspace(T)
    ws.fill_(0xA5)
    out = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    w.check(x, w.plan.forward(x, w.kernel, out=out, workspace=ws))
    assert w.plan.last_status(ws) == 0


@pytest.mark.parametrize("T,stride,offset", [(600, 8, 8), (1000, 3, 5)])
def test_strides_and_what_lies_around(pkg, T, stride, offset):  # noqa: F811
    N, K = 3900, 352
    rng = np.random.default_rng(T)
    w = Weight(pkg, N, K, 64, True, torch.bfloat16)
    x = activations(rng, T, K, K + stride, offset)
    wide = torch.full((T + 2, N + 7), 7.0, dtype=torch.bfloat16, device="cuda")
    w.check(x, w.plan.forward(x, w.kernel, out=wide[1:-1, 3:3 + N]))
    for rest in (wide[0], wide[-1], wide[:, :3], wide[:, 3 + N:]):
        assert (rest == 7).all()


def test_rows_and_columns_do_not_mix(pkg):  # noqa: F811
    T, N, K = 800, 4500, 256
    w = Weight(pkg, N, K, 64, False, torch.bfloat16)
    x = activations(np.random.default_rng(1), T, K)
    clean = w.plan.forward(x, w.kernel)
    w.scales[4321, 3] = float("nan")
    bad = w.plan.transform_weight(w.codes, w.scales)
    x[777, 5] = float("inf")
    got = w.plan.forward(x, bad)
    assert torch.isnan(got[:, 4321]).all()
    keep = torch.ones_like(got, dtype=torch.bool)
    keep[:, 4321] = False
    keep[777] = False
    assert torch.equal(got[keep], clean[keep])
    assert not torch.isfinite(got[777]).any()


def test_same_bits_captured_and_beside_another(pkg):  # noqa: F811
    T, N, K = 1500, 4096, 1024
    w = Weight(pkg, N, K, 128, False, torch.bfloat16)
    x = activations(np.random.default_rng(2), T, K)
    want = w.plan.forward(x, w.kernel)
    outs = [torch.empty_like(want) for _ in range(2)]
    wss = [w.plan.alloc_workspace(T) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):  # two at once: their CTA pairs share the SMs as these come free
        for st, o, ws in zip(streams, outs, wss):
            w.plan.forward(x, w.kernel, out=o, workspace=ws, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.plan.forward(x, w.kernel, out=outs[0], workspace=wss[0])
    outs[0].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want)


def test_waits_of_pairs_that_run_out(pkg):  # noqa: F811
    T, N, K = 700, 8000, 1024
    w = Weight(pkg, N, K, 128, False, torch.bfloat16)
    x = activations(np.random.default_rng(5), T, K)
    ws = w.plan.alloc_workspace(T)
    for limit in (0, 1, 0):
        w.plan.set_wait_timeout(limit)
        got = w.plan.forward(x, w.kernel, workspace=ws)
        assert w.plan.last_status(ws) == (7 if limit else 0)
    w.check(x, got)
