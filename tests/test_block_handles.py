"""What the handles of the operators around the experts refuse on the host, before any launch: stand-ins
take the place of the library and of device tensors, so no GPU is needed."""
import dataclasses

import pytest
import torch

import serving_topk_permute_gb300 as pkg
from serving_topk_permute_gb300 import block


class Library:
    """Stands in for the library: every call succeeds and is recorded; sizes are 4096 bytes."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            if name.endswith("_size"):
                args[-1]._obj.value = 4096
            return 0
        return call

    def launches(self):
        return [c for c in self.calls if c[0].split("_")[-1] in ("forward", "quantized", "backward", "quantize",
                                                                 "rmsnorm", "weight", "status")]


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(block, "_fns", lib)
    monkeypatch.setattr(block, "_raw_stream", lambda device: 1000 + device)
    return lib


def test_a_configuration_cannot_be_changed_under_its_handle(library):
    cfg = pkg.RouterConfig(64, 8, True, 0.1)
    router = pkg.Router(cfg)
    with pytest.raises(dataclasses.FrozenInstanceError):
        cfg.top_k = 1
    with pytest.raises(dataclasses.FrozenInstanceError):
        cfg.balance_coef = 0.0
    with pytest.raises(AttributeError):
        router.cfg = pkg.RouterConfig(64, 1)
    assert router.cfg is cfg and dataclasses.replace(cfg, top_k=1).top_k == 1
    lin = pkg.LinearConfig(64, 128, 16)
    plan = pkg.LinearPlan(lin)
    with pytest.raises(dataclasses.FrozenInstanceError):
        lin.out_features = 32
    with pytest.raises(AttributeError):
        plan.cfg = pkg.LinearConfig(32, 128, 16)
    assert plan.cfg is lin


def test_buffers_follow_what_the_library_was_told(library):
    """Also where a configuration is forced to another value: sizes are those of the handle's creation."""
    cfg = pkg.RouterConfig(64, 8)
    router = pkg.Router(cfg)
    object.__setattr__(cfg, "top_k", 1)
    o = router.alloc(5, device=torch.device("cpu"))
    assert o.topk_ids.shape == (5, 8) and router._c[torch.float32].top_k == 8
