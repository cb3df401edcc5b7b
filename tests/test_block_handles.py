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


class Tensor:
    """Stands in for a contiguous tensor on a device of that number (-1: the host); strides may be given."""

    _next = [1 << 20]

    def __init__(self, shape, dtype=torch.uint8, device=0, stride=None):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, device
        self._stride = stride or torch.empty(shape, dtype=dtype, device="meta").stride()
        self.address = Tensor._next[0]
        Tensor._next[0] += (self.numel() * self.element_size() + 4095) // 4096 * 4096 + 4096

    is_cuda = property(lambda self: self.index >= 0)
    device = property(lambda self: torch.device("cpu") if self.index < 0 else torch.device("cuda", self.index))

    def get_device(self): return self.index
    def data_ptr(self): return self.address
    def numel(self): return self.shape.numel()
    def element_size(self): return self.dtype.itemsize
    def stride(self): return self._stride
    def is_contiguous(self): return self._stride == torch.empty(self.shape, device="meta").stride()


BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
SF_BYTES = 4096  # what the stand-in library gives for every size


def linear(library, N=64, K=128, fmt="nvfp4"):
    return pkg.LinearPlan(pkg.LinearConfig(N, K, 16, fmt))


def weight(N=64, K=128, fmt="nvfp4", sf_bytes=SF_BYTES, known=True, device=0):
    return pkg.LinearWeight(Tensor((N, K // block.VALUES_PER_BYTE[fmt]), device=device), Tensor((sf_bytes,), device=device),
                            Tensor((1,), F32, device) if fmt == "nvfp4" else None, *((fmt, (N, K)) if known else ()))


def run_linear(plan, w, T=4, device=0, N=64, K=128, **kw):
    kw.setdefault("x", Tensor((T, K), BF16, device))
    kw.setdefault("out", Tensor((T, N), BF16, device))
    kw.setdefault("workspace", Tensor((SF_BYTES,), U8, device))
    return plan.forward(weight=w, **kw)


@pytest.mark.parametrize("kw", [
    dict(N=32), dict(K=64), dict(fmt="mxfp4"), dict(fmt="mxfp8"), dict(sf_bytes=2048),
    dict(N=128, K=64),                                # as many bytes, another shape
    dict(N=32, known=False), dict(K=64, known=False), dict(fmt="mxfp4", known=False), dict(sf_bytes=2048, known=False),
])
def test_a_weight_of_another_plan_is_refused(library, kw):
    plan = linear(library)
    w = weight(**kw)
    before = len(library.launches())
    with pytest.raises(ValueError):
        run_linear(plan, w)
    assert len(library.launches()) == before
    run_linear(plan, weight())
    run_linear(plan, weight(known=False))
    assert len(library.launches()) == before + 2


@pytest.mark.parametrize("codes,sf,gs", [
    (Tensor((64, 64), F32), Tensor((SF_BYTES,)), None),
    (Tensor((64, 64), device=-1), Tensor((SF_BYTES,)), None),
    (Tensor((64, 64), stride=(65, 1)), Tensor((SF_BYTES,)), None),
    (Tensor((64, 64)), Tensor((SF_BYTES,), I32), None),
    (Tensor((64, 64)), Tensor((SF_BYTES,), device=-1), None),
    (Tensor((64, 64)), Tensor((SF_BYTES,)), Tensor((1,), F32, -1)),
    (Tensor((64, 64)), Tensor((SF_BYTES,)), Tensor((2,), F32)),
    (Tensor((64, 64)), Tensor((SF_BYTES,)), Tensor((1,), torch.float64)),
])
def test_a_weight_of_unfit_tensors_is_refused(library, codes, sf, gs):
    with pytest.raises(ValueError):
        pkg.LinearWeight(codes, sf, gs)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4", "mxfp4"])
def test_a_weight_of_another_plan_is_refused_by_the_library_at_hand(fmt):
    def made(N, K):
        q = pkg.quantize(torch.randn((N, K), device="cuda").bfloat16(), fmt, "rows")
        plan = pkg.LinearPlan(pkg.LinearConfig(N, K, 8, fmt))
        return plan, plan.transform_weight(q.codes, q.sf.view(N, -1),
                                           torch.ones(1, device="cuda") if fmt == "nvfp4" else None)

    plan, w = made(320, 512)
    x = torch.randn((8, 512), device="cuda").bfloat16()
    want = plan.forward(x, w)
    for N, K in ((64, 512), (320, 256), (640, 256), (319, 512)):
        with pytest.raises(ValueError):
            plan.forward(x, made(N, K)[1])
    same = pkg.LinearWeight(w.codes, w.sf, w.global_scale)  # format and shape not said: told by its bytes
    assert torch.equal(plan.forward(x, same), want)
