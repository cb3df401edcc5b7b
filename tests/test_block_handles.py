"""What the handles of the operators around the experts refuse on the host, before any launch: stand-ins
take the place of the library and of device tensors, so no GPU is needed."""
import copy
import dataclasses
from contextlib import contextmanager

import pytest
import torch

import serving_topk_permute_gb300 as pkg
from serving_topk_permute_gb300 import block


class Library:
    """Stands in for the library: every call succeeds and is recorded, with the device that was current; sizes
    are 4096 bytes."""

    def __init__(self):
        self.calls, self.current, self.at = [], 0, []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            self.at.append(self.current)
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
    monkeypatch.setattr(block, "_current_device", lambda: lib.current, raising=False)

    @contextmanager
    def device(index):
        before, lib.current = lib.current, index
        yield
        lib.current = before

    monkeypatch.setattr(block, "_device", device, raising=False)
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


def contiguous(shape):
    strides = [1]
    for n in reversed(shape[1:]):
        strides.insert(0, strides[0] * n)
    return tuple(strides[:len(shape)])


class Tensor:
    """Stands in for a contiguous tensor on a device of that number (-1: the host); strides may be given."""

    _next = [1 << 20]

    def __init__(self, shape, dtype=torch.uint8, device=0, stride=None):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, device
        self._stride = stride or contiguous(shape)
        self.address = Tensor._next[0]
        Tensor._next[0] += (self.numel() * self.element_size() + 4095) // 4096 * 4096 + 4096

    is_cuda = property(lambda self: self.index >= 0)
    device = property(lambda self: torch.device("cpu") if self.index < 0 else torch.device("cuda", self.index))

    def get_device(self): return self.index
    def data_ptr(self): return self.address
    def numel(self): return self.shape.numel()
    def element_size(self): return self.dtype.itemsize
    def stride(self): return self._stride
    def is_contiguous(self): return self._stride == contiguous(self.shape)


BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
SF_BYTES = 4096  # what the stand-in library gives for every size


def linear(library, N=64, K=128, fmt="nvfp4"):
    return pkg.LinearPlan(pkg.LinearConfig(N, K, 16, fmt))


def weight(N=64, K=128, fmt="nvfp4", sf_bytes=SF_BYTES, known=True, device=0):
    return pkg.LinearWeight(Tensor((N, K // block.VALUES_PER_BYTE[fmt]), device=device),
                            Tensor((sf_bytes,), device=device),
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


# ----------------------------------------------------------------------------- memory that moves

def moved(t, shape=None):
    """What resize_, set_ or an assignment to .data does to a tensor that a handle holds."""
    if shape is not None:
        t.shape, t._stride = torch.Size(shape), contiguous(shape)
    t.address += 1 << 30


def router_output(T=5, E=8, k=2, device=0, bytes_=4096):
    return pkg.RouterOutput(Tensor((T, k), I32, device), Tensor((T, k), F32, device), Tensor((E,), I32, device),
                            Tensor((1,), I32, device), Tensor((E,), F32, device), Tensor((1,), F32, device),
                            Tensor((bytes_,), U8, device))


BUFFERS = ("topk_ids", "topk_weights", "counts", "num_valid", "prob_mean", "loss", "workspace")


@pytest.mark.parametrize("name", BUFFERS)
def test_a_router_follows_a_buffer_that_moved(library, name):
    router, o, logits = pkg.Router(pkg.RouterConfig(8, 2)), router_output(), Tensor((5, 8), F32)
    router.forward(logits, out=o)
    moved(getattr(o, name))
    router.forward(logits, out=o)
    args = library.launches()[-1][1]
    assert list(args[5:12]) == [getattr(o, b).data_ptr() for b in BUFFERS]


@pytest.mark.parametrize("name", BUFFERS)
def test_a_router_refuses_a_buffer_without_memory(library, name):
    router, o, logits = pkg.Router(pkg.RouterConfig(8, 2)), router_output(), Tensor((5, 8), F32)
    router.forward(logits, out=o)
    before = len(library.launches())
    getattr(o, name).address = 0  # its storage was freed: to the library no buffer at all
    with pytest.raises(ValueError):
        router.forward(logits, out=o)
    assert len(library.launches()) == before


@pytest.mark.parametrize("name", BUFFERS[:-1])
def test_a_router_refuses_a_buffer_that_shrank(library, name):
    router, o, logits = pkg.Router(pkg.RouterConfig(8, 2)), router_output(), Tensor((5, 8), F32)
    router.forward(logits, out=o)
    before = len(library.launches())
    t = getattr(o, name)
    t.shape, t._stride = torch.Size((t.numel() - 1,)), (1,)
    with pytest.raises(ValueError):
        router.forward(logits, out=o)
    assert len(library.launches()) == before


def test_a_router_passes_on_what_is_left_of_its_workspace(library):
    router, o, logits = pkg.Router(pkg.RouterConfig(8, 2)), router_output(), Tensor((5, 8), F32)
    router.forward(logits, out=o)
    o.workspace.shape = torch.Size((512,))
    router.forward(logits, out=o)
    assert library.launches()[-1][1][12] == 512  # which the library then refuses if it is too small


def test_a_copied_router_output_writes_its_own_buffers(library):
    router, o, logits = pkg.Router(pkg.RouterConfig(8, 2)), router_output(), Tensor((5, 8), F32)
    router.forward(logits, out=o)
    twin = copy.deepcopy(o)
    for b in BUFFERS:
        moved(getattr(twin, b))
    router.forward(logits, out=twin)
    assert list(library.launches()[-1][1][5:12]) == [getattr(twin, b).data_ptr() for b in BUFFERS]
    router.forward(logits, out=o)
    assert list(library.launches()[-1][1][5:12]) == [getattr(o, b).data_ptr() for b in BUFFERS]


def quantized(T=4, K=128, fmt="nvfp4", device=0):
    return pkg.Quantized(fmt, (T, K), Tensor((T, K // block.VALUES_PER_BYTE[fmt]), device=device),
                         Tensor((SF_BYTES,), device=device), Tensor((T,), F32, device) if fmt == "nvfp4" else None,
                         "atoms")


@pytest.mark.parametrize("shape", [None, (2, 64)])
@pytest.mark.parametrize("name", ["codes", "sf", "row_scale"])
def test_quantised_rows_whose_memory_moved_are_refused(library, name, shape):
    q, x, plan = quantized(), Tensor((4, 128), BF16), linear(library)
    pkg.quantize(x, "nvfp4", out=q)
    pkg.add_rmsnorm(x, Tensor((128,), F32), quantized=q)
    run_linear(plan, weight(), x=q)
    before = len(library.launches())
    moved(getattr(q, name), shape)
    for call in (lambda: pkg.quantize(x, "nvfp4", out=q), lambda: pkg.add_rmsnorm(x, Tensor((128,), F32), quantized=q),
                 lambda: run_linear(plan, weight(), x=q)):
        with pytest.raises(ValueError):
            call()
    assert len(library.launches()) == before


@pytest.mark.parametrize("name", ["codes", "sf", "global_scale"])
def test_a_weight_whose_memory_moved_is_refused(library, name):
    w, plan = weight(), linear(library)
    run_linear(plan, w)
    before = len(library.launches())
    moved(getattr(w, name))
    with pytest.raises(ValueError):
        run_linear(plan, w)
    with pytest.raises(ValueError):
        run_linear(plan, w, x=quantized())
    assert len(library.launches()) == before


# ----------------------------------------------------------------------------- devices

class Stream:
    def __init__(self, device):
        self.device_index, self.cuda_stream = device, 77


def calls_on(library, dev, other=None, **kw):
    """Every launching call with its tensors on device dev; the tensor named `other` on the device after it."""
    d = lambda name: dev + 1 if name == other else dev  # noqa: E731
    library.current = dev
    plan = linear(library)
    library.current = 0
    router = pkg.Router(pkg.RouterConfig(8, 2))
    T, x, logits = 4, Tensor((4, 128), BF16, d("x")), Tensor((4, 8), F32, d("logits"))
    o = router_output(T, device=dev)
    if other in BUFFERS:
        t = getattr(o, other)
        t.index = dev + 1
    grad = dict(counts=Tensor((8,), I32, d("counts")), num_valid=Tensor((1,), I32, d("num_valid")),
                d_weights=Tensor((T, 2), F32, d("d_weights")), d_loss=Tensor((1,), F32, d("d_loss")),
                token_mask=Tensor((T,), torch.bool, d("mask")), out=Tensor((T, 8), F32, d("out")))
    src = (Tensor((64, 64), U8, d("w_codes")), Tensor((64, 8), U8, d("w_sf")), Tensor((1,), F32, d("w_scale")))
    return {
        "quantize": lambda: pkg.quantize(x, "nvfp4", out=quantized(device=d("q")), **kw),
        "norm": lambda: pkg.add_rmsnorm(x, Tensor((128,), F32, d("gamma")),
                                        residual=Tensor((4, 128), BF16, d("residual")),
                                        sum_out=Tensor((4, 128), BF16, d("sum")), out=Tensor((4, 128), BF16, d("out")),
                                        quantized=quantized(device=d("q")), **kw),
        "router": lambda: router.forward(logits, token_mask=Tensor((T,), torch.bool, d("mask")), out=o, **kw),
        "gradient": lambda: router.backward(logits, Tensor((T, 2), I32, d("ids")), **grad, **kw),
        "linear": lambda: run_linear(plan, weight(device=d("weight")), x=x, out=Tensor((T, 64), BF16, d("out")),
                                     workspace=Tensor((SF_BYTES,), U8, d("ws")), **kw),
        "linear from quantised rows": lambda: run_linear(
            plan, weight(device=d("weight")), x=quantized(device=d("q")), out=Tensor((T, 64), BF16, d("out")),
            workspace=Tensor((SF_BYTES,), U8, d("ws")), **kw),
        "transform": lambda: plan.transform_weight(*src, **kw),
        "status": lambda: plan.last_status(Tensor((SF_BYTES,), U8, d("ws")), **kw),
    }


NAMES = ("quantize", "norm", "router", "gradient", "linear", "linear from quantised rows", "transform", "status")


@pytest.fixture
def no_allocation(monkeypatch):
    monkeypatch.setattr(block.torch, "empty", lambda shape, dtype=None, device=None: Tensor(
        (shape,) if isinstance(shape, int) else shape, dtype or F32, device.index))


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("dev", [0, 1])
def test_a_call_runs_with_its_tensors_device_current(library, no_allocation, name, dev):
    """On that device's current stream, and the device that was current is current again afterwards."""
    calls_on(library, dev)[name]()
    (_, args), at = library.launches()[-1], library.at[-1]
    assert at == dev and library.current == 0
    assert 1000 + dev in args


@pytest.mark.parametrize("name,other", [
    ("quantize", "x"), ("quantize", "q"), ("norm", "x"), ("norm", "gamma"), ("norm", "residual"), ("norm", "sum"),
    ("norm", "out"), ("norm", "q"), ("router", "logits"), ("router", "mask"), *(("router", b) for b in BUFFERS),
    ("gradient", "logits"), ("gradient", "ids"), ("gradient", "counts"), ("gradient", "num_valid"),
    ("gradient", "d_weights"), ("gradient", "d_loss"), ("gradient", "mask"), ("gradient", "out"), ("linear", "x"),
    ("linear", "weight"), ("linear", "out"), ("linear", "ws"), ("linear from quantised rows", "q"),
    ("linear from quantised rows", "weight"), ("transform", "w_codes"), ("transform", "w_sf"), ("transform", "w_scale"),
    ("status", "ws"),
])
@pytest.mark.parametrize("dev", [0, 1])
def test_tensors_on_two_devices_are_refused(library, no_allocation, name, other, dev):
    call = calls_on(library, dev, other)[name]
    before = len(library.launches())
    with pytest.raises(ValueError):
        call()
    assert len(library.launches()) == before


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_device_is_refused(library, no_allocation, monkeypatch, name):
    monkeypatch.setattr(block, "_on", lambda stream: block.nullcontext())
    calls_on(library, 1, stream=Stream(1))[name]()
    assert 77 in library.launches()[-1][1]
    call = calls_on(library, 1, stream=Stream(0))[name]
    before = len(library.launches())
    with pytest.raises(ValueError):
        call()
    assert len(library.launches()) == before


def test_buffers_that_were_checked_on_one_device_are_not_taken_for_another(library):
    router, o = pkg.Router(pkg.RouterConfig(8, 2)), router_output()
    router.forward(Tensor((5, 8), F32), out=o)
    with pytest.raises(ValueError):
        router.forward(Tensor((5, 8), F32, 1), out=o)


@pytest.mark.parametrize("codes,sf,scale", [(0, 1, 0), (0, 0, 1), (1, 0, 0), (-1, 0, 0), (0, -1, 0)])
def test_the_tensors_of_a_handle_are_on_one_device(library, codes, sf, scale):
    c, s, g = Tensor((4, 64), device=codes), Tensor((SF_BYTES,), device=sf), Tensor((4,), F32, scale)
    with pytest.raises(ValueError):
        pkg.Quantized("nvfp4", (4, 128), c, s, g, "atoms")
    with pytest.raises(ValueError):
        pkg.LinearWeight(c, s, Tensor((1,), F32, scale), "nvfp4", (4, 128))


@pytest.mark.parametrize("workspace", [Tensor((SF_BYTES - 1,)), Tensor((16,)), Tensor((0,)), Tensor((SF_BYTES,), I32),
                                       Tensor((SF_BYTES,), stride=(2,))])
def test_a_status_is_read_from_a_whole_workspace_only(library, workspace):
    plan = linear(library)
    before = len(library.launches())
    with pytest.raises(ValueError):
        plan.last_status(workspace)
    assert len(library.launches()) == before
    assert plan.last_status(Tensor((SF_BYTES,))) == 0


# ----------------------------------------------------------------------------- on the device

@pytest.mark.gpu
def test_real_tensors_that_move():
    """resize_, set_, .data and a resized storage, on the device."""
    router, logits = pkg.Router(pkg.RouterConfig(64, 8)), torch.randn((33, 64), device="cuda")
    want = router.forward(logits, training=True)
    taken = []
    for how in ("set_", "data", "resize_", "storage"):
        o = router.alloc(33, training=True)
        router.forward(logits, out=o)
        for name in BUFFERS:
            t = getattr(o, name)
            fresh = torch.zeros_like(t)
            if how == "set_":
                t.set_(fresh)
            elif how == "data":
                t.data = fresh
            elif how == "resize_":
                shape = t.shape
                t.resize_(1 << 22).resize_(shape).zero_()
            else:
                n = t.untyped_storage().nbytes()
                t.untyped_storage().resize_(0)
                taken.append(torch.empty(n, dtype=torch.uint8, device="cuda"))  # the old place
                t.untyped_storage().resize_(n)
                t.zero_()
        router.forward(logits, out=o)
        for name in BUFFERS[:-1]:
            assert torch.equal(getattr(o, name), getattr(want, name)), (how, name)
    x = torch.randn((33, 64), device="cuda").bfloat16()
    q = pkg.quantize(x, "nvfp4")
    q.codes.set_(torch.zeros_like(q.codes))
    with pytest.raises(ValueError):
        pkg.quantize(x, "nvfp4", out=q)
