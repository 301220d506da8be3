"""Which device and stream the plans of a linear layer and of an update hand to the library, with
another device current: fakes of the library and of torch's device calls, no GPU."""
import contextlib

import pytest
import torch

import megatron_tensor_transformer_tma_gb300 as mlpb


class _Tensor:
    """Stands for a CUDA tensor of a plan or a call."""

    def __init__(self, shape, dtype, device, stream):
        self.shape, self.dtype, self.device, self.stream = torch.Size(shape), dtype, device, stream

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return 4096

    @property
    def nbytes(self):
        return self.numel()

    def __getitem__(self, _):
        return self

    def view(self, *_):
        return self


@pytest.fixture
def fake(monkeypatch):
    """A library and two devices; the current stream of device d is 1000 + d."""
    state = {"device": 1, "calls": [], "made": [], "streams": []}

    class Lib:
        def __getattr__(self, name):
            def fn(*args):
                state["calls"].append((name, state["device"], args[-1] if args else None))
                return mlpb.MLPB_OK
            return fn

    @contextlib.contextmanager
    def device(d):
        before = state["device"]
        state["device"] = d.index if isinstance(d, torch.device) else int(d)
        yield
        state["device"] = before

    class External:
        def __init__(self, ptr, device=None):
            self.cuda_stream, self.device = ptr, torch.device(device)

    @contextlib.contextmanager
    def stream(s):
        state["streams"].append(s)
        yield
        state["streams"].pop()

    def empty(shape, dtype=None, device=None):
        d = torch.device(device)
        here = [s.cuda_stream for s in state["streams"] if s.device == d]
        shape = (shape,) if isinstance(shape, int) else shape
        state["made"].append(_Tensor(shape, dtype, d, here[-1] if here else 1000 + d.index))
        return state["made"][-1]
    lib = Lib()
    monkeypatch.setattr(mlpb.mlpb, "load_library", lambda: lib)
    monkeypatch.setattr(mlpb.mlpb, "_raw_stream", lambda d: 1000 + d)
    monkeypatch.setattr(mlpb.mlpb, "_arg", lambda t, *a: None if t is None else t.data_ptr())
    monkeypatch.setattr(mlpb.mlpb, "_cuda_index", lambda t, name: t.device.index)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: state["device"])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "ExternalStream", External)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch, "empty", empty)
    mlpb.mlpb.mlpb_b128_sizes.cache_clear()
    yield state
    mlpb.mlpb.mlpb_b128_sizes.cache_clear()


@pytest.mark.parametrize("stream", [None, 5])
@pytest.mark.parametrize("name", ["linear", "muon"])
def test_plans_stay_on_their_device_and_stream(fake, name, stream):
    if name == "linear":
        plan = mlpb.Linear8(8, 64, 32)
    else:
        plan = mlpb.Muon(24, 40, 2)
    assert plan.handle.device == 1 and plan.device.index == 1
    assert all(t.device.index == 1 for t in fake["made"])
    fake["device"] = 0
    fake["made"].clear()
    fake["calls"].clear()
    dev = torch.device("cuda", 1)
    if name == "linear":
        plan.load(_Tensor((32, 64), torch.bfloat16, dev, None), stream=stream)
        plan.forward(_Tensor((8, 64), torch.bfloat16, dev, None), stream=stream)
        plan.backward(_Tensor((8, 32), torch.bfloat16, dev, None), stream=stream)
        made = 3
    else:
        t = _Tensor((2, 24, 40), torch.float32, dev, None)
        plan.orthogonalize(t, stream=stream)
        plan.step(t, t, t, t, stream=stream)
        made = 1
    want = 1001 if stream is None else stream
    assert fake["calls"] and all(c[1:] == (1, want) for c in fake["calls"])
    assert len(fake["made"]) == made and all(t.stream == want for t in fake["made"])
    plan.handle.ptr = 0  # nothing to destroy


@pytest.mark.parametrize("name", ["linear", "muon"])
def test_tensors_of_another_device_are_refused(fake, name):
    dev = torch.device("cuda", 0)
    if name == "linear":
        plan = mlpb.Linear8(8, 64, 32)
        with pytest.raises(ValueError, match="the handle on cuda:1"):
            plan.forward(_Tensor((8, 64), torch.bfloat16, dev, None))
    else:
        plan = mlpb.Muon(24, 40, 2)
        with pytest.raises(ValueError, match="the handle on cuda:1"):
            plan.orthogonalize(_Tensor((2, 24, 40), torch.float32, dev, None))
    plan.handle.ptr = 0


def test_a_layer_without_a_weight_is_refused(fake):
    dev = torch.device("cuda", 1)
    X, dY = (_Tensor((8, n), torch.bfloat16, dev, None) for n in (64, 32))
    plan = mlpb.Linear8(8, 64, 32)
    serving = mlpb.Linear8(8, 64, 32, training=False)
    fake["calls"].clear()
    for call in (lambda: plan.forward(X), lambda: serving.forward(X), lambda: plan.backward(dY),
                 lambda: plan.backward(dY, Xt=plan.saved(8))):
        with pytest.raises(ValueError, match="no weight yet"):
            call()
    with pytest.raises(ValueError, match="shape"):  # a refused weight is none
        plan.load(_Tensor((64, 32), torch.bfloat16, dev, None))
    with pytest.raises(ValueError, match="no weight yet"):
        plan.forward(X)
    assert not fake["calls"]
    plan.load(_Tensor((32, 64), torch.bfloat16, dev, None))
    plan.forward(X)
    plan.backward(dY)
    assert [c[0] for c in fake["calls"]] == ["mlpb_b128_quantize", "mlpb_linear8_forward",
                                             "mlpb_linear8_backward"]
    plan.handle.ptr = serving.handle.ptr = 0


def test_a_backward_takes_the_rows_of_the_last_forward(fake):
    """After a forward into an Xt of the caller's, the X^T of an earlier forward is not taken for
    its rows; it can be named."""
    dev = torch.device("cuda", 1)
    X, dY = (_Tensor((8, n), torch.bfloat16, dev, None) for n in (64, 32))
    plan = mlpb.Linear8(8, 64, 32)
    plan.load(_Tensor((32, 64), torch.bfloat16, dev, None))
    with pytest.raises(ValueError, match="the last forward kept no rows here"):
        plan.backward(dY)
    plan.forward(X)
    kept = mlpb.b128_empty(64, 8, dev)
    plan.forward(X, Xt=kept)
    fake["calls"].clear()
    with pytest.raises(ValueError, match="the last forward kept no rows here"):
        plan.backward(dY)
    assert not fake["calls"]
    plan.backward(dY, Xt=kept)
    plan.backward(dY, Xt=plan.saved(8))
    plan.forward(X)
    plan.backward(dY)
    plan.handle.ptr = 0
