"""Which device and stream the bindings hand to the library, with another device current: fakes of
the library and of torch's device calls, no GPU."""
import contextlib

import pytest
import torch

import megatron_tensor_transformer_tma_gb300 as mlpb


class _Lib:
    """Notes the arguments and the device that is current at each call."""

    def __init__(self, state):
        self.state, self.calls, self.result = state, [], mlpb.MLPB_OK

    def __getattr__(self, name):
        def fn(*args):
            self.calls.append((name, args, self.state["device"]))
            return self.result
        return fn


@pytest.fixture
def fake(monkeypatch):
    """A library and two devices, 0 current; the current stream of device d is 1000 + d."""
    state = {"device": 0}

    @contextlib.contextmanager
    def device(d):
        before = state["device"]
        state["device"] = d.index if isinstance(d, torch.device) else int(d)
        yield
        state["device"] = before
    lib = _Lib(state)
    monkeypatch.setattr(mlpb.mlpb, "load_library", lambda: lib)
    monkeypatch.setattr(mlpb.mlpb, "_raw_stream", lambda d: 1000 + d)
    monkeypatch.setattr(mlpb.mlpb, "_stream",
                        lambda s: 1000 + state["device"] if s is None else int(s))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: state["device"])
    monkeypatch.setattr(torch.cuda, "device", device)
    return lib


@pytest.mark.parametrize("dev", [0, 1])
def test_moe_error_is_read_on_the_handles_device(fake, dev):
    h = mlpb.MoEHandle(77, mlpb.make_moe_config(4, 64, 32, 8, 2), dev)
    fake.result = mlpb.MLPB_ETIMEOUT
    assert mlpb.mlpb_moe_last_device_error(h) == mlpb.MLPB_ETIMEOUT
    assert mlpb.mlpb_moe_last_device_error(h, 5) == mlpb.MLPB_ETIMEOUT
    h.ptr = 0
    assert fake.calls == [("mlpb_moe_last_device_error", (77, 1000 + dev), dev),
                          ("mlpb_moe_last_device_error", (77, 5), dev)]


class _Out:
    """Stands for a tensor of a plan or a call."""

    def __init__(self, shape, device, stream):
        self.shape, self.device, self.stream = shape, device, stream


@pytest.fixture
def made(fake, monkeypatch):
    """The tensors that torch.empty made: their device, and the stream that was current there."""
    out, now = [], []

    class External:
        def __init__(self, ptr, device=None):
            self.cuda_stream = ptr
            self.device = torch.device("cuda", fake.state["device"] if device is None
                                       else torch.device(device).index)

    @contextlib.contextmanager
    def stream(s):
        now.append(s)
        yield
        now.pop()

    def empty(shape, dtype=None, device=None):
        d = torch.device(device)
        d = torch.device("cuda", fake.state["device"] if d.index is None else d.index)
        here = [s.cuda_stream for s in now if s.device == d]
        out.append(_Out(shape, d, here[-1] if here else 1000 + d.index))
        return out[-1]
    monkeypatch.setattr(torch.cuda, "ExternalStream", External)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch, "empty", empty)
    for name in ("mlpb_act8_save", "mlpb_act8_grad", "mlpb_join_fwd", "mlpb_join_bwd",
                 "mlpb_moe_forward"):
        monkeypatch.setattr(mlpb.mlpb, name, lambda *a, **k: None)
    caches = (mlpb.mlpb.mlpb_act8_scales, mlpb.mlpb._join_ws_of)
    for c in caches:
        c.cache_clear()
    yield out
    for c in caches:
        c.cache_clear()


@pytest.mark.parametrize("name", ["act8", "join", "moe"])
@pytest.mark.parametrize("stream", [None, 5])
def test_a_plans_tensors_stay_on_its_device_and_stream(fake, made, name, stream):
    """A plan made with device 1 current, called with device 0 current and a raw stream handle."""
    fake.state["device"] = 1
    if name == "act8":
        plan = mlpb.ActCheckpoint8(3, 64)
    elif name == "join":
        plan = mlpb.Join(3, 64, "rms", "rms")
    else:
        plan = mlpb.MoEDecode(4, 64, 32, 8, 2)
        plan.handle.ptr = 0  # nothing to destroy
    assert made and all(t.device.index == 1 for t in made)
    fake.state["device"] = 0
    made.clear()
    x = _Out((3, 64), torch.device("cuda", 1), None)
    if name == "act8":
        plan.save(x, stream=stream)
        plan.grad(x, stream=stream)
    elif name == "join":
        plan.forward(x, x, stream=stream)
        plan.backward(x, x, x, x, x, x, stream=stream)
    else:
        plan.forward(x, x, x, x, stream=stream)
    assert len(made) >= 3
    assert all(t.device.index == 1 for t in made)
    assert all(t.stream == (1001 if stream is None else stream) for t in made)
