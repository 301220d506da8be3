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
