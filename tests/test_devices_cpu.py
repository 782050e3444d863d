"""Tensors on a GPU that is not the current one: every call reaches the
library with the tensors' device current and on that device's stream. On the
host, with stand-ins for the devices and the library."""
import contextlib

import pytest
import torch

import maxsim_scoring_gb300 as ms
from maxsim_scoring_gb300 import _native, ops


class FakeLibrary:
    """Records (entry point, current device, stream) of every call; answers OK."""

    def __init__(self, devices):
        self.devices, self.calls = devices, []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, self.devices.current, args[-1]))
            return 0
        return call


class Devices:
    def __init__(self):
        self.current = 0

    @contextlib.contextmanager
    def device(self, index):
        before, self.current = self.current, getattr(index, "index", index)
        try:
            yield
        finally:
            self.current = before


@pytest.fixture
def fake(monkeypatch):
    """Two devices, 0 current; CPU tensors pass for tensors on device 1."""
    devices = Devices()
    library = FakeLibrary(devices)
    monkeypatch.setattr(_native, "lib", lambda: library)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 1)
    monkeypatch.setattr(ops, "_current_device", lambda: devices.current, raising=False)
    monkeypatch.setattr(ops, "_raw_stream", lambda index: 100 + index)
    monkeypatch.setattr(torch.cuda, "device", devices.device)
    return devices, library


def operators():
    x, i8, one = torch.zeros(4, 8), torch.zeros(4, 8, dtype=torch.int8), torch.ones(4)
    return {"maxsim_quantize_rows": lambda: ms.quantize_rows(x, normalize=True),
            "maxsim_linear_int8": lambda: ms.linear_int8(i8, one, i8, one, one, out_dtype=torch.float32),
            "maxsim_dropout_fwd": lambda: ms.dropout_fwd(x, 0.5, 1, 2, x),
            "maxsim_dropout_bwd": lambda: ms.dropout_bwd(x, 0.5, 1, 2)}


@pytest.mark.parametrize("name", ["maxsim_quantize_rows", "maxsim_linear_int8", "maxsim_dropout_fwd", "maxsim_dropout_bwd"])
@pytest.mark.parametrize("current", [0, 1])
def test_token_head_calls_with_the_tensors_device_current(fake, name, current):
    devices, library = fake
    devices.current = current
    operators()[name]()
    assert library.calls == [(name, 1, 101)] and devices.current == current


def test_other_entry_points_run_with_the_tensors_device_current(fake):
    devices, _ = fake
    seen = []

    @ops._on_tensors_device
    def entry(Q, D=None):
        seen.append(devices.current)
        if D is not None:
            raise ValueError("no")

    entry(torch.zeros(1))
    entry(Q=torch.zeros(1))
    with pytest.raises(ValueError):
        entry(torch.zeros(1), D=1)
    assert seen == [1, 1, 1] and devices.current == 0
    for fn in (ms.maxsim_fwd, ms.maxsim_fwd_varlen, ms.maxsim_score_pairs_packed, ms.maxsim_bwd, ms.maxsim_bwd_varlen,
               ms.maxsim_fwd_int8, ms.chamfer_fwd, ms.chamfer_bwd, ms.maxsim_topk, ms.maxsim_two_stage_topk,
               ms.maxsim_fwd_streamed, ms.maxsim_fwd_varlen_streamed):
        assert fn.__wrapped__.__name__ == fn.__name__


@pytest.mark.parametrize("workspace", [torch.zeros(64, dtype=torch.uint8), torch.zeros(64, 2, dtype=torch.uint8, device="meta")[:, 0]])
def test_workspace_elsewhere_or_strided_is_refused(workspace):
    # its bytes from data_ptr() on would not be the device's, or not the tensor's
    with pytest.raises(ValueError):
        ops._workspace(32, torch.device("meta"), workspace)
    assert ops._workspace(32, torch.device("meta"), torch.zeros(64, dtype=torch.uint8, device="meta"))[1] == 64
    with pytest.raises(ValueError):
        ops._workspace(65, torch.device("meta"), torch.zeros(64, dtype=torch.uint8, device="meta"))
