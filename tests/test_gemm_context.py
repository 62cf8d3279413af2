"""Where gemm and gemm_scaled allocate and launch, with a fake library and
fake tensors (no GPU needed)."""
import contextlib
import types

import pytest
import torch

import bit_weight_only_g128_gb300 as w4

DEV = torch.device("cuda", 1)


class Tensor:
    """What the two functions ask of a tensor."""

    def __init__(self, shape, dtype, device=DEV):
        self.shape, self.dtype, self.device, self.is_cuda = shape, dtype, device, True

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def element_size(self):
        return 2

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000


class Stream:
    def __init__(self, device=DEV, handle=0x77):
        self.device, self.cuda_stream = device, handle


@pytest.fixture
def seen(monkeypatch):
    """What is current when: a list of (what, device index, stream handle)."""
    log = []
    current = dict(device=0, streams={0: 0x50, 1: 0x51})

    def note(what):
        log.append((what, current["device"], current["streams"][1]))

    @contextlib.contextmanager
    def on_device(d):
        before, current["device"] = current["device"], torch.device(d).index
        yield
        current["device"] = before

    @contextlib.contextmanager
    def on_stream(s):
        before = current["streams"][s.device.index]
        with on_device(s.device):
            current["streams"][s.device.index] = s.cuda_stream
            yield
        current["streams"][s.device.index] = before

    def empty(shape, dtype, device):
        note("result")
        return Tensor(shape, dtype, device)

    def workspace(need, device, stream):
        assert stream == current["streams"][device]
        note("workspace")
        return Tensor((need,), torch.uint8)

    def launch(*args):
        assert args[-1] == current["streams"][1]
        note("launch")
        return 0

    def size(*args):
        note("size")
        return 4096

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", on_stream)
    monkeypatch.setattr(torch.cuda, "device", on_device)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: current["streams"][d], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current["device"], raising=False)
    monkeypatch.setattr(w4, "stream_workspace", workspace)
    monkeypatch.setattr(w4, "workspace_size", size)
    monkeypatch.setattr(w4, "lib", lambda: types.SimpleNamespace(w4a16_gemm_ex=launch, w4a16_gemm_scaled=launch))
    return log, current


PW = w4.PackedWeight(Tensor((64,), torch.int32), Tensor((64,), torch.float16), Tensor((64,), torch.int32), 128, 64, 128)
X, S = Tensor((40, 128), torch.float16), Tensor((40,), torch.float32)
CALLS = [lambda **k: w4.gemm(X, PW, **k), lambda **k: w4.gemm_scaled(X, S, PW, **k)]


@pytest.mark.parametrize("call", CALLS)
def test_results_and_workspaces_belong_to_the_given_stream(seen, call):
    log, current = seen
    current["device"] = 1
    call(stream=Stream())
    assert {what for what, _, _ in log} == {"result", "size", "workspace", "launch"}
    assert all(stream == 0x77 for _, _, stream in log), log
    assert current["streams"][1] == 0x51
    log.clear()
    call()
    assert len(log) == 4 and all(stream == 0x51 for _, _, stream in log), log


@pytest.mark.parametrize("call", CALLS)
def test_a_stream_of_another_device_is_refused(seen, call):
    log, current = seen
    current["device"] = 1
    with pytest.raises(ValueError, match="stream is on cuda:0"):
        call(stream=Stream(torch.device("cuda", 0)))
    assert not [what for what, _, _ in log if what == "launch"]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("stream", [None, Stream()])
def test_the_tensors_device_is_the_current_one_for_the_call(seen, call, stream):
    log, current = seen
    call(stream=stream)
    assert log and all(device == 1 for _, device, _ in log), log
    assert current["device"] == 0
