"""Which device and stream a call of the binding allocates and launches on, with the
runtime's queries replaced: tensors on device 1 while device 0 is current."""
import contextlib
import types

import pytest
import torch

import precision_weight_quantization_amd as lpq


@pytest.fixture
def runtime(monkeypatch):
    log = types.SimpleNamespace(current=0, external=[], streams=[])

    @contextlib.contextmanager
    def device(index):
        before, log.current = log.current, index
        try:
            yield
        finally:
            log.current = before

    @contextlib.contextmanager
    def stream(s):
        log.streams.append(s)
        yield

    def external(handle, device=None):
        log.external.append((handle, device))
        return ("external", handle)

    monkeypatch.setattr(torch.cuda, "current_device", lambda: log.current)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 1000 + index, raising=False)
    return log


def like(index):
    return types.SimpleNamespace(device=torch.device("cuda", index))


@pytest.mark.parametrize("index", [0, 1])
@pytest.mark.parametrize("stream,want", [(None, None), (77, 77), (0, 0)])
def test_launch(runtime, index, stream, want):
    calls = []

    def fn(*args):
        calls.append((runtime.current, args))
        return 0

    lpq._launch(fn, "fn", like(index), stream, 5)
    assert calls == [(index, (5, 1000 + index if want is None else want))]
    assert runtime.current == 0


@pytest.mark.parametrize("index", [0, 1])
def test_launch_restores_the_device_behind_an_error(runtime, index):
    with pytest.raises(lpq.LpqError):
        lpq._launch(lambda *a: 1, "fn", like(index), None)
    assert runtime.current == 0


@pytest.mark.parametrize("handle", [0, 77])
def test_a_handle_is_a_stream_of_the_tensors_device(runtime, handle):
    with lpq._on(handle, like(1)):
        pass
    assert runtime.external == [(handle, torch.device("cuda", 1))]
    assert runtime.streams == [("external", handle)]


def test_no_stream_means_the_current_one(runtime):
    with lpq._on(None, like(1)):
        pass
    assert runtime.streams == []
