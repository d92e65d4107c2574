"""Every call of the binding runs with its tensors' device as the current one: a default
stream's handle is the same on every device, and a launch on it goes to the current
device. Without a GPU: the queries of torch that say which device is current are replaced."""
import contextlib
import inspect
import re

import pytest
import torch

import bit_quantized_matmul_col_amd as lm


class On:
    """A tensor, as far as _launch looks at it."""

    def __init__(self, index):
        self.index = index

    def get_device(self):
        return self.index


@pytest.fixture
def devices(monkeypatch):
    state = {"current": 0}

    @contextlib.contextmanager
    def device(index):
        before, state["current"] = state["current"], index
        try:
            yield
        finally:
            state["current"] = before
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state["current"])
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 1000 + index)
    monkeypatch.setattr(torch.cuda, "device", device)
    return state


@pytest.mark.parametrize("index", [0, 1])
def test_a_call_runs_on_the_device_of_its_tensors(devices, index):
    seen = []

    def call(*args):
        seen.append((devices["current"], args))
        return lm.LLMINT8_OK
    lm._launch(call, On(index), 7, 8)
    lm._launch(call, On(index), 7, opts=(9,))
    assert seen == [(index, (7, 8, 1000 + index)), (index, (7, 1000 + index, 9))]
    assert devices["current"] == 0


@pytest.mark.parametrize("index", [0, 1])
def test_errors_are_raised_and_leave_the_device(devices, index, built_library):
    with pytest.raises(lm.Llmint8Error) as e:
        lm._launch(lambda *args: lm.LLMINT8_ERR_WORKSPACE, On(index))
    assert e.value.status == lm.LLMINT8_ERR_WORKSPACE and devices["current"] == 0


def test_every_call_goes_that_way():
    source = inspect.getsource(lm)
    calls = set(re.findall(r"_launch\((?:lib\(\)|L)\.(\w+)", source))
    assert calls == {n for n in re.findall(r"def (llmint8_\w+)\(", source)
                     if not n.endswith("_workspace_size")} - {"llmint8_status_string"} | {
                         "llmint8_linear_ex"}
    assert not re.search(r"_check\((?:lib\(\)|L)\.", source)
