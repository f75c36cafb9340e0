"""Which GPU and stream the binding launches on, with the library and the GPU stubbed: the arguments'
GPU and its current stream, whichever GPU is the current one."""
import contextlib

import pytest
import torch

import mixture_experts_layer_logits_amd as m


class Stub:
    """As much of a GPU tensor as the binding looks at."""
    is_cuda = True

    def __init__(self, device, n=0, dtype=torch.float32):
        self.device_, self.n, self.dtype, self.shape = device, n, dtype, (n,)

    def get_device(self):
        return self.device_

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096

    def numel(self):
        return self.n

    def element_size(self):
        return self.dtype.itemsize


@pytest.fixture
def calls(monkeypatch):
    """(entry point, current GPU, stream) of each launch; GPU 0 is the current one outside."""
    log, current = [], [0]

    class Lib:
        def __getattr__(self, name):
            def entry(*args):
                log.append((name, current[-1], args[-1]))
                return 0
            return entry

    @contextlib.contextmanager
    def device(d):
        current.append(d)
        yield
        current.pop()

    class Stream:
        @property
        def cuda_stream(self):
            return 100 + current[-1]

    monkeypatch.setattr(m, "_lib", Lib())
    monkeypatch.setattr(m, "_device", lambda: current[-1])
    monkeypatch.setattr(m, "_raw_stream", lambda d: 100 + d)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream())
    return log


S = m.make_shape(4, 64, 64, 8, 2, m.MOE_F32)


def _launch_each(dev, stream=None):
    t = lambda n=0, dtype=torch.float32: Stub(dev, n, dtype)  # noqa: E731
    i32 = torch.int32
    m.moe_combine(S, t(), t(), t(), None, t(), stream=stream)
    m.moe_route(S, t(), t(), t(), t(), t(), t(), t(64, torch.uint8), stream=stream)
    m.moe_mx_quantize(4, 64, 0, None, 0, t(), t(), t(), stream=stream)
    m.moe_balance_bwd(S, t(32), t(4), t(9, i32), t(2), None, None, None, t(32), stream=stream)


NAMES = ["moe_combine", "moe_route", "moe_mx_quantize", "moe_balance_bwd"]


@pytest.mark.parametrize("dev", [0, 1, 3])
def test_launches_go_to_the_arguments_gpu(calls, dev):
    _launch_each(dev)
    assert calls == [(n, dev, 100 + dev) for n in NAMES]


@pytest.mark.parametrize("dev", [0, 1])
def test_a_given_stream_is_used_on_the_arguments_gpu(calls, dev):
    _launch_each(dev, stream=77)
    assert calls == [(n, dev, 77) for n in NAMES]


def test_raw_pointers_run_on_the_current_gpu(calls):
    m.moe_combine(S, 4096, 4096, 4096, None, 4096)
    m.moe_combine(S, 4096, 4096, 4096, None, 4096, stream=77)
    assert calls == [("moe_combine", 0, 100), ("moe_combine", 0, 77)]
