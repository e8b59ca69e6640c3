"""The verify step's ordering and the binding's shared state, without a GPU."""
import contextlib
import importlib.util
import sys
import threading

import numpy as np
import pytest

from adapter_lora_bgmv_amd import binding as B
from adapter_lora_bgmv_amd import verify_step as V

torch = pytest.importorskip("torch")


class Record:
    """In the place of a device array: which stream its copies were made on."""

    def __init__(self, log, name):
        self.log, self.name = log, name

    def copy_(self, _):
        self.log.append((self.name, self.log.stream))


class Log(list):
    stream = "current"


@pytest.mark.parametrize("handle", [None, 77, 0])  # a torch stream, and raw handles: 0 is the default stream
def test_inputs_are_copied_on_the_stream_of_the_kernels(monkeypatch, handle):
    """Lengths and ids may be rewritten only behind the kernels of the step
    before, which read them on the caller's stream."""
    log = Log()

    class Stream:
        def __init__(self, handle=77):
            self.cuda_stream = handle

    @contextlib.contextmanager
    def on(stream):
        log.stream = stream.cuda_stream
        yield
        log.stream = "current"

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: Stream(0))
    step = V.VerifyStep.__new__(V.VerifyStep)
    step.ids, step.scores = Record(log, "ids"), {}
    step.seqs = type("Seqs", (), {"kv_len": Record(log, "kv_len")})
    step.parts = lambda x, stream: {"call": lambda: log.append(("call", getattr(stream, "cuda_stream", stream)))}
    step.run(None, [3, 4], np.arange(2), Stream() if handle is None else handle)
    want = 77 if handle is None else handle
    assert log == [("kv_len", want), ("ids", want), ("call", want)]


def test_first_stream_lookup_from_two_threads(monkeypatch):
    """Two threads held together between finding no lookup and setting it: both
    get the stream, and so does every later call."""
    fresh = importlib.util.module_from_spec(B.__spec__)
    B.__spec__.loader.exec_module(fresh)  # a binding whose lookup is not made yet
    together = threading.Barrier(2, timeout=20)
    waits = threading.local()

    class Torch:
        """torch, where reading it for the lookup first waits for the other thread."""

        def __getattr__(self, name):
            if not getattr(waits, "done", False):
                waits.done = True
                together.wait()
            return getattr(torch, name)

    monkeypatch.setitem(sys.modules, "torch", Torch())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 100 + device, raising=False)
    got = []
    threads = [threading.Thread(target=lambda: got.append(fresh._stream(None))) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(30)
    assert got == [103, 103] and fresh._stream(None) == 103
