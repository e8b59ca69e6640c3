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


def small(**options):
    return V.Sizes(hidden=272, heads=4, kv_heads=2, head_dim=64, vocab=1000, page_tokens=16, slots=3, rank=16, top=4, **options)


def tensors(o, at="step"):
    """(where, tensor) of everything that an object holds."""
    if isinstance(o, torch.Tensor):
        yield at, o
    elif isinstance(o, dict):
        for k, v in o.items():
            yield from tensors(v, f"{at}[{k!r}]")
    elif isinstance(o, (list, tuple)):
        for i, v in enumerate(o):
            yield from tensors(v, f"{at}[{i}]")
    elif type(o).__module__.startswith("adapter_lora_bgmv_amd") and hasattr(o, "__dict__"):
        for k, v in vars(o).items():
            yield from tensors(v, f"{at}.{k}")


def test_a_step_with_all_options_lies_on_its_device(monkeypatch):
    """Here the CPU, with the quantisation of the weights left out; no array goes to the default GPU."""
    monkeypatch.setattr(V.VerifyStep, "_quantize", staticmethod(lambda *a, **k: None))
    step = V.VerifyStep(small(base8=True, theta=10000.0, sample=True), n_seqs=2, draft=3, max_tokens=32, device="cpu")
    found = dict(tensors(step))
    assert {"step.w_qkv8[0]", "step.x8[1]", "step.rotary.inv_freq", "step.uniform"} <= set(found)
    assert all(t.device.type == "cpu" for t in found.values())


def test_next_tokens_take_numbers_and_other_steps_none():
    """No step draws with the numbers of the one before: run refuses a missing
    argument, and one that nothing would use, before it does anything."""
    log = Log()
    for options, uniform in ((dict(sample=True), None), ({}, np.zeros(6))):
        step = V.VerifyStep(small(**options), n_seqs=2, draft=3, max_tokens=32, device="cpu")
        step.ids, step.seqs = Record(log, "ids"), type("Seqs", (), {"kv_len": Record(log, "kv_len")})
        step.parts = lambda x, stream: {"call": lambda: log.append("call")}
        with pytest.raises(ValueError, match="uniform"):
            step.run(None, [3, 4], np.arange(6), stream=77, uniform=uniform)
    assert log == []


def test_a_step_holds_its_base_weights_once(monkeypatch):
    """As codes or in 16 bits, not both."""
    monkeypatch.setattr(V.VerifyStep, "_quantize", staticmethod(lambda *a, **k: None))
    for base8, size in ((False, 2), (True, 1)):
        step = V.VerifyStep(small(base8=base8), n_seqs=2, draft=3, max_tokens=32, device="cpu")
        for shape in ((step.row, step.s.hidden), (step.s.vocab, step.q_dim)):
            held = [t.element_size() for _, t in tensors(step) if tuple(t.shape) == shape]
            assert held == [size], (base8, shape, held)
