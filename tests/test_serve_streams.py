"""Allocations of a packed call on a named stream belong to that stream on the
tensors' device, which need not be the current one (host logic, no GPU)."""
import contextlib

import torch

from gated_delta_rule_117_b200 import kda


def test_a_handle_is_taken_on_the_tensors_device(monkeypatch):
    kda._torch or kda._init()
    made, entered = [], []

    class External:
        cuda_stream = 77

        def __init__(self, handle, device=None):
            made.append((handle, device))

    @contextlib.contextmanager
    def on(stream):
        entered.append(stream)
        yield

    monkeypatch.setattr(torch.cuda, "ExternalStream", External)
    monkeypatch.setattr(torch.cuda, "stream", on)
    assert kda._fresh(1234, 3, lambda n: n + 1, 5) == 6
    assert made == [(1234, 3)] and isinstance(entered[0], External)
    named = External(9, device=2)  # a stream object brings its device with it
    assert kda._fresh(named, 2, lambda: "t") == "t" and entered[1] is named and len(made) == 2
    assert kda._fresh(None, 3, lambda: "t") == "t" and len(entered) == 2  # the current stream: nothing to enter
