"""The workspace of calls made without one, on the CPU: who shares it, when it is replaced, and what a
capture gets. CPU tensors stand for the device's, a variable for the current stream."""
import threading

import pytest
import torch


@pytest.fixture
def m(monkeypatch):
    from nvfp4_mixture_experts_02_gb300 import ftmoe
    state = dict(stream=5, capturing=False, made=[])
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: state["stream"], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: state["capturing"], raising=False)

    def make(n, dev, head=True):
        ws = torch.zeros(n, dtype=torch.uint8)
        state["made"].append((n, head))
        return ws

    monkeypatch.setattr(ftmoe, "_new_scratch", make)
    ftmoe.state = state
    yield ftmoe
    del ftmoe.state
    ftmoe._KEPT.by_stream.clear()


def in_thread(fn):
    got = []
    t = threading.Thread(target=lambda: got.append(fn()))
    t.start()
    t.join()
    return got[0]


def test_one_per_stream_and_thread(m):
    a = m._scratch(100, 0)
    assert m._scratch(100, 0) is a and m._scratch(50, 0) is a and m._scratch(70, 0, True) is a
    other = in_thread(lambda: m._scratch(100, 0))
    assert other is not a and m._scratch(100, 0) is a
    m.state["stream"] = 6
    assert m._scratch(100, 0) is not a
    assert m.state["made"] == [(100, True)] * 3


def test_it_grows_and_keeps_its_flags(m):
    a = m._scratch(100, 0)
    a[0], a[90] = 4, 9
    b = m._scratch(101, 0)
    assert b is not a and b.numel() == 101 and b[0] == 4 and not b[1:].any()
    assert m._scratch(100, 0) is b


def test_a_capture_has_its_own(m):
    a = m._scratch(100, 0)
    m.state["capturing"] = True
    b, c = m._scratch(100, 0), m._scratch(100, 0, True)
    assert a is not b and b is not c and a is not c
    assert m.state["made"][1:] == [(100, False), (100, True)]   # the layer's counters are zeroed in the graph
    assert m._scratch(200, 0).numel() == 200
    m.state["capturing"] = False
    assert m._scratch(100, 0) is a                              # nothing of the capture is kept, nothing replaced
