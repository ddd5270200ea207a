"""Workspaces that the package keeps for its callers, on stand-ins for the GPU: a call
under capture gets one of its own, since a graph's replays go on using its address
after the kept one has been replaced by a larger one."""
from __future__ import annotations

import contextlib
import types

import pytest

import sparse_linear_layers_02_amd as sbn
from sparse_linear_layers_02_amd import training


class Cuda:
    """Stand-in for torch, with host memory: one stream, under capture or not."""

    def __init__(self):
        import torch
        self.capturing = False
        self.uint8 = torch.uint8
        here = types.SimpleNamespace(cuda_stream=7)
        same = lambda *a, **k: contextlib.nullcontext()  # noqa: E731
        self.cuda = types.SimpleNamespace(device=same, stream=same, current_stream=lambda *a: here,
                                          is_current_stream_capturing=lambda: self.capturing)
        self._C = types.SimpleNamespace(_cuda_isCurrentStreamCapturing=lambda: self.capturing,
                                        _cuda_getDevice=lambda: 0, _cuda_getCurrentRawStream=lambda i: 7)

    def empty(self, n, dtype, device):
        import torch
        return torch.empty(n, dtype=dtype)


@pytest.fixture(params=["training", "layer"])
def scratch(request, monkeypatch):
    """(the stand-in, a function bytes -> workspace) of either part of the package."""
    import torch
    fake = Cuda()
    dev = torch.device("cuda", 0)
    monkeypatch.setattr(training, "_torch_module", fake)
    monkeypatch.setattr(sbn, "_torch", lambda: fake)
    if request.param == "training":
        return fake, lambda n: training._scratch("test", n, dev, 7)
    return fake, lambda n: sbn._workspace("test2", n, dev, None)


def test_a_captured_call_has_a_workspace_of_its_own(scratch):
    fake, get = scratch
    kept = get(1000)
    assert get(500) is kept                                        # eager calls share one
    fake.capturing = True
    first, second = get(600), get(600)
    assert first is not kept and second is not kept and first is not second
    assert first.numel() >= 600
    large = get(5000)
    fake.capturing = False
    assert get(1000) is kept and get(3000) is not large            # and what a graph got serves no eager call


def test_the_kept_workspace_grows(scratch):
    _, get = scratch
    a = get(300)
    b = get(4000)
    assert b is not a and b.numel() >= 4000 and get(4000) is b and get(20) is b


def test_threads_do_not_share_a_workspace(scratch):
    """A call is several launches, between which another thread may enqueue its own on the same stream."""
    import gc
    import threading
    import weakref
    _, get = scratch
    mine, seen, gone = get(1000), [], []

    def other():
        buf = get(1000)
        seen.append(buf is mine)
        seen.append(get(800) is buf)
        gone.append(weakref.ref(buf))

    t = threading.Thread(target=other)
    t.start()
    t.join()
    assert seen == [False, True] and get(1000) is mine
    del t
    gc.collect()
    assert gone[0]() is None                                       # a thread's workspaces end with it
