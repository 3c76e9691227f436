"""What the Python calls hand to the library, without a GPU: the library, the streams and the current device
are stand-ins, and the tensors are host tensors that say they are on a device."""

from __future__ import annotations

import contextlib

import pytest
import torch

import sparse_latent_attention_gb300 as sa

DEV = 1  # the device that the tensors say they are on


class OnDevice(torch.Tensor):
    """A host tensor that says it is on device DEV."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", DEV))

    def get_device(self):
        return DEV


def on_device(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)


class Stream:
    cuda_stream = 77


@pytest.fixture
def calls(monkeypatch):
    """The library's calls as (name, current device, stream argument), and the streams that outputs were
    asked for on; device 0 is the current one."""
    log = {"calls": [], "new": []}
    now = [0]

    class Library:
        def __getattr__(self, name):
            def f(*args):
                log["calls"].append((name, now[0], args[-1]))
                return 1 << 20 if name == "sa_sparse_attn_workspace_size" else 0
            return f

    @contextlib.contextmanager
    def device(d):
        before, now[0] = now[0], d if isinstance(d, int) else torch.device(d).index
        yield
        now[0] = before

    def new(stream, make):
        log["new"].append(stream)
        with monkeypatch.context() as m:  # what it makes is a host tensor
            for name in ("empty", "zeros"):
                m.setattr(torch, name, lambda *shape, _f=getattr(torch, name), **kw:
                          _f(*shape, **{**kw, "device": "cpu"}).as_subclass(OnDevice))
            return make()

    monkeypatch.setattr(sa, "load", Library)
    monkeypatch.setattr(sa, "_raw_stream", lambda d: 1000 + d)
    monkeypatch.setattr(sa, "_new", new)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    return log


bf16, i32, u8 = torch.bfloat16, torch.int32, torch.uint8

MAKE_OUTPUTS = {
    "hc_split_sinkhorn": lambda st: sa.hc_split_sinkhorn(on_device(3, 24), on_device(3), on_device(24), stream=st),
    "candidate_blocks": lambda st: sa.candidate_blocks(on_device(1, 8, 2), 0, 4, 1, 1, stream=st),
    "indexer_topk": lambda st: sa.indexer_topk(on_device(1, 8, 2), 0, 4, 2, 0, stream=st),
    "window_idxs": lambda st: sa.window_idxs(0, 8, 4, stream=st),
}


@pytest.mark.parametrize("name", MAKE_OUTPUTS)
def test_outputs_come_from_the_given_stream(calls, name):
    st = Stream()
    MAKE_OUTPUTS[name](st)
    assert [c[2] for c in calls["calls"]] == [77]
    assert calls["new"] and all(s is st for s in calls["new"])
