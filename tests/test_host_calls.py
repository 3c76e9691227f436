"""What the Python calls hand to the library, without a GPU: the library, the streams and the current device
are stand-ins, and the tensors are host tensors that say they are on a device."""

from __future__ import annotations

import contextlib
import os
import subprocess
import sys

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


def _attn(**more):
    return sa.sparse_attn(on_device(1, 2, 4, 64, dtype=bf16), on_device(1, 8, 64, dtype=bf16), on_device(4),
                          on_device(1, 2, 4, dtype=i32), 0.1, **more)


ROT = (on_device(16, 8, 2), 3)
CALLS = {
    "sa_sparse_attn": lambda: _attn(),
    "sa_sparse_attn_family": lambda: _attn(family="mma"),
    "sa_sparse_attn_rope": lambda: _attn(rope=ROT),
    "sa_sparse_attn_lse": lambda: _attn(lse=on_device(1, 2, 4)),
    "sa_hc_split_sinkhorn": lambda: MAKE_OUTPUTS["hc_split_sinkhorn"](None),
    "sa_candidate_blocks": lambda: MAKE_OUTPUTS["candidate_blocks"](None),
    "sa_indexer_topk": lambda: MAKE_OUTPUTS["indexer_topk"](None),
    "sa_window_idxs": lambda: sa.window_idxs(0, 8, 4, out=on_device(8, 4, dtype=i32)),
    "sa_act_quant_fp8": lambda: sa.act_quant_fp8(on_device(2, 64, dtype=bf16), codes=on_device(2, 64, dtype=u8)),
    "sa_window_write": lambda: sa.window_write(on_device(1, 2, 64, dtype=bf16), 0,
                                               codes=on_device(1, 8, 64, dtype=u8)),
    "sa_act_quant_fp4": lambda: sa.act_quant_fp4(on_device(2, 64, dtype=bf16), codes=on_device(2, 32, dtype=u8)),
    "sa_window_write_fp4": lambda: sa.window_write_fp4(on_device(1, 2, 64, dtype=bf16), 0,
                                                       codes=on_device(1, 8, 32, dtype=u8)),
    "sa_row_weights": lambda: sa.row_weights(
        on_device(1, 2, 4, 64, dtype=bf16), on_device(1, 8, 64, dtype=bf16), on_device(1, 2, 4),
        on_device(1, 2, 4, dtype=i32), 0.1, on_device(1, 8, dtype=torch.int64)),
    "sa_evict_select": lambda: sa.evict_select(on_device(1, 8, dtype=torch.int64), 4),
    "sa_compact_rows": lambda: sa.compact_rows([on_device(1, 8)], on_device(1, 4, dtype=i32)),
    "sa_remap_idx": lambda: sa.remap_idx(on_device(1, 4, dtype=i32), on_device(1, 8, dtype=i32)),
    "sa_read_status": lambda: sa.read_status(on_device(256, dtype=u8)),
}


@pytest.mark.parametrize("name", CALLS)
def test_calls_run_on_their_tensors_device(calls, name):
    """With another device current: that of the tensors is current for the call, on its own stream."""
    CALLS[name]()
    assert [c for c in calls["calls"] if c[0] != "sa_sparse_attn_workspace_size"] == [(name, DEV, 1000 + DEV)]
    assert torch.cuda.current_device() == 0


def test_status_of_a_host_tensor_is_refused():
    with pytest.raises(TypeError):
        sa.read_status(torch.zeros(256, dtype=u8))


ELSEWHERE = {
    "candidate_blocks out": lambda: sa.candidate_blocks(on_device(1, 8, 2), 0, 4, 1, 1,
                                                        out=torch.zeros(1, 8, 2, dtype=torch.bool)),
    "indexer_topk candidates": lambda: sa.indexer_topk(on_device(1, 8, 2), 0, 4, 2, 0,
                                                       candidates=torch.zeros(1, 8, 2, dtype=torch.bool)),
    "act_quant_fp8 out_rt": lambda: sa.act_quant_fp8(on_device(2, 64, dtype=bf16),
                                                     out_rt=torch.zeros(2, 64, dtype=bf16)),
    "act_quant_fp8 codes": lambda: sa.act_quant_fp8(on_device(2, 64, dtype=bf16),
                                                    codes=torch.zeros(2, 64, dtype=u8)),
    "act_quant_fp8 scales": lambda: sa.act_quant_fp8(on_device(2, 64, dtype=bf16),
                                                     scales=torch.zeros(2, 2, dtype=u8)),
    "window_write ring_rt": lambda: sa.window_write(on_device(1, 2, 64, dtype=bf16), 0,
                                                    ring_rt=torch.zeros(1, 8, 64, dtype=bf16)),
    "window_write codes": lambda: sa.window_write(on_device(1, 2, 64, dtype=bf16), 0,
                                                  codes=torch.zeros(1, 8, 64, dtype=u8)),
    "window_write scales": lambda: sa.window_write(on_device(1, 2, 64, dtype=bf16), 0,
                                                   scales=torch.zeros(1, 8, 2, dtype=u8)),
}


@pytest.mark.parametrize("name", ELSEWHERE)
def test_tensors_elsewhere_are_refused(calls, name):
    """A tensor that is not on the call's device, a host tensor here: its address never reaches a kernel."""
    with pytest.raises(ValueError):
        ELSEWHERE[name]()
    assert not calls["calls"]


def test_imports_with_a_pytorch_without_cuda():
    code = ("import torch\ndel torch._C._cuda_getCurrentRawStream\n"
            "import sparse_latent_attention_gb300 as sa\nassert sa.workspace_size and sa.WEIGHT_UNIT")
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                          cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert done.returncode == 0, done.stderr


def test_an_empty_rotation_table(calls):
    """None of the positions: fine where there are no tokens, refused where there are some."""
    rope = (on_device(0, 8, 2), 0)
    for lse in (None, on_device(1, 0, 4)):
        o = sa.sparse_attn(on_device(1, 0, 4, 512, dtype=bf16), on_device(1, 8, 512, dtype=bf16), on_device(4),
                           on_device(1, 0, 4, dtype=i32), 0.1, rope=rope, lse=lse,
                           out=on_device(1, 0, 4, 512, dtype=bf16))
        assert o.shape == (1, 0, 4, 512)
    with pytest.raises(ValueError):
        _attn(rope=rope, lse=on_device(1, 2, 4))
