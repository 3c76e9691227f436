"""Calls on a stream of their own: where their outputs come from."""

from __future__ import annotations

import pytest
import torch

import sparse_latent_attention_gb300 as sa
from tests.test_gpu_cache import dev  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("call", ["hc_split_sinkhorn", "candidate_blocks", "indexer_topk", "window_idxs"])
def test_outputs_of_a_call_on_another_stream(dev, call):  # noqa: F811
    """A call on a stream of its own does not write into memory that the current stream still reads."""
    g = torch.Generator(device=dev).manual_seed(3)
    mixes = torch.randn(70000, 24, device=dev, generator=g)
    hc_scale, hc_base = torch.ones(3, device=dev), torch.randn(24, device=dev, generator=g)
    score = torch.randn(1, 4096, 1024, device=dev, generator=g)
    run = {"hc_split_sinkhorn": lambda st: sa.hc_split_sinkhorn(mixes, hc_scale, hc_base, stream=st),
           "candidate_blocks": lambda st: [sa.candidate_blocks(score, 0, 4, 64, 8, stream=st)],
           "indexer_topk": lambda st: [sa.indexer_topk(score, 0, 4, 512, 128, stream=st)],
           "window_idxs": lambda st: [sa.window_idxs(0, 4096, 128, stream=st)]}[call]
    want = [t.clone() for t in run(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    nbytes = want[-1].numel() * want[-1].element_size()
    old, copy = (torch.full((nbytes,), 7, dtype=torch.uint8, device=dev) for _ in range(2))
    copy.zero_()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # some 50 ms
    copy.copy_(old)
    del old
    got = run(side)
    side.synchronize()
    torch.cuda.synchronize()
    assert (copy == 7).all()
    assert all(torch.equal(g_, w) for g_, w in zip(got, want))
