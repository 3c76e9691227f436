"""Two host threads that call at the same time, each on a stream of its own."""

from __future__ import annotations

import threading

import pytest
import torch

import sparse_latent_attention_gb300 as sa
from tests.test_gpu_cache import dev  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu

ROUNDS = 400


def at_once(calls):
    """Runs each of the calls (of a stream, returning a tensor) ROUNDS times in a thread of its own, and
    returns what went wrong: errors, and results that differ from the thread's first."""
    wrong = []

    def work(call):
        try:
            st = torch.cuda.Stream()
            first = None
            with torch.cuda.stream(st):
                start.wait()
                for _ in range(ROUNDS):
                    got = call()
                    first = got if first is None else first
                    last = got
                st.synchronize()
                if not torch.equal(first, last):
                    wrong.append("results differ")
        except Exception as e:  # noqa: BLE001 (reported by the caller)
            wrong.append(e)

    start = threading.Barrier(len(calls))
    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return wrong


def test_evict_select_of_two_sizes_at_once(dev):  # noqa: F811
    """Rows that take 33 KB of shared memory, and rows that take 160 KB of one CTA's."""
    g = torch.Generator(device=dev).manual_seed(1)
    small = torch.randint(0, 1 << 40, (1, 8320), device=dev, generator=g)
    large = torch.randint(0, 1 << 40, (160, 40000), device=dev, generator=g)
    assert not at_once([lambda: sa.evict_select(small, 4000)[0], lambda: sa.evict_select(large, 20000)[0]])


def test_indexer_topk_of_two_sizes_at_once(dev):  # noqa: F811
    """Rows that take 52 KB of shared memory, and rows that take 192 KB."""
    g = torch.Generator(device=dev).manual_seed(2)
    small = torch.randn(4, 1, 13000, device=dev, generator=g)
    large = torch.randn(4, 1, 49152, device=dev, generator=g)
    assert not at_once([lambda: sa.indexer_topk(small, 4 * 13000 - 1, 4, 512, 0),
                        lambda: sa.indexer_topk(large, 4 * 49152 - 1, 4, 512, 0)])
