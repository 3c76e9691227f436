"""The 4-bit quantiser on enough rows for two groups a thread (2048 groups of eight an SM): bit-exact."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import sparse_latent_attention_gb300 as sa
from tests import _cache, _gpu
from tests.test_gpu_cache import _rows, dev  # noqa: F401 (dev is a fixture)

pytestmark = pytest.mark.gpu

GROUPS = 160 * 2048  # at least as many as any GPU that the library runs on calls for


# d / 8 groups a row divide the block's 128 threads, or do not, or are more of them
@pytest.mark.parametrize("n,d,stride", [(5201, 512, 512), (27501, 96, 104), (13901, 192, 192), (2101, 1280, 1288),
                                        (82001, 32, 32)])
def test_act_quant_fp4_of_many_rows(dev, n, d, stride):  # noqa: F811
    assert n * (d // 8) >= GROUPS and n * (d // 8) % 256  # (the last block is not full)
    bits = _rows(np.random.default_rng(n), n, d)
    want_c, want_s, want_v = _cache.quantise(bits)
    x = torch.full((n + 1, stride), 7.0, dtype=torch.bfloat16, device=dev)
    x[:n, :d] = _gpu.u16_to_bf16_tensor(bits, dev)
    codes = torch.full((n + 1, d // 2), 0xAB, dtype=torch.uint8, device=dev)
    scales = torch.full((n + 1, d // 32), 0x55, dtype=torch.uint8, device=dev)
    sa.act_quant_fp4(x[:n, :d], out_rt=x[:n, :d], codes=codes[:n], scales=scales[:n])
    assert (codes[:n].cpu().numpy() == want_c).all() and (scales[:n].cpu().numpy() == want_s).all()
    got = x[:n, :d].double().cpu().numpy()
    assert np.array_equal(got, want_v) and np.array_equal(np.signbit(got), np.signbit(want_v))
    assert (codes[n] == 0xAB).all() and (scales[n] == 0x55).all()
    assert (x[n] == 7.0).all() and (x[:, d:] == 7.0).all()


@pytest.mark.parametrize("nb,seqlen,start,window,rows,d", [(41, 128, 77, 128, 140, 512), (40, 800, 0, 701, 705, 96),
                                                           (5, 1000, 12, 600, 600, 1280)])
def test_window_write_fp4_of_many_rows(dev, nb, seqlen, start, window, rows, d):  # noqa: F811
    assert nb * min(seqlen, window) * (d // 8) >= GROUPS
    bits = _rows(np.random.default_rng(nb), nb * seqlen, d)
    codes, scales, values = (a.reshape(nb, seqlen, -1) for a in _cache.quantise(bits))
    want_c = np.full((nb, rows, d // 2), 0xAB, np.uint8)
    want_s = np.full((nb, rows, d // 32), 0x55, np.uint8)
    want_v = np.full((nb, rows, d), 7.0)
    for t in range(seqlen):
        slot = (start + t) % window
        want_c[:, slot], want_s[:, slot], want_v[:, slot] = codes[:, t], scales[:, t], values[:, t]
    c = torch.full((nb, rows, d // 2), 0xAB, dtype=torch.uint8, device=dev)
    s = torch.full((nb, rows, d // 32), 0x55, dtype=torch.uint8, device=dev)
    rt = torch.full((nb, rows, d), 7.0, dtype=torch.bfloat16, device=dev)
    x = _gpu.u16_to_bf16_tensor(bits, dev).view(nb, seqlen, d)
    sa.window_write_fp4(x, start, codes=c[:, :window], scales=s[:, :window], ring_rt=rt[:, :window])
    assert (c.cpu().numpy() == want_c).all() and (s.cpu().numpy() == want_s).all()
    assert np.array_equal(rt.double().cpu().numpy(), want_v)
