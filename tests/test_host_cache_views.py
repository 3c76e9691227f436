"""The C ABI's checks of parts of larger buffers, on the CPU."""

from __future__ import annotations

import pytest

from sparse_latent_attention_gb300._lib import SA_ERR_CUDA as CUDA
from tests.test_host_cache import INVALID, WORKSPACE, at, lib  # noqa: F401 (lib is a fixture)


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("d,offset,code", [
    (64, 2, WORKSPACE), (64, 1, INVALID), (192, 6, WORKSPACE), (448, 14, WORKSPACE), (320, 5, INVALID),
    (128, 4, WORKSPACE), (128, 2, INVALID), (384, 12, WORKSPACE), (256, 8, WORKSPACE), (512, 16, WORKSPACE),
    (512, 8, INVALID)])
def test_row_weights_scales_of_a_later_sequence(lib, fmt, d, offset, code):  # noqa: F811
    """kv_scale where a sequence of a packed cache with an odd number of rows puts it (nothing else is
    wrong with the call but its missing workspace)."""
    a = dict(q=at(1), kv=at(2), kv_scale=at(9, offset), fmt=fmt, lse=at(3), idx=at(4), scale=0.1, b=1, s=2, h=64,
             d=d, rows=8, topk=4, acc=at(6), ws=None, ws_bytes=0)
    assert lib.sa_row_weights(*a.values(), None) == code


N = 1 << 37  # rows: more blocks than a grid has, so a call whose arguments are right launches nothing


@pytest.mark.parametrize("change,code", [
    # codes and scales of a row side by side: 32 + 2 bytes, 40 apart
    (dict(codes=at(5120), cs=40, scales=at(5120, 32), ss=40), CUDA),
    (dict(codes=at(5120, 8), cs=40, scales=at(5120, 6), ss=40), CUDA),             # the scales in front
    (dict(codes=at(5120), cs=40, scales=at(5120, 31), ss=40), INVALID),            # in the codes' last byte
    (dict(codes=at(5120), cs=40, scales=at(5120, 39), ss=40), INVALID),            # into the next row's codes
    (dict(codes=at(5120), cs=40, scales=at(5120, 32), ss=42), INVALID),            # other distances
    (dict(codes=at(5120), cs=40, scales=at(5120, 32 + 40 * (N - 1)), ss=40), CUDA),    # from the last row's side on
    (dict(codes=at(5120), cs=40, scales=at(5120, 31 + 40 * (N - 1)), ss=40), INVALID),
    (dict(codes=at(5120), cs=40, scales=at(5120, 40 * (N - 1) + 32), ss=2), CUDA),     # right behind them
    (dict(codes=at(5120), cs=40, scales=at(5120, 40 * (N - 1) + 31), ss=2), INVALID),
    # x, its round trip, codes and scales of a row in 320 bytes
    (dict(xs=160, rt=at(1024, 128), rts=160, codes=at(1024, 256), cs=320, scales=at(1024, 288), ss=320), CUDA),
    (dict(xs=160, rt=at(1024, 126), rts=160, codes=at(1024, 256), cs=320, scales=at(1024, 288), ss=320), INVALID),
    (dict(xs=160, rt=at(1024, 128), rts=160, codes=at(1024, 252), cs=320, scales=at(1024, 288), ss=320), INVALID),
    (dict(xs=160, rt=at(1024, 128), rts=160, codes=at(1024, 256), cs=320, scales=at(1024, 319), ss=320), INVALID),
    (dict(xs=160, rt=at(1024, 128), rts=168, codes=None, scales=None), INVALID),
    (dict(rt=at(1024), codes=None, scales=None), CUDA),                            # in place
])
def test_act_quant_fp4_rows_between_one_another(lib, change, code):  # noqa: F811
    a = dict(x=at(1024), n=N, d=64, xs=64, rt=at(2048), rts=64, codes=at(5120), cs=32, scales=at(4096), ss=2)
    a.update(change)
    assert lib.sa_act_quant_fp4(*a.values(), None) == code
