"""The C ABI's checks of parts of larger buffers, on the CPU."""

from __future__ import annotations

import pytest

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
