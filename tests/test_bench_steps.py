"""The timed steps of the bench and the interpreter's garbage collection (stand-ins for the GPU)."""

from __future__ import annotations

import gc

import pytest

import bench


class Event:
    def __init__(self, enable_timing):
        pass

    def record(self):
        pass

    def elapsed_time(self, other):
        return 1.0


class Torch:
    class cuda:
        Event = Event
        _sleep = staticmethod(lambda cycles: None)
        synchronize = staticmethod(lambda: None)


class Flush:
    def zero_(self):
        pass


@pytest.mark.parametrize("fails", [False, True])
@pytest.mark.parametrize("enabled", [True, False])
def test_no_collection_in_or_before_the_timed_steps(fails, enabled):
    seen, collections = [], []

    class Path:
        def step(self, ev=None):
            seen.append(gc.isenabled())
            if fails:
                raise RuntimeError("step")

    def note(phase, info):
        collections.append(phase)

    was = gc.isenabled()
    gc.collect()
    (gc.enable if enabled else gc.disable)()
    gc.callbacks.append(note)
    try:
        if fails:
            with pytest.raises(RuntimeError):
                bench.time_device_steps(Torch, Path(), Flush(), 3, 0)
        else:
            assert bench.time_device_steps(Torch, Path(), Flush(), 3, 0) == ([1.0] * 3, [1.0] * 3)
        assert gc.isenabled() is enabled
    finally:
        gc.callbacks.remove(note)
        (gc.enable if was else gc.disable)()
    assert seen == [False] * (1 if fails else 3)
    assert not collections
