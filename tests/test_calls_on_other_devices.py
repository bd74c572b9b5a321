"""Calls on tensors of a device that is not the current one (stand-ins, no GPU):
the C call runs with the tensors' device current, where its stream's launches
belong (the default streams of all devices share one handle), on that
device's stream, and a stream of another device is refused."""
import pytest

from tests.standins import Gpus, Stream, calls

NAMES = sorted(calls())


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("own,current", [(0, 0), (1, 0), (0, 1), (1, 1)])
def test_the_tensors_device_is_current(monkeypatch, name, own, current):
    gpus = Gpus(monkeypatch)
    gpus.dev = current
    side = Stream(own)
    calls(own)[name]()
    with gpus.stream(side):
        gpus.dev = current
        calls(own)[name]()
    calls(own)[name](stream=side)
    assert [dev for _, dev, _ in gpus.lib.calls] == [own] * 3
    assert [side.cuda_stream in args for _, _, args in gpus.lib.calls] == [False, True, True]
    assert all(t.device.index == own for t in gpus.made) and gpus.dev == current


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_device_is_refused(monkeypatch, name):
    gpus = Gpus(monkeypatch)
    with pytest.raises(ValueError):
        calls(0)[name](stream=Stream(1))
    assert not gpus.lib.calls
