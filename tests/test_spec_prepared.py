"""Prepared calls of the speculative step used by several threads, on the CPU:
a stand-in for the library's function records which stream each call is given."""
import threading
import time
import types

import pytest
import torch

from gated_deltanet_recurrent_sigmoid_b200 import binding, speculative as spec
from test_spec_abi import make_commit, make_maps


@pytest.fixture(scope="module", autouse=True)
def _lib(gdn_lib):
    return spec.load()


@pytest.mark.parametrize("cls,make", [(spec.PreparedCommitStates, make_commit), (spec.PreparedStepMaps, make_maps)])
def test_one_object_on_two_threads_streams(cls, make, monkeypatch):
    here, seen = threading.local(), []

    def recorded(*args):
        """The library's function, which runs without the interpreter's lock."""
        if cls is spec.PreparedStepMaps:
            extra = spec.GdnStepMapsCall.from_address(args[0].value).extra.contents
        else:
            extra = binding.GdnExtra.from_address(args[-1].value)
        time.sleep(0.0005)
        seen.append((here.stream, extra.stream))
        return binding.OK

    real = spec.load()
    name = {spec.PreparedCommitStates: "gdn_commit_states", spec.PreparedStepMaps: "gdn_step_maps"}[cls]
    lib = types.SimpleNamespace(untyped=types.SimpleNamespace(**{name: recorded}), **{name: getattr(real, name)})
    monkeypatch.setattr(spec, "_LIB", lib)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: here.stream, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    call = cls.__new__(cls)
    with pytest.raises(ValueError):                      # host tensors
        call.__init__(**make()[1])
    call._device = 0
    call._ready()

    def run(streams):
        for k in range(40):
            here.stream = streams[k % len(streams)]
            call()

    threads = [threading.Thread(target=run, args=(s,)) for s in ((0x1000,), (0x2000, 0x3000))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(seen) == 80 and all(own == given for own, given in seen)


def test_streams_that_come_and_go(monkeypatch):
    """What is kept for a stream does not grow without bound."""
    streams, seen = [], []
    real = spec.load()
    lib = types.SimpleNamespace(
        untyped=types.SimpleNamespace(gdn_commit_states=lambda *args: seen.append(binding.GdnExtra.from_address(args[-1].value).stream) or 0),
        gdn_commit_states=real.gdn_commit_states)
    monkeypatch.setattr(spec, "_LIB", lib)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: streams[-1], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    call = spec.PreparedCommitStates.__new__(spec.PreparedCommitStates)
    with pytest.raises(ValueError):
        call.__init__(**make_commit()[1])
    call._device = 0
    call._ready()
    for k in range(1000):
        streams.append(0x1000 + 64 * k)
        call()
    assert seen == streams and len(call._by_stream) <= 64
