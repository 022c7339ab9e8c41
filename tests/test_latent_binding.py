"""What the latent entry points hand to the library, without a GPU: CPU tensors stand in for
the current device's, and a recorder for the library."""
import contextlib

import pytest
import torch

from paged_kv_attention_32_gb300 import _lib as L
from paged_kv_attention_32_gb300 import api

BF = torch.bfloat16


class Recorder:
    """Any entry point: keeps its arguments and succeeds."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


class Streams:
    """The current stream's raw handle, as torch keeps it."""

    def __init__(self):
        self.now = 11

    @contextlib.contextmanager
    def on(self, stream):
        before, self.now = self.now, int(stream)
        try:
            yield
        finally:
            self.now = before


@pytest.fixture
def streams(monkeypatch):
    s = Streams()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)   # a CPU tensor's get_device()
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: s.now, raising=False)
    monkeypatch.setattr(api, "_on_stream", s.on)
    return s


@pytest.fixture
def library(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(L, "lib", lambda: r)
    return r


@pytest.mark.parametrize("stream,handle", [(None, 11), (77, 77), (0, 0)])
def test_append_is_queued_on_the_given_stream(streams, library, stream, handle):
    rows, pages = torch.zeros((3, 64), dtype=BF), torch.zeros((2, 8, 64), dtype=BF)
    got = api.paged_latent_append(rows[:, :56], rows[:, 56:], torch.arange(3), pages, stream=stream)
    assert got is pages
    (name, args), = library.calls
    assert name == "paged_latent_append" and args[-1] == handle
    assert streams.now == 11


@pytest.mark.parametrize("given,made", [(0, "default"), (99, "external 99")])
def test_raw_handles_become_the_stream_they_name(monkeypatch, given, made):
    """0 is the default stream's handle; torch makes a stream of its own of it."""
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: "default")
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h: f"external {h}")
    monkeypatch.setattr(torch.cuda, "stream", lambda s: s)
    assert api._on_stream(given) == made
