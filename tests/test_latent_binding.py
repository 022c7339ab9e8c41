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


def _plan(batch):
    return api.paged_latent_decode_plan([20] * batch, num_heads=8, page_size=16, max_pages_per_seq=4,
                                        num_pages=8, scale=0.1, latent_dim=256, num_sms=8, host_only=True)


def _tables(table):
    z = torch.zeros(table.shape[0], dtype=torch.int32)
    return api.paged_kv_tables(z, z.clone(), torch.zeros(3, dtype=torch.int32),
                               torch.zeros(1, dtype=torch.int32), table, page_size=16, num_slots=2)


def _decode(table):
    q, pages = torch.zeros((table.shape[0], 8, 320), dtype=BF), torch.zeros((8, 16, 320), dtype=BF)
    return api.paged_latent_decode_run(_plan(table.shape[0]), q, pages, table)


BASE = torch.zeros(40, dtype=torch.int32)


@pytest.mark.parametrize("call,at", [(_tables, 8), (_decode, 7)])
@pytest.mark.parametrize("rows,stride,given", [
    (3, 0, 0), (3, 2, 2),              # rows over one another: as they are, for the library to refuse
    (3, 4, 4), (3, 9, 9),
    (1, 0, 4), (1, 1, 4), (1, 9, 9),   # of one row the stride says nothing
])
def test_table_rows_keep_their_stride(streams, monkeypatch, call, at, rows, stride, given):
    plan = _plan(rows)
    r = Recorder()
    table = BASE.as_strided((rows, 4), (stride, 1))
    monkeypatch.setattr(api, "paged_latent_decode_plan", lambda *a, **k: plan)
    with monkeypatch.context() as m:
        m.setattr(L, "lib", lambda: r)
        call(table)
    (name, args), = r.calls
    assert args[at] == given


def test_tables_over_one_another_are_refused(streams):
    """By the library, before anything is launched: two requests would write one row."""
    for table in (BASE[:4].expand(3, 4), BASE.as_strided((3, 4), (2, 1))):
        with pytest.raises(L.PkaError, match="row stride") as e:
            _tables(table)
        assert e.value.code == L.PKA_ERR_INVALID_ARG
