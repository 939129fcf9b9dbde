"""What the operators' bindings do around the library calls, without a GPU: the
library is replaced by one that accepts everything, and tensors by host tensors
that note the stream whose pool they came from."""
import contextlib

import pytest
import torch

from context_attention_long_b200 import _native, api

CURRENT, OTHER = "current stream", "other stream"


class Library:
    """Accepts every call; sizes of workspaces are small numbers."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 64 if name.endswith("_bytes") else 0
        return call


class Stream:
    cuda_stream = 5

    def __init__(self, name):
        self.name = name

    def __eq__(self, other):
        return self.name == other.name


class Host(torch.Tensor):
    """A host tensor that the bindings take for a device tensor; `made`
    collects what is allocated from it, with the pool it came from."""
    made, active = [], [CURRENT]

    def new_empty(self, shape, dtype=None):
        t = torch.empty(shape, dtype=dtype or self.dtype).as_subclass(Host)
        t.pool, t.recorded = Host.active[-1], []
        Host.made.append(t)
        return t

    def record_stream(self, stream):
        self.recorded.append(stream.name)


@pytest.fixture()
def host(monkeypatch):
    lib = Library()

    @contextlib.contextmanager
    def on(stream):
        Host.active.append(stream.name)
        yield
        Host.active.pop()

    def address(t, *_):
        return None if t is None else t.data_ptr()
    monkeypatch.setattr(_native, "load", lambda: lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *_: Stream(Host.active[-1]))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(api, "_view", lambda t, *_: (address(t), None))
    monkeypatch.setattr(api, "_plain", address)
    monkeypatch.setattr(api, "_ptr", address)
    monkeypatch.setattr(api, "_raw_stream", lambda stream, device: 0)
    monkeypatch.setattr(Host, "made", [])
    monkeypatch.setattr(Host, "active", [CURRENT])
    return lib


def _host(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(Host)


def _calls(stream):
    q, k = _host(2, 3, 4, 64), _host(2, 5, 2, 64)
    t, w = _host(2, 3, 2, 64), _host(64, dtype=torch.float32)
    lse = _host(2, 4, 3, dtype=torch.float32)
    return [lambda: api.cpattn_qk_norm_rope(q, t, w, w, stream=stream),
            lambda: api.cpattn_qk_norm_rope_backward(q, t, q, t, w, w, stream=stream),
            lambda: api.cpattn_cross_attention(q, k, k, stream=stream),
            lambda: api.cpattn_cross_attention_backward(q, k, k, q, lse, q, stream=stream)]


@pytest.mark.parametrize("i", range(4))
@pytest.mark.parametrize("stream", [None, Stream(CURRENT), Stream(OTHER)])
def test_allocations_come_from_the_pool_of_the_launch_stream(host, i, stream):
    returned = _calls(stream)[i]()
    pool = CURRENT if stream is None else stream.name
    assert Host.made and all(t.pool == pool for t in Host.made)
    # what the caller reads on the current stream is noted as used there
    for t in Host.made:
        seen = any(t is r for r in returned)
        assert t.recorded == ([CURRENT] if pool == OTHER and seen else [])


MB = 1 << 20


@pytest.mark.parametrize("pair,free,idle,ds_budget,pairs", [
    (200 * MB, 100 << 30, 0, None, 4),          # all there is
    (200 * MB, 1000 * MB, 0, None, 2),          # within half of what is free
    (200 * MB, 300 * MB, 0, None, 1),           # half is less than what is always taken: 256 MB, one pair
    (200 * MB, 300 * MB, 650 * MB, None, 3),    # or than what torch holds unused
    (200 * MB, None, 800 * MB, None, 4),        # which is enough: the device is not asked
    (200 * MB, None, 0, 800 * MB, 4),           # the caller's own budget
    (200 * MB, None, 0, 0, 1),
    (64 * MB, None, None, None, 4),             # 256 MB in all
])
def test_scratch_of_the_cross_backward_leaves_free_memory(host, monkeypatch, pair, free, idle, ds_budget, pairs):
    def mem_get_info(device):
        assert free is not None
        return free, 180 << 30

    def stats(device):
        assert idle is not None
        return {"reserved_bytes": {"all": {"current": 7 * MB + idle}}, "allocated_bytes": {"all": {"current": 7 * MB}}}
    monkeypatch.setattr(torch.cuda, "mem_get_info", mem_get_info)
    monkeypatch.setattr(torch.cuda, "memory_stats_as_nested_dict", stats)
    monkeypatch.setattr(api, "cpattn_cross_attention_backward_ds_bytes", lambda *_: pair)
    monkeypatch.setattr(api, "cpattn_cross_attention_backward_workspace_bytes", lambda *_: 1000 + pair)
    q, k, lse = _host(2, 3, 4, 64), _host(2, 5, 2, 64), _host(2, 4, 3, dtype=torch.float32)
    api.cpattn_cross_attention_backward(q, k, k, q, lse, q, ds_budget=ds_budget)
    assert [t.numel() for t in Host.made if t.dtype is torch.uint8] == [1000 + pairs * pair]
