"""What a call that is given a stream makes, it makes with that stream current:
seen on the host, with stand-ins for the library's entries, for the tensors'
device and for torch's stream context."""
import contextlib

import pytest
import torch

from linear_attention_video_relu_b200 import _native as C
from linear_attention_video_relu_b200 import api

SIDE = object()


@pytest.fixture
def seen(monkeypatch):
    """Records, for every allocation and every launch, the stream current then."""
    log, current = [], []

    @contextlib.contextmanager
    def on_stream(t, stream=None, makes=True):
        current.append(stream)
        yield
        current.pop()

    def entry(*a):
        log.append(("launch", current[-1] if current else None))
        return C.LA_OK

    def make(f, what):
        def g(*a, **k):
            log.append((what, current[-1] if current else None))
            return f(*a, **k)
        return g

    monkeypatch.setattr(api, "_on_stream", on_stream)
    monkeypatch.setattr(api, "_on_device", on_stream)
    monkeypatch.setattr(api, "_check_io", lambda *a, **k: None)
    monkeypatch.setattr(api, "_same_device", lambda *a: None)
    monkeypatch.setattr(api, "_stream", lambda *a: 0)
    monkeypatch.setattr(torch, "empty_like", make(torch.empty_like, "result"))
    monkeypatch.setattr(api, "Workspace", make(lambda n, dev: type("W", (), {
        "ptr": 0, "nbytes": n, "buf": torch.zeros(1)})(), "workspace"))
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    for f in ("lin_attn_forward", "lin_attn_cross_forward", "lin_attn_block_step",
              "lin_attn_state_update"):
        monkeypatch.setattr(C, f, entry)
    for f in ("lin_attn_workspace_size", "lin_attn_block_step_workspace_size",
              "lin_attn_cross_workspace_size"):
        monkeypatch.setattr(C, f, lambda *a: 256)
    return log


def _state():
    st = object.__new__(api.BlockState)
    st.S, st._st, st._ws, st._plans = torch.zeros(1), None, {}, {}
    return st


CALLS = {
    "forward": (lambda q: api.forward(q, q, q, stream=SIDE), 3),
    "cross_forward": (lambda q: api.cross_forward(q, q, q, stream=SIDE), 3),
    "step": (lambda q: _state().step(q, q, q, stream=SIDE), 3),
    "update": (lambda q: _state().update(q, q, stream=SIDE), 2),
}


@pytest.mark.parametrize("name", CALLS)
def test_made_on_the_calls_stream(seen, name):
    call, n = CALLS[name]
    call(torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16))
    assert len(seen) == n and all(s is SIDE for _, s in seen), seen
