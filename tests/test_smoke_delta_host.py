"""The delta rule's part of smoke() on the CPU, through stand-ins for the CUDA
calls (the oracle, rounded to bf16 like the GPU's results), as test_smoke_host.py
does for the rest. It checks the harness, not the kernels."""
import types

import numpy as np
import pytest
import torch

import __graft_entry__
from oracle import delta, rotary


def _f64(t):
    return t.float().numpy().astype(np.float64)


def _bf16(x):
    return torch.from_numpy(np.asarray(x)).to(torch.bfloat16)


def _stand_in(calls, wrong=None):
    names = ("q", "k", "v", "log_decay", "beta")

    def turn(x, offset, dim, style, back):
        pos = np.arange(offset, offset + x.shape[2])[None]
        return _bf16(rotary.rotate(_f64(x), pos, dim, style, transpose=back))

    def f(name, back):
        def call(q, k, *, offset, dim, style):
            calls.append(name)
            return tuple(turn(x, offset, dim, style, back) for x in (q, k))
        return call

    class State:
        def __init__(self, B, H, D, device):
            self.S = torch.zeros(B, H, D, D)

        def step(self, *t):
            calls.append("step")
            out, S = delta.forward(scale=t[0].shape[-1] ** -0.5, state=self.S.numpy(),
                                   **dict(zip(names, map(_f64, t))))
            self.S = torch.from_numpy(S).float()
            return _bf16(out)

    def backward(do, *t):
        calls.append("backward")
        r = [_bf16(x) for x in delta.backward(_f64(do), scale=t[0].shape[-1] ** -0.5,
                                              **dict(zip(names, map(_f64, t))))[:5]]
        if wrong is not None:
            r[wrong] = r[wrong] * 1.02
        return tuple(r) + (None,)

    return types.SimpleNamespace(rotary=f("rotary", False), rotary_backward=f("rotary_backward", True),
                                 DeltaState=State, delta_backward=backward)


def test_smoke_logic_with_stand_ins(capsys):
    calls = []
    __graft_entry__._smoke_delta(torch.device("cpu"), _stand_in(calls), lambda: None)
    assert calls == ["rotary", "step", "step", "backward", "rotary_backward"]
    out = capsys.readouterr().out
    for name in ("rotary q", "delta_forward", "delta state", "delta_backward dbeta",
                 "rotary_backward dk"):
        assert "smoke %s ok" % name in out


@pytest.mark.parametrize("wrong", range(5))
def test_a_gradient_that_is_off_is_seen(wrong):
    with pytest.raises(AssertionError, match="delta_backward"):
        __graft_entry__._smoke_delta(torch.device("cpu"), _stand_in([], wrong), lambda: None)
