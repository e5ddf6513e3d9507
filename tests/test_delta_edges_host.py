"""Refusals of the delta rule's calls that test_delta_rotary_host.py leaves out,
through the C ABI with fake device addresses that no rejected call touches."""
import pytest

import __graft_entry__
from linear_attention_video_relu_b200 import _native as C
from test_delta_rotary_host import DK, DQ, K, LEN, Q, _backward, _delta, _forward


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()


def test_gradients_without_value_heads():
    """dq and dk are written all the same, so they are checked."""
    p = _delta(H=0, Hk=2)
    for bad in (dict(dq=None), dict(dk=None), dict(dq=DQ + 8), dict(dk=DK + 2), dict(dq=Q), dict(dk=K),
                dict(dk=DQ), dict(dq=LEN), dict(lengths=LEN + 2)):
        assert _backward(p, **bad) == C.LA_ERR_INVALID_ARG, bad
    assert _backward(_delta(H=0, Hk=0)) == C.LA_OK
    assert _backward(_delta(H=0, Hk=2, N=0), dq=None) == C.LA_OK
    assert _backward(_delta(B=0), dq=None) == C.LA_OK
    assert _forward(p) == C.LA_OK
