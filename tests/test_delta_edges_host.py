"""Refusals of the delta rule's calls that test_delta_rotary_host.py leaves out,
through the C ABI with fake device addresses that no rejected call touches."""
import pytest

import __graft_entry__
from linear_attention_video_relu_b200 import _native as C
from test_delta_rotary_host import DK, DQ, G, K, LEN, O, Q, S0, S1, V, _backward, _delta, _forward


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


BLOCK = C.LA_WORKSPACE_CONTROL_BYTES


@pytest.mark.parametrize("other", [Q, K, V, G, S0, O, S1, LEN])
def test_the_flag_word_of_a_workspace_that_is_not_needed(other):
    """It is written all the same, so it may lie in nothing else."""
    p = _delta(N=1)
    assert C.lin_attn_delta_workspace_size(p) == 0
    assert _forward(p, workspace=other, workspace_bytes=BLOCK) == C.LA_ERR_INVALID_ARG


def test_the_flag_word_of_calls_without_tokens_or_value_heads():
    for ws in (S0, S1):
        assert _forward(_delta(N=0), workspace=ws, workspace_bytes=BLOCK) == C.LA_ERR_INVALID_ARG
        assert _backward(_delta(N=0), dstate_out=S0, workspace=ws,
                         workspace_bytes=BLOCK) == C.LA_ERR_INVALID_ARG
    for ws in (Q, K, DQ, DK, LEN):
        assert _backward(_delta(H=0, Hk=2), workspace=ws,
                         workspace_bytes=BLOCK) == C.LA_ERR_INVALID_ARG
