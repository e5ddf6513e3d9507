"""Calls that are given a stream: what they make (results, and a workspace whose
control block has to be zero) and where they work is that stream's. What the
current stream still has to do cannot reach into it, and memory that a call is
done with on the host is not handed to the current stream."""
import pytest
import torch

import linear_attention_video_relu_b200 as la

pytestmark = pytest.mark.gpu


def _inputs(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _attention(s, **kw):
    q, k, v, g = (_inputs(i, 1, 4, 1000, 64) for i in range(4))
    if kw.pop("fp32", False):
        q, k, v, g = (t.float() for t in (q, k, v, g))
    return lambda: la.forward(q, k, v, g, stream=s, **kw)


def _cross(s):
    q, k, v = (_inputs(i, 1, 4, n, 64) for i, n in enumerate((1000, 300, 300)))
    return lambda: la.cross_forward(q, k, v, stream=s)


def _conv(s):
    x, w = _inputs(5, 1, 6, 40, 64), torch.ones(3, 64, device="cuda")
    return lambda: la.temporal_conv(x, w, stream=s)


CALLS = {
    "forward": _attention,
    "block_causal": lambda s: _attention(s, mode="block_causal", block_tokens=100),
    "token_causal": lambda s: _attention(s, mode="token_causal"),
    "fp32": lambda s: _attention(s, fp32=True),
    "cross": _cross,
    "temporal_conv": _conv,
}


def _junk(value):
    """Every small block of the current stream's pool, filled on that stream."""
    return [torch.full((n,), value, device="cuda") for n in (1 << 12, 1 << 16, 1 << 20)
            for _ in range(20)]


@pytest.mark.parametrize("name", CALLS)
def test_a_call_on_another_stream_is_that_streams_altogether(name):
    want = CALLS[name](None)()
    side = torch.cuda.Stream()
    call = CALLS[name](side)
    torch.cuda.synchronize()
    call()   # its allocations first: new memory from the driver may wait for the device
    junk = _junk(float("nan"))
    del junk
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)   # a fifth of a second
    got = call()
    junk = _junk(float("nan"))
    torch.cuda.synchronize()
    assert torch.equal(got, want) and len(junk) == 60


def test_block_steps_on_another_stream():
    """The state's workspace is made by its first step, on that step's stream."""
    parts = [[_inputs(10 * i + j, 1, 4, 96, 64) for j in range(3)] for i in range(2)]

    def steps(st, stream):
        outs = [st.step(*p, stream=stream) for p in parts]
        st.update(parts[0][1], parts[0][2], stream=stream)
        return outs + [st.S, st.z]

    want = steps(la.BlockState(1, 4, 64), None)
    side = torch.cuda.Stream()
    first, second = la.BlockState(1, 4, 64), la.BlockState(1, 4, 64)
    torch.cuda.synchronize()
    steps(first, side)
    junk = _junk(float("nan"))
    del junk
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)
    got = steps(second, side)
    junk = _junk(float("nan"))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and len(junk) == 60


def test_a_stream_of_another_device_is_refused():
    class Other:   # what the check looks at
        device = torch.device("cuda", torch.cuda.device_count())
        cuda_stream = 0

    q = _inputs(0, 1, 2, 64, 64)
    x = _inputs(1, 1, 2, 8, 64)
    for call in (lambda: la.forward(q, q, q, stream=Other), lambda: la.cross_forward(q, q, q, stream=Other),
                 lambda: la.temporal_conv(x, torch.ones(3, 64, device="cuda"), stream=Other)):
        with pytest.raises(ValueError, match="stream"):
            call()
