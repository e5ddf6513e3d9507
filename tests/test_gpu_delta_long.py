"""The gated delta rule over long sequences and far into large tensors, against
the fp64 oracle. Tolerances as in test_gpu_delta.py: a chunk's errors are of
random signs from chunk to chunk, and what later writes replace of the state they
replace of its error, so that both grow alike with the number of chunks."""
import numpy as np
import pytest
import torch

import linear_attention_video_relu_b200 as la
from oracle import delta
from test_gpu_delta import DT, INNER, args, check, first, make, put

pytestmark = pytest.mark.gpu

NAMES = ("dq", "dk", "dv", "dlog_decay", "dbeta")


@pytest.mark.parametrize("dt,H,Hk,N,D,Dv", [("bf16", 2, 1, 4100, 64, 64), ("bf16", 2, 2, 3001, 128, 128),
                                            ("bf16", 1, 1, 3500, 112, 40), ("fp32", 1, 1, 2500, 64, 72)])
def test_thousands_of_tokens(dt, H, Hk, N, D, Dv):
    """Log decays near 0, so that what is written stays for the whole sequence
    unless another write replaces it: with the initial state's gradient and,
    by chains of fewer bits in bf16, without."""
    dtype, scale = DT[dt], D ** -0.5
    x, S0 = make(N, 1, H, Hk, N, D, Dv, dtype, decay=0.002)
    r = np.random.default_rng(1)
    do = torch.from_numpy(r.standard_normal((1, H, N, Dv))).to(dtype).double().numpy()
    want = delta.forward(scale=scale, state=S0, **x)
    grad = delta.backward(do, scale=scale, state=S0, **x)
    t, st = args(x, dtype), put(S0, torch.float32)
    out, S1 = la.delta_forward(*t, state=st)
    check(out, want[0], INNER[dtype], "out")
    check(S1, want[1], INNER[torch.float32], "state")
    got = la.delta_backward(put(do, dtype), *t, state=st)
    for name, g, w in zip(NAMES, got, grad):
        check(g, w, INNER[dtype], name)
    check(got[5], grad[5], INNER[torch.float32], "dstate")
    # and from no initial state
    grad = delta.backward(do, scale=scale, **x)
    for name, g, w in zip(NAMES, la.delta_backward(put(do, dtype), *t), grad):
        check(g, w, INNER[dtype], name)


@pytest.mark.parametrize("layout,Hk", [("bhnd", 140), ("bnhd", 70)])
def test_gradients_past_32_bits(layout, Hk):
    """The last tokens of the last head of tensors of more than 2^31 elements
    (heads of their own) or bytes, after a reset; zeros before them. The
    workspace's images, records and shared heads' parts lie further on still."""
    B, H, N, D, Dv, n, dtype = 1, 140, 128 * 1024, 128, 64, 130, torch.bfloat16
    x, _ = make(12, 1, 1, 1, n, D, Dv, dtype, state=False)
    x["log_decay"][:, :, 0] = -100.0

    def far(heads, a):
        t = torch.zeros((B, heads, N) + a.shape[3:] if layout == "bhnd" else
                        (B, N, heads) + a.shape[3:], device="cuda", dtype=dtype)
        first(t, layout)[0, heads - 1, N - n:] = put(a, dtype)[0, 0]
        return t

    do = np.random.default_rng(9).standard_normal((1, 1, n, Dv))
    do = torch.from_numpy(do).to(dtype).double().numpy()
    t = [far(Hk, x["q"]), far(Hk, x["k"]), far(H, x["v"]), far(H, x["log_decay"]), far(H, x["beta"])]
    assert t[0].numel() > 2 ** 31 or 2 * t[0].numel() > 2 ** 31 and layout == "bnhd"
    want = delta.forward(scale=D ** -0.5, **x)
    out, S = la.delta_forward(*t, layout=layout)
    check(first(out, layout)[:, H - 1:, N - n:], want[0], INNER[dtype], "out")
    check(S[:, H - 1:], want[1], INNER[torch.float32], "state")
    assert not first(out, layout)[0, :H - 1].any() and not S[0, :H - 1].any()
    del out, S
    got = la.delta_backward(far(H, do), *t, layout=layout)
    for name, g, w in zip(NAMES, got, delta.backward(do, scale=D ** -0.5, **x)):
        g = first(g, layout)
        check(g[:, -1:, N - n:], w, INNER[dtype], name)
        assert not g[0, :-1].any() and not g[0, -1, :N - n].any(), name
