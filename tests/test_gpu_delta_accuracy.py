"""How exact the gated delta rule's results are, on the GPU against the fp64
oracle: beyond the norms that test_gpu_delta.py bounds."""
import numpy as np
import pytest
import torch

import linear_attention_video_relu_b200 as la
from oracle import delta
from test_gpu_delta import args, make, put

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,N,D,Dv", [(4, 1024, 64, 64), (4, 1024, 128, 128), (3, 500, 112, 40),
                                      (80, 200, 64, 64), (40, 200, 128, 128)])
def test_outputs_are_those_of_an_fp32_computation(H, N, D, Dv):
    """Few heads (16 value columns to a chain) and many (32).

    Sums of up to 192 terms in fp32, each off by at most 2^-24 and of random
    signs, are off by sqrt(192) 2^-24 < 2^-20 of the tensor's root mean square.
    An error e before the rounding to bf16 changes the result in a share
    e / step of the elements, by a step (at most 2^-7 of the value, 2^-8 on
    average over mantissas and less where values are below the mean): a mean
    square of e step <= 2^-20 2^-8. So the 2-norm of the difference to the exact
    values' roundings is at most 2^-14 of theirs. (Operands of 17 bits, off by
    2^-17, would give 2^-12.)"""
    x, S0 = make(D + H, 1, H, H, N, D, Dv, torch.bfloat16)
    want, _ = delta.forward(scale=D ** -0.5, state=S0, **x)
    out, _ = la.delta_forward(*args(x, torch.bfloat16), state=put(S0, torch.float32))
    want = torch.from_numpy(want).to(torch.bfloat16).double().numpy()
    err = out.double().cpu().numpy() - want
    assert np.linalg.norm(err) <= 2.0 ** -14 * np.linalg.norm(want)


def decay_scales(x, S0, do, dS, scale):
    """|exp(log_decay_t) S_{t-1}| |dS_t| by token, the 2-norms of the two states
    whose product dlog_decay_t is (of value heads with keys of their own)."""
    states, n = [], np.zeros_like(x["log_decay"])
    delta.forward(scale=scale, state=S0, states=states, **x)
    G = np.array(dS)
    for t in reversed(range(n.shape[2])):
        k, q, b = (x[i][:, :, t] for i in ("k", "q", "beta"))
        a = np.exp(x["log_decay"][:, :, t])[..., None, None]
        G = G + scale * q[..., :, None] * do[:, :, t, None, :]
        G = G - b[..., None, None] * k[..., :, None] * (k[..., None, :] @ G)
        n[:, :, t] = (np.linalg.norm(a * states[t], axis=(-2, -1)) *
                      np.linalg.norm(G, axis=(-2, -1)))
        G = a * G
    return n


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("D,Dv,with_dstate", [(64, 32, True), (64, 96, False), (128, 128, True),
                                              (112, 40, False)])
def test_gradients_of_strong_decays_have_digits_of_their_own(dtype, D, Dv, with_dstate):
    """A decay that forgets nearly all has a gradient of that size. dlog_decay_t is
    the product of two states with exp(log_decay_t) in one of them; its sums are off
    by INNER (test_gpu_delta.py) of the states' norms, of which 8 times are allowed
    an element, and by the rounding."""
    N, H, scale = 200, 3, D ** -0.5
    inner = 2.0 ** -12 if dtype is torch.bfloat16 else 2.0 ** -16
    x, S0 = make(D + Dv, 1, H, H, N, D, Dv, dtype)
    r = np.random.default_rng(5)
    for t, g in ((3, -12.0), (15, -30.0), (16, -8.0), (40, -50.0), (63, -20.0), (64, -20.0),
                 (90, -60.0), (91, -2.0), (128, -60.0), (150, -16.0), (191, -40.0), (199, -40.0)):
        x["log_decay"][:, :, t] = g
    x["log_decay"][:, 2] = -np.float32(0.5) * r.integers(0, 20, (1, N))   # up to -9.5 everywhere

    def hold(a, dt):
        return torch.from_numpy(a).to(dt).double().numpy()

    do = hold(r.standard_normal((1, H, N, Dv)), dtype)
    dS = hold(r.standard_normal((1, H, D, Dv)), torch.float32)
    want = delta.backward(do, scale=scale, state=S0, dstate_out=dS, **x)[3]
    bound = decay_scales(x, S0, do, dS, scale)
    st = put(S0, torch.float32)
    if with_dstate:
        got = la.delta_backward(put(do, dtype), *args(x, dtype), state=st,
                                dstate_out=put(dS, torch.float32))[3]
    else:   # the initial state's gradient is not asked for (C ABI)
        C, t = la._native, args(x, dtype)
        out = [torch.empty_like(a) for a in t]
        p = la.api._delta_params(*t, None, "bhnd")
        ws = la.Workspace(C.lin_attn_delta_backward_workspace_size(p), "cuda")
        dot, dst = put(do, dtype), put(dS, torch.float32)
        C.check(C.lin_attn_delta_backward(p, dot.data_ptr(), *(a.data_ptr() for a in t),
                                          st.data_ptr(), dst.data_ptr(), None,
                                          *(a.data_ptr() for a in out), None, ws.ptr, ws.nbytes,
                                          torch.cuda.current_stream().cuda_stream), "backward")
        got = out[3]
    err = np.abs(got.double().cpu().numpy() - want)
    half = torch.finfo(dtype).eps / 2
    assert (err <= half * np.abs(want) + 8 * inner * bound).all()
