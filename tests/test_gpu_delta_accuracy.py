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
