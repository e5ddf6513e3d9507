"""The gated delta rule's calls that the other tests leave out: no value heads,
workspaces' status, long offsets."""
import pytest
import torch

import linear_attention_video_relu_b200 as la

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["bhnd", "bnhd"])
@pytest.mark.parametrize("lengths", [None, [5, 70, -1]], ids=["whole", "ragged"])
def test_gradients_without_value_heads(dtype, layout, lengths):
    """Keys that no value head reads have gradients of zero."""
    B, Hk, N, D = 3, 2, 70, 40
    shape = (lambda h, w: (B, h, N, w)) if layout == "bhnd" else (lambda h, w: (B, N, h, w))
    q = torch.randn(shape(Hk, D), device="cuda").to(dtype)
    v = torch.empty(shape(0, 16), device="cuda", dtype=dtype)
    g = v[..., 0]
    ln = None if lengths is None else torch.tensor(lengths, device="cuda", dtype=torch.int32)
    junk = [torch.full_like(q, float("nan")) for _ in range(4)]
    del junk
    for a in la.delta_backward(v, q, q, v, g, g, lengths=ln, layout=layout)[:2]:
        assert a.shape == q.shape and not a.any()
    out = [torch.full_like(t, 7.0) for t in (q, q, v, g, g)]
    la.delta_backward(v, q, q, v, g, g, lengths=ln, layout=layout, out=out)
    live = torch.arange(N, device="cuda") < (N if ln is None else ln[:, None])
    live = live.expand(B, N)[:, None, :, None] if layout == "bhnd" else live.expand(B, N)[:, :, None, None]
    for a in out[:2]:
        assert torch.equal(a, torch.where(live, 0.0, 7.0).to(dtype).expand_as(a))
