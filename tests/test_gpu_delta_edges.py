"""The gated delta rule's calls that the other tests leave out: no value heads,
workspaces' status, long offsets."""
import os
import shutil
import subprocess

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


def _inputs(B, H, N, D=64, dtype=torch.bfloat16):
    q = torch.nn.functional.normalize(torch.randn(B, H, N, D, device="cuda"), dim=-1).to(dtype)
    g = torch.zeros(B, H, N, device="cuda", dtype=dtype)
    return q, q, q, g - 0.5, g + 0.5


@pytest.mark.parametrize("flag", [-1, 8], ids=["junk", "set"])
def test_a_status_is_that_of_the_last_call(flag):
    """Whatever the flag word holds before, and whether the call needs a workspace."""
    OK = la._native.LA_OK
    few, many, chunks = _inputs(1, 2, 1), _inputs(16, 16, 20), _inputs(1, 2, 100)
    S = torch.randn(1, 2, 64, 64, device="cuda")
    nothing = [t[:, :, :0] for t in few]
    no_heads = [few[0], few[1]] + [t[:, :0] for t in few[2:]]
    p = la.api._delta_params(*chunks, None, "bhnd")
    ws = la.Workspace(la._native.lin_attn_delta_backward_workspace_size(p), "cuda")
    for call in (lambda: la.delta_forward(*few, workspace=ws), lambda: la.delta_forward(*many, workspace=ws),
                 lambda: la.delta_forward(*chunks, workspace=ws),
                 lambda: la.delta_forward(*nothing, state=S, workspace=ws),
                 lambda: la.delta_forward(*nothing, workspace=ws),
                 lambda: la.delta_backward(torch.ones_like(chunks[2]), *chunks, workspace=ws),
                 lambda: la.delta_backward(torch.ones_like(few[2]), *few, workspace=ws),
                 lambda: la.delta_backward(nothing[2], *nothing, state=S, dstate_out=S, workspace=ws),
                 lambda: la.delta_backward(no_heads[2], *no_heads, workspace=ws)):
        ws.buf.view(torch.int32)[:] = flag
        call()
        assert ws.status() == OK


def test_a_workspace_without_a_control_block_is_left_alone():
    ws = la.Workspace(256, "cuda")
    ws.buf.fill_(255)
    la.delta_forward(*_inputs(1, 2, 1), workspace=ws)
    assert (ws.buf == 255).all()


@pytest.mark.skipif(shutil.which("nvcc") is None, reason="needs nvcc")
def test_a_wait_that_nothing_ends_gives_up(tmp_path):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = str(tmp_path / "wait_check")
    subprocess.check_call(["nvcc", "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "-O2",
                           "--expt-relaxed-constexpr", "-I",
                           os.path.join(root, "linear_attention_video_relu_b200", "csrc"), "-I",
                           os.path.join(root, "include"),
                           os.path.join(root, "tests", "c", "wait_check.cu"), "-o", exe])
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout + r.stderr
