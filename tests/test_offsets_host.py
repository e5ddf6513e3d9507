"""Positions and sizes that no 32-bit int holds are refused, not cut off to one
that another call could have meant."""
import pytest
import torch

import linear_attention_video_relu_b200 as la


@pytest.mark.parametrize("call", [la.rotary, la.rotary_backward])
@pytest.mark.parametrize("bad", [
    dict(offset=2 ** 32 + 5), dict(offset=2 ** 31), dict(offset=-2 ** 31 - 1), dict(dim=2 ** 32 + 16),
    dict(grid=(2 ** 32 + 2, 2, 2), rope_split=(16, 24, 24)),
    dict(grid=(2, 2, 2), rope_split=(16, 24, 2 ** 32 + 24))], ids=str)
def test_values_past_32_bits(call, bad):
    with pytest.raises(ValueError, match="32-bit"):
        call(torch.zeros(1, 2, 8, 64), **bad)


@pytest.mark.parametrize("bad", [2 ** 32 + 5, 2 ** 31])
def test_block_offsets_past_32_bits(bad):
    st = object.__new__(la.BlockState)   # refused before anything of it is read
    x = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="32-bit"):
        st.step(x, x, x, t_offset=bad)
    with pytest.raises(ValueError, match="32-bit"):
        st.update(x, x, t_offset=bad)
