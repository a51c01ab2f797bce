"""How the binding reads and checks its arguments for the grouped router and
block-scaled e4m3 (host only; no GPU needed)."""
import pytest
import torch

import moe_layer_topk_amd as moe


@pytest.mark.parametrize("E,N,K", [(4, 512, 256), (1, 512, 256), (3, 256, 256), (16, 512, 128)])
@pytest.mark.parametrize("shape", ["E11", "1E1", "11E"])
def test_one_scale_an_expert_in_three_dimensions(E, N, K, shape):
    """What amax(dim=(1, 2), keepdim=True) gives is still one scale per expert."""
    w = torch.zeros(E, N, K, dtype=torch.float8_e4m3fn)
    s = torch.ones({"E11": (E, 1, 1), "1E1": (1, E, 1), "11E": (1, 1, E)}[shape])
    assert moe._layer_dtype(w, s) == moe.MOE_FP8_E4M3
    assert moe._layer_dtype(w, s.view(E)) == moe.MOE_FP8_E4M3


@pytest.mark.parametrize("E,N,K", [(4, 512, 256), (1, 512, 128), (8, 128, 128), (1, 128, 128), (2, 128, 256)])
def test_block_scales(E, N, K):
    w = torch.zeros(E, N, K, dtype=torch.float8_e4m3fn)
    assert moe._layer_dtype(w, torch.ones(E, N // 128, K // 128)) == moe.MOE_FP8_BLOCK
    assert moe._layer_dtype(w, torch.ones(E, N // 128 + 2, K // 128)) == moe.MOE_FP8_BLOCK  # (refused by its shape later)
