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


class OnDevice(torch.Tensor):
    """A host tensor that says it is on a GPU: only its address is asked for."""
    is_cuda = True


def on_device(t):
    return t.as_subclass(OnDevice)


def test_routing_reads_the_bias_it_has():
    a, b = on_device(torch.zeros(8)), on_device(torch.ones(8))
    r = moe.Routing(bias=a)
    r._check(8, a.device)
    assert r.args.bias == a.data_ptr()
    r.bias = b  # another tensor
    r._check(8, b.device)
    assert r.args.bias == b.data_ptr() and r.bias is b
    b.set_(torch.ones(8))  # the same tensor with another storage
    r._check(8, b.device)
    assert r.args.bias == b.data_ptr()
    r.bias = None
    r._check(8, b.device)
    assert r.args.bias is None and r.bias is None


def test_routing_refuses_a_bias_it_cannot_read():
    r = moe.Routing()
    with pytest.raises(ValueError, match="CPU"):
        r.bias = torch.zeros(8)
    with pytest.raises(ValueError, match="float32"):
        r.bias = on_device(torch.zeros(8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="contiguous"):
        r.bias = on_device(torch.zeros(16))[::2]
    assert r.bias is None
    r.bias = on_device(torch.zeros(8))
    with pytest.raises(ValueError, match="bias"):
        r._check(16, r.bias.device)
    r.bias.resize_(4)
    with pytest.raises(ValueError, match="bias"):
        r._check(8, r.bias.device)
    assert (moe.Routing("sigmoid", r.bias, 4, 2, 2, False, 2.5).args.n_groups == 4)
