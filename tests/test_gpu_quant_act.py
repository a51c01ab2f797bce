"""Codes of moe_quant_act against IEEE float32 quotients on the CPU, bit for bit,
from the smallest scales to the largest: values on, and up to two float32 steps
beside, every border between two codes."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_layer_topk_amd as moe
    moe.lib()
    return torch.device("cuda:0")


@pytest.mark.parametrize("exp", [-149, -140, -127, -126, -123, -120, -115, -110, -104, -100, -90, -81, -80, -79, -64, 0, 64, 118])
def test_borders(dev, exp):
    import moe_layer_topk_amd as moe
    g = torch.Generator().manual_seed(exp + 200)
    codes = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    mid = (codes[1:] + codes[:-1]) / 2
    for _ in range(8):
        amax = ((448.0 * (1.0 + torch.rand(1, generator=g).double())) * 2.0 ** exp).float().clamp_max(3e38)
        s = amax / 448.0
        a = (mid * s.double()).float()
        bits = a.view(torch.int32)[None, :] + torch.arange(-2, 3, dtype=torch.int32)[:, None]
        a = bits.clamp_min(0).view(torch.float32)
        a = torch.cat([a, -a]).flatten()
        a = torch.cat([a, a.new_zeros(-a.numel() % 16)])
        q = moe.moe_quant_act(a.to(dev), amax.to(dev)).cpu()
        want = (a / s).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        assert torch.equal(q.view(torch.uint8), want.view(torch.uint8)), float(s)
