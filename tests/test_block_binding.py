"""How the binding reads and checks its arguments for the grouped router and
block-scaled e4m3 (host only; no GPU needed)."""
import os

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


@pytest.mark.parametrize("name", ["n_groups", "topk_groups", "group_top"])
@pytest.mark.parametrize("v", [2 ** 32 + 1, 2 ** 31, -2 ** 32 + 1, -1])
def test_routing_refuses_numbers_it_would_cut(name, v):
    with pytest.raises(ValueError, match=name):
        moe.Routing(**{name: v})


# ------------------------------------------------- fused_moe_grouped, any dtype

E, K, H, I, M = 4, 2, 512, 256, 3
DTYPES = ["f32", "bf16", "e4m3", "w4a16", "block"]


def layer_args(name):
    """Tensors of a layer of this dtype, as fused_moe_grouped takes them."""
    f8, dt = torch.float8_e4m3fn, {"f32": torch.float32, "bf16": torch.bfloat16}.get(name)
    a = dict(x=torch.zeros(M, H, dtype=dt or (f8 if name == "e4m3" else torch.bfloat16)), router_logits=torch.zeros(M, E),
             w1=torch.zeros(E, 2 * I, H, dtype=dt or f8), w2=torch.zeros(E, H, I, dtype=dt or f8))
    if name == "e4m3":
        a.update(x_scale=torch.ones(1), w1_scale=torch.ones(E), w2_scale=torch.ones(E, 1, 1))
    if name == "w4a16":
        a.update(w1=torch.zeros(E, 2 * I, H // 2, dtype=torch.uint8), w2=torch.zeros(E, H, I // 2, dtype=torch.uint8),
                 w1_scale=torch.ones(E, H // 128, 2 * I), w2_scale=torch.ones(E, I // 128, H))
    if name == "block":
        a.update(w1_scale=torch.ones(E, 2 * I // 128, H // 128), w2_scale=torch.ones(E, H // 128, I // 128))
    return a


@pytest.fixture
def calls(monkeypatch):
    """What the binding would have handed to the library."""
    from moe_layer_topk_amd import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    got = []
    monkeypatch.setattr(moe, "_stream", lambda t: None)
    monkeypatch.setattr(moe, "_call", lambda fn, what, dev, *args: got.append(what))
    return got


@pytest.mark.parametrize("name", DTYPES)
def test_grouped_layer_takes_its_dtypes(calls, name):
    moe.fused_moe_grouped(topk=K, routing=moe.Routing(), **layer_args(name))
    assert calls == ["fused_moe_grouped"]


WRONG = {
    "x strided": lambda a: dict(x=a["x"].new_zeros(M, 2 * H)[:, ::2]),
    "x narrow": lambda a: dict(x=a["x"].new_zeros(M, H - 128)),
    "x of another dtype": lambda a: dict(x=torch.zeros(M, H, dtype=torch.float64)),
    "x elsewhere": lambda a: dict(w1=a["w1"].to("meta"), w2=a["w2"].to("meta")),
    "w1 strided": lambda a: dict(w1=a["w1"].new_zeros(*a["w1"].shape[:2], 2 * a["w1"].shape[2])[:, :, ::2]),
    "w1 odd": lambda a: dict(w1=a["w1"].new_zeros(E, 2 * I - 1, a["w1"].shape[2])),
    "w2 of fewer experts": lambda a: dict(w2=a["w2"].new_zeros(E - 1, *a["w2"].shape[1:])),
    "w2 transposed": lambda a: dict(w2=a["w2"].new_zeros(E, a["w2"].shape[2], H).transpose(1, 2)),
    "w2 short": lambda a: dict(w2=a["w2"].new_zeros(E, H, a["w2"].shape[2] // 2)),
    "w2 of another dtype": lambda a: dict(w2=torch.zeros(a["w2"].shape, dtype=torch.int8)),
    "logits of fewer experts": lambda a: dict(router_logits=torch.zeros(M, E - 1)),
}
SCALES = {
    "missing": lambda s: None,
    "short": lambda s: s.reshape(-1)[:-1],
    "strided": lambda s: s.new_zeros(*s.shape, 2)[..., 1] if s.numel() > 1 else s.new_zeros(2),
    "of another dtype": lambda s: s.double(),
}


@pytest.mark.parametrize("name", DTYPES)
@pytest.mark.parametrize("wrong", WRONG)
def test_grouped_layer_refuses_tensors_it_would_misread(calls, name, wrong):
    a = layer_args(name)
    a.update(WRONG[wrong](a))
    with pytest.raises(ValueError):
        moe.fused_moe_grouped(topk=K, routing=moe.Routing(), **a)
    assert calls == []


@pytest.mark.parametrize("name,scale", [("e4m3", "x_scale"), ("e4m3", "w1_scale"), ("e4m3", "w2_scale"), ("w4a16", "w1_scale"),
                                        ("w4a16", "w2_scale"), ("block", "w2_scale")])
@pytest.mark.parametrize("wrong", SCALES)
def test_grouped_layer_refuses_scales_it_would_misread(calls, name, scale, wrong):
    a = layer_args(name)
    a[scale] = SCALES[wrong](a[scale])
    with pytest.raises(ValueError):
        moe.fused_moe_grouped(topk=K, routing=moe.Routing(), **a)
    assert calls == []


@pytest.mark.parametrize("name", DTYPES)
def test_grouped_layer_refuses_a_workspace_smaller_than_it_looks(calls, name):
    n = moe.fused_moe_workspace_size(moe._layer_dtype(layer_args(name)["w1"], layer_args(name).get("w1_scale")), M, E, K, H, I)
    one = torch.zeros(1, dtype=torch.uint8)
    for ws in (one.expand(n), one.expand(2, n), torch.zeros(2 * n, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            moe.fused_moe_grouped(topk=K, routing=moe.Routing(), workspace=ws, **layer_args(name))
    assert calls == []
    moe.fused_moe_grouped(topk=K, routing=moe.Routing(), workspace=torch.zeros(n + 9, dtype=torch.uint8)[:n], **layer_args(name))
    assert calls == ["fused_moe_grouped"]
