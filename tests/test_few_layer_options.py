"""MoeFFN's router option and MoeFew: which buffers and calls they make, and what they refuse (CPU only: nothing runs)."""
import pytest
import torch

import load_balanced_dispatch_amd as m

DIMS = (2, 4, 1, 6, 2, 64, 32)
FEW = (2, 4, 3, 2, 64, 32)


def names(calls):
    return [n for n, _ in calls]


def test_router_in_front_of_the_planned_layer():
    plain = m.MoeFFN(*DIMS, device="cpu", backward=True)
    L = m.MoeFFN(*DIMS, device="cpu", backward=True, router="sigmoid", router_bias=True, route_scale=2.5)
    assert names(L.forward_calls()) == ["route"] + names(plain.forward_calls())
    assert names(L.backward_calls()) == names(plain.backward_calls()) + ["route_backward"]
    assert L.logits.shape == L.dlogits.shape == (2, 6, 4) and L.bias.shape == (4,)
    assert plain.logits is None and plain.bias is None and not hasattr(plain, "dlogits")
    assert not hasattr(m.MoeFFN(*DIMS, device="cpu", router="softmax"), "dlogits")
    with pytest.raises(ValueError, match="unknown router score"):
        m.MoeFFN(*DIMS, device="cpu", router="tanh")
    with pytest.raises(ValueError, match="router_bias"):
        m.MoeFFN(*DIMS, device="cpu", router_bias=True)


def test_calls_of_each_form():
    assert names(m.MoeFew(*FEW, device="cpu").forward_calls()) == ["few_ffn"]
    L = m.MoeFew(*FEW, device="cpu", bits=4, G=64, norm=True, router="softmax")
    assert names(L.forward_calls()) == ["route", "layernorm", "few_ffn4"]
    assert L.gu_codes.shape == (4, 8, 64) and L.gu_scales.shape == (4, 1, 64)
    assert L.down_codes.shape == (4, 4, 64) and L.down_scales.shape == (4, 1, 64)


def test_weights_of_another_layer():
    ffn = m.MoeFFN(*DIMS, device="cpu")
    L = m.MoeFew(*FEW, device="cpu", weights=(ffn.W_gu_home, ffn.W_down_home))
    assert L.W_gu.data_ptr() == ffn.W_gu_home.data_ptr() and L.W_down.data_ptr() == ffn.W_down_home.data_ptr()
    a = m.MoeFew(*FEW, device="cpu", bits=4)
    b = m.MoeFew(*FEW, device="cpu", bits=4, weights=(a.gu_codes, a.gu_scales, a.down_codes, a.down_scales))
    assert b.down_scales.data_ptr() == a.down_scales.data_ptr() and b.out.data_ptr() != a.out.data_ptr()
    with pytest.raises(ValueError, match="W_gu must be"):
        m.MoeFew(*FEW, device="cpu", weights=(ffn.W_gu_home.float(), ffn.W_down_home))
    with pytest.raises(ValueError, match="W_down must be"):
        m.MoeFew(*FEW, device="cpu", weights=(ffn.W_gu_home, ffn.W_gu_home))
    with pytest.raises(ValueError, match="contiguous"):
        m.MoeFew(*FEW, device="cpu", weights=(ffn.W_gu_home.transpose(0, 1).contiguous().transpose(0, 1), ffn.W_down_home))
    with pytest.raises(ValueError, match="weights must be gu_codes"):
        m.MoeFew(*FEW, device="cpu", bits=4, weights=(ffn.W_gu_home, ffn.W_down_home))
    with pytest.raises(ValueError, match="gu_scales must be"):
        m.MoeFew(*FEW, device="cpu", bits=4, G=32,
                 weights=(a.gu_codes, torch.zeros(4, 1, 64, dtype=torch.bfloat16), a.down_codes, a.down_scales))


def test_refusals():
    with pytest.raises(ValueError, match="bits"):
        m.MoeFew(*FEW, device="cpu", bits=8)
    with pytest.raises(ValueError, match="G must be"):
        m.MoeFew(*FEW, device="cpu", bits=4, G=16)
    with pytest.raises(ValueError, match="exceeds 1024"):
        m.MoeFew(2, 4, 257, 2, 64, 32, device="cpu")
    with pytest.raises(ValueError, match="unknown router score"):
        m.MoeFew(*FEW, device="cpu", router="none")


def test_weights_are_copied_as_they_are():
    L = m.MoeFew(*FEW, device="cpu", dtype=torch.float32)
    g, w = torch.randn(4, 64, 64), torch.randn(4, 32, 64)
    L.save_weights(g, w)
    assert torch.equal(L.W_gu, g) and torch.equal(L.W_down, w)


def test_weights_of_another_shape_are_refused():
    # copy_ alone would repeat one expert's for all, and save4 read a transposed tensor of as many elements
    g, w = torch.randn(4, 64, 64), torch.randn(4, 32, 64)
    for L in (m.MoeFew(*FEW, device="cpu"), m.MoeFew(*FEW, device="cpu", bits=4)):
        with pytest.raises(ValueError, match="W_gu must be"):
            L.save_weights(g[:1], w)
        with pytest.raises(ValueError, match="W_down must be"):
            L.save_weights(g, w.transpose(1, 2).contiguous())
