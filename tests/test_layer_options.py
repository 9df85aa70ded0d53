"""MoeFFN's norm, save8 and scratch options: which buffers it makes, and what it refuses (CPU only: nothing runs)."""
import pytest
import torch

import load_balanced_dispatch_amd as m

DIMS = (2, 4, 1, 6, 2, 64, 32)


def make(**kw):
    return m.MoeFFN(*DIMS, device="cpu", **kw)


def test_calls_of_each_form():
    names = lambda L: [n for n, _ in L.forward_calls() + L.backward_calls()]  # noqa: E731
    plain = ["plan", "prefetch", "dispatch", "gemm_gate_up", "swiglu", "gemm_down", "combine", "combine_backward",
             "dgrad_down", "wgrad_down", "swiglu_backward", "dgrad_gate_up", "wgrad_gate_up", "dispatch_backward",
             "reduce_grad"]
    assert names(make(backward=True)) == plain
    with_norm = names(make(backward=True, norm=True))
    assert with_norm == plain[:2] + ["layernorm_dispatch"] + plain[3:] + ["layernorm_backward"]
    kept = names(make(backward=True, save8=True))
    assert kept[2] == "save8" and "swiglu_save8" in kept and "swiglu_backward8" in kept and "dispatch8" in kept
    assert "save8" not in names(make(backward=True, save8=True, norm=True))


def test_kept_bytes():
    # what a layer holds between its passes: 8-bit rows of the tokens and of the activation's input
    L = make(backward=True, norm=True, save8=True)
    R, S, K, H, Hp = 2, 6, 2, 64, 32
    N = R * S * K
    kept = [L.x_codes, L.x_exps, L.ygu_codes, L.ygu_exps]
    assert sum(t.numel() * t.element_size() for t in kept) == (R * S * H + N * 2 * Hp) * 33 // 32
    assert L.dZp.data_ptr() == L.Zp.data_ptr() and L.dYgu.data_ptr() == L.Ygu.data_ptr()


def test_shared_rows():
    a = make(backward=True, save8=True)
    b = make(backward=True, save8=True, scratch=a.scratch)
    assert b.Xp.data_ptr() == a.Xp.data_ptr() and b.x_codes.data_ptr() != a.x_codes.data_ptr()
    make(scratch=a.scratch)  # a layer without a backward may share too
    with pytest.raises(ValueError, match="save8=True"):
        make(backward=True, scratch=a.scratch)
    with pytest.raises(ValueError, match="scratch must hold"):
        m.MoeFFN(2, 4, 1, 6, 2, 64, 48, device="cpu", backward=True, save8=True, scratch=a.scratch)
    with pytest.raises(ValueError, match="scratch must hold"):
        m.MoeFFN(*DIMS, device="cpu", dtype=torch.float32, backward=True, save8=True, scratch=a.scratch)
    with pytest.raises(ValueError, match="scratch must hold dA"):
        make(backward=True, save8=True, scratch={k: v for k, v in a.scratch.items() if k != "dA"})


def test_save8_needs_a_backward():
    with pytest.raises(ValueError, match="backward=True"):
        make(save8=True)
