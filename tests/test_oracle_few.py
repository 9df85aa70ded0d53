"""Pins the router, the 4-bit weights and the layer for few tokens in the oracle (CPU only).

Pins: the choice on hand-worked rows (ties, masks, a bias that changes the choice and not the gates, tokens with too few
experts); scores against float64 torch; the gates' gradient against central differences and float64 autograd; 4-bit codes
on hand-worked groups, their bound (half a scale) and their word layout bit by bit; the layer for few tokens against the
plain definitions of the whole layer.
"""
import numpy as np
import pytest
import torch

from oracle import few, layer

INF = float("inf")


def test_choice_hand_worked():
    l = np.array([[1.0, 3.0, 3.0, 2.0], [0.0, 0.0, 0.0, 0.0], [-INF, 5.0, np.nan, -1.0], [-INF] * 4, [INF, 1.0, INF, 0.0]])
    ids, gates = few.route(l, None, 3, "softmax", True, 1.0)
    assert ids.tolist() == [[1, 2, 3], [0, 1, 2], [1, 3, -1], [-1, -1, -1], [0, 2, 1]]
    assert np.allclose(gates.sum(1), [1, 1, 1, 0, 1])
    assert gates[2, 2] == 0 and gates[4].tolist() == [0.5, 0.5, 0.0]
    _, whole = few.route(l, None, 3, "softmax", False, 2.0)
    assert np.allclose(whole[1], 0.5)
    # a bias changes who is chosen, not the scores that are handed on
    ids, gates = few.route(l[:1], np.array([0.9, 0, 0, -np.inf]), 2, "sigmoid", False, 1.0)
    assert ids.tolist() == [[0, 1]]
    assert np.allclose(gates, 1 / (1 + np.exp(-np.array([[1.0, 3.0]]))))
    ids, _ = few.route(l[:1], np.array([-np.inf, np.nan, 0, -np.inf]), 3, "sigmoid", True, 1.0)
    assert ids.tolist() == [[2, -1, -1]]


def test_lowest_values():
    low = -few.LARGEST
    l = np.array([[low, low, low], [low, 0.0, few.LARGEST]])
    ids, gates = few.route(l, None, 2, "softmax", False, 1.0)
    assert ids.tolist() == [[0, 1], [2, 1]]
    assert np.allclose(gates, [[1 / 3, 1 / 3], [1, 0]])
    ids, gates = few.route(np.array([[-200.0, -201.0, -300.0]]), None, 2, "sigmoid", True, 1.0)
    assert np.allclose(gates, [[1 / (1 + np.exp(-1)), 1 / (1 + np.exp(1))]])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_are_torch(score):
    l = np.random.default_rng(1).standard_normal((9, 13)) * 4
    t = torch.tensor(l)
    ref = torch.softmax(t, 1) if score == "softmax" else torch.sigmoid(t)
    assert np.allclose(few.scores(l, score), ref.numpy(), rtol=1e-13)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_is_differences_and_autograd(score, renorm):
    rng = np.random.default_rng(3)
    T, E, K, scale = 4, 7, 3, 2.5
    l, dg = rng.standard_normal((T, E)), rng.standard_normal((T, K))
    ids, gates = few.route(l, None, K, score, renorm, scale)
    ids[1, 2] = -1           # a place without an expert
    ids[2, 1] = ids[2, 0]    # the same expert twice
    dl, size = few.route_backward(l, ids, dg, score, renorm, scale)
    for t in range(T):
        for e in range(E):
            h = np.zeros((T, E))
            h[t, e] = 1e-6
            up = few.gates_of(l + h, ids, score, renorm, scale)
            down = few.gates_of(l - h, ids, score, renorm, scale)
            assert abs(((up - down) * dg).sum() / 2e-6 - dl[t, e]) < 1e-8
    x = torch.tensor(l, requires_grad=True)
    s = torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x)
    on = torch.tensor(ids >= 0)
    w = s.gather(1, torch.tensor(np.maximum(ids, 0))) * on
    g = scale * (w / w.sum(1, keepdim=True) if renorm else w)
    (g * torch.tensor(dg)).sum().backward()
    assert np.allclose(dl, x.grad.numpy(), atol=1e-14)
    assert np.all(np.abs(dl) <= size * (1 + 1e-12))


def test_gradient_of_masked_experts_is_zero():
    l = np.array([[-INF, 1.0, np.nan, 2.0], [-INF] * 4])
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            ids, _ = few.route(l, None, 3, score, renorm, 1.0)
            dl, _ = few.route_backward(l, ids, np.ones((2, 3)) * [1, 2, 5], score, renorm, 1.0)
            assert np.isfinite(dl).all() and not dl[1].any() and not dl[0, [0, 2]].any()


def test_save4_hand_worked():
    W = np.zeros((1, 40, 3), dtype=np.float32)
    W[0, :4, 0] = [7.0, -7.0, 2.5, 1.5]     # scale 1: 2.5 rounds to 2, 1.5 to 2
    W[0, 33, 1] = -3.5                       # the second group: scale 0.5
    W[0, 5, 2] = np.inf
    codes, scales = few.save4(W, 32)
    assert scales[0, :, 0].tolist() == [1.0, 0.0] and scales[0, 1, 1] == 0.5 and np.isnan(scales[0, 0, 2])
    assert codes[0, :4, 0].tolist() == [7, -7, 2, 2] and codes[0, 33, 1] == -7
    v = few.load4(codes, scales, 32)
    assert v[0, 33, 1] == -3.5 and np.isnan(v[0, :32, 2]).all() and not v[0, 32:, 2].any()


def test_words_bit_by_bit():
    codes = np.full((1, 11, 1), 0)
    for i in range(8):
        codes[:] = -8
        codes[0, i] = 7
        words = few.pack4(codes)
        assert words.shape == (1, 2, 1)
        # rows 0, 2, 4, 6 in the low half from the lowest bits on, rows 1, 3, 5, 7 in the high half
        assert int(words[0, 0, 0]) & 0xFFFFFFFF == 15 << (4 * (i // 2) + (16 if i % 2 else 0))
        assert int(words[0, 1, 0]) & 0xFFFFFFFF == 0x88808800  # rows 8, 9, 10 (bits 0, 16, 4) hold 0, rows past H the code 0
    rng = np.random.default_rng(0)
    codes = rng.integers(-8, 8, (3, 21, 5))
    assert np.array_equal(few.unpack4(few.pack4(codes), 21), codes)


@pytest.mark.parametrize("G", [32, 64, 128])
def test_save4_bound(G):
    rng = np.random.default_rng(G)
    W = (rng.standard_normal((2, 200, 9)) * np.exp2(rng.integers(-30, 30, (2, 1, 9)))).astype(np.float32)
    codes, scales = few.save4(W, G)
    s = np.repeat(scales, G, axis=1)[:, :200]
    # half a step, and the float32 quotient's rounding; a scale rounded down leaves the largest 7.03 steps long
    assert np.all(np.abs(few.load4(codes, scales, G) - W) <= (0.5 + 2 ** -18) * s)
    assert codes.max() <= 7 and codes.min() >= -7


def test_few_layer_and_ffn_are_the_layer():
    rng = np.random.default_rng(4)
    R, S, E, K, H, Hp = 2, 3, 5, 2, 6, 4
    X = rng.standard_normal((R, S, H))
    ids = np.stack([rng.permutation(E)[:K] for _ in range(R * S)]).reshape(R, S, K)
    gates = rng.random((R, S, K))
    W, W_gu, W_down = (rng.standard_normal(s) for s in ((E, H, Hp), (E, H, 2 * Hp), (E, Hp, H)))
    flat = (X.reshape(-1, H), ids.reshape(-1, K), gates.reshape(-1, K))
    out, size = few.few_layer(*flat, W)
    assert np.allclose(out, layer.moe_forward(X, W, ids, gates).reshape(R * S, -1)) and np.all(np.abs(out) <= size)
    out, bound = few.few_ffn(*flat, W_gu, W_down, 1e-9)
    assert np.allclose(out, layer.moe_ffn_forward(X, W_gu, W_down, ids, gates).reshape(R * S, -1))
    # the bound holds for products that are off by as much as it says
    off = few.few_ffn(flat[0], flat[1], flat[2], W_gu * (1 + 1e-9 * np.sign(W_gu) * rng.random(W_gu.shape)), W_down, 0)[0]
    assert np.all(np.abs(off - out) <= bound + 1e-15)
    none = flat[1] * 0 - 1
    assert not few.few_layer(flat[0], none, flat[2], W)[0].any()
