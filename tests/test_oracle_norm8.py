"""Pins the layer norm, the 8-bit rows and the FFN backward from 8-bit checkpoints in the oracle (CPU only).

Pins: 8-bit rows on hand-worked blocks; the error bound of every kept value (half a step, a step next to
the clamp) and the step's bound (1/64 of the block's largest magnitude) on random rows over 60 binary
orders; values are bf16 numbers; blocks that are zero, denormal, or not finite.  The norm equals float64
torch; its gradient equals central differences and float64 autograd.  The backward with the gates on the
expert's side (ungated output gradient, <dA, h> as the gate's gradient) equals float64 autograd of the
plain forward, on random plans.
"""
import numpy as np
import pytest
import torch

from oracle import layer, norm8, planner
from tests.test_oracle_ffn import _ffn_case


def test_save8_hand_worked():
    x = np.zeros((1, 40))
    x[0, :4] = [1.0, -0.5, 0.3, 127.0 / 64]   # block 0: b = 127, step 2^-6
    x[0, 32:35] = [4.0, 4.0 + 1 / 32, -6.1]   # block 1 (8 columns): b = 129, step 2^-4
    codes, exps = norm8.save8(x)
    assert exps.tolist() == [[127, 129]]
    assert codes[0, :4].tolist() == [64, -32, 19, 127]
    assert codes[0, 32:35].tolist() == [64, 64, -98]  # 64.5 steps round to the even 64
    assert norm8.load8(codes, exps)[0, 34] == -98 / 16


def test_save8_bounds_on_random_rows():
    rng = np.random.default_rng(5)
    for C in (1, 7, 31, 32, 33, 100):
        x = (rng.standard_normal((200, C)) * np.exp2(rng.integers(-30, 30, (200, 1)))).astype(np.float32)
        codes, exps = norm8.save8(x)
        v, st = norm8.load8(codes, exps), norm8.steps(exps, C)
        near_clamp = np.abs(x) > 127.5 * st
        assert np.all(np.abs(v - x) <= np.where(near_clamp, 1.0, 0.5) * st)
        top = np.stack([np.abs(x[:, j * 32:(j + 1) * 32]).max(1) for j in range(norm8.blocks(C))], 1)
        assert np.all(norm8.steps(exps, 32 * exps.shape[1])[:, ::32] * 64 <= top)
        assert np.array_equal(torch.tensor(v).to(torch.bfloat16).double().numpy(), v)


def test_save8_edges():
    tiny, big = np.float32(1e-45), np.float32(3.4028235e38)
    x = np.stack([np.zeros(5), np.full(5, tiny), np.full(5, big), [1, np.inf, 0, 0, 2], [np.nan, 0, 1, 0, 0]])
    codes, exps = norm8.save8(x)
    assert exps[:, 0].tolist() == [1, 1, 254, 255, 255]
    v = norm8.load8(codes, exps)
    assert not v[:2].any()                                # far below the smallest step, 2^-132
    assert np.all(v[2] == 127 * 2.0 ** 121)               # clamped, and finite
    assert np.isnan(v[3:]).all()


def test_layernorm_is_torch():
    rng = np.random.default_rng(2)
    x, g, b = rng.standard_normal((6, 17)) + 3, rng.standard_normal(17), rng.standard_normal(17)
    y, m, r, z = norm8.layernorm(x, g, b, 1e-5)
    ref = torch.nn.functional.layer_norm(torch.tensor(x), (17,), torch.tensor(g), torch.tensor(b), 1e-5)
    assert np.allclose(y, ref.numpy(), rtol=1e-13, atol=1e-13)
    assert np.allclose(z.mean(1), 0, atol=1e-14)
    assert np.allclose(m, x.mean(1)) and np.allclose(r, 1 / np.sqrt(x.var(1) + 1e-5))


@pytest.mark.parametrize("H", [1, 2, 9, 33])
def test_layernorm_gradient_is_differences_and_autograd(H):
    rng = np.random.default_rng(H)
    eps = 1e-3
    x, g, b = rng.standard_normal((4, H)) * 2 + 1, rng.standard_normal(H), rng.standard_normal(H)
    dy = rng.standard_normal((4, H))
    _, m, r, z = norm8.layernorm(x, g, b, eps)
    dx, dg, db = norm8.layernorm_backward(dy, z, r, g)
    h = 1e-6
    loss = lambda x_, g_, b_: np.sum(dy * norm8.layernorm(x_, g_, b_, eps)[0])  # noqa: E731
    for i in range(4):
        for j in range(H):
            e = np.zeros((4, H))
            e[i, j] = h
            assert abs((loss(x + e, g, b) - loss(x - e, g, b)) / (2 * h) - dx[i, j]) < 1e-6
    for j in range(H):
        e = np.zeros(H)
        e[j] = h
        assert abs((loss(x, g + e, b) - loss(x, g - e, b)) / (2 * h) - dg[j]) < 1e-6
        assert abs((loss(x, g, b + e) - loss(x, g, b - e)) / (2 * h) - db[j]) < 1e-6
    xt, gt, bt = (torch.tensor(a, requires_grad=True) for a in (x, g, b))
    (torch.nn.functional.layer_norm(xt, (H,), gt, bt, eps) * torch.tensor(dy)).sum().backward()
    for got, ref in ((dx, xt), (dg, gt), (db, bt)):
        assert np.allclose(got, ref.grad.numpy(), rtol=1e-10, atol=1e-10)


@pytest.mark.parametrize("seed", range(8))
def test_backward_with_gates_on_the_experts_side_equals_autograd(seed):
    c = _ffn_case(seed)
    R, S, K, E, H, Hp = c["R"], c["S"], c["K"], c["E"], c["H"], c["Hp"]
    rng = c["rng"]
    gamma, beta, x0 = rng.standard_normal(H), rng.standard_normal(H), rng.standard_normal((R, S, H)) + 0.5
    dout = rng.standard_normal((R, S, H))
    p = planner.plan(c["idx"], E, c["B"])
    P = S * K
    xn, _, r, z = norm8.layernorm(x0.reshape(-1, H), gamma, beta, 1e-5)
    Wgus, Wds = layer.prefetch(c["Wgu"], p.slot_expert), layer.prefetch(c["Wd"], p.slot_expert)
    Xp = norm8.dispatch8(z.reshape(R, S, H), gamma, beta, p.dest_idx)
    assert np.allclose(Xp, layer.dispatch(xn.reshape(R, S, H), p.dest_idx), rtol=1e-14, atol=1e-14)
    Ygu = layer.group_gemm(Xp, c["Wgu"], Wgus, p.cu_seqlens, P)
    # backward, nothing kept but z and Ygu
    dZ = norm8.combine_backward_ungated(dout, p.dest_idx)
    dA = layer.group_gemm_dgrad(dZ, c["Wd"], Wds, p.cu_seqlens, P)
    src = np.empty(R * P, dtype=np.int64)
    src[p.dest_idx.reshape(-1)] = np.arange(R * P)
    A, dYgu, dgate_row = norm8.swiglu_backward8(Ygu, dA, c["gates"].reshape(-1)[src])
    dgate = np.empty(R * P)
    dgate[src] = dgate_row
    dXn = layer.dispatch_backward(layer.group_gemm_dgrad(dYgu, c["Wgu"], Wgus, p.cu_seqlens, P), p.dest_idx)
    dX, dgamma, dbeta = norm8.layernorm_backward(dXn.reshape(-1, H), z, r, gamma)
    B = max(c["B"], 0)
    dWd, dWds = np.zeros((E, Hp, H)), np.zeros((R, B, Hp, H))
    layer.wgrad(A, dZ, p.cu_seqlens, P, dWd, dWds)
    layer.reduce_grad(p.slot_expert, dWd, dWds)
    # float64 autograd of the plain forward (CPU)
    X, G0, B0, Wgu, Wd, G = (torch.tensor(a, requires_grad=True)
                             for a in (x0, gamma, beta, c["Wgu"], c["Wd"], c["gates"]))
    ids = torch.tensor(np.asarray(c["idx"]), dtype=torch.int64)
    xt = torch.nn.functional.layer_norm(X, (H,), G0, B0, 1e-5)
    y = torch.einsum("rsh,rskhn->rskn", xt, Wgu[ids])
    a = torch.nn.functional.silu(y[..., :Hp]) * y[..., Hp:]
    o = (G.unsqueeze(-1) * torch.einsum("rskn,rsknh->rskh", a, Wd[ids])).sum(dim=2)
    (o * torch.tensor(dout)).sum().backward()
    for got, ref in ((dX.reshape(R, S, H), X), (dgamma, G0), (dbeta, B0), (dgate.reshape(R, S, K), G), (dWd, Wd)):
        assert np.allclose(got, ref.grad.numpy(), rtol=1e-10, atol=1e-10)
