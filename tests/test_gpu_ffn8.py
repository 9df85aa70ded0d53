"""The gated expert FFN with a layer norm in front and 8-bit checkpoints, as one run (GPU).

  * Inputs that 8 bits hold without loss (rows of +-1, so that the norm's rows are +-1; weights that select
    one column, so that the activation's input stays on the 8-bit grid): the gradients are those of the FFN
    that keeps everything, held to the float64 oracle within rel (1 + |ref|), rel = 1e-4 for float32 (as the
    tiny float32 FFN).
  * Ordinary bf16 inputs: the gradients against the FFN that keeps everything.  A kept value is off by at
    most half a step, at most 1/128 of its block's largest magnitude (about 3 deviations at most of 32 normal
    values), evenly spread: 0.29 steps rms, below 1.4% of a deviation.  A gradient has one such factor from the
    rows and one from the activation, whose derivative multiplies it by at most about 2: within 5% of the
    gradient's norm.
  * Layers that share their row buffers, a pass captured in a graph and replayed, and calls whose outputs pass
    256 MB: the same bits as without.
"""
import numpy as np
import pytest
import torch

from oracle import layer as olayer
from oracle import norm8
from oracle import planner as oplanner
from tests.gpu_util import DEV, assert_gemm_close, i32, np64, npi, rand_tensor, say
from tests.plan_checks import random_routing

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def m():
    import load_balanced_dispatch_amd as mod
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    return mod


def routed(L, seed, skew=1.5):
    d = L.d
    rng = np.random.default_rng(seed)
    idx = random_routing(rng, d.R, d.S, d.K, d.E, skew)
    gates = rng.dirichlet(np.ones(d.K), size=(d.R, d.S)).astype(np.float32)
    L.topk_idx.copy_(torch.as_tensor(np.asarray(idx, dtype=np.int32)))
    L.gates.copy_(torch.as_tensor(gates))
    return np.asarray(idx), gates


def grads(L):
    names = ["out", "dgates", "dX", "dW_down_home", "dW_gu_home"] + (["dgamma", "dbeta"] if L.norm else [])
    return {n: getattr(L, n).clone() for n in names}


@pytest.mark.parametrize("norm", [True, False])
def test_lossless_checkpoints_against_the_oracle(m, norm):
    R, E, B, S, K, H, Hp = 4, 16, 4, 32, 2, 128, 96
    L = m.MoeFFN(R, E, B, S, K, H, Hp, dtype=F32, backward=True, norm=norm, eps=2.0 ** -30, save8=True)
    idx, gates = routed(L, 21)
    rng = np.random.default_rng(22)
    # rows with as many +1 as -1: mean 0, variance 1, 1 / sqrt(1 + 2^-30) = 1 in float32
    x = np.stack([rng.permutation(np.repeat([1.0, -1.0], H // 2)) for _ in range(R * S)]).reshape(R, S, H)
    gamma, beta = rng.integers(8, 33, H) / 32.0, rng.integers(-16, 17, H) / 64.0
    if not norm:
        x = x * gamma + beta
    pick = rng.integers(0, H, (E, 2 * Hp))
    Wgu = np.zeros((E, H, 2 * Hp))
    for e in range(E):
        Wgu[e, pick[e], np.arange(2 * Hp)] = rng.choice([1.0, -1.0], 2 * Hp)
    Wd = rng.standard_normal((E, Hp, H)) * Hp ** -0.5
    dout = rng.standard_normal((R, S, H))
    for t, v in ((L.X, x), (L.W_gu_home, Wgu), (L.W_down_home, Wd), (L.dout, dout)):
        t.copy_(torch.as_tensor(v, dtype=F32))
    if norm:
        L.gamma.copy_(torch.as_tensor(gamma))
        L.beta.copy_(torch.as_tensor(beta))
    say("lossless checkpoints", "norm" if norm else "no norm")
    L.forward()
    L.backward()
    torch.cuda.synchronize()
    Wd, dout = np64(L.W_down_home), np64(L.dout)
    g64 = gates.astype(np.float64)
    z = x.reshape(-1, H)
    rstd = np.ones(R * S)
    xn = x
    if norm:
        y, _, rstd, z = norm8.layernorm(z, gamma, beta, 2.0 ** -30)
        xn = y.reshape(R, S, H)
    kept = norm8.load8(npi(L.ygu_codes).reshape(-1, Hp), npi(L.ygu_exps).reshape(-1, norm8.blocks(Hp)))
    p = oplanner.plan(idx, E, B)
    P = S * K
    Xp = olayer.dispatch(xn, p.dest_idx)
    Wgus, Wds = olayer.prefetch(Wgu, p.slot_expert), olayer.prefetch(Wd, p.slot_expert)
    Ygu = olayer.group_gemm(Xp, Wgu, Wgus, p.cu_seqlens, P)
    # the checkpoint holds what the oracle computes, to the norm's rounding: the case is lossless
    assert np.abs(kept.reshape(Ygu.shape) - Ygu).max() < 1e-6
    A = olayer.swiglu(Ygu)
    Zp = olayer.group_gemm(A, Wd, Wds, p.cu_seqlens, P)
    dZp, dgate = olayer.combine_backward(dout, Zp, p.dest_idx, g64)
    dA = olayer.group_gemm_dgrad(dZp, Wd, Wds, p.cu_seqlens, P)
    dYgu = olayer.swiglu_backward(Ygu, dA)
    dXn = olayer.dispatch_backward(olayer.group_gemm_dgrad(dYgu, Wgu, Wgus, p.cu_seqlens, P), p.dest_idx)
    dWd, dWds = np.zeros((E, Hp, H)), np.zeros((R, B, Hp, H))
    dWgu, dWgus = np.zeros(Wgu.shape), np.zeros((R, B) + Wgu.shape[1:])
    olayer.wgrad(A, dZp, p.cu_seqlens, P, dWd, dWds)
    olayer.reduce_grad(p.slot_expert, dWd, dWds)
    olayer.wgrad(Xp, dYgu, p.cu_seqlens, P, dWgu, dWgus)
    olayer.reduce_grad(p.slot_expert, dWgu, dWgus)
    assert_gemm_close(np64(L.out), olayer.combine(Zp, p.dest_idx, g64), 1e-4, "out")
    assert_gemm_close(np64(L.dgates), dgate, 1e-4, "dgates")
    assert_gemm_close(np64(L.dW_down_home), dWd, 1e-4, "dW_down")
    assert_gemm_close(np64(L.dW_gu_home), dWgu, 1e-4, "dW_gate_up")
    if norm:
        dX, dgamma, dbeta = norm8.layernorm_backward(dXn.reshape(-1, H), z, rstd, gamma)
        assert_gemm_close(np64(L.dX).reshape(-1, H), dX, 1e-4, "dX")
        assert_gemm_close(np64(L.dgamma), dgamma, 1e-4, "dgamma")
        assert_gemm_close(np64(L.dbeta), dbeta, 1e-4, "dbeta")
    else:
        assert_gemm_close(np64(L.dX), dXn, 1e-4, "dX")


def fill(L, seed):
    d, H, Hp = L.d, L.H, L.Hp
    routed(L, seed)
    L.X.copy_(rand_tensor((d.R, d.S, H), L.dtype, seed + 1))
    L.W_gu_home.copy_(rand_tensor((d.E, H, 2 * Hp), L.dtype, seed + 2, std=H ** -0.5))
    L.W_down_home.copy_(rand_tensor((d.E, Hp, H), L.dtype, seed + 3, std=Hp ** -0.5))
    L.dout.copy_(rand_tensor((d.R, d.S, H), F32, seed + 4))
    if L.norm:
        L.gamma.copy_(1 + rand_tensor((H,), F32, seed + 5, std=0.2))
        L.beta.copy_(rand_tensor((H,), F32, seed + 6, std=0.1))


DIMS = (4, 16, 2, 128, 4, 256, 192)


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("dims,dtype", [(DIMS, BF), ((2, 6, 0, 75, 3, 100, 37), F32), ((3, 3, 1, 41, 1, 61, 45), BF)])
def test_checkpoints_against_keeping_everything(m, dims, dtype, norm):
    whole = m.MoeFFN(*dims, dtype=dtype, backward=True, norm=norm)
    kept8 = m.MoeFFN(*dims, dtype=dtype, backward=True, norm=norm, save8=True)
    for L in (whole, kept8):
        fill(L, 31)
        say("FFN", "save8" if L.save8 else "whole", "norm" if norm else "no norm")
        L.forward()
        L.backward()
    torch.cuda.synchronize()
    a, b = grads(whole), grads(kept8)
    assert torch.equal(a["out"], b["out"])
    for n in a:
        off = float((a[n].double() - b[n].double()).norm() / a[n].double().norm())
        assert off <= 0.05, (n, off)


def test_norm_without_checkpoints_against_the_plain_ffn(m):
    # the norm's own calls around an FFN that gets its rows from outside: the same bits
    L = m.MoeFFN(*DIMS, backward=True, norm=True)
    fill(L, 41)
    L.forward()
    L.backward()
    plain = m.MoeFFN(*DIMS, backward=True)
    fill(plain, 41)
    m.moonep_layernorm(L.d, L.H, L.X, L.gamma, L.beta, L.eps, plain.X, None, None)
    plain.forward()
    plain.backward()
    torch.cuda.synchronize()
    assert torch.equal(plain.out, L.out) and torch.equal(plain.dX, L.dXn)
    assert torch.equal(plain.dW_gu_home, L.dW_gu_home) and torch.equal(plain.dgates, L.dgates)
    dx, dg, db = norm8.layernorm_backward(np64(L.dXn).reshape(-1, L.H),
                                          norm8.layernorm(np64(L.X).reshape(-1, L.H), np64(L.gamma), None, L.eps)[3],
                                          np64(L.rstd).reshape(-1), np64(L.gamma))
    assert_gemm_close(np64(L.dX).reshape(-1, L.H), dx, 1e-4, "dX")
    assert_gemm_close(np64(L.dgamma), dg, 1e-4, "dgamma")
    assert_gemm_close(np64(L.dbeta), db, 1e-4, "dbeta")


@pytest.mark.parametrize("kw", [dict(), dict(norm=True), dict(norm=True, save8=True)])
def test_buffers_given_by_assignment(m, kw):
    # a program may put its own tensors in the place of the layer's
    a, b = (m.MoeFFN(*DIMS, backward=True, **kw) for _ in range(2))
    for L in (a, b):
        fill(L, 45)
    b.X, b.dX, b.dout = b.X.clone(), torch.empty_like(b.dX), b.dout.clone()
    a.X.zero_()
    fill(a, 45)
    for L in (a, b):
        L.forward()
        L.backward()
    torch.cuda.synchronize()
    ga, gb = grads(a), grads(b)
    assert all(torch.equal(ga[n], gb[n]) for n in ga)


def test_layers_share_their_row_buffers(m):
    alone = [m.MoeFFN(*DIMS, backward=True, norm=True, save8=True) for _ in range(2)]
    first = m.MoeFFN(*DIMS, backward=True, norm=True, save8=True)
    shared = [first, m.MoeFFN(*DIMS, backward=True, norm=True, save8=True, scratch=first.scratch)]
    for L, seed in zip(alone + shared, (51, 61, 51, 61)):
        fill(L, seed)
    say("shared row buffers")
    for L in alone:
        L.forward()
        L.backward()
    shared[0].forward()
    shared[1].forward()   # overwrites the first layer's rows
    shared[1].backward()
    shared[0].backward()
    torch.cuda.synchronize()
    for a, b in zip(alone, shared):
        ga, gb = grads(a), grads(b)
        assert all(torch.equal(ga[n], gb[n]) for n in ga)


@pytest.mark.parametrize("dims", [DIMS, (4, 16, 2, 160, 4, 256, 192)])  # the norm's backward in one launch, in two
def test_captured_and_replayed(m, dims):
    L, E = (m.MoeFFN(*dims, backward=True, norm=True, save8=True) for _ in range(2))
    sums = lambda x: [x.dW_gu_home, x.dW_down_home, x.dgamma, x.dbeta]  # noqa: E731

    def step(x):
        for t in sums(x):
            t.zero_()
        x.forward()
        x.backward()

    fill(L, 71)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(L)  # once before the capture, as torch asks
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(L)
    for seed in (81, 91, 101, 81):
        fill(L, seed)
        fill(E, seed)
        say("replay", seed)
        g.replay()
        step(E)  # the program's own eager work between the replays
        torch.cuda.synchronize()
        a, b = grads(L), grads(E)
        assert all(torch.equal(a[n], b[n]) for n in a)


def test_outputs_past_256_mb_hold_the_same_bits(m):
    # outputs this large are stored another way; halves of them are not
    H, rows = 4096, 36000  # 295 MB of bf16
    x = rand_tensor((rows, H), BF, 1)
    gamma, beta = rand_tensor((H,), F32, 2), rand_tensor((H,), F32, 3)

    def norm(x_):
        n = x_.shape[0]
        d = m.make_dims(1, 1, 0, n, 1)
        Y = torch.empty_like(x_)
        codes = torch.empty((n, H), dtype=torch.int8, device=DEV)
        exps = torch.empty((n, H // 32), dtype=torch.uint8, device=DEV)
        v = torch.empty_like(x_)
        Xp = torch.empty_like(x_)
        m.moonep_layernorm(d, H, x_, gamma, beta, 1e-5, Y, None, None, codes, exps)
        m.moonep_load8(n, H, codes, exps, v)
        dest = torch.arange(n, dtype=torch.int32, device=DEV)
        m.moonep_dispatch8(d, H, codes, exps, gamma, beta, dest, Xp)
        return Y, codes, exps, v, Xp

    say("norm, load8, dispatch8 past 256 MB")
    whole = norm(x)
    cut = rows // 2
    lo, hi = norm(x[:cut]), norm(x[cut:].clone())
    for w, a, b in zip(whole, lo, hi):
        assert torch.equal(w[:cut], a) and torch.equal(w[cut:], b)

    def act(y, dA, rows_):
        d = m.make_dims(1, 1, 0, rows_, 1)
        A, A2, dY = torch.empty_like(dA), torch.empty_like(dA), torch.empty_like(y)
        codes = torch.empty((rows_, 2, H), dtype=torch.int8, device=DEV)
        exps = torch.empty((rows_, 2, H // 32), dtype=torch.uint8, device=DEV)
        m.moonep_swiglu_save8(d, H, y, A, codes, exps)
        m.moonep_swiglu_backward8(d, H, codes, exps, dA, None, None, A2, dY, None)
        return A, codes, exps, A2, dY

    y, dA = torch.cat([x, x.flip(0)], 1).contiguous(), x.flip(1).contiguous()
    say("swiglu_save8, swiglu_backward8 past 256 MB")
    whole = act(y, dA, rows)
    lo, hi = act(y[:cut], dA[:cut], cut), act(y[cut:].clone(), dA[cut:].clone(), rows - cut)
    for w, a, b in zip(whole, lo, hi):
        assert torch.equal(w[:cut], a) and torch.equal(w[cut:], b)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_activation_is_the_plain_ones_bit_for_bit(m, dtype):
    # keeping a checkpoint does not change the forward pass: random values over many orders of magnitude, every
    # pair of special ones
    vals = torch.tensor([0.0, -0.0, 1e-30, -90.0, 90.0, -200.0, 200.0, 3e38, -3e38, float("inf"), float("-inf"),
                         float("nan")], device=DEV)
    g, u = torch.meshgrid(vals, vals, indexing="ij")
    n, Hp = 257, 1024
    y = rand_tensor((n, 2 * Hp), F32, 1) * torch.exp2(rand_tensor((n, 2 * Hp), F32, 2, std=3.0))
    y[0, :144], y[0, Hp:Hp + 144] = g.reshape(-1), u.reshape(-1)
    y = y.to(dtype)
    d = m.make_dims(1, 1, 0, n, 1)
    a, b = torch.empty((n, Hp), dtype=dtype, device=DEV), torch.empty((n, Hp), dtype=dtype, device=DEV)
    codes = torch.empty((n, 2, Hp), dtype=torch.int8, device=DEV)
    exps = torch.empty((n, 2, Hp // 32), dtype=torch.uint8, device=DEV)
    m.moonep_swiglu(d, Hp, y, a)
    m.moonep_swiglu_save8(d, Hp, y, b, codes, exps)
    torch.cuda.synchronize()
    same = (a == b) | (torch.isnan(a) & torch.isnan(b))
    assert bool(same.all())


def test_offsets_past_32_bits(m):
    # 310 000 rows of 7168 columns are 2.2e9 elements: the last rows must be those of a call on them alone
    n, H, last = 310_000, 7168, 6
    g = torch.Generator(device=DEV).manual_seed(9)
    gamma, beta = rand_tensor((H,), F32, 2), rand_tensor((H,), F32, 3)

    def norm(x):
        rows = x.shape[0]
        d = m.make_dims(1, 1, 0, rows, 1)
        Y, v, Xp = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
        rstd = torch.empty(rows, device=DEV)
        codes = torch.empty((rows, H), dtype=torch.int8, device=DEV)
        exps = torch.empty((rows, H // 32), dtype=torch.uint8, device=DEV)
        m.moonep_layernorm(d, H, x, gamma, beta, 1e-5, Y, None, rstd, codes, exps)
        m.moonep_load8(rows, H, codes, exps, v)
        m.moonep_dispatch8(d, H, codes, exps, gamma, beta, torch.arange(rows, dtype=torch.int32, device=DEV), Xp)
        return Y, v, Xp, codes, exps, rstd

    x = torch.randn((n, H), generator=g, device=DEV, dtype=BF)
    say("norm, load8, dispatch8 of", n, "rows")
    whole = norm(x)
    tail = norm(x[-last:].clone())
    for a, b in zip(whole, tail):
        assert torch.equal(a[-last:], b)
    codes, exps, rstd = whole[3:]
    del whole, x
    dY = torch.randn((n, H), generator=g, device=DEV)

    def back(rows, dY_, codes_, exps_, rstd_):
        d = m.make_dims(1, 1, 0, rows, 1)
        dX, dg, Xp = torch.empty_like(dY_), torch.zeros(H, device=DEV), torch.empty((rows, H), dtype=BF, device=DEV)
        ws = torch.empty(m.moonep_layernorm_backward_workspace_bytes(d, H), dtype=torch.uint8, device=DEV)
        m.moonep_layernorm_backward8(d, H, dY_, codes_, exps_, rstd_, gamma, dX, dg, None, ws)
        m.moonep_combine_backward_ungated(d, H, dY_, torch.arange(rows, dtype=torch.int32, device=DEV), Xp)
        return dX, Xp

    say("norm backward, ungated rows of", n, "rows")
    dX, Xp = back(n, dY, codes, exps, rstd)
    dXt, Xpt = back(last, dY[-last:].clone(), codes[-last:].clone(), exps[-last:].clone(), rstd[-last:].clone())
    assert torch.equal(Xp[-last:], Xpt)
    # few rows take another kernel, which sums the means in another order: 65 u of the terms (test_gpu_norm8.py)
    z = np64(tail[1])
    gy = np.abs(np64(dY[-last:]) * np64(gamma))
    terms = gy + gy.mean(axis=1, keepdims=True) + np.abs(z) * (gy * np.abs(z)).mean(axis=1, keepdims=True)
    tol = 2 * 65 * 2.0 ** -24 * np64(rstd[-last:])[:, None] * terms
    assert np.all(np.abs(np64(dX[-last:]) - np64(dXt)) <= tol)
    del dX, Xp, dY, codes, exps
    Hp = H // 2
    y = torch.randn((n, 2 * Hp), generator=g, device=DEV, dtype=BF)

    def act(rows, y_):
        d = m.make_dims(1, 1, 0, rows, 1)
        A, A2, dYgu = (torch.empty((rows, w), dtype=BF, device=DEV) for w in (Hp, Hp, 2 * Hp))
        c = torch.empty((rows, 2, Hp), dtype=torch.int8, device=DEV)
        e = torch.empty((rows, 2, Hp // 32), dtype=torch.uint8, device=DEV)
        m.moonep_swiglu_save8(d, Hp, y_, A, c, e)
        m.moonep_swiglu_backward8(d, Hp, c, e, A, None, None, A2, dYgu, None)
        return A, c, e, A2, dYgu

    say("swiglu_save8, swiglu_backward8 of", n, "rows")
    for a, b in zip(act(n, y), act(last, y[-last:].clone())):
        assert torch.equal(a[-last:], b)
