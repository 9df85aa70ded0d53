"""Forms of the layer norm and of the 8-bit checkpoint kernels that a launch chooses by width and row count (GPU):
widths of each lane layout, more rows than a launch holds at a time, more columns than a wave takes at a time, and the
reciprocal behind the activation.

Tolerances are those derived at the head of test_gpu_norm8.py.
"""
import numpy as np
import pytest
import torch

from oracle import norm8
from tests import test_gpu_norm8 as base
from tests.gpu_util import DEV, np64, npi, rand_tensor, say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def m():
    import load_balanced_dispatch_amd as mod
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    return mod


# rows of three waves of one chunk a lane, in whole chunks: the layout's first and last width, and one between
THREE_WAVES = [1032, 1408, 1536]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H", THREE_WAVES)
def test_layernorm_of_three_waves(m, dtype, H):
    base.test_layernorm(m, dtype, H)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,K", [(1032, 3), (1408, 6), (1536, 1)])
def test_layernorm_dispatch_of_three_waves(m, dtype, H, K):
    base.test_layernorm_dispatch_is_the_two_calls(m, dtype, H, K)


@pytest.mark.parametrize("H", THREE_WAVES)
def test_layernorm_checkpoint_of_three_waves(m, H):
    base.test_layernorm_checkpoint_is_save8_of_its_rows(m, H)


# A launch of the forward has at most 64 waves' worth of blocks on each of 256 compute units: 16 384 rows of one wave,
# 5 376 of three, 2 048 of eight, 1 792 of nine.  Each case has more.
MANY_ROWS = [(40_000, 64, BF), (40_000, 61, BF), (33_000, 520, F32), (20_000, 1000, BF), (20_000, 1408, BF),
             (12_000, 1408, F32), (20_000, 1413, BF), (17_000, 2048, BF), (5_000, 8192, BF), (5_000, 8190, F32),
             (4_000, 16400, BF), (4_000, 16401, F32)]


@pytest.mark.parametrize("rows,H,dtype", MANY_ROWS)
def test_layernorm_of_more_rows_than_a_launch_holds(m, rows, H, dtype):
    eps = 1e-5
    nb = m.moonep_save8_blocks(H)
    x = base.norm_rows(rows, H, dtype, H)
    gamma, beta = rand_tensor((H,), F32, 1), rand_tensor((H,), F32, 2)

    def call(x_):
        n = x_.shape[0]
        Y, codes = torch.empty_like(x_), torch.empty((n, H), dtype=torch.int8, device=DEV)
        mean, rstd = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
        exps = torch.empty((n, nb), dtype=torch.uint8, device=DEV)
        m.moonep_layernorm(m.make_dims(1, 1, 0, n, 1), H, x_, gamma, beta, eps, Y, mean, rstd, codes, exps)
        return Y, mean, rstd, codes, exps

    say("layernorm, many rows", rows, H, dtype)
    whole = call(x)
    # a row's bits do not depend on where in the launch it runs: pieces of 1500 rows run all at a time
    for at in range(0, rows, 1500):
        for w, piece in zip(whole, call(base.at_offset(x[at:at + 1500], 0))):
            assert torch.equal(w[at:at + 1500], piece), at
    # and the oracle, on the last rows
    Y, mean, rstd, codes, exps = (t[-96:] for t in whole)
    x64 = np64(x[-96:])
    ref, rm, rr, rz = norm8.layernorm(x64, np64(gamma), np64(beta), eps)
    dm = 57 * U * np.abs(x64).mean(axis=1)
    rv = rr ** -2 - eps
    assert np.all(np.abs(np64(mean) - rm) <= dm)
    assert np.all(np.abs(np64(rstd) / rr - 1) <= 40 * U + (dm ** 2 + 2 * U * (rv + dm ** 2)) * rr ** 2)
    zb = base.z_bound(x64, rm, rr, rz) + np.abs(rz) * ((dm * rr) ** 2)[:, None]
    g = np.abs(np64(gamma))
    tol = g * zb + U * (np.abs(rz) * g + np.abs(ref)) + base.half(dtype) * (np.abs(ref) + g * zb)
    assert np.all(np.abs(np64(Y) - ref) <= tol)
    st = norm8.steps(npi(exps), H)
    near = np.abs(rz) + zb > 127.5 * st
    assert np.all(np.abs(norm8.load8(npi(codes), npi(exps)) - rz) <= np.where(near, 1.0, 0.5) * st + zb)


@pytest.mark.parametrize("rows,H,dtype", MANY_ROWS)
def test_layernorm_dispatch_of_more_rows_than_a_launch_holds(m, rows, H, dtype):
    # bit for bit what the two calls give, two places a row
    K = 2
    d = m.make_dims(1, 4, 0, rows, K)
    nb = m.moonep_save8_blocks(H)
    x = base.norm_rows(rows, H, dtype, H)
    gamma, beta = rand_tensor((H,), F32, 1), rand_tensor((H,), F32, 2)
    g = torch.Generator().manual_seed(rows + H)
    dest = torch.randperm(rows * K, generator=g).to(torch.int32).to(DEV)
    outs = []
    for fused in (False, True):
        Xp = torch.empty((rows * K, H), dtype=dtype, device=DEV)
        mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
        codes = torch.empty((rows, H), dtype=torch.int8, device=DEV)
        exps = torch.empty((rows, nb), dtype=torch.uint8, device=DEV)
        say("layernorm_dispatch" if fused else "layernorm, dispatch", "many rows", rows, H, dtype)
        if fused:
            m.moonep_layernorm_dispatch(d, H, x, gamma, beta, 1e-5, dest, Xp, mean, rstd, codes, exps)
        else:
            Y = torch.empty_like(x)
            m.moonep_layernorm(d, H, x, gamma, beta, 1e-5, Y, mean, rstd, codes, exps)
            m.moonep_dispatch(d, H, Y, dest, Xp)
        torch.cuda.synchronize()
        outs.append((Xp, mean, rstd, codes, exps))
    assert all(torch.equal(a, b) for a, b in zip(*outs))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hp", [2056, 2561, 4104, 6145])  # a wave takes 2048 columns at a time: two and more passes
@pytest.mark.parametrize("gated", [True, False])
def test_swiglu_backward8_of_wide_rows(m, dtype, Hp, gated):
    base.test_swiglu_backward8(m, dtype, Hp, gated)


@pytest.mark.parametrize("up", [1.0, 1.2345678, -0.7654321])
def test_activation_over_every_sigmoid_denominator(m, up):
    # the sigmoid's denominator 1 + exp(-|g|) takes the float32 values of [1, 2]; with |g| = -log(k 2^-23), k from 1 to
    # 2^23, it takes (nearly) each of them, with either sign of g.  The activation with a checkpoint, which has its
    # own reciprocal for that range, must give the plain one's bits throughout
    n, Hp = 4096, 4096
    k = torch.arange(1, 2 ** 23 + 1, dtype=torch.float64, device=DEV)
    g = torch.log(k * 2.0 ** -23).to(F32)
    y = torch.empty((n, 2 * Hp), device=DEV)
    y[:, :Hp] = torch.cat([g, -g]).view(n, Hp)
    y[:, Hp:] = up
    d = m.make_dims(1, 1, 0, n, 1)
    a, b = torch.empty((n, Hp), device=DEV), torch.empty((n, Hp), device=DEV)
    codes = torch.empty((n, 2, Hp), dtype=torch.int8, device=DEV)
    exps = torch.empty((n, 2, Hp // 32), dtype=torch.uint8, device=DEV)
    say("swiglu and swiglu_save8, every denominator, up", up)
    m.moonep_swiglu(d, Hp, y, a)
    m.moonep_swiglu_save8(d, Hp, y, b, codes, exps)
    torch.cuda.synchronize()
    assert torch.equal(a.view(torch.int32), b.view(torch.int32))
