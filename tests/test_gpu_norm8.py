"""Parity of the layer norm and of the 8-bit checkpoint kernels against the float64 oracle (GPU).

Bounds, with u = 2^-24 (half a step of float32) and half = 2^-8 for bf16 results, u for float32 ones:
  * 8-bit rows: codes, exponents and values bit for bit (x / step and code * step are exact).
  * swiglu and its gradient: at most 12 float32 roundings behind each factor (exp's own error of 2 steps
    among them), so (16 u + half) |ref| and, where 1 + g (1 - s) crosses zero, 16 u times its terms' size;
    a gate's gradient is a sum of up to 1 + Hp / 64 terms a lane and 6 more additions.
  * the norm: a mean is a sum of at most 32 terms a lane, 6 additions across lanes and 16 across waves, and
    a division: 56 roundings of partial sums of size at most the sum of |x|.  So m is off by 56 u mean|x| at
    most, z by r times that and, from the variance (60 roundings, halved by the root), the root, the quotient
    and the product, by 40 u |z|; y adds u (|z gamma| + |y|) and its own rounding.
  * its gradient: each mean 56 u times the mean of magnitudes, the products and the three subtractions 8 u
    times the terms; dgamma and dbeta sums of `rows` terms: (rows + 32) u times the sum of magnitudes.
"""
import numpy as np
import pytest
import torch

from oracle import norm8
from oracle import planner as oplanner
from tests.gpu_util import DEV, Guarded, f32, i32, np64, npi, rand_tensor, say
from tests.plan_checks import random_routing

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def m():
    import load_balanced_dispatch_amd as mod
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    return mod


def half(dtype):
    return 2.0 ** -8 if dtype == BF else U


def at_offset(t, by):
    """A contiguous copy of t that starts `by` elements into its allocation."""
    buf = torch.empty(t.numel() + by + 64, dtype=t.dtype, device=DEV)
    v = buf[by:by + t.numel()].view(t.shape)
    v.copy_(t)
    return v


class Bytes:
    """Guarded uint8/int8 buffer of `shape`, `by` bytes off its alignment."""

    def __init__(self, shape, dtype, by=0):
        self.n, self.by = int(np.prod(shape)), by
        self.buf = torch.full((self.n + 1024 + by,), 0x5A, dtype=torch.uint8, device=DEV)
        self.view = self.buf[512 + by:512 + by + self.n].view(dtype).view(shape)

    def intact(self):
        lo, hi = self.buf[:512 + self.by], self.buf[512 + self.by + self.n:]
        return bool((lo == 0x5A).all()) and bool((hi == 0x5A).all())


def rows_of(shape, dtype, seed):
    """Rows with several binary orders of magnitude between blocks, a zero block and a constant one."""
    x = rand_tensor(shape, F32, seed)
    g = torch.Generator().manual_seed(seed + 1)
    s = torch.exp2(torch.randint(-20, 20, (shape[0], -(-shape[1] // 32)), generator=g).float()).to(DEV)
    x = x * s.repeat_interleave(32, 1)[:, :shape[1]]
    x[0, :32] = 0.0
    x[-1, -5:] = 1.0
    return x.to(dtype)



WIDTHS = [1, 7, 8, 31, 32, 33, 40, 100, 253, 256, 1408, 2049]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("C", WIDTHS)
def test_save8_and_load8_bit_for_bit(m, dtype, C):
    rows = 37
    x = rows_of((rows, C), dtype, C)
    nb = m.moonep_save8_blocks(C)
    rc, re = norm8.save8(np64(x))
    for by in (0, 1):  # by 1: rows off the wide accesses' alignment
        xo = at_offset(x, by)
        codes, exps = Bytes((rows, C), torch.int8, by), Bytes((rows, nb), torch.uint8, by)
        say("save8", dtype, C, "offset", by)
        m.moonep_save8(rows, C, xo, codes.view, exps.view)
        torch.cuda.synchronize()
        assert np.array_equal(npi(exps.view), re)
        assert np.array_equal(npi(codes.view), rc)
        assert codes.intact() and exps.intact()
        for out in (BF, F32):
            v = Guarded((rows, C), out)
            say("load8", out, C, "offset", by)
            m.moonep_load8(rows, C, codes.view, exps.view, v.view)
            torch.cuda.synchronize()
            assert np.array_equal(np64(v.view), norm8.load8(rc, re))
            assert v.intact()


def test_save8_extremes(m):
    big, tiny = 3.4028235e38, 1e-45
    x = torch.tensor([[0.0] * 40, [tiny] * 40, [1e-38] * 40, [-big] * 40, [1.0] * 31 + [float("inf")] + [2.0] * 8,
                      [3.0] * 39 + [float("nan")], [-127.75, 127.25, 126.5, 125.5, 64.0] * 8], device=DEV)
    rows, C = x.shape
    codes = torch.empty((rows, C), dtype=torch.int8, device=DEV)
    exps = torch.empty((rows, 2), dtype=torch.uint8, device=DEV)
    v = torch.empty((rows, C), device=DEV)
    say("save8 extremes")
    m.moonep_save8(rows, C, x, codes, exps)
    m.moonep_load8(rows, C, codes, exps, v)
    torch.cuda.synchronize()
    rc, re = norm8.save8(np64(x))
    assert np.array_equal(npi(exps), re)
    ref = norm8.load8(rc, re)
    assert np.array_equal(np64(v), ref, equal_nan=True)
    assert np.isnan(ref[4, :32]).all() and not np.isnan(ref[4, 32:]).any()
    assert np.isnan(ref[5, 32:]).all() and not np.isnan(ref[5, :32]).any()
    assert ref[6, :5].tolist() == [-127.0, 127.0, 126.0, 126.0, 64.0]


def test_denormal_blocks_in_bf16(m):
    # bf16 rows whose blocks reach below 2^-126: the codes, and the values written back as bf16 and float32
    x = (torch.arange(-32, 32, device=DEV).float() * 2.0 ** -131).to(BF).reshape(1, 64)
    x[0, 40] = 1.5 * 2.0 ** -127
    codes = torch.empty((1, 64), dtype=torch.int8, device=DEV)
    exps = torch.empty((1, 2), dtype=torch.uint8, device=DEV)
    m.moonep_save8(1, 64, x, codes, exps)
    rc, re = norm8.save8(np64(x))
    for out in (BF, F32):
        v = torch.empty((1, 64), dtype=out, device=DEV)
        m.moonep_load8(1, 64, codes, exps, v)
        torch.cuda.synchronize()
        # read as bits: the host may flush denormals in a conversion
        bits = v.view(torch.int16 if out == BF else torch.int32).cpu().numpy().astype(np.int64) & 0xFFFFFFFF
        got = (bits & 0xFFFF) << 16 if out == BF else bits
        got = got.astype(np.uint32).view(np.float32).astype(np.float64)
        assert np.array_equal(got, norm8.load8(rc, re))
    assert np.array_equal(npi(exps), re) and np.array_equal(npi(codes), rc)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hp", [1, 13, 32, 253, 256, 1408, 2048])
def test_swiglu_save8(m, dtype, Hp):
    d = m.make_dims(2, 4, 1, 11, 3)
    N = d.N
    y = rand_tensor((N, 2 * Hp), dtype, seed=Hp, std=3.0)
    nb = m.moonep_save8_blocks(Hp)
    for by in (0, 1):
        yo = at_offset(y, by)
        A = Guarded((N, Hp), dtype)
        codes, exps = Bytes((N, 2, Hp), torch.int8, by), Bytes((N, 2, nb), torch.uint8, by)
        say("swiglu_save8", dtype, Hp, "offset", by)
        m.moonep_swiglu_save8(d, Hp, yo, A.view, codes.view, exps.view)
        torch.cuda.synchronize()
        rc, re = norm8.save8(np64(y).reshape(2 * N, Hp))
        assert np.array_equal(npi(codes.view).reshape(2 * N, Hp), rc)
        assert np.array_equal(npi(exps.view).reshape(2 * N, nb), re)
        from oracle import layer as olayer
        ref = olayer.swiglu(np64(y))
        assert np.all(np.abs(np64(A.view) - ref) <= (16 * U + half(dtype)) * np.abs(ref))
        assert A.intact() and codes.intact() and exps.intact()


def _backward8_case(m, dtype, Hp, seed, R=2, E=4, S=11, K=3):
    rng = np.random.default_rng(seed)
    p = oplanner.plan(random_routing(rng, R, S, K, E, 1.0), E, 1)
    N = R * S * K
    src = np.empty(N, dtype=np.int64)
    src[p.dest_idx.reshape(-1)] = np.arange(N)
    gates = rng.dirichlet(np.ones(K), size=(R, S)).astype(np.float32)
    gates[0, 0, 0] = 0.0
    rc, re = norm8.save8(np64(rand_tensor((2 * N, Hp), dtype, seed, std=2.0)))
    dA = rand_tensor((N, Hp), dtype, seed + 1)
    codes = torch.as_tensor(rc.astype(np.int8), device=DEV)
    exps = torch.as_tensor(re.astype(np.uint8), device=DEV)
    return m.make_dims(R, E, 1, S, K), rc, re, codes, exps, dA, src, gates


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hp", [1, 13, 32, 253, 256, 520, 1408, 2048])
@pytest.mark.parametrize("gated", [True, False])
def test_swiglu_backward8(m, dtype, Hp, gated):
    d, rc, re, codes, exps, dA, src, gates = _backward8_case(m, dtype, Hp, 70 + Hp)
    N = d.N
    A, dY = Guarded((N, Hp), dtype), Guarded((N, 2 * Hp), dtype)
    dg = Guarded((d.R, d.S, d.K), F32)
    dg.view.fill_(7.0)
    by = Hp % 2  # the odd widths also with everything off its wide alignment
    say("swiglu_backward8", dtype, Hp, gated)
    m.moonep_swiglu_backward8(d, Hp, at_offset(codes, by), exps, at_offset(dA, by), i32(src) if gated else None,
                              f32(gates) if gated else None, A.view, dY.view, dg.view if gated else None)
    torch.cuda.synchronize()
    y = norm8.load8(rc, re).reshape(N, 2 * Hp)
    w = gates.astype(np.float64).reshape(-1)[src] if gated else np.ones(N)
    da = np64(dA)
    rA, rdY, rdg = norm8.swiglu_backward8(y, da, w)
    g, u = y[:, :Hp], y[:, Hp:]
    s = 1 / (1 + np.exp(-g))
    scale = np.concatenate([np.abs(da * u) * s * (1 + np.abs(g)), np.abs(da * g) * s], axis=1) * w[:, None]
    h = half(dtype)
    assert np.all(np.abs(np64(A.view) - rA) <= (16 * U + h) * np.abs(rA))
    assert np.all(np.abs(np64(dY.view) - rdY) <= h * np.abs(rdY) + 16 * U * scale)
    assert A.intact() and dY.intact() and dg.intact()
    if gated:
        terms = (np.abs(da) * np.abs(g * s * u)).sum(axis=1)
        got = np64(dg.view).reshape(-1)[src]
        assert np.all(np.abs(got - rdg) <= (16 + 8 * (Hp // 512 + 1) + 6) * U * terms)


def test_swiglu_backward8_rows_without_a_pair(m):
    # a row whose pair id is out of range counts as gate 0; the gates' gradients of pairs without a row stay
    d, rc, re, codes, exps, dA, src, gates = _backward8_case(m, BF, 64, 5)
    N = d.N
    src = src.copy()
    lost = [int(src[4]), int(src[9])]
    src[4], src[9] = -1, N
    A = torch.full((N, 64), 9.0, dtype=BF, device=DEV)
    dY = torch.full((N, 128), 9.0, dtype=BF, device=DEV)
    dg = torch.full((d.R, d.S, d.K), 7.0, device=DEV)
    say("swiglu_backward8 rows without a pair")
    m.moonep_swiglu_backward8(d, 64, codes, exps, dA, i32(src), f32(gates), A, dY, dg)
    torch.cuda.synchronize()
    assert not np64(A)[[4, 9]].any() and not np64(dY)[[4, 9]].any()
    got = np64(dg).reshape(-1)
    assert np.all(got[lost] == 7.0) and (got == 7.0).sum() == 2


def test_swiglu_backward8_nan_block(m):
    # a block that held an infinity makes its own row's gradients NaN, and no other row's
    d, rc, re, codes, exps, dA, src, gates = _backward8_case(m, F32, 45, 6)
    exps = exps.clone()
    exps[2 * 3 + 1, 1] = 255  # row 3, up half, its short last block
    A = torch.empty((d.N, 45), device=DEV)
    dY = torch.empty((d.N, 90), device=DEV)
    dg = torch.empty((d.R, d.S, d.K), device=DEV)
    m.moonep_swiglu_backward8(d, 45, codes, exps, dA, i32(src), f32(gates), A, dY, dg)
    torch.cuda.synchronize()
    bad = np.isnan(np64(dY)).any(axis=1)
    assert np.nonzero(bad)[0].tolist() == [3]
    assert np.isnan(np64(A)[3, 32:]).all() and not np.isnan(np64(A)[3, :32]).any()
    assert np.nonzero(np.isnan(np64(dg).reshape(-1)))[0].tolist() == [int(src[3])]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H", [1, 9, 32, 100, 253, 512, 520, 2048, 7168])
@pytest.mark.parametrize("affine", ["both", "gamma", "none"])
def test_dispatch8(m, dtype, H, affine):
    R, E, S, K = 2, 4, 9, 3
    rng = np.random.default_rng(H)
    p = oplanner.plan(random_routing(rng, R, S, K, E, 1.0), E, 1)
    d = m.make_dims(R, E, 1, S, K)
    rc, re = norm8.save8(np64(rows_of((R * S, H), dtype, H)))
    gamma = rand_tensor((H,), F32, 1) if affine != "none" else None
    beta = rand_tensor((H,), F32, 2) if affine == "both" else None
    Xp = Guarded((d.N, H), dtype)
    by = H % 2
    say("dispatch8", dtype, H, affine)
    m.moonep_dispatch8(d, H, at_offset(torch.as_tensor(rc.astype(np.int8), device=DEV), by),
                       torch.as_tensor(re.astype(np.uint8), device=DEV), gamma, beta, i32(p.dest_idx), Xp.view)
    torch.cuda.synchronize()
    v = norm8.load8(rc, re).reshape(R, S, H)
    g64 = None if gamma is None else np64(gamma)
    b64 = None if beta is None else np64(beta)
    ref = norm8.dispatch8(v, g64, b64, p.dest_idx)
    # one fused multiply-add and one rounding to the row type (none without gamma: bf16 holds the values)
    bound = 0.0 if affine == "none" else (U + half(dtype)) * np.abs(ref)
    assert np.all(np.abs(np64(Xp.view) - ref) <= bound)
    assert Xp.intact()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,K", [(1, 1), (9, 2), (253, 3), (520, 12), (2048, 6)])
def test_combine_backward_ungated(m, dtype, D, K):
    R, E, S = 2, 16, 9
    rng = np.random.default_rng(D)
    p = oplanner.plan(random_routing(rng, R, S, K, E, 1.0), E, 1)
    d = m.make_dims(R, E, 1, S, K)
    dest = p.dest_idx.copy()
    gone = int(dest[1, 2, 0])
    dest[1, 2, 0] = -1
    dout = rand_tensor((R, S, D), F32, D)
    out = Guarded((d.N, D), dtype)
    out.view.fill_(3.0)
    say("combine_backward_ungated", dtype, D, K)
    m.moonep_combine_backward_ungated(d, D, at_offset(dout, D % 2), i32(dest), out.view)
    torch.cuda.synchronize()
    ref = norm8.combine_backward_ungated(dout.to(dtype).double().cpu().numpy(), p.dest_idx)
    ref[gone] = 3.0
    assert np.array_equal(np64(out.view), ref)
    assert out.intact()


# ------------------------------------------------------------------ layer norm

# forward: a wave per row with 1 and 2 chunks a lane, a block per row with 1 (three waves), 2 and 4; backward: a wave per
# row with 1, 2 and 4, groups of waves, a block per row with 2, 4 and 8; odd widths among them
NORM_WIDTHS = [1, 2, 7, 8, 33, 128, 253, 512, 513, 1000, 1024, 1413, 2048, 2056, 2500, 7168, 16384, 16392, 20001,
               32768]


def norm_rows(rows, H, dtype, seed):
    """Rows at several offsets and scales, one constant and one of zeros."""
    x = rand_tensor((rows, H), F32, seed)
    x = x * torch.tensor([1.0, 30.0, 0.01], device=DEV).repeat(rows)[:rows, None]
    x = x + torch.tensor([0.0, -5.0, 3.0, 100.0], device=DEV).repeat(rows)[:rows, None]
    x[min(1, rows - 1)] = 2.5
    x[min(4, rows - 1)] = 0.0
    return x.to(dtype)


def z_bound(x, m_, r, z):
    return 57 * U * r[:, None] * np.abs(x).mean(axis=1, keepdims=True) + 40 * U * np.abs(z)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H", NORM_WIDTHS)
def test_layernorm(m, dtype, H):
    R, S = 3, 3
    rows = R * S
    d = m.make_dims(R, R, 0, S, 1)
    nb = m.moonep_save8_blocks(H)
    x = norm_rows(rows, H, dtype, H)
    gamma, beta = rand_tensor((H,), F32, 1), rand_tensor((H,), F32, 2)
    eps = 1e-5
    ref, rm, rr, rz = norm8.layernorm(np64(x), np64(gamma), np64(beta), eps)
    for by, save in ((0, True), (1, True), (0, False)):
        Y, mean, rstd = Guarded((rows, H), dtype), Guarded((rows,), F32), Guarded((rows,), F32)
        codes, exps = Bytes((rows, H), torch.int8, by), Bytes((rows, nb), torch.uint8, by)
        say("layernorm", dtype, H, "offset", by, "save", save)
        m.moonep_layernorm(d, H, at_offset(x, by), gamma, beta, eps, Y.view, mean.view, rstd.view,
                           codes.view if save else None, exps.view if save else None)
        torch.cuda.synchronize()
        assert Y.intact() and mean.intact() and rstd.intact() and codes.intact() and exps.intact()
        x64 = np64(x)
        assert np.all(np.abs(np64(mean.view) - rm) <= 57 * U * np.abs(x64).mean(axis=1))
        zb = z_bound(x64, rm, rr, rz)
        # the variance sees the mean's error squared and the centred values' roundings
        dm = 57 * U * np.abs(x64).mean(axis=1)
        rv = rr ** -2 - eps
        assert np.all(np.abs(np64(rstd.view) / rr - 1) <= 40 * U + (dm ** 2 + 2 * U * (rv + dm ** 2)) * rr ** 2)
        zb = zb + np.abs(rz) * ((dm * rr) ** 2)[:, None]
        g = np.abs(np64(gamma))
        tol = g * zb + U * (np.abs(rz) * g + np.abs(ref)) + half(dtype) * (np.abs(ref) + g * zb)
        assert np.all(np.abs(np64(Y.view) - ref) <= tol)
        if save:
            v = norm8.load8(npi(codes.view), npi(exps.view))
            st = norm8.steps(npi(exps.view), H)
            near = np.abs(rz) + zb > 127.5 * st
            assert np.all(np.abs(v - rz) <= np.where(near, 1.0, 0.5) * st + zb)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,K", [(1, 1), (40, 3), (253, 2), (512, 9), (1000, 4), (1413, 3), (2048, 6), (7168, 2),
                                 (16392, 2)])
def test_layernorm_dispatch_is_the_two_calls(m, dtype, H, K):
    # bit for bit: the rows, the statistics and the checkpoint; rows without a destination are left alone
    R, S, E = 2, 9, 16
    p = oplanner.plan(random_routing(np.random.default_rng(H), R, S, K, E, 1.0), E, 1)
    d = m.make_dims(R, E, 1, S, K)
    dest = p.dest_idx.copy()
    gone = int(dest[1, 3, 0])
    dest[1, 3, 0] = -1
    dest = i32(dest)
    x = norm_rows(R * S, H, dtype, H)
    gamma, beta = rand_tensor((H,), F32, 1), rand_tensor((H,), F32, 2)
    nb = m.moonep_save8_blocks(H)
    for by in (0, 1):
        xo = at_offset(x, by)
        outs = []
        for fused in (False, True):
            Xp = Guarded((d.N, H), dtype)
            Xp.view.fill_(3.0)
            mean, rstd = Guarded((R * S,), F32), Guarded((R * S,), F32)
            codes, exps = Bytes((R * S, H), torch.int8, by), Bytes((R * S, nb), torch.uint8, by)
            tail = (mean.view, rstd.view, codes.view, exps.view)
            say("layernorm_dispatch" if fused else "layernorm, dispatch", dtype, H, K, "offset", by)
            if fused:
                m.moonep_layernorm_dispatch(d, H, xo, gamma, beta, 1e-5, dest, Xp.view, *tail)
            else:
                Y = torch.empty((R * S, H), dtype=dtype, device=DEV)
                m.moonep_layernorm(d, H, xo, gamma, beta, 1e-5, Y, *tail)
                m.moonep_dispatch(d, H, Y, dest, Xp.view)
            torch.cuda.synchronize()
            assert all(b.intact() for b in (Xp, mean, rstd, codes, exps))
            outs.append((Xp.view, *tail))
        assert all(torch.equal(a, b) for a, b in zip(*outs))
        assert bool((outs[1][0][gone] == 3.0).all())
    Xp = torch.empty((d.N, H), dtype=dtype, device=DEV)
    m.moonep_layernorm_dispatch(d, H, x, gamma, None, 1e-5, i32(p.dest_idx), Xp, None, None)
    Y = torch.empty((R * S, H), dtype=dtype, device=DEV)
    m.moonep_layernorm(d, H, x, gamma, None, 1e-5, Y, None, None)
    torch.cuda.synchronize()
    assert torch.equal(Xp[torch.as_tensor(p.dest_idx.reshape(-1), device=DEV)], Y.repeat_interleave(K, 0))


@pytest.mark.parametrize("H", [40, 253, 2048, 7168])
def test_layernorm_checkpoint_is_save8_of_its_rows(m, H):
    # with weight 1 and no bias the float32 output is z itself, and the codes must be its 8-bit rows
    rows = 6
    d = m.make_dims(1, 1, 0, rows, 1)
    x = norm_rows(rows, H, F32, 3 * H)
    Y = torch.empty((rows, H), device=DEV)
    codes = torch.empty((rows, H), dtype=torch.int8, device=DEV)
    exps = torch.empty((rows, m.moonep_save8_blocks(H)), dtype=torch.uint8, device=DEV)
    say("layernorm checkpoint", H)
    m.moonep_layernorm(d, H, x, torch.ones(H, device=DEV), None, 1e-5, Y, None, None, codes, exps)
    torch.cuda.synchronize()
    rc, re = norm8.save8(np64(Y))
    assert np.array_equal(npi(exps), re) and np.array_equal(npi(codes), rc)


@pytest.mark.parametrize("dtype", [BF, F32, "8"])
@pytest.mark.parametrize("H", NORM_WIDTHS)
def test_layernorm_backward(m, dtype, H):
    # few rows: one launch
    backward_case(m, dtype, H, 3, 7 if H > 4096 else 43)


@pytest.mark.parametrize("dtype", [BF, F32, "8"])
@pytest.mark.parametrize("H", [1, 7, 64, 253, 512, 1000, 1024, 1413, 2048, 2500, 2560, 4096, 7168, 8192, 16384, 20001, 32768])
def test_layernorm_backward_more_rows(m, dtype, H):
    # more than 512 rows: the rows' blocks leave partial sums, a second launch folds them
    backward_case(m, dtype, H, 3, 173)


@pytest.mark.parametrize("rows", [1, 2, 63, 64, 65, 256, 257, 511, 512, 513, 1027, 2051])
@pytest.mark.parametrize("H", [72, 520, 1100, 1413, 2050, 2560, 2564])
def test_layernorm_backward_row_counts(m, rows, H):
    backward_case(m, BF, H, 1, rows)


def backward_case(m, dtype, H, R, S):
    rows = R * S
    d = m.make_dims(R, R, 0, S, 1)
    x = norm_rows(rows, H, F32 if dtype == "8" else dtype, H)
    gamma, dY = rand_tensor((H,), F32, 1), rand_tensor((rows, H), F32, 2)
    _, rm, rr, rz = norm8.layernorm(np64(x), np64(gamma), None, 1e-3)
    mean, rstd = f32(rm), f32(rr)
    if dtype == "8":
        rc, re = norm8.save8(rz.astype(np.float32))
        z = norm8.load8(rc, re)
        rc, re = torch.as_tensor(rc.astype(np.int8), device=DEV), torch.as_tensor(re.astype(np.uint8), device=DEV)
    else:
        z = (np64(x) - np64(mean)[:, None]) * np64(rstd)[:, None]
    r = np64(rstd)
    dx, dg, db = norm8.layernorm_backward(np64(dY), z, r, np64(gamma))
    ws = torch.empty(m.moonep_layernorm_backward_workspace_bytes(d, H), dtype=torch.uint8, device=DEV)
    dg0, db0 = rand_tensor((H,), F32, 5), rand_tensor((H,), F32, 6)
    for by, bias in ((0, True), (1, True), (0, False)):
        dX, dgam, dbet = Guarded((rows, H), F32), Guarded((H,), F32), Guarded((H,), F32)
        dgam.view.copy_(dg0)
        dbet.view.copy_(db0)
        say("layernorm_backward", dtype, H, "offset", by, "bias", bias)
        tail = (rstd, gamma, dX.view, dgam.view, dbet.view if bias else None, ws)
        if dtype == "8":
            m.moonep_layernorm_backward8(d, H, at_offset(dY, by), at_offset(rc, by), re, *tail)
        else:
            m.moonep_layernorm_backward(d, H, at_offset(dY, by), at_offset(x, by), mean, *tail)
        torch.cuda.synchronize()
        assert dX.intact() and dgam.intact() and dbet.intact()
        gy = np.abs(np64(dY) * np64(gamma))
        terms = gy + gy.mean(axis=1, keepdims=True) + np.abs(z) * (gy * np.abs(z)).mean(axis=1, keepdims=True)
        assert np.all(np.abs(np64(dX.view) - dx) <= (57 + 8) * U * r[:, None] * terms)
        sums = ((dgam.view, dg, dg0, np64(dY) * z), (dbet.view, db, db0, np64(dY)))
        for got, ref, start, each in sums[:2 if bias else 1]:
            bound = (rows + 32) * U * np.abs(each).sum(axis=0) + U * np.abs(ref + np64(start))
            assert np.all(np.abs(np64(got) - ref - np64(start)) <= bound)
        if not bias:
            assert np.array_equal(np64(dbet.view), np64(db0))


def test_layernorm_backward_many_rows_is_deterministic(m):
    # more rows than blocks: every block sums several rows, and a second run gives the same bits
    R, S, H = 4, 2500, 72
    d = m.make_dims(R, R, 0, S, 1)
    rows = R * S
    x, dY = norm_rows(rows, H, BF, 1), rand_tensor((rows, H), F32, 2)
    gamma = rand_tensor((H,), F32, 3)
    _, rm, rr, _ = norm8.layernorm(np64(x), np64(gamma), None, 1e-3)
    mean, rstd = f32(rm), f32(rr)
    ws = torch.empty(m.moonep_layernorm_backward_workspace_bytes(d, H), dtype=torch.uint8, device=DEV)
    outs = []
    for _ in range(2):
        dX, dg, db = torch.empty((rows, H), device=DEV), torch.zeros(H, device=DEV), torch.zeros(H, device=DEV)
        ws.fill_(0xFF)
        say("layernorm_backward many rows")
        m.moonep_layernorm_backward(d, H, dY, x, mean, rstd, gamma, dX, dg, db, ws)
        torch.cuda.synchronize()
        outs.append((dX, dg, db))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    z = (np64(x) - np64(mean)[:, None]) * np64(rstd)[:, None]
    _, dg, db = norm8.layernorm_backward(np64(dY), z, np64(rstd), np64(gamma))
    for got, ref, each in ((outs[0][1], dg, np64(dY) * z), (outs[0][2], db, np64(dY))):
        assert np.all(np.abs(np64(got) - ref) <= (rows + 32) * U * np.abs(each).sum(axis=0))


def test_layernorm_gradient_is_the_forwards_difference(m):
    # a float32 forward at x + h v and x - h v: the loss's difference over 2 h against <dX, v>.  The central
    # difference is off by h^2/6 times the third derivative (of order r^3: here r ~ 1, |v| = 1 a row) and by the
    # forwards' roundings, 60 u |dy y| over h: with h = 0.02, 1e-4 and 2e-4 of sqrt(H) |dy||y| per row.
    R, S, H = 2, 4, 256
    d = m.make_dims(R, R, 0, S, 1)
    rows = R * S
    x, dY, v = (rand_tensor((rows, H), F32, s) for s in (1, 2, 3))
    v = v / v.norm(dim=1, keepdim=True)
    gamma, beta = rand_tensor((H,), F32, 4), rand_tensor((H,), F32, 5)
    h = 0.02
    Y, mean, rstd = (torch.empty(s, device=DEV) for s in ((rows, H), (rows,), (rows,)))

    def loss(t):
        m.moonep_layernorm(d, H, t.contiguous(), gamma, beta, 1e-5, Y, None, None)
        return (dY.double() * Y.double()).sum(dim=1)

    diff = (loss(x + h * v) - loss(x - h * v)) / (2 * h)
    m.moonep_layernorm(d, H, x, gamma, beta, 1e-5, Y, mean, rstd)
    dX, dg, db = torch.empty((rows, H), device=DEV), torch.zeros(H, device=DEV), torch.zeros(H, device=DEV)
    ws = torch.empty(m.moonep_layernorm_backward_workspace_bytes(d, H), dtype=torch.uint8, device=DEV)
    m.moonep_layernorm_backward(d, H, dY, x, mean, rstd, gamma, dX, dg, db, ws)
    got = (dX.double() * v.double()).sum(dim=1)
    scale = dY.double().norm(dim=1) * gamma.double().abs().max()
    assert bool(((got - diff).abs() <= 1e-3 * scale).all())


def test_layernorm_not_finite_stays_in_its_row(m):
    R, S, H = 2, 3, 100
    d = m.make_dims(R, R, 0, S, 1)
    x = norm_rows(6, H, BF, 1)
    x[2, 17] = float("inf")
    x[5, 99] = float("nan")
    Y = torch.empty((6, H), dtype=BF, device=DEV)
    codes = torch.empty((6, H), dtype=torch.int8, device=DEV)
    exps = torch.empty((6, 4), dtype=torch.uint8, device=DEV)
    rstd = torch.empty(6, device=DEV)
    m.moonep_layernorm(d, H, x, torch.ones(H, device=DEV), None, 1e-5, Y, None, rstd, codes, exps)
    torch.cuda.synchronize()
    bad = np.isnan(np64(Y)).all(axis=1)
    assert np.nonzero(bad)[0].tolist() == [2, 5] and not np.isnan(np64(Y)[~bad]).any()
    assert (npi(exps)[[2, 5]] == 255).all() and (npi(exps)[[0, 1, 3, 4]] < 255).all()


def test_calls_on_another_stream(m):
    # inputs made on the default stream, the calls on another one that waits for them
    R, S, H = 2, 64, 512
    d = m.make_dims(R, R, 0, S, 1)
    x = norm_rows(R * S, H, BF, 1)
    gamma = rand_tensor((H,), F32, 2)
    outs = []
    for other in (False, True):
        st = torch.cuda.Stream() if other else torch.cuda.current_stream()
        Y = torch.empty((R * S, H), dtype=BF, device=DEV)
        codes = torch.empty((R * S, H), dtype=torch.int8, device=DEV)
        exps = torch.empty((R * S, H // 32), dtype=torch.uint8, device=DEV)
        v = torch.empty((R * S, H), dtype=BF, device=DEV)
        if other:
            st.wait_stream(torch.cuda.current_stream())
        m.moonep_layernorm(d, H, x, gamma, None, 1e-5, Y, None, None, codes, exps, stream=st)
        m.moonep_load8(R * S, H, codes, exps, v, stream=st)
        torch.cuda.synchronize()
        outs.append((Y, v))
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_binding_checks_on_device_tensors(m):
    d = m.make_dims(2, 4, 0, 4, 1)
    x = torch.zeros((8, 16), dtype=BF, device=DEV)
    g = torch.zeros(16, device=DEV)
    with pytest.raises(ValueError, match="codes must be"):
        m.moonep_save8(8, 16, x, x, torch.zeros((8, 1), dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="exps must hold 8"):
        m.moonep_save8(8, 16, x, torch.zeros((8, 16), dtype=torch.int8, device=DEV),
                       torch.zeros((9, 1), dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="contiguous"):
        m.moonep_layernorm(d, 16, x.t(), g, None, 1e-5, x, None, None)
    with pytest.raises(ValueError, match="gamma must be"):
        m.moonep_layernorm(d, 16, x, g.to(BF), None, 1e-5, x, None, None)
    with pytest.raises(m.MoonepError, match="go together"):
        m.moonep_layernorm(d, 16, x, g, None, 1e-5, torch.empty_like(x), None, None,
                           torch.empty((8, 16), dtype=torch.int8, device=DEV))
    with pytest.raises(ValueError, match="workspace too small"):
        m.moonep_layernorm_backward(d, 16, torch.zeros((8, 16), device=DEV), x, torch.zeros(8, device=DEV),
                                    torch.zeros(8, device=DEV), g, torch.zeros((8, 16), device=DEV), g.clone(),
                                    None, torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="unsupported dtype"):
        m.moonep_load8(8, 16, torch.zeros((8, 16), dtype=torch.int8, device=DEV),
                       torch.zeros((8, 1), dtype=torch.uint8, device=DEV), torch.empty((8, 16), dtype=torch.float16,
                                                                                       device=DEV))
