"""Parity of the 4-bit weights and of the expert layer for few tokens against the float64 oracle (GPU).

Bounds, with u = 2^-24.  4-bit codes and scales, and the float32 values that they stand for: equal; bfloat16 values: half a
step, 2^-8.  A product of rows of H elements and its sum over K: products of the operands' bits are exact in a matrix
instruction, every addition rounds (up to 2 u where an instruction cuts off instead) a partial sum that is at most the sum
of the terms' magnitudes, so 2 (H + K + 16) u times that sum.  With 4-bit weights the terms that are added are x times a
code plus 24 and x times 24 (at most 32 + 24 steps), times the scale.  The whole layer: tests take the three products'
errors through the activation as oracle.few.few_ffn does, the two projections with the longer row's unit.
"""
import numpy as np
import pytest
import torch

from oracle import few
from tests.gpu_util import DEV, Guarded, f32, i32, np64, npi, rand_tensor, say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def m():
    import load_balanced_dispatch_amd as mod
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    return mod


def off_by(t, by):
    """A contiguous copy of t that starts `by` elements into its allocation."""
    buf = torch.empty(t.numel() + by + 64, dtype=t.dtype, device=DEV)
    v = buf[by:by + t.numel()].view(t.shape)
    v.copy_(t)
    return v


def workspace(m, d, H, Hp):
    """A guarded workspace, full of NaN."""
    w = Guarded((m.moonep_few_workspace_bytes(d, H, Hp) // 4,), torch.int32)
    w.view.fill_(-1)
    return w


def routing(T, E, K, seed, one=None):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:K] for _ in range(T)])
    if one is not None:  # every token chooses it
        for t in range(T):
            if one not in ids[t]:
                ids[t, t % K] = one
    gates = rng.random((T, K)).astype(np.float32)
    return ids, gates / gates.sum(1, keepdims=True)


# ------------------------------------------------------------------ 4-bit weights

def weights_of(shape, dtype, seed):
    """Weights over many binary orders from column to column, with zero, constant and tiny columns."""
    w = rand_tensor(shape, F32, seed)
    g = torch.Generator().manual_seed(seed + 1)
    w = w * torch.exp2(torch.randint(-20, 20, (shape[0], 1, shape[2]), generator=g).float()).to(DEV)
    w[0, :, 0] = 0.0
    w[-1, :, -1] = 1.0
    if shape[2] > 2:
        w[0, :, 1] *= 2.0 ** -140  # denormal: scales of a few steps, or 0
    return w.to(dtype)


SHAPES4 = [(1, 1, 1), (2, 7, 3), (1, 8, 5), (3, 31, 16), (2, 32, 64), (1, 33, 100), (2, 64, 257), (1, 100, 8),
           (2, 128, 128), (1, 129, 31), (3, 200, 66), (1, 1408, 256), (2, 253, 512)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("E,H,N", SHAPES4)
def test_save4_and_load4(m, dtype, E, H, N):
    w = weights_of((E, H, N), dtype, seed=H + N)
    for G in (32, 64, 128):
        rc, rs = few.save4(np64(w), G)
        for by in (0, 1):
            codes = Guarded((E, -(-H // 8), N), torch.int32)
            scales = Guarded((E, -(-H // G), N), BF)
            wo = off_by(w, by)
            say("save4", dtype, E, H, N, G, "offset", by)
            m.moonep_save4(E, H, N, G, wo, codes.view, scales.view)
            torch.cuda.synchronize()
            assert np.array_equal(np64(scales.view), rs)
            words = codes.view.cpu().numpy()
            assert np.array_equal(few.unpack4(words, H), rc)
            assert np.array_equal(words, few.pack4(rc))  # rows past H hold the code 0
            assert codes.intact() and scales.intact()
            for out in (BF, F32):
                v = Guarded((E, H, N), out)
                co, so = off_by(codes.view, by), off_by(scales.view, by)
                say("load4", out, "offset", by)
                m.moonep_load4(E, H, N, G, co, so, v.view)
                torch.cuda.synchronize()
                ref = few.load4(rc, rs, G)
                if out == F32:
                    assert np.array_equal(np64(v.view), ref.astype(np.float32))
                else:
                    assert np.array_equal(np64(v.view), np64(torch.tensor(ref, dtype=F32).to(BF)))
                assert v.intact()


def test_save4_not_finite(m):
    w = torch.ones(1, 70, 6, device=DEV)
    w[0, 3, 0], w[0, 40, 1], w[0, 69, 2], w[0, 0, 3] = float("inf"), float("nan"), float("-inf"), few.LARGEST
    codes = torch.empty((1, 9, 6), dtype=torch.int32, device=DEV)
    scales = torch.empty((1, 3, 6), dtype=BF, device=DEV)
    v = torch.empty((1, 70, 6), device=DEV)
    say("save4 not finite")
    m.moonep_save4(1, 70, 6, 32, w, codes, scales)
    m.moonep_load4(1, 70, 6, 32, codes, scales, v)
    torch.cuda.synchronize()
    rc, rs = few.save4(np64(w), 32)
    assert np.array_equal(np64(v), few.load4(rc, rs, 32).astype(np.float32), equal_nan=True)
    nan = torch.isnan(v[0])
    assert nan[:32, 0].all() and nan[32:64, 1].all() and nan[64:, 2].all() and nan.sum() == 32 + 32 + 6
    assert torch.isfinite(v[0, :, 3]).all()


# ------------------------------------------------------------------ the layer

def four(W, G):
    """4-bit weights of float64 values: what the calls take, their values and the size of what is added for them."""
    codes, scales = few.save4(W, G)
    rng = np.random.default_rng(codes.size)
    codes = np.where(rng.random(codes.shape) < 0.02, -8, codes)  # also the code that save4 never writes
    words = few.pack4(codes)
    if W.shape[1] % 8:  # rows past H hold whatever they hold
        words[:, -1] ^= np.int32(sum(5 << (4 * (i // 2) + 16 * (i % 2)) for i in range(W.shape[1] % 8, 8)) & 0x7FFFFFFF)
    tensors = (torch.as_tensor(words).to(DEV), torch.tensor(scales, dtype=F32).to(BF).to(DEV))
    steps = np.repeat(scales, G, axis=1)[:, :W.shape[1]]
    return tensors, few.load4(codes, scales, G), 56 * steps


class Case:
    """Inputs of a layer and its results in float64."""

    def __init__(self, m, T, E, K, H, Hp, dtype, bits, seed=0, G=32, one=None, R=1, gates=True):
        rng = np.random.default_rng(seed)
        self.m, self.d, self.H, self.Hp, self.G, self.bits = m, m.make_dims(R, E, 0, T // R, K), H, Hp, G, bits
        self.T, self.K, self.dtype = T, K, dtype
        self.ids, self.g = routing(T, E, K, seed, one)
        if not gates:
            self.g = np.ones((T, K), np.float32)
        self.gates = f32(self.g) if gates else None
        self.X = rand_tensor((T, H), dtype, seed)
        mk = lambda rows, cols, s: rand_tensor((E, rows, cols), dtype if bits == 16 else F32, s, 1 / np.sqrt(rows))  # noqa: E731
        self.w = {"w": mk(H, Hp, seed + 1), "gu": mk(H, 2 * Hp, seed + 2), "down": mk(Hp, H, seed + 3)}
        self.values, self.size = {}, {}
        for k, w in self.w.items():
            if bits == 4:
                self.w[k], self.values[k], self.size[k] = four(np64(w), G)
            else:
                self.values[k] = np64(w)
                self.size[k] = np.abs(self.values[k])

    def layer(self, X=None, stream=None, ws=None, out=None):
        d, H, Hp, m = self.d, self.H, self.Hp, self.m
        X = self.X if X is None else X
        out = Guarded((self.T, Hp), F32) if out is None else out
        ws = ws or workspace(m, d, H, Hp)
        out.view.fill_(float("nan"))
        say("few_layer", self.bits, self.dtype, d, H, Hp, self.G)
        if self.bits == 4:
            m.moonep_few_layer4(d, H, Hp, self.G, X, i32(self.ids), self.gates, *self.w["w"], out.view, ws.view, stream)
        else:
            m.moonep_few_layer(d, H, Hp, X, i32(self.ids), self.gates, self.w["w"], out.view, ws.view, stream)
        torch.cuda.synchronize()
        assert out.intact() and ws.intact()
        return out.view

    def ffn(self, X=None, stream=None, ws=None):
        d, H, Hp, m = self.d, self.H, self.Hp, self.m
        X = self.X if X is None else X
        out = Guarded((self.T, H), F32)
        ws = ws or workspace(m, d, H, Hp)
        out.view.fill_(float("nan"))
        say("few_ffn", self.bits, self.dtype, d, H, Hp, self.G)
        if self.bits == 4:
            m.moonep_few_ffn4(d, H, Hp, self.G, X, i32(self.ids), self.gates, *self.w["gu"], *self.w["down"], out.view,
                              ws.view, stream)
        else:
            m.moonep_few_ffn(d, H, Hp, X, i32(self.ids), self.gates, self.w["gu"], self.w["down"], out.view, ws.view,
                             stream)
        torch.cuda.synchronize()
        assert out.intact() and ws.intact()
        return out.view

    def check(self, what=("layer", "ffn")):
        x = np64(self.X)
        if "layer" in what:
            size = {e: self.size["w"][e] for e in range(self.d.E)}
            ref, _ = few.few_layer(x, self.ids, self.g, self.values["w"])
            scale = few.few_layer(np.abs(x), self.ids, np.abs(self.g), size)[0]
            err = np.abs(np64(self.layer()) - ref)
            bound = 2 * (self.H + self.K + 16) * U * scale
            assert np.all(err <= bound), float((err / np.maximum(bound, 1e-300)).max())
        if "ffn" in what:
            self.check_ffn(x)

    def check_ffn(self, x):
        # the sizes go with the expert: few_ffn asks for them by its weights
        by = {id(self.values[k][e]): self.size[k][e] for k in ("gu", "down") for e in range(self.d.E)}
        rows = {k: [self.values[k][e] for e in range(self.d.E)] for k in ("gu", "down")}
        by = {id(w): s for k in rows for w, s in zip(rows[k], self.size[k])}
        unit = 2 * (max(self.H, self.Hp) + self.K + 16) * U
        ref, bound = few.few_ffn(x, self.ids, self.g, rows["gu"], rows["down"], unit, lambda w: by[id(w)],
                                 lambda w: by[id(w)])
        err = np.abs(np64(self.ffn()) - ref)
        assert np.all(err <= bound), float((err / np.maximum(bound, 1e-300)).max())


DTYPES = [(BF, 16), (F32, 16), (BF, 4), (F32, 4)]
# T, E, K, H, Hp
LAYERS = [(1, 1, 1, 1, 1), (1, 2, 2, 7, 3), (3, 4, 2, 8, 8), (2, 5, 3, 31, 9), (5, 8, 2, 32, 16), (4, 3, 1, 33, 17),
          (1, 16, 8, 64, 64), (16, 4, 2, 65, 65), (17, 3, 2, 100, 127), (8, 16, 4, 128, 128), (3, 6, 2, 253, 130),
          (33, 5, 3, 96, 40), (2, 4, 2, 1413, 259), (64, 8, 2, 72, 136), (1, 4, 2, 2048, 1408)]
# enough tiles for wide ones and for few waves to each; more than 64 pairs with more experts yet; more than 8 and 16 choices
LAYERS += [(40, 64, 2, 64, 1030), (40, 48, 2, 70, 1030), (40, 64, 2, 1030, 40), (40, 48, 2, 1100, 70), (40, 100, 2, 65, 70),
           (3, 16, 11, 40, 24), (6, 16, 11, 40, 24), (2, 20, 17, 33, 20), (4, 20, 16, 33, 20)]


@pytest.mark.parametrize("dtype,bits", DTYPES)
@pytest.mark.parametrize("T,E,K,H,Hp", LAYERS)
def test_sizes(m, dtype, bits, T, E, K, H, Hp):
    Case(m, T, E, K, H, Hp, dtype, bits, seed=H, G=(32, 64, 128)[H % 3]).check()


@pytest.mark.parametrize("dtype,bits", DTYPES)
@pytest.mark.parametrize("T,K", [(16, 2), (17, 2), (64, 1), (65, 2), (128, 8), (200, 3)])
def test_one_expert_takes_every_token(m, dtype, bits, T, K):
    Case(m, T, 9, K, 96, 48, dtype, bits, seed=T, one=4).check()


@pytest.mark.parametrize("bits", [16, 4])
def test_group_sizes_and_tails(m, bits):
    for H, Hp, G in ((127, 24, 64), (128, 24, 64), (129, 40, 128), (257, 72, 128), (191, 33, 32)):
        Case(m, 3, 4, 2, H, Hp, BF, bits, seed=H, G=G).check()


@pytest.mark.parametrize("dtype,bits", DTYPES)
def test_invalid_and_repeated_ids(m, dtype, bits):
    c = Case(m, 6, 5, 3, 70, 33, dtype, bits, seed=1)
    c.ids = np.array([[0, 1, 2], [-1, 3, 5], [-1, -2 ** 31, 2 ** 31 - 1], [4, 4, 4], [1, 1, 0], [5, 6, -1]])
    c.check()
    assert not c.layer()[[2, 5]].any() and not c.ffn()[[2, 5]].any()


@pytest.mark.parametrize("dtype,bits", DTYPES)
def test_no_gates_is_gate_1(m, dtype, bits):
    Case(m, 5, 4, 2, 48, 40, dtype, bits, seed=3, gates=False).check()
    Case(m, 1, 1, 1, 300, 77, dtype, bits, seed=4, gates=False, G=64).check(("layer",))


@pytest.mark.parametrize("dtype,bits", DTYPES)
def test_pointers_at_any_element(m, dtype, bits):
    c = Case(m, 4, 5, 2, 64, 40, dtype, bits, seed=5)
    want = c.layer().clone(), c.ffn().clone()
    c.X = off_by(c.X, 1)
    for k in c.w:
        c.w[k] = tuple(off_by(t, 1) for t in c.w[k]) if bits == 4 else off_by(c.w[k], 1)
    c.gates = off_by(c.gates, 1)
    assert torch.equal(c.layer(), want[0]) and torch.equal(c.ffn(), want[1])
    c.check()


@pytest.mark.parametrize("dtype,bits", DTYPES)
def test_rows_do_not_meet(m, dtype, bits):
    # a token's NaN, infinity or large values stay its own, and weights that no token chooses are not read into any
    c = Case(m, 18, 6, 2, 64, 48, dtype, bits, seed=6)
    c.ids = c.ids % 5  # expert 5 is nobody's
    want = c.layer().clone(), c.ffn().clone()
    X = c.X.clone()
    X[3, 5], X[7, 0], X[11] = float("nan"), float("inf"), 2.0 ** 100
    if bits == 4:
        for k in c.w:
            c.w[k][1][5] = float("nan")
    else:
        for k in c.w:
            c.w[k][5] = float("nan")
    rest = [t for t in range(18) if t not in (3, 7, 11)]
    a, b = c.layer(X), c.ffn(X)
    assert torch.equal(a[rest], want[0][rest]) and torch.equal(b[rest], want[1][rest])
    assert torch.isnan(a[3]).all() and not torch.isfinite(a[7]).any()
    assert torch.isfinite(a[11]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_infinite_weights(m, dtype):
    # rows past the end are not multiplied: an infinity in the last row of an odd width stays one
    c = Case(m, 2, 2, 1, 37, 20, dtype, 16, seed=7)
    c.w["w"][:, -1, 3] = float("inf")
    out = c.layer()
    assert torch.isinf(out[:, 3]).all()
    assert torch.isfinite(out[:, [i for i in range(20) if i != 3]]).all()


@pytest.mark.parametrize("dtype,bits", DTYPES)
def test_same_results_again(m, dtype, bits):
    # partial sums are added in one order, whatever finishes first
    c = Case(m, 32, 8, 4, 512, 384, dtype, bits, seed=8)
    first = c.layer().clone(), c.ffn().clone()
    for _ in range(5):
        assert torch.equal(c.layer(), first[0]) and torch.equal(c.ffn(), first[1])


@pytest.mark.parametrize("bits", [16, 4])
def test_ranks_are_tokens(m, bits):
    a = Case(m, 12, 8, 2, 96, 40, BF, bits, seed=9, R=1)
    b = Case(m, 12, 8, 2, 96, 40, BF, bits, seed=9, R=4)
    assert torch.equal(a.layer(), b.layer()) and torch.equal(a.ffn(), b.ffn())


@pytest.mark.parametrize("dtype,bits", DTYPES)
def test_graphs_and_streams(m, dtype, bits):
    """Two graphs with workspaces of their own replayed on two streams, inputs changed between replays."""
    cases = [Case(m, 8, 8, 2, 256, 128, dtype, bits, seed=s) for s in (10, 11)]
    ids = [i32(c.ids) for c in cases]
    outs = [torch.empty((8, 256), device=DEV) for _ in cases]
    spaces = [workspace(m, c.d, c.H, c.Hp) for c in cases]

    def call(i, stream=None):
        c = cases[i]
        if bits == 4:
            m.moonep_few_ffn4(c.d, c.H, c.Hp, c.G, c.X, ids[i], c.gates, *c.w["gu"], *c.w["down"], outs[i],
                              spaces[i].view, stream)
        else:
            m.moonep_few_ffn(c.d, c.H, c.Hp, c.X, ids[i], c.gates, c.w["gu"], c.w["down"], outs[i], spaces[i].view,
                             stream)
    streams, graphs = [torch.cuda.Stream() for _ in cases], []
    for i, s in enumerate(streams):
        s.wait_stream(torch.cuda.current_stream())
        call(i, s)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call(i)
        graphs.append(g)
    for r in range(4):
        for i, c in enumerate(cases):
            c.X.copy_(rand_tensor(tuple(c.X.shape), dtype, 100 * r + i))
            ids[i].copy_(i32(routing(8, 8, 2, 7 * r + i)[0]))
            call(i)
        torch.cuda.synchronize()
        want = [o.clone() for o in outs]
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        say("replays", r)
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


@pytest.mark.parametrize("bits", [16, 4])
def test_offsets_past_32_bits(m, bits):
    """The last experts of a weight tensor of more than 2^32 elements."""
    E, H, Hp, T, K = (160, 7168, 2048, 2, 2) if bits == 16 else (320, 7168, 2048, 2, 2)
    assert E * H * 2 * Hp > 2 ** 32 * (1 if bits == 16 else 2)  # 4 bits: more than 2^31 bytes of words, 2^30 words
    d = m.make_dims(1, E, 0, T, K)
    ids = np.array([[E - 1, 0], [E - 2, E - 1]])
    gates = np.array([[0.5, 0.25], [1.0, -0.5]], np.float32)
    X = rand_tensor((T, H), BF, 0)
    used = sorted(set(ids.ravel().tolist()))
    shapes = {"gu": (H, 2 * Hp), "down": (Hp, H)}
    w, values = {}, {k: {} for k in shapes}
    for k, (rows, cols) in shapes.items():
        if bits == 16:
            w[k] = (torch.empty((E, rows, cols), dtype=BF, device=DEV),)
        else:
            w[k] = (torch.empty((E, rows // 8, cols), dtype=torch.int32, device=DEV),
                    torch.empty((E, rows // 32, cols), dtype=BF, device=DEV))
        for e in used:
            v = rand_tensor((1, rows, cols), BF, 10 + e, 1 / np.sqrt(rows))
            if bits == 16:
                w[k][0][e] = v[0]
            else:
                m.moonep_save4(1, rows, cols, 32, v, w[k][0][e:e + 1], w[k][1][e:e + 1])
                m.moonep_load4(1, rows, cols, 32, w[k][0][e:e + 1], w[k][1][e:e + 1], v)
                torch.cuda.synchronize()
                v = torch.empty((1, rows, cols), device=DEV)
                m.moonep_load4(1, rows, cols, 32, w[k][0][e:e + 1], w[k][1][e:e + 1], v)
            values[k][e] = v[0].double()
    out = torch.empty((T, H), device=DEV)
    ws = workspace(m, d, H, Hp)
    say("few_ffn past 2^32", bits)
    if bits == 16:
        m.moonep_few_ffn(d, H, Hp, X, i32(ids), f32(gates), w["gu"][0], w["down"][0], out, ws.view)
    else:
        m.moonep_few_ffn4(d, H, Hp, 32, X, i32(ids), f32(gates), *w["gu"], *w["down"], out, ws.view)
    torch.cuda.synchronize()
    ref, size = torch.zeros((T, H), dtype=torch.float64, device=DEV), torch.zeros((T, H), dtype=torch.float64, device=DEV)
    for t in range(T):
        for k in range(K):
            e = int(ids[t, k])
            y = X[t].double() @ values["gu"][e]
            a = y[:Hp] * torch.sigmoid(y[:Hp]) * y[Hp:]
            ref[t] += float(gates[t, k]) * (a @ values["down"][e])
            size[t] += abs(float(gates[t, k])) * (a.abs() @ values["down"][e].abs())
    # a wrong expert or row is off by the size of the terms; the products' roundings are far below a thousandth of it
    assert float(((out.double() - ref).abs() / size).max()) < 1e-3


def test_layer_through_save4(m):
    """Router, weights into 4 bits and the layer from them, as a program runs them together."""
    R, S, E, K, H, Hp, G = 2, 3, 16, 4, 192, 88, 64
    T = R * S
    d = m.make_dims(R, E, 0, S, K)
    W_gu, W_down = rand_tensor((E, H, 2 * Hp), BF, 1, H ** -0.5), rand_tensor((E, Hp, H), BF, 2, Hp ** -0.5)
    X, logits = rand_tensor((R, S, H), BF, 3), rand_tensor((R, S, E), F32, 4)
    words = lambda r, c: (torch.empty((E, -(-r // 8), c), dtype=torch.int32, device=DEV),  # noqa: E731
                          torch.empty((E, -(-r // G), c), dtype=BF, device=DEV))
    gu, down = words(H, 2 * Hp), words(Hp, H)
    ids = torch.empty((R, S, K), dtype=torch.int32, device=DEV)
    gates, out = torch.empty((R, S, K), device=DEV), torch.empty((R, S, H), device=DEV)
    ws = workspace(m, d, H, Hp)
    say("route, save4, few_ffn4")
    m.moonep_save4(E, H, 2 * Hp, G, W_gu, *gu)
    m.moonep_save4(E, Hp, H, G, W_down, *down)
    m.moonep_route(d, "sigmoid", True, 2.5, logits, None, ids, gates)
    m.moonep_few_ffn4(d, H, Hp, G, X, ids, gates, *gu, *down, out, ws.view)
    torch.cuda.synchronize()
    ri, rg = few.route(np64(logits).reshape(T, E), None, K, "sigmoid", True, 2.5)
    assert np.array_equal(npi(ids).reshape(T, K), ri)
    kept = [few.save4(np64(w), G) for w in (W_gu, W_down)]
    values = [few.load4(*k, G) for k in kept]
    sizes = [56 * np.repeat(k[1], G, axis=1)[:, :v.shape[1]] for k, v in zip(kept, values)]
    rows = [[v[e] for e in range(E)] for v in values]
    by = {id(w): s for r, z in zip(rows, sizes) for w, s in zip(r, z)}
    size = lambda w: by[id(w)]  # noqa: E731
    ref, bound = few.few_ffn(np64(X).reshape(T, H), ri, rg, *rows, 2 * (H + K + 16) * U, size, size)
    # the gates' own error, (E + 40) u of each pair's term (see the router's tests), one pair at a time
    for k in range(K):
        one = few.few_ffn(np64(X).reshape(T, H), ri[:, k:k + 1], rg[:, k:k + 1], *rows, 0.0)[0]
        bound = bound + (E + 40) * U * np.abs(one)
    assert np.all(np.abs(np64(out).reshape(T, H) - ref) <= bound)


# T, E, K, H, Hp: long inputs with so few tiles that they are cut narrower, in either product; rows for one and for two
# matrix instructions, few and many waves' steps, widths off the tiles' and down to one column
NARROW = [(24, 2, 2, 3503, 141), (3, 4, 2, 769, 40), (5, 8, 3, 1536, 2), (4, 3, 1, 800, 1), (40, 3, 2, 33, 770),
          (7, 16, 4, 1024, 65), (33, 2, 1, 775, 800), (9, 2, 2, 2080, 3)]


@pytest.mark.parametrize("dtype,bits", DTYPES)
@pytest.mark.parametrize("T,E,K,H,Hp", NARROW)
def test_long_inputs_of_few_tiles(m, dtype, bits, T, E, K, H, Hp):
    Case(m, T, E, K, H, Hp, dtype, bits, seed=T + H).check()
