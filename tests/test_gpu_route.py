"""Parity of the router and its gradient against the float64 oracle (GPU).

Bounds, with u = 2^-24 (half a step of float32).  The choice: equal.  Gates: the exponential's argument l - max is rounded
once (u |l - max| of the result, the spread), its own error is at most 4 u, a sum of E positive terms at most E u, and at
most 12 roundings follow (quotient, product, the sigmoid's terms): (E + 2 spread + 20) u of the gate, and 2^-126 for
results that leave float32's normal range.  Gradients: sums over the K chosen on top of that, so the same with K more,
times the size of the terms that are subtracted.
"""
import numpy as np
import pytest
import torch

from oracle import few
from tests.gpu_util import DEV, Guarded, f32, i32, np64, npi, say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
LOW = -few.LARGEST
KINDS = [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)]


@pytest.fixture(scope="module")
def m():
    import load_balanced_dispatch_amd as mod
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    return mod


def spread(l, ids):
    """How far below the largest logit the chosen ones lie, [T, K]."""
    l = few._masked(l)
    x = np.take_along_axis(l, np.maximum(ids, 0), axis=1)
    top = l.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        return np.where((ids >= 0) & np.isfinite(x), np.minimum(np.abs(top - x), 200.0), 0.0)


def off_by(t, by):
    """A contiguous copy of t that starts `by` elements into its allocation."""
    buf = torch.empty(t.numel() + by + 64, dtype=t.dtype, device=DEV)
    v = buf[by:by + t.numel()].view(t.shape)
    v.copy_(t)
    return v


def check(m, l, bias, K, score, renorm, scale, seed=0, by=0):
    """Forward and backward of logits [T, E] against the oracle."""
    T, E = l.shape
    d = m.make_dims(1, E, 0, T, K)
    x = off_by(f32(l), by)
    b = None if bias is None else off_by(f32(bias), by)
    ids, gates = Guarded((T, K), torch.int32), Guarded((T, K), torch.float32)
    say("route", T, E, K, score, renorm, "bias" if bias is not None else "", "offset", by)
    m.moonep_route(d, score, renorm, scale, x, b, ids.view, gates.view)
    torch.cuda.synchronize()
    ri, rg = few.route(l, bias, K, score, renorm, scale)
    assert np.array_equal(npi(ids.view), ri)
    sp = spread(l, ri)
    bound = (E + 2 * sp + 20) * U * np.abs(rg) + 2.0 ** -126 * abs(scale)
    err = np.abs(np64(gates.view) - rg)
    assert np.all(err <= bound), float((err - bound).max())
    assert ids.intact() and gates.intact()
    dg = np.random.default_rng(seed + 9).standard_normal((T, K)).astype(np.float32)
    dl = Guarded((T, E), torch.float32)
    say("route_backward")
    m.moonep_route_backward(d, score, renorm, scale, x, i32(ri), f32(dg), dl.view)
    torch.cuda.synchronize()
    rd, size = few.route_backward(l, ri, dg, score, renorm, scale)
    each = np.minimum(np.abs(few._masked(l).max(axis=1, keepdims=True) - np.where(np.isfinite(l), l, 0)), 200.0)
    each = np.where(np.isfinite(each), each, 0)
    bound = (E + K + 2 * each + 2 * sp.max(axis=1, keepdims=True) + 40) * U * size + 2.0 ** -120
    err = np.abs(np64(dl.view) - rd)
    assert np.all(err <= bound), float((err - bound).max())
    assert dl.intact()
    return ids.view, gates.view


def logits(T, E, seed, std=1.0):
    return (np.random.default_rng(seed).standard_normal((T, E)) * std).astype(np.float32)


SIZES = [(1, 1, 1), (5, 2, 2), (3, 5, 5), (7, 15, 4), (9, 16, 16), (33, 17, 3), (64, 63, 6), (130, 64, 6), (67, 65, 8),
         (9, 100, 7), (41, 128, 1), (19, 160, 8), (50, 256, 8), (3, 256, 9), (2, 256, 256), (17, 257, 8), (21, 384, 8),
         (5, 512, 17), (18, 512, 15), (5, 512, 16), (21, 64, 15), (21, 60, 16), (6, 1000, 12), (3, 1024, 33), (4, 2500, 8), (2, 4096, 5)]


@pytest.mark.parametrize("T,E,K", SIZES)
def test_sizes(m, T, E, K):
    for i, (score, renorm) in enumerate(KINDS):
        l = logits(T, E, seed=E + i)
        check(m, l, None, K, score, renorm, 1.0, by=i % 2)
        bias = (np.random.default_rng(E).standard_normal(E) * 0.1).astype(np.float32)
        check(m, l, bias, K, score, renorm, 2.5, by=(i + 1) % 2)


@pytest.mark.parametrize("E", [16, 100, 256, 700])
def test_ties_go_to_the_lowest(m, E):
    rng = np.random.default_rng(E)
    l = rng.integers(-2, 3, (40, E)).astype(np.float32)
    l[0] = 0.0
    l[1] = np.where(np.arange(E) % 2 == 0, -0.0, 0.0)  # equal zeros of both signs
    for score, renorm in KINDS:
        check(m, l, None, 8, score, renorm, 1.0)
        check(m, l, (rng.integers(0, 2, E) * 0.5).astype(np.float32), 8, score, renorm, 1.0)
        check(m, l, np.zeros(E, np.float32), 8, score, renorm, 1.0)


@pytest.mark.parametrize("E", [8, 64, 200, 256, 300])
def test_masks_and_extremes(m, E):
    l = logits(12, E, seed=E, std=3.0)
    l[0] = -np.inf                                  # nothing to choose
    l[1, 3:] = -np.inf                              # fewer than K
    l[2] = np.nan
    l[3, 1::2] = np.nan
    l[4] = LOW                                      # finite masks of the type's lowest value: all alike
    l[5, 2:] = LOW
    l[6, :2] = np.inf
    l[7] = few.LARGEST
    l[8, 0] = few.LARGEST                           # the others' exponentials are 0
    l[9] = -np.abs(l[9]) - 150.0                    # sigmoids below float32's range
    l[10] = np.linspace(0, 120, E)                  # scores from 1e-52 to 1
    bias = logits(1, E, seed=1)[0] * np.float32(0.1)
    bias[::3] = -np.inf
    bias[1] = np.nan
    bias[2] = np.inf
    for score, renorm in KINDS:
        ids, gates = check(m, l, None, 6, score, renorm, 1.0)
        assert npi(ids)[0].tolist() == [-1] * 6 and not np64(gates)[0].any()
        # the rows whose scores all vanish (9: sigmoid) or saturate would be ties of rounding: not with a bias
        rows = [i for i in range(12) if i not in (8, 9, 10)]
        check(m, l[rows], bias, 6, score, renorm, 1.5)


@pytest.mark.parametrize("E", [128, 192, 256, 384, 512])
def test_the_largest_lie_together(m, E):
    # more of the largest keys than the sorted ones of a lane hold: columns 4 j .. 4 j + 3 of every 64, in any order,
    # far above the others, a little above and below them, and next to each other within float32's error of a score
    rng = np.random.default_rng(E)
    T = 48
    l = (rng.standard_normal((T, E)) * 0.01).astype(np.float32)
    bias = np.zeros(E, np.float32)
    for t in range(T):
        lane = rng.integers(0, 16)
        cols = np.concatenate([64 * q + 4 * lane + np.arange(4) for q in range(E // 64)])
        lift = [1.0, 0.02, 0.0][t % 3]
        l[t, cols] = lift + rng.permutation(len(cols)) * [1e-2, 2.0 ** -22, 0.0, 2.0 ** -23][t % 4]
    for score, renorm in KINDS:
        for K in (3, 4, 5, 8, 15):
            check(m, l, None, K, score, renorm, 1.0)
            check(m, l, bias, K, score, renorm, 1.0)


@pytest.mark.parametrize("E", [8, 64, 256, 300])
def test_infinite_and_largest_biases_are_alike(m, E):
    # both count as the largest float, so that the scores do not matter: the lowest index first
    l = logits(9, E, seed=E)
    bias = np.zeros(E, np.float32)
    bias[1], bias[3], bias[E - 2] = few.LARGEST, np.inf, few.LARGEST
    for score, renorm in KINDS:
        for K in (1, 2, 3, 5):
            ids, _ = check(m, l, bias, K, score, renorm, 1.0)
            assert npi(ids)[:, :min(K, 3)].tolist() == [[1, 3, E - 2][:min(K, 3)]] * 9


def test_backward_takes_any_ids(m):
    # ids outside [0, E) are left out, the same expert twice adds up, and so does a masked one's nothing
    T, E, K = 6, 40, 4
    l = logits(T, E, seed=2)
    l[3, 5] = -np.inf
    ids = np.array([[0, 0, 1, 2], [-1, 40, 3, 2 ** 31 - 1], [-1] * 4, [5, 6, 7, 8], [9, 9, 9, 9], [-2 ** 31, 0, 39, 39]])
    dg = np.random.default_rng(0).standard_normal((T, K)).astype(np.float32)
    d = m.make_dims(1, E, 0, T, K)
    for score, renorm in KINDS:
        dl = Guarded((T, E), torch.float32)
        say("route_backward ids", score, renorm)
        m.moonep_route_backward(d, score, renorm, 1.0, f32(l), i32(ids), f32(dg), dl.view)
        torch.cuda.synchronize()
        ref, size = few.route_backward(l, ids, dg, score, renorm, 1.0)
        assert np.all(np.abs(np64(dl.view) - ref) <= (E + K + 40) * U * size + 2.0 ** -120)
        assert dl.intact()


def test_gradient_is_the_forwards_differences(m):
    # float32 gates of shifted logits: their rounding over the shift bounds what the quotient can say
    T, E, K, h = 8, 24, 4, 2.0 ** -6
    l = logits(T, E, seed=5)
    d = m.make_dims(1, E, 0, T, K)
    dg = np.random.default_rng(1).standard_normal((T, K))
    for score, renorm in KINDS:
        ids, gates = torch.empty((T, K), dtype=torch.int32, device=DEV), torch.empty((T, K), device=DEV)
        m.moonep_route(d, score, renorm, 1.0, f32(l), None, ids, gates)
        dl = torch.empty((T, E), device=DEV)
        m.moonep_route_backward(d, score, renorm, 1.0, f32(l), ids, f32(dg), dl)
        torch.cuda.synchronize()
        chosen = npi(ids)
        got = np64(dl)
        for e in (0, 7, 23, int(chosen[0, 0]), int(chosen[1, 2])):
            side = []
            for s in (h, -h):
                x = l.copy()
                x[:, e] += np.float32(s)
                side.append((few.gates_of(x, chosen, score, renorm, 1.0) * dg).sum(1))
            # third derivatives of both score functions' gates are at most 1 in size: h^2 / 6 per unit of dgates
            assert np.all(np.abs((side[0] - side[1]) / (2 * h) - got[:, e]) <= h * h / 6 * np.abs(dg).sum(1) + 1e-5)


def test_plan_takes_what_route_gives(m):
    """A layer's forward and backward from logits: route, plan, dispatch, ..., combine backward, route backward."""
    R, E, B, S, K, H = 2, 8, 4, 32, 2, 64
    l = logits(R * S, E, seed=8)
    l[5] = -np.inf  # a token without an expert: its pairs are left out everywhere
    L = m.MoeLayer(R, E, B, S, K, H, 32, dtype=torch.float32, device=DEV, backward=True, data_grad=True)
    g = torch.Generator().manual_seed(0)
    L.X.copy_(torch.randn(R, S, H, generator=g))
    L.W_home.copy_(torch.randn(E, H, 32, generator=g) / 8)
    L.dout.copy_(torch.randn(R, S, 32, generator=g))
    x = f32(l).view(R, S, E)
    say("route in front of a layer")
    m.moonep_route(L.d, "softmax", True, 1.0, x, None, L.topk_idx, L.gates)
    L.forward()
    L.backward_data()
    dl = torch.empty_like(x)
    m.moonep_route_backward(L.d, "softmax", True, 1.0, x, L.topk_idx, L.dgates, dl)
    torch.cuda.synchronize()
    assert L.stats[3].item() == K and not L.out.view(-1, 32)[5].any()
    t = torch.tensor(l, dtype=torch.float64, requires_grad=True)
    ids = L.topk_idx.view(-1, K).cpu().long()
    rows = [i for i in range(R * S) if i != 5]
    w = torch.softmax(t[rows], 1).gather(1, ids[rows])
    gates = w / w.sum(1, keepdim=True)
    X, W = L.X.view(-1, H).cpu().double()[rows], L.W_home.cpu().double()
    out = sum(gates[:, k:k + 1] * (X.unsqueeze(1) @ W[ids[rows, k]]).squeeze(1) for k in range(K))
    (out * L.dout.view(-1, 32).cpu().double()[rows]).sum().backward()
    ref = t.grad.numpy()
    # dgates is a float32 sum of 32 products of sums of 64
    assert np.all(np.abs(np64(dl).reshape(ref.shape) - ref) <= 1e-4)


def test_graph_and_streams(m):
    T, E, K = 64, 256, 8
    d = m.make_dims(8, E, 0, T // 8, K)
    x, b = f32(logits(T, E, 3)), f32(logits(1, E, 4)[0] * np.float32(0.1))
    ids = torch.zeros((T, K), dtype=torch.int32, device=DEV)
    gates, dl = torch.zeros((T, K), device=DEV), torch.zeros((T, E), device=DEV)

    def step():
        m.moonep_route(d, "sigmoid", True, 2.5, x, b, ids, gates)
        m.moonep_route_backward(d, "sigmoid", True, 2.5, x, ids, gates, dl)
    say("route on a stream of its own")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for i in range(3):
        x.copy_(f32(logits(T, E, 20 + i)))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (ids, gates, dl)]
        for t in (ids, gates, dl):
            t.zero_()
        say("replay", i)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, w) for a, w in zip((ids, gates, dl), want))
