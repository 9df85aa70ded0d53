"""Gradients of the router where dgates are no finite numbers (GPU).

Nothing is bounded here: what is masked has the gradient 0, the rest of such a token is not finite, and other tokens keep
theirs to the last bit.
"""
import numpy as np
import pytest
import torch

from oracle import few
from tests.gpu_util import DEV, f32, i32, np64, say

pytestmark = pytest.mark.gpu

KINDS = [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)]


@pytest.fixture(scope="module")
def m():
    import load_balanced_dispatch_amd as mod
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    return mod


@pytest.mark.parametrize("E,K", [(12, 3), (64, 4), (190, 8), (512, 15), (300, 16), (700, 5)])
@pytest.mark.parametrize("score,renorm", KINDS)
def test_masked_experts_have_gradient_0_whatever_dgates_are(m, E, K, score, renorm):
    rng = np.random.default_rng(E)
    T = 9
    l = rng.standard_normal((T, E)).astype(np.float32)
    l[:, 1::4] = -np.inf
    l[:, 2::4] = np.nan
    ids = np.stack([rng.permutation(np.flatnonzero(l[t] > -np.inf))[:K] for t in range(T)])
    dg = rng.standard_normal((T, K)).astype(np.float32)
    d = m.make_dims(1, E, 0, T, K)
    plain, dl = torch.empty((T, E), device=DEV), torch.empty((T, E), device=DEV)
    say("route_backward, finite dgates", E, K, score, renorm)
    m.moonep_route_backward(d, score, renorm, 1.0, f32(l), i32(ids), f32(dg), plain)
    dg[1, 0], dg[4, K - 1], dg[6, 1] = np.nan, np.inf, -np.inf
    say("route_backward, dgates of NaN and infinity")
    m.moonep_route_backward(d, score, renorm, 1.0, f32(l), i32(ids), f32(dg), dl)
    torch.cuda.synchronize()
    got, masked = np64(dl), ~(l > -np.inf)
    assert not got[masked].any()  # NaN would be true
    for t in range(T):
        if t not in (1, 4, 6):
            assert torch.equal(dl[t], plain[t])
    for t, k in ((1, 0), (4, K - 1), (6, 1)):
        assert not np.isfinite(got[t, ids[t, k]])
    with np.errstate(invalid="ignore"):
        ref, _ = few.route_backward(l, ids, dg, score, renorm, 1.0)
    assert not ref[masked].any()


@pytest.mark.parametrize("E,K", [(64, 8), (700, 40)])
@pytest.mark.parametrize("score,renorm", KINDS)
def test_gradients_of_repeated_ids_are_the_same_again(m, E, K, score, renorm):
    # an id that a token holds many times: its sum is taken in one order
    rng = np.random.default_rng(K)
    T = 33
    d = m.make_dims(1, E, 0, T, K)
    l, dg = f32(rng.standard_normal((T, E))), f32(rng.standard_normal((T, K)) * np.exp(rng.standard_normal((T, K)) * 4))
    ids = i32(rng.integers(0, 3, (T, K)))
    first = torch.empty((T, E), device=DEV)
    m.moonep_route_backward(d, score, renorm, 1.0, l, ids, dg, first)
    say("route_backward repeated ids", E, K, score, renorm)
    for _ in range(20):
        again = torch.empty((T, E), device=DEV)
        m.moonep_route_backward(d, score, renorm, 1.0, l, ids, dg, again)
        assert torch.equal(again, first)


@pytest.mark.parametrize("save8", [False, True])
def test_a_training_pass_with_a_router_captured(m, save8):
    R, E, B, S, K, H, Hp = 2, 8, 4, 24, 2, 64, 32
    L = m.MoeFFN(R, E, B, S, K, H, Hp, dtype=torch.float32, device=DEV, backward=True, router="softmax", renorm=False,
                 router_bias=True, save8=save8)
    g = torch.Generator().manual_seed(0)
    draw = lambda t, std=1.0: t.copy_(torch.randn(t.shape, generator=g) * std)  # noqa: E731
    draw(L.W_gu_home, H ** -0.5)
    draw(L.W_down_home, Hp ** -0.5)
    results = ("topk_idx", "gates", "out", "dX", "dgates", "dlogits", "dW_gu_home", "dW_down_home")

    def inputs():
        for t in (L.X, L.logits, L.dout):
            draw(t)
        draw(L.bias, 0.1)
        L.logits[0, 1] = -float("inf")

    def step():
        L.forward()
        L.backward()
    inputs()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    say("MoeFFN with a router captured", save8)
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    for r in range(3):
        inputs()
        L.dW_gu_home.zero_()
        L.dW_down_home.zero_()
        step()
        torch.cuda.synchronize()
        want = {n: getattr(L, n).clone() for n in results}
        for n in results:
            getattr(L, n).zero_()
        torch.cuda.synchronize()
        say("replay", r)
        graph.replay()
        torch.cuda.synchronize()
        for n in results:
            assert torch.equal(getattr(L, n), want[n]), n
