"""MoeFFN's router and MoeFew on the GPU: the calls together, as programs use them.

Bounds: float32 layers against float64 autograd of the plain formula, 1e-4 (1 + |ref|) as for the tiny float32 layer
elsewhere (sums of at most 256 terms of size about 1, three of them behind each other: below 1e-5).  The router's gradient
from the layer's own dgates: as in the router's tests, with logits at most 20 apart.  MoeFew from a MoeFFN's
bf16 weights against that layer's planned pass, which rounds Ygu, A and the output rows to bf16 (2^-8 each): per
output, (2^-8 for each of the three, and 2^-8 for gate and up behind each other) of the sum of its terms' magnitudes.
"""
import numpy as np
import pytest
import torch

from oracle import few
from tests.gpu_util import DEV, np64, npi, rand_tensor, say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def m():
    import load_balanced_dispatch_amd as mod
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    return mod


def fill(L, seed):
    """Random inputs, weights and output gradient of a MoeFFN."""
    E, H, Hp = L.d.E, L.H, L.Hp
    L.X.copy_(rand_tensor(tuple(L.X.shape), L.dtype, seed))
    L.W_gu_home.copy_(rand_tensor((E, H, 2 * Hp), L.dtype, seed + 1, H ** -0.5))
    L.W_down_home.copy_(rand_tensor((E, Hp, H), L.dtype, seed + 2, Hp ** -0.5))
    if L.logits is not None:
        L.logits.copy_(rand_tensor(tuple(L.logits.shape), F32, seed + 3))
    if hasattr(L, "dout"):
        L.dout.copy_(rand_tensor(tuple(L.dout.shape), F32, seed + 4))


@pytest.mark.parametrize("score,renorm,biased", [("softmax", True, False), ("softmax", False, True),
                                                 ("sigmoid", True, True), ("sigmoid", False, False)])
@pytest.mark.parametrize("save8", [False, True])
def test_router_through_a_training_pass(m, score, renorm, biased, save8):
    R, E, B, S, K, H, Hp = 2, 8, 4, 24, 2, 64, 32
    L = m.MoeFFN(R, E, B, S, K, H, Hp, dtype=F32, device=DEV, backward=True, router=score, renorm=renorm,
                 route_scale=1.5, router_bias=biased, save8=save8)
    fill(L, 11)
    if biased:
        L.bias.copy_(rand_tensor((E,), F32, 5, 0.1))
    L.logits[1, 3] = -float("inf")  # a token without an expert
    say("MoeFFN with a router", score, renorm, biased, save8)
    L.forward()
    L.backward()
    torch.cuda.synchronize()
    T = R * S
    l = np64(L.logits).reshape(T, E)
    ids, gates = few.route(l, np64(L.bias) if biased else None, K, score, renorm, 1.5)
    assert np.array_equal(npi(L.topk_idx).reshape(T, K), ids)
    assert np.all(np.abs(np64(L.gates).reshape(T, K) - gates) <= (E + 40) * 2.0 ** -24 * np.abs(gates))
    # float64 autograd of the whole layer
    rows = [t for t in range(T) if t != S + 3]
    t64 = lambda a: torch.tensor(np64(a), dtype=torch.float64)  # noqa: E731
    x, wg, wd = t64(L.X).view(T, H)[rows], t64(L.W_gu_home), t64(L.W_down_home)
    lt = torch.tensor(l[rows], requires_grad=True)
    s = torch.softmax(lt, 1) if score == "softmax" else torch.sigmoid(lt)
    it = torch.tensor(ids[rows])
    w = s.gather(1, it)
    g = 1.5 * (w / w.sum(1, keepdim=True) if renorm else w)
    y = x.view(-1, 1, 1, H) @ wg[it]
    a = torch.nn.functional.silu(y[..., :Hp]) * y[..., Hp:]
    out = (g[..., None] * (a @ wd[it]).squeeze(2)).sum(1)
    assert not L.out.view(T, H)[S + 3].any()
    ref = out.detach().numpy()
    assert np.all(np.abs(np64(L.out).reshape(T, H)[rows] - ref) <= 1e-4 * (1 + np.abs(ref)))
    (out * t64(L.dout).view(T, H)[rows]).sum().backward()
    dl = np64(L.dlogits).reshape(T, E)
    assert not dl[S + 3].any()
    # the router's gradient from the layer's own dgates, whose parity with 8-bit checkpoints is tested with those
    dg = np64(L.dgates).reshape(T, K)
    ref, size = few.route_backward(l, ids, np.where(ids >= 0, dg, 0.0), score, renorm, 1.5)
    assert np.all(np.abs(dl - ref) <= (E + K + 80) * 2.0 ** -24 * size)
    if not save8:
        assert np.all(np.abs(dl[rows] - lt.grad.numpy()) <= 1e-4 * (1 + np.abs(lt.grad.numpy())))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_few_is_the_planned_layer(m, dtype):
    R, E, B, S, K, H, Hp = 4, 16, 4, 8, 4, 192, 128
    L = m.MoeFFN(R, E, B, S, K, H, Hp, dtype=dtype, device=DEV, router="softmax")
    fill(L, 21)
    F = m.MoeFew(R, E, S, K, H, Hp, dtype=dtype, device=DEV, router="softmax", weights=(L.W_gu_home, L.W_down_home))
    F.X.copy_(L.X)
    F.logits.copy_(L.logits)
    say("MoeFew and MoeFFN", dtype)
    L.forward()
    F.forward()
    torch.cuda.synchronize()
    assert torch.equal(F.topk_idx, L.topk_idx) and torch.equal(F.gates, L.gates)
    T = R * S
    ids, gates = npi(F.topk_idx).reshape(T, K), np64(F.gates).reshape(T, K)
    rows = [[w for w in np64(t)] for t in (L.W_gu_home, L.W_down_home)]
    # a planned bf16 layer: Ygu, A and the output rows each rounded, half a step 2^-8 of their own size; float32: sums
    h = 2.0 ** -8 if dtype == BF else 2 * (H + 16) * 2.0 ** -24
    ref, bound = few.few_ffn(np64(F.X).reshape(T, H), ids, gates, *rows, h)
    assert np.all(np.abs(np64(F.out) - np64(L.out)).reshape(T, H) <= bound + h * bound)
    exact = few.few_ffn(np64(F.X).reshape(T, H), ids, gates, *rows, 2 * (H + K + 16) * 2.0 ** -24)[1]
    assert np.all(np.abs(np64(F.out).reshape(T, H) - ref) <= exact)


@pytest.mark.parametrize("bits", [16, 4])
def test_few_with_norm_and_router_captured(m, bits):
    R, E, S, K, H, Hp = 2, 8, 2, 2, 160, 72
    F = m.MoeFew(R, E, S, K, H, Hp, device=DEV, bits=bits, G=32, norm=True, router="sigmoid", router_bias=True,
                 route_scale=2.0)
    W_gu, W_down = rand_tensor((E, H, 2 * Hp), BF, 1, H ** -0.5), rand_tensor((E, Hp, H), BF, 2, Hp ** -0.5)
    F.save_weights(W_gu, W_down)
    F.gamma.copy_(1 + rand_tensor((H,), F32, 3, 0.1))
    F.beta.copy_(rand_tensor((H,), F32, 4, 0.1))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    say("MoeFew captured", bits)
    with torch.cuda.stream(stream):
        F.forward()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        F.forward()
    for r in range(3):
        F.X.copy_(rand_tensor((R, S, H), BF, 50 + r))
        F.logits.copy_(rand_tensor((R, S, E), F32, 60 + r))
        F.bias.copy_(rand_tensor((E,), F32, 70 + r, 0.1))
        F.forward()
        torch.cuda.synchronize()
        want = F.out.clone()
        F.out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(F.out, want)
    T = R * S
    ids, gates = few.route(np64(F.logits).reshape(T, E), np64(F.bias), K, "sigmoid", True, 2.0)
    assert np.array_equal(npi(F.topk_idx).reshape(T, K), ids)
    values = [np64(w) for w in (W_gu, W_down)]
    sizes = [np.abs(v) for v in values]
    if bits == 4:
        kept = [few.save4(v, 32) for v in values]
        values = [few.load4(*k, 32) for k in kept]
        sizes = [56 * np.repeat(k[1], 32, axis=1)[:, :v.shape[1]] for k, v in zip(kept, values)]
    rows = [[w for w in v] for v in values]
    by = {id(w): s for ws, z in zip(rows, sizes) for w, s in zip(ws, z)}
    size = lambda w: by[id(w)]  # noqa: E731
    # the rows that the experts read are the norm's own, whose parity is tested with the norm
    ref, bound = few.few_ffn(np64(F.Xn).reshape(T, H), ids, np64(F.gates).reshape(T, K), *rows,
                             2 * (H + K + 16) * 2.0 ** -24, size, size)
    assert np.all(np.abs(np64(F.out).reshape(T, H) - ref) <= bound)
