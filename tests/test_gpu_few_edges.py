"""The layer for few tokens and the 4-bit weights at the ends of their ranges (GPU).

Bounds, with u = 2^-24, are those of the products' roundings: 2 (H + K + 16) u of the sum of the terms' magnitudes, where
with 4-bit weights a term counts as 56 times the scale times the row's value, whatever its code (32 + 24 steps, as the
products are with code + 24, less 24).  Small rows lose what leaves float32 and bf16: 4-bit sums are taken in units of 2^-10,
so each of at most 6 (H + 32) products and additions is off by 2^-149 of them, 2^-139 times the scale, as are the sums'
own, 2^-139 each; a float32 row's parts are off by bf16's last place, 2^-133, times 56 scales.
"""
import numpy as np
import pytest
import torch

from oracle import few
from tests.gpu_util import DEV, Guarded, f32, i32, np64, rand_tensor, say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def m():
    import load_balanced_dispatch_amd as mod
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    return mod


def space(m, d, H, Hp):
    w = Guarded((m.moonep_few_workspace_bytes(d, H, Hp) // 4,), torch.int32)
    w.view.fill_(-1)
    return w


def four(E, rows, cols, G, seed, std):
    """4-bit weights of random values: what the calls take, the values, and 56 scales for every row."""
    rng = np.random.default_rng(seed)
    codes, scales = few.save4(rng.standard_normal((E, rows, cols)) * std, G)
    tensors = torch.as_tensor(few.pack4(codes)).to(DEV), torch.tensor(scales, dtype=F32).to(BF).to(DEV)
    return tensors, few.load4(codes, scales, G), 56 * np.repeat(scales, G, axis=1)[:, :rows]


def routing(T, E, K, seed):
    rng = np.random.default_rng(seed)
    g = rng.random((T, K)).astype(np.float32)
    return np.stack([rng.permutation(E)[:K] for _ in range(T)]), g / g.sum(1, keepdims=True)


# T, E, K, H, Hp: a token's block, an expert's, narrow tiles, more pairs of an expert than packed float32 rows hold
FORMS = [(1, 2, 1, 100, 40), (6, 3, 2, 100, 70), (7, 2, 1, 800, 24), (12, 2, 2, 96, 65)]
SIZES = [-122, -100, -60, 60, 100, 112, 120, 126]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,E,K,H,Hp", FORMS)
def test_layer4_of_rows_of_any_size(m, dtype, T, E, K, H, Hp):
    G = 32
    d = m.make_dims(1, E, 0, T, K)
    ids, gates = routing(T, E, K, 1)
    (words, scales), values, size = four(E, H, Hp, G, 2, 2.0 ** -12 / np.sqrt(H))
    base = rand_tensor((T, H), F32, 3).clamp(-1.9, 1.9)
    for b in SIZES:
        X = (base * 2.0 ** b).to(dtype)
        out, ws = Guarded((T, Hp), F32), space(m, d, H, Hp)
        say("few_layer4 rows of 2 ^", b, dtype, T, E, K, H, Hp)
        m.moonep_few_layer4(d, H, Hp, G, X, i32(ids), f32(gates), words, scales, out.view, ws.view)
        torch.cuda.synchronize()
        x = X.double().cpu().numpy()
        ref, _ = few.few_layer(x, ids, gates, values)
        scale = few.few_layer(np.abs(x), ids, gates, size)[0]
        top = float(scales.float().max())
        lost = K * (6 * (H + 32) * 2.0 ** -139 * (1 + top) + H * 56 * 2.0 ** -133 * top)
        err = np.abs(out.view.double().cpu().numpy() - ref)
        assert np.all(err <= 2 * (H + K + 16) * U * scale + lost), b
        assert out.intact() and ws.intact()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,E,K,H,Hp", FORMS)
def test_ffn4_with_activations_of_any_size(m, dtype, T, E, K, H, Hp):
    # rows of 2^56 make activations of about 2^110, which take part in the second product as rows do in the first
    G = 32
    d = m.make_dims(1, E, 0, T, K)
    ids, gates = routing(T, E, K, 4)
    gu, gu_values, gu_size = four(E, H, 2 * Hp, G, 5, 1 / np.sqrt(H))
    down, down_values, down_size = four(E, Hp, H, G, 6, 2.0 ** -10 / np.sqrt(Hp))
    rows = [[v[e] for e in range(E)] for v in (gu_values, down_values)]
    by = {id(w): s for ws_, z in zip(rows, (gu_size, down_size)) for w, s in zip(ws_, z)}
    base = rand_tensor((T, H), F32, 7).clamp(-1.9, 1.9)
    for b in (0, 50, 56, 60, 61):
        X = (base * 2.0 ** b).to(dtype)
        out, ws = Guarded((T, H), F32), space(m, d, H, Hp)
        say("few_ffn4 rows of 2 ^", b, dtype, T, E, K, H, Hp)
        m.moonep_few_ffn4(d, H, Hp, G, X, i32(ids), f32(gates), *gu, *down, out.view, ws.view)
        torch.cuda.synchronize()
        x = X.double().cpu().numpy()
        with np.errstate(over="ignore"):
            ref, bound = few.few_ffn(x, ids, gates, *rows, 2 * (max(H, Hp) + K + 16) * U, lambda w: by[id(w)],
                                     lambda w: by[id(w)])
        err = np.abs(out.view.double().cpu().numpy() - ref)
        assert np.all(err <= bound + 2.0 ** -100), b
        assert out.intact() and ws.intact()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 6, 12])
def test_an_outlier_on_zero_codes(m, dtype, T):
    # a row's value that only meets the code 0 is still added, and taken off: what it leaves is within the stated bound
    E, H, Hp, G, K = 1, 64, 48, 32, 1
    d = m.make_dims(1, E, 0, T, K)
    codes = np.random.default_rng(0).integers(-8, 8, (E, H, Hp))
    codes[:, 5] = codes[:, 40] = 0
    scales = np.full((E, H // G, Hp), 0.5)
    words, s = torch.as_tensor(few.pack4(codes)).to(DEV), torch.tensor(scales, dtype=F32).to(BF).to(DEV)
    values, ids, gates = few.load4(codes, scales, G), np.zeros((T, K), np.int64), np.ones((T, K), np.float32)
    for b in (4, 8, 16, 24, 40):
        X = rand_tensor((T, H), dtype, 8)
        X[:, 5], X[:, 40] = 2.0 ** b, -1.5 * 2.0 ** b
        out, ws = Guarded((T, Hp), F32), space(m, d, H, Hp)
        say("few_layer4 outlier 2 ^", b, dtype, T)
        m.moonep_few_layer4(d, H, Hp, G, X, i32(ids), None, words, s, out.view, ws.view)
        torch.cuda.synchronize()
        x = X.double().cpu().numpy()
        ref, _ = few.few_layer(x, ids, gates, values)
        bound = 2 * (H + K + 16) * U * 56 * 0.5 * np.abs(x).sum(1, keepdims=True)
        err = np.abs(out.view.double().cpu().numpy() - ref)
        assert np.all(err <= bound), (b, float((err / bound).max()))
        assert out.intact() and ws.intact()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,H,Hp", [(6, 37, 20), (40, 37, 130), (7, 803, 20), (6, 803, 200)])
def test_infinite_weights_in_an_experts_block(m, dtype, T, H, Hp):
    # rows past the end are not multiplied: an infinity in the last row of an odd width stays one
    E, K = 3, 2
    d = m.make_dims(1, E, 0, T, K)
    ids, gates = routing(T, E, K, 9)
    w = rand_tensor((E, H, Hp), dtype, 10, H ** -0.5)
    w[:, -1, 3] = float("inf")
    X = rand_tensor((T, H), dtype, 11)
    X[:, -1] = X[:, -1].abs() + 0.5
    out, ws = Guarded((T, Hp), F32), space(m, d, H, Hp)
    say("few_layer infinite weights", dtype, T, H, Hp)
    m.moonep_few_layer(d, H, Hp, X, i32(ids), f32(gates), w, out.view, ws.view)
    torch.cuda.synchronize()
    assert torch.isposinf(out.view[:, 3]).all()
    assert torch.isfinite(out.view[:, [i for i in range(Hp) if i != 3]]).all()
    assert out.intact() and ws.intact()


def test_words_and_scales_of_4_bits_past_32_bits(m):
    """The last experts of more than 2^33 words and 2^31 scales."""
    E, H, Hp, G, T, K = 2400, 7168, 4096, 32, 6, 2
    assert E * (H // 8) * Hp > 2 ** 33 and E * (H // G) * Hp > 2 ** 31
    d = m.make_dims(1, E, 0, T, K)
    ids = np.array([[E - 1, 0], [E - 2, E - 1], [0, E - 2], [E - 1, E - 2], [E - 2, 0], [0, E - 1]])
    gates = routing(T, E, K, 12)[1]
    words = torch.empty((E, H // 8, Hp), dtype=torch.int32, device=DEV)
    scales = torch.empty((E, H // G, Hp), dtype=BF, device=DEV)
    values = {}
    for e in (0, E - 2, E - 1):
        v = torch.empty((1, H, Hp), device=DEV)
        say("weights of expert", e)
        m.moonep_save4(1, H, Hp, G, rand_tensor((1, H, Hp), BF, e, H ** -0.5), words[e:e + 1], scales[e:e + 1])
        m.moonep_load4(1, H, Hp, G, words[e:e + 1], scales[e:e + 1], v)
        values[e] = v[0].double()
    X = rand_tensor((T, H), BF, 13)
    for rows in (T, 1):  # an expert's block, and a token's
        dr = m.make_dims(1, E, 0, rows, K)
        out, ws = Guarded((rows, Hp), F32), space(m, dr, H, Hp)
        say("few_layer4 past 2^33 words", rows)
        m.moonep_few_layer4(dr, H, Hp, G, X[:rows], i32(ids[:rows]), f32(gates[:rows]), words, scales, out.view, ws.view)
        torch.cuda.synchronize()
        for t in range(rows):
            terms = [(float(gates[t, k]), values[int(ids[t, k])]) for k in range(K)]
            ref = sum(g * (X[t].double() @ w) for g, w in terms)
            size = sum(g * (X[t].double().abs() @ w.abs()) for g, w in terms)
            # a wrong expert or scale is off by the size of the terms, of which the roundings are far below a thousandth
            assert float(((out.view[t].double() - ref).abs() / size).max()) < 1e-3
        assert out.intact() and ws.intact()


def test_save4_and_load4_past_32_bits(m):
    """Expert offsets past 2^31 words and 2^34 weights, within one call."""
    E, H, N, G = 2100, 2048, 4096, 64
    assert E * H * N > 2 ** 34 and E * (H // 8) * N > 2 ** 31
    few_experts = (0, 1049, E - 1)
    W = torch.zeros((E, H, N), dtype=BF, device=DEV)
    for e in few_experts:
        W[e] = rand_tensor((H, N), BF, e, 0.1)
    words = torch.empty((E, H // 8, N), dtype=torch.int32, device=DEV)
    scales = torch.empty((E, H // G, N), dtype=BF, device=DEV)
    say("save4 past 2^31 words")
    m.moonep_save4(E, H, N, G, W, words, scales)
    torch.cuda.synchronize()
    kept = {}
    for e in few_experts:
        one = torch.empty((1, H // 8, N), dtype=torch.int32, device=DEV), torch.empty((1, H // G, N), dtype=BF, device=DEV)
        m.moonep_save4(1, H, N, G, W[e:e + 1].clone(), *one)
        torch.cuda.synchronize()
        assert torch.equal(words[e], one[0][0]) and torch.equal(scales[e], one[1][0])
        kept[e] = torch.empty((1, H, N), dtype=BF, device=DEV)
        m.moonep_load4(1, H, N, G, *one, kept[e])
    assert not scales[E - 2].any() and torch.equal(words[E - 2], words[1])
    W.fill_(1.0)
    say("load4 past 2^31 words")
    m.moonep_load4(E, H, N, G, words, scales, W)
    torch.cuda.synchronize()
    for e in few_experts:
        assert torch.equal(W[e], kept[e][0])
    assert not W[E - 2].any() and not W[1].any()


@pytest.mark.parametrize("T", [6, 40])
def test_wide_tiles_captured(m, T):
    # eight columns to a lane: sums in more than 64 KB of LDS, which the launch asks for while a graph is captured too
    E, K, H, Hp = 8, 2, 96, 6200
    d = m.make_dims(1, E, 0, T, K)
    w = rand_tensor((E, H, Hp), BF, 20, H ** -0.5)
    X, ids, gates = rand_tensor((T, H), BF, 21), i32(routing(T, E, K, 22)[0]), f32(routing(T, E, K, 22)[1])
    out, ws = Guarded((T, Hp), F32), space(m, d, H, Hp)

    def call():
        m.moonep_few_layer(d, H, Hp, X, ids, gates, w, out.view, ws.view)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    say("few_layer wide tiles captured", T)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        call()
    for r in range(3):
        X.copy_(rand_tensor((T, H), BF, 30 + r))
        ids.copy_(i32(routing(T, E, K, 40 + r)[0]))
        call()
        torch.cuda.synchronize()
        want = out.view.clone()
        out.view.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view, want)
    x, idn = np64(X), ids.cpu().numpy()
    ref, size = few.few_layer(x, idn, np64(gates), np64(w))
    scale = few.few_layer(np.abs(x), idn, np64(gates), np.abs(np64(w)))[0]
    assert np.all(np.abs(np64(out.view) - ref) <= 2 * (H + K + 16) * U * scale)
    assert out.intact() and ws.intact()


@pytest.mark.parametrize("bits", [16, 4])
def test_no_tokens(m, bits):
    L = m.MoeFew(2, 8, 0, 2, 64, 32, device=DEV, bits=bits, norm=True, router="sigmoid", router_bias=True)
    say("MoeFew without tokens", bits)
    L.forward()
    torch.cuda.synchronize()
    assert L.out.numel() == 0 and L.topk_idx.numel() == 0
    F = m.MoeFFN(2, 8, 4, 0, 2, 64, 32, device=DEV, router="softmax", backward=True)
    say("MoeFFN with a router without tokens")
    F.forward()
    F.backward()
    torch.cuda.synchronize()
    assert F.dlogits.numel() == 0
