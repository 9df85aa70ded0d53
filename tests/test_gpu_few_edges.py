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
