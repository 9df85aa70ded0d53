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
