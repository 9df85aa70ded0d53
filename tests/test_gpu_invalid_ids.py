"""Routing ids outside [0, E): their pairs get no row, some rows no pair, and the gated FFN that keeps 8-bit checkpoints
must give what the one that keeps everything gives (GPU)."""
import numpy as np
import pytest
import torch

from tests import test_gpu_ffn8 as ffn8
from tests import test_gpu_stages as stages
from tests.gpu_util import npi, say
from tests.plan_checks import random_routing

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def m():
    import load_balanced_dispatch_amd as mod
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    return mod


def some_invalid(rng, idx, E, share):
    idx = np.array(idx)
    bad = rng.random(idx.shape) < share
    return np.where(bad, rng.choice([-1, E, E + 7, -2 ** 31, 2 ** 31 - 1], idx.shape), idx), bad


@pytest.mark.parametrize("planner", ["prefix", "mincopy"])
@pytest.mark.parametrize("share", [0.0, 0.02, 0.5, 1.0])
@pytest.mark.parametrize("R,E,B,S,K", [(2, 8, 2, 50, 3), (1, 4, 0, 700, 2), (4, 16, 4, 1, 2), (8, 64, 8, 301, 6),
                                       (3, 6, 1, 1, 1), (2, 2048, 1, 3, 1030)])
def test_plan_tells_rows_without_a_pair(m, R, E, B, S, K, share, planner):
    rng = np.random.default_rng(S)
    idx, bad = some_invalid(rng, random_routing(rng, R, S, K, E, 1.5), E, share)
    say("plan", R, E, B, S, K, "invalid share", share, planner)
    _, out = stages.gpu_plan(m, idx.astype(np.int32), E, B, planner=planner)
    dest = npi(out["dest"]).reshape(-1)
    assert np.array_equal(dest < 0, bad.reshape(-1)) and np.all(dest[bad.reshape(-1)] == -1)
    src = np.full(R * S * K, -1)
    src[dest[dest >= 0]] = np.nonzero(dest >= 0)[0]
    assert np.array_equal(npi(out["src"]), src)


# The two FFNs' gradients are within 5% of their norms of each other (derived at the head of test_gpu_ffn8.py).
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("norm", [True, False])
def test_ffn_with_checkpoints_and_invalid_ids(m, dtype, norm):
    dims = (4, 16, 2, 128, 4, 256, 192)
    whole, kept, again = (m.MoeFFN(*dims, dtype=dtype, backward=True, norm=norm, save8=s) for s in (False, True, True))
    rng = np.random.default_rng(11)
    for step, share in enumerate((0.1, 0.0, 0.3, 1.0)):
        for L in (whole, kept, again):
            ffn8.fill(L, 40 + step)
            for t in (L.dW_gu_home, L.dW_down_home) + ((L.dgamma, L.dbeta) if norm else ()):
                t.zero_()
        idx, bad = some_invalid(rng, npi(kept.topk_idx), kept.d.E, share)
        for L in (whole, kept, again):
            L.topk_idx.copy_(torch.as_tensor(idx.astype(np.int32)))
        for t in again.scratch.values():  # rows without a pair hold whatever was there: it must not matter
            t.fill_(float("nan"))
        for L in (whole, kept, again):
            say("FFN", "save8" if L.save8 else "whole", dtype, "invalid share", share)
            L.forward()
            L.backward()
        torch.cuda.synchronize()
        a, b, c = ffn8.grads(whole), ffn8.grads(kept), ffn8.grads(again)
        valid = torch.as_tensor(~bad, device=kept.dgates.device)
        for g in (a, b, c):
            g["dgates"] = g["dgates"][valid]
        assert torch.equal(a["out"], b["out"])
        for n in a:
            off = float((a[n].double() - b[n].double()).norm())
            assert off <= 0.05 * float(a[n].double().norm()), (step, n, off)
            assert torch.equal(b[n], c[n]), (step, n)


@pytest.mark.parametrize("kw", [dict(), dict(save8=True), dict(save8=True, norm=True)])
def test_gates_of_invalid_ids_have_no_gradient(m, kw):
    # whatever an earlier step left there
    L = m.MoeFFN(4, 16, 2, 128, 4, 256, 192, backward=True, **kw)
    rng = np.random.default_rng(12)
    for step in range(2):
        ffn8.fill(L, 60 + step)
        idx, bad = some_invalid(rng, npi(L.topk_idx), L.d.E, 0.2)
        L.topk_idx.copy_(torch.as_tensor(idx.astype(np.int32)))
        L.dgates.fill_(7.0)
        say("FFN", kw, "gates of invalid ids, step", step)
        L.forward()
        L.backward()
        torch.cuda.synchronize()
        dropped = torch.as_tensor(bad, device=L.dgates.device)
        assert not bool(L.dgates[dropped].any())
        assert bool((L.dgates[~dropped] != 7.0).all())
