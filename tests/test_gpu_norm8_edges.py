"""Edges of the layer norm and of the 8-bit checkpoint kernels (GPU): magnitudes near float32's end.

Tolerances are those derived at the head of test_gpu_norm8.py.
"""
import numpy as np
import pytest
import torch

from oracle import norm8
from tests import test_gpu_norm8 as base
from tests.gpu_util import DEV, Guarded, f32, np64, rand_tensor, say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def m():
    import load_balanced_dispatch_amd as mod
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    return mod


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [40, 600])  # one launch; row blocks and a fold
@pytest.mark.parametrize("H", [100, 1100, 4000, 8200, 16400])  # each layout of the backward, lanes past the row's end
def test_layernorm_backward_of_large_constant_rows(m, dtype, rows, H):
    # mean * rstd passes float32's end, but z is 0 in every column and the gradient is finite.  Magnitudes up to
    # 2^120 and rstd = 1 / sqrt(1e-5), both exactly representable as given, so z = (x - mean) rstd is exact here
    d = m.make_dims(1, 1, 0, rows, 1)
    x = rand_tensor((rows, H), F32, H).to(dtype)
    big = [0, rows // 2, rows - 1]
    x[big] = torch.tensor([[2.0 ** 120], [-(2.0 ** 120)], [2.0 ** 126]], device=DEV).to(dtype)
    x64 = np64(x)
    rm = x64.mean(axis=1)
    rr = 1 / np.sqrt(x64.var(axis=1) + 1e-5)
    mean, rstd = f32(rm), f32(rr)
    assert np.array_equal(np64(mean)[big], x64[big, 0])
    z = (x64 - np64(mean)[:, None]) * np64(rstd)[:, None]
    gamma, dY = rand_tensor((H,), F32, 1), rand_tensor((rows, H), F32, 2)
    dx, dg, db = norm8.layernorm_backward(np64(dY), z, np64(rstd), np64(gamma))
    gy = np.abs(np64(dY) * np64(gamma))
    terms = gy + gy.mean(axis=1, keepdims=True) + np.abs(z) * (gy * np.abs(z)).mean(axis=1, keepdims=True)
    ws = torch.empty(m.moonep_layernorm_backward_workspace_bytes(d, H), dtype=torch.uint8, device=DEV)
    for by in (0, 1):
        dX, dgam, dbet = Guarded((rows, H), F32), Guarded((H,), F32), Guarded((H,), F32)
        dgam.view.zero_()
        dbet.view.zero_()
        say("layernorm_backward, large constant rows", dtype, rows, H, "offset", by)
        m.moonep_layernorm_backward(d, H, base.at_offset(dY, by), base.at_offset(x, by), mean, rstd, gamma, dX.view,
                                    dgam.view, dbet.view, ws)
        torch.cuda.synchronize()
        assert dX.intact() and dgam.intact() and dbet.intact()
        assert np.all(np.abs(np64(dX.view) - dx) <= (57 + 8) * U * np64(rstd)[:, None] * terms)
        for got, ref, each in ((dgam.view, dg, np64(dY) * z), (dbet.view, db, np64(dY))):
            assert np.all(np.abs(np64(got) - ref) <= (rows + 32) * U * np.abs(each).sum(axis=0) + U * np.abs(ref))
