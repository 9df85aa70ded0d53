"""Refusals of the router, the layer for few tokens and the 4-bit weights: all on the host, before anything is enqueued
(CPU only: no call here reaches a kernel, and no pointer is dereferenced)."""
import pytest
import torch

import load_balanced_dispatch_amd as m
from load_balanced_dispatch_amd import _lib

L = _lib.lib()
BF, F32 = _lib.MOONEP_BF16, _lib.MOONEP_F32
D = m.make_dims(2, 4, 0, 3, 2)
P = [0x10000 * (i + 1) for i in range(12)]  # never dereferenced

# name -> (call with dims, width, type and a list of pointers, number of pointers, of which optional, of which workspace)
FEW = {
    "moonep_few_layer": (lambda d, w, t, p: L.moonep_few_layer(d, w, w, t, *p, None), 6, (2,), 5),
    "moonep_few_ffn": (lambda d, w, t, p: L.moonep_few_ffn(d, w, w, t, *p, None), 7, (2,), 6),
    "moonep_few_layer4": (lambda d, w, t, p: L.moonep_few_layer4(d, w, w, 32, t, *p, None), 7, (2,), 6),
    "moonep_few_ffn4": (lambda d, w, t, p: L.moonep_few_ffn4(d, w, w, 32, t, *p, None), 9, (2,), 8),
}
ROUTE = {
    "moonep_route": (lambda d, p, score=0, scale=1.0: L.moonep_route(d, score, 1, scale, *p, None), 4, (1,)),
    "moonep_route_backward":
        (lambda d, p, score=0, scale=1.0: L.moonep_route_backward(d, score, 1, scale, *p, None), 4, ()),
}
FOUR = {
    "moonep_save4": lambda E, H, N, G, t, p: L.moonep_save4(E, H, N, G, t, *p, None),
    "moonep_load4": lambda E, H, N, G, t, p: L.moonep_load4(E, H, N, G, t, *p, None),
}
BAD_DIMS = [((8, 63, 8, 16, 2), "multiple of R"), ((2, 4, 1, -1, 2), "S must be"), ((2, 4, 1, 3, 5), "K must be"),
            ((1024, 1024, 1, 1 << 20, 8), "2^31")]


@pytest.mark.parametrize("dims,msg", BAD_DIMS)
def test_bad_dims(dims, msg):
    d = m.make_dims(*dims)
    for name, (call, n, *_) in FEW.items():
        assert call(d, 8, BF, P[:n]) == _lib.MOONEP_EINVAL
        assert msg in m.last_error() and name in m.last_error()
    for name, (call, n, _) in ROUTE.items():
        assert call(d, P[:n]) == _lib.MOONEP_EINVAL
        assert msg in m.last_error() and name in m.last_error()
    assert m.moonep_few_workspace_bytes(d, 8, 8) == 0


def test_too_many_pairs():
    assert m.MOONEP_FEW_PAIRS == 1024
    d = m.make_dims(1, 4, 0, 513, 2)
    for name, (call, n, *_) in FEW.items():
        assert call(d, 8, BF, P[:n]) == _lib.MOONEP_EINVAL
        assert "exceeds 1024" in m.last_error()
    assert m.moonep_few_workspace_bytes(d, 8, 8) == 0
    assert m.moonep_few_workspace_bytes(m.make_dims(1, 4, 0, 512, 2), 8, 8) > 0


def test_bad_width_and_type():
    for name, (call, n, *_) in FEW.items():
        for w in (0, -3, 65537):
            assert call(D, w, BF, P[:n]) == _lib.MOONEP_EINVAL
            assert "must be in [1" in m.last_error()
            assert m.moonep_few_workspace_bytes(D, w, 8) == 0 and m.moonep_few_workspace_bytes(D, 8, w) == 0
        assert call(D, 8, 7, P[:n]) == _lib.MOONEP_EINVAL
        assert "dtype" in m.last_error()


def test_group_sizes():
    for G in (0, 16, 33, 96, 256, -32):
        assert L.moonep_few_layer4(D, 8, 8, G, BF, *P[:7], None) == _lib.MOONEP_EINVAL
        assert "G must be" in m.last_error()
        assert L.moonep_few_ffn4(D, 8, 8, G, BF, *P[:9], None) == _lib.MOONEP_EINVAL
        for name, call in FOUR.items():
            assert call(2, 8, 8, G, BF, P[:3]) == _lib.MOONEP_EINVAL
            assert "G must be" in m.last_error() and name in m.last_error()


def test_null_pointers():
    for name, (call, n, optional, _) in FEW.items():
        for i in range(n):
            if i not in optional:
                assert call(D, 8, BF, P[:i] + [None] + P[i + 1:n]) == _lib.MOONEP_EINVAL, (name, i)
                assert "null" in m.last_error()
    for name, (call, n, optional) in ROUTE.items():
        for i in range(n):
            if i not in optional:
                assert call(D, P[:i] + [None] + P[i + 1:n]) == _lib.MOONEP_EINVAL, (name, i)
                assert "null" in m.last_error()
    for name, call in FOUR.items():
        for i in range(3):
            assert call(2, 8, 8, 32, BF, P[:i] + [None] + P[i + 1:3]) == _lib.MOONEP_EINVAL, (name, i)
            assert "null" in m.last_error()


def test_alignment():
    for name, (call, n, optional, ws) in FEW.items():
        p = list(P[:n])
        p[ws] += 128
        assert call(D, 8, BF, p) == _lib.MOONEP_EINVAL
        assert "256-byte" in m.last_error()
        for i in range(n):
            if i == ws:
                continue
            p = list(P[:n])
            p[i] += 1
            assert call(D, 8, BF, p) == _lib.MOONEP_EINVAL, (name, i)
            assert "aligned" in m.last_error()
    for name, (call, n, _) in ROUTE.items():
        for i in range(n):
            p = list(P[:n])
            p[i] += 2
            assert call(D, p) == _lib.MOONEP_EINVAL, (name, i)
            assert "aligned" in m.last_error()
    for name, call in FOUR.items():
        for i in range(3):
            p = list(P[:3])
            p[i] += 1
            assert call(2, 8, 8, 32, BF, p) == _lib.MOONEP_EINVAL, (name, i)
            assert "aligned" in m.last_error()


def test_router_arguments():
    for name, (call, n, _) in ROUTE.items():
        assert call(D, P[:n], score=2) == _lib.MOONEP_EINVAL
        assert "score" in m.last_error()
        for scale in (float("nan"), float("inf")):
            assert call(D, P[:n], scale=scale) == _lib.MOONEP_EINVAL
            assert "scale" in m.last_error()
        assert call(m.make_dims(1, 4097, 0, 3, 2), P[:n]) == _lib.MOONEP_EINVAL
        assert "exceeds 4096" in m.last_error()
        assert call(m.make_dims(1, 4, 0, (1 << 25) + 1, 2), P[:n]) == _lib.MOONEP_EINVAL
        assert "exceeds 33554432" in m.last_error()
    with pytest.raises(ValueError, match="unknown score"):
        m.moonep_route(D, "tanh", True, 1.0, None, None, None, None)


def test_sizes_of_4_bit_weights():
    for name, call in FOUR.items():
        for E, H, N in ((-1, 8, 8), (2, 0, 8), (2, 8, 0), (2, 65537, 8), (2, 8, 65537)):
            assert call(E, H, N, 32, BF, P[:3]) == _lib.MOONEP_EINVAL
            assert "must be" in m.last_error()
        assert call(1 << 20, 4096, 8192, 32, BF, P[:3]) == _lib.MOONEP_EINVAL
        assert "grid too large" in m.last_error()
        assert call(2, 8, 8, 32, 9, P[:3]) == _lib.MOONEP_EINVAL
        assert "dtype" in m.last_error()


def test_grid_of_4_bit_weights():
    # 8 waves to 128 rows and 256 columns: from 2^23 such tiles on the grid would have 2^32 threads
    for name, call in FOUR.items():
        for E, H, N in ((1 << 23, 8, 8), (1 << 22, 129, 8), (1 << 22, 8, 257), ((1 << 24) - 1, 8, 8)):
            assert call(E, H, N, 32, BF, P[:3]) == _lib.MOONEP_EINVAL
            assert "grid too large" in m.last_error() and name in m.last_error()


def test_nothing_to_do_is_ok():
    d = m.make_dims(2, 4, 1, 0, 2)
    for call, n, *_ in FEW.values():
        assert call(d, 8, BF, [None] * n) == _lib.MOONEP_OK, m.last_error()
    for call, n, _ in ROUTE.values():
        assert call(d, [None] * n) == _lib.MOONEP_OK, m.last_error()
    for call in FOUR.values():
        assert call(0, 8, 8, 32, F32, [None] * 3) == _lib.MOONEP_OK, m.last_error()


def test_binding_refuses_host_and_wrong_tensors():
    x = torch.zeros(2, 3, 8)
    with pytest.raises(ValueError, match="device tensor"):
        m.moonep_few_layer(D, 8, 8, x, x, x, x, x, None)
    with pytest.raises(ValueError, match="too small"):
        m.moonep_few_layer(D, 8, 8, x, x, x, x, x, torch.zeros(1))
    with pytest.raises(ValueError, match="required"):
        m.moonep_few_ffn(D, 8, 8, None, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="device tensor"):
        m.moonep_route(D, "sigmoid", True, 1.0, torch.zeros(2, 3, 4), None, torch.zeros(2, 3, 2), torch.zeros(2, 3, 2))
    with pytest.raises(ValueError, match="device tensor"):
        m.moonep_save4(1, 8, 8, 32, torch.zeros(1, 8, 8), None, None)
