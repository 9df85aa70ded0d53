"""Refusals of the layer norm and the 8-bit checkpoint calls: all on the host, before anything is enqueued
(CPU only: no call here reaches a kernel, and no pointer is dereferenced)."""
import pytest
import torch

import load_balanced_dispatch_amd as m
from load_balanced_dispatch_amd import _lib

L = _lib.lib()
BF, F32 = _lib.MOONEP_BF16, _lib.MOONEP_F32
D = m.make_dims(2, 4, 1, 3, 2)
P = [0x10000 * (i + 1) for i in range(12)]  # never dereferenced

# name -> (call with a list of pointers, number of pointers, of which optional)
CALLS = {
    "moonep_save8": (lambda d, w, t, p: L.moonep_save8(4, w, t, *p, None), 3, ()),
    "moonep_load8": (lambda d, w, t, p: L.moonep_load8(4, w, t, *p, None), 3, ()),
    "moonep_swiglu_save8": (lambda d, w, t, p: L.moonep_swiglu_save8(d, w, t, *p, None), 4, ()),
    "moonep_swiglu_backward8": (lambda d, w, t, p: L.moonep_swiglu_backward8(d, w, t, *p, None), 8, ()),
    "moonep_dispatch8": (lambda d, w, t, p: L.moonep_dispatch8(d, w, t, *p, None), 6, (2, 3)),
    "moonep_combine_backward_ungated":
        (lambda d, w, t, p: L.moonep_combine_backward_ungated(d, w, t, *p, None), 3, ()),
    "moonep_layernorm": (lambda d, w, t, p: L.moonep_layernorm(d, w, t, *p[:3], 1e-5, *p[3:], None), 8, (2, 4, 5)),
    "moonep_layernorm_dispatch":
        (lambda d, w, t, p: L.moonep_layernorm_dispatch(d, w, t, *p[:3], 1e-5, *p[3:], None), 9, (2, 5, 6)),
    "moonep_layernorm_backward": (lambda d, w, t, p: L.moonep_layernorm_backward(d, w, t, *p, None), 9, (7,)),
    "moonep_layernorm_backward8":
        (lambda d, w, t, p: L.moonep_layernorm_backward8(d, w, *p, None), 9, (7,)),
}
WITH_DIMS = [n for n in CALLS if n not in ("moonep_save8", "moonep_load8")]
WITH_TYPE = [n for n in CALLS if n != "moonep_layernorm_backward8"]


@pytest.mark.parametrize("name", WITH_DIMS)
@pytest.mark.parametrize("dims,msg", [((8, 63, 8, 16, 2), "multiple of R"), ((2, 4, 1, -1, 2), "S must be"),
                                      ((2, 4, 1, 3, 5), "K must be"), ((1024, 1024, 1, 1 << 20, 8), "2^31")])
def test_bad_dims(name, dims, msg):
    call, n, _ = CALLS[name]
    assert call(m.make_dims(*dims), 8, BF, P[:n]) == _lib.MOONEP_EINVAL
    assert msg in m.last_error() and name in m.last_error()
    assert m.moonep_layernorm_backward_workspace_bytes(m.make_dims(*dims), 8) == 0


@pytest.mark.parametrize("name", list(CALLS))
def test_bad_width(name):
    call, n, _ = CALLS[name]
    too_wide = 32769 if "layernorm" in name else (1 << 30) + 1
    for w in (0, -3, too_wide):
        assert call(D, w, BF, P[:n]) == _lib.MOONEP_EINVAL
        assert "must be in [1" in m.last_error()


@pytest.mark.parametrize("name", WITH_TYPE)
def test_bad_dtype(name):
    call, n, _ = CALLS[name]
    assert call(D, 8, 7, P[:n]) == _lib.MOONEP_EINVAL
    assert "dtype" in m.last_error()


@pytest.mark.parametrize("name", list(CALLS))
def test_null_pointers(name):
    call, n, optional = CALLS[name]
    for i in range(n):
        if i in optional:
            continue
        p = list(P[:n])
        p[i] = None
        assert call(D, 8, BF, p) == _lib.MOONEP_EINVAL, i
        assert any(s in m.last_error() for s in ("null", "go together")), m.last_error()


def test_arguments_that_go_together():
    assert L.moonep_dispatch8(D, 8, BF, P[0], P[1], None, P[3], P[4], P[5], None) == _lib.MOONEP_EINVAL
    assert "beta without gamma" in m.last_error()
    for eps in (0.0, -1e-5, float("nan"), float("inf")):
        assert L.moonep_layernorm(D, 8, BF, P[0], P[1], None, eps, P[2], None, None, None, None, None) == \
            _lib.MOONEP_EINVAL
        assert "eps" in m.last_error()


@pytest.mark.parametrize("name,which", [("moonep_save8", 0), ("moonep_load8", 2), ("moonep_swiglu_save8", 0),
                                        ("moonep_swiglu_save8", 1), ("moonep_swiglu_backward8", 2),
                                        ("moonep_swiglu_backward8", 5), ("moonep_swiglu_backward8", 6),
                                        ("moonep_dispatch8", 5), ("moonep_combine_backward_ungated", 0),
                                        ("moonep_combine_backward_ungated", 2), ("moonep_layernorm_backward", 0),
                                        ("moonep_layernorm_backward8", 0), ("moonep_layernorm_backward8", 5),
                                        ("moonep_layernorm", 0), ("moonep_layernorm", 3),
                                        ("moonep_layernorm_dispatch", 0), ("moonep_layernorm_dispatch", 4),
                                        ("moonep_layernorm_backward", 1)])
def test_rows_off_their_elements_alignment(name, which):
    call, n, _ = CALLS[name]
    p = list(P[:n])
    p[which] += 1
    assert call(D, 8, BF, p) == _lib.MOONEP_EINVAL
    assert "aligned" in m.last_error()


def test_workspace_alignment_and_rows():
    for name, at in (("moonep_layernorm_backward", 8), ("moonep_layernorm_backward8", 8)):
        call, n, _ = CALLS[name]
        p = list(P[:n])
        p[at] += 128
        assert call(D, 8, BF, p) == _lib.MOONEP_EINVAL
        assert "256-byte" in m.last_error()
    assert L.moonep_save8(-1, 8, BF, *P[:3], None) == _lib.MOONEP_EINVAL
    assert L.moonep_load8(1 << 60, 8, BF, *P[:3], None) == _lib.MOONEP_EINVAL


def test_nothing_to_do_is_ok():
    d = m.make_dims(2, 4, 1, 0, 2)
    for name, (call, n, _) in CALLS.items():
        if name in WITH_DIMS:
            assert call(d, 8, BF, [None] * n) == _lib.MOONEP_OK, m.last_error()
    assert L.moonep_save8(0, 8, BF, None, None, None, None) == _lib.MOONEP_OK
    assert L.moonep_load8(0, 8, F32, None, None, None, None) == _lib.MOONEP_OK


def test_block_counts():
    assert [m.moonep_save8_blocks(c) for c in (-1, 0, 1, 32, 33, 2 ** 31 - 1)] == [0, 0, 1, 1, 2, 2 ** 26]


def test_binding_refuses_host_and_wrong_tensors():
    t = dict(dtype=torch.int8)
    with pytest.raises(ValueError, match="device tensor"):
        m.moonep_save8(4, 8, torch.zeros(4, 8), torch.zeros(4, 8, **t), torch.zeros(4, 1, dtype=torch.uint8))
    with pytest.raises(ValueError, match="required"):
        m.moonep_layernorm(D, 8, None, None, None, 1e-5, None, None, None)
