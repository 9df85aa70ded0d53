"""Which row buffers layers may share, and on which device a layer's calls and checks run (CPU only: nothing runs)."""
import pytest
import torch

import load_balanced_dispatch_amd as m

DIMS = (2, 4, 1, 6, 2, 64, 32)


def make(**kw):
    return m.MoeFFN(*DIMS, device="cpu", **kw)


@pytest.mark.parametrize("norm", [False, True])
def test_a_layer_whose_backward_reads_its_rows_gives_none_away(norm):
    a = make(backward=True, norm=norm)
    assert a.scratch is None
    for kw in (dict(), dict(backward=True, save8=True)):
        b = make(scratch=a.scratch, **kw)  # None: buffers of its own
        mine = {t.data_ptr() for t in (a.Xp, a.Ygu, a.A, a.Zp, a.dZp, a.dA, a.dYgu, a.dXp)}
        assert not mine & {t.data_ptr() for t in (b.Xp, b.Ygu, b.A, b.Zp)}


def test_layers_without_a_backward_share():
    a = make()
    b = make(scratch=a.scratch)
    assert b.Ygu.data_ptr() == a.Ygu.data_ptr()


def test_rows_on_another_device_are_refused():
    a = make(backward=True, save8=True)
    for name in a.scratch:
        other = {k: torch.empty_like(v, device="meta") if k == name else v for k, v in a.scratch.items()}
        with pytest.raises(ValueError, match=f"scratch must hold {name} .*on cpu"):
            make(backward=True, save8=True, scratch=other)
