"""Which row buffers layers may share, and on which device a layer's calls and checks run (CPU only: nothing runs)."""
import pytest
import torch

import load_balanced_dispatch_amd as m
from load_balanced_dispatch_amd import _lib

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


class FakeDevices:
    """Stands for two GPUs whose launches differ in size: what the binding asks of torch and of the library."""

    def __init__(self, monkeypatch, sizes):
        self.current, self.sizes = 0, sizes
        outer = self

        class on:
            def __init__(self, device):
                self.to = torch.device(device).index if not isinstance(device, int) else device

            def __enter__(self):
                self.back, outer.current = outer.current, self.to

            def __exit__(self, *exc):
                outer.current = self.back

        class Library:
            moonep_layernorm_backward_workspace_bytes = staticmethod(lambda d, H: sizes[outer.current])
            moonep_layernorm_backward8 = moonep_layernorm_backward = None

        monkeypatch.setattr(torch.cuda, "device", on)
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: self.current)
        monkeypatch.setattr(_lib, "_LIB", Library)


class FakeBytes:
    """A uint8 tensor of n bytes on a device."""

    def __init__(self, n, device):
        self.n, self.device = n, device

    def numel(self):
        return self.n

    def element_size(self):
        return 1

    def get_device(self):
        return self.device


def test_the_workspace_is_sized_by_its_own_device(monkeypatch):
    # 100 bytes are enough on the current device, not on the one that the tensors are on and the launch goes to
    gpus = FakeDevices(monkeypatch, [64, 4096])
    d = m.make_dims(2, 4, 1, 6, 2)
    f32 = torch.zeros(1)
    for call in (lambda ws: m.moonep_layernorm_backward8(d, 64, f32, f32, f32, f32, f32, f32, f32, None, ws),
                 lambda ws: m.moonep_layernorm_backward(d, 64, f32, f32, f32, f32, f32, f32, f32, None, ws)):
        with pytest.raises(ValueError, match="workspace too small: 4096 bytes"):
            call(FakeBytes(100, 1))
        with pytest.raises(ValueError, match="dY must be a device tensor"):  # the size is enough: the next check
            call(FakeBytes(4096, 1))
        with pytest.raises(ValueError, match="dY must be a device tensor"):
            call(FakeBytes(100, 0))
    assert gpus.current == 0


def test_a_layers_workspace_is_sized_by_its_device(monkeypatch):
    FakeDevices(monkeypatch, {0: 64, -1: 4096})  # the layer is on the host, which counts as device -1
    monkeypatch.setattr(_lib, "moonep_plan_workspace_bytes", lambda d: 1)
    monkeypatch.setattr(_lib, "moonep_group_gemm_workspace_bytes", lambda d: 1)
    monkeypatch.setattr(_lib, "moonep_wgrad_workspace_bytes", lambda d: 1)
    assert make(backward=True, norm=True).ws_norm.numel() == 4096


@pytest.mark.parametrize("kw", [dict(), dict(norm=True), dict(norm=True, save8=True)])
def test_a_layers_passes_run_on_its_device(monkeypatch, kw):
    # some of the calls go to the current device's stream and some to their tensors': both are the layer's
    L = make(backward=True, **kw)
    gpus = FakeDevices(monkeypatch, [64, 4096])
    L.X = FakeBytes(1, 1)
    seen = []
    L.forward_calls = L.backward_calls = lambda: [("step", lambda: seen.append(gpus.current))] * 2
    L.forward()
    L.backward()
    assert seen == [1] * 4 and gpus.current == 0


def test_the_gradient_of_the_norms_rows_is_shared_too():
    # it lives inside one backward pass only, like the row buffers
    a = make(backward=True, norm=True, save8=True)
    b = make(backward=True, norm=True, save8=True, scratch=a.scratch)
    assert b.dXn.data_ptr() == a.dXn.data_ptr() and b.dX.data_ptr() != a.dX.data_ptr()
    assert a.dXn.shape == a.dX.shape and a.dXn.dtype == torch.float32
    # buffers from a layer without a norm get one with the first layer that has
    c = make(backward=True, save8=True)
    assert "dXn" not in c.scratch
    d, e = (make(backward=True, norm=True, save8=True, scratch=c.scratch) for _ in range(2))
    assert d.Xp.data_ptr() == c.Xp.data_ptr() and e.dXn.data_ptr() == d.dXn.data_ptr()
    # the same rows of other tokens (12 of one pair each for 6 of two): its own, the others' stays
    f = m.MoeFFN(2, 4, 1, 12, 1, 64, 32, device="cpu", backward=True, norm=True, save8=True, scratch=a.scratch)
    assert f.Xp.data_ptr() == a.Xp.data_ptr() and f.dXn.shape == f.dX.shape
    assert a.scratch["dXn"].data_ptr() == a.dXn.data_ptr() != f.dXn.data_ptr()
    # a layer that keeps everything has its own
    assert make(backward=True, norm=True).dXn.shape == a.dXn.shape
