"""ctypes binding of libmoonep.so: the same entry points, taking torch tensors.

Argument marshalling only: every step of the layer runs in the HIP kernels of
libmoonep.so.  Tensors must be CUDA (HIP) tensors, contiguous, with the shapes
and dtypes that include/moonep.h documents; calls are enqueued on the current
torch stream (or the one passed) and never synchronise.  A nonzero return code
raises MoonepError carrying the library's message.

There is no fallback: if libmoonep.so is missing or fails to load, importing
this module raises.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoonep.so")

MOONEP_F32, MOONEP_BF16 = 0, 1
MOONEP_PLAN_PREFIX, MOONEP_PLAN_MINCOPY = 0, 1
MOONEP_SCORE_SOFTMAX, MOONEP_SCORE_SIGMOID = 0, 1
SCORES = {"softmax": MOONEP_SCORE_SOFTMAX, "sigmoid": MOONEP_SCORE_SIGMOID}
MOONEP_FEW_PAIRS = 1024
PLANNERS = {"prefix": MOONEP_PLAN_PREFIX, "mincopy": MOONEP_PLAN_MINCOPY}
MOONEP_OK, MOONEP_EINVAL, MOONEP_EHIP, MOONEP_EUNSUPPORTED = 0, -1, -2, -3
_CODES = {MOONEP_EINVAL: "EINVAL", MOONEP_EHIP: "EHIP", MOONEP_EUNSUPPORTED: "EUNSUPPORTED"}


class MoonepError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"{_CODES.get(code, code)}: {message}")
        self.code = code


class Dims(ctypes.Structure):
    _fields_ = [("R", ctypes.c_int32), ("E", ctypes.c_int32), ("B", ctypes.c_int32),
                ("S", ctypes.c_int32), ("K", ctypes.c_int32)]

    def __repr__(self):
        return f"Dims(R={self.R}, E={self.E}, B={self.B}, S={self.S}, K={self.K})"

    @property
    def P(self):
        return self.S * self.K

    @property
    def N(self):
        return self.R * self.S * self.K


def _load():
    # torch must bring in its HIP runtime first: libmoonep.so then binds to that same
    # libamdhip64 (same soname) instead of loading a second runtime from /opt/rocm,
    # and two HIP runtimes in one process leave the library's launches without a device.
    import torch  # noqa: F401
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python load_balanced_dispatch_amd/build.py`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    sig = {
        "moonep_last_error": (ctypes.c_char_p, []),
        "moonep_plan_workspace_bytes": (sz, [Dims]),
        "moonep_plan": (ctypes.c_int, [Dims, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "moonep_plan_ex": (ctypes.c_int, [Dims, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "moonep_plan_static_scratch_bytes": (sz, []),
        "moonep_plan_static": (ctypes.c_int, [Dims, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "moonep_dispatch": (ctypes.c_int, [Dims, i32, ctypes.c_int, vp, vp, vp, vp]),
        "moonep_prefetch": (ctypes.c_int, [Dims, i32, i32, ctypes.c_int, vp, vp, vp, vp]),
        "moonep_group_gemm_workspace_bytes": (sz, [Dims]),
        "moonep_group_gemm": (ctypes.c_int, [Dims, i32, i32, ctypes.c_int, vp, vp, vp, vp, vp, vp, vp]),
        "moonep_combine": (ctypes.c_int, [Dims, i32, ctypes.c_int, vp, vp, vp, vp, vp]),
        "moonep_wgrad_workspace_bytes": (sz, [Dims]),
        "moonep_wgrad": (ctypes.c_int, [Dims, i32, i32, ctypes.c_int, vp, vp, vp, vp, vp, vp, vp]),
        "moonep_reduce_grad": (ctypes.c_int, [Dims, i32, i32, vp, vp, vp, vp]),
        "moonep_combine_backward": (ctypes.c_int, [Dims, i32, ctypes.c_int, vp, vp, vp, vp, vp, vp, vp]),
        "moonep_group_gemm_dgrad": (ctypes.c_int, [Dims, i32, i32, ctypes.c_int, vp, vp, vp, vp, vp, vp, vp]),
        "moonep_dispatch_backward": (ctypes.c_int, [Dims, i32, ctypes.c_int, vp, vp, vp, vp]),
        "moonep_swiglu": (ctypes.c_int, [Dims, i32, ctypes.c_int, vp, vp, vp]),
        "moonep_swiglu_backward": (ctypes.c_int, [Dims, i32, ctypes.c_int, vp, vp, vp, vp]),
        "moonep_save8_blocks": (i32, [i32]),
        "moonep_save8": (ctypes.c_int, [i64, i32, ctypes.c_int, vp, vp, vp, vp]),
        "moonep_load8": (ctypes.c_int, [i64, i32, ctypes.c_int, vp, vp, vp, vp]),
        "moonep_swiglu_save8": (ctypes.c_int, [Dims, i32, ctypes.c_int, vp, vp, vp, vp, vp]),
        "moonep_swiglu_backward8": (ctypes.c_int, [Dims, i32, ctypes.c_int] + [vp] * 9),
        "moonep_dispatch8": (ctypes.c_int, [Dims, i32, ctypes.c_int] + [vp] * 7),
        "moonep_combine_backward_ungated": (ctypes.c_int, [Dims, i32, ctypes.c_int, vp, vp, vp, vp]),
        "moonep_layernorm": (ctypes.c_int, [Dims, i32, ctypes.c_int, vp, vp, vp, ctypes.c_float] + [vp] * 6),
        "moonep_layernorm_dispatch": (ctypes.c_int, [Dims, i32, ctypes.c_int, vp, vp, vp, ctypes.c_float] + [vp] * 7),
        "moonep_layernorm_backward_workspace_bytes": (sz, [Dims, i32]),
        "moonep_layernorm_backward": (ctypes.c_int, [Dims, i32, ctypes.c_int] + [vp] * 10),
        "moonep_layernorm_backward8": (ctypes.c_int, [Dims, i32] + [vp] * 10),
        "moonep_route": (ctypes.c_int, [Dims, i32, i32, ctypes.c_float] + [vp] * 5),
        "moonep_route_backward": (ctypes.c_int, [Dims, i32, i32, ctypes.c_float] + [vp] * 5),
        "moonep_few_workspace_bytes": (sz, [Dims, i32, i32]),
        "moonep_few_layer": (ctypes.c_int, [Dims, i32, i32, ctypes.c_int] + [vp] * 7),
        "moonep_few_ffn": (ctypes.c_int, [Dims, i32, i32, ctypes.c_int] + [vp] * 8),
        "moonep_save4": (ctypes.c_int, [i32, i32, i32, i32, ctypes.c_int] + [vp] * 4),
        "moonep_load4": (ctypes.c_int, [i32, i32, i32, i32, ctypes.c_int] + [vp] * 4),
        "moonep_few_layer4": (ctypes.c_int, [Dims, i32, i32, i32, ctypes.c_int] + [vp] * 8),
        "moonep_few_ffn4": (ctypes.c_int, [Dims, i32, i32, i32, ctypes.c_int] + [vp] * 10),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


_LIB = _load()

# exported symbol names, as declared in include/moonep.h
SYMBOLS = ("moonep_last_error", "moonep_plan_workspace_bytes", "moonep_plan", "moonep_plan_ex",
           "moonep_plan_static_scratch_bytes", "moonep_plan_static", "moonep_dispatch", "moonep_prefetch",
           "moonep_group_gemm_workspace_bytes", "moonep_group_gemm", "moonep_combine",
           "moonep_wgrad_workspace_bytes", "moonep_wgrad", "moonep_reduce_grad", "moonep_combine_backward",
           "moonep_group_gemm_dgrad", "moonep_dispatch_backward", "moonep_swiglu", "moonep_swiglu_backward",
           "moonep_save8_blocks", "moonep_save8", "moonep_load8", "moonep_swiglu_save8", "moonep_swiglu_backward8",
           "moonep_dispatch8", "moonep_combine_backward_ungated", "moonep_layernorm", "moonep_layernorm_dispatch",
           "moonep_layernorm_backward_workspace_bytes", "moonep_layernorm_backward", "moonep_layernorm_backward8",
           "moonep_route", "moonep_route_backward", "moonep_few_workspace_bytes", "moonep_few_layer",
           "moonep_few_ffn", "moonep_save4", "moonep_load4", "moonep_few_layer4", "moonep_few_ffn4")


def lib():
    return _LIB


def last_error() -> str:
    return _LIB.moonep_last_error().decode()


def _check(rc: int):
    if rc != MOONEP_OK:
        raise MoonepError(rc, last_error())


# ------------------------------------------------------------------ marshalling helpers

def _ptr(t, name, dtype=None, numel=None, optional=False):
    import torch
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor (got {t.device})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} (got {t.dtype})")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must hold {numel} elements (got {t.numel()})")
    return t.data_ptr()


def _dtype_enum(t):
    import torch
    if t.dtype == torch.bfloat16:
        return MOONEP_BF16
    if t.dtype == torch.float32:
        return MOONEP_F32
    raise ValueError(f"unsupported dtype {t.dtype}")


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def make_dims(R, E, B, S, K) -> Dims:
    return Dims(int(R), int(E), int(B), int(S), int(K))


# ------------------------------------------------------------------ entry points

def moonep_plan_workspace_bytes(d: Dims) -> int:
    return int(_LIB.moonep_plan_workspace_bytes(d))


def moonep_group_gemm_workspace_bytes(d: Dims) -> int:
    return int(_LIB.moonep_group_gemm_workspace_bytes(d))


def moonep_wgrad_workspace_bytes(d: Dims) -> int:
    return int(_LIB.moonep_wgrad_workspace_bytes(d))


def moonep_plan(d: Dims, topk_idx, expert_counts, maxvio, cu_seqlens, slot_expert, dest_idx, src_of_row, stats,
                workspace, stream=None):
    moonep_plan_ex(d, MOONEP_PLAN_PREFIX, topk_idx, expert_counts, maxvio, cu_seqlens, slot_expert, dest_idx,
                   src_of_row, stats, workspace, stream)


def _planner_code(planner) -> int:
    if isinstance(planner, str):
        if planner not in PLANNERS:
            raise ValueError(f"unknown planner {planner!r}; one of {sorted(PLANNERS)}")
        return PLANNERS[planner]
    return int(planner)


def moonep_plan_ex(d: Dims, planner, topk_idx, expert_counts, maxvio, cu_seqlens, slot_expert, dest_idx, src_of_row,
                   stats, workspace, stream=None):
    """moonep_plan with a planner: "prefix" (MOONEP_PLAN_PREFIX) or "mincopy" (MOONEP_PLAN_MINCOPY)."""
    import torch
    i32 = torch.int32
    args = (
        _ptr(topk_idx, "topk_idx", i32, d.N),
        _ptr(expert_counts, "expert_counts", i32, d.E),
        _ptr(maxvio, "maxvio", torch.float64, 1),
        _ptr(cu_seqlens, "cu_seqlens", i32, d.R * (d.E + d.B + 1)),
        _ptr(slot_expert, "slot_expert", i32, d.R * d.B, optional=d.B == 0),
        _ptr(dest_idx, "dest_idx", i32, d.N),
        _ptr(src_of_row, "src_of_row", i32, d.N, optional=True),
        _ptr(stats, "stats", i32, 4),
        _ptr(workspace, "workspace"),
    )
    if workspace.numel() * workspace.element_size() < moonep_plan_workspace_bytes(d):
        raise ValueError("plan workspace too small")
    _check(_LIB.moonep_plan_ex(d, _planner_code(planner), *args, _stream(stream)))


def moonep_plan_static_scratch_bytes() -> int:
    return int(_LIB.moonep_plan_static_scratch_bytes())


def moonep_plan_static(d: Dims, planner, topk_idx, expert_counts, maxvio, cu_seqlens, slot_expert, dest_idx,
                       src_of_row, stats, stream=None):
    """moonep_plan_ex without a workspace: the library's own per-GPU scratch array serves instead (calls that
    overlap on one GPU race on it)."""
    import torch
    i32 = torch.int32
    _check(_LIB.moonep_plan_static(
        d, _planner_code(planner), _ptr(topk_idx, "topk_idx", i32, d.N),
        _ptr(expert_counts, "expert_counts", i32, d.E), _ptr(maxvio, "maxvio", torch.float64, 1),
        _ptr(cu_seqlens, "cu_seqlens", i32, d.R * (d.E + d.B + 1)),
        _ptr(slot_expert, "slot_expert", i32, d.R * d.B, optional=d.B == 0), _ptr(dest_idx, "dest_idx", i32, d.N),
        _ptr(src_of_row, "src_of_row", i32, d.N, optional=True), _ptr(stats, "stats", i32, 4), _stream(stream)))


def moonep_dispatch(d: Dims, H: int, X, dest_idx, Xp, stream=None):
    import torch
    t = _dtype_enum(X)
    _check(_LIB.moonep_dispatch(d, int(H), t, _ptr(X, "X", X.dtype, d.R * d.S * H),
                                _ptr(dest_idx, "dest_idx", torch.int32, d.N),
                                _ptr(Xp, "Xp", X.dtype, d.N * H), _stream(stream)))


def moonep_prefetch(d: Dims, H: int, Hp: int, W_home, slot_expert, W_slots, stream=None):
    import torch
    t = _dtype_enum(W_home)
    _check(_LIB.moonep_prefetch(d, int(H), int(Hp), t, _ptr(W_home, "W_home", W_home.dtype, d.E * H * Hp),
                                _ptr(slot_expert, "slot_expert", torch.int32, d.R * d.B, optional=d.B == 0),
                                _ptr(W_slots, "W_slots", W_home.dtype, d.R * d.B * H * Hp, optional=d.B == 0),
                                _stream(stream)))


def moonep_group_gemm(d: Dims, H: int, Hp: int, Xp, W_home, W_slots, cu_seqlens, Yp, workspace, stream=None):
    import torch
    t = _dtype_enum(Xp)
    if workspace.numel() * workspace.element_size() < moonep_group_gemm_workspace_bytes(d):
        raise ValueError("group GEMM workspace too small")
    _check(_LIB.moonep_group_gemm(d, int(H), int(Hp), t, _ptr(Xp, "Xp", Xp.dtype, d.N * H),
                                  _ptr(W_home, "W_home", Xp.dtype, d.E * H * Hp),
                                  _ptr(W_slots, "W_slots", Xp.dtype, d.R * d.B * H * Hp, optional=d.B == 0),
                                  _ptr(cu_seqlens, "cu_seqlens", torch.int32, d.R * (d.E + d.B + 1)),
                                  _ptr(Yp, "Yp", Xp.dtype, d.N * Hp), _ptr(workspace, "workspace"),
                                  _stream(stream)))


def moonep_combine(d: Dims, D: int, Yp, dest_idx, gates, out, stream=None):
    import torch
    t = _dtype_enum(Yp)
    _check(_LIB.moonep_combine(d, int(D), t, _ptr(Yp, "Yp", Yp.dtype, d.N * D),
                               _ptr(dest_idx, "dest_idx", torch.int32, d.N),
                               _ptr(gates, "gates", torch.float32, d.N),
                               _ptr(out, "out", torch.float32, d.R * d.S * D), _stream(stream)))


def moonep_wgrad(d: Dims, H: int, Hp: int, Xp, dY, cu_seqlens, dW_home, dW_slots, workspace, stream=None):
    import torch
    t = _dtype_enum(Xp)
    if workspace.numel() * workspace.element_size() < moonep_wgrad_workspace_bytes(d):
        raise ValueError("wgrad workspace too small")
    _check(_LIB.moonep_wgrad(d, int(H), int(Hp), t, _ptr(Xp, "Xp", Xp.dtype, d.N * H),
                             _ptr(dY, "dY", Xp.dtype, d.N * Hp),
                             _ptr(cu_seqlens, "cu_seqlens", torch.int32, d.R * (d.E + d.B + 1)),
                             _ptr(dW_home, "dW_home", torch.float32, d.E * H * Hp),
                             _ptr(dW_slots, "dW_slots", torch.float32, d.R * d.B * H * Hp, optional=d.B == 0),
                             _ptr(workspace, "workspace"), _stream(stream)))


def moonep_reduce_grad(d: Dims, H: int, Hp: int, slot_expert, dW_home, dW_slots, stream=None):
    import torch
    _check(_LIB.moonep_reduce_grad(d, int(H), int(Hp),
                                   _ptr(slot_expert, "slot_expert", torch.int32, d.R * d.B, optional=d.B == 0),
                                   _ptr(dW_home, "dW_home", torch.float32, d.E * H * Hp),
                                   _ptr(dW_slots, "dW_slots", torch.float32, d.R * d.B * H * Hp, optional=d.B == 0),
                                   _stream(stream)))


def moonep_combine_backward(d: Dims, D: int, dout, Yp, dest_idx, gates, dYp, dgates, stream=None):
    import torch
    t = _dtype_enum(Yp)
    _check(_LIB.moonep_combine_backward(d, int(D), t, _ptr(dout, "dout", torch.float32, d.R * d.S * D),
                                        _ptr(Yp, "Yp", Yp.dtype, d.N * D),
                                        _ptr(dest_idx, "dest_idx", torch.int32, d.N),
                                        _ptr(gates, "gates", torch.float32, d.N),
                                        _ptr(dYp, "dYp", Yp.dtype, d.N * D),
                                        _ptr(dgates, "dgates", torch.float32, d.N), _stream(stream)))


def moonep_group_gemm_dgrad(d: Dims, H: int, Hp: int, dYp, W_home, W_slots, cu_seqlens, dXp, workspace,
                            stream=None):
    import torch
    t = _dtype_enum(dYp)
    if workspace.numel() * workspace.element_size() < moonep_group_gemm_workspace_bytes(d):
        raise ValueError("group GEMM workspace too small")
    _check(_LIB.moonep_group_gemm_dgrad(d, int(H), int(Hp), t, _ptr(dYp, "dYp", dYp.dtype, d.N * Hp),
                                        _ptr(W_home, "W_home", dYp.dtype, d.E * H * Hp),
                                        _ptr(W_slots, "W_slots", dYp.dtype, d.R * d.B * H * Hp, optional=d.B == 0),
                                        _ptr(cu_seqlens, "cu_seqlens", torch.int32, d.R * (d.E + d.B + 1)),
                                        _ptr(dXp, "dXp", dYp.dtype, d.N * H), _ptr(workspace, "workspace"),
                                        _stream(stream)))


def moonep_dispatch_backward(d: Dims, H: int, dXp, dest_idx, dX, stream=None):
    import torch
    t = _dtype_enum(dXp)
    _check(_LIB.moonep_dispatch_backward(d, int(H), t, _ptr(dXp, "dXp", dXp.dtype, d.N * H),
                                         _ptr(dest_idx, "dest_idx", torch.int32, d.N),
                                         _ptr(dX, "dX", torch.float32, d.R * d.S * H), _stream(stream)))


def moonep_swiglu(d: Dims, Hp: int, Ygu, A, stream=None):
    t = _dtype_enum(Ygu)
    _check(_LIB.moonep_swiglu(d, int(Hp), t, _ptr(Ygu, "Ygu", Ygu.dtype, d.N * 2 * Hp),
                              _ptr(A, "A", Ygu.dtype, d.N * Hp), _stream(stream)))


def moonep_swiglu_backward(d: Dims, Hp: int, Ygu, dA, dYgu, stream=None):
    t = _dtype_enum(Ygu)
    _check(_LIB.moonep_swiglu_backward(d, int(Hp), t, _ptr(Ygu, "Ygu", Ygu.dtype, d.N * 2 * Hp),
                                       _ptr(dA, "dA", Ygu.dtype, d.N * Hp),
                                       _ptr(dYgu, "dYgu", Ygu.dtype, d.N * 2 * Hp), _stream(stream)))


# ------------------------------------------------------------------ layer norm and 8-bit checkpoints
import torch  # noqa: E402  (already loaded with the library)

_Tensor = torch.Tensor


def _launch(entry, *args, stream=None):
    """Calls `entry` with its arguments, tensors given as (tensor, name, dtype, elements) and passed as pointers, on the
    current stream of the device that they all lie on (or the stream passed), whatever device is current."""
    device, values = None, []
    for a in args:
        if a.__class__ is tuple:
            t, name, dtype, numel = a
            if device is None and t.__class__ is _Tensor and t.is_cuda:
                device = t.get_device()
            # what every tensor passes by, if nothing is wrong with it
            if not (t.__class__ is _Tensor and t.dtype is dtype and t.numel() == numel and t.is_contiguous()
                    and t.get_device() == device):
                _ptr(t, name, dtype, numel)
                at = t.get_device()
                if device is None:
                    device = at
                elif at != device:
                    raise ValueError(f"{name} is on cuda:{at}, the tensors before it on cuda:{device}")
            a = t.data_ptr()
        values.append(a)
    if stream is None:
        # the handle alone: torch.cuda.current_stream() costs 2-3 us, as much as a small kernel
        values.append(torch._C._cuda_getCurrentRawStream(device))
    elif stream.device.index != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{device}")
    else:
        values.append(stream.cuda_stream)
    if device == torch._C._cuda_getDevice():
        rc = entry(*values)
    else:
        with torch.cuda.device(device):
            rc = entry(*values)
    if rc != MOONEP_OK:
        _check(rc)


def _row_type(t, name):
    """The row type of the tensor that sets the call's, and the library's code for it."""
    if t is None:
        raise ValueError(f"{name} is required")
    return t.dtype, _dtype_enum(t)


def _or_none(t, *spec):
    """An optional tensor's argument: None where it is not given."""
    return None if t is None else (t, *spec)


def moonep_save8_blocks(C: int) -> int:
    """Exponent bytes of an 8-bit row of C columns."""
    return int(_LIB.moonep_save8_blocks(int(C)))


def _rows8(codes, exps, rows, C):
    """8-bit rows [rows, C] as arguments."""
    return (codes, "codes", torch.int8, rows * C), (exps, "exps", torch.uint8, rows * -(-C // 32))


def moonep_save8(rows: int, C: int, X, codes, exps, stream=None):
    """Keeps X [rows, C] in 8 bits: codes int8 [rows, C], exps uint8 [rows, moonep_save8_blocks(C)]."""
    t, code = _row_type(X, "X")
    _launch(_LIB.moonep_save8, int(rows), int(C), code, (X, "X", t, rows * C), *_rows8(codes, exps, rows, C),
            stream=stream)


def moonep_load8(rows: int, C: int, codes, exps, X, stream=None):
    """Writes the values of 8-bit rows to X [rows, C] (bfloat16 or float32, both exact)."""
    t, code = _row_type(X, "X")
    _launch(_LIB.moonep_load8, int(rows), int(C), code, *_rows8(codes, exps, rows, C), (X, "X", t, rows * C),
            stream=stream)


def moonep_swiglu_save8(d: Dims, Hp: int, Ygu, A, codes, exps, stream=None):
    """moonep_swiglu, and Ygu kept in 8 bits (its gate and up halves as rows of their own)."""
    N = d.N
    t, code = _row_type(Ygu, "Ygu")
    _launch(_LIB.moonep_swiglu_save8, d, int(Hp), code, (Ygu, "Ygu", t, N * 2 * Hp), (A, "A", t, N * Hp),
            *_rows8(codes, exps, 2 * N, Hp), stream=stream)


def moonep_swiglu_backward8(d: Dims, Hp: int, codes, exps, dA, src_of_row, gates, A, dYgu, dgates, stream=None):
    """Gradient of moonep_swiglu from its 8-bit input; with src_of_row, gates and dgates (all or none) the gates
    are applied here: A and dYgu come out times the gate, and dgates is <dA, silu(g) u> per pair."""
    N = d.N
    t, code = _row_type(dA, "dA")
    _launch(_LIB.moonep_swiglu_backward8, d, int(Hp), code, *_rows8(codes, exps, 2 * N, Hp), (dA, "dA", t, N * Hp),
            _or_none(src_of_row, "src_of_row", torch.int32, N), _or_none(gates, "gates", torch.float32, N),
            (A, "A", t, N * Hp), (dYgu, "dYgu", t, N * 2 * Hp), _or_none(dgates, "dgates", torch.float32, N),
            stream=stream)


def moonep_dispatch8(d: Dims, H: int, codes, exps, gamma, beta, dest_idx, Xp, stream=None):
    """moonep_dispatch from 8-bit token rows, times gamma plus beta (float32 [H], or None)."""
    t, code = _row_type(Xp, "Xp")
    _launch(_LIB.moonep_dispatch8, d, int(H), code, *_rows8(codes, exps, d.R * d.S, H),
            _or_none(gamma, "gamma", torch.float32, H), _or_none(beta, "beta", torch.float32, H),
            (dest_idx, "dest_idx", torch.int32, d.N), (Xp, "Xp", t, d.N * H), stream=stream)


def moonep_combine_backward_ungated(d: Dims, D: int, dout, dest_idx, dYp, stream=None):
    """The output gradient's rows laid out by expert, without gates."""
    t, code = _row_type(dYp, "dYp")
    _launch(_LIB.moonep_combine_backward_ungated, d, int(D), code, (dout, "dout", torch.float32, d.R * d.S * D),
            (dest_idx, "dest_idx", torch.int32, d.N), (dYp, "dYp", t, d.N * D), stream=stream)


def moonep_layernorm(d: Dims, H: int, X, gamma, beta, eps: float, Y, mean, rstd, codes=None, exps=None, stream=None):
    """Layer norm of X [R,S,H]; mean and rstd [R,S] may be None, and codes and exps keep the normalised rows in
    8 bits."""
    t, code = _row_type(X, "X")
    T, f32 = d.R * d.S, torch.float32
    c8, e8 = _rows8(codes, exps, T, H)
    _launch(_LIB.moonep_layernorm, d, int(H), code, (X, "X", t, T * H), (gamma, "gamma", f32, H),
            _or_none(beta, "beta", f32, H), float(eps), (Y, "Y", t, T * H), _or_none(mean, "mean", f32, T),
            _or_none(rstd, "rstd", f32, T), None if codes is None else c8, None if exps is None else e8, stream=stream)


def moonep_layernorm_dispatch(d: Dims, H: int, X, gamma, beta, eps: float, dest_idx, Xp, mean, rstd, codes=None,
                              exps=None, stream=None):
    """moonep_layernorm and moonep_dispatch of its rows in one pass; the normalised rows themselves are not stored."""
    t, code = _row_type(X, "X")
    T, f32 = d.R * d.S, torch.float32
    c8, e8 = _rows8(codes, exps, T, H)
    _launch(_LIB.moonep_layernorm_dispatch, d, int(H), code, (X, "X", t, T * H), (gamma, "gamma", f32, H),
            _or_none(beta, "beta", f32, H), float(eps), (dest_idx, "dest_idx", torch.int32, d.N),
            (Xp, "Xp", t, d.N * H), _or_none(mean, "mean", f32, T), _or_none(rstd, "rstd", f32, T),
            None if codes is None else c8, None if exps is None else e8, stream=stream)


def moonep_layernorm_backward_workspace_bytes(d: Dims, H: int) -> int:
    return int(_LIB.moonep_layernorm_backward_workspace_bytes(d, int(H)))


def _layernorm_backward(entry, d, H, code, dY, z, rstd, gamma, dX, dgamma, dbeta, workspace, stream):
    T, f32 = d.R * d.S, torch.float32
    if workspace is not None:
        at = workspace.get_device()
        if at < 0 or at == torch._C._cuda_getDevice():
            needed = moonep_layernorm_backward_workspace_bytes(d, H)
        else:  # the launch, whose size sets the workspace's, is for the tensors' device
            with torch.cuda.device(at):
                needed = moonep_layernorm_backward_workspace_bytes(d, H)
        if workspace.numel() * workspace.element_size() < needed:
            raise ValueError(f"workspace too small: {needed} bytes needed")
    _launch(entry, d, int(H), *code, (dY, "dY", f32, T * H), *z, (rstd, "rstd", f32, T), (gamma, "gamma", f32, H),
            (dX, "dX", f32, T * H), (dgamma, "dgamma", f32, H), _or_none(dbeta, "dbeta", f32, H),
            (workspace, "workspace", None, None), stream=stream)


def moonep_layernorm_backward(d: Dims, H: int, dY, X, mean, rstd, gamma, dX, dgamma, dbeta, workspace, stream=None):
    """Gradients of moonep_layernorm from its input: writes dX, adds into dgamma and dbeta (or None)."""
    t, code = _row_type(X, "X")
    T = d.R * d.S
    _layernorm_backward(_LIB.moonep_layernorm_backward, d, H, (code,), dY,
                        ((X, "X", t, T * H), (mean, "mean", torch.float32, T)), rstd, gamma, dX, dgamma, dbeta,
                        workspace, stream)


def moonep_layernorm_backward8(d: Dims, H: int, dY, codes, exps, rstd, gamma, dX, dgamma, dbeta, workspace,
                               stream=None):
    """moonep_layernorm_backward from the 8-bit normalised rows."""
    _layernorm_backward(_LIB.moonep_layernorm_backward8, d, H, (), dY, _rows8(codes, exps, d.R * d.S, H), rstd, gamma,
                        dX, dgamma, dbeta, workspace, stream)


# ------------------------------------------------------------------ router, layer for few tokens, 4-bit weights

def _score_code(score) -> int:
    if isinstance(score, str):
        if score not in SCORES:
            raise ValueError(f"unknown score {score!r}; one of {sorted(SCORES)}")
        return SCORES[score]
    return int(score)


def moonep_route(d: Dims, score, renorm: bool, scale: float, logits, bias, topk_idx, gates, stream=None):
    """The K experts of every token of logits [R,S,E], and their gates: score "softmax" or "sigmoid"; bias (float32 [E]
    or None) corrects the choice only."""
    f32 = torch.float32
    _launch(_LIB.moonep_route, d, _score_code(score), int(bool(renorm)), float(scale),
            (logits, "logits", f32, d.R * d.S * d.E), _or_none(bias, "bias", f32, d.E),
            (topk_idx, "topk_idx", torch.int32, d.N), (gates, "gates", f32, d.N), stream=stream)


def moonep_route_backward(d: Dims, score, renorm: bool, scale: float, logits, topk_idx, dgates, dlogits, stream=None):
    """Gradient of moonep_route's gates: writes dlogits [R,S,E] from dgates [R,S,K]."""
    f32 = torch.float32
    n = d.R * d.S * d.E
    _launch(_LIB.moonep_route_backward, d, _score_code(score), int(bool(renorm)), float(scale),
            (logits, "logits", f32, n), (topk_idx, "topk_idx", torch.int32, d.N), (dgates, "dgates", f32, d.N),
            (dlogits, "dlogits", f32, n), stream=stream)


def moonep_few_workspace_bytes(d: Dims, H: int, Hp: int) -> int:
    """Bytes of workspace of the calls for few tokens (0 for dims that they refuse)."""
    return int(_LIB.moonep_few_workspace_bytes(d, int(H), int(Hp)))


def _few(entry, d, H, Hp, G, row_type, X, topk_idx, gates, weights, out, wide, workspace, stream):
    t, code = row_type
    ws = (workspace, "workspace", None, None)
    if workspace is not None:
        n = workspace.numel()
        if n * workspace.element_size() < _LIB.moonep_few_workspace_bytes(d, H, Hp):
            raise ValueError(f"workspace too small: {moonep_few_workspace_bytes(d, H, Hp)} bytes needed")
        ws = (workspace, "workspace", workspace.dtype, n)
    T, f32 = d.R * d.S, torch.float32
    N = T * d.K
    _launch(entry, d, H, Hp, *G, code, (X, "X", t, T * H), (topk_idx, "topk_idx", torch.int32, N),
            None if gates is None else (gates, "gates", f32, N), *weights, (out, "out", f32, T * wide), ws,
            stream=stream)


def _weights4(codes, scales, E, H, N, G, name):
    """4-bit weights [E, H, N] as arguments (a refused G is left to the library)."""
    return ((codes, name + "codes", torch.int32, E * -(-H // 8) * N),
            (scales, name + "scales", torch.bfloat16, E * -(-H // max(1, G)) * N))


def moonep_few_layer(d: Dims, H: int, Hp: int, X, topk_idx, gates, W_home, out, workspace, stream=None):
    """One expert projection and the combine for few tokens, without a plan: out [R,S,Hp] float32."""
    t = _row_type(X, "X")
    _few(_LIB.moonep_few_layer, d, H, Hp, (), t, X, topk_idx, gates, ((W_home, "W_home", t[0], d.E * H * Hp),), out, Hp,
         workspace, stream)


def moonep_few_ffn(d: Dims, H: int, Hp: int, X, topk_idx, gates, W_gu, W_down, out, workspace, stream=None):
    """The whole gated expert layer for few tokens, without a plan: out [R,S,H] float32."""
    t = _row_type(X, "X")
    n = d.E * H * Hp
    _few(_LIB.moonep_few_ffn, d, H, Hp, (), t, X, topk_idx, gates,
         ((W_gu, "W_gu", t[0], 2 * n), (W_down, "W_down", t[0], n)), out, H, workspace, stream)


def moonep_few_layer4(d: Dims, H: int, Hp: int, G: int, X, topk_idx, gates, codes, scales, out, workspace, stream=None):
    """moonep_few_layer with 4-bit weights."""
    _few(_LIB.moonep_few_layer4, d, H, Hp, (G,), _row_type(X, "X"), X, topk_idx, gates,
         _weights4(codes, scales, d.E, H, Hp, G, ""), out, Hp, workspace, stream)


def moonep_few_ffn4(d: Dims, H: int, Hp: int, G: int, X, topk_idx, gates, gu_codes, gu_scales, down_codes, down_scales,
                    out, workspace, stream=None):
    """moonep_few_ffn with 4-bit weights."""
    _few(_LIB.moonep_few_ffn4, d, H, Hp, (G,), _row_type(X, "X"), X, topk_idx, gates,
         _weights4(gu_codes, gu_scales, d.E, H, 2 * Hp, G, "gu_") + _weights4(down_codes, down_scales, d.E, Hp, H, G,
                                                                               "down_"), out, H, workspace, stream)


def moonep_save4(E: int, H: int, N: int, G: int, W, codes, scales, stream=None):
    """Weights W [E,H,N] into 4 bits: codes int32 [E, ceil(H/8), N], scales bfloat16 [E, ceil(H/G), N]."""
    t, code = _row_type(W, "W")
    _launch(_LIB.moonep_save4, int(E), int(H), int(N), int(G), code, (W, "W", t, E * H * N),
            *_weights4(codes, scales, E, H, N, G, ""), stream=stream)


def moonep_load4(E: int, H: int, N: int, G: int, codes, scales, W, stream=None):
    """Writes the values of 4-bit weights to W [E,H,N] (float32 exactly, bfloat16 rounded)."""
    t, code = _row_type(W, "W")
    _launch(_LIB.moonep_load4, int(E), int(H), int(N), int(G), code, *_weights4(codes, scales, E, H, N, G, ""),
            (W, "W", t, E * H * N), stream=stream)
