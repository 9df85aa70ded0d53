"""Static buffers for one balanced MoE layer and the call sequence through libmoonep.

Every buffer is allocated once, with shapes fixed by (R, E, B, S, K, H, Hp):
nothing depends on the routing, so repeated passes allocate nothing and a
pass can be captured in a HIP graph.  The forward pass is
plan -> prefetch -> dispatch -> group GEMM -> combine (the prefetch needs only
the plan); the weight backward is
wgrad -> reduce_grad; with data_grad=True the data backward is
combine_backward (writes dY and dgates from dout) -> dgrad -> dispatch_backward
(dX).  Each step is one C-ABI call whose kernels do all the work; this class
only owns memory and passes pointers.  MoeFFN is the same for experts that are
gated FFNs, and MoeFew that layer for few tokens, without a plan.
"""
from __future__ import annotations

import torch

from . import _lib
from ._lib import Dims, make_dims


class MoeLayer:
    """One balanced MoE projection layer.

    `slot_pool` = (W_slots [R,B,H,Hp] of the layer dtype, dW_slots [R,B,H,Hp] float32 or None) makes the
    layer use a caller's slot buffers instead of its own: the pages keep one process-wide pool of B
    slots that every layer shares, so the extra memory is B experts in total, not B per layer.  Layers
    sharing a pool run one after another; a layer's backward that follows other layers' forward passes
    re-runs its prefetch first (the pool then holds the other layers' slots), and its reduce_grad leaves
    the slot gradients at zero for the next layer.
    """

    def __init__(self, R, E, B, S, K, H, Hp=None, dtype=torch.bfloat16, device="cuda", backward=False,
                 src_of_row=True, data_grad=False, planner="prefix", slot_pool=None):
        self.d: Dims = make_dims(R, E, B, S, K)
        self.planner = planner  # "prefix" (home-first) or "mincopy" (fewest copies)
        d = self.d
        self.H, self.Hp, self.dtype, self.device = H, Hp, dtype, device
        i32 = dict(dtype=torch.int32, device=device)
        N = d.N
        # routing (inputs)
        self.topk_idx = torch.zeros((R, S, K), **i32)
        self.gates = torch.zeros((R, S, K), dtype=torch.float32, device=device)
        # plan outputs
        self.expert_counts = torch.zeros(E, **i32)
        self.maxvio = torch.zeros(1, dtype=torch.float64, device=device)
        self.cu_seqlens = torch.zeros((R, E + B + 1), **i32)
        self.slot_expert = torch.full((R, max(B, 0)), -1, **i32)
        self.dest_idx = torch.zeros((R, S, K), **i32)
        self.src_of_row = torch.zeros(N, **i32) if src_of_row else None
        self.stats = torch.zeros(4, **i32)
        self.ws_plan = torch.empty(max(1, _lib.moonep_plan_workspace_bytes(d)), dtype=torch.uint8, device=device)
        # activations
        self.X = torch.zeros((R, S, H), dtype=dtype, device=device)
        self.Xp = torch.empty((N, H), dtype=dtype, device=device)
        pool_w, pool_dw = slot_pool if slot_pool is not None else (None, None)
        if Hp is not None:
            self.W_home = torch.zeros((E, H, Hp), dtype=dtype, device=device)
            if pool_w is not None:
                if tuple(pool_w.shape) != (R, B, H, Hp) or pool_w.dtype != dtype:
                    raise ValueError(f"slot pool must be [{R},{B},{H},{Hp}] {dtype}")
                self.W_slots = pool_w
            else:
                self.W_slots = torch.zeros((R, B, H, Hp), dtype=dtype, device=device)
            self.Yp = torch.empty((N, Hp), dtype=dtype, device=device)
            self.ws_gemm = torch.empty(max(1, _lib.moonep_group_gemm_workspace_bytes(d)), dtype=torch.uint8,
                                       device=device)
            self.out = torch.empty((R, S, Hp), dtype=torch.float32, device=device)
            if backward:
                self.dY = torch.zeros((N, Hp), dtype=dtype, device=device)
                self.dW_home = torch.zeros((E, H, Hp), dtype=torch.float32, device=device)
                if pool_dw is not None:
                    if tuple(pool_dw.shape) != (R, B, H, Hp) or pool_dw.dtype != torch.float32:
                        raise ValueError(f"slot gradient pool must be [{R},{B},{H},{Hp}] float32")
                    self.dW_slots = pool_dw
                else:
                    self.dW_slots = torch.zeros((R, B, H, Hp), dtype=torch.float32, device=device)
                self.ws_wgrad = torch.empty(max(1, _lib.moonep_wgrad_workspace_bytes(d)), dtype=torch.uint8,
                                            device=device)
                if data_grad:
                    self.dout = torch.zeros((R, S, Hp), dtype=torch.float32, device=device)
                    self.dgates = torch.zeros((R, S, K), dtype=torch.float32, device=device)
                    self.dXp = torch.empty((N, H), dtype=dtype, device=device)
                    self.dX = torch.empty((R, S, H), dtype=torch.float32, device=device)

    # ---------------------------------------------------------------- steps
    def plan(self, stream=None):
        _lib.moonep_plan_ex(self.d, self.planner, self.topk_idx, self.expert_counts, self.maxvio, self.cu_seqlens,
                            self.slot_expert if self.d.B > 0 else None, self.dest_idx, self.src_of_row, self.stats,
                            self.ws_plan, stream)

    def dispatch(self, stream=None):
        _lib.moonep_dispatch(self.d, self.H, self.X, self.dest_idx, self.Xp, stream)

    def prefetch(self, stream=None):
        _lib.moonep_prefetch(self.d, self.H, self.Hp, self.W_home, self.slot_expert if self.d.B > 0 else None,
                             self.W_slots if self.d.B > 0 else None, stream)

    def group_gemm(self, stream=None):
        _lib.moonep_group_gemm(self.d, self.H, self.Hp, self.Xp, self.W_home,
                               self.W_slots if self.d.B > 0 else None, self.cu_seqlens, self.Yp, self.ws_gemm, stream)

    def combine(self, stream=None):
        _lib.moonep_combine(self.d, self.Hp, self.Yp, self.dest_idx, self.gates, self.out, stream)

    def wgrad(self, stream=None):
        _lib.moonep_wgrad(self.d, self.H, self.Hp, self.Xp, self.dY, self.cu_seqlens, self.dW_home,
                          self.dW_slots if self.d.B > 0 else None, self.ws_wgrad, stream)

    def reduce_grad(self, stream=None):
        _lib.moonep_reduce_grad(self.d, self.H, self.Hp, self.slot_expert if self.d.B > 0 else None, self.dW_home,
                                self.dW_slots if self.d.B > 0 else None, stream)

    def combine_backward(self, stream=None):
        _lib.moonep_combine_backward(self.d, self.Hp, self.dout, self.Yp, self.dest_idx, self.gates, self.dY,
                                     self.dgates, stream)

    def dgrad(self, stream=None):
        _lib.moonep_group_gemm_dgrad(self.d, self.H, self.Hp, self.dY, self.W_home,
                                     self.W_slots if self.d.B > 0 else None, self.cu_seqlens, self.dXp, self.ws_gemm,
                                     stream)

    def dispatch_backward(self, stream=None):
        _lib.moonep_dispatch_backward(self.d, self.H, self.dXp, self.dest_idx, self.dX, stream)

    def backward_data(self, stream=None):
        self.combine_backward(stream)
        self.dgrad(stream)
        self.dispatch_backward(stream)

    def forward(self, stream=None):
        self.plan(stream)
        if self.Hp is None:
            self.dispatch(stream)
            return
        # the weight prefetch needs only the plan, so it runs while (here: before) tokens dispatch
        self.prefetch(stream)
        self.dispatch(stream)
        self.group_gemm(stream)
        self.combine(stream)

    def backward(self, stream=None):
        self.wgrad(stream)
        self.reduce_grad(stream)


class MoeFFN:
    """Static buffers for one balanced MoE layer whose experts are gated FFNs, and the call sequence.

    Forward: plan -> dispatch -> prefetch (both projections) -> group GEMM with the gate|up weights
    [E+B, H, 2H'] -> swiglu -> group GEMM with the down weights [E+B, H', H] -> combine to [R, S, H].
    Backward (backward=True): combine backward -> dgrad and wgrad of the down projection -> swiglu
    backward -> dgrad and wgrad of the gate|up projection -> dispatch backward -> reduce_grad of both
    projections.  Every buffer has a shape fixed by (R, E, B, S, K, H, H'); nothing depends on the
    routing, so passes allocate nothing.

    `norm=True` puts a layer norm (gamma, beta [H] float32, eps) in front: X is then its input, dispatch lays
    out its rows in the same pass, and backward() continues through it from their gradient dXn to dX, adding into
    dgamma and dbeta.  The norm's backward reads X again unless save8=True, so X must keep its values until then
    (without a norm a program may overwrite X once forward() is over).

    `save8=True` (with backward=True) keeps only 8 bits of two activations from forward() to backward(): the
    rows that the experts read (normalised rows with norm=True, else X) in x_codes, x_exps [R, S, ...] and the
    activation's input Ygu in ygu_codes, ygu_exps.  The row buffers of the forward pass are then free once it
    is over: they are in the dict `scratch`, which layers of one shape can share by passing one's to the
    others' constructor (layers sharing it run one after another, as on one stream); with norm=True dXn, which is
    used inside backward() only, is there as well.  A layer without a backward has such a dict too; with
    backward=True and save8=False `scratch` is None.  backward() applies the gates on the experts' side: ungated
    output-gradient rows -> dgrad of the down projection -> swiglu backward from 8 bits (which also gives the gated
    activation and dgates) -> wgrad of the down projection -> dispatch from 8 bits -> dgrad and wgrad of the
    gate|up projection -> dispatch backward -> reduce_grad.

    `router="softmax"` or `"sigmoid"` puts the router's choice in front: forward() makes topk_idx and gates from the
    scores `logits` [R, S, E] (float32, which the caller's router projection writes) and, with router_bias=True, from
    `bias` [E], which corrects the choice only; `renorm` and `route_scale` are moonep_route's renorm and scale.
    backward() ends with `dlogits` from dgates.
    """

    def __init__(self, R, E, B, S, K, H, Hp, dtype=torch.bfloat16, device="cuda", backward=False, norm=False,
                 eps=1e-5, save8=False, scratch=None, router=None, renorm=True, route_scale=1.0, router_bias=False):
        if save8 and not backward:
            raise ValueError("save8 keeps activations for the backward pass: it needs backward=True")
        if scratch is not None and backward and not save8:
            raise ValueError("the backward pass reads the row buffers unless save8=True: they cannot be shared")
        self.d: Dims = make_dims(R, E, B, S, K)
        d = self.d
        self.H, self.Hp, self.dtype, self.device = H, Hp, dtype, device
        self.norm, self.eps, self.save8 = norm, eps, save8
        i32 = dict(dtype=torch.int32, device=device)
        act = dict(dtype=dtype, device=device)
        f32 = dict(dtype=torch.float32, device=device)
        N = d.N
        self.topk_idx = torch.zeros((R, S, K), **i32)
        self.gates = torch.zeros((R, S, K), **f32)
        _router_buffers(self, router, renorm, route_scale, router_bias, f32)
        if router is not None and backward:
            self.dlogits = torch.empty((R, S, E), **f32)
        self.expert_counts = torch.zeros(E, **i32)
        self.maxvio = torch.zeros(1, dtype=torch.float64, device=device)
        self.cu_seqlens = torch.zeros((R, E + B + 1), **i32)
        self.slot_expert = torch.full((R, max(B, 0)), -1, **i32)
        self.dest_idx = torch.zeros((R, S, K), **i32)
        self.src_of_row = torch.zeros(N, **i32) if save8 else None
        self.stats = torch.zeros(4, **i32)
        self.ws_plan = torch.empty(max(1, _lib.moonep_plan_workspace_bytes(d)), dtype=torch.uint8, device=device)
        self.ws_gemm = torch.empty(max(1, _lib.moonep_group_gemm_workspace_bytes(d)), dtype=torch.uint8,
                                   device=device)
        self.X = torch.zeros((R, S, H), **act)
        if norm:
            self.gamma = torch.ones(H, **f32)
            self.beta = torch.zeros(H, **f32)
            self.mean = torch.empty((R, S), **f32)
            self.rstd = torch.empty((R, S), **f32)
        rows = {"Xp": (N, H), "Ygu": (N, 2 * Hp), "A": (N, Hp), "Zp": (N, H)}
        if save8:  # the backward's rows of these shapes take the places of Zp and Ygu
            rows.update(dA=(N, Hp), dXp=(N, H))
        if scratch is None:
            scratch = {name: torch.empty(shape, **act) for name, shape in rows.items()}
        for name, shape in rows.items():
            t = scratch.get(name)
            if (t is None or tuple(t.shape) != shape or t.dtype != dtype or not t.is_contiguous()
                    or t.device != self.X.device):
                raise ValueError(f"scratch must hold {name} {list(shape)} {dtype} on {self.X.device}")
        # the backward of a layer that keeps everything reads these rows: no other layer may write them
        self.scratch = scratch if save8 or not backward else None
        self.Xp, self.Ygu, self.A, self.Zp = (scratch[name] for name in ("Xp", "Ygu", "A", "Zp"))
        self.W_gu_home = torch.zeros((E, H, 2 * Hp), **act)
        self.W_gu_slots = torch.zeros((R, B, H, 2 * Hp), **act)
        self.W_down_home = torch.zeros((E, Hp, H), **act)
        self.W_down_slots = torch.zeros((R, B, Hp, H), **act)
        self.out = torch.empty((R, S, H), **f32)
        if save8:
            codes = lambda *shape: (torch.empty(shape, dtype=torch.int8, device=device),  # noqa: E731
                                    torch.empty(shape[:-1] + (_lib.moonep_save8_blocks(shape[-1]),),
                                                dtype=torch.uint8, device=device))
            self.x_codes, self.x_exps = codes(R, S, H)
            self.ygu_codes, self.ygu_exps = codes(N, 2, Hp)
        if backward:
            self.ws_wgrad = torch.empty(max(1, _lib.moonep_wgrad_workspace_bytes(d)), dtype=torch.uint8,
                                        device=device)
            self.dout = torch.zeros((R, S, H), **f32)
            self.dgates = torch.zeros((R, S, K), **f32)
            if save8:
                self.dZp, self.dYgu, self.dA, self.dXp = self.Zp, self.Ygu, scratch["dA"], scratch["dXp"]
            else:
                self.dZp = torch.empty((N, H), **act)
                self.dA = torch.empty((N, Hp), **act)
                self.dYgu = torch.empty((N, 2 * Hp), **act)
                self.dXp = torch.empty((N, H), **act)
            self.dX = torch.empty((R, S, H), **f32)
            if norm:
                # inside one backward pass only, so save8's layers of the same tokens share it with their rows
                kind = lambda t: (t.shape, t.dtype, t.device, t.is_contiguous())  # noqa: E731
                self.dXn = scratch.get("dXn") if save8 else None
                if self.dXn is None or kind(self.dXn) != kind(self.dX):
                    self.dXn = torch.empty((R, S, H), **f32)
                    if save8:
                        scratch.setdefault("dXn", self.dXn)
                self.dgamma = torch.zeros(H, **f32)
                self.dbeta = torch.zeros(H, **f32)
                with torch.cuda.device(self.X.get_device()):  # its size is for the current device
                    nbytes = _lib.moonep_layernorm_backward_workspace_bytes(d, H)
                self.ws_norm = torch.empty(max(1, nbytes), dtype=torch.uint8, device=device)
            self.dW_gu_home = torch.zeros((E, H, 2 * Hp), **f32)
            self.dW_gu_slots = torch.zeros((R, B, H, 2 * Hp), **f32)
            self.dW_down_home = torch.zeros((E, Hp, H), **f32)
            self.dW_down_slots = torch.zeros((R, B, Hp, H), **f32)

    def _slots(self, t):
        return t if self.d.B > 0 else None

    def forward_calls(self):
        d, H, Hp, L = self.d, self.H, self.Hp, _lib
        sl = self._slots
        calls = _route_calls(self) + [
            ("plan", lambda: L.moonep_plan(d, self.topk_idx, self.expert_counts, self.maxvio, self.cu_seqlens,
                                           sl(self.slot_expert), self.dest_idx, self.src_of_row, self.stats,
                                           self.ws_plan)),
            ("prefetch", lambda: (L.moonep_prefetch(d, H, 2 * Hp, self.W_gu_home, sl(self.slot_expert),
                                                    sl(self.W_gu_slots)),
                                  L.moonep_prefetch(d, Hp, H, self.W_down_home, sl(self.slot_expert),
                                                    sl(self.W_down_slots)))),
        ]
        if self.norm:
            dispatch = ("layernorm_dispatch", lambda: L.moonep_layernorm_dispatch(
                d, H, self.X, self.gamma, self.beta, self.eps, self.dest_idx, self.Xp, self.mean, self.rstd,
                self.x_codes if self.save8 else None, self.x_exps if self.save8 else None))
        else:
            dispatch = ("dispatch", lambda: L.moonep_dispatch(d, H, self.X, self.dest_idx, self.Xp))
            if self.save8:
                calls.append(("save8", lambda: L.moonep_save8(d.R * d.S, H, self.X, self.x_codes, self.x_exps)))
        calls += [
            dispatch,
            ("gemm_gate_up", lambda: L.moonep_group_gemm(d, H, 2 * Hp, self.Xp, self.W_gu_home, sl(self.W_gu_slots),
                                                         self.cu_seqlens, self.Ygu, self.ws_gemm)),
            ("swiglu_save8", lambda: L.moonep_swiglu_save8(d, Hp, self.Ygu, self.A, self.ygu_codes, self.ygu_exps))
            if self.save8 else ("swiglu", lambda: L.moonep_swiglu(d, Hp, self.Ygu, self.A)),
            ("gemm_down", lambda: L.moonep_group_gemm(d, Hp, H, self.A, self.W_down_home, sl(self.W_down_slots),
                                                      self.cu_seqlens, self.Zp, self.ws_gemm)),
            ("combine", lambda: L.moonep_combine(d, H, self.Zp, self.dest_idx, self.gates, self.out)),
        ]
        return calls

    def backward_calls(self):
        d, H, Hp, L = self.d, self.H, self.Hp, _lib
        sl = self._slots
        dgrad_down = ("dgrad_down", lambda: L.moonep_group_gemm_dgrad(d, Hp, H, self.dZp, self.W_down_home,
                                                                      sl(self.W_down_slots), self.cu_seqlens,
                                                                      self.dA, self.ws_gemm))
        wgrad_down = ("wgrad_down", lambda: L.moonep_wgrad(d, Hp, H, self.A, self.dZp, self.cu_seqlens,
                                                           self.dW_down_home, sl(self.dW_down_slots),
                                                           self.ws_wgrad))
        if self.save8:
            affine = (self.gamma, self.beta) if self.norm else (None, None)
            calls = [
                ("combine_backward", lambda: L.moonep_combine_backward_ungated(d, H, self.dout, self.dest_idx,
                                                                               self.dZp)),
                dgrad_down,
                # a pair whose id is outside [0, E) has no row, from which the call would write its gradient: it is 0
                ("swiglu_backward8", lambda: (self.dgates.zero_(),
                                              L.moonep_swiglu_backward8(d, Hp, self.ygu_codes, self.ygu_exps, self.dA,
                                                                        self.src_of_row, self.gates, self.A,
                                                                        self.dYgu, self.dgates))),
                wgrad_down,
                ("dispatch8", lambda: L.moonep_dispatch8(d, H, self.x_codes, self.x_exps, *affine, self.dest_idx,
                                                         self.Xp)),
            ]
        else:
            calls = [
                ("combine_backward", lambda: L.moonep_combine_backward(d, H, self.dout, self.Zp, self.dest_idx,
                                                                       self.gates, self.dZp, self.dgates)),
                dgrad_down,
                wgrad_down,
                ("swiglu_backward", lambda: L.moonep_swiglu_backward(d, Hp, self.Ygu, self.dA, self.dYgu)),
            ]
        calls += [
            ("dgrad_gate_up", lambda: L.moonep_group_gemm_dgrad(d, H, 2 * Hp, self.dYgu, self.W_gu_home,
                                                                sl(self.W_gu_slots), self.cu_seqlens, self.dXp,
                                                                self.ws_gemm)),
            ("wgrad_gate_up", lambda: L.moonep_wgrad(d, H, 2 * Hp, self.Xp, self.dYgu, self.cu_seqlens,
                                                     self.dW_gu_home, sl(self.dW_gu_slots), self.ws_wgrad)),
            ("dispatch_backward", lambda: L.moonep_dispatch_backward(d, H, self.dXp, self.dest_idx,
                                                                     self.dXn if self.norm else self.dX)),
            ("reduce_grad", lambda: (L.moonep_reduce_grad(d, H, 2 * Hp, sl(self.slot_expert), self.dW_gu_home,
                                                          sl(self.dW_gu_slots)),
                                     L.moonep_reduce_grad(d, Hp, H, sl(self.slot_expert), self.dW_down_home,
                                                          sl(self.dW_down_slots)))),
        ]
        if self.norm and self.save8:
            calls.append(("layernorm_backward", lambda: L.moonep_layernorm_backward8(
                d, H, self.dXn, self.x_codes, self.x_exps, self.rstd, self.gamma, self.dX, self.dgamma, self.dbeta,
                self.ws_norm)))
        elif self.norm:
            calls.append(("layernorm_backward", lambda: L.moonep_layernorm_backward(
                d, H, self.dXn, self.X, self.mean, self.rstd, self.gamma, self.dX, self.dgamma, self.dbeta,
                self.ws_norm)))
        if self.router is not None:
            calls.append(("route_backward", lambda: L.moonep_route_backward(
                d, self.router, self.renorm, self.route_scale, self.logits, self.topk_idx, self.dgates, self.dlogits)))
        return calls

    def forward(self):
        self._run(self.forward_calls())

    def backward(self):
        self._run(self.backward_calls())

    def _run(self, calls):
        # some calls are enqueued on the current device's stream, some on their tensors': one stream if that is current
        with torch.cuda.device(self.X.get_device()):
            for _, f in calls:
                f()


def _router_buffers(layer, router, renorm, route_scale, router_bias, f32):
    """The router's options and buffers of a layer, whose topk_idx and gates forward() then writes."""
    d = layer.d
    if router is not None and router not in _lib.SCORES:
        raise ValueError(f"unknown router score {router!r}; one of {sorted(_lib.SCORES)}")
    if router_bias and router is None:
        raise ValueError("router_bias corrects the choice of a router")
    layer.router, layer.renorm, layer.route_scale = router, renorm, route_scale
    layer.logits = torch.zeros((d.R, d.S, d.E), **f32) if router is not None else None
    layer.bias = torch.zeros(d.E, **f32) if router_bias else None


def _route_calls(layer):
    if layer.router is None:
        return []
    return [("route", lambda: _lib.moonep_route(layer.d, layer.router, layer.renorm, layer.route_scale, layer.logits,
                                                layer.bias, layer.topk_idx, layer.gates))]


class MoeFew:
    """Static buffers for one gated expert layer that serves few tokens (R*S*K <= MOONEP_FEW_PAIRS), and its calls.

    forward() writes out [R, S, H] (float32) from X [R, S, H], topk_idx and gates, without a plan: the chosen experts'
    weights are read where they lie, once for up to ten pairs of an expert (moonep_few_ffn has the numbers).  `router`,
    `renorm`, `route_scale`, `router_bias`: as in MoeFFN, topk_idx and gates are then made from `logits`.  `norm=True` puts the layer norm of MoeFFN in front (gamma, beta, eps; its rows, rounded to
    dtype, are in Xn).

    The weights are the home weights of MoeFFN, W_gu [E, H, 2H'] and W_down [E, H', H] of `dtype`, or with bits=4 their
    4-bit form with groups of G input rows: gu_codes, gu_scales, down_codes, down_scales, which save_weights() writes.
    `weights` = those tensors in that order makes the layer use a caller's, such as a MoeFFN's W_gu_home and
    W_down_home or another MoeFew's.
    """

    def __init__(self, R, E, S, K, H, Hp, dtype=torch.bfloat16, device="cuda", norm=False, eps=1e-5, bits=16, G=32,
                 weights=None, router=None, renorm=True, route_scale=1.0, router_bias=False):
        if bits not in (4, 16):
            raise ValueError(f"bits must be 16 (weights of dtype) or 4 (got {bits})")
        if bits == 4 and G not in (32, 64, 128):
            raise ValueError(f"G must be 32, 64 or 128 (got {G})")
        self.d: Dims = make_dims(R, E, 0, S, K)
        d = self.d
        if d.N > _lib.MOONEP_FEW_PAIRS:
            raise ValueError(f"R*S*K ({d.N}) exceeds {_lib.MOONEP_FEW_PAIRS}: MoeFFN is for as many tokens")
        self.H, self.Hp, self.dtype, self.device = H, Hp, dtype, device
        self.norm, self.eps, self.bits, self.G = norm, eps, bits, G
        f32 = dict(dtype=torch.float32, device=device)
        self.topk_idx = torch.zeros((R, S, K), dtype=torch.int32, device=device)
        self.gates = torch.zeros((R, S, K), **f32)
        _router_buffers(self, router, renorm, route_scale, router_bias, f32)
        self.X = torch.zeros((R, S, H), dtype=dtype, device=device)
        if norm:
            self.gamma = torch.ones(H, **f32)
            self.beta = torch.zeros(H, **f32)
            self.Xn = torch.empty((R, S, H), dtype=dtype, device=device)
        self.out = torch.empty((R, S, H), **f32)
        self.workspace = torch.empty(max(1, _lib.moonep_few_workspace_bytes(d, H, Hp)), dtype=torch.uint8, device=device)
        if bits == 4:
            i32, bf16 = dict(dtype=torch.int32, device=device), dict(dtype=torch.bfloat16, device=device)
            form = []
            for rows, cols in ((H, 2 * Hp), (Hp, H)):
                form += [((E, -(-rows // 8), cols), i32), ((E, -(-rows // G), cols), bf16)]
            names = ("gu_codes", "gu_scales", "down_codes", "down_scales")
        else:
            form = [(shape, dict(dtype=dtype, device=device)) for shape in ((E, H, 2 * Hp), (E, Hp, H))]
            names = ("W_gu", "W_down")
        if weights is None:
            weights = [torch.zeros(shape, **kind) for shape, kind in form]
        if len(weights) != len(form):
            raise ValueError(f"weights must be {', '.join(names)}")
        for name, t, (shape, kind) in zip(names, weights, form):
            if tuple(t.shape) != shape or t.dtype != kind["dtype"] or not t.is_contiguous() or t.device != self.X.device:
                raise ValueError(f"{name} must be {list(shape)} {kind['dtype']}, contiguous, on {self.X.device}")
            setattr(self, name, t)

    def save_weights(self, W_gu, W_down):
        """Writes weights [E, H, 2H'] and [E, H', H] (bfloat16 or float32) as the layer keeps them."""
        E, H, Hp = self.d.E, self.H, self.Hp
        for name, t, shape in (("W_gu", W_gu, (E, H, 2 * Hp)), ("W_down", W_down, (E, Hp, H))):
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} must be {list(shape)} (got {list(t.shape)})")
        if self.bits == 4:
            _lib.moonep_save4(E, H, 2 * Hp, self.G, W_gu, self.gu_codes, self.gu_scales)
            _lib.moonep_save4(E, Hp, H, self.G, W_down, self.down_codes, self.down_scales)
        else:
            self.W_gu.copy_(W_gu)
            self.W_down.copy_(W_down)

    def forward_calls(self):
        d, H, Hp, L = self.d, self.H, self.Hp, _lib
        calls = _route_calls(self)
        if self.norm:
            calls.append(("layernorm", lambda: L.moonep_layernorm(d, H, self.X, self.gamma, self.beta, self.eps, self.Xn,
                                                                  None, None)))
        rows = (self.Xn if self.norm else self.X, self.topk_idx, self.gates)
        if self.bits == 4:
            calls.append(("few_ffn4", lambda: L.moonep_few_ffn4(d, H, Hp, self.G, *rows, self.gu_codes, self.gu_scales,
                                                                self.down_codes, self.down_scales, self.out,
                                                                self.workspace)))
        else:
            calls.append(("few_ffn", lambda: L.moonep_few_ffn(d, H, Hp, *rows, self.W_gu, self.W_down, self.out,
                                                              self.workspace)))
        return calls

    def forward(self):
        for _, f in self.forward_calls():
            f()
