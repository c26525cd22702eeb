"""A DeepSeekMoE layer on one GPU: device buffers plus the C-ABI calls of a forward
(five of them), and of a training step.

torch is used for device memory and the stream only; each step of the layer
runs in the HIP kernels behind include/moe.h.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import numpy as np
import torch

from . import _lib

_TORCH_STORAGE = {"f32": torch.float32, "bf16": torch.int16, "e4m3": torch.uint8}


def _dev(a, device):
    """Host numpy array -> device tensor with the same bytes."""
    t = torch.from_numpy(a)
    if t.dtype == torch.uint16:
        t = t.view(torch.int16)
    return t.to(device, non_blocking=False)


class Checkpoint(NamedTuple):
    """What MoeLayer.checkpoint() kept of a forward."""
    x: tuple  # (values or codes, scales or None, format)
    y_perm: tuple
    routing: torch.Tensor  # as MoeLayer.routing
    forward: Optional[int]  # whose buffers of the layer they are; None: they are the checkpoint's own


class MoeLayer:
    """Weights and scratch of one layer; ``forward`` runs route -> dispatch ->
    expert FFN -> combine, ``update_bias`` the sign step, ``step`` both.

    router: how the experts are chosen, where not by moe_route's rule: the keywords of
    ``selection`` (score, n_group, topk_group, group_score, renorm, scale).  The forward
    then computes the logits (kept in ``logits``) and chooses from them.

    A training step is ``forward``, ``checkpoint`` (what the backward needs of it, in 8
    bits or as it is) and ``backward``; with a router also ``balance_loss``; then
    ``adamw_step``.  ``checkpoint`` and ``balance_loss`` go by the last forward,
    ``backward`` by the forward whose checkpoint it is given.

    ``pack_experts`` keeps the routed experts in four bits beside their bf16 weights; the
    forward then runs on those (the backward on the bf16 ones they were packed from)."""

    def __init__(self, T, d, I, act, wt, wr, experts: dict, shared: dict, E=256, k=8, device="cuda", router=None):
        self.T, self.d, self.I, self.E, self.k = T, d, I, E, k
        self.act, self.wt = act, wt
        self.device = torch.device(device)
        self.desc = _lib.desc(T, d, E, k, I, act, wt)
        self.packed = None  # the routed experts in four bits (x's format, gate, up, down): pack_experts()
        self._packed_room = {}  # by x's format: codes and scales of x, workspace
        self.forwards = 0  # run so far: a checkpoint that reads the layer's own buffers knows whose they are
        self.sel = _lib.selection(T, E, k, **router) if router is not None else None
        self.wr = _dev(wr, self.device)
        self.ex = {n: (_dev(a, self.device) if a is not None else None) for n, a in experts.items()}
        self.sh = {n: (_dev(a, self.device) if a is not None else None) for n, a in shared.items()}
        self.ex_w = _lib.ffn_weights(*(self.ex[n] for n in ("gate", "up", "down", "s_gate", "s_up", "s_down")))
        self.sh_w = _lib.ffn_weights(*(self.sh[n] for n in ("gate", "up", "down", "s_gate", "s_up", "s_down")))
        self._alloc()

    def _alloc(self):
        dev, T, d, E, k = self.device, self.T, self.d, self.E, self.k
        A = T * k
        i32 = dict(dtype=torch.int32, device=dev)
        # one buffer, so that a checkpoint's copy is one
        self.routing = torch.empty(4 * A + (T * E if self.sel is not None else 0) + E + 1, **i32)
        self.idx, self.w, self.offsets, self.row_src, self.row_of, self.logits = self._parts(self.routing)
        self.gap = torch.empty(T, dtype=torch.float32, device=dev)
        self.counts = torch.empty(E, **i32)
        self.x_perm = self.x_perm_scale = None  # allocated on first use of the materialised dispatch
        self.y_perm = torch.empty((A, d), dtype=torch.float32 if self.wt == "f32" else torch.int16, device=dev)
        self.y = torch.empty((T, d), dtype=torch.float32, device=dev)
        ws = max(_lib.workspace_bytes(self.desc, s) for s in (0, 1, 2, 3, _lib.MOE_WS_ROUTER_LOGITS))
        self.ws = torch.empty(max(ws, 256), dtype=torch.uint8, device=dev)

    def _parts(self, routing):
        """idx, w, offsets, row_src, row_of and logits (None without a router) of a routing buffer."""
        T, E, k = self.T, self.E, self.k
        idx, w, row_src, row_of, logits, offsets = routing.split([T * k] * 4 + [routing.numel() - 4 * T * k - E - 1, E + 1])
        return (idx.view(T, k), w.view(torch.float32).view(T, k), offsets, row_src, row_of,
                logits.view(torch.float32).view(T, E) if self.sel is not None else None)

    def ensure_x_perm(self):
        if self.x_perm is None:
            A, d = self.T * self.k, self.d
            self.x_perm = torch.empty((A, d), dtype=_TORCH_STORAGE[self.wt], device=self.device)
            self.x_perm_scale = (torch.empty((A, d // 128), dtype=torch.uint8, device=self.device)
                                 if self.wt == "e4m3" else None)

    def forward(self, x, bias, gap=False, stream=None, gather_in_gemm=True):
        """One pass of the layer.  gather_in_gemm: the gate/up GEMM reads the
        token rows through row_src (no x_perm); otherwise moe_dispatch
        materialises x_perm and moe_expert_ffn consumes it.  Both give the
        same y bit for bit.  (Experts in four bits always gather.)"""
        D = self.desc
        self.forwards += 1
        if self.sel is None:
            _lib.moe_route(D, x, self.wr, bias, self.idx, self.w, self.gap if gap else None, self.ws, stream)
        else:
            if gap:
                raise ValueError("the gap is moe_route's: a layer with a router has none")
            _lib.moe_router_logits(D, x, self.wr, self.logits, self.ws, stream)
            _lib.moe_select(self.sel, self.logits, bias, self.idx, self.w, stream)
        if gather_in_gemm or self.packed is not None:
            _lib.moe_dispatch(D, self.idx, x, self.counts, self.offsets, self.row_src, self.row_of, None, None,
                              self.ws, stream)
        if self.packed is not None:
            fmt, mats = self.packed
            codes, scales, ws = self._packed_room[fmt]
            _lib.moe_mx_pack(x, codes, scales, fmt, stream)
            _lib.moe_mx_expert_ffn(_lib.mx(codes, scales, fmt), *mats, self.offsets, self.y_perm, ws, self.row_src, self.k,
                                   stream)
        elif gather_in_gemm:
            _lib.moe_expert_gate_up_rows(D, x, self.row_src, self.offsets, self.ex_w, self.ws, stream)
            _lib.moe_expert_down(D, self.offsets, self.ex_w, self.y_perm, self.ws, stream)
        else:
            self.ensure_x_perm()
            _lib.moe_dispatch(D, self.idx, x, self.counts, self.offsets, self.row_src, self.row_of, self.x_perm,
                              self.x_perm_scale, self.ws, stream)
            _lib.moe_expert_ffn(D, self.x_perm, self.x_perm_scale, self.offsets, self.ex_w, self.y_perm, self.ws,
                                stream)
        _lib.moe_combine(D, x, self.sh_w, self.y_perm, self.row_of, self.w, self.y, self.ws, stream)
        return self.y

    def checkpoint(self, x, fmt="e4m3", stream=None) -> Checkpoint:
        """What the backward needs of the last forward: x and the routed outputs in 8 bits ("e4m3" or "i8", half the
        memory of "bf16") and the routing, its own copies: any number of forwards may come before the backward.  "bf16"
        keeps x and the layer's buffers themselves, which the next forward overwrites: backward() refuses it then."""
        if fmt == "bf16":
            return Checkpoint((x, None, fmt), (self.y_perm, None, fmt), self.routing, self.forwards)
        kept = []
        with torch.cuda.stream(stream):
            for t in (x, self.y_perm):
                codes = torch.empty(t.shape, dtype=torch.uint8, device=t.device)
                scales = torch.empty((t.shape[0], (t.shape[1] + 127) // 128), dtype=torch.uint8, device=t.device)
                _lib.moe_checkpoint_pack(t, codes, scales, fmt)
                kept.append((codes, scales, fmt))
            return Checkpoint(*kept, self.routing.clone(), None)

    def balance_loss(self, seq_offsets, alpha, stream=None):
        """The last forward's sequence-wise balance loss [n_seq] and the loads [n_seq, E] that its gradient needs."""
        if self.sel is None:
            raise ValueError("the balance loss needs a layer with a router: the logits are not kept without one")
        n = seq_offsets.numel() - 1
        with torch.cuda.stream(stream):
            loss = torch.empty(max(n, 0), dtype=torch.float32, device=self.device)
            load = torch.empty((max(n, 0), self.E), dtype=torch.float32, device=self.device)
            ws = torch.empty(max(_lib.balance_workspace_bytes(self.sel, n), 1), dtype=torch.uint8, device=self.device)
            _lib.moe_balance_loss(self.sel, self.logits, self.idx, seq_offsets, alpha, loss, load, ws)
        return loss, load

    def backward(self, x, kept, dy, seq_offsets=None, load=None, dloss=None, alpha=0.0, stream=None) -> dict:
        """Gradients of a forward's output (dy [T, d] fp32), as moe_backward names them, from what checkpoint() kept of
        that forward.  Where there is a router, its projection's gradient reads x, the forward's input, or with None the
        checkpoint's values of it, so that x need not be kept beside them.  With a router, dloss [n_seq] adds the gradient
        of balance_loss(seq_offsets, alpha) of that forward."""
        if kept.forward not in (None, self.forwards):
            raise ValueError("this checkpoint's routing and outputs were overwritten by a later forward: keep them in 8 bits")
        if self.sel is None and dloss is not None:
            raise ValueError("the balance loss needs a layer with a router")
        self._need_weights()
        if dloss is None:
            seq_offsets = load = None
        # results and workspaces are the stream's own: freed here, they serve only what follows on it
        with torch.cuda.stream(stream):
            return self._backward(x, kept, dy, seq_offsets, load, dloss, alpha)

    def _backward(self, x, kept, dy, seq_offsets, load, dloss, alpha) -> dict:
        D, f32 = self.desc, dict(dtype=torch.float32, device=self.device)
        T, d, I, E, k = self.T, self.d, self.I, self.E, self.k
        grads = {n: torch.empty(s, **f32) for n, s in (
            ("dx", (T, d)), ("dw_gate", (E, I, d)), ("dw_up", (E, I, d)), ("dw_down", (E, d, I)), ("ds_gate", (I, d)),
            ("ds_up", (I, d)), ("ds_down", (d, I)), ("dg", (T, k)), ("dw_router", (E, d)))}
        xs, ys = _lib.saved(*kept.x), _lib.saved(*kept.y_perm)
        idx, w, offsets, row_src, row_of, logits = self._parts(kept.routing)
        ws = torch.empty(_lib.workspace_bytes(D, _lib.MOE_WS_BACKWARD_SAVED), dtype=torch.uint8, device=self.device)
        experts = (w, offsets, row_src, row_of, self.ex_w, self.sh_w, ys, dy)
        if self.sel is None:
            _lib.moe_backward_saved(D, xs, self.wr, idx, *experts, grads, ws)
            return grads
        _lib.moe_backward_saved(D, xs, None, None, *experts, {n: g for n, g in grads.items() if n != "dw_router"}, ws)
        dlogits = torch.empty((T, E), **f32)
        _lib.moe_select_backward(self.sel, logits, idx, grads["dg"], dlogits, seq_offsets, load, dloss, alpha)
        if x is None:
            data, scales, fmt = kept.x
            x = data if fmt == "bf16" else torch.empty((T, d), dtype=torch.bfloat16, device=self.device)
            if fmt != "bf16":
                _lib.moe_checkpoint_unpack(data, scales, fmt, x)
        ws = torch.empty(_lib.workspace_bytes(D, _lib.MOE_WS_ROUTER_GRAD), dtype=torch.uint8, device=self.device)
        _lib.moe_router_logits_backward(D, x, self.wr, dlogits, grads["dx"], grads["dx"], grads["dw_router"], ws)
        return grads

    def pack_experts(self, fmt="e4m3", keep=True, stream=None):
        """The routed experts' weights (bf16) as they are now in four bits (MX e2m1), for the forwards from here on; x and
        the experts' inner activations are packed in fmt, "e4m3" or "e2m1".  Called again it packs anew, in place (what a
        graph captured stays what it was captured with); adamw_step does.  keep=False lets go of the bf16 weights, once all that
        was launched and may read them has ended (not while a graph is captured): the layer then only serves, and a graph
        that captured them is not replayed any more."""
        if self.wt != "bf16":
            raise ValueError(f"experts are packed from bf16 weights, not {self.wt}")
        self._need_weights()
        if fmt not in _lib.MX_FORMATS:
            raise ValueError(f"format {fmt!r}")
        if not keep and torch.cuda.is_current_stream_capturing():
            raise ValueError("the experts' bf16 weights cannot be let go of while a graph is captured")
        E, T, d, I, A = self.E, self.T, self.d, self.I, self.T * self.k
        need = _lib.mx_ffn_workspace_bytes(E, A, d, I, fmt)
        if need == 0 or T * _lib.mx_code_bytes(d, fmt) > _lib.MX_GATHERED_BYTES:  # (found out before any weights are let go of)
            raise ValueError(f"{T} tokens of {d} in {fmt} are more than moe_mx_expert_ffn takes")
        with torch.cuda.stream(stream):
            if fmt not in self._packed_room:
                ws = torch.empty(need, dtype=torch.uint8, device=self.device)
                self._packed_room[fmt] = (*_lib.mx_empty(T, d, fmt, self.device), ws)
            mats = self.packed[1] if self.packed is not None else []
            if not mats:
                for N, K in ((I, d), (I, d), (d, I)):
                    codes, scales = _lib.mx_empty(E * N, K, "e2m1", self.device)
                    mats.append(_lib.mx(codes.view(E, N, K // 2), scales, "e2m1"))
            for n, m in zip(("gate", "up", "down"), mats):
                codes, scales = m.tensors
                _lib.moe_mx_pack(self.ex[n].view(-1, 2 * codes.shape[2]), codes.view(-1, codes.shape[2]), scales, "e2m1")
        self.packed = (fmt, mats)
        if not keep:
            # the packing on its stream, and forwards on any other: freed before those have read them, the weights' memory
            # would be handed out anew on the stream that they were allocated on
            torch.cuda.synchronize(self.ex["gate"].device)
            self.ex.update(gate=None, up=None, down=None)
            self.ex_w = None

    def _need_weights(self):
        if self.ex_w is None:
            raise ValueError("the experts' bf16 weights were let go of (pack_experts(keep=False))")

    def _weights(self):
        """The weights by their gradients' names (``backward``)."""
        ex, sh = self.ex, self.sh
        return {"dw_router": self.wr, "dw_gate": ex["gate"], "dw_up": ex["up"], "dw_down": ex["down"],
                "ds_gate": sh["gate"], "ds_up": sh["up"], "ds_down": sh["down"]}

    def adamw_state(self, states=8, masters=False) -> dict:
        """The optimizer's state of the layer's weights (bf16 experts, fp32 router), nothing seen yet: m and v in 8 or 32
        bits (in 8, a quarter of the memory, the second moments' roots are off by 11 to 18 %, one deviation), and with
        masters the fp32 weights that the bf16 ones are rounded from."""
        if self.wt == "e4m3":
            raise ValueError("weights in e4m3 have no step: keep bf16 ones")
        self._need_weights()
        if states not in (8, 32):
            raise ValueError(f"states of {states} bits")
        kind, kept = (torch.uint8 if states == 8 else torch.float32), {}
        for n, w in self._weights().items():
            new = lambda *shape: torch.zeros(*shape, dtype=kind, device=self.device)  # noqa: E731
            tiles = (w.numel() + 127) // 128
            kept[n] = {"m": new(w.shape), "v": new(w.shape), "m_scales": new(tiles) if states == 8 else None,
                       "v_scales": new(tiles) if states == 8 else None,
                       "master": w.view(torch.bfloat16).float() if masters and w.dtype == torch.int16 else None}
        return kept

    def adamw_step(self, grads, state, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, step=1, seed=0, grad_scale=None,
                   stream=None):
        """One moe_adamw step of the layer's weights, in place, by the gradients that ``backward`` returned; experts that
        are packed are packed anew."""
        self._need_weights()
        weights = self._weights()
        with torch.cuda.stream(stream):
            tensors = _lib.adamw_tensors(
                list(weights.values()), [grads[n].view(w.shape) for n, w in weights.items()],
                *([state[n][k] for n in weights] for k in ("m", "v", "m_scales", "v_scales", "master")))
            _lib.moe_adamw(tensors, lr, betas, eps, weight_decay, step, seed, grad_scale)
            if self.packed is not None:
                self.pack_experts(self.packed[0])

    def update_bias(self, bias, gamma=1e-3, stream=None):
        _lib.moe_bias_update(self.desc, self.counts, gamma, bias, stream)

    def step(self, x, bias, gamma=None, tokens_seen=0, stream=None):
        """One training step's forward and bias update; gamma defaults to the
        schedule's value for a step starting after `tokens_seen` tokens."""
        y = self.forward(x, bias, stream=stream)
        self.update_bias(bias, bias_gamma(tokens_seen) if gamma is None else gamma, stream)
        return y


# kbwen.com DeepSeek feed, "A bias term for each expert": the bias moves by
# 0.001 per step for the first 14.3T training tokens and by 0 for the rest.
# Reading: a step that starts before 14.3T tokens have been consumed uses
# 0.001.
GAMMA = 1e-3
GAMMA_TOKENS = 14.3e12


def bias_gamma(tokens_seen: float) -> float:
    """The bias step size for a training step that starts after `tokens_seen` tokens."""
    return GAMMA if tokens_seen < GAMMA_TOKENS else 0.0


def save_bias(path, bias) -> None:
    """Checkpoint the balancing state: the fp32 bias is the layer's only state
    that changes from step to step (DeepSeek V3 From Scratch, "In code":
    update_bias returns the new bias; kbwen.com DeepSeek feed, "A bias term
    for each expert").  Written as a .npy file holding the exact fp32 bits."""
    if isinstance(bias, torch.Tensor):
        bias = bias.detach().to("cpu").numpy()
    np.save(path, np.ascontiguousarray(bias, dtype=np.float32), allow_pickle=False)


def load_bias(path, device="cuda") -> torch.Tensor:
    """The bias saved by save_bias, as an fp32 tensor on `device` (bit-exact)."""
    b = np.load(path, allow_pickle=False)
    if b.dtype != np.float32 or b.ndim != 1:
        raise ValueError(f"{path}: expected a 1-D float32 bias, got {b.dtype} {b.shape}")
    return torch.from_numpy(b).to(device)


def layer_from_inputs(inp: dict, device="cuda", router=None) -> MoeLayer:
    """Build a layer from a synth.make_inputs() dict (weights uploaded once)."""
    c = inp["cfg"]
    return MoeLayer(c.T, c.d, c.I, c.act, c.wt, inp["wr"], inp["experts"], inp["shared"], c.E, c.k, device, router)


def upload(a, device="cuda"):
    return _dev(a, torch.device(device))
