"""ctypes binding of libmoe.so (include/moe.h): argument marshalling only.

Every function takes torch tensors that already live on the GPU, passes their
device pointers and the current HIP stream to the C ABI, and raises MoeError
on a non-zero status.  No arithmetic of the layer happens here.  If the
library has not been built this module fails loudly: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")

MOE_OK, MOE_EINVAL, MOE_ENOTSUP, MOE_EWORKSPACE, MOE_EHIP, MOE_ESCRATCH = range(6)
MOE_F32, MOE_BF16, MOE_E4M3 = 0, 1, 2
MOE_WS_DISPATCH, MOE_WS_FFN, MOE_WS_COMBINE, MOE_WS_ROUTE, MOE_WS_BACKWARD = 0, 1, 2, 3, 4
MOE_WS_ROUTER_LOGITS, MOE_WS_ROUTER_GRAD, MOE_WS_BACKWARD_SAVED = 5, 6, 7
MOE_SIGMOID, MOE_SOFTMAX = 0, 1
MOE_GROUP_MAX, MOE_GROUP_TOP_TWO = 0, 1
MOE_SAVED_BF16, MOE_SAVED_E4M3, MOE_SAVED_I8 = 0, 1, 2
DTYPES = {"f32": MOE_F32, "bf16": MOE_BF16, "e4m3": MOE_E4M3}
SCORES = {"sigmoid": MOE_SIGMOID, "softmax": MOE_SOFTMAX}
GROUP_SCORES = {"max": MOE_GROUP_MAX, "top2": MOE_GROUP_TOP_TWO}
MOE_MX_E4M3, MOE_MX_E2M1 = 0, 1
MX_FORMATS = {"e4m3": MOE_MX_E4M3, "e2m1": MOE_MX_E2M1}
MX_GATHERED_BYTES = (1 << 32) - (1 << 20)  # of x's codes, at most, where its rows are gathered
SAVED_FORMATS = {"bf16": MOE_SAVED_BF16, "e4m3": MOE_SAVED_E4M3, "i8": MOE_SAVED_I8}

EXPORTS = ("moe_route", "moe_dispatch", "moe_dispatch_noalloc", "moe_expert_ffn", "moe_expert_gate_up", "moe_expert_gate_up_rows",
           "moe_expert_down", "moe_combine", "moe_bias_update", "moe_backward", "moe_workspace_bytes",
           "moe_status_str", "moe_router_logits", "moe_router_logits_backward", "moe_select", "moe_select_backward",
           "moe_balance_loss", "moe_balance_workspace_bytes", "moe_checkpoint_pack", "moe_checkpoint_unpack",
           "moe_combine_backward", "moe_backward_saved", "moe_mx_pack", "moe_mx_unpack", "moe_mx_product",
           "moe_mx_product_workspace_bytes", "moe_mx_expert_ffn", "moe_mx_ffn_workspace_bytes", "moe_adamw")


class MoeError(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__(f"{fn} failed: {msg}")
        self.status = status


class Desc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32),
                ("I", ctypes.c_int32), ("act", ctypes.c_int32), ("wt", ctypes.c_int32)]


class FfnWeights(ctypes.Structure):
    _fields_ = [("gate", ctypes.c_void_p), ("up", ctypes.c_void_p), ("down", ctypes.c_void_p),
                ("s_gate", ctypes.c_void_p), ("s_up", ctypes.c_void_p), ("s_down", ctypes.c_void_p)]


class Select(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("score", ctypes.c_int32),
                ("n_group", ctypes.c_int32), ("topk_group", ctypes.c_int32), ("group_score", ctypes.c_int32),
                ("renorm", ctypes.c_int32), ("scale", ctypes.c_float), ("logits", ctypes.c_int32)]


class Saved(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("format", ctypes.c_int32)]


class Mx(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("format", ctypes.c_int32)]


class MxGroups(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("G", "M", "N", "K", "x_rows", "k")]


class AdamWTensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("w", "g", "m", "v", "m_scales", "v_scales", "master")] + [
        ("n", ctypes.c_int64), ("w_type", ctypes.c_int32), ("g_type", ctypes.c_int32), ("states", ctypes.c_int32)]


class AdamW(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps", "weight_decay")] + [
        ("step", ctypes.c_int64), ("seed", ctypes.c_uint64), ("grad_scale", ctypes.c_void_p), ("step_ptr", ctypes.c_void_p),
        ("lr_ptr", ctypes.c_void_p)]


_lib = None


def load(path: str = LIB_PATH):
    """Load libmoe.so (raises if it is missing: build it first)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build the HIP library first "
                           "(python -m sparse_expert_routing_amd.build); there is no CPU fallback")
    L = ctypes.CDLL(path)
    vp, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
    pd = ctypes.POINTER(Desc)
    pw = ctypes.POINTER(FfnWeights)
    L.moe_route.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_dispatch.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_dispatch_noalloc.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.moe_expert_ffn.argtypes = [pd, vp, vp, vp, pw, vp, vp, sz, vp]
    L.moe_expert_gate_up.argtypes = [pd, vp, vp, vp, pw, vp, sz, vp]
    L.moe_expert_gate_up_rows.argtypes = [pd, vp, vp, vp, pw, vp, sz, vp]
    L.moe_expert_down.argtypes = [pd, vp, pw, vp, vp, sz, vp]
    L.moe_combine.argtypes = [pd, vp, pw, vp, vp, vp, vp, vp, sz, vp]
    L.moe_bias_update.argtypes = [pd, vp, f32, vp, vp]
    L.moe_backward.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, pw, pw, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                               vp, sz, vp]
    i64, psel, psav = ctypes.c_int64, ctypes.POINTER(Select), ctypes.POINTER(Saved)
    L.moe_router_logits.argtypes = [pd, vp, vp, vp, vp, sz, vp]
    L.moe_router_logits_backward.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_select.argtypes = [psel, vp, i64, vp, vp, vp, vp]
    L.moe_select_backward.argtypes = [psel, vp, i64, vp, vp, vp, i32, vp, vp, f32, vp, vp]
    L.moe_balance_loss.argtypes = [psel, vp, i64, vp, vp, i32, f32, vp, vp, vp, sz, vp]
    L.moe_balance_workspace_bytes.argtypes = [psel, i32]
    L.moe_balance_workspace_bytes.restype = sz
    L.moe_checkpoint_pack.argtypes = [i64, i32, i32, vp, i64, i32, vp, vp, vp]
    L.moe_checkpoint_unpack.argtypes = [i64, i32, i32, vp, vp, i32, vp, i64, vp]
    L.moe_combine_backward.argtypes = [pd, vp, psav, vp, vp, vp, vp, vp]
    L.moe_backward_saved.argtypes = [pd, psav, vp, vp, vp, vp, vp, vp, pw, pw, psav, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                     vp, vp, sz, vp]
    pmx, pgr = ctypes.POINTER(Mx), ctypes.POINTER(MxGroups)
    L.moe_mx_pack.argtypes = [i64, i32, i32, vp, i64, i32, vp, vp, vp]
    L.moe_mx_unpack.argtypes = [i64, i32, i32, vp, vp, i32, vp, i64, vp]
    L.moe_mx_product.argtypes = [pgr, pmx, vp, vp, pmx, i32, vp, vp, sz, vp]
    L.moe_mx_product_workspace_bytes.argtypes = [pgr, i32]
    L.moe_mx_product_workspace_bytes.restype = sz
    L.moe_mx_expert_ffn.argtypes = [pgr, pmx, vp, vp, pmx, pmx, pmx, vp, vp, sz, vp]
    L.moe_mx_ffn_workspace_bytes.argtypes = [pgr, i32]
    L.moe_mx_ffn_workspace_bytes.restype = sz
    L.moe_adamw.argtypes = [ctypes.POINTER(AdamW), ctypes.POINTER(AdamWTensor), i32, vp]
    for fn in ("moe_mx_pack", "moe_mx_unpack", "moe_mx_product", "moe_mx_expert_ffn", "moe_adamw"):
        getattr(L, fn).restype = ctypes.c_int
    for fn in ("moe_router_logits", "moe_router_logits_backward", "moe_select", "moe_select_backward",
               "moe_balance_loss", "moe_checkpoint_pack", "moe_checkpoint_unpack", "moe_combine_backward",
               "moe_backward_saved"):
        getattr(L, fn).restype = ctypes.c_int
    for fn in ("moe_route", "moe_dispatch", "moe_dispatch_noalloc", "moe_expert_ffn", "moe_expert_gate_up", "moe_expert_gate_up_rows",
               "moe_expert_down", "moe_combine", "moe_bias_update", "moe_backward"):
        getattr(L, fn).restype = ctypes.c_int
    L.moe_workspace_bytes.argtypes = [pd, i32]
    L.moe_workspace_bytes.restype = sz
    L.moe_status_str.argtypes = [ctypes.c_int]
    L.moe_status_str.restype = ctypes.c_char_p
    _lib = L
    return L


def desc(T, d, E, k, I, act="bf16", wt="bf16") -> Desc:
    return Desc(T, d, E, k, I, DTYPES[act], DTYPES[wt])


def _ptr(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(fn, st):
    if st != MOE_OK:
        raise MoeError(fn, st, load().moe_status_str(st).decode())


def ffn_weights(gate, up, down, s_gate=None, s_up=None, s_down=None) -> FfnWeights:
    return FfnWeights(*[t.data_ptr() if t is not None else None for t in (gate, up, down, s_gate, s_up, s_down)])


def workspace_bytes(ds: Desc, stage: int) -> int:
    return load().moe_workspace_bytes(ctypes.byref(ds), stage)


def moe_route(ds, x, w_router, bias, idx, weights, gap=None, workspace=None, stream=None):
    nb = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("moe_route", load().moe_route(ctypes.byref(ds), _ptr(x), _ptr(w_router), _ptr(bias), _ptr(idx),
                                         _ptr(weights), _ptr(gap), _ptr(workspace), nb, _stream(stream)))


def moe_dispatch(ds, idx, x, counts, offsets, row_src, row_of, x_perm, x_perm_scale, workspace, stream=None):
    _check("moe_dispatch", load().moe_dispatch(
        ctypes.byref(ds), _ptr(idx), _ptr(x), _ptr(counts), _ptr(offsets), _ptr(row_src), _ptr(row_of),
        _ptr(x_perm), _ptr(x_perm_scale), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))


def moe_dispatch_noalloc(ds, idx, x, counts, offsets, row_src, row_of, x_perm, x_perm_scale, stream=None):
    _check("moe_dispatch_noalloc", load().moe_dispatch_noalloc(
        ctypes.byref(ds), _ptr(idx), _ptr(x), _ptr(counts), _ptr(offsets), _ptr(row_src), _ptr(row_of),
        _ptr(x_perm), _ptr(x_perm_scale), _stream(stream)))


def moe_expert_ffn(ds, x_perm, x_perm_scale, offsets, experts: FfnWeights, y_perm, workspace, stream=None):
    _check("moe_expert_ffn", load().moe_expert_ffn(
        ctypes.byref(ds), _ptr(x_perm), _ptr(x_perm_scale), _ptr(offsets), ctypes.byref(experts), _ptr(y_perm),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def moe_expert_gate_up(ds, x_perm, x_perm_scale, offsets, experts: FfnWeights, workspace, stream=None):
    _check("moe_expert_gate_up", load().moe_expert_gate_up(
        ctypes.byref(ds), _ptr(x_perm), _ptr(x_perm_scale), _ptr(offsets), ctypes.byref(experts),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def moe_expert_gate_up_rows(ds, x, row_src, offsets, experts: FfnWeights, workspace, stream=None):
    _check("moe_expert_gate_up_rows", load().moe_expert_gate_up_rows(
        ctypes.byref(ds), _ptr(x), _ptr(row_src), _ptr(offsets), ctypes.byref(experts),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def moe_expert_down(ds, offsets, experts: FfnWeights, y_perm, workspace, stream=None):
    _check("moe_expert_down", load().moe_expert_down(
        ctypes.byref(ds), _ptr(offsets), ctypes.byref(experts), _ptr(y_perm), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def moe_combine(ds, x, shared: FfnWeights, y_perm, row_of, weights, y, workspace, stream=None):
    _check("moe_combine", load().moe_combine(
        ctypes.byref(ds), _ptr(x), ctypes.byref(shared), _ptr(y_perm), _ptr(row_of), _ptr(weights), _ptr(y),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def moe_backward(ds, x, w_router, idx, weights, offsets, row_src, row_of, experts: FfnWeights,
                 shared: FfnWeights, y_perm, dy, grads: dict, workspace, stream=None):
    """grads: device tensors dx, dw_router, dw_gate, dw_up, dw_down, ds_gate, ds_up, ds_down, and
    optionally dg (fp32, written)."""
    _check("moe_backward", load().moe_backward(
        ctypes.byref(ds), _ptr(x), _ptr(w_router), _ptr(idx), _ptr(weights), _ptr(offsets), _ptr(row_src),
        _ptr(row_of), ctypes.byref(experts), ctypes.byref(shared), _ptr(y_perm), _ptr(dy),
        *[_ptr(grads[n]) for n in ("dx", "dw_router", "dw_gate", "dw_up", "dw_down", "ds_gate", "ds_up",
                                    "ds_down")],
        _ptr(grads.get("dg")), _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def moe_bias_update(ds, counts, gamma, bias, stream=None):
    _check("moe_bias_update", load().moe_bias_update(ctypes.byref(ds), _ptr(counts), gamma, _ptr(bias),
                                                     _stream(stream)))


# ------------------------------------------------- routing from logits, checkpoints
#
# These entry points check their tensors (type, shape, contiguity, device) and
# run on the device that holds them, whichever is current.

def selection(T, E, k, score="sigmoid", n_group=1, topk_group=1, group_score="top2", renorm=True, scale=1.0,
              logits="f32") -> Select:
    """The rule by which k of E experts are chosen for each of T tokens (moe_select_t)."""
    return Select(T, E, k, SCORES[score], n_group, topk_group, GROUP_SCORES[group_score], int(renorm), scale,
                  DTYPES[logits])


def saved(data, scales=None, fmt="bf16") -> Saved:
    """A saved activation (moe_saved_t): bf16 values, or 8-bit codes and their tiles' scales, which it keeps alive."""
    s = Saved(data.data_ptr(), scales.data_ptr() if scales is not None else None, SAVED_FORMATS[fmt])
    s.tensors = (data, scales)
    return s


def balance_workspace_bytes(sel: Select, n_seq: int) -> int:
    return load().moe_balance_workspace_bytes(ctypes.byref(sel), n_seq)


def _library():
    return load()


_torch = _raw_stream = _current_device = None
_KINDS = {}


def _bind_torch():
    global _torch, _raw_stream, _current_device
    import torch
    # the current stream's handle and the current device without an object made for them
    _raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    # the torch types a storage type travels in (bf16 also as its 16-bit patterns)
    _KINDS.update({MOE_F32: (torch.float32,), MOE_BF16: (torch.bfloat16, torch.int16), MOE_E4M3: (torch.uint8,),
                   "i32": (torch.int32,), "i64": (torch.int64,), "byte": (torch.uint8, torch.int8)})
    _torch = torch


class _Call:
    """Checks of one call's tensors, which have to lie on one GPU, and its launch there."""

    __slots__ = ("fn", "index", "elsewhere")

    def __init__(self, fn):
        if _torch is None:
            _bind_torch()
        self.fn, self.index, self.elsewhere = fn, -2, None  # (-1 is the CPU)

    def refuse(self, what):
        raise MoeError(self.fn, MOE_EINVAL, "MOE_EINVAL: " + what)

    def int32(self, name, n):
        """A size that the C ABI takes in 32 bits."""
        if n >= 1 << 31:
            self.refuse(f"{name}, {n}, is not below 2^31")
        return n

    def ptr(self, name, t, kind, shape, optional=False):
        """The address of a contiguous tensor of that type and shape."""
        if t is None:
            if not optional:
                self.refuse(f"{name} is missing")
            return None
        if t.dtype not in _KINDS[kind]:
            self.refuse(f"{name} has type {t.dtype}")
        if t.shape != shape:
            self.refuse(f"{name} has shape {tuple(t.shape)}, not {shape}")
        if not t.is_contiguous():
            self.refuse(f"{name} is not contiguous")
        if t.get_device() != self.index:
            self.on(name, t)
        return t.data_ptr()

    def fits(self, t, kind, shape):
        """Whether ptr would take a tensor that lies where the call's others do (where not, ptr says why)."""
        return (t is not None and t.get_device() == self.index and t.shape == shape and t.dtype in _KINDS[kind]
                and t.is_contiguous())

    def rows(self, name, t, kind, shape):
        """The address and row stride of a tensor whose rows are contiguous."""
        if t is None:
            self.refuse(f"{name} is missing")
        if t.dtype not in _KINDS[kind]:
            self.refuse(f"{name} has type {t.dtype}")
        if t.shape != shape:
            self.refuse(f"{name} has shape {tuple(t.shape)}, not {shape}")
        ld, step = t.stride()
        if shape[0] == 1:
            ld = max(ld, shape[1])
        if (shape[1] > 1 and step != 1) or ld < shape[1]:
            self.refuse(f"{name} has strides {tuple(t.stride())}: its rows have to be contiguous and apart")
        if t.get_device() != self.index:
            self.on(name, t)
        return t.data_ptr(), ld

    def saved(self, name, s, rows, cols):
        """A saved activation of that shape (its tensors are looked at where saved() made it)."""
        if s is None:
            self.refuse(f"{name} is missing")
        data, scales = getattr(s, "tensors", (None, None))
        if data is not None:
            plain = s.format == MOE_SAVED_BF16
            self.ptr(f"{name}'s values" if plain else f"{name}'s codes", data, MOE_BF16 if plain else "byte", (rows, cols))
            self.ptr(f"{name}'s scales", scales, MOE_E4M3, (rows, (cols + 127) // 128), plain)
        return ctypes.byref(s)

    def on(self, name, t):
        if self.index < 0 and t.is_cuda:
            self.index = t.get_device()
        elif self.elsewhere is None:  # reported behind the types and shapes
            self.elsewhere = f"{name} is on {t.device}" + (f", not cuda:{self.index}" if self.index >= 0 else "")

    def workspace(self, t):
        """Address and size of a workspace (None: none)."""
        if t is None:
            return None, 0
        if not t.is_contiguous():
            self.refuse("the workspace is not contiguous")
        if t.get_device() != self.index:
            self.on("the workspace", t)
        return t.data_ptr(), t.numel() * t.element_size()

    def nothing(self, stream):
        """A call of no rows: where run would look, and no launch."""
        if self.elsewhere is not None:
            self.refuse(self.elsewhere)
        if stream is not None and stream.device.index != self.index:
            self.refuse(f"the stream is on {stream.device}, not cuda:{self.index}")

    def no_rows(self, x_rows, row_src, k, stream):
        """A product of no rows (a shard that no token chose), which the C ABI does not take: nothing, if its x is fit for it."""
        if row_src is None and (k != 1 or x_rows != 0):
            self.refuse(f"x's {x_rows} rows and k = {k} are not those of no rows")
        self.nothing(stream)

    def run(self, call, *args, stream=None):
        if self.elsewhere is not None:
            self.refuse(self.elsewhere)
        index = self.index
        if stream is None:
            raw = _raw_stream(index)
        elif stream.device.index != index:
            self.refuse(f"the stream is on {stream.device}, not cuda:{index}")
        else:
            raw = stream.cuda_stream
        if _current_device() == index:
            st = call(*args, raw)
        else:
            with _torch.cuda.device(index):
                st = call(*args, raw)
        if st != MOE_OK:
            _check(self.fn, st)


def moe_router_logits(ds, x, w_router, logits, workspace=None, stream=None):
    """logits [T, E] = x . w_router^T in fp32."""
    c = _Call("moe_router_logits")
    args = (c.ptr("x", x, ds.act, (ds.T, ds.d)), c.ptr("w_router", w_router, MOE_F32, (ds.E, ds.d)),
            c.ptr("logits", logits, MOE_F32, (ds.T, ds.E)))
    c.run(load().moe_router_logits, ctypes.byref(ds), *args, *c.workspace(workspace), stream=stream)


def moe_router_logits_backward(ds, x, w_router, dlogits, dx_in, dx, dw_router, workspace=None, stream=None):
    """dx = dx_in + dlogits . w_router (dx_in may be None, or dx itself), dw_router = dlogits^T . x."""
    c = _Call("moe_router_logits_backward")
    args = (c.ptr("x", x, ds.act, (ds.T, ds.d)), c.ptr("w_router", w_router, MOE_F32, (ds.E, ds.d)),
            c.ptr("dlogits", dlogits, MOE_F32, (ds.T, ds.E)), c.ptr("dx_in", dx_in, MOE_F32, (ds.T, ds.d), True),
            c.ptr("dx", dx, MOE_F32, (ds.T, ds.d)), c.ptr("dw_router", dw_router, MOE_F32, (ds.E, ds.d)))
    c.run(load().moe_router_logits_backward, ctypes.byref(ds), *args, *c.workspace(workspace), stream=stream)


def moe_select(sel: Select, logits, bias, idx, weights, stream=None):
    """The choice of experts and its combine weights; logits [T, E] with any row stride, bias [E] or None."""
    c = _Call("moe_select")
    p, ld = c.rows("logits", logits, sel.logits, (sel.T, sel.E))
    args = (c.ptr("bias", bias, MOE_F32, (sel.E,), True), c.ptr("idx", idx, "i32", (sel.T, sel.k)),
            c.ptr("weights", weights, MOE_F32, (sel.T, sel.k)))
    c.run(load().moe_select, ctypes.byref(sel), p, ld, *args, stream=stream)


def moe_select_backward(sel: Select, logits, idx, dweights, dlogits, seq_offsets=None, load=None, dloss=None, alpha=0.0,
                        stream=None):
    """dlogits [T, E] through the weights (dweights [T, k], or None) and the balance loss (seq_offsets, load and dloss
    of moe_balance_loss, or None)."""
    c = _Call("moe_select_backward")
    if seq_offsets is None and (load is not None or dloss is not None):
        c.refuse("load and dloss need seq_offsets")
    p, ld = c.rows("logits", logits, sel.logits, (sel.T, sel.E))
    n = c.int32("seq_offsets' count", seq_offsets.numel() - 1) if seq_offsets is not None else 0
    on = seq_offsets is None
    args = (c.ptr("idx", idx, "i32", (sel.T, sel.k), dweights is None),
            c.ptr("dweights", dweights, MOE_F32, (sel.T, sel.k), True),
            c.ptr("seq_offsets", seq_offsets, "i32", (n + 1,), True), n,
            c.ptr("load", load, MOE_F32, (n, sel.E), on), c.ptr("dloss", dloss, MOE_F32, (n,), on), alpha,
            c.ptr("dlogits", dlogits, MOE_F32, (sel.T, sel.E)))
    c.run(_library().moe_select_backward, ctypes.byref(sel), p, ld, *args, stream=stream)


def moe_balance_loss(sel: Select, logits, idx, seq_offsets, alpha, loss, load, workspace, stream=None):
    """The sequence-wise balance loss [n_seq] and each expert's load [n_seq, E]."""
    c = _Call("moe_balance_loss")
    p, ld = c.rows("logits", logits, sel.logits, (sel.T, sel.E))
    if seq_offsets is None or seq_offsets.numel() < 2:
        c.refuse("seq_offsets holds no sequence")
    n = c.int32("seq_offsets' count", seq_offsets.numel() - 1)
    args = (c.ptr("idx", idx, "i32", (sel.T, sel.k)), c.ptr("seq_offsets", seq_offsets, "i32", (n + 1,)), n, alpha,
            c.ptr("loss", loss, MOE_F32, (n,)), c.ptr("load", load, MOE_F32, (n, sel.E)))
    c.run(_library().moe_balance_loss, ctypes.byref(sel), p, ld, *args, *c.workspace(workspace), stream=stream)


def _plain_type(c, name, t):
    """MOE_F32 or MOE_BF16 of a plain 2-D tensor."""
    if t is None or t.dim() != 2:
        c.refuse(f"{name} has to be a matrix")
    if t.shape[1] >= 1 << 31:
        c.int32(f"{name}'s columns", t.shape[1])
    for kind in (MOE_F32, MOE_BF16):
        if t.dtype in _KINDS[kind]:
            return kind
    c.refuse(f"{name} has type {t.dtype}")


def _codes(c, codes, scales, fmt, rows, cols):
    if fmt not in ("e4m3", "i8"):
        c.refuse(f"format {fmt!r}")
    return (c.ptr("codes", codes, "byte", (rows, cols)),
            c.ptr("scales", scales, MOE_E4M3, (rows, (cols + 127) // 128)))


def moe_checkpoint_pack(src, codes, scales, fmt, stream=None):
    """src [rows, cols] (fp32 or bf16, any row stride) as 8-bit codes [rows, cols] and scales [rows, ceil(cols/128)];
    fmt: "e4m3" or "i8"."""
    c = _Call("moe_checkpoint_pack")
    kind = _plain_type(c, "src", src)
    rows, cols = src.shape
    p, ld = c.rows("src", src, kind, (rows, cols))
    q, s = _codes(c, codes, scales, fmt, rows, cols)
    c.run(load().moe_checkpoint_pack, rows, cols, kind, p, ld, SAVED_FORMATS[fmt], q, s, stream=stream)


def moe_checkpoint_unpack(codes, scales, fmt, dst, stream=None):
    """The values of 8-bit codes into dst [rows, cols] (fp32 or bf16, any row stride)."""
    c = _Call("moe_checkpoint_unpack")
    kind = _plain_type(c, "dst", dst)
    rows, cols = dst.shape
    q, s = _codes(c, codes, scales, fmt, rows, cols)
    p, ld = c.rows("dst", dst, kind, (rows, cols))
    c.run(load().moe_checkpoint_unpack, rows, cols, kind, q, s, SAVED_FORMATS[fmt], p, ld, stream=stream)


def moe_combine_backward(ds, dy, y_perm: Saved, row_of, weights, dy_perm, dg, stream=None):
    """The combine's gradient from saved routed outputs: dy_perm [T*k, d] bf16 and dg [T, k]."""
    c = _Call("moe_combine_backward")
    args = (c.ptr("dy", dy, MOE_F32, (ds.T, ds.d)), c.saved("y_perm", y_perm, ds.T * ds.k, ds.d), c.ptr("row_of", row_of, "i32", (ds.T * ds.k,)),
            c.ptr("weights", weights, MOE_F32, (ds.T, ds.k)), c.ptr("dy_perm", dy_perm, MOE_BF16, (ds.T * ds.k, ds.d)),
            c.ptr("dg", dg, MOE_F32, (ds.T, ds.k)))
    c.run(load().moe_combine_backward, ctypes.byref(ds), *args, stream=stream)


def moe_backward_saved(ds, x: Saved, w_router, idx, weights, offsets, row_src, row_of, experts: FfnWeights,
                       shared: FfnWeights, y_perm: Saved, dy, grads: dict, workspace, stream=None):
    """moe_backward from saved activations; w_router None leaves the router's share to the caller (grads then has no
    dw_router and has dg)."""
    c = _Call("moe_backward_saved")
    A, T, d, E, I = ds.T * ds.k, ds.T, ds.d, ds.E, ds.I
    own = w_router is None
    head = (c.saved("x", x, T, d), c.ptr("w_router", w_router, MOE_F32, (E, d), True),
            c.ptr("idx", idx, "i32", (T, ds.k), own), c.ptr("weights", weights, MOE_F32, (T, ds.k)),
            c.ptr("offsets", offsets, "i32", (E + 1,)), c.ptr("row_src", row_src, "i32", (A,)),
            c.ptr("row_of", row_of, "i32", (A,)), ctypes.byref(experts), ctypes.byref(shared),
            c.saved("y_perm", y_perm, A, d), c.ptr("dy", dy, MOE_F32, (T, d)))
    out = [c.ptr(n, grads.get(n), MOE_F32, s, n == "dg" or (n == "dw_router" and own))
           for n, s in (("dx", (T, d)), ("dw_router", (E, d)), ("dw_gate", (E, I, d)), ("dw_up", (E, I, d)),
                        ("dw_down", (E, d, I)), ("ds_gate", (I, d)), ("ds_up", (I, d)), ("ds_down", (d, I)),
                        ("dg", (T, ds.k)))]
    c.run(load().moe_backward_saved, ctypes.byref(ds), *head, *out, *c.workspace(workspace), stream=stream)


# ------------------------------------------------- microscaled operands, products by expert

def mx(codes, scales, fmt) -> Mx:
    """A microscaled matrix (moe_mx_t): codes and their blocks' scale bytes, which it keeps alive; fmt "e4m3" or "e2m1"."""
    m = Mx(codes.data_ptr(), scales.data_ptr(), MX_FORMATS[fmt])
    m.tensors = (codes, scales)
    return m


def mx_code_bytes(cols, fmt):
    """Bytes of a row's codes."""
    return cols if fmt == "e4m3" else (cols + 1) // 2


def mx_empty(rows, cols, fmt, device="cuda"):
    """Room for a packed matrix [rows, cols]: codes and scales."""
    import torch
    return (torch.empty((rows, mx_code_bytes(cols, fmt)), dtype=torch.uint8, device=device),
            torch.empty(((cols + 127) // 128, rows, 4), dtype=torch.uint8, device=device))


def _mx_matrix(c, codes, scales, fmt, rows, cols):
    if fmt not in MX_FORMATS:
        c.refuse(f"format {fmt!r}")
    return (c.ptr("codes", codes, "byte", (rows, mx_code_bytes(cols, fmt))),
            c.ptr("scales", scales, MOE_E4M3, ((cols + 127) // 128, rows, 4)))


def moe_mx_pack(src, codes, scales, fmt, stream=None):
    """src [rows, cols] (fp32 or bf16, any row stride) as microscaled codes [rows, cols] ("e4m3") or [rows, ceil(cols/2)]
    ("e2m1") and scales [ceil(cols/128), rows, 4].  No rows are allowed."""
    c = _Call("moe_mx_pack")
    kind = _plain_type(c, "src", src)
    rows, cols = src.shape
    p, ld = c.rows("src", src, kind, (rows, cols))
    q, s = _mx_matrix(c, codes, scales, fmt, rows, cols)
    if rows == 0:  # (the C ABI takes no empty matrix)
        return c.nothing(stream)
    c.run(load().moe_mx_pack, rows, cols, kind, p, ld, MX_FORMATS[fmt], q, s, stream=stream)


def moe_mx_unpack(codes, scales, fmt, dst, stream=None):
    """The values of microscaled codes into dst [rows, cols] (fp32 or bf16, any row stride)."""
    c = _Call("moe_mx_unpack")
    kind = _plain_type(c, "dst", dst)
    rows, cols = dst.shape
    q, s = _mx_matrix(c, codes, scales, fmt, rows, cols)
    p, ld = c.rows("dst", dst, kind, (rows, cols))
    if rows == 0:  # (the C ABI takes no empty matrix)
        return c.nothing(stream)
    c.run(load().moe_mx_unpack, rows, cols, kind, q, s, MX_FORMATS[fmt], p, ld, stream=stream)


def mx_product_workspace_bytes(G, M, N, K, out="bf16") -> int:
    if max(G, M, N, K) >= 1 << 31:  # (past the C ABI's 32 bits: no product that it takes)
        return 0
    return load().moe_mx_product_workspace_bytes(ctypes.byref(MxGroups(G, M, N, K, M, 1)), DTYPES[out])


def mx_ffn_workspace_bytes(E, M, d, I, fmt) -> int:
    if max(E, M, d, I) >= 1 << 31:
        return 0
    return load().moe_mx_ffn_workspace_bytes(ctypes.byref(MxGroups(E, M, I, d, M, 1)), MX_FORMATS[fmt])


def _mx_weights(c, name, m, shape=None):
    """(G, N, K) of packed matrices [G, N, K], checked (against a shape)."""
    if m is None or getattr(m, "tensors", None) is None:
        c.refuse(f"{name} has to be packed matrices (mx)")
    codes, scales = m.tensors
    if m.format != MOE_MX_E2M1:
        raise MoeError(c.fn, MOE_ENOTSUP, f"MOE_ENOTSUP: {name} has to be in e2m1")
    size = codes.shape
    if len(size) != 3:
        c.refuse(f"{name}'s codes have shape {tuple(size)}, not [G, N, K / 2]")
    G, N, K = shape or (size[0], size[1], 2 * size[2])
    if not c.fits(codes, "byte", (G, N, K // 2)):
        c.ptr(f"{name}'s codes", codes, "byte", (G, N, K // 2))
    if not c.fits(scales, MOE_E4M3, ((K + 127) // 128, G * N, 4)):
        c.ptr(f"{name}'s scales", scales, MOE_E4M3, ((K + 127) // 128, G * N, 4))
    return c.int32("matrices", G), c.int32("weights' rows", N), c.int32("weights' columns", K)


def _mx_rows(c, x, K, M, row_src, k):
    """The rows of x [x_rows, K], checked, and row_src's address."""
    if x is None or getattr(x, "tensors", None) is None:
        c.refuse("x has to be a packed matrix (mx)")
    codes, scales = x.tensors
    size = codes.shape
    rows = size[0] if len(size) == 2 else 0
    wide, scale = (rows, K if x.format == MOE_MX_E4M3 else K // 2), ((K + 127) // 128, rows, 4)
    if not c.fits(codes, "byte", wide):
        c.ptr("x's codes", codes, "byte", wide)
    if not c.fits(scales, MOE_E4M3, scale):
        c.ptr("x's scales", scales, MOE_E4M3, scale)
    if not 0 < k < 1 << 31:
        c.refuse(f"k, {k}, is not from 1 to 2^31 - 1")
    return c.int32("x's rows", rows), None if row_src is None else c.ptr("row_src", row_src, "i32", (M,))


def moe_mx_product(x: Mx, w: Mx, offsets, out, workspace=None, row_src=None, k=1, stream=None):
    """out [M, N] (fp32 or bf16): rows offsets[g] .. offsets[g+1] are x's (row r: x's row r, or row_src[r] // k) times
    w[g]^T, w [G, N, K] in four bits.  M = 0 is allowed (a shard that no token chose)."""
    c = _Call("moe_mx_product")
    G, N, K = _mx_weights(c, "w", w)
    kind = _plain_type(c, "out", out)
    M = c.int32("out's rows", out.shape[0])
    rows, src = _mx_rows(c, x, K, M, row_src, k)
    args = (c.ptr("offsets", offsets, "i32", (G + 1,)), ctypes.byref(w), kind, c.ptr("out", out, kind, (M, N)))
    if M == 0:
        return c.no_rows(rows, row_src, k, stream)
    c.run(load().moe_mx_product, ctypes.byref(MxGroups(G, M, N, K, rows, k)), ctypes.byref(x), src, *args,
          *c.workspace(workspace), stream=stream)


def moe_mx_expert_ffn(x: Mx, gate: Mx, up: Mx, down: Mx, offsets, y, workspace, row_src=None, k=1, stream=None):
    """The routed experts' SwiGLU FFN on weights in four bits (gate, up [G, I, d], down [G, d, I]): y [M, d] bf16 for
    the rows of moe_mx_product (or none); h is packed in x's format."""
    c = _Call("moe_mx_expert_ffn")
    G, I, d = _mx_weights(c, "gate", gate)
    _mx_weights(c, "up", up, (G, I, d))
    _mx_weights(c, "down", down, (G, d, I))
    if y is None or y.dim() != 2:
        c.refuse("y has to be a matrix")
    M = c.int32("y's rows", y.shape[0])
    rows, src = _mx_rows(c, x, d, M, row_src, k)
    args = (c.ptr("offsets", offsets, "i32", (G + 1,)), ctypes.byref(gate), ctypes.byref(up), ctypes.byref(down),
            c.ptr("y", y, MOE_BF16, (M, d)))
    if M == 0:
        return c.no_rows(rows, row_src, k, stream)
    c.run(load().moe_mx_expert_ffn, ctypes.byref(MxGroups(G, M, I, d, rows, k)), ctypes.byref(x), src, *args,
          *c.workspace(workspace), stream=stream)


# ------------------------------------------------- the optimizer's step

class AdamWTensors:
    """The tensors of a step: their addresses for moe_adamw, and themselves, which it keeps alive."""

    def __init__(self, table, index, tensors):
        self.table, self.index, self.tensors = table, index, tensors


def adamw_tensors(weights, grads, m, v, m_scales=None, v_scales=None, masters=None) -> AdamWTensors:
    """Lists of contiguous tensors of equal length each: weights and gradients in fp32 or bf16; states in fp32, or in
    8 bits (uint8 codes) with m_scales and v_scales [ceil(n/128)]; masters: fp32 weights that the step works on (an entry
    or the list may be None).  What a step writes may not overlap with anything else of it: a weight that a model uses
    twice is listed once.  Made once for the tensors of a model, for moe_adamw."""
    c = _Call("moe_adamw")
    n = len(weights)
    empty = [None] * n
    lists = [list(t) if t is not None else empty for t in (weights, grads, m, v, m_scales, v_scales, masters)]
    if any(len(t) != n for t in lists):
        c.refuse(f"lists of {', '.join(str(len(t)) for t in lists)} tensors")
    table = (AdamWTensor * n)()
    for i, (w, g, mi, vi, ms, vs, ma) in enumerate(zip(*lists)):
        if w is None:
            c.refuse(f"weight {i} is missing")
        kinds = []
        for name, t in (("weight", w), ("gradient", g)):
            kind = next((q for q in (MOE_F32, MOE_BF16) if t is not None and t.dtype in _KINDS[q]), None)
            if kind is None:
                c.refuse(f"{name} {i} is missing" if t is None else f"{name} {i} has type {t.dtype}")
            kinds.append(kind)
        wide = mi is not None and mi.dtype in _KINDS[MOE_F32]
        state = MOE_F32 if wide else MOE_E4M3
        tiles = ((w.numel() + 127) // 128,)
        table[i] = AdamWTensor(
            c.ptr(f"weight {i}", w, kinds[0], w.shape), c.ptr(f"gradient {i}", g, kinds[1], w.shape),
            c.ptr(f"m {i}", mi, state, w.shape), c.ptr(f"v {i}", vi, state, w.shape),
            c.ptr(f"m's scales {i}", ms, MOE_E4M3, tiles, wide), c.ptr(f"v's scales {i}", vs, MOE_E4M3, tiles, wide),
            c.ptr(f"master {i}", ma, MOE_F32, w.shape, True), w.numel(), kinds[0], kinds[1], 32 if wide else 8)
    _apart(c, lists)
    if c.elsewhere is not None:
        c.refuse(c.elsewhere)
    return AdamWTensors(table, c.index, lists)


def _apart(c, lists):
    """Refuses a step that writes what it reads or writes elsewhere (its workgroups would race)."""
    names = ("weight", "gradient", "m", "v", "m's scales", "v's scales", "master")
    places = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), k, i)
                    for k, ts in enumerate(lists) for i, t in enumerate(ts) if t is not None and t.numel())
    last = written = (0, 0, 0, 0)  # those that reach furthest, of all so far and of those that the step writes
    for p in places:
        other = written if p[2] == 1 else last
        if p[0] < other[1]:
            c.refuse(f"{names[p[2]]} {p[3]} and {names[other[2]]} {other[3]} overlap")
        if p[1] > last[1]:
            last = p
        if p[2] != 1 and p[1] > written[1]:
            written = p


def moe_adamw(tensors: AdamWTensors, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, step=1, seed=0, grad_scale=None,
              stream=None):
    """One AdamW step of adamw_tensors(...).  lr and step: numbers, or tensors of one element on the device (fp32,
    int64), which a replayed graph reads anew; grad_scale: one fp32 on the device that the gradients are multiplied by
    (not finite: nothing changes); seed: of the stochastic rounding of 8-bit states and of bf16 weights without
    masters, which with step and the element's place gives its random numbers."""
    c = _Call("moe_adamw")
    c.index = tensors.index
    n = len(tensors.table)
    if n == 0:
        return
    on_device = [hasattr(t, "data_ptr") for t in (lr, step)]
    if not on_device[1] and not 0 < step < 1 << 63:
        c.refuse(f"step, {step}, is not from 1 to 2^63 - 1")
    rule = AdamW(0.0 if on_device[0] else lr, betas[0], betas[1], eps, weight_decay, 1 if on_device[1] else step,
                 seed & 0xFFFFFFFFFFFFFFFF,
                 c.ptr("grad_scale", grad_scale, MOE_F32, (1,)) if grad_scale is not None else None,
                 c.ptr("step", step, "i64", (1,)) if on_device[1] else None,
                 c.ptr("lr", lr, MOE_F32, (1,)) if on_device[0] else None)
    c.run(load().moe_adamw, ctypes.byref(rule), tensors.table, n, stream=stream)
