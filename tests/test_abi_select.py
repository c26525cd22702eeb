"""Refusals of the routing-from-logits and checkpoint entry points, on the CPU: by the
C ABI's host checks (every call here fails them, so no kernel is launched) and by
the binding's checks of its tensors."""
import ctypes

import pytest
import torch

from sparse_expert_routing_amd import _lib

P = 0x1000  # an address that no call gets to read
OK, EINVAL, ENOTSUP, EWORKSPACE = _lib.MOE_OK, _lib.MOE_EINVAL, _lib.MOE_ENOTSUP, _lib.MOE_EWORKSPACE


def rule(**kw):
    d = dict(T=16, E=256, k=8, n_group=8, topk_group=4)
    raw = {n: kw.pop(n) for n in list(kw) if n in ("score_", "logits_", "group_score_", "renorm_")}
    s = _lib.selection(**{**d, **kw})
    for n, v in raw.items():
        setattr(s, n[:-1], v)
    return s


BAD_RULES = [
    (dict(T=0), EINVAL), (dict(T=-3), EINVAL), (dict(E=0), EINVAL), (dict(k=0), EINVAL), (dict(k=257), EINVAL),
    (dict(n_group=0), EINVAL), (dict(n_group=7), EINVAL), (dict(topk_group=0), EINVAL), (dict(topk_group=9), EINVAL),
    (dict(n_group=64, topk_group=1), EINVAL), (dict(score_=2), EINVAL), (dict(group_score_=-1), EINVAL),
    (dict(renorm_=2), EINVAL), (dict(scale=float("inf")), EINVAL), (dict(scale=float("nan")), EINVAL),
    (dict(logits_=_lib.MOE_E4M3), ENOTSUP), (dict(logits_=9), EINVAL), (dict(E=1032, n_group=1, topk_group=1), ENOTSUP),
    (dict(k=65, n_group=1, topk_group=1), ENOTSUP), (dict(T=1 << 28), ENOTSUP),
]


@pytest.mark.parametrize("kw,status", BAD_RULES)
def test_rules_refused_by_every_call(kw, status):
    L, s = _lib.load(), rule(**kw)
    r = ctypes.byref(s)
    assert L.moe_select(r, P, 4096, P, P, P, None) == status
    assert L.moe_select_backward(r, P, 4096, P, P, None, 0, None, None, 0.0, P, None) == status
    assert L.moe_balance_loss(r, P, 4096, P, P, 1, 0.1, P, P, P, 1 << 40, None) == status
    assert L.moe_balance_workspace_bytes(r, 1) == 0


def test_null_rule_and_pointers():
    L, r = _lib.load(), ctypes.byref(rule())
    assert L.moe_select(None, P, 256, None, P, P, None) == EINVAL
    for args in ((None, 256, None, P, P), (P, 255, None, P, P), (P, 256, None, None, P), (P, 256, None, P, None)):
        assert L.moe_select(r, *args, None) == EINVAL
    bad = [
        (None, 256, P, P, None, 0, None, None, 0.0, P), (P, 255, P, P, None, 0, None, None, 0.0, P),
        (P, 256, P, P, None, 0, None, None, 0.0, None), (P, 256, P, None, None, 0, None, None, 0.0, P),  # nothing to do
        (P, 256, None, P, None, 0, None, None, 0.0, P),  # weights without ids
        (P, 256, P, P, P, 0, P, P, 0.0, P), (P, 256, P, P, P, 1, None, P, 0.0, P), (P, 256, P, P, P, 1, P, None, 0.0, P),
    ]
    for args in bad:
        assert L.moe_select_backward(r, *args, None) == EINVAL
    need = L.moe_balance_workspace_bytes(r, 5)
    assert need >= 5 * 256 * 8
    for args, st in (((P, 256, P, P, 0, 0.1, P, P, P, need), EINVAL), ((P, 256, P, None, 5, 0.1, P, P, P, need), EINVAL),
                     ((P, 256, None, P, 5, 0.1, P, P, P, need), EINVAL), ((P, 256, P, P, 5, 0.1, None, P, P, need), EINVAL),
                     ((P, 256, P, P, 5, 0.1, P, None, P, need), EINVAL), ((P, 200, P, P, 5, 0.1, P, P, P, need), EINVAL),
                     ((P, 256, P, P, 5, 0.1, P, P, P + 4, need), EINVAL),
                     ((P, 256, P, P, 5, 0.1, P, P, P, need - 1), EWORKSPACE),
                     ((P, 256, P, P, 5, 0.1, P, P, None, need), EWORKSPACE)):
        assert L.moe_balance_loss(r, *args, None) == st
    assert L.moe_balance_workspace_bytes(r, 0) == 0 and L.moe_balance_workspace_bytes(None, 1) == 0


@pytest.mark.parametrize("rows,cols,kind,ld,fmt,status", [
    (0, 8, 1, 8, 1, EINVAL), (-1, 8, 1, 8, 1, EINVAL), (8, 0, 1, 8, 1, EINVAL), (8, 8, 1, 7, 1, EINVAL),
    (8, 8, 2, 8, 1, ENOTSUP), (8, 8, 5, 8, 1, EINVAL), (8, 8, 0, 8, 0, EINVAL), (8, 8, 0, 8, 3, EINVAL),
    (1 << 60, 8, 0, 8, 1, ENOTSUP), (1, 8, 0, 1 << 62, 1, ENOTSUP)])
def test_checkpoint_shapes(rows, cols, kind, ld, fmt, status):
    L = _lib.load()
    assert L.moe_checkpoint_pack(rows, cols, kind, P, ld, fmt, P, P, None) == status
    assert L.moe_checkpoint_unpack(rows, cols, kind, P, P, fmt, P, ld, None) == status


def test_checkpoint_null_pointers():
    L = _lib.load()
    for i in range(3):
        p = [None if i == j else P for j in range(3)]
        assert L.moe_checkpoint_pack(8, 8, 1, p[0], 8, 1, p[1], p[2], None) == EINVAL
        assert L.moe_checkpoint_unpack(8, 8, 1, p[0], p[1], 1, p[2], 8, None) == EINVAL


def good_desc(**kw):
    d = dict(T=64, d=256, E=256, k=8, I=128, act="bf16", wt="bf16")
    return _lib.desc(**{**d, **kw})


SAVED_BAD = [_lib.Saved(None, None, 0), _lib.Saved(P, None, 1), _lib.Saved(P, None, 2), _lib.Saved(P, P, 3),
             _lib.Saved(P + 8, None, 0)]


def test_combine_backward_refusals():
    L, ds = _lib.load(), ctypes.byref(good_desc())
    ok = _lib.Saved(P, P, 1)
    for i in (0, 2, 3, 4, 5):
        a = [P, ctypes.byref(ok), P, P, P, P]
        a[i] = None
        assert L.moe_combine_backward(ds, *a, None) == EINVAL
    for s in SAVED_BAD:
        assert L.moe_combine_backward(ds, P, ctypes.byref(s), P, P, P, P, None) == EINVAL
    assert L.moe_combine_backward(ds, P, None, P, P, P, P, None) == EINVAL
    assert L.moe_combine_backward(ds, P + 4, ctypes.byref(ok), P, P, P, P, None) == EINVAL
    assert L.moe_combine_backward(ds, P, ctypes.byref(ok), P, P, P + 2, P, None) == EINVAL
    assert L.moe_combine_backward(ctypes.byref(good_desc(k=4)), P, ctypes.byref(ok), P, P, P, P, None) == ENOTSUP


def call_backward_saved(ds, x, y, w_router=P, idx=P, dw_router=P, dg=P, ws=P, nb=1 << 50, w=None):
    w = ctypes.byref(w or _lib.FfnWeights(P, P, P, P, P, P))
    return _lib.load().moe_backward_saved(ctypes.byref(ds), x, w_router, idx, P, P, P, P, w, w, y, P, P, dw_router, P, P, P,
                                          P, P, P, dg, ws, nb, None)


def test_backward_saved_refusals():
    ok, ds = ctypes.byref(_lib.Saved(P, P, 1)), good_desc()
    for s in SAVED_BAD:
        assert call_backward_saved(ds, ctypes.byref(s), ok) == EINVAL
        assert call_backward_saved(ds, ok, ctypes.byref(s)) == EINVAL
    assert call_backward_saved(ds, None, ok) == EINVAL
    assert call_backward_saved(ds, ok, ok, w_router=None) == EINVAL               # dw_router without w_router
    assert call_backward_saved(ds, ok, ok, w_router=None, dw_router=None, dg=None) == EINVAL  # the gradient would be lost
    assert call_backward_saved(ds, ok, ok, dw_router=None) == EINVAL
    assert call_backward_saved(ds, ok, ok, idx=None) == EINVAL
    assert call_backward_saved(ds, ok, ok, w=_lib.FfnWeights(P, P, None, P, P, P)) == EINVAL
    need = _lib.workspace_bytes(ds, _lib.MOE_WS_BACKWARD_SAVED)
    assert need >= _lib.workspace_bytes(ds, _lib.MOE_WS_BACKWARD) + 64 * 256 * 2
    assert call_backward_saved(ds, ok, ok, nb=need - 1) == EWORKSPACE
    assert call_backward_saved(ds, ok, ok, ws=None) == EWORKSPACE
    assert call_backward_saved(ds, ok, ok, ws=P + 8) == EINVAL
    assert call_backward_saved(good_desc(act="f32", wt="f32"), ok, ok) == ENOTSUP
    assert _lib.workspace_bytes(good_desc(act="f32", wt="f32"), _lib.MOE_WS_BACKWARD_SAVED) == 0


def test_router_logits_refusals():
    L, ds = _lib.load(), good_desc()
    need = _lib.workspace_bytes(ds, _lib.MOE_WS_ROUTER_LOGITS)
    assert need == _lib.workspace_bytes(ds, _lib.MOE_WS_ROUTE)
    for i in range(3):
        a = [None if i == j else P for j in range(3)]
        assert L.moe_router_logits(ctypes.byref(ds), *a, P, need, None) == EINVAL
    assert L.moe_router_logits(ctypes.byref(ds), P, P, P, P, need - 1, None) == EWORKSPACE
    assert L.moe_router_logits(ctypes.byref(ds), P + 2, P, P, P, need, None) == EINVAL
    assert L.moe_router_logits(ctypes.byref(ds), P, P, P + 4, P, need, None) == EINVAL
    need = _lib.workspace_bytes(ds, _lib.MOE_WS_ROUTER_GRAD)
    for i in (0, 1, 2, 4, 5):
        a = [None if i == j else P for j in range(6)]
        assert L.moe_router_logits_backward(ctypes.byref(ds), *a, P, need, None) == EINVAL
    assert need > 0
    for i in (0, 2, 5):  # not 16-byte aligned
        a = [P + 4 if i == j else P for j in range(6)]
        assert L.moe_router_logits_backward(ctypes.byref(ds), *a, P, need, None) == EINVAL
    if need:
        assert L.moe_router_logits_backward(ctypes.byref(ds), P, P, P, None, P, P, P, need - 1, None) == EWORKSPACE
    assert L.moe_router_logits_backward(ctypes.byref(good_desc(E=64)), P, P, P, None, P, P, P, need, None) == ENOTSUP


# ---------------------------------------------------------------- the binding's checks

def refused(call, *args, **kw):
    with pytest.raises(_lib.MoeError) as e:
        call(*args, **kw)
    assert e.value.status == EINVAL
    return str(e.value)


def test_binding_checks_types_shapes_and_devices():
    s = _lib.selection(4, 16, 2)
    l, i, w = torch.zeros(4, 16), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    assert "is on cpu" in refused(_lib.moe_select, s, l, None, i, w)
    assert "type" in refused(_lib.moe_select, s, l.double(), None, i, w)
    assert "shape" in refused(_lib.moe_select, s, l[:3], None, i, w)
    assert "strides" in refused(_lib.moe_select, s, torch.zeros(16, 4).t(), None, i, w)
    assert "strides" in refused(_lib.moe_select, s, torch.zeros(16).expand(4, 16), None, i, w)  # rows on top of each other
    assert "missing" in refused(_lib.moe_select, s, None, None, i, w)
    b = torch.zeros(4, 16, dtype=torch.bfloat16)
    assert "type" in refused(_lib.moe_select, s, b, None, i, w)
    x = torch.zeros(3, 200)
    q, c = torch.zeros(3, 200, dtype=torch.uint8), torch.zeros(3, 2, dtype=torch.uint8)
    assert "format" in refused(_lib.moe_checkpoint_pack, x, q, c, "bf16")
    assert "shape" in refused(_lib.moe_checkpoint_unpack, q, c[:, :1].contiguous(), "i8", x)
    assert "type" in refused(_lib.moe_checkpoint_pack, x.double(), q, c, "e4m3")
    assert "matrix" in refused(_lib.moe_checkpoint_pack, x[0], q, c, "e4m3")
    assert "no sequence" in refused(_lib.moe_balance_loss, s, l, i, torch.zeros(1, dtype=torch.int32), 0.1, w, w, w)


def test_binding_checks_come_in_front_of_the_device():
    """meta tensors have a device that is not the GPU: every pointer argument is asked for one."""
    m = dict(device="meta")
    s = _lib.selection(4, 16, 2)
    assert "is on meta" in refused(_lib.moe_select, s, torch.zeros(4, 16, **m), None, torch.zeros(4, 2, dtype=torch.int32, **m),
                                   torch.zeros(4, 2, **m))


def test_binding_checks_saved_activations():
    ds = good_desc(T=4)
    dy, row_of, w = torch.zeros(4, 256), torch.zeros(32, dtype=torch.int32), torch.zeros(4, 8)
    out, dg = torch.zeros(32, 256, dtype=torch.bfloat16), torch.zeros(4, 8)
    q, s = torch.zeros(32, 256, dtype=torch.uint8), torch.zeros(32, 2, dtype=torch.uint8)

    def why(saved):
        return refused(_lib.moe_combine_backward, ds, dy, saved, row_of, w, out, dg)

    assert "is on cpu" in why(_lib.saved(q, s, "e4m3"))
    assert "missing" in why(None)
    assert "codes has shape" in why(_lib.saved(q[:8], s, "i8"))
    assert "scales has shape" in why(_lib.saved(q, s[:, :1].contiguous(), "i8"))
    assert "scales is missing" in why(_lib.saved(q, None, "i8"))
    assert "values has type" in why(_lib.saved(q))
    assert "values has shape" in why(_lib.saved(out[:, :128].contiguous()))
