"""The host code of the microscaled and optimizer calls up to their launches, where there is no
GPU to launch on: workspace layouts, grids and a step's tables over the range of sizes.
Every call gets through its checks and reports that the launch failed."""
import ctypes

import pytest
import torch

from sparse_expert_routing_amd import _lib

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="with a GPU these calls would be launched on addresses that hold nothing")

P = 0x100000
BIG = 1 << 60
EHIP, OK = _lib.MOE_EHIP, _lib.MOE_OK


def mat(fmt):
    return ctypes.byref(_lib.Mx(P, P, fmt))


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1000, 7), (1 << 20, 8192), (1 << 40, 512), (3, 2**31 - 1000)])
def test_packing(rows, cols, kind, fmt):
    L = _lib.load()
    assert L.moe_mx_pack(rows, cols, kind, P, cols, fmt, P, P, None) == EHIP
    assert L.moe_mx_unpack(rows, cols, kind, P, P, fmt, P, cols + 5, None) == EHIP


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("G,M,N,K", [(1, 1, 32, 32), (1, 300, 4096, 4096), (7, 4000, 96, 64), (1024, 1500, 32, 32), (1024, 200000, 2048, 7168),
                                     (1, (1 << 29) - 1, 32, 32), (1024, (1 << 29) - 1, 96, 64), (1, 1, (1 << 21) - 32, 64), (3, 70, 64, (1 << 21) - 32)])
def test_products(G, M, N, K, fmt):
    L = _lib.load()
    w = mat(1)
    g = _lib.MxGroups(G, M, N, K, M, 1)
    few = _lib.MxGroups(G, M, N, K, min(M, 100), 2**31 - 1)
    for out in (0, 1):
        need = L.moe_mx_product_workspace_bytes(ctypes.byref(g), out)
        for src, groups in ((None, g), (P, few)):
            assert L.moe_mx_product(ctypes.byref(groups), mat(fmt), src, P, w, out, P, P, BIG, None) == EHIP
        if need:
            assert L.moe_mx_product(ctypes.byref(g), mat(fmt), None, P, w, out, P, P, need - 1, None) == _lib.MOE_EWORKSPACE
    assert L.moe_mx_ffn_workspace_bytes(ctypes.byref(g), fmt) > M * (N // 2)
    assert L.moe_mx_expert_ffn(ctypes.byref(g), mat(fmt), None, P, w, w, w, P, P, BIG, None) == EHIP


def tensors(kind, sizes):
    w_type, g_type, states, master = kind
    return (_lib.AdamWTensor * max(len(sizes), 1))(
        *[_lib.AdamWTensor(P, P, P, P, P, P, P if master else None, n, w_type, g_type, states) for n in sizes])


KINDS = [(w, g, s, m) for w in (0, 1) for g in (0, 1) for s in (8, 32) for m in ((False, True) if w else (False,))]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("step", [1, 10**12])
def test_steps(kind, step):
    L = _lib.load()
    for beta1, beta2 in ((0.9, 0.999), (0.0, 0.0)):
        rule = _lib.AdamW(1e-3, beta1, beta2, 1e-8, 0.1, step, 2**64 - 1, P, P, P)
        for sizes in ([1], [4096] * 58, [5] * 59, [7] * 60, [4097] * 94, [1 << 22] * 130, [(1 << 35) - 1], [(1 << 35) - 1, 3, (1 << 34) + 5], [0, 0, 9]):
            assert L.moe_adamw(ctypes.byref(rule), tensors(kind, sizes), len(sizes), None) == EHIP
        assert L.moe_adamw(ctypes.byref(rule), tensors(kind, [0] * 300), 300, None) == OK


def test_steps_of_every_kind_at_once():
    L = _lib.load()
    all_kinds = [t for i in range(400) for t in tensors(KINDS[i % len(KINDS)], [i])]
    many = (_lib.AdamWTensor * len(all_kinds))(*all_kinds)
    rule = _lib.AdamW(1e-3, 0.9, 0.999, 1e-8, 0.1, 3, 0, None, None, None)
    assert L.moe_adamw(ctypes.byref(rule), many, len(all_kinds), None) == EHIP
