"""Packing and products of no rows: a shard that no token chose.  Nothing is launched."""
import pytest
import torch

from sparse_expert_routing_amd import _lib


@pytest.fixture(params=["cpu", pytest.param("cuda", marks=pytest.mark.gpu)])
def where(request, monkeypatch):
    if request.param == "cpu":  # tensors in host memory count as lying on a GPU
        monkeypatch.setattr(_lib._Call, "on", lambda self, name, t: setattr(self, "index", 0))
    return request.param


def weights(G, N, K, where):
    codes, scales = _lib.mx_empty(G * N, K, "e2m1", where)
    return _lib.mx(codes.view(G, N, K // 2), scales, "e2m1")


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_packing(where, fmt):
    for t in (torch.float32, torch.bfloat16):
        x = torch.zeros(0, 100, dtype=t, device=where)
        codes, scales = _lib.mx_empty(0, 100, fmt, where)
        _lib.moe_mx_pack(x, codes, scales, fmt)
        _lib.moe_mx_unpack(codes, scales, fmt, x)
        with pytest.raises(_lib.MoeError):
            _lib.moe_mx_pack(x, codes, scales[:, :, :3], fmt)
        with pytest.raises(_lib.MoeError):
            _lib.moe_mx_unpack(codes, scales, fmt, x[:, :97])


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_products(where, fmt):
    G, N, K = 3, 64, 96
    new = dict(device=where)
    x, some = (_lib.mx(*_lib.mx_empty(rows, K, fmt, where), fmt) for rows in (0, 5))
    w, down = weights(G, N, K, where), weights(G, K, N, where)
    off, out = torch.zeros(G + 1, dtype=torch.int32, **new), torch.zeros(0, N, **new)
    y, src = torch.zeros(0, K, dtype=torch.bfloat16, **new), torch.zeros(0, dtype=torch.int32, **new)
    ws = torch.empty(_lib.mx_ffn_workspace_bytes(G, 0, K, N, fmt), dtype=torch.uint8, **new)
    _lib.moe_mx_product(x, w, off, out)
    _lib.moe_mx_product(x, w, off, out, ws, src, 2)
    _lib.moe_mx_product(some, w, off, out, ws, src, 2)  # a shard that none of the tokens chose
    _lib.moe_mx_expert_ffn(x, w, w, down, off, y, ws)
    _lib.moe_mx_expert_ffn(some, w, w, down, off, y, ws, src, 2)
    for bad in (lambda: _lib.moe_mx_product(some, w, off, out), lambda: _lib.moe_mx_product(x, w, off, out, None, src, 0),
                lambda: _lib.moe_mx_product(x, w, off[:-1], out), lambda: _lib.moe_mx_product(x, w, off, out, None, off, 1),
                lambda: _lib.moe_mx_expert_ffn(some, w, w, down, off, y, ws), lambda: _lib.moe_mx_expert_ffn(x, w, w, w, off, y, ws)):
        with pytest.raises(_lib.MoeError):
            bad()
    if where == "cuda":
        host = torch.zeros(0, N)
        with pytest.raises(_lib.MoeError):
            _lib.moe_mx_product(x, w, off, host)
