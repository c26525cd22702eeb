"""Numbers past the C ABI's integers are refused by the binding, where they would be cut to
small ones (on the CPU: nothing is launched)."""
import pytest
import torch

from sparse_expert_routing_amd import _lib


def refusal(call, *a, **k):
    with pytest.raises(_lib.MoeError) as e:
        call(*a, **k)
    assert e.value.status == _lib.MOE_EINVAL
    return str(e.value)


@pytest.mark.parametrize("k", [0, -1, 1 << 31, (1 << 32) + 1, 1 - (1 << 32)])
def test_k(k):
    codes, scales = _lib.mx_empty(3 * 64, 96, "e2m1", "cpu")
    w = _lib.mx(codes.view(3, 64, 48), scales, "e2m1")
    down_codes, down_scales = _lib.mx_empty(3 * 96, 64, "e2m1", "cpu")
    down = _lib.mx(down_codes.view(3, 96, 32), down_scales, "e2m1")
    x = _lib.mx(*_lib.mx_empty(10, 96, "e4m3", "cpu"), "e4m3")
    off, src = torch.zeros(4, dtype=torch.int32), torch.zeros(10, dtype=torch.int32)
    assert "k," in refusal(_lib.moe_mx_product, x, w, off, torch.zeros(10, 64), None, src, k)
    assert "k," in refusal(_lib.moe_mx_expert_ffn, x, w, w, down, off, torch.zeros(10, 96, dtype=torch.bfloat16), None, src, k)


@pytest.mark.parametrize("step", [0, -3, 1 << 63, (1 << 64) + 1, 1 - (1 << 64)])
def test_step(step):
    one = _lib.AdamWTensors((_lib.AdamWTensor * 1)(), 0, [])
    assert "step," in refusal(_lib.moe_adamw, one, 1e-3, step=step)


def test_workspaces():
    far = 1 << 32
    sizes = (4, 5000, 512, 128)
    assert _lib.mx_product_workspace_bytes(*sizes) > 0 and _lib.mx_ffn_workspace_bytes(*sizes, "e4m3") > 0
    for i in range(4):
        more = [n + far * (i == j) for j, n in enumerate(sizes)]
        assert _lib.mx_product_workspace_bytes(*more) == 0 and _lib.mx_ffn_workspace_bytes(*more, "e4m3") == 0
