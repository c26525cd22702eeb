"""Refusals at the edges of the routing-from-logits entry points' ranges, on the CPU."""
import ctypes

import pytest
import torch

from sparse_expert_routing_amd import _lib


def test_a_loss_gradient_without_its_sequences_is_refused():
    """load or dloss without seq_offsets: the gradient of the loss would be left out in silence."""
    T, E, k = 4, 16, 2
    s = _lib.selection(T, E, k)
    l, i, w, out = torch.zeros(T, E), torch.zeros(T, k, dtype=torch.int32), torch.zeros(T, k), torch.zeros(T, E)
    for kw in (dict(dloss=torch.ones(1)), dict(load=torch.ones(1, E)), dict(load=torch.ones(1, E), dloss=torch.ones(1))):
        with pytest.raises(_lib.MoeError) as e:
            _lib.moe_select_backward(s, l, i, w, out, alpha=0.1, **kw)
        assert e.value.status == _lib.MOE_EINVAL and "seq_offsets" in str(e.value)


P = 0x1000  # an address that no call gets to read


@pytest.mark.parametrize("T", [1 << 28, (1 << 31) - 64, (1 << 31) - 1])
def test_more_tokens_than_a_launch_takes_are_refused(T):
    """A launch has fewer than 2^32 threads and a token up to sixteen."""
    L, r = _lib.load(), ctypes.byref(_lib.selection(T, 4, 1))
    assert L.moe_select(r, P, 4, P, P, P, None) == _lib.MOE_ENOTSUP
    assert L.moe_select_backward(r, P, 4, P, P, None, 0, None, None, 0.0, P, None) == _lib.MOE_ENOTSUP
    assert L.moe_balance_loss(r, P, 4, P, P, 1, 0.1, P, P, P, 1 << 60, None) == _lib.MOE_ENOTSUP
    assert L.moe_balance_workspace_bytes(r, 1) == 0


def test_the_largest_balance_workspace():
    L, T, E, n = _lib.load(), (1 << 28) - 1, 4, (1 << 22) - 1
    r = ctypes.byref(_lib.selection(T, E, 1))
    for n_seq in (1, n):
        need = (-(-T // 64) + n_seq) * E * 8  # a partial share and a count per expert and slot
        assert need <= L.moe_balance_workspace_bytes(r, n_seq) < need + 256
        assert L.moe_balance_loss(r, P, 4, P, P, n_seq, 0.1, P, P, P, need - 1, None) == _lib.MOE_EWORKSPACE
    assert L.moe_balance_workspace_bytes(r, n + 1) == 0
    assert L.moe_balance_loss(r, P, 4, P, P, n + 1, 0.1, P, P, P, 1 << 60, None) == _lib.MOE_ENOTSUP


@pytest.mark.parametrize("T,d", [(1 << 26, 64), ((1 << 28) - 1, 1024), (1 << 24, 2048)])
def test_more_tokens_than_the_combines_gradient_takes_are_refused(T, d):
    """A wave of 64 threads per token, four from 2048 columns on, and fewer than 2^32 threads to a launch."""
    L, ds, y = _lib.load(), _lib.desc(T, d, 256, 8, 128), _lib.Saved(P, P, 1)
    assert L.moe_combine_backward(ctypes.byref(ds), P, ctypes.byref(y), P, P, P, P, None) == _lib.MOE_ENOTSUP
