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
