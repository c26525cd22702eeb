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


@pytest.mark.parametrize("d", [1 << 30, (1 << 31) - 64])
def test_columns_past_the_combine_gradients_index_are_refused(d):
    """Its column index steps past d by up to 2048 before it ends."""
    L, ds, y = _lib.load(), _lib.desc(1, d, 256, 8, 128), _lib.Saved(P, P, 1)
    assert L.moe_combine_backward(ctypes.byref(ds), P, ctypes.byref(y), P, P, P, P, None) == _lib.MOE_ENOTSUP


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_columns_past_the_router_weights_index_are_refused(act):
    """256 rows of 2^23 columns are 2^31 weights."""
    L, ds = _lib.load(), _lib.desc(1, 1 << 23, 256, 8, 128, act, act)
    assert L.moe_router_logits(ctypes.byref(ds), P, P, P, P, 1 << 60, None) == _lib.MOE_ENOTSUP


def test_sizes_past_32_bits_are_refused():
    """A size that the C ABI's 32 bits would cut to a small one (meta tensors: nothing is allocated)."""
    many = (1 << 32) + 8
    m = dict(device="meta")
    x, q = torch.empty(1, many, dtype=torch.bfloat16, **m), torch.empty(1, many, dtype=torch.uint8, **m)
    s = torch.empty(1, -(-many // 128), dtype=torch.uint8, **m)
    sel = _lib.selection(4, 16, 2)
    l, i, off = torch.empty(4, 16, **m), torch.empty(4, 2, dtype=torch.int32, **m), torch.empty(many + 1, dtype=torch.int32, **m)
    load, loss = torch.empty(many, 16, **m), torch.empty(many, **m)
    for call, args in ((_lib.moe_checkpoint_pack, (x, q, s, "e4m3")), (_lib.moe_checkpoint_unpack, (q, s, "e4m3", x)),
                       (_lib.moe_balance_loss, (sel, l, i, off, 0.1, loss, load, None)),
                       (_lib.moe_select_backward, (sel, l, i, None, l, off, load, loss, 0.1))):
        with pytest.raises(_lib.MoeError) as e:
            call(*args)
        assert e.value.status == _lib.MOE_EINVAL and "2^31" in str(e.value), str(e.value)
