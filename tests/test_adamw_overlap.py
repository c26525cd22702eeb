"""Tensors of an AdamW step that share memory are refused when the step's table is made (on the
CPU: no step runs)."""
import pytest
import torch

from sparse_expert_routing_amd import _lib


def refusal(*a, **k):
    with pytest.raises(_lib.MoeError) as e:
        _lib.adamw_tensors(*a, **k)
    return str(e.value)


def f(n=300, t=torch.float32):
    return torch.zeros(n, dtype=t)


def test_a_weight_that_is_listed_twice():
    w = f()
    assert "weight 0" in (r := refusal([w, w], [f(), f()], [f(), f()], [f(), f()])) and "weight 1" in r and "overlap" in r
    # views of it, by an element at the end of one
    flat = f(700)
    assert "overlap" in refusal([flat[:300], flat[299:599]], [f(), f()], [f(), f()], [f(), f()])
    assert "overlap" in refusal([flat[10:20], flat], [f(10), f(700)], [f(10), f(700)], [f(10), f(700)])


def test_states_masters_and_gradients():
    m, u8 = f(), torch.uint8
    assert "overlap" in refusal([f(), f()], [f(), f()], [m, m], [f(), f()])
    assert "overlap" in refusal([f()], [f()], [m], [m])
    assert "overlap" in refusal([m], [m], [f()], [f()])  # a gradient that the step would write
    s = torch.zeros(4, dtype=u8)
    assert "overlap" in refusal([f()], [f()], [f(300, u8)], [f(300, u8)], [s[:3]], [s[1:]])
    half = f(300, torch.bfloat16)
    master = f(300)
    assert "overlap" in refusal([half, f(300, torch.bfloat16)], [f(), f()], [f(), f()], [f(), f()], masters=[master, master])
    long = f(600)
    assert "overlap" in refusal([f(300), f(20)], [long[:300], f(20)], [f(300), f(20)], [f(300), long[290:310]])


def test_what_lies_side_by_side_and_shared_gradients_are_taken():
    """As far as the check of the device, which is the last."""
    flat, g = f(4 * 257), f(257)
    cut = flat.split(257)
    assert "cpu" in refusal([cut[0], cut[2]], [g, g], [cut[1], f(257)], [cut[3], f(257)])
    e = f(0)
    assert "cpu" in refusal([e, e], [e, e], [e, e], [e, e])
    flat = f(900)  # a gradient may hold another's
    assert "cpu" in refusal([f(900), f(100)], [flat, flat[100:200]], [f(900), f(100)], [f(900), f(100)])
