"""Expert choice, its gradient and the balance loss where fp32 is at its edge: crowded keys, far
logits, large scales, gradients that are zero, and bounds in the gradient's own size."""
import numpy as np
import pytest
import torch

from sparse_expert_routing_amd import _lib
from tests import plain64
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    _lib.load()


def f64(t):
    return t.detach().cpu().double().numpy()


def select(l, bias, k, **kw):
    T, E = l.shape
    sel = _lib.selection(T, E, k, logits="bf16" if l.dtype == torch.bfloat16 else "f32", **kw)
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -7.0, device="cuda")
    _lib.moe_select(sel, l, bias, idx, w)
    torch.cuda.synchronize()
    return sel, idx, w


@pytest.mark.parametrize("G,KG,gs", [(1, 1, "max"), (8, 4, "max"), (8, 4, "top2"), (16, 5, "max")], ids=str)
@pytest.mark.parametrize("E", [256, 208])
def test_fewer_distinct_scores_than_choices(E, G, KG, gs):
    """k experts with one fp32 score, and all others a rounding below it in fp32, above it in 64 bits: fewer distinct
    scores than choices, and the ones on top are not the ones chosen."""
    k, T = 8, 40
    say(f"[select-edges] E={E} {G} {KG} {gs}: few distinct scores")
    per = E // G
    high = torch.arange(k) + (100 if G == 1 else 100 // per * per)  # all of them in one group
    g = torch.Generator().manual_seed(E + G)
    l = torch.tensor([16.58, 16.6, 16.62])[torch.randint(0, 3, (T, E), generator=g)]
    l[0] = 16.6
    l[:, high] = 30.0
    bias = torch.full((E,), 8e-8)
    bias[high] = 0.0
    _, idx, _ = select(l.cuda(), bias.cuda(), k, n_group=G, topk_group=KG, group_score=gs)
    ri, _ = plain64.select(f64(l), f64(bias), k, "sigmoid", G, KG, gs)
    assert not np.isin(high.numpy(), ri[0]).all()  # the definition's choice is another one
    assert np.array_equal(idx.cpu().numpy(), ri)
