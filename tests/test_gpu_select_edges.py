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


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("G,KG", [(1, 1), (32, 32), (32, 31)])
def test_a_large_finite_scale_gives_finite_weights(score, G, KG):
    """scale * (s / sum): the product of the scale and the sum's reciprocal alone may be past fp32."""
    T, E, k, scale = 9, 64, 4, 1e30
    say(f"[select-edges] scale {scale} {score} {KG} of {G}")
    l = -27.0 - torch.rand(T, E, generator=torch.Generator().manual_seed(1))
    for renorm in (True, False):
        _, idx, w = select(l.cuda(), None, k, score=score, n_group=G, topk_group=KG, renorm=renorm, scale=scale)
        ri, rw = plain64.select(f64(l), None, k, score, G, KG, "top2", renorm, scale)
        assert np.array_equal(idx.cpu().numpy(), ri)
        np.testing.assert_allclose(f64(w), rw, rtol=40 * plain64.EPS32)


@pytest.mark.parametrize("score,renorm", [("sigmoid", True), ("sigmoid", False), ("softmax", True), ("softmax", False)])
def test_a_large_finite_scale_gives_finite_gradients(score, renorm):
    """Two chosen experts with scores of about 1e-9 and weight gradients whose product with the scale is past fp32."""
    T, E, k, scale = 5, 64, 8, 1e30
    say(f"[select-edges] gradient with scale {scale} {score} {renorm}")
    g = torch.Generator().manual_seed(3)
    l = torch.randn(T, E, generator=g)
    idx = torch.arange(k, dtype=torch.int32).repeat(T, 1)
    l[:, :2] = -20.0
    dw = torch.zeros(T, k)
    dw[:, :2] = 1e10 * (1 + torch.rand(T, 2, generator=g))
    sel = _lib.selection(T, E, k, score=score, renorm=renorm, scale=scale)
    out = torch.full((T, E), float("nan"), device="cuda")
    _lib.moe_select_backward(sel, l.cuda(), idx.cuda(), dw.cuda(), out)
    ref = plain64.select_grad(f64(l), idx.numpy(), f64(dw), score, renorm, scale)
    assert np.abs(ref).max() < 1e38
    # products and sums of a row's E terms, exps of logits up to 24 below the largest
    size = np.abs(ref).max(axis=1, keepdims=True)
    assert (np.abs(f64(out) - ref) <= 80 * plain64.EPS32 * size).all()


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("G,KG", [(1, 1), (4, 4), (32, 32), (4, 3), (32, 31)])
def test_weights_of_far_logits(G, KG, renorm):
    """Sigmoids of logits down to -32.  Half steps: 2 for the exp, 1 each for the sum and quotient of a score; with
    renormalisation the same for the denominator's, 1 for its sum of two, 1 for the quotient: 10 (4 without)."""
    T, E, k = 4000, 64, 2
    say(f"[select-edges] far logits, {KG} of {G} groups, renorm={renorm}")
    l = -32.0 + 24.0 * torch.rand(T, E, generator=torch.Generator().manual_seed(7))
    _, idx, w = select(l.cuda(), -l.mean(0).cuda(), k, n_group=G, topk_group=KG, renorm=renorm)
    i = idx.cpu().numpy()
    np.testing.assert_allclose(f64(w), plain64.weights(f64(l), i, "sigmoid", renorm, 1.0),
                               rtol=(10 if renorm else 4) * plain64.EPS32, atol=0)


def shares_tolerance(E, span):
    """Half steps of a share p_e / sum p: an exp 4 (span: the rounding of l - m, relative to e^(l-m)), 1 + x 1, its
    reciprocal 2, the same again for the denominator's terms, their sum over E / 16 of a lane and four exchanges, the
    reciprocal of the sum 2 and the product 1."""
    return (14 + 2 * span + E / 16 + 4 + 3) * plain64.EPS32


def span_of(l, score):
    return float((l.amax(1) - l.amin(1)).max()) if score == "softmax" else 0.0


def far_logits(T, E, seed):
    return -32.0 + 14.0 * torch.rand(T, E, generator=torch.Generator().manual_seed(seed))


@pytest.mark.parametrize("E", [16, 13])
def test_balance_loss_of_far_logits(E):
    """One token and one choice per sequence: the loss is alpha E p_e, and shows the share's own error."""
    T = 4000
    say(f"[select-edges] balance loss, far logits E={E}")
    l = far_logits(T, E, E)
    idx = torch.randint(0, E, (T, 1), generator=torch.Generator().manual_seed(2)).to(torch.int32)
    off = torch.arange(T + 1, dtype=torch.int32)
    sel = _lib.selection(T, E, 1)
    loss, load = torch.empty(T, device="cuda"), torch.empty(T, E, device="cuda")
    ws = torch.empty(_lib.balance_workspace_bytes(sel, T), dtype=torch.uint8, device="cuda")
    _lib.moe_balance_loss(sel, l.cuda(), idx.cuda(), off.cuda(), 0.5, loss, load, ws)
    rl, _ = plain64.balance(f64(l), idx.numpy(), off.numpy(), 0.5, "sigmoid")
    np.testing.assert_allclose(f64(loss), rl, rtol=shares_tolerance(E, 0) + plain64.EPS32, atol=0)
