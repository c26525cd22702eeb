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


def balance_grad_bound(l, off, load, dloss, alpha, score):
    """What the balance gradient's elements may be off by: each is p'_e (f_e - sum_i f_i p'_i), times 1 - s_e for a
    sigmoid, with p' the shares and f = alpha dloss (load - 1) / n: relative to the shares' errors and a few
    roundings of each term, so to p'_e (|f_e| + sum |f| p')."""
    T, E = l.shape
    p = plain64.shares(f64(l), score)
    rest = plain64.sigmoid(-f64(l)) if score == "sigmoid" else 1.0
    size = np.zeros((T, E))
    for q, (a, b) in enumerate(zip(off[:-1], off[1:])):
        if b > a:
            f = np.abs(alpha * dloss[q] * (load[q] - 1.0) / (b - a))
            size[a:b] = f + (p[a:b] * f).sum(1, keepdims=True)
    # two shares in a row (p' and the one inside the sum), the sum's E / 16 + 4 additions, f's 3 roundings and the
    # difference, product and 1 - s (7) behind them
    c = 2 * shares_tolerance(E, span_of(l, score)) + (E / 16 + 4 + 12) * plain64.EPS32
    return c * p * rest * size + 1e-37


BALANCE = [(300, 256, 8, "sigmoid", "f32", 5), (1000, 60, 4, "softmax", "bf16", 9), (1000, 64, 6, "softmax", "f32", 200),
           (200, 1000, 20, "sigmoid", "bf16", 3), (5000, 256, 8, "sigmoid", "f32", 2), (4096, 8, 2, "softmax", "f32", 1),
           (64, 17, 3, "sigmoid", "f32", 64), (501, 255, 8, "sigmoid", "f32", 4)]


def sequences(T, n, seed):
    cuts = torch.randint(0, T + 1, (n - 1,), generator=torch.Generator().manual_seed(seed)).sort().values
    return torch.cat([torch.tensor([0]), cuts, torch.tensor([T])]).to(torch.int32)


def balance_case(T, E, k, score, dtype, n):
    g = torch.Generator().manual_seed(T + E)
    l = (1.5 * torch.randn(T, E, generator=g)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    idx = torch.rand(T, E, generator=g).topk(k, dim=1).indices.sort(dim=1).values.to(torch.int32)
    sel = _lib.selection(T, E, k, score=score, logits=dtype)
    off = sequences(T, n, n)
    loss, load = torch.empty(n, device="cuda"), torch.empty(n, E, device="cuda")
    ws = torch.empty(_lib.balance_workspace_bytes(sel, n), dtype=torch.uint8, device="cuda")
    _lib.moe_balance_loss(sel, l.cuda(), idx.cuda(), off.cuda(), 0.5, loss, load, ws)
    return l, idx, sel, off, load, torch.rand(n, generator=g) + 0.5


def check_balance_grad(l, got, off, load, dloss, alpha, score):
    ref = plain64.select_grad(f64(l), None, None, score, True, 1.0, off.numpy(), f64(load), f64(dloss), alpha)
    bound = balance_grad_bound(l, off.numpy(), f64(load), f64(dloss), alpha, score)
    # a gradient of zeros would be found at nearly every element
    inside = np.abs(ref) > 0
    assert not inside.any() or (np.abs(ref) > bound)[inside].mean() > 0.95
    assert (np.abs(got - ref) <= bound).all()


@pytest.mark.parametrize("T,E,k,score,dtype,n", BALANCE)
def test_balance_gradient_in_its_own_size(T, E, k, score, dtype, n):
    say(f"[select-edges] balance gradient T={T} E={E} {score} {dtype} n_seq={n}")
    l, idx, sel, off, load, dloss = balance_case(T, E, k, score, dtype, n)
    out = torch.full((T, E), float("nan"), device="cuda")
    _lib.moe_select_backward(sel, l.cuda(), None, None, out, off.cuda(), load, dloss.cuda(), 0.5)
    check_balance_grad(l, f64(out), off, load, dloss, 0.5, score)


@pytest.mark.parametrize("E", [64, 61])
def test_balance_gradient_of_far_logits(E):
    say(f"[select-edges] balance gradient, far logits E={E}")
    T, n = 700, 3
    l, off = far_logits(T, E, E), sequences(T, n, 5)
    sel = _lib.selection(T, E, 4)
    load = 2 * torch.rand(n, E, generator=torch.Generator().manual_seed(1))
    dloss = torch.ones(n)
    out = torch.full((T, E), float("nan"), device="cuda")
    _lib.moe_select_backward(sel, l.cuda(), None, None, out, off.cuda(), load.cuda(), dloss.cuda(), 0.5)
    check_balance_grad(l, f64(out), off, load, dloss, 0.5, "sigmoid")


@pytest.mark.parametrize("T,E,k,score,dtype,n", BALANCE)
def test_balance_gradient_beside_the_weights(T, E, k, score, dtype, n):
    """Both gradients in one call are the sum of each alone: the balance share, which may be far below the weights',
    is found where no expert is chosen, and to one rounding of the sum where one is."""
    say(f"[select-edges] both gradients T={T} E={E} {score} {dtype} n_seq={n}")
    l, idx, sel, off, load, dloss = balance_case(T, E, k, score, dtype, n)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(9)).cuda()
    seq = dict(seq_offsets=off.cuda(), load=load, dloss=dloss.cuda(), alpha=0.5)
    outs = [torch.full((T, E), float("nan"), device="cuda") for _ in range(3)]
    for out, d, kw in zip(outs, (dw, None, dw), (seq, seq, {})):
        _lib.moe_select_backward(sel, l.cuda(), idx.cuda() if d is not None else None, d, out, **kw)
    both, loss, weights = (f64(o) for o in outs)
    assert (loss != 0).mean() > 0.9
    # renormalised weights: zero but for the chosen
    assert (np.abs(both - (loss + weights)) <= 2 * plain64.EPS32 * (np.abs(loss) + np.abs(weights))).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_gradients_that_are_zero_by_definition(score):
    """One renormalised choice has the weight `scale` whatever its logit; where every expert is chosen, every load is
    1 and the loss alpha sum p' = alpha: no gradient, and none of the formula's roundings in its place."""
    say(f"[select-edges] zero gradients {score}")
    T, E = 133, 40
    g = torch.Generator().manual_seed(4)
    for seed in range(2):
        l = torch.randn(T, E, generator=g).cuda()
        sel, idx, w = select(l, None, 1, score=score, scale=2.5)
        assert (w == 2.5).all()
        out = torch.full((T, E), float("nan"), device="cuda")
        _lib.moe_select_backward(sel, l, idx, torch.randn(T, 1, generator=g).cuda(), out)
        assert (out == 0).all()
        sel = _lib.selection(T, E, E, score=score)
        idx = torch.arange(E, dtype=torch.int32).repeat(T, 1).cuda()
        off = torch.tensor([0, 50, T], dtype=torch.int32, device="cuda")
        loss, load = torch.empty(2, device="cuda"), torch.empty(2, E, device="cuda")
        ws = torch.empty(_lib.balance_workspace_bytes(sel, 2), dtype=torch.uint8, device="cuda")
        _lib.moe_balance_loss(sel, l, idx, off, 0.25, loss, load, ws)
        assert (load == 1).all()
        np.testing.assert_allclose(f64(loss), 0.25, rtol=shares_tolerance(E, 10) + plain64.EPS32)
        _lib.moe_select_backward(sel, l, None, None, out.fill_(float("nan")), off, load, torch.ones(2, device="cuda"), 0.25)
        assert (out == 0).all()


def test_more_tokens_than_one_launch_of_waves():
    """A wave per token, 64 threads: 2^26 tokens and more in several launches, the last tokens as a call of their own."""
    T, E, k, n = (1 << 26) + 7, 34, 2, 300
    say(f"[select-edges] T={T} E={E}")
    l = torch.empty(T, E, dtype=torch.bfloat16, device="cuda").normal_()
    bias = torch.linspace(-0.05, 0.05, E).cuda()
    kw = dict(n_group=17, topk_group=16)
    _, idx, w = select(l, bias, k, **kw)
    for part in (slice(0, n), slice((1 << 25) - n, (1 << 25) + n), slice(T - n, T)):
        _, fi, fw = select(l[part].clone(), bias, k, **kw)
        assert torch.equal(idx[part], fi) and torch.equal(w[part], fw)
    ri, _ = plain64.select(f64(l[-n:]), f64(bias), k, "sigmoid", 17, 16)
    assert np.array_equal(idx[-n:].cpu().numpy(), ri)
