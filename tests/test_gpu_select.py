"""Expert choice from logits, its gradient and the sequence-wise balance loss on the
GPU against their definitions in 64 bits: ids exactly, weights and gradients to
a few fp32 roundings.

Tolerances (half a step of fp32, EPS32 = 2^-24): a score is off by its exp (2), the
subtraction or negation before it (the logits' range, absolutely), one addition
and one division, a share by a sum of up to E terms over 64 lanes (E/64 + 6) and
one more division; so 32 + E/64 + range half steps hold with room."""
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


def logits_of(T, E, dtype, seed, std=1.5):
    g = torch.Generator().manual_seed(seed)
    l = std * torch.randn(T, E, generator=g)
    return l.to(torch.bfloat16 if dtype == "bf16" else torch.float32)


def f64(t):
    return t.detach().cpu().double().numpy()


def run_select(l, bias, **kw):
    T, E = l.shape
    k = kw.pop("k")
    sel = _lib.selection(T, E, k, logits="bf16" if l.dtype == torch.bfloat16 else "f32", **kw)
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -7.0, device="cuda")
    _lib.moe_select(sel, l, bias, idx, w)
    torch.cuda.synchronize()
    return sel, idx, w


def rtol(l, E):
    finite = l[torch.isfinite(l)].float()
    span = float(finite.max() - finite.min()) if finite.numel() else 0.0
    return plain64.EPS32 * (32 + E / 64 + min(span, 200.0))


RULES = [
    # T, E, k, score, n_group, topk_group, group_score, renorm, scale, bias, dtype
    (1, 256, 8, "sigmoid", 8, 4, "top2", True, 2.5, True, "f32"),
    (33, 256, 8, "sigmoid", 1, 1, "max", True, 1.0, True, "f32"),
    (517, 256, 8, "sigmoid", 8, 4, "top2", True, 2.5, True, "f32"),
    (130, 256, 8, "sigmoid", 8, 4, "max", True, 1.0, False, "bf16"),
    (64, 256, 8, "softmax", 8, 3, "max", False, 16.0, False, "f32"),
    (77, 160, 6, "softmax", 8, 3, "max", False, 16.0, False, "bf16"),
    (301, 60, 4, "softmax", 1, 1, "max", False, 1.0, False, "bf16"),
    (301, 64, 6, "softmax", 1, 1, "max", True, 1.0, True, "f32"),
    (40, 7, 3, "sigmoid", 7, 5, "max", True, 1.0, True, "f32"),
    (40, 7, 5, "sigmoid", 7, 5, "top2", True, 1.0, True, "f32"),
    (21, 66, 9, "sigmoid", 6, 2, "top2", False, 1.0, False, "f32"),
    (21, 1, 1, "softmax", 1, 1, "max", True, 1.0, False, "f32"),
    (5, 2, 2, "sigmoid", 2, 2, "max", True, 1.0, True, "bf16"),
    (50, 512, 16, "sigmoid", 16, 4, "top2", True, 1.0, True, "f32"),
    (50, 500, 16, "softmax", 4, 2, "top2", True, 1.0, True, "bf16"),
    (20, 1024, 64, "sigmoid", 32, 7, "top2", True, 1.0, True, "f32"),
    (20, 1023, 33, "softmax", 1, 1, "max", False, 1.0, True, "f32"),
    (20, 768, 64, "softmax", 3, 1, "max", True, 1.0, False, "f32"),
    (9, 128, 64, "sigmoid", 2, 1, "max", True, 1.0, False, "f32"),
]


@pytest.mark.parametrize("rule", RULES, ids=lambda r: "-".join(map(str, r)))
def test_select_matches_the_definition(rule):
    T, E, k, score, G, KG, gs, renorm, scale, biased, dtype = rule
    say(f"[select] {rule}")
    l = logits_of(T, E, dtype, seed=T * 31 + E).cuda()
    bias = (0.2 * torch.rand(E, generator=torch.Generator().manual_seed(E)) - 0.1).cuda() if biased else None
    _, idx, w = run_select(l, bias, k=k, score=score, n_group=G, topk_group=KG, group_score=gs, renorm=renorm, scale=scale)
    ri, rw = plain64.select(f64(l), f64(bias) if biased else None, k, score, G, KG, gs, renorm, scale)
    assert np.array_equal(idx.cpu().numpy(), ri)
    np.testing.assert_allclose(f64(w), rw, rtol=rtol(l, E), atol=1e-38)


def test_select_large_batch_of_the_layers_rule():
    """Every token of a prefill-sized batch, with the balancing bias: the border decides 64-bit scores."""
    T, E = 16384, 256
    say(f"[select] T={T} E={E}: whole batch")
    l = logits_of(T, E, "f32", 5).cuda()
    bias = (0.1 * torch.rand(E, generator=torch.Generator().manual_seed(3)) - 0.05).cuda()
    _, idx, w = run_select(l, bias, k=8, n_group=8, topk_group=4, scale=2.5)
    p = torch.sigmoid(l.double()) + bias.double()
    g = p.view(T, 8, 32).topk(2, dim=2).values.sum(2)
    best = g.sort(dim=1, descending=True, stable=True).indices[:, :4]
    shut = torch.ones(T, 8, dtype=torch.bool, device="cuda").scatter_(1, best, False).repeat_interleave(32, dim=1)
    ref = p.masked_fill(shut, -9.0).sort(dim=1, descending=True, stable=True).indices[:, :8].sort(dim=1).values
    assert torch.equal(idx.long(), ref)
    assert torch.allclose(w.sum(dim=1), torch.full((T,), 2.5, device="cuda"), rtol=1e-6)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups", [(1, 1, "max"), (8, 3, "max"), (8, 3, "top2")], ids=str)
@pytest.mark.parametrize("biased", [False, True])
def test_select_near_the_border(score, groups, biased):
    """Scores that differ by less than fp32 keeps of them, exact ties, signed zeros, and the two together."""
    T, E, k = 64, 256, 8
    say(f"[select] border {score} {groups} bias={biased}")
    g = torch.Generator().manual_seed(11)
    l = torch.zeros(T, E)
    l[0:16] = 1.0 + 1e-7 * torch.randint(-3, 4, (16, E), generator=g)  # neighbouring floats
    l[16:32] = torch.randint(0, 3, (16, E), generator=g).float()       # many exact ties
    l[32:40] = torch.where(torch.rand(8, E, generator=g) < 0.5, -0.0, 0.0)
    l[40:48] = 8.0 + 1e-6 * torch.randint(-3, 4, (8, E), generator=g)  # a flat sigmoid
    l[48:64] = logits_of(16, E, "bf16", 4).float()
    bias = None
    if biased:  # neighbouring biases, many of them equal
        bias = (0.01 + 1e-9 * torch.randint(0, 5, (E,), generator=g)).float()
    G, KG, gs = groups
    lc, bc = l.cuda(), bias.cuda() if biased else None
    _, idx, w = run_select(lc, bc, k=k, score=score, n_group=G, topk_group=KG, group_score=gs)
    ri, rw = plain64.select(l.double().numpy(), f64(bias) if biased else None, k, score, G, KG, gs)
    got = idx.cpu().numpy()
    if score == "sigmoid" or (gs == "max" and not biased):
        assert np.array_equal(got, ri)
    else:
        # a softmax's 64-bit denominator depends on the order of its sum (2^-53 of it): the choices'
        # total may differ by that much and by no more
        a = plain64.scores(l.double().numpy(), score) + (f64(bias) if biased else 0.0)
        for t in range(T):
            assert len(set(got[t])) == k
            assert abs(a[t][got[t]].sum() - a[t][ri[t]].sum()) <= 256 * 2.0**-53 * np.abs(a[t]).sum()
    np.testing.assert_allclose(f64(w), plain64.weights(l.double().numpy(), got, score, True, 1.0), rtol=rtol(l, E))


@pytest.mark.parametrize("E,k,G,KG,gs", [(256, 8, 1, 1, "max"), (256, 8, 8, 4, "top2"), (150, 6, 3, 2, "max"),
                                         (165, 9, 5, 2, "top2"), (496, 12, 16, 5, "top2"), (500, 8, 2, 1, "top2"),
                                         (16, 5, 16, 7, "top2"), (64, 64, 4, 4, "max"), (510, 3, 3, 1, "max"),
                                         (600, 8, 4, 3, "max"), (68, 7, 17, 5, "top2")], ids=str)
@pytest.mark.parametrize("std", [1.0, 1e-2, 1e-4])
def test_select_crowded_scores(E, k, G, KG, gs, std):
    """The narrower the scores, the more tokens have a border that only 64 bits decide, of experts and of groups."""
    T = 300
    say(f"[select] crowded E={E} k={k} groups {KG} of {G} {gs} std={std}")
    for dtype in ("f32", "bf16"):
        l = logits_of(T, E, dtype, E + k, std=std)
        bias = 0.05 * std * torch.randn(E, generator=torch.Generator().manual_seed(k))
        for b in (bias, torch.zeros(E), None):
            _, idx, w = run_select(l.cuda(), b.cuda() if b is not None else None, k=k, n_group=G, topk_group=KG,
                                   group_score=gs)
            ri, rw = plain64.select(f64(l), f64(b) if b is not None else None, k, "sigmoid", G, KG, gs)
            assert np.array_equal(idx.cpu().numpy(), ri), (dtype, b is None)
            np.testing.assert_allclose(f64(w), rw, rtol=rtol(l, E))


def test_select_special_rows():
    """Masked logits (-inf, the type's lowest), NaN, infinities: ids stay distinct and in range, as documented."""
    E, k = 256, 8
    inf, nan, low = float("inf"), float("nan"), torch.finfo(torch.float32).min
    l = logits_of(10, E, "f32", 8)
    l[0] = -inf
    l[1, :] = -inf
    l[1, 200:204] = 1.0          # fewer than k left
    l[2] = low
    l[3, 7:] = nan               # seven numbers
    l[4] = nan
    l[5, 100] = inf
    l[6, 0:255] = -inf
    l[7, 5] = nan
    l[8] = -200.0                # every sigmoid underflows in fp32
    l[9] = 500.0
    bias = (0.2 * torch.rand(E, generator=torch.Generator().manual_seed(1)) - 0.1)
    for score in ("sigmoid", "softmax"):
        for G, KG, gs in ((1, 1, "max"), (8, 4, "max"), (8, 4, "top2")):
            for b in (None, bias):
                say(f"[select] special rows {score} {G} {KG} {gs} bias={b is not None}")
                _, idx, w = run_select(l.cuda(), b.cuda() if b is not None else None, k=k, score=score, n_group=G,
                                       topk_group=KG, group_score=gs)
                i = idx.cpu().numpy()
                assert ((i >= 0) & (i < E)).all() and all(len(set(r)) == k for r in i)
                assert (np.diff(i, axis=1) > 0).all()
                rows = [0, 1, 2, 6, 8, 9] + ([5] if score == "sigmoid" else [])
                if score == "sigmoid":
                    rows += [3, 4, 7]
                with np.errstate(all="ignore"):
                    ri, rw = plain64.select(l[rows].double().numpy(), f64(b) if b is not None else None, k, score, G, KG,
                                            gs)
                if score == "sigmoid" or b is None and gs == "max":
                    assert np.array_equal(i[rows], ri)
                got = f64(w)
                assert np.isfinite(got[[0, 1, 2, 6, 8, 9]]).all()
                if score == "sigmoid":
                    assert (got[0] == 0).all() and (got[8] == 0).all()  # no score at all: weight 0


def test_select_past_32_bit_offsets():
    """More than 2^31 logits: the last tokens as a call of their own has them, their gradient and their loss too."""
    T, E, k, n = 8_400_003, 256, 2, 500
    say(f"[select] T={T} E={E}")
    l = torch.empty(T, E, dtype=torch.bfloat16, device="cuda").normal_()
    bias = (0.1 * torch.rand(E, generator=torch.Generator().manual_seed(1)) - 0.05).cuda()
    sel, idx, w = run_select(l, bias, k=k)
    few, fi, fw = run_select(l[-n:].clone(), bias, k=k)
    assert torch.equal(idx[-n:], fi) and torch.equal(w[-n:], fw)
    ri, _ = plain64.select(f64(l[-n:]), f64(bias), k, "sigmoid")
    assert np.array_equal(fi.cpu().numpy(), ri)
    off = torch.tensor([T - n, T], dtype=torch.int32, device="cuda")
    loss, load = torch.empty(1, device="cuda"), torch.empty(1, E, device="cuda")
    ws = torch.empty(_lib.balance_workspace_bytes(sel, 1), dtype=torch.uint8, device="cuda")
    _lib.moe_balance_loss(sel, l, idx, off, 0.5, loss, load, ws)
    rl, rf = plain64.balance(f64(l[-n:]), ri, [0, n], 0.5, "sigmoid")
    np.testing.assert_allclose(f64(loss), rl, rtol=1e-5)
    np.testing.assert_allclose(f64(load), rf, rtol=1e-6)
    dw = torch.randn(T, k, device="cuda")
    out = torch.empty(T, E, device="cuda")
    _lib.moe_select_backward(sel, l, idx, dw, out, off, load, torch.ones(1, device="cuda"), 0.5)
    ref = plain64.select_grad(f64(l[-n:]), ri, f64(dw[-n:]), "sigmoid", True, 1.0, [0, n], f64(load), np.ones(1), 0.5)
    assert np.abs(f64(out[-n:]) - ref).max() <= 2 * rtol(l[-n:], E) * float(dw[-n:].abs().max() + 1)


def test_select_unaligned_inputs():
    """Logits, bias and gradients that begin at any element."""
    T, E, k = 70, 128, 6
    say("[select] unaligned")
    for dtype in ("f32", "bf16"):
        flat = logits_of(1, T * E + 1, dtype, 5).cuda().view(-1)
        b = (0.1 * torch.rand(E + 1, generator=torch.Generator().manual_seed(2))).cuda()[1:]
        l = flat[1:].view(T, E)
        _, idx, w = run_select(l, b, k=k, n_group=4, topk_group=2)
        ri, rw = plain64.select(f64(l), f64(b), k, "sigmoid", 4, 2)
        assert np.array_equal(idx.cpu().numpy(), ri)
        np.testing.assert_allclose(f64(w), rw, rtol=rtol(l, E))
        sel = _lib.selection(T, E, k, logits=dtype)
        out = torch.empty(T * E + 1, device="cuda")[1:].view(T, E)
        dw = torch.randn(T * k + 1, device="cuda")[1:].view(T, k)
        off = torch.tensor([0, 0, 50], dtype=torch.int32, device="cuda")[1:]
        load = torch.rand(E + 1, device="cuda")[1:].view(1, E)
        _lib.moe_select_backward(sel, l, idx, dw, out, off, load, torch.ones(1, device="cuda"), 0.1)
        ref = plain64.select_grad(f64(l), ri, f64(dw), "sigmoid", True, 1.0, [0, 50], f64(load), np.ones(1), 0.1)
        assert np.abs(f64(out) - ref).max() <= 2 * rtol(l, E) * float(dw.abs().max() + 1)


def test_select_strided_rows_and_neighbours():
    T, E, k = 37, 200, 5
    say("[select] strided logits")
    wide = logits_of(T, 333, "bf16", 2).cuda()
    l = wide[:, 60:260]
    out = torch.full((T + 2, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 2, k), -7.0, device="cuda")
    sel = _lib.selection(T, E, k, logits="bf16")
    _lib.moe_select(sel, l, None, out[1:-1], w[1:-1])
    torch.cuda.synchronize()
    ri, rw = plain64.select(f64(l), None, k, "sigmoid")
    assert np.array_equal(out[1:-1].cpu().numpy(), ri)
    np.testing.assert_allclose(f64(w[1:-1]), rw, rtol=rtol(l, E))
    assert (out[[0, -1]] == -7).all() and (w[[0, -1]] == -7).all()


def test_select_agrees_with_the_layers_router():
    """Logits from moe_router_logits, ungrouped biased sigmoid choice: moe_route's ids and weights."""
    for T, d, act in ((300, 512, "bf16"), (2000, 1024, "bf16"), (33, 256, "f32")):
        say(f"[select] router logits T={T} d={d} {act}")
        g = torch.Generator().manual_seed(T)
        x = torch.randn(T, d, generator=g)
        x = (x.bfloat16() if act == "bf16" else x).cuda()
        wr = (torch.randn(256, d, generator=g) * d**-0.5).cuda()
        bias = (0.1 * torch.rand(256, generator=g) - 0.05).cuda()
        ds = _lib.desc(T, d, 256, 8, 128, act, act)
        ws = torch.empty(max(1, _lib.workspace_bytes(ds, _lib.MOE_WS_ROUTER_LOGITS)), dtype=torch.uint8, device="cuda")
        logits = torch.empty(T, 256, device="cuda")
        _lib.moe_router_logits(ds, x, wr, logits, ws)
        ref = f64(x) @ f64(wr).T
        # d fp32 additions of products |x| |w|
        bound = (d / 512 + 512) * 2 * plain64.EPS32 * (np.abs(f64(x)) @ np.abs(f64(wr)).T)
        assert (np.abs(f64(logits) - ref) <= bound).all()
        idx = torch.empty(T, 8, dtype=torch.int32, device="cuda")
        w, gap = torch.empty(T, 8, device="cuda"), torch.empty(T, device="cuda")
        _lib.moe_route(ds, x, wr, bias, idx, w, gap, ws)
        _, i2, w2 = run_select(logits, bias, k=8)
        clear = gap > 1e-6
        assert torch.equal(idx[clear], i2[clear]) and int(clear.sum()) > 0.99 * T
        assert torch.allclose(w[clear], w2[clear], rtol=1e-5)


# ---------------------------------------------------------------- gradients

def seqs(T, n, seed, first=0, last=None):
    g = torch.Generator().manual_seed(seed)
    last = T if last is None else last
    cuts = torch.randint(first, last + 1, (n - 1,), generator=g).sort().values if n > 1 else torch.empty(0, dtype=torch.long)
    return torch.cat([torch.tensor([first]), cuts, torch.tensor([last])]).to(torch.int32)


def ids_of(T, E, k, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.rand(T, E, generator=g).topk(k, dim=1).indices.sort(dim=1).values.to(torch.int32)


GRADS = [
    # T, E, k, score, renorm, scale, dtype, weights, sequences
    (1, 256, 8, "sigmoid", True, 2.5, "f32", True, 0),
    (300, 256, 8, "sigmoid", True, 2.5, "f32", True, 3),
    (300, 256, 8, "sigmoid", False, 1.0, "bf16", True, 0),
    (300, 60, 4, "softmax", False, 1.0, "bf16", True, 0),
    (300, 60, 4, "softmax", True, 1.0, "f32", True, 5),
    (301, 64, 6, "softmax", False, 2.0, "f32", True, 70),
    (300, 256, 8, "sigmoid", True, 1.0, "f32", False, 9),
    (55, 1000, 64, "softmax", True, 1.0, "f32", True, 2),
    (55, 513, 33, "sigmoid", False, 1.0, "bf16", True, 1),
    (13, 3, 3, "sigmoid", True, 1.0, "f32", True, 20),
    (13, 1, 1, "softmax", True, 1.0, "f32", True, 1),
]


@pytest.mark.parametrize("case", GRADS, ids=lambda r: "-".join(map(str, r)))
def test_select_backward_matches_the_formula(case):
    T, E, k, score, renorm, scale, dtype, with_w, n = case
    say(f"[select-grad] {case}")
    l = logits_of(T, E, dtype, T + E).cuda()
    idx = ids_of(T, E, k, 7).cuda()
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(9)).cuda() if with_w else None
    kw, ref_kw, f = {}, {}, 0.0
    if n:
        off = seqs(T, n, 3)
        load, dloss = torch.rand(n, E, generator=torch.Generator().manual_seed(1)) * 2, torch.rand(n) + 0.5
        kw = dict(seq_offsets=off.cuda(), load=load.cuda(), dloss=dloss.cuda(), alpha=0.3)
        ref_kw = dict(off=off.numpy(), load=load.numpy(), dloss=dloss.numpy(), alpha=0.3)
        f = 0.3 * 1.5 * 2
    sel = _lib.selection(T, E, k, score=score, renorm=renorm, scale=scale, logits=dtype)
    out = torch.full((T + 1, E), -7.0, device="cuda")
    _lib.moe_select_backward(sel, l, idx, dw, out[:T], **kw)
    torch.cuda.synchronize()
    ref = plain64.select_grad(f64(l), idx.cpu().numpy(), f64(dw) if with_w else None, score, renorm, scale, **ref_kw)
    big = (scale * float(dw.abs().max()) if with_w else 0.0) + f
    assert np.abs(f64(out[:T]) - ref).max() <= 2 * rtol(l, E) * big
    assert (out[T:] == -7).all()


@pytest.mark.parametrize("score,renorm", [("sigmoid", True), ("sigmoid", False), ("softmax", True), ("softmax", False)])
def test_select_backward_against_differences(score, renorm):
    """Central differences, in 64 bits, of sum w dw + sum dloss loss at the kernel's own choice and load."""
    T, E, k, alpha = 6, 24, 4, 0.7
    say(f"[select-grad] differences {score} {renorm}")
    l = logits_of(T, E, "f32", 21).cuda()
    sel, idx, w = run_select(l, None, k=k, score=score, renorm=renorm, scale=1.5)
    off = torch.tensor([0, 2, 2, 6], dtype=torch.int32)
    loss, load = torch.empty(3, device="cuda"), torch.empty(3, E, device="cuda")
    ws = torch.empty(_lib.balance_workspace_bytes(sel, 3), dtype=torch.uint8, device="cuda")
    _lib.moe_balance_loss(sel, l, idx, off.cuda(), alpha, loss, load, ws)
    g = torch.Generator().manual_seed(5)
    dw, dloss = torch.randn(T, k, generator=g), torch.rand(3, generator=g)
    out = torch.empty(T, E, device="cuda")
    _lib.moe_select_backward(sel, l, idx, dw.cuda(), out, seq_offsets=off.cuda(), load=load, dloss=dloss.cuda(),
                             alpha=alpha)
    i = idx.cpu().numpy()

    def value(v):
        total = float((plain64.weights(v, i, score, renorm, 1.5) * dw.double().numpy()).sum())
        return total + float((plain64.balance(v, i, off.numpy(), alpha, score)[0] * dloss.double().numpy()).sum())

    base, h = f64(l), 1e-5
    for t in range(T):
        for e in range(E):
            up, dn = base.copy(), base.copy()
            up[t, e] += h
            dn[t, e] -= h
            # h^2/6 of a third derivative of order one, rounding 1e-16 / h, and the kernel's fp32
            assert abs((value(up) - value(dn)) / (2 * h) - float(out[t, e])) <= 2e-6


def test_select_backward_tiny_scores_and_skipped_ids():
    """Rows whose scores underflow or are masked have finite gradients; an id outside the experts is skipped."""
    T, E, k = 5, 256, 8
    say("[select-grad] tiny scores")
    l = logits_of(T, E, "f32", 3)
    l[0] = -float("inf")
    l[1] = -200.0
    l[2, 10:] = -90.0
    idx = ids_of(T, E, k, 2)
    idx[3, 0], idx[4, 7] = -1, E + 5
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(2))
    off = torch.tensor([0, T], dtype=torch.int32)
    for score in ("sigmoid", "softmax"):
        for renorm in (True, False):
            sel = _lib.selection(T, E, k, score=score, renorm=renorm)
            out = torch.full((T, E), float("nan"), device="cuda")
            _lib.moe_select_backward(sel, l.cuda(), idx.cuda(), dw.cuda(), out, seq_offsets=off.cuda(),
                                     load=torch.ones(1, E, device="cuda"), dloss=torch.ones(1, device="cuda"), alpha=0.1)
            assert torch.isfinite(out).all()
            assert (out[0] == 0).all()
            for t, j in ((3, 0), (4, 7)):  # the others as if the skipped one had a score of zero
                keep = [i for i in range(k) if i != j]
                ref = plain64.select_grad(l[t:t + 1].double().numpy(), idx[t:t + 1, keep].numpy(),
                                          dw[t:t + 1, keep].double().numpy(), score, renorm, 1.0, off=[0, 1],
                                          load=np.ones((1, E)), dloss=[1.0], alpha=0.1 / T)
                assert np.abs(f64(out[t]) - ref[0]).max() <= 2 * rtol(l[t], E) * 5


# ---------------------------------------------------------------- the balance loss

@pytest.mark.parametrize("T,E,k,score,dtype,n,first,last", [
    (1, 256, 8, "sigmoid", "f32", 1, 0, 1), (300, 256, 8, "sigmoid", "f32", 5, 0, 300),
    (1000, 60, 4, "softmax", "bf16", 9, 0, 1000), (1000, 64, 6, "softmax", "f32", 200, 17, 900),
    (200, 1000, 20, "sigmoid", "bf16", 3, 100, 130), (5000, 256, 8, "sigmoid", "f32", 4600, 0, 5000),
    (4096, 8, 2, "softmax", "f32", 1, 0, 4096), (64, 17, 3, "sigmoid", "f32", 64, 0, 0)])
def test_balance_loss_and_its_gradient(T, E, k, score, dtype, n, first, last):
    say(f"[balance] T={T} E={E} {score} n_seq={n} [{first}, {last})")
    l, idx = logits_of(T, E, dtype, T).cuda(), ids_of(T, E, k, T).cuda()
    off = seqs(T, n, n, first, last)
    sel = _lib.selection(T, E, k, score=score, logits=dtype)
    ws = torch.full((_lib.balance_workspace_bytes(sel, n),), 255, dtype=torch.uint8, device="cuda")
    loss, load = torch.full((n,), -7.0, device="cuda"), torch.full((n, E), -7.0, device="cuda")
    _lib.moe_balance_loss(sel, l, idx, off.cuda(), 0.5, loss, load, ws)
    rl, rf = plain64.balance(f64(l), idx.cpu().numpy(), off.numpy(), 0.5, score)
    np.testing.assert_allclose(f64(load), rf, rtol=2 * plain64.EPS32, atol=0)
    # shares to rtol(), 16 of them added per wave, then 64-bit sums
    np.testing.assert_allclose(f64(loss), rl, rtol=rtol(l, E) + 20 * plain64.EPS32)
    again, load2 = torch.empty_like(loss), torch.empty_like(load)
    _lib.moe_balance_loss(sel, l, idx, off.cuda(), 0.5, again, load2, ws)
    assert torch.equal(loss, again) and torch.equal(load, load2)
    out = torch.empty(T, E, device="cuda")
    dloss = torch.ones(n, device="cuda")
    _lib.moe_select_backward(sel, l, None, None, out, seq_offsets=off.cuda(), load=load, dloss=dloss, alpha=0.5)
    ref = plain64.select_grad(f64(l), idx.cpu().numpy(), None, score, True, 1.0, off.numpy(), f64(load), np.ones(n), 0.5)
    assert np.abs(f64(out) - ref).max() <= 2 * rtol(l, E) * 0.5 * max(1.0, float(load.max()))
    outside = torch.ones(T, dtype=torch.bool)
    outside[first:last] = False
    assert (out[outside.cuda()] == 0).all()


def test_balance_loss_of_as_many_choices_as_there_may_be():
    """T * k = 2^31 - 64, the most that is taken: every expert chosen by every token."""
    E = k = 64
    T = (1 << 25) - 1
    say(f"[balance] T={T} k={k}")
    l = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    idx = torch.arange(E, dtype=torch.int32, device="cuda").repeat(T, 1)
    off = torch.tensor([0, 5, T - 3, T], dtype=torch.int32, device="cuda")
    sel = _lib.selection(T, E, k, logits="bf16")
    ws = torch.empty(_lib.balance_workspace_bytes(sel, 3), dtype=torch.uint8, device="cuda")
    loss, load = torch.empty(3, device="cuda"), torch.empty(3, E, device="cuda")
    _lib.moe_balance_loss(sel, l, idx, off, 0.25, loss, load, ws)
    assert (load == 1).all()
    np.testing.assert_allclose(f64(loss), 0.25, rtol=1e-6)


def test_balance_loss_of_a_balanced_sequence_is_alpha():
    say("[balance] balanced")
    T, E, k = 64, 64, 4
    idx = (torch.arange(T)[:, None] * k + torch.arange(k)) % E
    sel = _lib.selection(T, E, k)
    ws = torch.empty(_lib.balance_workspace_bytes(sel, 1), dtype=torch.uint8, device="cuda")
    loss, load = torch.empty(1, device="cuda"), torch.empty(1, E, device="cuda")
    _lib.moe_balance_loss(sel, torch.zeros(T, E, device="cuda"), idx.to(torch.int32).cuda(),
                          torch.tensor([0, T], dtype=torch.int32, device="cuda"), 0.25, loss, load, ws)
    assert float(loss) == 0.25 and (load == 1).all()


# ---------------------------------------------------------------- streams and graphs

def test_select_path_on_a_side_stream_and_from_a_graph():
    """The choice, the loss and the gradient captured once and replayed on new inputs, beside eager work."""
    T, E, k, n = 500, 256, 8, 3
    say("[select] graph replays")
    static = logits_of(T, E, "f32", 1).cuda()
    bias = (0.1 * torch.rand(E) - 0.05).cuda()
    off = seqs(T, n, 4).cuda()
    sel = _lib.selection(T, E, k, n_group=8, topk_group=4)
    dw, dloss = torch.randn(T, k, device="cuda"), torch.ones(n, device="cuda")
    o = dict(idx=torch.empty(T, k, dtype=torch.int32, device="cuda"), w=torch.empty(T, k, device="cuda"),
             loss=torch.empty(n, device="cuda"), load=torch.empty(n, E, device="cuda"), dl=torch.empty(T, E, device="cuda"))
    ws = torch.empty(_lib.balance_workspace_bytes(sel, n), dtype=torch.uint8, device="cuda")

    def step(l, b):
        _lib.moe_select(sel, l, bias, b["idx"], b["w"])
        _lib.moe_balance_loss(sel, l, b["idx"], off, 0.1, b["loss"], b["load"], ws)
        _lib.moe_select_backward(sel, l, b["idx"], dw, b["dl"], seq_offsets=off, load=b["load"], dloss=dloss, alpha=0.1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(static, o)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    first = {m: t.clone() for m, t in o.items()}
    e = {m: torch.empty_like(t) for m, t in o.items()}
    step(static, e)
    assert all(torch.equal(first[m], e[m]) for m in e)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(static, o)
    for r in range(3):
        l = logits_of(T, E, "f32", 50 + r).cuda()
        static.copy_(l)
        graph.replay()
        torch.cuda.synchronize()
        step(l, e)
        torch.cuda.synchronize()
        assert all(torch.equal(o[m], e[m]) for m in e), f"replay {r}"
