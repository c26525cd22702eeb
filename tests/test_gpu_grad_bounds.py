"""Bounds in the gradients' own sizes, element by element, where a norm or a worst case hides a wrong one: the router
projection's weight gradient over very many tokens, and the balance loss's share of a layer's router gradient."""
import numpy as np
import pytest
import torch

import synth
from sparse_expert_routing_amd import _lib
from sparse_expert_routing_amd.layer import layer_from_inputs, upload
from tests import plain64
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    _lib.load()


@pytest.mark.parametrize("T,d,splits", [(2_100_003, 1024, 64), (16_400, 1024, 64), (300_001, 256, 256)])
def test_router_grad_dw_elements(T, d, splits):
    """dw is summed in fp32 over T / splits tokens (blocks of 256 columns, a split per CU), three terms of 16 tokens at a
    time, so in n = 3 T / splits / 16 additions, the splits' sums behind one another.  An addition rounds to nearest:
    off by at most u = 2^-24 of the sum so far, about u / sqrt 3 of it on average and of either sign.  The sums so far
    are a random walk's, sqrt(i / n) of the split's last, so that the roundings add up to
    u sqrt(n / 6) sqrt(sum of squared products).  Four times u sqrt(n) is ten times that, which none of the elements
    comes near by chance, and far below the elements themselves."""
    say(f"[grad-bounds] dw T={T} d={d}")
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.empty(T, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w = torch.randn(256, d, device="cuda", generator=g) * d**-0.5
    dl = torch.randn(T, 256, device="cuda", generator=g)
    ds = _lib.desc(T, d, 256, 8, 128)
    ws = torch.full((_lib.workspace_bytes(ds, _lib.MOE_WS_ROUTER_GRAD),), 0xFF, dtype=torch.uint8, device="cuda")
    dx, dw = torch.empty(T, d, device="cuda"), torch.full((256, d), float("nan"), device="cuda")
    _lib.moe_router_logits_backward(ds, x, w, dl, None, dx, dw, ws)
    ref, square = 0, 0
    for xs, ls in zip(x.split(1 << 18), dl.split(1 << 18)):
        xs, ls = xs.double(), ls.double()
        ref = ref + ls.t() @ xs
        square = square + (ls**2).t() @ xs**2
    n = 3 * T / splits / 16
    bound = 4 * plain64.EPS32 * (n + splits) ** 0.5 * square.sqrt()
    assert ((dw.double() - ref).abs() <= bound).all()
    assert float((ref.abs() > bound).double().mean()) > 0.99  # a lost element is found


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_the_balance_loss_reaches_the_routers_weights(score):
    """dw_router with the balance loss less that without it is the loss's dlogits^T x, element by element."""
    say(f"[grad-bounds] dw_router's balance share {score}")
    cfg = synth.CONFIGS[2].with_(name=f"balance {score}", T=300, d=256, I=128, wt="bf16", act="bf16", seed=9)
    inp = synth.make_inputs(cfg)
    layer = layer_from_inputs(inp, router=dict(score=score))
    x, bias = upload(inp["x"]), upload(inp["bias"])
    layer.forward(x, bias)
    alpha = 200.0  # beside weight gradients of order one a token
    off = torch.tensor([0, 100, 100, 290], dtype=torch.int32, device="cuda")
    _, load = layer.balance_loss(off, alpha)
    dloss = torch.tensor([1.0, 5.0, 0.5], device="cuda")
    dy = torch.randn(layer.T, layer.d, generator=torch.Generator().manual_seed(1)).cuda()
    none = layer.backward(x, layer.checkpoint(x, "bf16"), dy)
    whole = layer.backward(x, layer.checkpoint(x, "bf16"), dy, off, load, dloss, alpha)

    def f64(t):
        return t.detach().cpu().double().numpy()

    l, i, xv = f64(layer.logits), layer.idx.cpu().numpy(), f64(x.view(torch.bfloat16))
    more = dict(off=off.cpu().numpy(), load=f64(load), dloss=f64(dloss), alpha=alpha)
    share = plain64.select_grad(l, i, None, score, True, 1.0, **more)
    weights = plain64.select_grad(l, i, f64(none["dg"]), score, True, 1.0)
    ref = share.T @ xv
    # T fp32 products added, of each of the two gradients; their dlogits to some tens of half steps
    bound = 2 * (layer.T + 100) * plain64.EPS32 * (np.abs(share).T + np.abs(weights).T) @ np.abs(xv)
    assert (np.abs(f64(whole["dw_router"]) - f64(none["dw_router"]) - ref) <= bound).all()
    assert (np.abs(ref) > bound).mean() > 0.5
