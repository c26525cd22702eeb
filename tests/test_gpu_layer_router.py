"""The layer with a router of its own: a forward chosen from logits, its balance loss, its
checkpoints and its backward, as a training step runs them, eagerly and from a graph."""
import numpy as np
import pytest
import torch

import synth
from sparse_expert_routing_amd import _lib
from sparse_expert_routing_amd.layer import layer_from_inputs, upload
from tests import plain64
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

ROUTERS = {
    "grouped sigmoid": dict(score="sigmoid", n_group=8, topk_group=4, group_score="top2", scale=2.5),
    "softmax as it is": dict(score="softmax", renorm=False, scale=4.0),
}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    _lib.load()


def f64(t):
    return t.detach().cpu().double().numpy()


def case(wt, T=300, d=256, I=128, router=None):
    act = "f32" if wt == "f32" else "bf16"
    cfg = synth.CONFIGS[2].with_(name=f"router {wt}", T=T, d=d, I=I, wt=wt, act=act, seed=9)
    inp = synth.make_inputs(cfg)
    return inp, layer_from_inputs(inp, router=router), upload(inp["x"]), upload(inp["bias"])


def values(t, wt):
    return t.double() if wt == "f32" else t.view(torch.bfloat16).double()


def routed(layer, wt):
    """sum_j w_j y_perm_j of the last forward, in 64 bits."""
    y = values(layer.y_perm, wt)[layer.row_of.long()].view(layer.T, 8, layer.d)
    return (layer.w.double()[:, :, None] * y).sum(1)


@pytest.mark.parametrize("wt", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("name", list(ROUTERS))
def test_forward_with_a_router(name, wt):
    say(f"[layer-router] forward {name} {wt}")
    router = ROUTERS[name]
    inp, layer, x, bias = case(wt, router=router)
    plain = layer_from_inputs(inp)
    y = layer.forward(x, bias)
    other = layer.forward(x, bias, gather_in_gemm=False).clone()
    assert torch.equal(y, other)
    kw = {n: v for n, v in router.items()}
    ri, rw = plain64.select(f64(layer.logits), f64(bias), 8, **kw)
    assert np.array_equal(layer.idx.cpu().numpy(), ri)
    np.testing.assert_allclose(f64(layer.w), rw, rtol=plain64.EPS32 * 64)
    # the shared expert's part is the same whatever the routing
    plain.forward(x, bias)
    shared = plain.y.double() - routed(plain, wt)
    want = shared + routed(layer, wt)
    assert float((y.double() - want).abs().max()) <= 1e-4 * float(want.abs().max())
    with pytest.raises(ValueError):
        layer.forward(x, bias, gap=True)


@pytest.mark.parametrize("wt", ["bf16", "e4m3"])
@pytest.mark.parametrize("name", list(ROUTERS))
def test_training_step_with_a_router(name, wt):
    """Router gradients of the whole step against the formulas: dlogits from the layer's own dg, dw_router and dx
    from them; the balance loss beside them."""
    say(f"[layer-router] training step {name} {wt}")
    router = ROUTERS[name]
    _, layer, x, bias = case(wt, router=router)
    T, d, alpha = layer.T, layer.d, 0.02
    layer.forward(x, bias)
    off = torch.tensor([0, 100, 100, 290], dtype=torch.int32, device="cuda")
    loss, load = layer.balance_loss(off, alpha)
    rl, rf = plain64.balance(f64(layer.logits), layer.idx.cpu().numpy(), off.cpu().numpy(), alpha, router["score"])
    np.testing.assert_allclose(f64(loss), rl, rtol=1e-5)
    np.testing.assert_allclose(f64(load), rf, rtol=1e-6)
    dy = torch.randn(T, d, generator=torch.Generator().manual_seed(1)).cuda()
    dloss = torch.tensor([1.0, 5.0, 0.5], device="cuda")
    none = layer.backward(x, layer.checkpoint(x, "bf16"), dy)
    whole = layer.backward(x, layer.checkpoint(x, "bf16"), dy, off, load, dloss, alpha)
    score, renorm, scale = router["score"], router.get("renorm", True), router["scale"]
    xv, wr = values(x, "bf16"), layer.wr.double()
    i = layer.idx.cpu().numpy()
    for g, more in ((none, {}), (whole, dict(off=off.cpu().numpy(), load=f64(load), dloss=f64(dloss), alpha=alpha))):
        dl = torch.from_numpy(plain64.select_grad(f64(layer.logits), i, f64(g["dg"]), score, renorm, scale, **more)).cuda()
        ref = dl.t() @ xv
        assert float((g["dw_router"].double() - ref).norm()) <= 1e-5 * float(ref.norm())
        # dx without the router's share: the same for both
        assert torch.equal(g["dw_down"], none["dw_down"]) and torch.equal(g["dg"], none["dg"])
        g["rest"] = g["dx"].double() - dl @ wr
    scale_of = float(none["rest"].abs().max())
    assert float((none["rest"] - whole["rest"]).abs().max()) <= 1e-5 * scale_of
    # 8 bits: about their rounding away (e4m3 2^-4, int8 a step of the tile's largest), not more
    # With e4m3 weights the backward rounds x to e4m3 again.  That leaves an e4m3 checkpoint's values as they are, but
    # an int8 one's, off by a mean of at most m / 127 / 2 for a tile's largest m (about 3 sigma: 0.012 sigma), moves
    # that share of a step of the values over a border of e4m3, by a whole step of up to 2^-3 sigma: a mean square of
    # 0.012 * 2^-3, 0.038 sigma, in both factors of a SwiGLU's gradient: 0.08.
    for fmt, tol in (("e4m3", 0.06), ("i8", 0.03 if wt == "bf16" else 0.08)):
        g = layer.backward(x, layer.checkpoint(x, fmt), dy)
        for n in ("dx", "dw_gate", "dw_down", "dw_router", "dg", "ds_up"):
            assert torch.isfinite(g[n]).all()
            assert float((g[n] - none[n]).norm()) <= tol * float(none[n].norm()), (fmt, n)


def test_layer_without_a_router_trains_by_moe_backward():
    say("[layer-router] fused router")
    _, layer, x, bias = case("bf16")
    layer.forward(x, bias)
    dy = torch.randn(layer.T, layer.d, generator=torch.Generator().manual_seed(1)).cuda()
    g = layer.backward(x, layer.checkpoint(x, "bf16"), dy)
    ref = {n: torch.empty_like(t) for n, t in g.items()}
    ws = torch.empty(_lib.workspace_bytes(layer.desc, _lib.MOE_WS_BACKWARD), dtype=torch.uint8, device="cuda")
    _lib.moe_backward(layer.desc, x, layer.wr, layer.idx, layer.w, layer.offsets, layer.row_src, layer.row_of, layer.ex_w,
                      layer.sh_w, layer.y_perm, dy, ref, ws)
    assert all(torch.equal(g[n], ref[n]) for n in ref)
    with pytest.raises(ValueError):
        layer.balance_loss(torch.tensor([0, 5], dtype=torch.int32, device="cuda"), 0.1)
    with pytest.raises(ValueError):
        layer.backward(x, layer.checkpoint(x, "bf16"), dy, dloss=torch.ones(1, device="cuda"))


def test_training_step_on_a_side_stream():
    """A step whose calls are given a stream other than the current one, while the current one allocates and
    overwrites: everything of it belongs to that stream."""
    say("[layer-router] side stream")
    _, layer, x, bias = case("bf16", router=ROUTERS["grouped sigmoid"])
    off = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
    dy = torch.randn(layer.T, layer.d, generator=torch.Generator().manual_seed(1)).cuda()
    dloss = torch.ones(2, device="cuda")

    def step(stream):
        layer.forward(x, bias, stream=stream)
        loss, load = layer.balance_loss(off, 0.01, stream=stream)
        kept = layer.checkpoint(x, "i8", stream=stream)
        if stream is not None:
            junk = [torch.full((1 << 22,), 7.0, device="cuda") for _ in range(8)]
        g = layer.backward(x, kept, dy, off, load, dloss, 0.01, stream=stream)
        if stream is not None:
            junk += [torch.full((1 << 24,), 7.0, device="cuda") for _ in range(8)]
        return dict(loss=loss, load=load, **g)

    ref = {n: t.clone() for n, t in step(None).items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    torch.cuda.synchronize()
    assert all(torch.equal(ref[n], got[n]) for n in ref)


def test_training_step_replays_from_a_graph():
    """One captured step (forward, loss, checkpoint, backward, bias step) replayed on new inputs beside eager work,
    each replay against the eager step on a layer of its own."""
    say("[layer-router] graph")
    inp, layer, x, bias = case("bf16", router=ROUTERS["grouped sigmoid"])
    eager = layer_from_inputs(inp, router=ROUTERS["grouped sigmoid"])
    off = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
    dy = torch.randn(layer.T, layer.d, generator=torch.Generator().manual_seed(1)).cuda()
    dloss = torch.ones(2, device="cuda")

    def step(lay, xx, b):
        lay.forward(xx, b)
        loss, load = lay.balance_loss(off, 0.01)
        g = lay.backward(xx, lay.checkpoint(xx), dy, off, load, dloss, 0.01)
        lay.update_bias(b)
        return dict(loss=loss, y=lay.y, bias=b, **g)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(layer, x, bias.clone())
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    mine, theirs = bias.clone(), bias.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(layer, x, mine)
    for r in range(3):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(r)).bfloat16().view(torch.int16))
        graph.replay()
        torch.cuda.synchronize()
        ref = step(eager, x, theirs)
        torch.cuda.synchronize()
        for n in ref:
            assert torch.equal(ref[n], out[n]), (r, n)
