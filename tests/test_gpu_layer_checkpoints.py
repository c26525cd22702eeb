"""Checkpoints that outlive later forwards: several micro-batches in flight, in any order, and a layer whose input is
kept in 8 bits alone."""
import pytest
import torch

import synth
from sparse_expert_routing_amd import _lib
from sparse_expert_routing_amd.layer import layer_from_inputs, upload
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

ROUTERS = {"fused": None, "logits": dict(score="sigmoid", n_group=8, topk_group=4, group_score="top2", scale=2.5)}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    _lib.load()


def case(router, wt="bf16", T=200, d=256, I=128):
    cfg = synth.CONFIGS[2].with_(name="micro-batches", T=T, d=d, I=I, wt=wt, act="bf16", seed=5)
    inp = synth.make_inputs(cfg)
    layer = layer_from_inputs(inp, router=ROUTERS[router])
    bias = upload(inp["bias"])
    xs = [torch.randn(T, d, generator=torch.Generator().manual_seed(s)).bfloat16().view(torch.int16).cuda() for s in range(3)]
    dys = [torch.randn(T, d, generator=torch.Generator().manual_seed(9 + s)).cuda() for s in range(3)]
    return layer, xs, dys, bias


def equal(a, b):
    return [n for n in a if not torch.equal(a[n], b[n])]


@pytest.mark.parametrize("router", list(ROUTERS))
@pytest.mark.parametrize("wt,fmt", [("bf16", "e4m3"), ("bf16", "i8"), ("e4m3", "e4m3")])
def test_forwards_before_the_first_backward(router, wt, fmt):
    say(f"[layer-checkpoints] {router} {wt} {fmt}")
    layer, xs, dys, bias = case(router, wt)
    off = torch.tensor([0, 90, 200], dtype=torch.int32, device="cuda")
    dloss = torch.tensor([1.0, 0.5], device="cuda")

    def forward(x):
        layer.forward(x, bias)
        load = layer.balance_loss(off, 0.1)[1] if ROUTERS[router] else None
        return layer.checkpoint(x, fmt), load

    def backward(x, dy, kept, load):
        more = (off, load, dloss, 0.1) if ROUTERS[router] else ()
        return layer.backward(x, kept, dy, *more)

    want = []
    for x, dy in zip(xs, dys):
        kept, load = forward(x)
        want.append({n: t.clone() for n, t in backward(x, dy, kept, load).items()})
    flying = [forward(x) for x in xs]
    for b in (1, 0, 2, 0):
        assert not equal(want[b], backward(xs[b], dys[b], *flying[b])), b


@pytest.mark.parametrize("router", list(ROUTERS))
def test_plain_checkpoints_are_refused_behind_the_next_forward(router):
    """fmt "bf16" keeps the layer's own buffers."""
    say(f"[layer-checkpoints] plain {router}")
    layer, xs, dys, bias = case(router)
    layer.forward(xs[0], bias)
    kept = layer.checkpoint(xs[0], "bf16")
    layer.backward(xs[0], kept, dys[0])
    layer.backward(xs[0], kept, dys[0])
    layer.forward(xs[1], bias)
    with pytest.raises(ValueError, match="forward"):
        layer.backward(xs[0], kept, dys[0])
    layer.backward(xs[1], layer.checkpoint(xs[1], "bf16"), dys[1])


def test_micro_batches_replay_from_a_graph():
    """Two forwards, then their backwards, captured and replayed on new inputs beside eager work."""
    say("[layer-checkpoints] graph")
    layer, xs, dys, bias = case("logits")
    other, *_ = case("logits")

    def step(lay):
        kept = []
        for x in xs[:2]:
            lay.forward(x, bias)
            kept.append(lay.checkpoint(x))
        return [lay.backward(x, k, dy) for x, k, dy in zip(xs, kept, dys)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(layer)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(layer)
    for r in range(4):
        for j, x in enumerate(xs[:2]):
            x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(20 + 2 * r + j)).bfloat16().view(torch.int16))
        graph.replay()
        torch.cuda.synchronize()
        ref = step(other)
        torch.cuda.synchronize()
        for a, b in zip(ref, out):
            assert not equal(a, b), r


@pytest.mark.parametrize("wt,fmt", [("bf16", "e4m3"), ("bf16", "i8"), ("e4m3", "i8"), ("bf16", "bf16")])
def test_a_layer_with_a_router_can_do_without_its_input(wt, fmt):
    """x None: the router projection's gradient takes the checkpoint's values too."""
    say(f"[layer-checkpoints] no x {wt} {fmt}")
    layer, xs, dys, bias = case("logits", wt)
    x, dy = xs[0], dys[0]
    layer.forward(x, bias)
    kept = layer.checkpoint(x, fmt)
    got = layer.backward(None, kept, dy)
    if fmt == "bf16":
        seen = x
    else:
        seen = torch.empty(x.shape, dtype=torch.bfloat16, device="cuda")
        _lib.moe_checkpoint_unpack(kept[0][0], kept[0][1], fmt, seen)
    assert not equal(layer.backward(seen, kept, dy), got)
    assert not equal(layer.backward(x, kept, dy), {**got, "dw_router": layer.backward(x, kept, dy)["dw_router"]})
