"""The layer's packed experts where another stream is behind."""
import pytest
import torch

from tests.gpu_util import say
from tests.test_gpu_layer_packed import case

pytestmark = pytest.mark.gpu


def busy(stream):
    """Some milliseconds of work on a stream."""
    with torch.cuda.stream(stream):
        a = torch.ones(4096, 4096, device="cuda")
        for _ in range(20):
            a = a @ a * 2.0**-12
    return a


def overwrite(layer_weights):
    """New tensors of the sizes that were let go of, on the current stream, filled with something else."""
    return [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda") for n in layer_weights for _ in range(3)]


@pytest.mark.parametrize("packing_is_behind", [True, False])
def test_weights_let_go_of_while_a_side_stream_is_behind(packing_is_behind):
    """The side stream's packing, or its forward on the bf16 weights, reads them late: new tensors on the first stream change
    neither."""
    say("[layer streams]", packing_is_behind)
    layer, x, bias = case(T=64, d=512, I=512)
    want = layer.forward(x, bias).clone()
    layer.pack_experts()
    served = layer.forward(x, bias).clone()
    mats = [[t.clone() for t in m.tensors] for m in layer.packed[1]]
    fresh, _, _ = case(T=64, d=512, I=512)
    sizes = [fresh.ex[n].numel() * 2 for n in ("gate", "up", "down")]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    kept = [busy(side)]
    if packing_is_behind:
        fresh.pack_experts(keep=False, stream=side)
        kept += overwrite(sizes)
        side.synchronize()
        for m, tensors in zip(fresh.packed[1], mats):
            assert all(torch.equal(a, b) for a, b in zip(m.tensors, tensors))
        torch.cuda.synchronize()
        assert torch.equal(fresh.forward(x, bias), served)
    else:
        y = fresh.forward(x, bias, stream=side)
        fresh.pack_experts(keep=False)
        kept += overwrite(sizes)
        side.synchronize()
        assert torch.equal(y, want)


def test_weights_are_not_let_go_of_in_a_capture():
    layer, x, bias = case(T=16, d=128, I=64)
    layer.pack_experts()
    layer.forward(x, bias)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError):
            layer.pack_experts(keep=False)
        layer.forward(x, bias)
    want = layer.forward(x, bias).clone()
    for _ in range(3):
        layer.y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(layer.y, want)
