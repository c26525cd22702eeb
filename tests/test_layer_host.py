"""What the layer does on the host, on the CPU: kernels are not launched."""
import pytest
import torch

import synth
from sparse_expert_routing_amd import layer as L


@pytest.fixture
def layer(monkeypatch):
    """A layer in host memory, whose packing launches nothing."""
    cfg = synth.CONFIGS[2].with_(name="host", T=8, d=128, I=64, seed=3)
    made = L.layer_from_inputs(synth.make_inputs(cfg), device="cpu")
    monkeypatch.setattr(L._lib, "moe_mx_pack", lambda *a, **k: None)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return made


def test_weights_are_let_go_of_behind_all_that_reads_them(layer, monkeypatch):
    waited = []
    monkeypatch.setattr(torch.cuda, "synchronize", lambda device=None: waited.append(layer.ex["gate"] is not None and layer.ex_w is not None))
    layer.pack_experts()
    assert waited == [] and layer.ex_w is not None
    layer.pack_experts(keep=False)
    assert waited == [True] and layer.ex_w is None and layer.ex["gate"] is None


def test_weights_are_not_let_go_of_in_a_capture(layer, monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(ValueError):
        layer.pack_experts(keep=False)
    assert layer.ex_w is not None and layer.packed is None
    layer.pack_experts()


@pytest.mark.parametrize("T,fmt", [(1 << 25, "e4m3"), ((1 << 26) - 100, "e2m1"), (1 << 28, "e2m1")])
def test_more_tokens_than_the_products_take_are_refused_before_weights_are_let_go_of(layer, T, fmt):
    """Codes of the gathered rows past 2^32 - 2^20 bytes, rows past 2^29 or 2^31."""
    layer.T = T
    with pytest.raises(ValueError):
        layer.pack_experts(fmt, keep=False)
    assert layer.ex_w is not None and layer.packed is None and not layer._packed_room


def test_the_device_that_is_waited_for_is_the_weights(layer, monkeypatch):
    """A layer made on "cuda" lies on the device that was current then, not on the one that is."""
    waited = []
    monkeypatch.setattr(torch.cuda, "synchronize", lambda device=None: waited.append(device))
    where = layer.ex["gate"].device
    layer.device = torch.device("meta")
    layer.pack_experts(keep=False)
    assert waited == [where]
