"""The router projection's gradient on the GPU against float64, elementwise to the
rounding of fp32 sums."""
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


def inputs(T, d, act, seed, sparse=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, d, generator=g)
    x = (x.bfloat16() if act == "bf16" else x).cuda()
    w = (torch.randn(256, d, generator=g) * d**-0.5).cuda()
    dl = torch.randn(T, 256, generator=g) * torch.exp(4 * torch.randn(T, 1, generator=g))
    if sparse:
        dl *= torch.rand(T, 256, generator=g) < 8 / 256
    return x, w, dl.cuda(), torch.randn(T, d, generator=g).cuda()


def run(x, w, dl, dx_in, dx, act):
    T, d = x.shape
    ds = _lib.desc(T, d, 256, 8, 128, act, act)
    ws = torch.full((max(1, _lib.workspace_bytes(ds, _lib.MOE_WS_ROUTER_GRAD)),), 0xFF, dtype=torch.uint8, device="cuda")
    dw = torch.full((256, d), float("nan"), device="cuda")
    _lib.moe_router_logits_backward(ds, x, w, dl, dx_in, dx, dw, ws)
    torch.cuda.synchronize()
    return dw


def check(x, w, dl, dx_in, dx, dw):
    X, W, L = x.double(), w.double(), dl.double()
    ref, size = L @ W, L.abs() @ W.abs()
    if dx_in is not None:
        ref, size = ref + dx_in.double(), size + dx_in.double().abs()
    # 256 fp32 additions and the terms' own roundings (or the split's, 2^-22 of the row's and column's largest)
    row, col = L.abs().amax(1, keepdim=True), W.abs().amax(0, keepdim=True)
    # A product or sum below fp32's smallest normal number, 2^-126, has no 24 bits to be held in: the row of
    # 1e-30 times the column of 1e-25 is 1e-55, which fp32 can only give as 0.  So each of the 256 products and
    # sums may be off by up to 2^-126 absolutely, beside its relative rounding.
    assert ((dx.double() - ref).abs() <= 260 * plain64.EPS32 * size + 256 * 2.0**-38 * row * col + 512 * 2.0**-126).all()
    ref, size = L.t() @ X, L.abs().t() @ X.abs()
    n = min(x.shape[0], 4096) + 32
    assert ((dw.double() - ref).abs() <= n * plain64.EPS32 * size + 2 * x.shape[0] * 2.0**-126).all()


@pytest.mark.parametrize("T,d,act", [(1, 128, "bf16"), (1, 64, "f32"), (37, 256, "bf16"), (129, 896, "bf16"),
                                     (64, 192, "f32"), (1000, 1024, "f32"), (2049, 2048, "bf16"), (4100, 512, "bf16"),
                                     (3000, 7168, "bf16")])
@pytest.mark.parametrize("sparse", [False, True])
def test_router_grad(T, d, act, sparse):
    say(f"[router-grad] T={T} d={d} {act} sparse={sparse}")
    x, w, dl, dx_in = inputs(T, d, act, T + d, sparse)
    dx = torch.full((T + 1, d), -7.0, device="cuda")
    dw = run(x, w, dl, dx_in, dx[:T], act)
    check(x, w, dl, dx_in, dx[:T], dw)
    assert (dx[T:] == -7).all()
    # no dx_in; and dx_in as dx itself, twice the same bits
    dx2 = torch.full((T, d), float("nan"), device="cuda")
    assert torch.equal(run(x, w, dl, None, dx2, act), dw)
    check(x, w, dl, None, dx2, dw)
    dx3 = dx_in.clone()
    assert torch.equal(run(x, w, dl, dx3, dx3, act), dw) and torch.equal(dx3, dx[:T])


@pytest.mark.parametrize("T,d,act", [(4099, 4096, "f32"), (4500, 4032, "f32"), (9001, 1920, "bf16"), (3900, 4096, "bf16")])
def test_router_grad_about_the_large_tiles(T, d, act):
    """The first sizes of the large tiles, ragged in both directions, and the last of the small ones."""
    say(f"[router-grad] T={T} d={d} {act}")
    x, w, dl, dx_in = inputs(T, d, act, T + d, False)
    dx = torch.full((T + 1, d), -7.0, device="cuda")
    dw = run(x, w, dl, dx_in, dx[:T], act)
    check(x, w, dl, dx_in, dx[:T], dw)
    assert (dx[T:] == -7).all()


def test_router_grad_past_32_bit_offsets():
    T, d = 2_100_003, 1024  # 2.15e9 values of x
    say(f"[router-grad] T={T} d={d}")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(T, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w = torch.randn(256, d, device="cuda", generator=g) * d**-0.5
    dl = torch.randn(T, 256, device="cuda", generator=g)
    dx = torch.empty(T, d, device="cuda")
    dw = run(x, w, dl, None, dx, "bf16")
    for part in (slice(0, 300), slice(T - 300, T)):
        L, W = dl[part].double(), w.double()
        assert ((dx[part].double() - L @ W).abs() <= 260 * plain64.EPS32 * (L.abs() @ W.abs()) + 1e-9).all()
    ref, size = 0, 0
    for xs, ls in zip(x.split(1 << 18), dl.split(1 << 18)):
        ref = ref + ls.double().t() @ xs.double()
        size = size + ls.double().abs().t() @ xs.double().abs()
    # a split's 4096-odd products at a time in fp32, the splits' sums behind one another
    assert ((dw.double() - ref).abs() <= (T / 16 + 300) * plain64.EPS32 * size).all()
    assert float((dw.double() - ref).norm()) <= 1e-5 * float(ref.norm())


def test_router_grad_zeros_and_extremes():
    """Rows and columns of zeros, tiny and large magnitudes."""
    T, d = 200, 256
    say("[router-grad] extremes")
    x, w, dl, dx_in = inputs(T, d, "bf16", 5)
    dl[0] = 0
    dl[1] *= 1e-30
    dl[2] *= 1e20
    dl[3, 1:] = 0
    dl[:, 17] = 0
    w[:, 3] = 0
    w[:, 4] *= 1e-25
    w[:, 5] *= 1e10
    w[9] = 0
    dx = torch.empty(T, d, device="cuda")
    dw = run(x, w, dl, None, dx, "bf16")
    check(x, w, dl, None, dx, dw)
    assert (dx[0] == 0).all() and (dx[:, 3] == 0).all() and (dw[17] == 0).all()


def test_router_grad_replays_from_a_graph():
    T, d = 700, 512
    say("[router-grad] graph")
    x, w, dl, dx_in = inputs(T, d, "bf16", 8)
    ds = _lib.desc(T, d, 256, 8, 128)
    ws = torch.empty(max(1, _lib.workspace_bytes(ds, _lib.MOE_WS_ROUTER_GRAD)), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty_like(ws)
    dx, dw = torch.empty(T, d, device="cuda"), torch.empty(256, d, device="cuda")
    ex, ew = torch.empty_like(dx), torch.empty_like(dw)
    _lib.moe_router_logits_backward(ds, x, w, dl, dx_in, dx, dw, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _lib.moe_router_logits_backward(ds, x, w, dl, dx_in, dx, dw, ws)
    for r in range(3):
        dl.copy_(torch.randn(T, 256, generator=torch.Generator().manual_seed(r)))
        g.replay()
        torch.cuda.synchronize()
        _lib.moe_router_logits_backward(ds, x, w, dl, dx_in, ex, ew, ws2)
        torch.cuda.synchronize()
        assert torch.equal(dx, ex) and torch.equal(dw, ew), f"replay {r}"
