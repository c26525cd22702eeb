"""8-bit activation checkpoints on the GPU: codes against their definition exactly,
the combine's gradient and the layer's backward from them."""
import numpy as np
import pytest
import torch

import synth
from sparse_expert_routing_amd import _lib
from sparse_expert_routing_amd.layer import layer_from_inputs, upload
from tests import plain64
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    _lib.load()


def f64(t):
    return t.detach().cpu().double().numpy()


def pack(x, fmt):
    rows, cols = x.shape
    codes = torch.full((rows, cols), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, -(-cols // 128)), 0x55, dtype=torch.uint8, device="cuda")
    _lib.moe_checkpoint_pack(x, codes, scales, fmt)
    return codes, scales


def unpack(codes, scales, fmt, dtype):
    out = torch.full(codes.shape, -7.0, dtype=dtype, device="cuda")
    _lib.moe_checkpoint_unpack(codes, scales, fmt, out)
    return out


def code_values(codes, fmt):
    return f64((codes.view(torch.float8_e4m3fn) if fmt == "e4m3" else codes.view(torch.int8)).float())


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 128), (17, 130), (33, 255), (9, 1024), (301, 1001), (64, 7168),
                                       (2000, 64)])
def test_pack_and_unpack(rows, cols, dtype, fmt):
    say(f"[ckpt] {rows}x{cols} {dtype} {fmt}")
    g = torch.Generator().manual_seed(rows * 7 + cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp(3 * torch.randn(rows, 1, generator=g))
    x = x.to(TYPES[dtype])
    codes, scales = pack(x.cuda(), fmt)
    u, byte = plain64.pack(f64(x), fmt)
    assert np.array_equal(scales.cpu().numpy(), byte)
    assert np.array_equal(code_values(codes, fmt), u)
    for out in ("bf16", "f32"):  # three (e4m3) and seven (int8) bits fit either type: nothing is rounded
        assert np.array_equal(f64(unpack(codes, scales, fmt, TYPES[out])), plain64.unpack(u, byte))


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
def test_special_tiles(fmt):
    """Zeros, subnormals, the largest numbers, ties of the rounding, the borders of a scale, infinities and NaN."""
    say(f"[ckpt] special tiles {fmt}")
    top = plain64.TOP[fmt]
    x = torch.zeros(12, 256)
    x[1, 3] = -0.0
    x[2, :4] = torch.tensor([1e-45, -3e-45, 1e-40, 5e-39])
    x[3, :3] = torch.tensor([3.4028234663852886e38, -1e38, 1.0])
    x[4] = torch.arange(256) * 0.5 - 64.0
    x[5, 0] = top
    x[6, 0] = float(np.nextafter(np.float32(top), np.float32(1e9)))
    x[7, 0] = float(np.nextafter(np.float32(top), np.float32(0)))
    x[8, 5], x[8, 140] = float("inf"), 2.0
    x[9, 200], x[9, 1] = float("nan"), 3.0
    x[10, 130] = -float("inf")
    x[11] = 2.0**-130 * torch.arange(256)
    codes, scales = pack(x.cuda(), fmt)
    with np.errstate(invalid="ignore"):
        u, byte = plain64.pack(f64(x), fmt)
    assert np.array_equal(scales.cpu().numpy(), byte)
    ok = np.repeat(byte != 255, 128, axis=1)
    assert np.array_equal(code_values(codes, fmt)[ok], u[ok])
    got = f64(unpack(codes, scales, fmt, torch.float32))
    with np.errstate(over="ignore"):
        want = plain64.unpack(u, byte).astype(np.float32).astype(np.float64)
    assert np.array_equal(np.isnan(got), ~ok)
    assert np.array_equal(got[ok], want[ok])


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
def test_every_code_and_scale_byte_unpacks(fmt):
    say(f"[ckpt] all codes {fmt}")
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1).cuda()
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 2).cuda()
    got = f64(unpack(codes, scales, fmt, torch.float32))
    with np.errstate(over="ignore"):
        want = (code_values(codes, fmt) * np.where(np.arange(256) == 255, np.nan, 2.0 ** (np.arange(256.0) - 127))[:, None])
        want = want.astype(np.float32).astype(np.float64)
    assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("cols,ld,first", [(100, 131, 3), (128, 136, 8), (256, 520, 4), (1000, 1001, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_rows(cols, ld, first, dtype):
    """Rows inside wider ones, at addresses of any alignment; what lies between them stays."""
    say(f"[ckpt] strided {cols} in {ld} from {first} {dtype}")
    rows = 21
    wide = torch.randn(rows, ld, generator=torch.Generator().manual_seed(cols)).to(TYPES[dtype]).cuda()
    x = torch.as_strided(wide, (rows, cols), (ld, 1), first) if first + cols <= ld else wide[:, :cols]
    codes, scales = pack(x, "e4m3")
    ref_c, ref_s = pack(x.contiguous(), "e4m3")
    assert torch.equal(codes, ref_c) and torch.equal(scales, ref_s)
    out = torch.full((rows, ld), -7.0, dtype=TYPES[dtype], device="cuda")
    view = torch.as_strided(out, x.shape, (ld, 1), x.storage_offset())
    _lib.moe_checkpoint_unpack(codes, scales, "e4m3", view)
    assert torch.equal(view, unpack(codes, scales, "e4m3", TYPES[dtype]))
    view.fill_(-7.0)
    assert (out == -7).all()


def test_past_32_bit_offsets():
    rows, cols = 70001, 32768  # 2.3e9 values
    say(f"[ckpt] {rows}x{cols}")
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    x.normal_()
    codes, scales = pack(x, "i8")
    back = unpack(codes, scales, "i8", torch.bfloat16)
    for r in (0, 65535, 65536, rows - 1):
        u, byte = plain64.pack(f64(x[r:r + 1]), "i8")
        assert np.array_equal(f64(back[r:r + 1]), plain64.unpack(u, byte))


# ---------------------------------------------------------------- the combine's gradient

def combine_inputs(T, d, fmt, seed):
    g = torch.Generator().manual_seed(seed)
    y = torch.randn(T * 8, d, generator=g).bfloat16().cuda()
    if fmt == "bf16":
        s, vals = (y, None), y.double()
    else:
        s = pack(y, fmt)
        vals = unpack(*s, fmt, torch.float32).double()
    row_of = torch.randperm(T * 8, generator=g).to(torch.int32).cuda()
    w = (torch.rand(T, 8, generator=g) + 0.1).cuda()
    dy = torch.randn(T, d, generator=g).cuda()
    return s, vals, row_of, w, dy


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("T,d", [(1, 64), (5, 192), (3, 7168), (33, 320), (257, 1024), (1000, 2048), (70, 4096)])
def test_combine_backward(T, d, fmt):
    say(f"[combine-grad] T={T} d={d} {fmt}")
    s, vals, row_of, w, dy = combine_inputs(T, d, fmt, T + d)
    gone = [0, T * 8 - 1] if T > 1 else [3]
    kept = row_of.clone()
    row_of[gone] = torch.tensor([-1, T * 8][:len(gone)], dtype=torch.int32, device="cuda")
    dyp = torch.full((T * 8, d), -7.0, dtype=torch.bfloat16, device="cuda")
    dg = torch.full((T, 8), -7.0, device="cuda")
    ds = _lib.desc(T, d, 256, 8, 128) if d % 128 == 0 else _lib.desc(T, d, 256, 8, 128, "f32", "f32")
    saved = _lib.saved(s[0], s[1], fmt)
    _lib.moe_combine_backward(ds, dy, saved, row_of, w, dyp, dg)
    prod = vals[kept.long()].view(T, 8, d) * dy.double()[:, None, :]
    ref, size = prod.sum(2), prod.abs().sum(2)
    want = torch.empty_like(dyp)
    want[kept.long()] = (w[:, :, None] * dy[:, None, :]).view(T * 8, d).bfloat16()
    for i in gone:
        ref.view(-1)[i] = 0
        want[kept[i].long()] = -7.0
    # d/64 additions in a lane and 6 across, one rounding per product: all relative to the sum of magnitudes
    assert ((dg.double() - ref).abs() <= (d / 64 + 8) * plain64.EPS32 * size).all()
    assert torch.equal(dyp, want)


@pytest.mark.parametrize("T,d", [(3, 64), (1101, 320), (77, 2112)])
@pytest.mark.parametrize("fmt", ["e4m3", "i8", "bf16"])
def test_combine_backward_takes_half_a_tile_with_any_types(T, d, fmt):
    """d of 64 more than a multiple of 128, which the products with bf16 weights refuse: as with fp32 ones."""
    say(f"[combine-grad] T={T} d={d} {fmt}, both pairs of types")
    s, _, row_of, w, dy = combine_inputs(T, d, fmt, T + d)
    got = []
    for types in ("f32", "bf16"):
        dyp = torch.full((T * 8, d), -7.0, dtype=torch.bfloat16, device="cuda")
        dg = torch.full((T, 8), -7.0, device="cuda")
        _lib.moe_combine_backward(_lib.desc(T, d, 256, 8, 128, types, types), dy, _lib.saved(s[0], s[1], fmt), row_of, w,
                                  dyp, dg)
        got.append((dyp, dg))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert (got[1][1] != -7).all()


def test_combine_backward_past_32_bit_offsets():
    T, d = 270_001, 1024  # 2.2e9 routed values
    say(f"[combine-grad] T={T} d={d}")
    codes = torch.randint(0, 255, (T * 8, d), dtype=torch.uint8, device="cuda")
    scales = torch.full((T * 8, d // 128), 120, dtype=torch.uint8, device="cuda")
    row_of = torch.arange(T * 8 - 1, -1, -1, dtype=torch.int32, device="cuda")  # the first token's rows last
    w, dy = torch.rand(T, 8, device="cuda"), torch.randn(T, d, device="cuda")
    dyp = torch.empty(T * 8, d, dtype=torch.bfloat16, device="cuda")
    dg = torch.empty(T, 8, device="cuda")
    _lib.moe_combine_backward(_lib.desc(T, d, 256, 8, 128), dy, _lib.saved(codes, scales, "i8"), row_of, w, dyp, dg)
    for t in (0, 1, T // 2, T - 1):
        rows = row_of[8 * t:8 * t + 8].long()
        y = codes[rows].view(torch.int8).double() * 2.0**-7
        prod = y * dy[t].double()
        assert ((dg[t].double() - prod.sum(1)).abs() <= (d / 64 + 8) * plain64.EPS32 * prod.abs().sum(1)).all()
        assert torch.equal(dyp[rows], (w[t][:, None] * dy[t]).bfloat16())


# ---------------------------------------------------------------- the layer's backward

def layer_case(wt, T=600, d=256, I=256, seed=3):
    cfg = synth.CONFIGS[2].with_(name=f"saved {wt}", T=T, d=d, I=I, wt=wt, seed=seed)
    inp = synth.make_inputs(cfg)
    layer = layer_from_inputs(inp)
    x, b = upload(inp["x"]), upload(inp["bias"])
    layer.forward(x, b)
    return layer, x, b


def grads_of(layer, router=True):
    T, d, I, E = layer.T, layer.d, layer.I, layer.E
    shapes = dict(dx=(T, d), dw_router=(E, d), dw_gate=(E, I, d), dw_up=(E, I, d), dw_down=(E, d, I), ds_gate=(I, d),
                  ds_up=(I, d), ds_down=(d, I), dg=(T, 8))
    if not router:
        del shapes["dw_router"]
    return {n: torch.full(s, float("nan"), device="cuda") for n, s in shapes.items()}


def backward(layer, x, y_perm, dy, router=True, plain=False):
    g = grads_of(layer, router)
    args = (layer.wr if router else None, layer.idx if router else None, layer.w, layer.offsets, layer.row_src,
            layer.row_of, layer.ex_w, layer.sh_w)
    stage = _lib.MOE_WS_BACKWARD if plain else _lib.MOE_WS_BACKWARD_SAVED
    ws = torch.full((_lib.workspace_bytes(layer.desc, stage),), 0xFF, dtype=torch.uint8, device="cuda")
    (_lib.moe_backward if plain else _lib.moe_backward_saved)(layer.desc, x, *args, y_perm, dy, g, ws)
    torch.cuda.synchronize()
    return g


@pytest.mark.parametrize("wt", ["bf16", "e4m3"])
def test_backward_saved(wt):
    """bf16 activations: moe_backward bit for bit.  8-bit ones: moe_backward of the values that they stand for
    (dg and what follows from it to the rounding of its sum)."""
    say(f"[backward-saved] {wt}")
    layer, x, _ = layer_case(wt)
    T, d = layer.T, layer.d
    dy = torch.randn(T, d, generator=torch.Generator().manual_seed(4)).cuda()
    ref = backward(layer, x, layer.y_perm, dy, plain=True)
    got = backward(layer, _lib.saved(x), _lib.saved(layer.y_perm), dy)
    for n in ref:
        assert torch.equal(ref[n], got[n]), n
    for fmt in ("e4m3", "i8"):
        say(f"[backward-saved] {wt} {fmt}")
        xs, ys = pack(x.view(torch.bfloat16), fmt), pack(layer.y_perm.view(torch.bfloat16), fmt)
        xv, yv = unpack(*xs, fmt, torch.bfloat16), unpack(*ys, fmt, torch.bfloat16)
        ref = backward(layer, xv, yv, dy, plain=True)
        got = backward(layer, _lib.saved(*xs, fmt), _lib.saved(*ys, fmt), dy)
        size = (yv.double()[layer.row_of.long()].view(T, 8, d) * dy.double()[:, None]).abs().sum(2)
        # both sides of the comparison are sums in some order
        assert ((ref["dg"] - got["dg"]).abs() <= 2 * (d / 64 + 8) * plain64.EPS32 * size).all()
        for n in ref:
            if n in ("dg", "dx", "dw_router"):  # the last two hold the router's share, linear in dg
                assert float((ref[n] - got[n]).norm()) <= 1e-5 * float(ref[n].norm()), n
            else:
                assert torch.equal(ref[n], got[n]), n


@pytest.mark.parametrize("wt", ["bf16", "e4m3"])
def test_a_training_step_routed_from_logits(wt):
    """Logits, choice, experts, combine, checkpoints, backward without the fused router, the choice's and the
    projection's gradients: where the rule is the fused router's, its gradients."""
    say(f"[train] from logits {wt}")
    layer, x, bias = layer_case(wt)
    T, d = layer.T, layer.d
    sel = _lib.selection(T, 256, 8)
    logits = torch.empty(T, 256, device="cuda")
    ws = torch.empty(_lib.workspace_bytes(layer.desc, _lib.MOE_WS_ROUTER_LOGITS), dtype=torch.uint8, device="cuda")
    _lib.moe_router_logits(layer.desc, x, layer.wr, logits, ws)
    idx, w = torch.empty_like(layer.idx), torch.empty_like(layer.w)
    _lib.moe_select(sel, logits, bias, idx, w)
    assert torch.equal(idx, layer.idx)
    assert torch.allclose(w, layer.w, rtol=1e-6)
    dy = torch.randn(T, d, generator=torch.Generator().manual_seed(4)).cuda()
    fused = backward(layer, x, layer.y_perm, dy, plain=True)
    g = backward(layer, _lib.saved(x), _lib.saved(layer.y_perm), dy, router=False)
    assert torch.equal(g["dg"], fused["dg"]) and torch.equal(g["dw_gate"], fused["dw_gate"])
    dl = torch.empty(T, 256, device="cuda")
    _lib.moe_select_backward(sel, logits, idx, g["dg"], dl)
    dwr = torch.empty(256, d, device="cuda")
    ws = torch.empty(max(1, _lib.workspace_bytes(layer.desc, _lib.MOE_WS_ROUTER_GRAD)), dtype=torch.uint8, device="cuda")
    _lib.moe_router_logits_backward(layer.desc, x, layer.wr, dl, g["dx"], g["dx"], dwr, ws)
    for a, b in ((g["dx"], fused["dx"]), (dwr, fused["dw_router"])):
        assert float((a - b).norm()) <= 1e-5 * float(b.norm())
