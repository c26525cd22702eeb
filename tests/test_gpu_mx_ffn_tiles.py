"""The experts' FFN on weights in four bits over more tiles than the card takes at once: several
tiles to a workgroup, at every tile size, in the SwiGLU product too."""
import numpy as np
import pytest
import torch

from tests import mx64, test_gpu_mx_product as products
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("E,M,d,I,some", [(256, 2048, 416, 1024, 32), (64, 3200, 416, 2048, 16), (4, 6000, 608, 4096, 1)])  # 32 rows, 64, 256
def test_all_groups_at_once_as_a_few_at_a_time(E, M, d, I, some, fmt):
    """A tile's result depends on its own rows and weights: the FFN of all groups, 768 and more tiles of gate and up, equals
    bit for bit the FFN of `some` groups at a time, a tile to a workgroup; rows of other groups are left alone."""
    import sparse_expert_routing_amd as moe
    say("[mx ffn tiles]", E, M, d, I, fmt)
    gen = torch.Generator(device="cuda").manual_seed(M)
    rng = np.random.default_rng(M)
    normal = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731

    def packed(rows, cols, f, size):
        codes, scales = moe.mx_empty(rows, cols, f)
        moe.moe_mx_pack(normal(rows, cols) * size, codes, scales, f)
        return codes, scales

    x = moe.mx(*packed(M // 2, d, fmt, 1.0), fmt)
    mats = []
    for r, c in ((I, d), (I, d), (d, I)):
        codes, scales = packed(E * r, c, "e2m1", c**-0.5)
        mats.append(moe.mx(codes.view(E, r, c // 2), scales, "e2m1"))
    # sizes about the average, so that no few groups have more tiles than there are workgroups
    share = rng.uniform(0.6, 1.4, E)
    off = np.concatenate(([0], np.floor(np.cumsum(share) / share.sum() * M))).astype(np.int32)
    off[-1] = M
    src = mx64.cuda(rng.permutation(M).astype(np.int32))
    ws = torch.empty(moe.mx_ffn_workspace_bytes(E, M, d, I, fmt), dtype=torch.uint8, device="cuda")

    def run(offsets):
        ws.fill_(0xFF)
        y = torch.full((M, d), 7.0, dtype=torch.bfloat16, device="cuda")
        moe.moe_mx_expert_ffn(x, *mats, mx64.cuda(offsets), y, ws, row_src=src, k=2)
        return y

    whole = run(off)
    assert bool(torch.isfinite(whole).all())
    rows = 32 if M // E <= 16 else 64 if M // E <= 64 else 256
    tiles = lambda o: int(np.sum(-(-np.diff(o) // rows))) * -(-I // 128)  # noqa: E731
    assert tiles(off) > 2 * (256 if rows == 256 else 512)
    for a in range(0, E, some):
        part = np.clip(off, off[a], off[a + some])
        assert tiles(part) <= (256 if rows == 256 else 512)
        y = run(part)
        assert torch.equal(y[off[a] : off[a + some]], whole[off[a] : off[a + some]]), a
        assert bool((y[: off[a]] == 7).all()) and bool((y[off[a + some] :] == 7).all()), a
    for _ in range(2):
        assert torch.equal(run(off), whole)


@pytest.mark.parametrize("E,T,k,d,I", [(2, 1300, 2, 288, 4608), (40, 60, 8, 96, 1920)])
def test_expert_ffn_of_many_tiles(E, T, k, d, I):
    """Against the definition, e2m1 rows."""
    products.test_expert_ffn(E, T, k, d, I, "e2m1")
