"""8-bit checkpoints of the widest rows."""
import pytest
import torch

from sparse_expert_routing_amd import _lib
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    _lib.load()


def there_and_back(x, fmt):
    codes = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
    scales = torch.empty(x.shape[0], -(-x.shape[1] // 128), dtype=torch.uint8, device="cuda")
    back = torch.full_like(x, -7.0)
    _lib.moe_checkpoint_pack(x, codes, scales, fmt)
    _lib.moe_checkpoint_unpack(codes, scales, fmt, back)
    return codes, scales, back


@pytest.mark.parametrize("cols", [(1 << 31) - 1, (1 << 31) - 8, (1 << 31) - 128])
def test_rows_as_wide_as_their_index(cols):
    """The first, a middle and the last tiles as a call of their own has them."""
    say(f"[ckpt-edges] 1x{cols}")
    x = torch.empty(1, cols, dtype=torch.bfloat16, device="cuda").normal_()
    codes, scales, back = there_and_back(x, "e4m3")
    last = (cols - 1) // 128 * 128
    for a, b in ((0, 1000 * 128), ((1 << 30) - 1280, (1 << 30) + 1280), (last - 1280, cols)):
        c, s, v = there_and_back(x[:, a:b].clone(), "e4m3")
        assert torch.equal(codes[:, a:b], c) and torch.equal(back[:, a:b], v)
        assert torch.equal(scales[:, a // 128:-(-b // 128)], s)
