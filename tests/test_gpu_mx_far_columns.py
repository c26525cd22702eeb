"""Products on weights in four bits whose rows are longer than 2^16 bytes: what a tile's rows
past their group compute is stored nowhere, whatever the column."""
import numpy as np
import pytest

from tests import mx64, test_gpu_mx_product as products
from tests.gpu_util import say
from tests.test_gpu_mx_wide import exact_operands

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("N,out", [(16640, "f32"), (20001, "f32"), (33024, "bf16"), (40001, "bf16")])
@pytest.mark.parametrize("G,M", [(3, 40), (3, 150), (2, 300)])  # tiles of 32 rows, of 64, of 256
def test_rows_past_a_group_are_stored_nowhere(G, M, N, out, fmt):
    """Every element of every row equals the sum, which is exact (rounded once); a weight row that is no number shows in its
    own column alone."""
    say("[mx far columns]", G, M, N, out, fmt)
    K = 96
    rng = np.random.default_rng(M + N)
    xc, xs, wc, ws, x, w = exact_operands(rng, G, M, N, K, fmt)
    off = np.linspace(2, M - 3, G + 1).astype(np.int32)
    assert np.all(np.diff(off) % 32 != 0)
    want, _ = products.grouped(x, w, off, M)
    if out == "bf16":
        inside = ~np.isnan(want)
        want[inside] = mx64.bf16_round(want[inside])
    want[: off[0]], want[off[-1] :] = 7.0, 7.0  # rows of no group, as they were
    ws[0, N + N - 9, 1] = 255
    want[off[1] : off[2], N - 9] = np.nan
    got = products.run(xc, xs, fmt, wc, ws, off, M, N, out)
    assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("E,T,k,d,I", [(3, 20, 2, 33024, 32), (2, 300, 1, 32800, 64)])
def test_expert_ffn_of_long_rows(E, T, k, d, I, fmt):
    products.test_expert_ffn(E, T, k, d, I, fmt)
