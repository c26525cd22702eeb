"""The AdamW step: a step number and a rate on the device element by element against the host's,
and what many steps make of second moments in 8 bits."""
import numpy as np
import pytest
import torch

from tests import mx64
from tests.gpu_util import say
from tests.test_gpu_adamw import make, read, table

pytestmark = pytest.mark.gpu
U = mx64.EPS32


@pytest.mark.parametrize("step", [1, 2, 3, 10, 1000, 100000, 2**40])
@pytest.mark.parametrize("betas", [(0.9, 0.999), (0.0, 0.0), (0.99, 0.9999)])
def test_numbers_on_the_device_and_on_the_host(step, betas):
    """m and v are equal.  The weights may differ by the update's error: each bias correction by a step of fp32 (2 u; its
    fp64 values round to neighbours at most), and behind them the product with m, the product with the root and the sum with
    eps (1 u each on either side: 6), the reciprocal (2 u on either side: 4), its product and lr's (4): 18 u of the update;
    and by the two last roundings of the weight, 1 u each."""
    import sparse_expert_routing_amd as moe
    say("[adamw] numbers on the device", step, betas)
    rng = np.random.default_rng(step % 1000)
    n, lr, eps, decay = 3000, 1e-3, 1e-8, 0.01
    a = make(rng, n, "f32", "f32", 32, False)
    b = {k: t.clone() if t is not None else None for k, t in a.items()}
    before = read(a, n, 32)
    rule = dict(betas=betas, eps=eps, weight_decay=decay)
    moe.moe_adamw(table([a], [n], 32), lr=lr, step=step, **rule)
    moe.moe_adamw(table([b], [n], 32), lr=torch.tensor([lr], device="cuda"), step=torch.tensor([step], device="cuda"), **rule)
    assert torch.equal(a["m"], b["m"]) and torch.equal(a["v"], b["v"])
    want, m, v = mx64.adamw(before["w"], before["g"], before["m"], before["v"], lr, betas, eps, decay, step)
    update = lr * np.abs(m) / (1 - betas[0] ** step) / (np.sqrt(v / (1 - betas[1] ** step)) + eps)
    x, y = (t["w"][:n].double().cpu().numpy() for t in (a, b))
    # (m and v carry errors of their own, 5 u of their terms, equal on both sides: the update's size is theirs to 2^-10 where
    # the terms do not cancel, and no more than the terms' sum where they do)
    terms = np.abs(betas[0] * before["m"]) + np.abs((1 - betas[0]) * before["g"])
    update = np.maximum(update, 5 * U * terms / np.maximum(np.abs(m), 1e-300) * update) * (1 + 2.0**-10)
    tol = 18 * U * update + 2 * U * np.maximum(np.abs(x), np.abs(y))
    assert np.all(np.abs(x - y) <= tol), float((np.abs(x - y) / tol).max())


@pytest.mark.parametrize("b2", [0.999, 0.95])
@pytest.mark.parametrize("kind", ["ones", "normal"])
def test_spread_of_the_roots_of_8_bit_second_moments(kind, b2):
    """600 steps.  The root is rounded without bias, to steps of 1/16 to 1/8 of it.  A step moves it by (1 - b2) / 2 of itself
    times d = |1 - g^2 / v|, so its rounding adds a variance of (1 - b2) / 2 d / 8 at most, of the root's square, of which what
    is 1 / (1 - b2) steps old is forgotten: in all d / 32 at most, with d at 1 or less in the mean (normal gradients: 0.97,
    gradients of 1: the spread itself), a deviation of 0.18.  The mean root is right to half the variance and to the
    deviation of 4096 of them: 2 %; the mean square is up by the variance, 3 % at most, and the same deviation twice."""
    import sparse_expert_routing_amd as moe
    say("[adamw] spread of roots", kind, b2)
    n, steps = 4096, 600
    rng = np.random.default_rng(7)
    w = torch.zeros(n, device="cuda")
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    s = [torch.full((n // 128,), 127, dtype=torch.uint8, device="cuda") for _ in range(2)]
    g = torch.ones(n, device="cuda")
    tab = moe.adamw_tensors([w], [g], [m], [v], m_scales=[s[0]], v_scales=[s[1]])
    exact = np.zeros(n)
    for step in range(1, steps + 1):
        if kind == "normal":
            g.copy_(torch.from_numpy(rng.standard_normal(n)).float())
        exact = b2 * exact + (1 - b2) * g.double().cpu().numpy() ** 2
        moe.moe_adamw(tab, lr=1e-4, betas=(0.9, b2), step=step, seed=3)
    root = mx64.grid_values(v.cpu().numpy(), "e4m3") * np.repeat(mx64.scale_value(s[1].cpu().numpy()), 128)
    q = root / np.sqrt(exact)
    say(f"[adamw] roots {kind} {b2}: mean {q.mean():.4f}, deviation {q.std():.4f}, mean square {(root**2).mean() / exact.mean():.4f}")
    assert abs(q.mean() - 1) <= 0.02
    assert q.std() <= 0.18
    assert abs((root**2).mean() / exact.mean() - 1) <= 0.04
