"""q4 attention of scores far below 0: the softmax is that of their differences, however far they are."""
import numpy as np
import pytest
import torch

from _beam_raw import Raw, TYPE

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("beams", [1, 3])
@pytest.mark.parametrize("scale,kind,size", [(1e30, "f16", 1.0), (3e34, "f16", 1.0), (0.125, "bf16", 2.0 ** 98)])
def test_only_scores_far_below_zero(kvq, cuda_dev, D, beams, scale, kind, size):
    """Every score is below -1e30; the largest one has all the weight, two of them half each."""
    n, best = 300, [41, 250]
    kc = np.full((n, D), -7)
    kc[best] = -3
    r = np.random.default_rng(D)
    c = Raw(kvq, cuda_dev, [(kc, np.ones(n), r.integers(-7, 8, (n, D)), np.ones(n))], beams)
    q = torch.full((beams, 4, D), size, dtype=TYPE[kind], device=cuda_dev)
    got, err = c.call(q, scale, [n] if beams > 1 else None)
    assert err == 0
    want = c.rows[0][1][best].mean(0)            # halves of whole numbers: exact in either type
    assert (got.double().cpu().numpy() == want).all()


@pytest.mark.parametrize("D,beams", [(64, 1), (128, 4), (256, 3)])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_whose_neighbours_are_far_apart(kvq, cuda_dev, D, beams, sign):
    """Scores of 2^20 to 2^31 that rise by a float32 step or two: what is rounded there decides weights, but
    results stay between the smallest and the largest value, whatever V's scale is."""
    n = 700
    r = np.random.default_rng(D)
    kc = np.zeros((n, D), np.int64)
    kc[:, 0], kc[:, 2] = 7, np.arange(n) * 15 // n - 7
    q = torch.zeros((beams, 4, D))
    q[..., 0], q[..., 2] = sign, torch.tensor([2.0 ** -20, 2.0 ** -19, 2.0 ** -17, 2.0 ** -21])
    q = q.to(torch.bfloat16).to(cuda_dev)
    for power in (-24, -5, -1, 0, 3, 6, 9, 12, 15):
        vc = r.integers(1, 8, (n, D))
        v_scale = 2.0 ** power
        c = Raw(kvq, cuda_dev, [(kc, np.ones(n), vc, np.full(n, v_scale))], beams, seed=D)
        for k in range(20, 32):
            for m in (1.0, 1.3, 1.7):
                got, err = c.call(q, 2.0 ** k * m / 7, [n] if beams > 1 else None)
                assert err == 0
                got = got.double() / v_scale
                assert (got >= 1 - 2.0 ** -7).all() and (got <= 7 * (1 + 2.0 ** -7)).all(), (power, k, m)
