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
