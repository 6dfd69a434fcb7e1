"""The order of selection within a beam is that of its logits, also where their t are one number in 64 bits."""
import numpy as np
import pytest
import torch

from test_gpu_beam_select import TYPES, _call

pytestmark = pytest.mark.gpu


def _best(row, k):
    """Tokens of the k largest logits, equal ones by token."""
    return np.argsort(-row.double().cpu().numpy(), kind="stable")[:k]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("score", [-1e30, float(np.finfo(np.float32).min), 1e35])
@pytest.mark.parametrize("V,k", [(300, 4), (70001, 4), (70001, 40)])
def test_scores_that_swallow_the_logits(kvq, cuda_dev, dtype, score, V, k):
    """All t of such a beam are one number, of equal beams too: beam 0's best logits, in their order."""
    g = torch.Generator().manual_seed(V)
    x = (torch.randn((6, V), generator=g) * 2.5).to(TYPES[dtype]).to(cuda_dev)
    s = torch.full((2, 3), score, device=cuda_dev)
    v, par, tok = _call(kvq, cuda_dev, x, s, k)
    assert (v == np.float32(score)).all()
    for i in range(2):
        assert (par[i] == 3 * i).all() and np.array_equal(tok[i], _best(x[3 * i], k))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logits_nearer_than_their_distance_to_the_sum(kvq, cuda_dev, dtype):
    """Logits of 1e-30 and less: t is the same in 64 bits for all of them."""
    V = 40001
    g = torch.Generator().manual_seed(3)
    x = (torch.rand((4, V), generator=g) * 1e-30).to(TYPES[dtype]).to(cuda_dev)
    s = torch.tensor([[0.0, -1.0], [-2.0, -1.0]], device=cuda_dev)
    v, par, tok = _call(kvq, cuda_dev, x, s, 20)
    for i, b in enumerate((0, 1)):
        assert (par[i] == 2 * i + b).all() and np.array_equal(tok[i], _best(x[2 * i + b], 20))
        assert np.abs(v[i] - (s[i, b].item() - np.log(V))).max() < 1e-5
