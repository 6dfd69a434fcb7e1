"""The log-sum of exponentials of selection's rows against float64, row by row, at the accuracy that its steps
have.  A beam's score is chosen so that t is near 0, where float32 shows some 1e-9.

Relative to the sum: a term's exponential is 2^-22 off, its argument d = x - max has two roundings (of the
difference and of the product with log2 e, 2^-24 |d| each); 32 terms are added in float32 in 6 steps, the
rest in pairs of floats and in float64.  A thread that meets a larger logit than before scales its sum (2^-22,
2^-23 of the rise, half a step), at most once a batch of 32 elements, and twice when the block ends."""
import numpy as np
import pytest
import torch

from test_gpu_beam_select import TYPES, _call

pytestmark = pytest.mark.gpu


def _rows(kind, V):
    g = torch.Generator().manual_seed(V)
    i = torch.arange(V, dtype=torch.float32)
    if kind == "one above many":
        x = torch.full((V,), -11.21875)
        x[3] = 0
    elif kind == "two levels":
        x = torch.where(i % 2 == 0, -5.6875, -5.75)
        x[1] = 0
    elif kind == "ordinary":
        x = torch.randn(V, generator=g) * 2.5
    elif kind == "near":
        x = torch.randn(V, generator=g) * 0.01 + 7
    elif kind == "rising":
        x = i * (8.0 / V)
    else:
        x = torch.full((V,), -23.1)
        x[V // 2:] = -22.7
    return x


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("kind", ["one above many", "two levels", "ordinary", "near", "rising", "far below 0"])
@pytest.mark.parametrize("V", [5000, 131072, 1000003])
def test_sums(kvq, cuda_dev, dtype, kind, V):
    x = _rows(kind, V).to(TYPES[dtype])
    xd = x.double().numpy()
    most = xd.max()
    e = np.exp(xd - most)
    lse = most + np.log(e.sum())
    score = np.float32(lse - most)
    batch = 8192 if dtype == "f32" else 16384            # elements of a block's batch
    rises = int((np.diff(np.maximum.accumulate(xd[::2048])) > 0).any()) * (V // batch + 1)
    bound = ((e * (2.0 ** -22 + (most - xd) * 2.0 ** -23)).sum() / e.sum() + 6 * 2.0 ** -24
             + (rises + 2) * 2.0 ** -22 + (most - xd.min()) * 2.0 ** -23 * (rises > 0) + 2.0 ** -30)
    s = torch.full((1, 1), float(score), device=cuda_dev)
    v, _, _ = _call(kvq, cuda_dev, x[None].to(cuda_dev), s, 1)
    off = abs(float(v[0, 0]) - (most - lse + float(score)))
    assert off <= bound
    if V <= 131072:
        assert bound < 2.0 ** -16                       # what the header states
