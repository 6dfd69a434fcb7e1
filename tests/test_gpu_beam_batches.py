"""q4 attention of batches whose longest prefix and longest own part belong to different groups."""
import numpy as np
import pytest
import torch

from _beam_raw import TYPE
from _gpu_util import i32
from test_gpu_beam_attn import Cache, _call, _check, _q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,beams", [(64, 2), (128, 1), (256, 3)])
@pytest.mark.parametrize("exact", [False, True])
def test_long_prefix_beside_long_own_part(kvq, cuda_dev, D, beams, exact):
    """A table of as many entries as the longest sequence has pages."""
    shared = [900, 0, 17]
    lens = [shared[g] + own for g, own in enumerate((28, 928, 300)) for _ in range(beams)]
    c = Cache(kvq, cuda_dev, D, 2, 16, beams, shared, lens, seed=D)
    width = 928 // 16
    c.table = c.table[:, :width].contiguous()
    q = _q(cuda_dev, (1, len(lens), 8, D), "f16")
    bounds = dict(max_own=928) if exact else dict(max_shared=928, max_own=928)
    out, err = _call(kvq, cuda_dev, [c], q, D ** -0.5, **bounds)
    assert err == 0
    _check(out[0], c, q[0], D ** -0.5, "f16")


@pytest.mark.parametrize("beams", [1, 2])
def test_sequences_longer_than_their_row_of_the_table(kvq, cuda_dev, beams):
    """Bounds that reach beyond the table do not: such a group gets 0 and the error word its bit."""
    lens = [100] * beams + [60] * beams
    c = Cache(kvq, cuda_dev, 64, 1, 16, beams, [50, 20], lens)
    c.table = c.table[:, :6].contiguous()            # 96 tokens
    q = _q(cuda_dev, (1, len(lens), 4, 64), "f16")
    out, err = _call(kvq, cuda_dev, [c], q, 0.125, max_shared=96, max_own=96)
    assert err == kvq.KVQ_DEVERR_INDEX and (out[0, :beams] == 0).all()
    ok, err = _call(kvq, cuda_dev, [c], q, 0.125, lens=[96] * beams + [60] * beams, max_shared=50, max_own=46)
    assert err == 0 and torch.equal(out[0, beams:], ok[0, beams:])
