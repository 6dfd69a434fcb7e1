"""Selection at the largest vocabulary that a call may have: places in the row up to the end of 31 bits."""
import numpy as np
import pytest
import torch

from test_gpu_beam_select import TYPES, _call

pytestmark = pytest.mark.gpu

V = 2 ** 31 - 1 - 65536


@pytest.mark.parametrize("dtype,beams", [("bf16", 1), ("bf16", 2), ("f16", 4), ("f32", 3)])
def test_largest_vocabulary(kvq, cuda_dev, dtype, beams):
    """Rows of -20 with some larger logits: at both ends, and around a border of the slices.

    The sum's terms are equal: each is 2^-22 and 2 |x - max| 2^-24 off, |x - max| < 27, and so is the sum."""
    x = torch.full((beams, V), -20.0, dtype=TYPES[dtype], device=cuda_dev)
    at = [0, 1, 4095, 4096, V // 129, V // 2, V - 65536, V - 4097, V - 2, V - 1]
    for b in range(beams):
        for i, token in enumerate(at):
            x[b, token] = (i * 7 + b) % 10 * 0.5 + 1
    s = torch.tensor([[-0.03125 * b for b in range(beams)]], device=cuda_dev)    # no two t are equal
    v, par, tok = _call(kvq, cuda_dev, x, s, 10)
    del x
    want = []
    for b in range(beams):
        big = np.array([(i * 7 + b) % 10 * 0.5 + 1 for i in range(len(at))])
        lse = np.log((V - len(at)) * np.exp(-20.0) + np.exp(big).sum())
        want += [(float(g - lse - 0.03125 * b), b, token) for g, token in zip(big, at)]
    want = sorted(want, key=lambda w: (-w[0], w[1], w[2]))[:10]
    assert par[0].tolist() == [w[1] for w in want] and tok[0].tolist() == [w[2] for w in want]
    assert np.abs(v[0] - [w[0] for w in want]).max() < 2.0 ** -22 + 54 * 2.0 ** -24 + 2.0 ** -20
    with pytest.raises(kvq.KVQError):
        kvq._check(kvq._lib.kvq_beam_select(kvq.KVQ_BF16, 1 << 20, V + 1, 1 << 20, 1, 1, V + 1, 1, 1 << 20,
                                            1 << 20, 1 << 20, 1 << 20, 1 << 40, None))
