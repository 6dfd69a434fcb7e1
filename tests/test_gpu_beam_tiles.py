"""q4 attention with every tile visible: a tile's values lie in a channel of its own or of few others, so that
one lost, read twice or from another place, and scores that are a few per cent off, are far outside the
tolerance (tests/test_beam_sensitivity.py shows that of the oracle)."""
import pytest
import torch

from _beam_raw import Raw, TYPE, tiles, tolerance

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,beams,heads", [(64, 1, 4), (64, 5, 8), (128, 1, 4), (128, 4, 4), (128, 2, 9),
                                           (256, 1, 6), (256, 8, 6)])
@pytest.mark.parametrize("lens,own", [([20011], 1), ([9001, 300, 17], 133), ([60013, 40000], 16),
                                      ([1000 + 37 * i for i in range(40)], 500)])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_every_tile(kvq, cuda_dev, D, beams, heads, lens, own, kind):
    """own: tokens that each sequence of a group reads for itself, at most (all of them without beams)."""
    c = Raw(kvq, cuda_dev, [tiles(D, n, D + i) for i, n in enumerate(lens)], beams, seed=len(lens))
    f = torch.tensor([1.0, 0.5, 0.25, 0.75, -0.5]).repeat(heads)[:heads]
    q = f[None, :, None].expand(len(c.lens), heads, D).to(TYPE[kind]).contiguous().to(cuda_dev)
    shared = [max(0, n - own) for n in lens] if beams > 1 else None
    got, err = c.call(q, 1 / D, shared)
    assert err == 0
    got = got.double().cpu().numpy()
    for s in range(0, len(c.lens), beams):
        o, size, score, top = c.reference(q, 1 / D, s)
        tol = tolerance(c.lens[s], o, size, score, top, 1.75, kind)
        for b in range(s, s + beams):
            assert (abs(got[b] - o) <= tol).all()
