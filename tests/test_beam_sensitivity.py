"""The q4 attention checks over distinguishable tiles see one that is lost, repeated or misread, a lost token,
and scores that are off (CPU, oracle only).

The oracle's result over the tests' own data is compared, with their tolerance, against its result with the
mistake in its input.  Mistakes are made on the CPU, never in a kernel."""
import numpy as np
import pytest

from oracle import beams as ob
from oracle import prompt as op
from _beam_raw import pack, tiles, tolerance


def _rows(D, n):
    kc, ks, vc, vs = tiles(D, n, D)
    return [ob.q4_rows(pack(c), np.asarray(s, np.float16)) for c, s in ((kc, ks), (vc, vs))]


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("D,n", [(64, 20011), (128, 20011), (256, 60013), (256, 9001)])
def test_mistakes_are_outside_the_tolerance(D, n, kind):
    k, v = _rows(D, n)
    q = np.ones((1, D))
    seen = np.ones((1, n), bool)

    def attend(k, v, seen=seen, scale=1 / D):
        return op.attend(q, k, v, seen, scale)

    o, _, size, _ = attend(k, v)
    x = k @ q[0] / D
    tol = tolerance(n, o, size, np.abs(x).max()[None], 1 / np.exp(x - x.max()).sum()[None], 1.75, kind)
    outside = lambda other: (np.abs(other - o) / tol).max()
    tiles_of = -(-n // 16)
    for tile in (0, 1, 7, 8, tiles_of // 3, tiles_of // 2, tiles_of - 2):
        lost = seen.copy()
        lost[0, 16 * tile:16 * tile + 16] = False
        assert outside(attend(k, v, lost)[0]) > 2, ("lost", tile)
        token = seen.copy()
        token[0, 16 * tile + 5] = False
        assert kind == "bf16" or n > 30000 or outside(attend(k, v, token)[0]) > 1, ("a token", tile)
        at = np.arange(n)
        at[16 * tile:16 * tile + 16] += 16 if tile < tiles_of - 2 else -16
        assert outside(attend(k, v[at])[0]) > 2, ("the next tile's values", tile)
        assert outside(attend(k[at], v)[0]) > 1 or (x[at] == x).all(), ("the next tile's keys", tile)
    for factor in (0.97, 1.03):
        assert outside(attend(k, v, scale=factor / D)[0]) > 2, ("scores", factor)
    assert outside(o * (1 + (0.01 if kind == "bf16" else 0.003))) > 1
