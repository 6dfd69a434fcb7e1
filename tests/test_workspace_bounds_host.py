"""A workspace sized for a program's largest bounds suffices for its smaller calls: the sizes that the
library gives never fall as the bounds grow (no GPU needed)."""
import numpy as np
import pytest


def _bounds(r):
    top = lambda n: int(np.exp(r.uniform(0, np.log(n))))
    return dict(nseq=top(200), total_q=top(70000), max_q=top(40000), max_k=top(300000))


@pytest.mark.parametrize("Hq,H,D", [(24, 4, 256), (16, 4, 128), (32, 8, 64), (6, 6, 256), (5, 1, 64),
                                    (128, 1, 128)])
def test_prompt_workspace_never_falls_as_the_bounds_grow(kvq, Hq, H, D):
    size = lambda b: kvq.kvq_prompt_attn_workspace(b["nseq"], b["total_q"], Hq, H, D, b["max_q"],
                                                   b["max_k"])
    r = np.random.default_rng(D + Hq)
    # at most: two blocks on each of 152 SMs, 128 rows of 128 channels and 4 more floats
    for _ in range(400):
        large = _bounds(r)
        small = {k: int(r.integers(1, v + 1)) for k, v in large.items()}
        assert 16 <= size(small) <= size(large) <= 304 * 128 * 132 * 4, (small, large)
    step = dict(nseq=1, total_q=1, max_q=1, max_k=16384)
    assert size(step) <= size(dict(nseq=1, total_q=16384, max_q=16384, max_k=16384))


def test_tree_workspace_never_falls_as_the_bounds_grow(kvq):
    size = lambda b, H, Hq: kvq.kvq_tree_attn_workspace(b["layers"], b["nseq"], b["total"], H, Hq, 256,
                                                        b["nodes"], b["len"])
    r = np.random.default_rng(3)
    for _ in range(1000):
        H = int(r.integers(1, 9))
        Hq = H * int(r.integers(1, 17))
        nseq = int(r.integers(1, 100))
        large = dict(layers=int(r.integers(1, 65)), nseq=nseq, total=int(r.integers(1, 64 * nseq + 1)),
                     nodes=int(r.integers(1, 65)), len=int(np.exp(r.uniform(0, 13))))
        small = {k: int(r.integers(1, v + 1)) for k, v in large.items()}
        assert 16 <= size(small, H, Hq) <= size(large, H, Hq), (small, large)
