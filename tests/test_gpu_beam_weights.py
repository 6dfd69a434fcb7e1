"""q4 attention where weights times V's scales span many magnitudes: one token that has nearly all of the
weight before tens of thousands of others, values of small and of mixed scales.  Values are of one sign, so
that what is rounded away is not averaged out."""
import numpy as np
import pytest
import torch

from _beam_raw import Raw, TYPE, tolerance

pytestmark = pytest.mark.gpu


def _group(r, D, n, v_scales, dominant=None):
    """Keys of code 0 (score 0) but the dominant one's; value codes 1 .. 7."""
    kc = np.zeros((n, D), np.int64)
    if dominant is not None:
        kc[dominant] = 1
    return kc, np.ones(n), r.integers(1, 8, (n, D)), v_scales


def _check(c, q, scale, kind, got, only=None):
    for s in range(len(c.lens)) if only is None else only:
        o, size, score, top = c.reference(q, scale, s)
        v_most = np.abs(c.rows[s // c.beams][1]).max()
        tol = tolerance(c.lens[s], o, size, score, top, v_most, kind)
        off = np.abs(got[s].double().cpu().numpy() - o)
        assert (off <= tol).all(), (s, (off / tol).max())


def _q(dev, n, heads, D, kind, seed=0):
    """Rows of one power of two each: 1, 1/2, 1/4 and 0."""
    f = torch.tensor([1.0, 0.5, 0.25, 0.0]).repeat(heads)[:heads]
    return f[None, :, None].expand(n, heads, D).to(TYPE[kind]).contiguous().to(dev)


@pytest.mark.parametrize("D,beams,heads", [(64, 1, 4), (128, 1, 4), (256, 1, 4), (64, 3, 8), (128, 4, 4),
                                           (256, 3, 6)])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("n,weight,lo,hi,sink", [(32768, 0.99, 0.05, 0.1, 1.0), (32768, 0.99, 0.05, 0.1, 0.0),
                                                 (50001, 0.5, 0.004, 0.004, 1.0), (40000, 0.9, 0.005, 0.02, 50.0),
                                                 (3001, 0.999, 0.0001, 0.0002, 1.0)])
def test_one_token_has_the_weight(kvq, cuda_dev, D, beams, heads, kind, n, weight, lo, hi, sink):
    """`sink`: the dominant token's scale of V over the others' (0: its values are 0)."""
    r = np.random.default_rng(n + D)
    at = int(r.integers(n))
    vs = r.uniform(lo, hi, n)
    vs[at] *= sink
    c = Raw(kvq, cuda_dev, [_group(r, D, n, vs, at)], beams, seed=D)
    scale = float(np.float32(np.log(weight / (1 - weight) * (n - 1)) / D))
    q = _q(cuda_dev, beams, heads, D, kind)
    got, err = c.call(q, scale, [n] if beams > 1 else None)
    assert err == 0
    _check(c, q, scale, kind, got)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("beams", [1, 4])
@pytest.mark.parametrize("v_scale", [1e-4, 1e-5, 1e-6, 6e-8])
def test_small_values(kvq, cuda_dev, D, beams, v_scale):
    r = np.random.default_rng(D)
    n = 8192
    c = Raw(kvq, cuda_dev, [_group(r, D, n, np.full(n, v_scale), 77), _group(r, D, 100, np.full(100, v_scale))],
            beams, seed=D)
    q = _q(cuda_dev, 2 * beams, 4, D, "bf16")
    got, err = c.call(q, 4 / D, [n, 100] if beams > 1 else None)
    assert err == 0
    _check(c, q, 4 / D, "bf16", got)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("beams", [1, 3])
def test_values_of_all_magnitudes(kvq, cuda_dev, D, beams):
    """Scales of V from 2^-24 to 2^15 in any order, with scores that rise by 30 along the tokens."""
    r = np.random.default_rng(D)
    groups = []
    for n in (5000, 700, 33):
        vs = 2.0 ** r.integers(-24, 16, n)
        for order in (slice(None), np.argsort(vs), np.argsort(-vs)):
            kc = np.ones((n, D), np.int64)
            groups.append((kc, np.linspace(0, 1, n), r.integers(1, 8, (n, D)), vs[order]))
    c = Raw(kvq, cuda_dev, groups, beams, seed=D)
    q = _q(cuda_dev, len(c.lens), 4, D, "bf16")
    got, err = c.call(q, 30 / D, [len(g[0]) for g in groups] if beams > 1 else None)
    assert err == 0
    _check(c, q, 30 / D, "bf16", got)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_small_values_of_many_short_sequences(kvq, cuda_dev, D):
    """So many short ones that each is a warp's."""
    r = np.random.default_rng(D)
    groups = [_group(r, D, n, np.full(n, 2.0 ** -int(r.integers(0, 25))), 0) for n in r.integers(1, 100, 420)]
    c = Raw(kvq, cuda_dev, groups, seed=D)
    q = _q(cuda_dev, 420, 4, D, "bf16")
    got, err = c.call(q, 12 / D)
    assert err == 0
    _check(c, q, 12 / D, "bf16", got, range(0, 420, 7))
