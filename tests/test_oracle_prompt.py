"""The prompt oracle's pins: closed forms and an independent float64 computation."""
import numpy as np
import pytest
import torch

from oracle import attention as oa
from oracle import prompt as op


def _rand(*shape, seed=0):
    return np.random.default_rng(seed).standard_normal(shape)


def test_causal_attention_matches_a_dense_float64_softmax():
    q, k, v = _rand(7, 4, 16, seed=1), _rand(11, 2, 16, seed=2), _rand(11, 2, 16, seed=3)
    r = op.prompt_attention(q, k, v, [0, 7], [0, 11], 0.3)
    tq, tk, tv = (torch.from_numpy(x).transpose(0, 1) for x in (q, k, v))
    s = tq @ tk.repeat_interleave(2, 0).transpose(-1, -2) * 0.3
    mask = torch.ones(7, 11, dtype=torch.bool).tril(4)
    s = s.masked_fill(~mask, -torch.inf)
    o = (s.softmax(-1) @ tv.repeat_interleave(2, 0)).transpose(0, 1).numpy()
    assert np.allclose(r["out"], o, atol=1e-12)
    assert np.allclose(r["lse"], s.logsumexp(-1).T.numpy(), atol=1e-12)


def test_rows_before_the_first_key_are_zero_and_unseen_values_do_not_matter():
    q, k, v = _rand(5, 1, 8, seed=4), _rand(2, 1, 8, seed=5), _rand(2, 1, 8, seed=6)
    v[1] = np.nan
    r = op.prompt_attention(q, k, v, [0, 5], [0, 2], 1.0)
    assert list(op.causal_limits(5, 2)) == [0, 0, 0, 1, 2]
    assert np.all(r["out"][:3] == 0) and np.all(np.isneginf(r["lse"][:3]))
    assert np.allclose(r["out"][3], v[0]) and np.isnan(r["out"][4]).all()


def test_a_chain_of_drafts_is_causal_attention_and_a_node_is_one_decode_step():
    q, k, v = _rand(4, 2, 8, seed=7), _rand(10, 1, 8, seed=8), _rand(10, 1, 8, seed=9)
    out, _, _ = op.tree_attention(q, k, v, 6, [-1, 0, 1, 2], 0.5)
    assert np.allclose(out, op.prompt_attention(q, k, v, [0, 4], [0, 10], 0.5)["out"])
    one = oa.attend(q[0].astype(np.float16), k[:7].astype(np.float16), v[:7].astype(np.float16), .5)
    o1, _, _ = op.tree_attention(q[:1].astype(np.float16), k[:7].astype(np.float16),
                                 v[:7].astype(np.float16), 6, [-1], 0.5)
    assert np.allclose(o1[0], one, atol=1e-12)


def test_siblings_do_not_see_each_other():
    see = op.ancestors([-1, 0, 0, 1, -1])
    want = np.eye(5, dtype=bool)
    want[1, 0] = want[2, 0] = want[3, 0] = want[3, 1] = True
    assert np.array_equal(see, want)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_depends_on_the_distance_only(interleaved):
    f = 1e4 ** (-np.arange(4) / 4)
    x, y = _rand(1, 1, 12, seed=10), _rand(1, 1, 12, seed=11)
    a = op.norm_rope(x, None, [5], f, 0, interleaved)
    assert np.isclose(np.linalg.norm(a), np.linalg.norm(x)) and np.array_equal(a[..., 8:], x[..., 8:])
    d = [float((op.norm_rope(x, None, [p + 9], f, 0, interleaved)
                * op.norm_rope(y, None, [p], f, 0, interleaved)).sum()) for p in (0, 1000)]
    assert np.isclose(d[0], d[1])
    pair = np.zeros((1, 1, 12))
    pair[..., 0] = 1
    r = op.norm_rope(pair, None, [1], f, 0, interleaved)[0, 0]
    assert np.isclose(r[0], np.cos(1.0)) and np.isclose(r[1 if interleaved else 4], np.sin(1.0))


def test_norm_of_a_constant_row_is_its_sign_times_the_weight():
    w = np.linspace(0.5, 1.5, 8)
    assert np.allclose(op.norm_rope(np.full((1, 1, 8), -3.0), w, [0], [], 0, False)[0, 0], -w)
