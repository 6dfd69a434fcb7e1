"""Refusals of the norm, prompt, tree and commit entry points (no GPU needed): every invalid
argument is turned into a status on the host, before anything is launched.  The C entry points are
called with made-up addresses that no check dereferences."""
import ctypes

import numpy as np
import pytest
import torch

A = 1 << 20            # an aligned address that is never read
SHAPE, NULL, ALIGN, RANGE, WORKSPACE, BITS = 2, 3, 4, 5, 8, 1
NAN, INF = float("nan"), float("inf")


def _call(kvq, fn, args, **over):
    assert set(over) <= set(args), over
    return getattr(kvq._lib, fn)(*{**args, **over}.values())


def _norm(kvq):
    return dict(dtype=0, q=A, qs=6 * 64, k=A, ks=2 * 64, qo=A, qos=6 * 64, ko=A, kos=2 * 64, n=3,
                hq=6, h=2, d=64, rd=32, inter=0, pos=A, phases=A, qw=A, kw=A, eps=1e-6, stream=None)


def _prompt(kvq):
    ws = kvq.kvq_prompt_attn_workspace(2, 100, 6, 2, 128, 60, 60)
    return dict(dtype=0, q=A, qs=6 * 128, k=A, ks=256, v=A, vs=256, hq=6, h=2, d=128, cu_q=A, cu_k=A,
                nseq=2, tq=100, tk=100, mq=60, mk=60, scale=0.1, out=A, lse=A, ws=A, wsb=ws, err=None,
                stream=None)


def _pools(kvq, n=1, **over):
    arr = (kvq.kvq_pool * n)()
    for i in range(n):
        f = dict(bits=6, num_heads=2, head_dim=256, page_size=16, num_pages=10, codes=A, scales=A)
        f.update(over)
        arr[i] = kvq.kvq_pool(*f.values())
    return arr


def _tree(kvq):
    ws = kvq.kvq_tree_attn_workspace(1, 2, 9, 2, 12, 256, 8, 100)
    return dict(k=_pools(kvq), v=_pools(kvq), n=1, q=A, hq=12, table=A, mp=10, lens=A, cu=A, par=A,
                nseq=2, total=9, nodes=8, ml=100, scale=0.1, out=A, ws=A, wsb=ws, err=None, stream=None)


def _commit(kvq):
    return dict(pools=_pools(kvq), n=1, table=A, mp=10, lens=A, cu=A, acc=A, nseq=2, total=5, err=None,
                stream=None)


@pytest.mark.parametrize("over,status", [
    (dict(dtype=2), SHAPE), (dict(dtype=-1), SHAPE), (dict(hq=0), SHAPE), (dict(h=0), SHAPE),
    (dict(d=60), SHAPE), (dict(d=264), SHAPE), (dict(d=0), SHAPE), (dict(rd=24), SHAPE),
    (dict(rd=80), SHAPE), (dict(rd=-16), SHAPE), (dict(qs=6 * 64 - 8), SHAPE),
    (dict(ks=2 * 64 + 4), SHAPE), (dict(qos=8), SHAPE), (dict(kos=2 * 64 + 1), SHAPE),
    (dict(qos=7 * 64), SHAPE), (dict(n=-1), RANGE), (dict(eps=-1.0), RANGE), (dict(eps=NAN), RANGE),
    (dict(eps=INF), RANGE), (dict(q=None), NULL), (dict(ko=None), NULL), (dict(pos=None), NULL),
    (dict(phases=None), NULL), (dict(q=A + 2), ALIGN), (dict(ko=A + 8), ALIGN),
    (dict(qw=A + 4), ALIGN), (dict(phases=A + 4), ALIGN), (dict(pos=A + 2), ALIGN),
    (dict(n=0, q=None, phases=None), 0)])
def test_norm_rope_refusals(kvq, over, status):
    assert _call(kvq, "kvq_qk_norm_rope", _norm(kvq), **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(dtype=2), SHAPE), (dict(d=96), SHAPE), (dict(d=512), SHAPE), (dict(h=0), SHAPE),
    (dict(hq=7), SHAPE), (dict(hq=1), SHAPE), (dict(hq=258, h=2), SHAPE), (dict(qs=6 * 128 - 8), SHAPE),
    (dict(ks=260), SHAPE), (dict(vs=128), SHAPE), (dict(nseq=-1), RANGE), (dict(tq=-1), RANGE),
    (dict(tk=-1), RANGE), (dict(mq=-1), RANGE), (dict(mk=-1), RANGE), (dict(scale=0.0), RANGE),
    (dict(scale=-1.0), RANGE), (dict(scale=NAN), RANGE), (dict(scale=INF), RANGE),
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(cu_q=None), NULL),
    (dict(cu_k=None), NULL), (dict(out=None), NULL), (dict(ws=None), NULL), (dict(q=A + 8), ALIGN),
    (dict(v=A + 2), ALIGN), (dict(out=A + 4), ALIGN), (dict(ws=A + 8), ALIGN), (dict(lse=A + 2), ALIGN),
    (dict(wsb=0), WORKSPACE), (dict(nseq=0, q=None), 0), (dict(tq=0, cu_q=None), 0)])
def test_prompt_refusals(kvq, over, status):
    assert _call(kvq, "kvq_prompt_attn", _prompt(kvq), **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(n=0), RANGE), (dict(n=65), RANGE), (dict(hq=13), SHAPE), (dict(hq=34), SHAPE),
    (dict(hq=0), SHAPE), (dict(mp=0), RANGE), (dict(nseq=-1), RANGE), (dict(total=-1), RANGE),
    (dict(nodes=0), RANGE), (dict(nodes=65), RANGE), (dict(ml=-1), RANGE), (dict(ml=161), RANGE),
    (dict(scale=NAN), RANGE), (dict(scale=0.0), RANGE), (dict(q=None), NULL), (dict(par=None), NULL),
    (dict(cu=None), NULL), (dict(lens=None), NULL), (dict(table=None), NULL), (dict(out=None), NULL),
    (dict(ws=None), NULL), (dict(q=A + 2), ALIGN), (dict(out=A + 8), ALIGN), (dict(ws=A + 4), ALIGN),
    (dict(wsb=0), WORKSPACE), (dict(k=None), NULL), (dict(nseq=0, q=None), 0),
    (dict(total=0, q=None), 0)])
def test_tree_refusals(kvq, over, status):
    assert _call(kvq, "kvq_tree_attn", _tree(kvq), **over) == status


@pytest.mark.parametrize("pool,status", [
    (dict(bits=5), BITS), (dict(head_dim=128), SHAPE), (dict(page_size=8), SHAPE),
    (dict(num_heads=1), SHAPE), (dict(num_pages=0), RANGE), (dict(codes=None), NULL),
    (dict(scales=A + 2), ALIGN)])
def test_tree_refuses_pools(kvq, pool, status):
    assert _call(kvq, "kvq_tree_attn", _tree(kvq), v=_pools(kvq, **pool)) == status


@pytest.mark.parametrize("over,status", [
    (dict(n=0), RANGE), (dict(n=65), RANGE), (dict(nseq=-1), RANGE), (dict(total=-1), RANGE),
    (dict(mp=0), RANGE), (dict(table=None), NULL), (dict(lens=None), NULL), (dict(cu=None), NULL),
    (dict(acc=None), NULL), (dict(pools=None), NULL), (dict(nseq=0, cu=None), 0),
    (dict(total=0, acc=None), 0)])
def test_commit_refusals(kvq, over, status):
    assert _call(kvq, "kvq_tree_commit", _commit(kvq), **over) == status
    assert _call(kvq, "kvq_tree_commit", _commit(kvq), pools=_pools(kvq, bits=7)) == BITS


def test_rope_phases(kvq):
    f = [0.0, 1.0, 1e-6, 2 * np.pi, 100.0]
    p = kvq.kvq_rope_phases(f, "cpu").numpy().view(np.uint64)
    assert p[0] == 0
    for x, got in zip(f, p):
        turns = x / (2 * np.pi) % 1.0
        d = abs(float(got) / 2.0 ** 64 - turns)
        assert min(d, 1 - d) < 2.0 ** -50 * max(1.0, x)
    for bad in ([NAN], [INF], [-1.0], [1.0] * 129):
        with pytest.raises(kvq.KVQError):
            kvq.kvq_rope_phases(bad, "cpu")
    out = (ctypes.c_uint64 * 1)()
    assert kvq._lib.kvq_rope_phases(None, 1, out) == NULL


def test_workspace_sizes_reject_nonsense(kvq):
    assert kvq.kvq_prompt_attn_workspace(0, 1, 1, 1, 64, 1, 1) == 0
    assert kvq.kvq_prompt_attn_workspace(1, 1, 1, 1, 64, -1, 1) == 0
    assert kvq.kvq_tree_attn_workspace(1, 0, 1, 1, 1, 256, 1, 1) == 0
    assert kvq.kvq_tree_attn_workspace(1, 1, 1, 1, 1, 256, 1, -1) == 0
    assert kvq.kvq_prompt_attn_workspace(1, 1, 1, 1, 64, 1, 1) >= 16
    assert kvq.kvq_tree_attn_workspace(1, 1, 1, 1, 1, 256, 1, 1) >= 16


def test_host_tensors_are_refused_by_the_binding(kvq):
    x = torch.zeros((2, 2, 64), dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        kvq.kvq_qk_norm_rope(x, x, x, x, i)
    with pytest.raises(TypeError):
        kvq.kvq_prompt_attn(x, x, x, i, i, 1, 1, 1.0, x, i)
    pool = kvq.Pool.empty(6, 1, 256, 16, 1, "cpu")
    q = torch.zeros((1, 1, 1, 256), dtype=torch.float16)
    with pytest.raises(TypeError):
        kvq.kvq_tree_attn([pool], [pool], q, i[None], i[:1], i, i[:1], 1, 16, 1.0, q, i)
    with pytest.raises(TypeError):
        kvq.kvq_tree_commit([pool], i[None], i[:1], i, i)


BIG = 2 ** 31 - 1


@pytest.mark.parametrize("over,status", [
    (dict(scale=3e38), RANGE),                    # finite, but not once it is in powers of two
    (dict(tk=BIG), RANGE), (dict(tk=BIG - 127), RANGE)])
def test_prompt_refuses_the_ends_of_the_range(kvq, over, status):
    assert _call(kvq, "kvq_prompt_attn", _prompt(kvq), **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(scale=3e38), RANGE), (dict(ml=BIG, mp=BIG), RANGE), (dict(ml=BIG - 63, mp=BIG), RANGE),
    # 2^30 tiles: 2 sequences x 2 heads x 1 row tile x 2^31 / 64 tokens x 9 layers and more
    (dict(ml=BIG - 64, mp=BIG, n=9, k=9, v=9, wsb=1 << 40), RANGE)])
def test_tree_refuses_the_ends_of_the_range(kvq, over, status):
    over = {k: _pools(kvq, x) if k in ("k", "v") else x for k, x in over.items()}
    assert _call(kvq, "kvq_tree_attn", _tree(kvq), **over) == status


@pytest.mark.parametrize("D", [64, 128, 256])
def test_generous_bounds_plan_like_exact_ones(kvq, D):
    # 128 keys below 2^31 are one tile fewer: the plans differ by no more than their rounding
    a = kvq.kvq_prompt_attn_workspace(1, 1, 6, 1, D, 1, BIG)
    b = kvq.kvq_prompt_attn_workspace(1, 1, 6, 1, D, 1, BIG - 1000)
    assert a == b > kvq.kvq_prompt_attn_workspace(1, 1, 6, 1, D, 1, 100)
    assert kvq.kvq_prompt_attn_workspace(2, 9, 6, 1, D, BIG, 100) > 0
