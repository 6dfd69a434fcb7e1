"""Tree attention on device data that contradicts the call: nothing is read or written outside what
the call's bounds describe, and the contradiction is reported (GPU)."""
import numpy as np
import pytest
import torch

import kvgen
from oracle import prompt as op
from _gpu_util import dev_tensor, i32
from _operator_checks import assert_rows_close
from test_gpu_tree_attn import Cache

pytestmark = pytest.mark.gpu

D = 256


@pytest.mark.parametrize("length", [20, 700])      # whole units, and tiles dealt in equal shares
@pytest.mark.parametrize("H", [1, 3])
def test_offsets_that_give_drafts_to_too_many_sequences_attend_nothing(kvq, cuda_dev, length, H):
    """Three of five sequences hold all 64 drafts: 24 row tiles of 128 (16 heads each), where the
    bounds (64 drafts in all) have 13 at most."""
    G, nodes, nseq = 16, 64, 5
    c = Cache(kvq, cuda_dev, 6, H, 16, [length] * nseq, [nodes] * nseq, seed=1)
    q = dev_tensor(kvgen.queries_np(2, 1, nodes, H * G, D), cuda_dev)
    lens, par = i32([length] * nseq, cuda_dev), i32([-1] * nodes, cuda_dev)
    ws = kvq.tree_workspace(c.kp, nseq, nodes, H * G, nodes, length + nodes, cuda_dev)
    for cu, skipped in (([0, 64, 0, 64, 0, 64], True), ([0, 64, 64, 64, 64, 64], False)):
        out, err = torch.full_like(q, 7.0), i32([0], cuda_dev)
        ws.fill_(255)
        kvq.kvq_tree_attn(c.kp, c.vp, q, c.pt, lens, i32(cu, cuda_dev), par, nodes, length + nodes,
                          1 / 16, out, ws, err)
        torch.cuda.synchronize()
        if skipped:
            assert int(err.item()) == kvq.KVQ_DEVERR_INDEX and (out == 7).all()
        else:      # as many row tiles as one sequence can have
            assert int(err.item()) == 0
            ref, size, span = op.tree_attention(q[0].cpu().numpy(), c.k_hat[0][:length + nodes],
                                                c.v_hat[0][:length + nodes], length, [-1] * nodes, 1 / 16)
            assert_rows_close(out[0].double().cpu().numpy(), ref, size, span, "f16")


@pytest.mark.parametrize("fewer", ["K", "V"])
@pytest.mark.parametrize("length", [10, 1002])
def test_drafts_on_a_page_that_one_pool_lacks_are_not_attended(kvq, cuda_dev, fewer, length):
    """The last drafts lie on a page number that only one of K and V has, with infinite values there
    and in one earlier draft: those on the page are not attended, by themselves either."""
    ps, nodes, G = 16, 10, 6
    c = Cache(kvq, cuda_dev, 8, 1, ps, [length], [nodes], seed=3)
    first = (length + nodes - 1) // ps * ps - length        # the first draft on the last page
    assert 4 <= first < nodes - 2
    last = c.pt_np.size                                      # page ids so far: 0 .. last - 1
    old = int(c.pt_np[0, (length + nodes - 1) // ps])
    for pools, lacks in ((c.kp, fewer == "K"), (c.vp, fewer == "V")):
        p = pools[0]
        if not lacks:
            q = kvq.Pool.empty(8, 1, D, ps, last + 1, cuda_dev)
            q.codes[:last], q.scales[:last] = p.codes, p.scales
            q.codes[last], q.scales[last] = p.codes[old], p.scales[old]
            pools[0] = q
    pt = c.pt.clone()
    pt[0, (length + nodes - 1) // ps] = last
    if fewer == "K":
        c.vp[0].scales[last] = float("inf")
    t = length + 1                                           # draft 1's values: the rows below do not see it
    c.vp[0].scales[int(c.pt_np[0, t // ps]), 0, t % ps] = float("inf")
    parents = [-1, -1, 0, 2, 3] + [4] * (nodes - 5)
    q_np = kvgen.queries_np(4, 1, nodes, G, D)
    q = dev_tensor(q_np, cuda_dev)
    out, err = torch.full_like(q, 7.0), i32([0], cuda_dev)
    ws = kvq.tree_workspace(c.kp, 1, nodes, G, nodes, length + nodes, cuda_dev)
    kvq.kvq_tree_attn(c.kp, c.vp, q, pt, i32([length], cuda_dev), i32([0, nodes], cuda_dev),
                      i32(parents, cuda_dev), nodes, length + nodes, 1 / 16, out, ws, err)
    torch.cuda.synchronize()
    assert int(err.item()) == kvq.KVQ_DEVERR_PAGE_RANGE
    see = op.ancestors(parents)
    see[:, first:] = False
    keep = length + first
    seen = np.concatenate([np.ones((nodes, length), dtype=bool), see[:, :first]], axis=1)
    rows = [i for i in range(nodes) if i != 1]
    for g in range(G):
        ref, _, size, span = op.attend(q_np[0, rows, g], c.k_hat[0][:keep, 0], c.v_hat[0][:keep, 0],
                                       seen[rows], 1 / 16)
        assert_rows_close(out[0, rows, g].double().cpu().numpy(), ref, size, span, "f16")


@pytest.mark.parametrize("bits", [8, 6, 4])
def test_a_long_cache(kvq, cuda_dev, bits):
    length, nodes, G = 131000, 5, 6
    c = Cache(kvq, cuda_dev, bits, 1, 16, [length], [nodes], seed=bits)
    parents = [-1, 0, 0, 1, 2]
    q_np = kvgen.queries_np(bits, 1, nodes, G, D)
    q = dev_tensor(q_np, cuda_dev)
    out, err = torch.full_like(q, 7.0), i32([0], cuda_dev)
    ws = kvq.tree_workspace(c.kp, 1, nodes, G, nodes, length + nodes, cuda_dev)
    kvq.kvq_tree_attn(c.kp, c.vp, q, c.pt, i32([length], cuda_dev), i32([0, nodes], cuda_dev),
                      i32(parents, cuda_dev), nodes, length + nodes, 1 / 16, out, ws, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    ref, size, span = op.tree_attention(q_np[0], c.k_hat[0], c.v_hat[0], length, parents, 1 / 16)
    assert_rows_close(out[0].double().cpu().numpy(), ref, size, span, "f16")
