"""Tree attention on device data that contradicts the call: nothing is read or written outside what
the call's bounds describe, and the contradiction is reported (GPU)."""
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
