"""Which sequences prompt attention skips when its offsets or lengths contradict the call, row by row;
and long caches (GPU)."""
import numpy as np
import pytest
import torch

from oracle import prompt as op
from _gpu_util import cu_of, i32
from _operator_checks import assert_lse_close, assert_rows_close

pytestmark = pytest.mark.gpu


def _rand(g, n, h, d, dev):
    return torch.randn((n, h, d), generator=g).half().to(dev)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("over,valid", [
    (dict(max_q=45), (0, 2)), (dict(max_k=45), (0, 2)),
    (dict(cu_k=[0, 40, 30, 120]), (0,)),      # falls for 1, and leaves 2 with 90 keys, above the bound
    (dict(cu_k=[0, 40, 90, 121]), (0, 1)), (dict(cu_q=[0, 40, 90, 121]), (0, 1)),
    (dict(cu_q=[-1, 40, 90, 120]), (1, 2)), (dict(cu_q=[0, 40, 30, 120]), (0,)),
    (dict(cu_k=[0, -1, 90, 120]), (2,))])     # 0 falls, 1 starts below 0
def test_exactly_the_contradicting_sequences_are_skipped(kvq, cuda_dev, D, over, valid):
    new, Hq, H = [40, 50, 30], 4, 2
    g = torch.Generator().manual_seed(D)
    q, k, v = (_rand(g, 120, h, D, cuda_dev) for h in (Hq, H, H))
    a = dict(max_q=50, max_k=50, cu_q=cu_of(new), cu_k=cu_of(new))
    a.update(over)
    out, err = torch.full_like(q, 7.0), i32([0], cuda_dev)
    lse = torch.full((120, Hq), 7.0, device=cuda_dev)
    ws = kvq.prompt_workspace(3, 120, Hq, H, D, a["max_q"], a["max_k"], cuda_dev)
    kvq.kvq_prompt_attn(q, k, v, i32(a["cu_q"], cuda_dev), i32(a["cu_k"], cuda_dev), a["max_q"],
                        a["max_k"], D ** -0.5, out, ws, lse, err)
    torch.cuda.synchronize()
    assert int(err.item()) == kvq.KVQ_DEVERR_INDEX
    r = op.prompt_attention(*(x.double().cpu().numpy() for x in (q, k, v)), cu_of(new), cu_of(new),
                            D ** -0.5)
    rows = np.zeros(120, dtype=bool)
    for s in valid:
        rows[cu_of(new)[s]:cu_of(new)[s + 1]] = True
    assert_rows_close(out[rows].double().cpu().numpy(), r["out"][rows], r["size"][rows],
                      r["span"][rows], "f16")
    assert_lse_close(lse[rows].cpu().numpy(), r["lse"][rows], r["span"][rows], D)
    assert (out[~rows] == 7).all() and (lse[~rows] == 7).all()


@pytest.mark.parametrize("D,Hq,H", [(64, 8, 2), (128, 4, 1), (256, 6, 1)])
@pytest.mark.parametrize("new,keys", [([1], [131072]), ([5, 1], [70001, 131])])
def test_long_caches_of_16_bit_keys(kvq, cuda_dev, D, Hq, H, new, keys):
    g = torch.Generator().manual_seed(D)
    q, k, v = (_rand(g, n, h, D, cuda_dev) for n, h in ((sum(new), Hq), (sum(keys), H), (sum(keys), H)))
    out, err = torch.full_like(q, 7.0), i32([0], cuda_dev)
    lse = torch.empty((sum(new), Hq), device=cuda_dev)
    ws = kvq.prompt_workspace(len(new), sum(new), Hq, H, D, max(new), max(keys), cuda_dev)
    kvq.kvq_prompt_attn(q, k, v, i32(cu_of(new), cuda_dev), i32(cu_of(keys), cuda_dev), max(new),
                        max(keys), D ** -0.5, out, ws, lse, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    r = op.prompt_attention(*(x.double().cpu().numpy() for x in (q, k, v)), cu_of(new), cu_of(keys),
                            D ** -0.5)
    assert_rows_close(out.double().cpu().numpy(), r["out"], r["size"], r["span"], "f16")
    assert_lse_close(lse.cpu().numpy(), r["lse"], r["span"], D)
