"""One workspace, sized for a program's largest call, serves its smaller ones (GPU)."""
import pytest
import torch

from oracle import prompt as op
from _gpu_util import cu_of, i32
from _operator_checks import assert_rows_close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,Hq,H", [(64, 8, 2), (128, 6, 2), (256, 6, 1)])
def test_prompt_chunks_and_single_tokens_share_the_largest_calls_workspace(kvq, cuda_dev, D, Hq, H):
    top = 16384
    ws = kvq.prompt_workspace(4, top, Hq, H, D, top, top, cuda_dev)   # by itself, one split
    g = torch.Generator().manual_seed(D)
    for new, keys in (([1], [3000]), ([1, 1, 1, 1], [900, 3000, 64, 1]), ([64], [2500]), ([300, 9], [300, 700])):
        q, k, v = (torch.randn((n, h, D), generator=g).half().to(cuda_dev)
                   for n, h in ((sum(new), Hq), (sum(keys), H), (sum(keys), H)))
        out, err = torch.full_like(q, 7.0), i32([0], cuda_dev)
        ws.fill_(255)
        kvq.kvq_prompt_attn(q, k, v, i32(cu_of(new), cuda_dev), i32(cu_of(keys), cuda_dev), max(new),
                            max(keys), D ** -0.5, out, ws, dev_err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        r = op.prompt_attention(*(x.double().cpu().numpy() for x in (q, k, v)), cu_of(new), cu_of(keys),
                                D ** -0.5)
        assert_rows_close(out.double().cpu().numpy(), r["out"], r["size"], r["span"], "f16")
