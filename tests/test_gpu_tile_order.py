"""Scores and weights of neighbouring tiles share tensor memory in prompt and tree attention: a score
that landed before the product of the weights under it had read them would change bits from run to
run.  Forty runs each, on two streams at once so that the blocks' timing varies, give the same bits
(GPU)."""
import pytest
import torch

import kvgen
from _gpu_util import cu_of, dev_tensor, i32
from test_gpu_tree_attn import Cache, _parents

pytestmark = pytest.mark.gpu


def _same_bits(run, like):
    """run(i, out, stream): call number i mod 2's own workspace and output."""
    first = torch.zeros_like(like)
    run(0, first, None)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [torch.zeros_like(like) for _ in range(2)]
    for _ in range(20):
        for i in range(2):
            outs[i].zero_()
        torch.cuda.synchronize()
        for i in range(2):
            run(i, outs[i], streams[i])
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i].view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("D,Hq,H", [(64, 32, 8), (128, 16, 4), (256, 24, 4)])
@pytest.mark.parametrize("new,keys", [([700, 90], [700, 1500]), ([30], [9000])])
def test_prompt_attention_gives_the_same_bits(kvq, cuda_dev, D, Hq, H, new, keys):
    g = torch.Generator().manual_seed(D)
    q, k, v = (torch.randn((n, h, D), generator=g).half().to(cuda_dev)
               for n, h in ((sum(new), Hq), (sum(keys), H), (sum(keys), H)))
    cu_q, cu_k = i32(cu_of(new), cuda_dev), i32(cu_of(keys), cuda_dev)
    ws = [kvq.prompt_workspace(len(new), sum(new), Hq, H, D, max(new), max(keys), cuda_dev)
          for _ in range(2)]
    _same_bits(lambda i, out, stream: kvq.kvq_prompt_attn(q, k, v, cu_q, cu_k, max(new), max(keys),
                                                          D ** -0.5, out, ws[i], stream=stream), q)


@pytest.mark.parametrize("bits", [8, 6, 4])
@pytest.mark.parametrize("lens,nodes", [([9000, 100, 4001], [16, 64, 3]), ([300, 77], [20, 64])])
def test_tree_attention_gives_the_same_bits(kvq, cuda_dev, bits, lens, nodes):
    c = Cache(kvq, cuda_dev, bits, 2, 16, lens, nodes, seed=bits)
    q = dev_tensor(kvgen.queries_np(bits, 1, sum(nodes), 12, 256), cuda_dev)
    lens_t, cu = i32(lens, cuda_dev), i32(cu_of(nodes), cuda_dev)
    par = i32(sum((_parents(n, n) for n in nodes), []), cuda_dev)
    longest = max(a + b for a, b in zip(lens, nodes))
    ws = [kvq.tree_workspace(c.kp, len(lens), sum(nodes), 12, max(nodes), longest, cuda_dev)
          for _ in range(2)]
    _same_bits(lambda i, out, stream: kvq.kvq_tree_attn(c.kp, c.vp, q, c.pt, lens_t, cu, par,
                                                        max(nodes), longest, 1 / 16, out, ws[i],
                                                        stream=stream), q)
