"""GPU parity of kvq_qk_norm_rope against the float64 oracle, within half a step of the output type
plus the float32 terms derived in _operator_checks."""
import numpy as np
import pytest
import torch

from oracle import prompt as op
from _operator_checks import norm_rope_tolerance

pytestmark = pytest.mark.gpu

KINDS = {"f16": torch.float16, "bf16": torch.bfloat16}


def _run(kvq, dev, T, Hq, H, D, rd, inter, kind, weights=True, far=1 << 20, eps=1e-6, seed=0,
         strided=False, in_place=False, magnitude=1.0):
    g = torch.Generator().manual_seed(seed)
    dt = KINDS[kind]
    pad = 8 if strided else 0
    buf = (torch.randn((T, (Hq + H) * D + pad), generator=g) * magnitude).to(dt).to(dev)
    q = buf[:, :Hq * D].unflatten(1, (Hq, D))
    k = buf[:, Hq * D:(Hq + H) * D].unflatten(1, (H, D))
    if not strided:
        q, k = q.contiguous(), k.contiguous()
    qn, kn = q.double().cpu().numpy(), k.double().cpu().numpy()
    pos = torch.randint(0, far, (T,), generator=g, dtype=torch.int32)
    inv = 1e6 ** (-np.arange(rd // 2) / max(rd // 2, 1))
    qw = (1 + 0.3 * torch.randn(D, generator=g)) if weights else None
    kw = (1 + 0.3 * torch.randn(D, generator=g)) if weights else None
    qo = q if in_place else torch.full((T, Hq, D), float("nan"), dtype=dt, device=dev)
    ko = k if in_place else torch.full((T, H, D), float("nan"), dtype=dt, device=dev)
    kvq.kvq_qk_norm_rope(q, k, qo, ko, pos.to(dev),
                         kvq.kvq_rope_phases(inv, dev) if rd else None,
                         None if qw is None else qw.to(dev), None if kw is None else kw.to(dev),
                         eps, inter)
    torch.cuda.synchronize()
    for x, w, got in ((qn, qw, qo), (kn, kw, ko)):
        wn = None if w is None else w.numpy()
        ref = op.norm_rope(x, wn, pos.numpy(), inv, eps, inter)
        tol = norm_rope_tolerance(x, wn, ref, eps, kind)
        d = np.abs(got.double().cpu().numpy() - ref)
        assert (d <= tol).all(), f"worst {np.nanmax(d / tol):.3g} of the tolerance"


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("D,rd,inter", [(256, 256, False), (256, 64, True), (128, 128, False),
                                        (64, 32, True), (64, 16, False), (80, 48, False),
                                        (8, 0, False), (200, 112, True), (136, 128, False)])
def test_head_sizes_and_pairings(kvq, cuda_dev, kind, D, rd, inter):
    _run(kvq, cuda_dev, 37, 5, 2, D, rd, inter, kind, seed=D + rd)


@pytest.mark.parametrize("T,Hq,H", [(1, 1, 1), (1, 24, 4), (3, 32, 8), (1000, 7, 1), (4097, 24, 4)])
def test_token_and_head_counts(kvq, cuda_dev, T, Hq, H):
    _run(kvq, cuda_dev, T, Hq, H, 256 if T < 4000 else 64, 64, False, "f16", seed=T)


def test_views_of_a_fused_buffer_and_in_place(kvq, cuda_dev):
    _run(kvq, cuda_dev, 65, 6, 2, 128, 128, False, "f16", strided=True)
    _run(kvq, cuda_dev, 65, 6, 2, 128, 64, True, "bf16", strided=True, in_place=True)
    _run(kvq, cuda_dev, 9, 24, 4, 256, 256, False, "f16", in_place=True)


def test_rotation_without_norm_far_positions_and_small_and_large_rows(kvq, cuda_dev):
    _run(kvq, cuda_dev, 50, 3, 1, 64, 64, False, "f16", weights=False, far=2 ** 31 - 1)
    _run(kvq, cuda_dev, 50, 3, 1, 256, 256, True, "f16", far=2 ** 31 - 1, magnitude=2.0 ** -20)
    _run(kvq, cuda_dev, 50, 3, 1, 256, 256, False, "f16", magnitude=2.0 ** 12)


def test_a_zero_row_stays_zero_and_other_rows_do_not_matter(kvq, cuda_dev):
    q = torch.randn((4, 2, 64), device=cuda_dev).half()
    q[1] = 0
    q[2, 1, 5] = float("inf")
    k = torch.zeros((4, 1, 64), device=cuda_dev).half()
    w = torch.ones(64, device=cuda_dev)
    pos = torch.arange(4, dtype=torch.int32, device=cuda_dev)
    ph = kvq.kvq_rope_phases(np.ones(32), cuda_dev)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    kvq.kvq_qk_norm_rope(q, k, qo, ko, pos, ph, w, w)
    assert (qo[1] == 0).all() and (ko == 0).all()
    assert torch.isfinite(qo[[0, 1, 3]]).all() and torch.isfinite(qo[2, 0]).all()


def test_no_tokens(kvq, cuda_dev):
    e = torch.empty((0, 2, 64), dtype=torch.float16, device=cuda_dev)
    kvq.kvq_qk_norm_rope(e, e, e, e, torch.empty(0, dtype=torch.int32, device=cuda_dev))


def test_captured_and_replayed_on_another_stream(kvq, cuda_dev):
    q = torch.randn((16, 3, 128), device=cuda_dev).bfloat16()
    k = torch.randn((16, 1, 128), device=cuda_dev).bfloat16()
    pos = torch.arange(16, dtype=torch.int32, device=cuda_dev) * 1000
    ph = kvq.kvq_rope_phases(1e4 ** (-np.arange(64) / 64), cuda_dev)
    want = torch.empty_like(q), torch.empty_like(k)
    kvq.kvq_qk_norm_rope(q, k, *want, pos, ph)
    got = torch.zeros_like(q), torch.zeros_like(k)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvq.kvq_qk_norm_rope(q, k, *got, pos, ph)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rows_behind_two_billion_elements(kvq, cuda_dev):
    n, hq, h, d, stride = 270010, 2, 1, 64, 8192
    buf = torch.empty((n, stride), dtype=torch.bfloat16, device=cuda_dev)
    q, k = buf[:, :hq * d].unflatten(1, (hq, d)), buf[:, hq * d:(hq + h) * d].unflatten(1, (h, d))
    g = torch.Generator().manual_seed(51)
    buf[:, :(hq + h) * d] = torch.randn((n, 1), generator=g).to(torch.bfloat16).to(cuda_dev)
    last = torch.randn((64, hq + h, d), generator=g).to(torch.bfloat16).to(cuda_dev)
    q[-64:], k[-64:] = last[:, :hq], last[:, hq:]
    phases = kvq.kvq_rope_phases([1.0 / (i + 1) for i in range(d // 2)])
    pos = torch.arange(n, dtype=torch.int32, device=cuda_dev)
    qo, ko = last[:, :hq].contiguous(), last[:, hq:].contiguous()
    kvq.kvq_qk_norm_rope(qo, ko, qo, ko, pos[-64:].contiguous(), phases)
    kvq.kvq_qk_norm_rope(q, k, q, k, pos, phases)
    assert torch.equal(q[-64:], qo) and torch.equal(k[-64:], ko)
