"""GPU parity of kvq_prompt_attn against the float64 oracle, within the tolerance derived in
_operator_checks (the rounding of the softmax weights and of the result to 16 bits)."""
import numpy as np
import pytest
import torch

from oracle import prompt as op
from _gpu_util import cu_of, i32
from _operator_checks import assert_lse_close, assert_rows_close

pytestmark = pytest.mark.gpu

KINDS = {"f16": torch.float16, "bf16": torch.bfloat16}


def _inputs(dev, kind, new, keys, Hq, H, D, seed, fused=False, tail=0, magnitude=1.0):
    g = torch.Generator().manual_seed(seed)
    dt = KINDS[kind]
    tq, tk = sum(new) + tail, sum(keys) + tail
    if fused:
        buf = torch.randn((tq, (Hq + 2 * H) * D + 8), generator=g).mul(magnitude).to(dt).to(dev)
        q = buf[:, :Hq * D].unflatten(1, (Hq, D))
        k = buf[:, Hq * D:(Hq + H) * D].unflatten(1, (H, D))
        v = buf[:, (Hq + H) * D:(Hq + 2 * H) * D].unflatten(1, (H, D))
        return q, k, v
    q = torch.randn((tq, Hq, D), generator=g).mul(magnitude).to(dt).to(dev)
    k = torch.randn((tk, H, D), generator=g).to(dt).to(dev)
    v = torch.randn((tk, H, D), generator=g).to(dt).to(dev)
    return q, k, v


def _call(kvq, q, k, v, new, keys, scale, lse=True, max_q=None, max_k=None, cu_q=None, cu_k=None):
    dev = q.device
    cu_q, cu_k = i32(cu_of(new) if cu_q is None else cu_q, dev), i32(cu_of(keys) if cu_k is None else cu_k, dev)
    max_q, max_k = max_q or max(new), max_k if max_k is not None else max(keys)
    out = torch.full((q.shape[0], q.shape[1], q.shape[2]), 7.0, dtype=q.dtype, device=dev)
    st = torch.full(q.shape[:2], 7.0, dtype=torch.float32, device=dev) if lse else None
    ws = kvq.prompt_workspace(len(cu_q) - 1, q.shape[0], q.shape[1], k.shape[1], q.shape[2],
                              max_q, max_k, dev)
    ws.fill_(255)                                       # NaNs: nothing may be read before written
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    kvq.kvq_prompt_attn(q, k, v, cu_q, cu_k, max_q, max_k, scale, out, ws, st, err)
    torch.cuda.synchronize()
    return out, st, int(err.item())


def _check(kvq, dev, kind, new, keys, Hq, H, D, seed=0, fused=False, tail=0, magnitude=1.0):
    q, k, v = _inputs(dev, kind, new, keys, Hq, H, D, seed, fused, tail, magnitude)
    scale = D ** -0.5
    out, lse, err = _call(kvq, q, k, v, new, keys, scale)
    assert err == 0
    f = [x.double().cpu().numpy() for x in (q, k, v)]
    r = op.prompt_attention(*f, cu_of(new), cu_of(keys), scale)
    n = sum(new)
    assert_rows_close(out[:n].double().cpu().numpy(), r["out"][:n], r["size"][:n], r["span"][:n], kind)
    assert_lse_close(lse[:n].cpu().numpy(), r["lse"][:n], r["span"][:n], D)
    assert (out[n:] == 7).all() and (lse[n:] == 7).all()     # rows of no sequence
    return out


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,H", [(6, 1), (4, 4), (5, 1), (16, 2)])
def test_ragged_prompts(kvq, cuda_dev, kind, D, Hq, H):
    new = [1, 2, 63, 0, 64, 65, 127, 128, 129, 200]
    _check(kvq, cuda_dev, kind, new, new, Hq, H, D, seed=D + Hq, tail=3)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new,keys", [
    ([1], [1]), ([1], [5000]), ([1, 1, 1], [1, 700, 64]), ([37, 5], [400, 5]), ([300], [2500]),
    ([5, 9], [2, 0]), ([130], [100]), ([64], [64 * 20 + 1]), ([3, 200], [3000, 200])])
def test_chunks_single_tokens_and_rows_without_keys(kvq, cuda_dev, D, new, keys):
    _check(kvq, cuda_dev, "f16", new, keys, 12, 2, D, seed=D + sum(keys))
    if D == 64:
        _check(kvq, cuda_dev, "bf16", new, keys, 32, 8, D, seed=D + sum(keys))


@pytest.mark.parametrize("G", [3, 7, 16, 48, 127, 128])
def test_group_sizes(kvq, cuda_dev, G):
    _check(kvq, cuda_dev, "f16", [3, 70], [3, 150], G, 1, 64, seed=G)


def test_more_sequences_than_a_warp_has_lanes(kvq, cuda_dev):
    """33 sequences and more are laid out in another order; empty ones among them."""
    r = np.random.default_rng(1)
    for n, top, past, D in ((33, 60, 0, 64), (70, 9, 300, 128), (100, 3, 2, 256)):
        new = [int(x) for x in r.integers(0, top, n)]
        keys = [a + int(x) for a, x in zip(new, r.integers(0, past + 1, n))]
        _check(kvq, cuda_dev, "f16", new, keys, 4, 2, D, seed=n, tail=2)


def test_tiles_that_end_at_the_view_of_their_first_row(kvq, cuda_dev):
    """Key counts around multiples of the key tile, one row and several."""
    for D, nb in ((256, 128), (128, 64), (64, 64)):
        for keys in (nb - 1, nb, nb + 1, 2 * nb, 5 * nb, 5 * nb + 1):
            _check(kvq, cuda_dev, "f16", [1, 3], [keys, keys], 6, 1, D, seed=keys)


def test_a_non_finite_query_spoils_its_own_row_only(kvq, cuda_dev):
    q, k, v = _inputs(cuda_dev, "f16", [90], [90], 6, 1, 128, 21)
    clean, _, _ = _call(kvq, q, k, v, [90], [90], 0.088)
    q[40, 2, 5], q[41, 3, 0] = float("nan"), float("inf")
    out, _, err = _call(kvq, q, k, v, [90], [90], 0.088)
    assert err == 0 and torch.isnan(out[40, 2]).all() and torch.isnan(out[41, 3]).any()
    keep = torch.ones((90, 6), dtype=torch.bool)
    keep[40, 2] = keep[41, 3] = False
    assert torch.equal(out[keep], clean[keep])


def test_views_of_a_fused_projection(kvq, cuda_dev):
    for D in (64, 256):
        _check(kvq, cuda_dev, "f16", [100, 33], [100, 33], 6, 2, D, fused=True)


def test_longer_prompt_and_sharp_softmax(kvq, cuda_dev):
    _check(kvq, cuda_dev, "f16", [700], [700], 6, 1, 256, seed=3)
    _check(kvq, cuda_dev, "f16", [200], [900], 2, 1, 128, seed=4, magnitude=20.0)
    _check(kvq, cuda_dev, "bf16", [200], [900], 2, 1, 64, seed=5, magnitude=20.0)


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("order", ["rising", "falling"])
def test_scores_that_rise_or_fall_along_the_keys(kvq, cuda_dev, D, order):
    """The running maximum moves in every tile (or only in the first)."""
    n = 600
    t = torch.arange(n, dtype=torch.float32) / n * 60
    if order == "falling":
        t = t.flip(0)
    q = torch.ones((n, 2, D), device=cuda_dev).half()
    k = (t[:, None, None] / D ** 0.5 * torch.ones((1, 1, D))).half().to(cuda_dev)
    v = torch.randn((n, 1, D), generator=torch.Generator().manual_seed(1)).half().to(cuda_dev)
    out, lse, err = _call(kvq, q, k, v, [n], [n], D ** -0.5)
    r = op.prompt_attention(*[x.double().cpu().numpy() for x in (q, k, v)], [0, n], [0, n], D ** -0.5)
    assert err == 0
    assert_rows_close(out.double().cpu().numpy(), r["out"], r["size"], r["span"], "f16")
    assert_lse_close(lse.cpu().numpy(), r["lse"], r["span"], D)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_unseen_infinities_and_nans_do_not_reach_a_row(kvq, cuda_dev, D, kind):
    """A later token's key and value, the next sequence's and the rows behind the last one."""
    new, keys = [150, 60], [150, 90]
    q, k, v = _inputs(cuda_dev, kind, new, keys, 6, 1, D, 9, tail=70)
    clean = [x.double().cpu().numpy() for x in (q, k, v)]
    for t, x in ((100, float("nan")), (140, float("inf")), (239, float("-inf"))):
        k[t, :, 3] = x
        v[t, :, 5] = x
        v[t, :, D - 1] = x
    q[sum(new):], k[sum(keys):], v[sum(keys):] = float("nan"), float("nan"), float("inf")
    out, lse, err = _call(kvq, q, k, v, new, keys, D ** -0.5)
    assert err == 0
    r = op.prompt_attention(*clean, cu_of(new), cu_of(keys), D ** -0.5)
    rows = list(range(100)) + list(range(150, 209))           # rows that see none of them
    assert_rows_close(out[rows].double().cpu().numpy(), r["out"][rows], r["size"][rows],
                      r["span"][rows], kind)
    assert_lse_close(lse[rows].cpu().numpy(), r["lse"][rows], r["span"][rows], D)
    assert torch.isnan(out[100:150]).all()                    # these see a NaN score


@pytest.mark.parametrize("D", [64, 256])
def test_seen_infinite_values_reach_their_rows_and_channels_only(kvq, cuda_dev, D):
    n = 200
    q, k, v = _inputs(cuda_dev, "f16", [n], [n], 2, 1, D, 11)
    v[20, 0, 7], v[180, 0, 9] = float("inf"), float("-inf")
    out, _, err = _call(kvq, q, k, v, [n], [n], D ** -0.5)
    assert err == 0
    o = out.float()
    assert torch.isposinf(o[20:, :, 7]).all() and torch.isneginf(o[180:, :, 9]).all()
    o[20:, :, 7], o[180:, :, 9] = 0, 0
    assert torch.isfinite(o).all()


def test_sequences_that_contradict_the_bounds_are_skipped_and_reported(kvq, cuda_dev):
    new = [40, 50, 30]
    q, k, v = _inputs(cuda_dev, "f16", new, new, 4, 2, 64, 12)
    want, _, _ = _call(kvq, q, k, v, new, new, 0.125)
    for over in (dict(max_q=45), dict(max_k=45), dict(cu_k=[0, 40, 30, 120]),
                 dict(cu_k=[0, 40, 90, 121]), dict(cu_q=[0, 40, 90, 121]), dict(cu_q=[-1, 40, 90, 120])):
        out, _, err = _call(kvq, q, k, v, new, new, 0.125, **over)
        assert err == kvq.KVQ_DEVERR_INDEX, over
        rows = (out != 7).any(-1).any(-1)
        assert rows.any() and not rows.all(), over
        assert torch.allclose(out[rows].float(), want[rows].float(), atol=4e-3) or "cu_k" in over


def test_no_tokens_and_no_keys(kvq, cuda_dev):
    q, k, v = _inputs(cuda_dev, "f16", [4], [4], 2, 1, 64, 13)
    out, lse, err = _call(kvq, q, k[:0], v[:0], [4], [0], 0.125)
    assert err == 0 and (out == 0).all() and torch.isneginf(lse).all()
    e = q[:0]
    out, _, err = _call(kvq, e, k, v, [0], [4], 0.125, max_q=1)
    assert err == 0


def test_same_bits_every_time_on_two_streams_and_replayed(kvq, cuda_dev):
    new, keys = [3, 90, 1], [4000, 90, 333]
    q, k, v = _inputs(cuda_dev, "f16", new, keys, 12, 2, 128, 14)
    a, la, _ = _call(kvq, q, k, v, new, keys, 0.088)
    b, lb, _ = _call(kvq, q, k, v, new, keys, 0.088)
    assert torch.equal(a, b) and torch.equal(la, lb)
    cq, ck = i32(cu_of(new), cuda_dev), i32(cu_of(keys), cuda_dev)
    ws = [kvq.prompt_workspace(3, q.shape[0], 12, 2, 128, 90, 4000, cuda_dev) for _ in range(2)]
    outs = [torch.zeros_like(q) for _ in range(2)]
    s = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            kvq.kvq_prompt_attn(q, k, v, cq, ck, 90, 4000, 0.088, outs[i], ws[i], stream=s[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], a) and torch.equal(outs[1], a)
    g, got = torch.cuda.CUDAGraph(), torch.zeros_like(q)
    with torch.cuda.graph(g):
        kvq.kvq_prompt_attn(q, k, v, cq, ck, 90, 4000, 0.088, got, ws[0])
    for _ in range(3):
        got.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, a)


def test_a_chunk_joined_to_earlier_keys_by_lse_is_the_whole(kvq, cuda_dev):
    """Attention over the first keys and over the rest, joined by the row statistics."""
    q, k, v = _inputs(cuda_dev, "f16", [1], [900], 6, 1, 128, 15)
    whole, lw, _ = _call(kvq, q, k, v, [1], [900], 0.088)
    a, la, _ = _call(kvq, q, k[:500], v[:500], [1], [500], 0.088)
    b, lb, _ = _call(kvq, q, k[500:], v[500:], [1], [400], 0.088)
    l = torch.logaddexp(la, lb)
    joined = a.float() * (la - l).exp()[..., None] + b.float() * (lb - l).exp()[..., None]
    assert torch.allclose(l, lw, atol=1e-5) and torch.allclose(joined, whole.float(), atol=1e-3)


@pytest.mark.parametrize("D", [64, 256])
def test_bounds_far_above_the_lengths(kvq, cuda_dev, D):
    new, keys = [1, 40], [300, 900]
    q, k, v = _inputs(cuda_dev, "f16", new, keys, 6, 1, D, 31)
    exact, lse, _ = _call(kvq, q, k, v, new, keys, 0.1)
    far, far_lse, err = _call(kvq, q, k, v, new, keys, 0.1, max_q=2 ** 31 - 1, max_k=2 ** 31 - 1)
    assert err == 0
    # one split instead of several: the same sums in another order, each result rounded once
    f = [x.double().cpu().numpy() for x in (q, k, v)]
    r = op.prompt_attention(*f, cu_of(new), cu_of(keys), 0.1)
    for o, s in ((exact, lse), (far, far_lse)):
        assert_rows_close(o.double().cpu().numpy(), r["out"], r["size"], r["span"], "f16")
        assert_lse_close(s.cpu().numpy(), r["lse"], r["span"], D)


@pytest.mark.parametrize("keys", [90, 5000])
def test_lse_of_a_row_of_nan_scores_is_nan(kvq, cuda_dev, keys):
    q, k, v = _inputs(cuda_dev, "f16", [90], [keys], 6, 1, 256, 33)
    q[40, 2] = float("nan")
    out, lse, err = _call(kvq, q, k, v, [90], [keys], 0.0625)
    assert err == 0 and torch.isnan(out[40, 2]).all()
    bad = torch.isnan(lse)
    assert bad[40, 2] and int(bad.sum()) == 1 and torch.isfinite(lse[~bad]).all()


def test_rows_behind_two_billion_elements(kvq, cuda_dev):
    """The same bits as from a small buffer: offsets of q, k, v and out pass 32 bits."""
    Hq, H, D, at, stride = 6, 1, 128, 270000, 8192
    new, keys = [40, 1], [40, 90]
    q, k, v = _inputs(cuda_dev, "f16", new, keys, Hq, H, D, 41)
    v[60, 0, 3] = float("inf")                       # also the values that are read one by one
    small, lse, _ = _call(kvq, q, k, v, new, keys, 0.1)
    buf = torch.empty((at + sum(keys), stride), dtype=torch.float16, device=cuda_dev)
    rows = lambda lo, x: buf[:at + x.shape[0], lo:lo + x.shape[1] * D].unflatten(1, x.shape[1:])
    views = []
    for lo, x in ((0, q), (Hq * D, k), ((Hq + H) * D, v)):
        w = rows(lo, x)
        w[at:] = x
        views.append(w)
    cu_q, cu_k = [[at + c for c in cu_of(n)] for n in (new, keys)]
    big, big_lse, err = _call(kvq, *views, new, keys, 0.1, cu_q=cu_q, cu_k=cu_k)
    assert err == 0
    assert torch.equal(big[at:].view(torch.int16), small.view(torch.int16))
    assert torch.equal(big_lse[at:], lse) and (big[:at] == 7).all()
