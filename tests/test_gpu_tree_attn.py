"""GPU parity of kvq_tree_attn and kvq_tree_commit against the oracle, and the run of a serving
step: projection rows -> norm and rotation -> pages -> tree attention -> commit -> decode."""
import numpy as np
import pytest
import torch

import kvgen
from oracle import prompt as op
from oracle import symmetric as osym
from _gpu_util import cu_of, dev_tensor, i32
from _operator_checks import assert_rows_close

pytestmark = pytest.mark.gpu

D = 256


def _parents(n, seed, chain=False):
    r = np.random.default_rng(seed)
    return [i - 1 if chain else int(r.integers(max(-1, i - 5), i)) for i in range(n)]


class Cache:
    """Pools (one layer) of sequences with `lens` cached tokens and `nodes` drafts behind them."""

    def __init__(self, kvq, dev, bits, H, ps, lens, nodes, seed=0, layers=1, extra_pages=0):
        self.lens, self.nodes, self.ps, self.bits, self.H = lens, nodes, ps, bits, H
        tot = [a + b for a, b in zip(lens, nodes)]
        per = max(-(-t // ps) for t in tot) + extra_pages
        per = max(per, 1)
        self.pt_np = kvgen.random_page_table(seed + 1, len(lens), per)
        self.pt = i32(self.pt_np, dev)
        self.kp, self.vp, self.k_hat, self.v_hat = [], [], [], []
        for layer in range(layers):
            for key, pools, hats in ((True, self.kp, self.k_hat), (False, self.vp, self.v_hat)):
                x = kvgen.KVSpec(seed=seed, layer=layer, is_key=key, n_seq=1, n_tok=max(sum(tot), 1),
                                 num_heads=H, head_dim=D).full_np()[:sum(tot)]
                p = kvq.Pool.empty(bits, H, D, ps, self.pt_np.size, dev)
                p.codes.fill_(0xFF)
                p.scales.fill_(float("nan"))              # what no token wrote must not matter
                kvq.kvq_quant_pack_paged([p], [dev_tensor(x, dev)], self.pt, i32(cu_of(tot), dev),
                                         i32([0] * len(lens), dev))
                s, c = osym.quantize_rows(x, bits)
                pools.append(p)
                hats.append(osym.dequantize_rows(c, s))
        self.cu_tot = cu_of(tot)


def _call(kvq, dev, c, q, parents, scale=1 / 16, lens=None, max_nodes=None, max_len=None, pt=None):
    nodes = c.nodes
    lens = c.lens if lens is None else lens
    max_nodes = max_nodes or max(nodes)
    max_len = max_len or max(a + b for a, b in zip(c.lens, nodes))
    out = torch.full(q.shape, 7.0, dtype=torch.float16, device=dev)
    ws = kvq.tree_workspace(c.kp, len(lens), q.shape[1], q.shape[2], max_nodes, max_len, dev)
    ws.fill_(255)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    kvq.kvq_tree_attn(c.kp, c.vp, q, c.pt if pt is None else pt, i32(lens, dev),
                      i32(cu_of(nodes), dev), i32(sum(parents, []) + [-1] * (q.shape[1] - sum(nodes)), dev),
                      max_nodes, max_len, scale, out, ws, err)
    torch.cuda.synchronize()
    return out, int(err.item())


def _reference(c, q_np, parents, layer=0, scale=1 / 16):
    outs = [op.tree_attention(q_np[cu0:cu1], c.k_hat[layer][t0:t1], c.v_hat[layer][t0:t1], n, par, scale)
            for cu0, cu1, t0, t1, n, par in zip(cu_of(c.nodes), cu_of(c.nodes)[1:], c.cu_tot,
                                                c.cu_tot[1:], c.lens, parents)]
    return [np.concatenate([o[i] for o in outs]) for i in range(3)]


def _check(kvq, dev, bits, H, G, lens, nodes, ps=16, seed=0, layers=1, chain=False, tail=0):
    c = Cache(kvq, dev, bits, H, ps, lens, nodes, seed, layers)
    parents = [_parents(n, seed + i, chain) for i, n in enumerate(nodes)]
    q_np = kvgen.queries_np(seed + 2, layers, sum(nodes) + tail, H * G, D)
    out, err = _call(kvq, dev, c, dev_tensor(q_np, dev), parents)
    assert err == 0
    n = sum(nodes)
    for l in range(layers):
        ref, size, span = _reference(c, q_np[l, :n], parents, l)
        assert_rows_close(out[l, :n].double().cpu().numpy(), ref, size, span, "f16", f"layer {l}")
    assert (out[:, n:] == 7).all()
    return c, parents, q_np, out


@pytest.mark.parametrize("bits", [8, 6, 4])
@pytest.mark.parametrize("H,G", [(1, 1), (4, 6), (2, 8), (1, 16)])
def test_small_caches_and_trees(kvq, cuda_dev, bits, H, G):
    _check(kvq, cuda_dev, bits, H, G, [0, 1, 15, 16, 17, 63, 64, 65, 300, 5],
           [1, 4, 64, 16, 21, 1, 22, 7, 33, 0], seed=bits + G, tail=2)


@pytest.mark.parametrize("bits", [8, 6, 4])
@pytest.mark.parametrize("lens,nodes", [([5000], [1]), ([9000, 100, 4001], [16, 64, 3]),
                                        ([2048], [64]), ([1, 2, 3], [1, 1, 1])])
def test_longer_caches(kvq, cuda_dev, bits, lens, nodes):
    _check(kvq, cuda_dev, bits, 1, 6, lens, nodes, seed=bits)


@pytest.mark.parametrize("ps", [16, 32, 48, 128])
def test_page_sizes(kvq, cuda_dev, ps):
    _check(kvq, cuda_dev, 6, 2, 3, [1000, 37, 128], [10, 64, 5], ps=ps, seed=ps)


def test_layers_in_one_call(kvq, cuda_dev):
    _check(kvq, cuda_dev, 4, 2, 6, [77, 200], [5, 12], layers=3, seed=3)


def test_many_sequences_and_units(kvq, cuda_dev):
    """More units than SMs, with short caches (whole units per CTA) and longer ones (several
    segments, cut units in the middle of a share), empty trees among them."""
    r = np.random.default_rng(3)
    for n, top, most in ((90, 200, 4), (70, 1400, 3)):
        lens = [int(x) for x in r.integers(0, top, n)]
        nodes = [int(x) for x in r.integers(0, most, n)]
        _check(kvq, cuda_dev, 6, 4, 2, lens, nodes, seed=n, tail=1)


def test_layers_and_cut_units(kvq, cuda_dev):
    _check(kvq, cuda_dev, 8, 2, 6, [700, 1500, 30], [30, 2, 64], layers=2, seed=5)


def test_scores_that_rise_along_the_cache(kvq, cuda_dev):
    """The running maximum moves in every tile."""
    n, nodes = 900, 5
    c = Cache(kvq, cuda_dev, 8, 1, 16, [n], [nodes], seed=11)
    t = np.arange(n + nodes, dtype=np.float64)
    k = np.repeat((t / n * 40)[:, None, None], D, 2).astype(np.float16)
    kvq.kvq_quant_pack_paged(c.kp, [dev_tensor(k, cuda_dev)], c.pt, i32([0, n + nodes], cuda_dev),
                             i32([0], cuda_dev))
    s, codes = osym.quantize_rows(k, 8)
    c.k_hat[0] = osym.dequantize_rows(codes, s)
    q_np = np.full((1, nodes, 6, D), 0.25, dtype=np.float16)
    parents = [_parents(nodes, 1)]
    out, err = _call(kvq, cuda_dev, c, dev_tensor(q_np, cuda_dev), parents)
    assert err == 0
    ref, size, span = _reference(c, q_np[0], parents)
    assert_rows_close(out[0].double().cpu().numpy(), ref, size, span, "f16")


def test_a_chain_equals_single_decode_steps(kvq, cuda_dev):
    """Node i of a chain attends as kvq_decode_attn does over the tokens up to it."""
    c, _, q_np, out = _check(kvq, cuda_dev, 6, 2, 6, [333, 70], [9, 9], chain=True, seed=4)
    for i in range(9):
        lens = [n + i + 1 for n in c.lens]
        q = dev_tensor(q_np[:, [i, 9 + i]].copy(), cuda_dev)
        o = torch.empty(q.shape, dtype=torch.float32, device=cuda_dev)
        ws = kvq.decode_workspace(c.kp, 2, 12, max(lens), cuda_dev)
        kvq.kvq_decode_attn(c.kp, c.vp, q, c.pt, i32(lens, cuda_dev), max(lens),
                            1 / 16, o, ws)
        assert torch.allclose(o, out[:, [i, 9 + i]].float(), atol=2e-3)


def test_drafts_that_a_node_does_not_see_do_not_reach_it(kvq, cuda_dev):
    """A sibling's infinite scales: K (its score is masked) and V (its weight is zero)."""
    c = Cache(kvq, cuda_dev, 6, 1, 16, [100], [6], seed=5)
    parents = [[-1, 0, 0, 1, 2, -1]]
    q_np = kvgen.queries_np(6, 1, 6, 6, D)
    for pools in (c.kp, c.vp):
        for node, x in ((2, float("inf")), (4, float("nan"))):
            t = 100 + node
            pools[0].scales[int(c.pt_np[0, t // 16]), 0, t % 16] = x
    out, err = _call(kvq, cuda_dev, c, dev_tensor(q_np, cuda_dev), parents)
    assert err == 0
    ref, size, span = _reference(c, q_np[0], parents)
    rows = [0, 1, 3, 5]
    assert_rows_close(out[0, rows].double().cpu().numpy(), ref[rows], size[rows], span[rows], "f16")
    assert torch.isnan(out[0, [2, 4]]).any(-1).all()


def test_bad_pages_lengths_and_parents_are_reported_and_skipped(kvq, cuda_dev):
    c = Cache(kvq, cuda_dev, 8, 1, 16, [200, 90], [4, 5], seed=7)
    parents = [_parents(4, 1), _parents(5, 2)]
    q_np = kvgen.queries_np(8, 1, 9, 6, D)
    q = dev_tensor(q_np, cuda_dev)
    good, err = _call(kvq, cuda_dev, c, q, parents)
    assert err == 0
    pt = c.pt.clone()
    pt[0, 3], pt[0, 5] = -1, 10 ** 6
    out, err = _call(kvq, cuda_dev, c, q, parents, pt=pt)
    assert err == kvq.KVQ_DEVERR_PAGE_RANGE
    keep = np.array([t for t in range(204) if t // 16 not in (3, 5)])
    ref, size, span = op.tree_attention(q_np[0, :4], c.k_hat[0][keep], c.v_hat[0][keep], 168,
                                        parents[0], 1 / 16)
    assert_rows_close(out[0, :4].double().cpu().numpy(), ref, size, span, "f16")
    assert torch.equal(out[0, 4:], good[0, 4:])
    for lens, kw in (([200, -1], {}), ([200, 500], {}), (None, dict(max_nodes=4))):
        out, err = _call(kvq, cuda_dev, c, q, parents, lens=lens, **kw)
        assert err == kvq.KVQ_DEVERR_INDEX and (out[0, 4:] == 7).all()
        assert torch.allclose(out[0, :4].float(), good[0, :4].float(), atol=2e-3)
    for bad in (1, 7, -2):
        out, err = _call(kvq, cuda_dev, c, q, [parents[0][:1] + [bad] + parents[0][2:], parents[1]])
        want, _ = _call(kvq, cuda_dev, c, q, [parents[0][:1] + [-1] + parents[0][2:], parents[1]])
        assert err == kvq.KVQ_DEVERR_INDEX and torch.equal(out, want)


def test_all_pages_missing_gives_zero(kvq, cuda_dev):
    c = Cache(kvq, cuda_dev, 6, 1, 16, [40], [2], seed=9)
    q = dev_tensor(kvgen.queries_np(9, 1, 2, 6, D), cuda_dev)
    out, err = _call(kvq, cuda_dev, c, q, [[-1, 0]], pt=torch.full_like(c.pt, -1))
    assert err == kvq.KVQ_DEVERR_PAGE_RANGE and (out == 0).all()


def test_same_bits_every_time_on_two_streams_and_replayed(kvq, cuda_dev):
    c = Cache(kvq, cuda_dev, 6, 2, 16, [3000, 50], [16, 3], seed=10)
    parents = [_parents(16, 1), _parents(3, 2)]
    q = dev_tensor(kvgen.queries_np(10, 1, 19, 12, D), cuda_dev)
    a, _ = _call(kvq, cuda_dev, c, q, parents)
    b, _ = _call(kvq, cuda_dev, c, q, parents)
    assert torch.equal(a, b)
    lens, cu, par = i32(c.lens, cuda_dev), i32(cu_of(c.nodes), cuda_dev), i32(sum(parents, []), cuda_dev)
    ws = [kvq.tree_workspace(c.kp, 2, 19, 12, 16, 3016, cuda_dev) for _ in range(2)]
    outs, s = [torch.zeros_like(q) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            kvq.kvq_tree_attn(c.kp, c.vp, q, c.pt, lens, cu, par, 16, 3016, 1 / 16, outs[i], ws[i],
                              stream=s[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], a) and torch.equal(outs[1], a)
    g, got = torch.cuda.CUDAGraph(), torch.zeros_like(q)
    with torch.cuda.graph(g):
        kvq.kvq_tree_attn(c.kp, c.vp, q, c.pt, lens, cu, par, 16, 3016, 1 / 16, got, ws[0])
    for _ in range(3):
        got.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, a)


# ---------------------------------------------------------------------------------------- commit
@pytest.mark.parametrize("bits,dim,ps", [(6, 256, 16), (8, 256, 16), (4, 128, 32), (8, 50, 7),
                                         (4, 6, 5), (6, 20, 16), (8, 256, 1)])
def test_commit_moves_packed_rows(kvq, cuda_dev, bits, dim, ps):
    lens, H, tensors = [0, 30, 6, 129], 3, 2
    accept = [[0, 2, 3, 9], [63, 5, 5, 0, 1], [], list(range(1, 64))]
    per = -(-(129 + 64) // ps) + 1
    pt_np = kvgen.random_page_table(2, 4, per)
    pools, want = [], []
    g = torch.Generator(device=cuda_dev).manual_seed(1)
    for _ in range(tensors):
        p = kvq.Pool.empty(bits, H, dim, ps, pt_np.size, cuda_dev)
        p.codes.random_(0, 256, generator=g)
        p.scales.copy_(torch.randn(p.scales.shape, generator=g, device=cuda_dev))
        pools.append(p)
        want.append((p.codes.cpu().numpy().copy(), p.scales.cpu().numpy().copy()))
    for codes, scales in want:
        old_c, old_s = codes.copy(), scales.copy()
        for s, (n, path) in enumerate(zip(lens, accept)):
            for i, a in enumerate(path):
                f, t = n + a, n + i
                fp, tp = pt_np[s, f // ps], pt_np[s, t // ps]
                codes[tp, :, t % ps] = old_c[fp, :, f % ps]
                scales[tp, :, t % ps] = old_s[fp, :, f % ps]
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    kvq.kvq_tree_commit(pools, i32(pt_np, cuda_dev), i32(lens, cuda_dev),
                        i32(cu_of([len(a) for a in accept]), cuda_dev),
                        i32(sum(accept, []), cuda_dev), err)
    assert int(err.item()) == 0
    for p, (codes, scales) in zip(pools, want):
        assert np.array_equal(p.codes.cpu().numpy(), codes)
        assert np.array_equal(p.scales.cpu().numpy().view(np.uint16), scales.view(np.uint16))


def test_commit_reports_and_skips_what_is_out_of_range(kvq, cuda_dev):
    p = kvq.Pool.empty(6, 2, 256, 16, 8, cuda_dev)
    p.codes.random_(0, 256)
    p.scales.fill_(1.0)
    before = p.codes.clone()

    def call(table, lens, cu, accept):
        err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
        kvq.kvq_tree_commit([p], i32(table, cuda_dev), i32(lens, cuda_dev), i32(cu, cuda_dev),
                            i32(accept, cuda_dev), err)
        return int(err.item())

    table = [[0, 1], [2, 3]]
    assert call(table, [0, 0], [0, 1, 2], [64, -1]) == kvq.KVQ_DEVERR_INDEX
    assert call(table, [0, -5], [0, 0, 1], [3]) == kvq.KVQ_DEVERR_INDEX
    assert call(table, [0, 0], [0, 5, 2], [1] * 2) == kvq.KVQ_DEVERR_INDEX
    assert call(table, [0, 0], [0, 0, 70], [1] * 70) == kvq.KVQ_DEVERR_INDEX
    assert call(table, [0, 30], [0, 0, 1], [9]) == kvq.KVQ_DEVERR_PAGE_RANGE
    assert call([[0, 1], [8, -1]], [0, 0], [0, 0, 2], [1, 20]) == kvq.KVQ_DEVERR_PAGE_RANGE
    assert torch.equal(p.codes, before)


def test_a_speculative_step_end_to_end(kvq, cuda_dev):
    """Two sequences: prompt through norm, rotation, prompt attention and pages; a drafted tree is
    appended and attended; one path is committed; the cache then decodes as if those tokens had
    been appended alone."""
    Hq, H, bits, ps = 12, 2, 6, 16
    lens, nodes = [50, 33], [7, 5]
    parents = [[-1, 0, 0, 1, 1, 2, 3], [-1, -1, 1, 2, 2]]
    paths = [[0, 1, 3, 6], [1, 2, 4]]
    inv = 1e4 ** (-np.arange(128) / 128)
    ph = kvq.kvq_rope_phases(inv, cuda_dev)
    w = torch.ones(D, device=cuda_dev)
    g = torch.Generator().manual_seed(3)

    def project(n, pos):
        """Rows as a projection leaves them, normed and rotated; V as it is."""
        buf = torch.randn((n, Hq + 2 * H, D), generator=g).half().to(cuda_dev)
        q, k = torch.empty((n, Hq, D), dtype=torch.float16, device=cuda_dev), torch.empty(
            (n, H, D), dtype=torch.float16, device=cuda_dev)
        kvq.kvq_qk_norm_rope(buf[:, :Hq], buf[:, Hq:Hq + H], q, k, i32(pos, cuda_dev), ph, w, w)
        return q, k, buf[:, Hq + H:].contiguous()

    q, k, v = project(sum(lens), list(range(50)) + list(range(33)))
    cu = i32(cu_of(lens), cuda_dev)
    out = torch.empty_like(q)
    kvq.kvq_prompt_attn(q, k, v, cu, cu, 50, 50, 1 / 16, out,
                        kvq.prompt_workspace(2, 83, Hq, H, D, 50, 50, cuda_dev))
    f = [x.double().cpu().numpy() for x in (q, k, v)]
    r = op.prompt_attention(*f, cu_of(lens), cu_of(lens), 1 / 16)
    assert_rows_close(out.double().cpu().numpy(), r["out"], r["size"], r["span"], "f16")

    pt = i32(kvgen.random_page_table(5, 2, 5), cuda_dev)
    kp, vp = (kvq.Pool.empty(bits, H, D, ps, 10, cuda_dev) for _ in range(2))
    zero, lens_t = i32([0, 0], cuda_dev), i32(lens, cuda_dev)
    kvq.kvq_quant_pack_paged([kp, vp], [k, v], pt, cu, zero)
    depth = [[50, 51, 51, 52, 52, 52, 53], [33, 33, 34, 35, 35]]
    dq, dk, dv = project(sum(nodes), sum(depth, []))
    cu_n = i32(cu_of(nodes), cuda_dev)
    kvq.kvq_quant_pack_paged([kp, vp], [dk, dv], pt, cu_n, lens_t)
    out = torch.empty((1, 12, Hq, D), dtype=torch.float16, device=cuda_dev)
    kvq.kvq_tree_attn([kp], [vp], dq[None], pt, lens_t, cu_n, i32(sum(parents, []), cuda_dev), 7, 57,
                      1 / 16, out, kvq.tree_workspace([kp], 2, 12, Hq, 7, 57, cuda_dev))

    def hat(a, b):
        x = torch.cat([a, b]).cpu().numpy()
        s, c = osym.quantize_rows(x, bits)
        return osym.dequantize_rows(c, s)

    for s, (a, b) in enumerate(((0, 50), (50, 83))):
        n0, n1 = cu_of(nodes)[s], cu_of(nodes)[s + 1]
        ref, size, span = op.tree_attention(dq[n0:n1].double().cpu().numpy(),
                                            hat(k[a:b], dk[n0:n1]), hat(v[a:b], dv[n0:n1]),
                                            b - a, parents[s], 1 / 16)
        assert_rows_close(out[0, n0:n1].double().cpu().numpy(), ref, size, span, "f16")

    kvq.kvq_tree_commit([kp, vp], pt, lens_t, i32([0, 4, 7], cuda_dev), i32(sum(paths, []), cuda_dev))
    after = i32([54, 36], cuda_dev)
    q1 = torch.randn((1, 2, Hq, D), generator=g).half().to(cuda_dev)
    got = torch.empty(q1.shape, dtype=torch.float32, device=cuda_dev)
    ws = kvq.decode_workspace([kp], 2, Hq, 60, cuda_dev)
    kvq.kvq_decode_attn([kp], [vp], q1, pt, after, 60, 1 / 16, got, ws)
    kq, vq = (kvq.Pool.empty(bits, H, D, ps, 10, cuda_dev) for _ in range(2))
    kvq.kvq_quant_pack_paged([kq, vq], [k, v], pt, cu, zero)
    keep = torch.tensor(paths[0] + [7 + i for i in paths[1]], device=cuda_dev)
    kvq.kvq_quant_pack_paged([kq, vq], [dk[keep].contiguous(), dv[keep].contiguous()], pt,
                             i32([0, 4, 7], cuda_dev), lens_t)
    want = torch.empty_like(got)
    kvq.kvq_decode_attn([kq], [vq], q1, pt, after, 60, 1 / 16, want, ws)
    assert torch.equal(got, want)


@pytest.mark.parametrize("bits", [8, 6, 4])
@pytest.mark.parametrize("G", [3, 5, 6, 7, 16])
def test_row_tiles_that_cut_a_drafts_heads(kvq, cuda_dev, bits, G):
    nodes = [64, 43, 22, 21, 1]
    _check(kvq, cuda_dev, bits, 2, G, [70, 300, 5, 0, 129], nodes, seed=50 + G)     # whole units
    _check(kvq, cuda_dev, bits, 2, G, [2600, 300, 1500, 0, 129], nodes, ps=32, seed=60 + G, tail=1)


@pytest.mark.parametrize("bits", [8, 6, 4])
@pytest.mark.parametrize("length", [100, 2500])     # a whole unit, a unit cut over several CTAs
def test_seen_infinite_values_reach_their_rows_and_channels_only(kvq, cuda_dev, bits, length):
    c = Cache(kvq, cuda_dev, bits, 1, 16, [length], [30], seed=7)
    parents = [[-1, 0, 0, 1, 2, -1, 4, 3] + [3] * 22]
    q_np = kvgen.queries_np(8, 1, 30, 6, D)
    t = length + 2
    c.vp[0].scales[int(c.pt_np[0, t // 16]), 0, t % 16] = float("inf")
    out, err = _call(kvq, cuda_dev, c, dev_tensor(q_np, cuda_dev), parents)
    assert err == 0
    out = out[0].double().cpu().numpy()
    ref, size, span = _reference(c, q_np[0], parents)
    sees = [i for i in range(30) if i == 2 or op.ancestors(parents[0])[i, 2]]
    rest = [i for i in range(30) if i not in sees]
    assert sees == [2, 4, 6]
    assert_rows_close(out[rest], ref[rest], size[rest], span[rest], "f16")
    v = c.v_hat[0].reshape(-1, D)[t].astype(np.float64)       # its codes' signs; code 0: 0 * inf
    want = np.where(v > 0, np.inf, np.where(v < 0, -np.inf, np.nan))
    for i in sees:
        for g in range(6):
            assert np.array_equal(out[i, g], want, equal_nan=True)


def test_pages_behind_four_billion_bytes(kvq, cuda_dev):
    """The same bits from small pools and from pools whose pages lie past 2^32 bytes."""
    c = Cache(kvq, cuda_dev, 8, 4, 16, [150], [9], seed=9)
    parents = [[-1, 0, 0, 1, 2, 2, 4, -1, 7]]
    q = dev_tensor(kvgen.queries_np(10, 1, 9, 8, D), cuda_dev)
    small, err = _call(kvq, cuda_dev, c, q, parents)
    assert err == 0
    first = 265000                                     # pages of 16 KB
    accept, cu = i32([0, 2, 4], cuda_dev), i32([0, 3], cuda_dev)
    pools = []
    for p in c.kp + c.vp:
        b = kvq.Pool.empty(8, 4, D, 16, first + p.codes.shape[0], cuda_dev)
        b.codes[first:], b.scales[first:] = p.codes, p.scales
        pools.append(b)
    small_pools, pt = c.kp + c.vp, c.pt + first
    c.kp, c.vp = pools[:1], pools[1:]
    big, err = _call(kvq, cuda_dev, c, q, parents, pt=pt)
    assert err == 0 and torch.equal(big, small)
    lens = i32([150], cuda_dev)
    kvq.kvq_tree_commit(small_pools, c.pt, lens, cu, accept)
    kvq.kvq_tree_commit(pools, pt, lens, cu, accept)
    for a, b in zip(small_pools, pools):
        assert torch.equal(a.codes, b.codes[first:])
        assert torch.equal(a.scales.view(torch.int16), b.scales[first:].view(torch.int16))
