"""The plan of large page tables gives up cleanly when its blocks do not meet (GPU).

The blocks of a cooperative grid wait for each other a bounded number of polls.  Here the kernels are built
again with limits of 0 polls (every block gives up at once) and of a few (some blocks meet, others have left
by then).  The workspace holds what a complete call on another state left there, so that moves by what a
missing block did not write would be moves of pages.  Each call has to return; one that reports the time-out
leaves the pools as they were, one that does not is right; the context stays usable.  Nothing waits without
a bound, and no limit makes an access leave its buffers: a plan that gave up moves nothing."""
import concurrent.futures as cf
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from conftest import ROOT
from oracle import beams as ob
from _gpu_util import i32
from test_gpu_tables import State, _bytes, _pools

pytestmark = pytest.mark.gpu

CSRC = os.path.join(ROOT, "paged_kv_cache_fp16_gb300", "csrc")
LIMITS = (0, 1, 8, 60)


@pytest.fixture(scope="module")
def short_meet_libs(kvq):
    out_dir = os.path.join(ROOT, "tests", "_build")
    os.makedirs(out_dir, exist_ok=True)
    nvcc = os.environ.get("NVCC", "nvcc")
    arch = ["-gencode", "arch=compute_103a,code=sm_103a"]
    flags = arch + ["-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
                    "-I", os.path.join(ROOT, "include"), "-I", CSRC, "--expt-relaxed-constexpr",
                    "-diag-suppress", "177"]

    def compile_one(job):
        name, limit = job
        obj = os.path.join(out_dir, f"meet_wait{limit}_{name}.o")
        subprocess.run([nvcc] + flags + [f"-DKVQ_MEET_WAIT_LIMIT={limit}", "-c", os.path.join(CSRC, name),
                                         "-o", obj], check=True, capture_output=True)
        return obj

    names = ["table_ops.cu", "host.cpp"]
    with cf.ThreadPoolExecutor(8) as ex:
        objs = list(ex.map(compile_one, [(n, x) for x in LIMITS for n in names]))
    libs = {}
    for i, limit in enumerate(LIMITS):
        so = os.path.join(out_dir, f"kvq_meet_wait{limit}.so")
        subprocess.run([nvcc] + arch + ["-shared", "-o", so] + objs[2 * i:2 * i + 2], check=True,
                       capture_output=True)
        libs[limit] = ctypes.CDLL(so)
        for name in ("kvq_table_update", "kvq_table_compact"):
            fn, like = getattr(libs[limit], name), getattr(kvq._lib, name)
            fn.restype, fn.argtypes = like.restype, like.argtypes
    return libs


def _same(pools, want):
    return all(np.array_equal(a, c) and np.array_equal(b, s)
               for (a, b), (c, s) in zip(_bytes(pools), want))


@pytest.mark.parametrize("limit", LIMITS)
def test_update_gives_up_cleanly(kvq, cuda_dev, short_meet_libs, limit):
    n = 64
    st = State(9, n, 16, 40000, spare=4 * n, outside=False)
    assert st.num_pages + n * st.width > 1 << 17              # beyond a cluster's share
    pools = _pools(kvq, cuda_dev, st, 4, 2, 64, 2)
    before = _bytes(pools)
    parents = np.random.default_rng(1).integers(0, n, n).tolist()
    rows, lens, refs, copies = ob.table_update(st.table, st.lens, st.held, st.refs, parents, [3] * n, 16)
    after = [(c.copy(), s.copy()) for c, s in before]
    for c, s in after:
        for a, b, k in copies:
            c[b, :, :k], s[b, :, :k] = c[a, :, :k], s[a, :, :k]
    assert copies
    other = [0] * n                                           # the call before: copies of one page
    ins = [i32(x, cuda_dev) for x in (st.table, st.lens, st.held, st.refs, other, [3] * n)]
    outs = [torch.full((n, st.width), -7, dtype=torch.int32, device=cuda_dev),
            *(torch.empty(n, dtype=torch.int32, device=cuda_dev) for _ in range(2)),
            torch.empty(st.num_pages, dtype=torch.int32, device=cuda_dev)]
    ws, err = kvq.table_workspace(st.num_pages, n, cuda_dev), i32([0], cuda_dev)
    words = kvq._pool_array(pools)

    def call(fn, par):
        ins[4].copy_(i32(par, cuda_dev))
        err.zero_()
        assert fn(words, len(pools), ins[0].data_ptr(), st.width, ins[1].data_ptr(), ins[2].data_ptr(), n,
                  ins[3].data_ptr(), ins[4].data_ptr(), ins[5].data_ptr(), n, outs[0].data_ptr(),
                  outs[1].data_ptr(), outs[2].data_ptr(), outs[3].data_ptr(), ws.data_ptr(), ws.numel(),
                  err.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        return int(err.item())

    def right():
        assert outs[1].tolist() == lens and np.array_equal(outs[3].cpu().numpy(), refs)
        assert all(outs[0][s, :len(r)].tolist() == r for s, r in enumerate(rows)) and _same(pools, after)

    for _ in range(6):
        assert call(kvq._lib.kvq_table_update, other) == 0
        for p, (c, s) in zip(pools, before):
            p.codes.copy_(torch.from_numpy(c))
            p.scales.copy_(torch.from_numpy(s.view(np.float16)))
        got = call(short_meet_libs[limit].kvq_table_update, parents)
        assert got in (0, kvq.KVQ_DEVERR_TIMEOUT) and (limit or got)
        if got:
            assert _same(pools, before)
        else:
            right()
    assert call(kvq._lib.kvq_table_update, parents) == 0
    right()


@pytest.mark.parametrize("limit", LIMITS)
def test_compaction_gives_up_cleanly(kvq, cuda_dev, short_meet_libs, limit):
    n = 30
    st = State(4, n, 16, 3000, spare=140000)
    pools = _pools(kvq, cuda_dev, st, 4, 1, 64, 2)
    before = _bytes(pools)
    rows, refs, live, moves = ob.table_compact(st.table, st.held, st.refs)
    after = [(c.copy(), s.copy()) for c, s in before]
    for c, s in after:
        for a, b in moves:
            c[b], s[b] = c[a], s[a]
    other = np.random.default_rng(5).permutation(st.refs)     # the call before: other pages in use
    ins = [i32(x, cuda_dev) for x in (st.table, st.held, st.refs)]
    outs = [torch.full(st.table.shape, -7, dtype=torch.int32, device=cuda_dev),
            torch.empty(st.num_pages, dtype=torch.int32, device=cuda_dev), i32([0], cuda_dev)]
    ws, err = kvq.table_workspace(st.num_pages, n, cuda_dev), i32([0], cuda_dev)
    words = kvq._pool_array(pools)

    def call(fn, counts, held):
        ins[1].copy_(i32(held, cuda_dev))
        ins[2].copy_(i32(counts, cuda_dev))
        err.zero_()
        assert fn(words, len(pools), ins[0].data_ptr(), st.width, ins[1].data_ptr(), n, ins[2].data_ptr(),
                  outs[0].data_ptr(), outs[1].data_ptr(), outs[2].data_ptr(), ws.data_ptr(), ws.numel(),
                  err.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        return int(err.item())

    def right():
        assert outs[2].item() == live and np.array_equal(outs[1].cpu().numpy(), refs)
        assert all(outs[0][s, :len(r)].tolist() == r for s, r in enumerate(rows)) and _same(pools, after)

    for _ in range(6):
        assert call(kvq._lib.kvq_table_compact, other, [0] * n) == 0
        for p, (c, s) in zip(pools, before):
            p.codes.copy_(torch.from_numpy(c))
            p.scales.copy_(torch.from_numpy(s.view(np.float16)))
        got = call(short_meet_libs[limit].kvq_table_compact, st.refs, st.held)
        assert got in (0, kvq.KVQ_DEVERR_TIMEOUT) and (limit or got)
        if got:
            assert _same(pools, before)
        else:
            right()
    assert call(kvq._lib.kvq_table_compact, st.refs, st.held) == 0
    right()
