"""The tiled attention kernels give up cleanly when a wait between their roles runs out (GPU).

Every wait of prompt and tree attention for a copy, a product or another role is bounded; one that
runs out sets KVQ_DEVERR_TIMEOUT, every role leaves (meeting the others at the barriers that have no
limit of their own), and the block ends with no copy or product in flight.
Here the kernels are built again with limits of 0 polls (every wait gives up at once, while the first
copies are in flight), 1 and 20 (some waits succeed, so that roles give up at different places, or
none does).  Each call has to return, report the time-out or be right, leave the rows that belong to
no sequence alone, and leave the context usable: the library's own build then computes the same
call correctly.  No fault is planted and nothing waits without a bound."""
import concurrent.futures as cf
import ctypes
import os
import subprocess

import pytest
import torch

import kvgen
from conftest import ROOT
from oracle import prompt as op
from _gpu_util import cu_of, dev_tensor, i32
from _operator_checks import assert_rows_close
from test_gpu_tree_attn import Cache, _parents, _reference

pytestmark = pytest.mark.gpu

CSRC = os.path.join(ROOT, "paged_kv_cache_fp16_gb300", "csrc")
LIMITS = (0, 1, 20)


@pytest.fixture(scope="module")
def short_wait_libs(kvq):
    out_dir = os.path.join(ROOT, "tests", "_build")
    os.makedirs(out_dir, exist_ok=True)
    nvcc = os.environ.get("NVCC", "nvcc")
    arch = ["-gencode", "arch=compute_103a,code=sm_103a"]
    flags = arch + ["-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
                    "-I", os.path.join(ROOT, "include"), "-I", CSRC, "--expt-relaxed-constexpr",
                    "-diag-suppress", "177"]

    def compile_one(job):
        name, limit = job
        obj = os.path.join(out_dir, f"tile_wait{limit}_{name}.o")
        subprocess.run([nvcc] + flags + [f"-DKVQ_TILE_WAIT_LIMIT={limit}", "-c",
                                         os.path.join(CSRC, name), "-o", obj],
                       check=True, capture_output=True)
        return obj

    names = ["prompt_attn.cu", "tree_attn.cu", "host.cpp"]
    jobs = [(n, x) for x in LIMITS for n in names]
    with cf.ThreadPoolExecutor(len(jobs)) as ex:
        objs = list(ex.map(compile_one, jobs))
    libs = {}
    for i, limit in enumerate(LIMITS):
        so = os.path.join(out_dir, f"kvq_tile_wait{limit}.so")
        subprocess.run([nvcc] + arch + ["-shared", "-o", so] + objs[i * len(names):(i + 1) * len(names)],
                       check=True, capture_output=True)
        libs[limit] = ctypes.CDLL(so)
        for name in ("kvq_prompt_attn", "kvq_tree_attn"):
            fn, like = getattr(libs[limit], name), getattr(kvq._lib, name)
            fn.restype, fn.argtypes = like.restype, like.argtypes
    return libs


def _outcome(kvq, err, limit, check):
    """A call with a short limit: the time-out, or the right result."""
    assert err in (0, kvq.KVQ_DEVERR_TIMEOUT)
    if limit == 0:
        assert err == kvq.KVQ_DEVERR_TIMEOUT
    if err == 0:
        check()


@pytest.mark.parametrize("limit", LIMITS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new,keys", [([130, 40], [300, 40]), ([1], [3000]), ([700], [700])])
def test_prompt_attention_gives_up_cleanly(kvq, cuda_dev, short_wait_libs, limit, D, new, keys):
    Hq, H, tail, scale = 6, 2, 3, D ** -0.5
    g = torch.Generator().manual_seed(D + sum(keys))
    q, k, v = (torch.randn((n, h, D), generator=g).half().to(cuda_dev)
               for n, h in ((sum(new) + tail, Hq), (sum(keys), H), (sum(keys), H)))
    cu_q, cu_k = i32(cu_of(new), cuda_dev), i32(cu_of(keys), cuda_dev)
    ws = kvq.prompt_workspace(len(new), sum(new) + tail, Hq, H, D, max(new), max(keys), cuda_dev)
    out, err = torch.full_like(q, 7.0), i32([0], cuda_dev)
    ref = op.prompt_attention(*(x.double().cpu().numpy() for x in (q, k, v)), cu_of(new), cu_of(keys),
                              scale)
    n = sum(new)
    right = lambda: assert_rows_close(out[:n].double().cpu().numpy(), ref["out"][:n], ref["size"][:n],
                                      ref["span"][:n], "f16")
    for _ in range(3):
        ws.fill_(255)
        out.fill_(7.0)
        err.zero_()
        st = short_wait_libs[limit].kvq_prompt_attn(
            kvq.KVQ_F16, q.data_ptr(), Hq * D, k.data_ptr(), H * D, v.data_ptr(), H * D, Hq, H, D,
            cu_q.data_ptr(), cu_k.data_ptr(), len(new), q.shape[0], k.shape[0], max(new), max(keys),
            scale, out.data_ptr(), None, ws.data_ptr(), ws.numel(), err.data_ptr(),
            torch.cuda.current_stream().cuda_stream)
        assert st == 0
        torch.cuda.synchronize()
        _outcome(kvq, int(err.item()), limit, right)
        assert (out[n:] == 7).all()
    err.zero_()
    kvq.kvq_prompt_attn(q, k, v, cu_q, cu_k, max(new), max(keys), scale, out, ws, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and (out[n:] == 7).all()
    right()


@pytest.mark.parametrize("limit", LIMITS)
@pytest.mark.parametrize("bits", [8, 6, 4])
@pytest.mark.parametrize("H,G,lens,nodes", [
    (2, 6, [300, 0, 70], [20, 64, 1]),            # whole units, idle row warps among them
    (4, 2, [40, 90] * 50, [3, 2] * 50),           # several units per CTA
    (1, 6, [9000, 100, 4001], [16, 64, 3]),       # cut units, joined
    (4, 2, [700, 1400] * 20, [2, 5] * 20)])       # several segments per share, cut at both ends
def test_tree_attention_gives_up_cleanly(kvq, cuda_dev, short_wait_libs, limit, bits, H, G, lens,
                                         nodes):
    tail, scale, n = 2, 1 / 16, sum(nodes)
    c = Cache(kvq, cuda_dev, bits, H, 16, lens, nodes, seed=bits + G)
    parents = [_parents(x, i) for i, x in enumerate(nodes)]
    q_np = kvgen.queries_np(7, 1, n + tail, H * G, 256)
    q = dev_tensor(q_np, cuda_dev)
    lens_t, cu, par = (i32(x, cuda_dev) for x in (lens, cu_of(nodes), sum(parents, []) + [-1] * tail))
    most, longest = max(nodes), max(a + b for a, b in zip(lens, nodes))
    ws = kvq.tree_workspace(c.kp, len(lens), n + tail, H * G, most, longest, cuda_dev)
    out, err = torch.full_like(q, 7.0), i32([0], cuda_dev)
    ref, size, span = _reference(c, q_np[0, :n], parents)
    right = lambda: assert_rows_close(out[0, :n].double().cpu().numpy(), ref, size, span, "f16")
    for _ in range(3):
        ws.fill_(255)
        out.fill_(7.0)
        err.zero_()
        st = short_wait_libs[limit].kvq_tree_attn(
            kvq._pool_array(c.kp), kvq._pool_array(c.vp), 1, q.data_ptr(), H * G, c.pt.data_ptr(),
            c.pt.shape[1], lens_t.data_ptr(), cu.data_ptr(), par.data_ptr(), len(lens), n + tail, most,
            longest, scale, out.data_ptr(), ws.data_ptr(), ws.numel(), err.data_ptr(),
            torch.cuda.current_stream().cuda_stream)
        assert st == 0
        torch.cuda.synchronize()
        _outcome(kvq, int(err.item()), limit, right)
        assert (out[:, n:] == 7).all()
    err.zero_()
    kvq.kvq_tree_attn(c.kp, c.vp, q, c.pt, lens_t, cu, par, most, longest, scale, out, ws, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and (out[:, n:] == 7).all()
    right()
