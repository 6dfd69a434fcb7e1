"""Workloads of the serving operators around the packed cache: per-head query/key norm with the
position rotation, attention over whole prompts, attention of a tree of drafted tokens over the
packed pages, and the commit of the accepted drafts.

Each case is a dict of plain values.  `run` computes a case's operator on what `prepare` made:
in elementary torch operations where `own` is false, and through this library's entry points
where it is true.  `exact` is the operator's definition in 64 bits.

The sizes are those of the library's own workloads: 24 query heads over 4 KV heads of 256 channels
(the paged cache), 32 over 8 of 64 (the KIVI cache), and 16 over 4 of 128 between the two; 16-token
pages in a random order; up to 262,144 cached tokens.
"""
from __future__ import annotations

import math
import random

import torch

own = False

HEADS = {256: (24, 4), 128: (16, 4), 64: (32, 8)}     # head_dim -> query heads, KV heads
QMAX = {8: 127, 6: 31, 4: 7}
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
PAGE = 16
MAX_NODES = 64


# ------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of 64 sequences: every token's 28 rows, positions up to 64k
        dict(name="norm_rope step 64", op="norm_rope", tokens=64, dim=256, dtype="f16",
             rotary=256, interleaved=False, far=65536),
        # a 32,768-token prompt, read from the fused projection's output
        dict(name="norm_rope prompt 32768", op="norm_rope", tokens=32768, dim=256, dtype="f16",
             rotary=256, interleaved=False, far=262144),
        # bf16 rows of 64 channels, half of them rotated, pairs interleaved, an odd count
        dict(name="norm_rope bf16 5003", op="norm_rope", tokens=5003, dim=64, dtype="bf16",
             rotary=32, interleaved=True, far=262144),
        # one short prompt: latency
        dict(name="prompt 1x128", op="prompt", nseq=1, new=128, past=0, ragged=False, dim=256,
             dtype="f16", lse=False, mix=1),
        # one long prompt
        dict(name="prompt 1x16384", op="prompt", nseq=1, new=16384, past=0, ragged=False, dim=256,
             dtype="f16", lse=False, mix=2),
        # a batch of prompts of very different lengths, 64-channel heads
        dict(name="prompt 8 ragged bf16", op="prompt", nseq=8, new=2501, past=0, ragged=True,
             dim=64, dtype="bf16", lse=False, mix=3),
        # a prompt's next chunk over what is already there, for four sequences; with the row
        # statistics that a merge with other keys needs
        dict(name="prompt 4x37 over 20011", op="prompt", nseq=4, new=37, past=20011, ragged=True,
             dim=128, dtype="f16", lse=True, mix=4),
        # a small draft over a short cache: latency
        dict(name="tree q4 1x300", op="tree", bits=4, nseq=1, length=300, nodes=4, ragged=False,
             chain=False, mix=5),
        # a 16-node tree over the full context
        dict(name="tree q6 1x262144", op="tree", bits=6, nseq=1, length=262144, nodes=16,
             ragged=False, chain=False, mix=6),
        # eight sequences of different lengths with trees of up to 64 nodes
        dict(name="tree q8 8 ragged", op="tree", bits=8, nseq=8, length=32768, nodes=64,
             ragged=True, chain=False, mix=7),
        # the accepted path of one sequence, one layer
        dict(name="commit q4 1x1", op="commit", bits=4, layers=1, nseq=1, nodes=16, mix=8),
        # the accepted paths of 64 sequences in all 16 layers
        dict(name="commit q6 16x64", op="commit", bits=6, layers=16, nseq=64, nodes=32, mix=9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "prompt", "prompt", "tree", "tree", "commit"])
    mix = rng.randrange(1 << 30)
    if op == "norm_rope":
        dim = rng.choice([64, 128, 256])
        return dict(op=op, tokens=_log(rng, 1, 32768), dim=dim, dtype=rng.choice(["f16", "bf16"]),
                    rotary=rng.choice([dim, dim // 2]), interleaved=rng.random() < 0.5,
                    far=_log(rng, 32768, 1 << 20))
    if op == "prompt":
        dim = rng.choice([64, 128, 256])
        nseq = _log(rng, 1, 16)
        kind = rng.choice(["prompt", "chunk", "step"])
        if kind == "prompt":
            new, past = _log(rng, 1, 8192 // nseq), 0
        elif kind == "chunk":
            new = _log(rng, 2, 512)
            past = _log(rng, 1, 32768 // nseq)
        else:
            new, past = 1, _log(rng, 1, 131072 // nseq)
        return dict(op=op, nseq=nseq, new=new, past=past, ragged=rng.random() < 0.7, dim=dim,
                    dtype=rng.choice(["f16", "bf16"]), lse=rng.random() < 0.5, mix=mix)
    if op == "tree":
        nseq = _log(rng, 1, 64)
        return dict(op=op, bits=rng.choice([8, 6, 4]), nseq=nseq,
                    length=_log(rng, 1, 262144 // nseq), nodes=_log(rng, 1, MAX_NODES),
                    ragged=rng.random() < 0.7, chain=rng.random() < 0.25, mix=mix)
    return dict(op=op, bits=rng.choice([8, 6, 4]), layers=_log(rng, 1, 16), nseq=_log(rng, 1, 64),
                nodes=_log(rng, 1, MAX_NODES), mix=mix)


# ------------------------------------------------------------------ what a case alone determines
def _lens(case):
    """Per sequence: (new tokens, all keys) of a prompt; (cached, nodes) of a tree or a commit."""
    r = random.Random(case["mix"])
    n = case["nseq"]
    if case["op"] == "prompt":
        new = [case["new"]] * n
        past = [case["past"]] * n
        if case["ragged"]:
            new = [case["new"]] + [r.randint(1, case["new"]) for _ in range(n - 1)]
            past = [case["past"]] + [r.randint(0, case["past"]) for _ in range(n - 1)]
        return new, [a + b for a, b in zip(new, past)]
    if case["op"] == "commit":
        return [r.randint(0, 65536) for _ in range(n)], [case["nodes"]] * n
    length = [case["length"]] * n
    nodes = [case["nodes"]] * n
    if case["ragged"]:
        length = [case["length"]] + [r.randint(case["length"] // 32, case["length"])
                                     for _ in range(n - 1)]
        nodes = [case["nodes"]] + [r.randint(1, case["nodes"]) for _ in range(n - 1)]
    return length, nodes


def _parents(case, nodes):
    """A draft tree per sequence: node i hangs on one of the nodes before it, or on the cache."""
    r = random.Random(case["mix"] + 1)
    return [[i - 1 if case.get("chain") else r.randint(max(-1, i - 6), i - 1) for i in range(n)]
            for n in nodes]


def _accepted(case, nodes):
    """One root-to-leaf path per sequence, as ascending node numbers."""
    out = []
    for par in _parents(case, nodes):
        i, path = len(par) - 1, []
        while i >= 0:
            path.append(i)
            i = par[i]
        out.append(path[::-1])
    return out


def _packed_dim(bits):
    return 256 * bits // 8


def work(case):
    if case["op"] == "norm_rope":
        hq, h = HEADS[case["dim"]]
        n = case["tokens"] * (hq + h) * case["dim"]
        return {"bytes": 4 * n + 4 * case["tokens"], "flops": 8 * n}
    if case["op"] == "prompt":
        hq, h = HEADS[case["dim"]]
        new, keys = _lens(case)
        seen = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(new, keys))
        return {"bytes": 2 * case["dim"] * (2 * hq * sum(new) + 2 * h * sum(keys)),
                "flops": 4 * case["dim"] * hq * seen}
    if case["op"] == "tree":
        hq, h = HEADS[256]
        length, nodes = _lens(case)
        rows = sum(length) + sum(nodes)
        return {"bytes": 2 * h * rows * (_packed_dim(case["bits"]) + 2) + 4 * 256 * hq * sum(nodes)
                + 4 * (rows // PAGE), "flops": 4 * 256 * hq * sum(a * b for a, b in zip(length, nodes))}
    _, nodes = _lens(case)
    rows = sum(len(p) for p in _accepted(case, nodes)) * 2 * case["layers"] * HEADS[256][1]
    return {"bytes": 2 * rows * (_packed_dim(case["bits"]) + 2), "flops": 0}


# ------------------------------------------------------------------------------------ the inputs
def _cu(lens):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()


def _pack(codes, bits):
    """Signed codes int8 [..., 256] -> the packed bytes of a row."""
    if bits == 8:
        return codes.view(torch.uint8)
    if bits == 4:
        u = (codes + 8).to(torch.uint8).unflatten(-1, (-1, 2))
        return u[..., 0] | (u[..., 1] << 4)
    u = (codes + 32).to(torch.uint8).unflatten(-1, (-1, 4))
    a, b, c, d = u.unbind(-1)
    return torch.stack([a | ((b & 3) << 6), (b >> 2) | ((c & 15) << 4), (c >> 4) | (d << 2)],
                       -1).flatten(-2)


def _pool(case, pages, gen, key):
    """Codes and scales of a pool as the symmetric quantizer leaves them: N(0,1) rows, keys with
    four channels x10."""
    h, bits = HEADS[256][1], case["bits"]
    x = torch.randn((pages, h, PAGE, 256), generator=gen, device="cuda", dtype=torch.float16)
    if key:
        x[..., [5, 77, 130, 201]] *= 10
    scale = (x.abs().amax(-1).float() / QMAX[bits]).half()
    codes = torch.round(x.float() / scale.float()[..., None]).clamp_(-QMAX[bits], QMAX[bits])
    return _pack(codes.to(torch.int8), bits).contiguous(), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float16):
        return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)

    st = dict(case=case)
    if case["op"] == "norm_rope":
        t, dim, dt = case["tokens"], case["dim"], DTYPES[case["dtype"]]
        hq, h = HEADS[dim]
        qkv = normal(t, hq + 2 * h, dim, dtype=dt)      # the fused projection's output
        st["q"], st["k"] = qkv[:, :hq], qkv[:, hq:hq + h]
        st["qo"] = torch.empty((t, hq, dim), dtype=dt, device="cuda")
        st["ko"] = torch.empty((t, h, dim), dtype=dt, device="cuda")
        st["qw"] = 1 + 0.2 * normal(dim, dtype=torch.float32)
        st["kw"] = 1 + 0.2 * normal(dim, dtype=torch.float32)
        st["pos"] = torch.randint(0, case["far"], (t,), generator=gen, device="cuda",
                                  dtype=torch.int32)
        half = case["rotary"] // 2
        st["inv_freq"] = 1e6 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        if own:   # the frequencies in the form that the kernel reads, made once per model
            import paged_kv_cache_fp16_gb300 as kvq
            st["phases"] = kvq.kvq_rope_phases(st["inv_freq"])
        return st
    if case["op"] == "prompt":
        dim, dt = case["dim"], DTYPES[case["dtype"]]
        hq, h = HEADS[dim]
        new, keys = _lens(case)
        if case["past"] == 0:    # a prompt's own keys: all three out of the fused projection
            qkv = normal(sum(new), hq + 2 * h, dim, dtype=dt)
            st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + h], qkv[:, hq + h:]
        else:
            st["q"] = normal(sum(new), hq, dim, dtype=dt)
            st["k"] = normal(sum(keys), h, dim, dtype=dt)
            st["v"] = normal(sum(keys), h, dim, dtype=dt)
        st["cu_q"], st["cu_k"] = _cu(new), _cu(keys)
        st["max_q"], st["max_k"] = max(new), max(keys)
        st["out"] = torch.empty((sum(new), hq, dim), dtype=dt, device="cuda")
        st["lse"] = (torch.empty((sum(new), hq), dtype=torch.float32, device="cuda")
                     if case["lse"] else None)
        if own:   # scratch that a program keeps
            import paged_kv_cache_fp16_gb300 as kvq
            st["ws"] = kvq.prompt_workspace(case["nseq"], sum(new), hq, h, dim, max(new), max(keys))
        return st
    hq, h = HEADS[256]
    length, nodes = _lens(case)
    n = case["nseq"]
    host = torch.Generator().manual_seed(seed)
    st["seq_lens"] = torch.tensor(length, dtype=torch.int32).cuda()
    if case["op"] == "tree":
        width = max(-(-(a + b) // PAGE) for a, b in zip(length, nodes))
        pages = n * width
        st["table"] = torch.randperm(pages, generator=host).to(torch.int32).view(n, width).cuda()
        st["kc"], st["ks"] = _pool(case, pages, gen, True)
        st["vc"], st["vs"] = _pool(case, pages, gen, False)
        st["q"] = normal(1, sum(nodes), hq, 256)
        st["cu_nodes"] = _cu(nodes)
        st["parents"] = torch.tensor(sum(_parents(case, nodes), []), dtype=torch.int32).cuda()
        st["max_nodes"], st["max_len"] = max(nodes), max(a + b for a, b in zip(length, nodes))
        st["out"] = torch.empty_like(st["q"])
        if own:   # the pools' descriptions and scratch that a program keeps
            import paged_kv_cache_fp16_gb300 as kvq
            st["kp"] = [kvq.Pool(case["bits"], h, 256, PAGE, st["kc"], st["ks"])]
            st["vp"] = [kvq.Pool(case["bits"], h, 256, PAGE, st["vc"], st["vs"])]
            st["ws"] = kvq.tree_workspace(st["kp"], n, sum(nodes), hq, max(nodes), st["max_len"])
        return st
    # commit: only the pages that hold drafts are mapped (the others are not touched)
    per = -(-case["nodes"] // PAGE) + 1
    table = torch.full((n, 65536 // PAGE + per + 1), -1, dtype=torch.int32)
    first = torch.tensor(length)[:, None] // PAGE + torch.arange(per)
    table.scatter_(1, first, torch.randperm(n * per, generator=host).to(torch.int32).view(n, per))
    st["table"] = table.cuda()
    st["pools"] = [_pool(case, n * per, gen, i % 2 == 0) for i in range(2 * case["layers"])]
    path = _accepted(case, nodes)
    st["accept"] = torch.tensor(sum(path, []), dtype=torch.int32).cuda()
    st["cu_accept"] = _cu([len(p) for p in path])
    if own:
        import paged_kv_cache_fp16_gb300 as kvq
        st["kp"] = [kvq.Pool(case["bits"], h, 256, PAGE, c, s) for c, s in st["pools"]]
    return st


# ----------------------------------------------------------------------------- the plain forms
def _plain_norm_rope(x, w, cos, sin, interleaved):
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
    half = cos.shape[-1]
    rot, rest = y[..., :2 * half], y[..., 2 * half:]
    if interleaved:
        a, b = rot[..., 0::2], rot[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = rot[..., :half], rot[..., half:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, rest], -1)


def _padded(x, cu, most):
    """Rows of packed sequences [total, H, D] -> float32 [nseq, H, most, D] and which are real."""
    at = cu[:-1, None].long() + torch.arange(most, device="cuda")
    real = at < cu[1:, None]
    return x[at.clamp(max=x.shape[0] - 1)].float().transpose(1, 2), real


def _softmax_v(s, seen, v):
    """s [..., rows, keys] (overwritten), seen broadcastable to it: sum of softmax(s) v, and the
    logarithm of the sum of exponentials; rows that see nothing are 0 and -inf."""
    s.masked_fill_(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total == 0, 1.0, total)
    return out, (top + total.log()).squeeze(-1)


def _plain_prompt(st):
    case = st["case"]
    hq, h = HEADS[case["dim"]]
    mq, mk, n = st["max_q"], st["max_k"], case["nseq"]
    q, q_real = _padded(st["q"], st["cu_q"], mq)
    k, k_real = _padded(st["k"], st["cu_k"], mk)
    v, _ = _padded(st["v"], st["cu_k"], mk)
    lq, lk = st["cu_q"].diff()[:, None], st["cu_k"].diff()[:, None]
    last = torch.arange(mq, device="cuda") + lk - lq                    # the last key each row sees
    seen = (torch.arange(mk, device="cuda") <= last[..., None]) & k_real[:, None]
    s = (q.reshape(n, h, -1, case["dim"]) @ k.transpose(-1, -2)).mul_(case["dim"] ** -0.5)
    o, lse = _softmax_v(s.view(n, h, hq // h, mq, mk), seen[:, None, None],
                        v.masked_fill(~k_real[:, None, :, None], 0)[:, :, None])
    o = o.reshape(n, hq, mq, -1).transpose(1, 2)[q_real].to(st["q"].dtype)
    return (o, lse.reshape(n, hq, mq).transpose(1, 2)[q_real]) if case["lse"] else o


def _unpack(b, bits):
    if bits == 8:
        return b.view(torch.int8).float()
    if bits == 4:
        return torch.stack([b & 15, b >> 4], -1).flatten(-2).float() - 8
    x, y, z = b.unflatten(-1, (-1, 3)).unbind(-1)
    return torch.stack([x & 63, (x >> 6) | ((y & 15) << 2), (y >> 4) | ((z & 3) << 4), z >> 2],
                       -1).flatten(-2).float() - 32


def _rows(codes, scales, table, most, bits):
    """The first `most` tokens of every sequence as the cache stands for them, [nseq, H, most, D]."""
    t = torch.arange(most, device="cuda")
    page = table[:, t // PAGE].long()
    x = _unpack(codes[page, :, t % PAGE], bits) * scales[page, :, t % PAGE].float()[..., None]
    return x.half().float().transpose(1, 2)


def _closure(m):
    return (m @ m > 0).float()


def _plain_tree(st):
    case = st["case"]
    hq, h = HEADS[256]
    n, most, mn = case["nseq"], st["max_len"], st["max_nodes"]
    q, q_real = _padded(st["q"][0], st["cu_nodes"], mn)
    at = (st["cu_nodes"][:-1, None].long() + torch.arange(mn, device="cuda"))
    par = torch.where(q_real, st["parents"][at.clamp(max=st["parents"].numel() - 1)].long(), -1)
    node = torch.arange(mn, device="cuda")
    up = ((par[..., None] == node) | (node[:, None] == node)).float()   # itself and its parent
    up = _closure(_closure(_closure(_closure(_closure(_closure(up))))))  # 64 steps up
    t = torch.arange(most, device="cuda") - st["seq_lens"][:, None]     # node number of a token
    inside = t < st["cu_nodes"].diff()[:, None]
    draft = up.gather(2, t.clamp(0, mn - 1)[:, None].expand(n, mn, most)) > 0
    seen = ((t < 0)[:, None] | (draft & (t >= 0)[:, None])) & inside[:, None]
    k = _rows(st["kc"], st["ks"], st["table"], most, case["bits"])
    v = _rows(st["vc"], st["vs"], st["table"], most, case["bits"])
    s = (q.reshape(n, h, -1, 256) @ k.transpose(-1, -2)).mul_(1 / 16)
    o, _ = _softmax_v(s.view(n, h, hq // h, mn, most), seen[:, None, None],
                      v.masked_fill(~inside[:, None, :, None], 0)[:, :, None])
    return o.reshape(n, hq, mn, 256).transpose(1, 2)[q_real][None].half()


def _plain_commit(st):
    n = st["case"]["nseq"]
    count = st["cu_accept"].diff().long()
    seq = torch.repeat_interleave(torch.arange(n, device="cuda"), count,
                                  output_size=st["accept"].numel())
    to = st["seq_lens"][seq] + torch.arange(seq.numel(), device="cuda") - st["cu_accept"][seq]
    fr = st["seq_lens"][seq] + st["accept"]
    pt, ps, ft, fs = (st["table"][seq, to // PAGE].long(), to % PAGE,
                      st["table"][seq, fr // PAGE].long(), fr % PAGE)
    out = []
    for codes, scales in st["pools"]:
        codes[pt, :, ps] = codes[ft, :, fs]
        scales[pt, :, ps] = scales[ft, :, fs]
        out += [codes, scales.view(torch.int16)]
    return out


def run(st):
    case = st["case"]
    if own:
        import paged_kv_cache_fp16_gb300 as kvq
        if case["op"] == "norm_rope":
            kvq.kvq_qk_norm_rope(st["q"], st["k"], st["qo"], st["ko"], st["pos"], st["phases"],
                                 st["qw"], st["kw"], 1e-6, case["interleaved"])
            return st["qo"], st["ko"]
        if case["op"] == "prompt":
            kvq.kvq_prompt_attn(st["q"], st["k"], st["v"], st["cu_q"], st["cu_k"], st["max_q"],
                                st["max_k"], case["dim"] ** -0.5, st["out"], st["ws"], st["lse"])
            return (st["out"], st["lse"]) if case["lse"] else st["out"]
        if case["op"] == "tree":
            kvq.kvq_tree_attn(st["kp"], st["vp"], st["q"], st["table"], st["seq_lens"],
                              st["cu_nodes"], st["parents"], st["max_nodes"], st["max_len"],
                              1 / 16, st["out"], st["ws"])
            return st["out"]
        kvq.kvq_tree_commit(st["kp"], st["table"], st["seq_lens"], st["cu_accept"], st["accept"])
        return [x for c, s in st["pools"] for x in (c, s.view(torch.int16))]
    if case["op"] == "norm_rope":
        angle = st["pos"].double()[:, None, None] * st["inv_freq"]
        cos, sin = angle.cos().float(), angle.sin().float()
        return tuple(_plain_norm_rope(x, w, cos, sin, case["interleaved"]).to(x.dtype)
                     for x, w in ((st["q"], st["qw"]), (st["k"], st["kw"])))
    return {"prompt": _plain_prompt, "tree": _plain_tree, "commit": _plain_commit}[case["op"]](st)


# --------------------------------------------------------------------- the definitions in 64 bits
def _attend64(q, k, v, limit_mask, scale):
    """q [rows, D], k and v [keys, D] float64, mask [rows, keys] -> out, lse of one KV head."""
    s = (q @ k.T) * scale
    s[~limit_mask] = -math.inf
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[:, None])
    return p @ v, lse


def _value64(byte, i, bits):
    """The code of channel i of a row's bytes, from the storage format's definition."""
    bit = i * bits
    lo = byte[..., bit // 8]
    hi = byte[..., torch.clamp((bit + bits - 1) // 8, max=byte.shape[-1] - 1)]
    u = ((lo | (hi << 8)) >> (bit % 8)) & ((1 << bits) - 1)
    return torch.where(u > 127, u - 256, u) if bits == 8 else u - (1 << (bits - 1))


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "commit":
        return None                                     # whole numbers
    if case["op"] == "norm_rope":
        outs = []
        angle = st["pos"].double()[:, None, None] * st["inv_freq"]
        turn = torch.polar(torch.ones_like(angle), angle)
        for x, w in ((st["q"], st["qw"]), (st["k"], st["kw"])):
            y = x.double()
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / case["dim"] + 1e-6) * w.double()
            half = case["rotary"] // 2
            i = torch.arange(half, device="cuda")
            a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
            z = torch.complex(y[..., a], y[..., b]) * turn
            y[..., a], y[..., b] = z.real, z.imag
            outs.append(y)
        return tuple(outs)
    if case["op"] == "prompt":
        hq, h = HEADS[case["dim"]]
        g = hq // h
        new, keys = _lens(case)
        out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros(st["q"].shape[:2], dtype=torch.float64, device="cuda")
        q0 = k0 = 0
        for a, b in zip(new, keys):
            for r0 in range(0, a, 2048):                # rows in pieces: each sees a prefix
                r1 = min(a, r0 + 2048)
                end = r1 + b - a
                mask = (torch.arange(end, device="cuda")
                        <= torch.arange(r0, r1, device="cuda")[:, None] + b - a)
                for j in range(hq):
                    o, e = _attend64(st["q"][q0 + r0:q0 + r1, j].double(),
                                     st["k"][k0:k0 + end, j // g].double(),
                                     st["v"][k0:k0 + end, j // g].double(), mask,
                                     case["dim"] ** -0.5)
                    out[q0 + r0:q0 + r1, j], lse[q0 + r0:q0 + r1, j] = o, e
            q0, k0 = q0 + a, k0 + b
        return (out, lse) if case["lse"] else out
    hq, h = HEADS[256]
    g, bits = hq // h, case["bits"]
    length, nodes = _lens(case)
    parents = _parents(case, nodes)
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    i = torch.arange(256, device="cuda")
    n0 = 0
    for s, (a, b) in enumerate(zip(length, nodes)):
        t = torch.arange(a + b, device="cuda")
        page = st["table"][s].long()[t // PAGE]
        mask = torch.zeros((b, a + b), dtype=torch.bool)
        mask[:, :a] = True
        for node in range(b):
            up = node
            while up >= 0:
                mask[node, a + up] = True
                up = parents[s][up]
        for head in range(h):
            kv = []
            for codes, scales in ((st["kc"], st["ks"]), (st["vc"], st["vs"])):
                byte = codes[page, head, t % PAGE].int()
                x = _value64(byte, i, bits).double() * scales[page, head, t % PAGE].double()[:, None]
                kv.append(x.half().double())            # a row stands for its fp16 values
            rows = st["q"][0, n0:n0 + b, head * g:(head + 1) * g].double()
            o, _ = _attend64(rows.reshape(-1, 256), kv[0], kv[1],
                             mask.cuda().repeat_interleave(g, 0), 1 / 16)
            out[0, n0:n0 + b, head * g:(head + 1) * g] = o.view(b, g, 256)
        n0 += b
    return out
