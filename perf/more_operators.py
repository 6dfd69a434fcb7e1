"""Workloads of beam search over the paged cache: the selection of the next beams over beams and
vocabulary, the update of the page tables that follows it (beams forked, pages shared, copied, freed
and mapped), the compaction of the pages in use, and the decode attention of beams that share a
prefix over a cache held in 4 bits.

Each case is a dict of plain values.  `run` computes a case's operator on what `prepare` made: in
elementary torch operations where `own` is false, and through this library's entry points where it is
true.  `exact` is the operator's definition in 64 bits.

The sizes are those of the library's own workloads: 24 query heads over 4 KV heads of 256 channels,
32 over 8 of 64, and 16 over 4 of 128 between the two; 16-token pages in a random order; 16 layers; up
to 262,144 cached tokens.  Vocabularies are generic.
"""
from __future__ import annotations

import math
import random

import torch

own = False

HEADS = {256: (24, 4), 128: (16, 4), 64: (32, 8)}     # head_dim -> query heads, KV heads
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
PAGE = 16
INT_MAX = 2 ** 31 - 1


# ------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one sequence's first step (one live beam): latency
        dict(name="select 1x4 f16", op="select", nseq=1, beams=4, vocab=32768, out=8, dtype="f16",
             masked=0.0, first=True),
        # the step of a batch, bf16 logits with the many ties that they have
        dict(name="select 64x4 bf16", op="select", nseq=64, beams=4, vocab=131072, out=8,
             dtype="bf16", masked=0.0, first=False),
        # an odd vocabulary with banned tokens, wide beams, float32
        dict(name="select 16x16 f32", op="select", nseq=16, beams=16, vocab=50021, out=32,
             dtype="f32", masked=0.02, first=False),
        # four beams of one short text, K and V of one layer: latency
        dict(name="update 1x4", op="update", bits=4, dim=256, tensors=2, groups=1, beams=4,
             prompt=300, made=21, room=1, spare=0.25, mix=1),
        # a batch of beams in all 16 layers: what the copies of the tails cost
        dict(name="update 32x4, 16 layers", op="update", bits=4, dim=256, tensors=32, groups=32,
             beams=4, prompt=1500, made=150, room=1, spare=0.25, mix=2),
        # beams over full contexts: what the tables and counts cost
        dict(name="update 8x8 long", op="update", bits=4, dim=64, tensors=2, groups=8, beams=8,
             prompt=262000, made=100, room=17, spare=0.1, mix=3),
        # a small pool of one layer, a third of it free
        dict(name="compact 2x500", op="compact", bits=6, dim=256, tensors=2, groups=4, beams=2,
             prompt=1000, made=60, spare=0.5, mix=4),
        # the pools of 16 layers, a third of them free
        dict(name="compact 32x9000", op="compact", bits=4, dim=128, tensors=32, groups=32, beams=4,
             prompt=2000, made=300, spare=0.5, mix=5),
        # four beams of one short text: latency
        dict(name="attn 1x4 short", op="attn", dim=64, dtype="f16", layers=1, groups=1, beams=4,
             prompt=200, made=100, mix=6),
        # a batch of beams behind long prompts of different lengths
        dict(name="attn 8x4 bf16", op="attn", dim=128, dtype="bf16", layers=1, groups=8, beams=4,
             prompt=32768, made=500, mix=7),
        # a batch without beams: the plain decode step of 64 sequences
        dict(name="attn 64x1", op="attn", dim=128, dtype="f16", layers=1, groups=64, beams=1,
             prompt=0, made=8192, mix=8),
        # eight beams over one full context
        dict(name="attn 1x8 long", op="attn", dim=256, dtype="f16", layers=1, groups=1, beams=8,
             prompt=200000, made=700, mix=9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["select", "select", "update", "compact", "attn", "attn"])
    mix = rng.randrange(1 << 30)
    if op == "select":
        beams = _log(rng, 1, 16)
        nseq = _log(rng, 1, 64)
        most = min(131072, (1 << 25) // (nseq * beams))
        return dict(op=op, nseq=nseq, beams=beams, vocab=_log(rng, 100, most),
                    out=min(beams * rng.choice([1, 2]), 32), dtype=rng.choice(["f16", "bf16", "f32"]),
                    masked=rng.choice([0.0, 0.0, 0.02, 0.5]), first=rng.random() < 0.2)
    dim = rng.choice([64, 128, 256])
    beams = _log(rng, 1, 8)
    if op == "attn":
        groups = _log(rng, 1, 64)
        total = 262144 // groups if dim == 64 else 131072 // groups
        made = _log(rng, 1, max(2, min(1024, total // beams)))
        return dict(op=op, dim=dim, dtype=rng.choice(["f16", "bf16"]), layers=1, groups=groups,
                    beams=beams, prompt=rng.choice([0, 1, 1]) * _log(rng, 1, max(2, total // 4)),
                    made=made, mix=mix)
    groups = _log(rng, 1, 32)
    case = dict(op=op, bits=rng.choice([8, 6, 4]), dim=dim, tensors=2 * _log(rng, 1, 8),
                groups=groups, beams=beams, prompt=_log(rng, 1, 16384 // groups),
                made=_log(rng, 1, 256), spare=rng.choice([0.1, 0.3, 0.9]), mix=mix)
    return dict(case, room=_log(rng, 1, 40)) if op == "update" else case


# ------------------------------------------------------------------ what a case alone determines
def _pages(n):
    return -(-n // PAGE)


def _lens(case):
    """Per group: the prompt's length and that of its beams."""
    r = random.Random(case["mix"])
    prompt = [case["prompt"]] + [r.randint(case["prompt"] // 8, case["prompt"])
                                 for _ in range(case["groups"] - 1)]
    made = [case["made"]] + [r.randint(max(1, case["made"] // 8), case["made"])
                             for _ in range(case["groups"] - 1)]
    return prompt, [a + b for a, b in zip(prompt, made)]


def _parents(case):
    """Which beam each new beam continues: any of its group, some of them by several."""
    r = random.Random(case["mix"] + 1)
    b = case["beams"]
    return [g * b + r.randrange(b) for g in range(case["groups"]) for _ in range(b)]


def _layout(case):
    """Logical pages -> numbers in the order of first use (-1: none), and how many there are.  A
    group's beams share its prompt's full pages; the second beam of each pair also shares its
    sibling's pages up to the middle of what was generated."""
    prompt, length = _lens(case)
    b = case["beams"]
    width = max(_pages(n) for n in length) + _pages(case.get("room", 0)) + 1
    table = torch.full((case["groups"] * b, width), -1, dtype=torch.int32)
    used = 0
    for g, (p, n) in enumerate(zip(prompt, length)):
        for i in range(b):
            row, full, end = table[g * b + i], p // PAGE, _pages(n)
            same = 0
            if i:
                same = full if i % 2 == 0 else max(full, (p + n) // 2 // PAGE)
                row[:same] = table[g * b + (i - i % 2 if same > full else 0), :same]
            row[same:end] = torch.arange(used, used + end - same, dtype=torch.int32)
            used += end - same
    return table, used


def _packed_dim(case):
    return case["dim"] * case.get("bits", 4) // 8


def _page_bytes(case):
    return HEADS[case["dim"]][1] * PAGE * (_packed_dim(case) + 2)


def work(case):
    if case["op"] == "select":
        n = case["nseq"] * case["beams"] * case["vocab"]
        return {"bytes": n * (4 if case["dtype"] == "f32" else 2) + 12 * case["nseq"] * case["out"],
                "flops": 3 * n}
    prompt, length = _lens(case)
    b = case["beams"]
    if case["op"] == "attn":
        hq, h = HEADS[case["dim"]]
        rows = sum(p + b * (n - p) for p, n in zip(prompt, length))
        return {"bytes": case["layers"] * (2 * h * rows * (_packed_dim(case) + 2)
                                           + 4 * case["groups"] * b * hq * case["dim"])
                + 4 * sum(_pages(n) * b for n in length),
                "flops": 4 * case["layers"] * case["dim"] * hq * b * sum(length)}
    table, used = _layout(case)
    pages = used + int(used * case["spare"]) + 8
    entries = sum(_pages(n) * b for n in length)
    if case["op"] == "compact":
        moved = used * (pages - used) // pages
        return {"bytes": 2 * moved * _page_bytes(case) * case["tensors"] + 8 * entries + 8 * pages,
                "flops": 0}
    children = _parents(case)
    rows = 0
    for g, n in enumerate(length):                    # the tails of all children but the first
        mine = [p for p in children if p // b == g]
        rows += (len(mine) - len(set(mine))) * (n % PAGE)
    return {"bytes": 2 * rows * _page_bytes(case) // PAGE * case["tensors"] + 8 * entries + 8 * pages,
            "flops": 0}


# ------------------------------------------------------------------------------------ the inputs
def _pack(codes, bits):
    """Signed codes int8 [..., D] -> the packed bytes of a row."""
    if bits == 8:
        return codes.view(torch.uint8)
    if bits == 4:
        u = (codes + 8).to(torch.uint8).unflatten(-1, (-1, 2))
        return u[..., 0] | (u[..., 1] << 4)
    a, b, c, d = (codes + 32).to(torch.uint8).unflatten(-1, (-1, 4)).unbind(-1)
    return torch.stack([a | ((b & 3) << 6), (b >> 2) | ((c & 15) << 4), (c >> 4) | (d << 2)],
                       -1).flatten(-2)


def _filled(gen, pages, heads, dim, key):
    """q4 codes and scales of a pool as the symmetric quantizer leaves them: N(0,1) rows, keys with
    four channels x10."""
    x = torch.randn((pages, heads, PAGE, dim), generator=gen, device="cuda", dtype=torch.float16)
    if key:
        x[..., [5, dim // 3, dim // 2 + 2, dim - 10]] *= 10
    scale = (x.abs().amax(-1).float() / 7).half()
    codes = torch.round(x.float() / scale.float()[..., None]).clamp_(-7, 7)
    return _pack(codes.to(torch.int8), 4).contiguous(), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    st = dict(case=case)
    if case["op"] == "select":
        n, b, v = case["nseq"], case["beams"], case["vocab"]
        x = torch.randn((n * b, v), generator=gen, device="cuda") * 2.5
        if case["masked"]:
            x.masked_fill_(torch.rand((n * b, v), generator=gen, device="cuda") < case["masked"],
                           -math.inf)
        st["logits"] = x.to(DTYPES[case["dtype"]])
        st["scores"] = -30 * torch.rand((n, b), generator=gen, device="cuda")
        if case["first"]:                             # all beams but one still empty
            st["scores"][:, 1:] = -math.inf
        k = case["out"]
        st["out"] = (torch.empty((n, k), device="cuda"),
                     torch.empty((n, k), dtype=torch.int32, device="cuda"),
                     torch.empty((n, k), dtype=torch.int32, device="cuda"))
        if own:   # scratch that a program keeps
            import paged_kv_cache_fp16_gb300 as kvq
            st["ws"] = kvq.beam_select_workspace(n, b, v, k)
        return st
    table, used = _layout(case)
    prompt, length = _lens(case)
    b, dim = case["beams"], case["dim"]
    hq, h = HEADS[dim]
    pages = used + int(used * case.get("spare", 0)) + 8
    place = torch.randperm(pages, generator=host).to(torch.int32)
    table = torch.where(table >= 0, place[table.clamp(min=0).long()], -1)
    lens = torch.tensor(length, dtype=torch.int32).repeat_interleave(b)
    held = (lens + PAGE - 1) // PAGE
    st["table"], st["lens"] = table.cuda(), lens.cuda()
    if case["op"] == "attn":
        st["shared"] = torch.tensor(prompt, dtype=torch.int32).cuda()
        st["max_shared"] = max(prompt)
        st["max_own"] = max(n - p for p, n in zip(prompt, length))
        kv = [[_filled(gen, pages, h, dim, key) for _ in range(case["layers"])]
              for key in (True, False)]
        tail = st["shared"].long()                    # the prompt's last page: a copy for each beam
        for codes, scales in kv[0] + kv[1]:
            for i in range(1, b):
                dst = st["table"][i::b].gather(1, tail[:, None] // PAGE)[:, 0].long()
                src = st["table"][::b].gather(1, tail[:, None] // PAGE)[:, 0].long()
                codes[dst], scales[dst] = codes[src], scales[src]
        st["kv"] = kv
        st["q"] = torch.randn((case["layers"], case["groups"] * b, hq, dim), generator=gen,
                              device="cuda").to(DTYPES[case["dtype"]])
        st["out"] = torch.empty_like(st["q"])
        if own:   # the pools' descriptions and scratch that a program keeps
            import paged_kv_cache_fp16_gb300 as kvq
            st["kp"], st["vp"] = ([kvq.Pool(4, h, dim, PAGE, c, s) for c, s in x] for x in kv)
            st["ws"] = kvq.beam_attn_workspace(st["kp"], case["groups"] * b, b, hq, st["max_shared"],
                                               st["max_own"])
        return st
    st["held"] = held.cuda()
    refs = torch.zeros(pages + 1, dtype=torch.int32)
    refs.index_add_(0, torch.where(table >= 0, table, pages).flatten().long(),
                    torch.ones(table.numel(), dtype=torch.int32))
    refs = refs[:pages]
    kept = table[:case["groups"] // 2 * b:b, :_pages(case["prompt"])].flatten()   # a prefix cache's own
    kept = kept[kept >= 0].unique().long()
    refs[kept] += 1
    st["refs"] = refs.cuda()
    st["table_out"], st["refs_out"] = torch.full_like(st["table"], -1), torch.empty_like(st["refs"])
    t = case["tensors"]
    st["codes"] = torch.randint(0, 256, (t, pages, h, PAGE, _packed_dim(case)), generator=gen,
                                device="cuda", dtype=torch.uint8)
    st["scales"] = torch.rand((t, pages, h, PAGE), generator=gen, device="cuda").half()
    if case["op"] == "update":
        st["parents"] = torch.tensor(_parents(case), dtype=torch.int32).cuda()
        st["room"] = torch.full((len(lens),), case["room"], dtype=torch.int32, device="cuda")
        st["lens_out"], st["held_out"] = torch.empty_like(st["lens"]), torch.empty_like(st["lens"])
    else:
        st["live"] = torch.empty(1, dtype=torch.int32, device="cuda")
    if own:
        import paged_kv_cache_fp16_gb300 as kvq
        st["pools"] = [kvq.Pool(case["bits"], h, dim, PAGE, st["codes"][i], st["scales"][i])
                       for i in range(t)]
        st["ws"] = kvq.table_workspace(pages, len(lens))
    return st


# ----------------------------------------------------------------------------- the plain forms
def _plain_select(st):
    case = st["case"]
    n, b, v, k = case["nseq"], case["beams"], case["vocab"], case["out"]
    x = st["logits"].double().view(n, b, v)           # in 64 bits: neighbours are close
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    x = x - (top + (x - top).exp().sum(-1, keepdim=True).log()) + st["scores"].double()[..., None]
    x = torch.where(x.isnan(), -math.inf, x).view(n, b * v)
    score, at = x.sort(dim=-1, descending=True, stable=True)
    score, at = score[:, :k], at[:, :k]
    if b * v < k:
        score = torch.nn.functional.pad(score, (0, k - b * v), value=-math.inf)
        at = torch.nn.functional.pad(at, (0, k - b * v))
    none = score == -math.inf
    row = at // v + b * torch.arange(n, device="cuda")[:, None]
    return (score.float(), torch.where(none, -1, row).int(), torch.where(none, -1, at % v).int())


def _plain_update(st):
    table, lens, held = st["table"], st["lens"].long(), st["held"].long()
    par, room = st["parents"].long(), st["room"].long()
    n_in, n_out, width = table.shape[0], par.numel(), table.shape[1]
    j = torch.arange(width, device="cuda")
    keep = (lens + PAGE - 1) // PAGE
    children = torch.zeros(n_in, dtype=torch.int32, device="cuda").index_add_(
        0, par, torch.ones_like(par, dtype=torch.int32))
    # every page loses its old owners and gains its heirs
    change = torch.where(j < keep[:, None], children[:, None], 0) - 1
    listed_ = j < held[:, None]
    refs = st["refs"].clone().index_add_(0, table.clamp(min=0).flatten().long(),
                                         torch.where(listed_, change, 0).int().flatten())
    new_len, new_keep = lens[par], keep[par]
    out = table[par]
    fill = new_len % PAGE
    writes = (fill > 0) & (room > 0)
    tail = out.gather(1, (new_keep - 1).clamp(min=0)[:, None])[:, 0].long()
    # of the beams that will write into a page, the first keeps it unless somebody else reads it
    s = torch.arange(n_out, device="cuda")
    w_tail = torch.where(writes, tail, refs.numel())
    count = torch.zeros(refs.numel() + 1, dtype=torch.int32, device="cuda").index_add_(
        0, w_tail, torch.ones_like(w_tail, dtype=torch.int32))
    first = torch.full((refs.numel() + 1,), INT_MAX, device="cuda").scatter_reduce_(
        0, w_tail, s, "amin")
    copy = writes & ~((refs[tail] == count[tail]) & (first[tail] == s))
    total_pages = (new_len + room + PAGE - 1) // PAGE
    total_pages = torch.where(room > 0, total_pages, new_keep)
    need = total_pages - new_keep + copy
    start = need.cumsum(0) - need
    begin = new_keep - copy.long()
    refs.index_add_(0, tail, -copy.int())
    free = torch.argsort((refs != 0).int(), stable=True)
    fresh = (j >= begin[:, None]) & (j < total_pages[:, None])
    page = free[(start[:, None] + j - begin[:, None]).clamp(0, refs.numel() - 1)]
    refs.index_add_(0, page.flatten(), fresh.flatten().int())
    out = torch.where(fresh, page.int(), torch.where(j < new_keep[:, None], out, -1))
    at = copy.nonzero()[:, 0]
    src = tail[at]
    dst = out[at, new_keep[at] - 1].long()
    part = torch.arange(PAGE, device="cuda") < fill[at, None]
    codes, scales = st["codes"], st["scales"]
    codes[:, dst] = torch.where(part[:, None, :, None], codes[:, src], codes[:, dst])
    scales[:, dst] = torch.where(part[:, None], scales[:, src], scales[:, dst])
    return out, new_len.int(), total_pages.int(), refs, codes, scales.view(torch.int16)


def _plain_compact(st):
    refs, table = st["refs"], st["table"]
    page = torch.arange(refs.numel(), device="cuda")
    live = refs != 0
    n = live.sum()
    src = (live & (page >= n)).nonzero()[:, 0]
    dst = (~live & (page < n)).nonzero()[:, 0]
    to = page.scatter(0, src, dst)
    out = torch.where(torch.arange(table.shape[1], device="cuda") < st["held"][:, None],
                      to[table.clamp(min=0).long()].int(), -1)
    refs = refs.scatter(0, dst, refs[src]).scatter(0, src, 0)
    codes, scales = st["codes"], st["scales"]
    codes[:, dst], scales[:, dst] = codes[:, src], scales[:, src]
    return out, refs, n.int()[None], codes, scales.view(torch.int16)


def _rows(codes, scales, table, most):
    """The first `most` tokens of every sequence as the codes and scales stand for, in float32,
    [sequences, H, most, D]."""
    t = torch.arange(most, device="cuda")
    page = table[:, t // PAGE].clamp(min=0).long()
    x = codes[page, :, t % PAGE]
    x = torch.stack([x & 15, x >> 4], -1).flatten(-2).float().sub_(8)
    return x.mul_(scales[page, :, t % PAGE].float()[..., None]).transpose(1, 2)


def _plain_attn(st, layer):
    case = st["case"]
    hq, h = HEADS[case["dim"]]
    q = st["q"][layer].float()
    most = int(st["max_shared"] + st["max_own"])
    seen = torch.arange(most, device="cuda") < st["lens"][:, None]
    s = q.view(len(q), h, hq // h, -1) @ _rows(*st["kv"][0][layer], st["table"], most).transpose(-1, -2)
    s.mul_(case["dim"] ** -0.5).masked_fill_(~seen[:, None, None], -math.inf)
    p = s.sub_(s.amax(-1, keepdim=True)).exp_()
    o = p @ _rows(*st["kv"][1][layer], st["table"], most).masked_fill_(~seen[:, None, :, None], 0)
    return (o / p.sum(-1, keepdim=True)).view(q.shape).to(st["q"].dtype)


def run(st):
    case = st["case"]
    if own:
        import paged_kv_cache_fp16_gb300 as kvq
        if case["op"] == "select":
            kvq.kvq_beam_select(st["logits"], st["scores"], *st["out"], st["ws"])
            return st["out"]
        if case["op"] == "update":
            kvq.kvq_table_update(st["pools"], st["table"], st["lens"], st["held"], st["refs"],
                                 st["parents"], st["room"], st["table_out"], st["lens_out"],
                                 st["held_out"], st["refs_out"], st["ws"])
            return (st["table_out"], st["lens_out"], st["held_out"], st["refs_out"], st["codes"],
                    st["scales"].view(torch.int16))
        if case["op"] == "compact":
            kvq.kvq_table_compact(st["pools"], st["table"], st["held"], st["refs"], st["table_out"],
                                  st["refs_out"], st["live"], st["ws"])
            return (st["table_out"], st["refs_out"], st["live"], st["codes"],
                    st["scales"].view(torch.int16))
        kvq.kvq_beam_attn(st["kp"], st["vp"], st["q"], st["table"], st["lens"], st["shared"],
                          case["beams"], st["max_shared"], st["max_own"], case["dim"] ** -0.5,
                          st["out"], st["ws"])
        return st["out"]
    if case["op"] == "attn":
        return torch.stack([_plain_attn(st, layer) for layer in range(case["layers"])])
    return {"select": _plain_select, "update": _plain_update, "compact": _plain_compact}[case["op"]](st)


# --------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    if case["op"] in ("update", "compact"):
        return None                                   # whole numbers
    st = prepare(case, seed)
    if case["op"] == "select":
        n, b, v, k = case["nseq"], case["beams"], case["vocab"], case["out"]
        best = torch.full((n, k), -math.inf, dtype=torch.float64, device="cuda")
        for i in range(n):
            lp = torch.log_softmax(st["logits"][i * b:(i + 1) * b].double(), -1)
            lp = (lp + st["scores"][i].double()[:, None]).flatten()
            lp = torch.topk(lp.nan_to_num(nan=-math.inf, neginf=-math.inf), min(k, b * v)).values
            best[i, :len(lp)] = lp
        return best, None, None
    hq, h = HEADS[case["dim"]]
    g, b = hq // h, case["beams"]
    _, length = _lens(case)
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    for layer in range(case["layers"]):
        for s in range(case["groups"] * b):
            t = torch.arange(length[s // b], device="cuda")
            page = st["table"][s].long()[t // PAGE]
            for head in range(h):
                kv = []
                for codes, scales in (st["kv"][0][layer], st["kv"][1][layer]):
                    byte = codes[page, head, t % PAGE].int()
                    x = torch.empty((len(t), case["dim"]), dtype=torch.float64, device="cuda")
                    x[:, 0::2], x[:, 1::2] = byte % 16 - 8, byte // 16 - 8
                    kv.append(x * scales[page, head, t % PAGE].double()[:, None])
                w = st["q"][layer, s, head * g:(head + 1) * g].double() @ kv[0].T
                out[layer, s, head * g:(head + 1) * g] = torch.softmax(
                    w / math.sqrt(case["dim"]), -1) @ kv[1]
    return out
