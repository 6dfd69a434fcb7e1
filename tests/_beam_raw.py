"""q4 caches of one KV head with given codes and scales, and attention over them (not a test module).

With queries whose entries are all one power of two, a score is a sum of whole numbers below 2^24 units: exact
in float32, so that what is left are the roundings behind it (see `tolerance`)."""
from __future__ import annotations

import numpy as np
import torch

from oracle import beams as ob
from oracle import prompt as op
from _gpu_util import i32

STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TYPE = {"f16": torch.float16, "bf16": torch.bfloat16}


def pack(codes):
    """Codes -8 .. 7, int [T, D] -> bytes [T, D / 2]."""
    u = (np.asarray(codes) + 8).astype(np.uint8)
    return u[:, 0::2] | u[:, 1::2] << 4


class Raw:
    """groups: per group (key codes [T, D], key scales [T], value codes, value scales); a group's `beams`
    sequences have all of its tokens in common.  Pages are in a random order."""

    def __init__(self, kvq, dev, groups, beams=1, ps=16, seed=0, wide=0):
        self.D, self.beams, self.dev, self.kvq = groups[0][0].shape[1], beams, dev, kvq
        self.lens = [len(g[0]) for g in groups for _ in range(beams)]
        per = [-(-len(g[0]) // ps) for g in groups]
        order = np.random.default_rng(seed).permutation(sum(per)).astype(np.int32)
        table = np.full((len(self.lens), max(per) + wide), -1, np.int32)
        pools = [kvq.Pool.empty(4, 1, self.D, ps, sum(per), "cpu") for _ in range(2)]
        for p in pools:
            p.codes.fill_(0xFF)
            p.scales.fill_(float("nan"))
        at = 0
        self.rows = []
        for g, (kc, ks, vc, vs) in enumerate(groups):
            pages = order[at:at + per[g]]
            at += per[g]
            table[g * beams:(g + 1) * beams, :per[g]] = pages
            t = np.arange(len(kc))
            page, slot = torch.from_numpy(pages[t // ps].astype(np.int64)), torch.from_numpy(t % ps)
            sub = []
            for p, codes, scales in zip(pools, (kc, vc), (ks, vs)):
                scales = np.asarray(scales, dtype=np.float16)
                p.codes[page, 0, slot] = torch.from_numpy(pack(codes))
                p.scales[page, 0, slot] = torch.from_numpy(scales)
                sub.append(ob.q4_rows(pack(codes), scales))
            self.rows.append(sub)
        self.pools = [kvq.Pool(4, 1, self.D, ps, p.codes.to(dev), p.scales.to(dev)) for p in pools]
        self.table = i32(table, dev)

    def call(self, q, scale, shared=None, **over):
        """q [sequences, heads, D] -> out, the error word; max_shared and max_own are exact unless given."""
        kvq, n = self.kvq, len(self.lens)
        own = [a - (shared[s // self.beams] if shared is not None else 0) for s, a in enumerate(self.lens)]
        ms = over.get("max_shared", max(shared) if shared is not None else 0)
        mo = over.get("max_own", max(own))
        kp, vp = self.pools[:1], self.pools[1:]
        ws = kvq.beam_attn_workspace(kp, n, self.beams, q.shape[1], ms, mo, self.dev)
        ws.fill_(255)
        out, err = torch.full_like(q, 7.0), i32([0], self.dev)
        kvq.kvq_beam_attn(kp, vp, q[None], self.table, i32(self.lens, self.dev),
                          None if shared is None else i32(shared, self.dev), self.beams, ms, mo, scale,
                          out[None], ws, err)
        torch.cuda.synchronize()
        return out, int(err.item())

    def reference(self, q, scale, s):
        """Of sequence s: out, size = sum p |v|, the largest |score|, the largest weight (of all: 1) per head."""
        k, v = self.rows[s // self.beams]
        qn = q[s].double().cpu().numpy()
        o, _, size, span = op.attend(qn, k, v, np.ones((len(qn), len(k)), bool), scale)
        x = k @ qn.T * scale
        p = np.exp(x - x.max(0))
        return o, size, np.abs(x).max(0), 1 / p.sum(0)


def tolerance(n, o, size, score, top, v_most, kind):
    """Of an attention row over n tokens whose scores are exact sums: a weight times its value's scale is
    rounded to fp16, 2^-11 of itself, or 2^-35 of the row's largest weight and scale where it is smaller than
    2^-24 of them (times a code of at most 8); a weight has four roundings of its score (2^-24 each), one of
    its distance to the reference (below 64: 2^-19), and 2^-22 of the exponential, and so have their sums
    twice; sums in float32 2^-17; the result's own rounding."""
    e = 4 * 2.0 ** -24 * score + 2.0 ** -19 + 2.0 ** -22
    least = 2.0 ** -25 if kind == "f16" else 0.0
    return (size * (2.0 ** -11 + 2 * e[:, None] + 2.0 ** -17) + 1.001 * STEP[kind] * np.abs(o) + least
            + (8 * n * 2.0 ** -35 * v_most * top)[:, None])


def tiles(D, n, seed):
    """A group whose tiles of 16 tokens can be told apart: a tile's values are 7 in one channel (tiles take the
    channels in turn), and its score is one of 16 levels that the channel has, over a range of some 5."""
    t = np.arange(n) // 16 % D
    level = np.random.default_rng(seed).permutation(D) % 16
    vc = np.zeros((n, D), np.int64)
    vc[np.arange(n), t] = 7
    return np.ones((n, D), np.int64), level[t] / 3 + 0.25, vc, np.full(n, 0.25)
