"""Shared helpers of the tests of include/kvq_tokens.h: each operator in plain
fp64 or Python."""
import math

import numpy as np

from quantized_kv_cache_03_gb300 import kvq


def rates(n_rot, base=10000.0, scaling=kvq.ROPE_PLAIN, factor=1.0, original=0.0, fast=0.0, slow=0.0):
    """(radians per position of each pair, amplitude), pair by pair as the header states them."""
    got = []
    if scaling == kvq.ROPE_BASE and n_rot:
        base = base * factor ** (n_rot / (n_rot - 2))
    for i in range(n_rot // 2):
        r = base ** (-2 * i / n_rot)
        turns = original * r / (2 * math.pi)   # within the original context
        share = 0.0                            # of the slowed rate
        if scaling == kvq.ROPE_LINEAR:
            share = 1.0
        elif scaling == kvq.ROPE_BY_INDEX:
            def pair_of(n):
                return n_rot * math.log(original / (2 * math.pi * n)) / (2 * math.log(base))
            lo, hi = max(math.floor(pair_of(fast)), 0), min(math.ceil(pair_of(slow)), n_rot - 1)
            share = (i - lo) / max(hi - lo, 1e-3)
        elif scaling == kvq.ROPE_BY_TURNS:
            share = (fast - turns) / (fast - slow)
        share = min(max(share, 0.0), 1.0)
        got.append(share * r / factor + (1 - share) * r if share else r)
    return np.array(got), 0.1 * math.log(factor) + 1 if scaling == kvq.ROPE_BY_INDEX else 1.0


def rotated(x, pos, f, amplitude, layout):
    """fp64 x [tokens][heads][128] at positions pos; and |a| + |b| of each value's pair (0 where nothing rotates)."""
    n = 2 * len(f)
    y, size = x.copy(), np.zeros_like(x)
    if n == 0:
        return y, size
    angle = np.asarray(pos, np.float64)[:, None] * f
    c, s = (amplitude * t[:, None, :] for t in (np.cos(angle), np.sin(angle)))
    first = np.arange(n // 2) if layout == kvq.ROPE_HALF else 2 * np.arange(n // 2)
    second = first + (n // 2 if layout == kvq.ROPE_HALF else 1)
    a, b = x[..., first], x[..., second]
    y[..., first], y[..., second] = a * c - b * s, a * s + b * c
    size[..., first] = size[..., second] = amplitude * (np.abs(a) + np.abs(b))
    return y, size


def normalized(x, w, eps):
    x = x.astype(np.float64)
    return x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w.astype(np.float64)


# What fp32 arithmetic may add, relative to |a| + |b| of a pair: the norm (twelve sums and a fused one, halved by the
# root; the reciprocal root, 2^-22; three products), cos and sin (an angle known to 1.9e-7, 2^-23 of the function, 2^-24
# of the amplitude's product) and two products with a sum.
FP32 = 6 * 2.0 ** -24 + 2.0 ** -22 + 3 * 2.0 ** -24 + 1.9e-7 + 2.0 ** -23 + 2.0 ** -24 + 2 * 2.0 ** -24


def fp16_bound(y, size):
    """How far an fp16 result may be from y: half a step of it (2^-11, or 2^-25 among the subnormals) and the fp32 arithmetic."""
    e = FP32 * np.where(size == 0, np.abs(y), size)
    return (np.abs(y) + e) * 2.0 ** -11 + 2.0 ** -25 + e


def fork_ref(page, n_pages, lens, table, free, n_free, out, most, parent=None, keep=None):
    """kvq_page_fork in plain Python: lists of pages, one place after another."""
    B = len(lens)
    lens = [min(max(int(x), 0), most * page) for x in lens]
    n_free = min(max(n_free, 0), n_pages)

    def blocks(n):
        return -(-n // page)

    rows, kept = [], []
    for b in range(B):
        p = b if parent is None else int(parent[b])
        n = 0
        if 0 <= p < B:
            n = lens[p] if keep is None else min(max(int(keep[b]), 0), lens[p])
        kept.append(n)
        rows.append([int(x) for x in table[p, :blocks(n)]] if n else [])
    there = {int(x) for b in range(B) for x in table[b, :blocks(lens[b])] if 0 <= x < n_pages}
    still = {x for r in rows for x in r if 0 <= x < n_pages}
    stack = [int(x) for x in free[:n_free]] + sorted(there - still)
    stack = stack[:n_pages]
    free, out = free.copy(), out.copy()
    free[n_free:len(stack)] = stack[n_free:]
    whole = {x for b, r in enumerate(rows) for x in r[:kept[b] // page]}
    tails = set()
    res = dict(lens=[], copy_from=[], copy_to=[], copy_held=[], status=[])
    for b, r in enumerate(rows):
        n, frm, to, held, st = kept[b], -1, -1, 0, 0
        if n % page and 0 <= r[-1] < n_pages:
            if r[-1] in whole or r[-1] in tails:
                if stack:
                    frm, to, held = r[-1], stack.pop(), n % page
                    r[-1] = to
                else:
                    n, st = n // page * page, 1
            else:
                tails.add(r[-1])
        out[b, :blocks(n)] = r[:blocks(n)]
        for k, v in (("lens", n), ("copy_from", frm), ("copy_to", to), ("copy_held", held), ("status", st)):
            res[k].append(v)
    return dict({k: np.array(v, np.int32) for k, v in res.items()}, table_out=out, free=free, n_free=np.array([len(stack)]))
