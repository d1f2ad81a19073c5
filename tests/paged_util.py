"""Batches over a paged cache for the tests, and the tolerance of attention.

Everything that an operator must not look at is hostile: slots of the pool that
no sequence's length covers hold NaN, and so do pages that nobody names; table
entries behind a sequence's last page are far out of range.
"""
from __future__ import annotations

import numpy as np
import torch

from swiglu_ar_tts_b200 import inputs
from tolerance import to_f64

UNUSED = 0x7FFFFFF0  # a table entry that must never be followed


def table_for(lens, page, free, extra=1):
    """Block table for the given lengths from the list of free pages."""
    counts = [-(-max(n, 0) // page) for n in lens]
    table = np.full((len(lens), max(counts + [0]) + extra), UNUSED, dtype=np.int32)
    for s, c in enumerate(counts):
        for i in range(c):
            table[s, i] = free.pop()
    return table


def fill_pool(pages, hk, page, d, dtype, seed, tables_lens):
    """k and v pools: NaN but for the slots that the (table, lens) pairs cover."""
    pools = []
    for i in range(2):
        t = torch.full((pages, hk, page, d), float("nan"), dtype=inputs.torch_dtype(dtype))
        for k, (table, lens) in enumerate(tables_lens):
            for s, n in enumerate(lens):
                for p0 in range(0, max(n, 0), page):
                    m = min(page, n - p0)
                    t[table[s, p0 // page], :, :m] = inputs.normal(
                        (hk, m, d), seed + 1_000_003 * i + 7919 * k + 101 * s + p0, dtype=dtype)
        pools.append(t)
    return pools


class Batch:
    """A ragged batch: new[s] query tokens and lens[s] cache positions each."""

    def __init__(self, new, lens, hq, hk, d, page, dtype="bf16", seed=0, pad=0, spare=3, q_std=1.0):
        rng = np.random.default_rng(seed)
        self.new, self.lens = list(new), list(lens)
        need = sum(-(-max(n, 0) // page) for n in lens)
        free = list(rng.permutation(need + spare))
        self.table = table_for(self.lens, page, free)
        self.q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.tokens = int(self.q_start[-1]) + pad
        self.kv_lens = np.array(lens, dtype=np.int32)
        self.k_pages, self.v_pages = fill_pool(need + spare, hk, page, d, dtype, seed + 17,
                                               [(self.table, self.lens)])
        self.q = inputs.normal((self.tokens, hq, d), seed + 5, std=q_std, dtype=dtype)
        self.dtype, self.hq, self.hk, self.d, self.page = dtype, hq, hk, d, page

    def arrays(self):
        return [torch.from_numpy(a).cuda() for a in (self.q_start, self.kv_lens, self.table)]


class Groups:
    """Candidates that share prompts: members[g] sequences on prefix[g]
    positions, lens[s] of their own."""

    def __init__(self, members, prefix, lens, hq, hk, d, page, dtype="bf16", seed=0, pad=0, spare=3):
        rng = np.random.default_rng(seed)
        need = sum(-(-n // page) for n in list(prefix) + list(lens))
        free = list(rng.permutation(need + spare))
        self.prefix, self.lens = list(prefix), list(lens)
        self.prefix_table = table_for(prefix, page, free)
        self.table = table_for(lens, page, free)
        self.group_start = np.concatenate([[0], np.cumsum(members)]).astype(np.int32)
        self.n = len(lens)
        assert self.group_start[-1] + pad == self.n
        self.prefix_lens = np.array(prefix, dtype=np.int32)
        self.kv_lens = np.array(lens, dtype=np.int32)
        self.k_pages, self.v_pages = fill_pool(
            need + spare, hk, page, d, dtype, seed + 17,
            [(self.prefix_table, self.prefix), (self.table, self.lens)])
        self.q = inputs.normal((self.n, hq, d), seed + 5, dtype=dtype)
        self.dtype = dtype

    def arrays(self):
        return [torch.from_numpy(a).cuda() for a in (self.group_start, self.prefix_lens,
                                                     self.prefix_table, self.kv_lens, self.table)]




# Size of the errors in the scores and of the sums, from the arithmetic:
#   * q.k: products of bf16 are exact in fp32, D of them are added at 2^-23
#     each (round toward zero counted): D * 2^-23 * scale * sum|q k|.  In fp32
#     every operand is split into two tf32 parts; a part is rounded by at most
#     2^-11 of its size, so what is left out is 2^-22 an operand, and the
#     product of the two small parts, 2^-22, is dropped: 3 * 2^-22 more.
#   * scale, cap, bias and the change of base are a handful of fp32 roundings
#     of numbers no larger than |s|, cap and bias, and the exponential's own
#     error is 2^-22: together at most 2^-21 * (1 + |s| + bias + cap).
#   * n weights are added in fp32: n * 2^-23 of sum p|v|; before the second
#     product a weight is rounded to bf16 (half a step: 2^-8) or split (3 * 2^-22).
#   * the result is rounded to its type: half a step of it.
def score_constants(dtype, d):
    return dict(c_dot=d * 2.0 ** -23 + (0.0 if dtype == "bf16" else 3 * 2.0 ** -22),
                c_abs=2.0 ** -21)


def check_attention(gpu, expected, dtype, keys, what=""):
    out, mass, err = expected
    g = to_f64(gpu)
    assert g.shape == out.shape
    weight = 2.0 ** -8 if dtype == "bf16" else 3 * 2.0 ** -22
    tol = (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * np.abs(out)
    tol += (weight + keys * 2.0 ** -23) * mass + err + 2.0 ** -120
    bad = ~(np.abs(g - out) <= tol)
    if bad.any():
        i = np.argwhere(bad)[:4]
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} values off; first at {i.tolist()}: "
                             f"{[(g[tuple(x)], out[tuple(x)], tol[tuple(x)]) for x in i]}")
