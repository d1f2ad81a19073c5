"""Attention row by row: a result depends on its own query and on nothing that
stands beside it in a tile, and every key counts once."""
import numpy as np
import pytest
import torch

from gpu_util import dev
from paged_util import Batch, Groups
from test_gpu_paged_attention import _slopes, expected, run, shared_expected, shared_run
from tolerance import to_f64

pytestmark = pytest.mark.gpu

OPTS = [{}, {"softcap": 20.0}, {"softcap": 3.0, "slopes": _slopes(16)}, {"slopes": _slopes(16)}]
VALUES = [0.0, 30.0, -1e4, float("inf"), float("nan")]


def _changed(q, where, value):
    """q with the rows of `where` multiplied by `value` (infinite where it is)."""
    q = q.clone()
    q[where] = q[where] * value if np.isfinite(value) else value
    return q


# rows of the tile kernel in the first two (tokens that end inside a warp's 32
# rows), of the row kernel in the others
@pytest.mark.parametrize("new,lens,dtype", [([50, 37, 61], [50, 137, 461], "bf16"), ([203, 5], [703, 300], "bf16"),
                                            ([1, 1, 3], [40, 900, 65], "bf16"), ([50, 9], [130, 70], "f32")])
@pytest.mark.parametrize("opt", OPTS)
def test_a_row_depends_on_its_own_query(new, lens, dtype, opt):
    b = Batch(new, lens, 16, 8, 128, 16, dtype, seed=95, pad=5)
    q = dev(b.q)
    first = run(b, q=q, **opt)
    n = int(b.q_start[-1])
    for value in VALUES:
        # padding tokens; the last sequence; one token of the first sequence
        for lo, hi in ((n, b.tokens), (int(b.q_start[-2]), n), (new[0] // 2, new[0] // 2 + 1)):
            got = run(b, q=_changed(q, slice(lo, hi), value), **opt)
            what = f"tokens {lo}..{hi} times {value}"
            assert torch.equal(got[:lo], first[:lo]), what
            assert torch.equal(got[hi:], first[hi:]), what
        # one head of one token
        other = torch.ones(b.tokens, 16, dtype=torch.bool)
        other[new[0] // 2, 7] = False
        got = run(b, q=_changed(q, (new[0] // 2, 7), value), **opt)
        assert torch.equal(got[other.cuda()], first[other.cuda()]), f"head times {value}"


@pytest.mark.parametrize("members,prefix", [([270], [300]), ([150, 119], [500, 70]), ([5, 3], [300, 40])])
@pytest.mark.parametrize("opt", OPTS)
def test_a_candidate_depends_on_its_own_query(members, prefix, opt):
    n, pad = sum(members), 3
    b = Groups(members, prefix, [1 + 7 * i % 40 for i in range(n)] + [9] * pad, 16, 8, 128, 16, "bf16", seed=96,
               pad=pad)
    q = dev(b.q)
    first = shared_run(b, q=q, **opt)
    for value in VALUES:
        for lo, hi in ((n, n + pad), (members[0] - 1, n), (members[0] // 2, members[0] // 2 + 1)):
            got = shared_run(b, q=_changed(q, slice(lo, hi), value), **opt)
            what = f"sequences {lo}..{hi} times {value}"
            assert torch.equal(got[:lo], first[:lo]), what
            assert torch.equal(got[hi:], first[hi:]), what


def _count_pools(b):
    """Values that count: key x of the cache is a 1 in one column, which its place
    in the pool chooses; every column collects about one key in d."""
    at = torch.arange(b.v_pages.shape[0] * b.v_pages.shape[2]).view(b.v_pages.shape[0], -1)
    hot = (at * 40503 % 65537) % b.v_pages.shape[3]
    v = torch.nn.functional.one_hot(hot, b.v_pages.shape[3]).to(b.v_pages.dtype)
    return torch.where(torch.isnan(b.v_pages), b.v_pages, v[:, None].expand(b.v_pages.shape))


def _check_counts(got, exact, dtype, n):
    # all scores are 0: the weights are 1 and their sums whole numbers, exact in
    # fp32; left are the reciprocal, the product and the rounding to the type.  A
    # key that is left out or counted twice changes its column by 1 / count.
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    g = to_f64(got)[:n]
    assert np.all(np.abs(g - exact[:n]) <= (half + 2.0 ** -22) * exact[:n])
    assert exact[:n][exact[:n] > 0].size


# A column collects fewer than 100 keys: one key is more than 2^-8 of it twice over.
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new,lens,page,opt", [
    ([1, 1, 1, 1], [11000, 1, 700, 64], 16, {}), ([130], [9130], 64, {}), ([300, 77], [300, 2077], 8, {}),
    ([200, 50], [1500, 50], 24, {"window": 333}), ([120, 1], [900, 5000], 16, {"bidir_lens": [850, 10]}),
    ([96, 1], [6000, 33], 20, {})])
def test_every_key_counts_once(new, lens, page, opt, dtype):
    if dtype == "f32":
        new = [min(n, 20) for n in new]
    b = Batch(new, lens, 4, 2, 128, page, dtype, seed=97, pad=1)
    b.q.zero_()
    b.v_pages = _count_pools(b)
    opt = {k: np.array(v, dtype=np.int32) if k == "bidir_lens" else v for k, v in opt.items()}
    _check_counts(run(b, **opt), expected(b, **opt)[0], dtype, int(b.q_start[-1]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("members,prefix", [([6], [9000]), ([290], [9000]), ([280, 30], [700, 65])])
def test_every_key_of_a_group_counts_once(members, prefix, dtype):
    n = sum(members)
    b = Groups(members, prefix, [7 * i % 90 for i in range(n)], 4, 2, 128, 16, dtype, seed=98)
    b.q.zero_()
    b.v_pages = _count_pools(b)
    _check_counts(shared_run(b), shared_expected(b)[0], dtype, n)
