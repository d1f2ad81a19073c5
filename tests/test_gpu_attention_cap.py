"""Attention whose scores are capped by a tanh, for caps from a fraction of the
scores to the largest that the type holds, against the formula in fp64 with a
tolerance that does not grow with the cap."""
import numpy as np
import pytest
import torch

from gpu_util import dev
from paged_util import Batch, Groups, check_attention, score_constants
from test_gpu_paged_attention import _slopes, run, shared_run

pytestmark = pytest.mark.gpu


def _gather(pool, row, n, page):
    p = np.arange(n)
    return pool[row[p // page], :, p % page].double().transpose(0, 1)  # [hk, n, d]


def _attend(q, k, v, at, cap, slopes, dtype):
    """(out, mass, err) as oracle_attention's, of queries q [t, hq, d] at
    positions `at` on the keys k, v [hk, n, d]."""
    hq, d = q.shape[1:]
    g = hq // k.shape[0]
    q = q.double().transpose(0, 1)  # [hq, t, d]
    k, v = (x.repeat_interleave(g, 0) for x in (k, v))
    scale = float(np.float32(d ** -0.5))
    cap = float(np.float32(cap))
    s = scale * (q @ k.transpose(1, 2))
    large = s.abs() > 0.499 * cap
    mag = scale * (q.abs() @ k.abs().transpose(1, 2))
    x = cap * torch.tanh(s / cap)
    gap = (at[:, None] - torch.arange(k.shape[1])[None]).double()
    bias = 0.0 if slopes is None else slopes.double()[:, None, None] * gap.abs()
    # What a cap may cost, of the capped score:
    #   |s| <= cap / 2, a polynomial: in fp32 s (1 + y Q(y)), y = (s / cap)^2: 2^-26 of
    #   Q, 5 roundings of y weighted by at most 1/12, 2 of Q likewise, the last one:
    #   below 2^-23.  In bf16 x P(y) with P off by 5.4e-7 and six roundings: 2^-20.
    #   |s| > cap / 2: 1 - 2 / (1 + e^2|x|), |x| > 1/2.  The exponential's argument has
    #   three roundings and a half (2|x| 3.5 2^-24) and its own error 2^-22; that is
    #   weighted by 2 e / (1 + e)^2, 0.39 at |x| = 1/2 and less above: 3 2^-24 of the cap.
    #   The sum, the reciprocal (2^-23) and the last two roundings: 2.6 2^-24.  The
    #   capped score is 0.46 of the cap at least: 2^-20.
    small = 2.0 ** -23 if dtype == "f32" else 2.0 ** -20
    c_cap = torch.where(large, torch.full_like(s, 2.0 ** -20), torch.full_like(s, small))
    delta = score_constants(dtype, d)["c_dot"] * mag + 2.0 ** -21 * (1 + x.abs() + bias) + c_cap * x.abs()
    w = (x - bias).masked_fill(gap < 0, -float("inf"))
    p = torch.softmax(w, -1)
    out = p @ v
    err = (p * delta) @ v.abs() + out.abs() * (p * delta).sum(-1, keepdim=True)
    return [y.transpose(0, 1).numpy() for y in (out, p @ v.abs(), err)]


def check(b, got, cap, slopes=None, what=""):
    parts = []
    for s, n in enumerate(b.lens):
        t0, t1 = int(b.q_start[s]), int(b.q_start[s + 1])
        at = torch.arange(n - (t1 - t0), n)
        k, v = (_gather(x, b.table[s], n, b.page) for x in (b.k_pages, b.v_pages))
        parts.append(_attend(b.q[t0:t1], k, v, at, cap, slopes, b.dtype))
    e = [np.concatenate(x) for x in zip(*parts)]
    check_attention(got[:e[0].shape[0]], e, b.dtype, max(b.lens), what)


CAPS = (2.0, 8.0, 1e2, 1e4, 1e5, 1e6, 1e8, 1e30, 3e38)
# decode steps; prompts (the tile kernel in bf16); pages that the tile kernel does not take
SHAPES = (([1, 1, 1], [300, 20, 65], 16), ([130, 60], [130, 200], 16), ([70, 3], [70, 90], 20))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("new,lens,page", SHAPES)
@pytest.mark.parametrize("biased", [False, True])
def test_caps_of_every_size(new, lens, page, cap, biased, dtype):
    b = Batch(new, lens, 8, 4, 128, page, dtype, seed=91, q_std=4.0)
    opt = dict(softcap=cap, **({"slopes": _slopes(8)} if biased else {}))
    check(b, run(b, **opt), cap, opt.get("slopes"), f"cap {cap} {dtype} {new}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cap", [50.0, 1e6, 1e8])
@pytest.mark.parametrize("new,lens,page", SHAPES)
@pytest.mark.parametrize("biased", [False, True])
def test_scores_on_both_sides_of_half_a_cap(new, lens, page, cap, biased, dtype):
    """One query of a batch far above its neighbours' scores, up to many caps."""
    b = Batch(new, lens, 8, 4, 128, page, dtype, seed=92, q_std=2.0)
    t = b.tokens // 2
    b.q[t, 3] = (b.q[t, 3].float() * cap).to(b.q.dtype)
    b.q[t, 5] = (b.q[t, 5].float() * cap / 8).to(b.q.dtype)
    opt = dict(softcap=cap, **({"slopes": _slopes(8)} if biased else {}))
    check(b, run(b, **opt), cap, opt.get("slopes"), f"outlier {cap} {dtype} {new}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cap", [8.0, 1e4, 1e8, 1e30])
@pytest.mark.parametrize("members", [5, 300])
def test_caps_of_a_group(members, cap, dtype):
    """A prefix and the members' own keys, of either kernel, under one cap."""
    b = Groups([members], [260], [1 + 7 * i % 50 for i in range(members)], 8, 4, 128, 16, dtype, seed=93)
    b.q = (b.q.float() * 4).to(b.q.dtype)
    got = shared_run(b, softcap=cap)
    k0, v0 = (_gather(x, b.prefix_table[0], 260, 16) for x in (b.k_pages, b.v_pages))
    parts = []
    for s, n in enumerate(b.lens):
        k, v = (torch.cat([x0, _gather(x, b.table[s], n, 16)], 1)
                for x0, x in ((k0, b.k_pages), (v0, b.v_pages)))
        parts.append(_attend(b.q[s:s + 1], k, v, torch.tensor([260 + n - 1]), cap, None, dtype))
    e = [np.concatenate(x) for x in zip(*parts)]
    check_attention(got, e, dtype, 260 + max(b.lens), f"group of {members}, cap {cap}")


def test_a_cap_far_above_the_scores_is_no_cap():
    """fp32 and bf16, both kernels: a cap of 2^100 changes nothing but roundings."""
    for dtype, shapes in (("bf16", SHAPES), ("f32", SHAPES)):
        for new, lens, page in shapes:
            b = Batch(new, lens, 8, 4, 128, page, dtype, seed=94, q_std=4.0)
            x, y = run(b).double(), run(b, softcap=2.0 ** 100).double()
            # bf16: two roundings to bf16, of the weights and of the result, on either
            # side.  fp32: sums of up to 300 weights at 2^-23 on either side, and scores
            # of up to 20 that differ by four roundings
            limit = 2.0 ** -6 if dtype == "bf16" else 2 * 300 * 2.0 ** -23 + 2 * 20 * 2.0 ** -22
            assert float((x - y).abs().max()) <= limit * float(dev(b.v_pages).nan_to_num().abs().max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new,lens,page", SHAPES)
@pytest.mark.parametrize("biased", [False, True])
def test_a_cap_far_below_the_scale(new, lens, page, biased, dtype):
    """Queries 2^24 times smaller under a scale 2^24 times larger: the same scores
    and cap, but for a polynomial on the products themselves nothing is left."""
    b = Batch(new, lens, 8, 4, 128, page, dtype, seed=99, q_std=4.0)
    opt = dict(softcap=6.0, **({"slopes": _slopes(8)} if biased else {}))
    got = run(b, q=dev(b.q) * 2.0 ** -24, scale=2.0 ** 24 * 128 ** -0.5, **opt)
    check(b, got, 6.0, opt.get("slopes"), f"far below {dtype} {new}")
