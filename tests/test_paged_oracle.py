"""The paged-cache oracle against closed forms and an independent fp64 formula
(CPU only): what it takes from the pages, which keys it counts as seen, and the
score options."""
import math

import numpy as np
import pytest
import torch

import oracle
from paged_util import Batch, Groups


def _dense(b, s):
    """Positions of sequence s, gathered page by page."""
    def take(pool):
        rows = [pool[b.table[s, p // b.page], :, p % b.page] for p in range(b.lens[s])]
        return torch.stack(rows, 1).double() if rows else torch.zeros(b.hk, 0, b.d).double()
    return take(b.k_pages), take(b.v_pages)


def _formula(q, k, v, first, scale, cap=0.0, window=0, slopes=None, bidir=0):
    """softmax over seen keys, one query and head at a time, in torch fp64."""
    n, hq, d = q.shape
    out = torch.zeros(n, hq, d, dtype=torch.float64)
    for t in range(n):
        i = first + t
        j = torch.arange(k.shape[1])
        seen = (j <= i) | (j < bidir)
        if window:
            seen &= j > i - window
        if not bool(seen.any()):
            continue
        for h in range(hq):
            s = scale * (k[h // (hq // k.shape[0])] @ q[t, h].double())
            if cap:
                s = cap * torch.tanh(s / cap)
            if slopes is not None:
                s = s - float(slopes[h]) * (i - j).abs().double()
            w = torch.softmax(s[seen], 0)
            out[t, h] = w @ v[h // (hq // k.shape[0])][seen]
    return out


@pytest.mark.parametrize("opt", [{}, dict(softcap=2.0), dict(window=5), dict(slopes=[0.5, 0.25, 0.1, 0.0]),
                                 dict(bidir_lens=[9, 0, 100]), dict(softcap=3.0, window=7, slopes=[1, .1, .2, .3],
                                                                    bidir_lens=[4, 4, 4])])
def test_against_a_formula(opt):
    b = Batch([3, 1, 12], [20, 9, 12], 4, 2, 8, 4, "f32", seed=1)
    out, mass, err = oracle.get().paged_attention(b.q, b.k_pages, b.v_pages, b.q_start, b.kv_lens, b.table,
                                                  c_dot=1e-7, c_abs=1e-7, **opt)
    for s in range(3):
        k, v = _dense(b, s)
        t0, t1 = b.q_start[s], b.q_start[s + 1]
        want = _formula(b.q[t0:t1], k, v, b.lens[s] - (t1 - t0), 8 ** -0.5, opt.get("softcap", 0.0),
                        opt.get("window", 0), opt.get("slopes"), opt.get("bidir_lens", [0] * 3)[s])
        np.testing.assert_allclose(out[t0:t1], want.numpy(), rtol=1e-12, atol=1e-13)
    assert np.all(mass >= np.abs(out) - 1e-12) and np.all(err >= 0)


def test_closed_forms():
    b = Batch([1, 2, 1], [10, 1, 0], 2, 1, 4, 3, "f32", seed=2)
    orc = oracle.get()
    # q = 0: the mean of the seen values; one seen key: that value; none: zero
    out, _, _ = orc.paged_attention(b.q * 0, b.k_pages, b.v_pages, b.q_start, b.kv_lens, b.table)
    _, v = _dense(b, 0)
    np.testing.assert_allclose(out[0, 0], v[0].mean(0).numpy(), rtol=1e-12)
    assert np.array_equal(out[1], np.zeros((2, 4)))  # position -1
    _, v1 = _dense(b, 1)
    np.testing.assert_allclose(out[2, 1], v1[0, 0].numpy(), rtol=1e-12)
    assert np.array_equal(out[3], np.zeros((2, 4)))
    # a slope of ln 2 halves the weight a position
    out, _, _ = orc.paged_attention(b.q * 0, b.k_pages, b.v_pages, b.q_start, b.kv_lens, b.table,
                                    slopes=[math.log(2)] * 2)
    w = 0.5 ** np.arange(9, -1, -1)
    np.testing.assert_allclose(out[0, 0], (w[:, None] * v[0].numpy()).sum(0) / w.sum(), rtol=1e-12)


def test_shared_prefix_is_joined_keys():
    b = Groups([2, 1], [7, 0], [3, 0, 5], 4, 2, 8, 4, "f32", seed=3)
    out, _, _ = oracle.get().shared_prefix_attention(b.q, b.k_pages, b.v_pages, b.group_start, b.prefix_lens,
                                                     b.prefix_table, b.kv_lens, b.table, window=9)
    for s, g in ((0, 0), (1, 0), (2, 1)):
        rows = [(b.prefix_table[g, p // 4], p % 4) for p in range(b.prefix[g])]
        rows += [(b.table[s, p // 4], p % 4) for p in range(b.lens[s])]
        k = torch.stack([b.k_pages[p, :, i] for p, i in rows], 1).double()
        v = torch.stack([b.v_pages[p, :, i] for p, i in rows], 1).double()
        want = _formula(b.q[s:s + 1], k, v, len(rows) - 1, 8 ** -0.5, window=9)
        np.testing.assert_allclose(out[s], want[0].numpy(), rtol=1e-12, atol=1e-13)


def test_pages_outside_the_pool_are_zeros():
    b = Batch([1], [10], 2, 1, 4, 3, "f32", seed=4)
    b.table[0, 1] = 999
    out, _, _ = oracle.get().paged_attention(b.q * 0, b.k_pages, b.v_pages, b.q_start, b.kv_lens, b.table)
    v = np.zeros(4)
    for p in (0, 1, 2, 6, 7, 8, 9):
        v += b.v_pages[b.table[0, p // 3], 0, p % 3].double().numpy()
    np.testing.assert_allclose(out[0, 0], v / 10, rtol=1e-12)


def test_append_goes_where_the_table_says():
    rng = np.random.default_rng(5)
    q, k, v = (torch.from_numpy(rng.standard_normal((4, h, 6))) for h in (2, 1, 1))
    pos = np.zeros((3, 4), dtype=np.int32)  # no rotation
    kp, vp = np.full((5, 1, 2, 6), 9.0), np.full((5, 1, 2, 6), 9.0)
    table = np.array([[3, 0], [1, 4]], dtype=np.int32)
    out, kn, vn = oracle.get().mrope_paged_append(q, k, v, pos, [0, 3, 3], [3, 0], table, kp, vp, (1, 1, 1),
                                                  q_out=np.full((4, 2, 6), 7.0))
    assert np.array_equal(out[:3], q[:3].numpy()) and np.all(out[3] == 7.0)  # the last token is padding
    for t, (p, s) in enumerate(((3, 0), (3, 1), (0, 0))):
        assert np.array_equal(kn[p, 0, s], k[t, 0].numpy()) and np.array_equal(vn[p, 0, s], v[t, 0].numpy())
    assert np.count_nonzero(kn != 9.0) == 18
    # with weights: RMSNorm a head first
    out, _, _ = oracle.get().mrope_paged_append(q, k, v, pos, [0, 3, 3], [3, 0], table, kp, vp, (1, 1, 1),
                                                gamma_q=np.full(6, 2.0), eps=0.0, q_out=np.zeros((4, 2, 6)))
    x = q[:3].numpy()
    np.testing.assert_allclose(out[:3], 2 * x / np.sqrt((x ** 2).mean(-1, keepdims=True)), rtol=1e-12)
