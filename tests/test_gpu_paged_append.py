"""M-RoPE with the paged append on the GPU against the oracle."""
import numpy as np
import pytest
import torch

import oracle
import swiglu_ar_tts_b200 as ops
from swiglu_ar_tts_b200 import inputs
from gpu_util import dev, misaligned
from paged_util import UNUSED, table_for
from tolerance import check, to_f64

pytestmark = pytest.mark.gpu


def _pair_scale(x):
    half = x.shape[-1] // 2
    m = np.maximum(np.abs(x[..., :half]), np.abs(x[..., half:]))
    return np.concatenate([m, m], axis=-1)


class Case:
    def __init__(self, new, lens, hq=16, hk=8, d=128, page=16, dtype="bf16", norm="qk", seed=0,
                 pad=0, sections=None):
        rng = np.random.default_rng(seed)
        need = sum(-(-max(n, 0) // page) for n in lens)
        self.table = table_for(lens, page, list(rng.permutation(need + 3)))
        self.q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.lens = np.array(lens, dtype=np.int32)
        t = int(self.q_start[-1]) + pad
        self.q = inputs.normal((t, hq, d), seed, std=3.0, dtype=dtype)
        self.k = inputs.normal((t, hk, d), seed + 1, dtype=dtype)
        self.v = inputs.normal((t, hk, d), seed + 2, dtype=dtype)
        self.kp = inputs.normal((need + 3, hk, page, d), seed + 3, dtype=dtype)
        self.vp = inputs.normal((need + 3, hk, page, d), seed + 4, dtype=dtype)
        g = [inputs.normal((d,), seed + 5 + i, mean=1.0, std=0.1, dtype=dtype) for i in range(2)]
        self.gq = g[0] if "q" in norm else None
        self.gk = g[1] if "k" in norm else None
        self.pos = torch.from_numpy(rng.integers(0, 5000, size=(3, t)).astype(np.int32))
        self.sections = sections or (d // 2 - 2 * (d // 6), d // 6, d // 6)
        self.dtype = dtype

    def expected(self, q_out):
        return oracle.get().mrope_paged_append(
            self.q, self.k, self.v, self.pos, self.q_start, self.lens, self.table, self.kp,
            self.vp, self.sections, 1e6, self.gq, self.gk, 1e-6, q_out)

    def run(self, q=None, k=None, v=None, kp=None, vp=None, q_out=None):
        a = [dev(self.q) if q is None else q, dev(self.k) if k is None else k,
             dev(self.v) if v is None else v]
        kp = dev(self.kp) if kp is None else kp
        vp = dev(self.vp) if vp is None else vp
        if q_out is None:
            q_out = torch.full_like(self.q, 7.0, device="cuda")
        ops.mrope_paged_append(*a, dev(self.pos), dev(torch.from_numpy(self.q_start)),
                               dev(torch.from_numpy(self.lens)), dev(torch.from_numpy(self.table)),
                               kp, vp, self.sections, 1e6,
                               None if self.gq is None else dev(self.gq),
                               None if self.gk is None else dev(self.gk), 1e-6, q_out)
        torch.cuda.synchronize()
        return q_out, kp, vp

    def check(self, got, what=""):
        q_out, kp, vp = got
        qe, ke, ve = self.expected(np.full(self.q.shape, 7.0))
        orc = oracle.get()
        d = self.q.shape[-1]
        qs, ks = to_f64(self.q), to_f64(self.k)
        if self.gq is not None:
            qs = orc.rmsnorm(qs.reshape(-1, d), self.gq, 1e-6).reshape(qs.shape)
        if self.gk is not None:
            ks = orc.rmsnorm(ks.reshape(-1, d), self.gk, 1e-6).reshape(ks.shape)
        check(q_out, qe, self.dtype, _pair_scale(qs), what=f"{what} q")
        assert np.array_equal(to_f64(vp), ve), f"{what} v"
        # k slots within tolerance; slots that no token names keep their bits
        changed = (ke != to_f64(self.kp)).any(-1)
        assert np.array_equal(to_f64(kp)[~changed], ke[~changed]), f"{what} untouched k"
        scale = np.full(ke.shape, np.abs(ks).max() if ks.size else 0.0)
        page = self.kp.shape[2]
        for s in range(self.lens.size):
            for t in range(self.q_start[s], self.q_start[s + 1]):
                p = self.lens[s] - (self.q_start[s + 1] - t)
                if p >= 0 and p // page < self.table.shape[1]:
                    pg = self.table[s, p // page]
                    if 0 <= pg < ke.shape[0]:
                        scale[pg, :, p % page] = _pair_scale(ks[t])
        check(kp, ke, self.dtype, scale, what=f"{what} k")


@pytest.mark.parametrize("norm", ["", "q", "k", "qk"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_and_prompts(dtype, norm):
    # one token each; prompts from nothing; a chunk onto a past; an empty sequence
    for new, lens in (([1] * 5, [1, 17, 32, 33, 100]), ([40, 0, 7, 300], [40, 12, 20, 333])):
        c = Case(new, lens, dtype=dtype, norm=norm, seed=len(new))
        c.check(c.run(), f"{dtype} {norm} {new}")


@pytest.mark.parametrize("tokens", [1, 256, 1500])
def test_many_sequences_and_launch_shapes(tokens):
    new = [1] * tokens
    c = Case(new, [1 + i % 40 for i in range(tokens)], hq=4, hk=2, d=64, seed=tokens)
    c.check(c.run())


@pytest.mark.parametrize("hq,hk,d,page", [(3, 2, 96, 20), (7, 7, 80, 1), (2, 1, 10, 5), (24, 3, 256, 48),
                                          (5, 5, 512, 7), (16, 2, 32, 128), (8, 1, 16, 3), (0, 4, 128, 16),
                                          (4, 0, 128, 16)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_head_layouts_and_pages(dtype, hq, hk, d, page):
    c = Case([9, 1, 30], [9, 50, 44], hq, hk, d, page, dtype, seed=d)
    if hk == 0:  # a pool without heads: only q is rotated
        q_out, _, _ = c.run()
        qe, _, _ = c.expected(None)
        check(q_out, qe, dtype, _pair_scale(to_f64(q_out)) * 2)
        return
    c.check(c.run(), f"{dtype} {hq}/{hk}/{d}/{page}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("extra", [0, 8, 3])
def test_slices_of_a_packed_projection(dtype, extra):
    """q, k, v from one buffer (strides kept, or misaligned by an odd extra)."""
    c = Case([33, 5], [40, 5], dtype=dtype, seed=3)
    t, hq, d = c.q.shape
    hk = c.k.shape[1]
    flat = torch.zeros(t, (hq + 2 * hk) * d + extra, dtype=c.q.dtype, device="cuda")
    q = flat[:, :hq * d].unflatten(1, (hq, d))
    k = flat[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
    v = flat[:, (hq + hk) * d:(hq + 2 * hk) * d].unflatten(1, (hk, d))
    q.copy_(c.q), k.copy_(c.k), v.copy_(c.v)
    before = flat.clone()
    c.check(c.run(q, k, v), "packed")
    assert torch.equal(flat, before)
    # q rotated in place, the rest of the buffer as it was
    got = c.run(q, k, v, q_out=q)
    c2 = torch.equal(flat[:, hq * d:], before[:, hq * d:])
    assert c2
    c.check((q.contiguous(), got[1], got[2]), "in place")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_misaligned_buffers(dtype):
    c = Case([33, 5], [40, 5], dtype=dtype, seed=4)
    c.check(c.run(kp=misaligned(c.kp), vp=misaligned(c.vp)), "misaligned pages")
    c.check(c.run(q=misaligned(c.q)), "misaligned q")


def test_padding_is_left_as_it_was():
    c = Case([3, 2], [30, 2], pad=6, seed=5)
    q_out, kp, vp = c.run()
    assert bool((q_out[5:] == 7.0).all())
    c.check((q_out, kp, vp), "padded")


def test_bad_pages_and_positions_are_skipped_and_flagged():
    for d in (128, 80):
        c = Case([2, 2, 5, 1], [40, 40, 3, 5000], d=d, page=16, seed=6)
        # page past the pool, negative page, more tokens than positions, a
        # length past the table
        c.table[0, 2], c.table[1, 2], c.table[3, :] = 10_000, -5, UNUSED
        c.lens[3] = 5000
        c.table = c.table[:, :4].copy()
        ops.device_errors(clear=True)
        got = c.run()
        assert ops.device_errors(clear=True) == 2
        c.check(got, f"bad {d}")


def test_malformed_starts_write_nothing_out_of_place():
    c = Case([4, 4], [20, 20], seed=7)
    c.q_start = np.array([0, 6, 4], dtype=np.int32)  # decreasing: sequence 1 has no tokens
    q_out, kp, vp = c.run()
    # tokens 0..5 belong to sequence 0 (its last six positions), 6 and 7 to none
    assert bool((q_out[6:] == 7.0).all())
    c.q_start = np.array([0, 6, 6], dtype=np.int32)
    c.check((q_out, kp, vp), "decreasing")


def test_graph_replay_follows_the_lengths():
    c = Case([1] * 5, [1, 17, 32, 33, 100], seed=8)
    q, k, v, pos = dev(c.q), dev(c.k), dev(c.v), dev(c.pos)
    start, lens, table = (dev(torch.from_numpy(a)) for a in (c.q_start, c.lens, c.table))
    kp, vp, q_out = dev(c.kp), dev(c.vp), torch.zeros_like(q)
    gq, gk = dev(c.gq), dev(c.gk)

    def step():
        ops.mrope_paged_append(q, k, v, pos, start, lens, table, kp, vp, c.sections, 1e6, gq, gk,
                               q_out=q_out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    c.lens = np.array([2, 16, 31, 1, 97], dtype=np.int32)
    kp.copy_(c.kp), vp.copy_(c.vp), lens.copy_(torch.from_numpy(c.lens))
    g.replay()
    torch.cuda.synchronize()
    c.check((q_out, kp, vp), "replay")


def test_offsets_past_32_bits():
    """A pool of more than 2^31 elements: the slots lie at its far end."""
    hk, page, d = 2, 16, 128
    pages = (1 << 31) // (hk * page * d) + 40
    c = Case([4, 1], [20, 33], hq=4, hk=hk, d=d, page=page, seed=9)
    small = c.kp.shape[0]
    kp = torch.zeros(pages, hk, page, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    kp[-small:].copy_(c.kp), vp[-small:].copy_(c.vp)
    table = c.table.copy()
    c.table = np.where(table < small, table + pages - small, table).astype(np.int32)
    q_out, _, _ = c.run(kp=kp, vp=vp)
    c.table = table
    assert not bool(kp[:-small].any()) and not bool(vp[:-small].any())
    c.check((q_out, kp[-small:], vp[-small:]), "far")
