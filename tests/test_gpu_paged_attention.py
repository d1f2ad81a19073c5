"""Attention over the paged cache, and with shared prefixes, on the GPU against
the oracle.  Unused slots hold NaN and unused table entries lead nowhere."""
import numpy as np
import pytest
import torch

import oracle
import swiglu_ar_tts_b200 as ops
from swiglu_ar_tts_b200 import inputs
from gpu_util import dev, misaligned
from paged_util import UNUSED, Batch, Groups, check_attention, score_constants
from tolerance import to_f64

pytestmark = pytest.mark.gpu


def _slopes(hq):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], dtype=torch.float32)


def expected(b, **opt):
    return oracle.get_omp().paged_attention(b.q, b.k_pages, b.v_pages, b.q_start, b.kv_lens,
                                            b.table, **opt, **score_constants(b.dtype, b.d))


def run(b, q=None, pools=None, workspace=None, **opt):
    kp, vp = pools or (dev(b.k_pages), dev(b.v_pages))
    opt = {k: dev(torch.as_tensor(v)) if k in ("slopes", "bidir_lens") else v
           for k, v in opt.items()}
    out = torch.full(b.q.shape, 7.0, dtype=b.q.dtype, device="cuda")
    ops.paged_attention(dev(b.q) if q is None else q, kp, vp, *b.arrays(), workspace=workspace,
                        out=out, **opt)
    torch.cuda.synchronize()
    return out


def check(b, got, what="", **opt):
    e = expected(b, **opt)
    n = int(b.q_start[-1])
    check_attention(got[:n], [x[:n] for x in e], b.dtype, max(b.lens + [0]), what)
    assert bool((got[n:] == 7.0).all()), f"{what}: padding written"


# (new tokens, cache lengths) of each sequence
MIXES = {
    "one": ([1], [1]),
    "decode": ([1] * 6, [1, 2, 15, 16, 17, 700]),
    "empty cache": ([1, 1, 0, 1], [0, 5, 9, 64]),
    "prompts": ([1, 63, 64, 65, 130], [1, 63, 64, 65, 130]),
    "chunks": ([5, 17, 100], [300, 129, 411]),
    "more queries than keys": ([8, 20], [3, 0]),
    "long prompt": ([700], [700]),
    "many more queries than keys": ([80, 70, 1], [3, 0, 200]),
    "prompt and steps": ([400, 1, 1, 1, 3], [400, 900, 33, 2, 65]),
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mix", MIXES)
def test_mixes(mix, dtype):
    new, lens = MIXES[mix]
    b = Batch(new, lens, 16, 8, 128, 16, dtype, seed=len(mix), pad=3)
    check(b, run(b), f"{mix} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hk,d,page", [(8, 1, 128, 16), (7, 7, 64, 24), (24, 3, 96, 20), (40, 2, 80, 64),
                                          (4, 4, 33, 1), (6, 2, 8, 128), (16, 8, 128, 512), (12, 4, 1, 5),
                                          (2, 2, 100, 8), (34, 1, 64, 32)])
def test_head_layouts_and_pages(hq, hk, d, page, dtype):
    for new, lens in (([1, 1, 4], [200, 33, 77]), ([90, 150, 2], [90, 301, 64])):
        b = Batch(new, lens, hq, hk, d, page, dtype, seed=d + page)
        check(b, run(b), f"{dtype} {hq}/{hk}/{d}/{page} {new}")


@pytest.mark.parametrize("hq,hk,d,page", [(128, 1, 64, 16), (256, 2, 16, 8), (48, 1, 120, 16), (5, 1, 24, 40),
                                          (260, 1, 72, 256)])
def test_tile_kernel_heads(hq, hk, d, page):
    """Heads a token that fill, divide and outnumber the rows of a tile; narrow ones."""
    b = Batch([3, 40, 0, 1], [100, 290, 7, 140], hq, hk, d, page, "bf16", seed=hq + d, pad=1)
    check(b, run(b), f"{hq}/{hk}/{d}/{page}")
    opt = dict(softcap=4.0, slopes=_slopes(hq), window=90)
    check(b, run(b, **opt), f"{hq}/{hk}/{d}/{page} options", **opt)


@pytest.mark.parametrize("d", [136, 192, 255, 256])
def test_wide_heads(d):
    for new, lens in (([1, 1, 4], [200, 33, 77]), ([60, 2], [90, 301])):
        b = Batch(new, lens, 8, 2, d, 16, "bf16", seed=d)
        check(b, run(b), f"{d} {new}")


OPTIONS = {
    "cap": dict(softcap=5.0),
    "window": dict(window=40),
    "window 1": dict(window=1),
    "slopes": dict(slopes=True),
    "bidirectional start": dict(bidir_lens=[0, 50, 10_000, 7]),
    "all": dict(softcap=20.0, window=100, slopes=True, bidir_lens=[3, 90, 1, 0]),
    "scale": dict(scale=-0.3),
    "scale 0": dict(scale=0.0),
    "tiny cap": dict(softcap=1e-20),
    "huge window": dict(window=2 ** 31 - 1),
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", OPTIONS)
@pytest.mark.parametrize("new,lens", [([1, 1, 1, 1], [300, 20, 65, 128]), ([130, 60, 20, 5], [130, 200, 20, 300]),
                                      ([2, 9, 1, 3], [1, 4, 0, 300])])
def test_score_options(name, new, lens, dtype):
    opt = dict(OPTIONS[name])
    if "slopes" in opt:
        opt["slopes"] = _slopes(16)
    if "bidir_lens" in opt:
        opt["bidir_lens"] = np.array(opt["bidir_lens"], dtype=np.int32)
    b = Batch(new, lens, 16, 8, 128, 16, dtype, seed=11)
    check(b, run(b, **opt), f"{name} {dtype} {new}", **opt)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 128)])
def test_long_axis_is_split_and_joined(dtype, d):
    b = Batch([1, 3], [20000, 12345], 16, 8, d, 64, dtype, seed=12)
    ws = ops.attention_prepare(torch.empty(ops.attention_workspace(b.tokens, 16, d),
                                           dtype=torch.uint8, device="cuda"))
    first = run(b, workspace=ws)
    check(b, first, "split")
    # the counters were left at zero, and the order of arrival changes no bit
    for _ in range(5):
        assert torch.equal(run(b, workspace=ws), first)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_chunk_on_a_long_cache(dtype):
    n = 96 if dtype == "bf16" else 12
    b = Batch([n, 40], [9000, 40], 16, 8, 128, 32, dtype, seed=13)
    opt = dict(softcap=30.0, slopes=_slopes(16))
    ws = ops.attention_prepare(torch.empty(ops.attention_workspace(b.tokens, 16, 128),
                                           dtype=torch.uint8, device="cuda"))
    first = run(b, workspace=ws, **opt)
    check(b, first, "chunk", **opt)
    for _ in range(3):
        assert torch.equal(run(b, workspace=ws, **opt), first)


def test_large_and_small_scores():
    """Scores far apart: one key takes all, or the running maximum keeps growing."""
    b = Batch([64, 1, 200], [64, 500, 900], 16, 8, 128, 16, "bf16", seed=14, q_std=30.0)
    check(b, run(b), "large")
    for s in range(3):  # keys growing along the sequence: the maximum moves every tile
        for p in range(b.lens[s]):
            pg, sl = b.table[s, p // 16], p % 16
            b.k_pages[pg, :, sl] = b.k_pages[pg, :, sl] * 0.0 + (p / 300.0) * b.q[int(b.q_start[s]), ::2] / 30
    check(b, run(b), "growing")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_and_misaligned(dtype):
    b = Batch([1, 70, 1], [65, 200, 300], 16, 8, 128, 16, dtype, seed=15)
    want = run(b)
    check(b, want)
    packed = torch.zeros(b.tokens, 32 * 128 + 8, dtype=b.q.dtype, device="cuda")
    q = packed[:, :2048].unflatten(1, (16, 128))
    q.copy_(b.q)
    assert torch.equal(run(b, q=q), want)
    check(b, run(b, q=misaligned(b.q)), "misaligned q")
    check(b, run(b, pools=(misaligned(b.k_pages), misaligned(b.v_pages))), "misaligned pages")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 70])
def test_pages_in_front_of_a_window_may_be_gone(new, dtype):
    """With a sliding window the table's first entries may lead nowhere."""
    window = 100
    b = Batch([new] * 2, [900, 1300], 16, 8, 128, 16, dtype, seed=23)
    whole = b.table.copy()
    got = run(b, window=window)
    e = expected(b, window=window)
    for s, n in enumerate(b.lens):
        b.table[s, :(n - new - window + 1) // 16] = UNUSED
    again = run(b, window=window)
    assert ops.device_errors(clear=True) == 0
    assert torch.equal(got, again)
    check_attention(again, e, dtype, 200, "gone")
    assert not np.array_equal(whole, b.table)


def test_more_sequences_than_the_kernel_keeps_counts_of():
    n = 9001
    b = Batch([1] * n, [1 + i % 5 for i in range(n)], 2, 1, 64, 8, "bf16", seed=24)
    check(b, run(b), "9001 sequences")


def test_negative_lengths_are_empty():
    b = Batch([1, 2, 60], [20, 0, 0], 16, 8, 128, 16, "bf16", seed=25)
    b.kv_lens[1:] = [-5, -2 ** 31]
    got = run(b)
    assert not bool(got[1:63].any())


@pytest.mark.parametrize("n", [1, 120])
def test_dependent_launches(n):
    """With programmatic dependent launch every kernel still waits for the one
    before it: append, attention, append, attention without a pause."""
    c = Batch([n], [n + 40], 16, 8, 128, 16, "bf16", seed=26)
    start, lens, table = c.arrays()
    k = inputs.normal((n, 8, 128), 27).cuda()
    q, pos = dev(c.q), torch.zeros(3, n, dtype=torch.int32, device="cuda")
    ws = ops.attention_prepare(torch.empty(ops.attention_workspace(n, 16, 128), dtype=torch.uint8,
                                           device="cuda"))
    results = []
    for pdl in (False, True):
        kp, vp = dev(c.k_pages), dev(c.v_pages)
        out = [torch.empty_like(q) for _ in range(6)]
        old = ops.set_pdl(pdl)
        try:
            torch.cuda._sleep(1_000_000)
            for i in range(6):
                ops.mrope_paged_append(q, k if i % 2 else -k, k if i % 2 else 2 * k, pos, start, lens, table,
                                       kp, vp)
                ops.paged_attention(q, kp, vp, start, lens, table, workspace=ws, out=out[i])
        finally:
            ops.set_pdl(old)
        torch.cuda.synchronize()
        results.append(torch.stack(out))
    assert torch.equal(results[0], results[1])
    assert torch.equal(results[0][0], results[0][2]) and not torch.equal(results[0][0], results[0][1])


def test_workspace_that_was_not_cleared_is_flagged():
    b = Batch([1], [20000], 16, 8, 128, 16, "bf16", seed=28)
    ws = torch.full((ops.attention_workspace(1, 16, 128),), 0x11, dtype=torch.uint8, device="cuda")
    ops.device_errors(clear=True)
    run(b, workspace=ws)
    assert ops.device_errors(clear=True) == 4  # AROPS_DEVICE_ERR_WORKSPACE


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("opt", [{}, {"softcap": 5.0}])
@pytest.mark.parametrize("new,lens", [([1, 1, 1], [1, 40, 900]), ([1], [9000]), ([3, 40], [3, 70]),
                                      ([130, 60], [130, 200]), ([40], [6000])])
def test_nan_query_row_stays_nan(new, lens, opt, dtype):
    """All of a NaN query's scores are NaN: whichever parts its row is joined
    from, it is not an empty row.  Other rows are what they were."""
    b = Batch(new, lens, 16, 8, 128, 16, dtype, seed=81)
    q = dev(b.q).clone()
    t, h = b.tokens - 1, 5
    q[t, h, 3] = float("nan")
    got = run(b, q=q, **opt)
    assert bool(torch.isnan(got[t, h]).all())
    got[t, h] = torch.from_numpy(expected(b, **opt)[0][t, h]).to(got)
    check(b, got, f"nan {new}", **opt)


@pytest.mark.parametrize("new,lens", [([1, 1], [30, 700]), ([100, 30], [100, 230]), ([7, 60], [1000, 99])])
@pytest.mark.parametrize("opt", [{}, {"softcap": 20.0}, {"softcap": 3.0, "slopes": _slopes(16)}])
def test_what_lies_behind_a_length_changes_no_bit(new, lens, opt):
    b = Batch(new, lens, 16, 8, 128, 16, "bf16", seed=85)
    first = run(b, **opt)
    check(b, first, "NaN behind", **opt)
    for value in (0.0, 3e4, float("inf")):
        pools = [dev(torch.nan_to_num(x, nan=value)) for x in (b.k_pages, b.v_pages)]
        assert torch.equal(run(b, pools=pools, **opt), first), f"{value} behind"


def test_numbers_that_a_field_cannot_hold_are_refused():
    """2^32 + 5 must not come out as a window of 5."""
    b = Batch([1], [20], 16, 8, 128, 16, "bf16", seed=88)
    for bad in (dict(window=2 ** 32 + 5), dict(window=-(2 ** 31) - 1), dict(window=2.5),
                dict(softcap=1e300), dict(scale="a")):
        with pytest.raises((ValueError, ops.ArOpsError)):
            run(b, **bad)


def test_very_wide_tables():
    """Tables for more positions than the tile kernel takes, and one for exactly as many."""
    for pages in (2 ** 16, 2 ** 16 + 1):
        b = Batch([100, 30], [300, 30], 16, 8, 128, 128, "bf16", seed=87)
        wide = np.full((2, pages), UNUSED, dtype=np.int32)
        wide[:, :b.table.shape[1]] = b.table
        b.table = wide
        check(b, run(b), f"{pages} pages")


def test_dense_cache_is_one_page_a_row():
    """The dense cache of mrope_kv_append: rows are pages, the table the identity."""
    b = Batch([1] * 4, [300, 20, 1, 299], 16, 8, 128, 300, "bf16", seed=16, spare=0)
    check(b, run(b), "dense")


def test_bad_pages_read_as_zeros_and_are_flagged():
    for new in ([1, 1, 1], [40, 40, 30]):
        b = Batch(new, [100, 100, 64], 16, 8, 128, 16, "bf16", seed=17)
        b.table[0, 2], b.table[1, 5] = -1, b.k_pages.shape[0]
        b.kv_lens[2] = 5000  # behind the table: counts as its capacity
        b.table = b.table[:, :7].copy()
        b.table[2, 4:] = b.table[2, :3]
        b.lens[2] = 112
        ops.device_errors(clear=True)
        got = run(b)
        assert ops.device_errors(clear=True) == 2
        check(b, got, f"bad {new}")


def test_malformed_starts_stay_in_bounds():
    b = Batch([4, 4], [20, 20], 16, 8, 128, 16, "bf16", seed=18)
    for start in ([0, 6, 4], [0, 4, 9999], [-3, 4, 8], [0, 2 ** 31 - 1, -(2 ** 31)]):
        b.q_start = np.array(start, dtype=np.int32)
        ops.device_errors(clear=True)
        got = run(b)
        ops.device_errors(clear=True)
        assert not bool(torch.isnan(got).any())


def test_graph_replay_follows_lengths_on_another_stream():
    b = Batch([1] * 5, [900, 17, 32, 33, 100], 16, 8, 128, 16, "bf16", seed=19)
    start, lens, table = b.arrays()
    q, kp, vp = dev(b.q), dev(b.k_pages), dev(b.v_pages)
    ws = ops.attention_prepare(torch.empty(ops.attention_workspace(5, 16, 128), dtype=torch.uint8,
                                           device="cuda"))
    out = torch.empty_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ops.paged_attention(q, kp, vp, start, lens, table, workspace=ws, out=out)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            ops.paged_attention(q, kp, vp, start, lens, table, workspace=ws, out=out)
    torch.cuda.synchronize()
    for n in ([900, 17, 32, 33, 100], [1, 16, 5, 30, 99], [700, 0, 31, 2, 64]):
        b.kv_lens = np.array(n, dtype=np.int32)
        lens.copy_(torch.from_numpy(b.kv_lens))
        torch.cuda.synchronize()
        out.fill_(7.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        torch.cuda.synchronize()
        check(b, out, f"replay {n}")


def test_two_calls_at_once_with_workspaces_of_their_own():
    a = Batch([1, 2], [9000, 5000], 16, 8, 128, 16, "bf16", seed=20)
    b = Batch([300, 1], [300, 8000], 16, 8, 128, 16, "bf16", seed=21)
    want = [run(a), run(b)]
    sets = []
    for x in (a, b):
        ws = ops.attention_prepare(torch.empty(ops.attention_workspace(x.tokens, 16, 128),
                                               dtype=torch.uint8, device="cuda"))
        sets.append((dev(x.q), dev(x.k_pages), dev(x.v_pages), x.arrays(), ws, torch.empty_like(dev(x.q))))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, (q, kp, vp, arr, ws, out) in zip(streams, sets):
            with torch.cuda.stream(s):
                ops.paged_attention(q, kp, vp, *arr, workspace=ws, out=out)
    torch.cuda.synchronize()
    for w, x in zip(want, sets):
        assert torch.equal(w, x[5])


def test_offsets_past_32_bits():
    hk, page, d = 2, 16, 128
    pages = (1 << 31) // (hk * page * d) + 60
    for new in ([1, 3], [200, 70]):
        b = Batch(new, [500, 300], 4, hk, d, page, "bf16", seed=22)
        small = b.k_pages.shape[0]
        kp = torch.zeros(pages, hk, page, d, dtype=torch.bfloat16, device="cuda")
        vp = torch.zeros_like(kp)
        kp[-small:].copy_(b.k_pages), vp[-small:].copy_(b.v_pages)
        table = b.table.copy()
        b.table = np.where(table < small, table + pages - small, table).astype(np.int32)
        got = run(b, pools=(kp, vp))
        b.table = table
        check(b, got, f"far {new}")


# -- shared prefixes -----------------------------------------------------------
def shared_expected(b, **opt):
    return oracle.get_omp().shared_prefix_attention(
        b.q, b.k_pages, b.v_pages, b.group_start, b.prefix_lens, b.prefix_table, b.kv_lens,
        b.table, **opt, **score_constants(b.dtype, b.q.shape[2]))


def shared_run(b, workspace=None, pools=None, q=None, **opt):
    kp, vp = pools or (dev(b.k_pages), dev(b.v_pages))
    opt = {k: dev(v) if k == "slopes" else v for k, v in opt.items()}
    out = torch.full(b.q.shape, 7.0, dtype=b.q.dtype, device="cuda")
    ops.shared_prefix_attention(dev(b.q) if q is None else q, kp, vp, *b.arrays(),
                                workspace=workspace, out=out, **opt)
    torch.cuda.synchronize()
    return out


def shared_check(b, got, what="", **opt):
    e = shared_expected(b, **opt)
    n = int(b.group_start[-1])
    keys = max(b.prefix + [0]) + max(b.lens + [0])
    check_attention(got[:n], [x[:n] for x in e], b.dtype, keys, what)
    assert bool((got[n:] == 7.0).all()), f"{what}: padding written"


GROUPS = {
    "five candidates": ([5], [333], [1, 40, 17, 64, 200]),
    "one": ([1], [1], [1]),
    "no own keys": ([3], [100], [0, 0, 5]),
    "no prefix": ([2, 2], [0, 40], [3, 50, 0, 7]),
    "nothing": ([2, 1], [0, 5], [0, 0, 1]),
    "ragged": ([1, 9, 0, 4], [50, 129, 10, 64], [1 + 13 * i % 70 for i in range(14)]),
    "many": ([70], [500], [1 + 7 * i % 90 for i in range(70)]),
    "two large": ([100, 33], [300, 700], [1 + 5 * i % 50 for i in range(133)]),
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", GROUPS)
def test_groups(name, dtype):
    members, prefix, lens = GROUPS[name]
    pad = 2
    b = Groups(members, prefix, lens + [9] * pad, 16, 8, 128, 16, dtype, seed=30, pad=pad)
    shared_check(b, shared_run(b), f"{name} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hk,d,page", [(8, 1, 128, 16), (7, 7, 64, 24), (24, 3, 96, 20), (40, 2, 80, 64),
                                          (4, 4, 33, 1), (34, 1, 64, 32), (8, 2, 128, 8)])
def test_group_head_layouts(hq, hk, d, page, dtype):
    for members, prefix, lens in (([5, 2], [200, 31], [3, 60, 1, 0, 17, 90, 2]),
                                  ([80], [260], [1 + 3 * i % 40 for i in range(80)])):
        b = Groups(members, prefix, lens, hq, hk, d, page, dtype, seed=31)
        shared_check(b, shared_run(b), f"{dtype} {hq}/{hk}/{d}/{page} {members}")


# enough rows a group for the prefix to go to the tile kernel
@pytest.mark.parametrize("hq,hk,d,page,members,prefix", [
    (16, 8, 128, 16, [270], [500]), (16, 8, 128, 64, [150, 0, 128], [700, 9, 0]), (8, 1, 64, 32, [66], [129]),
    (24, 3, 96, 24, [40, 40], [260, 1]), (40, 2, 80, 8, [30], [333]), (34, 1, 128, 16, [20], [128])])
@pytest.mark.parametrize("opt", ["", "cap", "slopes", "all"])
def test_groups_of_many_rows(hq, hk, d, page, members, prefix, opt):
    o = {"": {}, "cap": dict(softcap=5.0), "slopes": dict(slopes=_slopes(hq)),
         "all": dict(softcap=15.0, scale=-0.1, slopes=_slopes(hq))}[opt]
    n, pad = sum(members), 3
    b = Groups(members, prefix, [5 * i % 70 for i in range(n)] + [9] * pad, hq, hk, d, page, "bf16", seed=37,
               pad=pad)
    ws = ops.attention_prepare(torch.empty(ops.attention_workspace(n + pad, hq, d), dtype=torch.uint8,
                                           device="cuda"))
    got = shared_run(b, workspace=ws, **o)
    shared_check(b, got, f"{hq}/{hk}/{d} {opt}", **o)
    assert torch.equal(shared_run(b, workspace=ws, **o), got)


def test_many_rows_bad_pages_and_lengths():
    b = Groups([280], [400], [20] * 280, 16, 8, 128, 16, "bf16", seed=38)
    b.prefix_table[0, 3] = -7
    b.table[2, 1] = 1 << 30
    b.prefix_lens[0] = 10 ** 6  # counts as the table's capacity
    b.prefix_table = b.prefix_table[:, :25].copy()
    ops.device_errors(clear=True)
    got = shared_run(b)
    assert ops.device_errors(clear=True) == 2
    shared_check(b, got, "bad")
    for start in ([0, 400], [-1, 280], [280, 0]):
        b.group_start = np.array(start, dtype=np.int32)
        assert bool((shared_run(b) == 7.0).all())
        assert ops.device_errors(clear=True) == 2


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("opt", ["cap", "window", "long window", "slopes", "all"])
@pytest.mark.parametrize("members", [[5, 3], [80]])
def test_group_score_options(opt, members, dtype):
    o = {"cap": dict(softcap=5.0), "window": dict(window=30), "long window": dict(window=150),
         "slopes": dict(slopes=_slopes(16)),
         "all": dict(softcap=15.0, window=120, slopes=_slopes(16))}[opt]
    n = sum(members)
    b = Groups(members, [300, 100][:len(members)], [1 + 11 * i % 60 for i in range(n)], 16, 8, 128, 16,
               dtype, seed=32)
    shared_check(b, shared_run(b, **o), f"{opt} {members} {dtype}", **o)


def test_group_long_prefix_split_and_repeated():
    for members in ([5], [130]):
        n = sum(members)
        b = Groups(members, [9000], [1 + 11 * i % 300 for i in range(n)], 16, 8, 128, 64, "bf16", seed=33)
        ws = ops.attention_prepare(torch.empty(ops.attention_workspace(n, 16, 128), dtype=torch.uint8,
                                               device="cuda"))
        first = shared_run(b, workspace=ws)
        shared_check(b, first, f"long {members}")
        for _ in range(3):
            assert torch.equal(shared_run(b, workspace=ws), first)


def test_group_equals_attention_over_joined_pages():
    """Candidates whose tables start with the prompt's whole pages, through
    paged_attention: the same keys in the same order."""
    page, prefix = 16, 160
    b = Groups([6], [prefix], [1, 9, 16, 30, 47, 200], 16, 8, 128, page, "bf16", seed=34)
    got = shared_run(b)
    table = np.concatenate([np.repeat(b.prefix_table[:, :prefix // page], 6, 0), b.table], 1)
    out = torch.empty_like(got)
    ops.paged_attention(dev(b.q), dev(b.k_pages), dev(b.v_pages),
                        torch.arange(7, dtype=torch.int32, device="cuda"),
                        dev(torch.from_numpy(b.kv_lens + prefix)),
                        dev(torch.from_numpy(np.ascontiguousarray(table))), out=out)
    torch.cuda.synchronize()
    e = shared_expected(b)
    check_attention(out, e, "bf16", 400, "joined")
    check_attention(got, e, "bf16", 400, "shared")


def test_group_bad_pages_are_flagged():
    for members in ([5], [90]):
        n = sum(members)
        b = Groups(members, [100], [20] * n, 16, 8, 128, 16, "bf16", seed=35)
        b.prefix_table[0, 3] = -7
        b.table[2, 1] = 1 << 30
        ops.device_errors(clear=True)
        got = shared_run(b)
        assert ops.device_errors(clear=True) == 2
        shared_check(b, got, f"bad {members}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("members,prefix,own", [([5], [300], 20), ([80], [300], 20), ([80], [300], 0),
                                                ([300], [4000], 70)])
def test_nan_query_of_a_group_stays_nan(members, prefix, own, dtype):
    b = Groups(members, prefix, [own] * sum(members), 16, 8, 128, 16, dtype, seed=83)
    q = dev(b.q).clone()
    t, h = b.n - 2, 9
    q[t, h, 100] = float("nan")
    got = shared_run(b, q=q)
    assert bool(torch.isnan(got[t, h]).all())
    got[t, h] = torch.from_numpy(shared_expected(b)[0][t, h]).to(got)
    shared_check(b, got, f"nan {members}")


@pytest.mark.parametrize("members,prefix", [([5], [300]), ([80], [300])])
@pytest.mark.parametrize("opt", [{}, {"softcap": 20.0}])
def test_what_lies_behind_a_prefix_changes_no_bit(members, prefix, opt):
    b = Groups(members, prefix, [20] * sum(members), 16, 8, 128, 16, "bf16", seed=86)
    first = shared_run(b, **opt)
    for value in (0.0, 3e4, float("inf")):
        pools = [dev(torch.nan_to_num(x, nan=value)) for x in (b.k_pages, b.v_pages)]
        assert torch.equal(shared_run(b, pools=pools, **opt), first), f"{value} behind"


def test_malformed_groups_stay_in_bounds():
    b = Groups([3, 2], [40, 30], [5] * 5, 16, 8, 128, 16, "bf16", seed=36)
    for start in ([0, 4, 2], [0, 3, 999], [-4, 3, 5], [2 ** 31 - 1, 0, -1]):
        b.group_start = np.array(start, dtype=np.int32)
        ops.device_errors(clear=True)
        got = shared_run(b)
        ops.device_errors(clear=True)
        assert not bool(torch.isnan(got).any())


# -- together ------------------------------------------------------------------
def test_prompt_candidates_and_steps_together():
    """A prompt is appended and attended to; five candidates of it then take
    decode steps that append to pages of their own and attend to both.  Every
    step's output is checked against the oracle on the cache of that moment."""
    hq, hk, d, page, prompt, n, steps = 16, 8, 128, 16, 75, 5, 20
    orc, omp = oracle.get(), oracle.get_omp()
    rng = np.random.default_rng(40)
    order = rng.permutation(40).astype(np.int32)
    ptab, own = order[:5][None].copy(), order[5:5 + n * 2].reshape(n, 2).copy()
    kp = torch.full((40, hk, page, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vp = torch.full_like(kp, float("nan"))
    gq, gk = (inputs.normal((d,), 41 + i, mean=1.0, std=0.1) for i in range(2))
    ws = ops.attention_prepare(torch.empty(ops.attention_workspace(max(n, prompt), hq, d),
                                           dtype=torch.uint8, device="cuda"))
    i32 = lambda a: torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731

    def qkv(tokens, seed):
        x = inputs.normal((tokens, (hq + 2 * hk) * d), seed)
        g = x.cuda()
        return (x, g[:, :hq * d].unflatten(1, (hq, d)), g[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d)),
                g[:, (hq + hk) * d:].unflatten(1, (hk, d)))

    _, q, k, v = qkv(prompt, 50)
    pos = torch.arange(prompt, dtype=torch.int32).repeat(3, 1)
    args = (i32([0, prompt]), i32([prompt]), i32(ptab))
    ops.mrope_paged_append(q, k, v, pos.cuda(), *args, kp, vp, gamma_q=dev(gq), gamma_k=dev(gk))
    out = ops.paged_attention(q, kp, vp, *args, workspace=ws)
    torch.cuda.synchronize()
    e = omp.paged_attention(q.cpu(), kp.cpu(), vp.cpu(), [0, prompt], [prompt], ptab,
                            **score_constants("bf16", d))
    check_attention(out, e, "bf16", prompt, "prompt")
    for step in range(steps):
        before_k, before_v = kp.cpu(), vp.cpu()
        _, q, k, v = qkv(n, 60 + step)
        q0 = q.cpu().clone()
        pos = torch.full((3, n), prompt + step, dtype=torch.int32)
        lens = np.full(n, step + 1, dtype=np.int32)
        ops.mrope_paged_append(q, k, v, pos.cuda(), i32(np.arange(n + 1)), i32(lens), i32(own), kp, vp,
                               gamma_q=dev(gq), gamma_k=dev(gk))
        out = ops.shared_prefix_attention(q, kp, vp, i32([0, n]), i32([prompt]), i32(ptab), i32(lens),
                                          i32(own), workspace=ws)
        torch.cuda.synchronize()
        if step % 6 == 0 or step == steps - 1:
            qe, ke, _ = orc.mrope_paged_append(q0, k.cpu(), v.cpu(), pos, np.arange(n + 1), lens, own,
                                               torch.nan_to_num(before_k), torch.nan_to_num(before_v),
                                               gamma_q=gq, gamma_k=gk)
            assert np.abs(to_f64(q) - qe).max() <= 2.0 ** -7 * np.abs(qe).max()
            assert np.abs(np.nan_to_num(to_f64(kp)) - ke).max() <= 2.0 ** -7 * np.abs(ke).max()
            e = omp.shared_prefix_attention(q.cpu(), kp.cpu(), vp.cpu(), [0, n], [prompt], ptab, lens, own,
                                            **score_constants("bf16", d))
            check_attention(out, e, "bf16", prompt + step + 1, f"step {step}")
