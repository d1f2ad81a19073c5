"""Host-side checks of the paged-cache entry points: what is refused, and that
nothing is launched for it (no GPU needed)."""
import ctypes as C

import pytest
import torch

import swiglu_ar_tts_b200 as ops
from swiglu_ar_tts_b200 import _AttentionOptions, _PagedBatch, _PagedCache, _PrefixGroups

SEC = (C.c_int32 * 3)(24, 20, 20)
P = 1 << 20  # stands for a device pointer; never followed on the host


@pytest.fixture(scope="module")
def L():
    return ops.lib()


def cache(k=P, v=2 * P, pages=10, page=16, heads=8, d=128, dtype=1):
    return _PagedCache(k, v, pages, page, heads, d, dtype)


def batch(start=P, lens=P, table=P, n=2, max_pages=4):
    return _PagedBatch(start, lens, table, n, max_pages)


def options(scale=0.1, cap=0.0, window=0, slopes=None, bidir=None):
    return _AttentionOptions(scale, cap, window, slopes, bidir)


def groups(start=P, lens=P, table=P, n=1, max_pages=4):
    return _PrefixGroups(start, lens, table, n, max_pages)


def append(L, c=None, b=None, q=P, k=P, v=P, out=2 * P, strides=(2048, 1024, 1024, 2048), gq=None,
           eps=1e-6, pos=P, tokens=2, hq=16, sec=SEC, theta=1e6):
    return L.arops_mrope_paged_append(
        q, strides[0], k, strides[1], v, strides[2], out, strides[3], c or cache(), b or batch(),
        gq, None, eps, pos, tokens, hq, sec, theta, None)


def attend(L, c=None, b=None, o=None, q=P, stride=2048, out=2 * P, tokens=2, hq=16, ws=16,
           ws_bytes=1 << 40):
    return L.arops_paged_attention(q, stride, out, c or cache(), b or batch(), o or options(),
                                   tokens, hq, ws, ws_bytes, None)


def shared(L, c=None, b=None, g=None, o=None, q=P, stride=2048, out=2 * P, hq=16, ws=16,
           ws_bytes=1 << 40):
    return L.arops_shared_prefix_attention(q, stride, out, c or cache(), b or batch(),
                                           g or groups(), o or options(), hq, ws, ws_bytes, None)


BAD_CACHES = [
    (dict(dtype=5), 1), (dict(pages=0), 1), (dict(pages=-1), 1), (dict(page=0), 1), (dict(d=0), 1),
    (dict(heads=-1), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(v=P), 1), (dict(pages=1 << 31), 2),
    (dict(d=1024), 2),
]
BAD_BATCHES = [
    (dict(n=-1), 1), (dict(max_pages=-1), 1), (dict(lens=None), 1), (dict(table=None), 1),
    (dict(max_pages=1 << 28), 2),
]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
@pytest.mark.parametrize("op", [append, attend, shared])
def test_bad_caches(L, op, kw, status):
    before = L.arops_launch_count()
    assert op(L, c=cache(**kw)) == status, L.arops_last_error()
    assert L.arops_last_error() != b"" and L.arops_launch_count() == before


@pytest.mark.parametrize("kw,status", BAD_BATCHES)
@pytest.mark.parametrize("op", [append, attend, shared])
def test_bad_batches(L, op, kw, status):
    before = L.arops_launch_count()
    assert op(L, b=batch(**kw)) == status, L.arops_last_error()
    assert L.arops_launch_count() == before


@pytest.mark.parametrize("kw,status", [
    (dict(b=batch(start=None)), 1), (dict(tokens=-1), 1), (dict(tokens=1 << 31), 2), (dict(hq=-1), 1),
    (dict(sec=None), 1), (dict(sec=(C.c_int32 * 3)(24, 20, 19)), 1), (dict(sec=(C.c_int32 * 3)(65, -1, 0)), 1),
    (dict(theta=0.0), 1), (dict(theta=float("inf")), 1), (dict(theta=float("nan")), 1),
    (dict(gq=P, eps=-1.0), 1), (dict(gq=P, eps=float("nan")), 1), (dict(c=cache(d=127)), 1),
    (dict(strides=(2047, 1024, 1024, 2048)), 1), (dict(strides=(2048, 1023, 1024, 2048)), 1),
    (dict(strides=(2048, 1024, 0, 2048)), 1), (dict(strides=(2048, 1024, 1024, -1)), 1),
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(out=None), 1), (dict(pos=None), 1),
    (dict(out=P, strides=(4096, 1024, 1024, 2048)), 1),
    (dict(tokens=0, q=None, k=None, v=None, out=None, pos=None), 0),
    (dict(b=batch(None, None, None, 0, 0)), 0),
])
def test_append_arguments(L, kw, status):
    before = L.arops_launch_count()
    assert append(L, **kw) == status, L.arops_last_error()
    assert L.arops_launch_count() == before


def test_append_null_structs(L):
    f = L.arops_mrope_paged_append
    tail = (None, None, 1e-6, P, 2, 16, SEC, 1e6, None)
    assert f(P, 2048, P, 1024, P, 1024, P, 2048, None, batch(), *tail) == 1
    assert f(P, 2048, P, 1024, P, 1024, P, 2048, cache(), None, *tail) == 1


ATTENTION_ARGUMENTS = [
    (dict(o=options(scale=float("nan"))), 1), (dict(o=options(scale=float("inf"))), 1),
    (dict(o=options(cap=-1.0)), 1), (dict(o=options(cap=float("inf"))), 1), (dict(o=options(window=-1)), 1),
    (dict(hq=15), 1), (dict(hq=0), 1), (dict(hq=-8), 1), (dict(c=cache(heads=0)), 1),
    (dict(c=cache(d=257), stride=1 << 20), 2), (dict(c=cache(d=129, dtype=0), stride=1 << 20), 2),
    (dict(stride=2047), 1), (dict(q=None), 1), (dict(out=None), 1), (dict(out=P), 1),
    (dict(ws=None), 1), (dict(ws=24), 1), (dict(ws_bytes=1000), 1), (dict(b=batch(n=65536)), 2),
]


@pytest.mark.parametrize("kw,status", ATTENTION_ARGUMENTS)
@pytest.mark.parametrize("op", [attend, shared])
def test_attention_arguments(L, op, kw, status):
    before = L.arops_launch_count()
    assert op(L, **kw) == status, L.arops_last_error()
    assert L.arops_launch_count() == before


def test_attention_only(L):
    before = L.arops_launch_count()
    assert attend(L, b=batch(start=None)) == 1
    assert attend(L, tokens=-1) == 1
    assert attend(L, tokens=1 << 31) == 2
    assert attend(L, tokens=0, q=None, out=None, ws=None, ws_bytes=0) == 0
    assert attend(L, b=batch(None, None, None, 0, 0), q=None, out=None, ws=None, ws_bytes=0) == 0
    assert L.arops_paged_attention(P, 2048, 2 * P, cache(), batch(), None, 2, 16, 16, 1 << 40, None) == 1
    assert L.arops_launch_count() == before


def test_shared_only(L):
    before = L.arops_launch_count()
    for g in (groups(n=-1), groups(max_pages=-1), groups(start=None), groups(lens=None), groups(table=None),
              groups(n=3)):
        assert shared(L, g=g) == 1, L.arops_last_error()
    assert shared(L, g=groups(max_pages=1 << 27), b=batch(max_pages=1 << 20)) == 2
    assert shared(L, o=options(bidir=P)) == 1
    assert shared(L, g=groups(None, None, None, 0, 0), q=None, out=None, ws=None, ws_bytes=0) == 0
    assert L.arops_shared_prefix_attention(P, 2048, 2 * P, cache(), batch(), None, options(), 16, 16, 1 << 40,
                                           None) == 1
    assert L.arops_launch_count() == before


def test_workspace_sizes(L):
    n = C.c_size_t(0)
    f = L.arops_attention_workspace
    assert f(5, 16, 128, C.byref(n)) == 0 and n.value >= 16384
    small = n.value
    assert f(4096, 16, 128, C.byref(n)) == 0 and n.value >= small
    assert f(0, 16, 128, C.byref(n)) == 0
    assert f(5, 16, 128, None) == 1
    assert f(-1, 16, 128, C.byref(n)) == 1 and f(5, 0, 128, C.byref(n)) == 1 and f(5, 16, 0, C.byref(n)) == 1
    assert f(1 << 31, 16, 128, C.byref(n)) == 2 and f(5, 16, 512, C.byref(n)) == 2
    assert L.arops_attention_prepare(None, 1 << 20, None) == 1
    assert L.arops_attention_prepare(16, 1000, None) == 1
    assert L.arops_attention_prepare(8, 1 << 20, None) == 1


def test_binding_rejects_wrong_tensors():
    q = torch.zeros(2, 16, 128, dtype=torch.bfloat16)
    kv = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    pool = torch.zeros(4, 8, 16, 128, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        ops.mrope_paged_append(q, kv, kv, i, i, i, i, pool, pool.clone())
    with pytest.raises(ValueError):
        ops.paged_attention(q, pool, pool.clone(), i, i[:2], torch.zeros(2, 1, dtype=torch.int32))
    with pytest.raises(ValueError):
        ops.shared_prefix_attention(q, pool, pool.clone(), i, i[:2], torch.zeros(2, 1, dtype=torch.int32),
                                    i[:2], torch.zeros(2, 1, dtype=torch.int32))


@pytest.mark.parametrize("t", [
    torch.zeros(2, 16, 256)[:, :, ::2], torch.zeros(2, 32, 128)[:, ::2], torch.zeros(1, 16, 128).expand(2, 16, 128),
    torch.zeros(2, 16 * 128),
])
def test_binding_rejects_strides(t):
    with pytest.raises(ValueError):
        ops._token_stride("q", t)


def test_binding_token_strides():
    assert ops._token_stride("q", torch.zeros(3, 16, 128)) == 2048
    assert ops._token_stride("q", torch.zeros(3, 5000)[:, :2048].unflatten(1, (16, 128))) == 5000
    assert ops._token_stride("q", torch.zeros(1, 16, 128).expand(1, 16, 128)) == 2048


def test_packed_structures_have_the_layout_of_the_structures():
    for make, cls, values in (
            (ops._pack_cache, _PagedCache, (P, 2 * P, 10, 16, 8, 128, 1)),
            (ops._pack_batch, _PagedBatch, (P, 0, 3 * P, 7, 4)),
            (ops._pack_options, _AttentionOptions, (0.5, 20.0, 300, P, 0)),
            (ops._pack_groups, _PrefixGroups, (P, 2 * P, 3 * P, 5, 6))):
        expected = cls(*[v or None if n in ("kv_lens", "bidir_lens") else v
                         for v, (n, _) in zip(values, cls._fields_)])
        assert len(make(*values)) == C.sizeof(cls)
        back = cls.from_buffer_copy(make(*values))
        for name, _ in cls._fields_:
            assert getattr(back, name) == getattr(expected, name)
