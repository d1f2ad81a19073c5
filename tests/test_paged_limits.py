"""Numbers that the paged-cache binding must not change on their way to the
library (no GPU needed)."""
import ctypes

import pytest

import swiglu_ar_tts_b200 as ops


@pytest.mark.parametrize("cap", [1e-50, -1e-50, 1e-46, 5e-324, 2.0 ** -150])
def test_a_cap_that_vanishes_as_a_float_is_refused(cap):
    """1e-50 must not come out as 0, which is no cap at all."""
    with pytest.raises(ValueError):
        ops._options(0.1, cap, 0, 0, 0)


def test_caps_that_a_float_holds():
    for cap in (0.0, 0, -0.0):
        assert ops._options(0.1, cap, 0, 0, 0) == ops._pack_options(0.1, cap, 0, 0, 0)
    # these are the library's to refuse or to take
    for cap in (2.0 ** -149, 1e-30, 30, 30.0, 3e38, -1.0, float("nan"), float("inf")):
        assert ops._options(0.1, cap, 5, 8, 16) == ops._pack_options(0.1, cap, 5, 8, 16)


@pytest.mark.parametrize("sizes", [(2 ** 64 + 5, 16, 128), (5, 2 ** 32 + 16, 128), (5, 16, 2 ** 32 + 128),
                                   (-(2 ** 63) - 1, 16, 128), (5.5, 16, 128)])
def test_workspace_sizes_that_a_field_cannot_hold(sizes):
    """2^32 + 16 heads must not come out as the workspace of 16."""
    with pytest.raises(ValueError):
        ops.attention_workspace(*sizes)
    assert ops.attention_workspace(5, 16, 128) > 0


@pytest.mark.parametrize("sections", [(2 ** 32 + 24, 20, 20), (24, 20, 20 - 2 ** 32), (24, 40), (24, 20, 10, 10),
                                      (24.5, 20, 19)])
def test_sections_that_a_field_cannot_hold(sections):
    with pytest.raises(ValueError):
        ops._pack(ops._pack_sections, *sections)
    assert ops._pack(ops._pack_sections, 24, 20, 20) == bytes((ops._i32 * 3)(24, 20, 20))


@pytest.mark.parametrize("tokens,heads,d", [(0, 1, 1), (5, 16, 128), (16384, 16, 128), (2000, 12, 64), (300, 8, 256),
                                            (100_000, 16, 128)])
def test_workspace_of_one_operator(tokens, heads, d):
    """Attention without shared prefixes keeps nothing per token: a prompt of any
    length takes the same space."""
    both = ops.attention_workspace(tokens, heads, d)
    alone = ops.attention_workspace(tokens, heads, d, shared_prefix=False)
    width = 64 if d <= 64 else 128
    prefixes = tokens * heads * (width + 2) * 4 if d <= 128 and tokens * heads >= 96 else 0
    assert both - alone == prefixes
    assert 16384 < alone < 64 << 20


def test_workspace_of_one_operator_refuses_as_the_other():
    n = ctypes.c_size_t(0)
    for f in (ops.lib().arops_attention_workspace, ops.lib().arops_paged_attention_workspace):
        assert f(5, 16, 128, None) == 1
        for bad in ((-1, 16, 128), (5, 0, 128), (5, 16, 0)):
            assert f(*bad, ctypes.byref(n)) == 1
        for bad in ((1 << 31, 16, 128), (5, 65536, 128), (5, 16, 257)):
            assert f(*bad, ctypes.byref(n)) == 2
