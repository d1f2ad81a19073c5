"""Calls of the paged-cache operators at the limits of what they take, on the GPU."""
import pytest
import torch

import swiglu_ar_tts_b200 as ops
from paged_util import Batch
from test_gpu_paged_append import Case
from test_gpu_paged_attention import run

pytestmark = pytest.mark.gpu


def test_a_cap_that_vanishes_as_a_float_launches_nothing():
    b = Batch([1], [20], 16, 8, 128, 16, "bf16", seed=101)
    before = ops.launch_count()
    for cap in (1e-50, 5e-324):
        with pytest.raises(ValueError):
            run(b, softcap=cap)
    assert ops.launch_count() == before


def test_sections_that_a_field_cannot_hold_launch_nothing():
    c = Case([3], [9], seed=102, sections=(2 ** 32 + 24, 20, 20))
    before = ops.launch_count()
    with pytest.raises(ValueError):
        c.run()
    assert ops.launch_count() == before
    c.sections = torch.tensor([24, 20, 20])  # whole numbers of any kind
    c.run()
    assert ops.launch_count() == before + 1
