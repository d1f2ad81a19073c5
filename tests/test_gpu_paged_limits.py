"""Calls of the paged-cache operators at the limits of what they take, on the GPU."""
import pytest
import torch

import swiglu_ar_tts_b200 as ops
from gpu_util import Guarded
from paged_util import Batch, Groups
from test_gpu_paged_append import Case
from test_gpu_paged_attention import check, run, shared_check, shared_run

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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new,lens,d", [([1, 1], [9000, 30], 128), ([700, 60], [700, 5000], 128), ([333], [333], 64),
                                        ([90], [2000], 256)])
def test_the_workspace_of_one_operator_is_enough(new, lens, d, dtype):
    d = min(d, 128) if dtype == "f32" else d
    b = Batch(new, lens, 16, 8, d, 16, dtype, seed=103)
    size = ops.attention_workspace(b.tokens, 16, d, shared_prefix=False)
    ws = Guarded((size // 4,), torch.float32, fill=torch.zeros(size // 4))
    for _ in range(2):  # split lines, joined: the counters are zero again
        check(b, run(b, workspace=ws.t), "its own workspace")
    ws.check()
    with pytest.raises(ops.ArOpsError):
        run(b, workspace=ws.t[:-4])


def test_a_shared_prefix_needs_the_larger_workspace():
    b = Groups([300], [4000], [20] * 300, 16, 8, 128, 16, "bf16", seed=104)
    small, large = (ops.attention_workspace(300, 16, 128, shared_prefix=x) for x in (False, True))
    with pytest.raises(ops.ArOpsError):
        shared_run(b, workspace=torch.zeros(small, dtype=torch.uint8, device="cuda"))
    ws = Guarded((large // 4,), torch.float32, fill=torch.zeros(large // 4))
    shared_check(b, shared_run(b, workspace=ws.t), "the larger workspace")
    ws.check()
    shared_check(b, shared_run(b), "a workspace of the call's own")


def test_a_long_prompt_allocates_no_prefix_results():
    b = Batch([4096], [4096], 16, 8, 128, 16, "bf16", seed=105)
    q, kp, vp = (x.cuda() for x in (b.q, b.k_pages, b.v_pages))
    arrays, out = b.arrays(), torch.empty_like(b.q, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    ops.paged_attention(q, kp, vp, *arrays, out=out)
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() - before < 64 << 20
