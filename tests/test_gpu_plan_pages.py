"""kvq_plan_step over a page index that is out of range: where it comes back, and where a
request takes it."""
import numpy as np
import pytest
import torch

from packed_ref import DEV, i32
from quantized_kv_cache_05_gb300 import build as kbuild
from quantized_kv_cache_05_gb300 import kvq
from test_gpu_plan import ALL, OnGpu, State

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    kbuild.build()
    kvq.lib()
    torch.cuda.init()
    torch.zeros(1, device=DEV)


@pytest.mark.parametrize("bad", [-1, 30, 2 ** 31 - 1])
def test_a_bad_page_that_comes_back(bad):
    """It is reported, goes on the stack as it is, and is reported again where it is taken:
    that request's tokens there have no slots, all else is as with any page."""
    s = State(3, 4, 16, 30, [10, 40, 0])
    s.bt[1, 2] = bad                    # of request 1's three pages the one on top, later
    g = OnGpu(s, 20)
    g.plan(g.lens, i32([0, ALL, 0]), error_flag=g.err)
    want = s.step([0, ALL, 0], 20)
    g.check(s, (*want[:4], kvq.KVQ_DEVERR_BAD_PAGE))
    assert int(g.free[int(g.count) - 1]) == bad
    g.err.zero_()
    g.plan(g.lens, i32([3, 0, 17]), error_flag=g.err)
    old, offs, slots, pos, _ = s.step([3, 0, 17], 20)
    slots[3:19] = -1                    # the first page of request 2
    g.check(s, (old, offs, slots, pos, kvq.KVQ_DEVERR_BAD_PAGE))
    assert int(slots[19]) >= 0 and (slots[:3] >= 0).all() and np.array_equal(pos[3:20], np.arange(17))


@pytest.mark.parametrize("outputs", [("slots", "positions"), ("slots",), ()])
def test_a_bad_page_that_is_taken(outputs):
    """It is reported whatever is asked for beside the block table."""
    s = State(2, 4, 16, 30, [10, 0])
    g = OnGpu(s, 20)
    g.free[s.count - 1] = 30
    p = kvq.kvq_page_plan.from_buffer_copy(g.plan._struct)
    for name in ("slots", "positions"):
        if name not in outputs:
            setattr(p, name, None)
    out = torch.zeros(2, dtype=torch.int32, device=DEV)
    p.seq_lens, p.add_lens, p.seq_lens_out = g.lens.data_ptr(), (add := i32([2, 5])).data_ptr(), out.data_ptr()
    p.free_count_out, p.error_flag = g.count.data_ptr(), g.err.data_ptr()
    kvq.check(kvq.kvq_plan_step(p), "kvq_plan_step")
    torch.cuda.synchronize()
    assert add.tolist() == [2, 5] and out.tolist() == [12, 5]
    assert int(g.err) == kvq.KVQ_DEVERR_BAD_PAGE and int(g.bt[1, 0]) == 30
