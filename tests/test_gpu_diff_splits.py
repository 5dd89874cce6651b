"""The differential decode's own number of chunks."""
import pytest
import torch

from packed_ref import DEV, Packed
from quantized_kv_cache_05_gb300 import build as kbuild
from quantized_kv_cache_05_gb300 import kvq

pytestmark = pytest.mark.gpu


def test_eight_heads_of_one_kv_head_are_not_mla():
    """As many chunks with NVFP4 as with FP8: both have two CTAs on an SM."""
    kbuild.build()
    kvq.lib()
    torch.cuda.init()
    torch.zeros(1, device=DEV)
    made = [Packed(fmt, 64, 8, 1, 64, [(4999, 1)] * 16, diff=True) for fmt in ("fp8", "nvfp4")]
    objs = [X.decode("f32") for X in made]
    assert objs[0].cfg.num_splits == objs[1].cfg.num_splits
    for X, d in zip(made, objs):
        X.check(d(X.q, X.lens_t), "f32")
