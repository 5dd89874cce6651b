"""kvq_chunk_attention's choice of the probabilities' parts on the host."""
import pytest

from quantized_kv_cache_05_gb300 import build as kbuild
from quantized_kv_cache_05_gb300 import kvq
from test_plan_host import INV, OK, chunk, diff, params


@pytest.fixture(scope="module", autouse=True)
def _lib():
    kbuild.build()
    kvq.lib()


@pytest.mark.parametrize("v", [-1, 2, 7])
def test_prefix_p_f16_is_0_or_1(v):
    assert chunk(p=params(batch=0, prefix_p_f16=v)) == INV
    for d in (None, diff()):
        assert chunk(p=params(batch=0, prefix_p_f16=1), d=d) == OK
