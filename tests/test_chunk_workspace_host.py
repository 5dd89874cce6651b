"""What kvq_chunk_attention's workspace holds for single tokens, on the host."""
import pytest

from quantized_kv_cache_05_gb300 import build as kbuild
from quantized_kv_cache_05_gb300 import kvq
from test_plan_host import cache, params


@pytest.fixture(scope="module", autouse=True)
def _lib():
    kbuild.build()
    kvq.lib()


@pytest.mark.parametrize("hkv", [1, 8])
def test_it_does_not_grow_with_the_longest_length(hkv):
    """A batch that fills the GPU anyway: four partials of a row at most, however long a
    request may become."""
    size = lambda batch, most: kvq.kvq_chunk_workspace_bytes(
        152, cache(num_kv_heads=hkv), params(batch=batch, num_q_heads=4 * hkv, max_kv_len=most), None)
    chunks = size(1, 1 << 17)
    for batch in (512, 8192):
        rows = batch * 4 * hkv
        assert size(batch, 1 << 17) <= chunks + 4 * rows * 129 * 4 + batch * (4 * hkv + 16) + 2048
    # one that does not: as many chunks as places, in all
    assert size(2, 1 << 17) <= chunks + 304 * 4 * 129 * 4 + 4096


def test_sixteen_rows_of_one_kv_head_are_not_mla():
    """The formats differ in nothing that the single tokens' partials depend on."""
    nv = dict(fmt=kvq.KVQ_NVFP4, k_bscale=1 << 20, v_bscale=1 << 20)
    size = lambda **kw: kvq.kvq_chunk_workspace_bytes(
        152, cache(num_kv_heads=1, **kw), params(batch=4, num_q_heads=16, max_kv_len=1 << 15), None)
    assert size(**nv) == size()
