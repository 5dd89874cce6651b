"""kvq_decode_shared and kvq_shared_splits on the host: refusals before any CUDA
call (the addresses are never touched) and the split rule."""
import math
import weakref

import pytest
import torch

from quantized_kv_cache_05_gb300 import build as kbuild
from quantized_kv_cache_05_gb300 import kvq, runtime

P = 1 << 20
OK, INV, UNS = kvq.KVQ_OK, kvq.KVQ_ERR_INVALID, kvq.KVQ_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def _lib():
    kbuild.build()
    kvq.lib()


def cache(**kw):
    c = kvq.kvq_cache(fmt=kvq.KVQ_FP8_E4M3, num_pages=64, page_size=16, num_kv_heads=2, head_dim=128,
                      k_codes=P, v_codes=P, k_scale=1.0, v_scale=1.0, block_table=P,
                      max_pages_per_seq=32)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def params(**kw):
    p = kvq.kvq_decode_params(batch=4, num_q_heads=8, qk_dim=128, v_dim=128, num_splits=2, seq_lens=P,
                              max_kv_len=512, sm_scale=0.1, out_dtype=kvq.KVQ_OUT_BF16, out_scale=1.0)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def call(c=None, p=None, prefix=256, table=None, sp=2, q=P, po=P, pl=P, cn=P, out=P):
    return kvq.kvq_decode_shared(c or cache(), p or params(), prefix, table, sp, q, po, pl, cn, out, 0)


def test_no_batch_is_a_noop():
    assert call(p=params(batch=0)) == OK


@pytest.mark.parametrize("kw,want", [
    (dict(prefix=-16), INV), (dict(prefix=250), INV), (dict(prefix=528), INV), (dict(sp=0), INV),
    (dict(sp=-1), INV), (dict(q=None), INV), (dict(q=P + 8), INV), (dict(po=None), INV),
    (dict(po=P + 16), INV), (dict(pl=None), INV), (dict(cn=None), INV), (dict(out=None), INV),
    (dict(p=params(num_splits=0)), INV), (dict(p=params(num_splits=63)), UNS),
    (dict(p=params(prob_scale=0.1)), UNS), (dict(p=params(num_q_heads=7)), INV),
    (dict(p=params(num_q_heads=34)), UNS), (dict(p=params(qk_dim=64)), INV),
    (dict(p=params(v_dim=64)), INV), (dict(p=params(max_kv_len=513)), INV),
    (dict(p=params(seq_lens=None)), INV), (dict(p=params(sm_scale=math.nan)), INV),
    (dict(p=params(q_fp8=1, q_scale=0.0)), INV), (dict(p=params(out_dtype=7)), INV),
    (dict(c=cache(head_dim=256, fmt=kvq.KVQ_NVFP4, k_bscale=P, v_bscale=P),
          p=params(qk_dim=256, v_dim=256)), UNS),
    (dict(c=cache(page_size=24)), INV), (dict(c=cache(v_codes=None)), INV),
    (dict(c=cache(num_kv_heads=70000, num_pages=1), p=params(num_q_heads=70000)), UNS)])
def test_refused(kw, want):
    assert call(**kw) == want


def test_mla_refused():
    c = kvq.kvq_cache(fmt=kvq.KVQ_NVFP4, num_pages=8, page_size=16, num_kv_heads=1, head_dim=512,
                      k_codes=P, k_bscale=P, k_scale=1.0, block_table=P, max_pages_per_seq=32,
                      rope_dim=64, k_pe=P, v_is_k_latent=1)
    assert call(c=c, p=params(num_q_heads=16, qk_dim=576, v_dim=512)) == UNS


def test_splits():
    f = kvq.kvq_shared_splits
    for batch in (1, 4, 31, 64, 200):
        for hkv, g in ((8, 4), (1, 16), (2, 7), (300, 1)):
            for prefix in (0, 16, 128, 1040, 32768):
                for own in (0, 1, 100, 5000):
                    st, sp, so = f(152, batch, hkv, g, prefix, own, 1)
                    assert st == OK and 1 <= so <= 16 and 1 <= sp
                    assert sp <= max(1, (prefix + 127) // 128) and sp + so <= 64
    # few own chunks: they fit beside the prefix (8 heads x splits CTAs, one per SM)
    sp, so = f(152, 16, 8, 4, 8192, 512, 1)[1:]
    assert 16 * 8 * so <= 2 * (152 - 8 * sp)
    assert f(152, 4, 8, 4, 1024, 60, 1)[1:] == (8, 1)      # one tile per split at most
    # nothing of its own: the prefix takes the whole GPU in one wave
    assert 8 * f(152, 8, 8, 4, 65536, 0, 1)[1] in range(128, 153)
    assert f(0, 4, 8, 4, 1024, 60, 1)[0] == INV and f(152, 4, 8, 0, 1024, 60, 1)[0] == INV
    assert f(152, 4, 8, 4, -1, 60, 1)[0] == INV and f(152, 4, 8, 4, 16, -1, 1)[0] == INV


@pytest.mark.parametrize("v", [-1, 2])
def test_prefix_p_f16_is_0_or_1(v):
    assert call(p=params(batch=0, prefix_p_f16=v)) == INV
    assert call(p=params(batch=0, prefix_p_f16=1)) == OK


def test_block_table_of_a_call():
    """The table as it is at the call: fewer rows, another type or strides, refused."""
    check = runtime._calls().block_table
    t = torch.zeros(3, 4, dtype=torch.int32)      # (device -1: host memory)
    for ok in ((t, 0), (t, 3), (t[:1], 1), (t[:0], 0), (torch.zeros(3, 1, dtype=torch.int32), 3)):
        check(-1, *ok)
    for bad in ((t, 4), (t[:2], 3), (t.long(), 0), (t.t(), 0), (t[:, :2], 0), (t[0], 0), (t[None], 0)):
        with pytest.raises(ValueError, match="block_table"):
            check(-1, *bad)
    with pytest.raises(ValueError, match="block_table"):
        check(0, t, 0)                            # of another device
    c = runtime.QuantizedKVCache("fp8", 8, 16, 2, 64, t, 1.0, 1.0, device="cpu")
    assert c.struct().max_pages_per_seq == 4
    c.block_table = t[:, :2].contiguous()         # a narrower table: its own width
    assert c.max_pages_per_seq == 2 and c.struct().max_pages_per_seq == 2


def test_a_shared_decode_keeps_what_it_is_made_with(monkeypatch):
    """Its parameters hold addresses, its scratch a size: neither can be replaced."""
    monkeypatch.setattr(runtime, "_here", lambda *a: None)      # host tensors do here
    c = runtime.QuantizedKVCache("fp8", 8, 16, 2, 64, torch.zeros(3, 4, dtype=torch.int32), 1.0, 1.0,
                                 device="cpu")
    scale, table = torch.ones(4), torch.zeros(2, dtype=torch.int32)
    plan = runtime.SharedDecode(c, 3, 4, 32, 64, 0.1, q_fp8=True, q_head_scale=scale, prefix_table=table,
                                splits=(1, 1))
    assert plan.cache is c and plan.prefix_table is table and plan.prefix_len == 32
    for name in ("cache", "prefix_len", "prefix_table", "prefix_splits", "ws", "cfg"):
        with pytest.raises(AttributeError):
            setattr(plan, name, getattr(plan, name))
    address, kept = scale.data_ptr(), weakref.ref(scale)
    plan.cfg.q_head_scale = None                                # a copy's
    del scale
    assert kept() is plan.cfg.q_head_scale and plan._params.q_head_scale == address


def host_cache(rows=3, **kw):
    """A cache in host memory, for what is refused before any CUDA call."""
    args = dict(fmt="fp8", num_pages=8, page_size=16, num_kv_heads=2, head_dim=64, k_scale=1.0, v_scale=1.0,
                block_table=torch.zeros(rows, 4, dtype=torch.int32), device="cpu")
    return runtime.QuantizedKVCache(**{**args, **kw})


@pytest.mark.parametrize("splits", [(0, 1), (1, 0), (-1, 8), (8, -1), (-7, 8)])
@pytest.mark.parametrize("prefix", [0, 32])
def test_splits_below_one_are_refused(splits, prefix):
    """The scratch holds the sum of both: one below zero would make it too small."""
    with pytest.raises(ValueError, match="splits"):
        runtime.SharedDecode(host_cache(), 3, 4, prefix, 64, 0.1, splits=splits)


def test_tensors_of_another_device_than_the_cache_are_refused():
    """Whatever device is current when the object is made."""
    c = host_cache()
    away = [dict(prefix_table=torch.zeros(2, dtype=torch.int32, device="meta")),
            dict(q_fp8=True, q_head_scale=torch.ones(4, device="meta"))]
    for kw in away:
        with pytest.raises(ValueError, match="expected .* on cpu"):
            runtime.SharedDecode(c, 3, 4, 32, 64, 0.1, splits=(1, 1), **kw)
    runtime.SharedDecode(c, 3, 4, 32, 64, 0.1, splits=(1, 1), q_fp8=True, q_head_scale=torch.ones(4),
                         prefix_table=torch.zeros(2, dtype=torch.int32))


def test_refused_at_the_making():
    """What no step of the object could do raises before its scratch is made."""
    def make(c, hq=4, prefix=32, cap=64, splits=(1, 1), **kw):
        return runtime.SharedDecode(c, 3, hq, prefix, cap, 0.1, splits=splits, **kw)

    mla = host_cache(fmt="nvfp4", num_kv_heads=1, head_dim=512, rope_dim=64)
    wide = host_cache(fmt="nvfp4", head_dim=256)
    for want, kw in ((UNS, dict(c=mla, hq=16)), (UNS, dict(c=wide)), (INV, dict(c=host_cache(), prefix=24)),
                     (UNS, dict(c=host_cache(), hq=34)), (INV, dict(c=host_cache(), cap=80)),
                     (UNS, dict(c=host_cache(), splits=(1, 64))), (UNS, dict(c=host_cache(), splits=(1, 65))),
                     (INV, dict(c=host_cache(k_scale=0.0))), (INV, dict(c=host_cache(), q_fp8=True, q_scale=0.0)),
                     (INV, dict(c=host_cache(), out="e4m3", out_scale=0.0))):
        with pytest.raises(kvq.KvqError) as e:
            make(**kw)
        assert e.value.status == want, kw
    # more prefix splits than tiles are lowered, and the scratch holds what is left
    assert make(host_cache(), splits=(200, 63)).ws.part_lse.numel() == 3 * 4 * 64


def test_prefixes_next_to_2_to_the_31_are_refused():
    """Token numbers past the prefix's last tile have to fit 32 bits."""
    c = cache(max_pages_per_seq=1 << 27)
    for prefix, want in ((2 ** 31 - 16, UNS), (2 ** 31 - 4096, UNS), (2 ** 31 - 4112, OK)):
        p = params(batch=0 if want == OK else 4, max_kv_len=prefix)
        assert call(c=c, p=p, prefix=prefix) == want


def test_no_requests_and_an_empty_table():
    """A step of no requests does nothing, so nothing of it is refused."""
    plan = runtime.SharedDecode(host_cache(rows=0), 0, 4, 32, 64, 0.1, splits=(1, 1))
    assert plan.ws.out.shape == (0, 4, 64)


def test_prefix_p_f16_is_nothing_to_the_other_calls():
    """They neither read nor check it."""
    p = params(batch=0, prefix_p_f16=7)
    assert kvq.kvq_decode(cache(), p, P, P, P, P, P, 0) == OK
    assert kvq.kvq_decode_partial(cache(), p, P, P, P, 0) == OK
