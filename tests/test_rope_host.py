"""kvq_norm_rope and kvq_rope_append refuse bad arguments before any CUDA call
(the addresses here are never touched)."""
import ctypes
import math
import os
import subprocess
import sys

import pytest
import torch

from quantized_kv_cache_05_gb300 import build as kbuild
from quantized_kv_cache_05_gb300 import kvq, runtime

P = 1 << 20   # an aligned address that nothing dereferences
OK, INV, UNS = kvq.KVQ_OK, kvq.KVQ_ERR_INVALID, kvq.KVQ_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def _lib():
    kbuild.build()
    kvq.lib()


def rotary(**kw):
    r = kvq.kvq_rotary(P, 1000, 128, 0, None, None, 1e-6)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def heads(n=8, ts=8 * 128, hs=128, p=P):
    return kvq.kvq_heads(p, ts, hs, n)


def norm_rope(r=None, dim=128, tokens=0, pos=P, q="d", qo="d", fp8=0, scale=1.0, k="d", ko="d"):
    d = lambda h: heads() if h == "d" else h
    return kvq.kvq_norm_rope(r or rotary(), dim, tokens, pos, d(q), d(qo), fp8, scale, None, d(k),
                             d(ko), None, 0)


def test_norm_rope_no_tokens_is_a_noop():
    assert norm_rope() == OK


@pytest.mark.parametrize("kw,want", [
    (dict(rot_dim=-2), INV), (dict(rot_dim=130), INV), (dict(rot_dim=256), INV),
    (dict(rot_dim=33), INV), (dict(rot_dim=48), UNS), (dict(rot_dim=16), UNS),
    (dict(interleaved=2), INV), (dict(cos_sin=None), INV), (dict(cos_sin=P + 4), INV),
    (dict(num_positions=0), INV), (dict(q_norm=P + 8), INV), (dict(k_norm=P + 4), INV),
    (dict(q_norm=P, eps=math.nan), INV), (dict(q_norm=P, eps=-1e-6), INV),
    (dict(k_norm=P, eps=math.inf), INV)])
def test_rotary_refused(kw, want):
    assert norm_rope(rotary(**kw)) == want
    assert append(r=rotary(**kw)) == want


@pytest.mark.parametrize("dim,want", [(0, INV), (-64, INV), (512, UNS), (192, UNS), (1024, UNS)])
def test_norm_rope_head_dim(dim, want):
    assert norm_rope(rotary(rot_dim=0, cos_sin=None), dim=dim) == want


BAD_ROWS = [
    (heads(p=None), INV), (heads(p=P + 8), INV), (heads(n=0), INV), (heads(ts=1028), INV),
    (heads(hs=132), INV), (heads(ts=-1024), INV), (heads(ts=1 << 31), UNS)]


@pytest.mark.parametrize("bad,want", BAD_ROWS)
def test_norm_rope_rows_refused(bad, want):
    for kw in (dict(q=bad), dict(qo=bad), dict(k=bad), dict(ko=bad)):
        assert norm_rope(tokens=4, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=None, k=None), INV), (dict(tokens=-1), INV), (dict(pos=None), INV),
    (dict(qo=None), INV), (dict(ko=None), INV), (dict(qo=heads(n=7)), INV),
    (dict(ko=heads(n=9, ts=9 * 128)), INV), (dict(fp8=2), INV), (dict(fp8=1, scale=0.0), INV),
    (dict(fp8=1, scale=math.inf), INV), (dict(tokens=1 << 28), UNS),
    # outputs that overlap themselves
    (dict(qo=heads(ts=512)), INV), (dict(ko=heads(hs=64)), INV), (dict(qo=heads(ts=0)), INV)])
def test_norm_rope_refused(kw, want):
    assert norm_rope(**{"tokens": 4, **kw}) == want


def cache(**kw):
    c = kvq.kvq_cache(fmt=kvq.KVQ_FP8_E4M3, num_pages=8, page_size=16, num_kv_heads=8, head_dim=128,
                      k_codes=P, v_codes=P, k_scale=1.0, v_scale=1.0, block_table=P,
                      max_pages_per_seq=4)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def mla_cache():
    return kvq.kvq_cache(fmt=kvq.KVQ_NVFP4, num_pages=8, page_size=16, num_kv_heads=1, head_dim=512,
                         k_codes=P, k_bscale=P, k_scale=1.0, block_table=P, max_pages_per_seq=4,
                         rope_dim=64, k_pe=P, v_is_k_latent=1)


def append(c=None, r=None, batch=0, tokens=4, start=P, k="d", v="d", kpe=None, q=None, qo=None,
           fp8=0, scale=1.0):
    d = lambda h: heads() if h == "d" else h
    return kvq.kvq_rope_append(c or cache(), r or rotary(), batch, tokens, start, None, d(k), d(v),
                               d(kpe), d(q), d(qo), fp8, scale, None, None, 0)


def test_append_nothing_is_a_noop():
    assert append() == OK
    assert append(batch=3, tokens=0) == OK


@pytest.mark.parametrize("bad,want", BAD_ROWS)
def test_append_rows_refused(bad, want):
    for kw in (dict(k=bad), dict(v=bad), dict(q=bad, qo="d"), dict(q="d", qo=bad)):
        assert append(batch=2, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(batch=-1), INV), (dict(tokens=-1), INV), (dict(start=None), INV), (dict(k=None), INV),
    (dict(v=None), INV), (dict(kpe="d"), INV), (dict(k=heads(n=4)), INV), (dict(v=heads(n=4)), INV),
    (dict(q="d"), INV), (dict(q="d", qo=heads(n=4)), INV), (dict(q="d", qo="d", fp8=3), INV),
    (dict(q="d", qo="d", fp8=1, scale=-1.0), INV), (dict(batch=1 << 20, tokens=1 << 10), UNS),
    (dict(c=cache(head_dim=96)), UNS), (dict(c=cache(page_size=20)), INV),
    (dict(c=cache(k_scale=0.0)), INV), (dict(c=cache(block_table=None)), INV)])
def test_append_refused(kw, want):
    r = rotary(rot_dim=64)
    assert append(**{"batch": 2, "r": r, **kw}) == want


def test_append_mla_refused():
    r = rotary(rot_dim=64)
    lat, pe = heads(1, 512, 512), heads(1, 64, 64)
    base = dict(c=mla_cache(), r=r, batch=2, k=lat, v=None, kpe=pe)
    assert append(**{**base, "v": lat}) == INV
    assert append(**{**base, "kpe": None}) == INV
    assert append(**{**base, "q": "d", "qo": "d"}) == UNS
    assert append(**{**base, "r": rotary(rot_dim=128)}) == INV
    assert append(**{**base, "k": heads(2, 1024, 512)}) == INV
    c = mla_cache()
    c.head_dim = 256
    assert append(**{**base, "c": c}) == UNS


def test_struct_sizes():
    # the C structs' layout (LP64)
    assert ctypes.sizeof(kvq.kvq_rotary) == 48 and ctypes.sizeof(kvq.kvq_heads) == 32


@pytest.mark.parametrize("flag", [torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int64),
                                  torch.zeros(1)])
def test_error_flags_of_another_type_or_device_are_refused(flag):
    """Kernels write the flag: a tensor elsewhere is refused before any launch."""
    call, ro = runtime._calls(), kvq.kvq_rotary()
    with pytest.raises(ValueError, match="error_flag"):
        call.norm_rope(0, None, ctypes.addressof(ro), -1, -1, None, None, None, None, None, False, 1.0,
                       None, flag)
    c = kvq.kvq_cache()
    with pytest.raises(ValueError, match="error_flag"):
        call.rope_append(0, None, ctypes.addressof(c), 1, ctypes.addressof(ro), -1, -1, None, None, None,
                         None, None, None, None, False, 1.0, None, flag)
    p = kvq.kvq_decode_params()
    with pytest.raises(ValueError, match="error_flag"):
        call.decode_shared(0, None, ctypes.addressof(c), ctypes.addressof(p), 0, None, 1, None, None, None,
                           None, None, None, flag)


def test_a_rotary_keeps_its_tensors(monkeypatch):
    """Its struct holds their addresses: they cannot be replaced."""
    monkeypatch.setattr(runtime, "_here", lambda *a: None)      # host tensors do here
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    table, w, v = torch.zeros(10, 64), torch.ones(64), torch.ones(64)
    ro = runtime.Rotary(table, False, w, v)
    for name, t in (("table", table), ("q_norm", w), ("k_norm", v)):
        assert getattr(ro, name) is t
        with pytest.raises(AttributeError):
            setattr(ro, name, torch.zeros(20, 64))
        with pytest.raises(AttributeError):
            delattr(ro, name)
    assert ro.struct().cos_sin == table.data_ptr() and ro.struct().q_norm == w.data_ptr()
    assert runtime.Rotary(None).table is None


def test_a_refused_type_is_named_while_it_lives():
    """A type object that only the attribute's reader holds: it is still there when the
    refusal names it (freed memory is overwritten under this allocator)."""
    code = """
from quantized_kv_cache_05_gb300 import runtime

class Type:
    def __repr__(self):
        return "a type of its own"

class Flag:
    dtype = property(lambda self: Type())

try:
    runtime._calls().block_table(0, Flag(), 0)
except ValueError as e:
    assert "a type of its own" in str(e), e
    print("refused")
"""
    r = subprocess.run([sys.executable, "-c", code], env={**os.environ, "PYTHONMALLOC": "debug"},
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "refused" in r.stdout, (r.returncode, r.stderr[-500:])
