"""The packed step's and the differential heads' calls on the host: refusals before any
CUDA call (the addresses are never touched)."""
import ctypes
import math

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


def mla_cache():
    return kvq.kvq_cache(fmt=kvq.KVQ_NVFP4, num_pages=8, page_size=16, num_kv_heads=1, head_dim=512,
                         k_codes=P, k_bscale=P, k_scale=1.0, block_table=P, max_pages_per_seq=32,
                         rope_dim=64, k_pe=P, v_is_k_latent=1)


def params(**kw):
    p = kvq.kvq_decode_params(batch=4, num_q_heads=8, qk_dim=128, v_dim=128, num_splits=2, seq_lens=P,
                              max_kv_len=512, sm_scale=0.1, out_dtype=kvq.KVQ_OUT_BF16, out_scale=1.0)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def diff(**kw):
    d = kvq.kvq_diff(lambda_=P, norm=P, eps=1e-5, gain=0.5)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def test_struct_sizes():
    assert ctypes.sizeof(kvq.kvq_page_plan) == 128 and ctypes.sizeof(kvq.kvq_diff) == 24


# ------------------------------------------------------------------------- plan
def plan(**kw):
    p = kvq.kvq_page_plan(batch=4, page_size=16, num_pages=64, max_pages_per_seq=8, max_tokens=64)
    for name in ("block_table", "seq_lens", "seq_lens_out", "add_lens", "free_pages", "free_count",
                 "free_count_out", "counter", "start_pos", "q_offsets", "slots", "positions"):
        setattr(p, name, P)
    for k, v in kw.items():
        setattr(p, k, v)
    return kvq.kvq_plan_step(p, 0)


@pytest.mark.parametrize("kw,want", [
    (dict(batch=-1), INV), (dict(page_size=0), INV), (dict(num_pages=0), INV),
    (dict(max_pages_per_seq=0), INV), (dict(max_tokens=-1), INV), (dict(block_table=None), INV),
    (dict(seq_lens=None), INV), (dict(seq_lens_out=None), INV), (dict(add_lens=None), INV),
    (dict(free_pages=None), INV), (dict(free_count=None), INV), (dict(free_count_out=None), INV),
    (dict(counter=None), INV), (dict(batch=8193), UNS),
    (dict(max_pages_per_seq=1 << 27), UNS), (dict(max_tokens=(1 << 30) + 1), UNS),
    (dict(num_pages=(1 << 30) + 1), UNS)])
def test_plan_refused(kw, want):
    assert plan(**kw) == want


# ------------------------------------------------------------------------ slots
def heads(n=2, ts=1024, hs=128, data=P):
    return kvq.kvq_heads(data=data, token_stride=ts, head_stride=hs, num_heads=n)


def slots(c=None, r=None, tokens=4, pos=P, slot=P, k="d", v="d", kpe=None, q=None, qo=None, fp8=0,
          scale=1.0):
    d = lambda h: heads() if h == "d" else h
    r = r or kvq.kvq_rotary(cos_sin=P, num_positions=100, rot_dim=64, eps=1e-6)
    return kvq.kvq_rope_append_slots(c or cache(), r, tokens, pos, slot, d(k), d(v), d(kpe), d(q), d(qo),
                                     fp8, scale, None, None, 0)


def test_no_tokens_are_a_noop():
    assert slots(tokens=0) == OK


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), INV), (dict(slot=None), INV), (dict(pos=None), INV), (dict(k=None), INV),
    (dict(v=None), INV), (dict(kpe="d"), INV), (dict(k=heads(4)), INV), (dict(v=heads(4)), INV),
    (dict(k=heads(data=P + 8)), INV), (dict(k=heads(ts=1025)), INV), (dict(q="d"), INV),
    (dict(q="d", qo=heads(4)), INV), (dict(q="d", qo="d", fp8=2), INV),
    (dict(q="d", qo="d", fp8=1, scale=0.0), INV), (dict(c=cache(head_dim=96)), UNS),
    (dict(c=mla_cache()), INV), (dict(tokens=1 << 30), UNS)])
def test_slots_refused(kw, want):
    assert slots(**kw) == want


# -------------------------------------------------------- attention of the step
def chunk(c=None, p=None, d=None, tokens=7, offs=P, q=P, ws=P, size=1 << 40, out=P):
    return kvq.kvq_chunk_attention(c or cache(), p or params(), d, tokens, offs, q, ws, size, out, 0)


def decode(c=None, p=None, d="d", q=P, po=P, pl=P, cn=P, out=P):
    return kvq.kvq_decode_diff(c or cache(), p or params(), diff() if d == "d" else d, q, po, pl, cn, out, 0)


def test_nothing_is_a_noop():
    assert chunk(tokens=0) == OK and chunk(p=params(batch=0)) == OK and chunk(d=diff(), tokens=0) == OK
    assert decode(p=params(batch=0)) == OK


BOTH = [(dict(p=params(prob_scale=0.1)), UNS), (dict(p=params(num_q_heads=7)), INV),
        (dict(p=params(qk_dim=64)), INV), (dict(p=params(v_dim=64)), INV),
        (dict(p=params(max_kv_len=513)), INV), (dict(p=params(seq_lens=None)), INV),
        (dict(p=params(sm_scale=math.nan)), INV), (dict(p=params(q_fp8=1, q_scale=0.0)), INV),
        (dict(p=params(out_dtype=7)), INV), (dict(c=cache(page_size=24)), INV),
        (dict(c=cache(v_codes=None)), INV), (dict(c=cache(head_dim=96), p=params(qk_dim=96, v_dim=96)), UNS),
        (dict(c=cache(head_dim=256), p=params(qk_dim=256, v_dim=256)), UNS),
        (dict(c=mla_cache(), p=params(num_q_heads=16, qk_dim=576, v_dim=512)), UNS),
        (dict(d=diff(lambda_=None)), INV), (dict(d=diff(norm=P + 4)), INV), (dict(d=diff(eps=-1.0)), INV),
        (dict(d=diff(eps=math.nan)), INV), (dict(d=diff(gain=math.inf)), INV)]


@pytest.mark.parametrize("kw,want", BOTH + [
    (dict(tokens=-1), INV), (dict(offs=None), INV), (dict(q=None), INV), (dict(q=P + 8), INV),
    (dict(out=None), INV), (dict(out=P + 16), INV), (dict(ws=None), INV), (dict(ws=P + 16), INV),
    (dict(tokens=1 << 30), UNS), (dict(p=params(batch=8193)), UNS),
    (dict(c=cache(head_dim=256, fmt=kvq.KVQ_NVFP4, k_bscale=P, v_bscale=P),
          p=params(qk_dim=256, v_dim=256)), UNS)])
def test_chunk_refused(kw, want):
    assert chunk(**kw) == want


@pytest.mark.parametrize("kw,want", BOTH + [
    (dict(d=None), INV), (dict(q=None), INV), (dict(q=P + 8), INV), (dict(po=None), INV), (dict(pl=None), INV),
    (dict(cn=None), INV), (dict(out=None), INV), (dict(p=params(num_splits=0)), INV),
    (dict(p=params(num_splits=65)), UNS), (dict(p=params(num_q_heads=18)), UNS),
    (dict(p=params(num_q_heads=0x7ffffffe)), UNS)])
def test_decode_refused(kw, want):
    assert decode(**kw) == want


def test_norm_options_are_read_with_a_norm_alone():
    assert chunk(d=diff(norm=None, eps=-1.0), tokens=0) == OK


def test_workspace_bytes():
    f = lambda sms=152, c=None, d=None, **kw: kvq.kvq_chunk_workspace_bytes(sms, c or cache(), params(**kw), d)
    assert f(0) == 0 and f(batch=-1) == 0 and f(num_q_heads=0) == 0 and f(max_kv_len=-1) == 0
    assert kvq.kvq_chunk_workspace_bytes(152, None, params(), None) == 0
    base = 152 * 2 * 256 * 129 * 4
    assert f(batch=0) == f(batch=1) >= base
    # the decode's counters and partials: 4 x 2 groups of 4 rows (8 differential ones)
    one = f(batch=4, max_kv_len=512)
    assert one > f(batch=1) + 4 * 8 * 129 * 4 and f(batch=4, max_kv_len=512, d=diff()) > one
    # rows that the decode does not take
    assert f(batch=4, num_q_heads=34) < one


# ---------------------------------------------------------------------- binding
@pytest.mark.parametrize("flag", [torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int64),
                                  torch.zeros(1)])
def test_error_flags_of_another_type_or_device_are_refused(flag):
    """Kernels write the flag: a tensor elsewhere is refused before any launch."""
    call = runtime._calls()
    a = ctypes.addressof
    ro, c, pl, dp, d = kvq.kvq_rotary(), kvq.kvq_cache(), kvq.kvq_page_plan(), kvq.kvq_decode_params(), diff()
    for name, args in (("plan_step", (0, None, a(pl), None, None, None, None)),
                       ("append_slots", (0, None, a(c), a(ro), -1, -1, None, None, None, None, None, None,
                                         None, False, 1.0, None)),
                       ("decode_diff", (0, None, a(c), a(dp), a(d), None, None, None, None, None, None)),
                       ("chunk_attention", (0, None, a(c), a(dp), 0, None, None, None, None, 0, None,
                                            torch.float32))):
        with pytest.raises(ValueError, match="error_flag"):
            getattr(call, name)(*args, flag)
        with pytest.raises(TypeError):
            getattr(call, name)(*args)


def test_objects_keep_what_their_structs_hold(monkeypatch):
    monkeypatch.setattr(runtime, "_here", lambda *a: None)      # host tensors do here
    lam, w = torch.zeros(4), torch.ones(64)
    d = runtime.Differential(lam, w)
    free, count = torch.arange(8, dtype=torch.int32), torch.tensor([8], dtype=torch.int32)
    pool = runtime.PagePool.wrap(free, count)
    bt = torch.zeros(2, 3, dtype=torch.int32)
    plan = runtime.StepPlan(bt, 16, pool, 10)
    for o, names in ((d, ("lam", "norm")), (pool, ("free", "count", "counter")),
                     (plan, ("block_table", "pool", "start_pos", "q_offsets", "slots", "positions"))):
        for n in names:
            with pytest.raises(AttributeError):
                setattr(o, n, torch.zeros(1))
    assert plan.slots.dtype == torch.int64 and plan.q_offsets.numel() == 3 and plan.slots.numel() == 10
    with pytest.raises(ValueError):
        runtime.StepPlan(bt.t(), 16, pool, 10)
    with pytest.raises(ValueError):
        runtime.StepPlan(bt.long(), 16, pool, 10)
    with pytest.raises(ValueError):
        runtime.StepPlan(bt, 16, pool, -1)
