"""kvq_decode_diff against the differential attention in 64 bits (bounds: packed_ref)."""
import numpy as np
import pytest
import torch

from packed_ref import DEV, Packed, i32
from quantized_kv_cache_05_gb300 import build as kbuild
from quantized_kv_cache_05_gb300 import kvq, runtime

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    kbuild.build()
    kvq.lib()
    torch.cuda.init()
    torch.zeros(1, device=DEV)


def one(lens):
    return [(n - 1, 1) for n in lens]


def run(X, out="f32", splits=None, **kw):
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    d = X.decode(out, splits, **kw)
    o = d(X.q, X.lens_t, error_flag=err).clone()
    torch.cuda.synchronize()
    assert int(err) == 0 and int(d._ws.counters.abs().sum()) == 0
    return o


@pytest.mark.parametrize("fmt,D", [("fp8", 64), ("fp8", 128), ("nvfp4", 64), ("nvfp4", 128), ("nvfp4", 256)])
@pytest.mark.parametrize("hq,hkv", [(4, 2), (3, 3), (8, 2), (5, 1), (8, 1), (14, 2)])
@pytest.mark.parametrize("norm", [False, True])
def test_shapes(fmt, D, hq, hkv, norm):
    X = Packed(fmt, D, hq, hkv, 16, one([1, 700, 16, 333, 129]), diff=True, norm=norm)
    ref = X.reference()
    for splits in (None, 1, 3, 64):
        X.check(run(X, "f32", splits), "f32", ref, what=f"splits {splits}")
    X.check(run(X, "bf16"), "bf16", ref)


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("out", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("q_fp8,head_scales", [(False, False), (True, False), (False, True), (True, True)])
def test_types(fmt, out, q_fp8, head_scales):
    for D, ps in ((64, 48), (128, 256)):
        X = Packed(fmt, D, 8, 2, ps, one([300, 1, 1000]), 3, q_fp8, head_scales, diff=True)
        X.check(run(X, out), out)


def test_query_head_scales():
    X = Packed("fp8", 128, 6, 2, 16, one([300, 50]), 3, True, diff=True)
    hs = torch.linspace(0.01, 0.02, 6, device=DEV)
    X.q64 = X.q.view(torch.float8_e4m3fn).double() * hs.double()[:, None]
    d = runtime.DiffDecode(X.cache, 2, 6, X.cap, X.sm, X.diff, out="f32", q_fp8=True, q_head_scale=hs)
    X.check(d(X.q, X.lens_t), "f32")


def test_empty_requests_and_rows_past_the_end():
    """Length 0 gives zeros, with a norm of eps 0 too; NaN codes past the end reach nothing."""
    for eps in (0.0, 1e-5):
        X = Packed("fp8", 128, 8, 2, 16, one([77, 40, 300]), diff=True, eps=eps)
        for b in (0, 2):
            for c in X.codes:
                c[int(X.bt[b, X.lens[b] // 16]), :, X.lens[b] % 16:] = 0x7F
        ref = X.reference()
        X.lens[1] = 0
        X.lens_t = i32(X.lens)
        o = run(X)
        X.check(o, "f32", ref, rows=[0, 2])
        assert (o[1] == 0).all()


def test_a_nan_stays_with_its_head():
    X = Packed("fp8", 128, 4, 2, 16, one([77, 40]), diff=True)
    ref = X.reference()
    X.codes[1][int(X.bt[0, 1]), 1, 3, 5] = 0x7F
    o = run(X)
    X.check(o[:, :2], "f32", tuple(r[:, :2] for r in ref))
    X.check(o[1:], "f32", tuple(r[1:] for r in ref))
    assert torch.isnan(o[0, 2:]).all()   # through the norm all of the head


def test_clamped_lengths_and_bad_pages():
    X = Packed("fp8", 64, 4, 2, 16, one([77, 160]), diff=True)
    d = X.decode("f32")
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    o = d(X.q, i32([77, 1 << 20]), error_flag=err).clone()
    assert int(err) == kvq.KVQ_DEVERR_SEQ_CLAMPED
    X.check(o, "f32")
    err.zero_()
    X.bt[0, 2] = -1
    o = d(X.q, X.lens_t, error_flag=err).clone()
    assert int(err) == kvq.KVQ_DEVERR_BAD_PAGE
    X.bt[0, 2] = 0
    X.check(o, "f32")


def test_behind_the_append():
    """fresh_tokens: the decode that starts while the append of the last rows runs."""
    X = Packed("fp8", 128, 8, 2, 16, one([500, 33]), diff=True)
    d = X.decode("f32", fresh_tokens=1)
    k, v = (torch.randn(2, 1, 2, 128, generator=X.g, device=DEV).bfloat16() for _ in range(2))
    start = X.lens_t - 1
    for _ in range(5):
        for c in X.codes:   # other rows at the last position
            for b in range(2):
                c[int(X.bt[b, (X.lens[b] - 1) // 16]), :, (X.lens[b] - 1) % 16] = 0x38
        X.cache.append(k, v, start)
        o = d(X.q, X.lens_t).clone()
    for x, c, s in zip(X.val, X.codes, (0.0137, 0.0119)):
        x.copy_(c.view(torch.float8_e4m3fn).double() * float(np.float32(s)))
    X.check(o, "f32")


def test_agrees_with_the_chunk():
    X = Packed("nvfp4", 128, 8, 2, 16, one([1500, 7, 640]), diff=True)
    ref = X.reference()
    X.check(run(X), "f32", ref)
    X.check(X.run("f32"), "f32", ref)


def test_streams_and_graphs():
    X = Packed("nvfp4", 128, 8, 2, 16, one([1500, 7, 640]), diff=True)
    ref = X.reference()
    d = X.decode("f32")
    first = d(X.q, X.lens_t).clone()
    X.check(first, "f32", ref)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        d(X.q, X.lens_t, stream=s)
    s.synchronize()
    assert torch.equal(d(X.q, X.lens_t), first)
    g = torch.cuda.CUDAGraph()
    lens = X.lens_t.clone()
    with torch.cuda.graph(g):
        o = d(X.q, lens)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, first)
    lens.copy_(i32([1499, 1, 200]))
    g.replay()
    torch.cuda.synchronize()
    X.lens = [1499, 1, 200]
    X.check(o, "f32")


def test_refused():
    X = Packed("fp8", 128, 8, 2, 16, one([50, 40]), diff=True)
    d = X.decode("bf16")
    for args in ((X.q.float(), X.lens_t), (X.q[:1], X.lens_t), (X.q, X.lens_t.long()), (X.q, X.lens_t[:1]),
                 (X.q[:, :4], X.lens_t), (X.q.cpu(), X.lens_t)):
        with pytest.raises(ValueError):
            d(*args)
    make = lambda hq=8, diff=X.diff, **kw: runtime.DiffDecode(X.cache, 2, hq, X.cap, X.sm, diff, **kw)
    lam = lambda n: runtime.Differential(torch.ones(n, device=DEV))
    with pytest.raises(kvq.KvqError):   # nine heads per kv head
        make(18, lam(18))
    with pytest.raises(ValueError):
        make(8, lam(4))
    with pytest.raises(kvq.KvqError):
        make(splits=65)
    with pytest.raises(kvq.KvqError):
        make(diff=runtime.Differential(torch.ones(8, device=DEV), gain=float("inf")))
    with pytest.raises(ValueError):
        runtime.Differential(torch.ones(8, device=DEV).double())
