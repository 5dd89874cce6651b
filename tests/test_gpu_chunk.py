"""kvq_chunk_attention, with plain and differential heads, against softmax attention in
64 bits over the dequantized cache (bounds: packed_ref)."""
import math

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


# (tokens before, new tokens): idle requests, single tokens, chunks at tile borders
MIXED = [(0, 1), (9, 0), (100, 1), (37, 50), (0, 200), (513, 3), (127, 1), (128, 128), (0, 0), (255, 2),
         (1000, 70), (0, 33)]


@pytest.mark.parametrize("diff", [False, True])
@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (3, 3), (14, 2), (20, 1)])
@pytest.mark.parametrize("ps", [16, 48, 256])
def test_mixed(diff, fmt, D, hq, hkv, ps):
    X = Packed(fmt, D, hq, hkv, ps, MIXED, diff=diff)
    ref = X.reference()
    for out in ("f32", "bf16"):
        X.check(X.run(out), out, ref, what=out)


@pytest.mark.parametrize("diff", [False, True])
@pytest.mark.parametrize("reqs", [[(0, 1)], [(15, 1)], [(0, 128)], [(0, 700)], [(3000, 1)], [(5000, 40)],
                                  [(2500, 513)], [(0, 2), (4000, 1)], [(17, 1)] * 130, [(0, 0), (0, 5)]])
def test_shapes(diff, reqs):
    """One token, one tile, several row tiles, long keys behind few rows (cut into many
    pieces), many single tokens."""
    for fmt, D, hq, hkv in (("fp8", 128, 8, 2), ("nvfp4", 64, 6, 2)):
        X = Packed(fmt, D, hq, hkv, 32, reqs, seed=len(reqs), diff=diff)
        ref = X.reference()
        for out in ("f32", "bf16"):
            X.check(X.run(out), out, ref, what=f"{fmt} {out}")


@pytest.mark.parametrize("diff", [False, True])
def test_many_requests(diff):
    """More requests, and more row tiles, than the shares' kernel has threads."""
    reqs = [((37 * b) % 90, [0, 1, 2, 5, 40][b % 5]) for b in range(700)]
    X = Packed("fp8", 64, 8, 4, 16, reqs, diff=diff)
    X.check(X.run("bf16"), "bf16")


@pytest.mark.parametrize("hq", [17, 130, 300])
def test_many_heads_of_one_kv_head(hq):
    """Groups larger than the decode takes, than an accumulator's rows, than a row tile."""
    X = Packed("nvfp4", 64, hq, 1, 16, [(200, 1), (30, 3), (0, 2), (500, 1)])
    X.check(X.run("f32"), "f32")


@pytest.mark.parametrize("diff", [False, True])
@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("out", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("q_fp8,head_scales", [(False, False), (True, False), (False, True), (True, True)])
def test_types(diff, fmt, out, q_fp8, head_scales):
    for D in (64, 128):
        X = Packed(fmt, D, 8, 2, 16, [(300, 1), (40, 60), (0, 7)], 3, q_fp8, head_scales, diff=diff)
        X.check(X.run(out), out, what=str(D))


def test_query_head_scales_and_signs():
    """Per-query-head scales, one below zero and one of zero among them."""
    for diff in (False, True):
        X = Packed("fp8", 128, 4, 2, 16, [(300, 1), (40, 60)], 3, True, diff=diff)
        hs = torch.tensor([0.017, -0.011, 0.0, 0.02], device=DEV)
        X.q64 = X.q.view(torch.float8_e4m3fn).double() * hs.double()[:, None]
        att = runtime.ChunkAttention(X.cache, X.B, 4, X.cap, X.sm, out="f32", q_fp8=True, q_head_scale=hs,
                                     diff=X.diff)
        X.check(att(X.q, X.offs_t, X.lens_t), "f32")


@pytest.mark.parametrize("norm", [False, True])
def test_differential_options(norm):
    for gain, eps in ((1.0, 0.0), (-0.7, 1e-3)):
        X = Packed("fp8", 128, 8, 4, 16, [(700, 1), (90, 130), (0, 5)], 4, diff=True, norm=norm, gain=gain, eps=eps)
        X.check(X.run("f32"), "f32")


def test_equal_maps_cancel():
    """Both maps the same and lambda 1: nothing is left, with a norm too."""
    X = Packed("fp8", 128, 4, 2, 16, [(700, 1), (90, 130)], 4, diff=True, norm=False)
    for c, v in ((X.codes[0], X.val[0]),):
        c[..., 64:] = c[..., :64]
        v[..., 64:] = v[..., :64]
    X.q[..., 64:] = X.q[..., :64]
    X.q64 = X.q.double()
    X.diff.lam.fill_(1.0)
    o, tol, _ = X.reference()
    got = X.run("f32").double().cpu().numpy()
    assert (np.abs(got) <= tol).all()


def test_rows_before_the_first_position_and_empty_requests():
    """More new rows than tokens: those before position 0 see nothing and give zeros, with
    a norm of eps 0 too; a request without tokens gives zeros."""
    for diff in (False, True):
        X = Packed("fp8", 128, 8, 2, 16, [(60, 5), (0, 40), (100, 150)], diff=diff, eps=0.0)
        X.lens = [65, 13, 0]
        X.lens_t = i32(X.lens)
        ref = X.reference()
        for out in ("f32", "bf16"):
            o = X.run(out)
            X.check(o, out, ref)
            assert (o[5:5 + 27] == 0).all() and (o[45:] == 0).all() and (o[32:45] != 0).any()


def test_rows_that_are_nobodys_stay():
    """Rows of out before the first offset, in gaps and past the last offset."""
    X = Packed("fp8", 64, 4, 2, 16, [(60, 5), (30, 20), (0, 1)])
    ref = X.reference()
    pad = lambda t, n: torch.cat([t.new_full((n, *t.shape[1:]), 99), t])
    q = torch.cat([pad(X.q[:25], 3), pad(X.q[25:], 0), X.q[:4]])
    out = torch.full(q.shape, 7.0, device=DEV)
    # request 1's rows follow request 0's, rows 0..2 and 29.. belong to nobody
    X.chunk("f32")(q, X.offs_t + 3, X.lens_t, out=out)
    X.check(out[3:29], "f32", ref)
    assert (out[:3] == 7).all() and (out[29:] == 7).all()


def test_offsets_and_lengths_out_of_range():
    """Offsets past the rows are cut, falling ones are no tokens, lengths are clamped."""
    X = Packed("fp8", 64, 4, 2, 16, [(60, 5), (30, 20), (40, 2)])
    ref = X.reference()
    out = torch.full(X.q.shape, 7.0, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    X.chunk("f32")(X.q, i32([0, 5, 2, 1 << 30]), X.lens_t, out=out, error_flag=err)
    assert int(err) == 0
    X.check(out, "f32", ref, rows=slice(0, 2))
    assert torch.isfinite(out).all()
    out.fill_(7.0)
    X.chunk("f32")(X.q, i32([-9, 0, 0, 0]), X.lens_t, out=out, error_flag=err)
    assert (out == 7).all() and int(err) == 0
    lens = i32([65, 1 << 30, -4])
    o = X.chunk("f32")(X.q, X.offs_t, lens, error_flag=err)
    assert int(err) == kvq.KVQ_DEVERR_SEQ_CLAMPED
    X.check(o, "f32", ref, rows=slice(0, 5))
    assert torch.isfinite(o[5:25]).all() and (o[25:] == 0).all()


def test_offsets_that_overlap():
    """Requests that share rows, more of them than the rows hold: nothing is written."""
    X = Packed("fp8", 64, 8, 2, 16, [(200, 200), (30, 20), (200, 200), (40, 2), (200, 200)])
    q = X.q[:200].contiguous()
    out = torch.full(q.shape, 7.0, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    X.chunk("f32")(q, i32([0, 200, 0, 200, 0, 200]), X.lens_t, out=out, error_flag=err)
    assert int(err) == kvq.KVQ_DEVERR_SEQ_CLAMPED and (out == 7).all()


def test_bad_pages():
    """A page out of range is read as page 0, with its error bit."""
    X = Packed("fp8", 64, 4, 2, 16, [(200, 5), (30, 20)])
    X.bt[0, 3], X.bt[1, 0] = -1, 1 << 20
    got = X.chunk("f32")
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    o = got(X.q, X.offs_t, X.lens_t, error_flag=err)
    assert int(err) == kvq.KVQ_DEVERR_BAD_PAGE
    X.bt[0, 3], X.bt[1, 0] = 0, 0
    X.check(o, "f32", X.reference())


@pytest.mark.parametrize("diff", [False, True])
@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
def test_values_that_nobody_attends_to(diff, fmt):
    """NaN after each sequence's end reaches nothing; NaN of a new token reaches exactly
    the rows that attend to it (in its own request and kv head)."""
    reqs = [(70, 60), (200, 1), (0, 9)]
    X = Packed(fmt, 128, 4, 2, 16, reqs, diff=diff)
    ref = X.reference()
    bad = X.codes if fmt == "fp8" else X.bscale
    for b, n in enumerate(X.lens):
        if n % 16:
            for c in bad:
                c[int(X.bt[b, n // 16]), :, n % 16:] = 0x7F
    X.check(X.run("f32"), "f32", ref)
    for which in (0, 1):   # keys, values: head 1 of request 0's tokens 100 and 129
        for tok in (129, 100):
            bad[which][int(X.bt[0, tok // 16]), 1, tok % 16] = 0xFF if fmt == "fp8" else 0x7F
            o = X.run("f32")
            rows = tok - 70
            X.check(o[:, :2], "f32", tuple(r[:, :2] for r in ref), what="the other kv head")
            X.check(o, "f32", ref, rows=np.r_[0:rows, 60:X.T], what="rows before")
            assert torch.isnan(o[rows:60, 2:]).all()
        for tok in (129, 100):
            page = int(X.bt[0, tok // 16])
            good = Packed(fmt, 128, 4, 2, 16, reqs, diff=diff)
            src = (good.codes if fmt == "fp8" else good.bscale)[which]
            bad[which][page, 1, tok % 16] = src[page, 1, tok % 16]


@pytest.mark.parametrize("ramp", [(0.05, 6.0), (6.0, 0.05), (1.0, 12.0)])
@pytest.mark.parametrize("reqs", [[(2000, 1)], [(1500, 100)]])
def test_moving_maxima(ramp, reqs):
    """Scores that grow by far more than the lazy maximum's headroom, tile by tile."""
    for diff in (False, True):
        X = Packed("fp8", 128, 8, 2, 16, reqs, 5, q_std=3.0, k_ramp=ramp, diff=diff, norm=False)
        o, tol, mag = X.reference()
        # the exponents here reach 2^9: their rounding is 2^-13 of a weight at most, 2^-12
        # of each map's A, which 4 covers (values up to 3.9 of their scale, lambda <= 1)
        tol = tol + 2.0 ** -12 * (mag if not diff else 4 * 2)
        for out in ("f32", "bf16"):
            X.check(X.run(out), out, (o, tol, mag), what=out)


def test_query_range():
    """Queries far outside f16: the scores keep their accuracy."""
    X = Packed("fp8", 64, 4, 2, 16, [(512, 3), (40, 150)], 2)
    for e in (-60, 40):
        old, sm = X.q, X.sm
        X.q64 = X.q.double() * 2.0 ** e
        X.q = X.q64.bfloat16()
        assert torch.equal(X.q.double(), X.q64)
        X.sm = sm * 2.0 ** -e
        X.check(X.run("f32"), "f32", what=str(e))
        X.q, X.sm = old, sm


def test_flat_tail_behind_one_large_weight():
    """2^13 tokens of weight 2^-20 each behind one of weight 1: all of them count."""
    X = Packed("fp8", 64, 1, 1, 64, [(8192, 1)])
    X.codes[0].zero_()
    X.val[0].zero_()
    X.q.zero_()
    X.q[..., 0] = 8.0
    X.q64 = X.q.double()
    page, one = int(X.bt[0, 0]), torch.tensor(1.0).to(torch.float8_e4m3fn).view(torch.uint8).item()
    X.codes[0][page, 0, 0, 0] = one
    X.val[0][page, 0, 0, 0] = float(np.float32(0.0137))
    X.sm = 20 * math.log(2) / (8 * 0.0137)
    ref = X.reference()
    for out in ("f32", "bf16"):
        X.check(X.run(out), out, ref)


@pytest.mark.parametrize("out,diff,rows,L,norm", [
    ("f32", False, 512, 6000, True), ("f32", True, 256, 14000, True), ("f32", True, 256, 14000, False),
    ("bf16", False, 512, 45000, True)])
def test_long_sums_of_one_sign(out, diff, rows, L, norm):
    """Long pieces whose products all have one sign: an accumulator that is cut off at each
    of its products loses more and more of it."""
    X = Packed("fp8", 128, 32, 8, 48, [(L - rows, rows)], diff=diff, norm=norm)
    X.codes[1] &= 0x7F
    X.val[1] = X.val[1].abs()
    o, tol, _ = ref = X.reference()
    got = X.run(out)
    X.check(got, out, ref)
    if not diff and out == "f32":   # fp32: also on the whole
        e = (got.double().cpu().numpy() - o) / o
        assert abs(e.mean()) < 2.0 ** -17


@pytest.mark.parametrize("out,diff,past", [("f32", False, 6000), ("f32", True, 6000), ("bf16", False, 70000)])
@pytest.mark.parametrize("ramp", [(0.2, 2.0), (2.0, 0.2)])
def test_long_sums_of_few_rows(out, diff, past, ramp):
    """Pieces of many key tiles with one accumulator's rows, whose maxima move."""
    X = Packed("fp8", 64, 8, 2, 64, [(past + 13 * b, 20) for b in range(40)], diff=diff, k_ramp=ramp)
    X.check(X.run(out), out)


def test_is_the_decode_and_the_prefill():
    """Single tokens and equal chunks: the library's other calls agree."""
    X = Packed("nvfp4", 128, 8, 2, 16, [(400, 1), (31, 1), (0, 1)])
    cfg = runtime.DecodeConfig(3, 8, 128, 128, 3, X.cap, X.sm, out="f32")
    ref = X.reference()
    X.check(runtime.decode_fused(X.cache, X.q, X.lens_t, cfg), "f32", ref)
    X.check(X.run("f32"), "f32", ref)
    X = Packed("fp8", 64, 6, 2, 16, [(100, 40), (3, 40)])
    cfg = runtime.DecodeConfig(2, 6, 64, 64, 1, X.cap, X.sm, out="f32")
    o = runtime.prefill(X.cache, X.q.view(2, 40, 6, 64), X.lens_t, cfg, 40)
    ref = X.reference()
    X.check(o.view(80, 6, 64), "f32", ref)
    X.check(X.run("f32"), "f32", ref)


@pytest.mark.parametrize("diff", [False, True])
def test_workspace_holds_nothing(diff):
    """Whatever the workspace holds, and after other steps in it: the same bits."""
    X = Packed("fp8", 128, 8, 2, 16, MIXED, diff=diff)
    att = X.chunk("bf16")
    first = att(X.q, X.offs_t, X.lens_t).clone()
    for fill in (0xFF, 0x7F, 0):
        att._ws.fill_(fill)
        assert torch.equal(att(X.q, X.offs_t, X.lens_t), first)
    att(X.q[:1], i32([0, 1] + [1] * (X.B - 1)), X.lens_t)
    assert torch.equal(att(X.q, X.offs_t, X.lens_t), first)


def test_streams_graphs_and_two_objects():
    """Back to back, on two streams at once with a workspace each, and replayed from a
    graph with lengths, offsets and queries that change in place."""
    X = Packed("fp8", 128, 8, 2, 16, [(500, 1), (300, 90), (0, 30)])
    Y = Packed("nvfp4", 64, 6, 3, 32, [(1500, 1)] * 20, diff=True)
    rx, ry = X.reference(), Y.reference()
    ax, ay = X.chunk("f32"), Y.chunk("f32")
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        outs.append((ax(X.q, X.offs_t, X.lens_t, stream=s), ay(Y.q, Y.offs_t, Y.lens_t, stream=t)))
    torch.cuda.synchronize()
    for ox, oy in outs:
        assert torch.equal(ox, outs[0][0]) and torch.equal(oy, outs[0][1])
    X.check(outs[0][0], "f32", rx)
    Y.check(outs[0][1], "f32", ry)
    q, offs, lens, out = X.q.clone(), X.offs_t.clone(), X.lens_t.clone(), torch.zeros(X.T, 8, 128, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ax(q, offs, lens, out=out)
        ay(Y.q, Y.offs_t, Y.lens_t, out=(oy := torch.empty(Y.T, 6, 64, device=DEV)))
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, outs[0][0]) and torch.equal(oy, outs[0][1])
    # other lengths: the first request takes the chunk, the second a single token
    X.reqs = [(440, 61), (389, 1), (0, 30)]
    X.lens, X.new = [501, 390, 30], [61, 1, 30]
    X.offs = np.array([0, 61, 62, 92])
    X.T = 92
    X.q, X.q64 = X.q[:92], X.q64[:92]
    offs.copy_(i32(X.offs.tolist()))
    lens.copy_(i32(X.lens))
    g.replay()
    torch.cuda.synchronize()
    X.check(out[:92], "f32")


def test_long_cache_offsets():
    """Rows of a cache past 2^31 bytes."""
    ps, hkv, D = 256, 8, 128
    pages = (1 << 31) // (ps * hkv * D) + 40
    kc = torch.zeros(pages, hkv, ps, D, dtype=torch.uint8, device=DEV)
    vc = torch.zeros_like(kc)
    X = Packed("fp8", D, 16, hkv, ps, [(700, 30)])
    n = X.bt.shape[1]
    far = torch.arange(pages - n, pages, device=DEV)
    kc[far], vc[far] = X.codes[0][X.bt[0].long()], X.codes[1][X.bt[0].long()]
    cache = runtime.QuantizedKVCache.wrap("fp8", kc, vc, far.int()[None].contiguous(), 0.0137, 0.0119)
    att = runtime.ChunkAttention(cache, 1, 16, X.cap, X.sm, out="f32")
    X.check(att(X.q, X.offs_t, X.lens_t), "f32")


def test_refused():
    X = Packed("fp8", 128, 8, 2, 16, [(50, 3), (0, 4)])
    att = X.chunk("bf16")
    for args in ((X.q.float(), X.offs_t, X.lens_t), (X.q[:, :4], X.offs_t, X.lens_t),
                 (X.q, X.offs_t[:2], X.lens_t), (X.q, X.offs_t, X.lens_t[:1]), (X.q, X.offs_t.long(), X.lens_t),
                 (X.q.cpu(), X.offs_t, X.lens_t), (X.q.transpose(0, 1), X.offs_t, X.lens_t)):
        with pytest.raises(ValueError):
            att(*args)
    for out in (torch.empty(7, 8, 128, device=DEV), torch.empty(6, 8, 128, device=DEV).bfloat16(),
                torch.empty(7, 8, 256, device=DEV).bfloat16()[..., ::2]):
        with pytest.raises(ValueError):
            att(X.q, X.offs_t, X.lens_t, out=out)
    with pytest.raises(ValueError):
        runtime.ChunkAttention(X.cache, 3, 8, X.cap, X.sm)
    with pytest.raises(kvq.KvqError):
        runtime.ChunkAttention(X.cache, 2, 7, X.cap, X.sm)
    with pytest.raises(ValueError):
        runtime.ChunkAttention(X.cache, 2, 8, X.cap, X.sm, diff=runtime.Differential(torch.ones(4, device=DEV)))
    with pytest.raises(ValueError):
        runtime.ChunkAttention(X.cache, 2, 8, X.cap, X.sm, diff=runtime.Differential(
            torch.ones(8, device=DEV), norm=torch.ones(64, device=DEV)))
    with pytest.raises(kvq.KvqError):
        runtime.ChunkAttention(X.cache, 2, 8, X.cap + 1, X.sm)
    assert att(X.q[:0], i32([0, 0, 0]), X.lens_t).shape == (0, 8, 128)
    p = att.cfg.params(X.lens_t)
    st = kvq.kvq_chunk_attention(X.cache.struct(), p, None, 7, X.offs_t, X.q, att._ws, att._ws.numel() - 1, X.q)
    assert st == kvq.KVQ_ERR_WORKSPACE
