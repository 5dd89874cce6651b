"""Norm and rotation of queries and keys, and the append that applies them,
against the formulas in 64 bits (tests/rope_ref.py derives the bounds); V's
codes against the plain append's, bit for bit; cache rows, outputs and padding
that a call does not own stay as they were."""
import math

import numpy as np
import pytest
import torch

import rope_ref as R
from quantized_kv_cache_05_gb300 import build as kbuild
from quantized_kv_cache_05_gb300 import kvq, runtime

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    kbuild.build()
    kvq.lib()
    torch.cuda.init()
    torch.zeros(1, device=DEV)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def rand(shape, seed, std=1.5):
    return (torch.randn(shape, generator=gen(seed), device=DEV) * std).bfloat16()


def weights(d, seed):
    return 1 + 0.3 * torch.randn(d, generator=gen(seed), device=DEV)


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def make_rotary(dim, rot, inter, norm, rows=700, seed=0):
    table = runtime.rope_table(rows, rot) if rot else None
    qw, kw = (weights(dim, seed + 1), weights(dim, seed + 2)) if norm else (None, None)
    return runtime.Rotary(table, inter, qw, kw, EPS)


def reference(x, w, pos, ro, dim):
    rot = 0 if ro.table is None else ro.table.shape[1]
    return R.turn(f64(x), f64(w), pos, f64(ro.table), rot, bool(ro.struct().interleaved), EPS)


CASES = [(d, rot, inter, norm) for d in (64, 128, 256) for rot in sorted({0, 32, 64, d})
         for inter in (False, True) for norm in (False, True) if rot or not inter]


@pytest.mark.parametrize("dim,rot,inter,norm", CASES)
def test_norm_rope(dim, rot, inter, norm):
    T, hq, hk = 37, 6, 2
    x = rand((T, (hq + hk) * dim), 11 * dim + rot)
    q, k = x[:, :hq * dim].unflatten(1, (hq, dim)), x[:, hq * dim:].unflatten(1, (hk, dim))
    ro = make_rotary(dim, rot, inter, norm)
    pos = torch.randint(0, 700, (T,), generator=gen(5), device=DEV).int()
    before = x.clone()
    qo, ko = runtime.norm_rope(ro, q, k, pos)
    p = pos.cpu().numpy()
    for got, inp, w, name in ((qo, q, ro.q_norm, "q"), (ko, k, ro.k_norm, "k")):
        R.check_bf16(f64(got), *reference(inp, w, p, ro, dim), name)
    assert torch.equal(before, x)
    # FP8 queries, a scale for all and one for each head
    for hs in (None, torch.linspace(0.01, 0.05, hq, device=DEV)):
        q8, none = runtime.norm_rope(ro, q, None, pos, q_out_type="e4m3", q_scale=0.021, q_head_scale=hs)
        assert none is None and q8.dtype == torch.uint8
        s = np.float64(np.float32(0.021)) if hs is None else f64(hs)[None, :, None]
        R.check_grid(R.e4m3_values(q8.cpu().numpy()), *reference(q, ro.q_norm, p, ro, dim), s, R.E4M3_POS, "q8")
    # the inputs' own rows as outputs
    runtime.norm_rope(ro, q, k, pos, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko)


@pytest.mark.parametrize("T", [1, 2, 33, 1000])
def test_norm_rope_keys_alone_and_strides(T):
    """Keys alone, heads further apart than the head dim (the last 64 of 192), one
    norm of the two given."""
    x = rand((T, 3, 192), T)
    k = x[:, :, 128:]
    ro = runtime.Rotary(runtime.rope_table(1200, 64), True, None, weights(64, 3), EPS)
    pos = torch.arange(T, device=DEV).int() + 100
    want = R.turn(f64(k), f64(ro.k_norm), pos.cpu().numpy(), f64(ro.table), 64, True, EPS)
    y = R.turn(f64(k), None, pos.cpu().numpy(), f64(ro.table), 64, True, EPS)
    keep = x[:, :, :128].clone()
    qo, _ = runtime.norm_rope(ro, k, None, pos)      # the queries' norm is absent
    R.check_bf16(f64(qo), *y, "q")
    _, ko = runtime.norm_rope(ro, None, k, pos, k_out=k)
    R.check_bf16(f64(ko), *want, "k")
    assert torch.equal(keep, x[:, :, :128])


def test_skipped_tokens_keep_their_rows():
    T, H, D = 9, 3, 64
    q = rand((T, H, D), 1)
    ro = make_rotary(D, 64, False, True, rows=50)
    pos = torch.tensor([0, -1, 49, 50, 3, -(2 ** 31), 2 ** 31 - 1, 7, 8], device=DEV).int()
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full((T, H, D), 7.0, device=DEV).bfloat16()
    runtime.norm_rope(ro, q, None, pos, q_out=out, error_flag=flag)
    live = [0, 2, 4, 7, 8]
    skipped = [1, 3, 5, 6]
    assert (out[skipped] == 7).all()
    R.check_bf16(f64(out[live]), *reference(q[live], ro.q_norm, pos[live].cpu().numpy(), ro, D))
    assert int(flag) == kvq.KVQ_DEVERR_BAD_POSITION
    flag.zero_()
    runtime.norm_rope(ro, q[:2], None, pos[:2], q_out=out[:2], error_flag=flag)
    assert int(flag) == 0     # padding is no error


def test_extreme_rows():
    """Zeros, the smallest and the largest inputs, infinities and NaN stay within
    their own row."""
    D = 128
    q = rand((6, 2, D), 4)
    q[0] = 0
    q[1] = 1e-38
    q[2] = 1e18
    q[3, 0, 5] = math.inf
    q[4, 1, 100] = math.nan
    ro = make_rotary(D, D, False, True)
    pos = torch.arange(6, device=DEV).int() + 1
    qo, _ = runtime.norm_rope(ro, q, None, pos)
    ok = [(0, 0), (0, 1), (1, 0), (1, 1), (2, 0), (2, 1), (3, 1), (4, 0), (5, 0), (5, 1)]
    with np.errstate(invalid="ignore"):
        y, mag = reference(q, ro.q_norm, pos.cpu().numpy(), ro, D)
    got = f64(qo)
    for t, h in ok:
        R.check_bf16(got[t, h], y[t, h], mag[t, h], f"row {t} {h}")
    assert np.isnan(got[3, 0]).any() and np.isnan(got[4, 1]).all()


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

def make_cache(fmt, B, per, ps, hkv, D, seed, head_scales=False, rope=0):
    bt = torch.randperm(B * per, generator=gen(seed), device=DEV).int().reshape(B, per)
    hs = [torch.linspace(lo, 3 * lo, hkv, device=DEV) if head_scales else None for lo in (0.011, 0.013)]
    c = runtime.QuantizedKVCache(fmt, B * per, ps, hkv, D, bt, 0.0213, 0.0171, rope_dim=rope,
                                 k_head_scale=hs[0], v_head_scale=hs[1])
    for t in (c.k_codes, c.v_codes, c.k_bscale, c.v_bscale):
        if t is not None:
            t.copy_(torch.randint(0, 120, t.shape, generator=gen(seed + 1), device=DEV))
    return c


def rows_of(cache, t, pos, b):
    """Cache rows [n][heads][row] of request b's positions."""
    page = cache.block_table[b].long()[pos // cache.page_size]
    return t[page, :, pos % cache.page_size]


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("dim,rot,inter,norm", [(64, 64, False, True), (64, 32, True, False),
                                                (128, 128, False, True), (128, 64, False, False),
                                                (128, 128, True, True), (256, 96, False, True)])
@pytest.mark.parametrize("B,T,q8,hs", [(3, 37, False, False), (5, 1, True, True)])
def test_append(fmt, dim, rot, inter, norm, B, T, q8, hs):
    hq, hkv, ps, per = 6, 3, 16, 8
    cache = make_cache(fmt, B, per, ps, hkv, dim, 3, hs)
    plain = make_cache(fmt, B, per, ps, hkv, dim, 3, hs)
    ro = make_rotary(dim, rot, inter, norm)
    x = rand((B, T, (hq + 2 * hkv) * dim), dim + T)
    cut = lambda a, n: x[..., a * dim:(a + n) * dim].unflatten(2, (n, dim))
    q, k, v = cut(0, hq), cut(hq, hkv), cut(hq + hkv, hkv)
    start = torch.randint(0, per * ps - T, (B,), generator=gen(9), device=DEV).int()
    lens = torch.randint(0, T + 1, (B,), generator=gen(10), device=DEV).int()
    lens[0] = T
    old = {n: getattr(cache, n).clone() for n in ("k_codes", "v_codes", "k_bscale", "v_bscale")
           if getattr(cache, n) is not None}
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    qo = torch.full((B, T, hq, dim), 3, device=DEV, dtype=torch.uint8 if q8 else torch.bfloat16)
    q_hs = torch.linspace(0.01, 0.05, hq, device=DEV) if q8 and hs else None
    cache.append_rope(ro, k, v, start, new_lens=lens, q=q, q_out=qo, q_scale=0.019, q_head_scale=q_hs,
                      error_flag=flag)
    plain.append(k.contiguous(), v.contiguous(), start)
    torch.cuda.synchronize()
    assert int(flag) == 0
    kg = f64(cache.k_head_scale)[None, :, None] if hs else np.float64(np.float32(0.0213))
    for b in range(B):
        n = int(lens[b])
        pos = int(start[b]) + torch.arange(n, device=DEV)
        p = pos.cpu().numpy()
        # V: the plain append's codes
        for name in ("v_codes", "v_bscale"):
            if name in old:
                assert torch.equal(rows_of(cache, getattr(cache, name), pos, b),
                                   rows_of(plain, getattr(plain, name), pos, b)), name
        yk = reference(k[b, :n], ro.k_norm, p, ro, dim)
        codes = rows_of(cache, cache.k_codes, pos, b).cpu().numpy()
        if fmt == "fp8":
            R.check_grid(R.e4m3_values(codes), *yk, kg, R.E4M3_POS, "K")
        else:
            R.check_nvfp4(codes, rows_of(cache, cache.k_bscale, pos, b).cpu().numpy(), *yk, kg, "K")
        yq = reference(q[b, :n], ro.q_norm, p, ro, dim)
        if q8:
            s = np.float64(np.float32(0.019)) if q_hs is None else f64(q_hs)[None, :, None]
            R.check_grid(R.e4m3_values(qo[b, :n].cpu().numpy()), *yq, s, R.E4M3_POS, "q")
        else:
            R.check_bf16(f64(qo[b, :n]), *yq, "q")
        assert (qo[b, n:] == 3).all()
        # everything else of the request's pages is untouched
        rest = torch.ones(per * ps, dtype=torch.bool, device=DEV)
        rest[pos] = False
        at = rest.nonzero()[:, 0]
        for name, t in old.items():
            assert torch.equal(rows_of(cache, getattr(cache, name), at, b), rows_of(cache, t, at, b)), name


def test_append_without_norm_or_rotation_is_the_plain_append():
    for fmt in ("fp8", "nvfp4"):
        a, b = (make_cache(fmt, 2, 4, 16, 2, 128, 1) for _ in range(2))
        k, v = rand((2, 20, 2, 128), 1), rand((2, 20, 2, 128), 2)
        start = torch.tensor([3, 40], device=DEV).int()
        a.append_rope(runtime.Rotary(None), k, v, start)
        b.append(k, v, start)
        for n in ("k_codes", "v_codes", "k_bscale", "v_bscale"):
            if getattr(a, n) is not None:
                assert torch.equal(getattr(a, n), getattr(b, n)), n


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("inter", [False, True])
def test_append_mla(inter, norm):
    B, T, ps, per = 3, 21, 16, 4
    cache = make_cache("nvfp4", B, per, ps, 1, 512, 5, rope=64)
    old = cache.k_codes.clone(), cache.k_pe.clone()
    x = rand((B, T, 1, 576), 8)           # latent and rope key side by side
    lat, pe = x[..., :512], x[..., 512:]
    ro = runtime.Rotary(runtime.rope_table(100, 64), inter, None, weights(512, 1) if norm else None, EPS)
    start = torch.tensor([0, 17, 40], device=DEV).int()
    lens = torch.tensor([21, 0, 20], device=DEV).int()
    cache.append_rope(ro, lat, None, start, kpe_new=pe, new_lens=lens)
    for b in range(B):
        n = int(lens[b])
        pos = int(start[b]) + torch.arange(n, device=DEV)
        p = pos.cpu().numpy()
        y = R.turn(f64(lat[b, :n]), f64(ro.k_norm), p, None, 0, inter, EPS)
        R.check_nvfp4(rows_of(cache, cache.k_codes, pos, b).cpu().numpy(),
                      rows_of(cache, cache.k_bscale, pos, b).cpu().numpy(), *y, float(np.float32(0.0213)), "latent")
        page = cache.block_table[b].long()[pos // ps]
        got = cache.k_pe[page, pos % ps]
        R.check_bf16(f64(got)[:, None], *R.turn(f64(pe[b, :n]), None, p, f64(ro.table), 64, inter, EPS), "k_pe")
        cache.k_pe[page, pos % ps] = old[1][page, pos % ps]
        cache.k_codes[page, :, pos % ps] = old[0][page, :, pos % ps]
    assert torch.equal(cache.k_pe, old[1]) and torch.equal(cache.k_codes, old[0])


def test_append_bad_positions_and_pages():
    """Rows that have no place are skipped, and what went wrong is flagged."""
    cache = make_cache("fp8", 4, 4, 16, 2, 64, 2)
    old = cache.k_codes.clone(), cache.v_codes.clone()
    ro = make_rotary(64, 64, False, False, rows=60)
    x = rand((4, 2, 2, 64), 3)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)

    def call(start):
        flag.zero_()
        q = torch.full((4, 2, 2, 64), 9.0, device=DEV).bfloat16()
        cache.append_rope(ro, x, x, torch.tensor(start, device=DEV).int(), q=x, q_out=q, error_flag=flag)
        return int(flag), (q != 9).flatten(2).any(-1)

    bits, wrote = call([-2, 60, 2 ** 31 - 1, -(2 ** 31)])
    assert bits == kvq.KVQ_DEVERR_BAD_POSITION and not wrote.any()
    assert torch.equal(cache.k_codes, old[0]) and torch.equal(cache.v_codes, old[1])
    bits, wrote = call([-1, 59, -5, -5])      # the second of two is in range, then the first
    assert bits == kvq.KVQ_DEVERR_BAD_POSITION
    assert wrote.tolist() == [[False, True], [True, False], [False, False], [False, False]]
    # positions that the rotation table covers and the block table does not: no cache row
    wide = runtime.Rotary(runtime.rope_table(400, 64))
    cache.k_codes.copy_(old[0])
    flag.zero_()
    cache.append_rope(wide, x, x, torch.tensor([64, 300, 64, 64], device=DEV).int(), error_flag=flag)
    assert int(flag) == 0 and torch.equal(cache.k_codes, old[0])
    cache.block_table[1, 0], cache.block_table[2, 0] = 16, -1
    flag.zero_()
    cache.append_rope(wide, x, x, torch.tensor([64, 0, 0, 64], device=DEV).int(), error_flag=flag)
    assert int(flag) == kvq.KVQ_DEVERR_BAD_PAGE and torch.equal(cache.k_codes, old[0])


def test_streams_graphs_and_two_calls():
    """On a stream of its own, and replayed from a graph with new inputs in place."""
    cache = make_cache("fp8", 2, 8, 16, 2, 128, 4)
    ro = make_rotary(128, 128, False, True)
    x, v = rand((2, 1, 2, 128), 1), rand((2, 1, 2, 128), 2)
    start = torch.tensor([5, 77], device=DEV).int()
    qo = torch.zeros(2, 1, 2, 128, device=DEV).bfloat16()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        cache.append_rope(ro, x, v, start, q=x, q_out=qo)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.append_rope(ro, x, v, start, q=x, q_out=qo)
        q2, k2 = runtime.norm_rope(ro, x[:, 0], x[:, 0], start)
    x.copy_(rand((2, 1, 2, 128), 7))
    start.add_(1)
    g.replay()
    torch.cuda.synchronize()
    y, mag = reference(x[:, 0], ro.q_norm, start.cpu().numpy(), ro, 128)
    R.check_bf16(f64(qo[:, 0]), y, mag)
    assert torch.equal(q2, qo[:, 0])
    yk = reference(x[:, 0], ro.k_norm, start.cpu().numpy(), ro, 128)
    R.check_bf16(f64(k2), *yk)
    for b in range(2):
        got = rows_of(cache, cache.k_codes, start[b:b + 1].long(), b).cpu().numpy()
        R.check_grid(R.e4m3_values(got), yk[0][b:b + 1], yk[1][b:b + 1], np.float64(np.float32(0.0213)), R.E4M3_POS)


def test_runtime_refuses():
    ro = make_rotary(64, 64, False, True)
    q, pos = rand((4, 2, 64), 1), torch.arange(4, device=DEV).int()
    for args in ((q.float(), None, pos), (q, None, pos.long()), (q, None, pos[:3]), (None, None, pos),
                 (q, q[:3], pos), (q[..., :32], None, pos), (q.transpose(1, 2), None, pos),
                 (q.cpu(), None, pos)):
        with pytest.raises(ValueError):
            runtime.norm_rope(ro, *args)
    with pytest.raises(ValueError):
        runtime.norm_rope(ro, q, None, pos, q_out_type="f16")
    with pytest.raises(kvq.KvqError):
        runtime.norm_rope(ro, q, None, pos, q_out_type="e4m3", q_scale=0.0)
    with pytest.raises(kvq.KvqError):
        runtime.norm_rope(ro, q, None, None)
    cache = make_cache("fp8", 2, 2, 16, 2, 64, 1)
    x, start = rand((2, 2, 2, 64), 1), torch.zeros(2, device=DEV).int()
    for kw in (dict(k_new=x[:, :, :1]), dict(v_new=None), dict(v_new=x[:1]), dict(start_pos=start[:1]),
               dict(start_pos=start.long()), dict(new_lens=start[:1]), dict(q=x[:1]), dict(q=x, q_out=x[:1]),
               dict(k_new=rand((3, 2, 2, 64), 1), v_new=rand((3, 2, 2, 64), 1)),
               dict(q=x, q_head_scale=torch.ones(3, device=DEV))):
        with pytest.raises(ValueError):
            cache.append_rope(ro, **{"k_new": x, "v_new": x, "start_pos": start, **kw})
    assert cache.append_rope(ro, x[:0], x[:0], start[:0]) is None
    empty, _ = runtime.norm_rope(ro, q[:0], None, pos[:0])
    assert empty.shape == (0, 2, 64)


def test_single_token_of_odd_stride():
    """A lone token's stride is never used, whatever torch says it is."""
    ro = make_rotary(64, 64, False, False)
    q = rand((1, 3, 64), 1)
    odd = torch.as_strided(q, (1, 1, 3, 64), (3, 5, 64, 1))
    pos = torch.tensor([9], device=DEV).int()
    want, _ = runtime.norm_rope(ro, q, None, pos)
    cache = make_cache("fp8", 1, 2, 16, 3, 64, 1)
    got = cache.append_rope(ro, odd, odd, pos, q=odd)
    assert torch.equal(got[0], want)
    one = torch.as_strided(q, (1, 1, 64), (7, 5, 1))
    assert torch.equal(runtime.norm_rope(ro, one, None, pos)[0], want[:, :1])


def test_pinned_host_rows():
    """New rows read from, and the queries written to, page-locked host memory."""
    cache, same = (make_cache("fp8", 3, 4, 16, 2, 64, 6) for _ in range(2))
    ro = make_rotary(64, 64, False, True)
    x = rand((3, 2, 2, 64), 2)
    start = torch.tensor([0, 9, 40], device=DEV).int()
    want = cache.append_rope(ro, x, x, start, q=x)
    h = x.cpu().pin_memory()
    out = torch.zeros(x.shape, dtype=torch.bfloat16).pin_memory()
    rows = lambda t: kvq.kvq_heads(t.data_ptr(), 128, 64, 2)
    kvq.check(kvq.kvq_rope_append(same.struct(), ro.struct(), 3, 2, start, None, rows(h), rows(h), None, rows(h),
                                  rows(out), 0, 1.0, None))
    torch.cuda.synchronize()
    assert torch.equal(out, want.cpu())
    assert torch.equal(same.k_codes, cache.k_codes) and torch.equal(same.v_codes, cache.v_codes)


def test_new_lens_beyond_the_batch_and_below_zero():
    cache, full = (make_cache("fp8", 3, 4, 16, 2, 64, 6) for _ in range(2))
    ro = make_rotary(64, 64, False, False)
    x = rand((3, 5, 2, 64), 2)
    start = torch.tensor([3, 0, 20], device=DEV).int()
    old = cache.k_codes.clone()
    cache.append_rope(ro, x, x, start, new_lens=torch.tensor([-3, -(2 ** 31), 0], device=DEV).int())
    assert torch.equal(cache.k_codes, old)
    cache.append_rope(ro, x, x, start, new_lens=torch.tensor([5, 6, 2 ** 31 - 1], device=DEV).int())
    full.append_rope(ro, x, x, start)
    assert torch.equal(cache.k_codes, full.k_codes) and torch.equal(cache.v_codes, full.v_codes)


def test_codes_next_to_boundaries_are_decided_in_64_bits():
    """Half a million values, the scale put so that some quotients lie on a rounding
    boundary: the codes are the 64-bit ones.  They have to be wherever fp32's error is
    within the 16 steps (each at least u of the value) that send a quotient to 48
    bits: 2 u of mag without a norm, so down to |y| = mag / 7 with the quotient's own
    step; with one 12.5 u (the squares' sum and eps 15 u, halved by the root, which is
    within 1 u itself, two products 2 u, the rotation 2 u), so from 0.9 mag on."""
    T, H, D = 512, 8, 128
    for inter in (False, True):
        for norm in (False, True):
            ro = make_rotary(D, D, inter, norm)
            q = rand((T, H, D), 3)
            pos = torch.randint(0, 700, (T,), generator=gen(4), device=DEV).int()
            y, mag = reference(q, ro.q_norm, pos.cpu().numpy(), ro, D)
            sure = np.abs(y) >= mag * (0.9 if norm else 1 / 7)
            for i in range(4):
                # |y[0, 0, i]| becomes 17 x 2: a boundary (17 has five bits)
                scale = float(np.float32(np.abs(y[0, 0, i]) / (17 * 2.0)))
                q8, _ = runtime.norm_rope(ro, q, None, pos, q_out_type="e4m3", q_scale=scale)
                got = R.e4m3_values(q8.cpu().numpy())
                want = R.round_value(y / np.float64(np.float32(scale)), R.E4M3_POS)
                assert np.array_equal(got[sure], want[sure])
                assert (got != want).sum() <= 4    # the rest: nearly all (cancelled sums may differ)


@pytest.mark.parametrize("append", [False, True])
def test_new_outputs_belong_to_the_stream_that_is_given(append):
    """A freed tensor that the current stream has yet to write is not the memory of an
    output that a kernel on another stream writes first."""
    ro = make_rotary(128, 128, False, True)
    x, start = rand((64, 1, 2, 128), 1), torch.zeros(64, device=DEV).int()
    cache = make_cache("fp8", 64, 2, 16, 2, 128, 1)
    want, _ = runtime.norm_rope(ro, x[:, 0], None, start)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    late = torch.empty_like(want)
    torch.cuda._sleep(20_000_000)   # about ten milliseconds
    late.fill_(7)
    del late
    if append:
        got = cache.append_rope(ro, x, x, start, q=x, stream=side)[:, 0]
    else:
        got, _ = runtime.norm_rope(ro, x[:, 0], None, start, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


# ---------------------------------------------------------------------------
# chunks: more lanes than fill the GPU, so that a lane group walks several rows
# of its token with the next row's loads in flight
# ---------------------------------------------------------------------------

def chunk_tokens(dim, heads, extra):
    """Tokens just past the launcher's change of geometry (152 x 2048 lanes), an odd count."""
    return (152 * 2048 // (dim // 16) // heads + extra) | 1


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("dim,rot,inter,norm,hq,hk", [
    (64, 64, False, True, 10, 3), (64, 32, True, False, 7, 2), (128, 128, True, True, 10, 3),
    (128, 64, False, False, 72, 9), (256, 256, False, True, 10, 3), (256, 96, True, False, 5, 2)])
def test_norm_rope_chunk(dim, rot, inter, norm, hq, hk, q8):
    T = chunk_tokens(dim, hq + hk, 40)
    assert T * (dim // 16) * (hq + hk) >= 152 * 2048
    x = rand((T, (hq + hk) * dim), 7 * dim + rot + q8)
    q, k = x[:, :hq * dim].unflatten(1, (hq, dim)), x[:, hq * dim:].unflatten(1, (hk, dim))
    ro = make_rotary(dim, rot, inter, norm)
    pos = torch.randint(0, 700, (T,), generator=gen(6), device=DEV).int()
    pos[3::17] = -1      # padding among the tokens
    fill = torch.uint8 if q8 else torch.bfloat16
    qo, ko = (torch.full((T, h, dim), 3, device=DEV, dtype=t) for h, t in ((hq, fill), (hk, torch.bfloat16)))
    runtime.norm_rope(ro, q, k, pos, q_out=qo, k_out=ko, q_out_type="e4m3" if q8 else "bf16", q_scale=0.021)
    live = pos >= 0
    assert (qo[~live] == 3).all() and (ko[~live] == 3).all()
    p = pos[live].cpu().numpy()
    R.check_bf16(f64(ko[live]), *reference(k[live], ro.k_norm, p, ro, dim), "k")
    y = reference(q[live], ro.q_norm, p, ro, dim)
    if q8:
        R.check_grid(R.e4m3_values(qo[live].cpu().numpy()), *y, np.float64(np.float32(0.021)), R.E4M3_POS, "q8")
    else:
        R.check_bf16(f64(qo[live]), *y, "q")


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("dim,rot,inter,norm,hq,hkv,q8,hs", [
    (64, 64, False, True, 7, 3, False, False), (64, 32, True, False, 7, 3, True, True),
    (128, 128, True, True, 7, 3, False, True), (128, 64, False, False, 55, 5, True, False),
    (256, 96, False, True, 7, 3, True, False), (256, 256, True, False, 0, 1, False, False)])
def test_append_chunk(fmt, dim, rot, inter, norm, hq, hkv, q8, hs):
    B, ps = 5, 48
    H = hq + 2 * hkv
    T = chunk_tokens(dim, H, 3) // B + 2
    assert B * T * (dim // 16) * H >= 152 * 2048
    per = (T + 90) // ps + 1
    cache = make_cache(fmt, B, per, ps, hkv, dim, 3, hs)
    plain = make_cache(fmt, B, per, ps, hkv, dim, 3, hs)
    ro = make_rotary(dim, rot, inter, norm, rows=T + 100)
    x = rand((B, T, H * dim), dim + T)
    cut = lambda a, n: x[..., a * dim:(a + n) * dim].unflatten(2, (n, dim))
    k, v = cut(hq, hkv), cut(hq + hkv, hkv)
    q = cut(0, hq) if hq else None
    start = torch.randint(0, 90, (B,), generator=gen(9), device=DEV).int()
    lens = torch.tensor([T, 0, T - 1, T // 3, 1], device=DEV).int()
    old = {n: getattr(cache, n).clone() for n in ("k_codes", "v_codes", "k_bscale", "v_bscale")
           if getattr(cache, n) is not None}
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    qo = torch.full((B, T, hq, dim), 3, device=DEV, dtype=torch.uint8 if q8 else torch.bfloat16) if hq else None
    cache.append_rope(ro, k, v, start, new_lens=lens, q=q, q_out=qo, q_scale=0.019, error_flag=flag)
    plain.append(k.contiguous(), v.contiguous(), start)
    torch.cuda.synchronize()
    assert int(flag) == 0
    kg = f64(cache.k_head_scale)[None, :, None] if hs else np.float64(np.float32(0.0213))
    for b in range(B):
        n = int(lens[b])
        pos = int(start[b]) + torch.arange(n, device=DEV)
        p = pos.cpu().numpy()
        for name in ("v_codes", "v_bscale"):
            if name in old:
                assert torch.equal(rows_of(cache, getattr(cache, name), pos, b),
                                   rows_of(plain, getattr(plain, name), pos, b)), name
        if n:
            yk = reference(k[b, :n], ro.k_norm, p, ro, dim)
            codes = rows_of(cache, cache.k_codes, pos, b).cpu().numpy()
            if fmt == "fp8":
                R.check_grid(R.e4m3_values(codes), *yk, kg, R.E4M3_POS, "K")
            else:
                R.check_nvfp4(codes, rows_of(cache, cache.k_bscale, pos, b).cpu().numpy(), *yk, kg, "K")
        if hq:
            if n:
                yq = reference(q[b, :n], ro.q_norm, p, ro, dim)
                if q8:
                    R.check_grid(R.e4m3_values(qo[b, :n].cpu().numpy()), *yq, np.float64(np.float32(0.019)),
                                 R.E4M3_POS, "q")
                else:
                    R.check_bf16(f64(qo[b, :n]), *yq, "q")
            assert (qo[b, n:] == 3).all()
        rest = torch.ones(per * ps, dtype=torch.bool, device=DEV)
        rest[pos] = False
        at = rest.nonzero()[:, 0]
        for name, t in old.items():
            assert torch.equal(rows_of(cache, getattr(cache, name), at, b), rows_of(cache, t, at, b)), name


@pytest.mark.parametrize("kind", ["fp8", "nvfp4", "mla"])
def test_append_in_the_plain_ones_place_before_an_overlapping_decode(kind):
    """Without queries the call stands where kvq_quantize_append does in the contract of
    fresh_tokens: the decode right behind it starts early and still reads the new rows
    (other ones at every step), bit for bit what it reads after a wait."""
    B, T, ps, per = 24, 3, 16, 40
    mla = kind == "mla"
    hq, hkv, D, qk = (16, 1, 512, 576) if mla else (8, 2, 128, 128)
    cache = make_cache("fp8" if kind == "fp8" else "nvfp4", B, per, ps, hkv, D, 3, rope=64 if mla else 0)
    ro = runtime.Rotary(runtime.rope_table(700, 64), False, None, weights(D, 1), EPS)
    start = torch.tensor([(37 * b) % 600 if b % 3 else b % 13 for b in range(B)], device=DEV).int()
    lens = start + T
    q = rand((B, hq, qk), 5)
    new = [(rand((B, T, hkv, D), 10 + k, 1 + k), None if mla else rand((B, T, hkv, D), 20 + k),
            rand((B, T, 1, 64), 30 + k) if mla else None) for k in range(3)]
    for splits in (1, 4):
        cfg = runtime.DecodeConfig(B, hq, qk, D, splits, per * ps, qk ** -0.5, out="f32")
        ws = runtime.FusedWorkspace(cfg, hkv)
        want = []
        for k, v, e in new:
            cache.append_rope(ro, k, v, start, kpe_new=e)
            torch.cuda.synchronize()
            want.append(runtime.decode_fused(cache, q, lens, cfg, ws).clone())
            torch.cuda.synchronize()
        assert not torch.equal(want[0], want[1])
        cfg.fresh_tokens = T
        got = []
        for i in range(30):
            k, v, e = new[i % 3]
            cache.append_rope(ro, k, v, start, kpe_new=e)
            got.append(runtime.decode_fused(cache, q, lens, cfg, ws).clone())
        torch.cuda.synchronize()
        for i, g in enumerate(got):
            assert torch.equal(g, want[i % 3]), i
