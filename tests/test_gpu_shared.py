"""Decode of a batch that shares a prefix (kvq_decode_shared) against softmax
attention in 64 bits over the dequantized cache.

Bounds.  With A = sum_j softmax_j |v_j| per output: a weight's relative error is
that of its exponent -- the score's fp32 accumulation, at most (D / 8) 2^-23 of
sum_d |q_d k_d| sm_scale (16 products per step, each step's sum rounded at worst
by one unit of 2^-23, twice that for the split accumulators), the exponent's own
rounding, below 2^-22 of its magnitude (at most 2^5 here), and 2^-22 of the
exponential -- and, where the output is not fp32, P's rounding to f16, at most
2^-11.  Numerator and denominator both carry the former.  Sums of up to 2^13
terms in fp32 add 2^-20 (the partials are short and the errors' signs random).
The output's own rounding is half a step: bf16 2^-8 of the value; an E4M3 code
lies between those of the interval's ends.
"""
import math

import numpy as np
import pytest
import torch

import rope_ref as R
from quantized_kv_cache_05_gb300 import build as kbuild
from quantized_kv_cache_05_gb300 import kvq, runtime

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    kbuild.build()
    kvq.lib()
    torch.cuda.init()
    torch.zeros(1, device=DEV)


class Batch:
    """A cache whose requests share `prefix` tokens; `own` tokens each of their own
    (None: a padded row of length 0; negative: a request of that many tokens
    altogether, in pages of its own)."""

    def __init__(self, fmt, D, hq, hkv, ps, prefix, own, seed=1, q_fp8=False, head_scales=False,
                 q_std=1.0, k_ramp=None):
        g = self.g = torch.Generator(device=DEV).manual_seed(seed)
        self.fmt, self.D, self.hq, self.hkv, self.ps, self.prefix, self.B = fmt, D, hq, hkv, ps, prefix, len(own)
        self.lens = [0 if n is None else -n if n < 0 else prefix + n for n in own]
        per = max(1, -(-(max([0] + self.lens)) // ps), prefix // ps)
        pre = prefix // ps
        pages = pre + self.B * per + 1
        perm = torch.randperm(pages - 1, generator=g, device=DEV).int() + 1   # page 0 is nobody's
        bt = torch.zeros(self.B, per, dtype=torch.int32, device=DEV)
        at = pre
        for b, n in enumerate(own):
            need = -(-self.lens[b] // ps)
            if n is not None and n >= 0:
                bt[b, :pre] = perm[:pre]
                bt[b, pre:need] = perm[at:at + need - pre]
                at += need - pre
            else:
                bt[b, :need] = perm[at:at + need]
                at += need
        self.shared_pages = perm[:pre].contiguous()
        self.bt = bt
        self.cap = per * ps
        x = [torch.randn(pages, hkv, ps, D, generator=g, device=DEV) for _ in range(2)]
        if k_ramp is not None:   # scores that grow (or shrink) along the shared tokens
            for i, page in enumerate(self.shared_pages.tolist()):
                t = i * ps + torch.arange(ps, device=DEV)
                x[0][page] *= (k_ramp[0] + (k_ramp[1] - k_ramp[0]) * t / prefix)[None, :, None]
        hs = [torch.linspace(0.009, 0.02, hkv, device=DEV) * s if head_scales else None for s in (1, 1.3)]
        sc = (0.0137, 0.0119) if fmt == "fp8" else (0.0023, 0.0029)
        if fmt == "nvfp4" and head_scales:
            hs = [h * 0.15 for h in hs]
        self.codes, self.bscale, self.val = [], [], []
        for t, h, s in zip(x, hs, sc):
            scale = h[None, :, None, None] if h is not None else torch.tensor(s, device=DEV)
            if fmt == "fp8":
                c = (t / scale).clamp(-448, 448).to(torch.float8_e4m3fn)
                self.codes.append(c.view(torch.uint8))
                self.bscale.append(None)
                self.val.append(c.double() * scale.double())
            else:
                blk = t.reshape(pages, hkv, ps, D // 16, 16)
                bs = (blk.abs().amax(-1) / 6 / scale).clamp(max=448).to(torch.float8_e4m3fn)
                es = bs.double() * scale.double()
                grid = torch.tensor(R.E2M1_POS, device=DEV)
                idx = ((blk.double().abs() / es[..., None])[..., None] - grid).abs().argmin(-1)
                sign = blk < 0
                nib = (idx + 8 * sign).to(torch.uint8).reshape(pages, hkv, ps, D // 2, 2)
                self.codes.append((nib[..., 0] | (nib[..., 1] << 4)).contiguous())
                self.bscale.append(bs.view(torch.uint8).contiguous())
                self.val.append((grid[idx] * torch.where(sign, -1.0, 1.0) * es[..., None]).reshape(pages, hkv, ps, D))
        self.cache = runtime.QuantizedKVCache.wrap(fmt, *self.codes, bt, *sc, *self.bscale, *hs)
        self.lens_t = torch.tensor(self.lens, device=DEV).int()
        q = torch.randn(self.B, hq, D, generator=g, device=DEV) * q_std
        self.q_fp8, self.q_scale = q_fp8, 0.017
        if q_fp8:
            c = (q / self.q_scale).clamp(-448, 448).to(torch.float8_e4m3fn)
            self.q, self.q64 = c.view(torch.uint8), c.double() * float(np.float32(self.q_scale))
        else:
            self.q = q.bfloat16()
            self.q64 = self.q.double()
        self.sm = 1 / math.sqrt(D)

    def reference(self):
        """(output, bound on the error before the output's rounding) in 64 bits; the
        bound without P's rounding."""
        G = self.hq // self.hkv
        sm = float(np.float32(self.sm))
        out = torch.zeros(self.B, self.hq, self.D, dtype=torch.float64, device=DEV)
        tol, mag = out.clone(), out.clone()
        for b, n in enumerate(self.lens):
            if not n:
                continue
            pg = self.bt[b, :-(-n // self.ps)].long()
            for h in range(self.hkv):
                k, v = (x[pg, h].reshape(-1, self.D)[:n] for x in self.val)
                q = self.q64[b, h * G:(h + 1) * G]
                s = q @ k.T * sm
                p = torch.softmax(s, 1)
                A = p @ v.abs()
                eps = (q.abs() @ k.abs().T * sm).amax(1, keepdim=True) * (self.D / 8) * 2.0 ** -23
                eps = eps + 2.0 ** -17 + 2.0 ** -22
                hs = slice(h * G, (h + 1) * G)
                out[b, hs], mag[b, hs] = p @ v, A
                tol[b, hs] = A * (2 * eps + 2.0 ** -20)
        return out.cpu().numpy(), tol.cpu().numpy(), mag.cpu().numpy()

    def plan(self, out="bf16", splits=None, **kw):
        return runtime.SharedDecode(self.cache, self.B, self.hq, self.prefix, self.cap, self.sm, out=out,
                                    out_scale=0.004, q_fp8=self.q_fp8, q_scale=self.q_scale, splits=splits, **kw)

    def check(self, got, out, ref=None, rows=None, what=""):
        o, tol, mag = ref or self.reference()
        if out != "f32":
            tol = tol + 2.0 ** -11 * mag
        if rows is not None:
            o, tol, got = o[rows], tol[rows], got[rows]
        g = got.double().cpu().numpy() if out != "e4m3" else R.e4m3_values(got.cpu().numpy())
        if out == "e4m3":
            s = float(np.float32(0.004))
            bad = ~((g >= R.round_value((o - tol) / s * (1 + 1e-6 * -np.sign(o - tol)), R.E4M3_POS)) &
                    (g <= R.round_value((o + tol) / s * (1 + 1e-6 * np.sign(o + tol)), R.E4M3_POS)))
        else:
            lim = tol + (np.abs(o) + tol) * (2.0 ** -8 if out == "bf16" else 2.0 ** -23)
            bad = ~(np.abs(g - o) <= lim)
        assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, worst "
                               f"{np.nanmax(np.abs(g - o)) if out != 'e4m3' else 'code'}, at {np.argwhere(bad)[0]}")


def run(B, out="bf16", splits=None, **kw):
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    plan = B.plan(out, splits, **kw)
    o = plan(B.q, B.lens_t, error_flag=flag).clone()
    torch.cuda.synchronize()
    assert int(flag) == 0
    assert int(plan.ws.counters.abs().sum()) == 0
    return o


OWN = [5, 0, 70, 1, 33]


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (3, 3), (14, 2), (16, 1)])
@pytest.mark.parametrize("ps,prefix", [(16, 16), (16, 400), (48, 768), (128, 1280), (256, 256)])
def test_few_rows(fmt, D, hq, hkv, ps, prefix):
    """Up to 128 rows per kv head: one row tile, token tiles in two alternating slots."""
    B = Batch(fmt, D, hq, hkv, ps, prefix, OWN)
    ref = B.reference()
    for splits in (None, (1, 1), (3, 2), (60, 4)):
        B.check(run(B, "bf16", splits), "bf16", ref, what=f"splits {splits}")


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,hq,hkv", [(16, 8, 1), (43, 6, 2), (70, 4, 1), (130, 4, 1)])
def test_many_rows(fmt, D, n, hq, hkv):
    """128 rows exactly, just over, several row tiles with a ragged last one."""
    own = [(7 * b) % 41 for b in range(n)]
    B = Batch(fmt, D, hq, hkv, 16, 656, own, seed=n)
    ref = B.reference()
    for splits in (None, (1, 1), (5, 1)):
        B.check(run(B, "bf16", splits), "bf16", ref, what=f"splits {splits}")


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("out", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("q_fp8,head_scales", [(False, False), (True, False), (False, True), (True, True)])
def test_types(fmt, out, q_fp8, head_scales):
    for n, D in ((3, 128), (50, 64)):
        B = Batch(fmt, D, 8, 2, 32, 608, [(11 * b) % 50 for b in range(n)], 3, q_fp8, head_scales)
        B.check(run(B, out), out)


@pytest.mark.parametrize("n", [6, 40])
def test_idle_and_short_requests(n):
    """Padded rows give zeros; requests shorter than the prefix read their own pages."""
    own = [[12, None, -1, 0, -303, None][b % 6] for b in range(n)]
    B = Batch("fp8", 128, 8, 2, 16, 320, own)
    for out in ("f32", "bf16"):
        o = run(B, out, prefix_table=B.shared_pages)
        B.check(o, out)
        assert (o[[b for b in range(n) if own[b] is None]] == 0).all()
    # nobody shares at all
    B = Batch("fp8", 128, 8, 2, 16, 320, [None, -5] * (n // 2))
    B.check(run(B, "f32", prefix_table=B.shared_pages), "f32")


def test_values_that_nobody_attends_to():
    """NaN codes after each sequence's end, and in the shared pages for requests that
    do not share them, reach no output."""
    own = [9, -40, None, 0]
    B = Batch("fp8", 128, 8, 2, 16, 160, own)
    ref = B.reference()
    for b, n in enumerate(B.lens):
        if n % 16:
            page = int(B.bt[b, n // 16])
            for c in B.codes:
                c[page, :, n % 16:] = 0x7F
    B.check(run(B, "f32", prefix_table=B.shared_pages), "f32", ref)
    for c in B.codes:
        c[int(B.shared_pages[3]), :, 5] = 0x7F
    o = B.plan("f32", prefix_table=B.shared_pages)(B.q, B.lens_t)
    B.check(o, "f32", ref, rows=[1, 2])
    assert torch.isnan(o[[0, 3]]).all()


@pytest.mark.parametrize("ramp", [(0.05, 6.0), (6.0, 0.05), (1.0, 12.0)])
@pytest.mark.parametrize("n", [3, 40])
def test_moving_maxima(ramp, n):
    """Scores that grow by far more than the lazy maximum's headroom, tile by tile."""
    B = Batch("fp8", 128, 8, 2, 16, 2048, [3] * n, 5, q_std=3.0, k_ramp=ramp)
    ref = B.reference()
    # the exponents here reach 2^9: their rounding is 2^-13 of a weight at most
    ref = (ref[0], ref[1] + 2.0 ** -12 * ref[2], ref[2])
    for out in ("f32", "bf16"):
        for splits in ((1, 1), (4, 1)):
            B.check(run(B, out, splits), out, ref, what=f"{out} {splits}")


def test_query_range():
    """Queries far outside f16: the scores keep their accuracy."""
    B = Batch("fp8", 64, 4, 2, 16, 512, [4, 20, 0], 2)
    for e in (-60, 40):
        B.q64 = (B.q.double() * 2.0 ** e)
        q = B.q64.bfloat16()
        assert torch.equal(q.double(), B.q64)
        old, B.q, sm = B.q, q, B.sm
        B.sm = sm * 2.0 ** -e
        B.check(run(B, "f32"), "f32", what=str(e))
        B.q, B.sm = old, sm


def test_is_kvq_decode():
    """The same call without sharing, and a prefix of length 0."""
    B = Batch("nvfp4", 128, 8, 2, 16, 480, OWN)
    cfg = runtime.DecodeConfig(B.B, 8, 128, 128, 3, B.cap, B.sm, out="f32")
    plain = runtime.decode_fused(B.cache, B.q, B.lens_t, cfg)
    o = run(B, "f32")
    tol = 2 * B.reference()[1]
    assert (np.abs((o - plain).double().cpu().numpy()) <= tol + 1e-9).all()
    zero = runtime.SharedDecode(B.cache, B.B, 8, 0, B.cap, B.sm, out="f32", splits=(1, 3))
    assert torch.equal(zero(B.q, B.lens_t), plain)


def test_bad_pages_and_lengths():
    B = Batch("fp8", 64, 4, 2, 16, 160, [4, 20])
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    table = B.shared_pages.clone()
    for bad in (-1, B.codes[0].shape[0], 2 ** 31 - 1):
        table[4] = bad
        flag.zero_()
        o = B.plan("f32", prefix_table=table)(B.q, B.lens_t, error_flag=flag).clone()
        assert int(flag) == kvq.KVQ_DEVERR_BAD_PAGE
        good = B.shared_pages.clone()
        good[4] = 0      # page 0 is read instead
        want = B.plan("f32", prefix_table=good)(B.q, B.lens_t)
        assert torch.equal(o, want)
    flag.zero_()
    lens = B.lens_t.clone()
    lens[0] = B.cap + 1
    full = B.lens_t.clone()
    full[0] = B.cap
    o = B.plan("f32")(B.q, lens, error_flag=flag).clone()
    assert int(flag) == kvq.KVQ_DEVERR_SEQ_CLAMPED
    assert torch.equal(o, B.plan("f32")(B.q, full))


def test_append_then_decode_in_a_graph():
    """The step of a serving loop: norm, rotate and append the new tokens, then the
    shared decode, captured once and replayed with new inputs; two plans of the same
    cache in one graph keep their scratch apart."""
    own = [5, 0, 40, 17]
    B = Batch("fp8", 128, 8, 2, 16, 288, [n + 4 for n in own])
    G = 4
    ro = runtime.Rotary(runtime.rope_table(1024, 128), False, 1 + 0.2 * torch.randn(128, device=DEV),
                        1 + 0.2 * torch.randn(128, device=DEV))
    x = torch.randn(4, 1, 12 * 128, device=DEV).bfloat16()
    cut = lambda a, n: x[..., a * 128:(a + n) * 128].unflatten(2, (n, 128))
    start = torch.tensor([288 + n for n in own], device=DEV).int()
    lens = start + 1
    qo = torch.zeros(4, 8, 128, device=DEV).bfloat16()
    pa, pb = B.plan("f32"), B.plan("bf16")

    def step():
        B.cache.append_rope(ro, cut(8, 2), cut(10, 2), start, q=cut(0, 8), q_out=qo)
        return pa(qo, lens), pb(qo, lens)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = step()
    for k in range(3):
        x.copy_(torch.randn(x.shape, generator=B.g, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        # the reference from the cache as it stands and the rotated queries
        B.lens, B.lens_t, B.q, B.q64 = lens.tolist(), lens, qo, qo.double()
        B.val = [c.view(torch.float8_e4m3fn).double() * float(np.float32(sc))
                 for c, sc in zip(B.codes, (0.0137, 0.0119))]
        ref = B.reference()
        B.check(a, "f32", ref)
        B.check(b, "bf16", ref)
        start.add_(1)
        lens.add_(1)


def test_back_to_back_steps_and_streams():
    """Steps that follow one another without a wait between them, each on new inputs,
    and two plans on two streams at once."""
    B = Batch("fp8", 128, 16, 4, 16, 1024, [30] * 20)
    C = Batch("nvfp4", 64, 8, 1, 16, 512, [10] * 9, seed=9)
    pb, pc = B.plan("f32"), C.plan("f32")
    want_b, want_c = pb(B.q, B.lens_t).clone(), pc(C.q, C.lens_t).clone()
    q2 = B.q.flip(0).contiguous()
    want2 = pb(q2, B.lens_t).clone()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for k in range(20):
        with torch.cuda.stream(s1):
            got.append((pb(B.q if k % 2 else q2, B.lens_t).clone(), want_b if k % 2 else want2))
        with torch.cuda.stream(s2):
            got.append((pc(C.q, C.lens_t).clone(), want_c))
    torch.cuda.synchronize()
    for g, w in got:
        assert torch.equal(g, w)


def test_pinned_host_queries_and_output():
    """Queries read from, and the output written to, page-locked host memory."""
    for n in (5, 40):      # one row tile, and two; both with few and many own chunks
        B = Batch("fp8", 128, 8, 2, 16, 320, [(9 * b) % 60 for b in range(n)])
        for splits in ((2, 1), (3, 4)):
            plan = B.plan("f32", splits)
            want = plan(B.q, B.lens_t).clone()
            q = B.q.cpu().pin_memory()
            out = torch.full(want.shape, math.nan).pin_memory()
            ws = plan.ws
            kvq.check(kvq.kvq_decode_shared(B.cache.struct(), plan.cfg.params(B.lens_t), 320, None, splits[0], q,
                                            ws.part_o, ws.part_lse, ws.counters, out))
            torch.cuda.synchronize()
            assert torch.equal(out, want.cpu())


def test_no_requests():
    B = Batch("fp8", 64, 4, 2, 16, 160, [4, 20])
    plan = runtime.SharedDecode(B.cache, 0, 4, 160, B.cap, B.sm)
    assert plan(B.q[:0], B.lens_t[:0]).shape == (0, 4, 64)


def test_more_own_chunks_than_fit_beside_the_prefix():
    """Own chunks in many waves behind a prefix that leaves no SM free, a merge of
    their own: requests of every kind, in every output type."""
    own = [None if b % 7 == 3 else -9 if b % 11 == 5 else (37 * b) % 700 for b in range(90)]
    B = Batch("nvfp4", 64, 16, 8, 16, 2560, own)
    ref = B.reference()
    for out in ("f32", "bf16", "e4m3"):
        for splits in ((19, 4), (20, 1)):
            B.check(run(B, out, splits, prefix_table=B.shared_pages), out, ref, what=f"{out} {splits}")


def test_objects_of_another_device_are_refused():
    B = Batch("fp8", 64, 4, 2, 16, 160, [4, 20])
    plan, ro = B.plan(), runtime.Rotary(runtime.rope_table(64, 64))
    ro.device = 1          # as if made there
    x = torch.zeros(2, 1, 2, 64, device=DEV).bfloat16()
    with pytest.raises(ValueError, match="cuda:1"):
        B.cache.append_rope(ro, x, x, B.lens_t)
    with pytest.raises(ValueError, match="cuda:1"):
        runtime.norm_rope(ro, x[:, 0], None, B.lens_t)
    assert runtime._launch_device(torch.cuda.current_device(), -1) == torch.cuda.current_device()
    assert plan(B.q, B.lens_t) is plan.ws.out


def test_runtime_refuses():
    B = Batch("fp8", 64, 4, 2, 16, 160, [4, 20])
    for kw in (dict(prefix_len=-16), dict(prefix_len=10 ** 6), dict(batch=3), dict(num_q_heads=5),
               dict(prefix_table=B.shared_pages[:5]), dict(prefix_table=B.shared_pages.long()),
               dict(q_head_scale=torch.ones(3, device=DEV))):
        with pytest.raises(ValueError):
            runtime.SharedDecode(**{"cache": B.cache, "batch": 2, "num_q_heads": 4, "prefix_len": 160,
                                    "max_kv_len": B.cap, "sm_scale": 0.1, **kw})
    plan = B.plan()
    for args in ((B.q.float(), B.lens_t), (B.q[:1], B.lens_t), (B.q, B.lens_t[:1]), (B.q, B.lens_t.long()),
                 (B.q.transpose(1, 2), B.lens_t), (B.q.cpu(), B.lens_t)):
        with pytest.raises(ValueError):
            plan(*args)
    with pytest.raises(kvq.KvqError):
        runtime.SharedDecode(B.cache, 2, 4, 150, B.cap, 0.1)(B.q, B.lens_t)


def round_bf16(x):
    """The nearest bf16 value (8 significant bits) of each 64-bit number."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256) / 256, e)


def check_rounded(B, got, out, ref, what=""):
    """Rounding is monotone: the output lies between the rounded ends of the interval
    of the fp32 result, whose bound holds P's two f16 parts: 2^-22 of a weight, and for
    each shared token 2^-32 of the row's largest weight."""
    o, tol, mag = ref
    vmax = float(B.val[1].abs().max())
    # + the last fp32 steps (normalisation, the quotient by the output's scale)
    tol = tol + 2.0 ** -22 * mag + 2.0 ** -32 * B.prefix * vmax + 2.0 ** -21 * np.abs(o)
    if out == "bf16":
        g, lo, hi = got.double().cpu().numpy(), round_bf16(o - tol), round_bf16(o + tol)
    else:
        s = float(np.float32(0.004))
        g = R.e4m3_values(got.cpu().numpy())
        lo, hi = R.round_value((o - tol) / s, R.E4M3_POS), R.round_value((o + tol) / s, R.E4M3_POS)
    bad = ~((g >= lo) & (g <= hi))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, at {np.argwhere(bad)[0]}"


@pytest.mark.parametrize("out", ["bf16", "e4m3"])
@pytest.mark.parametrize("fmt,D,n", [("fp8", 64, 12), ("fp8", 128, 40), ("nvfp4", 64, 40), ("nvfp4", 128, 12)])
def test_weights_keep_two_f16_parts(out, fmt, D, n):
    """A few large weights decide each row here: one f16 part (some 2^-12 of a weight)
    puts bf16 outputs on the other side of a rounding boundary, 3 to 55 of these cases'
    12288 to 81920 beyond the bound."""
    B = Batch(fmt, D, 16, 2, 16, 656, [(5 * b) % 7 for b in range(n)], 11, q_std=4.0)
    check_rounded(B, run(B, out), out, B.reference())


def test_one_f16_part_where_the_caller_asks_for_it():
    """prefix_p_f16: within 2^-11 of a weight for every output type, and not the default."""
    for n, D in ((5, 128), (40, 64)):
        B = Batch("fp8", D, 16, 2, 16, 656, [(5 * b) % 7 for b in range(n)], 11, q_std=4.0)
        ref = B.reference()
        for out in ("f32", "bf16", "e4m3"):
            o, tol, mag = ref
            narrow = run(B, out, prefix_p_f16=True)
            B.check(narrow, out, (o, tol + 2.0 ** -11 * mag, mag))
            assert not torch.equal(narrow, run(B, out))


@pytest.mark.parametrize("splits", [(4, 2), (9, 16), (17, 4)])
def test_inputs_written_right_before_the_call(splits):
    """Queries, lengths, block table and own pages written by the kernels right before
    the call in one graph, other values at every replay: the own chunks run on all SMs
    beside the prefix and have to see them (compared with the same call on its own)."""
    own = [200 + (29 * b) % 300 for b in range(24)]
    B = Batch("fp8", 128, 32, 8, 16, 2176, own, 21)
    plan = B.plan("bf16", splits)
    names = ("q", "lens", "bt", "v")
    live = dict(q=B.q, lens=B.lens_t, bt=B.bt, v=B.codes[1])
    sets = []
    for k in range(4):
        lens = torch.tensor([2176 + (v * (k + 3) + 11 * b) % 500 for b, v in enumerate(own)], device=DEV).int()
        lens = lens.clamp(max=B.cap)
        perm = torch.arange(B.B, device=DEV).roll(k)     # another request's pages behind the prefix
        # (every row long enough: entries past a request's own pages are page 0)
        bt, q, v = B.bt[perm].contiguous(), B.q.roll(k, 0).contiguous(), B.codes[1].roll(k, 0).contiguous()
        sets.append(dict(q=q, lens=torch.minimum(lens, B.lens_t[perm]).int(), bt=bt, v=v))
    want = []
    for s in sets:
        for n in names:
            live[n].copy_(s[n])
        torch.cuda.synchronize()
        want.append(plan(B.q, B.lens_t).clone())
        torch.cuda.synchronize()
    assert not torch.equal(want[0], want[1])
    src = {n: torch.empty_like(sets[0][n]) for n in names}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        # element kernels, not copies: their writes stay in the caches
        live["v"].copy_(src["v"] ^ 0)
        live["bt"].copy_(src["bt"] + 0)
        live["lens"].copy_(src["lens"] + 0)
        live["q"].copy_(src["q"] * 1)
        out = plan(B.q, B.lens_t)
    for k in range(300):
        for n in names:
            src[n].copy_(sets[k % 4][n])
        g.replay()
        got = out.clone()
        if k % 50 < 8:
            assert torch.equal(got, want[k % 4]), k
    torch.cuda.synchronize()
    assert int(plan.ws.counters.abs().sum()) == 0


@pytest.mark.parametrize("n", [5, 40])
@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
def test_head_scales_of_zero_and_below(n, fmt):
    """A scale of zero gives every token the same weight, one below zero turns the
    order round; the prefix ends inside a 128-token tile."""
    B = Batch(fmt, 64, 8, 2, 16, 400, [(7 * b) % 30 for b in range(n)], 4, q_fp8=True)
    hs = torch.tensor([0.0, 0.017, -0.017, -0.0, 0.03, 0.0, -0.03, 0.01], device=DEV)
    B.q64 = B.q.view(torch.float8_e4m3fn).double() * hs.double()[:, None]
    ref = B.reference()
    o = run(B, "f32", q_head_scale=hs)
    B.check(o, "f32", ref)
    cfg = runtime.DecodeConfig(B.B, 8, 64, 64, 2, B.cap, B.sm, out="f32", q_fp8=True, q_head_scale=hs)
    B.check(runtime.decode_fused(B.cache, B.q, B.lens_t, cfg), "f32", ref)


@pytest.mark.parametrize("n", [5, 40])
def test_queries_whose_scale_underflows(n):
    """|q| below 2^-113 and a small score scale: their product falls out of fp32's range,
    and every token has the same weight."""
    B = Batch("fp8", 64, 8, 2, 16, 400, [(7 * b) % 30 for b in range(n)], 4)
    B.q = (torch.randn(B.q.shape, generator=B.g, device=DEV) * 2.0 ** -118).bfloat16()
    B.q64, B.sm = B.q.double(), 2.0 ** -25
    B.check(run(B, "f32"), "f32")


@pytest.mark.parametrize("n", [6, 40, 70])
def test_the_prefix_comes_from_a_request_that_shares_it(n):
    """Without a table of its own: idle and shorter requests come first, with entries
    of no meaning (out of range, or other pages) in their rows of the block table."""
    for lead in ([None], [-40, None, -1], [None] * (n - 1)):
        own = lead + [(13 * b) % 50 for b in range(n - len(lead))]
        B = Batch("fp8", 128, 8, 2, 16, 320, own, n)
        for b, v in enumerate(own):
            if v is None:
                B.bt[b] = -1 if b % 2 == 0 else 2 ** 30
        for out in ("f32", "bf16"):
            B.check(run(B, out), out, what=f"{lead}")
    B = Batch("fp8", 128, 8, 2, 16, 320, [None, -5] * (n // 2))
    B.bt[0] = -1
    B.check(run(B, "f32"), "f32", what="nobody shares")


def test_first_call_of_a_thread():
    """Each entry point as the first CUDA call that a thread makes."""
    import threading
    B = Batch("fp8", 128, 16, 2, 16, 320, [30] * 4)
    plan = B.plan("f32")
    cfg = runtime.DecodeConfig(4, 16, 128, 128, 2, B.cap, B.sm, out="f32")
    ws = runtime.FusedWorkspace(cfg, 2)
    q = B.q.reshape(4, 1, 16, 128)
    calls = [lambda: plan(B.q, B.lens_t), lambda: runtime.decode_fused(B.cache, B.q, B.lens_t, cfg, ws),
             lambda: runtime.prefill(B.cache, q, B.lens_t, cfg, 1, want[2])]
    want = [None, None, torch.zeros(4, 1, 16, 128, device=DEV)]
    for i, c in enumerate(calls):
        want[i] = c().clone()
    torch.cuda.synchronize()
    for c, w in zip(calls, want):
        got = []

        def work():
            try:
                got.append(c())
            except Exception as e:   # noqa: BLE001 - shown by the assertion
                got.append(e)
        t = threading.Thread(target=work)
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert isinstance(got[0], torch.Tensor) and torch.equal(got[0], w), got


def test_two_threads_with_different_splits():
    """Calls of one kernel with different scratch sizes from two threads at once."""
    import threading
    B = Batch("fp8", 128, 16, 2, 16, 8192, [30] * 4)
    plans = [B.plan("f32", s) for s in ((1, 1), (60, 4))]
    cfgs = [runtime.DecodeConfig(4, 16, 128, 128, s, B.cap, B.sm, out="f32") for s in (1, 64)]
    calls = []
    for plan, cfg in zip(plans, cfgs):
        ws = runtime.FusedWorkspace(cfg, 2)
        calls.append((lambda plan=plan: plan(B.q, B.lens_t),
                      lambda cfg=cfg, ws=ws: runtime.decode_fused(B.cache, B.q, B.lens_t, cfg, ws)))
    want = [[c().clone() for c in pair] for pair in calls]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                torch.zeros(1, device=DEV)   # (a call that the thread's context comes from)
                for _ in range(400):
                    for c in calls[i]:
                        c()
                for c, w in zip(calls[i], want[i]):
                    got = c()
                    torch.cuda.current_stream().synchronize()
                    if not torch.equal(got, w):
                        wrong.append(i)
        except Exception as e:   # noqa: BLE001 - shown by the assertion
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


def test_block_tables_put_in_later():
    """The cache's table may be replaced between calls: by one as large it is used, a
    smaller one is refused before any launch."""
    B = Batch("fp8", 64, 4, 2, 16, 160, [4, 20])
    plan, x = B.plan("f32"), torch.zeros(2, 1, 2, 64, device=DEV).bfloat16()
    want = plan(B.q, B.lens_t).clone()
    old = B.cache.block_table
    B.cache.block_table = torch.cat([old, old])
    assert torch.equal(plan(B.q, B.lens_t), want)
    for bad, error in ((old[:1], ValueError), (old.long(), ValueError), (old[:, 1:], ValueError),
                       (old.cpu(), ValueError), (old[:, :4].contiguous(), kvq.KvqError)):
        B.cache.block_table = bad
        with pytest.raises(error):
            plan(B.q, B.lens_t)
        if error is ValueError:
            with pytest.raises(ValueError):
                B.cache.append_rope(runtime.Rotary(None), x, x, B.lens_t)


@pytest.mark.parametrize("gap", [12.0, 16.0, 19.0, 23.0])
@pytest.mark.parametrize("out", ["f32", "bf16", "e4m3"])
def test_a_long_flat_tail_behind_one_large_weight(gap, out):
    """One token far above 32767 equal ones, all in one split.  Bound: an absolute
    2^-32 of the largest weight for each token (the residual's step), 2048 steps of
    16 tokens that each add at most 2^-23 of the accumulator, and the exponents'."""
    B = Batch("fp8", 64, 2, 1, 128, 32768, [0, 0, 0], 3)
    q, k_scale = 1.0, float(np.float32(0.0137))
    B.q = torch.full_like(B.q, q)
    B.q64 = B.q.double()
    # scores: 64 dims of q k: the codes 0.5 everywhere and 8 at the large token
    B.codes[0].copy_(torch.tensor(0.5).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV))
    first = int(B.shared_pages[0])
    B.codes[0][first, :, 5] = torch.tensor(8.0).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
    B.codes[1].copy_(B.codes[1] & 0x7F)    # values of one sign: the tail adds up
    B.val = [c.view(torch.float8_e4m3fn).double() * float(np.float32(s)) for c, s in zip(B.codes, (0.0137, 0.0119))]
    B.sm = gap / (64 * q * 7.5 * k_scale)
    o, tol, mag = B.reference()
    vmax = float(B.val[1].abs().max())
    ref = (o, tol + 2.0 ** -12 * mag + 2.0 ** -32 * B.prefix * vmax, mag)
    o1 = run(B, out, (1, 1))
    if out == "f32":
        assert (np.abs(o1.double().cpu().numpy() - o) <= ref[1]).all()
    else:
        check_rounded(B, o1, out, ref)


@pytest.mark.parametrize("out", ["bf16", "e4m3"])
def test_the_rounded_bound_tells_one_part_from_two(out):
    """What check_rounded has to see: the same call with one f16 part fails it."""
    B = Batch("fp8", 64, 16, 2, 16, 656, [(5 * b) % 7 for b in range(40)], 11, q_std=4.0)
    ref = B.reference()
    check_rounded(B, run(B, out), out, ref)
    with pytest.raises(AssertionError):
        check_rounded(B, run(B, out, prefix_p_f16=True), out, ref)
