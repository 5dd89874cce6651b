"""Packed steps and differential heads from their formulas in 64 bits, with the bounds
that the fp32 kernels' results must keep.

Bounds.  With A = sum_j softmax_j |v_j| per output: a weight's relative error is that of
its exponent -- the score's fp32 accumulation, at most (D / 8) 2^-23 of sum_d |q_d k_d|
sm_scale (16 products per step, each step's sum rounded at worst by one unit of 2^-23,
twice that for split accumulators), the exponent's own rounding, below 2^-22 of its
magnitude (at most 2^5 here: 2^-17) -- and 2^-22 each of the exponential and of P in two
f16 parts, or 2^-11 of P in one.  Numerator and denominator both carry the former.  Sums
of up to 2^13 terms in fp32 add 2^-20 (partials are short, the errors' signs random).
    e = A (2 (E + 2^-17 + 2^-21) + 2^-20)  [+ 2^-11 A with P in one part]
Differential heads: o = o1 - lambda o2 is off by e1 + |lambda| e2 and its own roundings,
2^-22 (|o1| + |lambda o2|).  The norm's sum of D <= 256 squares is at most 64 adds in a
lane and 8 more, all of positive terms, 72 u with u = 2^-24, halved by the root; root,
quotient, mean, products are 8 u more: 2^-18 covers them.  With M = mean o^2 + eps the
errors of o move the root by mean(|o| e + e^2) / M at most (relative), so
    y = gain w o / sqrt(M):  |w gain| e / sqrt(M) + |y| (mean(|o| e + e^2) / M + 2^-18).
The output's own rounding is half a step: bf16 2^-8 of the value; an E4M3 code lies
between those of the interval's ends.
"""
import math

import numpy as np
import torch

import rope_ref as R
from quantized_kv_cache_05_gb300 import runtime

DEV = "cuda"
OUT_SCALE = 0.004


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def f32(x):
    """The fp32 number that a call gets."""
    return float(np.float32(x))


class Packed:
    """A cache whose request b holds past + new tokens (`reqs`: pairs), the new ones rows
    of a packed step, and queries for them.  diff: differential heads; norm: with weights."""

    def __init__(self, fmt, D, hq, hkv, ps, reqs, seed=1, q_fp8=False, head_scales=False, q_std=1.0,
                 diff=False, norm=True, k_ramp=None, extra_pages=1, gain=0.3, eps=1e-5):
        g = self.g = torch.Generator(device=DEV).manual_seed(seed)
        self.fmt, self.D, self.hq, self.hkv, self.ps, self.reqs = fmt, D, hq, hkv, ps, reqs
        self.B, self.G = len(reqs), hq // hkv
        self.lens, self.new = [p + n for p, n in reqs], [n for _, n in reqs]
        need = [-(-n // ps) for n in self.lens]
        per = max(1, max(need, default=1))
        pages = sum(need) + extra_pages
        perm = torch.randperm(pages - extra_pages, generator=g, device=DEV).int() + extra_pages
        self.bt = torch.zeros(max(self.B, 1), per, dtype=torch.int32, device=DEV)
        at = 0
        for b, n in enumerate(need):
            self.bt[b, :n] = perm[at:at + n]
            at += n
        self.cap = per * ps
        x = [torch.randn(pages, hkv, ps, D, generator=g, device=DEV) for _ in range(2)]
        if k_ramp is not None:   # scores that grow or shrink along each request's tokens
            for b, n in enumerate(need):
                for i, page in enumerate(self.bt[b, :n].tolist()):
                    t = i * ps + torch.arange(ps, device=DEV)
                    x[0][page] *= (k_ramp[0] + (k_ramp[1] - k_ramp[0]) * t / max(self.lens[b], 1))[None, :, None]
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
        self.cache = runtime.QuantizedKVCache.wrap(fmt, *self.codes, self.bt, *sc, *self.bscale, *hs)
        self.lens_t = i32(self.lens)
        self.offs = np.concatenate([[0], np.cumsum(self.new)]).astype(int)
        self.offs_t = i32(self.offs.tolist())
        self.T = int(self.offs[-1])
        q = torch.randn(self.T, hq, D, generator=g, device=DEV) * q_std
        self.q_fp8, self.q_scale = q_fp8, 0.017
        if q_fp8:
            c = (q / self.q_scale).clamp(-448, 448).to(torch.float8_e4m3fn)
            self.q, self.q64 = c.view(torch.uint8), c.double() * f32(self.q_scale)
        else:
            self.q = q.bfloat16()
            self.q64 = self.q.double()
        self.sm = 1 / math.sqrt(D // 2 if diff else D)
        self.diff = None
        if diff:
            lam = torch.rand(hq, generator=g, device=DEV) * 1.2 - 0.2
            w = 1 + 0.3 * torch.randn(D, generator=g, device=DEV) if norm else None
            self.diff = runtime.Differential(lam, norm=w, eps=eps, gain=gain)
            self.gain, self.eps = gain, eps

    # ------------------------------------------------------------- reference
    def _sums(self, q, k, v, hidden, sm, dims):
        """(o, bound without P's rounding, A) of one softmax map."""
        s = (q @ k.T * sm).masked_fill(hidden, -math.inf)
        p = torch.softmax(s, 1)
        p = torch.where(hidden.all(1, keepdim=True), torch.zeros_like(p), p)
        A = p @ v.abs()
        eps = (q.abs() @ k.abs().T * sm).amax(1, keepdim=True) * (dims / 8) * 2.0 ** -23
        eps = eps + 2.0 ** -17 + 2.0 ** -21
        return p @ v, A * (2 * eps + 2.0 ** -20), A

    def reference(self, only=None):
        """(output, bound before the output's rounding, magnitude for P's rounding)."""
        sm, G, D = f32(self.sm), self.G, self.D
        out = torch.zeros(self.T, self.hq, D, dtype=torch.float64, device=DEV)
        tol, mag = out.clone(), out.clone()
        for b, (L, n) in enumerate(zip(self.lens, self.new)):
            if not n or L <= 0 or (only is not None and b not in only):
                continue
            pg = self.bt[b, :-(-L // self.ps)].long()
            last = (L - n + torch.arange(n, device=DEV)).repeat_interleave(G)
            hidden = torch.arange(L, device=DEV)[None] > last[:, None]
            rows = slice(int(self.offs[b]), int(self.offs[b + 1]))
            for h in range(self.hkv):
                k, v = (x[pg, h].reshape(-1, D)[:L] for x in self.val)
                hs = slice(h * G, (h + 1) * G)
                q = self.q64[rows, hs].reshape(n * G, D)
                if self.diff is None:
                    o, e, A = self._sums(q, k, v, hidden, sm, D)
                else:
                    o, e = self._diff(q, k, v, hidden, sm, self.diff.lam.double()[hs].repeat(n)[:, None])
                    A = torch.zeros_like(o)
                for to, x in ((out, o), (tol, e), (mag, A)):
                    to[rows, hs] = x.reshape(n, G, D)
        return out.cpu().numpy(), tol.cpu().numpy(), mag.cpu().numpy()

    def _diff(self, q, k, v, hidden, sm, lam):
        d = self.D // 2
        o1, e1, _ = self._sums(q[:, :d], k[:, :d], v, hidden, sm, d)
        o2, e2, _ = self._sums(q[:, d:], k[:, d:], v, hidden, sm, d)
        o = o1 - lam * o2
        e = e1 + lam.abs() * e2 + 2.0 ** -22 * (o1.abs() + (lam * o2).abs())
        gain = f32(self.gain)
        if self.diff.norm is None:
            return gain * o, abs(gain) * (e + 2.0 ** -23 * o.abs())
        w = self.diff.norm.double() * gain
        M = (o * o).mean(1, keepdim=True) + f32(self.eps)
        live = M > 0
        M = torch.where(live, M, torch.ones_like(M))
        y = w * o / M.sqrt()
        move = (o.abs() * e + e * e).mean(1, keepdim=True) / M + 2.0 ** -18
        return y, w.abs() * e / M.sqrt() + y.abs() * move

    # ----------------------------------------------------------------- calls
    def chunk(self, out="f32", max_len=None):
        return runtime.ChunkAttention(self.cache, self.B, self.hq, max_len or self.cap, self.sm, out=out,
                                      out_scale=OUT_SCALE, q_fp8=self.q_fp8, q_scale=self.q_scale,
                                      diff=self.diff)

    def decode(self, out="f32", splits=None, **kw):
        return runtime.DiffDecode(self.cache, self.B, self.hq, self.cap, self.sm, self.diff, out=out,
                                  out_scale=OUT_SCALE, q_fp8=self.q_fp8, q_scale=self.q_scale,
                                  splits=splits, **kw)

    def run(self, out="f32", flag=0):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        o = self.chunk(out)(self.q, self.offs_t, self.lens_t, error_flag=err)
        torch.cuda.synchronize()
        assert int(err) == flag
        return o

    def check(self, got, out, ref=None, rows=None, what=""):
        o, tol, mag = ref if ref is not None else self.reference()
        if out != "f32" and self.diff is None:
            tol = tol + 2.0 ** -11 * mag
        if rows is not None:
            o, tol, got = o[rows], tol[rows], got[rows]
        g = got.double().cpu().numpy() if out != "e4m3" else R.e4m3_values(got.cpu().numpy())
        if out == "e4m3":
            s = f32(OUT_SCALE)
            lo, hi = (o - tol) / s, (o + tol) / s   # (the quotient's rounding: 2^-24 of it)
            bad = ~((g >= R.round_value(lo - 2.0 ** -23 * np.abs(lo), R.E4M3_POS)) &
                    (g <= R.round_value(hi + 2.0 ** -23 * np.abs(hi), R.E4M3_POS)))
        else:
            lim = tol + (np.abs(o) + tol) * (2.0 ** -8 if out == "bf16" else 2.0 ** -23)
            bad = ~(np.abs(g - o) <= lim)
        assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, worst "
                               f"{np.nanmax(np.abs(g - o)) if out != 'e4m3' else 'code'}, at {np.argwhere(bad)[0]}")
