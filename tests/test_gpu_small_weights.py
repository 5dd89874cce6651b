"""What is left of small weights in the packed step's attention and the
differential decode, against 64 bits (bounds: packed_ref, and those below).

A weight enters the products with V as f16 numbers of 2^7 times itself (the row's reference,
at most its largest weight, is 1).  Two parts keep 2^-21 of it, but f16's steps end at 2^-24:
each part is off by up to 2^-25 of 2^-7, so a weight is off by 2^-31 of the row's largest at
most where that is more.  One part: 2^-11 of it, or 2^-32."""
import math

import numpy as np
import pytest
import torch

from packed_ref import DEV, Packed
from quantized_kv_cache_05_gb300 import build as kbuild
from quantized_kv_cache_05_gb300 import kvq, runtime

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    kbuild.build()
    kvq.lib()
    torch.cuda.init()
    torch.zeros(1, device=DEV)


def tail(reqs, bits, diff, lead=0.0):
    """Requests whose first token has weight 1 (and values `lead`), all others 2^-bits and
    values of one sign.  Differential heads: the second map is not subtracted (lambda 0)."""
    X = Packed("fp8", 64, 2, 1, 64, reqs, diff=diff, norm=False, gain=1.0)
    if diff:
        X.diff.lam.zero_()
    X.codes[0].zero_()
    X.val[0].zero_()
    X.codes[1] &= 0x7F
    X.val[1].abs_()
    code = lambda x: torch.tensor(x).to(torch.float8_e4m3fn).view(torch.uint8).item()
    for b, n in enumerate(X.lens):
        if n:
            page = int(X.bt[b, 0])
            for t, scale, x in ((0, 0.0137, 1.0), (1, 0.0119, lead)):
                dims = slice(0, 1) if t == 0 else slice(None)
                X.codes[t][page, 0, 0, dims] = code(x)
                X.val[t][page, 0, 0, dims] = x * float(np.float32(scale))
    X.q.zero_()
    X.q[..., 0] = 8.0
    X.q64 = X.q.double()
    X.sm = bits * math.log(2) / (8 * 0.0137)
    return X


def with_floor(X, floor):
    """The reference, its bound wider by `floor` of each token's values."""
    o, tol, mag = X.reference()
    for b, n in enumerate(X.lens):
        pages = X.bt[b, :-(-n // X.ps)].long()
        v = X.val[1][pages, 0].reshape(-1, X.D)[:n].abs().sum(0).cpu().numpy()
        tol[X.offs[b]:X.offs[b + 1]] += floor * v
    return o, tol, mag


BITS = [15.3, 20.3, 21.7, 24.4]   # (no powers of two: those are exact in f16)


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("diff", [False, True])
@pytest.mark.parametrize("reqs", [[(16383, 1)], [(16383, 1), (12000, 1)],
                                  [(4000, 1), (3500, 1)] + [(0, 0)] * 151, [(16000, 20)]])
def test_tail_of_the_packed_step(reqs, diff, bits):
    """Whatever other requests the batch has: by the chunks' kernel, or as single tokens in
    many chunks (whose own largest weights the tail's are) and in one."""
    X = tail(reqs, bits, diff)
    ref = with_floor(X, 2.0 ** -31)
    for out in ("f32", "bf16"):
        X.check(X.run(out), out, ref, what=out)


@pytest.mark.parametrize("bits", BITS)
def test_tail_with_one_part(bits):
    X = tail([(16000, 20)], bits, False)
    o, tol, mag = with_floor(X, 2.0 ** -32)
    att = runtime.ChunkAttention(X.cache, X.B, X.hq, X.cap, X.sm, out="f32", p_f16=True)
    X.check(att(X.q, X.offs_t, X.lens_t), "f32", (o, tol + 2.0 ** -11 * mag, mag))


@pytest.mark.parametrize("bits", BITS)
def test_many_small_weights_behind_one_large_one(bits):
    """The header's figure for 131072 of them, with the large one's values in the sum."""
    X = tail([(131071, 20)], bits, False, lead=0.5)
    o, tol, mag = X.reference()
    vmax = float(X.val[1].abs().max())
    X.check(X.run("f32"), "f32", (o, tol + 131072 * 2.0 ** -31 * vmax, mag))


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("splits", [None, 1])
def test_tail_of_the_differential_decode(splits, bits):
    X = tail([(16383, 1), (12000, 1)], bits, True)
    ref = with_floor(X, 2.0 ** -31)
    X.check(X.decode("f32", splits)(X.q, X.lens_t), "f32", ref)
