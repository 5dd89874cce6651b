"""How many bits of the probabilities kvq_chunk_attention keeps: two f16 parts for every
output type, as the library's other attention, and one where the caller asks for it."""
import numpy as np
import pytest
import torch

import rope_ref as R
from packed_ref import DEV, OUT_SCALE, Packed, f32
from quantized_kv_cache_05_gb300 import build as kbuild
from quantized_kv_cache_05_gb300 import kvq, runtime

pytestmark = pytest.mark.gpu

REQS = [(600, 40), (300, 33), (0, 17), (77, 2)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    kbuild.build()
    kvq.lib()
    torch.cuda.init()
    torch.zeros(1, device=DEV)


def round_bf16(x):
    """The nearest bf16 value (ties to even) of each 64-bit value."""
    _, e = np.frexp(x)
    step = np.ldexp(1.0, np.maximum(e - 1, -126) - 7)
    return np.round(x / step) * step


def run(X, out, p_f16):
    att = runtime.ChunkAttention(X.cache, X.B, X.hq, X.cap, X.sm, out=out, out_scale=OUT_SCALE, p_f16=p_f16)
    return att(X.q, X.offs_t, X.lens_t)


def outside(got, out, ref):
    """Rounding is monotone: the output lies between the rounded ends of the interval of
    the fp32 result.  packed_ref's bound holds the two parts; 640 keys are 5 key tiles of 16
    accumulated products, each cut off by 2^-23 of the sum at most: 2^-16 of it."""
    o, tol, mag = ref
    tol = tol + 2.0 ** -16 * mag + 2.0 ** -21 * np.abs(o)
    if out == "bf16":
        g, lo, hi = got.double().cpu().numpy(), round_bf16(o - tol), round_bf16(o + tol)
    else:
        s = f32(OUT_SCALE)
        g = R.e4m3_values(got.cpu().numpy())
        lo, hi = R.round_value((o - tol) / s, R.E4M3_POS), R.round_value((o + tol) / s, R.E4M3_POS)
    return ~((g >= lo) & (g <= hi))


@pytest.mark.parametrize("out", ["bf16", "e4m3"])
@pytest.mark.parametrize("fmt,D", [("fp8", 64), ("fp8", 128), ("nvfp4", 64), ("nvfp4", 128)])
def test_two_f16_parts(out, fmt, D):
    """A few large weights decide each row here (some 2^-12 of a weight is what one f16
    part leaves)."""
    X = Packed(fmt, D, 16, 2, 16, REQS, 11, q_std=4.0)
    ref = X.reference()
    bad = outside(run(X, out, False), out, ref)
    assert not bad.any(), f"{bad.sum()} of {bad.size}, at {np.argwhere(bad)[0]}"


def test_the_bound_tells_one_part_from_two():
    X = Packed("fp8", 64, 16, 2, 16, REQS, 11, q_std=4.0)
    ref = X.reference()
    for out in ("bf16", "e4m3"):
        assert outside(run(X, out, True), out, ref).any()


def test_one_f16_part_where_the_caller_asks_for_it():
    """Within 2^-11 of a weight for every output type, and not the default; differential
    heads always have two."""
    for fmt, D in (("fp8", 128), ("nvfp4", 64)):
        X = Packed(fmt, D, 16, 2, 16, REQS, 11, q_std=4.0)
        o, tol, mag = X.reference()
        for out in ("f32", "bf16", "e4m3"):
            narrow = run(X, out, True)
            X.check(narrow, out, (o, tol + 2.0 ** -11 * mag, mag))
            assert not torch.equal(narrow, run(X, out, False))
    X = Packed("fp8", 128, 8, 2, 16, REQS, diff=True)
    two = X.chunk("bf16")(X.q, X.offs_t, X.lens_t)
    asked = runtime.ChunkAttention(X.cache, X.B, 8, X.cap, X.sm, diff=X.diff, p_f16=True)
    assert torch.equal(asked(X.q, X.offs_t, X.lens_t), two)


@pytest.mark.parametrize("out,p_f16", [("bf16", False), ("f32", True)])
@pytest.mark.parametrize("past", [9000, 45000])
def test_long_sums_of_one_sign(out, p_f16, past):
    """Past one chain of products in an accumulator (32 key tiles of a slot with two parts,
    64 with one): the header's 5e-5 of a sum, beside what the probabilities' parts leave."""
    X = Packed("fp8", 128, 32, 8, 48, [(past, 512)])
    X.codes[1] &= 0x7F
    X.val[1] = X.val[1].abs()
    o, tol, mag = X.reference()
    X.check(run(X, out, p_f16), out, (o, tol + 5e-5 * mag + (2.0 ** -11 * mag if p_f16 else 0), mag))
    # the roundings of P and of bf16 are unbiased, to far below this over 2 million outputs
    e = (run(X, out, p_f16).double().cpu().numpy() - o) / o
    assert abs(e.mean()) < 5e-5
