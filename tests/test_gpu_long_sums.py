"""Long sums of one sign in the decode of differential heads and of a packed step's single
tokens.  The matrix units cut off towards zero what does not fit an accumulator, so that
sums kept there lose ever more; fp32 sums rounded to nearest err in both directions, and
the mean over many outputs is far below the 2^-17 that is asked for."""
import pytest
import torch

from packed_ref import DEV, Packed
from quantized_kv_cache_05_gb300 import build as kbuild
from quantized_kv_cache_05_gb300 import kvq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    kbuild.build()
    kvq.lib()
    torch.cuda.init()
    torch.zeros(1, device=DEV)


def one_sign(fmt, hq, reqs, diff):
    """Values of one sign; differential heads: the second map is not subtracted."""
    X = Packed(fmt, 64, hq, 1, 64, reqs, diff=diff, norm=False, gain=1.0)
    if diff:
        X.diff.lam.zero_()
    X.codes[1] &= 0x7F if fmt == "fp8" else 0x77
    X.val[1].abs_()
    return X


def check(X, got, limit=2.0 ** -17):
    """The requests' rows: within packed_ref's bound, and on the whole."""
    o, _, _ = ref = X.reference()
    X.check(got, "f32", ref)
    rel = (got.double().cpu().numpy() - o) / o
    assert abs(rel.mean()) < limit


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("hq", [4, 8])
def test_differential_decode(fmt, hq):
    X = one_sign(fmt, hq, [(99999, 1), (70000, 1)], True)
    check(X, X.decode("f32", 1)(X.q, X.lens_t))


@pytest.mark.parametrize("diff", [False, True])
def test_single_tokens(diff):
    """Long single tokens in a batch so large that the split rule gives one chunk."""
    X = one_sign("fp8", 4, [(20000 + 7 * b, 1) for b in range(100)] + [(0, 0)] * 60, diff)
    check(X, X.run("f32"))


@pytest.mark.parametrize("diff", [False, True])
def test_two_single_tokens(diff):
    """Two of them alone count as chunks: what the header states for those."""
    X = one_sign("fp8", 4, [(99999, 1), (0, 0), (70000, 1)] + [(0, 0)] * 150, diff)
    check(X, X.run("f32"), 1.5e-5 if diff else 6e-6)
