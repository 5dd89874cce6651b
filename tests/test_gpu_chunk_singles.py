"""Single tokens of a packed step whose lengths have nothing to do with one another: the
longest are cut into shares with the chunks instead of keeping a few SMs busy."""
import pytest
import torch

from packed_ref import DEV, Packed, i32
from quantized_kv_cache_05_gb300 import build as kbuild
from quantized_kv_cache_05_gb300 import kvq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    kbuild.build()
    kvq.lib()
    torch.cuda.init()
    torch.zeros(1, device=DEV)


def as_chunks(att):
    """Requests of the last step that counted as chunks (the second word of the workspace)."""
    return int(att._ws[:8].view(torch.int32)[1])


# (tokens before, new tokens), requests that count as chunks
STEPS = [([(20000, 1)] + [(100, 1)] * 160, 1),                        # one long one among many
         ([(20000, 1)] * 2 + [(0, 0)] * 159, 2),
         ([(100, 1)] * 161, 0),
         ([(9000 + 10 * b, 1) for b in range(40)] + [(0, 0)] * 121, 40),  # on 40 of 304 places
         ([(4500, 1)] * 161, 0),                                          # long, but all of them
         ([(20000, 1), (50, 3), (100, 1)] + [(0, 0)] * 158, 2)]


@pytest.mark.parametrize("diff", [False, True])
@pytest.mark.parametrize("reqs,chunks", STEPS)
def test_long_single_tokens(reqs, chunks, diff):
    X = Packed("fp8", 64, 4, 1, 64, reqs, diff=diff)
    ref = X.reference()
    for out in ("f32", "bf16"):
        att = X.chunk(out)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        o = att(X.q, X.offs_t, X.lens_t, error_flag=err)
        X.check(o, out, ref, what=out)
        assert as_chunks(att) == chunks and int(err) == 0


def test_one_chunk_each_at_the_border():
    """161 requests of one kv head have one chunk each on 152 SMs: 4096 tokens are the
    decode's, whatever the others are, 4097 are not."""
    for n, chunks in ((4096, 0), (4097, 1)):
        X = Packed("nvfp4", 64, 4, 1, 64, [(n - 1, 1), (30, 1)] + [(0, 0)] * 159)
        att = X.chunk("f32")
        X.check(att(X.q, X.offs_t, X.lens_t), "f32")
        assert as_chunks(att) == chunks


def test_lengths_that_change_in_a_graph():
    """A captured step whose single tokens become long, and short again; the workspace is
    filled between the replays."""
    X = Packed("fp8", 64, 4, 1, 64, [(20000, 1)] + [(100, 1)] * 160)
    att = X.chunk("f32")
    lens = X.lens_t.clone()
    out = torch.zeros(X.T, 4, 64, device=DEV)
    att(X.q, X.offs_t, lens, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        att(X.q, X.offs_t, lens, out=out)
    for first, chunks in ((20001, 1), (101, 0), (20001, 1)):
        X.lens[0] = first
        lens.copy_(i32(X.lens))
        att._ws.fill_(0xFF)
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert as_chunks(att) == chunks
        X.check(out, "f32")


def test_lengths_past_the_most():
    """A clamped length is clamped for both kernels alike."""
    X = Packed("fp8", 64, 4, 1, 64, [(20000, 1)] + [(100, 1)] * 160)
    o, tol, mag = X.reference()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    lens = X.lens_t.clone()
    lens[0], lens[1] = 1 << 30, -5
    X.lens = [X.cap] + [0] + X.lens[2:]
    att = X.chunk("f32")
    got = att(X.q, X.offs_t, lens, error_flag=err)
    assert int(err) == kvq.KVQ_DEVERR_SEQ_CLAMPED and as_chunks(att) == 1
    X.check(got, "f32")
    assert (got[1] == 0).all()
