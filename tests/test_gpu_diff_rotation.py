"""Differential heads whose two queries and two keys are rotated each over its own half,
from the projection into the cache and to the output, in the ways that the header names."""
import numpy as np
import pytest
import torch

import rope_ref as R
from packed_ref import DEV, Packed, i32
from quantized_kv_cache_05_gb300 import build as kbuild
from quantized_kv_cache_05_gb300 import kvq, runtime
from test_gpu_plan import values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    kbuild.build()
    kvq.lib()
    torch.cuda.init()
    torch.zeros(1, device=DEV)


def turned(x, pos, table, interleaved):
    """x [tokens][heads][D] with each half turned by itself, in 64 bits: (y, magnitude)."""
    T, H, D = x.shape
    y, mag = R.turn(x.double().cpu().numpy().reshape(T, 2 * H, D // 2), None, pos.cpu().numpy(),
                    table.cpu().numpy(), D // 2, interleaved, 0.0)
    return y.reshape(T, H, D), mag.reshape(T, H, D)


def to_pairs(D):
    """Where the elements (i, i + D/4) of both halves go: (2i, 2i + 1)."""
    h = torch.arange(D // 2).view(2, D // 4).t().reshape(-1)
    return torch.cat([h, h + D // 2])


SCALES = {"fp8": (0.0137, 0.0119), "nvfp4": (0.0023, 0.0029)}


@pytest.mark.parametrize("order", ["interleaved", "halves"])
@pytest.mark.parametrize("fmt,D", [("fp8", 64), ("fp8", 128), ("nvfp4", 64), ("nvfp4", 128)])
def test_in_the_append(fmt, D, order):
    """A table that repeats its angles, interleaved; the half order with its rows permuted."""
    n, hq, hkv, ps = 50, 4, 2, 16
    g = torch.Generator(device=DEV).manual_seed(D)
    small = runtime.rope_table(512, D // 2)
    c, s = small.chunk(2, 1)
    ro = runtime.Rotary(torch.cat([c, c, s, s], 1), interleaved=True)
    q, k, v = (torch.randn(n, h, D, generator=g, device=DEV).bfloat16() for h in (hq, hkv, hkv))
    pos = torch.arange(n, device=DEV).int()
    wq, magq = turned(q, pos, small, order == "interleaved")
    wk, magk = turned(k, pos, small, order == "interleaved")
    if order == "halves":   # as a program whose projections' rows are permuted gets them
        perm = to_pairs(D)
        q, k = q[..., perm.to(DEV)].contiguous(), k[..., perm.to(DEV)].contiguous()
        wq, magq, wk, magk = (x[..., perm.numpy()] for x in (wq, magq, wk, magk))
    bt = torch.arange(1, 5).int()[None]
    cache = runtime.QuantizedKVCache(fmt, 5, ps, hkv, D, bt, *SCALES[fmt])
    qo = cache.append_slots(ro, k, v, pos.long() + ps, pos, q=q)
    R.check_bf16(qo.double().cpu().numpy(), wq, magq, "queries")
    rows = lambda x: x[1:5].transpose(1, 2).reshape(4 * ps, hkv, -1)[:n].cpu().numpy()
    if fmt == "fp8":
        R.check_grid(R.e4m3_values(rows(cache.k_codes)), wk, magk, np.float32(SCALES[fmt][0]), R.E4M3_POS, "keys")
    else:
        R.check_nvfp4(rows(cache.k_codes), rows(cache.k_bscale), wk, magk, np.float32(SCALES[fmt][0]), "keys")
    # and on to the outputs, over what the cache holds
    X = Packed(fmt, D, hq, hkv, ps, [(0, n)], diff=True)
    X.cache, X.bt, X.q, X.q64 = cache, cache.block_table, qo, qo.double()
    X.val = [values(a, b, x) for a, b, x in zip((cache.k_codes, cache.v_codes), (cache.k_bscale, cache.v_bscale),
                                                SCALES[fmt])]
    X.check(X.run("f32"), "f32")


@pytest.mark.parametrize("D", [128, 256])
def test_as_heads_of_their_own(D):
    """kvq_norm_rope over twice the heads, in the half order, then an append that turns nothing."""
    n, hq, hkv, ps = 50, 4, 2, 16
    g = torch.Generator(device=DEV).manual_seed(D)
    small = runtime.rope_table(512, D // 2)
    q, k, v = (torch.randn(n, h, D, generator=g, device=DEV).bfloat16() for h in (hq, hkv, hkv))
    pos = torch.arange(n, device=DEV).int()
    halves = lambda x: x.view(n, -1, D // 2)
    qo, ko = (x.view(n, -1, D) for x in runtime.norm_rope(runtime.Rotary(small), halves(q), halves(k), pos))
    for got, x in ((qo, q), (ko, k)):
        R.check_bf16(got.double().cpu().numpy(), *turned(x, pos, small, False))
    cache = runtime.QuantizedKVCache("nvfp4", 5, ps, hkv, D, torch.arange(1, 5).int()[None], *SCALES["nvfp4"])
    cache.append_slots(runtime.Rotary(None), ko, v, pos.long() + ps, pos)
    plain = runtime.QuantizedKVCache("nvfp4", 5, ps, hkv, D, torch.arange(1, 5).int()[None], *SCALES["nvfp4"])
    plain.append(ko[None].contiguous(), v[None].contiguous(), i32([0]))
    assert torch.equal(cache.k_codes, plain.k_codes) and torch.equal(cache.k_bscale, plain.k_bscale)
    # one token of the last position, over the cache's values
    X = Packed("nvfp4", D, hq, hkv, ps, [(n - 1, 1)], diff=True)
    X.cache, X.bt, X.q, X.q64 = cache, cache.block_table, qo[-1:].contiguous(), qo[-1:].double()
    X.cap = 4 * ps
    X.val = [values(a, b, x) for a, b, x in zip((cache.k_codes, cache.v_codes), (cache.k_bscale, cache.v_bscale),
                                                SCALES["nvfp4"])]
    X.check(X.decode("f32")(X.q, X.lens_t), "f32")
