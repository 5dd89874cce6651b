"""Block tables whose rows hold 2^31 tokens and more."""
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


@pytest.mark.parametrize("width", [1 << 27, 1 << 28])
def test_wide_tables(width):
    made = [Packed("fp8", 64, 8, 2, 16, [(300, 1)]), Packed("nvfp4", 64, 8, 2, 16, [(300, 1)], diff=True),
            Packed("fp8", 64, 8, 2, 16, [(300, 40)])]
    table = torch.zeros(1, width, dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    for i, X in enumerate(made):
        ref = X.reference()
        table[:, :X.bt.shape[1]] = X.bt
        X.cache.block_table = table
        X.check(X.chunk("f32")(X.q, X.offs_t, X.lens_t, error_flag=err), "f32", ref)
        if i == 0:
            cfg = runtime.DecodeConfig(1, 8, 64, 64, 2, X.cap, X.sm, out="f32")
            X.check(runtime.decode_fused(X.cache, X.q, X.lens_t, cfg, error_flag=err), "f32", ref)
            X.check(runtime.decode(X.cache, X.q, X.lens_t, cfg, error_flag=err), "f32", ref)
        elif i == 1:
            X.check(X.decode("f32")(X.q, X.lens_t, error_flag=err), "f32", ref)
        else:
            cfg = runtime.DecodeConfig(1, 8, 64, 64, 1, X.cap, X.sm, out="f32")
            o = runtime.prefill(X.cache, X.q.view(1, 40, 8, 64), X.lens_t, cfg, 40, error_flag=err)
            X.check(o.view(40, 8, 64), "f32", ref)
    # the append into such a table, and what it wrote
    X = made[0]
    table[:, :X.bt.shape[1]] = X.bt
    row = torch.randn(1, 1, 2, 64, device=DEV).bfloat16()
    X.cache.append(row, row, X.lens_t - 1)
    page, at = int(X.bt[0, 300 // 16]), 300 % 16
    for c, s in ((X.codes[0], 0.0137), (X.codes[1], 0.0119)):
        want = (row[0, 0].float() / s).clamp(-448, 448).to(torch.float8_e4m3fn).float()
        # (the quotient's rounding may move a code by one step)
        got = c[page, :, at].view(torch.float8_e4m3fn).float()
        assert ((got - want).abs() <= want.abs() / 8 + 2.0 ** -9).all()
    assert int(err) == 0


def test_wide_table_of_latents():
    """MLA: the same decode over the same pages, whatever the table's width."""
    ps, n = 16, 200
    g = torch.Generator(device=DEV).manual_seed(1)
    bt = torch.arange(1, 1 + (n + ps - 1) // ps).int()[None]
    cache = runtime.QuantizedKVCache("nvfp4", bt.numel() + 1, ps, 1, 512, bt, 0.002, 0.002, rope_dim=64)
    lat, pe = (torch.randn(1, n, 1, d, generator=g, device=DEV).bfloat16() for d in (512, 64))
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    cache.append(lat, None, zero, pe[:, :, 0].contiguous())
    q = torch.randn(1, 16, 576, generator=g, device=DEV).bfloat16()
    lens = zero + n
    err = zero.clone()
    cfg = runtime.DecodeConfig(1, 16, 576, 512, 2, 208, 0.1, out="f32")
    want = runtime.decode_fused(cache, q, lens, cfg, error_flag=err).clone()
    codes = cache.k_codes.clone()
    assert (want != 0).any()
    for width in (1 << 27, 1 << 28):
        wide = torch.zeros(1, width, dtype=torch.int32, device=DEV)
        wide[:, :bt.shape[1]] = cache.block_table[:, :bt.shape[1]]
        cache.block_table = wide
        cache.append(lat, None, zero, pe[:, :, 0].contiguous())
        assert torch.equal(runtime.decode_fused(cache, q, lens, cfg, error_flag=err), want)
        assert torch.equal(cache.k_codes, codes)
    assert int(err) == 0
