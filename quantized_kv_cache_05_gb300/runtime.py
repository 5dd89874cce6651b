"""Device-memory plumbing around the C ABI: a paged quantized KV cache held in
torch tensors, and one decode step (partial + combine).

Marshalling only -- torch allocates memory and supplies streams; every
computation is a libkvq.so kernel.  Nothing here falls back to torch math.

A call's ``stream`` (default: the current one) is where its kernels run, and nothing
more: what another stream still writes of the inputs, the cache or the scratch has to
be waited for first (``wait_stream``), and a tensor of another stream's memory has to
be kept, or marked with ``record_stream``, until the given one is done with it.  That
holds for the scratch too, which its object zeroes on the stream that is current when
it is made.
"""
from __future__ import annotations

import ctypes
import dataclasses
from typing import Optional

import torch

from . import kvq

FMT = {"fp8": kvq.KVQ_FP8_E4M3, "nvfp4": kvq.KVQ_NVFP4}
OUT = {"f32": kvq.KVQ_OUT_F32, "bf16": kvq.KVQ_OUT_BF16, "e4m3": kvq.KVQ_OUT_E4M3}
MAX_SPLITS = 64   # partials of a row that a call joins (kvq_decode_params)
OUT_TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.uint8}


def rope_table(num_positions: int, rot_dim: int, base: float = 10000.0,
               device: str | torch.device = "cuda") -> torch.Tensor:
    """Rotation table of ``kvq_rotary`` (fp32 [num_positions][rot_dim]: cosines, then
    sines) for the angles position * base^(-2i / rot_dim), formed in 64 bits."""
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device)
    ang = torch.arange(num_positions, dtype=torch.float64, device=device)[:, None] * \
        base ** (-i / rot_dim)
    return torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()


_call = None


def _calls():
    """The marshalling module, bound to the loaded library.  A missing one raises."""
    global _call
    if _call is None:
        L = kvq.lib()
        try:
            from . import _kvq_call as m
        except ImportError as e:
            raise RuntimeError("the _kvq_call module is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`") from e
        ptr = lambda f: ctypes.cast(f, ctypes.c_void_p).value
        m.bind(ptr(L.kvq_norm_rope), ptr(L.kvq_rope_append), ptr(L.kvq_decode_shared),
               torch.bfloat16, torch.uint8, torch.int32, torch.float32)
        _call = m
    return _call


def _check(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _here(t: torch.Tensor, dtype: torch.dtype, what: str) -> None:
    """A CUDA tensor of the current device (kernels launch there) and this type."""
    if t.dtype != dtype or not t.is_cuda or t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{what}: expected {dtype} on cuda:{torch.cuda.current_device()}, got "
                         f"{t.dtype} on {t.device}")


def _launch_device(*held: int) -> int:
    """The current device, on which the kernels launch: what an object holds (-1:
    nothing) has to be there."""
    dev = torch.cuda.current_device()
    for d in held:
        if d != dev and d != -1:
            raise ValueError(f"made on cuda:{d}, called with cuda:{dev} current")
    return dev


class Rotary:
    """The norm and rotation of a layer's queries and keys (``kvq_rotary``): the
    table of ``rope_table`` (None: no rotation) and the norms' weights (float32
    [head_dim] each; None: no norm).  It keeps these tensors, whose addresses its
    struct holds; others need a Rotary of their own."""

    def __init__(self, table: Optional[torch.Tensor], interleaved: bool = False,
                 q_norm: Optional[torch.Tensor] = None, k_norm: Optional[torch.Tensor] = None,
                 eps: float = 1e-6):
        for t, what in ((table, "table"), (q_norm, "q_norm"), (k_norm, "k_norm")):
            if t is not None:
                _here(t, torch.float32, what)
                _check(t.is_contiguous(), f"{what}: expected a contiguous tensor")
        _check(table is None or table.dim() == 2, "table: expected [positions][rot_dim]")
        self._tensors = table, q_norm, k_norm
        r = self._struct = kvq.kvq_rotary()
        if table is not None:
            r.cos_sin, r.num_positions, r.rot_dim = table.data_ptr(), *table.shape
        r.interleaved = 1 if interleaved else 0
        r.q_norm = q_norm.data_ptr() if q_norm is not None else None
        r.k_norm = k_norm.data_ptr() if k_norm is not None else None
        r.eps = eps
        # for the calls: the struct's address, the norms' lengths (-1: none); the
        # device that the tensors are on
        self._args = (ctypes.addressof(r), -1 if q_norm is None else q_norm.numel(),
                      -1 if k_norm is None else k_norm.numel())
        held = [t for t in (table, q_norm, k_norm) if t is not None]
        self.device = held[0].get_device() if held else -1

    # read-only: a tensor put in their place would leave the struct with the address of
    # one that is gone
    table = property(lambda self: self._tensors[0])
    q_norm = property(lambda self: self._tensors[1])
    k_norm = property(lambda self: self._tensors[2])

    def struct(self) -> kvq.kvq_rotary:
        return self._struct


def _rows_like(t: torch.Tensor, dtype: torch.dtype, stream) -> torch.Tensor:
    """A dense tensor of t's shape for a kernel on `stream` to write: from that stream's
    memory, since work that the current one has yet to do may use what it freed."""
    if stream is not None and kvq._stream(stream) != torch.cuda.current_stream().cuda_stream:
        with torch.cuda.stream(torch.cuda.ExternalStream(kvq._stream(stream))):
            return torch.empty_like(t, dtype=dtype, memory_format=torch.contiguous_format)
    return torch.empty_like(t, dtype=dtype, memory_format=torch.contiguous_format)


def _query_out(q: torch.Tensor, out: Optional[torch.Tensor], kind: str, stream) -> torch.Tensor:
    if kind not in OUT_TORCH or kind == "f32":
        raise ValueError("q_out_type: bf16 or e4m3")
    if out is None:
        return _rows_like(q, OUT_TORCH[kind], stream)
    if out.numel() != q.numel() or out.shape[-2:] != q.shape[-2:]:
        raise ValueError("q_out: expected q's shape")
    return out


def _with(t: torch.Tensor, dtype: torch.dtype, device: torch.device, what: str) -> None:
    """A tensor of this type on the device of the object that keeps it."""
    if t.dtype != dtype or t.device != device:
        raise ValueError(f"{what}: expected {dtype} on {device}, got {t.dtype} on {t.device}")


def _head_scale(t: Optional[torch.Tensor], heads: int,
                device: torch.device) -> Optional[torch.Tensor]:
    if t is not None:
        _with(t, torch.float32, device, "q_head_scale")
        _check(t.numel() == heads and t.is_contiguous(), "q_head_scale: one scale per query head")
    return t


def norm_rope(rotary: Rotary, q: Optional[torch.Tensor], k: Optional[torch.Tensor],
              positions: Optional[torch.Tensor], q_out: Optional[torch.Tensor] = None,
              k_out: Optional[torch.Tensor] = None, q_out_type: str = "bf16",
              q_scale: float = 1.0, q_head_scale: Optional[torch.Tensor] = None,
              error_flag: Optional[torch.Tensor] = None, stream=None):
    """Norm and rotation of queries and keys (kvq_norm_rope): q bf16 [T][Hq][D] and k
    bf16 [T][Hk][D], positions int32 [T].  Returns (q_out, k_out): new tensors, or the
    given ones (bf16 outputs may be the inputs).  q_out_type "e4m3": uint8 codes.
    New tensors belong to the stream that is given; inputs do not (see the top)."""
    if q is not None:
        q_out = _query_out(q, q_out, q_out_type, stream)
    if k is not None and k_out is None:
        k_out = _rows_like(k, k.dtype, stream)
    dev = _launch_device(rotary.device)
    addr, nq, nk = rotary._args
    st = (_call or _calls()).norm_rope(dev, kvq._stream(stream), addr, nq, nk,
                                       q, k, positions, q_out, k_out, q_out_type == "e4m3", q_scale,
                                       q_head_scale, error_flag)
    if st:
        kvq.check(st, "kvq_norm_rope")
    return q_out, k_out


class QuantizedKVCache:
    """Paged FP8 / NVFP4 KV cache (layout of ``kvq_cache`` in include/kvq.h).

    codes  uint8 [num_pages][Hkv][page_size][row]   row = D (FP8) or D/2 (NVFP4)
    bscale uint8 [num_pages][Hkv][page_size][D/16]  (NVFP4)
    k_pe   bf16  [num_pages][page_size][rope]       (MLA; V is the latent)
    """

    def __init__(self, fmt: str, num_pages: int, page_size: int, num_kv_heads: int,
                 head_dim: int, block_table: torch.Tensor, k_scale: float, v_scale: float,
                 rope_dim: int = 0, device: str | torch.device = "cuda",
                 k_head_scale: Optional[torch.Tensor] = None,
                 v_head_scale: Optional[torch.Tensor] = None):
        self.fmt = fmt
        self.num_pages, self.page_size = num_pages, page_size
        self.Hkv, self.D, self.rope = num_kv_heads, head_dim, rope_dim
        self.k_scale, self.v_scale = float(k_scale), float(v_scale)
        row = head_dim if fmt == "fp8" else head_dim // 2
        shape = (num_pages, num_kv_heads, page_size, row)
        self.k_codes = torch.zeros(shape, dtype=torch.uint8, device=device)
        self.v_codes = None if rope_dim else torch.zeros(shape, dtype=torch.uint8, device=device)
        self.k_bscale = self.v_bscale = None
        if fmt == "nvfp4":
            sshape = (num_pages, num_kv_heads, page_size, head_dim // 16)
            self.k_bscale = torch.zeros(sshape, dtype=torch.uint8, device=device)
            if not rope_dim:
                self.v_bscale = torch.zeros(sshape, dtype=torch.uint8, device=device)
        self.k_pe = (torch.zeros((num_pages, page_size, rope_dim), dtype=torch.bfloat16,
                                 device=device) if rope_dim else None)
        self.block_table = block_table.to(device=device, dtype=torch.int32).contiguous()
        # per-kv-head scales (float32 [Hkv] on the device), replacing k_scale / v_scale
        def _hs(t):
            if t is None:
                return None
            t = t.to(device=device, dtype=torch.float32).contiguous()
            assert t.numel() == num_kv_heads, "one scale per kv head"
            return t
        self.k_head_scale, self.v_head_scale = _hs(k_head_scale), _hs(v_head_scale)

    @classmethod
    def wrap(cls, fmt: str, k_codes: torch.Tensor, v_codes: torch.Tensor,
             block_table: torch.Tensor, k_scale: float, v_scale: float,
             k_bscale: Optional[torch.Tensor] = None, v_bscale: Optional[torch.Tensor] = None,
             k_head_scale: Optional[torch.Tensor] = None,
             v_head_scale: Optional[torch.Tensor] = None) -> "QuantizedKVCache":
        """A cache over tensors that the caller holds (K and V in the layout above;
        not MLA): nothing is allocated or copied."""
        _check(k_codes.dim() == 4 and k_codes.shape == v_codes.shape,
               "codes: expected [pages][kv heads][page size][row], K as V")
        pages, hkv, ps, row = k_codes.shape
        D = row if fmt == "fp8" else 2 * row
        arrays = [(k_codes, "k_codes"), (v_codes, "v_codes")]
        if fmt == "nvfp4":
            arrays += [(k_bscale, "k_bscale"), (v_bscale, "v_bscale")]
            for t in (k_bscale, v_bscale):
                _check(t is not None and t.shape == (pages, hkv, ps, D // 16),
                       "bscale: expected [pages][kv heads][page size][head_dim / 16]")
        for t, what in arrays:
            _here(t, torch.uint8, what)
            _check(t.is_contiguous(), f"{what}: expected a contiguous tensor")
        _here(block_table, torch.int32, "block_table")
        _check(block_table.dim() == 2 and block_table.is_contiguous(),
               "block_table: expected a contiguous [batch][pages]")
        for t in (k_head_scale, v_head_scale):
            if t is not None:
                _here(t, torch.float32, "head scales")
                _check(t.numel() == hkv and t.is_contiguous(), "head scales: one per kv head")
        self = cls.__new__(cls)
        self.fmt, self.num_pages, self.page_size = fmt, pages, ps
        self.Hkv, self.D, self.rope = hkv, D, 0
        self.k_scale, self.v_scale = float(k_scale), float(v_scale)
        self.k_codes, self.v_codes, self.k_pe = k_codes, v_codes, None
        self.k_bscale, self.v_bscale = k_bscale, v_bscale
        self.block_table = block_table
        self.k_head_scale, self.v_head_scale = k_head_scale, v_head_scale
        return self

    @property
    def mla(self) -> bool:
        return self.rope > 0

    @property
    def max_pages_per_seq(self) -> int:
        return self.block_table.shape[1]

    def struct(self) -> kvq.kvq_cache:
        # in the order of kvq_cache's fields
        ptr = lambda t: None if t is None else t.data_ptr()
        return kvq.kvq_cache(
            FMT[self.fmt], self.num_pages, self.page_size, self.Hkv, self.D, ptr(self.k_codes),
            ptr(self.v_codes), ptr(self.k_bscale), ptr(self.v_bscale), self.k_scale, self.v_scale,
            ptr(self.block_table), self.max_pages_per_seq, self.rope, ptr(self.k_pe),
            1 if self.mla else 0, ptr(self.k_head_scale), ptr(self.v_head_scale))

    def append(self, k_new: torch.Tensor, v_new: Optional[torch.Tensor],
               start_pos: torch.Tensor, kpe_new: Optional[torch.Tensor] = None,
               stream=None) -> None:
        """k_new/v_new bf16 [B][T][Hkv][D]; start_pos int32 [B] (device)."""
        B, T = k_new.shape[0], k_new.shape[1]
        kvq.check(kvq.kvq_quantize_append(self.struct(), k_new, v_new, kpe_new, start_pos, B, T,
                                          stream), "kvq_quantize_append")

    def append_rope(self, rotary: Rotary, k_new: torch.Tensor, v_new: Optional[torch.Tensor],
                    start_pos: torch.Tensor, kpe_new: Optional[torch.Tensor] = None,
                    new_lens: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                    q_out: Optional[torch.Tensor] = None, q_out_type: Optional[str] = None,
                    q_scale: float = 1.0, q_head_scale: Optional[torch.Tensor] = None,
                    error_flag: Optional[torch.Tensor] = None,
                    stream=None) -> Optional[torch.Tensor]:
        """Append with the keys' norm and rotation, and the queries' in the same launch
        (kvq_rope_append): k_new/v_new bf16 [B][T][Hkv][D], q bf16 [B][T][Hq][D], all of
        them strided as a packed projection's slices are; start_pos int32 [B]; new_lens
        int32 [B] or None (all T).  MLA: k_new the latents [B][T][1][512], kpe_new
        [B][T][1][64].  Returns q_out (q_out_type "bf16", or "e4m3": uint8 codes; by
        default q_out's own type, bf16 without one).  On a given stream: the result belongs
        to it, the inputs do not (see the top)."""
        fp8 = False
        if q is not None:
            kind = q_out_type or ("e4m3" if q_out is not None and q_out.dtype == torch.uint8 else "bf16")
            q_out = _query_out(q, q_out, kind, stream)
            fp8 = kind == "e4m3"
        dev = _launch_device(rotary.device, self.k_codes.get_device())
        call = _call or _calls()
        call.block_table(dev, self.block_table, 0)   # (it may be another one than at the start)
        c = self.struct()
        addr, nq, nk = rotary._args
        st = call.rope_append(
            dev, kvq._stream(stream), ctypes.addressof(c),
            self.block_table.shape[0], addr, nq, nk, k_new, v_new, kpe_new, start_pos, new_lens, q,
            q_out, fp8, q_scale, q_head_scale, error_flag)
        if st:
            kvq.check(st, "kvq_rope_append")
        return q_out


@dataclasses.dataclass
class DecodeConfig:
    batch: int
    num_q_heads: int
    qk_dim: int
    v_dim: int
    num_splits: int
    max_kv_len: int
    sm_scale: float
    prob_scale: float = 0.0
    out: str = "f32"
    out_scale: float = 1.0
    # > 0: the call right before on the stream is the append of the last
    # fresh_tokens positions, and the decode overlaps with it (kvq_decode_params)
    fresh_tokens: int = 0
    # FP8 query: q holds E4M3 codes, dequantized with q_scale or the per-head
    # q_head_scale tensor (float32 [num_q_heads] on the device)
    q_fp8: bool = False
    q_scale: float = 1.0
    q_head_scale: Optional[torch.Tensor] = None
    # SharedDecode: the prefix's probabilities in one f16 instead of two
    # (kvq_decode_params)
    prefix_p_f16: bool = False

    def params(self, seq_lens: Optional[torch.Tensor], error_flag: Optional[torch.Tensor] = None
               ) -> kvq.kvq_decode_params:
        # in the order of kvq_decode_params' fields
        ptr = lambda t: None if t is None else t.data_ptr()
        return kvq.kvq_decode_params(
            self.batch, self.num_q_heads, self.qk_dim, self.v_dim, self.num_splits,
            ptr(seq_lens), self.max_kv_len, self.sm_scale, self.prob_scale, OUT[self.out],
            self.out_scale, ptr(error_flag), self.fresh_tokens, 1 if self.q_fp8 else 0, self.q_scale,
            ptr(self.q_head_scale), 1 if self.prefix_p_f16 else 0)


class DecodeWorkspace:
    """Split partials for one decode configuration (caller-owned scratch)."""

    def __init__(self, cfg: DecodeConfig, device="cuda"):
        rows = cfg.batch * cfg.num_q_heads * cfg.num_splits
        self.part_o = torch.empty(rows * cfg.v_dim, dtype=torch.float32, device=device)
        self.part_lse = torch.empty(rows, dtype=torch.float32, device=device)
        self.out = torch.empty((cfg.batch, cfg.num_q_heads, cfg.v_dim), dtype=OUT_TORCH[cfg.out],
                               device=device)


class FusedWorkspace(DecodeWorkspace):
    """Scratch of kvq_decode: split partials plus arrival counters, which are
    zeroed once here; every call leaves them at zero again."""

    def __init__(self, cfg: DecodeConfig, num_kv_heads: int, device="cuda"):
        super().__init__(cfg, device)
        self.counters = torch.zeros(cfg.batch * num_kv_heads, dtype=torch.int32, device=device)


def decode_fused(cache: QuantizedKVCache, q: torch.Tensor, seq_lens: torch.Tensor,
                 cfg: DecodeConfig, ws: Optional[FusedWorkspace] = None,
                 error_flag: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One decode step in one launch (kvq_decode)."""
    ws = ws or FusedWorkspace(cfg, cache.Hkv, q.device)
    p = cfg.params(seq_lens, error_flag)
    kvq.check(kvq.kvq_decode(cache.struct(), p, q, ws.part_o, ws.part_lse, ws.counters, ws.out,
                             stream), "kvq_decode")
    return ws.out


def auto_splits(batch: int, num_kv_heads: int, q_per_kv: int, max_kv_len: int, fmt: str,
                device: int | None = None) -> int:
    if device is None:
        device = torch.cuda.current_device()
    sms = torch.cuda.get_device_properties(device).multi_processor_count
    st, s = kvq.kvq_auto_splits(sms, batch, num_kv_heads, q_per_kv, max_kv_len, FMT[fmt])
    kvq.check(st, "kvq_auto_splits")
    return s


def decode(cache: QuantizedKVCache, q: torch.Tensor, seq_lens: torch.Tensor, cfg: DecodeConfig,
           ws: Optional[DecodeWorkspace] = None, error_flag: Optional[torch.Tensor] = None,
           stream=None) -> torch.Tensor:
    """One decode step: kvq_decode_partial then kvq_decode_combine."""
    ws = ws or DecodeWorkspace(cfg, q.device)
    p = cfg.params(seq_lens, error_flag)
    c = cache.struct()
    kvq.check(kvq.kvq_decode_partial(c, p, q, ws.part_o, ws.part_lse, stream),
              "kvq_decode_partial")
    kvq.check(kvq.kvq_decode_combine(p, ws.part_o, ws.part_lse, ws.out, stream),
              "kvq_decode_combine")
    return ws.out


def prefill(cache: QuantizedKVCache, q: torch.Tensor, seq_lens: torch.Tensor, cfg: DecodeConfig,
            q_len: int, out: Optional[torch.Tensor] = None,
            error_flag: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Causal prefill attention of q_len new tokens per request (kvq_prefill):
    q bf16 [batch][q_len][Hq][D] -> out [batch][q_len][Hq][D]."""
    if out is None:
        out = torch.empty((cfg.batch, q_len, cfg.num_q_heads, cfg.v_dim), dtype=OUT_TORCH[cfg.out],
                          device=q.device)
    p = cfg.params(seq_lens, error_flag)
    kvq.check(kvq.kvq_prefill(cache.struct(), p, q_len, q, out, stream), "kvq_prefill")
    return out


class SharedDecode:
    """Decode steps of a batch whose requests share their first prefix_len tokens
    (kvq_decode_shared): the configuration and its scratch, kept between steps.
    Steps of one object must not overlap on the GPU (they share the scratch).  What it
    is made with stays as it is: another configuration needs an object of its own."""

    def __init__(self, cache: QuantizedKVCache, batch: int, num_q_heads: int, prefix_len: int,
                 max_kv_len: int, sm_scale: float, out: str = "bf16", out_scale: float = 1.0,
                 q_fp8: bool = False, q_scale: float = 1.0,
                 q_head_scale: Optional[torch.Tensor] = None,
                 prefix_table: Optional[torch.Tensor] = None,
                 splits: Optional[tuple[int, int]] = None, prefix_p_f16: bool = False):
        """prefix_table: the shared pages (int32; default: the first entries of the first
        request that is at least prefix_len long); splits: (prefix, own) chunks, by
        default kvq_shared_splits'; prefix_p_f16: the prefix's probabilities with 11 bits
        instead of 22, for bf16 outputs that need not be kvq_decode's to the last step."""
        _check(0 <= prefix_len <= max_kv_len, "prefix_len: expected 0 .. max_kv_len")
        _check(batch <= cache.block_table.shape[0], "more requests than the block table has")
        _check(num_q_heads % cache.Hkv == 0, "num_q_heads: a multiple of the kv heads")
        device = cache.k_codes.device
        if prefix_table is not None:
            _with(prefix_table, torch.int32, device, "prefix_table")
            _check(prefix_table.is_contiguous() and
                   prefix_table.numel() * cache.page_size >= prefix_len,
                   "prefix_table: one page per page_size shared tokens")
        if splits is None:
            sms = torch.cuda.get_device_properties(device).multi_processor_count
            st, sp, so = kvq.kvq_shared_splits(sms, max(batch, 1), cache.Hkv,
                                               num_q_heads // cache.Hkv, prefix_len,
                                               max_kv_len - prefix_len, FMT[cache.fmt])
            kvq.check(st, "kvq_shared_splits")
        else:
            sp, so = splits
            _check(sp >= 1 and so >= 1, "splits: at least one of the prefix and one of the own tokens")
            if prefix_len > 0:   # as the call lowers them
                sp = min(sp, (prefix_len + 127) // 128)
                if sp + so > MAX_SPLITS:
                    raise kvq.KvqError(kvq.KVQ_ERR_UNSUPPORTED, "SharedDecode: splits")
        self._cache, self._prefix = cache, (prefix_len, prefix_table, sp)
        cfg = self._cfg = DecodeConfig(batch, num_q_heads, cache.D, cache.D, so, max_kv_len, sm_scale,
                                      out=out, out_scale=out_scale, q_fp8=q_fp8, q_scale=q_scale,
                                      q_head_scale=_head_scale(q_head_scale, num_q_heads, device),
                                      prefix_p_f16=prefix_p_f16)
        # the call's own checks, without requests: what no step could do is refused here
        # (without any request a step does nothing)
        if batch > 0:
            none = dataclasses.replace(cfg, batch=0).params(None)
            kvq.check(kvq.kvq_decode_shared(cache.struct(), none, prefix_len, None, sp, None, None, None,
                                            None, None, 0), "SharedDecode")
        self._ws = FusedWorkspace(dataclasses.replace(cfg, num_splits=so + sp), cache.Hkv, device)
        self._params = cfg.params(None)   # the lengths and the flag come with each step

    # read-only, and the configuration as a copy: the parameters and the scratch were
    # made for these
    cache = property(lambda self: self._cache)
    prefix_len = property(lambda self: self._prefix[0])
    prefix_table = property(lambda self: self._prefix[1])
    prefix_splits = property(lambda self: self._prefix[2])
    ws = property(lambda self: self._ws)
    cfg = property(lambda self: dataclasses.replace(self._cfg))

    def __call__(self, q: torch.Tensor, seq_lens: torch.Tensor,
                 error_flag: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """q bf16 (FP8 query: uint8) [batch][Hq][D], seq_lens int32 [batch] (whole lengths)
        -> the output buffer [batch][Hq][D], overwritten by the next step.  On a given
        stream: ordered behind the object's making and kept as said at the top."""
        ws, cache = self._ws, self._cache
        prefix_len, prefix_table, prefix_splits = self._prefix
        dev = _launch_device(cache.k_codes.get_device())
        call = _call or _calls()
        call.block_table(dev, cache.block_table, self._cfg.batch)   # (as in append_rope)
        c = cache.struct()
        st = call.decode_shared(
            dev, kvq._stream(stream), ctypes.addressof(c),
            ctypes.addressof(self._params), prefix_len, prefix_table, prefix_splits, q,
            seq_lens, ws.part_o, ws.part_lse, ws.counters, ws.out, error_flag)
        if st:
            kvq.check(st, "kvq_decode_shared")
        return ws.out
