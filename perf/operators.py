"""The workloads of the serving operators that surround the quantized decode:
per-head norms with the position rotation, the rotating quantize-on-append, and
decode attention over a prefix that the whole batch shares.

A case is a dict of sizes and options; ``prepare`` makes what a serving program
holds before the call, ``run`` makes one call -- the plain torch form, or with
``own`` set the library's kernels through ``quantized_kv_cache_05_gb300.runtime``
-- and ``exact`` gives the same outputs from the definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _rope(name, tokens, hq, hk, dim, rot, inter, norm, fp8):
    return dict(name=name, op="norm_rope", tokens=tokens, hq=hq, hk=hk, dim=dim, rot=rot,
                inter=inter, norm=norm, fp8=fp8)


def _append(name, batch, tokens, hq, hkv, dim, rot, inter, norm, fp8q, page, past, ragged):
    return dict(name=name, op="append", batch=batch, tokens=tokens, hq=hq, hkv=hkv, dim=dim,
                rot=rot, inter=inter, norm=norm, fp8q=fp8q, page=page, past=past, ragged=ragged)


def _shared(name, batch, hq, hkv, dim, fmt, page, prefix, tail, idle, qfp8, out):
    return dict(name=name, op="shared", batch=batch, hq=hq, hkv=hkv, dim=dim, fmt=fmt, page=page,
                prefix=prefix, tail=tail, idle=idle, qfp8=qfp8, out=out)


def listed():
    return [
        # one decode step of 64 requests: latency
        _rope("rope step 64", 64, 32, 8, 128, 128, False, True, False),
        # a prefill chunk: bandwidth
        _rope("rope chunk 8192", 8192, 32, 8, 128, 128, False, True, False),
        # an odd packed batch, half of each head rotated, pairs side by side,
        # queries as E4M3 codes for the FP8-query decode
        _rope("rope odd 1003 fp8", 1003, 14, 2, 64, 32, True, False, True),
        # one decode step of 48 requests: queries, keys and values in one call
        _append("append step 48", 48, 1, 32, 8, 128, 128, False, True, False, 16, 900, False),
        # the padded prefill chunks of four requests, their lengths ragged
        _append("append chunk 4x2048", 4, 2048, 32, 8, 128, 128, False, True, False, 16, 700, True),
        # odd sizes: three kv heads, pages that are no power of two, FP8 queries
        _append("append odd 7x113", 7, 113, 12, 3, 64, 64, True, False, True, 48, 333, False),
        # a few requests behind a short system prompt: latency
        _shared("shared 4 x 1k", 4, 32, 8, 128, "fp8", 16, 1024, 60, 0, False, "bf16"),
        # an ordinary batch behind a long system prompt
        _shared("shared 16 x 8k", 16, 32, 8, 128, "fp8", 16, 8192, 512, 0, False, "bf16"),
        # NVFP4, a prefix that ends inside a tile, two idle rows of a padded batch
        _shared("shared nvfp4 48 x 16k", 48, 32, 8, 128, "nvfp4", 16, 16400, 300, 2, False, "bf16"),
        # seven queries per kv head, FP8 queries, fp32 output
        _shared("shared odd 13 x 4080", 13, 14, 2, 64, "fp8", 48, 4080, 77, 0, True, "f32"),
        # many requests about one long document
        _shared("shared 64 x 32k", 64, 32, 8, 128, "fp8", 64, 32768, 1024, 0, False, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _drawn(rng):
    op = rng.choice(["norm_rope", "append", "shared"])
    dim = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 8])
    hq = hkv * rng.choice([1, 3, 4, 7, 8])
    rot = dim if rng.random() < 0.6 else dim // 2
    inter, norm, fp8 = rng.random() < 0.4, rng.random() < 0.6, rng.random() < 0.4
    page = rng.choice([16, 16, 32, 48, 64])
    if op == "norm_rope":
        c = _rope("", _log(rng, 1, 8192), hq, hkv, dim, rot, inter, norm, fp8)
    elif op == "append":
        batch = _log(rng, 1, 64)
        tokens = _log(rng, 1, max(1, 8192 // batch))
        c = _append("", batch, tokens, hq, hkv, dim, rot, inter, norm, fp8, page,
                    rng.randrange(0, 900), tokens > 1 and rng.random() < 0.5)
    else:
        batch = _log(rng, 1, 96)
        prefix = max(1, _log(rng, 256, 40000) // page) * page
        out = rng.choice(["bf16", "bf16", "f32", "e4m3"])
        c = _shared("", batch, hq, hkv, dim, rng.choice(["fp8", "nvfp4"]), page, prefix,
                    _log(rng, 1, 1024), rng.choice([0, 0, min(1, batch - 1)]), fp8, out)
    del c["name"]
    return c


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        c = _drawn(rng)
        if _cost(c) <= most:
            return c


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def work(case):
    c = case
    if c["op"] == "norm_rope":
        t, heads = c["tokens"], c["hq"] + c["hk"]
        b = t * heads * c["dim"] * 2 + t * c["dim"] * (c["hq"] * (1 if c["fp8"] else 2) + c["hk"] * 2)
        return {"bytes": b + t * (4 * c["rot"] + 4), "flops": t * heads * (3 * c["rot"] + 4 * c["dim"])}
    if c["op"] == "append":
        t = c["batch"] * c["tokens"] * (0.5 if c["ragged"] else 1.0)
        rows = t * c["dim"]
        b = rows * (c["hq"] + 2 * c["hkv"]) * 2 + rows * (c["hq"] * (1 if c["fp8q"] else 2) + 2 * c["hkv"])
        heads = c["hq"] + c["hkv"]
        return {"bytes": b + t * 4 * c["rot"] + 8 * c["batch"],
                "flops": t * heads * (3 * c["rot"] + 4 * c["dim"]) + 2 * rows * c["hkv"]}
    live = c["batch"] - c["idle"]
    row = c["dim"] if c["fmt"] == "fp8" else c["dim"] // 2 + c["dim"] // 16
    tokens = c["prefix"] + live * (c["tail"] + 1) / 2
    seen = live * (c["prefix"] + (c["tail"] + 1) / 2)
    outb = {"f32": 4, "bf16": 2, "e4m3": 1}[c["out"]]
    io = c["batch"] * c["hq"] * c["dim"] * ((1 if c["qfp8"] else 2) + outb)
    return {"bytes": 2 * tokens * c["hkv"] * row + io + 4 * tokens / c["page"],
            "flops": 4 * seen * c["hq"] * c["dim"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _table(rows, rot):
    """cos and sin of every position's rot / 2 angles, base 10000, made in 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    ang = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def _codes_fp8(x, scale):
    return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _codes_nvfp4(x, scale):
    """x [..., D] -> packed E2M1 codes [..., D/2] and E4M3 block scales [..., D/16]."""
    blk = x.reshape(*x.shape[:-1], -1, 16)
    sc = (blk.abs().amax(-1) / 6 / scale).clamp(max=448).to(torch.float8_e4m3fn)
    es = (sc.float() * scale)[..., None]
    y = torch.where(es > 0, blk / es.clamp(min=1e-30), torch.zeros_like(blk))
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    code = torch.bucketize(y.abs(), edges).to(torch.uint8) | ((y < 0).to(torch.uint8) << 3)
    code = code.reshape(*x.shape[:-1], -1, 2)
    return (code[..., 0] | (code[..., 1] << 4)).contiguous(), sc.view(torch.uint8)


def _heads(x, first, n, dim):
    """Heads first .. first + n - 1 of the packed projection x [tokens][heads * dim]: a view."""
    return x[:, first * dim:(first + n) * dim].unflatten(1, (n, dim))


def _prepare_rope(c, g, s):
    t, hq, hk, d = c["tokens"], c["hq"], c["hk"], c["dim"]
    rows = 40960
    s["table"] = _table(rows, c["rot"])
    s["x"] = (torch.randn(t, (hq + hk) * d, generator=g, device=DEV) * 1.5).bfloat16()
    s["q"], s["k"] = _heads(s["x"], 0, hq, d), _heads(s["x"], hq, hk, d)
    start = int(torch.randint(0, rows - t, (1,), generator=g, device=DEV))
    s["pos"] = (start + torch.arange(t, device=DEV)).int()
    if c["norm"]:
        s["qw"] = 1 + 0.2 * torch.randn(d, generator=g, device=DEV)
        s["kw"] = 1 + 0.2 * torch.randn(d, generator=g, device=DEV)
    s["q_scale"] = torch.tensor(9.1372 / 448, device=DEV)


def _prepare_append(c, g, s):
    b, t, hq, hkv, d, ps = c["batch"], c["tokens"], c["hq"], c["hkv"], c["dim"], c["page"]
    n = b * t
    s["table"] = _table(16384, c["rot"])
    s["x"] = (torch.randn(n, (hq + 2 * hkv) * d, generator=g, device=DEV) * 1.5).bfloat16()
    s["q"], s["k"] = _heads(s["x"], 0, hq, d), _heads(s["x"], hq, hkv, d)
    s["v"] = _heads(s["x"], hq + hkv, hkv, d)
    if c["norm"]:
        s["qw"] = 1 + 0.2 * torch.randn(d, generator=g, device=DEV)
        s["kw"] = 1 + 0.2 * torch.randn(d, generator=g, device=DEV)
    per = (c["past"] + t + ps - 1) // ps
    s["bt"] = torch.randperm(b * per, generator=g, device=DEV).int().reshape(b, per)
    s["start"] = torch.randint(0, c["past"] + 1, (b,), generator=g, device=DEV).int()
    lens = torch.full((b,), t, device=DEV)
    if c["ragged"]:
        lens = torch.randint(0, t + 1, (b,), generator=g, device=DEV)
    s["lens"] = lens.int()
    # the real tokens of the padded batch, and the request of each
    s["valid"] = (torch.arange(t, device=DEV) < lens[:, None]).reshape(-1).nonzero()[:, 0]
    # a cache in use: what is not written has to stay
    shape = (b * per, hkv, ps, d)
    for name in ("kc", "vc"):
        s[name] = _codes_fp8(torch.randn(shape, generator=g, device=DEV), 0.02)
    # static scales as a calibration gives them: the largest magnitude seen / 448
    s["k_scale"], s["v_scale"] = torch.tensor(9.1372 / 448, device=DEV), torch.tensor(6.8419 / 448, device=DEV)
    s["q_scale"] = torch.tensor(9.1372 / 448, device=DEV)
    s["q_out"] = torch.zeros(n, hq, d, device=DEV, dtype=torch.uint8 if c["fp8q"] else torch.bfloat16)


def _prepare_shared(c, g, s):
    b, hq, hkv, d, ps = c["batch"], c["hq"], c["hkv"], c["dim"], c["page"]
    pre, per = c["prefix"] // ps, (c["tail"] + ps - 1) // ps
    pages = pre + b * per
    perm = torch.randperm(pages, generator=g, device=DEV).int()
    s["bt"] = torch.cat([perm[:pre].expand(b, pre), perm[pre:].reshape(b, per)], 1).contiguous()
    lens = c["prefix"] + torch.randint(1, c["tail"] + 1, (b,), generator=g, device=DEV)
    if c["idle"]:
        lens[b - c["idle"]:] = 0
    s["lens"] = lens.int()
    shape = (pages, hkv, ps, d)
    s["k_scale"], s["v_scale"] = (0.0125, 0.011) if c["fmt"] == "fp8" else (0.0021, 0.0019)
    for name in "kv":
        x = torch.randn(shape, generator=g, device=DEV)
        if c["fmt"] == "fp8":
            s[name + "c"] = _codes_fp8(x, s[name + "_scale"])
        else:
            s[name + "c"], s[name + "b"] = _codes_nvfp4(x, s[name + "_scale"])
    q = torch.randn(b, hq, d, generator=g, device=DEV) * 1.5
    s["q_scale"] = 0.02
    s["q"] = _codes_fp8(q, s["q_scale"]) if c["qfp8"] else q.bfloat16()
    s["sm_scale"], s["out_scale"] = 1 / math.sqrt(d), 0.004


def prepare(case, seed):
    g, s = _gen(seed), {"case": case}
    {"norm_rope": _prepare_rope, "append": _prepare_append, "shared": _prepare_shared}[case["op"]](case, g, s)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _norm_rotate(x, w, cos_sin, c):
    """x [tokens][heads][dim] in fp32: RMS norm of each head, then the rotation."""
    if w is not None:
        x = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w
    rot = c["rot"]
    cos, sin = cos_sin[:, None, :rot // 2], cos_sin[:, None, rot // 2:]
    r = x[..., :rot]
    if c["inter"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, x[..., rot:]], -1)


def _to_e4m3(x, scale):
    return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn)


def _plain_rope(s, c):
    cs = s["table"][s["pos"].long()]
    q = _norm_rotate(s["q"].float(), s.get("qw"), cs, c)
    k = _norm_rotate(s["k"].float(), s.get("kw"), cs, c)
    return {"q": _to_e4m3(q, s["q_scale"]) if c["fp8"] else q.bfloat16(), "k": k.bfloat16()}


def _plain_append(s, c):
    at = s["valid"]
    b, t = at // c["tokens"], at % c["tokens"]
    pos = s["start"].long()[b] + t
    cs = s["table"][pos]
    q = _norm_rotate(s["q"][at].float(), s.get("qw"), cs, c)
    k = _norm_rotate(s["k"][at].float(), s.get("kw"), cs, c)
    page, off = s["bt"].long()[b, pos // c["page"]], pos % c["page"]
    s["kc"][page, :, off] = _to_e4m3(k, s["k_scale"]).view(torch.uint8)
    s["vc"][page, :, off] = _to_e4m3(s["v"][at].float(), s["v_scale"]).view(torch.uint8)
    s["q_out"][at] = _to_e4m3(q, s["q_scale"]).view(torch.uint8) if c["fp8q"] else q.bfloat16()
    return _append_outputs(s, c)


def _append_outputs(s, c):
    e4m3 = torch.float8_e4m3fn
    return {"k": s["kc"].view(e4m3), "v": s["vc"].view(e4m3),
            "q": s["q_out"].view(e4m3) if c["fp8q"] else s["q_out"]}


def _values(s, name, pages, c):
    """The cached values of some pages in fp32: [..., kv heads, page size, dim]."""
    codes = s[name + "c"][pages]
    if c["fmt"] == "fp8":
        return codes.view(torch.float8_e4m3fn).float() * s[name + "_scale"]
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
    x = grid[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]
    sc = s[name + "b"][pages].view(torch.float8_e4m3fn).float() * s[name + "_scale"]
    return (x.unflatten(-1, (-1, 16)) * sc[..., None]).flatten(-2)


def _plain_shared(s, c):
    b, hq, hkv, d, ps = c["batch"], c["hq"], c["hkv"], c["dim"], c["page"]
    grp, pre = hq // hkv, c["prefix"] // ps
    q = s["q"].view(torch.float8_e4m3fn).float() * s["q_scale"] if c["qfp8"] else s["q"].float()
    q = q.reshape(b, hkv, grp, d) * s["sm_scale"]
    table, lens = s["bt"].long(), s["lens"].long()
    # the shared pages, once for every request
    first = table[0, :pre]
    k1 = _values(s, "k", first, c).transpose(0, 1).reshape(hkv, -1, d)
    v1 = _values(s, "v", first, c).transpose(0, 1).reshape(hkv, -1, d)
    # each request's own pages
    k2 = _values(s, "k", table[:, pre:], c).transpose(1, 2).reshape(b, hkv, -1, d)
    v2 = _values(s, "v", table[:, pre:], c).transpose(1, 2).reshape(b, hkv, -1, d)
    rows = q.transpose(0, 1).reshape(hkv, b * grp, d)
    s1 = (rows @ k1.transpose(1, 2)).reshape(hkv, b, grp, -1)
    s2 = (q @ k2.transpose(2, 3)).transpose(0, 1)
    at1, at2 = torch.arange(s1.shape[-1], device=DEV), torch.arange(s2.shape[-1], device=DEV)
    s1 = s1.masked_fill((at1 >= lens[:, None])[None, :, None], -math.inf)
    s2 = s2.masked_fill((at2 >= lens[:, None] - c["prefix"])[None, :, None], -math.inf)
    top = torch.maximum(s1.amax(-1, keepdim=True), s2.amax(-1, keepdim=True))
    top = top.masked_fill(top == -math.inf, 0.0)
    p1, p2 = (s1 - top).exp(), (s2 - top).exp()
    total = p1.sum(-1, keepdim=True) + p2.sum(-1, keepdim=True)
    o = (p1.reshape(hkv, b * grp, -1) @ v1).reshape(hkv, b, grp, d)
    o = o + (p2.transpose(0, 1) @ v2).transpose(0, 1)
    o = torch.where(total > 0, o / total, torch.zeros_like(o)).transpose(0, 1).reshape(b, hq, d)
    if c["out"] == "f32":
        return o
    return o.bfloat16() if c["out"] == "bf16" else _to_e4m3(o, torch.tensor(s["out_scale"], device=DEV))


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _handle(s, c):
    """What a serving program keeps beside its buffers: made on a state's first pass."""
    if "handle" not in s:
        from quantized_kv_cache_05_gb300 import runtime
        h = s["handle"] = {"rt": runtime}
        if c["op"] != "shared":
            h["rotary"] = runtime.Rotary(s["table"], interleaved=c["inter"], q_norm=s.get("qw"),
                                         k_norm=s.get("kw"), eps=EPS)
        if c["op"] == "append":
            h["cache"] = runtime.QuantizedKVCache.wrap("fp8", s["kc"], s["vc"], s["bt"], float(s["k_scale"]),
                                                       float(s["v_scale"]))
            h["shape"] = (c["batch"], c["tokens"])
        if c["op"] != "shared":
            h["q_scale"] = float(s["q_scale"])
        if c["op"] == "shared":
            h["cache"] = runtime.QuantizedKVCache.wrap(c["fmt"], s["kc"], s["vc"], s["bt"], s["k_scale"],
                                                       s["v_scale"], s.get("kb"), s.get("vb"))
            h["plan"] = runtime.SharedDecode(h["cache"], c["batch"], c["hq"], c["prefix"],
                                             c["prefix"] + c["tail"], s["sm_scale"], out=c["out"],
                                             out_scale=s["out_scale"], q_fp8=c["qfp8"], q_scale=s["q_scale"])
    return s["handle"]


def _own(s, c):
    h = _handle(s, c)
    if c["op"] == "norm_rope":
        q, k = h["rt"].norm_rope(h["rotary"], s["q"], s["k"], s["pos"],
                                 q_out_type="e4m3" if c["fp8"] else "bf16", q_scale=h["q_scale"])
        return {"q": q.view(torch.float8_e4m3fn) if c["fp8"] else q, "k": k}
    if c["op"] == "append":
        h["cache"].append_rope(h["rotary"], s["k"].unflatten(0, h["shape"]), s["v"].unflatten(0, h["shape"]),
                               s["start"], new_lens=s["lens"] if c["ragged"] else None,
                               q=s["q"].unflatten(0, h["shape"]), q_out=s["q_out"], q_scale=h["q_scale"])
        return _append_outputs(s, c)
    o = h["plan"](s["q"], s["lens"])
    return o.view(torch.float8_e4m3fn) if c["out"] == "e4m3" else o


def run(state):
    c = state["case"]
    if own:
        return _own(state, c)
    return {"norm_rope": _plain_rope, "append": _plain_append, "shared": _plain_shared}[c["op"]](state, c)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _e4m3_64(x):
    """The nearest E4M3 value (ties to even, saturating) of each 64-bit value."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return ((x / step).round() * step).clamp(-448, 448)


def _turn_64(x, w, pos, table, c):
    x = x.double()
    if w is not None:
        x = x * torch.rsqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
    half = c["rot"] // 2
    ang = torch.complex(table[pos][:, :half].double(), table[pos][:, half:].double())[:, None]
    i = torch.arange(half, device=DEV)
    lo, hi = (2 * i, 2 * i + 1) if c["inter"] else (i, i + half)
    z = torch.complex(x[..., lo], x[..., hi]) * ang
    y = x.clone()
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def _exact_rope(s, c):
    pos = s["pos"].long()
    q = _turn_64(s["q"], s.get("qw"), pos, s["table"], c)
    return {"q": _e4m3_64(q / s["q_scale"].double()) if c["fp8"] else q,
            "k": _turn_64(s["k"], s.get("kw"), pos, s["table"], c)}


def _exact_append(s, c):
    d = c["dim"]
    out = {n: s[n + "c"].view(torch.float8_e4m3fn).double() for n in "kv"}
    out["q"] = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["lens"].tolist()):
        at = slice(b * c["tokens"], b * c["tokens"] + n)
        pos = int(s["start"][b]) + torch.arange(n, device=DEV)
        slot = s["bt"][b].long()[pos // c["page"]] * c["page"] + pos % c["page"]
        rows = {"k": _turn_64(s["k"][at], s.get("kw"), pos, s["table"], c), "v": s["v"][at].double()}
        for name, x in rows.items():
            flat = out[name].transpose(1, 2).reshape(-1, c["hkv"], d)
            flat[slot] = _e4m3_64(x / s[name + "_scale"].double())
            out[name] = flat.reshape(-1, c["page"], c["hkv"], d).transpose(1, 2).contiguous()
        q = _turn_64(s["q"][at], s.get("qw"), pos, s["table"], c)
        out["q"][at] = _e4m3_64(q / s["q_scale"].double()) if c["fp8q"] else q
    return out


def _cached_64(s, name, h, pages, c):
    if c["fmt"] == "fp8":
        x = s[name + "c"][pages, h].view(torch.float8_e4m3fn).double()
    else:
        codes = s[name + "c"][pages, h].long()
        x = torch.empty(*codes.shape[:-1], c["dim"], dtype=torch.float64, device=DEV)
        grid = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
        for k in (0, 1):
            nib = (codes >> (4 * k)) & 15
            x[..., k::2] = grid[nib & 7] * (1.0 - 2.0 * (nib >> 3))
        x = x * s[name + "b"][pages, h].view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)
    return x.reshape(-1, c["dim"]) * s[name + "_scale"]


def _exact_shared(s, c):
    grp, pre = c["hq"] // c["hkv"], c["prefix"] // c["page"]
    q = s["q"].view(torch.float8_e4m3fn).double() * s["q_scale"] if c["qfp8"] else s["q"].double()
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lens, table = s["lens"].tolist(), s["bt"].long()
    for h in range(c["hkv"]):
        hs = slice(h * grp, (h + 1) * grp)
        k1, v1 = (_cached_64(s, n, h, table[0, :pre], c) for n in "kv")
        for b, n in enumerate(lens):
            if not n:
                continue
            k2, v2 = (_cached_64(s, m, h, table[b, pre:], c)[:n - c["prefix"]] for m in "kv")
            x = torch.cat([q[b, hs] @ k1.T, q[b, hs] @ k2.T], 1) * s["sm_scale"]
            out[b, hs] = torch.softmax(x, 1) @ torch.cat([v1, v2])
    if c["out"] == "e4m3":
        # the scale that the call gets is an fp32 number
        return _e4m3_64(out / float(torch.tensor(s["out_scale"])))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"norm_rope": _exact_rope, "append": _exact_append, "shared": _exact_shared}[case["op"]](s, case)
