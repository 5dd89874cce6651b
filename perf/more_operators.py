"""The workloads of the packed serving step over the paged quantised cache: the block
tables, slots and positions of a step's new tokens, planned from request lengths; the
append of packed rows into those slots; causal attention of a ragged batch of prompt
chunks and single tokens over the FP8 or NVFP4 cache; and differential attention (the
difference of two softmax maps) for single tokens and for chunks.

A case is a dict of sizes and options; ``prepare`` makes what a serving program holds
before the call, ``run`` makes one call -- the plain torch form, or with ``own`` set the
library's kernels through ``quantized_kv_cache_05_gb300.runtime`` -- and ``exact`` gives
the same outputs from the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6
DROP_ALL = -2 ** 31


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _plan(name, batch, page, past, single, chunk, done, padding):
    return dict(name=name, op="plan", batch=batch, page=page, past=past, single=single,
                chunk=chunk, done=done, padding=padding)


def _slots(name, tokens, padding, hq, hkv, dim, page, rot, inter, norm, fp8q):
    return dict(name=name, op="slots", tokens=tokens, padding=padding, hq=hq, hkv=hkv, dim=dim,
                fmt="fp8", page=page, rot=rot, inter=inter, norm=norm, fp8q=fp8q)


def _chunk(name, batch, single, chunk, past, hq, hkv, dim, fmt, page, qfp8, out, diff=False):
    return dict(name=name, op="chunk", batch=batch, single=single, chunk=chunk, past=past, hq=hq,
                hkv=hkv, dim=dim, fmt=fmt, page=page, qfp8=qfp8, out=out, diff=diff, norm=diff)


def _diff(name, batch, length, hq, hkv, dim, fmt, page, qfp8, out, norm):
    return dict(name=name, op="diff", batch=batch, length=length, hq=hq, hkv=hkv, dim=dim, fmt=fmt,
                page=page, qfp8=qfp8, out=out, norm=norm)


def listed():
    return [
        # a decode step of 256 requests, some of them starting a page: latency
        _plan("plan step 256", 256, 16, 900, 256, 0, 0, 0),
        # a large step: finished requests give their pages back, others bring prompts
        _plan("plan mixed 1500", 1500, 16, 2000, 1100, 900, 100, 1000),
        # the rows of a decode step, padded to a captured size: latency
        _slots("slots step 61", 64, 3, 32, 8, 128, 16, 128, False, True, False),
        # a packed step of prompt chunks: bandwidth
        _slots("slots 8000", 8000, 0, 32, 8, 128, 16, 128, False, True, False),
        # a small mixed step over a 4-bit cache: four single tokens and two short chunks
        _chunk("chunk small mixed nvfp4", 6, 4, 100, 900, 32, 8, 128, "nvfp4", 16, False, "bf16"),
        # an ordinary step: prompts of some requests beside single tokens of others
        _chunk("chunk 4 + 28 nvfp4", 32, 28, 700, 4000, 32, 8, 128, "nvfp4", 16, False, "bf16"),
        # odd sizes: seven query heads per kv head, FP8 queries, pages that are no power of two
        _chunk("chunk odd fp8 f32", 5, 1, 333, 1777, 14, 2, 64, "fp8", 48, True, "f32"),
        # a chunk of a long prompt: the tensor cores
        _chunk("chunk 4096 behind 12k", 1, 0, 4096, 12288, 32, 8, 128, "fp8", 64, False, "bf16"),
        # one token each of a few requests, differential heads: latency
        _diff("diff step 4 x 1k", 4, 1024, 16, 4, 128, "fp8", 16, False, "bf16", True),
        # an ordinary decode step of differential heads on a 4-bit cache
        _diff("diff step 48 x 8k nvfp4", 48, 8192, 32, 8, 128, "nvfp4", 16, False, "bf16", True),
        # differential heads of 32 + 32, fp32 output, in a ragged step
        _chunk("diff chunk odd", 9, 5, 211, 1500, 12, 3, 64, "fp8", 48, False, "f32", True),
        # prompt chunks of differential heads over a 4-bit cache
        _chunk("diff chunk 4 x 1024 nvfp4", 4, 0, 1024, 4096, 32, 8, 128, "nvfp4", 16, False,
               "bf16", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _drawn(rng):
    op = rng.choice(["plan", "slots", "chunk", "diff", "chunk"])
    dim = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 8])
    page = rng.choice([16, 16, 32, 48, 64])
    fmt = rng.choice(["fp8", "nvfp4"])
    qfp8 = rng.random() < 0.25
    out = rng.choice(["bf16", "bf16", "f32", "e4m3"])
    if op == "plan":
        batch = _log(rng, 1, 4000)
        single, done = int(batch * rng.random()), 0
        if batch > 2:
            done = int((batch - single) * rng.random() * 0.5)
        c = _plan("", batch, page, _log(rng, 1, 2000), single, _log(rng, 1, 900), done,
                  rng.choice([0, 0, 7, 1000]))
    elif op == "slots":
        rot = dim if rng.random() < 0.6 else dim // 2
        c = _slots("", _log(rng, 1, 8000), 0, hkv * rng.choice([1, 3, 4, 7, 8]), hkv, dim, page,
                   rot, rng.random() < 0.4, rng.random() < 0.6, qfp8)
        c["padding"] = int(c["tokens"] * rng.random() * 0.2)
    elif op == "chunk":
        batch = _log(rng, 1, 32)
        diff = rng.random() < 0.5
        c = _chunk("", batch, int(batch * rng.random()), _log(rng, 1, 4096), _log(rng, 1, 12288),
                   hkv * rng.choice([1, 2, 4, 7, 8]), hkv, dim, fmt, page, qfp8, out, diff)
        c["norm"] = diff and rng.random() < 0.7
    else:
        c = _diff("", _log(rng, 1, 64), _log(rng, 1, 16384), hkv * rng.choice([1, 2, 3, 4, 8]), hkv,
                  dim, fmt, page, qfp8, out, rng.random() < 0.7)
    del c["name"]
    return c


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        c = _drawn(rng)
        if _cost(c) <= most and (c["op"] != "plan" or sum(_plan_adds(c)) <= 200000):
            return c


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 280)


def _sizes(c):
    """A case's generator of request sizes: the same for every seed of the inputs."""
    return random.Random("/".join(str(c[k]) for k in sorted(c) if k != "name"))


def _lens(c):
    """(tokens held before, new tokens) of each request of a chunk case; (length, 1) of a
    differential decode step's."""
    rng = _sizes(c)
    if c["op"] == "diff":
        return [(rng.randint((c["length"] + 1) // 2, c["length"]), 1) for _ in range(c["batch"])]
    kinds = [1] * c["single"] + [0] * (c["batch"] - c["single"])
    rng.shuffle(kinds)
    one = c["batch"] - c["single"] == 1   # a chunk by itself has the sizes that are given
    size = lambda most: most if one else rng.randint((most + 1) // 2, most)
    return [(rng.randint((c["past"] + 1) // 2, c["past"]), 1) if k else (size(c["past"]), size(c["chunk"]))
            for k in kinds]


def _plan_olds(c):
    rng = _sizes(c)
    return [rng.randint(0, c["past"]) for _ in range(c["batch"])]


def _plan_adds(c):
    """New tokens of each request of a plan case (below zero: tokens that go)."""
    rng = _sizes(c)
    adds = [1] * c["single"] + [DROP_ALL] * c["done"]
    rest = c["batch"] - len(adds)
    # prompts' chunks; some requests wait, some take a few rejected tokens back
    adds += [rng.choice([c["chunk"], rng.randint(0, c["chunk"]), 0, -rng.randint(0, 5)])
             for _ in range(rest)]
    rng.shuffle(adds)
    return adds


def _plan_tokens(c):
    return max(1, sum(max(a, 0) for a in _plan_adds(c)) + c["padding"])


def _row_bytes(c):
    return c["dim"] if c["fmt"] == "fp8" else c["dim"] // 2 + c["dim"] // 16


def work(case):
    c = case
    if c["op"] == "plan":
        pages = 0
        for old, add in zip(_plan_olds(c), _plan_adds(c)):
            pages += abs(-(-max(old + add, 0) // c["page"]) + -old // c["page"])
        # lengths and changes in, lengths, starts and offsets out; pages moved; slots, positions
        return {"bytes": 20 * c["batch"] + 8 * pages + 12 * _plan_tokens(c), "flops": 0}
    if c["op"] == "slots":
        t, rows = c["tokens"], (c["tokens"] - c["padding"]) * c["dim"]
        b = rows * (c["hq"] + 2 * c["hkv"]) * 2 + rows * c["hq"] * (1 if c["fp8q"] else 2)
        b += 2 * (c["tokens"] - c["padding"]) * c["hkv"] * _row_bytes(c)
        heads = c["hq"] + c["hkv"]
        return {"bytes": b + t * (4 * c["rot"] + 12),
                "flops": t * heads * (3 * c["rot"] + 4 * c["dim"]) + 2 * rows * c["hkv"]}
    lens = _lens(c)
    diff = c["op"] == "diff" or c["diff"]
    outb = {"f32": 4, "bf16": 2, "e4m3": 1}[c["out"]]
    total = [p if c["op"] == "diff" else p + n for p, n in lens]
    new = sum(n for _, n in lens)
    io = new * c["hq"] * c["dim"] * ((1 if c["qfp8"] else 2) + outb)
    # keys that each new token sees: the held ones and, of the new, those up to itself
    seen = sum(t * n - n * (n - 1) // 2 for t, (_, n) in zip(total, lens))
    # two maps of half the dims and their values, or one map
    per = 6 * c["dim"] if diff else 4 * c["dim"]
    return {"bytes": 2 * sum(total) * c["hkv"] * _row_bytes(c) + io + 4 * sum(total) / c["page"],
            "flops": per * seen * c["hq"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


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


def _prepare_plan(c, g, s):
    olds, adds = _plan_olds(c), _plan_adds(c)
    held = [-(-n // c["page"]) for n in olds]
    want = [-(-max(n + a, 0) // c["page"]) for n, a in zip(olds, adds)]
    width = max(max(held), max(want), 1) + 1
    spare = sum(max(w - h, 0) for w, h in zip(want, held)) + 5
    pages = sum(held) + spare
    perm = torch.randperm(pages, generator=g, device=DEV).int()
    table = torch.full((c["batch"], width), -1, dtype=torch.int32, device=DEV)
    row = torch.repeat_interleave(torch.arange(c["batch"]), torch.tensor(held))
    col = torch.arange(sum(held)) - torch.repeat_interleave(
        torch.tensor([0] + held[:-1]).cumsum(0), torch.tensor(held))
    table[row.to(DEV), col.to(DEV)] = perm[spare:]
    s["bt"], s["pages"] = table, pages
    s["free"] = torch.full((pages,), -1, dtype=torch.int32, device=DEV)
    s["free"][:spare] = perm[:spare]
    s["count"], s["count_out"] = _i32([spare]), _i32([0])
    s["lens"], s["lens_out"], s["adds"] = _i32(olds), _i32([0] * c["batch"]), _i32(adds)
    s["max_tokens"] = _plan_tokens(c)


def _table(rows, rot):
    """cos and sin of every position's rot / 2 angles, base 10000, made in 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    ang = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def _heads(x, first, n, dim):
    """Heads first .. first + n - 1 of the packed projection x [tokens][heads * dim]: a view."""
    return x[:, first * dim:(first + n) * dim].unflatten(1, (n, dim))


def _cache(c, g, s, pages):
    """A cache in use: codes of normal values."""
    shape = (pages, c["hkv"], c["page"], c["dim"])
    s["k_scale"], s["v_scale"] = (0.0125, 0.011) if c["fmt"] == "fp8" else (0.0021, 0.0019)
    for name in "kv":
        x = torch.randn(shape, generator=g, device=DEV)
        if c["fmt"] == "fp8":
            s[name + "c"] = _codes_fp8(x, s[name + "_scale"])
        else:
            s[name + "c"], s[name + "b"] = _codes_nvfp4(x, s[name + "_scale"])


def _prepare_slots(c, g, s):
    t, hq, hkv, d, ps = c["tokens"], c["hq"], c["hkv"], c["dim"], c["page"]
    s["table"] = _table(16384, c["rot"])
    s["x"] = (torch.randn(t, (hq + 2 * hkv) * d, generator=g, device=DEV) * 1.5).bfloat16()
    s["q"], s["k"] = _heads(s["x"], 0, hq, d), _heads(s["x"], hq, hkv, d)
    s["v"] = _heads(s["x"], hq + hkv, hkv, d)
    if c["norm"]:
        s["qw"] = 1 + 0.2 * torch.randn(d, generator=g, device=DEV)
        s["kw"] = 1 + 0.2 * torch.randn(d, generator=g, device=DEV)
    live = t - c["padding"]
    pages = (2 * t + ps - 1) // ps
    _cache(c, g, s, pages)
    slots = torch.full((t,), -1, dtype=torch.int64, device=DEV)
    slots[:live] = torch.randperm(pages * ps, generator=g, device=DEV)[:live]
    pos = torch.full((t,), -1, dtype=torch.int32, device=DEV)
    pos[:live] = torch.randint(0, 16384, (live,), generator=g, device=DEV).int()
    s["slots"], s["pos"] = slots, pos
    s["bt"] = _i32([[0]])
    s["q_scale"] = 9.1372 / 448
    # static scales as a calibration gives them: the largest magnitude seen / 448
    s["k_scale"], s["v_scale"] = 9.1372 / 448, 6.8419 / 448
    s["q_out"] = torch.zeros(t, hq, d, device=DEV, dtype=torch.uint8 if c["fp8q"] else torch.bfloat16)


def _prepare_attention(c, g, s):
    hq, d, ps = c["hq"], c["dim"], c["page"]
    lens = _lens(c)
    s["total"] = [p if c["op"] == "diff" else p + n for p, n in lens]
    s["new"] = [n for _, n in lens]
    need = [-(-n // ps) for n in s["total"]]
    width = max(need)
    perm = torch.randperm(sum(need), generator=g, device=DEV).int()
    table = torch.zeros(c["batch"], width, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    s["bt"], s["lens"] = table, _i32(s["total"])
    s["offsets"] = _i32([0] + np.cumsum(s["new"]).tolist())
    _cache(c, g, s, sum(need))
    q = torch.randn(sum(s["new"]), hq, d, generator=g, device=DEV) * 1.5
    s["q_scale"] = 0.02
    s["q"] = _codes_fp8(q, s["q_scale"]) if c["qfp8"] else q.bfloat16()
    s["out_scale"] = 0.004
    s["sm_scale"] = 1 / math.sqrt(d)
    if c["op"] == "diff" or c["diff"]:
        s["sm_scale"] = 1 / math.sqrt(d // 2)
        # lambda = exp(a . b) - exp(c . d) + init of a deep layer's learned vectors
        init = 0.8 - 0.6 * math.exp(-0.3 * 12)
        w = 0.1 * torch.randn(4, hq, d // 2, generator=g, device=DEV, dtype=torch.float64)
        s["lam"] = ((w[0] * w[1]).sum(-1).exp() - (w[2] * w[3]).sum(-1).exp() + init).float()
        s["gain"], s["eps"] = 1 - init, 1e-5
        if c["norm"]:
            s["nw"] = 1 + 0.2 * torch.randn(d, generator=g, device=DEV)


PREPARE = {"plan": _prepare_plan, "slots": _prepare_slots, "chunk": _prepare_attention,
           "diff": _prepare_attention}


def prepare(case, seed):
    g, s = _gen(seed), {"case": case}
    PREPARE[case["op"]](case, g, s)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _plain_plan(s, c):
    ps, B, T = c["page"], c["batch"], s["max_tokens"]
    old, add, bt, free = s["lens"].long(), s["adds"].long(), s["bt"], s["free"]
    new = (old + add).clamp(min=0)
    held, want = (old + ps - 1) // ps, (new + ps - 1) // ps
    n = s["count"].long()
    # pages that go back, request by request
    back = (held - want).clamp(min=0)
    width = torch.arange(bt.shape[1], device=DEV)
    gone = (width >= want[:, None]) & (width < held[:, None])
    rank = (gone.reshape(-1).cumsum(0) - 1).reshape(gone.shape) + n
    keep = torch.where(gone, rank, torch.full_like(rank, free.numel()))
    pad = torch.cat([free, free.new_zeros(1)])
    pad.scatter_(0, keep.reshape(-1), bt.reshape(-1))
    free.copy_(pad[:-1])
    n = n + back.sum()
    # pages that are taken, from the stack's top; a request whose pages are not all there
    # gets none
    tokens = add.clamp(min=0)
    end = tokens.cumsum(0)
    need = (want - held).clamp(min=0)
    fits = (want <= bt.shape[1]) & (end <= T)
    need = torch.where(fits, need, torch.zeros_like(need))
    upto = need.cumsum(0)
    ok = (add <= 0) | (fits & ((need == 0) | (upto <= n)))
    need = torch.where(ok, need, torch.zeros_like(need))
    first = upto - need
    grown = (width >= held[:, None]) & (width < (held + need)[:, None])
    at = (n - 1 - (first[:, None] + width - held[:, None])).clamp(0, free.numel() - 1)
    bt.copy_(torch.where(grown, free[at], bt))
    s["count_out"].copy_(n - need.sum())
    s["lens_out"].copy_(torch.where(ok, new, old))
    offsets = torch.cat([end.new_zeros(1), end]).clamp(max=T)
    i = torch.arange(T, device=DEV)
    b = torch.searchsorted(offsets[1:].contiguous(), i, right=True).clamp(max=B - 1)
    pos = old[b] + i - offsets[b]
    live = (i < offsets[-1]) & ok[b]
    page = bt[b, (pos // ps).clamp(0, bt.shape[1] - 1)].long()
    none = torch.full_like(pos, -1)
    return {"bt": bt, "free": free, "count": s["count_out"], "lens": s["lens_out"],
            "start": old.int(), "offsets": offsets.int(),
            "slots": torch.where(live, page * ps + pos % ps, none),
            "positions": torch.where(live, pos, none).int()}


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


def _plain_slots(s, c):
    at = torch.arange(c["tokens"] - c["padding"], device=DEV)   # the real tokens come first
    cs = s["table"][s["pos"][at].long()]
    q = _norm_rotate(s["q"][at].float(), s.get("qw"), cs, c)
    k = _norm_rotate(s["k"][at].float(), s.get("kw"), cs, c)
    page, off = s["slots"][at] // c["page"], s["slots"][at] % c["page"]
    for name, x in (("k", k), ("v", s["v"][at].float())):
        s[name + "c"][page, :, off] = _codes_fp8(x, torch.tensor(s[name + "_scale"], device=DEV))
    qs = torch.tensor(s["q_scale"], device=DEV)
    s["q_out"][at] = _codes_fp8(q, qs) if c["fp8q"] else q.bfloat16()
    return _slots_outputs(s, c)


def _slots_outputs(s, c):
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


def _softmax(x):
    """Over the last axis; a row that sees nothing gives zeros."""
    top = x.amax(-1, keepdim=True)
    p = (x - top.masked_fill(top == -math.inf, 0.0)).exp()
    total = p.sum(-1, keepdim=True)
    return torch.where(total > 0, p / total, torch.zeros_like(p))


def _maps(x):
    """Both halves of the last axis."""
    return x[..., :x.shape[-1] // 2], x[..., x.shape[-1] // 2:]


def _attend(q, k, v, mask, s, c):
    """q [..., kv heads, group, rows, dim], k and v [..., kv heads, 1, keys, dim], mask True
    where a key is not seen; the operator's output before it is rounded."""
    def one(a, b):
        return _softmax((a @ b.transpose(-1, -2)).masked_fill(mask, -math.inf)) @ v
    q = q * s["sm_scale"]
    if not (c["op"] == "diff" or c["diff"]):
        return one(q, k)
    (q1, q2), (k1, k2) = _maps(q), _maps(k)
    o = one(q1, k1) - s["lam"].reshape(c["hkv"], -1, 1, 1) * one(q2, k2)
    if c["norm"]:
        o = o / (o.square().mean(-1, keepdim=True) + s["eps"]).sqrt() * s["nw"]
    return o * s["gain"]


def _rounded(o, s, c):
    if c["out"] == "f32":
        return o
    if c["out"] == "bf16":
        return o.bfloat16()
    return (o / torch.tensor(s["out_scale"], device=DEV)).clamp(-448, 448).to(torch.float8_e4m3fn)


def _queries(s, c):
    return s["q"].view(torch.float8_e4m3fn).float() * s["q_scale"] if c["qfp8"] else s["q"].float()


def _plain_chunk(s, c):
    hkv, d = c["hkv"], c["dim"]
    q = _queries(s, c).unflatten(1, (hkv, -1)).permute(1, 2, 0, 3)   # [kv heads][group][tokens][dim]
    out = torch.zeros_like(q)
    at = 0
    for b, (n, total) in enumerate(zip(s["new"], s["total"])):
        pages = s["bt"][b, :-(-total // c["page"])].long()
        k, v = (_values(s, x, pages, c).transpose(0, 1).reshape(hkv, 1, -1, d)[:, :, :total]
                for x in "kv")
        key = torch.arange(total, device=DEV)
        for i in range(0, n, 256):
            j = min(i + 256, n)
            pos = total - n + torch.arange(i, j, device=DEV)
            out[:, :, at + i:at + j] = _attend(q[:, :, at + i:at + j], k, v,
                                               key > pos[:, None], s, c)
        at += n
    return _rounded(out.permute(2, 0, 1, 3).flatten(1, 2).contiguous(), s, c)


def _plain_diff(s, c):
    q = _queries(s, c).unflatten(1, (c["hkv"], -1))[..., None, :]   # [batch][kv heads][group][1][dim]
    k, v = (_values(s, x, s["bt"].long(), c).transpose(1, 2).flatten(2, 3)[:, :, None] for x in "kv")
    mask = torch.arange(k.shape[3], device=DEV) >= s["lens"][:, None]
    o = _attend(q, k, v, mask[:, None, None, None], s, c)
    return _rounded(o.reshape(c["batch"], c["hq"], c["dim"]), s, c)


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _handle(s, c):
    """What a serving program keeps beside its buffers: made on a state's first pass."""
    if "handle" in s:
        return s["handle"]
    from quantized_kv_cache_05_gb300 import runtime
    h = s["handle"] = {"rt": runtime}
    if c["op"] == "plan":
        pool = runtime.PagePool.wrap(s["free"], s["count"])
        h["plan"] = runtime.StepPlan(s["bt"], c["page"], pool, s["max_tokens"])
        return h
    h["cache"] = runtime.QuantizedKVCache.wrap(c["fmt"], s["kc"], s["vc"], s["bt"], s["k_scale"],
                                               s["v_scale"], s.get("kb"), s.get("vb"))
    if c["op"] == "slots":
        h["rotary"] = runtime.Rotary(s["table"], interleaved=c["inter"], q_norm=s.get("qw"),
                                     k_norm=s.get("kw"), eps=EPS)
        return h
    diff = None
    if "lam" in s:
        diff = runtime.Differential(s["lam"], norm=s.get("nw"), eps=s["eps"], gain=s["gain"])
    options = dict(out=c["out"], out_scale=s["out_scale"], q_fp8=c["qfp8"], q_scale=s["q_scale"],
                   diff=diff)
    kind = runtime.DiffDecode if c["op"] == "diff" else runtime.ChunkAttention
    h["attend"] = kind(h["cache"], c["batch"], c["hq"], max(s["total"]), s["sm_scale"], **options)
    return h


def _own(s, c):
    h = _handle(s, c)
    if c["op"] == "plan":
        p = h["plan"]
        p(s["lens"], s["adds"], seq_lens_out=s["lens_out"], count_out=s["count_out"])
        return {"bt": s["bt"], "free": s["free"], "count": s["count_out"], "lens": s["lens_out"],
                "start": p.start_pos, "offsets": p.q_offsets, "slots": p.slots,
                "positions": p.positions}
    if c["op"] == "slots":
        h["cache"].append_slots(h["rotary"], s["k"], s["v"], s["slots"], s["pos"], q=s["q"],
                                q_out=s["q_out"], q_scale=s["q_scale"])
        return _slots_outputs(s, c)
    if c["op"] == "chunk":
        o = h["attend"](s["q"], s["offsets"], s["lens"])
    else:
        o = h["attend"](s["q"], s["lens"])
    return o.view(torch.float8_e4m3fn) if c["out"] == "e4m3" else o


PLAIN = {"plan": _plain_plan, "slots": _plain_slots, "chunk": _plain_chunk, "diff": _plain_diff}


def run(state):
    c = state["case"]
    return _own(state, c) if own else PLAIN[c["op"]](state, c)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _exact_plan(s, c):
    """Request by request, with a list for the stack of free pages."""
    ps, T = c["page"], s["max_tokens"]
    bt, free = s["bt"].cpu().numpy().copy(), s["free"].cpu().numpy().copy()
    stack = free[:int(s["count"])].tolist()
    old, add = s["lens"].tolist(), s["adds"].tolist()
    lens = list(old)
    for b, a in enumerate(add):          # what goes back, first
        if a < 0:
            lens[b] = max(old[b] + a, 0)
            for p in range(-(-lens[b] // ps), -(-old[b] // ps)):
                free[len(stack)] = bt[b, p]
                stack.append(int(bt[b, p]))
    slots, pos = np.full(T, -1, np.int64), np.full(T, -1, np.int32)
    offsets, out_of_pages = [0], False
    for b, a in enumerate(add):
        at = offsets[-1]
        offsets.append(min(at + max(a, 0), T))
        if a <= 0:
            continue
        have, want = -(-old[b] // ps), -(-(old[b] + a) // ps)
        if want > bt.shape[1] or at + a > T:
            continue
        if want > have:
            out_of_pages = out_of_pages or want - have > len(stack)
            if out_of_pages:
                continue
            for p in range(have, want):
                bt[b, p] = stack.pop()
        lens[b] = old[b] + a
        where = np.arange(old[b], old[b] + a)
        slots[at:at + a] = bt[b, where // ps].astype(np.int64) * ps + where % ps
        pos[at:at + a] = where
    t = lambda x: torch.as_tensor(np.asarray(x), device=DEV)
    return {"bt": t(bt), "free": t(free), "count": _i32([len(stack)]), "lens": _i32(lens),
            "start": _i32(old), "offsets": _i32(offsets), "slots": t(slots), "positions": t(pos)}


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


def _scale_64(x):
    """The fp32 number that a call gets for a scale."""
    return float(torch.tensor(x, dtype=torch.float32))


def _exact_slots(s, c):
    live, d, ps = c["tokens"] - c["padding"], c["dim"], c["page"]
    pos, slot = s["pos"][:live].long(), s["slots"][:live]
    rows = {"k": _turn_64(s["k"][:live], s.get("kw"), pos, s["table"], c), "v": s["v"][:live].double()}
    q = _turn_64(s["q"][:live], s.get("qw"), pos, s["table"], c)
    out = {"q": torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)}
    out["q"][:live] = _e4m3_64(q / _scale_64(s["q_scale"])) if c["fp8q"] else q
    for name, x in rows.items():
        flat = s[name + "c"].view(torch.float8_e4m3fn).double().transpose(1, 2).reshape(-1, c["hkv"], d)
        flat[slot] = _e4m3_64(x / _scale_64(s[name + "_scale"]))
        out[name] = flat.reshape(-1, ps, c["hkv"], d).transpose(1, 2).contiguous()
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
    return x.reshape(-1, c["dim"]) * _scale_64(s[name + "_scale"])


def _exact_attention(s, c):
    if work(c)["flops"] > 4e12:   # minutes in 64 bits
        return None
    grp, d = c["hq"] // c["hkv"], c["dim"]
    q = s["q"].double()
    if c["qfp8"]:
        q = s["q"].view(torch.float8_e4m3fn).double() * _scale_64(s["q_scale"])
    sm = _scale_64(s["sm_scale"])
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    first = s["offsets"].tolist()
    differ = c["op"] == "diff" or c["diff"]
    for b, total in enumerate(s["total"]):
        pages = s["bt"][b, :-(-total // c["page"])].long()
        n = s["new"][b]
        for h in range(c["hkv"]):
            k, v = (_cached_64(s, x, h, pages, c)[:total] for x in "kv")
            for i in range(0, n, 512):
                m = min(512, n - i)
                # rows in the order (token, query head)
                rows = q[first[b] + i:first[b] + i + m, h * grp:(h + 1) * grp].reshape(m * grp, d)
                last = (total - n + i + torch.arange(m, device=DEV)).repeat_interleave(grp)
                hidden = torch.arange(total, device=DEV)[None] > last[:, None]
                def probs(a, e):
                    return torch.softmax((a @ e.T * sm).masked_fill(hidden, -math.inf), 1)
                if differ:
                    lam = s["lam"].double()[h * grp:(h + 1) * grp].repeat(m)[:, None]
                    w = probs(rows[:, :d // 2], k[:, :d // 2]) - lam * probs(rows[:, d // 2:], k[:, d // 2:])
                    o = w @ v
                    if c["norm"]:
                        o = o * torch.rsqrt((o * o).sum(1, keepdim=True) / d + _scale_64(s["eps"])) * s["nw"].double()
                    o = o * _scale_64(s["gain"])
                else:
                    o = probs(rows, k) @ v
                out[first[b] + i:first[b] + i + m, h * grp:(h + 1) * grp] = o.reshape(m, grp, d)
    if c["out"] == "e4m3":
        return _e4m3_64(out / _scale_64(s["out_scale"]))
    return out


EXACT = {"plan": _exact_plan, "slots": _exact_slots, "chunk": _exact_attention,
         "diff": _exact_attention}


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return EXACT[case["op"]](s, case)
