"""kvq_plan_step against the step done request by request, kvq_rope_append_slots against
kvq_rope_append, and whole packed steps: plan, append, attention."""
import numpy as np
import pytest
import torch

from packed_ref import DEV, Packed, i32
from quantized_kv_cache_05_gb300 import build as kbuild
from quantized_kv_cache_05_gb300 import kvq, runtime

pytestmark = pytest.mark.gpu
ALL = -2 ** 31


@pytest.fixture(scope="module", autouse=True)
def _lib():
    kbuild.build()
    kvq.lib()
    torch.cuda.init()
    torch.zeros(1, device=DEV)


class State:
    """What a serving program holds, on the host: tables, lengths and the stack."""

    def __init__(self, B, width, ps, pages, lens, spare=None, seed=0):
        r = np.random.default_rng(seed)
        perm = r.permutation(pages).astype(np.int32)
        self.ps, self.pages, self.lens = ps, pages, list(lens)
        self.bt = np.full((B, width), -7, np.int32)
        at = 0
        for b, n in enumerate(lens):
            h = -(-n // ps)
            self.bt[b, :h] = perm[at:at + h]
            at += h
        self.free = np.full(pages, -9, np.int32)
        self.count = pages - at if spare is None else spare
        self.free[:self.count] = perm[at:at + self.count]

    def step(self, add, T):
        """One request after the other; the outputs, and the error bits."""
        ps, width = self.ps, self.bt.shape[1]
        old, stack, err = list(self.lens), self.free[:self.count].tolist(), 0
        for b, a in enumerate(add):
            if a < 0:
                self.lens[b] = max(old[b] + a, 0)
                for p in range(-(-self.lens[b] // ps), -(-old[b] // ps)):
                    self.free[len(stack)] = self.bt[b, p]
                    stack.append(self.bt[b, p])
        slots, pos, offs, out = np.full(T, -1, np.int64), np.full(T, -1, np.int32), [0], False
        for b, a in enumerate(add):
            at = offs[-1] if b == 0 else total
            total = (0 if b == 0 else total) + max(a, 0)
            offs.append(min(total, T))
            if a <= 0:
                continue
            at = total - a
            have, want = -(-old[b] // ps), -(-(old[b] + a) // ps)
            if want > width or old[b] + a > width * ps or total > T:
                err |= kvq.KVQ_DEVERR_REFUSED
                continue
            if want > have:
                out = out or want - have > len(stack)
                if out:
                    err |= kvq.KVQ_DEVERR_REFUSED
                    continue
                for p in range(have, want):
                    self.bt[b, p] = stack.pop()
            self.lens[b] = old[b] + a
            for i in range(a):
                t = old[b] + i
                slots[at + i] = int(self.bt[b, t // ps]) * ps + t % ps
                pos[at + i] = t
        self.count = len(stack)
        return old, offs, slots, pos, err


class OnGpu:
    def __init__(self, s, T):
        self.bt, self.free, self.count = (torch.from_numpy(s.bt.copy()).to(DEV),
                                          torch.from_numpy(s.free.copy()).to(DEV), i32([s.count]))
        self.lens = i32(s.lens)
        self.pool = runtime.PagePool.wrap(self.free, self.count)
        self.plan = runtime.StepPlan(self.bt, s.ps, self.pool, T)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def check(self, s, want, in_place=True):
        old, offs, slots, pos, err = want
        p = self.plan
        torch.cuda.synchronize()
        assert p.start_pos.tolist() == old and p.q_offsets.tolist() == offs
        assert np.array_equal(p.slots.cpu().numpy(), slots) and np.array_equal(p.positions.cpu().numpy(), pos)
        assert np.array_equal(self.bt.cpu().numpy(), s.bt) and np.array_equal(self.free.cpu().numpy(), s.free)
        if in_place:
            assert self.lens.tolist() == s.lens and self.count.tolist() == [s.count]
        assert int(self.err) == err and int(self.pool.counter) == 0


@pytest.mark.parametrize("B", [1, 5, 33, 1000, 1500, 8192])
@pytest.mark.parametrize("ps", [1, 16, 48])
def test_steps(B, ps):
    """Steps in a row, the lengths and the stack updated in place: single tokens, chunks,
    ends, tokens that go again, idle requests; then a pool that runs out."""
    r = np.random.default_rng(B + ps)
    width = 70
    lens = [int(x) for x in r.integers(0, min(30 * ps, 400), B)]
    held = sum(-(-n // ps) for n in lens)
    s = State(B, width, ps, held + 3 * B + 20, lens)
    T = 5000
    g = OnGpu(s, T)
    for step in range(6):
        kind = r.integers(0, 6, B)
        add = np.select([kind <= 2, kind == 3, kind == 4], [1, r.integers(0, 60, B), -r.integers(0, 40, B)], 0)
        add[r.random(B) < 0.05] = ALL
        if step == 4:
            add = np.full(B, 3 * ps)   # more than there are pages, or rows, or table entries
        add = [int(a) for a in add]
        g.err.zero_()
        want = s.step(add, T)
        g.plan(g.lens, i32(add), error_flag=g.err)
        g.check(s, want)


def test_out_of_place_leaves_the_inputs():
    s = State(40, 9, 16, 400, [(7 * b) % 100 for b in range(40)])
    g = OnGpu(s, 300)
    lens0, n0 = list(s.lens), s.count
    add = [[1, 17, 0, -20, ALL][b % 5] for b in range(40)]
    want = s.step(add, 300)
    out, n = i32([5] * 40), i32([5])
    for _ in range(3):   # the same call again gives the same
        g.plan(g.lens, i32(add), out, n, error_flag=g.err)
        g.check(s, want, in_place=False)
        assert out.tolist() == s.lens and n.tolist() == [s.count]
        assert g.lens.tolist() == lens0 and g.count.tolist() == [n0]


@pytest.mark.parametrize("spare", [0, 1, 2, 3, 4])
def test_a_pool_that_runs_out(spare):
    """Served in order, whole or not at all; requests that need no page go on; what comes
    back in the same step is taken at once."""
    s = State(7, 4, 16, 12 + spare, [15, 16, 32, 3, 16, 40, 0], spare=spare)
    g = OnGpu(s, 100)
    for add in ([1, 1, 2, 1, 17, 0, 1], [0, 30, 1, ALL, 1, -30, 20]):
        g.err.zero_()
        want = s.step(add, 100)
        g.plan(g.lens, i32(add), error_flag=g.err)
        g.check(s, want)


def test_rows_that_do_not_fit():
    """A request past the packed rows, or past its block-table row, and those behind."""
    s = State(4, 3, 16, 40, [10, 40, 0, 16])
    g = OnGpu(s, 20)
    for add in ([5, 9, 1, 1], [1, 0, 25, 1], [0, 0, 0, 2 ** 31 - 1], [2 ** 31 - 1] * 4, [0, 0, 20, 0]):
        g.err.zero_()
        want = s.step(add, 20)
        g.plan(g.lens, i32(add), error_flag=g.err)
        g.check(s, want)


def test_no_requests_and_no_rows():
    s = State(3, 4, 16, 30, [10, 40, 0])
    g = OnGpu(s, 0)
    want = s.step([0, -5, 0], 0)
    g.plan(g.lens, i32([0, -5, 0]), error_flag=g.err)
    g.check(s, want)
    pool = runtime.PagePool(5)
    p = runtime.StepPlan(torch.zeros(0, 3, dtype=torch.int32, device=DEV), 16, pool, 4)
    p(i32([]), i32([]))
    assert p.slots.tolist() == [-1] * 4 and p.q_offsets.tolist() == [0] and pool.count.tolist() == [5]
    assert pool.free.tolist() == [4, 3, 2, 1, 0]


def test_damaged_inputs():
    """Counts, lengths and pages out of range: clamped or dropped, with their bits; nothing
    outside the arrays is touched (the next call over sound ones is right)."""
    s = State(3, 4, 16, 30, [10, 40, 0])
    for count, bits in ((-5, 32), (99, 32)):
        g = OnGpu(s, 10)
        g.count.fill_(count)
        g.plan(g.lens, i32([1, 1, 0]), error_flag=g.err)
        assert int(g.err) & 32
    g = OnGpu(s, 10)
    g.plan(i32([-3, 1000, 0]), i32([1, -1, 0]), seq_lens_out=g.lens, error_flag=g.err)
    assert int(g.err) & 2 and g.lens.tolist() == [1, 63, 0]
    # a full pool that gets pages back
    g = OnGpu(s, 10)
    g.count.fill_(30)
    g.plan(g.lens, i32([ALL, 0, 0]), error_flag=g.err)
    assert int(g.err) == 32 and g.count.tolist() == [30]
    # a free page out of range: no slot
    g = OnGpu(s, 10)
    g.free[s.count - 1] = 30
    g.plan(g.lens, i32([0, 0, 2]), error_flag=g.err)
    assert int(g.err) == kvq.KVQ_DEVERR_BAD_PAGE and g.plan.slots.tolist() == [-1] * 10
    assert g.plan.positions.tolist() == [0, 1] + [-1] * 8


def test_replayed_steps():
    """Decode steps replayed from a graph: the lengths grow on the GPU."""
    s = State(60, 6, 16, 500, [(5 * b) % 50 for b in range(60)])
    g = OnGpu(s, 64)
    add = i32([1] * 60)
    g.plan(g.lens, add, error_flag=g.err)
    g.check(s, s.step([1] * 60, 64))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.plan(g.lens, add, error_flag=g.err)
    for _ in range(30):
        want = s.step([1] * 60, 64)
        graph.replay()
    g.check(s, want)


# ------------------------------------------------------------------------ slots
def table(rows, rot):
    return runtime.rope_table(rows, rot)


@pytest.mark.parametrize("fmt,D", [("fp8", 64), ("fp8", 128), ("fp8", 256), ("nvfp4", 64), ("nvfp4", 128),
                                   ("nvfp4", 256)])
@pytest.mark.parametrize("T", [1, 40, 1500])
@pytest.mark.parametrize("norm,rot,inter", [(True, 1.0, False), (False, 0.5, True), (False, 0.0, False)])
def test_slots_are_the_appends(fmt, D, T, norm, rot, inter):
    """The codes and queries of kvq_rope_append for the same tokens, bit for bit, in the
    slots' order; tokens without a slot and padded ones leave everything as it was."""
    hq, hkv, ps = 6, 2, 16
    g = torch.Generator(device=DEV).manual_seed(T)
    rot_dim = int(D * rot) // 32 * 32
    w = (lambda: 1 + 0.2 * torch.randn(D, generator=g, device=DEV)) if norm else (lambda: None)
    ro = runtime.Rotary(table(4096, rot_dim) if rot_dim else None, inter, w(), w())
    pages = (T + 15) // 16 + 5
    x = torch.randn(T, (hq + 2 * hkv) * D, generator=g, device=DEV).bfloat16()
    part = lambda a, n: x[:, a * D:(a + n) * D].unflatten(1, (n, D))
    q, k, v = part(0, hq), part(hq, hkv), part(hq + hkv, hkv)
    make = lambda bt: runtime.QuantizedKVCache(fmt, pages, ps, hkv, D, bt, 0.021 if fmt == "fp8" else 0.0021,
                                               0.017 if fmt == "fp8" else 0.0019)
    # the plain append of one request per token, at that token's position, into page t
    pos = torch.randint(0, ps, (T,), generator=g, device=DEV).int()
    one = runtime.QuantizedKVCache(fmt, T, ps, hkv, D, torch.arange(T).int()[:, None], 0.021 if fmt == "fp8" else 0.0021,
                                   0.017 if fmt == "fp8" else 0.0019)
    want_q = one.append_rope(ro, k[:, None], v[:, None], pos, q=q[:, None], q_out_type="e4m3", q_scale=0.02)
    cache = make(torch.zeros(1, 1, dtype=torch.int32))
    slots = torch.randperm(pages * ps, generator=g, device=DEV)[:T]
    slots[T // 3:T // 3 + 1] = -1
    real = torch.ones(T, dtype=torch.bool, device=DEV)
    real[T // 2 + 1:T // 2 + 4] = False          # padded rows: a negative position
    at = torch.where(real, pos, torch.full_like(pos, -1))
    for t in (cache.k_codes, cache.v_codes, cache.k_bscale, cache.v_bscale):
        if t is not None:
            t.fill_(0x5A)
    qo = torch.full((T, hq, D), 0x33, dtype=torch.uint8, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    # (without a rotation the positions tell the padded rows all the same)
    cache.append_slots(ro, k, v, slots, at, q=q, q_out=qo, q_scale=0.02, error_flag=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    assert torch.equal(qo[real], want_q[:, 0][real]) and (qo[~real] == 0x33).all()
    live = (real & (slots >= 0)).nonzero()[:, 0]
    for got, src in ((cache.k_codes, one.k_codes), (cache.v_codes, one.v_codes), (cache.k_bscale, one.k_bscale),
                     (cache.v_bscale, one.v_bscale)):
        if got is None:
            continue
        want = torch.full_like(got, 0x5A)
        want[slots[live] // ps, :, slots[live] % ps] = src[live, :, pos[live].long()]
        assert torch.equal(got, want)


def test_slots_mla():
    T, ps = 70, 16
    g = torch.Generator(device=DEV).manual_seed(1)
    ro = runtime.Rotary(table(512, 64), False, None, 1 + 0.2 * torch.randn(512, generator=g, device=DEV))
    lat, pe = (torch.randn(T, 1, n, generator=g, device=DEV).bfloat16() for n in (512, 64))
    make = lambda n, bt: runtime.QuantizedKVCache("nvfp4", n, ps, 1, 512, bt, 0.002, 0.002, rope_dim=64)
    pos = torch.randint(0, ps, (T,), generator=g, device=DEV).int()
    one, cache = make(T, torch.arange(T).int()[:, None]), make(9, torch.zeros(1, 1, dtype=torch.int32))
    one.append_rope(ro, lat[:, None], None, pos, pe[:, None])
    slots = torch.randperm(9 * ps, generator=g, device=DEV)[:T]
    cache.append_slots(ro, lat, None, slots, pos, kpe_new=pe)
    i = torch.arange(T, device=DEV)
    for got, src in ((cache.k_codes[:, 0], one.k_codes[:, 0]), (cache.k_bscale[:, 0], one.k_bscale[:, 0]),
                     (cache.k_pe, one.k_pe)):
        assert torch.equal(got[slots // ps, slots % ps], src[i, pos.long()])


def test_slots_out_of_range():
    g = torch.Generator(device=DEV).manual_seed(1)
    ro = runtime.Rotary(table(64, 64))
    k = torch.randn(4, 2, 64, generator=g, device=DEV).bfloat16()
    cache = runtime.QuantizedKVCache("fp8", 3, 16, 2, 64, torch.zeros(1, 1, dtype=torch.int32), 0.02, 0.02)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    for slots, pos, bits in (([48, 1 << 40, -1, -(1 << 40)], [0, 1, 2, 3], 4), ([1, 2, 3, 4], [64, 1 << 30, -1, 99], 8)):
        err.zero_()
        q = cache.append_slots(ro, k, k, torch.tensor(slots, device=DEV), i32(pos), q=k,
                               q_out=torch.zeros_like(k), error_flag=err)
        assert int(err) == bits and int(cache.k_codes.sum()) == 0
        assert (q != 0).any(-1).any(-1).tolist() == [bits == 4] * 4
    for args in ((k, k, i32([1, 2, 3, 4]), i32([0] * 4)), (k, k, torch.arange(3, device=DEV), i32([0] * 4)),
                 (k, k[:3], torch.arange(4, device=DEV), i32([0] * 4)), (k, None, torch.arange(4, device=DEV), None),
                 (k[:, :1], k, torch.arange(4, device=DEV), i32([0] * 4)),
                 (k, k, torch.arange(4, device=DEV), torch.arange(4, device=DEV))):
        with pytest.raises(ValueError):
            cache.append_slots(ro, *args)
    with pytest.raises(kvq.KvqError):
        cache.append_slots(ro, k, k, torch.arange(4, device=DEV), None)


# ------------------------------------------------------------------- whole steps
@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("diff", [False, True])
def test_packed_steps(fmt, diff):
    """Prompts, single tokens, ends, new requests in their rows: every step's plan, append
    and attention, against a cache with a page of its own for each request."""
    B, hq, hkv, D, ps, T, cap = 6, 8, 2, 128, 16, 256, 512
    X = Packed(fmt, D, hq, hkv, ps, [(0, 1)], diff=diff)   # (its reference serves any state)
    pages = 70
    pool = runtime.PagePool(pages)
    scale = (0.02, 0.02) if fmt == "fp8" else (0.003, 0.003)
    cache = runtime.QuantizedKVCache(fmt, pages, ps, hkv, D, torch.full((B, cap // ps), -1).int(), *scale)
    mirror = runtime.QuantizedKVCache(fmt, B, cap, hkv, D, torch.arange(B).int()[:, None], *scale)
    plan = runtime.StepPlan(cache.block_table, ps, pool, T)
    sm = X.sm
    att = runtime.ChunkAttention(cache, B, hq, cap, sm, out="f32", diff=X.diff)
    ro = runtime.Rotary(table(cap, D), k_norm=torch.ones(D, device=DEV), q_norm=torch.ones(D, device=DEV))
    lens = i32([0] * B)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(9)
    host = [0] * B
    steps = [[100, 0, 30, 1, 0, 0], [1, 77, 1, 1, 0, 3], [1, 1, ALL, 1, 100, 1], [1, 1, 64, -1, 1, 40],
             [ALL, 1, 1, 1, 1, 1], [130, 1, 1, 1, 1, 1]]
    for add in steps:
        x = torch.randn(T, (hq + 2 * hkv) * D, generator=g, device=DEV).bfloat16()
        part = lambda a, n: x[:, a * D:(a + n) * D].unflatten(1, (n, D))
        q, k, v = part(0, hq), part(hq, hkv), part(hq + hkv, hkv)
        plan(lens, i32(add), error_flag=err)
        qn = cache.append_slots(ro, k, v, plan.slots, plan.positions, q=q, error_flag=err)
        o = att(qn, plan.q_offsets, lens, error_flag=err)
        torch.cuda.synchronize()
        assert int(err) == 0
        # the mirror: padded rows, the plain rotating append
        new = [max(a, 0) for a in add]
        start = [max(h + min(a, 0), 0) for h, a in zip(host, add)]
        host = [s + n for s, n in zip(start, new)]
        assert lens.tolist() == host
        n = max(new)
        pad = torch.zeros(B, n, hq + 2 * hkv, D, device=DEV).bfloat16()
        at = 0
        for b, m in enumerate(new):
            pad[b, :m] = x[at:at + m].view(m, hq + 2 * hkv, D)
            at += m
        mq = mirror.append_rope(ro, pad[:, :, hq:hq + hkv], pad[:, :, hq + hkv:], i32(start), new_lens=i32(new),
                                q=pad[:, :, :hq])
        total = sum(new)
        assert torch.equal(qn[:total], torch.cat([mq[b, :m] for b, m in enumerate(new)]))
        bt = cache.block_table.long()
        for b, L in enumerate(host):
            for a, m in ((cache.k_codes, mirror.k_codes), (cache.v_codes, mirror.v_codes),
                         (cache.k_bscale, mirror.k_bscale), (cache.v_bscale, mirror.v_bscale)):
                if a is not None and L:
                    t = torch.arange(L, device=DEV)
                    assert torch.equal(a[bt[b, t // ps], :, t % ps], m[b, :, :L].transpose(0, 1))
        # attention over the mirror's values
        X.B, X.lens, X.new, X.bt, X.ps, X.T = B, host, new, mirror.block_table, cap, total
        X.offs = np.concatenate([[0], np.cumsum(new)]).astype(int)
        X.q64 = qn[:total].double()
        X.val = [values(c, s, sc) for c, s, sc in ((mirror.k_codes, mirror.k_bscale, scale[0]),
                                                    (mirror.v_codes, mirror.v_bscale, scale[1]))]
        X.check(o[:total], "f32")


def values(codes, bscale, scale):
    s = float(np.float32(scale))
    if bscale is None:
        return codes.view(torch.float8_e4m3fn).double() * s
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=DEV)
    nib = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    x = grid[nib & 7] * (1.0 - 2.0 * (nib >> 3))
    return (x.unflatten(-1, (-1, 16)) * bscale.view(torch.float8_e4m3fn).double()[..., None]).flatten(-2) * s
