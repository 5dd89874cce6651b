"""The norm-and-rotate operators from their formulas in 64 bits, and the
intervals that the fp32 kernels' results must lie in.

fp32 error of a kernel value y = n_a cos -+ n_b sin, u = 2^-24: the sum of at
most 512 squares is 8 fused steps per lane and at most 6 adds, all of positive
terms: 14 u; the mean's scaling is exact; + eps 1 u; half of that through the
root, whose own error is at most 2 units in the last place, 4 u: r within 12 u;
n = (x r) w adds 2 u; each product of the rotation is rounded once and the sum
once: 2 u more.  Altogether |y' - y| <= 16 u (|n_a cos| + |n_b sin|); 20 u leaves
room for the second-order terms.
"""
import numpy as np

U = 2.0 ** -24
ERR = 20 * U

E4M3_POS = np.array([(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                     for e in range(16) for m in range(8)][:127])   # codes 0..0x7E
E2M1_POS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def round_code(x, grid):
    """Index of the nearest grid value of |x| (ties to the even index, saturating)."""
    a = np.abs(np.asarray(x, np.float64))
    mid = (grid[1:] + grid[:-1]) / 2
    lo = np.searchsorted(mid, a, side="left")    # a <= mid[lo]
    tie = (lo < len(mid)) & (a == mid[np.minimum(lo, len(mid) - 1)])
    return np.where(tie & (lo % 2 == 1), lo + 1, lo)


def round_value(x, grid):
    return np.copysign(grid[round_code(x, grid)], x)


def turn(x, w, pos, table, rot, interleaved, eps):
    """x float64 [tokens][heads][dim] -> (y, the magnitude that the error is relative to)."""
    x = np.asarray(x, np.float64)
    if w is not None:
        x = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * np.asarray(w, np.float64)
    y, mag = x.copy(), np.abs(x)
    if rot:
        h = rot // 2
        cs = np.asarray(table, np.float64)[pos][:, None]
        c, s = cs[..., :h], cs[..., h:]
        i = np.arange(h)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
        xa, xb = x[..., a], x[..., b]
        y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
        mag[..., a] = np.abs(xa * c) + np.abs(xb * s)
        mag[..., b] = np.abs(xb * c) + np.abs(xa * s)
    return y, mag


def check_bf16(got, y, mag, what=""):
    """bf16 rounds by at most 2^-8 of the value."""
    lim = np.abs(y) * 2.0 ** -8 * (1 + ERR) + ERR * mag + 1e-40
    bad = ~(np.abs(got - y) <= lim)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, first {np.argwhere(bad)[0]}"


def check_grid(got, y, mag, scale, grid, what=""):
    """Rounding to a grid is monotone: the value lies between those of the interval's ends."""
    s = np.asarray(scale, np.float64)
    lo, hi = (y - ERR * mag) / s, (y + ERR * mag) / s
    lo, hi = lo - 2 * U * np.abs(lo), hi + 2 * U * np.abs(hi)
    bad = ~((got >= round_value(lo, grid)) & (got <= round_value(hi, grid)))
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size}, first {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} for {(y / s)[bad][0]}")


def e4m3_values(codes):
    codes = np.asarray(codes, np.uint8)
    return np.where(codes & 0x80, -1.0, 1.0) * E4M3_POS[np.minimum(codes & 0x7F, 0x7E)]


def e2m1_values(codes):
    """Packed nibbles [..., D/2] -> [..., D]."""
    codes = np.asarray(codes, np.uint8)
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    return np.where(nib & 8, -1.0, 1.0) * E2M1_POS[nib & 7]


def blocks(a):
    return a.reshape(*a.shape[:-1], a.shape[-1] // 16, 16)


def check_nvfp4(codes, bscale, y, mag, g, what=""):
    """Block scales within the interval of the block's largest magnitude; the codes
    against the scales that the kernel chose."""
    sc = e4m3_values(bscale)
    lo = np.maximum(blocks(np.abs(y) - ERR * mag).max(-1), 0) / 6 / g
    hi = blocks(np.abs(y) + ERR * mag).max(-1) / 6 / g
    lo, hi = lo * (1 - 4 * U), hi * (1 + 4 * U)
    bad = ~((sc >= round_value(lo, E4M3_POS)) & (sc <= round_value(hi, E4M3_POS)))
    assert not bad.any(), f"{what} block scales: {bad.sum()} of {bad.size}"
    es = (sc.astype(np.float32) * np.float32(g)).astype(np.float64)[..., None]
    got, yb, mb = blocks(e2m1_values(codes)), blocks(y), blocks(mag)
    zero = np.broadcast_to(es == 0, yb.shape)
    assert not got[zero].any(), f"{what}: codes of a zero scale"
    esb = np.where(es == 0, 1.0, es)
    live = ~zero
    check_grid(got[live], yb[live], mb[live], np.broadcast_to(esb, yb.shape)[live], E2M1_POS, what)
