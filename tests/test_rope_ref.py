"""The 64-bit form of the norm-and-rotate operators holds what it should: the
rotation keeps lengths and turns with relative positions only, and the grid
rounding is torch's cast; a mistake planted in it is seen by the checks."""
import numpy as np
import pytest
import torch

import rope_ref as R


def table(n, rot):
    ang = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [32, 64])
def test_rotation_depends_on_relative_positions(rot, interleaved):
    g = np.random.default_rng(1)
    q, k = g.normal(size=(1, 1, 64)), g.normal(size=(1, 1, 64))
    t = table(200, rot)
    dots = []
    for shift in (0, 17, 101):
        y = R.turn(q, None, np.array([shift + 40]), t, rot, interleaved, 0)[0]
        z = R.turn(k, None, np.array([shift + 3]), t, rot, interleaved, 0)[0]
        assert abs(np.linalg.norm(y) - np.linalg.norm(q)) < 1e-12
        dots.append(float((y * z).sum()))
    assert np.ptp(dots) < 1e-12


def test_grid_rounding_is_the_cast():
    g = np.random.default_rng(2)
    x = np.concatenate([g.normal(size=4000) * 100, g.normal(size=4000) * 0.01, R.E4M3_POS,
                        (R.E4M3_POS[1:] + R.E4M3_POS[:-1]) / 2, [500.0]]).astype(np.float32)
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.round_value(x, R.E4M3_POS), want)


def test_checks_see_planted_mistakes():
    g = np.random.default_rng(3)
    x = g.normal(size=(5, 2, 64))
    t = table(50, 64)
    pos = np.arange(5) + 7
    y, mag = R.turn(x, None, pos, t, 64, False, 0)
    R.check_bf16(torch.from_numpy(y).bfloat16().double().numpy(), y, mag)
    wrong = R.turn(x, None, pos + 1, t, 64, False, 0)[0]
    with pytest.raises(AssertionError):
        R.check_bf16(wrong, y, mag)
    R.check_grid(R.round_value(y / 0.02, R.E4M3_POS), y, mag, 0.02, R.E4M3_POS)
    with pytest.raises(AssertionError):
        R.check_grid(R.round_value(y / 0.021, R.E4M3_POS), y, mag, 0.02, R.E4M3_POS)
