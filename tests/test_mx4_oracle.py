"""Pins of the 4-bit oracle: hand-worked blocks, the grid's neighbours and ties
by brute force, and planted slips that the pins must catch."""
import numpy as np
import pytest

from oracle import moe_tokens as omt
from oracle import mx4 as ox


def one(vals):
    v = np.zeros((1, 32))
    v[0, :len(vals)] = vals
    c, s = ox.quantize(v)
    return c[0, :len(vals)].tolist(), int(s[0, 0])


@pytest.mark.parametrize("vals,codes,scale", [
    # m = 6: e = floor(log2 6) - 2 = 0; ties 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5 to even codes
    ([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -5], [7, 0, 2, 2, 4, 4, 6, 6, 8, 14], 127),
    # m = 7.9: e = 0 and 7.9 is clamped to 6; just below and above a middle
    ([7.9, 6.1, .2499, .2501, 4.999, 5.001], [7, 7, 0, 1, 6, 7], 127),
    ([8, 6, 1], [6, 5, 1], 128),             # m = 8: e = 1, in units of 2: 4, 3, 0.5
    ([0, -0.0, 0], [0, 8, 0], 0),            # nothing: the smallest scale
    ([2.0 ** -130], [0], 0),                 # 2^-130 / 2^-127 = 0.125 rounds to 0
    ([1.5 * 2.0 ** -128], [2], 0),           # 0.75 is a tie: to 1
    ([float("nan"), 5], [0, 0], 255), ([float("inf"), 5], [0, 0], 255),
])
def test_hand_worked_blocks(vals, codes, scale):
    assert one(vals) == (codes, scale)


def brute(a):
    """Index of the nearest grid value to 0 <= a, the even one of two nearest."""
    d = np.abs(ox.GRID - a)
    near = np.flatnonzero(d == d.min())
    return int(near[0]) if len(near) == 1 else int([i for i in near if i % 2 == 0][0])


def test_nearest_by_brute_force():
    a = np.arange(0, 8, 1 / 64)
    x = np.concatenate([[[7.0] + a[i:i + 31].tolist() + [0.0] * (31 - len(a[i:i + 31]))]
                        for i in range(0, len(a), 31)])
    codes, scales = ox.quantize(x)
    assert (scales == 127).all()
    got = codes[:, 1:].reshape(-1)[:len(a)]
    assert got.tolist() == [brute(min(v, 6.0)) for v in a]


def test_values_and_storage():
    rng = np.random.default_rng(0)
    codes = rng.integers(0, 16, (5, 96)).astype(np.uint8)
    scales = rng.integers(0, 255, (5, 3)).astype(np.uint8)
    pc, ps = ox.pack(codes, scales)
    assert pc.shape == (5, 48) and ps.shape == (5, 16) and (ps[:, 3:] == 0).all()
    assert pc[0, 0] == codes[0, 0] + 16 * codes[0, 1]
    c, s = ox.unpack(pc, ps)
    assert (c == codes).all() and (s == scales).all()
    v = ox.values(codes, scales, 70)
    assert v.shape == (5, 70)
    assert v[2, 33] == ox.GRID[codes[2, 33] & 7] * (-1.0 if codes[2, 33] & 8 else 1.0) * 2.0 ** (int(scales[2, 1]) - 127)
    assert np.isnan(ox.values(codes, np.full((5, 3), 255), 70)).all()


def test_quantising_what_was_quantised_changes_nothing():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((20, 96)) * np.exp(rng.standard_normal((20, 96)))
    v = ox.values(*ox.quantize(x), 96)
    np.testing.assert_array_equal(ox.values(*ox.quantize(v), 96), v)
    assert (np.abs(v - x) <= np.maximum(np.abs(x) / 4, 2.0 ** -2 * np.repeat(
        np.ldexp(1.0, ox.quantize(x)[1].astype(int) - 127), 32, axis=1))).all()


def test_layer_by_hand():
    """One token, two experts of width 1: silu(2) = 2 / (1 + e^-2)."""
    x = np.array([[1.0, 2.0]])
    w1 = np.array([[[2.0, 1.0], [0.0, 1.0]], [[0.0, 5.0], [1.0, 0.0]]])  # (E, H, 2I)
    w2 = np.array([[[1.0, -1.0]], [[3.0, 0.0]]])
    silu = 2 / (1 + np.exp(-2))
    out, _, bad = omt.layer(x, np.array([[0, 1]]), np.array([[0.5, 0.25]]), w1, w2, ep_rank=0,
                            num_experts=2)
    # expert 0: gate 2, up 3; expert 1: gate 2, up 5
    np.testing.assert_allclose(out, [[0.5 * silu * 3 + 0.25 * silu * 5 * 3, -0.5 * silu * 3]])
    assert not bad
    out, _, bad = omt.layer(x, np.array([[7, 1]]), np.array([[0.5, 0.25]]), w1[1:], w2[1:],
                            ep_rank=1, num_experts=2)
    np.testing.assert_allclose(out, [[0.25 * silu * 5 * 3, 0]])
    assert bad


@pytest.mark.parametrize("slip", ["floor", "ceil_exponent", "ties_up", "no_clamp"])
def test_planted_slips_are_caught(monkeypatch, slip):
    if slip == "no_clamp":
        monkeypatch.setattr(ox, "GRID", np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 8.0]))
    elif slip == "ceil_exponent":
        frexp = np.frexp
        monkeypatch.setattr(ox.np, "frexp", lambda v: (frexp(v)[0], frexp(v)[1] + 1))
    else:
        real = ox.quantize

        def wrong(x):
            c, s = real(x)
            a = np.abs(x) / np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, axis=1)[:, :x.shape[1]]
            shift = ox.GRID[c[:, :x.shape[1]] & 7]
            c[:, :x.shape[1]] += ((shift < a) if slip == "ties_up" else -(shift > a).astype(int)).astype(np.uint8)
            return c, s
        monkeypatch.setattr(ox, "quantize", wrong)
    with pytest.raises(AssertionError):
        test_hand_worked_blocks([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -5],
                                [7, 0, 2, 2, 4, 4, 6, 6, 8, 14], 127)
