"""Pins of the compression oracle: the 4-bit format and eviction, on CPU."""
import numpy as np
import pytest

from oracle import compress as oc


def test_bf16_rounding():
    assert oc.round_bf16(1.0) == 1.0
    assert oc.round_bf16(1 + 2 ** -8) == 1.0  # a tie goes to the even neighbour
    assert oc.round_bf16(1 + 3 * 2 ** -8) == 1 + 2 ** -6
    assert oc.round_bf16(-(1 + 2 ** -8 + 2 ** -20)) == -(1 + 2 ** -7)


@pytest.mark.parametrize("offset,size", [(0, 1), (3, 1), (100, 0.1), (-1e4, 1e-3), (0, 1e-6), (0, 3e4)])
def test_quantisation_error_is_half_a_step(offset, size):
    rng = np.random.default_rng(1)
    with np.errstate(over="ignore"):
        x = (offset + size * rng.standard_normal((50, 128))).astype(np.float16).astype(np.float64)
    n, s, z = oc.quantise(x)
    # at 3e4 a few of the fp16 inputs are infinities: their groups have no scale
    finite = np.isfinite(x.reshape(50, 2, 64)).all(-1)
    assert np.array_equal(np.isfinite(s), finite) and finite.any()
    step, whole = np.repeat(s, 64, -1), np.repeat(finite, 64, -1)
    err = np.abs(step * (n - np.repeat(z, 64, -1)) - np.where(whole, x, 0))
    # half a step; the scale was rounded by up to 2^-8 of itself, so 15 steps fall short by 15 / 256
    assert (err <= step * (0.5 + 15 / 256))[whole].all()
    assert n.max() <= 15 and np.abs(z).max() <= 2048


def test_constant_and_zero_groups():
    x = np.zeros((2, 64))
    x[1] = 5.0
    n, s, z = oc.quantise(x)
    assert s[0, 0] == 0 and z[0, 0] == 0 and (n[0] == 0).all()
    assert abs(s[1, 0] * (n[1, 0] - z[1, 0]) - 5.0) <= 0.51 * s[1, 0] and s[1, 0] < 0.003


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_groups_that_are_not_finite_read_back_as_nan(bad):
    x = np.ones((1, 128))
    x[0, 3] = bad
    pool = np.zeros((1, 1, 9 * 128), dtype=np.uint8)
    oc.store_row(pool, 0, 0, 5, x[0])
    v = oc.values(pool, 128)[0, 0, 5]
    assert np.isnan(v[:64]).all() and np.isfinite(v[64:]).all()


def test_rows_of_a_tile_are_independent():
    rng = np.random.default_rng(2)
    rows = rng.standard_normal((16, 128)).astype(np.float16).astype(np.float64)
    pool = rng.integers(0, 256, (2, 1, 9 * 128)).astype(np.uint8)
    before = pool[1].copy()
    for t in rng.permutation(16):
        oc.store_row(pool, 0, 0, int(t), rows[t])
    n, s, z = oc.quantise(rows)
    assert np.array_equal(oc.values(pool[:1], 128)[0, 0], np.repeat(s, 64, -1) * (n - np.repeat(z, 64, -1)))
    assert np.array_equal(pool[1], before)


def test_evict_worked_example():
    # 8 tokens, 4 stay: position 0 (sink), 7 (recent), then the masses 9 and 5
    mass = [0.0, 1, 9, 2, 5, 0, 3, 0]
    moves, m, p, h = oc.evict(mass, [0] * 8, (0, 0), 8, 4, 1, 1)
    assert moves == [(4, 1), (7, 3)]
    assert m == [0, 5, 9, 0, 0, 0, 0, 0] and p[:4] == [0, 4, 2, 7] and h == (4, 8)
    # three tokens later: slots 4.. hold positions 8, 9, 10; the newest two are protected
    m[4:7] = [1, 1, 1]
    moves, m, p, h = oc.evict(m, p, h, 7, 3, 0, 2)
    assert moves == [(5, 0), (6, 1)] and p[:3] == [9, 10, 2] and h == (3, 11)


def test_evict_ties_and_nan():
    moves, *_ = oc.evict([1.0, 1, 1, 1, 1], [0] * 5, (0, 0), 5, 2, 0, 0)
    assert moves == []  # the lowest slots stay
    moves, *_ = oc.evict([1.0, 2, np.inf, np.nan], [0] * 4, (0, 0), 4, 2, 0, 0)
    assert moves == [(2, 0), (3, 1)]
    assert oc.evict([1.0] * 4, [0] * 4, (0, 0), 4, 0, 1, 1)[3] == (0, 4)
