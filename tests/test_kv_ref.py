"""The tests' own reference of the 8-bit cache, on the CPU: its rounding against hand values, its scale rule by its definition."""

import numpy as np
import pytest

import _kv_ref as ref
from _gpu import fp8_table


@pytest.mark.parametrize("fmt", [0, 1])
def test_rounding_keeps_codes_and_takes_ties_to_even(fmt):
    t = fp8_table(fmt)
    t = t[np.isfinite(t)]
    assert np.array_equal(ref.fp8_round(t, fmt), t)
    assert np.isnan(ref.fp8_round(np.array([np.nan, np.inf]), fmt)).all()
    one = (1.0625, 1.0, 1.1875, 1.25) if fmt == 0 else (1.125, 1.0, 1.375, 1.5)
    assert ref.fp8_round(np.array([one[0], -one[0], one[2]]), fmt).tolist() == [one[1], -one[1], one[3]]
    tiny = t[t > 0].min()
    assert ref.fp8_round(np.array([tiny / 2, tiny * 0.75, tiny * 1.5]), fmt).tolist() == [0.0, tiny, 2 * tiny]
    assert ref.fp8_round(np.array([ref.FMAX[fmt] * 1.03]), fmt).tolist() == [ref.FMAX[fmt]]


@pytest.mark.parametrize("fmt", [0, 1])
def test_exponent_is_the_smallest_that_clips_nothing(fmt):
    f = ref.FMAX[fmt]
    for a in (f, np.nextafter(f, 2 * f), f / 2, 1.0, 3.7e-30, 1.75, 1.7500001, 2.0 ** 100):
        x = ref.exponent(a, fmt)
        assert a <= f * 2.0 ** x and (x == -127 or a > f * 2.0 ** (x - 1))
    assert ref.exponent(0.0, fmt) == -127 and ref.exponent(1e-45, fmt) == -127


def test_one_token_at_a_time_holds_what_a_page_at_once_holds_but_for_small_values():
    """Codes move by powers of two: a value that is normal at the final scale is rounded as if once."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((16, 2, 1, 64)) * np.exp2(rng.integers(-3, 4, (16, 1, 1, 1)))
    empty = lambda: {"k": np.zeros((1, 1, 16, 64)), "v": np.zeros((1, 1, 16, 64)), "kx": np.zeros((1, 1), int), "vx": np.zeros((1, 1), int)}
    whole, steps = empty(), empty()
    ref.append(whole, 0, 16, [[0]], [16], [(0, 16)], x)
    for t in range(16):
        ref.append(steps, 0, 16, [[0]], [t + 1], [(0, 1)], x[t:t + 1])
    for n in "kv":
        assert whole[n + "x"] == steps[n + "x"]
        normal = np.abs(whole[n]) >= 2.0 ** -6
        assert np.array_equal(whole[n][normal], steps[n][normal])
        assert np.abs(whole[n] - steps[n]).max() <= 2.0 ** -9


def test_attention_of_the_reference_is_softmax():
    rng = np.random.default_rng(1)
    cache = {"k": rng.standard_normal((3, 2, 16, 64)), "v": rng.standard_normal((3, 2, 16, 64)), "kx": np.full((3, 2), 1), "vx": np.full((3, 2), -1)}
    q = rng.standard_normal((2, 4, 64))
    att, size, lse, mag = ref.attend(cache, 16, [[2, 0]], [19], [(0, 2)], q)
    K = np.concatenate([cache["k"][2], cache["k"][0]], 1)[:, :18] * 2
    V = np.concatenate([cache["v"][2], cache["v"][0]], 1)[:, :18] / 2
    for h in range(4):
        e = np.exp(K[h // 2] @ q[0, h] / 8)
        assert np.allclose(att[0, h], e @ V[h // 2] / e.sum(), rtol=1e-12) and np.isclose(lse[h, 0], np.log(e.sum()), rtol=1e-12)
    att, _, lse, _ = ref.attend(cache, 16, [[2, 0]], [0], [(0, 2)], q)
    assert (att == 0).all() and np.isneginf(lse).all()
