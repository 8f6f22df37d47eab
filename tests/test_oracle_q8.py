"""Pins of the fp64 oracle of the 8-bit cache: code tables, rounding, the scale
rule and the append, against closed forms and torch's own 8-bit types."""

import numpy as np
import pytest
import torch

import oracle


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_code_values_and_bytes_are_inverse(fmt):
    b = np.arange(256, dtype=np.uint8)
    v = oracle.q8_values(b, fmt)
    if fmt == "e4m3":
        want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
        assert np.array_equal(v, want, equal_nan=True)
        keep = ~np.isnan(v)
        assert keep.sum() == 254 and np.nanmax(v) == 448
    else:
        assert np.array_equal(v, np.arange(256, dtype=np.uint8).view(np.int8))
        keep = np.ones(256, bool)
    assert np.array_equal(oracle.q8_bytes(v[keep], fmt), b[keep])


def test_e4m3_rounding_matches_torch_and_ties_go_to_even():
    rng = np.random.default_rng(3)
    x = np.concatenate([rng.normal(size=4096) * 2.0 ** rng.integers(-12, 9, 4096),
                        [0.0, 2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0, 447.9, 464.0]])
    x = np.clip(x, -448, 448).astype(np.float32).astype(np.float64)
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oracle.q8_round(x, "e4m3"), want)
    assert oracle.q8_round(17.0, "e4m3") == 16 and oracle.q8_round(19.0, "e4m3") == 20
    assert oracle.q8_round(2.0 ** -10, "e4m3") == 0
    assert oracle.q8_round(1e9, "e4m3") == 448 and oracle.q8_round(-1e9, "int8") == -127


@pytest.mark.parametrize("fmt,top", [("e4m3", 448.0), ("int8", 127.0)])
def test_scale_exponent_is_the_smallest_that_covers(fmt, top):
    assert oracle.q8_scale_exponent(top, fmt) == 0
    assert oracle.q8_scale_exponent(np.nextafter(top, 1e9), fmt) == 1
    assert oracle.q8_scale_exponent(top / 2, fmt) == -1
    assert oracle.q8_scale_exponent(0.0, fmt) == -64
    assert oracle.q8_scale_exponent(1e30, fmt) == 63


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_keeps_values_within_half_a_step_and_follows_growth(fmt):
    rng = np.random.default_rng(5)
    codes = oracle.q8_bytes(oracle.q8_round(rng.normal(size=(2, 32, 2, 8)) * 40, fmt), fmt)
    scales = np.full((2, 2, 2), 0.25)
    y = rng.normal(size=(3, 2, 8)) * [[[1.0]], [[300.0]], [[2.0]]]
    slots = [5, 6, 48 + 3]                   # one group grows, another one is extended
    c, s = oracle.q8_append(y, slots, codes, scales, fmt)
    before = oracle.q8_values(codes, fmt)
    assert (s[0, 0] > 0.25).all() and s[0, 1].tolist() == [0.25, 0.25]
    # appended: within half a code step of the value
    for t, slot in enumerate(slots):
        sc = s[slot // 32, slot % 32 // 16][:, None]
        got, want = c[slot // 32, slot % 32] * sc, y[t]
        half = np.maximum(np.abs(want) * 2.0 ** -4, sc * 2.0 ** -10) if fmt == "e4m3" else sc / 2
        assert (np.abs(got - want) <= half).all()
    # earlier tokens of the grown group: the rescaled code, everything else as it was
    rest = [o for o in range(16) if o not in (5, 6)]
    assert np.array_equal(c[0, rest],
                          oracle.q8_round(before[0, rest] * (0.25 / s[0, 0])[:, None], fmt))
    assert np.array_equal(c[0, 16:], before[0, 16:]) and np.array_equal(c[1, :16], before[1, :16])
    # slot 0 starts a group anew, whatever its scale was
    c2, s2 = oracle.q8_append(y[:1], [32], codes, np.full((2, 2, 2), 2.0 ** 20), fmt)
    assert (s2[1, 0] < 1).all() and np.array_equal(c2[1, 1:], before[1, 1:])


def test_append_of_non_finite_values():
    y = np.array([np.inf, -np.inf, np.nan, 1.0]).reshape(1, 1, 4)
    c, s = oracle.q8_append(y, [0], np.zeros((1, 16, 1, 4), np.uint8), np.ones((1, 1, 1)), "e4m3")
    assert s[0, 0, 0] == 2.0 ** oracle.q8_scale_exponent(1.0, "e4m3")
    assert c[0, 0, 0].tolist() == [448.0, -448.0, 0.0, 256.0]
