"""Pins of the oracle of the low-precision linear layer and the preference
loss (CPU): hand-built roundings and scales, and gradients by differences."""

import numpy as np
import pytest

from oracle import head_oracle as H


def test_e2m1_ties_go_to_the_even_code():
    row = np.zeros((1, 32))
    given = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -5.0, 0.26, 4.99]
    want = [6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 0.0, -4.0, 0.5, 4.0]
    row[0, :len(given)] = given
    assert H.quantize(row, "mx4")[1][0, 0] == 127
    np.testing.assert_array_equal(H.rounded(row, "mx4")[0, :len(want)], want)


@pytest.mark.parametrize("fmt,top,byte", [
    ("mx4", 6.0, 127), ("mx4", 6.0001, 128), ("mx4", 12.0, 128), ("mx4", 3.0, 126), ("mx4", 3.0001, 127),
    ("mx8", 448.0, 127), ("mx8", 449.0, 128), ("mx8", 224.0, 126), ("mx8", 225.0, 127),
    ("mx4", 0.0, 1), ("mx8", 0.0, 1), ("mx4", 1e-44, 1), ("mx4", 3e38, 127 + 126), ("mx4", np.inf, 255), ("mx8", np.nan, 255)])
def test_scale_is_the_least_that_fits(fmt, top, byte):
    x = np.zeros((1, 40))
    x[0, 3] = -top
    codes, scales = H.quantize(x, fmt)
    assert scales[0, 0] == byte and scales[0, 1] == 1
    if byte == 255:
        assert not codes.any() and np.isnan(H.rounded(x, fmt)[0, :32]).all() and not H.rounded(x, fmt)[0, 32:].any()


def test_values_are_fixed_points_and_errors_are_half_a_step():
    x = np.random.default_rng(0).standard_normal((7, 300)) * 5
    for fmt, eps in (("mx4", 2.0 ** -2), ("mx8", 2.0 ** -4)):
        r = H.rounded(x, fmt)
        np.testing.assert_array_equal(H.rounded(r, fmt), r)
        top = np.abs(np.pad(x, ((0, 0), (0, 20))).reshape(7, -1, 32)).max(2).repeat(32, 1)[:, :300]
        # half a step of the value, or of the smallest normal (1 of at most 12, 2^-6 of at most 896)
        floor = top / 3.0 if fmt == "mx4" else top / 224.0 * 2.0 ** -6
        assert (np.abs(r - x) <= eps * np.maximum(np.abs(x), floor)).all()


def test_mx4_codes_put_the_even_element_low():
    x = np.zeros((1, 2))
    x[0] = [1.0, -6.0]
    codes, scales = H.quantize(x, "mx4")
    assert codes.shape == (1, 64) and scales.shape == (1, 4) and codes[0, 0] == (2 | (15 << 4))


@pytest.mark.parametrize("kind,eps,average", [("logistic", 0.0, False), ("logistic", 0.2, True), ("squared", 0.0, False),
                                              ("squared", 0.0, True)])
def test_preference_gradient_by_differences(kind, eps, average):
    rng = np.random.default_rng(1)
    z, labels = rng.standard_normal((9, 5)), rng.integers(0, 5, 9)
    labels[[0, 4]] = -100
    offsets, ref, g = [0, 3, 5, 5, 9], rng.standard_normal(9), np.array([0.7, -1.3])

    def total(zz):
        return float(g @ H.preference(zz, labels, offsets, ref, 0.3, kind, eps, average)["loss"])

    d = H.preference(z, labels, offsets, ref, 0.3, kind, eps, average, g)["dlogits"]
    for t in range(9):
        for v in range(5):
            step = np.zeros_like(z)
            step[t, v] = 1e-5
            # central difference: error ~ third derivative * 1e-10 / 6 and 1e-16 * |loss| / 1e-5
            assert abs((total(z + step) - total(z - step)) / 2e-5 - d[t, v]) < 1e-8
    assert not d[[0, 4]].any()


def test_preference_closed_forms():
    z = np.zeros((2, 4))
    r = H.preference(z, np.array([1, 2]), [0, 1, 2], None, 0.1, grad_loss=np.ones(1))
    assert r["margin"][0] == 0 and abs(r["loss"][0] - np.log(2)) < 1e-15 and abs(r["slope"][0] + 0.05) < 1e-16
    np.testing.assert_allclose(r["dlogits"][0], -0.05 * (np.eye(4)[1] - 0.25), atol=1e-17)
    s = H.preference(z, np.array([1, 2]), [0, 1, 2], None, 0.5, "squared")
    assert s["loss"][0] == 1.0 and s["slope"][0] == -2.0
