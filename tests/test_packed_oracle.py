"""The oracle of the 4-bit latent row, pinned by hand-computed cases and by properties."""
import numpy as np

import oracle


def test_e4m3_values():
    assert oracle.e4m3_value(0x00) == 0 and oracle.e4m3_value(0x01) == 2.0 ** -9
    assert oracle.e4m3_value(0x08) == 2.0 ** -6 and oracle.e4m3_value(0x38) == 1.0
    assert oracle.e4m3_value(0x7E) == 448.0 and oracle.e4m3_value(0xB8) == -1.0
    assert np.isnan(oracle.e4m3_value(0x7F))


def test_rounding_ties_go_to_the_even_code():
    # scale 1 (the largest is 6): the values between two codes
    row = np.zeros(512)
    row[:16] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, 0.2501, 2.4999, 2.5001, 4.999, 5.001, -6]
    got = oracle.packed_values(oracle.packed_quantise(row))[:16]
    assert got.tolist() == [6, 0, 1, 1, 2, 2, 4, 4, 0, -1, 0.5, 2, 3, 4, 6, -6]


def test_layout_of_a_row():
    row = np.zeros(512)
    row[0], row[1], row[16] = 6.0, -3.0, 12.0
    p = oracle.packed_quantise(row)
    assert p.shape == (288,) and p.dtype == np.uint8
    assert p[0] == (0x7 | (0xD << 4))        # 6 -> code 7, -3 -> code 8 + 5
    assert p[8] == 0x7 and p[256] == 0x38 and p[257] == 0x40  # scales 1 and 2


def test_saturation_zero_and_non_finite_groups():
    row = np.zeros(512)
    row[0] = 1e6            # scale saturates at 448, the value at 6 * 448
    row[16] = 1e-5          # scale rounds to zero
    row[32], row[48] = np.inf, np.nan
    v = oracle.packed_values(oracle.packed_quantise(row))
    assert v[0] == 2688.0 and not v[16:32].any()
    assert np.isnan(v[32:64]).all() and not v[64:].any()


def test_error_is_half_a_step_and_unit_scales():
    rng = np.random.default_rng(0)
    rows = rng.standard_normal((50, 512)) * np.exp(rng.standard_normal(512))
    v = oracle.packed_values(oracle.packed_quantise(rows))
    amax = np.abs(rows.reshape(50, 32, 16)).max(-1).repeat(16, axis=-1).reshape(50, 512)
    # the scale is within 2^-4 of amax / 6; a step of the code grid is at most 2 scales (1 half
    # step), and an amax that the scale rounded down loses up to 2^-4 of itself at the top
    assert (np.abs(v - rows) <= amax / 6 * (1 + 2.0 ** -4) + 1e-12).all()
    assert np.array_equal(oracle.packed_quantise(rows * 8, 8.0), oracle.packed_quantise(rows))
    # quantising a quantised row again changes nothing in value when its largest code is 6
    again = oracle.packed_values(oracle.packed_quantise(v))
    six = np.abs(v.reshape(50, 32, 16)).max(-1) == 6 * oracle.e4m3_value(oracle.packed_quantise(rows)[:, 256:])
    assert np.array_equal(again.reshape(50, 32, 16)[six], v.reshape(50, 32, 16)[six])


def test_window_positions():
    f = oracle.window_positions
    assert f(10, 1, 0, 0, 3).tolist() == list(range(10))
    assert f(10, 1, 0, 4, 2).tolist() == [0, 1, 6, 7, 8, 9]
    assert f(10, 3, 0, 4, 2).tolist() == [0, 1, 4, 5, 6, 7]
    assert f(10, 1, 0, 4, 8).tolist() == list(range(10))
    assert f(2, 4, 0, 4, 8).size == 0 and f(2, 4, 2, 1, 0).tolist() == [0]
