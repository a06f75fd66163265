"""The oracle of the block operators: how a query is held."""
import numpy as np
import pytest

from oracle import block_oracle as B


def test_e2m3_rounds_to_nearest_even_and_ends_at_seven_and_a_half():
    assert len(B._E2M3) == 32 and B._E2M3[-1] == 7.5 and np.all(np.diff(B._E2M3) > 0)
    assert np.array_equal(B.e2m3(B._E2M3), B._E2M3) and np.array_equal(B.e2m3(-B._E2M3), -B._E2M3)
    for i in range(31):
        mid = (B._E2M3[i] + B._E2M3[i + 1]) / 2
        assert B.e2m3(np.array([mid]))[0] == B._E2M3[i + i % 2]
        assert B.e2m3(np.array([mid * (1 + 1e-12)]))[0] == B._E2M3[i + 1]
    assert np.array_equal(B.e2m3(np.array([7.6, 9.0, -1e9])), [7.5, 7.5, -7.5])


@pytest.mark.parametrize("largest", [1.0, 1.5, 1.8749, 1.875, 1.8751, 1.9, 1.9375, 1.99, 1.9996, 1.99999, 2 - 1e-9])
def test_three_terms_leave_less_than_a_part_in_8192(largest):
    """Of the block's largest element, whatever its mantissa: 2^-12 of 2^e, and 3.75 of 2^e at least."""
    rng = np.random.default_rng(int(largest * 1e6))
    for scale in (1.0, 2.0 ** -9, 2.0 ** 20):
        x = rng.uniform(-1, 1, (2000, 32)) * largest
        x[:, rng.integers(0, 32)] = largest * rng.choice([-1, 1], 2000)
        x[:, 0] *= 2.0 ** -rng.integers(0, 12, 2000)
        x *= scale
        left = np.abs(B.query_terms(x).sum(0) - x).max()
        assert left <= 2.0 ** -12 / 3.75 * largest * scale < 2.0 ** -13 * largest * scale * 1.1
        assert left <= 2.0 ** -13 * largest * scale
