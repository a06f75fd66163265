"""What the bounds of the attention's tests reject, by mistakes planted in a CPU form of its sums."""
import numpy as np
import pytest

from oracle import block_oracle as B
from tests import attention_check as A


def test_exact_scale_is_a_power_of_two_of_base_two():
    for had in (0, 32):
        for k in (0, 3, 7):
            c = np.float32(np.float32(A.exact_scale(k, had)) * A.LOG2E) / np.float32(32 if had else 1)
            assert abs(float(c) * 2.0 ** k - 1) <= 2.0 ** -23


@pytest.mark.parametrize("had", [0, 32])
def test_whole_queries_are_held_exactly(had):
    """Three FP6 terms hold the queries of these tests: whole numbers, transformed ones, patterns."""
    rng = np.random.default_rng(1)
    q = A.whole_queries(rng, 50, 3, 128, 2).astype(np.float64)
    c = A.climb_problem(1, "late", 64, 20, 2, 64, had)["q"].astype(np.float64)
    s = A.steep_problem(1, 64, 20, 2, 128, had, lambda r, shape: r.integers(125, 130, shape))["q"].astype(np.float64)
    for x in (q, c, s):
        x = B.hadamard_blocks(x) if had else x
        b = x.reshape(-1, 32)
        assert np.array_equal(B.query_terms(b).sum(0), b)


def _caught(kind, had, runs):
    """The planted mistakes that the room rejects, in a row of factor one (row 0) or over all rows;
    the right sums are inside it and zeros are not."""
    n, rows = 1300, 12
    p = A.climb_problem(5, kind, n, rows, 1, 64, had)
    out, _, room, _ = A.want(p["q"], p["arr"], p["table"], p["lens"], p["cu"], p["scale"], False, 64, had)
    k, v, _ = A.gathered(p["arr"], p["table"][0], n)
    s = A.scores(p["q"][:, 0], k[0], p["scale"], had)[0] / np.log(2.0)
    assert np.abs(s[0] - np.rint(s[0])).max() < 1e-4
    turned = lambda o: B.unrotated(o, had)[:64]       # noqa: E731
    right = np.stack([turned(A.summed(s[r], v[0], runs)) for r in range(rows)])
    assert A.outside(right, out[:, 0], room[:, 0]) == 0.0
    assert A.outside(0.0, out[:, 0], room[:, 0]) > 0.7
    caught = set()
    for m in A.MISTAKES:
        with np.errstate(over="ignore", invalid="ignore"):
            got = np.stack([turned(A.summed(s[r], v[0], runs, m)) for r in range(rows)])
        if A.outside(got[:1], out[:1, 0], room[:1, 0]) > 0.3 or A.outside(got, out[:, 0], room[:, 0]) > 0.15:
            caught.add(m)
    return caught


@pytest.mark.parametrize("had", [0, 32])
@pytest.mark.parametrize("runs", [1, 4])
def test_every_planted_mistake_is_rejected(had, runs):
    """By two of the climbs at least, and by every climb some."""
    caught = {k: _caught(k, had, runs) for k in A.CLIMBS}
    print(runs, {k: sorted(c) for k, c in caught.items()})
    for m in A.MISTAKES:
        if runs > 1 or m not in ("parts joined as they are", "one part lost"):
            assert sum(m in c for c in caught.values()) >= 2, m
    assert all(caught.values())
