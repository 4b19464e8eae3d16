"""The plain paged-cache and verification forms against invariants and brute force (no GPU)."""
import numpy as np
import pytest

from oracle import paged_oracle as P


@pytest.mark.parametrize("fmt,step", [("f16", 0.0), ("fp8", 2.0 ** -4), ("int4", 0.5 / 7 * 1.01)])
@pytest.mark.parametrize("d", [64, 128])
def test_quantised_rows_are_within_half_a_step(fmt, step, d):
    rng = np.random.default_rng(d)
    x = (rng.standard_normal((50, d)) * np.exp(rng.uniform(-4, 4, (50, 1)))).astype(np.float16)
    v = P.values(*P.quantise(x, fmt), fmt)
    if fmt == "fp8":       # half a step of a 4-bit significand, or of the smallest e4m3 step
        tol = np.maximum(np.abs(x.astype(np.float64)) * step, np.abs(x).max(-1, keepdims=True) / 448 * 2.0 ** -10) * 1.001
    else:                  # half a step of amax/7 (and the rounding of the scale to 11 bits)
        tol = np.abs(x.reshape(50, -1, 32)).max(-1).repeat(32, -1).astype(np.float64) * (step + (2.0 ** -11 if step else 0))
    assert (np.abs(v - x.astype(np.float64)) <= tol).all()


def test_quantised_special_rows():
    zero = np.zeros((1, 64), np.float16)
    for fmt in ("f16", "fp8", "int4"):
        assert (P.values(*P.quantise(zero, fmt), fmt) == 0).all()
    x = np.ones((1, 64), np.float16)
    x[0, 3] = np.nan
    v = P.values(*P.quantise(x, "int4"), "int4")
    assert np.isnan(v[0, :32]).all() and np.array_equal(v[0, 32:], np.full(32, float(np.float16(1 / 7)) * 7.0).astype(np.float16))


def test_4bit_rows_of_finite_values_are_finite():
    """Every f16 value as a group's largest, each value within half a step of what it was."""
    x = np.zeros((0x7c00, 64), np.float16)
    x[:, 40] = np.arange(0x7c00, dtype=np.uint16).view(np.float16)
    x[:, 3] = -x[:, 40]
    codes, scales = P.quantise(x, "int4")
    v = P.values(codes, scales, "int4")
    assert np.isfinite(scales).all() and np.isfinite(v).all() and scales.max() == 9352
    # half a step of the scale, and its and the product's rounding to f16 (of 7 scales: 2^-11 and 2^-24)
    step = np.maximum(scales.astype(np.float64), 2.0 ** -24)
    assert (np.abs(v - x.astype(np.float64)) <= 0.5 * step.repeat(32, -1) + np.abs(x.astype(np.float64)) * 2.0 ** -10 + 7 * 2.0 ** -25).all()


def test_attention_matches_brute_force_and_masks():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((3, 4, 8)), rng.standard_normal((6, 2, 8)), rng.standard_normal((6, 2, 8))
    out, lse, bound, depth = P.attention(q, k, v)
    for u in range(3):
        for h in range(4):
            n = 6 - 3 + u + 1
            z = [sum(q[u, h, d] * k[c, h // 2, d] for d in range(8)) / np.sqrt(8) for c in range(n)]
            w = np.exp(z)
            assert np.isclose(lse[u, h], np.log(w.sum()), rtol=1e-12)
            assert np.allclose(out[u, h], (w[:, None] * v[:n, h // 2]).sum(0) / w.sum(), rtol=1e-12)
    assert (np.abs(out) <= bound + 1e-15).all() and (depth > 0).all()
    out, lse, *_ = P.attention(q, k[:2], v[:2])      # fewer tokens than queries
    assert (out[0] == 0).all() and np.isinf(lse[0]).all() and np.isfinite(lse[1:]).all()


def test_verification_keeps_the_targets_distribution():
    """Summed over a fine grid of random numbers, the first emitted token has probability p."""
    p, q = np.array([[0.5, 0.25, 0.25], [1.0, 0.0, 0.0]]), np.array([[0.25, 0.5, 0.25]])
    n, count = 64, np.zeros(3)
    grid = (np.arange(n) + 0.5) / n
    for d in range(3):
        for a in grid:
            for b in grid:
                m, t = P.verify(p, q, [d], [a, b])
                count[d if m else t] += q[0, d] / n ** 2
    assert np.allclose(count, p[0], atol=1.5 / n)


@pytest.mark.parametrize("u,want", [(0.0, 1), (0.24, 1), (0.25, 3), (0.999, 3), (1.0, 3), (-1.0, 1), (float("nan"), 1)])
def test_verification_takes_the_lowest_token_past_the_threshold(u, want):
    p = [[0.0, 0.25, 0.0, 0.75, 0.0]]
    assert P.verify(p, None, [], [u]) == (0, want)


def test_verification_corner_cases():
    p = np.array([[0.5, 0.5, 0.0], [0.0, 0.25, 0.75]])
    assert P.verify(p, None, [0], [0.49, 0.5]) == (1, 2)     # kept, next from the row after it
    assert P.verify(p, None, [0], [0.5, 0.0]) == (0, 1)      # u q < p fails: the others are left
    assert P.verify(p, None, [7], [0.0, 0.0]) == (0, 0)      # no such token: rejected
    assert P.verify(p, p[:1], [1], [0.5, 0.9]) == (1, 2)
    assert P.verify([[0.1, 0.4, 0.4], [1, 0, 0]], [[0.5, 0.5, 0.5]], [0], [0.9, 0.3]) == (0, 1)  # nothing left: argmax


@pytest.mark.parametrize("u", [0.0, -0.0, -1.0, float("-inf"), float("nan")])
def test_a_draft_the_target_never_gives_is_rejected(u):
    p = np.array([[0.5, 0.5, 0.0], [0.0, 0.25, 0.75]])
    assert P.verify(p, [[0.2, 0.2, 0.6]], [2], [u, 0.0]) == (0, 0)
