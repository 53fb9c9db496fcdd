"""fp32 numbers as sums of three bf16 ones, each the nearest to what the ones before leave: a restatement of the split that
attention over packed prompts makes of fp32, at the mantissas that are worst for it."""

import numpy as np
import pytest


def nearest(x):
    """fp32 to bf16, ties to even, infinity for what lies beyond the largest."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return (((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32)).view(np.float32)


def cut(x):
    return (np.asarray(x, np.float32).view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)


def parts(x, to=nearest):
    """The first part no larger than the largest bf16 number."""
    out, left = [], np.asarray(x, np.float32)
    for i in range(3):
        p = to(left)
        if i == 0:
            p = np.clip(p, -np.float32(2.0 ** 127 * (2 - 2.0 ** -7)), np.float32(2.0 ** 127 * (2 - 2.0 ** -7)))
        out.append(p)
        left = (left - p).astype(np.float32)
    return out, left


def numbers(kind):
    rng = np.random.default_rng(0)
    m = rng.integers(0, 1 << 23, 200000)
    if kind == "runs":                        # of ones and zeros
        m = (1 << rng.integers(0, 24, m.size)) - (1 << rng.integers(0, 24, m.size))
    if kind == "halves":                      # near the middle between two steps of either part
        m = (rng.integers(0, 128, m.size) << 16) + 0x8000 + rng.integers(-3, 4, m.size) + (rng.integers(-1, 2, m.size) << 7)
    m = np.abs(m) & 0x7FFFFF
    return ((rng.integers(0, 2, m.size) << 31) | (127 << 23) | m).astype(np.uint32).view(np.float32)


@pytest.mark.parametrize("kind", ["any", "runs", "halves"])
def test_six_products_leave_out_a_step_of_24_bits_at_most(kind):
    """Their error: 2^-24 of the product and the two smallest parts' own."""
    a = numbers(kind)
    b = np.random.default_rng(1).permutation(a)
    pa, left_a = parts(a)
    pb, left_b = parts(b)
    assert not left_a.any() and not left_b.any()                    # the parts are the number
    a0, a1, a2 = (x.astype(np.float64) for x in pa)
    b0, b1, b2 = (x.astype(np.float64) for x in pb)
    assert np.array_equal(a0 + a1 + a2, a.astype(np.float64))
    off = (a1 * b2 + a2 * b1 + a2 * b2) / (a.astype(np.float64) * b.astype(np.float64))
    assert np.abs(off).max() <= 2.0 ** -24 * (1 + 2.0 ** -8)
    # cut off instead of rounded the parts lose more, and all to one side
    (_, c1, c2), (_, d1, d2) = ([x.astype(np.float64) for x in parts(y, cut)[0]] for y in (a, b))
    lost = (c1 * d2 + c2 * d1 + c2 * d2) / (a.astype(np.float64) * b.astype(np.float64))
    assert lost.min() >= 0 and np.abs(off.mean()) < 0.05 * lost.mean()
    assert kind == "halves" or lost.max() > 2.0 ** -23


def test_the_largest_numbers_have_finite_parts():
    x = np.array([0x7F7FFFFF, 0x7F7F8000, 0x7F7F7FFF, 0x7F7FC000, 0xFF7FFFFF, 0xFF7F8001], np.uint32).view(np.float32)
    p, left = parts(x)
    assert np.isfinite(np.stack(p)).all() and not left.any()
